// beam_api.hip -- the entry points of beam search (include/ssm.h): host-side validation, launch shapes and
// launches.
#include <hip/hip_runtime.h>

#include "../../include/ssm.h"
#include "beam.hpp"
#include "cache_host.hpp"

using namespace ssm_host;

namespace {

// How a row is cut: into stretches of at most what a workgroup holds, all about as long.
struct BeamShape {
  int64_t chunks, blocks, words, bytes;
};

ssm_status_t beam_shape(int64_t batch, int64_t rows, int64_t vocab, int64_t beams, bool bf16, BeamShape* out) {
  const int64_t epb = bf16 ? 8 : 4, blocks = (vocab + epb - 1) / epb;
  const int64_t group = ssm::kBeamThreads * (ssm::kBeamValues / epb);
  out->chunks = (blocks + group - 1) / group;
  out->blocks = (blocks + out->chunks - 1) / out->chunks;
  int64_t n;
  if (!mul_ok(batch * rows, out->chunks, &n) || !mul_ok(n, 8 * (beams + ssm::kBeamWaves), &out->bytes))
    return fail(SSM_ERR_INVALID_ARG, "workspace size overflows int64");
  if (n > kMaxBlocks) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  out->words = n;
  return SSM_OK;
}

ssm_status_t check_beams(int64_t batch, int64_t rows, int64_t vocab, int64_t beams, ssm_dtype_t dtype) {
  if (batch < 0 || rows < 1 || vocab < 1 || beams < 1 || batch > kMaxIndex || vocab > kMaxIndex)
    return fail(SSM_ERR_INVALID_ARG, "bad size (batch=%lld rows=%lld vocab=%lld beams=%lld)", (long long)batch,
                (long long)rows, (long long)vocab, (long long)beams);
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (rows > ssm::kBeamMost || beams > ssm::kBeamMost)
    return fail(SSM_ERR_UNSUPPORTED, "more than %d rows (%lld) or beams (%lld)", ssm::kBeamMost, (long long)rows,
                (long long)beams);
  if (beams > rows * vocab)
    return fail(SSM_ERR_INVALID_ARG, "%lld beams of %lld candidates", (long long)beams, (long long)(rows * vocab));
  return SSM_OK;
}

struct Reorder {
  void (*kernel)(const ssm::ReorderArgs);
  int64_t bytes;  // of an entry that a workgroup takes
};
template <int BEAMS, int COLUMNS, int WORDS>
constexpr Reorder reorder_with() {
  return {ssm::reorder_kernel<BEAMS, COLUMNS, WORDS>, int64_t{4} * WORDS * COLUMNS * ssm::kBeamThreads};
}
Reorder reorder_of(int64_t beams) {
  return beams <= 4 ? reorder_with<4, 2, 4>()
                    : beams <= 8 ? reorder_with<8, 2, 4>()
                                 : beams <= 16 ? reorder_with<16, 1, 4>()
                                               : beams <= 32 ? reorder_with<32, 1, 4>() : reorder_with<64, 1, 2>();
}

}  // namespace

extern "C" {

ssm_status_t ssm_beam_select_workspace(int64_t batch, int64_t rows, int64_t vocab, int64_t beams, ssm_dtype_t dtype,
                                       int64_t* bytes) {
  g_err[0] = '\0';
  if (!bytes) return fail(SSM_ERR_INVALID_ARG, "NULL bytes");
  SSM_TRY(check_beams(batch, rows, vocab, beams, dtype));
  BeamShape s;
  SSM_TRY(beam_shape(batch, rows, vocab, beams, dtype == SSM_BF16, &s));
  *bytes = s.bytes;
  return SSM_OK;
}

ssm_status_t ssm_beam_select(int64_t batch, int64_t rows, int64_t vocab, int64_t beams, ssm_dtype_t dtype,
                             const void* logits, int64_t stride_batch, int64_t stride_row, const float* scores,
                             const uint8_t* finished, int64_t eos, int32_t* parents, int32_t* tokens, float* out_scores,
                             uint8_t* out_finished, void* workspace, int64_t workspace_bytes, void* stream) {
  g_err[0] = '\0';
  SSM_TRY(check_beams(batch, rows, vocab, beams, dtype));
  BeamShape s;
  SSM_TRY(beam_shape(batch, rows, vocab, beams, dtype == SSM_BF16, &s));
  if (finished && (eos < 0 || eos >= vocab))
    return fail(SSM_ERR_INVALID_ARG, "eos %lld is not in 0..%lld", (long long)eos, (long long)(vocab - 1));
  if (out_finished && !finished) return fail(SSM_ERR_INVALID_ARG, "out_finished needs finished");
  if (stride_row == 0) stride_row = vocab;
  if (stride_batch == 0 && !mul_ok(rows, stride_row, &stride_batch))
    return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  int64_t span, n;
  if (stride_row < 0 || stride_batch < 0 || !mul_ok(batch > 0 ? batch - 1 : 0, stride_batch, &span) ||
      !mul_ok(rows - 1, stride_row, &n) || __builtin_add_overflow(span, n, &span) ||
      __builtin_add_overflow(span, vocab, &span) || !mul_ok(span, es, &span))
    return fail(SSM_ERR_INVALID_ARG, "bad strides (%lld, %lld)", (long long)stride_batch, (long long)stride_row);
  if (batch == 0) return SSM_OK;
  if (!logits || !scores || !parents || !tokens || !out_scores)
    return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (logits, scores, parents, tokens and out_scores)");
  const Arg args[] = {{logits, es, "logits"}, {scores, 4, "scores"}, {parents, 4, "parents"}, {tokens, 4, "tokens"},
                      {out_scores, 4, "out_scores"}, {workspace, 16, "workspace"}};
  if (const Arg* m = misaligned(args, sizeof args / sizeof *args))
    return fail(SSM_ERR_MISALIGNED, "%s (%p) is not aligned", m->name, m->p);
  if (!workspace || workspace_bytes < s.bytes)
    return fail(SSM_ERR_INVALID_ARG, "workspace of %lld bytes, need %lld", workspace ? (long long)workspace_bytes : 0ll,
                (long long)s.bytes);
  const Range outs[] = {{parents, batch * beams * 4}, {tokens, batch * beams * 4}, {out_scores, batch * beams * 4},
                        {out_finished, batch * beams}, {workspace, s.bytes}};
  const Range ins[] = {{logits, span}, {scores, batch * rows * 4}, {finished, batch * rows}};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));
  ssm::BeamArgs a{};
  a.logits = logits; a.sb = stride_batch; a.sr = stride_row; a.scores = scores; a.finished = finished;
  a.rows = static_cast<int32_t>(rows); a.beams = static_cast<int32_t>(beams); a.eos = static_cast<int32_t>(eos);
  a.vocab = vocab;
  a.chunks = static_cast<int32_t>(s.chunks); a.blocks = static_cast<int32_t>(s.blocks);
  a.best = static_cast<uint64_t*>(workspace);
  a.stats = reinterpret_cast<float*>(a.best + s.words * beams);
  a.parents = parents; a.tokens = tokens; a.out_scores = out_scores; a.out_finished = out_finished;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (batch > 0xffffffffll / 1024) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  const auto k = dtype == SSM_BF16 ? ssm::beam_rows_kernel<true> : ssm::beam_rows_kernel<false>;
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(s.words)), dim3(ssm::kBeamThreads), 0, st, a);
  SSM_TRY(check_launch("beam selection (rows)"));
  const unsigned threads = 64u * static_cast<unsigned>(rows < 16 ? rows : 16);
  hipLaunchKernelGGL(ssm::beam_join_kernel, dim3(static_cast<unsigned>(batch)), dim3(threads), 0, st, a);
  return check_launch("beam selection (join)");
}

ssm_status_t ssm_cache_reorder(int64_t batch, int64_t beams, const ssm_entries_t* caches, int64_t count,
                               const int32_t* cache_slots, const int32_t* parents, void* stream) {
  g_err[0] = '\0';
  if (batch < 0 || beams < 1 || count < 0 || batch > kMaxIndex)
    return fail(SSM_ERR_INVALID_ARG, "bad size (batch=%lld beams=%lld caches=%lld)", (long long)batch, (long long)beams,
                (long long)count);
  if (beams > ssm::kBeamMost)
    return fail(SSM_ERR_UNSUPPORTED, "more than %d beams (%lld)", ssm::kBeamMost, (long long)beams);
  if (count > 0 && !caches) return fail(SSM_ERR_INVALID_ARG, "NULL caches");
  const Reorder k = reorder_of(beams);
  uintptr_t last = 0;  // the highest address so far: layers mostly come in the order of their addresses
  for (int64_t i = 0; i < count; ++i) {
    const ssm_entries_t& c = caches[i];
    const uintptr_t at = reinterpret_cast<uintptr_t>(c.data);
    for (int64_t j = 0; at <= last && c.slots > 0 && c.bytes > 0 && j < i; ++j)
      if (caches[j].data == c.data && caches[j].slots > 0 && caches[j].bytes > 0)
        return fail(SSM_ERR_INVALID_ARG, "cache %lld is cache %lld again", (long long)i, (long long)j);
    last = at > last ? at : last;
    const int64_t stride = c.slot_stride == 0 ? c.bytes : c.slot_stride;
    int64_t span;
    if (c.slots < 0 || c.slots > kMaxIndex || c.bytes < 0 || stride < c.bytes || !mul_ok(c.slots, stride, &span))
      return fail(SSM_ERR_INVALID_ARG, "cache %lld: bad slots (%lld), bytes (%lld) or slot_stride (%lld)", (long long)i,
                  (long long)c.slots, (long long)c.bytes, (long long)c.slot_stride);
    if (!c.data && c.slots > 0 && c.bytes > 0) return fail(SSM_ERR_INVALID_ARG, "NULL cache data (%lld)", (long long)i);
    if (c.bytes / k.bytes >= kMaxBlocks / ssm::kReorderCaches)
      return fail(SSM_ERR_UNSUPPORTED, "grid too large");
    const Range r{c.data, c.slots > 0 ? (c.slots - 1) * stride + c.bytes : 0};
    if (overlap(r, {parents, batch * beams * 4}) || overlap(r, {cache_slots, batch * beams * 4}))
      return fail(SSM_ERR_INVALID_ARG, "a cache overlaps parents or cache_slots");
  }
  if (batch == 0 || beams == 1) return SSM_OK;
  bool any = false;
  for (int64_t i = 0; i < count; ++i) any |= caches[i].slots > 0 && caches[i].bytes > 0;
  if (!any) return SSM_OK;
  if (!parents) return fail(SSM_ERR_INVALID_ARG, "NULL parents");
  if (!aligned(parents, 4) || !aligned(cache_slots, 4))
    return fail(SSM_ERR_MISALIGNED, "parents or cache_slots is not 4-byte aligned");
  for (int64_t i = 0; i < count;) {
    ssm::ReorderArgs a{};
    a.slots = cache_slots; a.parents = parents; a.batch = batch; a.beams = static_cast<int32_t>(beams);
    int64_t blocks = 0;
    for (; i < count && a.caches < ssm::kReorderCaches; ++i) {
      const ssm_entries_t& c = caches[i];
      if (c.slots == 0 || c.bytes == 0) continue;
      a.c[a.caches++] = {static_cast<char*>(c.data), c.slots, c.slot_stride == 0 ? c.bytes : c.slot_stride, c.bytes, blocks};
      blocks += (c.bytes + k.bytes - 1) / k.bytes;
    }
    if (a.caches == 0) break;
    hipLaunchKernelGGL(k.kernel, dim3(static_cast<unsigned>(blocks), grid_y(batch)), dim3(ssm::kBeamThreads), 0,
                       static_cast<hipStream_t>(stream), a);
    SSM_TRY(check_launch("cache reorder"));
  }
  return SSM_OK;
}

}  // extern "C"
