// gated_api.hip -- the entry points of the gated recurrence (include/ssm.h): host-side validation, launch
// shapes and launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/ssm.h"
#include "cache_host.hpp"
#include "gated_scan.hpp"

using namespace ssm_host;

namespace {

// A kernel and the rows of its tiles.
struct Tiled {
  void (*kernel)(const ssm::GatedArgs);
  int64_t rows;
};
template <bool BF16, int V, int R>
Tiled forward_of(bool z) {
  return {z ? ssm::gated_scan_kernel<BF16, true, V, R> : ssm::gated_scan_kernel<BF16, false, V, R>,
          ssm::GatedShape<V, R>::kRows};
}
template <bool BF16, int V, int R>
Tiled backward_of(bool z) {
  return {z ? ssm::gated_scan_bwd_kernel<BF16, true, V, R> : ssm::gated_scan_bwd_kernel<BF16, false, V, R>,
          ssm::GatedShape<V, R>::kRows};
}

// The forward's shape: 8 bytes of a bf16 row or of an fp32 row a lane; the backward's two channels of 64 rows, what
// its registers hold.  Single channels below 4 (backward 2), since a lane's must lie in the row: 64 x 16384 x 3 bf16 rows
// take 391 us forward, in tiles of 32 rows, and 332 backward; of 4 channels, in tiles of 128, 147 and 309.
Tiled forward_kernel(bool bf16, int64_t dim, bool z) {
  if (dim < 4) return bf16 ? forward_of<true, 1, 8>(z) : forward_of<false, 1, 8>(z);
  return bf16 ? forward_of<true, 4, 8>(z) : forward_of<false, 2, 8>(z);
}
Tiled backward_kernel(bool bf16, int64_t dim, bool z) {
  if (dim < 2) return bf16 ? backward_of<true, 1, 16>(z) : backward_of<false, 1, 16>(z);
  return bf16 ? backward_of<true, 2, 8>(z) : backward_of<false, 2, 8>(z);
}

// How the rows are cut: tiles of sequences by themselves where these are long enough that a last, shorter tile
// of each costs little; tiles of several whole sequences where these fill three quarters of one or more (then no
// tile waits: 2000 x 40 x 1024 bf16 rows forward, 120 of 128, 207 us for 218, 60 x 40 x 1024 15 for 20; backward, 40
// of 64, 496 for 401); else of all rows, which may share tiles.  The tiles and the bytes that they publish through
// (0 where no tile enters another).
//
// Rows of a sequence from which on it has tiles of its own.  64 sequences of 1536 channels (bf16, us forward and backward) in
// tiles of their own and across sequences: 192 rows 67 and 97 for 58 and 100, 200 rows 67 and 113 for 61 and 104;
// 256 rows 71 and 121 for 72 and 125, 384 rows 98 and 170 for 101 and 178, 700 rows 169 and 288 for 171 and 325, 32 of
// 1024 rows 120 and 218 for 128 and 235.  Lengths whose last tile is nearly empty lose up to about 600 rows: 260 rows 89 and
// 138 for 74 and 129, 400 rows 118 and 190 for 105 and 186; so does the backward in fp32, 200 x 256 x 256 61 and 117 for 61 and
// 108, 200 x 700 x 256 147 and 276 for 151 and 275.  (The checkpoints' layout goes by this length.)
constexpr int64_t kOwnTiles = 256;
struct Cut {
  int64_t tiles, each, pitch, published, words;  // each: of a sequence (0: shared); words: where they begin
};
int64_t chains_of(int64_t dim) { return (dim + ssm::kGatedChannels - 1) / ssm::kGatedChannels; }
ssm_status_t cut_rows(const Tiled& t, int64_t sequences, int64_t seqlen, int64_t rows, int64_t dim, Cut* out) {
  *out = Cut{};
  if (sequences > 1 && seqlen >= kOwnTiles) out->each = (seqlen + t.rows - 1) / t.rows;
  const int64_t held = sequences > 1 && seqlen > 0 ? t.rows / seqlen * seqlen : 0;  // rows of whole sequences
  const bool whole = held * 4 >= t.rows * 3;
  out->pitch = whole ? held : t.rows;
  out->tiles = out->each ? out->each * sequences : (rows + out->pitch - 1) / out->pitch;
  int64_t n;
  if (!mul_ok(chains_of(dim), out->tiles, &n) || n > kMaxBlocks) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  if (out->tiles <= 1 || whole) return SSM_OK;
  out->words = int64_t{ssm::kGatedQueues} * ssm::kGatedQueueWords * 4;  // behind the queues' counters
  if (!mul_ok(out->tiles, dim, &n) || !mul_ok(n, 8, &n) || __builtin_add_overflow(n, out->words + 15, &n))
    return fail(SSM_ERR_INVALID_ARG, "workspace size overflows int64");
  out->published = n / 16 * 16;
  return SSM_OK;
}

// a tile's rows are reached by 32-bit byte offsets
constexpr int64_t kMaxRowStride = int64_t{1} << 23;
static_assert(128 * kMaxRowStride * 4 <= int64_t{1} << 32, "128 rows of fp32");

ssm_status_t check_sizes(int64_t rows, int64_t dim, ssm_dtype_t dtype) {
  if (dim < 0) return fail(SSM_ERR_INVALID_ARG, "negative size (dim=%lld)", (long long)dim);
  if (dim >= kMaxRowStride) return fail(SSM_ERR_UNSUPPORTED, "dim %lld is not below 2^23", (long long)dim);
  if (rows > kMaxIndex) return fail(SSM_ERR_UNSUPPORTED, "more than 2^31-1 rows");
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  return SSM_OK;
}

ssm_status_t workspace_of(int64_t sequences, int64_t seqlen, int64_t rows, int64_t dim, bool bf16, bool backward,
                          int64_t* bytes) {
  *bytes = 0;
  if (rows == 0 || dim == 0) return SSM_OK;
  Cut c;
  SSM_TRY(cut_rows(backward ? backward_kernel(bf16, dim, true) : forward_kernel(bf16, dim, true), sequences, seqlen, rows,
                   dim, &c));
  *bytes = c.published;
  if (backward) {
    int64_t n;
    if (!mul_ok(c.tiles, dim, &n) || !mul_ok(n, 12, &n) || __builtin_add_overflow(*bytes, n, bytes))
      return fail(SSM_ERR_INVALID_ARG, "workspace size overflows int64");
  }
  return SSM_OK;
}

ssm_status_t check_params(const float* param, const float* ab, const float* xb, float scale) {
  if (!aligned(param, 4) || !aligned(ab, 4) || !aligned(xb, 4))
    return fail(SSM_ERR_MISALIGNED, "a_param, a_bias or x_bias is not 4-byte aligned");
  if (!(scale >= 0.0f) || std::isinf(scale))
    return fail(SSM_ERR_INVALID_ARG, "a_scale %g is not a finite number of at least 0", (double)scale);
  return SSM_OK;
}

ssm_status_t check_workspace(const void* workspace, int64_t bytes, int64_t need) {
  if (need == 0) return SSM_OK;
  if (!workspace || bytes < need)
    return fail(SSM_ERR_INVALID_ARG, "workspace of %lld bytes, need %lld", workspace ? (long long)bytes : 0ll,
                (long long)need);
  if (!aligned(workspace, 16)) return fail(SSM_ERR_MISALIGNED, "workspace (%p) is not 16-byte aligned", workspace);
  return SSM_OK;
}

// Clears the words that tiles publish and launches the kernel over all tiles.
ssm_status_t launch_tiles(const Tiled& t, ssm::GatedArgs& a, const Cut& cut, void* workspace, hipStream_t st,
                          const char* what) {
  const int64_t chains = chains_of(a.dim), grid = chains * cut.tiles;
  const int64_t words = cut.published / 16, blocks = (words + 255) / 256;
  if (blocks > kMaxBlocks) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  a.tiles = cut.tiles;
  a.each = cut.each;
  a.pitch = cut.pitch;
  a.chains = static_cast<int32_t>(chains);
  if (cut.published) {
    char* w = static_cast<char*>(workspace);
    a.ticket = reinterpret_cast<uint32_t*>(w);
    a.words = reinterpret_cast<uint64_t*>(w + cut.words);
    hipLaunchKernelGGL(ssm::gated_clear_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st,
                       reinterpret_cast<ssm::U32x4*>(w), words);
    SSM_TRY(check_launch("gated scan (clear)"));
  }
  hipLaunchKernelGGL(t.kernel, dim3(static_cast<unsigned>(grid)), dim3(ssm::kGatedThreads), 0, st, a);
  return check_launch(what);
}

ssm_status_t keep_states(const float* in, float* out, int64_t n, hipStream_t st) {
  const int64_t blocks = (n + 255) / 256;
  if (blocks > kMaxBlocks) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  hipLaunchKernelGGL(ssm::gated_keep_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, in, out, n);
  return check_launch("gated scan (states of no rows)");
}

struct Batch {
  int64_t rows, elems, bytes, states;  // bytes of a (batch, seqlen, dim) tensor and of a (batch, dim) fp32 one
  int64_t saved;                       // checkpoints
};
ssm_status_t check_batch(int64_t batch, int64_t seqlen, int64_t dim, ssm_dtype_t dtype, Batch* b) {
  if (batch < 0 || seqlen < 0 || dim < 0)
    return fail(SSM_ERR_INVALID_ARG, "negative size (batch=%lld seqlen=%lld dim=%lld)", (long long)batch,
                (long long)seqlen, (long long)dim);
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  if (!mul_ok(batch, seqlen, &b->rows) || !mul_ok(b->rows, dim, &b->elems) || !mul_ok(b->elems, es, &b->bytes) ||
      !mul_ok(batch, dim, &b->states) || !mul_ok(b->states, 4, &b->states))
    return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  if (batch > kMaxIndex) return fail(SSM_ERR_UNSUPPORTED, "batch exceeds int32");
  b->saved = batch > 1 && seqlen >= kOwnTiles ? batch * (seqlen / ssm::kGatedSave) : b->rows / ssm::kGatedSave;
  return check_sizes(b->rows, dim, dtype);
}

ssm_status_t first_misaligned(const Arg* args, size_t n) {
  if (const Arg* m = misaligned(args, n))
    return fail(SSM_ERR_MISALIGNED, "%s (%p) is not aligned to its element size", m->name, m->p);
  return SSM_OK;
}

}  // namespace

extern "C" {

ssm_status_t ssm_gated_scan_workspace(int64_t batch, int64_t seqlen, int64_t dim, ssm_dtype_t dtype, int backward,
                                      int64_t* bytes) {
  g_err[0] = '\0';
  if (!bytes) return fail(SSM_ERR_INVALID_ARG, "NULL bytes");
  Batch n;
  SSM_TRY(check_batch(batch, seqlen, dim, dtype, &n));
  return workspace_of(batch, seqlen, n.rows, dim, dtype == SSM_BF16, backward != 0, bytes);
}

ssm_status_t ssm_gated_scan_fwd(int64_t batch, int64_t seqlen, int64_t dim, ssm_dtype_t dtype, const void* x,
                                const void* a_gate, const void* x_gate, const float* a_param, const float* a_bias,
                                const float* x_bias, const void* z, float a_scale, const float* initial_state, void* y,
                                float* last_state, float* checkpoints, void* workspace, int64_t workspace_bytes,
                                void* stream) {
  g_err[0] = '\0';
  Batch n;
  SSM_TRY(check_batch(batch, seqlen, dim, dtype, &n));
  SSM_TRY(check_params(a_param, a_bias, x_bias, a_scale));
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  const Arg args[] = {{x, es, "x"}, {a_gate, es, "a_gate"}, {x_gate, es, "x_gate"}, {z, es, "z"}, {y, es, "y"},
                      {initial_state, 4, "initial_state"}, {last_state, 4, "last_state"}, {checkpoints, 4, "checkpoints"}};
  SSM_TRY(first_misaligned(args, sizeof args / sizeof *args));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Range r0{initial_state, n.states}, r1{last_state, n.states};
  if (n.elems == 0) {
    if (overlap(r0, r1)) return fail(SSM_ERR_INVALID_ARG, "an output overlaps an input");
    if (!last_state || n.states == 0) return SSM_OK;
    return keep_states(initial_state, last_state, n.states / 4, st);
  }
  if (!x || !a_gate || !x_gate || !a_param || !y)
    return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (x, a_gate, x_gate, a_param and y)");
  const Tiled t = forward_kernel(dtype == SSM_BF16, dim, z != nullptr);
  Cut cut;
  SSM_TRY(cut_rows(t, batch, seqlen, n.rows, dim, &cut));
  SSM_TRY(check_workspace(workspace, workspace_bytes, cut.published));
  const Range outs[] = {{y, n.bytes}, r1, {checkpoints, n.saved * dim * 4}, {workspace, cut.published}};
  const Range ins[] = {{x, n.bytes}, {a_gate, n.bytes}, {x_gate, n.bytes}, {z, n.bytes}, r0,
                       {a_param, dim * 4}, {a_bias, dim * 4}, {x_bias, dim * 4}};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));
  ssm::GatedArgs a{};
  a.x = x; a.ag = a_gate; a.xg = x_gate; a.z = z; a.y = y;
  a.param = a_param; a.ab = a_bias; a.xb = x_bias; a.scale = a_scale;
  a.sx = a.sag = a.sxg = a.sz = a.sy = dim;
  a.total = n.rows; a.dim = dim; a.seqlen = seqlen; a.nseq = batch;
  a.in = {const_cast<float*>(initial_state), batch, dim};
  a.out = {last_state, batch, dim};
  a.ckpt = checkpoints;
  return launch_tiles(t, a, cut, workspace, st, "gated scan");
}

ssm_status_t ssm_gated_scan_bwd(int64_t batch, int64_t seqlen, int64_t dim, ssm_dtype_t dtype, const void* x,
                                const void* a_gate, const void* x_gate, const float* a_param, const float* a_bias,
                                const float* x_bias, const void* z, float a_scale, const float* initial_state,
                                const float* checkpoints, const void* dy, const float* dlast_state, void* dx,
                                void* da_gate, void* dx_gate, float* da_param, float* da_bias, float* dx_bias, void* dz,
                                float* dinitial_state, void* workspace, int64_t workspace_bytes, void* stream) {
  g_err[0] = '\0';
  Batch n;
  SSM_TRY(check_batch(batch, seqlen, dim, dtype, &n));
  SSM_TRY(check_params(a_param, a_bias, x_bias, a_scale));
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  const Arg args[] = {{x, es, "x"}, {a_gate, es, "a_gate"}, {x_gate, es, "x_gate"}, {z, es, "z"}, {dy, es, "dy"},
                      {dx, es, "dx"}, {da_gate, es, "da_gate"}, {dx_gate, es, "dx_gate"}, {dz, es, "dz"},
                      {initial_state, 4, "initial_state"}, {checkpoints, 4, "checkpoints"},
                      {dlast_state, 4, "dlast_state"}, {da_param, 4, "da_param"}, {da_bias, 4, "da_bias"},
                      {dx_bias, 4, "dx_bias"}, {dinitial_state, 4, "dinitial_state"}};
  SSM_TRY(first_misaligned(args, sizeof args / sizeof *args));
  if (dim == 0) return SSM_OK;
  if (!a_param || !da_param) return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (a_param and da_param)");
  if (n.elems > 0 && (!x || !a_gate || !x_gate || !dy || !dx || !da_gate || !dx_gate))
    return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (x, a_gate, x_gate, dy, dx, da_gate and dx_gate)");
  if (n.elems > 0 && z && !dz) return fail(SSM_ERR_INVALID_ARG, "z needs dz");
  const Tiled t = backward_kernel(dtype == SSM_BF16, dim, z != nullptr);
  Cut cut;
  int64_t need;
  SSM_TRY(cut_rows(t, batch, seqlen, n.rows, dim, &cut));
  SSM_TRY(workspace_of(batch, seqlen, n.rows, dim, dtype == SSM_BF16, true, &need));
  SSM_TRY(check_workspace(workspace, workspace_bytes, need));
  const int64_t saved = n.saved * dim * 4;
  if (cut.tiles > 1 && !checkpoints) return fail(SSM_ERR_INVALID_ARG, "NULL checkpoints");
  const Range outs[] = {{dx, n.bytes}, {da_gate, n.bytes}, {dx_gate, n.bytes}, {z ? dz : nullptr, n.bytes},
                        {da_param, dim * 4}, {da_bias, dim * 4}, {dx_bias, dim * 4}, {dinitial_state, n.states},
                        {workspace, need}};
  const Range ins[] = {{x, n.bytes}, {a_gate, n.bytes}, {x_gate, n.bytes}, {z, n.bytes}, {dy, n.bytes},
                       {initial_state, n.states}, {checkpoints, saved}, {dlast_state, n.states},
                       {a_param, dim * 4}, {a_bias, dim * 4}, {x_bias, dim * 4}};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));
  hipStream_t st = static_cast<hipStream_t>(stream);
  ssm::GatedSumArgs sum{};
  sum.param = a_param; sum.dparam = da_param; sum.dab = da_bias; sum.dxb = dx_bias; sum.dim = dim;
  if (n.elems > 0) {
    ssm::GatedArgs a{};
    a.x = x; a.ag = a_gate; a.xg = x_gate; a.z = z; a.dy = dy;
    a.param = a_param; a.ab = a_bias; a.xb = x_bias; a.scale = a_scale;
    a.total = n.rows; a.dim = dim; a.seqlen = seqlen; a.nseq = batch;
    a.in = {const_cast<float*>(initial_state), batch, dim};
    a.ckpt = const_cast<float*>(checkpoints);
    a.dlast = dlast_state; a.dx = dx; a.dag = da_gate; a.dxg = dx_gate; a.dz = dz; a.dh0 = dinitial_state;
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + cut.published);
    a.dparam = da_param; a.dab = da_bias; a.dxb = dx_bias;
    sum.partial = a.partial;
    sum.tiles = cut.tiles;
    SSM_TRY(launch_tiles(t, a, cut, workspace, st, "gated scan backward"));
    if (cut.tiles == 1) return SSM_OK;  // it has the sums
  } else if (dinitial_state && n.states > 0) {
    SSM_TRY(keep_states(dlast_state, dinitial_state, n.states / 4, st));
  }
  const int64_t blocks = (dim + 63) / 64;
  if (blocks > kMaxBlocks / 4) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  hipLaunchKernelGGL(ssm::gated_sum_kernel, dim3(static_cast<unsigned>(blocks), 3), dim3(ssm::kGatedSumThreads), 0, st,
                     sum);
  return check_launch("gated scan backward (sums)");
}

ssm_status_t ssm_gated_scan_packed_fwd(const ssm_packed_t* seqs, int64_t dim, ssm_dtype_t dtype, const void* x,
                                       const void* a_gate, const void* x_gate, const float* a_param,
                                       const float* a_bias, const float* x_bias, const void* z, float a_scale, void* y,
                                       const ssm_cache_t* cache, const ssm_gated_strides_t* strides, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
  g_err[0] = '\0';
  SSM_TRY(check_packed(seqs));
  SSM_TRY(check_sizes(seqs->total, dim, dtype));
  SSM_TRY(check_params(a_param, a_bias, x_bias, a_scale));
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  ssm::GatedArgs a{};
  Range rc{nullptr, 0};
  if (cache) SSM_TRY(check_cache(cache, dim, &a.in, &rc));
  ssm_gated_strides_t rs = strides ? *strides : ssm_gated_strides_t{};
  Rows t[] = {{x, dim, &rs.x, "x", 0}, {a_gate, dim, &rs.a_gate, "a_gate", 0}, {x_gate, dim, &rs.x_gate, "x_gate", 0},
              {z, dim, &rs.z, "z", 0}, {y, dim, &rs.y, "y", 0}};
  SSM_TRY(check_rows(t, 5, seqs->total, es));
  for (const Rows& r : t) {
    if (seqs->total <= 1) *r.stride = dim;  // there is no next row, whatever the distance to it
    if (*r.stride >= kMaxRowStride)
      return fail(SSM_ERR_UNSUPPORTED, "row stride %lld of %s is not below 2^23", (long long)*r.stride, r.name);
  }
  if (seqs->total == 0 || seqs->sequences == 0 || dim == 0) return SSM_OK;
  if (!x || !a_gate || !x_gate || !a_param || !y)
    return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (x, a_gate, x_gate, a_param and y)");
  Range idx[3];
  SSM_TRY(check_packed_pointers(seqs, idx));
  const Tiled k = forward_kernel(dtype == SSM_BF16, dim, z != nullptr);
  Cut cut;
  SSM_TRY(cut_rows(k, 1, seqs->total, seqs->total, dim, &cut));
  SSM_TRY(check_workspace(workspace, workspace_bytes, cut.published));
  const Range outs[] = {{y, t[4].bytes}, rc, {workspace, cut.published}};
  const Range ins[] = {{x, t[0].bytes}, {a_gate, t[1].bytes}, {x_gate, t[2].bytes}, {z, t[3].bytes}, {a_param, dim * 4},
                       {a_bias, dim * 4}, {x_bias, dim * 4}, idx[0], idx[1], idx[2]};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));
  a.x = x; a.ag = a_gate; a.xg = x_gate; a.z = z; a.y = y;
  a.param = a_param; a.ab = a_bias; a.xb = x_bias; a.scale = a_scale;
  a.sx = rs.x; a.sag = rs.a_gate; a.sxg = rs.x_gate; a.sz = rs.z; a.sy = rs.y;
  a.total = seqs->total; a.dim = dim; a.nseq = seqs->sequences;
  a.cu = seqs->cu_seqlens; a.slots = seqs->cache_slots; a.has_initial = seqs->has_initial;
  a.out = a.in;
  a.cb16 = cache && cache->dtype == SSM_BF16;
  return launch_tiles(k, a, cut, workspace, static_cast<hipStream_t>(stream), "gated scan (packed)");
}

ssm_status_t ssm_gated_update_cache(int64_t batch, int64_t dim, ssm_dtype_t dtype, const ssm_cache_t* cache,
                                    const int32_t* cache_slots, const void* x, const void* a_gate, const void* x_gate,
                                    const float* a_param, const float* a_bias, const float* x_bias, const void* z,
                                    float a_scale, void* y, const ssm_gated_strides_t* strides, void* stream) {
  g_err[0] = '\0';
  if (batch < 0) return fail(SSM_ERR_INVALID_ARG, "bad size (batch=%lld)", (long long)batch);
  SSM_TRY(check_sizes(batch, dim, dtype));
  SSM_TRY(check_params(a_param, a_bias, x_bias, a_scale));
  if (!cache) return fail(SSM_ERR_INVALID_ARG, "NULL cache");
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  ssm::GatedStepArgs q{};
  ssm::GatedArgs& a = q.g;
  Range rc;
  SSM_TRY(check_cache(cache, dim, &a.in, &rc));
  ssm_gated_strides_t rs = strides ? *strides : ssm_gated_strides_t{};
  Rows t[] = {{x, dim, &rs.x, "x", 0}, {a_gate, dim, &rs.a_gate, "a_gate", 0}, {x_gate, dim, &rs.x_gate, "x_gate", 0},
              {z, dim, &rs.z, "z", 0}, {y, dim, &rs.y, "y", 0}};
  SSM_TRY(check_rows(t, 5, batch, es));
  if (batch == 0 || dim == 0 || cache->slots == 0) return SSM_OK;
  if (!x || !a_gate || !x_gate || !a_param || !y)
    return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (x, a_gate, x_gate, a_param and y)");
  if (!aligned(cache_slots, 4)) return fail(SSM_ERR_MISALIGNED, "cache_slots is not 4-byte aligned");
  const Range outs[] = {{y, t[4].bytes}, rc};
  const Range ins[] = {{x, t[0].bytes}, {a_gate, t[1].bytes}, {x_gate, t[2].bytes}, {z, t[3].bytes}, {a_param, dim * 4},
                       {a_bias, dim * 4}, {x_bias, dim * 4}, {cache_slots, batch * 4}};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));
  a.x = x; a.ag = a_gate; a.xg = x_gate; a.z = z; a.y = y;
  a.param = a_param; a.ab = a_bias; a.xb = x_bias; a.scale = a_scale;
  a.sx = rs.x; a.sag = rs.a_gate; a.sxg = rs.x_gate; a.sz = rs.z; a.sy = rs.y;
  a.dim = dim; a.slots = cache_slots; q.batch = batch;
  const bool bf16 = dtype == SSM_BF16, cb16 = cache->dtype == SSM_BF16;
  using Kernel = void (*)(const ssm::GatedStepArgs);
  const int64_t v = dim < 4 ? 1 : 4;
  const int64_t blocks = ((dim + v - 1) / v + ssm::kGatedThreads - 1) / ssm::kGatedThreads;
  if (blocks > kMaxBlocks) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  const int R = v == 4 ? step_entries(blocks, batch) : 1;
  const auto pick = [&](auto B, auto C) -> Kernel {
    constexpr bool b = decltype(B)::value, c = decltype(C)::value;
    return v == 1 ? ssm::gated_step_kernel<b, c, 1, 1>
                  : R > 1 ? ssm::gated_step_kernel<b, c, 4, kStepEntries> : ssm::gated_step_kernel<b, c, 4, 1>;
  };
  using T = std::true_type;
  using F = std::false_type;
  const Kernel k = bf16 ? (cb16 ? pick(T{}, T{}) : pick(T{}, F{})) : (cb16 ? pick(F{}, T{}) : pick(F{}, F{}));
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(blocks), grid_y((batch + R - 1) / R)), dim3(ssm::kGatedThreads), 0,
                     static_cast<hipStream_t>(stream), q);
  return check_launch("gated step (cache)");
}

}  // extern "C"
