// cache_host.hpp -- host-side checks and launch helpers that the serving entry points share.
#pragma once

#include "cache.hpp"
#include "host_util.hpp"

namespace ssm_host {

constexpr int64_t kMaxIndex = 0x7fffffff;
// workgroups along x: a launch has at most 2^32 - 1 threads in a dimension
constexpr int64_t kMaxBlocks = 0xffffffffll / 256;

// bytes from the first to the last element of `rows` rows of `width` elements, or -1
inline int64_t span_bytes(int64_t rows, int64_t stride, int64_t width, int64_t es) {
  int64_t n;
  if (rows <= 0 || width <= 0) return 0;
  if (!mul_ok(rows - 1, stride, &n) || __builtin_add_overflow(n, width, &n) || !mul_ok(n, es, &n)) return -1;
  return n;
}

// a tensor of rows: its row stride checked and 0 replaced, its span for the overlap check
struct Rows {
  const void* p;
  int64_t width;
  int64_t* stride;
  const char* name;
  int64_t bytes;
};

inline ssm_status_t check_rows(Rows* r, size_t n, int64_t rows, int64_t es) {
  for (size_t i = 0; i < n; ++i) {
    if (*r[i].stride == 0) *r[i].stride = r[i].width;
    if (*r[i].stride < r[i].width)
      return fail(SSM_ERR_INVALID_ARG, "row stride %lld of %s is below its row of %lld elements",
                  (long long)*r[i].stride, r[i].name, (long long)r[i].width);
    if (!aligned(r[i].p, static_cast<uintptr_t>(es)))
      return fail(SSM_ERR_MISALIGNED, "%s (%p) is not aligned to its element size", r[i].name, r[i].p);
    r[i].bytes = span_bytes(rows, *r[i].stride, r[i].width, es);
    if (r[i].bytes < 0) return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  }
  return SSM_OK;
}

// The cache's fields, its entries of `entry` elements
inline ssm_status_t check_cache(const ssm_cache_t* c, int64_t entry, ssm::CacheRef* ref, Range* range) {
  if (c->reserved != 0) return fail(SSM_ERR_INVALID_ARG, "ssm_cache_t.reserved must be zero");
  if (c->dtype != SSM_F32 && c->dtype != SSM_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "unknown cache dtype %d", (int)c->dtype);
  if (c->slots < 0 || c->slots > kMaxIndex)
    return fail(SSM_ERR_INVALID_ARG, "cache slots %lld not in 0..2^31-1", (long long)c->slots);
  const int64_t es = c->dtype == SSM_BF16 ? 2 : 4;
  const int64_t stride = c->slot_stride == 0 ? entry : c->slot_stride;
  if (stride < entry)
    return fail(SSM_ERR_INVALID_ARG, "slot_stride %lld is below a slot's %lld elements", (long long)stride,
                (long long)entry);
  if (!c->data && c->slots > 0 && entry > 0) return fail(SSM_ERR_INVALID_ARG, "NULL cache data");
  if (!aligned(c->data, static_cast<uintptr_t>(es)))
    return fail(SSM_ERR_MISALIGNED, "cache (%p) is not aligned to its element size", c->data);
  const int64_t bytes = span_bytes(c->slots, stride, entry, es);
  if (bytes < 0) return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  ref->data = c->slots > 0 ? c->data : nullptr;
  ref->slots = c->slots;
  ref->stride = stride;
  *range = {c->data, bytes};
  return SSM_OK;
}

inline ssm_status_t check_packed(const ssm_packed_t* q) {
  if (!q) return fail(SSM_ERR_INVALID_ARG, "NULL seqs");
  if (q->total < 0 || q->sequences < 0 || q->max_seqlen < 0 || q->total > kMaxIndex || q->sequences > kMaxIndex ||
      q->max_seqlen > kMaxIndex)
    return fail(SSM_ERR_INVALID_ARG, "total %lld, sequences %lld and max_seqlen %lld must be in 0..2^31-1",
                (long long)q->total, (long long)q->sequences, (long long)q->max_seqlen);
  return SSM_OK;
}

inline ssm_status_t check_packed_pointers(const ssm_packed_t* q, Range out[3]) {
  if (!q->cu_seqlens) return fail(SSM_ERR_INVALID_ARG, "NULL cu_seqlens");
  if (!aligned(q->cu_seqlens, 4) || !aligned(q->cache_slots, 4))
    return fail(SSM_ERR_MISALIGNED, "cu_seqlens or cache_slots is not 4-byte aligned");
  out[0] = {q->cu_seqlens, (q->sequences + 1) * 4};
  out[1] = {q->cache_slots, q->sequences * 4};
  out[2] = {q->has_initial, q->sequences};
  return SSM_OK;
}

// outputs against inputs and against each other
inline ssm_status_t check_overlap(const Range* outs, size_t n_out, const Range* ins, size_t n_in) {
  for (size_t i = 0; i < n_out; ++i) {
    for (size_t j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j])) return fail(SSM_ERR_INVALID_ARG, "an output overlaps an input");
    for (size_t j = i + 1; j < n_out; ++j)
      if (overlap(outs[i], outs[j])) return fail(SSM_ERR_INVALID_ARG, "two outputs overlap");
  }
  return SSM_OK;
}

template <size_t N>
constexpr size_t count_of(const Range (&)[N]) {
  return N;
}

inline ssm_row_strides_t strides_or_zero(const ssm_row_strides_t* s) { return s ? *s : ssm_row_strides_t{}; }

// Entries of a batch that a thread of a step takes: several once that leaves a few workgroups per CU.
constexpr int kStepEntries = 4;
inline int step_entries(int64_t blocks, int64_t batch) {
  return blocks * ((batch + kStepEntries - 1) / kStepEntries) >= device_cus() ? kStepEntries : 1;
}

// rows of a batch along gridDim.y, whose limit the kernels' loops step over
inline unsigned grid_y(int64_t rows) { return static_cast<unsigned>(rows < 65535 ? rows : 65535); }

#define SSM_TRY(call)                       \
  do {                                      \
    const ssm_status_t st_ = (call);        \
    if (st_ != SSM_OK) return st_;          \
  } while (0)

}  // namespace ssm_host
