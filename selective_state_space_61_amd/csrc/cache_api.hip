// cache_api.hip -- the serving entry points of include/ssm.h (packed prompts, steps on a cache of
// slots, states set aside in 8 bits): host-side validation, launch shapes and launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/ssm.h"
#include "cache_host.hpp"
#include "cache_q8.hpp"
#include "cache_step.hpp"
#include "conv1d_packed.hpp"
#include "scan_packed.hpp"

using namespace ssm_host;

namespace {

using ConvPackedKernel = void (*)(const ssm::ConvPackedArgs);
template <bool BF16, int T>
ConvPackedKernel conv_packed_kernel(int64_t width) {
  switch (width) {
    case 1: return ssm::conv1d_packed_kernel<BF16, 1, T>;
    case 2: return ssm::conv1d_packed_kernel<BF16, 2, T>;
    case 3: return ssm::conv1d_packed_kernel<BF16, 3, T>;
    case 4: return ssm::conv1d_packed_kernel<BF16, 4, T>;
    default: return nullptr;
  }
}

using ConvStepKernel = void (*)(const ssm::ConvStepArgs);
template <bool BF16, int R>
ConvStepKernel conv_step_kernel(int64_t width) {
  switch (width) {
    case 1: return ssm::conv1d_update_cache_kernel<BF16, 1, R>;
    case 2: return ssm::conv1d_update_cache_kernel<BF16, 2, R>;
    case 3: return ssm::conv1d_update_cache_kernel<BF16, 3, R>;
    case 4: return ssm::conv1d_update_cache_kernel<BF16, 4, R>;
    default: return nullptr;
  }
}

// kernels by dstate: K<BF16, CB16, N> for the four pairs of storage types
template <template <bool, bool, int> class K, int... N>
auto by_dstate(bool bf16, bool cb16, int64_t n) {
  decltype(K<true, true, 16>::get()) k = nullptr;
  ((n == N ? (void)(k = bf16 ? (cb16 ? K<true, true, N>::get() : K<true, false, N>::get())
                              : (cb16 ? K<false, true, N>::get() : K<false, false, N>::get()))
           : (void)0),
   ...);
  return k;
}
template <int R>
struct StateStepOf {
  template <bool BF16, bool CB16, int N>
  struct K {
    static auto get() { return &ssm::state_update_cache_kernel<BF16, CB16, N, R>; }
  };
};
template <bool BF16, bool CB16, int N>
struct SsdStep {
  static auto get() { return &ssm::ssd_state_update_cache_kernel<BF16, CB16, N>; }
};
using Q8Kernel = void (*)(const ssm::Q8Args);
template <bool CB16>
Q8Kernel q8_kernel(bool store, int64_t n) {
  switch (n) {
#define SSM_Q8(N) \
  case N: return store ? ssm::cache_store_q8_kernel<CB16, N> : ssm::cache_load_q8_kernel<CB16, N>
    SSM_Q8(1);
    SSM_Q8(2);
    SSM_Q8(4);
    SSM_Q8(8);
    SSM_Q8(16);
    SSM_Q8(32);
    SSM_Q8(64);
    SSM_Q8(128);
    SSM_Q8(256);
#undef SSM_Q8
    default: return nullptr;
  }
}

ssm_status_t q8_call(bool store, int64_t count, int64_t rows, int64_t dstate, const ssm_cache_t* cache,
                     const int32_t* cache_slots, int64_t stored, int8_t* codes, float* scales,
                     const int32_t* store_slots, void* stream) {
  if (count < 0 || rows < 0 || dstate < 0 || stored < 0 || stored > kMaxIndex || count > kMaxIndex)
    return fail(SSM_ERR_INVALID_ARG, "bad size (count=%lld rows=%lld dstate=%lld stored=%lld)", (long long)count,
                (long long)rows, (long long)dstate, (long long)stored);
  if (!cache) return fail(SSM_ERR_INVALID_ARG, "NULL cache");
  const bool cb16 = cache->dtype == SSM_BF16;
  const Q8Kernel k = cb16 ? q8_kernel<true>(store, dstate) : q8_kernel<false>(store, dstate);
  if (!k) return fail(SSM_ERR_UNSUPPORTED, "dstate %lld is not a power of two up to 256", (long long)dstate);
  int64_t entry, entry_bytes, n_codes, n_scales;
  if (!mul_ok(rows, dstate, &entry) || !mul_ok(entry, 4, &entry_bytes) || !mul_ok(entry, stored, &n_codes) ||
      !mul_ok(rows * 4, stored, &n_scales))
    return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  ssm::Q8Args a{};
  Range rc;
  SSM_TRY(check_cache(cache, entry, &a.cache, &rc));
  if (count == 0 || rows == 0 || stored == 0 || cache->slots == 0) return SSM_OK;
  if (!codes || !scales) return fail(SSM_ERR_INVALID_ARG, "NULL codes or scales");
  if (!aligned(scales, 4) || !aligned(cache_slots, 4) || !aligned(store_slots, 4))
    return fail(SSM_ERR_MISALIGNED, "scales, cache_slots or store_slots is not 4-byte aligned");
  const Range rq{codes, n_codes}, rs{scales, n_scales}, i1{cache_slots, count * 4}, i2{store_slots, count * 4};
  const Range kept[] = {rq, rs}, live[] = {rc};
  const Range in_s[] = {rc, i1, i2}, in_l[] = {rq, rs, i1, i2};
  if (store) SSM_TRY(check_overlap(kept, 2, in_s, 3));
  else SSM_TRY(check_overlap(live, 1, in_l, 4));
  const int64_t v = cb16 ? (dstate < 8 ? dstate : 8) : (dstate < 4 ? dstate : 4);
  const int64_t per = static_cast<int64_t>(ssm::kQ8Threads) / (dstate / v) * ssm::kQ8Rows;
  const int64_t blocks = (rows + per - 1) / per;
  if (blocks > kMaxBlocks) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  a.cache_slots = cache_slots; a.codes = codes; a.scales = scales; a.store_slots = store_slots;
  a.stored = stored; a.count = count; a.rows = rows;
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(blocks), grid_y(count)), dim3(ssm::kQ8Threads), 0,
                     static_cast<hipStream_t>(stream), a);
  return check_launch(store ? "cache store (8 bits)" : "cache load (8 bits)");
}

// sizes, dtype and dstate of the packed scan
ssm_status_t check_scan_packed(const ssm_packed_t* seqs, int64_t dim, int64_t dstate, ssm_dtype_t dtype) {
  SSM_TRY(check_packed(seqs));
  if (dim < 0 || dstate < 0)
    return fail(SSM_ERR_INVALID_ARG, "negative size (dim=%lld dstate=%lld)", (long long)dim, (long long)dstate);
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (!ssm::scan_packed_kernels(dtype == SSM_BF16, dstate))
    return fail(SSM_ERR_UNSUPPORTED, "dstate %lld not in {1,2,4,8,16,32,64}", (long long)dstate);
  return SSM_OK;
}

// Launch shape of the packed scan: rows per piece (0: whole sequences), the bound on the pieces of
// all sequences and the workspace that they need.
struct ScanPackedShape {
  int64_t piece, pieces, ncb, floats;
};

// Rows per piece (0: whole sequences), by a model of the two launches from what was measured on MI355X
// (dstate 16, bf16; other dstates by the factors below): a wave alone on its SIMD takes 85 ns a row and
// m waves that share one 54 + 24 / m ns each (full pass), 62 and 34 + 32 / m ns without read-outs, where a
// sequence's last piece is left out; the second launch and the pieces' set-up take 8 us; composing the
// states of 8 pieces takes 2 us (linear in the pieces, where the reads of their states are not: too little
// past some 100000 rows).  Pieces are no longer than an eighth of the longest sequence, or 32 rows: of
// fewer, ragged ones the model knows too little (24 of 30000 x 1536: 402 us with 1024 rows, 300 with 384).
// Both sides, whole | in pieces of the chosen length, in us: one sequence of 8192 x 1536: 661 | 93; of 512:
// 45 | 19; 11 ragged ones of 11003 x 1536: 218 | 117; 8 of 2048 x 1536: 173 | 159; 16 of 512 x 1536: 71 | 79
// (whole is chosen); 32 of 2048 x 1536: 377 | 575 (whole).  Over 55 bf16 shapes (35 of dstate 16, the others
// of 1, 2, 4, 8, 32 and 64) the choice is 2.8% off the best of these lengths on average, 14% at worst; there
// is no term for fp32 rows.
int64_t scan_packed_piece(int64_t total, int64_t sequences, int64_t longest, int64_t waves, int64_t dstate) {
  const double per_simd = static_cast<double>(waves) / (4.0 * device_cus());  // waves of a sequence's channels
  const double states = static_cast<double>(dstate < 4 ? 4 : dstate);
  const double scale = 0.45 + 0.55 * states / 16.0;                            // of a wave alone
  const double work = dstate == 16 ? 1.0 : (139.0 + 20.0 * states) / 395.0;  // VALU instructions, where waves share
  const double rows = static_cast<double>(total), n = static_cast<double>(sequences);
  // a pass over `count` pieces of up to `length` rows, `sum` rows in all; the fullest SIMD has one of
  // `length` rows and others of `mean` where all run at once
  auto pass = [&](double length, double mean, double count, double sum, double alone, double shared, double rest) {
    const double m = std::ceil(count * per_simd);
    const double queue = m <= 4.0 ? length + (m - 1.0) * mean : sum * per_simd + 0.3 * length;
    const double busy = m <= 1.0 ? 0.0 : work * (shared + rest / (m < 4.0 ? m : 4.0)) * queue;
    const double one = scale * alone * length;
    return busy > one ? busy : one;
  };
  const double most = static_cast<double>(longest);
  double best = pass(most, rows / n, n, rows, 0.085, 0.054, 0.024);
  int64_t piece = 0;
  for (int64_t p : {32, 48, 64, 96, 128, 160, 192, 256, 384, 512, 768, 1024}) {
    if (p >= longest || (p > 32 && 8 * p > longest)) break;
    const double length = static_cast<double>(p);
    // of sequences of about one length every piece but the last is full; of others the last is half
    // full on average
    const double count = rows >= 0.9 * n * most ? n * std::ceil(most / length) : rows / length + 0.5 * n;
    const double first = count > n ? count - n : 0.0;
    const double t = pass(length, length, count, rows, 0.085, 0.054, 0.024) +
                     pass(length, length, first, first * length < rows ? first * length : rows, 0.062, 0.034, 0.032) +
                     8.0 + 2.0 * most / (8.0 * length);
    if (t < best) {
      best = t;
      piece = p;
    }
  }
  return piece;
}

ssm_status_t scan_packed_shape(const ssm_packed_t* seqs, int64_t dim, int64_t dstate, ScanPackedShape* out) {
  const int64_t ncb = (dim + 16 * ssm::kPackedWaves - 1) / (16 * ssm::kPackedWaves);
  const int64_t longest =
      seqs->max_seqlen > 0 && seqs->max_seqlen < seqs->total ? seqs->max_seqlen : seqs->total;
  const int64_t piece = scan_packed_piece(seqs->total, seqs->sequences, longest, (dim + 15) / 16, dstate);
  out->piece = piece;
  out->ncb = ncb;
  out->pieces = piece ? seqs->total / piece + seqs->sequences : seqs->sequences;
  out->floats = 0;
  if (piece && (!mul_ok(out->pieces, dim, &out->floats) || !mul_ok(out->floats, (dstate + 1) * 4, &out->floats)))
    return fail(SSM_ERR_INVALID_ARG, "workspace size overflows int64");
  out->floats /= 4;
  return SSM_OK;
}

}  // namespace

extern "C" {

ssm_status_t ssm_causal_conv1d_packed_fwd(const ssm_packed_t* seqs, int64_t dim, int64_t width, ssm_dtype_t dtype,
                                          const void* x, const float* weight, const float* bias, int silu, void* y,
                                          const ssm_cache_t* cache, const ssm_row_strides_t* strides, void* stream) {
  g_err[0] = '\0';
  SSM_TRY(check_packed(seqs));
  if (dim < 0 || width < 0)
    return fail(SSM_ERR_INVALID_ARG, "negative size (dim=%lld width=%lld)", (long long)dim, (long long)width);
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (width < 1 || width > 4) return fail(SSM_ERR_UNSUPPORTED, "width %lld not in 1..4", (long long)width);
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  int64_t n_w, entry;
  if (!mul_ok(dim, width * 4, &n_w) || !mul_ok(dim, width - 1, &entry))
    return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  ssm::ConvPackedArgs a{};
  Range rc{nullptr, 0};
  if (cache) {
    if (cache->dtype != dtype) return fail(SSM_ERR_INVALID_ARG, "the cache's dtype differs from x's");
    SSM_TRY(check_cache(cache, entry, &a.cache, &rc));
  }
  ssm_row_strides_t rs = strides_or_zero(strides);
  Rows t[] = {{x, dim, &rs.x, "x", 0}, {y, dim, &rs.y, "y", 0}};
  SSM_TRY(check_rows(t, 2, seqs->total, es));
  if (seqs->total == 0 || seqs->sequences == 0 || dim == 0) return SSM_OK;
  if (!x || !weight || !y) return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (x, weight and y)");
  Range idx[3];
  SSM_TRY(check_packed_pointers(seqs, idx));
  if (!aligned(weight, 4) || !aligned(bias, 4))
    return fail(SSM_ERR_MISALIGNED, "weight or bias is not 4-byte aligned");
  const Range outs[] = {{y, t[1].bytes}, rc};
  const Range ins[] = {{x, t[0].bytes}, {weight, n_w}, {bias, dim * 4}, idx[0], idx[1], idx[2]};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));

  const int64_t vec = dtype == SSM_BF16 ? ssm::kConvVec<true> : ssm::kConvVec<false>;
  a.x = x; a.weight = weight; a.bias = bias; a.y = y;
  a.cu = seqs->cu_seqlens; a.slots = seqs->cache_slots; a.has_initial = seqs->has_initial;
  a.total = seqs->total; a.nseq = seqs->sequences; a.dim = dim; a.sx = rs.x; a.sy = rs.y;
  a.silu = silu ? 1 : 0;
  const int64_t ncv = (dim + vec - 1) / vec;
  const int64_t ncb = (ncv + ssm::kConvThreads - 1) / ssm::kConvThreads;
  const int64_t large = (seqs->total + ssm::kPackTile - 1) / ssm::kPackTile;
  const bool small = large * ncb < 2 * device_cus() || seqs->sequences > large;
  const int64_t ntiles = small ? (seqs->total + ssm::kPackTileSmall - 1) / ssm::kPackTileSmall : large;
  int64_t grid;
  if (ncb > kMaxBlocks || !mul_ok(ncb, ntiles, &grid) || grid > kMaxBlocks)
    return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  a.ncb = static_cast<int32_t>(ncb);
  const bool bf16 = dtype == SSM_BF16;
  const ConvPackedKernel k =
      small ? (bf16 ? conv_packed_kernel<true, ssm::kPackTileSmall>(width) : conv_packed_kernel<false, ssm::kPackTileSmall>(width))
            : (bf16 ? conv_packed_kernel<true, ssm::kPackTile>(width) : conv_packed_kernel<false, ssm::kPackTile>(width));
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(grid)), dim3(ssm::kConvThreads), 0,
                     static_cast<hipStream_t>(stream), a);
  return check_launch("causal conv1d (packed)");
}

ssm_status_t ssm_scan_packed_workspace(const ssm_packed_t* seqs, int64_t dim, int64_t dstate, ssm_dtype_t dtype,
                                       int64_t* bytes) {
  g_err[0] = '\0';
  if (!bytes) return fail(SSM_ERR_INVALID_ARG, "NULL bytes");
  SSM_TRY(check_scan_packed(seqs, dim, dstate, dtype));
  *bytes = 0;
  if (seqs->total == 0 || seqs->sequences == 0 || dim == 0) return SSM_OK;
  ScanPackedShape shape;
  SSM_TRY(scan_packed_shape(seqs, dim, dstate, &shape));
  *bytes = shape.floats * 4;
  return SSM_OK;
}

ssm_status_t ssm_scan_packed_fwd(const ssm_packed_t* seqs, int64_t dim, int64_t dstate, ssm_dtype_t dtype,
                                 const void* x, const void* delta, const float* A, const void* B, const void* C,
                                 const float* D, const void* z, const float* delta_bias, int delta_softplus, void* y,
                                 const ssm_cache_t* cache, const ssm_row_strides_t* strides, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
  g_err[0] = '\0';
  SSM_TRY(check_scan_packed(seqs, dim, dstate, dtype));
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  int64_t entry, n_dn;
  if (!mul_ok(dim, dstate, &entry) || !mul_ok(entry, 4, &n_dn))
    return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  ssm::ScanPackedArgs a{};
  Range rc{nullptr, 0};
  const bool cb16 = cache && cache->dtype == SSM_BF16;
  if (cache) SSM_TRY(check_cache(cache, entry, &a.cache, &rc));
  ssm_row_strides_t rs = strides_or_zero(strides);
  Rows t[] = {{x, dim, &rs.x, "x", 0},        {delta, dim, &rs.delta, "delta", 0}, {B, dstate, &rs.B, "B", 0},
              {C, dstate, &rs.C, "C", 0},     {z, dim, &rs.z, "z", 0},             {y, dim, &rs.y, "y", 0}};
  SSM_TRY(check_rows(t, 6, seqs->total, es));
  if (seqs->total == 0 || seqs->sequences == 0 || dim == 0) return SSM_OK;
  if (!x || !delta || !A || !B || !C || !y)
    return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (x, delta, A, B, C and y)");
  Range idx[3];
  SSM_TRY(check_packed_pointers(seqs, idx));
  if (!aligned(A, 4) || !aligned(D, 4) || !aligned(delta_bias, 4))
    return fail(SSM_ERR_MISALIGNED, "A, D or delta_bias is not 4-byte aligned");
  for (const Rows& r : t)
    if (*r.stride >= ssm::kScanPackedMaxStride)
      return fail(SSM_ERR_UNSUPPORTED, "row stride %lld of %s is not below 2^24", (long long)*r.stride, r.name);
  ScanPackedShape shape;
  SSM_TRY(scan_packed_shape(seqs, dim, dstate, &shape));
  if (shape.floats > 0) {
    if (!workspace || workspace_bytes < shape.floats * 4)
      return fail(SSM_ERR_INVALID_ARG, "workspace of %lld bytes, %lld are needed",
                  (long long)(workspace ? workspace_bytes : 0), (long long)(shape.floats * 4));
    if (!aligned(workspace, 16)) return fail(SSM_ERR_MISALIGNED, "workspace (%p) is not 16-byte aligned", workspace);
  }
  const Range outs[] = {{y, t[5].bytes}, rc, {workspace, shape.floats * 4}};
  const Range ins[] = {{x, t[0].bytes}, {delta, t[1].bytes}, {B, t[2].bytes}, {C, t[3].bytes}, {z, t[4].bytes},
                       {A, n_dn},       {D, dim * 4},        {delta_bias, dim * 4}, idx[0], idx[1], idx[2]};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));

  a.x = x; a.delta = delta; a.A = A; a.B = B; a.C = C; a.Dskip = D; a.z = z; a.delta_bias = delta_bias; a.y = y;
  a.cu = seqs->cu_seqlens; a.slots = seqs->cache_slots; a.has_initial = seqs->has_initial;
  a.total = seqs->total; a.nseq = seqs->sequences; a.dim = dim;
  a.sx = rs.x; a.sdelta = rs.delta; a.sB = rs.B; a.sC = rs.C; a.sz = rs.z; a.sy = rs.y;
  a.softplus = delta_softplus ? 1 : 0;
  a.cache_bf16 = cb16 ? 1 : 0;
  a.piece = static_cast<int32_t>(shape.piece);
  a.pieces = shape.pieces;
  a.ncb = static_cast<int32_t>(shape.ncb);
  if (shape.piece) {
    a.seg_state = static_cast<float*>(workspace);
    a.seg_dsum = a.seg_state + shape.pieces * dim * dstate;
  }
  int64_t blocks;
  if (!mul_ok(shape.pieces, shape.ncb, &blocks) || blocks > kMaxBlocks)
    return fail(SSM_ERR_UNSUPPORTED, "grid of %lld x %lld workgroups is too large", (long long)shape.pieces,
                (long long)shape.ncb);
  const ssm::ScanPackedKernels& k = *ssm::scan_packed_kernels(dtype == SSM_BF16, dstate);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (shape.piece) {
    hipLaunchKernelGGL(k.agg, dim3(static_cast<unsigned>(blocks)), dim3(64 * ssm::kPackedWaves), 0, st, a);
    SSM_TRY(check_launch("scan (packed, pieces' states)"));
  }
  hipLaunchKernelGGL(k.full, dim3(static_cast<unsigned>(blocks)), dim3(64 * ssm::kPackedWaves), 0, st, a);
  return check_launch("scan (packed)");
}

ssm_status_t ssm_causal_conv1d_update_cache(int64_t batch, int64_t dim, int64_t width, ssm_dtype_t dtype,
                                            const ssm_cache_t* cache, const int32_t* cache_slots, const void* x,
                                            const float* weight, const float* bias, int silu, void* y,
                                            const ssm_row_strides_t* strides, void* stream) {
  g_err[0] = '\0';
  if (batch < 0 || dim < 0 || width < 0 || batch > kMaxIndex)
    return fail(SSM_ERR_INVALID_ARG, "bad size (batch=%lld dim=%lld width=%lld)", (long long)batch, (long long)dim,
                (long long)width);
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (width < 1 || width > 4) return fail(SSM_ERR_UNSUPPORTED, "width %lld not in 1..4", (long long)width);
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  int64_t n_w, entry;
  if (!mul_ok(dim, width * 4, &n_w) || !mul_ok(dim, width - 1, &entry))
    return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  if (!cache && width > 1) return fail(SSM_ERR_INVALID_ARG, "NULL cache");
  ssm::ConvStepArgs a{};
  Range rc{nullptr, 0};
  if (cache) {
    if (cache->dtype != dtype) return fail(SSM_ERR_INVALID_ARG, "the cache's dtype differs from x's");
    SSM_TRY(check_cache(cache, entry, &a.cache, &rc));
  } else {
    a.cache.slots = kMaxIndex + 1;  // any slot that is not negative
  }
  if (width == 1) a.cache.stride = 0;  // no windows: only which slots there are counts
  ssm_row_strides_t rs = strides_or_zero(strides);
  Rows t[] = {{x, dim, &rs.x, "x", 0}, {y, dim, &rs.y, "y", 0}};
  SSM_TRY(check_rows(t, 2, batch, es));
  if (batch == 0 || dim == 0 || (cache && cache->slots == 0)) return SSM_OK;
  if (!x || !weight || !y) return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (x, weight and y)");
  if (!aligned(weight, 4) || !aligned(bias, 4) || !aligned(cache_slots, 4))
    return fail(SSM_ERR_MISALIGNED, "weight, bias or cache_slots is not 4-byte aligned");
  const Range outs[] = {{y, t[1].bytes}, rc};
  const Range ins[] = {{x, t[0].bytes}, {weight, n_w}, {bias, dim * 4}, {cache_slots, batch * 4}};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));
  a.slots = cache_slots; a.x = x; a.weight = weight; a.bias = bias; a.y = y;
  a.batch = batch; a.dim = dim; a.sx = rs.x; a.sy = rs.y; a.silu = silu ? 1 : 0;
  const int64_t per = static_cast<int64_t>(ssm::kStepThreads) * ssm::kConvStepVec;
  const int64_t blocks = (dim + per - 1) / per;
  if (blocks > kMaxBlocks) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  const int R = step_entries(blocks, batch);
  const bool bf16 = dtype == SSM_BF16;
  const ConvStepKernel k =
      R > 1 ? (bf16 ? conv_step_kernel<true, kStepEntries>(width) : conv_step_kernel<false, kStepEntries>(width))
            : (bf16 ? conv_step_kernel<true, 1>(width) : conv_step_kernel<false, 1>(width));
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(blocks), grid_y((batch + R - 1) / R)), dim3(ssm::kStepThreads), 0,
                     static_cast<hipStream_t>(stream), a);
  return check_launch("causal conv1d step (cache)");
}

ssm_status_t ssm_state_update_cache(int64_t batch, int64_t dim, int64_t dstate, ssm_dtype_t dtype,
                                    const ssm_cache_t* cache, const int32_t* cache_slots, const void* x,
                                    const void* delta, const float* A, const void* B, const void* C, const float* D,
                                    const void* z, const float* delta_bias, int delta_softplus, void* y,
                                    const ssm_row_strides_t* strides, void* stream) {
  g_err[0] = '\0';
  if (batch < 0 || dim < 0 || dstate < 0 || batch > kMaxIndex)
    return fail(SSM_ERR_INVALID_ARG, "bad size (batch=%lld dim=%lld dstate=%lld)", (long long)batch, (long long)dim,
                (long long)dstate);
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (!cache) return fail(SSM_ERR_INVALID_ARG, "NULL cache");
  const bool cb16 = cache->dtype == SSM_BF16;
  auto k = by_dstate<StateStepOf<1>::K, 1, 2, 4, 8, 16, 32, 64>(dtype == SSM_BF16, cb16, dstate);
  if (!k) return fail(SSM_ERR_UNSUPPORTED, "dstate %lld not in {1,2,4,8,16,32,64}", (long long)dstate);
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  const int64_t spt = cb16 ? (dstate < 8 ? dstate : 8) : (dstate < 4 ? dstate : 4);  // kStepStates
  int64_t entry, n_dn;
  if (!mul_ok(dim, dstate, &entry) || !mul_ok(entry, 4, &n_dn))
    return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  ssm::StepArgs a{};
  Range rc;
  SSM_TRY(check_cache(cache, entry, &a.cache, &rc));
  ssm_row_strides_t rs = strides_or_zero(strides);
  Rows t[] = {{x, dim, &rs.x, "x", 0},    {delta, dim, &rs.delta, "delta", 0}, {B, dstate, &rs.B, "B", 0},
              {C, dstate, &rs.C, "C", 0}, {z, dim, &rs.z, "z", 0},             {y, dim, &rs.y, "y", 0}};
  SSM_TRY(check_rows(t, 6, batch, es));
  if (batch == 0 || dim == 0 || cache->slots == 0) return SSM_OK;
  if (!x || !delta || !A || !B || !C || !y)
    return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (x, delta, A, B, C and y)");
  if (!aligned(A, 4) || !aligned(D, 4) || !aligned(delta_bias, 4) || !aligned(cache_slots, 4))
    return fail(SSM_ERR_MISALIGNED, "A, D, delta_bias or cache_slots is not 4-byte aligned");
  const Range outs[] = {{y, t[5].bytes}, rc};
  const Range ins[] = {{x, t[0].bytes}, {delta, t[1].bytes}, {B, t[2].bytes}, {C, t[3].bytes}, {z, t[4].bytes},
                       {A, n_dn},       {D, dim * 4},        {delta_bias, dim * 4}, {cache_slots, batch * 4}};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));
  a.slots = cache_slots; a.x = x; a.delta = delta; a.A = A; a.B = B; a.C = C; a.Dskip = D; a.z = z;
  a.delta_bias = delta_bias; a.y = y; a.batch = batch; a.dim = dim;
  a.sx = rs.x; a.sdelta = rs.delta; a.sB = rs.B; a.sC = rs.C; a.sz = rs.z; a.sy = rs.y;
  a.softplus = delta_softplus ? 1 : 0;
  const int64_t blocks = (dim * (dstate / spt) + ssm::kStepThreads - 1) / ssm::kStepThreads;
  if (blocks > kMaxBlocks) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  const int R = step_entries(blocks, batch);
  if (R > 1) k = by_dstate<StateStepOf<kStepEntries>::K, 1, 2, 4, 8, 16, 32, 64>(dtype == SSM_BF16, cb16, dstate);
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(blocks), grid_y((batch + R - 1) / R)), dim3(ssm::kStepThreads), 0,
                     static_cast<hipStream_t>(stream), a);
  return check_launch("scan step (cache)");
}

ssm_status_t ssm_ssd_state_update_cache(int64_t batch, int64_t nheads, int64_t headdim, int64_t dstate,
                                        int64_t ngroups, ssm_dtype_t dtype, const ssm_cache_t* cache,
                                        const int32_t* cache_slots, const void* x, const void* dt, const float* A,
                                        const void* B, const void* C, const float* D, const void* z,
                                        const float* dt_bias, int dt_softplus, void* y,
                                        const ssm_row_strides_t* strides, void* stream) {
  g_err[0] = '\0';
  if (batch < 0 || nheads < 1 || headdim < 1 || dstate < 1 || ngroups < 1 || batch > kMaxIndex)
    return fail(SSM_ERR_INVALID_ARG, "bad size (batch=%lld nheads=%lld headdim=%lld dstate=%lld ngroups=%lld)",
                (long long)batch, (long long)nheads, (long long)headdim, (long long)dstate, (long long)ngroups);
  if (nheads % ngroups != 0)
    return fail(SSM_ERR_INVALID_ARG, "ngroups %lld does not divide nheads %lld", (long long)ngroups,
                (long long)nheads);
  if (nheads > kMaxIndex || headdim > kMaxIndex)
    return fail(SSM_ERR_INVALID_ARG, "nheads or headdim exceeds int32");
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (!cache) return fail(SSM_ERR_INVALID_ARG, "NULL cache");
  const bool cb16 = cache->dtype == SSM_BF16;
  const auto k = by_dstate<SsdStep, 16, 32, 64, 128, 256>(dtype == SSM_BF16, cb16, dstate);
  if (!k) return fail(SSM_ERR_UNSUPPORTED, "dstate %lld not in {16, 32, 64, 128, 256}", (long long)dstate);
  const int64_t es = dtype == SSM_BF16 ? 2 : 4;
  int64_t width, entry, bc;
  if (!mul_ok(nheads, headdim, &width) || !mul_ok(width, dstate, &entry) || !mul_ok(ngroups, dstate, &bc))
    return fail(SSM_ERR_INVALID_ARG, "tensor size overflows int64");
  ssm::SsdStepArgs a{};
  Range rc;
  SSM_TRY(check_cache(cache, entry, &a.cache, &rc));
  ssm_row_strides_t rs = strides_or_zero(strides);
  Rows t[] = {{x, width, &rs.x, "x", 0}, {dt, nheads, &rs.delta, "dt", 0}, {B, bc, &rs.B, "B", 0},
              {C, bc, &rs.C, "C", 0},    {z, width, &rs.z, "z", 0},        {y, width, &rs.y, "y", 0}};
  SSM_TRY(check_rows(t, 6, batch, es));
  if (batch == 0 || cache->slots == 0) return SSM_OK;
  if (!x || !dt || !A || !B || !C || !y)
    return fail(SSM_ERR_INVALID_ARG, "NULL required pointer (x, dt, A, B, C and y)");
  if (!aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(cache_slots, 4))
    return fail(SSM_ERR_MISALIGNED, "A, D, dt_bias or cache_slots is not 4-byte aligned");
  const Range outs[] = {{y, t[5].bytes}, rc};
  const Range ins[] = {{x, t[0].bytes}, {dt, t[1].bytes}, {B, t[2].bytes}, {C, t[3].bytes}, {z, t[4].bytes},
                       {A, nheads * 4}, {D, nheads * 4},  {dt_bias, nheads * 4}, {cache_slots, batch * 4}};
  SSM_TRY(check_overlap(outs, count_of(outs), ins, count_of(ins)));
  a.slots = cache_slots; a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.D = D; a.z = z; a.dt_bias = dt_bias;
  a.y = y; a.batch = batch; a.sx = rs.x; a.sdt = rs.delta; a.sB = rs.B; a.sC = rs.C; a.sz = rs.z; a.sy = rs.y;
  a.nheads = static_cast<int32_t>(nheads); a.headdim = static_cast<int32_t>(headdim);
  a.ngroups = static_cast<int32_t>(ngroups); a.softplus = dt_softplus ? 1 : 0;
  const int64_t spt = cb16 ? 8 : 4;
  const int64_t per = ssm::kSsdStepUnroll * ssm::kStepThreads * spt / dstate;
  const int64_t chunks = (headdim + per - 1) / per;
  int64_t blocks;
  if (!mul_ok(chunks, nheads, &blocks) || blocks > kMaxBlocks) return fail(SSM_ERR_UNSUPPORTED, "grid too large");
  a.chunks = static_cast<int32_t>(chunks);
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(blocks), grid_y(batch)), dim3(ssm::kStepThreads), 0,
                     static_cast<hipStream_t>(stream), a);
  return check_launch("SSD step (cache)");
}

ssm_status_t ssm_cache_store_q8(int64_t count, int64_t rows, int64_t dstate, const ssm_cache_t* cache,
                                const int32_t* cache_slots, int64_t stored, int8_t* codes, float* scales,
                                const int32_t* store_slots, void* stream) {
  g_err[0] = '\0';
  return q8_call(true, count, rows, dstate, cache, cache_slots, stored, codes, scales, store_slots, stream);
}

ssm_status_t ssm_cache_load_q8(int64_t count, int64_t rows, int64_t dstate, int64_t stored, const int8_t* codes,
                               const float* scales, const int32_t* store_slots, const ssm_cache_t* cache,
                               const int32_t* cache_slots, void* stream) {
  g_err[0] = '\0';
  return q8_call(false, count, rows, dstate, cache, cache_slots, stored, const_cast<int8_t*>(codes),
                 const_cast<float*>(scales), store_slots, stream);
}

}  // extern "C"
