// scan_packed.hpp -- the selective scan over packed prompts, for gfx950.
//
// The recurrence is scan_fwd.hpp's ("Mamba 论文精读" sec. 2.2 and sec. 3.3) for every sequence by
// itself, from its slot's state or from zeros.
#pragma once

#include "cache.hpp"

namespace ssm {

struct ScanPackedArgs {
  const void* x;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* Dskip;
  const void* z;
  const float* delta_bias;
  void* y;
  CacheRef cache;  // data NULL: none
  const int32_t* cu;
  const int32_t* slots;
  const uint8_t* has_initial;
  int64_t total;
  int64_t nseq;
  int64_t dim;
  int64_t sx, sdelta, sB, sC, sz, sy;
  int32_t softplus;
};

constexpr int kScanSimpleThreads = 256;
constexpr int kScanSimpleUnroll = 8;

// One workgroup: a block of channels of one sequence, SPT states of a channel per thread, the rows
// one after another with kScanSimpleUnroll rows' loads in flight.
template <bool BF16, bool CB16, int N>
__global__ __launch_bounds__(kScanSimpleThreads) void scan_packed_kernel(const ScanPackedArgs p) {
  constexpr int SPT = N < 4 ? N : 4, TPC = N / SPT, U = kScanSimpleUnroll;
  const int64_t s = blockIdx.y;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kScanSimpleThreads + threadIdx.x;
  const bool ok = t / TPC < p.dim;
  const int64_t d = ok ? t / TPC : p.dim - 1;
  const int n0 = static_cast<int>(t % TPC) * SPT;
  int64_t r0 = p.cu[s], r1 = p.cu[s + 1];
  r0 = r0 < 0 ? 0 : r0;
  r1 = r1 > p.total ? p.total : r1;
  if (r0 >= r1) return;
  const int64_t at = p.cache.data ? cache_offset(p.cache, p.slots, s) : -1;
  float a2[SPT], h[SPT];
  Run<CB16, SPT> st;
  if (at >= 0 && p.has_initial && p.has_initial[s]) {
    st.load(p.cache.data, at + d * N + n0, p.cache.vec_ok);
#pragma unroll
    for (int j = 0; j < SPT; ++j) h[j] = st.get(j);
  } else {
#pragma unroll
    for (int j = 0; j < SPT; ++j) h[j] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < SPT; ++j) a2[j] = p.A[d * N + n0 + j] * kLog2e;
  const float bias = p.delta_bias ? p.delta_bias[d] : 0.0f;
  const float dsk = p.Dskip ? p.Dskip[d] : 0.0f;
  for (int64_t r = r0; r < r1; r += U) {
    float xv[U], dv[U], zv[U];
    Run<BF16, SPT> bv[U], cv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t q = r + u < r1 ? r + u : r1 - 1;
      xv[u] = load_one<BF16>(p.x, q * p.sx + d);
      dv[u] = load_one<BF16>(p.delta, q * p.sdelta + d);
      zv[u] = p.z ? load_one<BF16>(p.z, q * p.sz + d) : 0.0f;
      bv[u].load(p.B, q * p.sB + n0, false);
      cv[u].load(p.C, q * p.sC + n0, false);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r + u >= r1) break;
      const float vb = dv[u] + bias;
      const float dt = p.softplus ? softplus_f32(vb) : vb;
      const float w = dt * xv[u];
      float yp = 0.0f;
#pragma unroll
      for (int j = 0; j < SPT; ++j) {
        h[j] = fmaf(hw_exp2(dt * a2[j]), h[j], w * bv[u].get(j));
        yp = fmaf(cv[u].get(j), h[j], yp);
      }
#pragma unroll
      for (int off = 1; off < TPC; off <<= 1) yp += __shfl_xor(yp, off, 64);
      if (ok && n0 == 0) {
        float yv = fmaf(dsk, xv[u], yp);
        if (p.z) yv *= silu_f32(zv[u]);
        store_one<BF16>(p.y, (r + u) * p.sy + d, yv);
      }
    }
  }
  if (at >= 0 && ok) {
    st.set(h);
    st.store(p.cache.data, at + d * N + n0, p.cache.vec_ok);
  }
}

}  // namespace ssm
