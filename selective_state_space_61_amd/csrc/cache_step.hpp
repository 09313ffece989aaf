// cache_step.hpp -- single-token steps on a cache of slots, for gfx950: the convolution's, the
// selective scan's and the Mamba-2 layer's.
//
// The formulas are those of conv1d.hpp, state_update.hpp and ssd_fwd.hpp ("Mamba 论文精读" sec. 3.4,
// sec. 2.2 and sec. 4.1; sec. 6: O(1) work per token).  What differs: entry i of the batch works
// on the slot that the device array names, entries without one (the padding of a batch that a
// graph was captured with) are skipped, rows of the inputs are strided, and the states are fp32
// or bf16.
#pragma once

#include "cache.hpp"

namespace ssm {

constexpr int kStepThreads = 256;

struct StepArgs {
  CacheRef cache;
  const int32_t* slots;
  const void* x;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* Dskip;
  const void* z;
  const float* delta_bias;
  void* y;
  int64_t batch;
  int64_t dim;
  int64_t sx, sdelta, sB, sC, sz, sy;  // elements between rows
  int32_t softplus;
};

// A thread owns SPT consecutive states of a channel (16 bytes), N / SPT lanes a channel.
template <bool BF16, bool CB16, int N>
__global__ __launch_bounds__(kStepThreads) void state_update_cache_kernel(const StepArgs p) {
  constexpr int SPT = CB16 ? (N < 8 ? N : 8) : (N < 4 ? N : 4);
  constexpr int TPC = N / SPT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kStepThreads + threadIdx.x;
  const bool ok = t / TPC < p.dim;
  const int64_t d = ok ? t / TPC : p.dim - 1;
  const int n0 = static_cast<int>(t % TPC) * SPT;
  Run<false, SPT> a;
  a.load(p.A, d * N + n0);
  const float bias = p.delta_bias ? p.delta_bias[d] : 0.0f;
  const float dsk = p.Dskip ? p.Dskip[d] : 0.0f;
  for (int64_t b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const int64_t at = cache_offset(p.cache, p.slots, b);
    if (at < 0) continue;
    Run<CB16, SPT, true> st;
    Run<BF16, SPT> bv, cv;
    st.load(p.cache.data, at + d * N + n0);
    bv.load(p.B, b * p.sB + n0);
    cv.load(p.C, b * p.sC + n0);
    const float xv = load_one<BF16>(p.x, b * p.sx + d);
    const float vb = load_one<BF16>(p.delta, b * p.sdelta + d) + bias;
    const float zv = p.z ? load_one<BF16>(p.z, b * p.sz + d) : 0.0f;
    const float dt = p.softplus ? softplus_f32(vb) : vb;
    const float w = dt * xv;
    float h[SPT], yp = 0.0f;
#pragma unroll
    for (int j = 0; j < SPT; ++j) {
      h[j] = fmaf(hw_exp2(dt * (a.get(j) * kLog2e)), st.get(j), w * bv.get(j));
      yp = fmaf(cv.get(j), h[j], yp);
    }
    st.set(h);
    if (ok) st.store(p.cache.data, at + d * N + n0);
#pragma unroll
    for (int off = 1; off < TPC; off <<= 1) yp += __shfl_xor(yp, off, 64);
    if (ok && n0 == 0) {
      float yv = fmaf(dsk, xv, yp);
      if (p.z) yv *= silu_f32(zv);
      store_one<BF16>(p.y, b * p.sy + d, yv);
    }
  }
}

struct ConvStepArgs {
  CacheRef cache;
  const int32_t* slots;
  const void* x;
  const float* weight;
  const float* bias;
  void* y;
  int64_t batch;
  int64_t dim;
  int64_t sx, sy;
  int32_t silu;
};

constexpr int kConvStepVec = 4;  // channels per thread

// A thread owns 4 channels of an entry: its windows are 4 (K - 1) consecutive elements.
template <bool BF16, int K>
__global__ __launch_bounds__(kStepThreads) void conv1d_update_cache_kernel(const ConvStepArgs p) {
  constexpr int V = kConvStepVec, W = K - 1;
  const int64_t d0 = (static_cast<int64_t>(blockIdx.x) * kStepThreads + threadIdx.x) * V;
  if (d0 >= p.dim) return;
  const int nv = static_cast<int>(p.dim - d0 < V ? p.dim - d0 : V);
  for (int64_t b = blockIdx.y; b < p.batch; b += gridDim.y) {
    // without windows (K 1) there is no slot to look up: only padding is skipped
    const int64_t at = W > 0 ? cache_offset(p.cache, p.slots, b) : (p.slots && p.slots[b] < 0 ? -1 : 0);
    if (at < 0) continue;
    if (nv == V) {
      Run<BF16, V> xr;
      Run<BF16, V * W + (W == 0)> win;
      xr.load(p.x, b * p.sx + d0);
      if constexpr (W > 0) win.load(p.cache.data, at + d0 * W);
      float out[V], keep[V * W + (W == 0)];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float* wt = p.weight + (d0 + v) * K;
        float acc = p.bias ? p.bias[d0 + v] : 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) acc = fmaf(wt[j], win.get(v * W + j), acc);
        acc = fmaf(wt[W], xr.get(v), acc);
        out[v] = p.silu ? silu_f32(acc) : acc;
#pragma unroll
        for (int j = 0; j < W; ++j) keep[v * W + j] = j + 1 < W ? win.get(v * W + j + 1) : xr.get(v);
      }
      Run<BF16, V> yr;
      yr.set(out);
      yr.store(p.y, b * p.sy + d0);
      if constexpr (W > 0) {
        win.set(keep);
        win.store(p.cache.data, at + d0 * W);
      }
      continue;
    }
    for (int v = 0; v < nv; ++v) {
      const int64_t d = d0 + v;
      const float xv = load_one<BF16>(p.x, b * p.sx + d);
      float acc = p.bias ? p.bias[d] : 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) acc = fmaf(p.weight[d * K + j], load_one<BF16>(p.cache.data, at + d * W + j), acc);
      acc = fmaf(p.weight[d * K + W], xv, acc);
      store_one<BF16>(p.y, b * p.sy + d, p.silu ? silu_f32(acc) : acc);
#pragma unroll
      for (int j = 0; j < W; ++j)
        store_one<BF16>(p.cache.data, at + d * W + j,
                        j + 1 < W ? load_one<BF16>(p.cache.data, at + d * W + j + 1) : xv);
    }
  }
}

struct SsdStepArgs {
  CacheRef cache;
  const int32_t* slots;
  const void* x;
  const void* dt;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* dt_bias;
  void* y;
  int64_t batch;
  int64_t sx, sdt, sB, sC, sz, sy;
  int32_t nheads, headdim, ngroups;
  int32_t chunks;  // workgroups per head
  int32_t softplus;
};

// channels of a head that one workgroup takes: U per 16-byte state access of its four waves
constexpr int kSsdStepUnroll = 4;
template <bool CB16, int N>
constexpr int kSsdStepChannels = kSsdStepUnroll * kStepThreads * (CB16 ? 8 : 4) / N;

// One workgroup: a stretch of the channels of one head of one entry.  N / SPT lanes share a
// channel; each lane's B and C values serve all of the channels that it takes.
template <bool BF16, bool CB16, int N>
__global__ __launch_bounds__(kStepThreads) void ssd_state_update_cache_kernel(const SsdStepArgs p) {
  constexpr int SPT = CB16 ? 8 : 4;
  constexpr int TPC = N / SPT;
  constexpr int CPB = kStepThreads / TPC;  // channels per access of the workgroup
  static_assert(TPC >= 1 && TPC <= 64, "a channel's lanes share one wave");
  const int64_t P = p.headdim;
  const int h = static_cast<int>(blockIdx.x / p.chunks);
  const int64_t p0 = static_cast<int64_t>(blockIdx.x % p.chunks) * kSsdStepChannels<CB16, N> + threadIdx.x / TPC;
  const int n0 = static_cast<int>(threadIdx.x % TPC) * SPT;
  const int g = h / (p.nheads / p.ngroups);
  const float al = p.A[h] * kLog2e;
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
  const float dsk = p.D ? p.D[h] : 0.0f;
  for (int64_t b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const int64_t at = cache_offset(p.cache, p.slots, b);
    if (at < 0) continue;
    Run<CB16, SPT, true> st[kSsdStepUnroll];
    float xv[kSsdStepUnroll], zv[kSsdStepUnroll];
    bool ok[kSsdStepUnroll];
    int64_t off[kSsdStepUnroll];
#pragma unroll
    for (int u = 0; u < kSsdStepUnroll; ++u) {
      const int64_t pc = p0 + u * CPB;
      ok[u] = pc < P;
      const int64_t c = static_cast<int64_t>(h) * P + (ok[u] ? pc : 0);
      off[u] = at + c * N + n0;
      st[u].load(p.cache.data, off[u]);
      xv[u] = load_one<BF16>(p.x, b * p.sx + c);
      zv[u] = p.z ? load_one<BF16>(p.z, b * p.sz + c) : 0.0f;
    }
    Run<BF16, SPT> bv, cv;
    bv.load(p.B, b * p.sB + static_cast<int64_t>(g) * N + n0);
    cv.load(p.C, b * p.sC + static_cast<int64_t>(g) * N + n0);
    const float v = load_one<BF16>(p.dt, b * p.sdt + h) + bias;
    const float dtv = p.softplus ? softplus_f32(v) : v;
    const float a = hw_exp2(dtv * al);
#pragma unroll
    for (int u = 0; u < kSsdStepUnroll; ++u) {
      const float w = dtv * xv[u];
      float s[SPT], yp = 0.0f;
#pragma unroll
      for (int j = 0; j < SPT; ++j) {
        s[j] = fmaf(a, st[u].get(j), w * bv.get(j));
        yp = fmaf(cv.get(j), s[j], yp);
      }
      st[u].set(s);
      if (ok[u]) st[u].store(p.cache.data, off[u]);
#pragma unroll
      for (int o = 1; o < TPC; o <<= 1) yp += __shfl_xor(yp, o, 64);
      if (ok[u] && n0 == 0) {
        float yv = fmaf(dsk, xv[u], yp);
        if (p.z) yv *= silu_f32(zv[u]);
        store_one<BF16>(p.y, b * p.sy + static_cast<int64_t>(h) * P + p0 + u * CPB, yv);
      }
    }
  }
}

}  // namespace ssm
