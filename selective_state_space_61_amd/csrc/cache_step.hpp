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

// The step's functions by the inputs' type.  bf16: the hardware exp2 with log2(e) in its factor and
// fused multiply-adds, as in the scan.  fp32: the library's exp and log1p and the formula's own
// roundings: exp2(dt (A log2 e)) is off by up to |dt A| 2^-24 more, which fp32 outputs would show,
// and a step is bound by its states' traffic, not by these.
template <bool BF16>
struct StepMath {
  static __device__ __forceinline__ float softplus(float v) {
    if constexpr (BF16) return softplus_f32(v);
    else return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v)));
  }
  static __device__ __forceinline__ float decay(float dt, float a) {
    if constexpr (BF16) return hw_exp2(dt * (a * kLog2e));
    else return expf(dt * a);
  }
  static __device__ __forceinline__ float state(float a, float h, float w, float b) {
    if constexpr (BF16) {
      return fmaf(a, h, w * b);
    } else {
#pragma clang fp contract(off)
      return a * h + w * b;
    }
  }
  static __device__ __forceinline__ float gate(float z) {
    if constexpr (BF16) return silu_f32(z);
    else return z / (1.0f + expf(-z));
  }
};

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

// States of a channel that a lane takes: 16 bytes
template <bool CB16, int N>
constexpr int kStepStates = CB16 ? (N < 8 ? N : 8) : (N < 4 ? N : 4);

// A thread owns SPT consecutive states of a channel, N / SPT lanes a channel, in R entries of
// the batch: A, D and the bias serve all of them, and their states' loads are in flight together.
// Bound by the states' traffic: 250 entries of 5120 x 16 take 33.3 us with fp32 states (174 MB, 5.2 TB/s,
// a copy's rate) and 21.5 us with bf16 ones (92 MB, 4.3 TB/s), with R 1 | 2 | 4 | 8 23.7 | 22.5 | 21.5 |
// 25.8 us; with 32 bytes of state a lane 24.2 us.
template <bool BF16, bool CB16, int N, int R>
__global__ __launch_bounds__(kStepThreads) void state_update_cache_kernel(const StepArgs p) {
  constexpr int SPT = kStepStates<CB16, N>, TPC = N / SPT;
  using M = StepMath<BF16>;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kStepThreads + threadIdx.x;
  const bool ok = t / TPC < p.dim;
  const int64_t d = ok ? t / TPC : p.dim - 1;
  const int n0 = static_cast<int>(t % TPC) * SPT;
  const bool has_z = p.z != nullptr;
  const void* zsrc = has_z ? p.z : p.x;
  const int64_t zstride = has_z ? p.sz : p.sx;
  for (int64_t b0 = static_cast<int64_t>(blockIdx.y) * R; b0 < p.batch; b0 += static_cast<int64_t>(gridDim.y) * R) {
    // every load on every path: an entry past the batch or without a slot reads entry b0 and slot 0
    int64_t at[R], b[R];
    Run<CB16, SPT, true> st[R];
    Run<BF16, SPT> bv[R], cv[R];
    Run<BF16, 1> xr[R], dr[R], zr[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      b[i] = b0 + i < p.batch ? b0 + i : b0;
      at[i] = b0 + i < p.batch ? cache_offset(p.cache, p.slots, b0 + i) : -1;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      st[i].load(p.cache.data, (at[i] < 0 ? 0 : at[i]) + d * N + n0);
      xr[i].load(p.x, b[i] * p.sx + d);
      dr[i].load(p.delta, b[i] * p.sdelta + d);
      zr[i].load(zsrc, b[i] * zstride + d);
      bv[i].load(p.B, b[i] * p.sB + n0);
      cv[i].load(p.C, b[i] * p.sC + n0);
    }
    Run<false, SPT> a;
    a.load(p.A, d * N + n0);
    const float bias = p.delta_bias ? p.delta_bias[d] : 0.0f;
    const float dsk = p.Dskip ? p.Dskip[d] : 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float xv = xr[i].get(0), vb = dr[i].get(0) + bias;
      const float dt = p.softplus ? M::softplus(vb) : vb;
      const float w = dt * xv;
      float h[SPT], yp = 0.0f;
#pragma unroll
      for (int j = 0; j < SPT; ++j) {
        h[j] = M::state(M::decay(dt, a.get(j)), st[i].get(j), w, bv[i].get(j));
        yp = fmaf(cv[i].get(j), h[j], yp);
      }
      st[i].set(h);
      if (ok && at[i] >= 0) st[i].store(p.cache.data, at[i] + d * N + n0);
      yp = group_sum<TPC>(yp);
      if (ok && at[i] >= 0 && n0 == 0) {
        float yv = p.Dskip ? fmaf(dsk, xv, yp) : yp;
        if (has_z) yv *= M::gate(zr[i].get(0));
        store_one<BF16>(p.y, b[i] * p.sy + d, yv);
      }
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

// A thread owns 4 channels of R entries: an entry's windows are 4 (K - 1) consecutive elements, and the
// weights serve all R.  250 entries of 5120 channels, width 4, bf16: 7.4 us (20 MB; 13 us with R 1 and the
// weights loaded one by one): the launch and one round trip to memory are half of it.
template <bool BF16, int K, int R>
__global__ __launch_bounds__(kStepThreads) void conv1d_update_cache_kernel(const ConvStepArgs p) {
  constexpr int V = kConvStepVec, W = K - 1, E = W > 0 ? V * W : 2;
  const int64_t d0 = (static_cast<int64_t>(blockIdx.x) * kStepThreads + threadIdx.x) * V;
  if (d0 >= p.dim) return;
  const int nv = static_cast<int>(p.dim - d0 < V ? p.dim - d0 : V);
  for (int64_t b0 = static_cast<int64_t>(blockIdx.y) * R; b0 < p.batch; b0 += static_cast<int64_t>(gridDim.y) * R) {
    int64_t at[R], b[R];
    Run<BF16, V> xr[R];
    Run<BF16, E> win[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      // (without windows, K 1, a slot only says whether the entry is padding)
      b[i] = b0 + i < p.batch ? b0 + i : b0;
      at[i] = b0 + i < p.batch ? cache_offset(p.cache, p.slots, b0 + i) : -1;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t from = (at[i] < 0 ? 0 : at[i]) + d0 * W;
      if (nv == V) {
        xr[i].load(p.x, b[i] * p.sx + d0);
        if constexpr (W > 0) win[i].load(p.cache.data, from);
      } else {
        xr[i].load_some(p.x, b[i] * p.sx + d0, nv);
        if constexpr (W > 0) win[i].load_some(p.cache.data, from, nv * W);
      }
    }
    Run<false, V * K> wt;
    Run<false, V> bias;
    if (nv == V) {
      wt.load(p.weight, d0 * K);
      if (p.bias) bias.load(p.bias, d0);
      else bias.load_some(p.weight, 0, 0);
    } else {
      wt.load_some(p.weight, d0 * K, nv * K);
      bias.load_some(p.bias, d0, p.bias ? nv : 0);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (at[i] < 0) continue;
      float out[V], keep[E] = {};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float acc = bias.get(v);
#pragma unroll
        for (int j = 0; j < W; ++j) acc = fmaf(wt.get(v * K + j), win[i].get(v * W + j), acc);
        acc = fmaf(wt.get(v * K + W), xr[i].get(v), acc);
        out[v] = p.silu ? silu_f32(acc) : acc;
#pragma unroll
        for (int j = 0; j < W; ++j) keep[v * W + j] = j + 1 < W ? win[i].get(v * W + j + 1) : xr[i].get(v);
      }
      Run<BF16, V> yr;
      yr.set(out);
      win[i].set(keep);
      if (nv == V) {
        yr.store(p.y, b[i] * p.sy + d0);
        if constexpr (W > 0) win[i].store(p.cache.data, at[i] + d0 * W);
      } else {
        yr.store_some(p.y, b[i] * p.sy + d0, nv);
        if constexpr (W > 0) win[i].store_some(p.cache.data, at[i] + d0 * W, nv * W);
      }
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
// channel; each lane's B and C values serve all of the channels that it takes, whose states' loads are in
// flight together.  Bound by the states' traffic: 96 entries of 64 heads x 64 x 128 in fp32 take 75.5 us
// (406 MB, 5.4 TB/s, a copy's rate).
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
  using M = StepMath<BF16>;
  const float ah = p.A[h];
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
    const float dtv = p.softplus ? M::softplus(v) : v;
    const float a = M::decay(dtv, ah);
#pragma unroll
    for (int u = 0; u < kSsdStepUnroll; ++u) {
      const float w = dtv * xv[u];
      float s[SPT], yp = 0.0f;
#pragma unroll
      for (int j = 0; j < SPT; ++j) {
        s[j] = M::state(a, st[u].get(j), w, bv.get(j));
        yp = fmaf(cv.get(j), s[j], yp);
      }
      st[u].set(s);
      if (ok[u]) st[u].store(p.cache.data, off[u]);
      yp = group_sum<TPC>(yp);
      if (ok[u] && n0 == 0) {
        float yv = p.D ? fmaf(dsk, xv[u], yp) : yp;
        if (p.z) yv *= M::gate(zv[u]);
        store_one<BF16>(p.y, b * p.sy + static_cast<int64_t>(h) * P + p0 + u * CPB, yv);
      }
    }
  }
}

}  // namespace ssm
