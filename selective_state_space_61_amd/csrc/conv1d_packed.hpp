// conv1d_packed.hpp -- the depthwise causal convolution over packed prompts, for gfx950.
//
// The formula is conv1d.hpp's ("Mamba 论文精读" sec. 3.4) for every sequence by itself: the inputs
// before a sequence's first row are its slot's window, or zeros.
//
// The packed axis is cut into tiles of kPackTile rows, whatever sequences they belong to, so that a
// batch of many short prompts fills the card as well as one long one.  A thread owns the channels
// of one 4-byte access and one tile; it goes through the tile sequence by sequence, with the K-1
// previous inputs in registers and kConvUnroll row loads in flight.
//
// The thread that meets a sequence's first row takes up the slot's window and, with the window in
// registers, stores the sequence's last K-1 inputs to the slot; it also computes the sequence's
// first K-1 rows where those reach into the next tile, which begins behind them.  So no other
// thread reads that window, and nothing has to order the read and the write.
#pragma once

#include "cache.hpp"

namespace ssm {

struct ConvPackedArgs {
  const void* x;
  const float* weight;
  const float* bias;
  void* y;
  CacheRef cache;  // data NULL: none
  const int32_t* cu;
  const int32_t* slots;
  const uint8_t* has_initial;
  int64_t total;
  int64_t nseq;
  int64_t dim;
  int64_t sx, sy;
  int32_t ncb;  // workgroups per tile
  int32_t silu;
};

constexpr int kPackTile = 32;

template <bool BF16, int K>
__global__ __launch_bounds__(kConvThreads) void conv1d_packed_kernel(const ConvPackedArgs p) {
  constexpr int V = kConvVec<BF16>, W = K - 1, T = kPackTile;
  const int64_t tile = blockIdx.x / p.ncb;
  const int64_t d0 = (static_cast<int64_t>(blockIdx.x % p.ncb) * kConvThreads + threadIdx.x) * V;
  const int64_t t0 = tile * T;
  const int64_t t1 = t0 + T < p.total ? t0 + T : p.total;
  // lanes without channels (nv 0) take part in the search for sequences
  const int nv = d0 >= p.dim ? 0 : static_cast<int>(p.dim - d0 < V ? p.dim - d0 : V);
  float w[K][V], bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][v] = v < nv ? p.weight[(d0 + v) * K + k] : 0.0f;
    bias[v] = v < nv && p.bias ? p.bias[d0 + v] : 0.0f;
  }
  // win[j]: the input K-1-j rows before the row at hand
  float win[W > 0 ? W : 1][V];
  // the inputs before the sequence's row `row`: at row 0 the slot's window, else rows (row >= W)
  auto take_window = [&](const RowOwner& o, int64_t row) {
    if constexpr (W > 0) {
      const int64_t at = p.cache.data ? cache_offset(p.cache, p.slots, o.s) : -1;
      const bool init = at >= 0 && p.has_initial && p.has_initial[o.s];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int64_t s = row - W + j;  // row of the sequence; negative: of the slot's window
        Run<BF16, V> q;
        q.load_some(p.x, (o.start + (s >= 0 ? s : 0)) * p.sx + d0, s >= 0 ? nv : 0);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          win[j][v] = q.get(v);
          if (s < 0 && init && v < nv) win[j][v] = load_one<BF16>(p.cache.data, at + (d0 + v) * W + W + s);
        }
      }
    }
  };
  // the sequence's last W inputs to its slot; `win` holds the window before its first row
  auto leave_window = [&](const RowOwner& o) {
    if constexpr (W > 0) {
      const int64_t at = p.cache.data ? cache_offset(p.cache, p.slots, o.s) : -1;
      if (at < 0) return;
      const int64_t len = o.end - o.start;
      float fin[W][V];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int64_t s = len - W + j;
        Run<BF16, V> q;
        q.load_some(p.x, (o.start + (s >= 0 ? s : 0)) * p.sx + d0, s >= 0 ? nv : 0);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          fin[j][v] = q.get(v);
#pragma unroll
          for (int i = 0; i < W; ++i)
            if (s == i - W) fin[j][v] = win[i][v];
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (v < nv) store_one<BF16>(p.cache.data, at + (d0 + v) * W + j, fin[j][v]);
    }
  };
  for (int64_t t = t0; t < t1;) {
    const RowOwner own = row_owner(p.cu, p.nseq, p.total, t);
    int64_t end = own.end < t1 ? own.end : t1;
    if (own.s < 0) {
      t = end;
      continue;
    }
    if (own.start < t0 && t < own.start + W) {  // the tile before computed these rows
      t = own.start + W < own.end ? own.start + W : own.end;
      if (t == own.end) continue;
    }
    if (own.end > t1 && own.start + W > t1) end = own.start + W < own.end ? own.start + W : own.end;
    take_window(own, t - own.start);
    if (t == own.start) leave_window(own);
    for (; t < end; t += kConvUnroll) {
      Run<BF16, V> r[kConvUnroll];
#pragma unroll
      for (int u = 0; u < kConvUnroll; ++u) {
        const int64_t at = (t + u < end ? t + u : end - 1) * p.sx + d0;
        if (nv == V) r[u].load(p.x, at);
        else r[u].load_some(p.x, at, nv);
      }
#pragma unroll
      for (int u = 0; u < kConvUnroll; ++u) {
        if (t + u >= end) break;
        float out[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float xv = r[u].get(v);
          float acc = bias[v];
#pragma unroll
          for (int j = 0; j < W; ++j) acc = fmaf(w[j][v], win[j][v], acc);
          acc = fmaf(w[W][v], xv, acc);
          out[v] = p.silu ? silu_f32(acc) : acc;
#pragma unroll
          for (int j = 0; j + 1 < W; ++j) win[j][v] = win[j + 1][v];
          if constexpr (W > 0) win[W - 1][v] = xv;
        }
        Run<BF16, V, true> o;  // written once and read by the next kernel
        o.set(out);
        if (nv == V) o.store(p.y, (t + u) * p.sy + d0);
        else o.store_some(p.y, (t + u) * p.sy + d0, nv);
      }
    }
    t = end;
  }
}

}  // namespace ssm
