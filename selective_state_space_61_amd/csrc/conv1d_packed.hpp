// conv1d_packed.hpp -- the depthwise causal convolution over packed prompts, for gfx950.
//
// The formula is conv1d.hpp's ("Mamba 论文精读" sec. 3.4) for every sequence by itself: the inputs
// before a sequence's first row are its slot's window, or zeros.
//
// The packed axis is cut into tiles of rows, whatever sequences they belong to, so that a batch of
// many short prompts fills the card as well as one long one.  A thread owns the channels of one
// 4-byte access and one tile, whose rows it loads before anything else; the K-1 inputs before a row
// run along in registers.
//
// The thread that meets a sequence's first row takes up the slot's window and, with the window in
// registers, stores the sequence's last K-1 inputs to the slot; it also computes the sequence's
// first K-1 rows where those reach into the next tile.  So no other thread reads that window, and
// nothing has to order the read and the write.
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

// Rows per tile: 32 (a sequence's 3 rows before a tile are a tenth of its reads), or 8 where that leaves
// fewer than two workgroups a CU, or where sequences are shorter than a tile on average (a tile takes
// its sequences one after another, about 2.5 us each).  bf16, us with 8 | 32: 171 rows of 1536 channels
// 8.0 | 15.5, 1000 of 1536 9.0 | 14.6, 4288 of 1536 13.2 | 16.0, 16384 of 1536 31 | 22.6 (4.4 TB/s; 25.8
// with the tiles dealt round robin to the XCDs), 12288 of 5120 78 | 55 (4.6 TB/s).
constexpr int kPackTile = 32, kPackTileSmall = 8;

template <bool BF16, int K, int T>
__global__ __launch_bounds__(kConvThreads) void conv1d_packed_kernel(const ConvPackedArgs p) {
  constexpr int V = kConvVec<BF16>, W = K - 1, WN = W > 0 ? W : 1;
  const int64_t blk = xcd_local(blockIdx.x, gridDim.x);  // a tile's last rows are the next one's first reads: one L2
  const int64_t tile = blk / p.ncb;
  const int64_t d0 = (blk % p.ncb * kConvThreads + threadIdx.x) * V;
  const int64_t t0 = tile * T;
  const int64_t t1 = t0 + T < p.total ? t0 + T : p.total;
  // lanes without channels (nv 0) take part in the search for sequences
  const int nv = d0 >= p.dim ? 0 : static_cast<int>(p.dim - d0 < V ? p.dim - d0 : V);
  auto load_row = [&](Run<BF16, V>& r, int64_t t) {
    if (nv == V) r.load(p.x, t * p.sx + d0);
    else r.load_some(p.x, t * p.sx + d0, nv);
  };
  // the tile's rows and the ones before it, whatever sequences they belong to: in flight while the
  // sequences are looked up
  Run<BF16, V> r[T], before[WN];
#pragma unroll
  for (int j = 0; j < W; ++j) load_row(before[j], t0 - W + j > 0 ? t0 - W + j : 0);
#pragma unroll
  for (int u = 0; u < T; ++u) load_row(r[u], t0 + u < t1 ? t0 + u : t1 - 1);
  float w[K][V], bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][v] = v < nv ? p.weight[(d0 + v) * K + k] : 0.0f;
    bias[v] = v < nv && p.bias ? p.bias[d0 + v] : 0.0f;
  }
  Sequences seqs(p.cu, p.slots, p.has_initial, p.nseq, p.total, t0);
  RowOwner own = seqs.owner(t0);
  // win[j]: the input W - j rows before the row at hand
  float win[WN][V];
  auto shift = [&](const Run<BF16, V>& x) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) win[j][v] = win[j + 1][v];
      if constexpr (W > 0) win[W - 1][v] = x.get(v);
    }
  };
  auto step = [&](const Run<BF16, V>& x, int64_t t) {
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float acc = bias[v];
#pragma unroll
      for (int j = 0; j < W; ++j) acc = fmaf(w[j][v], win[j][v], acc);
      acc = fmaf(w[W][v], x.get(v), acc);
      out[v] = p.silu ? silu_f32(acc) : acc;
    }
    shift(x);
    Run<BF16, V, true> o;  // written once and read by the next kernel
    o.set(out);
    if (nv == V) o.store(p.y, t * p.sy + d0);
    else o.store_some(p.y, t * p.sy + d0, nv);
  };
  if (own.s >= 0 && own.end >= t1 && t0 - own.start >= W) {  // one sequence, begun before the tile
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) win[j][v] = before[j].get(v);
#pragma unroll
    for (int u = 0; u < T; ++u)
      if (t0 + u < t1) step(r[u], t0 + u);
    return;
  }
  // Otherwise sequence by sequence.  What the next sequence needs (its slot's window, its last W inputs,
  // its first rows) is loaded before the rows of the one at hand are computed; its place, slot and flag
  // come from registers.  (Looked up in memory one after another, a sequence took 3.5 us, now 2.5.)
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) win[j][v] = before[j].get(v);
  constexpr int G = 8, E = W > 0 ? V * W : 2;
  struct Ahead {
    RowOwner o;
    int64_t at;  // its slot, -1: none, or not begun here
    bool init;   // it starts from the slot's window
    Run<BF16, E> window;
    Run<BF16, V> last[WN], q[G];
  };
  auto load_rows = [&](Run<BF16, V> (&q)[G], int64_t t, int64_t end) {
#pragma unroll
    for (int u = 0; u < G; ++u) load_row(q[u], t + u < end ? t + u : end - 1);
  };
  const bool cached = W > 0 && p.cache.data != nullptr;
  // Without branches around its loads, whose registers would have to meet again and wait: rows and slots
  // that are not needed are read from places that exist.
  auto look_up = [&](Ahead& f, const RowOwner& o, int64_t t) {
    f.o = o;
    load_rows(f.q, t, o.end < t1 ? o.end : t1);
    const bool first = o.s >= 0 && t == o.start;
    f.at = cached && first ? seqs.slot_offset(p.cache, o.s) : -1;
    f.init = f.at >= 0 && seqs.initial(o.s);
    if (!cached) return;
#pragma unroll
    for (int j = 0; j < W; ++j) load_row(f.last[j], o.end - W + j > o.start ? o.end - W + j : o.start);
    const int64_t from = (f.at < 0 ? 0 : f.at) + d0 * W;
    if (nv == V) f.window.load(p.cache.data, from);
    else f.window.load_some(p.cache.data, from, nv * W);
  };
  auto begin = [&](const Ahead& f) {
    if constexpr (W > 0) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) win[j][v] = f.init ? f.window.get(v * W + j) : 0.0f;
      if (f.at < 0) return;
      const int64_t len = f.o.end - f.o.start;
      float left[E];
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          left[v * W + j] = f.last[j].get(v);
#pragma unroll
          for (int i = 0; i < W; ++i)  // of a sequence shorter than W the window's later part stays
            if (len - W + j == i - W) left[v * W + j] = win[i][v];
        }
      Run<BF16, E> out;
      out.set(left);
      if (nv == V) out.store(p.cache.data, f.at + d0 * W);
      else out.store_some(p.cache.data, f.at + d0 * W, nv * W);
    }
  };
  Ahead cur;
  look_up(cur, own, t0);
  for (int64_t t = t0; t < t1;) {
    own = cur.o;
    const int64_t end = own.end < t1 ? own.end : t1;
    Ahead next;
    next.o = own;
    if (end < t1) look_up(next, seqs.owner(end), end);
    if (own.s >= 0) {
      if (t == own.start) begin(cur);
      while (true) {
#pragma unroll
        for (int u = 0; u < G; ++u) {
          if (t + u >= end) continue;
          // (the tile before computed the first W rows of a sequence that began in it)
          if (own.start >= t0 || t + u >= own.start + W) step(cur.q[u], t + u);
          else shift(cur.q[u]);
        }
        t += G;
        if (t >= end) break;
        load_rows(cur.q, t, end);
      }
    }
    t = end;
    cur = next;
  }
  // the first W rows of a sequence that began in this tile, where they reach into the next one
  for (int64_t t = t1; own.s >= 0 && own.start >= t0 && t < own.end && t < own.start + W; ++t) {
    Run<BF16, V> q;
    load_row(q, t);
    step(q, t);
  }
}

}  // namespace ssm
