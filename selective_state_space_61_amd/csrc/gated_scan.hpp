// gated_scan.hpp -- the gated linear recurrence for gfx950: forward over whole batches and packed
// prompts, and backward.
//
// Per channel d and row t (include/ssm.h, "Gated recurrence"):
//   r = sigmoid(a_gate + a_bias), i = sigmoid(x_gate + x_bias), l = -a_scale softplus(a_param) r
//   a = e^l, w = sqrt(1 - a^2), u = i x,  h_t = a h_{t-1} + w u,  y_t = h_t silu(z_t)
//
// One pass.  Rows of all sequences form one axis, cut into tiles; a workgroup takes one tile of 64
// channels, keeps it in registers, and composes its rows in three levels: a lane's rows one after
// another, the lanes of a channel through the LDS, tiles through memory.  A map h -> A h + B stands
// for a stretch of rows; a stretch that holds a sequence's first row has a state of its own whatever
// entered.  Each tile publishes its map as soon as it has it and its end state once it knows the
// entering one, and looks back over the maps of the tiles before it to the nearest end state
// (the look-back of Merrill and Garland, "Single-pass parallel prefix scan with decoupled look-back").
//  - Every wait ends: tiles are taken by tickets in the order of the axis, so that a tile waits only for
//    tiles that running workgroups have taken before it, the first tile waits for none, and a waiting
//    wave leaves its SIMD to others.
//  - Results do not depend on timing: whoever computes the end state of a tile does it by the same
//    operation, fma(A, entering state, B), from the same two words.
//  - No fences: a published word is written once, by a relaxed atomic store at agent scope (a state is 32
//    bits, a map 64), over a pattern that no published word has, and is itself the sign of its arrival.
#pragma once

#include "cache.hpp"

namespace ssm {

constexpr int kGatedThreads = 256;
constexpr int kGatedChannels = 64;   // channels of a workgroup: one 128-byte line of a bf16 row
constexpr uint32_t kEmpty = 0xffffffffu;
constexpr int kGatedWindow = 8;      // tiles that one look back covers
constexpr int kGatedSave = 64;       // rows between checkpoints

struct GatedArgs {
  const void *x, *ag, *xg, *z;
  void* y;
  const float *param, *ab, *xb;
  float scale;
  int64_t sx, sag, sxg, sz, sy;  // elements between rows
  int64_t total, dim;
  int64_t seqlen;                // rows of each sequence where cu is NULL
  const int32_t *cu, *slots;
  const uint8_t* has_initial;
  int64_t nseq;
  CacheRef in, out;              // initial and final states by slot
  int32_t cb16;                  // they are bf16
  float* ckpt;                   // state after every kGatedSave-th row
  uint32_t* ticket;              // NULL: one tile, nothing is published
  uint64_t* maps;
  uint32_t* ends;
  int64_t tiles;
  int32_t chains;                // blocks of kGatedChannels channels
  // backward
  const void* dy;
  const float* dlast;
  void *dx, *dag, *dxg, *dz;
  float* dh0;
  float* partial;                // (tiles, 3, dim): sums of E, da_gate, dx_gate
};

// Lanes of a workgroup: kLanes lanes of V channels, the others its rows, R each.
template <int V, int R>
struct GatedShape {
  static constexpr int kLanes = kGatedChannels / V;
  static constexpr int kParts = kGatedThreads / kLanes;  // row groups
  static constexpr int kRows = kParts * R;               // rows of a tile
};

__device__ __forceinline__ void publish(uint32_t* p, float v) {
  uint32_t b = __builtin_bit_cast(uint32_t, v);
  b = b == kEmpty ? 0x7fc00000u : b;
  __hip_atomic_store(p, b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint64_t* p, float a, float b) {
  uint32_t lo = __builtin_bit_cast(uint32_t, a);
  const uint32_t hi = __builtin_bit_cast(uint32_t, b);
  lo = lo == kEmpty && hi == kEmpty ? 0x7fc00000u : lo;
  __hip_atomic_store(p, (static_cast<uint64_t>(hi) << 32) | lo, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that leaves the k-th tile before this one (k = 0: the one just before), in the order in
// which tiles are taken; `first` of them exist.  maps and ends point at the nearest one's words, `step` elements apart.
// Every lane of the wave calls it; lanes with `on` false (no channel, or nothing enters) get 0.
__device__ __forceinline__ float look_back(const uint64_t* maps, const uint32_t* ends, int64_t step, int64_t first,
                                           bool on) {
  float h = 0.0f;
  bool done = !on;
  while (!__all(done)) {
    if (!done) {
      uint32_t e[kGatedWindow];
      uint64_t m[kGatedWindow];
#pragma unroll
      for (int k = 0; k < kGatedWindow; ++k) {
        // before the first tile the state is 0
        e[k] = k < first ? __hip_atomic_load(ends + k * step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0u;
        m[k] = k < first ? __hip_atomic_load(maps + k * step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0u;
      }
      int near = 0;  // tiles over whose maps the nearest end state comes here
      bool open = true;
#pragma unroll
      for (int k = 0; k < kGatedWindow; ++k) {
        if (open && e[k] != kEmpty) {
          done = true;
          open = false;
          near = k;
        }
        if (m[k] == ~0ull) open = false;
      }
      if (done) {
#pragma unroll
        for (int k = kGatedWindow - 1; k >= 0; --k) {
          const float a = __builtin_bit_cast(float, static_cast<uint32_t>(m[k]));
          const float b = __builtin_bit_cast(float, static_cast<uint32_t>(m[k] >> 32));
          if (k == near) h = __builtin_bit_cast(float, e[k]);
          else if (k < near) h = fmaf(a, h, b);
        }
      }
    }
    if (!__all(done)) __builtin_amdgcn_s_sleep(2);
  }
  return h;
}

// Which rows of a tile begin a sequence, end one, or belong to one.
template <int ROWS>
struct TileRows {
  int32_t seq[ROWS];
  uint64_t first[(ROWS + 63) / 64], last[(ROWS + 63) / 64], live[(ROWS + 63) / 64];
};

template <int ROWS>
__device__ __forceinline__ void find_rows(TileRows<ROWS>& t, const GatedArgs& p, int64_t row0) {
  for (int at = threadIdx.x; at < ROWS; at += kGatedThreads) {
    const int64_t row = row0 + at;
    bool first = false, last = false, live = row < p.total;
    int64_t s = -1;
    if (live) {
      if (!p.cu) {
        s = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.seqlen);
        const int64_t in = row - s * p.seqlen;
        first = in == 0;
        last = in == p.seqlen - 1;
      } else {
        // the last entry not above the row
        int64_t lo = -1, hi = p.nseq + 1;
        while (hi - lo > 1) {
          const int64_t mid = (lo + hi) >> 1;
          if (p.cu[mid] <= row) lo = mid;
          else hi = mid;
        }
        live = lo >= 0 && lo < p.nseq;
        if (live) {
          s = lo;
          first = p.cu[s] == row;
          last = p.cu[s + 1] == row + 1;
        }
      }
    }
    t.seq[at] = static_cast<int32_t>(s);
    const uint64_t f = __ballot(first), l = __ballot(last), v = __ballot(live);
    if ((threadIdx.x & 63) == 0) {
      t.first[at >> 6] = f;
      t.last[at >> 6] = l;
      t.live[at >> 6] = v;
    }
  }
}

// V consecutive channels of a state: of sequence s's slot, zeros where it has none.  Fills h and says
// whether there is one to read.
template <int V>
__device__ __forceinline__ void initial_state(const GatedArgs& p, int64_t s, int64_t d, float (&h)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.0f;
  if (!p.in.data || (p.cu && !(p.has_initial && p.has_initial[s]))) return;
  const int64_t at = cache_offset(p.in, p.slots, s);
  if (at < 0) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (p.cb16) h[v] = bf16_lo(static_cast<const uint16_t*>(p.in.data)[at + d + v]);
    else h[v] = static_cast<const float*>(p.in.data)[at + d + v];
  }
}

template <int V>
__device__ __forceinline__ void final_state(const GatedArgs& p, int64_t s, int64_t d, int own, const float (&h)[V]) {
  if (!p.out.data) return;
  const int64_t at = cache_offset(p.out, p.slots, s);
  if (at < 0) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v < own) continue;
    if (p.cb16) static_cast<uint16_t*>(p.out.data)[at + d + v] = to_bf16(h[v]);
    else static_cast<float*>(p.out.data)[at + d + v] = h[v];
  }
}

__device__ __forceinline__ float sigmoid_f32(float v) { return hw_rcp(1.0f + hw_exp2(-v * kLog2e)); }

// w = sqrt(1 - a^2) with a = e^l.  1 - a^2 = -expm1(2 l): from p = -2 l = 0.35 on the difference itself (its
// rounding errors are below 2^-24 / 0.29 of it), below it p times the series of (1 - e^-p) / p up to p^6,
// which leaves p^7 / 8! < 2^-25 of the result: a difference would lose every digit of a slow decay.
__device__ __forceinline__ float input_weight(float l, float a) {
  const float p = -2.0f * l;
  float s = 1.0f / 5040.0f;
  s = fmaf(s, p, -1.0f / 720.0f);
  s = fmaf(s, p, 1.0f / 120.0f);
  s = fmaf(s, p, -1.0f / 24.0f);
  s = fmaf(s, p, 1.0f / 6.0f);
  s = fmaf(s, p, -0.5f);
  s = fmaf(s, p, 1.0f);
  return __builtin_amdgcn_sqrtf(p < 0.35f ? s * p : fmaf(-a, a, 1.0f));
}

// The channels of a lane: V neighbouring ones.  Where dim is no multiple of V the last lane's begin
// further left, so that every load is a whole vector; what it shares with its neighbour it computes
// but does not store (channels below d + own are another lane's).
template <int V>
struct LaneChannels {
  int64_t d;
  int own;
  __device__ __forceinline__ LaneChannels(int64_t natural, int64_t dim) {
    d = natural < dim - V ? natural : dim - V;
    own = natural - d < V ? static_cast<int>(natural - d) : V;
  }
};

template <bool BF16, int V>
__device__ __forceinline__ void store_own(void* base, int64_t idx, int own, const float (&val)[V]) {
  Run<BF16, V> r;
  r.set(val);
  if (own == 0) {
    r.store(base, idx);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v < own) continue;
      if constexpr (BF16) static_cast<uint16_t*>(base)[idx + v] = static_cast<uint16_t>(r.w[v >> 1] >> (16 * (v & 1)));
      else static_cast<uint32_t*>(base)[idx + v] = r.w[v];
    }
  }
}

// Parameters of a lane's channels: biases, and l = k r
template <int V>
struct LaneParams {
  float ab[V], xb[V], k[V];
  __device__ __forceinline__ LaneParams(const GatedArgs& p, int64_t d) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ab[v] = p.ab ? p.ab[d + v] : 0.0f;
      xb[v] = p.xb ? p.xb[d + v] : 0.0f;
      const float q = p.param[d + v];
      // finite, so that l a is 0 and not NaN where a is 0
      k[v] = -fminf(p.scale * (fmaxf(q, 0.0f) + log1pf(expf(-fabsf(q)))), 1e30f);
    }
  }
};

// The maps of a channel's lanes in the LDS, then what enters each of them.
template <int PARTS>
struct PartMaps {
  float a[PARTS][kGatedChannels];
  float b[PARTS][kGatedChannels];
  uint8_t own[PARTS];  // the part holds a state of its own
};

// A tile's number, in the order in which tiles are taken
__device__ __forceinline__ int64_t take_ticket(const GatedArgs& p, uint32_t* shared) {
  if (!p.ticket) return blockIdx.x;
  if (threadIdx.x == 0)
    *shared = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;  // (cleared to ~0)
  __syncthreads();
  return *shared;
}

template <bool BF16, int V, int R>
__global__ __launch_bounds__(kGatedThreads) void gated_scan_kernel(const GatedArgs p) {
  using S = GatedShape<V, R>;
  __shared__ TileRows<S::kRows> rows;
  __shared__ PartMaps<S::kParts> maps;
  __shared__ float entering[kGatedChannels];
  __shared__ uint32_t ticket;
  const int64_t n = take_ticket(p, &ticket);
  const int64_t tile = n / p.chains;
  const int64_t c0 = (n - tile * p.chains) * kGatedChannels;
  const int lane = threadIdx.x % S::kLanes, part = threadIdx.x / S::kLanes;
  const int64_t row0 = tile * S::kRows + part * R;
  const LaneChannels<V> ch(c0 + lane * V, p.dim);

  Run<BF16, V> x[R], ag[R], xg[R], z[R];
  const bool has_z = p.z != nullptr;
  const void* zsrc = has_z ? p.z : p.x;
  const int64_t zstride = has_z ? p.sz : p.sx;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int64_t row = row0 + j < p.total ? row0 + j : p.total - 1;
    x[j].load(p.x, row * p.sx + ch.d);
    ag[j].load(p.ag, row * p.sag + ch.d);
    xg[j].load(p.xg, row * p.sxg + ch.d);
    z[j].load(zsrc, row * zstride + ch.d);
  }
  const LaneParams<V> par(p, ch.d);
  find_rows(rows, p, tile * S::kRows);
  __syncthreads();
  const int at0 = part * R;
  const uint32_t bits = (1u << R) - 1u;
  const uint32_t first = static_cast<uint32_t>(rows.first[at0 >> 6] >> (at0 & 63)) & bits;
  const uint32_t last = static_cast<uint32_t>(rows.last[at0 >> 6] >> (at0 & 63)) & bits;
  const uint32_t live = static_cast<uint32_t>(rows.live[at0 >> 6] >> (at0 & 63)) & bits;

  float a[R][V], b[R][V], A[V], B[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll
  for (int j = 0; j < R; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float l = par.k[v] * sigmoid_f32(ag[j].get(v) + par.ab[v]);
      const float i = sigmoid_f32(xg[j].get(v) + par.xb[v]);
      const float e = hw_exp2(l * kLog2e);
      const bool on = live >> j & 1;
      a[j][v] = on ? e : 1.0f;
      b[j][v] = on ? input_weight(l, e) * (i * x[j].get(v)) : 0.0f;
    }
    if (first >> j & 1) {
      float h[V];
      initial_state<V>(p, rows.seq[at0 + j], ch.d, h);
#pragma unroll
      for (int v = 0; v < V; ++v) b[j][v] = fmaf(a[j][v], h[v], b[j][v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      A[v] *= a[j][v];
      B[v] = first >> j & 1 ? b[j][v] : fmaf(a[j][v], B[v], b[j][v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    maps.a[part][lane * V + v] = A[v];
    maps.b[part][lane * V + v] = B[v];
  }
  if (lane == 0) maps.own[part] = first != 0;
  __syncthreads();

  if (threadIdx.x < kGatedChannels) {
    const int c = threadIdx.x, l = c / V, v = c - l * V;
    const LaneChannels<V> my(c0 + l * V, p.dim);
    const bool on = v >= my.own;
    const int64_t d = my.d + v;
    // what comes before each part, as a map of what enters the tile
    float ta = 1.0f, tb = 0.0f;
    bool own = false;
#pragma unroll
    for (int k = 0; k < S::kParts; ++k) {
      const float pa = maps.a[k][c], pb = maps.b[k][c];
      maps.a[k][c] = own ? 0.0f : ta;
      maps.b[k][c] = tb;
      if (maps.own[k]) {
        own = true;
        tb = pb;
      } else {
        ta *= pa;
        tb = fmaf(pa, tb, pb);
      }
    }
    float h = 0.0f;
    if (p.ticket) {
      const int64_t at = tile * p.dim + d;
      if (on && !own) publish(p.maps + at, ta, tb);
      if (on && own) publish(p.ends + at, tb);
      h = look_back(p.maps + at - p.dim, p.ends + at - p.dim, -p.dim, tile, on && !(rows.first[0] & 1));
      if (on && !own) publish(p.ends + at, fmaf(ta, h, tb));
    }
    entering[c] = h;
  }
  __syncthreads();

  float h[V];
  bool before = false;  // a part before this one has a state of its own
#pragma unroll
  for (int k = 0; k < S::kParts; ++k) before |= k < part && maps.own[k];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = lane * V + v;
    h[v] = before ? maps.b[part][c] : fmaf(maps.a[part][c], entering[c], maps.b[part][c]);
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = first >> j & 1 ? b[j][v] : fmaf(a[j][v], h[v], b[j][v]);
      o[v] = has_z ? h[v] * silu_f32(z[j].get(v)) : h[v];
    }
    if (live >> j & 1) store_own<BF16, V>(p.y, (row0 + j) * p.sy + ch.d, ch.own, o);
    if (last >> j & 1) final_state<V>(p, rows.seq[at0 + j], ch.d, ch.own, h);
  }
  static_assert(kGatedSave % R == 0, "a checkpoint is the state after a part");
  if (p.ckpt && (row0 + R) % kGatedSave == 0 && row0 + R <= p.total)
    store_own<false, V>(p.ckpt, (row0 / kGatedSave) * p.dim + ch.d, ch.own, h);
}

// Backward.  With g = dy silu(z) (+ dlast at a sequence's last row), from the last row on:
//   G_t = g_t + a_{t+1} G_{t+1},  q = -l e^{2l} / w,  E_t = G_t (l a h_{t-1} + u q)   (= l dL/dl)
//   da_gate = E (1 - r), dx = G w i, dx_gate = G w x i (1 - i), dz = dy h silu'(z), dh_0 = a_1 G_1
// q is 0 where w is (a = 1): l / w -> 0 as l -> 0, so the product has that limit though dw/dl has none.
// The states come from the checkpoint before the tile and the tile's own rows; a G is carried from tile
// to tile like the forward's state, tiles taken from the last one on.
template <bool BF16, int V, int R>
__global__ __launch_bounds__(kGatedThreads) void gated_scan_bwd_kernel(const GatedArgs p) {
  using S = GatedShape<V, R>;
  static_assert(S::kRows == kGatedSave, "a tile begins behind a checkpoint");
  __shared__ TileRows<S::kRows> rows;
  __shared__ PartMaps<S::kParts> fwd;      // the states' maps
  __shared__ float back[S::kParts][kGatedChannels];
  __shared__ uint8_t ends[S::kParts];      // the part holds a sequence's last row
  __shared__ uint32_t ticket;
  const int64_t n = take_ticket(p, &ticket);
  const int64_t turn = n / p.chains, tile = p.tiles - 1 - turn;
  const int64_t c0 = (n - turn * p.chains) * kGatedChannels;
  const int lane = threadIdx.x % S::kLanes, part = threadIdx.x / S::kLanes;
  const int64_t row0 = tile * S::kRows + part * R;
  const LaneChannels<V> ch(c0 + lane * V, p.dim);
  const bool has_z = p.z != nullptr;

  Run<BF16, V> x[R], ag[R], xg[R], z[R], dy[R];
  const void* zsrc = has_z ? p.z : p.x;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int64_t row = row0 + j < p.total ? row0 + j : p.total - 1;
    x[j].load(p.x, row * p.dim + ch.d);
    ag[j].load(p.ag, row * p.dim + ch.d);
    xg[j].load(p.xg, row * p.dim + ch.d);
    z[j].load(zsrc, row * p.dim + ch.d);
    dy[j].load(p.dy, row * p.dim + ch.d);
  }
  const LaneParams<V> par(p, ch.d);
  find_rows(rows, p, tile * S::kRows);
  __syncthreads();
  const int at0 = part * R;
  const uint32_t bits = (1u << R) - 1u;
  const uint32_t first = static_cast<uint32_t>(rows.first[at0 >> 6] >> (at0 & 63)) & bits;
  const uint32_t last = static_cast<uint32_t>(rows.last[at0 >> 6] >> (at0 & 63)) & bits;
  const uint32_t live = static_cast<uint32_t>(rows.live[at0 >> 6] >> (at0 & 63)) & bits;

  float a[R][V], h[R][V], g[R][V], f[R][V], r[R][V], i[R][V], w[R][V];
  float A[V], B[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const bool on = live >> j & 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      r[j][v] = sigmoid_f32(ag[j].get(v) + par.ab[v]);
      i[j][v] = sigmoid_f32(xg[j].get(v) + par.xb[v]);
      const float l = par.k[v] * r[j][v], e = hw_exp2(l * kLog2e);
      w[j][v] = input_weight(l, e);
      a[j][v] = on ? e : 1.0f;
      h[j][v] = on ? w[j][v] * (i[j][v] * x[j].get(v)) : 0.0f;
      const float d = on ? dy[j].get(v) : 0.0f, zv = z[j].get(v), o = sigmoid_f32(zv);
      g[j][v] = on && has_z ? d * (zv * o) : d;
      f[j][v] = d * (o * fmaf(zv, 1.0f - o, 1.0f));
    }
    if (first >> j & 1) {
      float h0[V];
      initial_state<V>(p, rows.seq[at0 + j], ch.d, h0);
#pragma unroll
      for (int v = 0; v < V; ++v) h[j][v] = fmaf(a[j][v], h0[v], h[j][v]);
    }
    if ((last >> j & 1) && p.dlast) {
#pragma unroll
      for (int v = 0; v < V; ++v) g[j][v] += p.dlast[static_cast<int64_t>(rows.seq[at0 + j]) * p.dim + ch.d + v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      A[v] *= a[j][v];
      B[v] = first >> j & 1 ? h[j][v] : fmaf(a[j][v], B[v], h[j][v]);
    }
  }
  float C[V];  // a G of the row that the part begins with
#pragma unroll
  for (int v = 0; v < V; ++v) C[v] = 0.0f;
#pragma unroll
  for (int j = R - 1; j >= 0; --j)
#pragma unroll
    for (int v = 0; v < V; ++v) C[v] = a[j][v] * (last >> j & 1 ? g[j][v] : g[j][v] + C[v]);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    fwd.a[part][lane * V + v] = A[v];
    fwd.b[part][lane * V + v] = B[v];
    back[part][lane * V + v] = C[v];
  }
  if (lane == 0) {
    fwd.own[part] = first != 0;
    ends[part] = last != 0;
  }
  __syncthreads();

  // the first wave runs the states through the parts, the second the adjoint
  const int wave = threadIdx.x / 64;
  if (wave < 2) {
    const int c = threadIdx.x & 63, l = c / V, v = c - l * V;
    const LaneChannels<V> my(c0 + l * V, p.dim);
    const bool on = v >= my.own;
    const int64_t d = my.d + v;
    float pa[S::kParts], pb[S::kParts];
#pragma unroll
    for (int k = 0; k < S::kParts; ++k) {
      pa[k] = fwd.a[k][c];
      pb[k] = wave == 0 ? fwd.b[k][c] : back[k][c];
    }
    if (wave == 0) {
      float s = tile > 0 ? p.ckpt[(tile - 1) * p.dim + d] : 0.0f;
#pragma unroll
      for (int k = 0; k < S::kParts; ++k) {
        fwd.b[k][c] = s;
        s = fwd.own[k] ? pb[k] : fmaf(pa[k], s, pb[k]);
      }
    } else {
      float ta = 1.0f, tb = 0.0f;
      bool own = false;
#pragma unroll
      for (int k = S::kParts - 1; k >= 0; --k) {
        if (ends[k]) {
          own = true;
          tb = pb[k];
        } else {
          ta *= pa[k];
          tb = fmaf(pa[k], tb, pb[k]);
        }
      }
      float s = 0.0f;
      if (p.ticket) {
        const int64_t at = tile * p.dim + d;
        if (on && !own) publish(p.maps + at, ta, tb);
        if (on && own) publish(p.ends + at, tb);
        s = look_back(p.maps + at + p.dim, p.ends + at + p.dim, p.dim, turn, on && !(rows.last[0] >> 63));
        if (on && !own) publish(p.ends + at, fmaf(ta, s, tb));
      }
#pragma unroll
      for (int k = S::kParts - 1; k >= 0; --k) {
        back[k][c] = s;
        s = ends[k] ? pb[k] : fmaf(pa[k], s, pb[k]);
      }
    }
  }
  __syncthreads();

  float enter[V], se[V], sa[V], sx[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    enter[v] = fwd.b[part][lane * V + v];
    C[v] = back[part][lane * V + v];
    se[v] = sa[v] = sx[v] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) h[j][v] = first >> j & 1 ? h[j][v] : fmaf(a[j][v], j > 0 ? h[j - 1][v] : enter[v], h[j][v]);
#pragma unroll
  for (int j = R - 1; j >= 0; --j) {
    float prev[V], odx[V], oda[V], odg[V], odz[V];
#pragma unroll
    for (int v = 0; v < V; ++v) prev[v] = j > 0 ? h[j > 0 ? j - 1 : 0][v] : enter[v];
    if (first >> j & 1) initial_state<V>(p, rows.seq[at0 + j], ch.d, prev);
    const bool on = live >> j & 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float G = last >> j & 1 ? g[j][v] : g[j][v] + C[v];
      const float xv = x[j].get(v), l = par.k[v] * r[j][v];
      const float la = l * a[j][v];
      const float q = w[j][v] > 0.0f ? -la * a[j][v] * hw_rcp(w[j][v]) : 0.0f;
      const float E = on ? G * fmaf(la, prev[v], i[j][v] * xv * q) : 0.0f;
      odz[v] = f[j][v] * h[j][v];
      oda[v] = E * (1.0f - r[j][v]);
      odx[v] = G * w[j][v] * i[j][v];
      odg[v] = on ? odx[v] * xv * (1.0f - i[j][v]) : 0.0f;
      se[v] += E;
      sa[v] += oda[v];
      sx[v] += odg[v];
      C[v] = a[j][v] * G;
    }
    if (on) {
      const int64_t at = (row0 + j) * p.dim + ch.d;
      store_own<BF16, V>(p.dx, at, ch.own, odx);
      store_own<BF16, V>(p.dag, at, ch.own, oda);
      store_own<BF16, V>(p.dxg, at, ch.own, odg);
      if (has_z) store_own<BF16, V>(p.dz, at, ch.own, odz);
      if ((first >> j & 1) && p.dh0)
        store_own<false, V>(p.dh0, static_cast<int64_t>(rows.seq[at0 + j]) * p.dim + ch.d, ch.own, C);
    }
  }
  // sums over the tile's rows, in the order of its parts
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    fwd.a[part][lane * V + v] = se[v];
    fwd.b[part][lane * V + v] = sa[v];
    back[part][lane * V + v] = sx[v];
  }
  __syncthreads();
  if (wave < 3) {
    const int c = threadIdx.x & 63, l = c / V, v = c - l * V;
    const LaneChannels<V> my(c0 + l * V, p.dim);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < S::kParts; ++k) s += wave == 0 ? fwd.a[k][c] : wave == 1 ? fwd.b[k][c] : back[k][c];
    if (v >= my.own) p.partial[(tile * 3 + wave) * p.dim + my.d + v] = s;
  }
}

struct GatedSumArgs {
  const float* partial;
  const float* param;
  float *dparam, *dab, *dxb;  // the last two may be NULL
  int64_t tiles, dim;
};

// Sums of the tiles' partial sums, 64 channels and one quantity a workgroup: 16 rows of tiles at a time.
constexpr int kGatedSumThreads = 1024;
__global__ __launch_bounds__(kGatedSumThreads) static void gated_sum_kernel(const GatedSumArgs p) {
  __shared__ float sums[16][64];
  const int c = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + c;
  const int k = blockIdx.y;
  float s = 0.0f;
  if (d < p.dim) {
    const float* q = p.partial + k * p.dim + d;
#pragma unroll 8
    for (int64_t t = part; t < p.tiles; t += 16) s += q[t * 3 * p.dim];
  }
  sums[part][c] = s;
  __syncthreads();
  if (part == 0 && d < p.dim) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += sums[i][c];
    if (k == 0) {
      // d softplus(v) / softplus(v): sigmoid(v) / softplus(v), 1 to fp32 below -17
      const float v = p.param[d];
      const float ratio = v < -17.0f ? 1.0f : 1.0f / (1.0f + expf(-v)) / (fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))));
      p.dparam[d] = s * ratio;
    } else if (float* out = k == 1 ? p.dab : p.dxb) {
      out[d] = s;
    }
  }
}

// The words that tiles publish, and the ticket: all ones.
__global__ __launch_bounds__(256) static void gated_clear_kernel(U32x4* p, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = U32x4{kEmpty, kEmpty, kEmpty, kEmpty};
}

// States of sequences of no rows (whole batches of them): the initial ones, or zeros.
__global__ __launch_bounds__(256) static void gated_keep_kernel(const float* in, float* out, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) out[i] = in ? in[i] : 0.0f;
}

// One token on a cache: a thread owns V channels of R entries.
struct GatedStepArgs {
  GatedArgs g;      // rows are the batch's entries; in: the cache
  int64_t batch;
};

template <bool BF16, bool CB16, int V, int R>
__global__ __launch_bounds__(kGatedThreads) void gated_step_kernel(const GatedStepArgs q) {
  const GatedArgs& p = q.g;
  const int64_t natural = (static_cast<int64_t>(blockIdx.x) * kGatedThreads + threadIdx.x) * V;
  if (natural >= p.dim) return;
  const LaneChannels<V> ch(natural, p.dim);
  const LaneParams<V> par(p, ch.d);
  const bool has_z = p.z != nullptr;
  const void* zsrc = has_z ? p.z : p.x;
  const int64_t zstride = has_z ? p.sz : p.sx;
  for (int64_t b0 = static_cast<int64_t>(blockIdx.y) * R; b0 < q.batch; b0 += static_cast<int64_t>(gridDim.y) * R) {
    int64_t at[R], e[R];
    Run<CB16, V> st[R];
    Run<BF16, V> x[R], ag[R], xg[R], z[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      e[k] = b0 + k < q.batch ? b0 + k : b0;
      at[k] = b0 + k < q.batch ? cache_offset(p.in, p.slots, b0 + k) : -1;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      // every load on every path: an entry past the batch or without a slot reads entry b0 and slot 0
      x[k].load(p.x, e[k] * p.sx + ch.d);
      ag[k].load(p.ag, e[k] * p.sag + ch.d);
      xg[k].load(p.xg, e[k] * p.sxg + ch.d);
      z[k].load(zsrc, e[k] * zstride + ch.d);
      st[k].load(p.in.data, (at[k] < 0 ? 0 : at[k]) + ch.d);
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float h[V], y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float l = par.k[v] * sigmoid_f32(ag[k].get(v) + par.ab[v]);
        const float i = sigmoid_f32(xg[k].get(v) + par.xb[v]);
        const float a = hw_exp2(l * kLog2e);
        h[v] = fmaf(a, st[k].get(v), input_weight(l, a) * (i * x[k].get(v)));
        y[v] = has_z ? h[v] * silu_f32(z[k].get(v)) : h[v];
      }
      if (at[k] < 0) continue;
      store_own<CB16, V>(p.in.data, at[k] + ch.d, ch.own, h);
      store_own<BF16, V>(p.y, (b0 + k) * p.sy + ch.d, ch.own, y);
    }
  }
}

}  // namespace ssm
