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
//  - Every wait ends: a channel's tiles are in one queue and taken from it in the order of the axis, so that a
//    tile waits only for tiles that running workgroups have taken before it, the first tile waits for none, and
//    a waiting wave leaves its SIMD to others.
//  - Results do not depend on timing: whoever computes the end state of a tile does it by the same
//    operation, fma(A, entering state, B), from the same two words.
//  - No fences: what a tile publishes is one 64-bit word a channel, written by relaxed atomic stores at agent scope,
//    and is itself the sign of its arrival.
#pragma once

#include "cache.hpp"

namespace ssm {

constexpr int kGatedThreads = 256;
constexpr int kGatedChannels = 64;   // channels of a workgroup: one 128-byte line of a bf16 row
constexpr int kGatedSave = 64;       // rows between checkpoints
constexpr uint32_t kGatedQueues = 4, kGatedQueueWords = 32;  // queues of tiles, and words from a counter to the next

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
  uint32_t* ticket;              // the queues' counters (NULL: no tile enters another)
  uint64_t* words;               // (tiles, dim), in the order in which tiles are taken
  int64_t tiles, each;           // tiles, and those of a sequence if none holds rows of two (else 0)
  int64_t pitch;                 // rows from a tile to the next, if tiles hold rows of several
  int32_t chains;                // blocks of kGatedChannels channels
  // backward
  const void* dy;
  const float* dlast;
  void *dx, *dag, *dxg, *dz;
  float* dh0;
  float* partial;                // (tiles, 3, dim): sums of E, da_gate, dx_gate
  float *dparam, *dab, *dxb;     // the sums over all rows; the last two may be NULL
};

// Lanes of a workgroup: kLanes lanes of V channels, the others its rows, R each.
template <int V, int R>
struct GatedShape {
  static constexpr int kLanes = kGatedChannels / V;
  static constexpr int kParts = kGatedThreads / kLanes;  // row groups
  static constexpr int kRows = kParts * R;               // rows of a tile
};

// A tile's word: nothing yet (all ones), then its map, then its end state.  A map's factor is in the low half, an end
// state in the high half above kEnd, which is no factor's.
constexpr uint32_t kEmpty = 0xffffffffu, kEnd = 0xfffffffeu;
__device__ __forceinline__ void publish(uint64_t* p, uint32_t lo, float hi) {
  __hip_atomic_store(p, (static_cast<uint64_t>(__builtin_bit_cast(uint32_t, hi)) << 32) | lo, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_end(uint64_t* p, float h) { publish(p, kEnd, h); }
__device__ __forceinline__ void publish_map(uint64_t* p, float a, float b) {
  const uint32_t lo = __builtin_bit_cast(uint32_t, a);
  publish(p, lo >= kEnd ? 0x7fc00000u : lo, b);  // (those are NaNs)
}

// The state that leaves the tile before this one.  words points at that tile's; those of the tiles before it lie
// `step` elements on each, `first` tiles in all.  WINDOW tiles' words are asked for at once, as many as leave the
// kernels' registers in place: forward with 4 and 8, 30000 x 256 bf16 rows take 56 and 43 us, but 8 x 2048 x 1536
// 67 and 69 and 12288 x 5120 packed ones 162 and 165; backward with 3, 4 and 5 30000 x 256 take 117, 101 and 91 us,
// 2000 x 40 x 1024 403, 408 and 425, and in fp32 with 2 and 3 400 x 33 x 1000 133 and 139.
// Every lane of the wave calls it; lanes with `on` false (no channel, or nothing enters) get 0.
template <int WINDOW>
__device__ __forceinline__ float look_back(const uint64_t* words, int64_t step, int64_t first, bool on) {
  float h = 0.0f;
  bool done = !on;
  while (!__all(done)) {
    if (!done) {
      uint64_t w[WINDOW];
#pragma unroll
      for (int k = 0; k < WINDOW; ++k)  // before the first tile the state is 0
        w[k] = k < first ? __hip_atomic_load(words + k * step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : uint64_t{kEnd};
      int near = 0;  // tiles over whose maps the nearest end state comes here
      bool open = true;
#pragma unroll
      for (int k = 0; k < WINDOW; ++k) {
        const uint32_t lo = static_cast<uint32_t>(w[k]);
        if (open && lo == kEnd) {
          done = true;
          near = k;
        }
        open = open && lo < kEnd;
      }
      if (done) {
#pragma unroll
        for (int k = WINDOW - 1; k >= 0; --k) {
          const float a = __builtin_bit_cast(float, static_cast<uint32_t>(w[k]));
          const float b = __builtin_bit_cast(float, static_cast<uint32_t>(w[k] >> 32));
          if (k == near) h = b;
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
  // all of one sequence, neither its first nor its last
  __device__ __forceinline__ bool inside() const {
    uint64_t other = 0;
#pragma unroll
    for (int i = 0; i < (ROWS + 63) / 64; ++i)
      other |= first[i] | last[i] | (live[i] ^ (ROWS < 64 ? (1ull << (ROWS & 63)) - 1 : ~0ull));
    return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(other) | static_cast<uint32_t>(other >> 32)) == 0;
  }
};

// The last sequence whose first row is not above `row`, as an index into cu (-1: none).  By one lane.
__device__ inline int64_t last_not_above(const int32_t* cu, int64_t nseq, int64_t row) {
  int64_t lo = -1, hi = nseq + 1;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (cu[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

// By the first threads, a row each.  Packed rows: a wave reads 64 entries of cu, from the last one that is
// not above its first row on (64 probes at a time: one round trip up to 63 sequences, two up to 4095), and
// its lanes search them in its registers.
template <int ROWS>
__device__ __forceinline__ void find_rows(TileRows<ROWS>& t, const GatedArgs& p, uint32_t row0, int64_t end) {
  const uint32_t at = threadIdx.x;
  if (at >= (ROWS < 64 ? 64 : ROWS)) return;  // whole waves
  const int32_t row = static_cast<int32_t>(row0 + at);  // (total is at most 2^31 - 1; rows behind it are not live)
  bool first = false, last = false, live = at < ROWS && row0 + at < end;
  int32_t s = -1;
  if (!p.cu) {
    if (live) {
      const uint32_t len = static_cast<uint32_t>(p.seqlen), n = (row0 + at) / len, in = row0 + at - n * len;
      s = static_cast<int32_t>(n);
      first = in == 0;
      last = in == len - 1;
    }
  } else {
    const int lane = threadIdx.x & 63;
    const int64_t from = static_cast<int64_t>(row0) + (at - lane);  // the wave's first row
    int64_t s0 = 0;
    for (int64_t left = p.nseq + 1; left > 64;) {
      const int64_t step = (left + 63) / 64, i = lane * step;
      const int c = __popcll(__ballot(i < left && p.cu[s0 + (i < left ? i : 0)] <= from));
      const int64_t skip = c > 0 ? (c - 1) * step : 0;
      s0 += skip;
      left = left - skip < step ? left - skip : step;
    }
    const int32_t entry = s0 + lane <= p.nseq ? p.cu[s0 + lane] : INT32_MAX;
    int c = 0;  // entries not above the row
#pragma unroll
    for (int k = 32; k; k >>= 1) c += __shfl(entry, c + k - 1) <= row ? k : 0;
    c += __shfl(entry, c < 64 ? c : 63) <= row && c < 64 ? 1 : 0;
    int32_t begin = __shfl(entry, c > 0 ? c - 1 : 0), stop = __shfl(entry, c < 64 ? c : 63);
    int64_t n = s0 + c - 1;
    if (live && c == 64) {  // more sequences than that begin here
      n = last_not_above(p.cu, p.nseq, row);
      begin = n >= 0 ? p.cu[n] : 0;
      stop = n >= 0 && n < p.nseq ? p.cu[n + 1] : 0;
    }
    live = live && c > 0 && n >= 0 && n < p.nseq;
    if (live) {
      s = static_cast<int32_t>(n);
      first = begin == row;
      last = stop == row + 1;
    }
  }
  if (at < ROWS) t.seq[at] = s;
  const uint64_t f = __ballot(first), l = __ballot(last), v = __ballot(live);
  if ((at & 63) == 0) {
    t.first[at >> 6] = f;
    t.last[at >> 6] = l;
    t.live[at >> 6] = v;
  }
}

// A part's rows of a tile as bits
template <int R>
struct PartRows {
  uint32_t first, last, live;
  template <int ROWS>
  __device__ __forceinline__ PartRows(const TileRows<ROWS>& t, int at) {
    constexpr uint32_t kAll = (1u << R) - 1u;
    first = static_cast<uint32_t>(t.first[at >> 6] >> (at & 63)) & kAll;
    last = static_cast<uint32_t>(t.last[at >> 6] >> (at & 63)) & kAll;
    live = static_cast<uint32_t>(t.live[at >> 6] >> (at & 63)) & kAll;
  }
};

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
__device__ __forceinline__ void final_state(const GatedArgs& p, int64_t s, int64_t d, const float (&h)[V]) {
  if (!p.out.data) return;
  const int64_t at = cache_offset(p.out, p.slots, s);
  if (at < 0) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (p.cb16) static_cast<uint16_t*>(p.out.data)[at + d + v] = to_bf16(h[v]);
    else static_cast<float*>(p.out.data)[at + d + v] = h[v];
  }
}

// sigmoid(v + bias) with c = -bias log2(e): one fused multiply-add, exp2, sum, reciprocal
__device__ __forceinline__ float sigmoid_f32(float v, float c) { return hw_rcp(1.0f + hw_exp2(fmaf(v, -kLog2e, c))); }
__device__ __forceinline__ float sigmoid_f32(float v) { return hw_rcp(1.0f + hw_exp2(v * -kLog2e)); }

// w = sqrt(1 - a^2) with a = e^l and p = -2 l.  1 - a^2 = -expm1(-p): from p = 0.35 on the difference itself (its
// rounding errors are below 2^-24 / 0.29 of it), below it p times a polynomial that is (1 - e^-p) / p there to
// 0.54 * 2^-24 (a minimax fit with these rounded coefficients): a difference would lose every digit of a
// slow decay.
__device__ __forceinline__ float input_weight(float p, float a) {
  float s = 0x1.d82f32p-8f;
  s = fmaf(s, p, -0x1.528dfp-5f);
  s = fmaf(s, p, 0x1.553f22p-3f);
  s = fmaf(s, p, -0x1.ffff82p-2f);
  s = fmaf(s, p, 1.0f);
  return __builtin_amdgcn_sqrtf(p < 0.35f ? s * p : fmaf(-a, a, 1.0f));
}

// The channels of a workgroup, a block of up to kGatedChannels, and of its lanes, V neighbouring ones each.
// Where the last lane's would pass dim they begin further left, so that every access is a whole vector: what
// it shares with its neighbour both compute and store alike.  A last block of fewer than V channels takes V
// more from the block before it, so that no two workgroups share a channel (a cached state is read and
// written by one alone).
template <int V>
struct Channels {
  int64_t first, dim;
  int32_t count;
  __device__ __forceinline__ Channels(uint32_t block, int64_t width) : first(int64_t{block} * kGatedChannels), dim(width) {
    const int64_t left = dim - first, next = left - kGatedChannels;
    count = static_cast<int32_t>(left < kGatedChannels ? left : kGatedChannels);
    if (block > 0 && left < V) {
      first -= V;
      count += V;
    } else if (next > 0 && next < V) {
      count -= V;
    }
  }
  // the first channel of lane l, and whether it has any
  __device__ __forceinline__ int64_t of(int l) const {
    const int64_t d = first + l * V;
    return d < dim - V ? d : dim - V;
  }
  __device__ __forceinline__ bool has(int l) const { return l * V < count; }
};

// l = k r of a channel: k = -a_scale softplus(a_param), by the library's exp and log1p (once a workgroup and
// channel, not once a lane).  Not infinite, so that l a is 0 and not NaN where a is 0; NaN where a_param is.
__device__ __forceinline__ float decay_rate(float scale, float q) {
  const float k = scale * (fmaxf(q, 0.0f) + log1pf(expf(-fabsf(q))));
  return k > 1e30f ? -1e30f : -k;
}

// -bias log2(e) of a lane's channels (sigmoid_f32)
template <int V>
__device__ __forceinline__ void load_bias(const float* bias, int64_t d, float (&c)[V]) {
  Run<false, V> r;
  if (bias) r.load(bias, d);
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = bias ? r.get(v) * -kLog2e : 0.0f;
}

// A lane's rows of a tensor, `stride` elements apart (not FULL: past the last row that row again).  The
// addresses are a base that the workgroup shares and a lane's 32-bit offset (row strides are below 2^23).
template <bool FULL, bool BF16, int V, int R>
__device__ __forceinline__ void load_rows(Run<BF16, V> (&out)[R], const void* base, int64_t stride, int64_t tile0,
                                          int at, int64_t d, int64_t total) {
  constexpr int ES = BF16 ? 2 : 4;
  const char* q = static_cast<const char*>(base) + tile0 * stride * ES;
  if constexpr (FULL) {
    const uint32_t off = (static_cast<uint32_t>(at) * static_cast<uint32_t>(stride) + static_cast<uint32_t>(d)) * ES;
#pragma unroll
    for (int j = 0; j < R; ++j) out[j].load_bytes(q + j * stride * ES + off);
  } else {
    const uint32_t left = static_cast<uint32_t>(total - tile0) - 1u;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const uint32_t row = static_cast<uint32_t>(at + j) < left ? static_cast<uint32_t>(at + j) : left;
      out[j].load_bytes(q + (row * static_cast<uint32_t>(stride) + static_cast<uint32_t>(d)) * ES);
    }
  }
}

// A row of no sequence leaves a state as it is: a decay of 1 (an a_gate of -inf) and no input
template <bool BF16, int V>
__device__ __forceinline__ void no_row(Run<BF16, V>& r, bool off, bool closed) {
#pragma unroll
  for (int i = 0; i < Run<BF16, V>::kWords; ++i) r.w[i] = off ? (closed ? (BF16 ? 0xff80ff80u : 0xff800000u) : 0u) : r.w[i];
}

// The decay of a stretch of steps, from the product of theirs and the least of them: 0 only if a step's is.  The
// product alone rounds to 0 after a few dozen ordinary steps and would make a NaN of an infinite state that each of
// them keeps, here or there as tiles happen to begin.  2^-149 in its place keeps that much of a finite state, twice what
// a product down there is rounded by: below 2^-24 up to states of 4e37.  (No decay exceeds 1, so the product is at
// most the least and the middle one of the three is meant.)
__device__ __forceinline__ float stretch_decay(float product, float least) {
  return __builtin_amdgcn_fmed3f(product, least, 0x1p-149f);
}
__device__ __forceinline__ float compose_decay(float a, float b) { return stretch_decay(a * b, fminf(a, b)); }
template <int V, int R>
__device__ __forceinline__ void compose_decays(const float (&a)[R][V], float (&out)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float least = a[0][v];
    out[v] = a[0][v];
#pragma unroll
    for (int j = 1; j < R; ++j) {
      out[v] *= a[j][v];
      least = fminf(least, a[j][v]);
    }
    out[v] = stretch_decay(out[v], least);
  }
}

// The maps of a channel's lanes in the LDS, then what enters each of them.
template <int PARTS>
struct PartMaps {
  float a[PARTS][kGatedChannels];
  float b[PARTS][kGatedChannels];
  uint8_t own[PARTS];  // the part holds a state of its own
};

// The tile that a workgroup takes: the next one of a queue.  Tiles of a sequence that share no row with another come
// in the order (their place in the sequence, sequence, channels), so that a tile waits for one that was taken a batch
// earlier: 8 x 2048 x 1536 bf16 rows take 10% less forward than in the order of the rows, and 15% less backward.
// The channels are shared among four queues, which the XCDs take from in turn: neighbouring channels, whose lines
// may be the same, stay on few XCDs, and fewer workgroups ask for one counter.  With 1, 2, 4 and 8 queues 8 x 2048 x
// 1536 take 72, 69, 68 and 68 us forward and 122, 119, 118 and 119 backward; 30011 x 2560 180, 180, 179, 185 and 337,
// 341, 344, 357 (the queues' rows drift apart); 30000 x 256 10% less each with 4 than with 1.
// (Workgroups that stay and take tile after tile with the next number asked for ahead: half as much again, since the
// tile that a number stands for waits.)
struct Turn {
  uint32_t block, turn;  // in the order in which tiles are taken
  uint32_t before;       // tiles before it that may enter it
  uint32_t apart;        // turns between those
  uint32_t s;            // its sequence, where tiles have one
  int64_t row0;          // its first row
  int64_t end;           // where its rows end at the latest
  template <int ROWS>
  __device__ __forceinline__ static Turn take(const GatedArgs& p, uint32_t (&shared)[2], bool backward) {
    Turn t;
    const uint32_t tiles = static_cast<uint32_t>(p.tiles), chains = static_cast<uint32_t>(p.chains);
    uint32_t n = blockIdx.x, first = 0, width = chains;
    if (p.ticket) {
      const uint32_t groups = chains < kGatedQueues ? chains : kGatedQueues;
      if (threadIdx.x == 0) {
        // Workgroups are as many as tiles and take one each, so a queue with one left is found within a round
        uint32_t g = n % kGatedQueues % groups, k;
        while (true) {
          k = __hip_atomic_fetch_add(p.ticket + g * kGatedQueueWords, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;  // (from ~0)
          if (k < ((g + 1) * chains / groups - g * chains / groups) * tiles) break;
          g = g + 1 < groups ? g + 1 : 0;
        }
        shared[0] = k;
        shared[1] = g;
      }
      __syncthreads();
      n = __builtin_amdgcn_readfirstlane(shared[0]);
      const uint32_t g = __builtin_amdgcn_readfirstlane(shared[1]);
      first = g * chains / groups;
      width = (g + 1) * chains / groups - first;
    }
    t.turn = n / width;
    t.block = first + n - t.turn * width;
    if (p.each) {
      const uint32_t each = static_cast<uint32_t>(p.each), batch = static_cast<uint32_t>(p.nseq);
      const uint32_t place = t.turn / batch;
      t.s = t.turn - place * batch;
      t.before = place;
      t.apart = batch;
      t.row0 = t.s * p.seqlen + static_cast<int64_t>(backward ? each - 1 - place : place) * ROWS;
      t.end = (t.s + int64_t{1}) * p.seqlen;
    } else {
      t.before = t.turn;
      t.apart = 1;
      t.s = 0;
      t.row0 = static_cast<int64_t>(backward ? tiles - 1 - t.turn : t.turn) * p.pitch;
      t.end = t.row0 + p.pitch < p.total ? t.row0 + p.pitch : p.total;
    }
    return t;
  }
};

// Checkpoints: the state after every kGatedSave-th row, of each sequence by itself where tiles are (`each`), else
// of the batch's rows.  The index of the one before row `next` (a multiple of kGatedSave from its sequence's or the
// batch's first on), or -1: none.
__device__ __forceinline__ int64_t checkpoint_after(const GatedArgs& p, const Turn& tile, int64_t next) {
  const uint32_t from = static_cast<uint32_t>(next - (p.each ? tile.end - p.seqlen : 0));
  if (next > tile.end || from < kGatedSave || from % kGatedSave) return -1;
  const uint32_t n = p.each ? tile.s * (static_cast<uint32_t>(p.seqlen) / kGatedSave) : 0;  // (fewer than rows)
  return n + from / kGatedSave - 1;
}

// Forward.  Bound by the memory, as far as loading, composing, waiting and storing of three workgroups a CU overlap:
// 8 x 2048 x 1536 bf16 take 64 us (251 MB, 3.9 TB/s, VALU 53% busy), 30011 x 2560 181 (4.3 TB/s), 12288 x 5120 packed
// columns of a wider tensor 161 (5.2 TB/s of what moves: rows that begin anywhere share lines).  Tiles of 128 rows
// and 64 channels: of half the rows 30% slower, workgroups of 384 or 512 threads 20% and more.
template <bool BF16, bool Z, int V, int R>
__global__ __launch_bounds__(kGatedThreads) void gated_scan_kernel(const GatedArgs p) {
  using S = GatedShape<V, R>;
  __shared__ TileRows<S::kRows> rows;
  __shared__ PartMaps<S::kParts> maps;
  __shared__ float entering[kGatedChannels], rate[kGatedChannels];
  __shared__ uint32_t ticket[2];
  const Turn tile = Turn::take<S::kRows>(p, ticket, false);
  const Channels<V> ch(tile.block, p.dim);
  const int lane = threadIdx.x % S::kLanes, part = threadIdx.x / S::kLanes, at0 = part * R;
  const int64_t tile0 = tile.row0, d = ch.of(lane);

  const float param = p.param[ch.of(threadIdx.x % kGatedChannels / V) + threadIdx.x % V];
  find_rows(rows, p, static_cast<uint32_t>(tile0), tile.end);
  __syncthreads();

  auto body = [&](auto edges) {
    constexpr bool EDGES = decltype(edges)::value;
    // (each variant loads for itself: rows loaded before the branch would stay in registers beside the other's)
    Run<BF16, V> x[R], ag[R], xg[R], z[R];
    load_rows<!EDGES>(ag, p.ag, p.sag, tile0, at0, d, tile.end);
    load_rows<!EDGES>(xg, p.xg, p.sxg, tile0, at0, d, tile.end);
    load_rows<!EDGES>(x, p.x, p.sx, tile0, at0, d, tile.end);
    float ab[V], xb[V];
    load_bias<V>(p.ab, d, ab);
    load_bias<V>(p.xb, d, xb);
    if (threadIdx.x < kGatedChannels) rate[threadIdx.x] = decay_rate(p.scale, param);
    __syncthreads();
    const PartRows<R> in(rows, at0);
    if constexpr (EDGES) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const bool off = !(in.live >> j & 1);
        no_row<BF16, V>(ag[j], off, true);
        no_row<BF16, V>(xg[j], off, false);
        no_row<BF16, V>(x[j], off, false);
      }
    }
    float a[R][V], b[R][V], A[V], B[V], kl[V], kp[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      B[v] = 0.0f;
      kl[v] = rate[lane * V + v] * kLog2e;
      kp[v] = rate[lane * V + v] * -2.0f;
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float r = sigmoid_f32(ag[j].get(v), ab[v]);
        a[j][v] = hw_exp2(kl[v] * r);
        b[j][v] = input_weight(kp[v] * r, a[j][v]) * (sigmoid_f32(xg[j].get(v), xb[v]) * x[j].get(v));
      }
    if constexpr (EDGES) {
      for (uint32_t bits = in.first; bits; bits &= bits - 1) {
        const int at = __builtin_ctz(bits);
        float h[V];
        initial_state<V>(p, rows.seq[at0 + at], d, h);
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) b[j][v] = j == at ? fmaf(a[j][v], h[v], b[j][v]) : b[j][v];
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) B[v] = EDGES && (in.first >> j & 1) ? b[j][v] : fmaf(a[j][v], B[v], b[j][v]);
    compose_decays(a, A);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      maps.a[part][lane * V + v] = A[v];
      maps.b[part][lane * V + v] = B[v];
    }
    // (not with the others: 12 registers fewer, and it arrives while the tile waits; 2% faster)
    if constexpr (Z) load_rows<!EDGES>(z, p.z, p.sz, tile0, at0, d, tile.end);
    if (EDGES && lane == 0) maps.own[part] = in.first != 0;
    __syncthreads();

    if (threadIdx.x < kGatedChannels) {
      const int c = threadIdx.x;
      const bool on = ch.has(c / V);
      // what comes before each part, as a map of what enters the tile
      float ta = 1.0f, tb = 0.0f;
      bool own = false;
#pragma unroll
      for (int i = 0; i < S::kParts; ++i) {
        const float pa = maps.a[i][c], pb = maps.b[i][c];
        maps.a[i][c] = ta;
        maps.b[i][c] = tb;
        const bool starts = EDGES && maps.own[i];
        own |= starts;
        ta = compose_decay(ta, pa);
        tb = starts ? pb : fmaf(pa, tb, pb);
      }
      float h = 0.0f;
      if (p.ticket) {
        const int64_t at = tile.turn * p.dim + ch.of(c / V) + c % V, step = -(tile.apart * p.dim);
        if (on && !own) publish_map(p.words + at, ta, tb);
        if (on && own) publish_end(p.words + at, tb);
        h = look_back<4>(p.words + at + step, step, tile.before, on && !(EDGES && (rows.first[0] & 1)));
        if (on && !own) publish_end(p.words + at, fmaf(ta, h, tb));
      }
      entering[c] = h;
    }
    __syncthreads();

    float h[V];
    bool before = false;  // a part before this one has a state of its own
    if constexpr (EDGES) {
#pragma unroll
      for (int i = 0; i < S::kParts; ++i) before |= i < part && maps.own[i];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = lane * V + v;
      h[v] = before ? maps.b[part][c] : fmaf(maps.a[part][c], entering[c], maps.b[part][c]);
    }
    if (!EDGES || ch.has(lane)) {
      constexpr int ES = BF16 ? 2 : 4;
      char* y = static_cast<char*>(p.y) + tile0 * p.sy * ES;
      const uint32_t off = (static_cast<uint32_t>(at0) * static_cast<uint32_t>(p.sy) + static_cast<uint32_t>(d)) * ES;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          h[v] = EDGES && (in.first >> j & 1) ? b[j][v] : fmaf(a[j][v], h[v], b[j][v]);
          if constexpr (EDGES) b[j][v] = h[v];
          if constexpr (Z) o[v] = h[v] * silu_f32(z[j].get(v));
          else o[v] = h[v];
        }
        Run<BF16, V, true> out;  // (non-temporal: 2% to 4% faster, forward and backward)
        out.set(o);
        if (!EDGES || (in.live >> j & 1)) out.store_bytes(y + j * p.sy * ES + off);
      }
      if constexpr (EDGES) {
        for (uint32_t bits = in.last; bits; bits &= bits - 1) {
          const int at = __builtin_ctz(bits);
          float e[V];
#pragma unroll
          for (int j = 0; j < R; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) e[v] = j == at || j == 0 ? b[j][v] : e[v];
          final_state<V>(p, rows.seq[at0 + at], d, e);
        }
      }
      static_assert(kGatedSave % R == 0, "inside a sequence a checkpoint is the state after a part");
      if (p.ckpt) {
        const int64_t from = tile0 + at0 - (p.each ? tile.end - p.seqlen : 0);
        const int at = EDGES ? kGatedSave - 1 - static_cast<int>(from % kGatedSave) : R - 1;
        const int64_t row = at < R ? checkpoint_after(p, tile, tile0 + at0 + at + 1) : -1;
        if (row >= 0) {
          if constexpr (EDGES) {
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
              for (int v = 0; v < V; ++v) h[v] = j == at ? b[j][v] : h[v];
          }
          Run<false, V> out;
          out.set(h);
          out.store(p.ckpt, row * p.dim + d);
        }
      }
    }
  };
  // most tiles lie inside a sequence: without the cases of the others they take half the instructions
  if (rows.inside() && ch.count == kGatedChannels) body(std::false_type{});
  else body(std::true_type{});
}

// Backward.  With g = dy silu(z) (+ dlast at a sequence's last row), from the last row on:
//   G_t = g_t + a_{t+1} G_{t+1},  E_t = G_t l a (h_{t-1} - u a / w)   (= l dL/dl)
//   da_gate = E (1 - r), dx = G w i, dx_gate = G w x i (1 - i), dz = dy h silu'(z), dh_0 = a_1 G_1
// E is 0 where w is (a = 1): l / w -> 0 as l -> 0, so the product has that limit though dw/dl has none.
// The states come from the checkpoint before the tile and the tile's own rows; a G is carried from tile
// to tile like the forward's state, tiles taken from the last one on.
// Bound like the forward: 8 x 2048 x 1536 bf16 take 104 us (453 MB, 4.4 TB/s, VALU 61% busy), 30011 x 2560 331 (4.2
// TB/s); with the arithmetic taken out the loads and stores alone took nine tenths of the time.

// Stores the sum over all rows of quantity k: E (da_param), da_gate (da_bias) or dx_gate (dx_bias).
__device__ __forceinline__ void store_sum(int k, int64_t d, float s, const float* param, float* dparam, float* dab, float* dxb) {
  if (k == 0) {
    // d softplus(v) / softplus(v): sigmoid(v) / softplus(v), 1 to fp32 below -17
    const float v = param[d];
    const float ratio = v < -17.0f ? 1.0f : 1.0f / (1.0f + expf(-v)) / (fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))));
    dparam[d] = s * ratio;
  } else if (float* out = k == 1 ? dab : dxb) {
    out[d] = s;
  }
}

// V channels of sequence s in a (batch, dim) tensor of states, zeros without one
template <int V>
__device__ __forceinline__ Run<false, V> batch_state(const void* states, int32_t s, int64_t dim, int64_t d) {
  Run<false, V> h;
#pragma unroll
  for (int v = 0; v < V; ++v) h.w[v] = 0u;
  if (states) h.load(states, s * dim + d);
  return h;
}

template <bool BF16, bool Z, int V, int R>
__global__ __launch_bounds__(kGatedThreads, 3) void gated_scan_bwd_kernel(const GatedArgs p) {
  using S = GatedShape<V, R>;
  static_assert(S::kRows == kGatedSave, "a tile begins behind a checkpoint");
  __shared__ TileRows<S::kRows> rows;
  __shared__ PartMaps<S::kParts> fwd;  // the states' maps
  __shared__ float back[S::kParts][kGatedChannels];
  __shared__ uint8_t ends[S::kParts];  // the part holds a sequence's last row
  __shared__ float rate[kGatedChannels];
  __shared__ float starts[S::kRows][kGatedChannels];  // where a sequence begins: its initial state, then that one's gradient
  __shared__ uint32_t ticket[2];
  const Turn tile = Turn::take<S::kRows>(p, ticket, true);
  const Channels<V> ch(tile.block, p.dim);
  const int lane = threadIdx.x % S::kLanes, part = threadIdx.x / S::kLanes, at0 = part * R, wave = threadIdx.x / 64;
  const int64_t tile0 = tile.row0, d = ch.of(lane);

  const float param = p.param[ch.of(threadIdx.x % kGatedChannels / V) + threadIdx.x % V];
  find_rows(rows, p, static_cast<uint32_t>(tile0), tile.end);
  float se[V], sa[V], sx[V];  // sums over the lane's rows
#pragma unroll
  for (int v = 0; v < V; ++v) se[v] = sa[v] = sx[v] = 0.0f;
  __syncthreads();
  auto body = [&](auto edges) {
    constexpr bool EDGES = decltype(edges)::value;
    Run<BF16, V> x[R], ag[R], xg[R], z[R], dy[R];
    load_rows<!EDGES>(ag, p.ag, p.dim, tile0, at0, d, tile.end);
    load_rows<!EDGES>(xg, p.xg, p.dim, tile0, at0, d, tile.end);
    load_rows<!EDGES>(x, p.x, p.dim, tile0, at0, d, tile.end);
    if constexpr (Z) load_rows<!EDGES>(z, p.z, p.dim, tile0, at0, d, tile.end);
    load_rows<!EDGES>(dy, p.dy, p.dim, tile0, at0, d, tile.end);
    float ab[V], xb[V], k[V];
    load_bias<V>(p.ab, d, ab);
    load_bias<V>(p.xb, d, xb);
    if (threadIdx.x < kGatedChannels) rate[threadIdx.x] = decay_rate(p.scale, param);
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) k[v] = rate[lane * V + v];
    const PartRows<R> in(rows, at0);
    if constexpr (EDGES) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const bool off = !(in.live >> j & 1);
        no_row<BF16, V>(ag[j], off, true);
        no_row<BF16, V>(xg[j], off, false);
        no_row<BF16, V>(x[j], off, false);
        if constexpr (Z) no_row<BF16, V>(z[j], off, false);
        no_row<BF16, V>(dy[j], off, false);
      }
    }
    float a[R][V], h[R][V], g[R][V], f[R][V], r[R][V], i[R][V], w[R][V];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        r[j][v] = sigmoid_f32(ag[j].get(v), ab[v]);
        i[j][v] = sigmoid_f32(xg[j].get(v), xb[v]);
        a[j][v] = hw_exp2(k[v] * kLog2e * r[j][v]);
        w[j][v] = input_weight(k[v] * -2.0f * r[j][v], a[j][v]);
        h[j][v] = w[j][v] * (i[j][v] * x[j].get(v));
        g[j][v] = dy[j].get(v);
        if constexpr (Z) {
          const float zv = z[j].get(v), o = sigmoid_f32(zv), od = g[j][v] * o;
          g[j][v] = od * zv;
          f[j][v] = fmaf(g[j][v], 1.0f - o, od);
          asm volatile("" : "+v"(f[j][v]));  // (worked out here, not where it is used: one register for three)
        }
      }
    if constexpr (EDGES) {
      for (uint32_t bits = in.first; bits; bits &= bits - 1) {
        const int at = __builtin_ctz(bits);
        const Run<false, V> h0 = batch_state<V>(p.in.data, rows.seq[at0 + at], p.dim, d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          starts[at0 + at][lane * V + v] = h0.get(v);
#pragma unroll
          for (int j = 0; j < R; ++j) h[j][v] = j == at ? fmaf(a[j][v], h0.get(v), h[j][v]) : h[j][v];
        }
      }
      if (p.dlast) {
        for (uint32_t bits = in.last; bits; bits &= bits - 1) {
          const int at = __builtin_ctz(bits);
          const Run<false, V> end = batch_state<V>(p.dlast, rows.seq[at0 + at], p.dim, d);
#pragma unroll
          for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < R; ++j) g[j][v] = j == at ? g[j][v] + end.get(v) : g[j][v];
        }
      }
    }
    float A[V], B[V], C[V];  // C: a G of the row that the part begins with
#pragma unroll
    for (int v = 0; v < V; ++v) B[v] = C[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) B[v] = EDGES && (in.first >> j & 1) ? h[j][v] : fmaf(a[j][v], B[v], h[j][v]);
    compose_decays(a, A);
#pragma unroll
    for (int j = R - 1; j >= 0; --j)
#pragma unroll
      for (int v = 0; v < V; ++v) C[v] = a[j][v] * (EDGES && (in.last >> j & 1) ? g[j][v] : g[j][v] + C[v]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      fwd.a[part][lane * V + v] = A[v];
      fwd.b[part][lane * V + v] = B[v];
      back[part][lane * V + v] = C[v];
    }
    if (EDGES && lane == 0) {
      fwd.own[part] = in.first != 0;
      ends[part] = in.last != 0;
    }
    __syncthreads();

    // The first wave runs the states through the parts, the second the adjoint.  (The parts' maps stay in the LDS:
    // in registers over the look-back they made the kernel spill, 8 x 2048 x 1536 in 126 us for 120.)
    if (wave < 2) {
      const int c = threadIdx.x & 63;
      const bool on = ch.has(c / V);
      const int64_t dc = ch.of(c / V) + c % V;
      if (wave == 0) {
        const int64_t saved = checkpoint_after(p, tile, tile0);
        float s = saved >= 0 ? p.ckpt[saved * p.dim + dc] : 0.0f;
#pragma unroll
        for (int q = 0; q < S::kParts; ++q) {
          const float pa = fwd.a[q][c], pb = fwd.b[q][c];
          fwd.b[q][c] = s;
          s = EDGES && fwd.own[q] ? pb : fmaf(pa, s, pb);
        }
      } else {
        float ta = 1.0f, tb = 0.0f;
        bool own = false;
#pragma unroll
        for (int q = S::kParts - 1; q >= 0; --q) {
          const bool stops = EDGES && ends[q];
          const float pa = fwd.a[q][c], pb = back[q][c];
          own |= stops;
          ta = compose_decay(ta, pa);
          tb = stops ? pb : fmaf(pa, tb, pb);
        }
        float s = 0.0f;
        if (p.ticket) {
          const int64_t at = tile.turn * p.dim + dc, step = -(tile.apart * p.dim);
          if (on && !own) publish_map(p.words + at, ta, tb);
          if (on && own) publish_end(p.words + at, tb);
          s = look_back<BF16 ? 3 : 2>(p.words + at + step, step, tile.before, on && !(EDGES && (rows.last[0] >> 63)));
          if (on && !own) publish_end(p.words + at, fmaf(ta, s, tb));
        }
#pragma unroll
        for (int q = S::kParts - 1; q >= 0; --q) {
          const float pa = fwd.a[q][c], pb = back[q][c];
          back[q][c] = s;
          s = EDGES && ends[q] ? pb : fmaf(pa, s, pb);
        }
      }
    }
    __syncthreads();

    // what the rest works out again rather than holds: the compiler would keep every common term in registers
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
      for (int q = 0; q < Run<BF16, V>::kWords; ++q) asm volatile("" : "+v"(x[j].w[q]));
#pragma unroll
      for (int v = 0; v < V; ++v) asm volatile("" : "+v"(r[j][v]), "+v"(i[j][v]));
    }
    if (!EDGES || ch.has(lane)) {
      float enter[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        enter[v] = fwd.b[part][lane * V + v];
        C[v] = back[part][lane * V + v];
      }
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float next = fmaf(a[j][v], j > 0 ? h[j > 0 ? j - 1 : 0][v] : enter[v], h[j][v]);
          h[j][v] = EDGES && (in.first >> j & 1) ? h[j][v] : next;
        }
#pragma unroll
      for (int j = R - 1; j >= 0; --j) {
        float prev[V], odx[V], oda[V], odg[V], odz[V];
        const bool on = !EDGES || (in.live >> j & 1);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          prev[v] = j > 0 ? h[j > 0 ? j - 1 : 0][v] : enter[v];
          if (EDGES && (in.first >> j & 1)) prev[v] = starts[at0 + j][lane * V + v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float G = EDGES && (in.last >> j & 1) ? g[j][v] : g[j][v] + C[v];
          const float xv = x[j].get(v), la = k[v] * r[j][v] * a[j][v];
          // l a^2 / w before x, whatever x is: at most w / 2, and 0 where l is (a w below 1e-19 has no normal l)
          const float q = la * a[j][v] * hw_rcp(fmaxf(w[j][v], 1e-19f));
          float E = G * fmaf(-i[j][v] * xv, q, la * prev[v]);
          odx[v] = G * w[j][v] * i[j][v];
          odg[v] = odx[v] * xv;
          odg[v] = fmaf(-odg[v], i[j][v], odg[v]);
          if (EDGES && !on) E = odg[v] = 0.0f;
          if constexpr (Z) odz[v] = f[j][v] * h[j][v];
          oda[v] = fmaf(-E, r[j][v], E);
          se[v] += E;
          sa[v] += oda[v];
          sx[v] += odg[v];
          C[v] = a[j][v] * G;
          if (EDGES && (in.first >> j & 1)) starts[at0 + j][lane * V + v] = C[v];
        }
        if (on) {
          constexpr int ES = BF16 ? 2 : 4;
          const uint32_t off = (static_cast<uint32_t>(at0) * static_cast<uint32_t>(p.dim) + static_cast<uint32_t>(d)) * ES;
          auto store = [&](void* base, const float(&val)[V]) {
            Run<BF16, V, true> out;
            out.set(val);
            out.store_bytes(static_cast<char*>(base) + (tile0 + j) * p.dim * ES + off);
          };
          store(p.dx, odx);
          store(p.dag, oda);
          store(p.dxg, odg);
          if constexpr (Z) store(p.dz, odz);
        }
      }
      if constexpr (EDGES) {
        if (p.dh0) {
          for (uint32_t bits = in.first; bits; bits &= bits - 1) {
            const int at = at0 + __builtin_ctz(bits);
            Run<false, V> out;
#pragma unroll
            for (int v = 0; v < V; ++v) out.w[v] = __builtin_bit_cast(uint32_t, starts[at][lane * V + v]);
            out.store(p.dh0, static_cast<int64_t>(rows.seq[at]) * p.dim + d);
          }
        }
      }
    }
  };
  if (rows.inside() && ch.count == kGatedChannels) body(std::false_type{});
  else body(std::true_type{});
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
    const int c = threadIdx.x & 63;
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < S::kParts; ++q) s += wave == 0 ? fwd.a[q][c] : wave == 1 ? fwd.b[q][c] : back[q][c];
    if (ch.has(c / V)) {
      const int64_t dc = ch.of(c / V) + c % V;
      if (p.tiles == 1) store_sum(wave, dc, s, p.param, p.dparam, p.dab, p.dxb);
      else p.partial[(static_cast<int64_t>(tile.turn) * 3 + wave) * p.dim + dc] = s;
    }
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
    store_sum(k, d, s, p.param, p.dparam, p.dab, p.dxb);
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

// V values from the skip-th on
template <bool BF16, int V>
__device__ __forceinline__ void store_from(void* base, int64_t idx, int skip, const float (&val)[V]) {
  Run<BF16, V> r;
  r.set(val);
  if (skip == 0) {
    r.store(base, idx);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v < skip) continue;
      if constexpr (BF16) static_cast<uint16_t*>(base)[idx + v] = static_cast<uint16_t>(r.w[v >> 1] >> (16 * (v & 1)));
      else static_cast<uint32_t*>(base)[idx + v] = r.w[v];
    }
  }
}

// One token on a cache: a thread owns V channels of R entries.  250 x 5120 on a bf16 cache take 9.6 us (launch, one
// round trip to the memory and 18 MB), less than the call on the host.
struct GatedStepArgs {
  GatedArgs g;      // rows are the batch's entries; in: the cache
  int64_t batch;
};

template <bool BF16, bool CB16, int V, int R>
__global__ __launch_bounds__(kGatedThreads) void gated_step_kernel(const GatedStepArgs q) {
  const GatedArgs& p = q.g;
  const int64_t natural = (static_cast<int64_t>(blockIdx.x) * kGatedThreads + threadIdx.x) * V;
  if (natural >= p.dim) return;
  // the last lane's channels begin further left where dim is no multiple of V; those that are its neighbour's
  // (the first `skip`) it does not store, since it may read their state after the neighbour has written it
  const int64_t d = natural < p.dim - V ? natural : p.dim - V;
  const int skip = static_cast<int>(natural - d);
  float ab[V], xb[V], rate[V];
  load_bias<V>(p.ab, d, ab);
  load_bias<V>(p.xb, d, xb);
#pragma unroll
  for (int v = 0; v < V; ++v) rate[v] = decay_rate(p.scale, p.param[d + v]);
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
      x[k].load(p.x, e[k] * p.sx + d);
      ag[k].load(p.ag, e[k] * p.sag + d);
      xg[k].load(p.xg, e[k] * p.sxg + d);
      z[k].load(zsrc, e[k] * zstride + d);
      st[k].load(p.in.data, (at[k] < 0 ? 0 : at[k]) + d);
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float h[V], y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float r = sigmoid_f32(ag[k].get(v), ab[v]), i = sigmoid_f32(xg[k].get(v), xb[v]);
        const float a = hw_exp2(rate[v] * kLog2e * r);
        h[v] = fmaf(a, st[k].get(v), input_weight(rate[v] * -2.0f * r, a) * (i * x[k].get(v)));
        y[v] = has_z ? h[v] * silu_f32(z[k].get(v)) : h[v];
      }
      if (at[k] < 0) continue;
      store_from<CB16, V>(p.in.data, at[k] + d, skip, h);
      store_from<BF16, V>(p.y, (b0 + k) * p.sy + d, skip, y);
    }
  }
}

}  // namespace ssm
