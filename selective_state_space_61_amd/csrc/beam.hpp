// beam.hpp -- beam search on cached states for gfx950: the selection over beams and vocabulary, and the
// reordering of the states that follows it.
//
// Selection.  A candidate (j, v) of a sequence has the value score_j + (logit[j, v] - lse_j) with lse_j =
// log sum_v exp(logit[j, v]); the `beams` largest are taken.  Two launches: a workgroup takes a stretch of
// one row into registers, sums exp(logit - a wave's largest) and keeps its largest `beams` logits; then a
// workgroup a sequence joins its rows' stretches, adds lse and score in 64 bits (they rank candidates of
// different rows) and ranks what is left.  Logits are read once.
//
// The largest k of a stretch: its values are taken for 64 columns, of which each lane of the four waves holds a
// quarter; the k-th largest of the columns' largest values is a bound that at least k values reach and few others
// do.  It is found bit by bit with a ballot each, what reaches it is gathered (by ballots again) and ranked by
// comparing all with all.
// Where more than 64 values reach it (rows of few different values) the k are found one after another.
#pragma once

#include "cache.hpp"

namespace ssm {

constexpr int kBeamThreads = 256;
constexpr int kBeamWaves = kBeamThreads / 64;
constexpr int kBeamValues = 32;  // of a row, a lane
constexpr int kBeamMost = 64;   // beams, and rows of a sequence

struct BeamArgs {
  const void* logits;
  int64_t sb, sr;           // elements between sequences and rows
  const float* scores;      // (batch, rows)
  const uint8_t* finished;  // (batch, rows) or NULL
  int32_t rows, beams, eos;
  int64_t vocab;
  int32_t chunks, blocks;   // stretches of a row, 16-byte blocks of a stretch
  uint64_t* best;           // (batch * rows, beams, chunks): key and token, a stretch's largest first
  float* stats;             // (batch * rows, chunks, waves, 2): largest logit, sum of exp(logit - it)
  int32_t *parents, *tokens;
  float* out_scores;
  uint8_t* out_finished;
};

// A value's key rises with it (-0 is 0); every key of a value is above 0.
__device__ __forceinline__ uint32_t beam_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float beam_logit(uint32_t key) {
  const uint32_t b = key ^ (static_cast<uint32_t>(static_cast<int32_t>(~key) >> 31) | 0x80000000u);
  return __builtin_bit_cast(float, b);
}
// Key and token in one word whose order is the candidates': equal keys by the lower token
__device__ __forceinline__ uint64_t beam_word(uint32_t key, uint32_t token) {
  return (static_cast<uint64_t>(key) << 32) | (0xffffffffu - token);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32);
  const uint32_t top = group_reduce<64>(hi, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
  const uint32_t lo = hi == top ? static_cast<uint32_t>(v) : 0u;
  return (static_cast<uint64_t>(top) << 32) | group_reduce<64>(lo, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// A bound that the keys of at least k lanes reach (k at most 64), near the k-th largest
__device__ __forceinline__ uint32_t kth_key(uint32_t key, int k) {
  const uint32_t hi = __builtin_amdgcn_readfirstlane(group_reduce<64>(key, [](uint32_t a, uint32_t b) { return a > b ? a : b; }));
  const uint32_t lo = __builtin_amdgcn_readfirstlane(group_reduce<64>(key, [](uint32_t a, uint32_t b) { return a < b ? a : b; }));
  if (hi == lo) return hi;
  int bit = 31 - __builtin_clz(hi ^ lo);
  uint32_t t = bit == 31 ? 0u : hi >> (bit + 1) << (bit + 1);
  for (; bit >= 12; --bit) {  // (11 bits of the mantissa: the few values more do not matter)
    const uint32_t c = t | (1u << bit);
    const int reach = __popcll(__ballot(key >= c));
    if (reach >= k) t = c;
    if (reach == k) break;
  }
  return t;
}

// Appends the words of the lanes in `on` to a wave's list of at most 64, `count` of which are there
__device__ __forceinline__ void append(uint64_t* list, int& count, uint64_t on, uint64_t word) {
  const int lane = threadIdx.x & 63;
  const int at = count + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(on >> 32),
                                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(on), 0));
  if ((on >> lane & 1) && at < 64) list[at] = word;
  count += __popcll(on);
}
// A wave's LDS writes before its reads
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Rank of a lane's word among those of the first n lanes (no two of which are equal)
__device__ __forceinline__ int rank_of(uint64_t w, int n) {
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const uint64_t o = (static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(w >> 32), i)) << 32) |
                       static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(w), i));
    rank += o > w;
  }
  return rank;
}

__device__ __forceinline__ bool is_finite(float v) { return __builtin_isfinite(v); }

// Neither the memory nor the VALU is busy (each near 60%): a workgroup loads, then ranks, and others fill in.  48 x 8
// rows of 50257 fp32 values take 16.8 us (4.6 TB/s), 20 x 16 of 131072 bf16 ones, a quarter finished, 20 (3.1 TB/s);
// seven waves a SIMD, three registers spilled, are 2% and 3% faster than six, eight 15% and 7% slower.  With half the
// values a lane, whose waves fit eight times, 0% and 16% slower.
template <bool BF16>
__global__ __launch_bounds__(kBeamThreads, 7) void beam_rows_kernel(const BeamArgs p) {
  constexpr int EPB = BF16 ? 8 : 4, IT = kBeamValues / EPB, ES = BF16 ? 2 : 4;
  __shared__ uint64_t lists[kBeamWaves][64];
  __shared__ float tops[kBeamWaves][64];
  __shared__ int32_t counts[kBeamWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t row = blockIdx.x / static_cast<uint32_t>(p.chunks), chunk = blockIdx.x - row * static_cast<uint32_t>(p.chunks);
  // what a finished or dead row holds does not matter
  if (!is_finite(p.scores[row]) || (p.finished && p.finished[row])) return;
  const uint32_t seq = row / static_cast<uint32_t>(p.rows);
  const char* base = static_cast<const char*>(p.logits) + (seq * p.sb + (row - seq * static_cast<uint32_t>(p.rows)) * p.sr) * ES;
  // Blocks of 16 bytes by token, at whatever alignment the row has (gfx950 takes wide loads at any), so that
  // rows of the same values have the same sums, and tie.
  const uint32_t token0 = chunk * static_cast<uint32_t>(p.blocks) * EPB;  // of the stretch
  const uint32_t vocab = static_cast<uint32_t>(p.vocab);
  // its values: of a vocabulary of very many stretches the last ones may have none
  const uint32_t rest = vocab > token0 ? vocab - token0 : 0u, most = static_cast<uint32_t>(p.blocks) * EPB;
  const uint32_t left = rest < most ? rest : most;
  base += static_cast<int64_t>(token0) * ES;
  uint32_t raw[IT][4];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const uint32_t first = (i * kBeamThreads + threadIdx.x) * EPB;
    raw[i][0] = raw[i][1] = raw[i][2] = raw[i][3] = BF16 ? 0xff80ff80u : 0xff800000u;  // -inf
    if (first + EPB <= left) {
      const U32x4 v = *reinterpret_cast<const typename Words<ES>::U4*>(base + first * ES);
      raw[i][0] = v.x; raw[i][1] = v.y; raw[i][2] = v.z; raw[i][3] = v.w;
    } else if (first < left) {
#pragma unroll
      for (int e = 0; e < EPB; ++e) {
        if (first + e >= left) continue;
        if constexpr (BF16) {
          const uint32_t h = reinterpret_cast<const uint16_t*>(base)[first + e];
          raw[i][e >> 1] = e & 1 ? (raw[i][e >> 1] & 0xffffu) | h << 16 : (raw[i][e >> 1] & 0xffff0000u) | h;
        } else {
          raw[i][e] = reinterpret_cast<const uint32_t*>(base)[first + e];
        }
      }
    }
  }
  auto value = [&](int i, int e) {
    if constexpr (BF16) return e & 1 ? bf16_hi(raw[i][e >> 1]) : bf16_lo(raw[i][e >> 1]);
    else return __builtin_bit_cast(float, raw[i][e]);
  };
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < EPB; ++e) top = fmaxf(top, value(i, e));
  const int k = p.beams;
  tops[wave][lane] = top;
  const float m = group_reduce<64>(top, [](float a, float b) { return fmaxf(a, b); });
  const float shift = m == -INFINITY ? 0.0f : m;  // (NaN and +inf leave a NaN in the sum)
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < EPB; ++e)
      s += hw_exp2((value(i, e) - shift) * kLog2e);  // (fused, a large shift's rounding would scale them all)
  s = group_sum<64>(s);
  if (lane == 0) {
    float* st = p.stats + 2 * (static_cast<int64_t>(blockIdx.x) * kBeamWaves + wave);
    st[0] = m;
    st[1] = s;
  }
  __syncthreads();

  top = tops[0][lane];
#pragma unroll
  for (int i = 1; i < kBeamWaves; ++i) top = fmaxf(top, tops[i][lane]);
  // (the first wave has the first blocks: its lanes without a value are those of columns without one)
  const uint32_t reach = kth_key(lane * EPB < left ? beam_key(top) : 0u, k);
  const float bound = reach >= 0x00800000u ? beam_logit(reach) : -INFINITY;  // (keys below are those of -inf and of no value)
  int count = 0;
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < EPB; ++e) {
      const uint32_t at = (i * kBeamThreads + threadIdx.x) * EPB + e;
      const uint64_t on = __ballot(value(i, e) >= bound);
      if (on) append(lists[wave], count, on & __ballot(at < left), beam_word(beam_key(value(i, e)), token0 + at));
    }
  if (lane == 0) counts[wave] = count;
  __syncthreads();

  uint64_t* out = p.best + static_cast<int64_t>(row) * k * p.chunks + chunk;
  int all = 0, before[kBeamWaves];
#pragma unroll
  for (int i = 0; i < kBeamWaves; ++i) {
    before[i] = all;
    all += counts[i];
  }
  all = __builtin_amdgcn_readfirstlane(all);
  if (all <= 64) {
    if (wave > 0) return;
    uint64_t w = 0u;
#pragma unroll
    for (int i = 0; i < kBeamWaves; ++i)
      if (lane >= before[i] && lane < before[i] + counts[i]) w = lists[i][lane - before[i]];
    const int rank = rank_of(w, all);
    if (lane < all && rank < k) out[rank * p.chunks] = w;
    if (lane >= all && lane < k) out[lane * p.chunks] = 0u;  // fewer values than beams
    return;
  }
  // each wave's largest one after another, then those of all four
  uint64_t last = ~0ull;
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0u;
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int e = 0; e < EPB; ++e) {
        const uint32_t at = (i * kBeamThreads + threadIdx.x) * EPB + e;
        const uint64_t w = beam_word(beam_key(value(i, e)), token0 + at);
        if (at < left && w < last && w > best) best = w;
      }
    last = wave_max(best);
    if (lane == 0) lists[wave][r] = last;
    if (last == 0u) last = 1u;  // none left: the rest is 0 too
  }
  __syncthreads();
  if (wave > 0) return;
  uint64_t words[kBeamWaves];
#pragma unroll
  for (int i = 0; i < kBeamWaves; ++i) words[i] = lane < k ? lists[i][lane] : 0u;
  last = ~0ull;
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0u;
#pragma unroll
    for (int i = 0; i < kBeamWaves; ++i)
      if (words[i] < last && words[i] > best) best = words[i];
    last = wave_max(best);
    if (lane == 0) out[r * p.chunks] = last;
    if (last == 0u) last = 1u;
  }
}

// One sequence a workgroup: a wave joins a row's stretches, then all rank the rows' candidates.
__global__ __launch_bounds__(1024) static void beam_join_kernel(const BeamArgs p) {
  __shared__ double values[kBeamMost * kBeamMost];  // of row j from j << shift on
  __shared__ int32_t tokens[kBeamMost * kBeamMost];
  __shared__ union {
    uint64_t lists[16][64];                // of the waves, while they join rows
    int32_t ranks[kBeamMost * kBeamMost];  // after that
  } room;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int k = static_cast<int>(p.vocab < p.beams ? p.vocab : p.beams);  // candidates of a row
  const int shift = k > 1 ? 32 - __builtin_clz(k - 1) : 0;
  const int64_t seq = blockIdx.x;
  for (int j = wave; j < p.rows; j += waves) {
    const int64_t row = seq * p.rows + j;
    const uint64_t* best = p.best + row * p.beams * p.chunks;
    const float* st = p.stats + 2 * row * p.chunks * kBeamWaves;
    const int sums = p.chunks * kBeamWaves;
    // The words by rank (all stretches' largest, then all second ones): the first 256, before it is known whether
    // the row counts.
    const int64_t n = static_cast<int64_t>(p.chunks) * k;
    constexpr int kAhead = 4;
    uint64_t word[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) word[i] = i * 64 + lane < n ? best[i * 64 + lane] : 0u;
    float m = -INFINITY, m0 = -INFINITY, s0 = 0.0f;
    if (lane < sums) m0 = st[2 * lane], s0 = st[2 * lane + 1];
    const float score = p.scores[row];
    const bool done = p.finished && p.finished[row];
    double lse = 0.0;
    bool dead = !is_finite(score);
    uint64_t* list = room.lists[wave];
    if (!dead && !done) {
      m = m0;
      for (int c = lane + 64; c < sums; c += 64) m = fmaxf(m, st[2 * c]);
      m = group_reduce<64>(m, [](float a, float b) { return fmaxf(a, b); });
      auto share = [&](float mc, float sc) { return sc * static_cast<double>(mc == m ? 1.0f : hw_exp2((mc - m) * kLog2e)); };
      double s = share(m0, s0);
      for (int c = lane + 64; c < sums; c += 64) s += share(st[2 * c], st[2 * c + 1]);
      for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
      lse = m + log(s);
      dead = !is_finite(m) || !(s > 0.0) || !__builtin_isfinite(lse);
    }
    if (dead || done) {
      // tokens in their order, all of no value but the end of a finished beam
      if (lane < k) {
        int t = lane;
        double v = -INFINITY;
        if (!dead) {
          t = lane == 0 ? p.eos : (lane <= p.eos ? lane - 1 : lane);
          if (lane == 0) v = score;
        }
        values[(j << shift) + lane] = v;
        tokens[(j << shift) + lane] = t;
      }
      continue;
    }
    uint64_t top = word[0];
#pragma unroll
    for (int i = 1; i < kAhead; ++i) top = word[i] > top ? word[i] : top;
    const uint32_t bound = kth_key(static_cast<uint32_t>(top >> 32), k);
    int count = 0, quiet = 0;  // words since the last that reaches the bound: a whole rank of them, and none follows
    for (int64_t i0 = 0; i0 < n && quiet < p.chunks; i0 += 64 * kAhead) {
      if (i0 > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) word[i] = i0 + i * 64 + lane < n ? best[i0 + i * 64 + lane] : 0u;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const uint64_t on = __ballot(word[i] != 0u && static_cast<uint32_t>(word[i] >> 32) >= bound);
        quiet = on ? 0 : quiet + 64;
        if (on) append(list, count, on, word[i]);
      }
    }
    uint64_t mine = 0u;  // the lane-th largest
    if (count <= 64) {
      wave_sync();
      const uint64_t w = lane < count ? list[lane] : 0u;
      const int rank = rank_of(w, count);
      wave_sync();
      if (lane < count) list[rank] = w;
      wave_sync();
      mine = lane < k ? list[lane] : 0u;
    } else {
      uint64_t last = ~0ull;
      for (int r = 0; r < k; ++r) {
        uint64_t b = 0u;
        for (int64_t i = lane; i < n; i += 64) {
          const uint64_t w = best[i];
          if (w < last && w > b) b = w;
        }
        last = wave_max(b);
        if (lane == r) mine = last;
      }
    }
    const double v = score + (static_cast<double>(beam_logit(static_cast<uint32_t>(mine >> 32))) - lse);
    const int32_t t = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(mine));
    int rank = lane;
    // by value now: logits that differ may give one value, which then goes by the token
    const double up = __shfl_up(v, 1);  // (by all lanes: one that is switched off gives its neighbour a 0)
    const bool tie = lane > 0 && lane < k && up == v;
    if (__any(tie)) {
      rank = 0;
      for (int i = 0; i < k; ++i) {
        const double o = __shfl(v, i);
        const int32_t u = __shfl(t, i);
        rank += o > v || (o == v && u < t);
      }
    }
    if (lane < k) {
      values[(j << shift) + rank] = v;
      tokens[(j << shift) + rank] = t;
    }
  }
  const int items = p.rows << shift;
  int32_t* ranks = room.ranks;
  __syncthreads();
  for (int i = threadIdx.x; i < items; i += blockDim.x) ranks[i] = i & ((1 << shift) - 1);  // its place in its own row
  __syncthreads();
  // how many of each other row come before each candidate: a row a wave, a candidate a lane
  for (int o = wave; o < p.rows; o += waves)
    for (int i = lane; i < items; i += 64) {
      const int j = i >> shift;
      if (j == o || (i & ((1 << shift) - 1)) >= k) continue;
      const double v = values[i];
      int lo = 0, hi = k;  // the first that does not come before (rows above win ties)
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const double w = values[(o << shift) + mid];
        if (w > v || (w == v && o < j)) lo = mid + 1;
        else hi = mid;
      }
      if (lo) atomicAdd(&ranks[i], lo);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < items; i += blockDim.x) {
    if ((i & ((1 << shift) - 1)) >= k || ranks[i] >= p.beams) continue;
    const int j = i >> shift;
    const int64_t at = seq * p.beams + ranks[i];
    p.parents[at] = j;
    p.tokens[at] = tokens[i];
    p.out_scores[at] = static_cast<float>(values[i]);
    if (p.out_finished) p.out_finished[at] = p.finished[seq * p.rows + j] || tokens[i] == p.eos;
  }
}

// Reordering.  Beam i of a sequence takes the entry of beam parents[i].  A thread owns 16 bytes (or 8) of the
// entry in every beam's slot: it reads what moves, then writes it, so that the order of beams does not
// matter and no copy of the cache is needed.  Bound by the memory: 128 slots of 2.6 MB (16 sequences of 8 beams, parents
// drawn) take 101 us, 4.8 TB/s; with one 16-byte column a thread 109, with four 102, with plain stores 5% more.
constexpr int kReorderCaches = 32;
struct ReorderCache {
  char* data;
  int64_t slots, stride, bytes;  // bytes between slots, bytes of an entry
  int64_t block0;                // the cache's first workgroup
};
struct ReorderArgs {
  ReorderCache c[kReorderCaches];
  const int32_t *slots, *parents;
  int64_t batch;
  int32_t beams, caches;
};

// COLUMNS of WORDS 32-bit words a thread, of BEAMS beams at most.  (64 beams of 16 bytes a thread spill: 4 sequences
// of 64 beams of 2.4 MB take 1507 us, of 8 bytes 401.)
template <int BEAMS, int COLUMNS, int WORDS>
__global__ __launch_bounds__(kBeamThreads) void reorder_kernel(const ReorderArgs p) {
  constexpr int BYTES = 4 * WORDS;
  using U = std::conditional_t<WORDS == 4, U32x4, U32x2>;
  int k = 0;
  while (k + 1 < p.caches && static_cast<int64_t>(blockIdx.x) >= p.c[k + 1].block0) ++k;
  const ReorderCache& c = p.c[k];
  const int64_t at = ((static_cast<int64_t>(blockIdx.x) - c.block0) * COLUMNS * kBeamThreads + threadIdx.x) * BYTES;
  for (int64_t b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const int32_t* parents = p.parents + b * p.beams;
    auto slot_of = [&](int i) -> int64_t { return p.slots ? p.slots[b * p.beams + i] : b * p.beams + i; };
    U v[BEAMS][COLUMNS];
    uint64_t moves = 0;
#pragma unroll
    for (int i = 0; i < BEAMS; ++i) {
      if (i >= p.beams) continue;
      const int from = parents[i];
      if (from < 0 || from >= p.beams || from == i) continue;
      const int64_t dst = slot_of(i), src = slot_of(from);
      if (dst < 0 || dst >= c.slots || src < 0 || src >= c.slots || dst == src) continue;
      moves |= 1ull << i;
#pragma unroll
      for (int j = 0; j < COLUMNS; ++j) {
        const int64_t first = at + j * kBeamThreads * BYTES, left = c.bytes - first;
        const char* q = c.data + src * c.stride + first;
        if (left >= BYTES) {
          if constexpr (WORDS == 4) v[i][j] = *reinterpret_cast<const Words<1>::U4*>(q);
          else v[i][j] = *reinterpret_cast<const Words<1>::U2*>(q);
        } else if (left > 0) {
          uint32_t w[WORDS] = {};
#pragma unroll
          for (int e = 0; e < BYTES; ++e)
            if (e < left) w[e >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(q[e])) << (8 * (e & 3));
#pragma unroll
          for (int e = 0; e < WORDS; ++e) v[i][j][e] = w[e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < BEAMS; ++i) {
      if (!(moves >> i & 1)) continue;
#pragma unroll
      for (int j = 0; j < COLUMNS; ++j) {
        const int64_t first = at + j * kBeamThreads * BYTES, left = c.bytes - first;
        char* q = c.data + slot_of(i) * c.stride + first;
        if (left >= BYTES) {
          if constexpr (WORDS == 4) __builtin_nontemporal_store(v[i][j], reinterpret_cast<Words<1>::U4*>(q));
          else __builtin_nontemporal_store(v[i][j], reinterpret_cast<Words<1>::U2*>(q));
        } else if (left > 0) {
#pragma unroll
          for (int e = 0; e < BYTES; ++e)
            if (e < left) q[e] = static_cast<char>(v[i][j][e >> 2] >> (8 * (e & 3)));
        }
      }
    }
  }
}

}  // namespace ssm
