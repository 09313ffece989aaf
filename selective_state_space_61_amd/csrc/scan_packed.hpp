// scan_packed.hpp -- the selective scan over packed prompts, for gfx950.
//
// The recurrence is scan_fwd.hpp's ("Mamba 论文精读" sec. 2.2 and sec. 3.3; "mamba->jamba" sec. 2.3)
// for every sequence by itself, from its slot's state or from zeros.
//
// Work decomposition.  A wave takes 16 channels of one piece of one sequence, and everything that
// they need, by itself: lane 16 r + k is channel k with states NPL r .. NPL r + NPL - 1 in registers
// (as in scan_rows.hpp; the states of dstate 1 and 2 are padded to 4 with A = B = C = 0).  Per chunk
// of 16 rows:
//   * the lanes load x, delta and z as (row lane / 4, four channels), one chunk ahead, and write
//     (dt, dt x) and (D x, silu z) to a part of the LDS that is the wave's own;
//   * lane k of row r loads step k's B and C of its NPL states: each step takes them through DPP
//     row broadcasts, so they need no LDS (but B goes there where the matrix cores take it, dstate 16);
//   * 16 steps of step_readout (ssm_device.hpp), or of decay_readout4 with the input terms from the
//     matrix cores;
//   * the read-outs of four steps, each spread over the four rows of lanes, are added with two
//     lane swaps and two adds a pair (v_permlane16_swap, v_permlane32_swap), which leaves step
//     t + r's sum in row r: skip term, gate and rounding then run once per value, not per state
//     group.  Rows of y go out as the rows of x came in.
// There are no barriers.  A sequence's channels are many small independent waves, several per
// SIMD, which cover each other's latencies and fill whatever CUs are free: with ragged prompts that
// balances better than workgroups that own a CU.  What bounds it is VALU issue: 399 VALU instructions
// per chunk, of them 80 transcendental ones, keep a SIMD with three waves busy for 82% of its cycles, and
// the matrix cores for 5%.  bf16, dstate 16: 32 prompts of 2048 x 1536 377 us (the dense scan's workgroups,
// one per CU: 490), 11 ragged ones of 11003 x 1536 117 us launched back to back, 119 to 126 from Python
// (workgroups of scan_rows.hpp's kind, in pieces or not: 176), one of 8192 x 1536 93 us (123).  Eight equal prompts of 2048 x 1536 fill the SIMDs with
// fewer than one wave each and take 172 us (in pieces 160), where the dense scan's wave specialisation
// takes 122: equal lengths are its case.
//
// Pieces.  Few long prompts have too few waves, so sequences are cut into pieces of `piece` rows: a
// first launch (AGG) runs every piece but a sequence's last one without read-outs and leaves its end
// state and its summed step, a second launch runs every piece from its entering state, which it
// composes from the states left by the pieces before it with (a1, h1) o (a2, h2) = (a1 a2, a2 h1 + h2),
// a = exp(A sum dt).  Which piece a wave has follows from cu_seqlens alone (it sums the piece counts
// of 64 sequences at a time), so the host needs no lengths and the launch can be captured.
//
// In-place states.  A sequence of one piece reads and writes its slot in the same wave.  With
// several pieces the slot is read by AGG's first piece only (which also leaves a copy of what it
// read for the second launch's first piece, in the last piece's unused place) and written by
// the second launch's last piece only.
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
  float* seg_state;  // (pieces, dim, N): a piece's end state (see above)
  float* seg_dsum;   // (pieces, dim): its summed step
  int64_t total;
  int64_t nseq;
  int64_t dim;
  int64_t sx, sdelta, sB, sC, sz, sy;
  int64_t pieces;      // bound on the pieces of all sequences: rows of seg_state
  int32_t piece;       // rows per piece, 0: whole sequences
  int32_t ncb;         // channel blocks of 64
  int32_t cache_bf16;
  int32_t softplus;
};

constexpr int64_t kScanPackedMaxStride = 1 << 24;  // elements between rows: a chunk's offsets fit 32 bits

// Piece g of all sequences: its sequence, which of the sequence's pieces it is, and its rows.
struct Piece {
  int64_t s;          // -1: no such piece
  int64_t k, count;   // the k-th of `count` pieces
  int64_t r0, r1;
};

__device__ __forceinline__ Piece find_piece(const ScanPackedArgs& p, int64_t g) {
  const int lane = threadIdx.x & 63;
  Piece q;
  q.s = -1;
  q.k = q.count = q.r0 = q.r1 = 0;
  auto rows = [&](int64_t s, int64_t* a, int64_t* b) {
    const int64_t c0 = p.cu[s], c1 = p.cu[s + 1];
    *a = c0 < 0 ? 0 : c0;
    *b = c1 > p.total ? p.total : c1;
  };
  if (p.piece == 0) {
    rows(g, &q.r0, &q.r1);
    if (q.r0 >= q.r1) return q;
    q.s = g;
    q.count = 1;
    return q;
  }
  int64_t base = 0;
  for (int64_t i = 0; i < p.nseq; i += 64) {
    int64_t a = 0, b = 0;
    if (i + lane < p.nseq) rows(i + lane, &a, &b);
    // lengths and piece lengths are below 2^31, counts of 64 sequences need more only for cu that falls
    const int64_t own = b > a ? (static_cast<uint32_t>(b - a) - 1u) / static_cast<uint32_t>(p.piece) + 1 : 0;
    int64_t upto = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t o = __shfl_up(upto, off, 64);
      upto += lane >= off ? o : 0;
    }
    const uint64_t past = __ballot(base + upto > g);
    if (past) {
      const int at = __ffsll(static_cast<unsigned long long>(past)) - 1;
      q.s = i + at;
      q.count = __shfl(own, at, 64);
      q.k = g - (base + __shfl(upto, at, 64) - q.count);
      const int64_t ra = __shfl(a, at, 64), rb = __shfl(b, at, 64);
      q.r0 = ra + q.k * p.piece;
      q.r1 = q.r0 + p.piece < rb ? q.r0 + p.piece : rb;
      return q;
    }
    base += __shfl(upto, 63, 64);
  }
  return q;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// One step without a read-out
template <int NPL, int K>
__device__ __forceinline__ void step_state(float dt, float w, const float* a2, const float* b, float* h) {
#pragma unroll
  for (int j = 0; j < NPL; ++j) h[j] = fmaf(hw_exp2(dt * a2[j]), h[j], row_bcast<K>(b[j]) * w);
}

// What a step needs besides its input term: its decays e[j] = exp2(dt a2[j]) and, while h is still the
// state before it, the read-out of the step before, sum_j C[j] h[j].  The order obeys step_readout's rules
// (ssm_device.hpp): each multiply-accumulate reads its accumulator three instructions after the last one,
// with decays in between.
template <int KC>
__device__ __forceinline__ float decay_readout4(float dt, const float* a2, const float* c, const float* h, float (&e)[4]) {
  float yp;
  asm("v_mul_f32 %[e0], %[dt], %[a0]\n\t"
      "v_mul_f32 %[e1], %[dt], %[a1]\n\t"
      "v_mul_f32_dpp %[yp], %[c0], %[h0] row_newbcast:%[kc] row_mask:0xf bank_mask:0xf\n\t"
      "v_exp_f32 %[e0], %[e0]\n\t"
      "v_exp_f32 %[e1], %[e1]\n\t"
      "v_fmac_f32_dpp %[yp], %[c1], %[h1] row_newbcast:%[kc] row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32 %[e2], %[dt], %[a2]\n\t"
      "v_mul_f32 %[e3], %[dt], %[a3]\n\t"
      "v_fmac_f32_dpp %[yp], %[c2], %[h2] row_newbcast:%[kc] row_mask:0xf bank_mask:0xf\n\t"
      "v_exp_f32 %[e2], %[e2]\n\t"
      "v_exp_f32 %[e3], %[e3]\n\t"
      "v_fmac_f32_dpp %[yp], %[c3], %[h3] row_newbcast:%[kc] row_mask:0xf bank_mask:0xf"
      : [e0] "=&v"(e[0]), [e1] "=&v"(e[1]), [e2] "=&v"(e[2]), [e3] "=&v"(e[3]), [yp] "=&v"(yp)
      : [dt] "v"(dt), [a0] "v"(a2[0]), [a1] "v"(a2[1]), [a2] "v"(a2[2]), [a3] "v"(a2[3]), [c0] "v"(c[0]),
        [c1] "v"(c[1]), [c2] "v"(c[2]), [c3] "v"(c[3]), [h0] "v"(h[0]), [h1] "v"(h[1]), [h2] "v"(h[2]), [h3] "v"(h[3]),
        [kc] "i"(KC));
  return yp;
}

// Orders a wave's LDS writes before its other lanes' reads (LDS serves a wave in order: this only
// keeps the compiler from moving them)
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Sums over the four 16-lane rows of four registers: row r of the result holds the sum of v[r].
// v_permlane16_swap exchanges the odd rows of its first operand with the even rows of its second,
// v_permlane32_swap the upper half with the lower half.  A lane swap may not follow a VALU write of
// its operand within two instructions, which the compiler cannot see where an asm block wrote v[3].
__device__ __forceinline__ float sum_rows4(const float (&v)[4]) {
  auto bits = [](float f) { return __builtin_bit_cast(uint32_t, f); };
  auto pair = [](auto q) {
    const uint32_t lo = q[0], hi = q[1];
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
  };
  float v3 = v[3];
  asm("s_nop 1" : "+v"(v3));
  const float a = pair(__builtin_amdgcn_permlane16_swap(bits(v[0]), bits(v[1]), false, false));
  const float b = pair(__builtin_amdgcn_permlane16_swap(bits(v[2]), bits(v3), false, false));
  return pair(__builtin_amdgcn_permlane32_swap(bits(a), bits(b), false, false));
}

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// Waves (of 16 channels) per workgroup: one for each SIMD of its CU, so that the SIMDs stay even.  32
// prompts of 2048 x 1536 with 1 | 2 | 4 | 8: 466 | 487 | 375 | 474 us, 11 ragged ones of 11003 rows
// 143 | 124 | 116 | 127.
constexpr int kPackedWaves = 4;
constexpr int kPackedChunk = 16;  // rows per chunk: lanes of a DPP row
constexpr int packed_states(int N) { return N < 4 ? 4 : N; }

template <bool BF16, int N, bool AGG>
__global__ __launch_bounds__(64 * kPackedWaves, packed_states(N) <= 16 ? 4 : 2) void scan_packed_kernel(const ScanPackedArgs p) {
  constexpr int NPL = packed_states(N) / 4, CH = kPackedChunk, ES = BF16 ? 2 : 4, V = 4;
  constexpr bool kOuter = N == 16;  // B (dt x) by the matrix cores
  constexpr int BS = CH + 4;  // floats between states of s_b: 64 lanes read 16 states of 4 rows from 64 banks
  // dt and dt x: [row][channel] float2, or (kOuter) all of dt before all of dt x
  __shared__ float4 s_dw_[kPackedWaves][CH * 8];
  __shared__ float4 s_xg_[kPackedWaves][AGG ? 1 : CH * 8];               // (D x, silu z)
  __shared__ float4 s_y_[kPackedWaves][AGG ? 1 : CH * 4];                // y: [row][channel]
  __shared__ float4 s_b_[kPackedWaves][kOuter ? N * BS / 4 : 1];         // B: [state][row]

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float2* const s_dw = reinterpret_cast<float2*>(s_dw_[wave]);
  [[maybe_unused]] float* const s_dt = reinterpret_cast<float*>(s_dw_[wave]);
  [[maybe_unused]] float* const s_w = s_dt + CH * 16;
  float2* const s_xg = reinterpret_cast<float2*>(s_xg_[wave]);
  float* const s_y = reinterpret_cast<float*>(s_y_[wave]);
  [[maybe_unused]] float* const s_b = reinterpret_cast<float*>(s_b_[wave]);

  const int64_t c0 = (static_cast<int64_t>(blockIdx.x % p.ncb) * kPackedWaves + wave) * 16;
  const int64_t g = blockIdx.x / p.ncb;
  if (c0 >= p.dim) return;
  const Piece pc = find_piece(p, g);
  const int64_t seq = uniform64(pc.s), kth = uniform64(pc.k), npieces = uniform64(pc.count);
  const int64_t row_base = uniform64(pc.r0);
  const int64_t rows = uniform64(pc.r1) - row_base;
  if (seq < 0 || rows <= 0) return;
  if (AGG && kth + 1 == npieces) return;
  const int nchunks = static_cast<int>((rows + CH - 1) / CH);
  const int last_row = static_cast<int>(rows - 1 - static_cast<int64_t>(nchunks - 1) * CH);  // of the last chunk

  // the lane's channel and states in the recurrence
  const int r = lane >> 4, k = lane & 15;
  const int n0 = NPL * r;
  const bool lane_ok = c0 + k < p.dim;
  const int64_t d = lane_ok ? c0 + k : p.dim - 1;  // a channel past dim computes the last one's states
  float A2[NPL], h[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    // finite below, so that steps past the piece (dt = 0) keep the state
    const float a = n0 + j < N ? p.A[d * N + n0 + j] * kLog2e : 0.0f;
    A2[j] = a < -3.0e38f ? -3.0e38f : a;
    h[j] = 0.0f;
  }

  // ---- the state entering the piece ---------------------------------------------------------------
  const int64_t at = p.cache.data ? uniform64(cache_offset(p.cache, p.slots, seq)) : -1;
  const bool from_slot = at >= 0 && p.has_initial && p.has_initial[seq] && kth == 0 && (AGG || npieces == 1);
  auto cache_index = [&](int j) { return at + d * N + n0 + j; };
  if (from_slot) {
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (n0 + j < N)
        h[j] = p.cache_bf16 ? load_one<true>(p.cache.data, cache_index(j)) : load_one<false>(p.cache.data, cache_index(j));
  }
  const int64_t spare = g - kth + npieces - 1;  // the last piece's place
  if constexpr (AGG) {
    if (kth == 0 && spare < p.pieces && lane_ok) {
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (n0 + j < N) p.seg_state[(spare * p.dim + d) * N + n0 + j] = h[j];
    }
  } else if (npieces > 1) {
    const int64_t first = g - kth;
    auto left = [&](int64_t i, int j) { return n0 + j < N ? p.seg_state[(i * p.dim + d) * N + n0 + j] : 0.0f; };
    if (kth == 0) {
      if (spare < p.pieces) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) h[j] = left(spare, j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NPL; ++j) h[j] = left(first, j);
      // states of the pieces between, kAhead of them in flight
      constexpr int kAhead = NPL <= 4 ? 8 : 2;
      for (int64_t i = 1; i < kth; i += kAhead) {
        float e[kAhead][NPL], ds[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int64_t w = first + (i + u < kth ? i + u : kth - 1);
          ds[u] = p.seg_dsum[w * p.dim + d];
#pragma unroll
          for (int j = 0; j < NPL; ++j) e[u][j] = left(w, j);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (i + u >= kth) break;
#pragma unroll
          for (int j = 0; j < NPL; ++j) {
            // a whole piece's decay is often 0 in fp32, which no step's is: an infinite state stays one
            const float a = hw_exp2(ds[u] * A2[j]), next = fmaf(a, h[j], e[u][j]);
            h[j] = a == 0.0f && fabsf(h[j]) == INFINITY ? h[j] + e[u][j] : next;
          }
        }
      }
    }
  }

  // ---- the rows -----------------------------------------------------------------------------------
  // Row addresses: a scalar base per tensor that moves on by a chunk (it stays at the last one) and
  // a 32-bit byte offset per lane that is the same in every chunk; in the last chunk rows past the
  // piece take its last row's.  (The host keeps strides below 2^24 elements: the offsets fit.)
  auto first_row = [&](const void* t, int64_t stride) { return static_cast<const char*>(t) + row_base * stride * ES; };
  auto offset = [&](int row, int64_t stride, int64_t col) {
    return static_cast<uint32_t>(row) * static_cast<uint32_t>(stride * ES) + static_cast<uint32_t>(col * ES);
  };
  const int lrow = lane >> 2, lcol = (lane & 3) * V;  // the row and channels that this lane loads
  const bool has_z = !AGG && p.z != nullptr, has_d = !AGG && p.Dskip != nullptr;
  const void* zsrc = has_z ? p.z : p.x;  // without a gate z is read from x and never used
  const int64_t zstride = has_z ? p.sz : p.sx;

  // kWhole: all 16 channels exist.  kVec: dim is at least V, so that a lane whose channels go past
  // dim can load the last V channels instead: it writes some of the values that the lanes beside it
  // write too, and none before the wave's first channel.
  auto run = [&](auto WHOLE, auto VEC_) {
    constexpr bool kWhole = decltype(WHOLE)::value, kVec = decltype(VEC_)::value;
    const int64_t left = p.dim - (c0 + lcol);
    const int nv = kWhole || left >= V ? V : static_cast<int>(left < 0 ? 0 : left);  // channels of this lane's rows of y
    const int64_t col = kWhole || left >= V ? c0 + lcol : (kVec ? p.dim - V : (nv > 0 ? c0 + lcol : c0));
    const int wcol = static_cast<int>(col - c0);  // negative where dim - V lies before the wave
    const int pv = kVec ? V : nv;                 // channels that it loads
    float bias[V], dsk[V], dsum[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bias[v] = p.delta_bias && v < pv ? p.delta_bias[col + v] : 0.0f;
      dsk[v] = has_d && v < pv ? p.Dskip[col + v] : 0.0f;
      dsum[v] = 0.0f;
    }
    const int row1 = lrow < last_row ? lrow : last_row, k1 = k < last_row ? k : last_row;
    const int nb = n0 < N ? n0 : 0;  // (rows of lanes past dstate read state 0 and use zeros)
    uint32_t ox = offset(lrow, p.sx, col), od = offset(lrow, p.sdelta, col), oz = offset(lrow, zstride, col);
    uint32_t ob = offset(k, p.sB, nb), oc = offset(k, p.sC, nb);
    const uint32_t oy = offset(lrow, p.sy, c0 + lcol);
    const char *bx = first_row(p.x, p.sx), *bd = first_row(p.delta, p.sdelta), *bz = first_row(zsrc, zstride);
    const char *bb = first_row(p.B, p.sB), *bc = first_row(p.C, p.sC);
    char* by = const_cast<char*>(first_row(p.y, p.sy));
    auto last_offsets = [&] {
      ox = offset(row1, p.sx, col);
      od = offset(row1, p.sdelta, col);
      oz = offset(row1, zstride, col);
      ob = offset(k1, p.sB, nb);
      oc = offset(k1, p.sC, nb);
    };
    Run<BF16, V> nx, nd, nz;
    constexpr int NB = N >= 4 ? NPL : 1;
    Run<BF16, NB> rb, rc;
    auto load = [&] {
      if constexpr (kVec) {
        nx.load_bytes(bx + ox);
        nd.load_bytes(bd + od);
        if constexpr (!AGG) nz.load_bytes(bz + oz);
      } else {
        nx.load_some_bytes(bx + ox, pv);
        nd.load_some_bytes(bd + od, pv);
        if constexpr (!AGG) nz.load_some_bytes(bz + oz, pv);
      }
      rb.load_bytes(bb + ob);
      if constexpr (!AGG) rc.load_bytes(bc + oc);
    };
    if (nchunks == 1) last_offsets();
    load();
    for (int c = 0; c < nchunks; ++c) {
      // ---- the chunk's values, from the registers loaded a chunk ago
      const bool full = c + 1 < nchunks || last_row == CH - 1;
      float dt[V], xv[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        dt[v] = nd.get(v) + bias[v];
        xv[v] = nx.get(v);
      }
      if (p.softplus) {
#pragma unroll
        for (int v = 0; v < V; ++v) dt[v] = softplus_f32(dt[v]);
      }
      float Bv[NPL], Cv[AGG ? 1 : NPL];
#pragma unroll
      for (int j = 0; j < NPL; ++j) {
        Bv[j] = n0 + j < N ? rb.get(j < NB ? j : 0) : 0.0f;
        if constexpr (!AGG) Cv[j] = n0 + j < N ? rc.get(j < NB ? j : 0) : 0.0f;
      }
      if (!full) {  // steps past the piece: dt = dt x = B = 0 keep the state
#pragma unroll
        for (int v = 0; v < V; ++v) {
          dt[v] = lrow <= last_row ? dt[v] : 0.0f;
          xv[v] = lrow <= last_row ? xv[v] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NPL; ++j) Bv[j] = k <= last_row ? Bv[j] : 0.0f;
      }
      float gate[V], skip[V];
      if constexpr (AGG) {
#pragma unroll
        for (int v = 0; v < V; ++v) dsum[v] += dt[v];
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          gate[v] = has_z ? silu_f32(nz.get(v)) : 1.0f;
          skip[v] = has_d ? dsk[v] * xv[v] : 0.0f;  // (without D an infinite x adds nothing here)
        }
      }
      if constexpr (kWhole) {
        if constexpr (kOuter) {
          *reinterpret_cast<float4*>(s_dt + lrow * 16 + lcol) = make_float4(dt[0], dt[1], dt[2], dt[3]);
          *reinterpret_cast<float4*>(s_w + lrow * 16 + lcol) =
              make_float4(dt[0] * xv[0], dt[1] * xv[1], dt[2] * xv[2], dt[3] * xv[3]);
        } else {
          float4* const qd = reinterpret_cast<float4*>(s_dw + lrow * 16 + lcol);
          qd[0] = make_float4(dt[0], dt[0] * xv[0], dt[1], dt[1] * xv[1]);
          qd[1] = make_float4(dt[2], dt[2] * xv[2], dt[3], dt[3] * xv[3]);
        }
        if constexpr (!AGG) {
          float4* const qx = reinterpret_cast<float4*>(s_xg + lrow * 16 + lcol);
          qx[0] = make_float4(skip[0], gate[0], skip[1], gate[1]);
          qx[1] = make_float4(skip[2], gate[2], skip[3], gate[3]);
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (v >= pv || wcol + v < 0) continue;
          if constexpr (kOuter) {
            s_dt[lrow * 16 + wcol + v] = dt[v];
            s_w[lrow * 16 + wcol + v] = dt[v] * xv[v];
          } else {
            s_dw[lrow * 16 + wcol + v] = make_float2(dt[v], dt[v] * xv[v]);
          }
          if constexpr (!AGG) s_xg[lrow * 16 + wcol + v] = make_float2(skip[v], gate[v]);
        }
      }
      if constexpr (kOuter) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) s_b[(n0 + j) * BS + k] = Bv[j];
      }
      wave_lds_fence();
      if (c + 1 < nchunks) {
        bx += CH * p.sx * ES;
        bd += CH * p.sdelta * ES;
        bz += CH * zstride * ES;
        bb += CH * p.sB * ES;
        bc += CH * p.sC * ES;
        if (c + 2 == nchunks) last_offsets();
      }
      load();
      // ---- 16 steps, four at a time
      [[maybe_unused]] float yp[4];
      auto finish = [&](int t) {  // read-outs of steps t .. t + 3
        if constexpr (N < 4) {  // a padding state that an infinity made NaN counts for nothing
#pragma unroll
          for (int u = 0; u < 4; ++u) yp[u] = r < N ? yp[u] : 0.0f;
        }
        const float y = sum_rows4(yp);
        const float2 xg = s_xg[(t + r) * 16 + k];
        s_y[(t + r) * 16 + k] = (y + xg.x) * xg.y;
      };
      if constexpr (kOuter) {
        // The input terms B (x) dt x of four steps are one 16x16x1 matrix instruction of four blocks: in
        // block b lane 16 b + m has B of step t + b, state m and dt x of channel m; of the result,
        // register 4 b + j of lane 16 r + k is step t + b, state 4 r + j, channel k: the recurrence's
        // own layout.  (A product of one term with a zero addend: rounded once, like a multiplication.)
        // It does not wait for the state, so the next four steps' goes out in the middle of these
        // four; the barrier keeps the compiler from moving it to where its result is used, at the
        // price of its whole latency.  bf16, us against the terms by DPP operands in every step: 32
        // prompts of 2048 x 1536 374 | 392, 8 of 2048 (whole) 172 | 178, one of 8192 92 | 96.  dstate 32 and 64
        // have no registers for the results of two groups (64: 536 | 480 us for 8 of 2048), and one
        // 4x4x1 instruction a step with exp(dt A) h as its addend is no faster than DPP (187 | 178).
        // The read-outs stay off the matrix cores: with them there too a full pass took 498 us for 397.
        const float* const t_b = s_b + k * BS + r;
        const float* const t_w = s_w + r * 16 + k;
        float dq[2][4];
        auto read_dt = [&](int t, float (&v)[4]) {
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = s_dt[(t + u) * 16 + k];
        };
        read_dt(0, dq[0]);
        float ob = t_b[0], ow = t_w[0];
        f32x16_t in[2];
        in[0] = __builtin_amdgcn_mfma_f32_16x16x1f32(ob, ow, f32x16_t{}, 0, 0, 0);
        ob = t_b[4], ow = t_w[4 * 16];
        static_for<CH / 4>([&](auto G) {
          constexpr int t = decltype(G)::value * 4, i = decltype(G)::value & 1;
          if constexpr (t + 4 < CH) read_dt(t + 4, dq[i ^ 1]);
          static_for<4>([&](auto U) {
            constexpr int u = decltype(U)::value, s = t + u;
            const float d = dq[i][u];
            if constexpr (u == 1 && t + 4 < CH) {
              in[i ^ 1] = __builtin_amdgcn_mfma_f32_16x16x1f32(ob, ow, f32x16_t{}, 0, 0, 0);
              if constexpr (t + 8 < CH) ob = t_b[t + 8], ow = t_w[(t + 8) * 16];
              __builtin_amdgcn_sched_barrier(0);
            }
            float e[4];
            if constexpr (AGG || s == 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j) e[j] = hw_exp2(d * A2[j]);
            } else {
              yp[(s - 1) & 3] = decay_readout4<s - 1>(d, A2, Cv, h, e);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = fmaf(e[j], h[j], in[i][4 * u + j]);
            if constexpr (!AGG && s > 0 && s % 4 == 0) finish(s - 4);
          });
        });
      } else {
        float2 dw[2][4];
        auto read_dw = [&](int t, float2 (&w)[4]) {
#pragma unroll
          for (int u = 0; u < 4; ++u) w[u] = s_dw[(t + u) * 16 + k];
        };
        read_dw(0, dw[0]);
        static_for<CH / 4>([&](auto G) {
          constexpr int t = decltype(G)::value * 4, i = decltype(G)::value & 1;
          if constexpr (t + 4 < CH) read_dw(t + 4, dw[i ^ 1]);
          static_for<4>([&](auto U) {
            constexpr int s = t + decltype(U)::value;
            const float2 w = dw[i][decltype(U)::value];
            if constexpr (AGG || s == 0) {
              step_state<NPL, s>(w.x, w.y, A2, Bv, h);
            } else {
              yp[(s - 1) & 3] = step_readout<NPL, s, s - 1>(w.x, w.y, A2, Bv, Cv, h);
              if constexpr (s % 4 == 0) finish(s - 4);
            }
          });
        });
      }
      if constexpr (!AGG) {
        float last = row_bcast<15>(Cv[0]) * h[0];
#pragma unroll
        for (int j = 1; j < NPL; ++j) last = fmaf(row_bcast<15>(Cv[j]), h[j], last);
        yp[3] = last;
        finish(CH - 4);
        wave_lds_fence();
        const float4 y4 = *reinterpret_cast<const float4*>(s_y + lrow * 16 + lcol);
        const float out[V] = {y4.x, y4.y, y4.z, y4.w};
        Run<BF16, V> o;
        o.set(out);
        if (full || lrow <= last_row) {
          if (kWhole || nv == V) o.store_bytes(by + oy);
          else o.store_some_bytes(by + oy, nv);
        }
        by += CH * p.sy * ES;
      }
      wave_lds_fence();  // before the next chunk's values
    }
    if constexpr (AGG) {
      // the summed step: over the 16 lanes that hold the same channels
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int off = 4; off < 64; off <<= 1) dsum[v] += __shfl_xor(dsum[v], off, 64);
        if (lrow == 0 && v < pv && wcol + v >= 0) p.seg_dsum[g * p.dim + col + v] = dsum[v];
      }
    }
  };
  if (c0 + 16 <= p.dim) run(std::true_type{}, std::true_type{});
  else if (p.dim >= V) run(std::false_type{}, std::true_type{});
  else run(std::false_type{}, std::false_type{});

  if (!lane_ok) return;
  if constexpr (AGG) {
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (n0 + j < N) p.seg_state[(g * p.dim + d) * N + n0 + j] = h[j];
  } else if (at >= 0 && kth + 1 == npieces) {
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      if (n0 + j >= N) continue;
      if (p.cache_bf16) store_one<true>(p.cache.data, cache_index(j), h[j]);
      else store_one<false>(p.cache.data, cache_index(j), h[j]);
    }
  }
}

struct ScanPackedKernels {
  void (*full)(const ScanPackedArgs);
  void (*agg)(const ScanPackedArgs);
};
const ScanPackedKernels* scan_packed_kernels(bool bf16, int64_t dstate);

}  // namespace ssm
