// cache_q8.hpp -- states of a cache set aside as int8 codes with a scale per row, and read back
// (gfx950).
//
//   scale = fl32(max_n |v_n| / 127),  code_n = rint(v_n / scale) (the exact quotient, ties to
//   even, clamped to +-127),  read back: fl(code_n * scale).
//
// The code is the rounding of the exact quotient: q0 = rint(v * (1 / scale)) is off by at most one
// and only next to a border between two codes; the remainder r = v - q0 scale is one fma and
// exact (it is below 0.51 scale and a multiple of the smaller of v's and scale's last places, or, at
// |q0| <= 1, a difference of neighbours), and 2 r against scale says on which side of the border v
// lies.  Rows whose scale is subnormal are computed 2^100 larger, which changes no code.
#pragma once

#include "cache.hpp"

namespace ssm {

struct Q8Args {
  CacheRef cache;
  const int32_t* cache_slots;
  int8_t* codes;
  float* scales;
  const int32_t* store_slots;
  int64_t stored;
  int64_t count;
  int64_t rows;
};

constexpr int kQ8Threads = 256;

// values of a row that one lane takes: 16 bytes of the cache
template <bool CB16, int N>
constexpr int kQ8Values = CB16 ? (N < 8 ? N : 8) : (N < 4 ? N : 4);

__device__ __forceinline__ float q8_code(float v, float scale, float inv) {
  float q = rintf(v * inv);
  const float r2 = 2.0f * fmaf(-q, scale, v);
  const float s = r2 < 0.0f ? -1.0f : 1.0f;
  const float m = fabsf(r2);
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (m > scale || (m == scale && odd)) q += s;
  return fminf(fmaxf(q, -127.0f), 127.0f);
}

// NV codes, the lowest byte first
template <int NV>
__device__ __forceinline__ void store_codes(int8_t* p, const int (&q)[NV]) {
  if constexpr (NV % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NV / 4; ++i)
      reinterpret_cast<Words<1>::U1*>(p)[i] = (q[4 * i] & 0xff) | (q[4 * i + 1] & 0xff) << 8 | (q[4 * i + 2] & 0xff) << 16 |
                                              static_cast<uint32_t>(q[4 * i + 3]) << 24;
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) p[v] = static_cast<int8_t>(q[v]);
  }
}

template <bool CB16, int N>
__global__ __launch_bounds__(kQ8Threads) void cache_store_q8_kernel(const Q8Args p) {
  constexpr int V = kQ8Values<CB16, N>, LPR = N / V;
  static_assert(LPR <= 64, "a row's lanes share one wave");
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kQ8Threads + threadIdx.x;
  const bool ok = t / LPR < p.rows;
  const int64_t row = ok ? t / LPR : p.rows - 1;
  const int n0 = static_cast<int>(t % LPR) * V;
  for (int64_t i = blockIdx.y; i < p.count; i += gridDim.y) {
    const int64_t at = cache_offset(p.cache, p.cache_slots, i);
    const int64_t to = p.store_slots ? p.store_slots[i] : i;
    if (at < 0 || to < 0 || to >= p.stored) continue;
    Run<CB16, V, true> r;
    r.load(p.cache.data, at + row * N + n0);
    // |v| as bits: their order is the values', with infinity and then NaN above every number
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t b = __builtin_bit_cast(uint32_t, r.get(v)) & 0x7fffffffu;
      top = b > top ? b : top;
    }
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) {
      const uint32_t o = __shfl_xor(top, off, 64);
      top = o > top ? o : top;
    }
    const bool bad = top >= 0x7f800000u;
    const float scale = bad ? __builtin_nanf("") : __builtin_bit_cast(float, top) / 127.0f;
    int q[V];
    if (bad || scale == 0.0f) {
#pragma unroll
      for (int v = 0; v < V; ++v) q[v] = 0;
    } else {
      const float up = scale < 1.17549435e-38f ? 1.2676506e30f : 1.0f;  // 2^100 where 1 / scale overflows
      const float sc = scale * up, inv = 1.0f / sc;
#pragma unroll
      for (int v = 0; v < V; ++v) q[v] = static_cast<int>(q8_code(r.get(v) * up, sc, inv));
    }
    if (ok) {
      const int64_t o = (to * p.rows + row) * N + n0;
      store_codes<V>(p.codes + o, q);
      if (n0 == 0) p.scales[to * p.rows + row] = scale;
    }
  }
}

template <bool CB16, int N>
__global__ __launch_bounds__(kQ8Threads) void cache_load_q8_kernel(const Q8Args p) {
  constexpr int V = kQ8Values<CB16, N>, LPR = N / V;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kQ8Threads + threadIdx.x;
  if (t / LPR >= p.rows) return;
  const int64_t row = t / LPR;
  const int n0 = static_cast<int>(t % LPR) * V;
  for (int64_t i = blockIdx.y; i < p.count; i += gridDim.y) {
    const int64_t at = cache_offset(p.cache, p.cache_slots, i);
    const int64_t from = p.store_slots ? p.store_slots[i] : i;
    if (at < 0 || from < 0 || from >= p.stored) continue;
    const int8_t* c = p.codes + (from * p.rows + row) * N + n0;
    const float scale = p.scales[from * p.rows + row];
    float val[V];
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const uint32_t w = reinterpret_cast<const Words<1>::U1*>(c)[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) val[4 * k + j] = static_cast<float>(static_cast<int8_t>(w >> (8 * j))) * scale;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) val[v] = static_cast<float>(c[v]) * scale;
    }
    Run<CB16, V, true> r;
    r.set(val);
    r.store(p.cache.data, at + row * N + n0);
  }
}

}  // namespace ssm
