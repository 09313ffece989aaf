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

template <int NV>
struct Codes {
  uint32_t w[(NV + 3) / 4];
  __device__ __forceinline__ void load(const int8_t* p) {
    if constexpr (NV % 4 == 0) {
#pragma unroll
      for (int i = 0; i < NV / 4; ++i) w[i] = reinterpret_cast<const Words<1>::U1*>(p)[i];
    } else {
      w[0] = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) w[0] |= static_cast<uint32_t>(static_cast<uint8_t>(p[v])) << (8 * v);
    }
  }
  __device__ __forceinline__ int get(int v) const { return static_cast<int8_t>(w[v / 4] >> (8 * (v % 4))); }
};

// Rows that a thread takes: their loads are in flight together.  61 states of 4096 x 128 fp32 are stored in
// 35 us (161 MB, 4.6 TB/s) with 4, in 47 us with one and reductions through the LDS, and read back in
// 24 us (161 MB: part of it comes out of the caches).
constexpr int kQ8Rows = 4;

template <bool CB16, int N>
__global__ __launch_bounds__(kQ8Threads) void cache_store_q8_kernel(const Q8Args p) {
  constexpr int V = kQ8Values<CB16, N>, LPR = N / V, RPB = kQ8Threads / LPR;
  static_assert(LPR <= 64, "a row's lanes share one wave");
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * (RPB * kQ8Rows) + threadIdx.x / LPR;
  const int n0 = static_cast<int>(threadIdx.x % LPR) * V;
  for (int64_t i = blockIdx.y; i < p.count; i += gridDim.y) {
    const int64_t at = cache_offset(p.cache, p.cache_slots, i);
    const int64_t to = p.store_slots ? p.store_slots[i] : i;
    if (at < 0 || to < 0 || to >= p.stored) continue;
    Run<CB16, V, true> r[kQ8Rows];
#pragma unroll
    for (int u = 0; u < kQ8Rows; ++u) {
      const int64_t row = row0 + u * RPB;
      r[u].load(p.cache.data, at + (row < p.rows ? row : p.rows - 1) * N + n0);
    }
#pragma unroll
    for (int u = 0; u < kQ8Rows; ++u) {
      const int64_t row = row0 + u * RPB;
      // |v| as bits: their order is the values', with infinity and then NaN above every number
      uint32_t top = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t b = __builtin_bit_cast(uint32_t, r[u].get(v)) & 0x7fffffffu;
        top = b > top ? b : top;
      }
      top = group_reduce<LPR>(top, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
      const bool bad = top >= 0x7f800000u;
      const float scale = bad ? __builtin_nanf("") : __builtin_bit_cast(float, top) / 127.0f;
      const float up = scale < 1.17549435e-38f ? 1.2676506e30f : 1.0f;  // 2^100 where 1 / scale overflows
      const float sc = scale * up, inv = 1.0f / sc;
      int q[V];
#pragma unroll
      for (int v = 0; v < V; ++v)
        q[v] = bad || scale == 0.0f ? 0 : static_cast<int>(q8_code(r[u].get(v) * up, sc, inv));
      if (row < p.rows) {
        const int64_t o = (to * p.rows + row) * N + n0;
        store_codes<V>(p.codes + o, q);
        if (n0 == 0) p.scales[to * p.rows + row] = scale;
      }
    }
  }
}

template <bool CB16, int N>
__global__ __launch_bounds__(kQ8Threads) void cache_load_q8_kernel(const Q8Args p) {
  constexpr int V = kQ8Values<CB16, N>, LPR = N / V, RPB = kQ8Threads / LPR;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * (RPB * kQ8Rows) + threadIdx.x / LPR;
  const int n0 = static_cast<int>(threadIdx.x % LPR) * V;
  for (int64_t i = blockIdx.y; i < p.count; i += gridDim.y) {
    const int64_t at = cache_offset(p.cache, p.cache_slots, i);
    const int64_t from = p.store_slots ? p.store_slots[i] : i;
    if (at < 0 || from < 0 || from >= p.stored) continue;
    Codes<V> c[kQ8Rows];
    float scale[kQ8Rows];
#pragma unroll
    for (int u = 0; u < kQ8Rows; ++u) {
      const int64_t row = from * p.rows + (row0 + u * RPB < p.rows ? row0 + u * RPB : p.rows - 1);
      c[u].load(p.codes + row * N + n0);
      scale[u] = p.scales[row];
    }
#pragma unroll
    for (int u = 0; u < kQ8Rows; ++u) {
      const int64_t row = row0 + u * RPB;
      if (row >= p.rows) break;
      float val[V];
#pragma unroll
      for (int v = 0; v < V; ++v) val[v] = static_cast<float>(c[u].get(v)) * scale[u];
      Run<CB16, V, true> r;
      r.set(val);
      r.store(p.cache.data, at + row * N + n0);
    }
  }
}

}  // namespace ssm
