// cache.hpp -- device helpers of the serving kernels: slots of a cache, runs of consecutive
// elements, and the sequence that a packed row belongs to.
#pragma once

#include "conv1d.hpp"

namespace ssm {

// `slots` entries `stride` elements apart
struct CacheRef {
  void* data;
  int64_t slots;
  int64_t stride;
};

// First element of entry i's slot, or -1 where it has none (padding, or out of range)
__device__ __forceinline__ int64_t cache_offset(const CacheRef& c, const int32_t* slots, int64_t i) {
  const int64_t s = slots ? slots[i] : i;
  return s >= 0 && s < c.slots ? s * c.stride : -1;
}

// Words of a run of elements that starts at a multiple of an element's size only.  gfx950 takes wide
// global accesses at any such address (the compiler's unaligned-access mode for this target), so
// rows of odd widths and columns of wider tensors take the same path as aligned ones: a 777-wide
// bf16 row costs the same instructions as a 776-wide one.
typedef uint32_t U32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t U32x2 __attribute__((ext_vector_type(2)));
template <int ALIGN>
struct Words;
#define SSM_WORDS(ALIGN)                                      \
  template <>                                                 \
  struct Words<ALIGN> {                                       \
    typedef U32x4 U4 __attribute__((aligned(ALIGN)));         \
    typedef U32x2 U2 __attribute__((aligned(ALIGN)));         \
    typedef uint32_t U1 __attribute__((aligned(ALIGN)));      \
  }
SSM_WORDS(1);
SSM_WORDS(2);
SSM_WORDS(4);
#undef SSM_WORDS

// NV consecutive elements as raw words, loaded with the widest pieces their size has.  NT:
// non-temporal, for state that the next use of is a whole model step away.
template <bool BF16, int NV, bool NT = false>
struct Run {
  static constexpr int kSize = BF16 ? 2 : 4;
  static constexpr int kBytes = NV * kSize;
  static constexpr int kWords = (kBytes + 3) / 4;
  using W = Words<kSize>;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* base, int64_t idx) {
    load_bytes(static_cast<const char*>(base) + idx * kSize);
  }
  __device__ __forceinline__ void load_bytes(const char* p) {
    if constexpr (kBytes == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      constexpr int n4 = kWords / 4, n2 = kWords % 4 / 2;
      static_assert(kBytes % 4 == 0, "whole words");
#pragma unroll
      for (int i = 0; i < n4; ++i) {
        const typename W::U4* q = reinterpret_cast<const typename W::U4*>(p) + i;
        const U32x4 v = NT ? __builtin_nontemporal_load(q) : *q;
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
      if constexpr (n2 > 0) {
        const typename W::U2* q = reinterpret_cast<const typename W::U2*>(p + 16 * n4);
        const U32x2 v = NT ? __builtin_nontemporal_load(q) : *q;
        w[4 * n4] = v.x; w[4 * n4 + 1] = v.y;
      }
      if constexpr (kWords % 2 > 0) {
        const typename W::U1* q = reinterpret_cast<const typename W::U1*>(p + 4 * (kWords - 1));
        w[kWords - 1] = NT ? __builtin_nontemporal_load(q) : *q;
      }
    }
  }

  // the first nv elements, the others zero
  __device__ __forceinline__ void load_some(const void* base, int64_t idx, int nv) {
    load_some_bytes(static_cast<const char*>(base) + idx * kSize, nv);
  }
  __device__ __forceinline__ void load_some_bytes(const char* p, int nv) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (v >= nv) continue;
      if constexpr (BF16) w[v >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[v]) << (16 * (v & 1));
      else w[v] = reinterpret_cast<const uint32_t*>(p)[v];
    }
  }

  __device__ __forceinline__ float get(int v) const {
    if constexpr (BF16) return (v & 1) ? bf16_hi(w[v >> 1]) : bf16_lo(w[v >> 1]);
    else return __builtin_bit_cast(float, w[v]);
  }

  // an (empty) use of the words: the compiler waits for their load here, on every path through it
  __device__ __forceinline__ void consume() const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" ::"v"(w[i]));
  }

  __device__ __forceinline__ void set(const float (&val)[NV]) {
    if constexpr (BF16) {
#pragma unroll
      for (int v = 0; v + 1 < NV; v += 2) w[v >> 1] = pack_bf16x2(val[v], val[v + 1]);
      if constexpr (NV % 2) w[NV >> 1] = to_bf16(val[NV - 1]);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) w[v] = __builtin_bit_cast(uint32_t, val[v]);
    }
  }

  __device__ __forceinline__ void store(void* base, int64_t idx) const {
    store_bytes(static_cast<char*>(base) + idx * kSize);
  }
  __device__ __forceinline__ void store_bytes(char* p) const {
    if constexpr (kBytes == 2) {
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    } else {
      constexpr int n4 = kWords / 4, n2 = kWords % 4 / 2;
#pragma unroll
      for (int i = 0; i < n4; ++i) {
        const U32x4 v = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        typename W::U4* q = reinterpret_cast<typename W::U4*>(p) + i;
        if constexpr (NT) __builtin_nontemporal_store(v, q);
        else *q = v;
      }
      if constexpr (n2 > 0) {
        const U32x2 v = {w[4 * n4], w[4 * n4 + 1]};
        typename W::U2* q = reinterpret_cast<typename W::U2*>(p + 16 * n4);
        if constexpr (NT) __builtin_nontemporal_store(v, q);
        else *q = v;
      }
      if constexpr (kWords % 2 > 0) {
        typename W::U1* q = reinterpret_cast<typename W::U1*>(p + 4 * (kWords - 1));
        if constexpr (NT) __builtin_nontemporal_store(w[kWords - 1], q);
        else *q = w[kWords - 1];
      }
    }
  }

  __device__ __forceinline__ void store_some(void* base, int64_t idx, int nv) const {
    store_some_bytes(static_cast<char*>(base) + idx * kSize, nv);
  }
  __device__ __forceinline__ void store_some_bytes(char* p, int nv) const {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (v >= nv) continue;
      if constexpr (BF16) reinterpret_cast<uint16_t*>(p)[v] = static_cast<uint16_t>(w[v >> 1] >> (16 * (v & 1)));
      else reinterpret_cast<uint32_t*>(p)[v] = w[v];
    }
  }
};

// The sequence of packed row t: `start` and `end` its rows (within 0..total, whatever cu holds),
// s its index, or -1 where the row is of none; then `end` is the first row that may be of one.
// Every lane of a wave calls it with the same t: 64 lanes compare 64 entries of cu at a time and
// count those not above t, so up to 63 sequences take one load.
struct RowOwner {
  int64_t s, start, end;
};
__device__ __forceinline__ RowOwner row_owner(const int32_t* cu, int64_t nseq, int64_t total, int64_t t) {
  const int lane = threadIdx.x & 63;
  int64_t n = 0;
  for (int64_t i = 0; i <= nseq; i += 64) {
    const bool in = i + lane <= nseq && cu[i + lane] <= t;
    n += __popcll(__ballot(in));
  }
  RowOwner r;
  r.s = n - 1;
  // with n == nseq + 1 the row lies behind the last sequence
  r.start = n > 0 ? cu[n - 1] : 0;
  r.end = n <= nseq ? cu[n] : total;
  if (n > nseq) r.s = -1;
  r.start = r.start < 0 ? 0 : (r.start > t ? t : r.start);
  r.end = r.end <= t ? t + 1 : (r.end > total ? total : r.end);
  return r;
}

}  // namespace ssm
