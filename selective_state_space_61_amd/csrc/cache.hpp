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

// A reduction over groups of LANES neighbouring lanes (a power of two), its result in every lane:
// DPP within a row of 16 (quad permutations, half-row and row mirrors), lane swaps across rows.  All
// of it VALU work; the shuffles through the LDS that it replaces set the pace of the 8-bit store.
template <int LANES, typename T, typename F>
__device__ __forceinline__ T group_reduce(T v, F op) {
  static_assert(sizeof(T) == 4 && LANES >= 1 && LANES <= 64 && (LANES & (LANES - 1)) == 0, "lanes of a wave");
  auto dpp = [&](auto CTRL) {
    return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(CTRL)::value, 0xF, 0xF, true));
  };
  if constexpr (LANES >= 2) v = op(v, dpp(std::integral_constant<int, 0xB1>{}));    // lane ^ 1
  if constexpr (LANES >= 4) v = op(v, dpp(std::integral_constant<int, 0x4E>{}));    // lane ^ 2
  if constexpr (LANES >= 8) v = op(v, dpp(std::integral_constant<int, 0x141>{}));   // the other half of 8
  if constexpr (LANES >= 16) v = op(v, dpp(std::integral_constant<int, 0x140>{}));  // the other half of 16
  auto swapped = [&](auto q) {
    const uint32_t a = q[0], b = q[1];
    return op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
  };
  if constexpr (LANES >= 32) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    v = swapped(__builtin_amdgcn_permlane16_swap(u, u, false, false));
  }
  if constexpr (LANES >= 64) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    v = swapped(__builtin_amdgcn_permlane32_swap(u, u, false, false));
  }
  return v;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<LANES>(v, [](float a, float b) { return a + b; });
}

// The sequence of a packed row: `start` and `end` its rows (within 0..total, whatever cu holds), s its
// index, or -1 where the row is of none.
struct RowOwner {
  int64_t s, start, end;
};

// The sequences from row t on, 64 of them at a time in a wave's registers: entry s0 + lane of cu, its slot
// and its flag.  Every lane of the wave makes the same calls, with rows that do not fall.
class Sequences {
 public:
  __device__ __forceinline__ Sequences(const int32_t* cu, const int32_t* slots, const uint8_t* has_initial,
                                       int64_t nseq, int64_t total, int64_t t)
      : cu_(cu), slots_(slots), has_initial_(has_initial), nseq_(nseq), total_(total), s0_(0) {
    // the last entry not above t, 64 probes at a time: none up to 63 sequences, one round up to 4095
    int64_t first = 0;
    for (int64_t left = nseq + 1; left > 64;) {
      const int64_t step = (left + 63) / 64, i = (threadIdx.x & 63) * step;
      const int c = __popcll(__ballot(i < left && cu[first + (i < left ? i : 0)] <= t));
      const int64_t skip = c > 0 ? (c - 1) * step : 0;
      first += skip;
      left = left - skip < step ? left - skip : step;
    }
    read(first);
  }

  __device__ __forceinline__ RowOwner owner(int64_t t) {
    int c = not_above(t);
    while (c == 64) {  // (ends: entries past nseq are above every row)
      read(s0_ + 63);
      c = not_above(t);
    }
    RowOwner r;
    const int64_t s = s0_ + c - 1;
    // with none the row lies before the first sequence, with all nseq + 1 behind the last
    r.s = c > 0 && s < nseq_ ? s : -1;
    r.start = c > 0 ? __builtin_amdgcn_readlane(entry_, c - 1) : 0;
    r.end = s < nseq_ ? __builtin_amdgcn_readlane(entry_, c) : total_;
    r.start = r.start < 0 ? 0 : (r.start > t ? t : r.start);
    r.end = r.end <= t ? t + 1 : (r.end > total_ ? total_ : r.end);
    return r;
  }

  // first element of the slot of sequence s (one that owner() gave last), -1: none
  __device__ __forceinline__ int64_t slot_offset(const CacheRef& c, int64_t s) const {
    const int64_t slot = slots_ ? __builtin_amdgcn_readlane(slot_, static_cast<int>(s - s0_)) : s;
    return slot >= 0 && slot < c.slots ? slot * c.stride : -1;
  }
  __device__ __forceinline__ bool initial(int64_t s) const {
    return __builtin_amdgcn_readlane(flag_, static_cast<int>(s - s0_)) != 0;
  }

 private:
  __device__ __forceinline__ int not_above(int64_t t) const {
    return __popcll(__ballot(static_cast<int64_t>(entry_) <= t));
  }
  __device__ __forceinline__ void read(int64_t s0) {
    s0_ = s0;
    const int64_t i = s0 + (threadIdx.x & 63);
    entry_ = i <= nseq_ ? cu_[i] : INT32_MAX;
    slot_ = slots_ && i < nseq_ ? slots_[i] : -1;
    flag_ = has_initial_ && i < nseq_ ? has_initial_[i] : 0;
  }
  const int32_t* cu_;
  const int32_t* slots_;
  const uint8_t* has_initial_;
  int64_t nseq_, total_, s0_;
  int32_t entry_, slot_;
  int32_t flag_;
};

}  // namespace ssm
