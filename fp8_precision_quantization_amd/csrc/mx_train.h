// Device helpers shared by the training-step operators (gfx950 only): moves
// between bf16 / binary32 memory and binary32 registers, and sums and maxima
// over lanes.  All arithmetic is binary32.
#pragma once

#include "mx_device.h"

namespace mx {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Two binary32 values -> packed bf16, nearest-even, the first in the low half
// (one v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// T: float, or uint16_t for bf16 bits.  N consecutive elements <-> binary32.
// N > 1 moves whole 16-byte words (N * sizeof(T) a multiple of 16, aligned),
// except for eight-byte halves of bf16 (N = 4).
template <int N>
__device__ __forceinline__ void unpack(const float* p, float (&f)[N]) {
  if constexpr (N == 1) {
    f[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(p + i);
      f[i] = v[0], f[i + 1] = v[1], f[i + 2] = v[2], f[i + 3] = v[3];
    }
  }
}
template <int N>
__device__ __forceinline__ void unpack(const uint16_t* p, float (&f)[N]) {
  if constexpr (N == 1) {
    f[0] = bf16_lo(*p);
  } else if constexpr (N == 4) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    f[0] = bf16_lo(v[0]), f[1] = bf16_hi(v[0]), f[2] = bf16_lo(v[1]), f[3] = bf16_hi(v[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[i + 2 * j] = bf16_lo(v[j]), f[i + 2 * j + 1] = bf16_hi(v[j]);
    }
  }
}

// Cache policies.  kCacheNT: memory that is not read again soon (a hint).
// kCacheThrough: stores go through to memory at once.
constexpr int kCacheNT = 2, kCacheThrough = 17;

// N elements as loaded, one register word per 4 bytes (a bf16 single fills
// one word): kept raw while in flight, turned into binary32 when used.
template <typename T, int N, int kPolicy = 0>
struct Raw {
  static constexpr int kWords = N == 1 ? 1 : N * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      w[i] = 0;
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (N == 1) {
      if constexpr (sizeof(T) == 2)
        w[0] = *p;
      else
        w[0] = __float_as_uint(*p);
    } else {
      static_assert(N * sizeof(T) == 16, "one 16-byte word");
      const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = v[i];
    }
  }
  // 16 bytes at any element
  __device__ __forceinline__ void load_ragged(const T* p) {
    static_assert(N * sizeof(T) == 16, "one 16-byte word");
    struct __attribute__((packed, aligned(sizeof(T)))) Word {
      u32x4 v;
    };
    const u32x4 v = reinterpret_cast<const Word*>(p)->v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = v[i];
  }
  // from a buffer's range, zeros past its end.  (The whole offset is the
  // lane's: a scalar one is taken off the range's size before the check, which
  // wraps where it is the larger.)
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rsrc, int offset) {
    if constexpr (N * sizeof(T) == 16) {
      const auto v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, offset, 0, kPolicy);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = v[i];
    } else if constexpr (sizeof(T) == 4) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, offset, 0, kPolicy);
    } else {
      w[0] = __builtin_amdgcn_raw_buffer_load_b16(rsrc, offset, 0, kPolicy);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i]);
    else if constexpr (N == 1)
      return bf16_lo(w[0]);
    else
      return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
};

// N binary32 values -> memory as T, rounded to nearest-even where T is bf16.
template <typename T, int N>
__device__ __forceinline__ void store(T* p, const float (&f)[N]) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (N == 1) {
      *p = f[0];
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<f32x4*>(p + i) = (f32x4){f[i], f[i + 1], f[i + 2], f[i + 3]};
    }
  } else {
    if constexpr (N == 1) {
      *p = (uint16_t)bf16_pair(f[0], f[0]);
    } else if constexpr (N == 4) {
      *reinterpret_cast<u32x2*>(p) = (u32x2){bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])};
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 8)
        *reinterpret_cast<u32x4*>(p + i) = (u32x4){bf16_pair(f[i], f[i + 1]), bf16_pair(f[i + 2], f[i + 3]),
                                                   bf16_pair(f[i + 4], f[i + 5]), bf16_pair(f[i + 6], f[i + 7])};
    }
  }
}

// The same at any element, 16 bytes.
template <typename T, int N>
__device__ __forceinline__ void store_ragged(T* p, const float (&f)[N]) {
  static_assert(N * sizeof(T) == 16, "one 16-byte word");
  struct __attribute__((packed, aligned(sizeof(T)))) Word {
    u32x4 v;
  };
  if constexpr (sizeof(T) == 4)
    reinterpret_cast<Word*>(p)->v = __builtin_bit_cast(u32x4, (f32x4){f[0], f[1], f[2], f[3]});
  else
    reinterpret_cast<Word*>(p)->v =
        (u32x4){bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
}

// The same into a buffer's range, dropped past its end; POLICY: the cache
// policy bits of the store.
template <typename T, int POLICY, int N>
__device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t rsrc, int offset, const float (&f)[N]) {
  if constexpr (N * sizeof(T) == 16 && sizeof(T) == 4)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, (f32x4){f[0], f[1], f[2], f[3]}), rsrc, offset, 0,
                                           POLICY);
  else if constexpr (N * sizeof(T) == 16)
    __builtin_amdgcn_raw_buffer_store_b128((u32x4){bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
                                                   bf16_pair(f[6], f[7])},
                                           rsrc, offset, 0, POLICY);
  else if constexpr (sizeof(T) == 4)
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f[0]), rsrc, offset, 0, POLICY);
  else
    __builtin_amdgcn_raw_buffer_store_b16((short)bf16_pair(f[0], f[0]), rsrc, offset, 0, POLICY);
}

// Lane moves inside rows of 16 lanes whose four steps visit every lane:
// neighbour, neighbouring pair, other half of 8, other half of 16.
template <int STEP>
__device__ __forceinline__ uint32_t row16_move(uint32_t v) {
  constexpr int ctrl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, true);
}

// op over the G lanes (16 or 64, aligned) a lane belongs to; every lane gets
// the result, the same bits in each (op is commutative and every step pairs
// lanes symmetrically).
template <int G, class Op>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, Op op) {
  v = op(v, row16_move<0>(v));
  v = op(v, row16_move<1>(v));
  v = op(v, row16_move<2>(v));
  v = op(v, row16_move<3>(v));
  if constexpr (G == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(b[0], b[1]);
  } else {
    static_assert(G == 16, "lanes of a group");
  }
  return v;
}
// Sum over the lanes l, l ^ 16, l ^ 32, l ^ 48; every lane gets it.
__device__ __forceinline__ float across_rows16(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
template <int G = 64>
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(lanes_reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int G>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return lanes_reduce<G>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int G>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
  return lanes_reduce<G>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}

// NaN if any is one (the maximum that keeps NaN).
template <int G>
__device__ __forceinline__ float lanes_fmax(float v) {
  return __uint_as_float(lanes_reduce<G>(__float_as_uint(v), [](uint32_t x, uint32_t y) {
    const float a = __uint_as_float(x), b = __uint_as_float(y);
    return __float_as_uint(__builtin_elementwise_maximum(a, b));
  }));
}

constexpr float kLog2E = 1.44269504088896341f;

// e^x from the hardware's 2^x: the product with log2(e) is rounded once, so
// the relative error grows like |x| * 2^-24, on top of the one or two ulp of
// v_exp_f32.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2E); }

}  // namespace mx
