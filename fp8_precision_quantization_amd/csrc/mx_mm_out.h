// The epilogues of the MX products (mx_mm.h): accumulators leave through a
// part of LDS that is the wave's own, 32 rows at a time, so that memory sees
// whole 16-byte words of whole row segments.
#pragma once

#include "mx_mm.h"
#include "mx_train.h"

namespace mx {

// 32 staged rows of BYTES each; a row's pitch is a word longer, which spreads
// the lanes of a write over the banks.
template <int BYTES>
struct Staged {
  static constexpr int kPitch = BYTES + 16;
  static constexpr int kSize = 32 * kPitch;
  static constexpr int kLanes = BYTES / 16, kRows = 64 / kLanes;   // of one access
  uint8_t* at;

  template <class V>
  __device__ __forceinline__ void put(int row, int byte, V v) const {
    *reinterpret_cast<V*>(at + row * kPitch + byte) = v;
  }
  template <class V>
  __device__ __forceinline__ V get(int row, int byte) const {
    return *reinterpret_cast<const V*>(at + row * kPitch + byte);
  }
  // To memory: the first `rows` rows' first `bytes` bytes (a multiple of 16),
  // rows ld bytes apart, everything 16-byte aligned.
  __device__ __forceinline__ void drain(uint8_t* dst, int64_t ld, int rows, int bytes) const {
    const int lane = threadIdx.x & 63, in = lane / kLanes, byte = 16 * (lane % kLanes);
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) {
      const int row = kRows * i + in;
      if (row < rows && byte < bytes)
        __builtin_nontemporal_store(get<u32x4>(row, byte), reinterpret_cast<u32x4*>(dst + row * ld + byte));
    }
  }
  // The same in elements of E at any alignment, `n` of them a row.
  template <class E>
  __device__ __forceinline__ void drain_each(E* dst, int64_t ld, int rows, int n) const {
    const int lane = threadIdx.x & 63;
    for (int row = 0; row < min(rows, 32); ++row)
      for (int e = lane; e < min(n, BYTES / (int)sizeof(E)); e += 64)
        dst[row * ld + e] = get<E>(row, e * (int)sizeof(E));
  }
  // From memory, as drain() writes; zeros elsewhere.
  __device__ __forceinline__ void fill(const uint8_t* src, int64_t ld, int rows, int bytes) const {
    const int lane = threadIdx.x & 63, in = lane / kLanes, byte = 16 * (lane % kLanes);
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) {
      const int row = kRows * i + in;
      u32x4 v = {0, 0, 0, 0};
      if (row < rows && byte < bytes)
        v = *reinterpret_cast<const u32x4*>(src + row * ld + byte);
      put(row, byte, v);
    }
  }
};

}  // namespace mx
