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
  // Buffer range and offsets of `rows` rows' first `bytes` bytes (a multiple of
  // 16), ld apart (32 ld < 2^31): what lies outside is dropped, or read as
  // zeros, without a branch.
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t range(const uint8_t* p, int64_t ld, int rows, int bytes) {
    return buffer_rsrc(p, (uint32_t)(min(rows, 32) - 1) * (uint32_t)ld + (uint32_t)min(bytes, BYTES));
  }
  static __device__ __forceinline__ uint32_t offset(int i, int64_t ld, int bytes, int& row, int& byte) {
    const int lane = threadIdx.x & 63;
    row = kRows * i + lane / kLanes, byte = 16 * (lane % kLanes);
    return byte < bytes ? (uint32_t)row * (uint32_t)ld + (uint32_t)byte : 0x80000000u;
  }
  // To memory, everything 16-byte aligned, past the caches that the operands use
  // (block 32768 x 2048 x 2048 in MXFP8 272 -> 259 us, 16640 x 4096 x 5120 even;
  // 4096 x 1024 x 1024 16.9 -> 17.2).
  __device__ __forceinline__ void drain(uint8_t* dst, int64_t ld, int rows, int bytes) const {
    const __amdgpu_buffer_rsrc_t rs = range(dst, ld, rows, bytes);
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) {
      int row, byte;
      const uint32_t off = offset(i, ld, bytes, row, byte);
      __builtin_amdgcn_raw_buffer_store_b128(get<u32x4>(row, byte), rs, off, 0, kCacheNT);
    }
  }
  // The same in elements of E at any alignment, `n` of them a row.  (16640 x 8191 x
  // 5120 in MXFP4 443-457 us where 8192 columns take 351-390; 1037 x 1001 x 1056 8.5-9.0
  // in binary32 and 7.7-8.0 in bf16 where 1000 columns take 7.1-7.7 and 6.8-7.2.)
  template <class E>
  __device__ __forceinline__ void drain_each(E* dst, int64_t ld, int rows, int n) const {
    const int lane = threadIdx.x & 63;
    for (int row = 0; row < min(rows, 32); ++row)
      for (int e = lane; e < min(n, BYTES / (int)sizeof(E)); e += 64)
        dst[row * ld + e] = get<E>(row, e * (int)sizeof(E));
  }
  // From memory, as drain() writes: the loads, and what they brought to its
  // place.
  struct Loads {
    u32x4 v[32 / kRows];
  };
  static __device__ __forceinline__ void load(Loads& w, const uint8_t* src, int64_t ld, int rows, int bytes) {
    const __amdgpu_buffer_rsrc_t rs = range(src, ld, rows, bytes);
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) {
      int row, byte;
      const uint32_t off = offset(i, ld, bytes, row, byte);
      w.v[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
    }
  }
  __device__ __forceinline__ void place(const Loads& w) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i)
      put(kRows * i + lane / kLanes, 16 * (lane % kLanes), w.v[i]);
  }
};

}  // namespace mx
