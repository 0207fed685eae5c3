// Products of a few bf16 rows with MX weights, for decoding:
//   y[t][j] = sum over k of x[t][k] * W(j, k), or with W's rows a gate and a
//   factor half, y = act(x Wg^T) (x Wu^T).
//
// Codes become bf16 in registers (exactly, but where 2^e leaves bf16's range)
// and meet x in v_mfma_f32_16x16x32_bf16: x is not rounded, and sums are
// binary32.  A chunk is 128 of K, four blocks and four MFMAs.  A lane holds one
// block of one row of W, its 16 or 32 bytes of codes under one scale, and MFMA u
// takes elements 8 u .. + 7 of every lane's block, of W and of x alike: the
// order of K inside a sum is free.
//
// Bound by the weights' bytes for a row or two of x, and then by x itself, which
// every workgroup reads.  Lanes of a load should be neighbours in memory (a load
// whose neighbouring lanes are 16 different rows moves a quarter of the bytes a
// cycle), while the MFMAs want 16 rows in neighbouring lanes: rows go straight
// from memory to LDS, whole 64-byte lines and more at a time, 16-byte pieces
// permuted by an XOR with the row so that the reads meet no bank twice.
//
// A workgroup owns 16 RB columns (of each half); its waves take chunks of K in
// turn, each through BUFS buffers of its own without any barrier, and their sums
// meet in LDS in a fixed order.
#include "mx_fp4_launch.h"
#include "mx_gate.h"
#include "mx_mm.h"
#include "mx_train.h"

namespace mx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct DecodeArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t *qw, *sw;
  int64_t n, k;
  int32_t m;
  void* c;
  bool f32, gelu;
};

// FW: codes of W; TB: blocks of 16 rows of x; KS: waves.
template <int FW, int TB, int RB, bool GATED>
struct DecodeBuffer {
  static constexpr int kRows = GATED ? 2 * RB : RB;                       // blocks of 16 rows of W
  static constexpr int kRow = FW == MX_FORMAT_E2M1 ? 64 : 128;            // bytes of a chunk of one
  static constexpr int kX = 0, kW = TB * 4096, kS = kW + kRows * 16 * kRow;
  static constexpr int kBytes = kS + 256;
  static constexpr int kLoadsW = kRows * kRow / 64, kLoads = TB * 4 + kLoadsW + 1;
  static_assert(kRows <= 4, "scales of 64 rows");
};

template <int FW, int TB, int RB, int KS, int BUFS, bool GATED>
__global__ __launch_bounds__(64 * KS) void decode_kernel(DecodeArgs a) {
  using B = DecodeBuffer<FW, TB, RB, GATED>;
  constexpr bool kFp4 = FW == MX_FORMAT_E2M1;
  constexpr int kRows = B::kRows, kPieces = B::kRow / 16, kWords = kFp4 ? 1 : 2;
  static_assert(128 % (16 * RB) == 0, "a workgroup's rows lie in one strip of a scale layout");
  constexpr int kSums = KS * kRows * TB * 1024;
  constexpr int kLds = KS * BUFS * B::kBytes > kSums ? KS * BUFS * B::kBytes : kSums;
  static_assert((BUFS - 1) * B::kLoads < 64 && kLds <= 163840, "the load counter and LDS");
  __shared__ __attribute__((aligned(256))) uint8_t lds[kLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int64_t j0 = (int64_t)blockIdx.x * 16 * RB;
  const int ldw = (int)(kFp4 ? a.k / 2 : a.k), strip = (int)((a.k / 32 + 3) / 4) * 512;
  const int chunks = (int)((a.k + 127) / 128);

  // Ranges over the workgroup's rows of each half of W, and four rows of x at a
  // time (which may lie far apart): rows past the end, and K past it (an offset
  // outside), read as zeros.
  const int64_t rows = min((int64_t)16 * RB, a.n - j0), up = GATED ? a.n : 0;
  const MmRange rw = mm_range(a.qw + j0 * ldw, (uint32_t)(rows * ldw));
  const MmRange ru = GATED ? mm_range(a.qw + (j0 + up) * ldw, (uint32_t)(rows * ldw)) : rw;
  auto four_rows = [&](int u) {
    const int rows = min(4, a.m - 4 * u);
    return mm_range(a.x + (rows > 0 ? 4 * u * a.ldx : 0), rows > 0 ? (uint32_t)(((rows - 1) * a.ldx + a.k) * 2) : 0u);
  };
  // scale words: lane l's is of W's row l of the workgroup's, gate's rows first
  const int64_t srow0 = j0 / 128 * 128, srows = (a.n + up + 127) / 128 * 128 - srow0;
  const MmRange rs = mm_range(a.sw + srow0 / 128 * strip, (uint32_t)(srows / 128 * strip));
  uint32_t soff;
  {
    const int64_t row = j0 - srow0 + lane % (16 * RB) + (lane >= 16 * RB ? up : 0);
    soff = lane < 16 * kRows ? (uint32_t)(row / 128 * strip + 16 * (row % 32) + 4 * (row % 128 / 32)) : 0x80000000u;
  }
  // x: load u brings rows 4 u .. + 3, a lane piece l % 16 ^ row % 16 of its
  // row; W: 64 / kPieces rows
  const int xrow = lane / 16, wrow = lane / kPieces;
  const uint32_t mine =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds) +
      wave * BUFS * B::kBytes;
  auto load = [&](int ch, int b) {
    const uint32_t to = mine + b * B::kBytes;
#pragma unroll
    for (int u = 0; u < TB * 4; ++u) {
      const int k = 128 * ch + 8 * ((lane % 16) ^ ((4 * u + xrow) % 16));
      mm_load<16>(to + B::kX + u * 1024, four_rows(u), k < a.k ? ((uint32_t)xrow * (uint32_t)a.ldx + k) * 2 : 0x80000000u);
    }
#pragma unroll
    for (int u = 0; u < B::kLoadsW; ++u) {
      constexpr int kEach = 64 / kPieces, kHalf = 16 * RB;
      const int row = u * kEach + wrow, byte = ch * B::kRow + 16 * ((lane % kPieces) ^ mm_swizzle<kPieces>(row));
      mm_load<16>(to + B::kW + u * 1024, u * kEach < kHalf ? rw : ru,
                  byte < ldw ? (uint32_t)(row % kHalf * ldw + byte) : 0x80000000u);
    }
    mm_load<4>(to + B::kS, rs, soff + ch * 512);
  };

  f32x4 acc[kRows][TB];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int t = 0; t < TB; ++t)
      acc[i][t] = (f32x4){};
  const int blocks = (int)(a.k / 32);
  auto multiply = [&](int ch, int b) {
    const uint8_t* at = lds + (wave * BUFS + b) * B::kBytes;
    // (scale 0 past K: the layout's padding may hold anything, a NaN too)
    const uint32_t keep = 4 * ch + q < blocks ? 0xFFu : 0u;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      u32x4 w[kWords];
#pragma unroll
      for (int v = 0; v < kWords; ++v)
        w[v] = *reinterpret_cast<const u32x4*>(at + B::kW + (16 * i + c) * B::kRow +
                                               16 * ((kWords * q + v) ^ mm_swizzle<kPieces>(c)));
      const uint32_t byte = at[B::kS + 4 * (16 * i + c) + q] & keep;
      const float scale = __uint_as_float(byte << 23);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t f[4];
        if constexpr (kFp4) {
          f[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0][u], scale, 0));
          f[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0][u], scale, 1));
          f[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0][u], scale, 2));
          f[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0][u], scale, 3));
        } else {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint32_t d = w[u / 2][2 * (u % 2) + v];
            f[2 * v] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, scale, false));
            f[2 * v + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, scale, true));
          }
        }
        // a NaN block (the convert knows no scale 0xFF)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[e] = byte == 0xFF ? 0x7FC07FC0u : f[e];
        const bf16x8 wf = __builtin_bit_cast(bf16x8, (u32x4){f[0], f[1], f[2], f[3]});
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(at + B::kX + (16 * t + c) * 256 + 16 * ((4 * q + u) ^ c));
          acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8, x), acc[i][t], 0, 0, 0);
        }
      }
    }
  };
  // The wave's chunks are wave + KS i.  Every turn issues a chunk's loads (past
  // K they bring zeros), so that one count of loads tells when a chunk is there.
#pragma unroll
  for (int i = 0; i < BUFS - 1; ++i)
    load(wave + KS * i, i);
  int b = 0;
  for (int ch = wave; ch < chunks; ch += KS) {
    load(ch + KS * (BUFS - 1), b == 0 ? BUFS - 1 : b - 1);
    mm_wait_loads<(BUFS - 1) * B::kLoads>();
    mm_wave_fence();
    multiply(ch, b);
    mm_wave_fence();
    __builtin_amdgcn_s_waitcnt(0xC07F);   // its reads are done (lgkmcnt 0) before the buffer is loaded again
    b = b + 1 == BUFS ? 0 : b + 1;
  }
  mm_wait_loads<0>();
  __syncthreads();

  // Register v of lane l: column 4 (l / 16) + v, row l % 16 of its block.
  float* sums = reinterpret_cast<float*>(lds);   // [wave][block][block of x][v][lane]
  auto sum_at = [](int u, int i, int t, int v, int l) { return (((u * kRows + i) * TB + t) * 4 + v) * 64 + l; };
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        sums[sum_at(wave, i, t, v, lane)] = acc[i][t][v];
  __syncthreads();
  auto total = [&](int i, int t, int v, int l) {
    float f = 0.0f;
#pragma unroll
    for (int u = 0; u < KS; ++u)
      f += sums[sum_at(u, i, t, v, l)];
    return f;
  };
  // element e of the workgroup's 16 TB rows of 16 RB columns
  for (int e = threadIdx.x; e < 256 * TB * RB; e += 64 * KS) {
    const int row = e / (16 * RB), col = e % (16 * RB);
    if (row >= a.m || j0 + col >= a.n)
      continue;
    const int i = col / 16, l = 16 * (col % 16 / 4) + row % 16, v = col % 4, t = row / 16;
    float f = total(i, t, v, l);
    if constexpr (GATED) {
      const float u = total(RB + i, t, v, l);
      f = (a.gelu ? act_of<true>(f) : act_of<false>(f)) * u;
    }
    const int64_t at = (int64_t)row * a.n + j0 + col;
    if (a.f32)
      static_cast<float*>(a.c)[at] = f;
    else
      static_cast<uint16_t*>(a.c)[at] = (uint16_t)bf16_pair(f, f);
  }
}

// Two blocks of 16 rows of W to a workgroup (half the reads of x that one
// makes), two buffers to a wave, eight waves for up to 16 rows of x and four (or
// what LDS holds) above: one or two to a SIMD.  Timed (us, best to median): on
// MXFP4 weights of 8192 x 5120 one row 6.9-7.6 (3.2 TB/s), 16 rows 8.4-8.9, 32 rows
// 10.8-11.3, 33 rows of 5120 x 8192 15.2-17.0, 64 rows 19.3-21.8; on MXFP8 weights of
// 8192 x 5120 one row 9.2-9.9 (4.7 TB/s), 16 rows 9.4-10.9, 32 rows 10.6-11.9; gated,
// 2 x 4096 x 5120: 3 rows 6.8-7.6 and, MXFP8, 9.3-10.0, 33 rows 11.7-13.0 and 11.7-14.0,
// 64 rows 14.5-16.4.  The choices when they were made: 1 x 8192 x 5120 6.7 (one block
// 8.1, four waves 7.2, four blocks 7.9), 32 x 8192 x 5120 9.4 (one block 14.6, three
// buffers 10.0, seven waves 10.9), 33 x 5120 x 8192 14.7 (one block 25.7, two waves
// 22, five 14.6), 64 x 5120 x 8192 18.6 (two waves 33).  From 33 rows on x is four
// times the bytes of the workgroup's W, and every workgroup takes all of it: what
// bounds these is x through LDS, with 96 of 256 CUs idle at 5120 columns.  Cutting K
// over workgroups would use them, with a workspace for the partial sums.
template <int FW, int TB, bool GATED>
static void launch(const DecodeArgs& a, hipStream_t stream) {
  constexpr int RB = GATED ? 1 : 2, kBufs = 2;
  constexpr int kFit = 163840 / (kBufs * DecodeBuffer<FW, TB, RB, GATED>::kBytes);
  constexpr int KS = TB == 1 && kFit >= 8 ? 8 : kFit >= 4 ? 4 : kFit;
  hipLaunchKernelGGL((decode_kernel<FW, TB, RB, KS, kBufs, GATED>), dim3((unsigned)((a.n + 16 * RB - 1) / (16 * RB))),
                     dim3(64 * KS), 0, stream, a);
}

template <int FW, bool GATED>
static void launch_rows(const DecodeArgs& a, hipStream_t stream) {
  if (a.m <= 16)
    launch<FW, 1, GATED>(a, stream);
  else if (a.m <= 32)
    launch<FW, 2, GATED>(a, stream);
  else if (a.m <= 48)
    launch<FW, 3, GATED>(a, stream);
  else
    launch<FW, 4, GATED>(a, stream);
}

hipError_t launch_decode(const void* x, int64_t ldx, const uint8_t* qw, const uint8_t* sw, int32_t w_format, int64_t m,
                         int64_t n, int64_t k, bool gated, bool gelu, void* c, bool f32, hipStream_t stream) {
  const DecodeArgs a = {static_cast<const uint16_t*>(x), ldx, qw, sw, n, k, (int32_t)m, c, f32, gelu};
  if (w_format == MX_FORMAT_E2M1)
    gated ? launch_rows<MX_FORMAT_E2M1, true>(a, stream) : launch_rows<MX_FORMAT_E2M1, false>(a, stream);
  else
    gated ? launch_rows<MX_FORMAT_E4M3, true>(a, stream) : launch_rows<MX_FORMAT_E4M3, false>(a, stream);
  return hipGetLastError();
}

}  // namespace mx
