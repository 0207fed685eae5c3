// MXFP4 cast along dim0 and dim1, and the way back.
//
// For a block of 32 with largest magnitude amax: e = floor(log2 amax) - 2,
// clamped to [-127, 127] (amax 0: -127), code = x / 2^e rounded to the nearest
// e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6), ties to even, at most 6.  gfx950's scaled
// converts do that in one instruction for two values: the scale's exponent
// field is used as is, halves go to even, and they saturate (checked on MI355X
// over every bf16 pattern under scale bytes from 0 to 254).
//
// Bound by memory: 2 or 4 bytes read and 17/32 written to an element and
// direction.
#include "mx_fp4_launch.h"
#include "mx_train.h"
#include "mxfp4.h"

namespace mx {

struct Cast4Args {
  const void* x;
  int64_t batch, rows, cols, ldx;
  uint8_t *q0, *s0, *q1, *s1;
  bool blocked;
  uint32_t row_tiles, col_tiles;   // of a matrix
};

// N consecutive elements of a row as loaded, from any element on.
template <typename T, int N = 8>
struct Run {
  static constexpr int kWords = N * (int)sizeof(T) / 16;
  u32x4 w[kWords];
  // (streaming: 8192 x 5120 binary32 in both directions 47.8 -> 40.8 us, 16640 x
  // 5120 bf16 along rows 38.5 -> 36.8; along rows of binary32 66.6 -> 68.7)
  template <bool STREAM>
  __device__ __forceinline__ void load(const T* p) {
    typedef u32x4 Word __attribute__((aligned(2)));   // (of binary32 4)
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      w[i] = STREAM ? __builtin_nontemporal_load(reinterpret_cast<const Word*>(p) + i)
                    : reinterpret_cast<const Word*>(p)[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      w[i] = (u32x4){0, 0, 0, 0};
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i / 4][i % 4]);
    else
      return (i & 1) ? bf16_hi(w[0][i / 2]) : bf16_lo(w[0][i / 2]);
  }
  // the largest magnitude's binary32 bits (NaN above Inf above the rest)
  __device__ __forceinline__ uint32_t amax() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
        m = max(m, w[i / 4][i % 4] & 0x7FFFFFFFu);
      return m;
    } else {
      const uint32_t m = max2(max2(mag2(w[0][0]), mag2(w[0][1])), max2(mag2(w[0][2]), mag2(w[0][3])));
      return max(m & 0xFFFFu, m >> 16) << 16;
    }
  }
};

// The scale byte of an amax given as binary32 magnitude bits, by the rule of
// the 8-bit casts with e2m1's largest exponent: 254 for a block with an Inf,
// 0xFF for one with a NaN.
__device__ __forceinline__ uint32_t scale4(uint32_t amax) {
  const uint32_t e = amax >> 23;
  if (amax >= 0x7F800000u)
    return amax == 0x7F800000u ? 254u : 255u;
  return e > 2 ? e - 2 : 0;
}
// Two elements -> codes in byte SEL of `old`.  A NaN block's codes are 0.
template <int SEL>
__device__ __forceinline__ uint32_t pair4(uint32_t old, float lo, float hi, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, lo, hi, scale, SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t pair4(uint32_t old, uint32_t bf16s, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, bf16s), scale, SEL);
}
// N codes, the first in the lowest bits.
template <typename T, int N>
__device__ __forceinline__ uint32_t codes(const Run<T, N>& d, uint32_t byte) {
  const float scale = __uint_as_float(byte << 23);
  uint32_t q = 0;
  if constexpr (sizeof(T) == 4) {
    q = pair4<0>(q, d.get(0), d.get(1), scale);
    q = pair4<1>(q, d.get(2), d.get(3), scale);
    if constexpr (N == 8) {
      q = pair4<2>(q, d.get(4), d.get(5), scale);
      q = pair4<3>(q, d.get(6), d.get(7), scale);
    }
  } else {
    q = pair4<0>(q, d.w[0][0], scale);
    q = pair4<1>(q, d.w[0][1], scale);
    q = pair4<2>(q, d.w[0][2], scale);
    q = pair4<3>(q, d.w[0][3], scale);
  }
  return byte == 0xFF ? 0u : q;
}

// Where scale (r, c) of a matrix of `strips`-byte 128-row strips lies in the
// blocked layout.
__device__ __forceinline__ int64_t blocked_at(int64_t r, int64_t c, int64_t strip) {
  return r / 128 * strip + c / 4 * 512 + 16 * (r % 32) + 4 * (r % 128 / 32) + c % 4;
}

constexpr int kCast4Threads = 256;

// dim0 alone: a lane owns eight columns of a row, a quad a block.  Of bf16 a lane
// has two of those, whose loads are on their way together (16640 x 5120: 44.0 ->
// 36.8 us, 5.9 TB/s; 34.7-37.4 on others); of binary32, 32 bytes each, one (66.6 us, 5.8
// TB/s, two 69.7; 73-76 on others).  Blocked scales: the lanes also cover the layout's padding, whose bytes
// they clear.
template <typename T>
constexpr int kCast4Runs = sizeof(T) == 2 ? 2 : 1;
template <typename T>
__global__ __launch_bounds__(kCast4Threads) void cast4_rows_kernel(Cast4Args a) {
  const uint32_t blocks = (uint32_t)(a.cols / 32), pblocks = a.blocked ? (blocks + 3) / 4 * 4 : blocks;
  const uint32_t prows = (uint32_t)(a.blocked ? (a.rows + 127) / 128 * 128 : a.rows), units = pblocks * 4;
  const uint32_t all = (uint32_t)a.batch * prows;
  constexpr int kRuns = kCast4Runs<T>;
  Run<T> d[kRuns];
  uint32_t row[kRuns], r[kRuns], c[kRuns];
  bool on[kRuns];
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const uint32_t unit = (blockIdx.x * kRuns + i) * kCast4Threads + threadIdx.x;
    row[i] = unit / units;   // of all matrices; whole quads (units is a multiple of 4)
    c[i] = (unit - row[i] * units) * 8;
    r[i] = row[i] % prows;
    on[i] = row[i] < all && r[i] < a.rows && c[i] < a.cols;
    d[i].clear();
    if (on[i])
      d[i].template load<sizeof(T) == 2>(static_cast<const T*>(a.x) + ((int64_t)(row[i] / prows) * a.rows + r[i]) * a.ldx + c[i]);
  }
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const int64_t b = row[i] / prows;
    uint32_t m = d[i].amax();
    m = max(m, quad_swap1(m));
    m = max(m, quad_swap2(m));
    const uint32_t byte = on[i] ? scale4(m) : 0;
    if (on[i])
      *reinterpret_cast<uint32_t*>(a.q0 + ((b * a.rows + r[i]) * a.cols + c[i]) / 2) = codes(d[i], byte);
    if ((threadIdx.x & 3) == 0 && row[i] < all) {
      const int64_t at = a.blocked ? b * prows * pblocks + blocked_at(r[i], c[i] / 32, (int64_t)pblocks * 128)
                                   : (int64_t)row[i] * blocks + c[i] / 32;
      a.s0[at] = (uint8_t)byte;
    }
  }
}

// Both directions, or dim1 alone: a workgroup of four waves owns 128 rows of 32 C
// columns, a wave 32 rows of them, a lane 16 rows of C columns, 16 bytes each,
// so that a block along the rows is 32 / C lanes' and one along the columns two
// lanes'.  Column codes and all scales leave through LDS: 64 bytes of a column's
// codes and four scales (a word of the blocked layout) at a time.  16640 x 5120
// bf16 49-53 us (4.9-5.3 TB/s; 61 on a slower card), 8192 x 5120 binary32 38-40
// (5.3-5.6 TB/s; eight columns to a lane took 158 registers, one workgroup to a CU:
// 62, where this took 41).  Eight waves and 128 bytes
// a column are even there and slower on small matrices (2048 x 2048 8.9 -> 9.9
// us); tiles in pieces per XCD, along rows or columns, gained nothing.
constexpr int kCast4Waves = 4, kCast4Rows = 32 * kCast4Waves;
constexpr int kCast4Pitch = kCast4Rows / 2 + 16;
template <typename T>
constexpr int kCast4Cols = 32 * 16 / (int)sizeof(T);

template <typename T>
__global__ __launch_bounds__(64 * kCast4Waves) void cast4_both_kernel(Cast4Args a) {
  constexpr int C = 16 / (int)sizeof(T), kCols = 32 * C;
  __shared__ __attribute__((aligned(16))) uint8_t qt[kCols * kCast4Pitch];
  __shared__ __attribute__((aligned(16))) uint8_t sr[kCast4Rows][kCols / 32], sc[kCols][kCast4Rows / 32];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t tiles = a.row_tiles * a.col_tiles;
  const int64_t b = blockIdx.x / tiles;
  const uint32_t tile = blockIdx.x % tiles;
  const int64_t row0 = (int64_t)(tile / a.col_tiles) * kCast4Rows, col0 = (int64_t)(tile % a.col_tiles) * kCols;
  const int lr = 32 * wave + 16 * (lane >> 5), lc = C * (lane & 31);
  const bool on = row0 + lr < a.rows && col0 + lc < a.cols;
  const T* x = static_cast<const T*>(a.x) + (b * a.rows + row0 + lr) * a.ldx + col0 + lc;
  Run<T, C> d[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    d[i].clear();
    if (on)
      d[i].template load<true>(x + i * a.ldx);
  }
  if (a.q0 != nullptr) {
    uint8_t* q0 = a.q0 + ((b * a.rows + row0 + lr) * a.cols + col0 + lc) / 2;
    uint32_t before = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint32_t m = d[i].amax();
      m = max(m, quad_swap1(m));
      m = max(m, quad_swap2(m));
      if constexpr (C == 4)
        m = max(m, half_row_mirror(m));
      const uint32_t byte = on ? scale4(m) : 0, q = codes(d[i], byte);
      if constexpr (C == 8) {
        if (on)
          *reinterpret_cast<uint32_t*>(q0 + i * (a.cols / 2)) = q;
      } else if (i % 2 == 0) {
        before = q;
      } else {
        // two rows' 2 bytes of two lanes: the even lane stores the first row's
        // 4 bytes, the odd lane the second's
        const bool odd = lane & 1;
        const uint32_t other = quad_swap1(odd ? before : q);
        if (on)
          *reinterpret_cast<uint32_t*>(q0 + (odd ? i * (a.cols / 2) - 2 : (i - 1) * (a.cols / 2))) =
              odd ? other | (q << 16) : before | (other << 16);
      }
      if ((lane & (32 / C - 1)) == 0)
        sr[lr + i][(lane & 31) * C / 32] = (uint8_t)byte;
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      m = max(m, __float_as_uint(d[i].get(c)) & 0x7FFFFFFFu);
    const auto o = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    const uint32_t byte = on ? scale4(max(o[0], o[1])) : 0;
    const float scale = __uint_as_float(byte << 23);
    u32x2 q = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q[i] = pair4<0>(q[i], d[8 * i].get(c), d[8 * i + 1].get(c), scale);
      q[i] = pair4<1>(q[i], d[8 * i + 2].get(c), d[8 * i + 3].get(c), scale);
      q[i] = pair4<2>(q[i], d[8 * i + 4].get(c), d[8 * i + 5].get(c), scale);
      q[i] = pair4<3>(q[i], d[8 * i + 6].get(c), d[8 * i + 7].get(c), scale);
    }
    if (byte == 0xFF)
      q = (u32x2){0, 0};
    *reinterpret_cast<u32x2*>(qt + (lc + c) * kCast4Pitch + lr / 2) = q;
    if (lane < 32)
      sc[lc + c][wave] = (uint8_t)byte;
  }
  __syncthreads();
  // rows are multiples of 32: a word holds whole blocks
#pragma unroll
  for (int i = 0; i < kCols / 64; ++i) {   // 16 bytes a thread, kCast4Waves of them a column
    const int c = 64 * i + threadIdx.x / kCast4Waves, byte = 16 * (threadIdx.x % kCast4Waves);
    if (col0 + c < a.cols && row0 + 2 * byte < a.rows)
      *reinterpret_cast<u32x4*>(a.q1 + ((b * a.cols + col0 + c) * a.rows + row0) / 2 + byte) =
          *reinterpret_cast<const u32x4*>(qt + c * kCast4Pitch + byte);
  }
  // four scales a thread: blocks `first` on of a line (a row, or a column)
  auto scales = [&](uint8_t* s, const uint8_t* from, int64_t line, int64_t lines, int64_t first, int64_t blocks) {
    const uint32_t word = *reinterpret_cast<const uint32_t*>(from);
    if (a.blocked) {
      const int64_t pl = (lines + 127) / 128 * 128, pb = (blocks + 3) / 4 * 4;
      if (line < pl && first < pb)
        *reinterpret_cast<uint32_t*>(s + b * pl * pb + blocked_at(line, first, pb * 128)) = word;
    } else if (line < lines) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (first + i < blocks)
          s[(b * lines + line) * blocks + first + i] = (uint8_t)(word >> (8 * i));
    }
  };
  constexpr int kRowWords = kCols / 128, kColWords = kCast4Waves / 4;   // words of a line's scales
  if (a.q0 != nullptr)
    for (int t = threadIdx.x; t < kCast4Rows * kRowWords; t += 64 * kCast4Waves)
      scales(a.s0, &sr[t / kRowWords][4 * (t % kRowWords)], row0 + t / kRowWords, a.rows,
             col0 / 32 + 4 * (t % kRowWords), a.cols / 32);
  for (int t = threadIdx.x; t < kCols * kColWords; t += 64 * kCast4Waves)
    scales(a.s1, &sc[t / kColWords][4 * (t % kColWords)], col0 + t / kColWords, a.cols,
           row0 / 32 + 4 * (t % kColWords), a.rows / 32);
}

static Cast4Args cast4_args(int64_t batch, int64_t rows, int64_t cols, int tile_cols) {
  Cast4Args a = {};
  a.batch = batch, a.rows = rows, a.cols = cols;
  a.row_tiles = (uint32_t)((rows + kCast4Rows - 1) / kCast4Rows);
  a.col_tiles = (uint32_t)((cols + tile_cols - 1) / tile_cols);
  return a;
}

static int64_t rows_blocks(int64_t batch, int64_t rows, int64_t cols, bool blocked, int runs) {
  const int64_t b = cols / 32, pb = blocked ? (b + 3) / 4 * 4 : b, pr = blocked ? (rows + 127) / 128 * 128 : rows;
  return (batch * pr * pb * 4 + kCast4Threads * runs - 1) / (kCast4Threads * runs);
}

hipError_t launch_cast4(const void* x, int64_t batch, int64_t rows, int64_t cols, int64_t ldx, bool f32, uint8_t* q0,
                        uint8_t* s0, uint8_t* q1, uint8_t* s1, bool blocked, hipStream_t stream) {
  Cast4Args a = cast4_args(batch, rows, cols, f32 ? kCast4Cols<float> : kCast4Cols<uint16_t>);
  a.x = x, a.ldx = ldx, a.q0 = q0, a.s0 = s0, a.q1 = q1, a.s1 = s1, a.blocked = blocked;
  if (q1 == nullptr) {
    const int runs = f32 ? kCast4Runs<float> : kCast4Runs<uint16_t>;
    const dim3 grid((unsigned)rows_blocks(batch, rows, cols, blocked, runs)), threads(kCast4Threads);
    if (f32)
      hipLaunchKernelGGL(cast4_rows_kernel<float>, grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL(cast4_rows_kernel<uint16_t>, grid, threads, 0, stream, a);
  } else {
    const dim3 grid((unsigned)(batch * a.row_tiles * a.col_tiles)), threads(64 * kCast4Waves);
    if (f32)
      hipLaunchKernelGGL(cast4_both_kernel<float>, grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL(cast4_both_kernel<uint16_t>, grid, threads, 0, stream, a);
  }
  return hipGetLastError();
}

// Back: a lane turns eight codes into 16 or 32 bytes.  Every value is a bf16
// number (or, above byte 252, past its range: Inf).  Bound by memory: 8192 x
// 5120 to bf16 19-20 us (5.3-5.6 TB/s), 16640 x 5120 34-39 (5.5-6.3 TB/s), to binary32
// 82-84 (4.6-4.7 TB/s).
template <bool F32>
__global__ __launch_bounds__(kCast4Threads) void dequantize4_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                                    int64_t batch, int64_t rows, int64_t cols,
                                                                    bool blocked, void* __restrict__ x) {
  const int64_t unit = (int64_t)blockIdx.x * kCast4Threads + threadIdx.x, units = cols / 8;
  const int64_t row = unit / units;
  if (row >= batch * rows)
    return;
  const int64_t blk = (unit - row * units) / 4, blocks = cols / 32;
  int64_t at = row * blocks + blk;
  if (blocked) {
    const int64_t pb = (blocks + 3) / 4 * 4, b = row / rows;
    at = b * ((rows + 127) / 128 * 128) * pb + blocked_at(row - b * rows, blk, pb * 128);
  }
  const uint32_t byte = s[at], c = reinterpret_cast<const uint32_t*>(q)[unit];
  const float scale = __uint_as_float(byte << 23);
  if constexpr (F32) {
    f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1),
                  __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3)};
    f32x4* out = static_cast<f32x4*>(x) + 2 * unit;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f32x4 o = {v[2 * i][0], v[2 * i][1], v[2 * i + 1][0], v[2 * i + 1][1]};
      if (byte == 0xFF)
        o = (f32x4)(__uint_as_float(0x7FC00000u));
      out[i] = o;
    }
  } else {
    u32x4 o = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3))};
    if (byte == 0xFF)
      o = (u32x4)(0x7FC07FC0u);
    static_cast<u32x4*>(x)[unit] = o;
  }
}

hipError_t launch_dequantize4(const uint8_t* q, const uint8_t* s, int64_t batch, int64_t rows, int64_t cols,
                              bool blocked, void* x, bool f32, hipStream_t stream) {
  const dim3 grid((unsigned)((batch * rows * (cols / 8) + kCast4Threads - 1) / kCast4Threads)), threads(kCast4Threads);
  if (f32)
    hipLaunchKernelGGL(dequantize4_kernel<true>, grid, threads, 0, stream, q, s, batch, rows, cols, blocked, x);
  else
    hipLaunchKernelGGL(dequantize4_kernel<false>, grid, threads, 0, stream, q, s, batch, rows, cols, blocked, x);
  return hipGetLastError();
}

}  // namespace mx
