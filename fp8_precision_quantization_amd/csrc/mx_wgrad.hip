// Weight gradient of a linear layer from the 8-bit checkpoint of its input:
//
//   dw_g[i][j] = sum over tokens t of group g of dy[t][i] * x[t][j],
//   x[t][j] = e4m3(q[t][j]) * 2^(s[t][j / 32] - 127).
//
// The sum runs over tokens, along which a checkpoint's scales change from
// element to element of a column, so the block-scaled MFMA does not apply:
// the codes are turned into bf16 (exact: four significant bits times a power
// of two) and the product runs on v_mfma_f32_32x32x16_bf16 with binary32
// accumulators.
//
// Work decomposition.  A 256-thread workgroup owns a 256 x 256 tile of one
// group's dw; wave w its (w / 2, w % 2) 128 x 128 quarter, 4 x 4 MFMA blocks.
// Tokens advance in stages of 64: the stage's 64 x 256 pieces of dy and x sit
// in LDS as bf16, token-major as in memory, double-buffered.  dy comes
// straight from memory into LDS (16 bytes per lane); the codes come through
// registers, where they are converted.
//
// An MFMA operand wants eight consecutive tokens of one column in a lane,
// which is down a column of the stage: gfx950's transposing LDS read delivers
// it.  ds_read_b64_tr_b16, its lane layout checked on MI355X: within each 16
// lanes, lane i addresses 8 bytes, and receives as element e the (i % 4)-th
// 16-bit value of the 8 bytes lane 4 e + i / 4 addressed; so with lane i on
// token i / 4, columns 4 (i % 4) .. + 3, lane i ends with column i of four
// tokens.  Two such reads make an operand.
//
// A stage row is 512 bytes, a multiple of the banks' period, and one read
// touches four tokens: the row's eight 64-byte pieces are permuted by the
// token, piece p at p ^ (token % 4), so that the four land on distinct banks.
//
// Rows past the end of the token range load as zero in both operands; columns
// past n or k may hold anything: they only reach outputs that are not stored.
#include "mx_train.h"
#include "mx_train_launch.h"
#include "mxtrain.h"

#include <type_traits>

namespace mx {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

constexpr int kWgThreads = 256;
constexpr int kWgTile = 256;
constexpr int kWgTokens = 64;                        // tokens per stage
constexpr int kWgRow = kWgTile * 2;                  // bytes of a stage row
constexpr int kWgHalf = kWgTokens * kWgRow;          // one operand's stage
constexpr int kWgBlocks = 4;                         // 32 x 32 blocks per wave each way

struct WgradArgs {
  const uint16_t* dy;
  const uint8_t *q, *s;
  const int32_t* ends;
  void* out;          // dw, or the pieces' sums
  int64_t lddy, n, k;
  int32_t rows, groups, splits;
  uint32_t tiles_n, tiles_k, per_xcd, total;
};

// Token range of group g: [min(max(0, ends_0 .. ends_{g-1}), rows), min(max(0,
// ends_0 .. ends_g), rows)), found by one wave's lanes together.
__device__ __forceinline__ void group_range(const int32_t* ends, int g, int32_t rows, int32_t& lo, int32_t& hi) {
  int32_t run = 0;
  for (int i = threadIdx.x & 63; i < g; i += 64)
    run = max(run, ends[i]);
  run = (int32_t)lanes_max<64>((uint32_t)run);   // not negative
  lo = __builtin_amdgcn_readfirstlane(min(run, rows));
  hi = __builtin_amdgcn_readfirstlane(min(max(run, ends[g]), rows));
}

// 16 bytes per lane from memory into LDS, in lane order from `to` on (the same
// in every lane).  As the compiler's own form of it, every later read from LDS
// would wait for the load, since the transposing reads carry nothing that
// tells the two halves apart; here the caller waits (vmcnt) and meets the
// other waves at a barrier before anything is read.  (m0, which holds the LDS
// address, is not a register the compiler keeps values in.)
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rsrc, const uint8_t* to, int offset) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)to;
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"(__builtin_amdgcn_readfirstlane(at)), "v"(offset), "s"(rsrc)
      : "memory");
}

template <bool VEC, bool BF16>
__global__ __launch_bounds__(kWgThreads) void wgrad_kernel(WgradArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][2][kWgHalf];   // [stage][dy, x]
  const uint32_t id = (blockIdx.x % 8) * a.per_xcd + blockIdx.x / 8;
  if (id >= a.total)
    return;   // uniform, before any barrier
  const uint32_t tiles = a.tiles_n * a.tiles_k;
  const uint32_t piece = id / tiles, tile = id % tiles;
  const int g = (int)(piece % (uint32_t)a.groups), split = (int)(piece / (uint32_t)a.groups);
  const int64_t i0 = (int64_t)(tile / a.tiles_k) * kWgTile, j0 = (int64_t)(tile % a.tiles_k) * kWgTile;

  int32_t lo = 0, hi = a.rows;
  if (a.ends != nullptr)
    group_range(a.ends, g, a.rows, lo, hi);
  if (a.splits > 1) {
    const int32_t each = ((hi - lo + a.splits - 1) / a.splits + kWgTokens - 1) / kWgTokens * kWgTokens;
    const int64_t first = lo + (int64_t)split * each;
    hi = (int32_t)min((int64_t)hi, first + each);
    lo = (int32_t)min((int64_t)hi, first);
  }

  const int t = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lane = t & 63;
  const int wi = wave >> 1, wj = wave & 1;
  const int stages = (hi - lo + kWgTokens - 1) / kWgTokens;
  const int64_t ks = a.k / MX_BLOCK;

  v16f acc[kWgBlocks][kWgBlocks];
#pragma unroll
  for (int i = 0; i < kWgBlocks; ++i)
#pragma unroll
    for (int j = 0; j < kWgBlocks; ++j)
      acc[i][j] = (v16f){};

  // Loader roles.  dy: load u of wave w fills rows 8 u + 2 w, + 1; lane l the
  // 16 bytes at position l % 32 of row 8 u + 2 w + l / 32, which hold chunk
  // (l % 32) ^ 4 (row % 4).  Codes: load u of thread t is row 16 u + t / 16,
  // columns 16 (t % 16) .. + 15.
  const int drow = 2 * wave + lane / 32;
  const int dchunk = (lane % 32) ^ ((drow & 3) << 2);
  const int xrow = t / 16, xcol = 16 * (t % 16);
  const int x_at = xrow * kWgRow + 16 * (((xcol / 8) ^ ((xrow & 3) << 2)) ^ ((xcol / 8) >> 4));   // the other chunk: ^ 16
  const int64_t dy_last = (int64_t)(a.rows - 1) * a.lddy + a.n;   // elements of dy
  u32x4 codes[4], dreg[VEC ? 1 : 8];
  uint32_t scales[4];

  // dy of stage st: straight into LDS half h, or into registers.
  auto load_dy = [&](auto h_c, int st) {
    constexpr int h = decltype(h_c)::value;
    const int32_t m0 = lo + st * kWgTokens;
    const int32_t left = min(hi - m0, kWgTokens);   // may be <= 0: nothing in range
    if constexpr (VEC) {
      const int64_t bytes = left > 0 ? ((left - 1) * a.lddy + (a.n - i0)) * 2 : 0;
      const __amdgpu_buffer_rsrc_t rd = buffer_rsrc(a.dy + (left > 0 ? m0 : 0) * a.lddy + i0, (uint32_t)bytes);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        load_to_lds(rd, lds[h][0] + (8 * u + 2 * wave) * kWgRow, (8 * u + drow) * (int)a.lddy * 2 + 16 * dchunk);
    } else {
      // 16 bytes at any alignment; what lies past column n belongs to columns
      // that are not stored.  Only at the very end of dy, element by element.
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int row = 8 * u + drow;
        const int64_t c = i0 + 8 * dchunk;
        dreg[u] = (u32x4){0, 0, 0, 0};
        if (row < left && c < a.n) {
          const int64_t at = (int64_t)(m0 + row) * a.lddy + c;
          if (at + 8 <= dy_last) {
            dreg[u] = *reinterpret_cast<const u32x4_any*>(a.dy + at);
          } else {
            for (int e = 0; e < dy_last - at; ++e)
              dreg[u][e / 2] |= (uint32_t)a.dy[at + e] << (16 * (e & 1));
          }
        }
      }
    }
  };
  auto load_codes = [&](int st) {
    const int32_t m0 = lo + st * kWgTokens;
    const int32_t left = min(hi - m0, kWgTokens);
    const int64_t qbytes = left > 0 ? (left - 1) * a.k + (a.k - j0) : 0;
    const int64_t sbytes = left > 0 ? (left - 1) * ks + (ks - j0 / MX_BLOCK) : 0;
    const __amdgpu_buffer_rsrc_t rq = buffer_rsrc(a.q + (left > 0 ? m0 : 0) * a.k + j0, (uint32_t)qbytes);
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(a.s + (left > 0 ? m0 : 0) * ks + j0 / MX_BLOCK, (uint32_t)sbytes);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      codes[u] = __builtin_amdgcn_raw_buffer_load_b128(rq, (16 * u + xrow) * (int)a.k + xcol, 0, 0);
      scales[u] = __builtin_amdgcn_raw_buffer_load_b8(rs, (16 * u + xrow) * (int)ks + xcol / MX_BLOCK, 0, 0);
    }
  };
  // Half e (eight codes) of code load u into LDS half h as bf16.
  auto put_codes = [&](auto h_c, int u, int e) {
    constexpr int h = decltype(h_c)::value;
    const float sc = __uint_as_float(scales[u] << 23);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[u][2 * e + i], sc, false));
      w[2 * i + 1] =
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[u][2 * e + i], sc, true));
    }
    *reinterpret_cast<u32x4*>(lds[h][1] + 16 * u * kWgRow + (x_at ^ (16 * e))) = (u32x4){w[0], w[1], w[2], w[3]};
  };
  auto put_dy = [&](auto h_c) {
    constexpr int h = decltype(h_c)::value;
    if constexpr (!VEC) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        *reinterpret_cast<u32x4*>(lds[h][0] + (8 * u + drow) * kWgRow + 16 * (lane % 32)) = dreg[u];
    }
  };

  // MFMA role: lane l reads token 8 (l / 32) + (l % 16) / 4 (+ 4), columns 16
  // ((l / 16) % 2) + 4 (l % 4) .. + 3 of a block.
  const int tok = 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int sub = 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
  int a_at[kWgBlocks], b_at[kWgBlocks];
#pragma unroll
  for (int b = 0; b < kWgBlocks; ++b) {
    a_at[b] = tok * kWgRow + 64 * ((4 * wi + b) ^ (tok & 3)) + sub;
    b_at[b] = tok * kWgRow + 64 * ((4 * wj + b) ^ (tok & 3)) + (sub ^ (16 * wj));
  }
  typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
  typedef s16x4 Step[2 * kWgBlocks][2];   // operands of 16 tokens: dy blocks, then x blocks, two reads each
  // Read r (0 .. 15) of step `step` from LDS half h, in the order the MFMAs
  // use the operands: dy 0, x 0 .. 3, dy 1 .. 3.
  auto read_one = [&](auto h_c, int step, int r, Step& f) {
    constexpr int h = decltype(h_c)::value;
    const int o = r / 2, e = r % 2;
    const bool is_x = o >= 1 && o <= kWgBlocks;
    const int b = o == 0 ? 0 : is_x ? o - 1 : o - kWgBlocks;
    const int at = (is_x ? b_at[b] : a_at[b]) + (16 * step + 4 * e) * kWgRow;
    f[is_x ? kWgBlocks + b : b][e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(lds[h][is_x] + at));
  };
  auto operand = [](const s16x4 (&f)[2]) {
    return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(f[0], f[1], 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto mfma = [&](int m, const Step& f) {
    const int i = m / kWgBlocks, j = m % kWgBlocks;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(f[i]), operand(f[kWgBlocks + j]), acc[i][j], 0, 0, 0);
  };

  // A stage is four steps of 16 tokens, 16 MFMAs each; there is one wave to a
  // SIMD, so nothing but this order hides a wait.  While a step's MFMAs run,
  // the next step's operands are read from LDS, two reads after each of the
  // first eight.  Before step 2 the wave waits for its loads of the next
  // stage, which have had three steps; step 2 turns the codes into bf16 in the
  // other LDS half.  The reads and writes of step 2 are done a few MFMAs
  // before its end, so that the stage's one barrier, between steps 2 and 3,
  // costs little.  Step 3 reads the next stage's first operands, and the loads
  // of the stage after that go into the half that the barrier has freed.
  auto stage = [&](auto h_c, int st, Step& f0, Step& f1) {
    constexpr int h = decltype(h_c)::value;
    using H = std::integral_constant<int, h>;
    using O = std::integral_constant<int, h ^ 1>;
    constexpr int kM = kWgBlocks * kWgBlocks;
    auto step = [&](auto from, int next, const Step& now, Step& then, bool put) {
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        mfma(m, now);
        if (m < kM / 2) {
          read_one(from, next, 2 * m, then);
          read_one(from, next, 2 * m + 1, then);
        }
        if (put && m >= 4 && m < 12)
          put_codes(O(), (m - 4) / 2, (m - 4) % 2);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    step(H(), 1, f0, f1, false);
    step(H(), 2, f1, f0, false);
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    put_dy(O());
    step(H(), 3, f0, f1, true);
    lds_barrier();
    load_dy(H(), st + 2);
    load_codes(st + 2);
    __builtin_amdgcn_sched_barrier(0);
    step(O(), 0, f1, f0, false);
  };
  if (stages > 0) {
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    Step f0, f1;
    load_dy(S0(), 0);
    load_codes(0);
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
#pragma unroll
    for (int u = 0; u < 8; ++u)
      put_codes(S0(), u / 2, u % 2);
    put_dy(S0());
    load_dy(S1(), 1);
    load_codes(1);
    lds_barrier();
#pragma unroll
    for (int r = 0; r < 4 * kWgBlocks; ++r)
      read_one(S0(), 0, r, f0);
    // stages past the last (an odd count runs one) load zeros and add nothing
    for (int st = 0; st < stages; st += 2) {
      stage(S0(), st, f0, f1);
      stage(S1(), st + 1, f0, f1);
    }
    // loads into LDS still in flight must land before it is used again
    __builtin_amdgcn_s_waitcnt(0x0F70);
  }

  // register v of lane l: row 8 (v / 4) + 4 (l / 32) + v % 4, column l % 32
  const int64_t plane = ((int64_t)split * a.groups + g) * a.n;
#pragma unroll
  for (int j = 0; j < kWgBlocks; ++j) {
    const int64_t col = j0 + wj * 128 + 32 * j + (lane & 31);
    if (col >= a.k)
      continue;
#pragma unroll
    for (int i = 0; i < kWgBlocks; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t row = i0 + wi * 128 + 32 * i + 8 * (v / 4) + 4 * (lane >> 5) + v % 4;
        if (row < a.n) {
          const int64_t at = (plane + row) * a.k + col;
          if constexpr (BF16)
            static_cast<uint16_t*>(a.out)[at] = (uint16_t)bf16_pair(acc[i][j][v], 0.0f);
          else
            static_cast<float*>(a.out)[at] = acc[i][j][v];
        }
      }
  }
}

// dw = the sum of the pieces, in order; four elements to a thread.
template <bool BF16>
__global__ __launch_bounds__(256) void wgrad_fold_kernel(const float* part, int32_t splits, int64_t elems, void* dw) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= elems)
    return;   // elems is a multiple of 32
  f32x4 sum = *reinterpret_cast<const f32x4*>(part + at);
#pragma unroll 4
  for (int s = 1; s < splits; ++s)
    sum += *reinterpret_cast<const f32x4*>(part + s * elems + at);
  if constexpr (BF16) {
    const u32x2 w = {bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
    uint16_t* p = static_cast<uint16_t*>(dw) + at;
    p[0] = (uint16_t)w[0], p[1] = (uint16_t)(w[0] >> 16), p[2] = (uint16_t)w[1], p[3] = (uint16_t)(w[1] >> 16);
  } else {
    float* p = static_cast<float*>(dw) + at;
    p[0] = sum[0], p[1] = sum[1], p[2] = sum[2], p[3] = sum[3];
  }
}

static int64_t wgrad_tiles(int64_t n, int64_t k, int32_t groups) {
  return ((n + kWgTile - 1) / kWgTile) * ((k + kWgTile - 1) / kWgTile) * groups;
}

// Pieces of the token axis: enough to give every CU a tile, as long as a
// piece keeps about four stages (of the groups' average length).
static int32_t wgrad_splits(int64_t rows, int64_t n, int64_t k, int32_t groups) {
  const int64_t tiles = wgrad_tiles(n, k, groups);
  if (tiles == 0 || tiles > 128)
    return 1;
  const int64_t by_cus = 256 / tiles, by_rows = rows / groups / (4 * kWgTokens);
  const int64_t s = by_cus < by_rows ? by_cus : by_rows;
  return s < 1 ? 1 : (int32_t)s;
}

int64_t wgrad_workspace_bytes(int64_t rows, int64_t n, int64_t k, int32_t groups) {
  const int32_t s = wgrad_splits(rows, n, k, groups);
  return s > 1 ? s * groups * n * k * 4 : 0;
}

int64_t wgrad_grid_blocks(int64_t rows, int64_t n, int64_t k, int32_t groups) {
  const int64_t total = wgrad_tiles(n, k, groups) * wgrad_splits(rows, n, k, groups);
  return (total + 7) / 8 * 8;
}

hipError_t launch_wgrad(const void* dy, int64_t lddy, const uint8_t* q, const uint8_t* s, int64_t rows, int64_t n,
                        int64_t k, const int32_t* ends, int32_t groups, void* dw, bool bf16, float* workspace,
                        bool vec, hipStream_t stream) {
  WgradArgs a = {};
  a.dy = static_cast<const uint16_t*>(dy), a.lddy = lddy, a.q = q, a.s = s, a.ends = ends, a.n = n, a.k = k;
  a.rows = (int32_t)rows, a.groups = groups, a.splits = wgrad_splits(rows, n, k, groups);
  a.tiles_n = (uint32_t)((n + kWgTile - 1) / kWgTile), a.tiles_k = (uint32_t)((k + kWgTile - 1) / kWgTile);
  a.total = (uint32_t)(wgrad_tiles(n, k, groups) * a.splits);
  a.per_xcd = (a.total + 7) / 8;
  const dim3 grid(a.per_xcd * 8), threads(kWgThreads);
  const bool half = bf16 && a.splits == 1;
  a.out = a.splits > 1 ? workspace : dw;
  if (vec) {
    if (half)
      hipLaunchKernelGGL((wgrad_kernel<true, true>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((wgrad_kernel<true, false>), grid, threads, 0, stream, a);
  } else {
    if (half)
      hipLaunchKernelGGL((wgrad_kernel<false, true>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((wgrad_kernel<false, false>), grid, threads, 0, stream, a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1)
    return e;
  const int64_t elems = groups * n * k;
  const dim3 fold((unsigned)((elems / 4 + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL((wgrad_fold_kernel<true>), fold, dim3(256), 0, stream, workspace, a.splits, elems, dw);
  else
    hipLaunchKernelGGL((wgrad_fold_kernel<false>), fold, dim3(256), 0, stream, workspace, a.splits, elems, dw);
  return hipGetLastError();
}

}  // namespace mx
