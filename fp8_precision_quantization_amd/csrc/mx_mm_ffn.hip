// The gated feed-forward block on MX operands: both projections, the
// activation and the product in one kernel, and its gradient.
//
// Forward: g = x Wg^T and u = x Wu^T stand in the same wave's accumulators
// (mx_mm.h, gated), so that y = act(g) u needs neither in memory:
// 8 bytes an element of y less than a product and the activation after it.
// The 8-bit checkpoint of (g, u) that the gradient reads is formed from the
// accumulators themselves: a block of 32 columns of a row is two lanes'
// registers.
//
// Backward: dy = do Wd, whose tile stays in the accumulators; the checkpoint's
// codes of the same tile come through LDS; dg = dy u act'(g), du = dy act(g).
//
// Timed at 16640 rows, 4096 columns, k 5120 (us, best to median): block in MXFP8
// with the checkpoint 536-621 (2.2-2.6 PFLOP/s), MXFP8 rows and MXFP4 weights
// 523-571, in MXFP4 380-408; gradient in MXFP8 331-359, MXFP4 weights 306-330, in
// MXFP4 with y again 270-292.  In 8 uneven groups: block 626-682 and 398-450,
// gradient 367-410 and 285-320 (a part-filled round and cut tiles to a group).
// Without their epilogues (copies): block in MXFP8 574 -> 508, in MXFP4 380 -> 313,
// gradient in MXFP8 334 -> 257, in MXFP4 269 -> 164: a workgroup has a CU to itself
// (its sums are half of the CU's registers), so nothing covers an epilogue, 300
// to 540 KB of loads and stores a tile.  Two workgroups of 128 x 128 a CU cover
// each other's, but load each operand twice as often: 710 for the block, 432 for
// its gradient in MXFP8, where large tiles took 585 and 376.  Four waves of 128 x
// 128 to a large tile, as the products take them, leave one wave a SIMD to run
// the epilogue: 626 and 417 then.  (Both
// were timed in MXFP8, with bands of eight tile rows and no quarters; the four
// waves in MXFP4 too, 503 against 420.)  Of the rest, a stage of MXFP8 moves 256
// KB through a CU's LDS, 2048 cycles at 128 bytes each, and keeps its MFMAs busy
// as long.
#include "mx_gate.h"
#include "mx_mm_out.h"

namespace mx {

struct FfnArgs {
  const uint8_t *q_in, *s_in;   // checkpoint (backward)
  uint16_t *y, *dh;             // y null: none (backward)
  uint8_t *q, *s;               // null: no checkpoint
  bool gelu;
};

// Everything a block's amax (binary32 magnitude bits) decides, by the MXFP8
// rule of the casts: kinds 0 finite, 1 with an Inf, 2 with a NaN.
struct Block8 {
  uint32_t byte;
  float limit, scale;   // 448 2^e; 2^e in its exponent field
  uint32_t kind;
};
__device__ __forceinline__ Block8 block8(uint32_t amax) {
  Block8 b;
  const uint32_t e = amax >> 23;
  b.kind = amax < 0x7F800000u ? 0 : amax == 0x7F800000u ? 1 : 2;
  b.byte = b.kind == 0 ? (e > 8 ? e - 8 : 0) : b.kind == 1 ? 254 : 0xFF;
  // (in a block with an Inf every finite element is below the limit)
  b.limit = __uint_as_float(b.kind == 0 ? ((b.byte + 8) << 23) | 0x600000u : 0x7F7FFFFFu);
  b.scale = __uint_as_float(b.byte << 23);
  return b;
}
__device__ __forceinline__ float clamp8(float f, const Block8& b) {
  return __builtin_amdgcn_fmed3f(f, -b.limit, b.limit);
}
// Four elements -> four e4m3 codes; the convert does not saturate.
__device__ __forceinline__ uint32_t quant8_f32(float f0, float f1, float f2, float f3, const Block8& b) {
  i16x2 r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32((i16x2){0, 0}, clamp8(f0, b), clamp8(f1, b), b.scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, clamp8(f2, b), clamp8(f3, b), b.scale, true);
  uint32_t c = as_u32(r);
  if (b.kind != 0) {
    const float f[4] = {f0, f1, f2, f3};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = __float_as_uint(f[i]);
      const uint32_t special = b.kind == 2 ? 0x7Fu : (bits & 0x7FFFFFFFu) == 0x7F800000u ? 0x7Eu : 0u;
      if (special != 0)
        c = (c & ~(0xFFu << (8 * i))) | ((special | ((bits >> 24) & 0x80u)) << (8 * i));
    }
  }
  return c;
}
// Largest magnitude's bits of a lane's 16 and the other half's 16.
__device__ __forceinline__ uint32_t amax32(const v16f& f) {
  uint32_t m = 0;
#pragma unroll
  for (int v = 0; v < 16; ++v)
    m = max(m, __float_as_uint(f[v]) & 0x7FFFFFFFu);
  const auto s = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  return max(s[0], s[1]);
}

template <class S, bool GELU>
__device__ __forceinline__ void ffn_store(const MmArgs& a, const FfnArgs& o, const MmPlace& p, int64_t col0,
                                          uint8_t* lds,
                                          const v16f (&acc)[S::kBW][S::kBX]) {
  constexpr int kCols = 16 * S::kBW;   // of this wave
  using StageY = Staged<kCols * 2>;
  using StageQ = Staged<kCols>;
  constexpr int kSize = StageY::kSize + 2 * StageQ::kSize;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* mine = lds + wave * kSize;
  const StageY sy = {mine};
  const StageQ sq[2] = {{mine + StageY::kSize}, {mine + StageY::kSize + StageQ::kSize}};
  const int row0 = wave / S::kWW * 32 * S::kBX;
  const int64_t c0 = col0 + wave % S::kWW * kCols;
  const int n = (int)min((int64_t)kCols, a.n - c0);   // a multiple of 32
#pragma unroll
  for (int j = 0; j < S::kBX; ++j) {
    const int rows = p.rows - row0 - 32 * j;
    if (rows <= 0 || n <= 0)
      break;
    const int64_t first = p.row0 + row0 + 32 * j;
#pragma unroll
    for (int i = 0; i < S::kBW / 2; ++i) {
      const v16f &g = acc[i][j], &u = acc[i + S::kBW / 2][j];
#pragma unroll
      for (int v = 0; v < 16; v += 4) {
        const int col = 32 * i + 2 * v + 4 * h;
        sy.put(r, col * 2, (u32x2){bf16_pair(act_of<GELU>(g[v]) * u[v], act_of<GELU>(g[v + 1]) * u[v + 1]),
                                   bf16_pair(act_of<GELU>(g[v + 2]) * u[v + 2], act_of<GELU>(g[v + 3]) * u[v + 3])});
      }
      if (o.q != nullptr) {
        const Block8 bg = block8(amax32(g)), bu = block8(amax32(u));
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
          const int col = 32 * i + 2 * v + 4 * h;
          sq[0].put(r, col, quant8_f32(g[v], g[v + 1], g[v + 2], g[v + 3], bg));
          sq[1].put(r, col, quant8_f32(u[v], u[v + 1], u[v + 2], u[v + 3], bu));
        }
        // the gate's scale byte by the lower lanes, the factor's by the others
        if (r < rows && 32 * i < n)
          o.s[(first + r) * (a.n / 16) + (c0 / 32 + i) + (h ? a.n / 32 : 0)] = (uint8_t)(h ? bu.byte : bg.byte);
      }
    }
    mm_wave_fence();
    sy.drain(reinterpret_cast<uint8_t*>(o.y + first * a.n + c0), a.n * 2, rows, n * 2);
    if (o.q != nullptr) {
      uint8_t* q = o.q + first * 2 * a.n + c0;
      sq[0].drain(q, 2 * a.n, rows, n);
      sq[1].drain(q + a.n, 2 * a.n, rows, n);
    }
    mm_wave_fence();
  }
}

// Tiles, and the quarters of the last ones in a launch of large tiles.
template <int FX, int FW>
using FfnQuarter = MmTile<FX, FW, false, false, true>;
template <int FX, int FW, bool LARGE, bool GROUPED>
constexpr int kFfnLds = LARGE && !GROUPED && FfnQuarter<FX, FW>::kLds > MmTile<FX, FW, LARGE>::kLds
                            ? FfnQuarter<FX, FW>::kLds
                            : MmTile<FX, FW, LARGE>::kLds;

template <int FX, int FW, bool LARGE, bool GROUPED>
__global__ __launch_bounds__(LARGE ? 512 : 256) __attribute__((amdgpu_waves_per_eu(2, 2)))
void ffn_kernel(MmArgs a, FfnArgs o) {
  using T = MmTile<FX, FW, LARGE>;
  __shared__ __attribute__((aligned(256))) uint8_t lds[kFfnLds<FX, FW, LARGE, GROUPED>];
  MmPlace p;
  if (!mm_place<GROUPED, T::kRowsX>(a, lds, p))
    return;
  int64_t col0 = (int64_t)p.tn * (T::kRowsW / 2);
  if constexpr (LARGE && !GROUPED) {
    if (p.quarter >= 0) {
      using Q = FfnQuarter<FX, FW>;
      if (!mm_quarter(a, p, T::kRowsX, col0, T::kRowsW / 2))
        return;
      v16f acc[Q::kBW][Q::kBX];
      mm_tile<FX, FW, Q, true>(a, p, col0, lds, acc);
      if (o.gelu)
        ffn_store<Q, true>(a, o, p, col0, lds, acc);
      else
        ffn_store<Q, false>(a, o, p, col0, lds, acc);
      return;
    }
  }
  v16f acc[T::kBW][T::kBX];
  mm_tile<FX, FW, T, true>(a, p, col0, lds, acc);
  if (o.gelu)
    ffn_store<T, true>(a, o, p, col0, lds, acc);
  else
    ffn_store<T, false>(a, o, p, col0, lds, acc);
}

// Backward.  The wave's rows of codes and, after them, of results go through
// one part of LDS.
template <class S, bool GELU>
__device__ __forceinline__ void ffn_bwd_store(const MmArgs& a, const FfnArgs& o, const MmPlace& p, int64_t col0,
                                              uint8_t* lds,
                                              const v16f (&acc)[S::kBW][S::kBX]) {
  constexpr int BW = S::kBW, kCols = 32 * BW;
  using StageQ = Staged<kCols>;
  using StageD = Staged<kCols * 2>;
  constexpr int kSize = 2 * StageQ::kSize > StageD::kSize ? 2 * StageQ::kSize : StageD::kSize;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* mine = lds + wave * kSize;
  const StageQ sg = {mine}, su = {mine + StageQ::kSize};
  const StageD sd = {mine};
  const int row0 = wave / S::kWW * 32 * S::kBX;
  const int64_t c0 = col0 + wave % S::kWW * kCols;
  const int n = (int)min((int64_t)kCols, a.n - c0);   // a multiple of 32
#pragma unroll
  for (int j = 0; j < S::kBX; ++j) {
    const int rows = p.rows - row0 - 32 * j;
    if (rows <= 0 || n <= 0)
      break;
    const int64_t first = p.row0 + row0 + 32 * j;
    // this row's scale bytes and the wave's rows of codes, all on their way at once
    const uint8_t* q = o.q_in + first * 2 * a.n + c0;
    typename StageQ::Loads lg, lu;
    StageQ::load(lg, q, 2 * a.n, rows, n);
    StageQ::load(lu, q + a.n, 2 * a.n, rows, n);
    const int lds = (int)(a.n / 16);
    const uint8_t* s = o.s_in + first * lds + c0 / 32;
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(s, (uint32_t)(min(rows, 32) * lds - c0 / 32));
    float vg[BW], vu[BW];
#pragma unroll
    for (int i = 0; i < BW; ++i) {   // (a block past the columns reads another's byte: it is not stored)
      vg[i] = scale_of(__builtin_amdgcn_raw_buffer_load_b8(rs, r * lds + i, 0, 0));
      vu[i] = scale_of(__builtin_amdgcn_raw_buffer_load_b8(rs, r * lds + i + lds / 2, 0, 0));
    }
    sg.place(lg);
    su.place(lu);
    mm_wave_fence();
    uint32_t cg[BW][4], cu[BW][4];
#pragma unroll
    for (int i = 0; i < BW; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        cg[i][v] = sg.template get<uint32_t>(r, 32 * i + 8 * v + 4 * h);
        cu[i][v] = su.template get<uint32_t>(r, 32 * i + 8 * v + 4 * h);
      }
    mm_wave_fence();
    // the checkpoint's values of four columns
    auto four = [](uint32_t c, float scale, float (&f)[4]) {
      const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
      f[0] = lo[0] * scale, f[1] = lo[1] * scale, f[2] = hi[0] * scale, f[3] = hi[1] * scale;
    };
    auto put = [&](int i, int v, const float (&f)[4]) {
      sd.put(r, (32 * i + 8 * v + 4 * h) * 2, (u32x2){bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])});
    };
    auto drain = [&](uint16_t* dst, int64_t ld) {
      mm_wave_fence();
      sd.drain(reinterpret_cast<uint8_t*>(dst), ld * 2, rows, n * 2);
      mm_wave_fence();
    };
    // (block by block: all at once would not fit the registers)
    u32x2 du[BW][4];
#pragma unroll
    for (int i = 0; i < BW; ++i) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float g[4], u[4], fg[4], fu[4];
        four(cg[i][v], vg[i], g);
        four(cu[i][v], vu[i], u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float s, dt;
          gate<GELU>(g[e], s, dt);
          const float dy = acc[i][j][4 * v + e];
          fu[e] = dy * (g[e] * s);
          fg[e] = dy * u[e] * (s + dt * s * (1.0f - s));
        }
        put(i, v, fg);
        du[i][v] = (u32x2){bf16_pair(fu[0], fu[1]), bf16_pair(fu[2], fu[3])};
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    uint16_t* dh = o.dh + first * 2 * a.n + c0;
    drain(dh, 2 * a.n);
#pragma unroll
    for (int i = 0; i < BW; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        sd.put(r, (32 * i + 8 * v + 4 * h) * 2, du[i][v]);
    drain(dh + a.n, 2 * a.n);
    if (o.y != nullptr) {
#pragma unroll
      for (int i = 0; i < BW; ++i) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float g[4], u[4], fy[4];
          // (formed again: kept from above, they would not fit the registers)
          asm volatile("" : "+v"(cg[i][v]), "+v"(cu[i][v]));
          four(cg[i][v], vg[i], g);
          four(cu[i][v], vu[i], u);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            fy[e] = act_of<GELU>(g[e]) * u[e];
          put(i, v, fy);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      drain(o.y + first * a.n + c0, a.n);
    }
  }
}

template <int FX, int FW, bool LARGE, bool GROUPED>
__global__ __launch_bounds__(LARGE ? 512 : 256) __attribute__((amdgpu_waves_per_eu(2, 2)))
void ffn_bwd_kernel(MmArgs a, FfnArgs o) {
  using T = MmTile<FX, FW, LARGE>;
  __shared__ __attribute__((aligned(256))) uint8_t lds[kFfnLds<FX, FW, LARGE, GROUPED>];
  static_assert(T::kWaves * 2 * Staged<32 * T::kBW>::kSize <= T::kLds &&
                T::kWaves * Staged<64 * T::kBW>::kSize <= T::kLds, "the epilogue's rows");
  MmPlace p;
  if (!mm_place<GROUPED, T::kRowsX>(a, lds, p))
    return;
  int64_t col0 = (int64_t)p.tn * T::kRowsW;
  if constexpr (LARGE && !GROUPED) {
    if (p.quarter >= 0) {
      using Q = FfnQuarter<FX, FW>;
      if (!mm_quarter(a, p, T::kRowsX, col0, T::kRowsW))
        return;
      v16f acc[Q::kBW][Q::kBX];
      mm_tile<FX, FW, Q, false>(a, p, col0, lds, acc);
      if (o.gelu)
        ffn_bwd_store<Q, true>(a, o, p, col0, lds, acc);
      else
        ffn_bwd_store<Q, false>(a, o, p, col0, lds, acc);
      return;
    }
  }
  v16f acc[T::kBW][T::kBX];
  mm_tile<FX, FW, T, false>(a, p, col0, lds, acc);
  if (o.gelu)
    ffn_bwd_store<T, true>(a, o, p, col0, lds, acc);
  else
    ffn_bwd_store<T, false>(a, o, p, col0, lds, acc);
}

static constexpr int32_t E4 = MX_FORMAT_E4M3, E2 = MX_FORMAT_E2M1;

template <int FX, int FW, bool LARGE>
static void launch_pair(bool bwd, const MmArgs& a, const FfnArgs& o, dim3 grid, hipStream_t stream) {
  const dim3 threads(MmTile<FX, FW, LARGE>::kThreads);
  if (bwd) {
    if (a.ends != nullptr)
      hipLaunchKernelGGL((ffn_bwd_kernel<FX, FW, LARGE, true>), grid, threads, 0, stream, a, o);
    else
      hipLaunchKernelGGL((ffn_bwd_kernel<FX, FW, LARGE, false>), grid, threads, 0, stream, a, o);
  } else {
    if (a.ends != nullptr)
      hipLaunchKernelGGL((ffn_kernel<FX, FW, LARGE, true>), grid, threads, 0, stream, a, o);
    else
      hipLaunchKernelGGL((ffn_kernel<FX, FW, LARGE, false>), grid, threads, 0, stream, a, o);
  }
}

template <bool LARGE>
static void launch_formats(bool bwd, int32_t fx, int32_t fw, const MmArgs& a, const FfnArgs& o, dim3 grid,
                           hipStream_t stream) {
  if (fx == E2)
    launch_pair<E2, E2, LARGE>(bwd, a, o, grid, stream);
  else if (fw == E2)
    launch_pair<E4, E2, LARGE>(bwd, a, o, grid, stream);
  else
    launch_pair<E4, E4, LARGE>(bwd, a, o, grid, stream);
}

static hipError_t launch_either(bool bwd, const MmOperands& in, int64_t m, int64_t n, int64_t k, const FfnArgs& o,
                                hipStream_t stream) {
  const bool large = mm_large(m, n, in.groups, bwd ? 256 : 128);
  MmArgs a = mm_args(in, m, n, bwd ? n : 2 * n, k);
  const int tile = large ? 256 : 128;
  const dim3 grid((unsigned)mm_grid(a, tile, bwd ? tile : tile / 2, large));
  if (large)
    launch_formats<true>(bwd, in.x_format, in.w_format, a, o, grid, stream);
  else
    launch_formats<false>(bwd, in.x_format, in.w_format, a, o, grid, stream);
  return hipGetLastError();
}

int64_t ffn_grid_blocks(int64_t m, int64_t n, int32_t groups) {
  MmArgs a = {};
  static const int32_t some = 0;
  a.m = m, a.n = n, a.ends = groups > 0 ? &some : nullptr, a.groups = groups;
  return mm_grid(a, 128, 64);   // the smaller tiles
}

hipError_t launch_ffn(const MmOperands& in, int64_t m, int64_t n, int64_t k, bool gelu, void* y, uint8_t* q, uint8_t* s,
                      hipStream_t stream) {
  FfnArgs o = {};
  o.y = static_cast<uint16_t*>(y), o.q = q, o.s = s, o.gelu = gelu;
  return launch_either(false, in, m, n, k, o, stream);
}

hipError_t launch_ffn_bwd(const MmOperands& in, int64_t m, int64_t n, int64_t k, bool gelu, const uint8_t* q,
                          const uint8_t* s, void* dh, void* y, hipStream_t stream) {
  FfnArgs o = {};
  o.q_in = q, o.s_in = s, o.dh = static_cast<uint16_t*>(dh), o.y = static_cast<uint16_t*>(y), o.gelu = gelu;
  return launch_either(true, in, m, n, k, o, stream);
}

}  // namespace mx
