// Products with MXFP4 weights: C[m][n] = sum over k of A(m, k) * B(n, k), A in
// MXFP4 or MXFP8, B in MXFP4, dense or grouped along M (mx_mm.h has the
// product itself).
//
// Timed (us, best to median): 16640 x 8192 x 5120 in MXFP4, bf16 out, 351-390
// (3.6-4.0 PFLOP/s), with MXFP8 rows 482-533 (2.6-2.9); 16640 x 2048 x 5120 in 16
// groups with MXFP8 rows 172-197, in MXFP4 129-138.
// What the MXFP4 product's 665 thousand cycles go to (copies with a part left
// out, thousands): its MFMAs are busy 333; without loads, LDS reads and epilogue
// 429 are left (starts, barriers, scales, the ends of rounds); loads and their
// waits cost 109 more, LDS reads 26 to 51, the epilogue 80.  So half of the cycles
// are waits that the one wave of a SIMD has nothing to cover with.  The clock
// stays at 1.8-1.95 GHz in all of these copies: power sets it, and with it the time
// of a cycle, not how many there are.  (It also bounds what fewer waits would bring:
// MFMAs alone and always busy hold the clock at 1.4-1.6 GHz and take 233 us.)
// Large tiles by four waves of 128 x 128 read a third less from LDS than by eight
// (375 against 360 us), and here the epilogue is short.
#include "mx_fp4_launch.h"
#include "mx_mm_out.h"

namespace mx {

struct MmGemmOut {
  void* c;
  bool f32, words;   // binary32 or bf16; rows of whole 16-byte words
};

template <class S, class E>
__device__ __forceinline__ void store_c(const MmArgs& a, const MmPlace& p, int64_t col0, uint8_t* lds, bool words,
                                        E* c, const v16f (&acc)[S::kBW][S::kBX]) {
  using Stage = Staged<32 * S::kBW * (int)sizeof(E)>;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Stage st = {lds + wave * Stage::kSize};
  const int row0 = wave / S::kWW * 32 * S::kBX;
  const int64_t c0 = col0 + wave % S::kWW * 32 * S::kBW;
  const int n = (int)min((int64_t)32 * S::kBW, a.n - c0);
#pragma unroll
  for (int j = 0; j < S::kBX; ++j) {
    const int rows = p.rows - row0 - 32 * j;
    if (rows <= 0 || n <= 0)
      break;
#pragma unroll
    for (int i = 0; i < S::kBW; ++i)
#pragma unroll
      for (int v = 0; v < 16; v += 4) {
        const int col = 32 * i + 2 * v + 4 * h;
        const v16f& f = acc[i][j];
        if constexpr (sizeof(E) == 4)
          st.put(r, col * 4, (f32x4){f[v], f[v + 1], f[v + 2], f[v + 3]});
        else
          st.put(r, col * 2, (u32x2){bf16_pair(f[v], f[v + 1]), bf16_pair(f[v + 2], f[v + 3])});
      }
    mm_wave_fence();
    E* dst = c + (p.row0 + row0 + 32 * j) * a.n + c0;
    if (words)
      st.drain(reinterpret_cast<uint8_t*>(dst), a.n * (int)sizeof(E), rows, n * (int)sizeof(E));
    else
      st.drain_each(dst, a.n, rows, n);
    mm_wave_fence();
  }
}

template <int FX, bool LARGE>
using GemmTile = MmTile<FX, MX_FORMAT_E2M1, LARGE, LARGE>;

template <int FX, bool LARGE, bool GROUPED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(LARGE ? 1 : 2, LARGE ? 1 : 2)))
void mm_gemm_kernel(MmArgs a, MmGemmOut o) {
  using T = GemmTile<FX, LARGE>;
  __shared__ __attribute__((aligned(256))) uint8_t lds[T::kLds];
  static_assert(T::kWaves * Staged<128 * T::kBW>::kSize <= T::kLds, "the epilogue's rows");
  MmPlace p;
  if (!mm_place<GROUPED, T::kRowsX>(a, lds, p))
    return;
  int64_t col0 = (int64_t)p.tn * T::kRowsW;
  if constexpr (LARGE && !GROUPED) {
    if (p.quarter >= 0) {
      using Q = GemmTile<FX, false>;
      if (!mm_quarter(a, p, T::kRowsX, col0, T::kRowsW))
        return;
      v16f acc[Q::kBW][Q::kBX];
      mm_tile<FX, MX_FORMAT_E2M1, Q, false>(a, p, col0, lds, acc);
      if (o.f32)
        store_c<Q>(a, p, col0, lds, o.words, static_cast<float*>(o.c), acc);
      else
        store_c<Q>(a, p, col0, lds, o.words, static_cast<uint16_t*>(o.c), acc);
      return;
    }
  }
  v16f acc[T::kBW][T::kBX];
  mm_tile<FX, MX_FORMAT_E2M1, T, false>(a, p, col0, lds, acc);
  if (o.f32)
    store_c<T>(a, p, col0, lds, o.words, static_cast<float*>(o.c), acc);
  else
    store_c<T>(a, p, col0, lds, o.words, static_cast<uint16_t*>(o.c), acc);
}

template <int FX, bool LARGE>
static void launch(const MmArgs& a, const MmGemmOut& o, dim3 grid, hipStream_t stream) {
  const dim3 threads(GemmTile<FX, LARGE>::kThreads);
  if (a.ends != nullptr)
    hipLaunchKernelGGL((mm_gemm_kernel<FX, LARGE, true>), grid, threads, 0, stream, a, o);
  else
    hipLaunchKernelGGL((mm_gemm_kernel<FX, LARGE, false>), grid, threads, 0, stream, a, o);
}

int64_t gemm4_grid_blocks(int64_t m, int64_t n, int32_t groups) {
  static const int32_t some = 0;
  MmArgs a = {};
  a.m = m, a.n = n, a.ends = groups > 0 ? &some : nullptr, a.groups = groups;
  return mm_grid(a, 128, 128);   // the smaller tiles
}

hipError_t launch_gemm4(const MmOperands& in, int64_t m, int64_t n, int64_t k, void* c, bool f32, hipStream_t stream) {
  const bool large = mm_large(m, n, in.groups, 256);
  MmArgs a = mm_args(in, m, n, n, k);
  const dim3 grid((unsigned)mm_grid(a, large ? 256 : 128, large ? 256 : 128, large));
  const MmGemmOut o = {c, f32, n * (f32 ? 4 : 2) % 16 == 0 && (uintptr_t)c % 16 == 0};
  if (in.x_format == MX_FORMAT_E2M1) {
    if (large)
      launch<MX_FORMAT_E2M1, true>(a, o, grid, stream);
    else
      launch<MX_FORMAT_E2M1, false>(a, o, grid, stream);
  } else {
    if (large)
      launch<MX_FORMAT_E4M3, true>(a, o, grid, stream);
    else
      launch<MX_FORMAT_E4M3, false>(a, o, grid, stream);
  }
  return hipGetLastError();
}

}  // namespace mx
