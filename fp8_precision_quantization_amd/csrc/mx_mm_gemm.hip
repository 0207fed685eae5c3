// Products with MXFP4 weights: C[m][n] = sum over k of A(m, k) * B(n, k), A in
// MXFP4 or MXFP8, B in MXFP4, dense or grouped along M (mx_mm.h has the
// product itself).
#include "mx_fp4_launch.h"
#include "mx_mm_out.h"

namespace mx {

struct MmGemmOut {
  void* c;
  bool f32, words;   // binary32 or bf16; rows of whole 16-byte words
};

template <int NB, class E>
__device__ __forceinline__ void store_c(const MmArgs& a, const MmPlace& p, int64_t col0, uint8_t* lds, bool words,
                                        E* c, const v16f (&acc)[NB][NB]) {
  using Stage = Staged<32 * NB * (int)sizeof(E)>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 31, h = lane >> 5;
  const Stage st = {lds + wave * Stage::kSize};
  const int row0 = (wave >> 1) * 32 * NB;
  const int64_t c0 = col0 + (wave & 1) * 32 * NB;
  const int n = (int)min((int64_t)32 * NB, a.n - c0);
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int rows = p.rows - row0 - 32 * j;
    if (rows <= 0 || n <= 0)
      break;
#pragma unroll
    for (int i = 0; i < NB; ++i)
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

template <int FX, int NB, bool GROUPED>
__global__ __launch_bounds__(kMmThreads) __attribute__((amdgpu_waves_per_eu(NB == 4 ? 1 : 2, NB == 4 ? 1 : 2)))
void mm_gemm_kernel(MmArgs a, MmGemmOut o) {
  using T = MmTile<FX, MX_FORMAT_E2M1, NB>;
  __shared__ __attribute__((aligned(256))) uint8_t lds[T::kLds];
  static_assert(4 * Staged<32 * NB * 4>::kSize <= T::kLds, "the epilogue's rows");
  MmPlace p;
  if (!mm_place<GROUPED, T::kTile>(a, lds, p))
    return;
  const int64_t col0 = (int64_t)p.tn * T::kTile;
  v16f acc[NB][NB];
  mm_tile<FX, MX_FORMAT_E2M1, NB, false>(a, p, col0, lds, acc);
  if (o.f32)
    store_c<NB>(a, p, col0, lds, o.words, static_cast<float*>(o.c), acc);
  else
    store_c<NB>(a, p, col0, lds, o.words, static_cast<uint16_t*>(o.c), acc);
}

template <int FX, int NB>
static void launch(const MmArgs& a, const MmGemmOut& o, dim3 grid, hipStream_t stream) {
  if (a.ends != nullptr)
    hipLaunchKernelGGL((mm_gemm_kernel<FX, NB, true>), grid, dim3(kMmThreads), 0, stream, a, o);
  else
    hipLaunchKernelGGL((mm_gemm_kernel<FX, NB, false>), grid, dim3(kMmThreads), 0, stream, a, o);
}

static MmArgs gemm4_args(const MmOperands& in, int64_t m, int64_t n, int64_t k, int nb, int64_t* blocks) {
  MmArgs a = mm_args(in, m, n, n, k);
  *blocks = mm_grid(a, 64 * nb, 64 * nb);
  return a;
}

int64_t gemm4_grid_blocks(int64_t m, int64_t n, int32_t groups) {
  MmOperands in = {};
  static const int32_t some = 0;
  in.ends = groups > 0 ? &some : nullptr, in.groups = groups;
  int64_t blocks;
  gemm4_args(in, m, n, 32, 2, &blocks);   // the smaller tiles
  return blocks;
}

hipError_t launch_gemm4(const MmOperands& in, int64_t m, int64_t n, int64_t k, void* c, bool f32, hipStream_t stream) {
  const int nb = mm_blocks(m, n, in.groups, 256);
  int64_t blocks;
  const MmArgs a = gemm4_args(in, m, n, k, nb, &blocks);
  const MmGemmOut o = {c, f32, n * (f32 ? 4 : 2) % 16 == 0 && (uintptr_t)c % 16 == 0};
  const dim3 grid((unsigned)blocks);
  if (in.x_format == MX_FORMAT_E2M1) {
    if (nb == 4)
      launch<MX_FORMAT_E2M1, 4>(a, o, grid, stream);
    else
      launch<MX_FORMAT_E2M1, 2>(a, o, grid, stream);
  } else {
    if (nb == 4)
      launch<MX_FORMAT_E4M3, 4>(a, o, grid, stream);
    else
      launch<MX_FORMAT_E4M3, 2>(a, o, grid, stream);
  }
  return hipGetLastError();
}

}  // namespace mx
