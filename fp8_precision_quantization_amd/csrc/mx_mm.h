// The MX product that the operators on MX operands share (gfx950 only):
//   R[t][j] = sum over k of X(t, k) * W(j, k)
// for a tile of rows t of X and rows j of W, both K-major codes with one
// e8m0 scale for every 32 of K in the 128 x 4 blocked layout, either of them
// e4m3 (a byte) or e2m1 (half a byte, the first of a byte's two in its low
// half).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes both formats, each side its own.
// Its lane layout (measured with in-bounds probes of random operands): lane l
// holds row l % 32; of e2m1 its 16 bytes are K 32 (l / 32) .. + 31 of the
// step's 64; of e4m3 its bytes 0-15 are K 16 (l / 32) .. + 15 of the first
// block of 32 and bytes 16-31 the same of the second.  The scale of block h
// of row r is the chosen byte of lane r + 32 h's scale register.  A step of
// e2m1 by e2m1 is summed to binary32's precision (1.6e-7 of its largest
// product); with an e4m3 operand to 4e-4 of it.  e2m1 by e2m1 takes half the
// cycles of any pair with an e4m3 side.
//
// W is the instruction's first operand, so that a lane's accumulators are one
// row t and runs of four columns j: register v of lane l is column 8 (v / 4)
// + 4 (l / 32) + v % 4, row l % 32 of a 32 x 32 block.  A block of 32 columns
// of a row is then two lanes' registers: the epilogues that need a block's
// largest magnitude exchange it once, and all of them write words.
//
// A workgroup of four waves owns a 64 NB x 64 NB tile of R, a wave its
// quarter in NB x NB blocks.  K advances in stages of 128: the waves bring
// stage rows (64 bytes of e2m1, 128 of e4m3) and the stage's scales straight
// from memory into one of kSlots LDS slots, kSlots - 1 stages ahead.  16-byte
// chunks of a row are permuted by an XOR with bits of the row (through the
// loads' source offsets, as a load to LDS writes in lane order), so that 16
// lanes that read one chunk of 16 rows reach all banks.  Operands are read
// from LDS one 64-deep step ahead of the MFMAs that use them; loads and reads
// stand between the MFMAs; one barrier a stage.
//
// Rows past the tile's end, K past the end and whole stages past it load as
// zeros: their offsets lie outside the buffer's range.
#pragma once

#include <type_traits>

#include "mx_device.h"
#include "mx_fp4_launch.h"
#include "mx_groups.h"
#include "mxfp4.h"

namespace mx {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kMmThreads = 256;
constexpr int kMmK = 128;     // K of a stage
constexpr int kMmBand = 8;    // tile rows to a band of the tile order

// Codes of a format: what the MFMA calls it, bytes of a stage's row.
template <int FMT>
struct MmFormat {
  static constexpr int kCode = FMT == MX_FORMAT_E2M1 ? 4 : 0;
  static constexpr int kRow = FMT == MX_FORMAT_E2M1 ? kMmK / 2 : kMmK;
  static constexpr int kChunks = kRow / 16;
  static constexpr int kWords = FMT == MX_FORMAT_E2M1 ? 1 : 2;   // 16-byte words of a lane's operand of a step
};

// The XOR of a stage row's chunk numbers.
template <int CHUNKS>
__device__ __forceinline__ int mm_swizzle(int row) {
  return CHUNKS == 8 ? (row & 7) ^ ((row >> 3) & 1) : (row >> 2) & 3;
}

template <int FX, int FW, int NB>
struct MmTile {
  static constexpr int kTile = 64 * NB;
  static constexpr int kX = 0;
  static constexpr int kW = kTile * MmFormat<FX>::kRow;
  static constexpr int kSX = kW + kTile * MmFormat<FW>::kRow;   // scales: 4 bytes a row
  static constexpr int kSW = kSX + kTile * 4;
  static constexpr int kSlot = kSW + kTile * 4;
  // slots that fit 160 KiB, or half of it where two workgroups share a CU
  static constexpr int kSlots = (NB == 4 ? 163840 : 81920) / kSlot > 4 ? 4 : (NB == 4 ? 163840 : 81920) / kSlot;
  static constexpr int kLds = kSlots * kSlot;
  static constexpr int kLoadsX = kTile * MmFormat<FX>::kRow / 4096;   // loads of a wave, 1 KiB each
  static constexpr int kLoadsW = kTile * MmFormat<FW>::kRow / 4096;
  static constexpr int kLoadsS = NB == 4 ? 2 : 1;
  static constexpr int kLoads = kLoadsX + kLoadsW + kLoadsS;
  static_assert(kSlots >= 2 && (kSlots - 1) * kLoads < 64, "slots and the load counter");
};

struct MmArgs {
  const uint8_t *qx, *sx, *qw, *sw;
  int64_t m, n, k;             // rows of X; columns of R to a group (of each half where gated); depth
  const int32_t* ends;         // null: one group
  int32_t groups;
  int64_t w_bytes, sw_bytes;   // codes and scales of one group's W
  uint32_t tiles_m, tiles_n, per_xcd;
};

// 16 or 4 bytes a lane from memory to LDS at `to` (the wave's; lane order).
template <int BYTES>
__device__ __forceinline__ void mm_load(uint32_t to, __amdgpu_buffer_rsrc_t rsrc, uint32_t offset) {
  static_assert(BYTES == 16 || BYTES == 4, "load sizes");
  // (a write of m0 and its use by a load to LDS need an instruction between)
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(offset),
                 "s"(rsrc)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to), "v"(offset),
                 "s"(rsrc)
                 : "memory");
}

// Until at most N of the wave's loads are in flight.
template <int N>
__device__ __forceinline__ void mm_wait_loads() {
  static_assert(N < 64, "the load counter has six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4 << 14));
}

// Orders a wave's LDS accesses by different lanes (LDS runs a wave's in order).
__device__ __forceinline__ void mm_wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// f(0) .. f(N - 1) with the numbers as constants.
template <class F, int... I>
__device__ __forceinline__ void mm_each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}

// Where a workgroup's tile lies.
struct MmPlace {
  int64_t row0;       // its first row of X and of the result
  int32_t rows;       // how many
  int64_t srow0;      // its first row in X's scale layout, a multiple of 128
  uint32_t tn;        // its tile column
  int32_t group;
};

// The tile of this workgroup: false if it has none (uniform; no barrier is
// left open).  XCD x (workgroups are dealt to the XCDs in turn) owns one of 8
// contiguous pieces of the ordered tiles: bands of 8 tile rows, column by
// column.  Grouped: a piece of each group's tiles, group after group.  `lds`
// holds the group table meanwhile.
template <bool GROUPED, int TILE>
__device__ __forceinline__ bool mm_place(const MmArgs& a, uint8_t* lds, MmPlace& p) {
  auto band_tile = [&](uint32_t i, uint32_t rows_of_tiles, uint32_t& tm) {
    const uint32_t band = i / (kMmBand * a.tiles_n);
    const uint32_t band_rows = min((uint32_t)kMmBand, rows_of_tiles - band * kMmBand);
    const uint32_t within = i - band * kMmBand * a.tiles_n;
    tm = band * kMmBand + within % band_rows;
    p.tn = within / band_rows;
  };
  uint32_t tm;
  if constexpr (!GROUPED) {
    const uint32_t id = (blockIdx.x % 8) * a.per_xcd + blockIdx.x / 8;
    if (blockIdx.x / 8 >= a.per_xcd || id >= a.tiles_m * a.tiles_n)
      return false;
    band_tile(id, a.tiles_m, tm);
    p.group = 0;
    p.row0 = (int64_t)tm * TILE;
    p.rows = (int32_t)min((int64_t)TILE, a.m - p.row0);
    p.srow0 = p.row0;
    return true;
  } else {
    GroupTable& table = *reinterpret_cast<GroupTable*>(lds);
    int32_t* xs = reinterpret_cast<int32_t*>(lds + sizeof(GroupTable));
    if (threadIdx.x < 64) {
      if (a.groups <= kScalarTableGroups)
        build_group_table_scalar(a.ends, a.groups, (int32_t)a.m, TILE, table);
      else
        build_group_table(a.ends, a.groups, (int32_t)a.m, TILE, table);
      build_piece_starts(table, a.groups, TILE, a.tiles_n, xs);
    }
    lds_barrier();
    const int32_t q = (int32_t)(blockIdx.x / 8), x = (int32_t)(blockIdx.x % 8);
    if (q >= __builtin_amdgcn_readfirstlane(xs[a.groups]))
      return false;
    int glo = 0, ghi = a.groups;   // xs[glo] <= q < xs[ghi]
    while (ghi - glo > 1) {
      const int mid = (glo + ghi) >> 1;
      if (xs[mid] <= q)
        glo = mid;
      else
        ghi = mid;
    }
    const int g = __builtin_amdgcn_readfirstlane(glo);
    const int32_t lo = __builtin_amdgcn_readfirstlane(table.lo[g]), hi = __builtin_amdgcn_readfirstlane(table.hi[g]);
    const uint32_t trows = (uint32_t)(__builtin_amdgcn_readfirstlane(table.start[g + 1]) -
                                      __builtin_amdgcn_readfirstlane(table.start[g])) / TILE;
    const uint32_t tg = trows * a.tiles_n, pg = (tg + 7) / 8;
    const uint32_t idx = (uint32_t)x * pg + (uint32_t)(q - __builtin_amdgcn_readfirstlane(xs[g]));
    if (idx >= tg)
      return false;
    band_tile(idx, trows, tm);
    const int32_t r0 = lo + (int32_t)tm * TILE;
    p.group = g;
    p.row0 = r0;
    p.rows = min(TILE, hi - r0);
    // group g starts in the scale layout at the earlier groups' sizes, each
    // rounded up to 128 rows
    int32_t part = 0;
    for (int h = threadIdx.x & 63; h < g; h += 64)
      part += (table.hi[h] - table.lo[h] + 127) / 128 * 128;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
      part += __shfl_xor(part, d);
    p.srow0 = __builtin_amdgcn_readfirstlane(part) + (r0 - lo);
    lds_barrier();   // every wave is done with the table
    return true;
  }
}

// The tile's accumulators: acc[i][j] is the block of W rows 32 i and X rows
// 32 j of this wave's quarter.  GATED: the wave's W rows are 16 NB rows from
// its columns' gate half and the same of the factor half (n rows on), blocks
// i < NB / 2 and the others.  col0: the tile's first column of R.
template <int FX, int FW, int NB, bool GATED>
__device__ __forceinline__ void mm_tile(const MmArgs& a, const MmPlace& p, int64_t col0, uint8_t* lds,
                                        v16f (&acc)[NB][NB]) {
  using T = MmTile<FX, FW, NB>;
  using X = MmFormat<FX>;
  using W = MmFormat<FW>;
  constexpr int kSlots = T::kSlots;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r = lane & 31, h = lane >> 5;

  const int ldx = (int)(FX == MX_FORMAT_E2M1 ? a.k / 2 : a.k), ldw = (int)(FW == MX_FORMAT_E2M1 ? a.k / 2 : a.k);
  const int strip = (int)((a.k / 32 + 3) / 4) * 512;   // a 128-row strip of a scale layout
  const int stages = (int)((a.k + kMmK - 1) / kMmK);

  const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.qx + p.row0 * ldx, (uint32_t)p.rows * (uint32_t)ldx);
  const __amdgpu_buffer_rsrc_t rsx =
      buffer_rsrc(a.sx + p.srow0 / 128 * strip, (uint32_t)((p.rows + 127) / 128 * strip));
  // W: one range, or the gate's and the factor's
  constexpr int kCols = GATED ? T::kTile / 2 : T::kTile;
  const int cols = (int)min((int64_t)kCols, a.n - col0);
  const uint8_t* wbase = a.qw + p.group * a.w_bytes + col0 * ldw;
  const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(wbase, (uint32_t)cols * (uint32_t)ldw);
  const __amdgpu_buffer_rsrc_t ru = GATED ? buffer_rsrc(wbase + a.n * ldw, (uint32_t)cols * (uint32_t)ldw) : rw;
  const int64_t strip0 = col0 / 128;
  const __amdgpu_buffer_rsrc_t rsw = buffer_rsrc(a.sw + p.group * a.sw_bytes + strip0 * strip,
                                                 (uint32_t)(a.sw_bytes - strip0 * strip));

  const uint32_t lds0 =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);

  // Loader roles.  Code load u of wave w fills 1 KiB, whole stage rows; the
  // lane's row of load 0, its chunk of memory, its offset.
  const int xrow = (64 / X::kChunks) * wave + lane / X::kChunks;
  const int xchunk = (lane % X::kChunks) ^ mm_swizzle<X::kChunks>(xrow);
  const uint32_t xoff = xrow * ldx + 16 * xchunk;
  const int wrow = (64 / W::kChunks) * wave + lane / W::kChunks;
  const int wchunk = (lane % W::kChunks) ^ mm_swizzle<W::kChunks>(wrow);
  const uint32_t woff = wrow * ldw + 16 * wchunk;
  constexpr int kXRows = 4 * 64 / X::kChunks, kWRows = 4 * 64 / W::kChunks;   // rows from load to load
  // Scales: word d of the stage's is row 32 NB (d / 32 NB) + 32 (d % NB) + d /
  // NB % 32 of the tile, so that a lane finds its row's words of its NB
  // blocks together.
  auto scale_row = [&](int d) { return 32 * NB * (d / (32 * NB)) + 32 * (d % NB) + d / NB % 32; };
  const int sd = NB == 4 ? threadIdx.x : threadIdx.x & 127;
  const int srow = scale_row(sd);
  auto scale_at = [&](int64_t row) {   // of a row of a scale layout, K 0
    return (uint32_t)(row / 128 * strip + 16 * (row % 32) + 4 * (row % 128 / 32));
  };
  const uint32_t sxoff = scale_at(srow);
  int64_t swrow = col0 % 128 + srow;
  if constexpr (GATED) {
    const int half = 16 * NB, quarter = srow / (2 * half), in = srow % (2 * half);
    swrow = col0 % 128 + half * quarter + in % half + (in >= half ? a.n : 0);
  }
  const uint32_t swoff = scale_at(swrow);

  // load i of stage t into slot b: X, W, scales.  Where the tile is 128 high
  // waves 0 and 1 bring X's scales and the others W's.
  auto load = [&](int i, int t, int b) {
    const uint32_t to = lds0 + b * T::kSlot;
    if (i < T::kLoadsX) {
      const uint32_t off = (16 * xchunk + t * X::kRow < ldx ? xoff + t * X::kRow : 0x80000000u) + (uint32_t)(i * kXRows * ldx);
      mm_load<16>(to + T::kX + i * 4096 + wave * 1024, rx, off);
    } else if (i < T::kLoadsX + T::kLoadsW) {
      const int u = i - T::kLoadsX;
      // rows of this load: kWRows u on, or in the gate or factor half
      int rows = u * kWRows;
      bool up = false;
      if constexpr (GATED) {
        constexpr int kHalf = 16 * NB;
        static_assert(kWRows <= kHalf || kWRows == 2 * kHalf, "a load's rows");
        if constexpr (kWRows <= kHalf) {
          up = rows % (2 * kHalf) >= kHalf;
          rows = rows / (2 * kHalf) * kHalf + rows % kHalf;
        } else {
          up = wave >= 2;   // waves 0 and 1 bring the gate's rows, the others the factor's
          rows = u * kHalf - (up ? kHalf : 0);
        }
      }
      const uint32_t off = (16 * wchunk + t * W::kRow < ldw ? woff + t * W::kRow : 0x80000000u) + (uint32_t)(rows * ldw);
      mm_load<16>(to + T::kW + u * 4096 + wave * 1024, GATED && up ? ru : rw, off);
    } else if constexpr (NB == 4) {
      if (i == T::kLoads - 2)
        mm_load<4>(to + T::kSX + wave * 256, rsx, sxoff + t * 512);
      else
        mm_load<4>(to + T::kSW + wave * 256, rsw, swoff + t * 512);
    } else {
      mm_load<4>(to + T::kSX + wave * 256, wave < 2 ? rsx : rsw, (wave < 2 ? sxoff : swoff) + t * 512);
    }
  };

  // Operands of a step: [block][word]; and the words of scales of a stage.
  typedef u32x4 OpX[NB][X::kWords];
  typedef u32x4 OpW[NB][W::kWords];
  typedef uint32_t Scales[NB];
  constexpr int kReads = NB * (X::kWords + W::kWords);
  const int fx = mm_swizzle<X::kChunks>(r), fw = mm_swizzle<W::kChunks>(r);
  const int xat = T::kX + (wm * 32 * NB + r) * X::kRow, wat = T::kW + (wn * 32 * NB + r) * W::kRow;
  // read q of step s from slot b: W's first block, X's blocks, W's others
  auto read = [&](int q, int s, int b, OpX& ox, OpW& ow) {
    const uint8_t* slot = lds + b * T::kSlot;
    auto one_w = [&](int i, int word) {
      const int chunk = W::kWords == 1 ? 2 * s + h : 4 * s + 2 * word + h;
      ow[i][word] = *reinterpret_cast<const u32x4*>(slot + wat + i * 32 * W::kRow + 16 * (chunk ^ fw));
    };
    auto one_x = [&](int j, int word) {
      const int chunk = X::kWords == 1 ? 2 * s + h : 4 * s + 2 * word + h;
      ox[j][word] = *reinterpret_cast<const u32x4*>(slot + xat + j * 32 * X::kRow + 16 * (chunk ^ fx));
    };
    if (q < W::kWords)
      one_w(0, q);
    else if (q < W::kWords + NB * X::kWords)
      one_x((q - W::kWords) / X::kWords, (q - W::kWords) % X::kWords);
    else
      one_w((q - NB * X::kWords) / W::kWords, (q - NB * X::kWords) % W::kWords);
  };
  auto read_scales = [&](int b, Scales& sx, Scales& sw) {
    const uint8_t* slot = lds + b * T::kSlot;
    if constexpr (NB == 4) {
      const u32x4 vx = *reinterpret_cast<const u32x4*>(slot + T::kSX + (wm * 32 + r) * 16);
      const u32x4 vw = *reinterpret_cast<const u32x4*>(slot + T::kSW + (wn * 32 + r) * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sx[i] = vx[i], sw[i] = vw[i];
    } else {
      const u32x2 vx = *reinterpret_cast<const u32x2*>(slot + T::kSX + (wm * 32 + r) * 8);
      const u32x2 vw = *reinterpret_cast<const u32x2*>(slot + T::kSW + (wn * 32 + r) * 8);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        sx[i] = vx[i], sw[i] = vw[i];
    }
  };
  auto wide_op = [](const auto& o) {
    if constexpr (std::extent_v<std::remove_reference_t<decltype(o)>> == 2)
      return (v8i){(int)o[0][0], (int)o[0][1], (int)o[0][2], (int)o[0][3],
                   (int)o[1][0], (int)o[1][1], (int)o[1][2], (int)o[1][3]};
    else
      return (v8i){(int)o[0][0], (int)o[0][1], (int)o[0][2], (int)o[0][3], 0, 0, 0, 0};
  };
  // MFMA q of step s: scale byte 2 s + h of a row's word, h shifted away before
  auto mfma = [&](auto s_c, int q, const OpX& ox, const OpW& ow, const Scales& sx, const Scales& sw) {
    constexpr int kByte = 2 * decltype(s_c)::value;
    const int i = q / NB, j = q % NB;
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide_op(ow[i]), wide_op(ox[j]), acc[i][j], W::kCode,
                                                                X::kCode, kByte, (int)sw[i], kByte, (int)sx[j]);
  };

#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      acc[i][j] = (v16f){};
  if (stages == 0)
    return;

#pragma unroll
  for (int t = 0; t < kSlots; ++t)
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i)
      load(i, t, t);
  mm_wait_loads<(kSlots - 1) * T::kLoads>();
  lds_barrier();
  OpX x0, x1;
  OpW w0, w1;
  Scales sx, sw, nx, nw;
  read_scales(0, nx, nw);
#pragma unroll
  for (int q = 0; q < kReads; ++q)
    read(q, 0, 0, x0, w0);

  // Stage t in slot b.  First step: its MFMAs, and the reads of the second
  // step's operands.  Then, once this wave's loads of stage t + 1 have landed
  // and every wave has read slot b, the second step: its MFMAs, the loads of
  // stage t + kSlots into slot b and the reads of stage t + 1's first step.
  constexpr int kMfmas = NB * NB;
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  int b = 0;
  for (int t = 0; t < stages; ++t) {
#pragma unroll
    for (int i = 0; i < NB; ++i)
      sx[i] = nx[i] >> (8 * h), sw[i] = nw[i] >> (8 * h);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < kMfmas; ++q) {
      mfma(S0(), q, x0, w0, sx, sw);
#pragma unroll
      for (int u = q * kReads / kMfmas; u < (q + 1) * kReads / kMfmas; ++u)
        read(u, 1, b, x1, w1);
      __builtin_amdgcn_sched_barrier(0);
    }
    mm_wait_loads<(kSlots - 2) * T::kLoads>();
    lds_barrier();
    const int nb = b + 1 == kSlots ? 0 : b + 1;
    read_scales(nb, nx, nw);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < kMfmas; ++q) {
      mfma(S1(), q, x1, w1, sx, sw);
#pragma unroll
      for (int i = q * T::kLoads / kMfmas; i < (q + 1) * T::kLoads / kMfmas; ++i)
        load(i, t + kSlots, b);
#pragma unroll
      for (int u = q * kReads / kMfmas; u < (q + 1) * kReads / kMfmas; ++u)
        read(u, 0, nb, x0, w0);
      __builtin_amdgcn_sched_barrier(0);
    }
    b = nb;
  }
  // the loads past K must land before the slots serve anything else
  mm_wait_loads<0>();
  lds_barrier();
}

// w_rows: rows of one group's W.
inline MmArgs mm_args(const MmOperands& in, int64_t m, int64_t n, int64_t w_rows, int64_t k) {
  MmArgs a = {};
  a.qx = in.qx, a.sx = in.sx, a.qw = in.qw, a.sw = in.sw;
  a.m = m, a.n = n, a.k = k;
  a.ends = in.ends, a.groups = in.groups;
  a.w_bytes = w_rows * (in.w_format == MX_FORMAT_E2M1 ? k / 2 : k);
  a.sw_bytes = (w_rows + 127) / 128 * 128 * ((k / 32 + 3) / 4 * 4);
  return a;
}

// NB for a result of m rows and n columns: 256 x 256 tiles where they fill
// the GPU, else 128 x 128.  tile_cols: columns of R that a large tile covers.
inline int mm_blocks(int64_t m, int64_t n, int32_t groups, int tile_cols) {
  const int64_t rows = groups > 1 ? m / groups : m;   // (of a group, if they were even)
  const int64_t tiles = (rows + 255) / 256 * (groups > 1 ? groups : 1) * ((n + tile_cols - 1) / tile_cols);
  return tiles >= 192 ? 4 : 2;
}

// Tiles of a launch, and its workgroups.  cols_tile: columns of R to a tile.
inline int64_t mm_grid(MmArgs& a, int tile, int cols_tile) {
  const int64_t groups = a.ends != nullptr ? a.groups : 0;
  const int64_t tm = (a.m + tile - 1) / tile + groups, tn = (a.n + cols_tile - 1) / cols_tile;
  const int64_t per = (tm * tn + 7) / 8 + groups;
  a.tiles_m = (uint32_t)tm, a.tiles_n = (uint32_t)tn, a.per_xcd = (uint32_t)per;
  return per * 8;
}

}  // namespace mx
