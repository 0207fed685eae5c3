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
// of row r is the chosen byte of lane r + 32 h's scale register.  The products of
// eight neighbouring k are added in fixed point, each cut toward zero at 2^-13 of
// the largest 2^(ea + eb) of their codes' exponents, and the groups of eight in
// binary32 (probed; random codes agree with this to 6e-7 of the largest product).
// e2m1 by e2m1 loses nothing by that, its products spanning eight bits.  With an
// e4m3 side a step loses 2e-4 of its largest product on average where all are of
// one sign (8e-4 at worst in 512 x 512 sums), a third of that of both signs.  The
// fp8 instructions without scales, and the 16 x 16 shape, cut at the same place.
// Exact sums would take codes as bf16, whose products reach half the rate (the
// library's 8192 cube 1.5 PFLOP/s against 2.5 in the gated block), for results
// that a bf16 rounding moves ten to a hundred times as far; what shows is the
// block's 8-bit checkpoint, 0.4% from the exact sums' in norm.  e2m1 by e2m1 takes
// half the cycles of any pair with an e4m3 side.
//
// W is the instruction's first operand, so that a lane's accumulators are one
// row t and runs of four columns j: register v of lane l is column 8 (v / 4)
// + 4 (l / 32) + v % 4, row l % 32 of a 32 x 32 block.  A block of 32 columns
// of a row is then two lanes' registers: the epilogues that need a block's
// largest magnitude exchange it once, and all of them write words.
//
// A workgroup of WX x WW waves owns a tile of R, a wave BX x BW blocks of 32 x
// 32 of it.  K advances in stages of 128: the waves bring stage rows (64 bytes
// of e2m1, 128 of e4m3) and the stage's scales straight from memory into one
// of kSlots LDS slots, kSlots - 1 stages ahead.  16-byte chunks of a row are
// permuted by an XOR with bits of the row (through the loads' source offsets,
// as a load to LDS writes in lane order), so that 16 lanes that read one chunk
// of 16 rows reach all banks.  Operands are read from LDS one 64-deep step
// ahead of the MFMAs that use them; loads and reads stand between the MFMAs;
// one barrier a stage.
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

constexpr int kMmK = 128;     // K of a stage
// Most tiles of an XCD's last round that are taken in quarters (us, whole and in
// quarters: 4 tiles, 16640 x 8192 x 5120 in MXFP4 356 and 343, gradient of 16640 x
// 4096 x 5120 in MXFP8 366 and 338; 5 tiles, 4352 x 4352 x 4096 60 and 48; 12 tiles,
// 5632 x 4096 x 4096 62.0 and 60.1; 16 tiles, 6144 x 4096 x 4096 63.1 and 61.3).
constexpr int kMmSplit = 16;
// Tile rows to a band of the tile order (the 32 CUs of an XCD then work on 5 x 6
// tiles or so).  Best of 30 in us, of 5, 7 and 8 (two runs each on one card, without
// quarters; 4 and 6 lost on the first shape and its gradient): block 16640 x 4096 x
// 5120 in MXFP8 567-569, 568-572, 586-591, in MXFP4 406-407, 406-408, 425-427, its
// gradient in MXFP8 364-366, 382-384, 377-379, block 32768 x 2048 x 2048 271-273,
// 273-275, 290; products in MXFP4: 16640 x 8192 x 5120 373, 377-379, 379-381, 16384
// x 4096 x 1024 59, 59, 63, 8192 x 4096 x 4096 74, 74, 76; 16 groups of 16640 x 2048
// x 5120 170-172, 174, 173.  Seven is ahead at 12000 x 5120 x 2048 (block in MXFP4
// 188-192, 184-185, 184) and 8192 x 4096 x 4096 (block in MXFP8 241-242, 234,
// 243-246); a launch of small tiles does not show it.
constexpr int kMmBand = 5;

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

// Tiles.  Large: 256 x 256, by eight waves, two to a SIMD, or WIDE by four of
// 128 x 128 each, which read a third less from LDS but leave an epilogue fewer
// registers.  Small: 128 x 128 by four, two workgroups to a CU, or EIGHT by eight
// of 32 x 64, a quarter of a large tile in a launch of these.
template <int FX, int FW, bool LARGE, bool WIDE = false, bool EIGHT = false>
struct MmTile {
  static constexpr int kBX = WIDE ? 4 : EIGHT ? 1 : 2, kBW = LARGE ? 4 : 2;
  static constexpr int kWX = (LARGE && !WIDE) || EIGHT ? 4 : 2, kWW = 2;
  static constexpr int kPerCu = LARGE || EIGHT ? 1 : 2;
  static constexpr int kWaves = kWX * kWW, kThreads = 64 * kWaves;
  static constexpr int kRowsX = 32 * kBX * kWX, kRowsW = 32 * kBW * kWW;
  static constexpr int kX = 0;
  static constexpr int kW = kRowsX * MmFormat<FX>::kRow;
  static constexpr int kSX = kW + kRowsW * MmFormat<FW>::kRow;   // scales: 4 bytes a row
  static constexpr int kSW = kSX + kRowsX * 4;
  static constexpr int kLoadsS = (kRowsX + kRowsW + 64 * kWaves - 1) / 64 / kWaves;   // of scales, 256 bytes each
  static constexpr int kSlot = kSX + kLoadsS * kWaves * 256;   // (of eight waves' loads the last four may be for none)
  // as many slots as a workgroup's share of a CU's LDS holds, four at most
  static constexpr int kFit = 163840 / kPerCu / kSlot;
  static constexpr int kSlots = kFit > 4 ? 4 : kFit;
  static constexpr int kLds = kSlots * kSlot;
  static constexpr int kLoadsX = kW / (1024 * kWaves);   // loads of a wave, 1 KiB each
  static constexpr int kLoadsW = (kSX - kW) / (1024 * kWaves);
  static constexpr int kLoads = kLoadsX + kLoadsW + kLoadsS;
  static_assert(kLoadsS * kWaves * 64 >= kRowsX + kRowsW && kRowsX % 64 == 0 && kRowsW % 64 == 0,
                "a load's scales are one operand's");
  static_assert(kSlots >= 2 && (kSlots - 1) * kLoads < 64, "slots and the load counter");
};

struct MmArgs {
  const uint8_t *qx, *sx, *qw, *sw;
  int64_t m, n, k;             // rows of X; columns of R to a group (of each half where gated); depth
  const int32_t* ends;         // null: one group
  int32_t groups;
  int64_t w_bytes, sw_bytes;   // codes and scales of one group's W
  uint32_t tiles_m, tiles_n, per_xcd;
  uint32_t split;              // of each XCD's tiles the last that are taken in quarters
};

// A buffer range [base, base + bytes) for mm_load, as the halves of its descriptor.
struct MmRange {
  uint64_t lo, hi;
};
__device__ __forceinline__ MmRange mm_range(const void* base, uint32_t bytes) {
  return {(uint64_t)(uintptr_t)base, (uint64_t)0x00020000u << 32 | bytes};   // (the raw-buffer format of buffer_rsrc())
}

// 16 or 4 bytes a lane from memory to LDS at `to` (the wave's; lane order).  The
// compiler does not look into the asm for hazards.  A load may follow a write of
// its descriptor by the vector unit (v_readlane, v_readfirstlane: also where the
// compiler restores a spilled register) by five wait states at the earliest, but
// one by the scalar unit at once: the block copies the descriptor, which is also
// what has to stand between the write of m0 and the load.  (Waiting five states
// instead cost 1 to 2% of the products and 7% of 33 rows; the copies 0 to 3%.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // (m0 is reserved: no write of it by the compiler may move across)
template <int BYTES>
__device__ __forceinline__ void mm_load(uint32_t to, const MmRange& range, uint32_t offset) {
  static_assert(BYTES == 16 || BYTES == 4, "load sizes");
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b64 s[92:93], %2\n\ts_mov_b64 s[94:95], %3\n\t"
                 "buffer_load_dwordx4 %1, s[92:95], 0 offen lds" ::"s"(to), "v"(offset), "s"(range.lo), "s"(range.hi)
                 : "memory", "m0", "s92", "s93", "s94", "s95");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b64 s[92:93], %2\n\ts_mov_b64 s[94:95], %3\n\t"
                 "buffer_load_dword %1, s[92:95], 0 offen lds" ::"s"(to), "v"(offset), "s"(range.lo), "s"(range.hi)
                 : "memory", "m0", "s92", "s93", "s94", "s95");
}
#pragma clang diagnostic pop

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

// Where a workgroup's tile lies.
struct MmPlace {
  int64_t row0;       // its first row of X and of the result
  int32_t rows;       // how many
  int64_t srow0;      // its first row in X's scale layout, a multiple of 128
  uint32_t tn;        // its tile column
  int32_t group;
  int32_t quarter;    // 0 to 3 of the tile, or -1: all of it
};

// The tile of this workgroup: false if it has none (uniform; no barrier is
// left open).  XCD x (workgroups are dealt to the XCDs in turn) owns one of 8
// contiguous pieces of the ordered tiles: bands of kMmBand tile rows, column by
// column.  Grouped: a piece of each group's tiles, group after group.  `lds`
// holds the table of many groups meanwhile.
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
    uint32_t i = blockIdx.x / 8;
    const uint32_t whole = a.per_xcd - a.split;
    p.quarter = -1;
    if (i >= whole) {
      p.quarter = (int32_t)((i - whole) % 4);
      i = whole + (i - whole) / 4;
    }
    const uint32_t id = (blockIdx.x % 8) * a.per_xcd + i;
    if (i >= a.per_xcd || id >= a.tiles_m * a.tiles_n)
      return false;
    band_tile(id, a.tiles_m, tm);
    p.group = 0;
    p.row0 = (int64_t)tm * TILE;
    p.rows = (int32_t)min((int64_t)TILE, a.m - p.row0);
    p.srow0 = p.row0;
    return true;
  } else {
    const int32_t q = (int32_t)(blockIdx.x / 8), x = (int32_t)(blockIdx.x % 8);
    // A few groups: every wave finds its tile by itself in a uniform loop, the
    // ends eight at a time (past the last they repeat it: no rows).
    if (a.groups <= kScalarTableGroups) {
      int32_t run = 0, lo = 0, hi = 0, first = 0, part = 0;   // first: the group's first of each XCD's workgroups
      uint32_t trows = 0, pg = 0;
      int g = -1;
      // (constant memory to the kernel: scalar loads)
      const auto* all = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)a.ends;
      for (int g0 = 0; g0 < a.groups && g < 0; g0 += 8) {
        int32_t ends[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          ends[i] = all[min(g0 + i, a.groups - 1)];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          asm volatile("" : "+s"(ends[i]));   // (all on their way before the first is waited for)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (g < 0) {
            run = max(run, ends[i]);
            first += (int32_t)pg, part += (hi - lo + 127) / 128 * 128;
            lo = hi, hi = min(run, (int32_t)a.m);
            trows = (uint32_t)(hi - lo + TILE - 1) / TILE, pg = (trows * a.tiles_n + 7) / 8;
            if ((uint32_t)(q - first) < pg)
              g = g0 + i;
          }
        }
      }
      const uint32_t idx = (uint32_t)x * pg + (uint32_t)(q - first);
      if (g < 0 || idx >= trows * a.tiles_n)
        return false;
      band_tile(idx, trows, tm);
      p.group = g;
      p.row0 = lo + (int32_t)tm * TILE;
      p.rows = min(TILE, hi - (int32_t)p.row0);
      p.srow0 = part + (int32_t)tm * TILE;
      return true;
    }
    GroupTable& table = *reinterpret_cast<GroupTable*>(lds);
    int32_t* xs = reinterpret_cast<int32_t*>(lds + sizeof(GroupTable));
    if (threadIdx.x < 64) {
      build_group_table(a.ends, a.groups, (int32_t)a.m, TILE, table);
      build_piece_starts(table, a.groups, TILE, a.tiles_n, xs);
    }
    lds_barrier();
    GroupPiece piece;
    if (!find_group_piece(table, xs, a.groups, TILE, a.tiles_n, q, x, piece))
      return false;
    band_tile(piece.tile, piece.tile_rows, tm);
    const int32_t r0 = piece.lo + (int32_t)tm * TILE;
    p.group = piece.g;
    p.row0 = r0;
    p.rows = min(TILE, piece.hi - r0);
    p.srow0 = group_scale_row(table, piece.g) + (r0 - piece.lo);
    lds_barrier();   // every wave is done with the table
    return true;
  }
}

// A quarter of the place: its first column, and whether it holds anything.
// tile, cols: rows and columns of R of the whole tile.
__device__ __forceinline__ bool mm_quarter(const MmArgs& a, MmPlace& p, int tile, int64_t& col0, int cols) {
  const int down = p.quarter / 2 * (tile / 2);
  p.row0 += down, p.srow0 += down, p.rows = min(tile / 2, p.rows - down);
  col0 += p.quarter % 2 * (cols / 2);
  return p.rows > 0 && col0 < a.n;
}

// The tile's accumulators: acc[i][j] is the block of W rows 32 i and X rows
// 32 j of this wave's part, wave w's at (w / WW, w % WW).  GATED: the wave's W
// rows are 16 BW rows from its columns' gate half and the same of the factor
// half (n rows on), blocks i < BW / 2 and the others.  col0: the tile's first
// column of R.
template <int FX, int FW, class T, bool GATED>
__device__ __forceinline__ void mm_tile(const MmArgs& a, const MmPlace& p, int64_t col0, uint8_t* lds,
                                        v16f (&acc)[T::kBW][T::kBX]) {
  using X = MmFormat<FX>;
  using W = MmFormat<FW>;
  constexpr int kSlots = T::kSlots, BX = T::kBX, BW = T::kBW;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wx = wave / T::kWW, ww = wave % T::kWW;
  const int r = lane & 31, h = lane >> 5;

  const int ldx = (int)(FX == MX_FORMAT_E2M1 ? a.k / 2 : a.k), ldw = (int)(FW == MX_FORMAT_E2M1 ? a.k / 2 : a.k);
  const int strip = (int)((a.k / 32 + 3) / 4) * 512;   // a 128-row strip of a scale layout
  const int stages = (int)((a.k + kMmK - 1) / kMmK);

  const MmRange rx = mm_range(a.qx + p.row0 * ldx, (uint32_t)p.rows * (uint32_t)ldx);
  // W: one range, or the gate's and the factor's
  constexpr int kCols = GATED ? T::kRowsW / 2 : T::kRowsW;
  const int cols = (int)min((int64_t)kCols, a.n - col0);
  const uint8_t* wbase = a.qw + p.group * a.w_bytes + col0 * ldw;
  const MmRange rw = mm_range(wbase, (uint32_t)cols * (uint32_t)ldw);
  const MmRange ru = GATED ? mm_range(wbase + a.n * ldw, (uint32_t)cols * (uint32_t)ldw) : rw;

  const uint32_t lds0 =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);

  // Loader roles.  Code load u of wave w fills 1 KiB: the stage rows from u *
  // kXRows + w * (64 / chunks) on; the lane's row of them, its chunk of memory.
  constexpr int kXEach = 64 / X::kChunks, kWEach = 64 / W::kChunks;             // rows of a load
  constexpr int kXRows = T::kWaves * kXEach, kWRows = T::kWaves * kWEach;       // rows from load to load
  const int xrow = kXEach * wave, wrow = kWEach * wave;
  const int xchunk = (lane % X::kChunks) ^ mm_swizzle<X::kChunks>(xrow + lane / X::kChunks);
  const int wchunk = (lane % W::kChunks) ^ mm_swizzle<W::kChunks>(wrow + lane / W::kChunks);
  const uint32_t xoff = lane / X::kChunks * ldx + 16 * xchunk, woff = lane / W::kChunks * ldw + 16 * wchunk;
  // Scales: word d of an operand's stage is row 32 B (d / 32 B) + 32 (d % B) +
  // d / B % 32 of the tile, B its blocks to a wave, so that a lane finds its
  // row's words of those blocks together.  Load u of wave w brings words 64 (u
  // * waves + w) on, X's first.
  const int64_t scol0 = col0 / 128 * 128;
  MmRange rs[T::kLoadsS];
  uint32_t soff[T::kLoadsS];
#pragma unroll
  for (int u = 0; u < T::kLoadsS; ++u) {
    const bool of_x = u * T::kWaves + wave < T::kRowsX / 64;
    rs[u] = of_x ? mm_range(a.sx + p.srow0 / 128 * strip, (uint32_t)((p.rows + 127) / 128 * strip))
                 : mm_range(a.sw + p.group * a.sw_bytes + scol0 / 128 * strip,
                               (uint32_t)(a.sw_bytes - scol0 / 128 * strip));
    const int d = threadIdx.x + u * T::kThreads - (of_x ? 0 : T::kRowsX), B = of_x ? BX : BW;
    int64_t row = 32 * B * (d / (32 * B)) + 32 * (d % B) + d / B % 32;   // in the scale layout, from the range's start
    if (!of_x) {
      if constexpr (GATED) {
        constexpr int kHalf = 16 * BW;
        const int in = (int)row % (2 * kHalf);
        row = (int)row / (2 * kHalf) * kHalf + in % kHalf + (in >= kHalf ? a.n : 0);
      }
      row += col0 - scol0;
    }
    soff[u] = (uint32_t)(row / 128 * strip + 16 * (row % 32) + 4 * (row % 128 / 32));
    if (u * T::kWaves + wave >= (T::kRowsX + T::kRowsW) / 64)
      soff[u] = 0, rs[u] = mm_range(a.sw, 0);
  }

  // load i of stage t into slot b: X, W, scales
  auto load = [&](int i, int t, int b) {
    const uint32_t to = lds0 + b * T::kSlot;
    if (i < T::kLoadsX) {
      const uint32_t off = 16 * xchunk + t * X::kRow < ldx ? xoff + t * X::kRow : 0x80000000u;
      mm_load<16>(to + T::kX + (i * T::kWaves + wave) * 1024, rx, off + (uint32_t)((i * kXRows + xrow) * ldx));
    } else if (i < T::kLoadsX + T::kLoadsW) {
      const int u = i - T::kLoadsX;
      int row = u * kWRows + wrow;
      bool up = false;
      if constexpr (GATED) {
        constexpr int kHalf = 16 * BW;   // (a multiple of kWEach: a load's rows are of one half)
        up = row % (2 * kHalf) >= kHalf;
        row = row / (2 * kHalf) * kHalf + row % kHalf;
      }
      const uint32_t off = 16 * wchunk + t * W::kRow < ldw ? woff + t * W::kRow : 0x80000000u;
      mm_load<16>(to + T::kW + (u * T::kWaves + wave) * 1024, GATED && up ? ru : rw, off + (uint32_t)(row * ldw));
    } else {
      const int u = i - T::kLoadsX - T::kLoadsW;
      mm_load<4>(to + T::kSX + (u * T::kWaves + wave) * 256, rs[u], soff[u] + t * 512);
    }
  };

  // Operands of a step: [block][word]; and the words of scales of a stage.
  typedef u32x4 OpX[BX][X::kWords];
  typedef u32x4 OpW[BW][W::kWords];
  constexpr int kReads = BX * X::kWords + BW * W::kWords;
  const int fx = mm_swizzle<X::kChunks>(r), fw = mm_swizzle<W::kChunks>(r);
  const int xat = T::kX + (wx * 32 * BX + r) * X::kRow, wat = T::kW + (ww * 32 * BW + r) * W::kRow;
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
    else if (q < W::kWords + BX * X::kWords)
      one_x((q - W::kWords) / X::kWords, (q - W::kWords) % X::kWords);
    else
      one_w((q - BX * X::kWords) / W::kWords, (q - BX * X::kWords) % W::kWords);
  };
  auto read_words = [&](const uint8_t* at, auto& s) {
    constexpr int B = (int)std::extent_v<std::remove_reference_t<decltype(s)>>;
    typedef uint32_t Words __attribute__((ext_vector_type(B)));
    const Words v = *reinterpret_cast<const Words*>(at + r * B * 4);
#pragma unroll
    for (int i = 0; i < B; ++i)
      s[i] = v[i];
  };
  uint32_t sx[BX], sw[BW], nx[BX], nw[BW];
  auto read_scales = [&](int b) {
    read_words(lds + b * T::kSlot + T::kSX + wx * 128 * BX, nx);
    read_words(lds + b * T::kSlot + T::kSW + ww * 128 * BW, nw);
  };
  auto wide_op = [](const auto& o) {
    if constexpr (std::extent_v<std::remove_reference_t<decltype(o)>> == 2)
      return (v8i){(int)o[0][0], (int)o[0][1], (int)o[0][2], (int)o[0][3],
                   (int)o[1][0], (int)o[1][1], (int)o[1][2], (int)o[1][3]};
    else
      return (v8i){(int)o[0][0], (int)o[0][1], (int)o[0][2], (int)o[0][3], 0, 0, 0, 0};
  };
  // MFMA q of step s: scale byte 2 s + h of a row's word, taken from 2 s on
  constexpr int kMfmas = BX * BW;
  auto mfma = [&](auto s_c, int q, const OpX& ox, const OpW& ow) {
    constexpr int kByte = 2 * decltype(s_c)::value;
    const int i = q / BX, j = q % BX;
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide_op(ow[i]), wide_op(ox[j]), acc[i][j], W::kCode,
                                                                X::kCode, kByte, (int)sw[i], kByte, (int)sx[j]);
  };

#pragma unroll
  for (int i = 0; i < BW; ++i)
#pragma unroll
    for (int j = 0; j < BX; ++j)
      acc[i][j] = (v16f){};
  if (stages == 0)
    return;

  // A stage's loads are issued in two steps, but with two slots in one (the
  // second would be late).
  constexpr int kFirst = kSlots > 2 ? (T::kLoads + 1) / 2 : T::kLoads, kSecond = T::kLoads - kFirst;
#pragma unroll
  for (int t = 0; t < kSlots; ++t)
#pragma unroll
    for (int i = 0; i < (t == kSlots - 1 ? kFirst : T::kLoads); ++i)
      load(i, t, t);
  mm_wait_loads<(kSlots - 2) * T::kLoads + kFirst>();
  lds_barrier();
  OpX x0, x1;
  OpW w0, w1;
  read_scales(0);
#pragma unroll
  for (int q = 0; q < kReads; ++q)
    read(q, 0, 0, x0, w0);

  // Stage t in slot b.  First step: its MFMAs, the reads of the second step's
  // operands and the last loads of stage t + kSlots - 1 into the slot before.
  // Then, once this wave's loads of stage t + 1 have landed and every wave has
  // read slot b, the second step: its MFMAs, the first loads of stage t +
  // kSlots into slot b and the reads of stage t + 1's first step.
  // The reads stand after the first half of the MFMAs, so that the others
  // cover their latency.
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  auto reads_by = [](int q) { return min(q * 2 * kReads / kMfmas, kReads); };
  // A row's scales of a stage: bytes h and h + 2 of a word to bits 0 and 16, and
  // 0 for blocks past K (the layout's padding may hold anything, a NaN too).
  const int tail = min(24, 8 * ((int)(a.k / 32) - 4 * (stages - 1) - h));
  int b = 0;
  for (int t = 0; t < stages; ++t) {
    const uint32_t bits = t == stages - 1 ? tail : 24;
#pragma unroll
    for (int i = 0; i < BW; ++i)
      sw[i] = __builtin_amdgcn_ubfe(nw[i], 8 * h, bits);
#pragma unroll
    for (int j = 0; j < BX; ++j)
      sx[j] = __builtin_amdgcn_ubfe(nx[j], 8 * h, bits);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < kMfmas; ++q) {
      mfma(S0(), q, x0, w0);
#pragma unroll
      for (int i = kFirst + q * kSecond / kMfmas; i < kFirst + (q + 1) * kSecond / kMfmas; ++i)
        load(i, t + kSlots - 1, b == 0 ? kSlots - 1 : b - 1);
#pragma unroll
      for (int u = reads_by(q); u < reads_by(q + 1); ++u)
        read(u, 1, b, x1, w1);
      __builtin_amdgcn_sched_barrier(0);
    }
    mm_wait_loads<(kSlots - 2) * T::kLoads>();
    lds_barrier();
    const int nb = b + 1 == kSlots ? 0 : b + 1;
    read_scales(nb);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < kMfmas; ++q) {
      mfma(S1(), q, x1, w1);
#pragma unroll
      for (int i = q * kFirst / kMfmas; i < (q + 1) * kFirst / kMfmas; ++i)
        load(i, t + kSlots, b);
#pragma unroll
      for (int u = reads_by(q); u < reads_by(q + 1); ++u)
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

// Whether a result of m rows and n columns is taken in large tiles: where they
// nearly fill the GPU.  tile_cols: columns of R that a large tile covers.
// (Timed, large against small, us: 256 tiles, 4096 x 4096 x 4096 with MXFP8 rows 52
// against 60; 128 tiles, 4096 x 2048 x 2048 25 against 18; 64 tiles, 2048 x 2048 x
// 4096 in 4 bits 27 against 14.  Groups are taken as even, and a tile counts whether
// it is full or not.  16640 rows of 2048 columns: 16 uneven groups, k 5120, 173
// against 189, in MXFP4 130 against 148; k 2048 in even groups: 32 of 520 rows 88
// against 88, in 64 of 260 in MXFP4 95 against 98.  It loses where groups end just
// past a large tile: 16 of 1040 rows 83 against 72, 64 of 260 121 against 112, 16 of
// 130 rows and 5120 columns 52 against 42; and a block of 4099 x 1056 x 1088 in 4
// groups takes 18.1 in small tiles where large ones take 16.1 to 17.1.)
inline bool mm_large(int64_t m, int64_t n, int32_t groups, int tile_cols) {
  const int64_t rows = groups > 1 ? m / groups : m;   // (of a group, if they were even)
  const int64_t tiles = (rows + 255) / 256 * (groups > 1 ? groups : 1) * ((n + tile_cols - 1) / tile_cols);
  return tiles >= 192;
}

// Tiles of a launch, and its workgroups.  cols_tile: columns of R to a tile.
// A workgroup with a large tile has a CU to itself, and an XCD 32 of them: where
// few of an XCD's tiles are left after whole rounds, these are taken in quarters.
inline int64_t mm_grid(MmArgs& a, int tile, int cols_tile, bool quarters = false) {
  const int64_t groups = a.ends != nullptr ? a.groups : 0;
  const int64_t tm = (a.m + tile - 1) / tile + groups, tn = (a.n + cols_tile - 1) / cols_tile;
  const int64_t per = (tm * tn + 7) / 8 + groups;
  a.tiles_m = (uint32_t)tm, a.tiles_n = (uint32_t)tn, a.per_xcd = (uint32_t)per;
  a.split = quarters && groups == 0 && per > 32 && per % 32 <= kMmSplit ? (uint32_t)(per % 32) : 0;
  return (per + 3 * a.split) * 8;
}

}  // namespace mx
