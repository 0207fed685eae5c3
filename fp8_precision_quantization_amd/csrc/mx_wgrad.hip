// Weight gradient of a linear layer from the 8-bit checkpoint of its input:
//
//   dw_g[i][j] = sum over tokens t of group g of dy[t][i] * x[t][j],
//   x[t][j] = e4m3(q[t][j]) * 2^(s[t][j / 32] - 127).
//
// The sum runs over tokens, along which a checkpoint's scales change from
// element to element of a column, so the block-scaled MFMA does not apply:
// the codes are turned into bf16 (exact: four significant bits times a power
// of two) and the product runs on the bf16 MFMA with binary32 accumulators.
//
// Work decomposition.  A 256-thread workgroup owns a tile of 32 NB x 32 NB of
// one group's dw, 256 x 256 (NB = 8, one workgroup to a CU) or 128 x 128 (NB =
// 4, two); wave w its (w / 2, w % 2) quarter, NB x NB blocks of
// v_mfma_f32_16x16x32_bf16, whose accumulators live in the accumulation
// registers.  Tokens advance in stages of 64.  A stage's pieces of dy (bf16),
// of the codes and of the scales lie in LDS token-major as in memory, three
// stages deep, brought there by loads that go straight from memory to LDS.
// Keeping the codes in LDS as codes halves what the waves read of x (LDS
// bandwidth, not the matrix cores, bound the kernel while LDS held bf16 x);
// each wave converts what it reads, between the MFMAs of the half stage
// before.  Tiles that do not fill a last round, and groups much longer than
// their share, are cut along the tokens; the pieces' sums are added up in a
// fixed order by a second kernel.
//
// Measured: 16640 x 8192 x 5120, bf16 out, 1030 - 1115 us from one MI355X to
// another (1.25 - 1.35 PFLOP/s; the library's bf16 product of that shape 0.91,
// of its best shape 1.58); the MFMAs take 68% of its cycles, at a clock that
// they pull down to 2.0 - 2.1 GHz.  16 groups of 16640 tokens, 1024 x 1024,
// binary32 out, 54 - 58 us; 4099 x 250 x 1056 19 us.  These wait for the start and
// the end of their workgroups (12 us a 256 x 256 tile, 5 us a 128 x 128 one):
// the first stages' loads, and stores that nothing overlaps.
//
// An MFMA operand is eight consecutive tokens of one column in a lane, down a
// column of the stage.
//  - dy: ds_read_b64_tr_b16, its lane layout checked on MI355X: within each 16
//    lanes, lane i addresses 8 bytes, and receives as element e the (i % 4)-th
//    16-bit value of the 8 bytes lane 4 e + i / 4 addressed; so with lane i on
//    token i / 4, columns 4 (i % 4) .. + 3, lane i ends with column i of four
//    tokens.  Two such reads make an operand.
//  - x: the lane takes 8 neighbouring columns of 8 tokens, 8 bytes from each,
//    and converts a token's column pairs under that token's scale (one
//    instruction a pair); byte permutes then bring the tokens of a column
//    together.  So column c of block b is column 8 c + b of the wave's 128,
//    and the 8 blocks' results of a lane are 8 neighbouring columns of dw:
//    the epilogue stores them as they are.
//
// LDS banks: dy's row is 512 bytes, a multiple of the banks' period, and one
// read touches tokens t .. t + 3 of two or four groups of eight: the 32-byte
// pieces of a row are permuted by XOR with (t % 4, t / 8 % 2), 3 bits, and the
// 128-byte halves of a row of codes by XOR with t / 8 % 2, both through the
// source addresses of the loads.
//
// Rows past the end of the token range load as zero in both operands; columns
// past n or k may hold anything: they only reach outputs that are not stored.
#include "mx_train.h"
#include "mx_train_launch.h"
#include "mxtrain.h"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace mx {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

constexpr int kWgThreads = 256;
constexpr int kWgTokens = 64;                        // tokens per stage
constexpr int kWgSlots = 3;                          // stages in LDS
constexpr int kWgCus = 256;
constexpr int kWgScaleRow = 4 * kWgTokens + 16;      // a block's scales (16 bytes more than the banks' period)

// Sizes of a tile of 32 NB x 32 NB: a wave has NB x NB blocks of 16 x 16.
template <int NB>
struct WgTile {
  static constexpr int kTile = 32 * NB;
  static constexpr int kRow = 2 * kTile;             // bytes of a stage row of dy
  static constexpr int kX = kWgTokens * kRow;        // where the codes start in a stage: rows of kTile bytes
  static constexpr int kS = kX + kWgTokens * kTile;  // where the scales start: a dword each, [block of 32][token]
  static constexpr int kSlot = (kS + NB * kWgScaleRow + 255) / 256 * 256;
  static constexpr int kPerCu = NB == 8 ? 1 : 2;     // workgroups
  static constexpr int kLoadsDy = NB, kLoadsX = NB / 2, kLoadsS = NB / 4;   // a wave's to a stage
  static constexpr int kLoads = kLoadsDy + kLoadsX + kLoadsS;
  static_assert(NB == 4 || NB == 8, "tiles");
  static_assert(kPerCu * kWgSlots * kSlot <= 160 * 1024, "stages fit LDS");
};

struct WgradArgs {
  const uint16_t* dy;
  int64_t n_read;          // columns of a row of dy that may be read, n or more
  const uint8_t *q, *s;
  const int32_t* ends;
  void* out;
  float* part;        // sums of pieces, a whole tile each
  int64_t lddy, n, k;
  int32_t rows, groups;
  uint32_t tiles_n, tiles_k;
  // One group: the first `whole` tiles are not cut, the others into `pieces`.
  // Several: `pieces` slots for groups or pieces of groups, a piece being
  // `piece_stages` long or thereabouts.
  uint32_t whole, pieces;
  int32_t piece_stages;
};

// What a workgroup works on: a tile of group g over tokens [lo, hi), into the
// output (part < 0) or into tile `part` of the pieces' sums.
struct WgradItem {
  int32_t g, lo, hi, part;
};

// Pieces of a group of `stages` stages, and the token range of one.
__device__ __forceinline__ int32_t group_pieces(int32_t stages, int32_t piece_stages) {
  return max(1, (stages + piece_stages / 2) / piece_stages);
}
__device__ __forceinline__ void piece_range(int32_t pieces, int32_t piece, int32_t& lo, int32_t& hi) {
  const int32_t stages = (hi - lo + kWgTokens - 1) / kWgTokens, each = (stages + pieces - 1) / pieces;
  const int32_t first = min(piece * each, stages);
  hi = min((int64_t)hi, (int64_t)lo + (int64_t)min(first + each, stages) * kWgTokens);
  lo = min((int64_t)hi, (int64_t)lo + (int64_t)first * kWgTokens);
}

// The groups' schedule, found by one wave with a group to a lane: which group
// and piece has slot `slot` (by_slot), or is the slot-th of the groups that
// are cut.  Group g's tokens are [min(max(0, ends_0 .. ends_{g-1}), rows),
// min(max(0, ends_0 .. ends_g), rows)).  Up to 64 groups come longest piece
// first, more in their own order.  Returns false past the last; g, lo, hi are
// the group's, `first_part` the number of pieces of cut groups before it.
__device__ __forceinline__ bool find_slot(const WgradArgs& a, int32_t slot, bool by_slot, int32_t& g, int32_t& lo,
                                          int32_t& hi, int32_t& pieces, int32_t& piece, int32_t& first_part) {
  const int lane = threadIdx.x & 63;
  int32_t run = 0, slots = 0, parts = 0, cuts = 0;   // of the groups before these 64
  for (int32_t g0 = 0; g0 < a.groups; g0 += 64) {
    const bool on = g0 + lane < a.groups;
    int32_t end = on ? max(a.ends[g0 + lane], 0) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(end, d);
      if (lane >= d)
        end = max(end, o);
    }
    end = min(max(end, run), a.rows);
    const int32_t up = __shfl_up(end, 1);
    const int32_t begin = lane == 0 ? min(run, a.rows) : up;
    run = __builtin_amdgcn_readlane(end, 63);
    const int32_t stages = (end - begin + kWgTokens - 1) / kWgTokens;
    const int32_t count = on ? group_pieces(stages, a.piece_stages) : 0;
    const int32_t len = (stages + max(count, 1) - 1) / max(count, 1);
    int32_t my_slots = 0, my_parts = 0, my_cuts = 0;
    const int n = min(a.groups - g0, 64);
    for (int q = 0; q < n; ++q) {
      const int32_t c = __builtin_amdgcn_readlane(count, q), l = __builtin_amdgcn_readlane(len, q);
      const bool before = a.groups <= 64 ? l > len || (l == len && q < lane) : q < lane;
      if (before) {
        my_slots += c;
        my_parts += c > 1 ? c : 0;
        my_cuts += c > 1;
      }
    }
    my_slots += slots, my_parts += parts, my_cuts += cuts;
    const bool hit = by_slot ? on && my_slots <= slot && slot < my_slots + count : on && count > 1 && my_cuts == slot;
    const uint64_t at = __ballot(hit);
    if (at != 0) {
      const int src = __builtin_ctzll(at);
      g = g0 + src;
      lo = __builtin_amdgcn_readlane(begin, src);
      hi = __builtin_amdgcn_readlane(end, src);
      pieces = __builtin_amdgcn_readlane(count, src);
      piece = slot - __builtin_amdgcn_readlane(my_slots, src);
      first_part = __builtin_amdgcn_readlane(my_parts, src);
      return true;
    }
    for (int q = 0; q < n; ++q) {
      const int32_t c = __builtin_amdgcn_readlane(count, q);
      slots += c;
      parts += c > 1 ? c : 0;
      cuts += c > 1;
    }
  }
  return false;
}

// Blocks of a segment of `tiles` tiles, and the tile of its block b, or -1.
// The workgroups of an XCD (every eighth) take neighbouring tiles, which share
// operands in its L2; few tiles go to the XCDs in turn instead, so that none
// is left without.
constexpr uint32_t kWgSpread = 64;
__host__ __device__ inline uint32_t segment_blocks(uint32_t tiles) {
  return tiles % 8 == 0 || tiles < kWgSpread ? tiles : (tiles + 7) / 8 * 8;
}
__device__ __forceinline__ int32_t segment_tile(uint32_t tiles, uint32_t b) {
  if (tiles % 8 != 0 && tiles < kWgSpread)
    return (int32_t)b;
  const uint32_t tile = b % 8 * ((tiles + 7) / 8) + b / 8;
  return tile < tiles ? (int32_t)tile : -1;
}

// 16 bytes per lane, or one byte widened to a dword, from memory into LDS, in
// lane order from `to` on (the same in every lane).  With the compiler's own
// form of it every later read from LDS would wait for the load, since the
// transposing reads carry nothing that tells the stages apart; here the caller
// waits (vmcnt) and meets the other waves at a barrier before anything is
// read.  (m0, which holds the LDS address, is not a register the compiler
// keeps values in.)
// lds_target() and the load have another instruction between them, as a write
// of m0 before its use asks for.
__device__ __forceinline__ void lds_target(uint32_t to) { asm volatile("s_mov_b32 m0, %0" ::"s"(to)); }
template <int BYTES>
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rsrc, int offset) {
  static_assert(BYTES == 16 || BYTES == 1, "load sizes");
  if constexpr (BYTES == 16)
    asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(offset), "s"(rsrc) : "memory");
  else
    asm volatile("buffer_load_ubyte %0, %1, 0 offen lds" ::"v"(offset), "s"(rsrc) : "memory");
}

// f(0), f(1), .. with the numbers as constants.
template <class F, int... I>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}

// A run of rows that loads walk through, a stage at a time: range checks see
// `left` bytes from `at` on.
struct Run {
  const uint8_t* at;
  int64_t left, by;
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc() const {
    return buffer_rsrc(at, (uint32_t)min(max(left, (int64_t)0), (int64_t)INT32_MAX));
  }
  __device__ __forceinline__ void next() {
    if (left > 0)
      at += by;   // (never far past the end of the array)
    left -= by;
  }
};

// Until at most N of the wave's loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "vmcnt has six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4 << 14));
}

template <int NB, bool VEC, bool BF16>
__global__ __launch_bounds__(kWgThreads)
    __attribute__((amdgpu_waves_per_eu(WgTile<NB>::kPerCu, WgTile<NB>::kPerCu))) void wgrad_kernel(WgradArgs a) {
  using Tile = WgTile<NB>;
  constexpr int kTile = Tile::kTile, kRow = Tile::kRow, kSlot = Tile::kSlot;
  __shared__ __attribute__((aligned(256))) uint8_t lds[kWgSlots * kSlot];
  const uint32_t tiles = a.tiles_n * a.tiles_k;
  WgradItem it = {0, 0, a.rows, -1};
  int32_t tile;
  if (a.groups == 1) {
    if (a.ends != nullptr)
      it.hi = min(max(a.ends[0], 0), a.rows);
    const uint32_t first = segment_blocks(a.whole);
    if (blockIdx.x < first) {
      tile = segment_tile(a.whole, blockIdx.x);
    } else {
      const uint32_t cut = tiles - a.whole, per = segment_blocks(cut), piece = (blockIdx.x - first) / per;
      tile = segment_tile(cut, (blockIdx.x - first) % per);
      it.part = tile < 0 ? 0 : (int32_t)(piece * cut + (uint32_t)tile);
      tile = tile < 0 ? tile : tile + (int32_t)a.whole;
      piece_range((int32_t)a.pieces, (int32_t)piece, it.lo, it.hi);
    }
  } else {
    const uint32_t per = segment_blocks(tiles);
    tile = segment_tile(tiles, blockIdx.x % per);
    int32_t pieces, piece, first_part;
    if (!find_slot(a, (int32_t)(blockIdx.x / per), true, it.g, it.lo, it.hi, pieces, piece, first_part))
      return;   // uniform, before any barrier
    if (pieces > 1) {
      it.part = (first_part + piece) * (int32_t)tiles + max(tile, 0);
      piece_range(pieces, piece, it.lo, it.hi);
    }
  }
  if (tile < 0)
    return;
  // values that came through vector registers, made scalar
  const int32_t g = __builtin_amdgcn_readfirstlane(it.g), part = __builtin_amdgcn_readfirstlane(it.part);
  const int32_t lo = __builtin_amdgcn_readfirstlane(it.lo), hi = __builtin_amdgcn_readfirstlane(it.hi);
  const int64_t i0 = (int64_t)((uint32_t)tile / a.tiles_k) * kTile, j0 = (int64_t)((uint32_t)tile % a.tiles_k) * kTile;

  const int t = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lane = t & 63;
  const int wi = wave >> 1, wj = wave & 1;
  const int64_t ks = a.k / MX_BLOCK;

  f32x4 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      acc[i][j] = (f32x4){};

  // Loader roles.  A load of a wave brings 1 KiB, whole rows of a stage:
  //  dy: kDyRows rows; lane l the 16 bytes at position l % kDyLanes of its
  //  row, whose source is chunk (l % kDyLanes) ^ 2 f, f = row % 4 + 4 (row / 8
  //  % 2).
  //  codes: kXRows rows; lane l position l % kXLanes of its row, whose source
  //  is chunk (l % kXLanes) ^ kXLanes / 2 (row / 8 % 2).
  //  scales: a block; lane l is token l.
  constexpr int kDyLanes = kRow / 16, kDyRows = 64 / kDyLanes, kXLanes = kTile / 16, kXRows = 64 / kXLanes;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);
  const int drow = kDyRows * wave + lane / kDyLanes;   // of load 0; load u: + 4 kDyRows u
  const int dchunk = (lane % kDyLanes) ^ (2 * (drow & 3)) ^ (drow & 8);
  auto dchunk_of = [&](int u) { return dchunk ^ (4 * kDyRows * u & 8); };
  const int doff = drow * (int)a.lddy * 2 + 16 * dchunk, doff1 = drow * (int)a.lddy * 2 + 16 * dchunk_of(1);
  const int xrow = kXRows * wave + lane / kXLanes;     // load u: + 4 kXRows u, a multiple of 16
  const int xoff = xrow * (int)a.k + 16 * ((lane % kXLanes) ^ (kXLanes / 2 * (xrow >> 3 & 1)));
  const int soff = lane * (int)ks + Tile::kLoadsS * wave;
  const int64_t dy_end = (int64_t)(a.rows - 1) * a.lddy + a.n;   // elements of dy
  u32x4 dreg[VEC ? 1 : Tile::kLoadsDy];

  // The next stage to load, and load i of it (dy, then codes, then scales;
  // from kFirstLoad on where dy goes through registers) into slot `slot`.
  // Past the last stage they load zeros.
  const int64_t tokens = hi - lo;
  Run run_dy = {reinterpret_cast<const uint8_t*>(a.dy + lo * a.lddy + i0), ((tokens - 1) * a.lddy + a.n_read - i0) * 2,
                kWgTokens * a.lddy * 2};
  Run run_q = {a.q + lo * a.k + j0, tokens * a.k - j0, kWgTokens * a.k};
  Run run_s = {a.s + lo * ks + j0 / MX_BLOCK, tokens * ks - j0 / MX_BLOCK, kWgTokens * ks};
  constexpr int kX0 = Tile::kLoadsDy, kS0 = kX0 + Tile::kLoadsX, kLoads = Tile::kLoads;
  auto target = [&](int i, int slot) {
    const uint32_t to = lds0 + slot * kSlot;
    lds_target(to + (i < kX0   ? (4 * i + wave) * kDyRows * kRow
                     : i < kS0 ? Tile::kX + (4 * (i - kX0) + wave) * kXRows * kTile
                               : Tile::kS + (Tile::kLoadsS * wave + i - kS0) * kWgScaleRow));
  };
  auto load = [&](int i) {
    if (i < kX0)
      load_to_lds<16>(run_dy.rsrc(), (i % 2 ? doff1 : doff) + 4 * i * kDyRows * (int)a.lddy * 2);
    else if (i < kS0)
      load_to_lds<16>(run_q.rsrc(), xoff + 4 * (i - kX0) * kXRows * (int)a.k);
    else
      load_to_lds<1>(run_s.rsrc(), soff + i - kS0);
  };
  auto next_stage = [&]() {
    run_dy.next();
    run_q.next();
    run_s.next();
  };
  constexpr int kFirstLoad = VEC ? 0 : kX0, kStageLoads = kLoads - kFirstLoad, kHalfLoads = kStageLoads / 2;
  auto load_stage = [&](int slot, int loads) {
#pragma unroll
    for (int i = kFirstLoad; i < kFirstLoad + loads; ++i) {
      target(i, slot);
      asm volatile("s_nop 0");
      load(i);
    }
  };
  // dy at any alignment: through registers, 16 bytes at a time; what lies
  // past column n belongs to columns that are not stored.  Only at the very
  // end of dy, element by element.
  auto load_dy = [&](int st) {
    if constexpr (!VEC) {
      const int32_t m0 = lo + st * kWgTokens;
      const int32_t left = min(hi - m0, kWgTokens);
#pragma unroll
      for (int u = 0; u < Tile::kLoadsDy; ++u) {
        const int row = 4 * kDyRows * u + drow;
        const int64_t c = i0 + 8 * dchunk_of(u);
        dreg[u] = (u32x4){0, 0, 0, 0};
        if (row < left && c < a.n) {
          const int64_t at = (int64_t)(m0 + row) * a.lddy + c;
          if (at + 8 <= dy_end) {
            dreg[u] = *reinterpret_cast<const u32x4_any*>(a.dy + at);
          } else {
            for (int e = 0; e < dy_end - at; ++e)
              dreg[u][e / 2] |= (uint32_t)a.dy[at + e] << (16 * (e & 1));
          }
        }
      }
    }
  };
  auto put_dy = [&](int slot) {
    if constexpr (!VEC) {
#pragma unroll
      for (int u = 0; u < Tile::kLoadsDy; ++u)
        *reinterpret_cast<u32x4*>(lds + slot * kSlot + (4 * kDyRows * u + drow) * kRow + 16 * (lane % kDyLanes)) = dreg[u];
    }
  };

  // MFMA role: lane l holds column (of dy or x) l % 16 of a block, tokens 8
  // (l / 16) .. + 7 of a step's 32.
  const int l16 = lane & 15, lg = lane >> 4;
  const int tok = 8 * lg + (l16 >> 2);                        // dy reads: this token, and + 4
  const int swz = (tok & 3) | ((lg & 1) << 2);
  typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
  typedef s16x4 Dy[NB][2];              // a step's dy operands: 8 tokens of a column, in two reads
  typedef uint32_t X[NB][4];            // ... and its x operands
  struct Codes {
    uint32_t q[8][NB / 4];              // NB columns of each of 8 tokens
    u32x4 s[2];                         // those tokens' scale bytes
  };
  // where the lane reads in the slot of the step that is read next
  int d_at[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
    d_at[i] = tok * kRow + 32 * ((NB * wi + i) ^ swz) + 8 * (lane & 3);
  int x_at = Tile::kX + 8 * lg * kTile + kTile / 2 * (wj ^ (lg & 1)) + NB * l16;
  int s_at = Tile::kS + (NB / 2 * wj + NB * l16 / 32) * kWgScaleRow + 32 * lg;
  auto read_dy = [&](int step, int r, Dy& d) {                // r: 0 .. 2 NB - 1
    const uint8_t* p = lds + d_at[r / 2] + (32 * step + 4 * (r % 2)) * kRow;
    d[r / 2][r % 2] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
  };
  auto read_scales = [&](int step, int r, Codes& c) {         // r: 0, 1
    c.s[r] = *reinterpret_cast<const u32x4*>(lds + s_at + 128 * step + 16 * r);
  };
  auto read_codes = [&](int step, int r, Codes& c) {          // r: 0 .. 7
    const uint8_t* p = lds + x_at + (32 * step + r) * kTile;
    if constexpr (NB == 8) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      c.q[r][0] = v[0], c.q[r][1] = v[1];
    } else {
      c.q[r][0] = *reinterpret_cast<const uint32_t*>(p);
    }
  };
  // Columns 2 p, 2 p + 1 of tokens 2 u, 2 u + 1: a dword of x blocks 2 p, 2 p
  // + 1, in three parts of two instructions.
  uint32_t pair[2];
  auto convert = [&](int p, int u, int part, const Codes& c, X& x) {
    if (part < 2) {
      const int tk = 2 * u + part;
      const float sc = __uint_as_float(c.s[tk / 4][tk % 4] << 23);
      pair[part] =
          __builtin_bit_cast(uint32_t, p % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.q[tk][p / 2], sc, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.q[tk][p / 2], sc, false));
    } else {
      x[2 * p][u] = __builtin_amdgcn_perm(pair[1], pair[0], 0x05040100u);
      x[2 * p + 1][u] = __builtin_amdgcn_perm(pair[1], pair[0], 0x07060302u);
    }
  };
  auto mfma = [&](int m, const Dy& d, const X& x) {
    const int i = m % NB, j = m / NB;
    const bf16x8 fa =
        __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(d[i][0], d[i][1], 0, 1, 2, 3, 4, 5, 6, 7));
    const bf16x8 fb = __builtin_bit_cast(bf16x8, (u32x4){x[j][0], x[j][1], x[j][2], x[j][3]});
    // v_mfma_f32_16x16x32_bf16 with the accumulators tied to accumulation
    // registers: given the intrinsic, the compiler moves NB = 8's 64 of them
    // about (428 register moves a stage).  Every operand was written at least
    // one MFMA earlier; the results are read after the wait below the loop.
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[i][j]) : "v"(fa), "v"(fb));
  };

  // A stage is two steps of 32 tokens, NB * NB MFMAs each, x block after x
  // block.  In the first step of stage st the wave waits for its loads of
  // stage st + 1 and meets the others at the stage's one barrier; all of stage
  // st has been read by then, and its slot takes the loads of stage st + 3:
  // half of them in the second step, half in the first of stage st + 1.
  constexpr int kM = NB * NB;
  auto arrive = [&](int to) {
    next_stage();
    put_dy(to);   // where dy comes through registers
    wait_loads<kStageLoads>();
    lds_barrier();
  };
  const int stages = (hi - lo + kWgTokens - 1) / kWgTokens;
  if (stages > 0) {
    load_dy(0);
    put_dy(0);
    load_dy(1);
    put_dy(1);
    load_dy(2);
    load_stage(0, kStageLoads);
    next_stage();
    load_stage(1, kStageLoads);
    next_stage();
    load_stage(2, kHalfLoads);
    wait_loads<kStageLoads + kHalfLoads>();   // stage 0 has landed
    lds_barrier();
  }
  int slot = 0, last = kWgSlots - 1;   // of this stage, of the one before
  Dy d0, d1;
  if constexpr (NB == 8) {
    // One wave to a SIMD: nothing but this order hides a wait.  During a step
    // the next step's codes and dy operands are read from LDS.  The codes are
    // converted in place, a pair of x blocks at a time once this step's MFMAs
    // are through with it; the last pair follows at the beginning of the next
    // step, and only then are the next codes read.  An MFMA takes 16 cycles,
    // in which two or three other instructions issue: the rest is spread out
    // accordingly, the loads (which queue up when they come together, and hold
    // up the MFMAs behind them) one to eight MFMAs.
    X x;
    Codes c;
    auto step = [&](int next, const Dy& now, Dy& then, auto first_c, int to) __attribute__((always_inline)) {
      constexpr bool first = decltype(first_c)::value;
      each(std::make_integer_sequence<int, kM>(), [&](auto m_c) __attribute__((always_inline)) {
        constexpr int m = decltype(m_c)::value;
        constexpr int i = m % 8 == 1 && m / 8 < kHalfLoads ? kFirstLoad + m / 8 + (first ? kHalfLoads : 0) : kLoads;
        if constexpr (i < kLoads)
          target(i, to);
        mfma(m, now, x);
        if constexpr (i < kLoads)
          load(i);
        if constexpr (m < 12)
          convert(3, m / 3, m % 3, c, x);
        if constexpr (m >= 12 && m < 14)
          read_scales(next, m - 12, c);
        if constexpr (m >= 14 && m < 22)
          read_codes(next, m - 14, c);
        if constexpr (m >= 22 && m < 28) {
          read_dy(next, 2 * (m - 22), then);
          read_dy(next, 2 * (m - 22) + 1, then);
        }
        if constexpr (m >= 28 && m < 32)
          read_dy(next, m - 16, then);
        if constexpr (m >= 28)
          convert((m - 28) / 12, (m - 28) % 12 / 3, m % 3 == 1 ? 0 : m % 3 == 2 ? 1 : 2, c, x);
        if constexpr (m == 58 && first)
          arrive(to);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    if (stages > 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        read_scales(0, r, c);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        read_codes(0, r, c);
#pragma unroll
      for (int r = 0; r < 2 * NB; ++r)
        read_dy(0, r, d0);
#pragma unroll
      for (int r = 0; r < 36; ++r)
        convert(r / 12, r % 12 / 3, r % 3, c, x);
    }
    for (int st = 0; st < stages; ++st) {
      const int next = slot + 1 == kWgSlots ? 0 : slot + 1, by = (next - slot) * kSlot;
      step(1, d0, d1, std::true_type(), last);
      load_dy(st + 3);
      x_at += by;
      s_at += by;
#pragma unroll
      for (int i = 0; i < NB; ++i)
        d_at[i] += by;
      step(0, d1, d0, std::false_type(), slot);
      last = slot;
      slot = next;
    }
  } else {
    // Two waves to a SIMD.  During a step the next step's dy operands are read
    // from LDS, its codes (read during the step before) are converted, and the
    // codes of the step after it are read.
    X x0, x1;
    Codes c0, c1;
    auto step = [&](int number, const Dy& d, const X& x, Dy& d_next, X& x_next, const Codes& c_next, Codes& c_then,
                    auto first_c, int to, int by) __attribute__((always_inline)) {
      constexpr bool first = decltype(first_c)::value;
      each(std::make_integer_sequence<int, kM>(), [&](auto m_c) __attribute__((always_inline)) {
        constexpr int m = decltype(m_c)::value;
        constexpr int n = (first ? kHalfLoads : 0) + m / 3;
        constexpr int i = m % 3 == 1 && n < (first ? kStageLoads : kHalfLoads) && m < 11 ? kFirstLoad + n : kLoads;
        if constexpr (i < kLoads)
          target(i, to);
        mfma(m, d, x);
        if constexpr (i < kLoads)
          load(i);
        if constexpr (m < 8)
          read_dy(number ^ 1, m, d_next);
        // 24 parts over 16 MFMAs
        each(std::make_integer_sequence<int, m % 2 + 1>(), [&](auto e_c) {
          constexpr int r = m / 2 * 3 + m % 2 + decltype(e_c)::value;
          convert(r / 12, r % 12 / 3, r % 3, c_next, x_next);
        });
        if constexpr (m == 11 && first) {
          arrive(to);
          x_at += by;
          s_at += by;
        }
        if constexpr (m >= 12) {
          if constexpr (m < 14)
            read_scales(number, m - 12, c_then);
          read_codes(number, 2 * (m - 12), c_then);
          read_codes(number, 2 * (m - 12) + 1, c_then);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    if (stages > 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        read_scales(0, r, c0);
        read_scales(1, r, c1);
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        read_codes(0, r, c0);
        read_codes(1, r, c1);
        read_dy(0, r, d0);
      }
#pragma unroll
      for (int r = 0; r < 24; ++r)
        convert(r / 12, r % 12 / 3, r % 3, c0, x0);
    }
    for (int st = 0; st < stages; ++st) {
      const int next = slot + 1 == kWgSlots ? 0 : slot + 1, by = (next - slot) * kSlot;
      step(0, d0, x0, d1, x1, c1, c0, std::true_type(), last, by);
      load_dy(st + 3);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        d_at[i] += by;
      step(1, d1, x1, d0, x0, c0, c1, std::false_type(), slot, by);
      last = slot;
      slot = next;
    }
  }
  // loads into LDS still in flight must land before the workgroup ends
  wait_loads<0>();
  // an MFMA's result may be read 18 cycles after it at the earliest
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      asm volatile("" : "+a"(acc[i][j]));

  // Register v of lane l: row 4 (l / 16) + v of its block; the lane's NB
  // blocks along k are NB neighbouring columns.
  const int64_t col = j0 + kTile / 2 * wj + NB * l16;
  if (part < 0 && col >= a.k)
    return;
  constexpr int kBytes = BF16 ? 2 : 4;
  const bool whole = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = kTile / 2 * wi + 16 * i + 4 * lg + v;
      float f[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j)
        f[j] = acc[i][j][v];
      if (part >= 0) {
        store(a.part + ((int64_t)part * kTile + row) * kTile + kTile / 2 * wj + NB * l16, f);
        continue;
      }
      if (i0 + row >= a.n)
        continue;
      void* at = static_cast<uint8_t*>(a.out) + (((int64_t)g * a.n + i0 + row) * a.k + col) * kBytes;
      if (whole) {
        if constexpr (BF16)
          store(static_cast<uint16_t*>(at), f);
        else
          store(static_cast<float*>(at), f);
      } else {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          if constexpr (BF16)
            static_cast<uint16_t*>(at)[j] = (uint16_t)bf16_pair(f[j], 0.0f);
          else
            static_cast<float*>(at)[j] = f[j];
        }
      }
    }
}

// The cut tiles: dw = the sum of a tile's pieces, in their order.  A
// workgroup adds up `rows` rows of a tile, a thread four columns.
template <int NB, bool BF16>
__global__ __launch_bounds__(256) void wgrad_fold_kernel(WgradArgs a, int32_t rows) {
  constexpr int kTile = 32 * NB, kAcross = kTile / 4, kDown = 256 / kAcross;
  const uint32_t tiles = a.tiles_n * a.tiles_k;
  int32_t g = 0, pieces = (int32_t)a.pieces;
  int64_t tile = blockIdx.y, part = blockIdx.y, stride = tiles - a.whole;   // first piece's part, parts from piece to piece
  if (a.groups == 1) {
    tile += a.whole;
  } else {
    int32_t lo, hi, piece, first_part;
    if (!find_slot(a, (int32_t)blockIdx.z, false, g, lo, hi, pieces, piece, first_part))
      return;
    part += (int64_t)first_part * tiles;
    stride = tiles;
  }
  const int64_t i0 = tile / a.tiles_k * kTile, j0 = tile % a.tiles_k * kTile;
  const int col = threadIdx.x % kAcross * 4;
  if (j0 + col >= a.k)
    return;
  const bool whole = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
  for (int row = blockIdx.x * rows + threadIdx.x / kAcross; row < (int)(blockIdx.x + 1) * rows && i0 + row < a.n;
       row += kDown) {
    const float* p = a.part + (part * kTile + row) * kTile + col;
    f32x4 sum = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 8
    for (int s = 1; s < pieces; ++s)
      sum += *reinterpret_cast<const f32x4*>(p + s * stride * kTile * kTile);
    const int64_t at = ((int64_t)g * a.n + i0 + row) * a.k + j0 + col;
    if constexpr (BF16) {
      const u32x2 w = {bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
      uint16_t* o = static_cast<uint16_t*>(a.out) + at;
      if (whole)
        *reinterpret_cast<u32x2*>(o) = w;
      else
        o[0] = (uint16_t)w[0], o[1] = (uint16_t)(w[0] >> 16), o[2] = (uint16_t)w[1], o[3] = (uint16_t)(w[1] >> 16);
    } else {
      float* o = static_cast<float*>(a.out) + at;
      if (whole)
        *reinterpret_cast<f32x4*>(o) = sum;
      else
        o[0] = sum[0], o[1] = sum[1], o[2] = sum[2], o[3] = sum[3];
    }
  }
}

// How a call is cut up, from its sizes alone.
struct WgradPlan {
  int nb;
  uint32_t tiles_n, tiles_k, whole, pieces;
  int32_t piece_stages;
  int64_t blocks, parts;   // workgroups; tiles of pieces' sums
  uint32_t cut;            // one group: tiles that are cut; several: groups that may be
  double work;             // us of the cost that a workgroup after another spends on stages
  int64_t copy_cols;       // dy is copied to rows of so many columns if it is not aligned; 0: it is not
};

// What a plan is weighed with, in us, measured on MI355X: a workgroup's start
// and end, one stage of it, and one piece's sums written and added up.
template <int NB>
struct WgradCost;
template <>
struct WgradCost<8> {
  static constexpr double kStart = 12.0, kStage = 1.4, kPart = 0.13;
};
template <>
struct WgradCost<4> {
  static constexpr double kStart = 5.0, kStage = 1.05, kPart = 0.033;
};
constexpr double kWgFold = 6.0;   // the kernel that adds pieces up, at least

// Tiles run in rounds of as many as the GPU holds.  One group: full rounds
// keep their tiles whole; what is left over is cut along the tokens into as
// many pieces as fill a round, but no more than balances the time saved with
// the traffic of the pieces' sums (the sum of stages / pieces and pieces *
// tiles, each at its cost, is least at a square root).
// Several groups: a group is cut where it is more than half as long again as
// its share of the GPU (and of 24 stages), if groups average 32 stages;
// shorter ones cost more in pieces than they save.
template <int NB>
static WgradPlan wgrad_plan_of(int64_t rows, int64_t n, int64_t k, int32_t groups, double& cost) {
  using Cost = WgradCost<NB>;
  constexpr int64_t kRound = kWgCus * WgTile<NB>::kPerCu, kSide = WgTile<NB>::kTile;
  WgradPlan p = {};
  p.nb = NB;
  p.tiles_n = (uint32_t)((n + kSide - 1) / kSide), p.tiles_k = (uint32_t)((k + kSide - 1) / kSide);
  const int64_t tiles = (int64_t)p.tiles_n * p.tiles_k;
  const int64_t stages = (rows + kWgTokens - 1) / kWgTokens;
  if (groups == 1) {
    const int64_t cut = tiles % kRound;
    int64_t pieces = 1;
    if (cut > 0) {
      const double most = Cost::kStage * (double)stages / (Cost::kPart * (double)cut);
      while ((double)((pieces + 1) * (pieces + 1)) <= most && (pieces + 1) * cut <= kRound && 2 * (pieces + 1) <= stages)
        ++pieces;
      if (Cost::kStage * (double)(stages - stages / pieces) < kWgFold + Cost::kPart * (double)(pieces * cut))
        pieces = 1;
    }
    p.cut = pieces > 1 ? (uint32_t)cut : 0;
    p.whole = (uint32_t)(tiles - p.cut), p.pieces = (uint32_t)pieces;
    p.parts = p.cut * pieces;
    p.blocks = segment_blocks(p.whole) + (int64_t)segment_blocks(p.cut) * pieces;
    cost = (double)(tiles / kRound) * (Cost::kStart + Cost::kStage * (double)stages);
    if (cut > 0)
      cost += Cost::kStart + Cost::kStage * (double)((stages + pieces - 1) / pieces);
    p.work = Cost::kStage * (double)(tiles / kRound * stages + (cut > 0 ? (stages + pieces - 1) / pieces : 0));
    if (pieces > 1)
      cost += kWgFold + Cost::kPart * (double)p.parts;
    return p;
  }
  const int64_t total = rows / kWgTokens + groups;   // at most: every group may end in a partial stage
  const int64_t share = (total * tiles + kRound - 1) / kRound, each = share < 24 ? 24 : share;
  const bool may_cut = rows / kWgTokens >= 32 * (int64_t)groups && tiles * groups < 8 * kRound;
  p.piece_stages = may_cut ? (int32_t)each : INT32_MAX / 2;
  p.pieces = (uint32_t)(may_cut ? total / each + groups : groups);
  const int64_t parts = may_cut ? total * 4 / (3 * each) : 0;   // a cut group is at least 1.5 pieces long
  p.cut = (uint32_t)(parts / 2);
  p.parts = p.cut > 0 ? parts * tiles : 0;
  p.blocks = (int64_t)segment_blocks((uint32_t)tiles) * p.pieces;
  // groups of uneven length: the longest of few tiles to a CU sets the time
  const double rounds = (double)(tiles * groups) / (double)kRound;
  const double even = (double)total / (double)groups;
  p.work = Cost::kStage * even * ((rounds < 1.0 ? 1.0 : rounds) + (rounds < 2.0 ? 1.0 : 0.0));
  cost = (rounds < 1.0 ? 1.0 : rounds) * (Cost::kStart + Cost::kStage * even) + (rounds < 2.0 ? Cost::kStage * even : 0.0);
  return p;
}

// 256 x 256 tiles move half as much per product as 128 x 128 tiles and keep
// the matrix cores busier (16640 x 4096 x 4096: 380 against 546 us); the
// smaller ones start and end sooner, two to a CU, and there are four times as
// many (1024 x 2048 x 2048: 16 against 29 us).
//
// Where n is not a multiple of 8, rows of dy are not aligned as a rule, and
// loads through registers (VEC false) make stages take about 1.55 times as
// long.  A copy in aligned rows costs a launch (3 us) and its bytes, and is
// made where that is less.  Without and with it: 16640 x 8191 x 5120 1538 and
// 1152 us, 16640 x 4095 x 4096 583 and 446, 1024 x 1023 x 1024 24 and 18; 8192 x
// 257 x 256, where it is not made, 17 and 20.  The workspace is sized by the
// lengths alone: rows of dy that are unaligned by their pitch or start only, n
// being a multiple of 8, find no room for a copy and go through registers at
// any size (16640 x 8192 x 5120 at a pitch of 8195: 1560 us).
static WgradPlan wgrad_plan(int64_t rows, int64_t n, int64_t k, int32_t groups) {
  double cost8, cost4;
  const WgradPlan p8 = wgrad_plan_of<8>(rows, n, k, groups, cost8);
  const WgradPlan p4 = wgrad_plan_of<4>(rows, n, k, groups, cost4);
  WgradPlan p = cost8 <= cost4 ? p8 : p4;
  const int64_t cols = (n + 7) / 8 * 8;
  if (n % 8 != 0 && 0.55 * p.work > 3.0 + (double)rows * (double)cols * 4.0 / 4.5e6)
    p.copy_cols = cols;
  return p;
}

static int64_t wgrad_part_bytes(const WgradPlan& p) { return p.parts * (32 * p.nb) * (32 * p.nb) * 4; }

int64_t wgrad_workspace_bytes(int64_t rows, int64_t n, int64_t k, int32_t groups) {
  const WgradPlan p = wgrad_plan(rows, n, k, groups);
  return wgrad_part_bytes(p) + rows * p.copy_cols * 2;
}

// dy in aligned rows of `cols` columns, zeros past column n: a wave to a row.
__global__ __launch_bounds__(256) void wgrad_copy_kernel(const uint16_t* dy, int64_t lddy, int64_t rows, int64_t n,
                                                         int64_t cols, uint16_t* out) {
  const int lane = threadIdx.x & 63;
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.x * 4) {
    const uint16_t* from = dy + row * lddy;
    for (int64_t c = 8 * lane; c < cols; c += 512) {
      u32x4 v = {0, 0, 0, 0};
      if (c + 8 <= n) {
        v = *reinterpret_cast<const u32x4_any*>(from + c);
      } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
          v[e / 2] |= c + e < n ? (uint32_t)from[c + e] << (16 * (e & 1)) : 0u;
      }
      *reinterpret_cast<u32x4*>(out + row * cols + c) = v;
    }
  }
}

int64_t wgrad_grid_blocks(int64_t rows, int64_t n, int64_t k, int32_t groups) {
  return wgrad_plan(rows, n, k, groups).blocks;
}

template <int NB, bool VEC, bool BF16>
static hipError_t launch_wgrad_tile(const WgradArgs& a, const WgradPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL((wgrad_kernel<NB, VEC, BF16>), dim3((unsigned)p.blocks), dim3(kWgThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.cut == 0)
    return e;
  // several groups: most of these find that their group is not cut, so fewer
  const int32_t rows = a.groups == 1 ? 32 / NB : 8 * NB;
  const dim3 fold(32 * NB / rows, a.groups == 1 ? p.cut : p.tiles_n * p.tiles_k, a.groups == 1 ? 1 : p.cut);
  hipLaunchKernelGGL((wgrad_fold_kernel<NB, BF16>), fold, dim3(256), 0, stream, a, rows);
  return hipGetLastError();
}

template <int NB>
static hipError_t launch_wgrad_any(const WgradArgs& a, const WgradPlan& p, bool vec, bool bf16, hipStream_t stream) {
  if (vec)
    return bf16 ? launch_wgrad_tile<NB, true, true>(a, p, stream) : launch_wgrad_tile<NB, true, false>(a, p, stream);
  return bf16 ? launch_wgrad_tile<NB, false, true>(a, p, stream) : launch_wgrad_tile<NB, false, false>(a, p, stream);
}

hipError_t launch_wgrad(const void* dy, int64_t lddy, const uint8_t* q, const uint8_t* s, int64_t rows, int64_t n,
                        int64_t k, const int32_t* ends, int32_t groups, void* dw, bool bf16, float* workspace,
                        bool vec, hipStream_t stream) {
  const WgradPlan p = wgrad_plan(rows, n, k, groups);
  WgradArgs a = {};
  a.dy = static_cast<const uint16_t*>(dy), a.lddy = lddy, a.n_read = n, a.q = q, a.s = s, a.ends = ends, a.n = n, a.k = k;
  a.out = dw, a.part = workspace, a.rows = (int32_t)rows, a.groups = groups;
  a.tiles_n = p.tiles_n, a.tiles_k = p.tiles_k, a.whole = p.whole, a.pieces = p.pieces, a.piece_stages = p.piece_stages;
  if (!vec && p.copy_cols > 0 && rows > 0) {
    uint16_t* copy = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(workspace) + wgrad_part_bytes(p));
    const int64_t blocks = std::min<int64_t>((rows + 3) / 4, 4096);
    hipLaunchKernelGGL(wgrad_copy_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a.dy, lddy, rows, n, p.copy_cols,
                       copy);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
      return e;
    a.dy = copy, a.lddy = a.n_read = p.copy_cols;
    vec = true;
  }
  return p.nb == 8 ? launch_wgrad_any<8>(a, p, vec, bf16, stream) : launch_wgrad_any<4>(a, p, vec, bf16, stream);
}

}  // namespace mx
