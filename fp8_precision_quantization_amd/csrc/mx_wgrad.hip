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
// Work decomposition.  A 256-thread workgroup owns a 256 x 256 tile of one
// group's dw; wave w its (w / 2, w % 2) 128 x 128 quarter, 8 x 8 blocks of
// v_mfma_f32_16x16x32_bf16, whose 256 accumulators live in the accumulation
// registers.  Tokens advance in stages of 64.  A stage's 64 x 256 pieces of dy
// (bf16), of the codes and of the scales lie in LDS token-major as in memory,
// three stages deep, brought there by loads that go straight from memory to
// LDS.  Keeping the codes in LDS as codes halves what the waves read of x
// (LDS bandwidth, not the matrix cores, bound the kernel while LDS held bf16
// x: 1293 us for 16640 x 8192 x 5120); each wave converts what it reads.
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

#include <type_traits>
#include <utility>

namespace mx {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

constexpr int kWgThreads = 256;
constexpr int kWgTile = 256;
constexpr int kWgTokens = 64;                        // tokens per stage
constexpr int kWgBlocks = 8;                         // 16 x 16 blocks per wave each way
constexpr int kWgRow = kWgTile * 2;                  // bytes of a stage row of dy
constexpr int kWgX = kWgTokens * kWgRow;             // where the codes start in a stage: rows of kWgTile bytes
constexpr int kWgS = kWgX + kWgTokens * kWgTile;     // where the scales start: a dword each, [block of 32][token]
constexpr int kWgScaleRow = 4 * kWgTokens + 16;      // (16 more than the banks' period)
constexpr int kWgSlot = kWgS + kWgTile / MX_BLOCK * kWgScaleRow + 128;
constexpr int kWgSlots = 3;
constexpr int kWgCus = 256;
static_assert(kWgSlot % 256 == 0 && kWgSlots * kWgSlot <= 160 * 1024, "stages fit LDS");

struct WgradArgs {
  const uint16_t* dy;
  const uint8_t *q, *s;
  const int32_t* ends;
  void* out;
  float* part;        // sums of pieces, a 256 x 256 tile each
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

template <bool VEC, bool BF16>
__global__ __launch_bounds__(kWgThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void wgrad_kernel(WgradArgs a) {
  __shared__ __attribute__((aligned(256))) uint8_t lds[kWgSlots * kWgSlot];
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
  const int64_t i0 = (int64_t)((uint32_t)tile / a.tiles_k) * kWgTile, j0 = (int64_t)((uint32_t)tile % a.tiles_k) * kWgTile;

  const int t = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lane = t & 63;
  const int wi = wave >> 1, wj = wave & 1;
  const int64_t ks = a.k / MX_BLOCK;

  f32x4 acc[kWgBlocks][kWgBlocks];
#pragma unroll
  for (int i = 0; i < kWgBlocks; ++i)
#pragma unroll
    for (int j = 0; j < kWgBlocks; ++j)
      acc[i][j] = (f32x4){};

  // Loader roles, 14 loads of a wave to a stage.
  //  dy: load u of wave w fills rows 8 u + 2 w, + 1; lane l the 16 bytes at
  //  position l % 32 of row 8 u + 2 w + l / 32, whose source is chunk (l % 32)
  //  ^ 2 f, f = row % 4 + 4 (row / 8 % 2).
  //  codes: load u fills rows 16 u + 4 w .. + 3; lane l position l % 16 of row
  //  16 u + 4 w + l / 16, source chunk (l % 16) ^ 8 (row / 8 % 2).
  //  scales: loads of blocks 2 w, 2 w + 1; lane l is token l.
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);
  const int drow = 2 * wave + lane / 32;
  const int dchunk = (lane % 32) ^ (2 * (drow & 3));   // of even u; odd u: ^ 8
  const int doff = drow * (int)a.lddy * 2 + 16 * dchunk, doff1 = drow * (int)a.lddy * 2 + 16 * (dchunk ^ 8);
  const int xoff = (4 * wave + lane / 16) * (int)a.k + 16 * ((lane % 16) ^ (8 * (wave >> 1)));
  const int soff = lane * (int)ks + 2 * wave;
  const int64_t dy_end = (int64_t)(a.rows - 1) * a.lddy + a.n;   // elements of dy
  u32x4 dreg[VEC ? 1 : 8];

  // The next stage to load, and load i of it (0 .. 13: eight of dy, four of
  // codes, two of scales; without the first eight where dy goes through
  // registers) into slot `slot`.  Past the last stage they load zeros.
  const int64_t tokens = hi - lo;
  Run run_dy = {reinterpret_cast<const uint8_t*>(a.dy + lo * a.lddy + i0), ((tokens - 1) * a.lddy + a.n - i0) * 2,
                kWgTokens * a.lddy * 2};
  Run run_q = {a.q + lo * a.k + j0, tokens * a.k - j0, kWgTokens * a.k};
  Run run_s = {a.s + lo * ks + j0 / MX_BLOCK, tokens * ks - j0 / MX_BLOCK, kWgTokens * ks};
  auto target = [&](int i, int slot) {
    const uint32_t to = lds0 + slot * kWgSlot;
    lds_target(to + (i < 8    ? (8 * i + 2 * wave) * kWgRow
                     : i < 12 ? kWgX + (16 * (i - 8) + 4 * wave) * kWgTile
                              : kWgS + (2 * wave + i - 12) * kWgScaleRow));
  };
  auto load = [&](int i) {
    if (i < 8)
      load_to_lds<16>(run_dy.rsrc(), (i % 2 ? doff1 : doff) + 8 * i * (int)a.lddy * 2);
    else if (i < 12)
      load_to_lds<16>(run_q.rsrc(), xoff + 16 * (i - 8) * (int)a.k);
    else
      load_to_lds<1>(run_s.rsrc(), soff + i - 12);
  };
  auto next_stage = [&]() {
    run_dy.next();
    run_q.next();
    run_s.next();
  };
  constexpr int kFirstLoad = VEC ? 0 : 8, kStageLoads = 14 - kFirstLoad, kHalfLoads = kStageLoads / 2;
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
      for (int u = 0; u < 8; ++u) {
        const int row = 8 * u + drow;
        const int64_t c = i0 + 8 * (u % 2 ? dchunk ^ 8 : dchunk);
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
      for (int u = 0; u < 8; ++u)
        *reinterpret_cast<u32x4*>(lds + slot * kWgSlot + (8 * u + drow) * kWgRow + 16 * (lane % 32)) = dreg[u];
    }
  };

  // MFMA role: lane l holds column (of dy or x) l % 16 of a block, tokens 8
  // (l / 16) .. + 7 of a step's 32.
  const int l16 = lane & 15, lg = lane >> 4;
  const int tok = 8 * lg + (l16 >> 2);                        // dy reads: this token, and + 4
  const int swz = (tok & 3) | ((lg & 1) << 2);
  const int a_at = tok * kWgRow + 256 * wi + 32 * swz + 8 * (lane & 3);   // block b at ^ 32 b
  const int x_at = kWgX + 8 * lg * kWgTile + 128 * (wj ^ (lg & 1)) + 8 * l16;
  const int s_at = kWgS + (4 * wj + l16 / 4) * kWgScaleRow + 32 * lg;
  typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
  typedef s16x4 Dy[kWgBlocks][2];   // a step's dy operands: 8 tokens of a column, in two reads
  Dy d0, d1;
  uint32_t x[kWgBlocks][4];         // a step's x operands
  u32x2 codes[8];                   // 8 columns of each of 8 tokens
  u32x4 scales[2];                  // those tokens' scale bytes

  // where the lane reads in the slot of the step that is read next
  int d_at[kWgBlocks], x_from = x_at, s_from = s_at;
#pragma unroll
  for (int i = 0; i < kWgBlocks; ++i)
    d_at[i] = a_at ^ (32 * i);
  auto read_dy = [&](int step, int r, Dy& d) {           // r: 0 .. 15
    const uint8_t* p = lds + d_at[r / 2] + (32 * step + 4 * (r % 2)) * kWgRow;
    d[r / 2][r % 2] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
  };
  auto read_x = [&](int step, int r) {                   // r: 0 .. 9, scales first
    if (r < 2)
      scales[r] = *reinterpret_cast<const u32x4*>(lds + s_from + 128 * step + 16 * r);
    else
      codes[r - 2] = *reinterpret_cast<const u32x2*>(lds + x_from + (32 * step + r - 2) * kWgTile);
  };
  // Columns 2 c, 2 c + 1 of tokens 2 u, 2 u + 1: a dword of x blocks 2 c, 2 c
  // + 1, in three parts of two instructions.
  uint32_t pair[2];
  auto convert = [&](int c, int u, int part) {
    if (part < 2) {
      const int t = 2 * u + part;
      const float sc = __uint_as_float(scales[t / 4][t % 4] << 23);
      pair[part] =
          __builtin_bit_cast(uint32_t, c % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[t][c / 2], sc, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[t][c / 2], sc, false));
    } else {
      x[2 * c][u] = __builtin_amdgcn_perm(pair[1], pair[0], 0x05040100u);
      x[2 * c + 1][u] = __builtin_amdgcn_perm(pair[1], pair[0], 0x07060302u);
    }
  };
  auto convert_part = [&](int c, int i) { convert(c, i / 3, i % 3); };   // i: 0 .. 11
  auto mfma = [&](int m, const Dy& d) {
    const int i = m % kWgBlocks, j = m / kWgBlocks;
    const bf16x8 fa =
        __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(d[i][0], d[i][1], 0, 1, 2, 3, 4, 5, 6, 7));
    const bf16x8 fb = __builtin_bit_cast(bf16x8, (u32x4){x[j][0], x[j][1], x[j][2], x[j][3]});
    // v_mfma_f32_16x16x32_bf16 with the accumulators tied to accumulation
    // registers: given the intrinsic, the compiler moves the 64 of them about
    // (428 register moves a stage).  Every operand was written at least four
    // MFMAs earlier; the results are read after drain() below.
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[i][j]) : "v"(fa), "v"(fb));
  };

  // A stage is two steps of 32 tokens, 64 MFMAs each, x block after x block;
  // there is one wave to a SIMD, so nothing but this order hides a wait.
  // During a step the next step's codes and dy operands are read from LDS.
  // The codes are converted in place, a pair of x blocks at a time once this
  // step's MFMAs are through with it; the last pair follows at the beginning
  // of the next step, and only then are the next codes read.
  // Late in the first step of stage st the wave waits for its loads of stage
  // st + 1 and meets the others at the stage's one barrier.  All of stage st
  // has been read by then, and its slot takes the loads of stage st + 3.
  // An MFMA takes 16 cycles, in which two or three other instructions issue:
  // the rest is spread out accordingly, the loads (which queue up when they
  // come together, and hold up the MFMAs behind them) one to eight MFMAs.
  auto step = [&](int next, const Dy& now, Dy& then, auto first_c, int to) __attribute__((always_inline)) {
    constexpr bool first = decltype(first_c)::value;
    each(std::make_integer_sequence<int, kWgBlocks * kWgBlocks>(), [&](auto m_c) __attribute__((always_inline)) {
      constexpr int m = decltype(m_c)::value;
      constexpr int i = m % 8 == 1 && m / 8 < kHalfLoads ? kFirstLoad + m / 8 + (first ? kHalfLoads : 0) : 14;
      if constexpr (i < 14)
        target(i, to);
      mfma(m, now);
      if constexpr (i < 14)
        load(i);
      if constexpr (m < 12)
        convert_part(3, m);
      if constexpr (m >= 12 && m < 22)
        read_x(next, m - 12);
      if constexpr (m >= 22 && m < 28) {
        read_dy(next, 2 * (m - 22), then);
        read_dy(next, 2 * (m - 22) + 1, then);
      }
      if constexpr (m >= 28 && m < 32)
        read_dy(next, m - 16, then);
      if constexpr (m >= 28)
        convert_part((m - 28) / 12, (m - 28) % 12);
      if constexpr (m == 58) {
        if (first) {
          next_stage();
          put_dy(to);   // where dy comes through registers
          wait_loads<kStageLoads>();
          lds_barrier();
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  if (hi > lo) {
    const int stages = (hi - lo + kWgTokens - 1) / kWgTokens;
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
#pragma unroll
    for (int r = 0; r < 10; ++r)
      read_x(0, r);
#pragma unroll
    for (int r = 0; r < 16; ++r)
      read_dy(0, r, d0);
#pragma unroll
    for (int r = 0; r < 36; ++r)
      convert_part(r / 12, r % 12);
    int slot = 0;
    for (int st = 0; st < stages; ++st) {
      step(1, d0, d1, std::true_type(), slot == 0 ? kWgSlots - 1 : slot - 1);
      load_dy(st + 3);
      const int to = slot + 1 == kWgSlots ? 0 : slot + 1;
      const int by = (to - slot) * kWgSlot;
      x_from += by;
      s_from += by;
#pragma unroll
      for (int i = 0; i < kWgBlocks; ++i)
        d_at[i] += by;
      step(0, d1, d0, std::false_type(), slot);
      slot = to;
    }
    // loads into LDS still in flight must land before the workgroup ends
    wait_loads<0>();
  }
  // an MFMA's result may be read 18 cycles after it at the earliest
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int i = 0; i < kWgBlocks; ++i)
#pragma unroll
    for (int j = 0; j < kWgBlocks; ++j)
      asm volatile("" : "+a"(acc[i][j]));

  // Register v of lane l: row 4 (l / 16) + v of its block; the lane's 8 blocks
  // along k are 8 neighbouring columns.
  const int64_t col = j0 + 128 * wj + 8 * l16;
  if (part < 0 && col >= a.k)
    return;
  constexpr int kBytes = BF16 ? 2 : 4;
  const bool whole = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
#pragma unroll
  for (int i = 0; i < kWgBlocks; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 128 * wi + 16 * i + 4 * lg + v;
      float f[8];
#pragma unroll
      for (int j = 0; j < kWgBlocks; ++j)
        f[j] = acc[i][j][v];
      if (part >= 0) {
        store(a.part + ((int64_t)part * kWgTile + row) * kWgTile + 128 * wj + 8 * l16, f);
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
        for (int j = 0; j < kWgBlocks; ++j) {
          if constexpr (BF16)
            static_cast<uint16_t*>(at)[j] = (uint16_t)bf16_pair(f[j], 0.0f);
          else
            static_cast<float*>(at)[j] = f[j];
        }
      }
    }
}

// The cut tiles: dw = the sum of a tile's pieces, in their order.  A
// workgroup adds up `rows` rows of a tile, four at a time, a thread four
// columns.
template <bool BF16>
__global__ __launch_bounds__(256) void wgrad_fold_kernel(WgradArgs a, int32_t rows) {
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
  const int64_t i0 = tile / a.tiles_k * kWgTile, j0 = tile % a.tiles_k * kWgTile;
  const int col = (threadIdx.x & 63) * 4;
  if (j0 + col >= a.k)
    return;
  const bool whole = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
  for (int row = blockIdx.x * rows + (threadIdx.x >> 6); row < (int)(blockIdx.x + 1) * rows && i0 + row < a.n; row += 4) {
    const float* p = a.part + (part * kWgTile + row) * kWgTile + col;
    f32x4 sum = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 8
    for (int s = 1; s < pieces; ++s)
      sum += *reinterpret_cast<const f32x4*>(p + s * stride * kWgTile * kWgTile);
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
  uint32_t tiles_n, tiles_k, whole, pieces;
  int32_t piece_stages;
  int64_t blocks, parts;   // workgroups; tiles of pieces' sums
  uint32_t cut;            // one group: tiles that are cut; several: groups that may be
};

// One workgroup fills a CU, so tiles run in rounds of 256.  One group: full
// rounds keep their tiles whole; what is left over is cut along the tokens
// into as many pieces as fill a round, but no more than balances the time
// saved with the traffic of the pieces' sums (about 1.3 us a stage against
// 0.13 us a piece and tile: pieces = sqrt(10 stages / tiles)).
// Several groups: a group is cut where it is more than half as long again as
// its share of the GPU (and of 24 stages); from eight rounds of tiles on, none.
static WgradPlan wgrad_plan(int64_t rows, int64_t n, int64_t k, int32_t groups) {
  WgradPlan p = {};
  p.tiles_n = (uint32_t)((n + kWgTile - 1) / kWgTile), p.tiles_k = (uint32_t)((k + kWgTile - 1) / kWgTile);
  const int64_t tiles = (int64_t)p.tiles_n * p.tiles_k;
  const int64_t stages = (rows + kWgTokens - 1) / kWgTokens;
  if (groups == 1) {
    const int64_t cut = tiles % kWgCus;
    int64_t pieces = 1;
    if (cut > 0) {
      while ((pieces + 1) * (pieces + 1) * cut <= 10 * stages && (pieces + 1) * cut <= kWgCus && 2 * (pieces + 1) <= stages)
        ++pieces;
    }
    p.cut = pieces > 1 ? (uint32_t)cut : 0;
    p.whole = (uint32_t)(tiles - p.cut), p.pieces = (uint32_t)pieces;
    p.parts = p.cut * pieces;
    p.blocks = segment_blocks(p.whole) + (int64_t)segment_blocks(p.cut) * pieces;
    return p;
  }
  const int64_t total = rows / kWgTokens + groups;   // at most: every group may end in a partial stage
  int64_t each = INT32_MAX / 2;
  if (tiles * groups < 8 * kWgCus) {
    each = (total * tiles + kWgCus - 1) / kWgCus;
    each = each < 24 ? 24 : each;
  }
  p.piece_stages = (int32_t)each;
  p.pieces = (uint32_t)(total / each + groups);
  const int64_t parts = total * 4 / (3 * each);      // a cut group is at least 1.5 pieces long
  p.cut = (uint32_t)(parts / 2);
  p.parts = p.cut > 0 ? parts * tiles : 0;
  p.blocks = (int64_t)segment_blocks((uint32_t)tiles) * p.pieces;
  return p;
}

int64_t wgrad_workspace_bytes(int64_t rows, int64_t n, int64_t k, int32_t groups) {
  return wgrad_plan(rows, n, k, groups).parts * kWgTile * kWgTile * 4;
}

int64_t wgrad_grid_blocks(int64_t rows, int64_t n, int64_t k, int32_t groups) {
  return wgrad_plan(rows, n, k, groups).blocks;
}

hipError_t launch_wgrad(const void* dy, int64_t lddy, const uint8_t* q, const uint8_t* s, int64_t rows, int64_t n,
                        int64_t k, const int32_t* ends, int32_t groups, void* dw, bool bf16, float* workspace,
                        bool vec, hipStream_t stream) {
  const WgradPlan p = wgrad_plan(rows, n, k, groups);
  WgradArgs a = {};
  a.dy = static_cast<const uint16_t*>(dy), a.lddy = lddy, a.q = q, a.s = s, a.ends = ends, a.n = n, a.k = k;
  a.out = dw, a.part = workspace, a.rows = (int32_t)rows, a.groups = groups;
  a.tiles_n = p.tiles_n, a.tiles_k = p.tiles_k, a.whole = p.whole, a.pieces = p.pieces, a.piece_stages = p.piece_stages;
  const dim3 grid((unsigned)p.blocks), threads(kWgThreads);
  if (vec) {
    if (bf16)
      hipLaunchKernelGGL((wgrad_kernel<true, true>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((wgrad_kernel<true, false>), grid, threads, 0, stream, a);
  } else {
    if (bf16)
      hipLaunchKernelGGL((wgrad_kernel<false, true>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((wgrad_kernel<false, false>), grid, threads, 0, stream, a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.cut == 0)
    return e;
  // several groups: most of these find that their group is not cut, so fewer
  const int32_t fold_rows = groups == 1 ? 4 : 32;
  const dim3 fold(kWgTile / fold_rows, groups == 1 ? p.cut : p.tiles_n * p.tiles_k, groups == 1 ? 1 : p.cut);
  if (bf16)
    hipLaunchKernelGGL((wgrad_fold_kernel<true>), fold, dim3(256), 0, stream, a, fold_rows);
  else
    hipLaunchKernelGGL((wgrad_fold_kernel<false>), fold, dim3(256), 0, stream, a, fold_rows);
  return hipGetLastError();
}

}  // namespace mx
