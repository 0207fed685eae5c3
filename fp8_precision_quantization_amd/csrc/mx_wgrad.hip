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
static_assert(kWgSlot % 256 == 0 && kWgSlots * kWgSlot <= 160 * 1024, "stages fit LDS");

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
  constexpr int kFirstLoad = VEC ? 0 : 8, kStageLoads = 14 - kFirstLoad;
  auto load_stage = [&](int slot) {
#pragma unroll
    for (int i = kFirstLoad; i < 14; ++i) {
      target(i, slot);
      asm volatile("s_nop 0");
      load(i);
    }
    next_stage();
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
  // come together, and hold up the MFMAs behind them) one to four MFMAs.
  auto step = [&](int next, const Dy& now, Dy& then, auto first_c, int slot) __attribute__((always_inline)) {
    constexpr bool first = decltype(first_c)::value;
    each(std::make_integer_sequence<int, kWgBlocks * kWgBlocks>(), [&](auto m_c) __attribute__((always_inline)) {
      constexpr int m = decltype(m_c)::value;
      constexpr int i = m % 4 == 1 ? m / 4 + kFirstLoad : 14;
      if constexpr (i < 14)
        if (!first)
          target(i, slot);
      mfma(m, now);
      if constexpr (i < 14)
        if (!first)
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
          put_dy(slot == 0 ? kWgSlots - 1 : slot - 1);   // stage st + 2, where dy comes through registers
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
    load_stage(0);
    load_stage(1);
    load_stage(2);
    wait_loads<2 * kStageLoads>();   // stage 0 has landed
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
      step(1, d0, d1, std::true_type(), slot);
      load_dy(st + 3);
      const int to = slot + 1 == kWgSlots ? 0 : slot + 1;
      const int by = (to - slot) * kWgSlot;
      x_from += by;
      s_from += by;
#pragma unroll
      for (int i = 0; i < kWgBlocks; ++i)
        d_at[i] += by;
      step(0, d1, d0, std::false_type(), slot);
      next_stage();
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
  if (col >= a.k)
    return;
  const int64_t plane = ((int64_t)split * a.groups + g) * a.n;
  constexpr int kBytes = BF16 ? 2 : 4;
  const bool whole = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
#pragma unroll
  for (int i = 0; i < kWgBlocks; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t row = i0 + 128 * wi + 16 * i + 4 * lg + v;
      if (row >= a.n)
        continue;
      float f[8];
#pragma unroll
      for (int j = 0; j < kWgBlocks; ++j)
        f[j] = acc[i][j][v];
      void* at = static_cast<uint8_t*>(a.out) + ((plane + row) * a.k + col) * kBytes;
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
