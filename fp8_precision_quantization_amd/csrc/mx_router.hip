// MoE router: expert choice, gates, per-expert counts and the balance loss;
// and the gradient of the logits.
//
//   p = softmax(z); chosen = the topk largest logits; gates = p[chosen]
//   (divided by their sum); counts, group ends; balance[e] = E counts[e] /
//   (topk N^2); loss = sum_e balance[e] sum_rows p[e].
//   dz[e] = p[e] (dp[e] - sum_i p[i] dp[i]),
//   dp[e] = dloss balance[e] + sum_j [chosen_j = e] d_j.
//
// A row belongs to G lanes: 16 (four rows to a wave) up to 256 experts, the
// wave for more.  A lane holds V logits, in pieces of U consecutive columns
// (U a 16-byte load where alignment allows, else 1); piece p of a row sits in
// lane p % G.  The row is read once: maximum, exponentials, their sum and the
// topk selections all work on registers and on lane moves.
//
// Selection.  A logit and its column become one integer below 2^31 that orders
// like (logit descending, column ascending): the logit's ordered bits above
// the reversed column, NaN highest, 0 for a closed expert.  They are distinct,
// so the next choice is the largest one below the last, and unsigned key -
// last puts those below (it wraps) above those already chosen: a subtraction
// and half a three-way maximum per logit and choice, nothing to clear.  bf16
// fits whole.  Of a binary32 the bits that do not fit are left off, and where
// two choices in a row (or the last and the first not chosen) then look alike,
// the wave chooses again with whole logits, the maximum first and then the
// lowest column that has it.  65536 rows of 256 bf16 logits, topk 8: 52 us
// with the second way for all, 26 us with the first (and 8 more to add the
// workgroups' sums up).  Vector instructions bound it, where memory would allow
// 7 us: 710 for a wave's four rows (19 us of issue), 285 of them the keys,
// maxima and exponentials before the choices, 245 the seven choices after the
// first, the rest gates, p sums and stores; four waves to a SIMD leave some of
// the loads' latency uncovered.  Binary32 logits: 32 us (and 8).  The gradient
// of 65536 x 256 binary32 logits takes 28 us, 5.1 TB/s; of bf16 ones 22 us.
//
// Sums over rows (p for the loss) stay in a lane's registers over all its
// rows, meet in LDS, and leave as one row of partial sums per workgroup; the
// last step adds these up in a fixed order.  Counts are integers: LDS atomics
// in any order give the same result.
#include "mx_train.h"
#include "mx_train_launch.h"
#include "mxtrain.h"

namespace mx {

constexpr int kRouterThreads = 1024;
constexpr int kRouterWaves = kRouterThreads / 64;
constexpr int64_t kRouterBlocks = 256;   // one workgroup to a CU

struct RouterArgs {
  const void* z;
  int64_t ld, rows;
  const uint8_t* valid;
  int32_t experts, topk, normalize, align;
  int32_t *chosen, *counts, *ends;
  float *gates, *lse, *balance, *loss;
  // workspace: per workgroup a row of p sums, then a row of counts, then the
  // number of rows that took part
  float* part_p;
  int32_t* part_n;
  int32_t* part_rows;
  // backward
  const int32_t* in_chosen;
  const float *in_lse, *in_gates, *in_balance, *dgates, *dloss;
  void* dz;
};

// Elements of a row of partial sums: whole 16-byte words.
__host__ __device__ inline int32_t router_stride(int32_t experts) { return (experts + 3) / 4 * 4; }

template <int G, int U>
__device__ __forceinline__ int router_col(int v, int gl) {
  return ((v / U) * G + gl) * U + v % U;
}

// This lane's logits of a row as they lie in memory, the next rows' while
// these are worked on.
template <typename T, int G, int V, int U>
struct RowWords {
  Raw<T, U> w[V / U];
  __device__ __forceinline__ void load(const T* row, int experts, int gl) {
#pragma unroll
    for (int p = 0; p < V / U; ++p) {
      const int c = router_col<G, U>(p * U, gl);
      if (c < experts)
        w[p].load(row + c);
    }
  }
};

// This lane's logits of a row as binary32; columns past the end give `pad`.
template <typename T, int G, int V, int U>
__device__ __forceinline__ void load_logits(const T* row, int experts, int gl, float pad, float (&z)[V]) {
#pragma unroll
  for (int p = 0; p < V / U; ++p) {
    const int c = router_col<G, U>(p * U, gl);
    float f[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      f[i] = pad;
    if (c < experts)
      unpack(row + c, f);
#pragma unroll
    for (int i = 0; i < U; ++i)
      z[p * U + i] = f[i];
  }
}

// Integer that orders like the logit, NaN highest, a closed expert's -inf
// lowest.  Adding +0 turns -0 into +0, which it equals.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return z != z ? 0xFFFFFFFFu : k;
}
constexpr uint32_t kClosedKey = 0x007FFFFFu;   // of -inf
// Its upper bits, at most BITS, counted from a closed expert's, which is 0.  T
// says what the logit was in memory: bf16 loses nothing, of a binary32 the
// lower bits go (those of -inf and of the lowest finite number differ).
template <typename T, int BITS>
__device__ __forceinline__ uint32_t short_key(float z) {
  static_assert(BITS >= 16 && BITS < 32, "key bits");
  constexpr int kShift = sizeof(T) == 2 ? 16 : 32 - BITS;
  return (order_key(z) >> kShift) - (kClosedKey >> kShift);
}

// counts, ends, balance and loss from totals in LDS (tot_p, tot_n) and the
// number of rows; by wave 0.
__device__ __forceinline__ void router_finish(const RouterArgs& a, const float* tot_p, const int32_t* tot_n,
                                              int32_t n_rows) {
  // lane l has the experts l per .. (l + 1) per - 1
  const int lane = threadIdx.x & 63;
  const int per = (a.experts + 63) / 64;
  const int e0 = min(lane * per, a.experts), e1 = min(e0 + per, a.experts);
  const float n = (float)n_rows;
  int32_t mine = 0;
  float loss = 0.0f;
  for (int e = e0; e < e1; ++e) {
    const int32_t c = tot_n[e];
    const float bal = n_rows > 0 ? (float)a.experts * (float)c / ((float)a.topk * n * n) : 0.0f;
    a.counts[e] = c;
    a.balance[e] = bal;
    if (n_rows > 0)
      loss += bal * tot_p[e];
    mine += (c + a.align - 1) / a.align * a.align;
  }
  int32_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(sum, d);
    if (lane >= d)
      sum += o;
  }
  int32_t end = sum - mine;
  for (int e = e0; e < e1; ++e) {
    end += (tot_n[e] + a.align - 1) / a.align * a.align;
    a.ends[e] = end;
  }
  loss = lanes_sum(loss);
  if (lane == 0)
    *a.loss = loss;
}

template <typename T, int G, int V, int U>
__global__ __launch_bounds__(kRouterThreads) void router_fwd_kernel(RouterArgs a) {
  constexpr int kRows = 64 / G;   // rows to a wave
  __shared__ float meet[kRouterWaves][G * V];   // the waves' p sums; their total in the first
  __shared__ int32_t tot_n[G * V];
  __shared__ int32_t tot_rows;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int gl = lane % G;
  for (int e = threadIdx.x; e < a.experts; e += kRouterThreads)
    tot_n[e] = 0;
  if (threadIdx.x == 0)
    tot_rows = 0;
  lds_barrier();

  float psum[V];
#pragma unroll
  for (int v = 0; v < V; ++v)
    psum[v] = 0.0f;
  int32_t rows_here = 0;

  const int64_t stride = (int64_t)gridDim.x * kRouterWaves * kRows;
  // (binary32 rows would take too many registers twice)
  constexpr bool kAhead = sizeof(T) == 2;
  RowWords<T, G, V, U> words;
  bool next_in = false;
  auto load_ahead = [&](int64_t row) {
    next_in = row < a.rows && (a.valid == nullptr || a.valid[row] != 0);
    if (next_in)
      words.load(static_cast<const T*>(a.z) + row * a.ld, a.experts, gl);
  };
  const int64_t start = ((int64_t)blockIdx.x * kRouterWaves + wave) * kRows;
  if constexpr (kAhead)
    load_ahead(start + lane / G);
  for (int64_t base = start; base < a.rows; base += stride) {
    const int64_t row = base + lane / G;
    float z[V];
    if constexpr (kAhead) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        z[v] = next_in && router_col<G, U>(v, gl) < a.experts ? words.w[v / U].get(v % U) : -INFINITY;
      load_ahead(row + stride);
    } else {
      const bool in = row < a.rows && (a.valid == nullptr || a.valid[row] != 0);
      load_logits<T, G, V, U>(static_cast<const T*>(a.z) + (in ? row : 0) * a.ld, in ? a.experts : 0, gl, -INFINITY, z);
    }
    // (a group's columns fit in kColBits)
    constexpr int kColBits = G == 16 ? 8 : 10, kKeyBits = 31 - kColBits;
    constexpr uint32_t kColMask = (1u << kColBits) - 1;
    uint32_t key[V], top = 0;
    float zmax = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      key[v] = short_key<T, kKeyBits>(z[v]) << kColBits | (kColMask - (uint32_t)router_col<G, U>(v, gl));
      top = max(top, key[v]);
      zmax = __builtin_elementwise_maximum(zmax, z[v]);
    }
    top = lanes_max<G>(top);
    zmax = lanes_fmax<G>(zmax);
    const bool part = top > kColMask;   // the row takes part
    if (!part)
      zmax = 0.0f;
    float e[V], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      e[v] = exp_fast(z[v] - zmax);
      sum += e[v];
    }
    sum = lanes_sum<G>(sum);
    const float inv = part ? 1.0f / sum : 0.0f;
    if (part) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        psum[v] += e[v] * inv;
    }
    rows_here += part && gl == 0;

    // lane j of the group keeps the choices j, j + G, ...
    constexpr int kKeep = (MX_MAX_TOPK + G - 1) / G;
    int32_t idx[kKeep];
    auto keep = [&](int j, int32_t col) {
      if (gl == j % G) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
          if (i == j / G)
            idx[i] = col;
      }
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      idx[i] = -1;
    uint32_t last = top;
    keep(0, part ? (int32_t)(kColMask - (top & kColMask)) : -1);
    bool alike = false;
    const int rounds = sizeof(T) == 2 ? a.topk : min(a.topk + 1, a.experts);
    for (int j = 1; j < rounds; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int v = 0; v < V; ++v)
        best = max(best, key[v] - last);
      best = lanes_max<G>(best) + last;
      const bool open = best > kColMask;
      alike |= open && best >> kColBits == last >> kColBits;
      last = best;
      if (j < a.topk)
        keep(j, open ? (int32_t)(kColMask - (best & kColMask)) : -1);
    }
    if (sizeof(T) == 4 && __any(alike)) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        key[v] = order_key(z[v]);
      for (int j = 0; j < a.topk; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
          best = max(best, key[v]);
        best = lanes_max<G>(best);
        uint32_t col = 0xFFFFFFFFu;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
          col = key[v] == best ? (uint32_t)router_col<G, U>(v, gl) : col;
        col = lanes_min<G>(col);
#pragma unroll
        for (int v = 0; v < V; ++v)
          key[v] = (uint32_t)router_col<G, U>(v, gl) == col ? 0u : key[v];
        keep(j, best > kClosedKey ? (int32_t)col : -1);
      }
    }
    float gate[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      gate[i] = 0.0f;
      if (idx[i] >= 0) {
        float f[1];
        unpack(static_cast<const T*>(a.z) + row * a.ld + idx[i], f);
        gate[i] = exp_fast(f[0] - zmax) * inv;
        atomicAdd(&tot_n[idx[i]], 1);
      }
    }
    if (a.normalize) {
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        total += gate[i];
      total = lanes_sum<G>(total);
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        gate[i] = part ? gate[i] / total : 0.0f;
    }
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int j = i * G + gl;
        if (j < a.topk) {
          a.chosen[row * a.topk + j] = idx[i];
          a.gates[row * a.topk + j] = idx[i] < 0 ? 0.0f : gate[i];
        }
      }
      if (gl == 0)
        a.lse[row] = part ? zmax + logf(sum) : 0.0f;
    }
  }

  // p sums: the groups of a wave by lane moves, then the waves in LDS
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (G == 16) {
      psum[v] = across_rows16(psum[v]);
    }
  }
  if (rows_here > 0)
    atomicAdd(&tot_rows, rows_here);
  if (lane < G) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      meet[wave][router_col<G, U>(v, gl)] = psum[v];
  }
  lds_barrier();
  float* tot_p = meet[0];
  for (int e = threadIdx.x; e < a.experts; e += kRouterThreads) {
    float p = tot_p[e];
#pragma unroll
    for (int w = 1; w < kRouterWaves; ++w)
      p += meet[w][e];
    tot_p[e] = p;
  }
  lds_barrier();
  if (gridDim.x == 1) {
    if (wave == 0)
      router_finish(a, tot_p, tot_n, tot_rows);
    return;
  }
  for (int c = threadIdx.x; c < a.experts; c += kRouterThreads) {
    a.part_p[(int64_t)blockIdx.x * router_stride(a.experts) + c] = tot_p[c];
    a.part_n[(int64_t)blockIdx.x * router_stride(a.experts) + c] = tot_n[c];
  }
  if (threadIdx.x == 0)
    a.part_rows[blockIdx.x] = tot_rows;
}

// Adds up the workgroups' rows: four columns belong to 1024 / width threads
// (width the power of two that holds a row), each taking every so many-th row,
// with many loads in flight: one workgroup has the whole workspace to read.
// (Sixteen workgroups, the last of which goes on to the ends and the loss: 7.7
// against 8.4 us for 65536 rows of 256, too little for what it takes.)
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
__global__ __launch_bounds__(kRouterThreads) void router_fold_kernel(RouterArgs a, int32_t blocks) {
  __shared__ f32x4 sum_p[kRouterThreads];
  __shared__ i32x4 sum_n[kRouterThreads];
  __shared__ int32_t rows_total;
  if (threadIdx.x == 0)
    rows_total = 0;
  lds_barrier();
  const int quads = router_stride(a.experts) / 4;
  int width = 1;
  while (width < quads)
    width *= 2;
  const int slices = kRouterThreads / width;
  const int c = threadIdx.x % width, slice = threadIdx.x / width;
  f32x4 p = {};
  i32x4 n = {};
  if (c < quads) {
    const f32x4* pp = reinterpret_cast<const f32x4*>(a.part_p) + c;
    const i32x4* pn = reinterpret_cast<const i32x4*>(a.part_n) + c;
#pragma unroll 8
    for (int b = slice; b < blocks; b += slices) {
      p += pp[(int64_t)b * quads];
      n += pn[(int64_t)b * quads];
    }
  }
  sum_p[threadIdx.x] = p;
  sum_n[threadIdx.x] = n;
  if ((int)threadIdx.x < blocks)
    atomicAdd(&rows_total, a.part_rows[threadIdx.x]);
  lds_barrier();
  if (slice == 0) {
    for (int s = 1; s < slices; ++s) {
      p += sum_p[s * width + c];
      n += sum_n[s * width + c];
    }
    sum_p[c] = p;
    sum_n[c] = n;
  }
  lds_barrier();
  if (threadIdx.x < 64)
    router_finish(a, reinterpret_cast<const float*>(sum_p), reinterpret_cast<const int32_t*>(sum_n), rows_total);
}

constexpr int kRouterBwdThreads = 256;
// Four workgroups to a CU, which go on to further rows: each sets up balance
// and its LDS once.  65536 rows of 256: 256 workgroups 44 us, 512 32, 1024 30,
// 2048 36, 4096 41.
constexpr int64_t kRouterBwdBlocks = 1024;

template <typename T, int G, int V, int U>
__global__ __launch_bounds__(kRouterBwdThreads) void router_bwd_kernel(RouterArgs a) {
  constexpr int kRows = 64 / G;
  constexpr int kWaves = kRouterBwdThreads / 64;
  constexpr int kKeep = (MX_MAX_TOPK + G - 1) / G;
  // The chosen experts' d_j of the wave's rows, 0 elsewhere, W of a lane's
  // logits side by side: the lanes that have them put them in, the lanes that
  // own the columns take them out (comparing each column with each choice
  // instead took 37 against 30 us for 65536 rows of 256, topk 8).
  constexpr int W = V < 4 ? V : 4;
  __shared__ __attribute__((aligned(16))) float sparse[kWaves][V / W][64][W];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int gl = lane % G;
  // place of column e of this lane's row
  auto sparse_at = [&](int e) -> float& {
    const int q = e / U, v = q / G * U + e % U;
    return sparse[wave][v / W][lane / G * G + q % G][v % W];
  };
#pragma unroll
  for (int v = 0; v < V; ++v)
    sparse[wave][v / W][lane][v % W] = 0.0f;
  const float dloss = a.dloss != nullptr ? *a.dloss : 0.0f;
  float bal[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = router_col<G, U>(v, gl);
    bal[v] = c < a.experts ? dloss * a.in_balance[c] : 0.0f;
  }
  const int64_t stride = (int64_t)gridDim.x * kWaves * kRows;
  const int64_t start = ((int64_t)blockIdx.x * kWaves + wave) * kRows;
  // the choices of the next rows, loaded a turn ahead: what they point at can
  // then be loaded together with everything else
  int32_t ahead[kKeep];
  auto load_chosen = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      ahead[i] = row < a.rows && i * G + gl < a.topk ? a.in_chosen[row * a.topk + i * G + gl] : -1;
  };
  load_chosen(start + lane / G);
  for (int64_t base = start; base < a.rows; base += stride) {
    const int64_t row = base + lane / G;
    const bool in = row < a.rows;
    // lane j of the group works out d_j, d_{j + G}, ... of the chosen experts
    int32_t idx[kKeep];
    float d[kKeep], pc[kKeep], dg = 0.0f, total = 0.0f;
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      idx[i] = ahead[i] < a.experts ? ahead[i] : -1;
    // a row that takes no part has -1 in its first slot (of the group's first
    // lane); what its logits hold is not used
    const bool part = __shfl(ahead[0], 0, G) >= 0;
    const T* zr = static_cast<const T*>(a.z) + (in ? row : 0) * a.ld;
    const float lse = in ? a.in_lse[row] : 0.0f;
    float z[V];
    load_logits<T, G, V, U>(zr, in ? a.experts : 0, gl, -INFINITY, z);
    float zc[kKeep], gate[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      d[i] = gate[i] = 0.0f;
      zc[i] = -INFINITY;
      if (idx[i] >= 0) {
        const int64_t at = row * a.topk + i * G + gl;
        float f[1];
        unpack(zr + idx[i], f);
        zc[i] = f[0];
        if (a.dgates != nullptr) {
          d[i] = a.dgates[at];
          gate[i] = a.in_gates[at];
        }
      }
    }
    load_chosen(row + stride);
    float p[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      p[v] = part ? exp_fast(z[v] - lse) : 0.0f;
    // p is e^(z - lse) over its sum, which is 1 but for lse's rounding: up to
    // |lse| = 16 that changes p by 2^-21, as the exponential's own error does,
    // and is left.  A far larger lse (of a row that a mask of the type's lowest
    // value covers, say) may have lost all of the sum's logarithm.
    float scale = 1.0f;
    const bool coarse = part && __builtin_fabsf(lse) > 16.0f;
    if (__any(coarse)) {
      float psum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        psum += p[v];
      psum = lanes_sum<G>(psum);
      scale = coarse ? 1.0f / psum : 1.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        p[v] *= scale;
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      pc[i] = exp_fast(zc[i] - lse) * scale;
      dg += d[i] * gate[i];
      total += pc[i];
    }
    if (a.normalize) {
      dg = lanes_sum<G>(dg);
      total = lanes_sum<G>(total);
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        d[i] = idx[i] >= 0 && a.dgates != nullptr ? (d[i] - dg) / total : 0.0f;
    }
    float along = 0.0f;
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      along += pc[i] * d[i];
    float dp[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      dp[v] = bal[v];
      along += p[v] * bal[v];
    }
    along = lanes_sum<G>(along);
    if (a.dgates != nullptr) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (idx[i] >= 0)
          sparse_at(idx[i]) = d[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int v = 0; v < V; ++v)
        dp[v] += sparse[wave][v / W][lane][v % W];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (idx[i] >= 0)
          sparse_at(idx[i]) = 0.0f;
    }
    if (in) {
      T* dr = static_cast<T*>(a.dz) + row * a.experts;
#pragma unroll
      for (int q = 0; q < V / U; ++q) {
        const int c = router_col<G, U>(q * U, gl);
        float f[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int v = q * U + i;
          // a closed expert's p is 0 and stays so
          f[i] = part ? p[v] * (dp[v] - along) : 0.0f;
        }
        if (c < a.experts)
          store(dr + c, f);
      }
    }
  }
}

static int64_t router_rows_per_block(int64_t experts, int waves) { return (experts <= 256 ? 4 : 1) * (int64_t)waves; }
static int64_t router_blocks(int64_t rows, int64_t experts) {
  const int64_t per = router_rows_per_block(experts, kRouterWaves);
  const int64_t want = (rows + per - 1) / per;
  return want < 1 ? 1 : want < kRouterBlocks ? want : kRouterBlocks;
}

int64_t router_workspace_bytes(int64_t rows, int64_t experts) {
  const int64_t blocks = router_blocks(rows, experts);
  return blocks == 1 ? 0 : blocks * (8 * (int64_t)router_stride((int32_t)experts) + 4);
}

template <typename T, int G, int V, int U>
static hipError_t launch_router(const RouterArgs& a, bool bwd, int64_t blocks, hipStream_t stream) {
  if (bwd) {
    hipLaunchKernelGGL((router_bwd_kernel<T, G, V, U>), dim3((unsigned)blocks), dim3(kRouterBwdThreads), 0, stream, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((router_fwd_kernel<T, G, V, U>), dim3((unsigned)blocks), dim3(kRouterThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1)
    return e;
  hipLaunchKernelGGL(router_fold_kernel, dim3(1), dim3(kRouterThreads), 0, stream, a, (int32_t)blocks);
  return hipGetLastError();
}

// Logits to a lane: the smallest power of two that holds the row, at least a
// 16-byte word's worth on the wide path.
template <typename T, int U>
static hipError_t launch_router_width(const RouterArgs& a, bool bwd, int64_t blocks, hipStream_t stream) {
  if (a.experts <= 256) {
    if constexpr (U == 1) {
      if (a.experts <= 16)
        return launch_router<T, 16, 1, U>(a, bwd, blocks, stream);
      if (a.experts <= 32)
        return launch_router<T, 16, 2, U>(a, bwd, blocks, stream);
    }
    if constexpr (U <= 4) {
      if (a.experts <= 64)
        return launch_router<T, 16, 4, U>(a, bwd, blocks, stream);
    }
    if (a.experts <= 128)
      return launch_router<T, 16, 8, U>(a, bwd, blocks, stream);
    return launch_router<T, 16, 16, U>(a, bwd, blocks, stream);
  }
  if (a.experts <= 512)
    return launch_router<T, 64, 8, U>(a, bwd, blocks, stream);
  return launch_router<T, 64, 16, U>(a, bwd, blocks, stream);
}

static hipError_t launch_router_any(const RouterArgs& a, bool f32, bool vec, bool bwd, int64_t blocks,
                                    hipStream_t stream) {
  // rows of at most 32 experts fit single loads
  vec = vec && a.experts > 32;
  if (f32)
    return vec ? launch_router_width<float, 4>(a, bwd, blocks, stream)
               : launch_router_width<float, 1>(a, bwd, blocks, stream);
  return vec ? launch_router_width<uint16_t, 8>(a, bwd, blocks, stream)
             : launch_router_width<uint16_t, 1>(a, bwd, blocks, stream);
}

hipError_t launch_router_fwd(const void* logits, int64_t ld, bool f32, const uint8_t* valid, int64_t rows,
                             int32_t experts, int32_t topk, bool normalize, int32_t align, int32_t* chosen,
                             float* gates, float* lse, int32_t* counts, int32_t* ends, float* balance, float* loss,
                             void* workspace, bool vec, hipStream_t stream) {
  RouterArgs a = {};
  a.z = logits, a.ld = ld, a.rows = rows, a.valid = valid, a.experts = experts, a.topk = topk;
  a.normalize = normalize, a.align = align, a.chosen = chosen, a.gates = gates, a.lse = lse, a.counts = counts;
  a.ends = ends, a.balance = balance, a.loss = loss;
  const int64_t blocks = router_blocks(rows, experts);
  a.part_p = static_cast<float*>(workspace);
  a.part_n = reinterpret_cast<int32_t*>(a.part_p + blocks * router_stride(experts));
  a.part_rows = a.part_n + blocks * router_stride(experts);
  return launch_router_any(a, f32, vec, false, blocks, stream);
}

hipError_t launch_router_bwd(const void* logits, int64_t ld, bool f32, const float* lse, const int32_t* chosen,
                             const float* gates, const float* balance, const float* dgates, const float* dloss,
                             int64_t rows, int32_t experts, int32_t topk, bool normalize, void* dlogits, bool vec,
                             hipStream_t stream) {
  RouterArgs a = {};
  a.z = logits, a.ld = ld, a.rows = rows, a.experts = experts, a.topk = topk, a.normalize = normalize;
  a.in_lse = lse, a.in_chosen = chosen, a.in_gates = gates, a.in_balance = balance, a.dgates = dgates;
  a.dloss = dloss, a.dz = dlogits;
  const int64_t per = router_rows_per_block(experts, kRouterBwdThreads / 64);
  const int64_t want = (rows + per - 1) / per;
  return launch_router_any(a, f32, vec, true, want < kRouterBwdBlocks ? want : kRouterBwdBlocks, stream);
}

}  // namespace mx
