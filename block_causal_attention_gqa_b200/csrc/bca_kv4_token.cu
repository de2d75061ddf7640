// Attention of a few query rows over the 4-bit cache, and the attention
// weight its keys receive (single tokens, short blocks of tokens).
//
// Mathematics.  The rows of a key/value head (group heads x queries) come in
// tiles of 8.  With Q^ = q r_q gamma_q gamma_k scale log2(e) (rotated first),
//   s_ij = Q^_i . K^_j,  o_i = sum_j 2^(s_ij - m) v_j / sum_j 2^(s_ij - m)
// with one pass over the history: a running reference m and sum per row.
//
// The bytes of the cache bound it (144 a token and head at head_dim 128), at
// 23 bytes a clock and SM.  CUDA cores could not keep up (each 4-bit value
// meets every row of the group), so the products are mma.m16n8k16 with fp16
// operands, and all the work per value left to the CUDA cores is half a
// conversion (e2m1x2 -> f16x2) and half a multiplication by the block's scale.
//   - The cached values are exact in fp16.  The other operands are split in
//     two fp16 numbers, x = hi + lo: the 8 rows fill M = 0..7 with hi and
//     M = 8..15 with lo, so the split costs no more matrix instructions than a
//     half-empty tile would, scores and sums are good to fp32's last bits, and
//     a lane finds both parts of a product in its own accumulator.
//   - The layouts of the fragments are met by renaming, not by moving data.
//     The features of a dot product may be summed in any order, so lane c of a
//     quad holds a contiguous quarter of a key row; and the columns of the
//     second product may stand in any order, so lane group g holds a contiguous
//     eighth of a value row, whose bytes hold two tokens each: a converted byte
//     is a fragment register.  Every shared-memory read of a warp is one
//     contiguous run.
//   - P is scaled by 2^7 (reference m - 7) and m moves only when a score passes
//     it by 8, so P stays below 2^15 in fp16 and loses nothing above 2^-31.
//   - Each warp streams its own steps of 32 tokens through its own ring of
//     bulk copies (one lane issues, mbarriers complete), so warps do not wait
//     for one another until the end.
// A history is cut into n_splits parts for different CTAs; kv4_combine_kernel
// joins their (m, l, O), launched early by programmatic dependent launch.
#include <algorithm>

#include "bca_kv4.cuh"
#include "bca_kv4_query.cuh"

namespace magi {
namespace kv4 {
namespace {

using namespace sm100;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kStep = 32;              // tokens of one step of a warp
constexpr float kMove = 8.f;           // log2 units a score may pass the reference by
constexpr float kLift = 7.f;           // P carries a factor 2^kLift

enum : int { kErrRing = 3101, kErrRingW = 3102 };

template <int D>
struct Ring {
  static constexpr int kKc = kStep * D / 2, kKs = kStep * D / 16, kVc = kStep / 2 * D, kVs = kStep * D / 16;
  static constexpr int kStage = kKc + kKs + kVc + kVs;
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kQ = D / 16 * 32 * 16;             // query fragments of a row tile
  static constexpr int kMergeRow = D + 4;                 // floats, padded
  static constexpr int kMerge = kWarps * 8 * kMergeRow * 4;
  static constexpr int kRing = kWarps * kWarp;
  static constexpr int kBody = kRing > kMerge ? kRing : kMerge;   // the merge reuses the ring
  static constexpr int kTotal = kBody + kQ + kWarps * 8 * 8 + kWarps * kStages * 8;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bounded wait whose outcome the whole warp agrees on.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status, int code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, code));
}

// Scores of 8 tokens (key rows kc, scales ks of the tile) against the row
// tile: acc[0..1] the hi part of tokens 2c, 2c + 1 for row g, acc[2..3] the lo part.
template <int D>
__device__ __forceinline__ void score_tile(const uint8_t* kc, const uint8_t* ks, int g, int c,
                                           const uint32_t (&q)[D / 16][4], float (&acc)[4]) {
  uint32_t w[D / 32];
  uint32_t sc[2];
  if constexpr (D == 128) {
    const uint4 x = *reinterpret_cast<const uint4*>(kc + g * 64 + c * 16);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    const uint32_t s2 = *reinterpret_cast<const uint16_t*>(ks + g * 8 + c * 2);
    sc[0] = scale_dup(s2 & 0xffu);
    sc[1] = scale_dup(s2 >> 8);
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(kc + g * 32 + c * 8);
    w[0] = x.x; w[1] = x.y;
    sc[0] = sc[1] = scale_dup(ks[g * 4 + c]);
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint32_t h[4];
    codes_f16x8(w[i], h);
    const uint32_t s = sc[i / 2];
    mma16816(acc, q[2 * i], hmul2(h[0], s), hmul2(h[1], s));
    mma16816(acc, q[2 * i + 1], hmul2(h[2], s), hmul2(h[3], s));
  }
}

template <int D>
__device__ __forceinline__ void load_query_fragments(const uint8_t* smem_q, int lane, uint32_t (&q)[D / 16][4]) {
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    const uint4 x = *reinterpret_cast<const uint4*>(smem_q + (j * 32 + lane) * 16);
    q[j][0] = x.x; q[j][1] = x.y; q[j][2] = x.z; q[j][3] = x.w;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 3) kv4_token_fwd_kernel(const FwdParams4 p) {
  using R = Ring<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* smem_q = smem + R::kBody;
  float2* smem_ml = reinterpret_cast<float2*>(smem_q + R::kQ);            // [warp][row]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_ml + kWarps * 8);     // [warp][stage]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x, row0 = blockIdx.y * kTokenRows, bh = blockIdx.z;
  const int b = bh / p.c.heads, hk = bh % p.c.heads;
  const int G = p.heads_q / p.c.heads, rows = G * p.sq;
  const int len = min(max(__ldg(p.lengths + b), 0), p.c.cap);
  const int steps = (len + kStep - 1) / kStep;
  const int s_begin = (int)((int64_t)steps * split / p.n_splits);
  const int s_end = (int)((int64_t)steps * (split + 1) / p.n_splits);
  uint8_t* ring = smem + warp * R::kWarp;
  uint64_t* bar = bars + warp * kStages;

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bar + i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int n_steps = s_end - s_begin > warp ? (s_end - s_begin - warp + kWarps - 1) / kWarps : 0;
  auto issue = [&](int k) {   // by lane 0
    const int64_t tok = (int64_t)(s_begin + warp + k * kWarps) * kStep;
    const int64_t at = (int64_t)bh * p.c.cap + tok;
    uint8_t* dst = ring + (k % kStages) * R::kStage;
    uint64_t* bb = bar + k % kStages;
    mbar_arrive_expect_tx(bb, R::kStage);
    bulk_load(dst, p.c.kc + at * (D / 2), R::kKc, bb);
    bulk_load(dst + R::kKc, p.c.ks + at * (D / 16), R::kKs, bb);
    bulk_load(dst + R::kKc + R::kKs, p.c.vc + at / 2 * D, R::kVc, bb);
    bulk_load(dst + R::kKc + R::kKs + R::kVc, p.c.vs + at * (D / 16), R::kVs, bb);
  };
  if (lane == 0)
    for (int k = 0; k < min(n_steps, kStages); ++k) issue(k);

  // the row tile's queries, while the first copies are under way
  for (int i = warp; i < kTokenRows; i += kWarps)
    fold_query_fragment<D>(p, b, hk, G, row0 + i, rows, i, lane, smem_q);
  __syncthreads();
  uint32_t q[D / 16][4];
  load_query_fragments<D>(smem_q, lane, q);

  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m = -INFINITY, l = 0.f;
  bool ok = true;
  for (int k = 0; k < n_steps; ++k) {
    ok = warp_wait(bar + k % kStages, (k / kStages) & 1, p.status, kErrRing);
    if (!ok) break;
    const uint8_t* kc = ring + (k % kStages) * R::kStage;
    const uint8_t* ks = kc + R::kKc;
    const uint8_t* vc = ks + R::kKs;
    const uint8_t* vs = vc + R::kVc;
    const int tok = (s_begin + warp + k * kWarps) * kStep;
    float x[4][2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      score_tile<D>(kc + t * 8 * (D / 2), ks + t * 8 * (D / 16), g, c, q, acc);
      x[t][0] = acc[0] + acc[2];
      x[t][1] = acc[1] + acc[3];
    }
    const bool tail = tok + kStep > len;
    if (tail) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (tok + t * 8 + 2 * c + i >= len) x[t][i] = -INFINITY;
    }
    const float top = fmaxf(fmax3(fmaxf(x[0][0], x[0][1]), x[1][0], x[1][1]),
                            fmax3(fmaxf(x[2][0], x[2][1]), x[3][0], x[3][1]));
    if (__any_sync(0xffffffffu, top > m + kMove)) {
      float t = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
      const float m1 = fmaxf(m, t);
      const float alpha = m1 == -INFINITY ? 1.f : fast_exp2(m - m1);
      m = m1;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] *= alpha;
    }
    const float shift = m == -INFINITY ? 0.f : kLift - m;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float p0 = fast_exp2(x[t][0] + shift), p1 = fast_exp2(x[t][1] + shift);
      l += p0 + p1;
      hi[t] = pack_f16x2(p0, p1);
      const float2 back = __half22float2(*reinterpret_cast<__half2*>(&hi[t]));
      lo[t] = pack_f16x2(p0 - back.x, p1 - back.y);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t a[4] = {hi[2 * u], lo[2 * u], hi[2 * u + 1], lo[2 * u + 1]};
      uint32_t v[2][D / 32], sc[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * u + 4 * i + c;    // tokens 2 row, 2 row + 1 of the step
        const uint8_t* src = vc + row * D + g * (D / 8);
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(src);
          v[i][0] = w.x; v[i][1] = w.y; v[i][2] = w.z; v[i][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(src);
          v[i][0] = w.x; v[i][1] = w.y;
        }
        const uint32_t s2 = *reinterpret_cast<const uint16_t*>(vs + (row * (D / 16) + g * (D / 8) / 16) * 2);
        sc[i] = scale_pair(s2 & 0xffu, s2 >> 8);
        if (tail) {   // rows behind the end may hold anything: their values count as zero
          if (tok + 2 * row >= len) sc[i] = 0u;
          else if (tok + 2 * row + 1 >= len) sc[i] &= 0xffffu;
        }
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t h0[4], h1[4];
        codes_f16x8(v[0][i], h0);
        codes_f16x8(v[1][i], h1);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(o[4 * i + j], a, hmul2(h0[j], sc[0]), hmul2(h1[j], sc[1]));
      }
    }
    __syncwarp();
    if (lane == 0 && k + kStages < n_steps) issue(k + kStages);
  }
  // join the warps: every issued copy has been waited for, so the ring is free
  if (__syncthreads_or(!ok)) return;
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  // scores that are NaN (a query that is) leave the reference at -inf: they must not pass for an empty row
  if (m == -INFINITY && !(l == 0.f)) m = kLift;
  float* merge = reinterpret_cast<float*>(smem) + warp * 8 * R::kMergeRow + g * R::kMergeRow;
#pragma unroll
  for (int j = 0; j < D / 8; j += 4) {
    float4 a, e;
    a.x = o[j][0] + o[j][2]; a.y = o[j + 1][0] + o[j + 1][2]; a.z = o[j + 2][0] + o[j + 2][2]; a.w = o[j + 3][0] + o[j + 3][2];
    e.x = o[j][1] + o[j][3]; e.y = o[j + 1][1] + o[j + 1][3]; e.z = o[j + 2][1] + o[j + 2][3]; e.w = o[j + 3][1] + o[j + 3][3];
    *reinterpret_cast<float4*>(merge + 2 * c * (D / 8) + j) = a;
    *reinterpret_cast<float4*>(merge + (2 * c + 1) * (D / 8) + j) = e;
  }
  if (c == 0) smem_ml[warp * 8 + g] = make_float2(m == -INFINITY ? -INFINITY : m - kLift, l);
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // 16 threads a row, D / 16 features each
  constexpr int F = D / 16;
  const int i = threadIdx.x >> 4, f0 = (threadIdx.x & 15) * F;
  const int row = row0 + i;
  float mm = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, smem_ml[w * 8 + i].x);
  float acc[F] = {}, ll = 0.f;
  if (mm != -INFINITY) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = smem_ml[w * 8 + i];
      const float s = fast_exp2(ml.x - mm);
      ll += ml.y * s;
      const float* src = reinterpret_cast<const float*>(smem) + (w * 8 + i) * R::kMergeRow + f0;
#pragma unroll
      for (int f = 0; f < F; ++f) acc[f] = fmaf(src[f], s, acc[f]);
    }
  }
  if (row >= rows) return;
  if (p.n_splits > 1) {
    const int64_t at = ((int64_t)split * gridDim.z + bh) * rows + row;
    if ((threadIdx.x & 15) == 0) p.part_ml[at] = make_float2(mm, ll);
    if (mm != -INFINITY) {
#pragma unroll
      for (int f = 0; f < F; f += 4)
        *reinterpret_cast<float4*>(p.part_o + at * D + f0 + f) = make_float4(acc[f], acc[f + 1], acc[f + 2], acc[f + 3]);
    }
  } else {
    finish_row<F>(p, b, hk, G, row, D, f0, mm, ll, acc);
  }
}

// Joins the parts of the rows: one warp a row.
template <int D>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const FwdParams4 p) {
  constexpr int F = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int G = p.heads_q / p.c.heads, rows = G * p.sq;
  const int64_t groups = (int64_t)p.c.batch * p.c.heads;
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= groups * rows) return;
  const int64_t stride = groups * rows;
  float mm = -INFINITY;
  for (int s = lane; s < p.n_splits; s += 32) mm = fmaxf(mm, p.part_ml[s * stride + r].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  float acc[F] = {}, ll = 0.f;
  if (mm != -INFINITY) {
#pragma unroll 4
    for (int s = 0; s < p.n_splits; ++s) {
      const int64_t at = s * stride + r;
      const float2 ml = p.part_ml[at];
      if (ml.x == -INFINITY) continue;     // an empty part wrote no O
      const float w = fast_exp2(ml.x - mm);
      ll += ml.y * w;
#pragma unroll
      for (int f = 0; f < F; ++f) acc[f] = fmaf(p.part_o[at * D + lane * F + f], w, acc[f]);
    }
  }
  const int bh = (int)(r / rows);
  finish_row<F>(p, bh / p.c.heads, bh % p.c.heads, G, (int)(r % rows), D, lane * F, mm, ll, acc);
}

// ------------------------------------------------------------------ weights
//
// w_j <- decay w_j + sum_i 2^(s_ij - lse_i log2 e): keys only.  A warp
// converts a step's 32 keys once and holds them as fragments while the row
// tiles pass, so any number of rows reads the cache once.
template <int D>
struct RingW {
  static constexpr int kKc = kStep * D / 2, kKs = kStep * D / 16, kW = kStep * 4;
  static constexpr int kStage = kKc + kKs + kW;
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kRing = kWarps * kWarp;
  static constexpr int kTileQ = D / 16 * 32 * 16 + 8 * 4;   // fragments, then the 8 rows' lse in log2 units
  static constexpr int bytes(int tiles) { return kRing + tiles * kTileQ + kWarps * kStages * 8; }
};

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_token_weights_kernel(const FwdParams4 p, int tiles) {
  using R = RingW<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + R::kRing);
  uint8_t* smem_q = smem + R::kRing + kWarps * kStages * 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int bh = blockIdx.y, b = bh / p.c.heads, hk = bh % p.c.heads;
  const int G = p.heads_q / p.c.heads, rows = G * p.sq;
  const int len = min(max(__ldg(p.lengths + b), 0), p.c.cap);
  const int steps = (len + kStep - 1) / kStep;
  const int s_begin = (int)((int64_t)steps * blockIdx.x / p.n_splits);
  const int s_end = (int)((int64_t)steps * (blockIdx.x + 1) / p.n_splits);
  uint8_t* ring = smem + warp * R::kWarp;
  uint64_t* bar = bars + warp * kStages;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bar + i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int n_steps = s_end - s_begin > warp ? (s_end - s_begin - warp + kWarps - 1) / kWarps : 0;
  const bool add = p.decay != 0.f;   // a factor of 0 replaces the weights, whatever they hold
  auto issue = [&](int k) {
    const int64_t at = (int64_t)bh * p.c.cap + (int64_t)(s_begin + warp + k * kWarps) * kStep;
    uint8_t* dst = ring + (k % kStages) * R::kStage;
    uint64_t* bb = bar + k % kStages;
    mbar_arrive_expect_tx(bb, R::kKc + R::kKs + (add ? R::kW : 0));
    bulk_load(dst, p.c.kc + at * (D / 2), R::kKc, bb);
    bulk_load(dst + R::kKc, p.c.ks + at * (D / 16), R::kKs, bb);
    if (add) bulk_load(dst + R::kKc + R::kKs, p.weights + at, R::kW, bb);
  };
  if (lane == 0)
    for (int k = 0; k < min(n_steps, kStages); ++k) issue(k);
  for (int i = warp; i < tiles * kTokenRows; i += kWarps) {
    uint8_t* tile = smem_q + (i >> 3) * R::kTileQ;
    fold_query_fragment<D>(p, b, hk, G, i, rows, i & 7, lane, tile);
    if (lane == 0) {
      // a row that saw nothing (lse = -inf) and rows behind the last give no weight
      float x = INFINITY;
      if (i < rows) x = p.w_lse[((int64_t)b * p.heads_q + hk * G + i / p.sq) * p.sq + i % p.sq] * kLog2e;
      reinterpret_cast<float*>(tile + D / 16 * 32 * 16)[i & 7] = x == -INFINITY ? INFINITY : x;
    }
  }
  __syncthreads();
  for (int k = 0; k < n_steps; ++k) {
    if (!warp_wait(bar + k % kStages, (k / kStages) & 1, p.status, kErrRingW)) break;
    const uint8_t* kc = ring + (k % kStages) * R::kStage;
    const uint8_t* ks = kc + R::kKc;
    const int tok = (s_begin + warp + k * kWarps) * kStep;
    float sum[4][2] = {};
    for (int t0 = 0; t0 < tiles; ++t0) {
      const uint8_t* tile = smem_q + t0 * R::kTileQ;
      uint32_t q[D / 16][4];
      load_query_fragments<D>(tile, lane, q);
      const float neg = -reinterpret_cast<const float*>(tile + D / 16 * 32 * 16)[g];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        score_tile<D>(kc + t * 8 * (D / 2), ks + t * 8 * (D / 16), g, c, q, acc);
        sum[t][0] += fast_exp2(acc[0] + acc[2] + neg);
        sum[t][1] += fast_exp2(acc[1] + acc[3] + neg);
      }
    }
    // Sum over the 8 lanes with the same c, each ending with one token: the
    // exchange halves the values each lane still carries.
    float v4[4], v2[2];
    const bool up16 = lane & 16, up8 = lane & 8, up4 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = sum[i >> 1][i & 1], e = sum[2 + (i >> 1)][i & 1];
      const float other = __shfl_xor_sync(0xffffffffu, up16 ? a : e, 16);
      v4[i] = (up16 ? e : a) + other;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, up8 ? v4[i] : v4[2 + i], 8);
      v2[i] = (up8 ? v4[2 + i] : v4[i]) + other;
    }
    const float other = __shfl_xor_sync(0xffffffffu, up4 ? v2[0] : v2[1], 4);
    const float total = (up4 ? v2[1] : v2[0]) + other;
    const int at = (up16 ? 16 : 0) + (up8 ? 8 : 0) + 2 * c + (up4 ? 1 : 0);
    if (tok + at < len) {
      const float old = add ? reinterpret_cast<const float*>(ks + R::kKs)[at] : 0.f;
      p.weights[(int64_t)bh * p.c.cap + tok + at] = add ? fmaf(p.decay, old, total) : total;
    }
    __syncwarp();
    if (lane == 0 && k + kStages < n_steps) issue(k + kStages);
  }
}

template <typename F>
cudaError_t allow_smem(F* f, int bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace

// Parts a history is cut into: enough CTAs for three on each of 148 SMs, of at
// least 128 tokens (a step of each warp) if the cache is full.
int token_splits(const Cache& c, int row_tiles) {
  const int64_t groups = (int64_t)c.batch * c.heads * row_tiles;
  const int64_t want = std::max<int64_t>(1, 148 * 3 / groups);
  return (int)std::min<int64_t>({want, (int64_t)(c.cap + kStep * kWarps - 1) / (kStep * kWarps), (int64_t)128});
}

template <int D>
static cudaError_t token_fwd_d(const FwdParams4& p, cudaStream_t s) {
  using R = Ring<D>;
  const int rows = p.heads_q / p.c.heads * p.sq;
  const cudaError_t e = allow_smem(kv4_token_fwd_kernel<D>, R::kTotal);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.n_splits, (rows + kTokenRows - 1) / kTokenRows, p.c.batch * p.c.heads);
  kv4_token_fwd_kernel<D><<<grid, kThreads, R::kTotal, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_token_fwd(const FwdParams4& p, cudaStream_t s) {
  return p.c.dim == 128 ? token_fwd_d<128>(p, s) : token_fwd_d<64>(p, s);
}

cudaError_t launch_combine(const FwdParams4& p, cudaStream_t s) {
  const int64_t rows = (int64_t)p.c.batch * p.heads_q * p.sq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return p.c.dim == 128 ? cudaLaunchKernelEx(&cfg, kv4_combine_kernel<128>, p)
                        : cudaLaunchKernelEx(&cfg, kv4_combine_kernel<64>, p);
}

template <int D>
static cudaError_t token_weights_d(const FwdParams4& p, cudaStream_t s) {
  const int rows = p.heads_q / p.c.heads * p.sq, tiles = (rows + kTokenRows - 1) / kTokenRows;
  const int bytes = RingW<D>::bytes(tiles);
  const cudaError_t e = allow_smem(kv4_token_weights_kernel<D>, bytes);
  if (e != cudaSuccess) return e;
  kv4_token_weights_kernel<D><<<dim3(p.n_splits, p.c.batch * p.c.heads), kThreads, bytes, s>>>(p, tiles);
  return cudaGetLastError();
}

cudaError_t launch_token_weights(const FwdParams4& p, cudaStream_t s) {
  return p.c.dim == 128 ? token_weights_d<128>(p, s) : token_weights_d<64>(p, s);
}

}  // namespace kv4
}  // namespace magi
