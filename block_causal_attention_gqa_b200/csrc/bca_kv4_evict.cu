// Eviction from the 4-bit cache by accumulated attention weight.
//
// Of the n tokens of a (batch element, head) the last `recent` stay, and of the
// others the `need` with the largest weight (equal weights: the lower index;
// NaN counts as -inf).  Order is kept.
//
// Selection (kv4_select_kernel).  A weight is mapped to an unsigned integer of
// the same order and the need-th largest is found digit by digit (11, 11 and
// 10 bits), a histogram of the candidates with the digits so far at each.  A
// cluster of 8 CTAs shares a head: each keeps the keys of an eighth in shared
// memory, counts them there and adds its counts that are not zero to the
// totals of all eight through distributed shared memory (a few hundred bins;
// reading all eight histograms whole took five times as long).  The kept
// tokens are then numbered in their order by ballots: a warp takes a
// contiguous run and starts at the counts of the runs before it.
//
// Moving (kv4_move_kernel).  Bound by bytes: a kept token is read and written
// once.  A row of the value cache holds two tokens, so a destination row is
// put together from the halves of two source rows.
#include <cooperative_groups.h>

#include <algorithm>

#include "bca_kv4.cuh"

namespace cg = cooperative_groups;

namespace magi {
namespace kv4 {
namespace {

constexpr int kCluster = 8;
constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;

// Order-preserving integer of a weight.
__device__ __forceinline__ uint32_t order_key(float w) {
  w = w == w ? w + 0.f : -INFINITY;   // + 0: -0 is 0
  const uint32_t u = __float_as_uint(w);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 40 * 1024;   // keys a CTA keeps; longer runs are read again each time

struct SelShared {
  uint32_t hist[kBins];      // this CTA's counts
  uint32_t total[3][kBins];  // the cluster's
  uint32_t scan[kSelWarps];
  uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  uint32_t cta_gt, cta_eq;
  uint32_t bin, above;
};

// Candidates of a CTA, and of one of its warps (a multiple of 128: a lane takes
// four neighbours at a time).
__host__ __device__ constexpr int cta_run(int n) { return (n + kCluster * 32 - 1) / (kCluster * 32) * 32; }
__host__ __device__ constexpr int warp_run(int cta) { return (cta + kSelThreads * 4 - 1) / (kSelThreads * 4) * 128; }

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSelThreads) kv4_select_kernel(const EvictParams p, bool held) {
  extern __shared__ __align__(16) uint8_t sel_smem[];
  SelShared& sh = *reinterpret_cast<SelShared*>(sel_smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.y, b = bh / p.src.heads;
  let_next_start();
  wait_for_previous();
  const int len = min(max(p.lengths[b], 0), p.src.cap);
  const int kept = min(len, p.keep);
  const int rec = min(p.recent, kept);
  const int n = len - rec;                      // candidates [0, n)
  const int need = kept - rec;
  const float* w = p.w_src + (int64_t)bh * p.src.cap;
  int32_t* index = p.index + (int64_t)bh * p.keep;
  const int seg = cta_run(n), run = warp_run(seg);
  // this warp's candidates: [a0, a0 + len_w), in steps of 128, a lane four of them
  const int i1 = min((rank + 1) * seg, n), a0 = rank * seg + warp * run;
  const int len_w = min(run, i1 - a0);
  uint32_t* keys = reinterpret_cast<uint32_t*>(sel_smem + sizeof(SelShared)) + warp * run;

  // the keys of four neighbours; 0, which no weight has, behind the last (the
  // row has 128-slot granularity, so reading four is always inside it)
  auto from_row = [&](int o) {
    const float4 x = *(reinterpret_cast<const float4*>(w + a0 + o));
    return make_uint4(order_key(x.x), o + 1 < len_w ? order_key(x.y) : 0u, o + 2 < len_w ? order_key(x.z) : 0u,
                      o + 3 < len_w ? order_key(x.w) : 0u);
  };
  if (held) {
#pragma unroll 4
    for (int o = lane * 4; o < len_w; o += 128) *reinterpret_cast<uint4*>(keys + o) = from_row(o);
  }
  auto four = [&](int o) {
    if (o >= len_w) return make_uint4(0, 0, 0, 0);
    return held ? *reinterpret_cast<const uint4*>(keys + o) : from_row(o);
  };

  // the need-th largest key and how many of those equal to it stay
  uint32_t top = need == 0 ? 0xffffffffu : 0u;   // all stay: every key is above
  uint32_t ties = 0;
  if (need > 0 && need < n) {                    // the same for the whole cluster
    uint32_t prefix = 0, left = (uint32_t)need;
    for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = sh.total[0][i] = sh.total[1][i] = sh.total[2][i] = 0;
    cluster.sync();
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
      auto count = [&](uint32_t key) {
        if (key != 0 && (pass == 0 || (key >> (shift + bits)) == prefix))
          atomicAdd(&sh.hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
      };
      for (int o = lane * 4; o < len_w; o += 128) {
        const uint4 k = four(o);
        count(k.x);
        count(k.y);
        count(k.z);
        count(k.w);
      }
      __syncthreads();
      for (int i = tid; i < kBins; i += kSelThreads) {
        const uint32_t v = sh.hist[i];
        if (v == 0) continue;
        sh.hist[i] = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) atomicAdd(cluster.map_shared_rank(&sh.total[pass][i], r), v);
      }
      cluster.sync();
      // thread t holds the counts of its bins from the top
      constexpr int kPer = kBins / kSelThreads;
      uint32_t cnt[kPer], mine = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) mine += cnt[k] = sh.total[pass][kBins - 1 - (tid * kPer + k)];
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      uint32_t before = incl - mine + __reduce_add_sync(0xffffffffu, lane < warp ? sh.scan[lane] : 0u);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (before < left && before + cnt[k] >= left) {   // exactly one bin
          sh.bin = (uint32_t)(kBins - 1 - (tid * kPer + k));
          sh.above = before;
        }
        before += cnt[k];
      }
      __syncthreads();
      prefix = (prefix << bits) | sh.bin;
      left -= sh.above;
    }
    top = prefix;
    ties = left;
  }
  __syncwarp();

  // number the kept tokens, warp by warp
  uint32_t gt = 0, eq = 0;
  for (int o = lane * 4; o < len_w; o += 128) {
    const uint4 k = four(o);
    gt += (k.x > top) + (k.y > top) + (k.z > top) + (k.w > top);
    eq += (k.x == top) + (k.y == top) + (k.z == top) + (k.w == top);   // (behind the last: 0, and top > 0 or no ties)
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    sh.warp_gt[warp] = gt;
    sh.warp_eq[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t g = __reduce_add_sync(0xffffffffu, sh.warp_gt[lane]), e = __reduce_add_sync(0xffffffffu, sh.warp_eq[lane]);
    if (lane == 0) {
      sh.cta_gt = g;
      sh.cta_eq = e;
    }
  }
  cluster.sync();
  uint32_t gt0 = lane < rank ? *cluster.map_shared_rank(&sh.cta_gt, lane) : 0u;
  uint32_t eq0 = lane < rank ? *cluster.map_shared_rank(&sh.cta_eq, lane) : 0u;
  gt0 = __reduce_add_sync(0xffffffffu, gt0 + (lane < warp ? sh.warp_gt[lane] : 0u));
  eq0 = __reduce_add_sync(0xffffffffu, eq0 + (lane < warp ? sh.warp_eq[lane] : 0u));
  cluster.sync();   // no CTA leaves while its shared memory is read
  const uint32_t below = (1u << lane) - 1u;
  for (int o0 = 0; o0 < len_w; o0 += 128) {
    const int o = o0 + lane * 4;
    const uint4 k4 = four(o);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    uint32_t g = gt0, e = eq0;   // before this lane's first
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t mg = __ballot_sync(0xffffffffu, k[c] > top), me = __ballot_sync(0xffffffffu, k[c] == top);
      g += __popc(mg & below);
      e += __popc(me & below);
      gt0 += __popc(mg);
      eq0 += __popc(me);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (k[c] > top) {
        index[g + min(e, ties)] = a0 + o + c;
        ++g;
      } else if (k[c] == top) {
        if (e < ties) index[g + e] = a0 + o + c;
        ++e;
      }
    }
  }
  for (int i = rank * kSelThreads + tid; i < p.keep - need; i += kCluster * kSelThreads)
    index[need + i] = i < rec ? n + i : -1;
  if (rank == 0 && tid == 0 && bh % p.src.heads == 0) p.new_lengths[b] = kept;
}

// One warp per 16 destination tokens (8 value rows), so that each lane has some
// hundred bytes under way.
template <int D>
__global__ void __launch_bounds__(256) kv4_move_kernel(const EvictParams p) {
  constexpr int kTok = 16;
  constexpr int kK = D / 32;       // 16-byte pieces of a key row
  constexpr int kV = D / 16;       // 16-byte pieces of a value row (two tokens)
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / p.src.heads;
  const int kept = min(min(max(p.lengths[b], 0), p.src.cap), p.keep);
  const int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kTok;
  const int n = min(kTok, kept - t0);
  if (n <= 0) return;
  const int64_t src = (int64_t)bh * p.src.cap, dst = (int64_t)bh * p.dst.cap + t0;
  // lane t (and t + 16): where token t of the sixteen comes from
  const int from = p.index[(int64_t)bh * p.keep + t0 + min(lane & 15, n - 1)];
  uint4 k[kK * kTok / 32], va[kV * kTok / 64], vb[kV * kTok / 64];
#pragma unroll
  for (int i = 0; i < kK * kTok / 32; ++i) {
    const int piece = i * 32 + lane, t = piece / kK;
    const int s = __shfl_sync(0xffffffffu, from, t);
    k[i] = *(reinterpret_cast<const uint4*>(p.src.kc + (src + s) * (D / 2)) + piece % kK);
  }
#pragma unroll
  for (int i = 0; i < kV * kTok / 64; ++i) {
    const int piece = i * 32 + lane, r = piece / kV;
    const int s0 = __shfl_sync(0xffffffffu, from, 2 * r), s1 = __shfl_sync(0xffffffffu, from, 2 * r + 1);
    va[i] = *(reinterpret_cast<const uint4*>(p.src.vc + (src / 2 + s0 / 2) * D) + piece % kV);
    vb[i] = *(reinterpret_cast<const uint4*>(p.src.vc + (src / 2 + s1 / 2) * D) + piece % kV);
  }
  // scales: lanes 0..15 a token's key and value scales each; lane t + 16 its weight
  uint2 ks = make_uint2(0, 0);
  uint4 vs = make_uint4(0, 0, 0, 0);
  float w = 0.f;
  if (lane < 16) {
    if constexpr (D == 128) {
      ks = *(reinterpret_cast<const uint2*>(p.src.ks + (src + from) * 8));
      vs = *(reinterpret_cast<const uint4*>(p.src.vs + (src / 2 + from / 2) * 16));
    } else {
      ks.x = *(reinterpret_cast<const uint32_t*>(p.src.ks + (src + from) * 4));
      const uint2 y = *(reinterpret_cast<const uint2*>(p.src.vs + (src / 2 + from / 2) * 8));
      vs.x = y.x;
      vs.y = y.y;
    }
  } else {
    w = *(p.w_src + src + from);
  }

#pragma unroll
  for (int i = 0; i < kK * kTok / 32; ++i) {
    const int piece = i * 32 + lane;
    if (piece / kK < n) reinterpret_cast<uint4*>(p.dst.kc + dst * (D / 2))[piece] = k[i];
  }
#pragma unroll
  for (int i = 0; i < kV * kTok / 64; ++i) {
    const int piece = i * 32 + lane, r = piece / kV;
    const int s0 = __shfl_sync(0xffffffffu, from, 2 * r), s1 = __shfl_sync(0xffffffffu, from, 2 * r + 1);
    if (2 * r >= n) continue;
    uint4* to = reinterpret_cast<uint4*>(p.dst.vc + dst / 2 * D) + piece;
    const bool two = 2 * r + 1 < n;
    const uint4 old = two ? make_uint4(0, 0, 0, 0) : *to;   // a half that no token takes stays
    const int h0 = 4 * (s0 & 1), h1 = 4 * (s1 & 1);
    auto join = [&](uint32_t a, uint32_t e, uint32_t o) {
      const uint32_t lo = (a >> h0) & 0x0f0f0f0fu;
      return two ? lo | (((e >> h1) & 0x0f0f0f0fu) << 4) : lo | (o & 0xf0f0f0f0u);
    };
    *to = make_uint4(join(va[i].x, vb[i].x, old.x), join(va[i].y, vb[i].y, old.y), join(va[i].z, vb[i].z, old.z),
                     join(va[i].w, vb[i].w, old.w));
  }
  if (lane < n) {
    uint8_t* to = p.dst.ks + (dst + lane) * (D / 16);
    if constexpr (D == 128) *reinterpret_cast<uint2*>(to) = ks;
    else *reinterpret_cast<uint32_t*>(to) = ks.x;
    // the token's bytes of its source row (every second one) to every second byte of the destination row
    const uint32_t x[4] = {vs.x, vs.y, vs.z, vs.w};
    uint8_t* vt = p.dst.vs + (dst / 2 + lane / 2) * (D / 8) + (lane & 1);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) vt[2 * i] = (uint8_t)(x[i / 2] >> (16 * (i & 1) + 8 * (from & 1)));
  }
  if (lane >= 16 && lane - 16 < n) p.w_dst[dst + lane - 16] = w;
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  const int BH = p.src.batch * p.src.heads;
  // room for the keys of an eighth of a full cache, if that is not too much
  const int keys = kSelWarps * warp_run(cta_run(p.src.cap));
  const bool held = keys <= kSelKeys;
  const int bytes = (int)sizeof(SelShared) + (held ? keys * 4 : 0);
  static SmemRecord have;
  cudaError_t e = allow_smem(kv4_select_kernel, bytes, have);
  if (e != cudaSuccess) return e;
  e = launch_early(kv4_select_kernel, dim3(kCluster, BH), kSelThreads, bytes, s, 0, p, held);
  if (e != cudaSuccess) return e;
  const int most = std::min(p.keep, p.src.cap);
  return launch_early(p.src.dim == 128 ? kv4_move_kernel<128> : kv4_move_kernel<64>,
                      dim3((unsigned)((most + 127) / 128), (unsigned)BH), 256, 0, s, 0, p);
}

}  // namespace kv4
}  // namespace magi
