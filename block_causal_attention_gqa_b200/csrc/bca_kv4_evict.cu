// Eviction from the 4-bit cache by accumulated attention weight.
//
// Of the n tokens of a (batch element, head) the last `recent` stay, and of the
// others the `need` with the largest weight (equal weights: the lower index;
// NaN counts as -inf).  Order is kept.
//
// Selection (kv4_select_kernel).  A weight is mapped to an unsigned integer of
// the same order and the need-th largest is found digit by digit (11, 11 and
// 10 bits), a histogram of the candidates with the digits so far at each.  A
// cluster of 8 CTAs shares a head: each counts an eighth, all read the eight
// histograms through distributed shared memory, so nothing but the index
// table goes through global memory.  The kept tokens are then numbered in
// their order by ballots: a warp takes a contiguous run and starts at the
// counts of the runs before it.
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
constexpr int kSelThreads = 512;
constexpr int kBins = 2048;

// Order-preserving integer of a weight.
__device__ __forceinline__ uint32_t order_key(float w) {
  w = w == w ? w + 0.f : -INFINITY;   // + 0: -0 is 0
  const uint32_t u = __float_as_uint(w);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

struct SelShared {
  uint32_t hist[3][kBins];
  uint32_t scan[kSelThreads / 32];
  uint32_t warp_gt[kSelThreads / 32], warp_eq[kSelThreads / 32];
  uint32_t cta_gt, cta_eq;
  uint32_t bin, above;
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSelThreads) kv4_select_kernel(const EvictParams p) {
  __shared__ SelShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.y, b = bh / p.src.heads;
  const int len = min(max(__ldg(p.lengths + b), 0), p.src.cap);
  const int kept = min(len, p.keep);
  const int rec = min(p.recent, kept);
  const int n = len - rec;                      // candidates [0, n)
  const int need = kept - rec;
  const float* w = p.w_src + (int64_t)bh * p.src.cap;
  int32_t* index = p.index + (int64_t)bh * p.keep;
  const int seg = (n + kCluster * 32 - 1) / (kCluster * 32) * 32;
  const int i0 = min(rank * seg, n), i1 = min(i0 + seg, n);

  // the need-th largest key and how many of those equal to it stay
  uint32_t top = need == 0 ? 0xffffffffu : 0u;   // all stay: every key is above or equal
  uint32_t ties = need == 0 ? 0u : 0x7fffffffu;
  if (need > 0 && need < n) {                    // the same for the whole cluster
    uint32_t prefix = 0, left = (uint32_t)need;
    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
      for (int i = i0 + tid; i < i1; i += kSelThreads) {
        const uint32_t key = order_key(__ldg(w + i));
        if (pass == 0 || (key >> (shift + bits)) == prefix)
          atomicAdd(&sh.hist[pass][(key >> shift) & ((1u << bits) - 1u)], 1u);
      }
      cluster.sync();
      // thread t holds the counts of bins 4t .. 4t+3 from the top, over the cluster
      constexpr int kPer = kBins / kSelThreads;
      uint32_t cnt[kPer] = {}, mine = 0;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) {
        const uint32_t* h = cluster.map_shared_rank(&sh.hist[pass][0], r);
#pragma unroll
        for (int k = 0; k < kPer; ++k) cnt[k] += h[kBins - 1 - (tid * kPer + k)];
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) mine += cnt[k];
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      uint32_t before = incl - mine;
      for (int k = 0; k < warp; ++k) before += sh.scan[k];
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

  // number the kept tokens of this CTA's run, warp by warp
  const int wseg = ((i1 - i0) + kSelThreads - 1) / kSelThreads * 32;
  const int a0 = min(i0 + warp * wseg, i1), a1 = min(a0 + wseg, i1);
  uint32_t gt = 0, eq = 0;
  for (int i = a0; i < a1; i += 32) {
    const uint32_t key = i + lane < a1 ? order_key(__ldg(w + i + lane)) : 0u;
    const bool in = i + lane < a1;
    gt += __popc(__ballot_sync(0xffffffffu, in && key > top));
    eq += __popc(__ballot_sync(0xffffffffu, in && key == top));
  }
  if (lane == 0) {
    sh.warp_gt[warp] = gt;
    sh.warp_eq[warp] = eq;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t a = 0, e = 0;
    for (int k = 0; k < kSelThreads / 32; ++k) {
      a += sh.warp_gt[k];
      e += sh.warp_eq[k];
    }
    sh.cta_gt = a;
    sh.cta_eq = e;
  }
  cluster.sync();
  uint32_t gt0 = 0, eq0 = 0;
  for (int r = 0; r < rank; ++r) {
    gt0 += *cluster.map_shared_rank(&sh.cta_gt, r);
    eq0 += *cluster.map_shared_rank(&sh.cta_eq, r);
  }
  cluster.sync();   // no CTA leaves while its shared memory is read
  for (int k = 0; k < warp; ++k) {
    gt0 += sh.warp_gt[k];
    eq0 += sh.warp_eq[k];
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i = a0; i < a1; i += 32) {
    const bool in = i + lane < a1;
    const uint32_t key = in ? order_key(__ldg(w + i + lane)) : 0u;
    const uint32_t mg = __ballot_sync(0xffffffffu, in && key > top);
    const uint32_t me = __ballot_sync(0xffffffffu, in && key == top);
    const uint32_t eq_rank = eq0 + __popc(me & below);
    if (in && (key > top || (key == top && eq_rank < ties)))
      index[gt0 + __popc(mg & below) + min(eq_rank, ties)] = i + lane;
    gt0 += __popc(mg);
    eq0 += __popc(me);
  }
  for (int i = rank * kSelThreads + tid; i < p.keep - need; i += kCluster * kSelThreads)
    index[need + i] = i < rec ? n + i : -1;
  if (rank == 0 && tid == 0 && bh % p.src.heads == 0) p.new_lengths[b] = kept;
}

// One warp per destination row of two tokens.
template <int D>
__global__ void __launch_bounds__(256) kv4_move_kernel(const EvictParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / p.src.heads;
  const int kept = min(min(max(__ldg(p.lengths + b), 0), p.src.cap), p.keep);
  const int pair = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (2 * pair >= kept) return;
  const bool two = 2 * pair + 1 < kept;
  const int32_t* index = p.index + (int64_t)bh * p.keep + 2 * pair;
  const int s0 = index[0], s1 = two ? index[1] : s0;
  const int64_t src = (int64_t)bh * p.src.cap, dst = (int64_t)bh * p.dst.cap + 2 * pair;
  constexpr int kRow = D / 8;     // words of a key row
  // keys: lanes [0, kRow) the first token, [kRow, 2 kRow) the second
  if (lane < (two ? 2 * kRow : kRow)) {
    const int64_t from = src + (lane < kRow ? s0 : s1);
    const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(p.src.kc + from * (D / 2)) + lane % kRow);
    (reinterpret_cast<uint32_t*>(p.dst.kc + dst * (D / 2)))[lane] = x;
  }
  // values: D bytes, a half from each source row
  if (lane < D / 4) {
    const uint32_t x0 = __ldg(reinterpret_cast<const uint32_t*>(p.src.vc + (src / 2 + s0 / 2) * D) + lane);
    const uint32_t x1 = __ldg(reinterpret_cast<const uint32_t*>(p.src.vc + (src / 2 + s1 / 2) * D) + lane);
    uint32_t* to = reinterpret_cast<uint32_t*>(p.dst.vc + dst / 2 * D) + lane;
    const uint32_t lo = (x0 >> (4 * (s0 & 1))) & 0x0f0f0f0fu, hi = (x1 >> (4 * (s1 & 1))) & 0x0f0f0f0fu;
    *to = lo | (two ? hi << 4 : *to & 0xf0f0f0f0u);
  }
  // scales and weights
  const int side = lane & 1, blk = lane >> 1;
  if (side == 0 || two) {
    const int s = side ? s1 : s0;
    if (blk < D / 16) {
      p.dst.ks[(dst + side) * (D / 16) + blk] = __ldg(p.src.ks + (src + s) * (D / 16) + blk);
      p.dst.vs[(dst / 2 * (D / 16) + blk) * 2 + side] = __ldg(p.src.vs + ((src / 2 + s / 2) * (D / 16) + blk) * 2 + (s & 1));
    }
    if (blk == 15) p.w_dst[dst + side] = __ldg(p.w_src + src + s);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  const int BH = p.src.batch * p.src.heads;
  kv4_select_kernel<<<dim3(kCluster, BH), kSelThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int most = std::min(p.keep, p.src.cap);
  cfg.gridDim = dim3((unsigned)(((most + 1) / 2 + 7) / 8), (unsigned)BH);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return p.src.dim == 128 ? cudaLaunchKernelEx(&cfg, kv4_move_kernel<128>, p)
                          : cudaLaunchKernelEx(&cfg, kv4_move_kernel<64>, p);
}

}  // namespace kv4
}  // namespace magi
