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
constexpr int kSelThreads = 512;
constexpr int kBins = 2048;

// Order-preserving integer of a weight.
__device__ __forceinline__ uint32_t order_key(float w) {
  w = w == w ? w + 0.f : -INFINITY;   // + 0: -0 is 0
  const uint32_t u = __float_as_uint(w);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

constexpr int kSelKeys = 40 * 1024;   // keys a CTA keeps; longer runs are read again each time

struct SelShared {
  uint32_t hist[kBins];      // this CTA's counts
  uint32_t total[3][kBins];  // the cluster's
  uint32_t scan[kSelThreads / 32];
  uint32_t warp_gt[kSelThreads / 32], warp_eq[kSelThreads / 32];
  uint32_t cta_gt, cta_eq;
  uint32_t bin, above;
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSelThreads) kv4_select_kernel(const EvictParams p, bool held) {
  extern __shared__ __align__(16) uint8_t sel_smem[];
  SelShared& sh = *reinterpret_cast<SelShared*>(sel_smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(sel_smem + sizeof(SelShared));
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
  if (held)
    for (int i = i0 + tid * 4; i < i1; i += kSelThreads * 4) {   // i0 and the row are multiples of 4 (or past n)
      const float4 x = __ldg(reinterpret_cast<const float4*>(w + i));
      *reinterpret_cast<uint4*>(keys + (i - i0)) = make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
    }
  auto key_at = [&](int i) { return held ? keys[i - i0] : order_key(__ldg(w + i)); };
  if (need > 0 && need < n) {                    // the same for the whole cluster
    uint32_t prefix = 0, left = (uint32_t)need;
    for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = sh.total[0][i] = sh.total[1][i] = sh.total[2][i] = 0;
    cluster.sync();
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
      for (int i = i0 + tid; i < i1; i += kSelThreads) {
        const uint32_t key = key_at(i);
        if (pass == 0 || (key >> (shift + bits)) == prefix) atomicAdd(&sh.hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      for (int i = tid; i < kBins; i += kSelThreads) {
        const uint32_t v = sh.hist[i];
        if (v == 0) continue;
        sh.hist[i] = 0;
        for (int r = 0; r < kCluster; ++r) atomicAdd(cluster.map_shared_rank(&sh.total[pass][i], r), v);
      }
      cluster.sync();
      // thread t holds the counts of bins 4t .. 4t+3 from the top
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
  } else {
    __syncthreads();
  }

  // number the kept tokens of this CTA's run, warp by warp
  const int wseg = ((i1 - i0) + kSelThreads - 1) / kSelThreads * 32;
  const int a0 = min(i0 + warp * wseg, i1), a1 = min(a0 + wseg, i1);
  uint32_t gt = 0, eq = 0;
  for (int i = a0; i < a1; i += 32) {
    const uint32_t key = i + lane < a1 ? key_at(i + lane) : 0u;
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
    const uint32_t key = in ? key_at(i + lane) : 0u;
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

// One warp per 16 destination tokens (8 value rows), so that each lane has some
// hundred bytes under way.
template <int D>
__global__ void __launch_bounds__(256) kv4_move_kernel(const EvictParams p) {
  constexpr int kTok = 16;
  constexpr int kK = D / 32;       // 16-byte pieces of a key row
  constexpr int kV = D / 16;       // 16-byte pieces of a value row (two tokens)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / p.src.heads;
  const int kept = min(min(max(__ldg(p.lengths + b), 0), p.src.cap), p.keep);
  const int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kTok;
  const int n = min(kTok, kept - t0);
  if (n <= 0) return;
  const int64_t src = (int64_t)bh * p.src.cap, dst = (int64_t)bh * p.dst.cap + t0;
  // lane t (and t + 16): where token t of the sixteen comes from
  const int from = p.index[(int64_t)bh * p.keep + t0 + min(lane & 15, n - 1)];   // not __ldg: written while this grid was starting
  uint4 k[kK * kTok / 32], va[kV * kTok / 64], vb[kV * kTok / 64];
#pragma unroll
  for (int i = 0; i < kK * kTok / 32; ++i) {
    const int piece = i * 32 + lane, t = piece / kK;
    const int s = __shfl_sync(0xffffffffu, from, t);
    k[i] = __ldg(reinterpret_cast<const uint4*>(p.src.kc + (src + s) * (D / 2)) + piece % kK);
  }
#pragma unroll
  for (int i = 0; i < kV * kTok / 64; ++i) {
    const int piece = i * 32 + lane, r = piece / kV;
    const int s0 = __shfl_sync(0xffffffffu, from, 2 * r), s1 = __shfl_sync(0xffffffffu, from, 2 * r + 1);
    va[i] = __ldg(reinterpret_cast<const uint4*>(p.src.vc + (src / 2 + s0 / 2) * D) + piece % kV);
    vb[i] = __ldg(reinterpret_cast<const uint4*>(p.src.vc + (src / 2 + s1 / 2) * D) + piece % kV);
  }
  // scales: lanes 0..15 a token's key and value scales each; lane t + 16 its weight
  uint2 ks = make_uint2(0, 0);
  uint4 vs = make_uint4(0, 0, 0, 0);
  float w = 0.f;
  if (lane < 16) {
    if constexpr (D == 128) {
      ks = __ldg(reinterpret_cast<const uint2*>(p.src.ks + (src + from) * 8));
      vs = __ldg(reinterpret_cast<const uint4*>(p.src.vs + (src / 2 + from / 2) * 16));
    } else {
      ks.x = __ldg(reinterpret_cast<const uint32_t*>(p.src.ks + (src + from) * 4));
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(p.src.vs + (src / 2 + from / 2) * 8));
      vs.x = y.x;
      vs.y = y.y;
    }
  } else {
    w = __ldg(p.w_src + src + from);
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
  const int seg = (p.src.cap + kCluster * 32 - 1) / (kCluster * 32) * 32;
  const int bytes = (int)sizeof(SelShared) + (seg <= kSelKeys ? seg * 4 : 0);
  static SmemRecord have;
  cudaError_t e = allow_smem(kv4_select_kernel, bytes, have);
  if (e != cudaSuccess) return e;
  kv4_select_kernel<<<dim3(kCluster, BH), kSelThreads, bytes, s>>>(p, seg <= kSelKeys);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int most = std::min(p.keep, p.src.cap);
  cfg.gridDim = dim3((unsigned)((most + 127) / 128), (unsigned)BH);
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
