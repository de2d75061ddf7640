// Eviction from the 4-bit cache by accumulated attention weight.
//
// Of the n tokens of a (batch element, head) the last `recent` stay, and of the
// others the `need` with the largest weight (equal weights: the lower index;
// NaN counts as -inf).  Order is kept.
//
// Selection (kv4_select_kernel).  A weight is mapped to an unsigned integer of
// the same order and the need-th largest is found digit by digit (12, 12 and 8
// bits), a histogram of the candidates with the digits so far at each.  A
// cluster of 8 CTAs shares a head: each keeps the keys of an eighth in shared
// memory and counts them there, by bin and by group of 64 bins.  One warp of
// each CTA then reads the eight CTAs' group counts through distributed shared
// memory, finds the group that holds the need-th, and in its 64 bins the bin.
// (Adding every count that is not zero to totals of all eight CTAs took up to
// 8300 cycles a digit: 66.7 us for 16 heads of 92160 against 60.3 in all, 10.8
// against 11.2 for 8 heads of 4097; sending the group counts instead of having
// them read 61.5 and 11.8.)
// The kept tokens are then numbered in their order: a warp takes a contiguous
// run and starts at the counts of the runs before it.
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
constexpr int kBins = 4096;         // of the first two digits
constexpr int kLastBins = 256;
constexpr int kGroup = 64, kGroups = kBins / kGroup;   // bins are counted by group too; two of each a lane

// Order-preserving integer of a weight.
__device__ __forceinline__ uint32_t order_key(float w) {
  w = w == w ? w + 0.f : -INFINITY;   // + 0: -0 is 0
  const uint32_t u = __float_as_uint(w);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 40 * 1024;   // keys a CTA keeps; longer runs are read again each time

struct SelShared {
  uint32_t hist[2 * kBins + kLastBins];   // this CTA's counts, each digit its own
  uint32_t group[3][kGroups];
  uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  uint32_t cta_gt, cta_eq;
  uint32_t bin, left;
};
static_assert(sizeof(SelShared) % 16 == 0, "the keys behind it are read 16 bytes at a time");

// Of 64 counts (two a lane, `at` summed over the cluster's CTAs) the one, from
// the top, in which the left-th lies; left becomes its place in there.
__device__ __forceinline__ uint32_t pick(cg::cluster_group& cluster, uint32_t* at, uint32_t& left) {
  const int lane = threadIdx.x & 31;
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int r = 0; r < kCluster; ++r) {
    const uint2 v = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(at, r) + 62 - 2 * lane);
    lo += v.x;
    hi += v.y;
  }
  uint32_t incl = lo + hi;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const uint32_t before = incl - lo - hi;
  const int at_lane = __ffs(__ballot_sync(0xffffffffu, incl >= left)) - 1;   // (the counts' sum is at least left)
  const bool in_hi = before + hi >= left;
  const uint32_t bin = in_hi ? 63 - 2 * lane : 62 - 2 * lane, place = left - before - (in_hi ? 0u : hi);
  left = __shfl_sync(0xffffffffu, place, at_lane);
  return __shfl_sync(0xffffffffu, bin, at_lane);
}

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
  for (int i = tid; i < (int)(sizeof(sh.hist) / 16); i += kSelThreads)
    reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
  if (tid < 3 * kGroups) (&sh.group[0][0])[tid] = 0;
  __syncthreads();
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
  auto four = [&](int o) {
    if (o >= len_w) return make_uint4(0, 0, 0, 0);
    return held ? *reinterpret_cast<const uint4*>(keys + o) : from_row(o);
  };
  const bool search = need > 0 && need < n;      // the same for the whole cluster
  auto count = [&](uint32_t key, int shift, uint32_t mask, uint32_t* hist) {
    if (key != 0) atomicAdd(hist + ((key >> shift) & mask), 1u);
  };

  // keys into shared memory and the first digit's counts, four loads under way a lane
  if (held || search)
    for (int o0 = lane * 4; o0 < len_w; o0 += 512) {
      uint4 k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        k[j] = o0 + 128 * j < len_w ? from_row(o0 + 128 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (o0 + 128 * j >= len_w) continue;
        if (held) *reinterpret_cast<uint4*>(keys + o0 + 128 * j) = k[j];
        if (search) {
          count(k[j].x, 20, kBins - 1, sh.hist);
          count(k[j].y, 20, kBins - 1, sh.hist);
          count(k[j].z, 20, kBins - 1, sh.hist);
          count(k[j].w, 20, kBins - 1, sh.hist);
        }
      }
    }

  // the need-th largest key and how many of those equal to it stay
  uint32_t top = need == 0 ? 0xffffffffu : 0u;   // all stay: every key is above
  uint32_t ties = 0;
  if (search) {
    uint32_t prefix = 0, left = (uint32_t)need;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 20 : pass == 1 ? 8 : 0;
      const int bits = pass == 2 ? 8 : 12;
      uint32_t* hist = sh.hist + pass * kBins;
      if (pass > 0) {
        auto of_prefix = [&](uint32_t key) {
          if ((key >> (shift + bits)) == prefix) count(key, shift, (1u << bits) - 1u, hist);
        };
        for (int o = lane * 4; o < len_w; o += 128) {
          const uint4 k = four(o);
          of_prefix(k.x);
          of_prefix(k.y);
          of_prefix(k.z);
          of_prefix(k.w);
        }
      }
      __syncthreads();
      if (tid < (1 << bits) / 4) {   // whole warps; 16 lanes a group
        const uint4 v = reinterpret_cast<const uint4*>(hist)[tid];
        uint32_t sum = v.x + v.y + v.z + v.w;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane % 16 == 0) sh.group[pass][tid / 16] = sum;
      }
      cluster.sync();
      if (warp == 0) {
        const uint32_t g = pick(cluster, sh.group[pass], left);
        const uint32_t in_group = pick(cluster, hist + g * kGroup, left);
        if (lane == 0) {
          sh.bin = g * kGroup + in_group;
          sh.left = left;
        }
      }
      __syncthreads();
      prefix = (prefix << bits) | sh.bin;
      left = sh.left;
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
  for (int o0 = 0; o0 < len_w; o0 += 128) {
    const int o = o0 + lane * 4;
    const uint4 k4 = four(o);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    uint32_t mine = 0;   // above the threshold, and equal to it in the upper half
#pragma unroll
    for (int c = 0; c < 4; ++c) mine += (k[c] > top ? 1u : 0u) + (k[c] == top ? 0x10000u : 0u);
    uint32_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += x;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
    uint32_t g = gt0 + ((incl - mine) & 0xffffu), e = eq0 + ((incl - mine) >> 16);   // before this lane's first
    gt0 += all & 0xffffu;
    eq0 += all >> 16;
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
