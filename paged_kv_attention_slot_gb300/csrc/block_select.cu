// The pages of every (token, KV head) that decode attention reads (pkv_block_select).
//
// For a request with one new token and N pages, and KV head h, of which the first S and the last R stay: the m = K - S - R
// others with the largest score (equal scores: the lower page),
//   score_b = sum_d w+_d hi_bd + w-_d lo_bd,   w+-_d = sum over the query heads g of h of max / min(c_gd, 0),
//   c_gd = rint(fl(fl(a_gd / M) T)),  a_gd = fl(q_gd scale_hd),  M = max |a_gd|,  T = floor(32767 / G),
// an upper bound of sum_g q_g.k over the page's keys, up to the codes' rounding.  Everything from c_gd on is whole numbers
// that 32 bits hold (2 D terms below 2^15 2^7), so neither the order of a sum nor the split of the work moves a page
// across the border, and a border is where the definition puts it.
//
// What bounds it: reading 2 D bytes of bounds per page, and the latency of the steps behind (a selection from
// numbers that a few thousand threads hold).  One launch: a cluster of C CTAs per (request, KV head) scores its pages in
// C slices, 8 lanes to a page (head_dim 128) by two-way 16 x 8 bit dot products; the scores go to the first
// CTA's shared memory, which selects: a radix select on the scores less their smallest, by the digits that their
// range has, then ballots and prefix counts that list the survivors in order.

#include <cooperative_groups.h>

#include <algorithm>

#include "decode_blocks.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBinBits = 11;
constexpr int kBins = 1 << kBinBits;
constexpr int kSelectMaxCluster = 8;

struct SelectShared {
  uint32_t hist[kBins];
  int32_t w[2][2][128];  // [half of the threads][lower, upper][channel]: whole-number weights
  float warp_max[kWarps];
  uint32_t warp_lo[kWarps], warp_hi[kWarps];
  uint64_t warp_sum[kWarps];
  uint32_t digit, rest, count;  // of the radix pass: the digit found, the keys to take inside it, its keys
};

// exclusive prefix over the block's threads of v, and the block's total
template <typename V>
__device__ __forceinline__ V block_prefix(V v, uint64_t* warp_sum, V& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();  // the previous use of warp_sum is over
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  V before = 0;
  total = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const V s = (V)warp_sum[k];
    before += k < warp ? s : (V)0;
    total += s;
  }
  return before + inc - v;
}

template <int D>
__global__ void __launch_bounds__(kThreads) block_select_kernel(const SelectParams p) {
  constexpr int LANES = D / 16;      // per page: 16 bytes of the lower and of the upper bounds each
  constexpr int PAGES = 32 / LANES;  // per warp-wide load
  constexpr int UNROLL = 4;          // such loads in flight
  constexpr int PARTS = kThreads / D;
  constexpr int HELD = 8;  // query values a thread keeps between the two looks at them
  extern __shared__ __align__(16) uint8_t smem[];
  SelectShared& sh = *reinterpret_cast<SelectShared*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(SelectShared));  // [body pages, rounded up to 32]
  uint32_t* gtw = keys + p.key_cap;                                           // a bit per key: above the threshold
  uint32_t* eqw = gtw + p.key_cap / 32;                                       // at the threshold

  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int unit = blockIdx.x / C;
  const int i = unit / p.num_kv_heads, h = unit - i * p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  pdl_wait();
  pdl_launch_dependents();
  const int4 rq = __ldg(reinterpret_cast<const int4*>(p.req + i));  // page_base, kv_len, q_begin, q_len
  if (rq.w == 0) return;  // (the whole cluster)
  const int N = (int)p.by_page.div((uint32_t)rq.y + (uint32_t)p.page_size - 1u);
  const int K = p.num_blocks, S = p.num_sink, R = p.num_recent;
  int32_t* out = p.blocks + ((int64_t)rq.z * p.num_kv_heads + h) * K;
  const int m = K - S - R;  // pages to find
  if (N <= K || m == 0) {   // (the whole cluster) nothing competes
    if (rank == 0)
      for (int j = tid; j < K; j += kThreads) out[j] = N <= K ? (j < N ? j : -1) : (j < S ? j : N - K + j);
    return;
  }
  const int nb = N - S - R;  // competing pages S .. N - R - 1
  if (C > 1) cluster.barrier_arrive();  // (every CTA of the cluster runs before its memory is written to)

  // ---- whole-number weights ----
  const int G = p.group;
  const int d = tid % D, part = tid / D;
  const float scale = __ldg(p.scale + h * D + d);
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + ((int64_t)rq.z * p.num_kv_heads + h) * G * D + d;
  auto value = [&](int g) -> float {
    const float a = __uint_as_float((uint32_t)__ldg(q + g * D) << 16) * scale;
    return fabsf(a) <= 3.402823466e38f ? a : 0.f;  // an infinity or a NaN counts as 0
  };
  float held[HELD], top = 0.f;
#pragma unroll
  for (int r = 0; r < HELD; ++r) {
    const int g = part + r * PARTS;
    held[r] = g < G ? value(g) : 0.f;
    top = fmaxf(top, fabsf(held[r]));
  }
  for (int g = part + HELD * PARTS; g < G; g += PARTS) top = fmaxf(top, fabsf(value(g)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) sh.warp_max[warp] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sh.warp_max[k]);
  const float T = (float)(32767 / G);
  int32_t neg = 0, pos = 0;
  auto add = [&](float a) {
    const int c = __float2int_rn(__fmul_rn(__fdiv_rn(a, top), T));
    neg += min(c, 0);
    pos += max(c, 0);
  };
  if (top > 0.f) {
#pragma unroll
    for (int r = 0; r < HELD; ++r)
      if (part + r * PARTS < G) add(held[r]);
    for (int g = part + HELD * PARTS; g < G; g += PARTS) add(value(g));
  }
  // (head_dim 64 has four parts: two of them to a half, one after the other)
  if (part < 2) {
    sh.w[part][0][d] = neg;
    sh.w[part][1][d] = pos;
  }
  __syncthreads();
  if constexpr (PARTS > 2) {
    if (part >= 2) {
      sh.w[part - 2][0][d] += neg;
      sh.w[part - 2][1][d] += pos;
    }
    __syncthreads();
  }
  // this lane's weights, two to a word: channels 16 lc .. 16 lc + 15 of the lower and of the upper bounds
  const int lc = lane % LANES, lp = lane / LANES;
  uint32_t w[2][8];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = 16 * lc + 2 * j;
      const int a = sh.w[0][s][at] + sh.w[1][s][at], b = sh.w[0][s][at + 1] + sh.w[1][s][at + 1];
      w[s][j] = ((uint32_t)a & 0xffffu) | ((uint32_t)b << 16);
    }

  // ---- scores of this CTA's slice ----
  if (C > 1) cluster.barrier_wait();
  uint32_t* to = C > 1 ? cluster.map_shared_rank(keys, 0) : keys;
  const int slice = ((nb + C - 1) / C + 31) / 32 * 32;
  const int lo = rank * slice, hi = min(nb, lo + slice);
  const int32_t* pages = p.kv_indices + rq.x + S;
  for (int b0 = lo + warp * PAGES; b0 < hi; b0 += kWarps * PAGES * UNROLL) {
    int page[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) page[u] = __ldg(pages + min(b0 + u * kWarps * PAGES + lp, hi - 1));
    uint4 x[UNROLL][2];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const uint4* at = reinterpret_cast<const uint4*>(p.codes + ((int64_t)page[u] * p.num_kv_heads + h) * (2 * D)) + lc;
      x[u][0] = __ldg(at);
      x[u][1] = __ldg(at + LANES);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      int acc = 0;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t b[4] = {x[u][s].x, x[u][s].y, x[u][s].z, x[u][s].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc = __dp2a_lo((int)w[s][2 * j], (int)b[j], acc);
          acc = __dp2a_hi((int)w[s][2 * j + 1], (int)b[j], acc);
        }
      }
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      const int b = b0 + u * kWarps * PAGES + lp;
      if (lc == 0 && b < hi) to[b] = (uint32_t)acc ^ 0x80000000u;
    }
  }
  if (C > 1) {
    cluster.sync();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  // ---- the m largest of nb keys ----
  uint32_t least = 0xffffffffu, most = 0u;
  for (int b = tid; b < nb; b += kThreads) {
    least = min(least, keys[b]);
    most = max(most, keys[b]);
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    sh.warp_lo[warp] = least;
    sh.warp_hi[warp] = most;
  }
  for (int k = tid; k < kBins; k += kThreads) sh.hist[k] = 0u;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    least = min(least, sh.warp_lo[k]);
    most = max(most, sh.warp_hi[k]);
  }
  // digits from the top of the range; `found`: the threshold's digits so far, keys >> shift compare with it
  int bits = 32 - __clz((int)(most - least));
  int shift = max(0, bits - kBinBits);
  uint32_t found = 0, rest = (uint32_t)m, count = 0;
  int above = 32;  // keys whose digits above bit `above` equal found's compete (all of them in the first pass)
  while (true) {
    for (int b = tid; b < nb; b += kThreads) {
      const uint32_t k = keys[b] - least;
      if (above == 32 || k >> above == found) atomicAdd(&sh.hist[(k >> shift) & (kBins - 1)], 1u);
    }
    __syncthreads();
    // the digit at which the count from the top reaches `rest`: each thread sums its bins from the top
    constexpr int PER = kBins / kThreads;
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) mine += sh.hist[kBins - 1 - (tid * PER + k)];
    uint32_t total;
    uint32_t before = block_prefix<uint32_t>(mine, sh.warp_sum, total);
    if (before < rest && before + mine >= rest) {
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const uint32_t n = sh.hist[kBins - 1 - (tid * PER + k)];
        if (before < rest && before + n >= rest) {
          sh.digit = (uint32_t)(kBins - 1 - (tid * PER + k));
          sh.rest = rest - before;
          sh.count = n;
        }
        before += n;
      }
    }
    __syncthreads();
    const int width = min(kBinBits, above - shift);
    found = above == 32 ? sh.digit : (found << width) | (sh.digit & ((1u << width) - 1u));
    rest = sh.rest;
    count = sh.count;
    if (rest == count || shift == 0) break;  // all of the digit's keys stay, or they are equal
    above = shift;
    shift = max(0, shift - kBinBits);
    for (int k = tid; k < kBins; k += kThreads) sh.hist[k] = 0u;
    __syncthreads();
  }

  // ---- the survivors, in order ----
  const int words = (nb + 31) / 32;
  for (int wd = warp; wd < words; wd += kWarps) {
    const int b = wd * 32 + lane;
    const uint32_t k = b < nb ? (keys[b] - least) >> shift : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, b < nb && k > found);
    const uint32_t eq = __ballot_sync(0xffffffffu, b < nb && k == found);
    if (lane == 0) {
      gtw[wd] = gt;
      eqw[wd] = eq;
    }
  }
  __syncthreads();
  // counts before each word: above the threshold (high half) and at it (low half), a thread per run of words
  const int run = (words + kThreads - 1) / kThreads;
  uint64_t mine = 0;
  for (int k = 0; k < run; ++k) {
    const int wd = tid * run + k;
    if (wd < words) mine += ((uint64_t)__popc(gtw[wd]) << 32) | (uint32_t)__popc(eqw[wd]);
  }
  uint64_t total;
  uint64_t before = block_prefix<uint64_t>(mine, sh.warp_sum, total);
  for (int k = 0; k < run; ++k) {
    const int wd = tid * run + k;
    if (wd >= words) break;
    const uint32_t gt = gtw[wd], eq = eqw[wd];
    uint32_t ties = (uint32_t)before;  // keys at the threshold before this word: the first `rest` of them stay
    uint32_t at = (uint32_t)(before >> 32) + min(ties, rest);
    for (uint32_t live = gt | eq; live; live &= live - 1u) {
      const int bit = __ffs(live) - 1;
      if (!(gt >> bit & 1u) && ties++ >= rest) continue;
      out[S + at++] = S + wd * 32 + bit;
    }
    before += ((uint64_t)__popc(gt) << 32) | (uint32_t)__popc(eq);
  }
  for (int j = tid; j < S; j += kThreads) out[j] = j;
  for (int j = tid; j < R; j += kThreads) out[K - R + j] = N - R + j;
}

template <int D>
cudaError_t launch_form(const SelectParams& p, int64_t units, int C, cudaStream_t s) {
  if (units * C > INT32_MAX) return cudaErrorInvalidValue;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(block_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(SelectShared) + (size_t)p.key_cap * 4 + (size_t)p.key_cap / 32 * 8;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, block_select_kernel<D>, p);
}

static_assert(sizeof(SelectShared) + (size_t)kSelectMaxBlocks * 4 + (size_t)kSelectMaxBlocks / 32 * 8 <= 232448,
              "the scores of the longest request fit the shared memory of one CTA");

}  // namespace

cudaError_t launch_block_select(SelectParams p, int32_t batch, int32_t max_blocks, int num_sms, cudaStream_t s) {
  const int64_t units = (int64_t)batch * p.num_kv_heads;
  const int32_t most = std::max(1, max_blocks - p.num_sink - p.num_recent);
  p.key_cap = (most + 31) / 32 * 32;
  p.by_page = divider(p.page_size);
  // clusters while their CTAs all run at once and a slice keeps a load per warp in flight
  int C = 1;
  while (C < kSelectMaxCluster && units * C * 2 <= 2 * (int64_t)num_sms && most / (2 * C) >= 128) C *= 2;
  return p.head_dim == 128 ? launch_form<128>(p, units, C, s) : launch_form<64>(p, units, C, s);
}

}  // namespace pkv
