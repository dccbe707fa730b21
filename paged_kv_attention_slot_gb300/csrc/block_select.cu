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
// What bounds it: reading 2 D bytes of bounds per page, and the latency of the steps before and behind.  One launch,
// a unit per (request, KV head), in one of two forms:
//   * narrow: a CTA of 256 threads per unit, four to an SM.  64 x 8 units of up to 256 pages (17.8 MB): 7.4 us, of which
//     reading takes 2.8 at the measured copy rate; the rest is the way to the first bounds (request, page ids: 0.6 us), the
//     weights (1.4), the selection (1.8) and the launch;
//   * wide, for few units of many pages: a cluster of C CTAs of 512 threads scores its pages in C slices; the scores go to
//     the first CTA's shared memory, which selects.  2 x 8 units of 8192 pages (33.5 MB): 14.3 us, 5.1 at the copy rate; the
//     slices stream for 7.9 us (16 clusters of 6: 96 SMs; of 7 or 8 no 16 run at once, and half-size CTAs in clusters
//     of 12 to 16 take 15.5), the selection behind them takes 3.7.
// A page takes 8 lanes (head_dim 128): two 16-byte loads each, past L1 (0.2 us of the 14.3), 16 two-way 16 x 8 bit dot
// products, three shuffles.  Loads through a ring in shared memory instead of registers: 15.5 us (4 to 8 in flight), 17.7 (12).
// The selection is a radix select on the scores less their smallest, cut by the digits that their range has (a range
// known before the scores, from the weights, is too coarse: 18.0 us); once a digit holds at most 256 keys they are
// compared with each other; then ballots and prefix counts list the survivors in order.

#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "decode_blocks.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pkv {

int32_t* device_error_ptr();

namespace {

constexpr int kSelectMaxCluster = 8;
constexpr int kFewPages = 768;     // competing pages that the narrow form takes in any case
constexpr int kCandidates = 256;   // keys of one digit that are compared with each other

// WIDE: a cluster of CTAs that have an SM each, for few units of many pages; narrow: a CTA of four on an SM.
// UNROLL: warp-wide loads in flight (of two vectors a lane each).
template <bool WIDE>
struct Form {
  static constexpr int THREADS = WIDE ? 512 : 256;
  static constexpr int WARPS = THREADS / 32;
  static constexpr int CTAS = WIDE ? 1 : 4;
  static constexpr int UNROLL = WIDE ? 8 : 2;
  static constexpr int BIN_BITS = WIDE ? 11 : 8;
  static constexpr int BINS = 1 << BIN_BITS;
  struct alignas(16) Shared {  // (packed and hist are read 16 bytes at a time)
    int32_t w[2][2][128];   // [half of the threads][lower, upper][channel]: whole-number weights
    alignas(16) uint32_t packed[2][2][8][4];  // [lower, upper][half of 16 channels][16 channels][pair]: two 16-bit weights to a word
    float warp_max[WARPS];
    uint32_t warp_sum[WARPS];
    uint32_t digit, rest, count;  // of the radix pass: the digit found, the keys to take inside it, its keys
    uint32_t candidates;
    uint32_t least, most;         // of the keys
    alignas(16) uint32_t hist[BINS];          // keys of each digit, the largest digit first
    alignas(16) uint2 candidate[kCandidates];  // (key, place)
  };
};

// exclusive prefix over the block's threads of v
template <int WARPS>
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();  // the previous use of warp_sum is over
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int k = 0; k < WARPS; ++k) {
    const uint32_t s = warp_sum[k];
    before += k < warp ? s : 0u;
  }
  return before + inc - v;
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(Form<WIDE>::THREADS, Form<WIDE>::CTAS) block_select_kernel(const SelectParams p) {
  using F = Form<WIDE>;
  constexpr int THREADS = F::THREADS, WARPS = F::WARPS, UNROLL = F::UNROLL;
  constexpr int LANES = D / 16;          // per page: 16 bytes of the lower and of the upper bounds each
  constexpr int PAGES = 32 / LANES;      // per warp-wide load
  constexpr int STEP = WARPS * PAGES;    // pages between the loads of one thread
  constexpr int PARTS = THREADS / D;     // threads per channel
  constexpr int BINS = F::BINS, BIN_BITS = F::BIN_BITS;
  constexpr int READ = WIDE ? 8 : 2;     // keys that a thread reads at once
  constexpr int HELD = 4;                // query values a thread keeps between the two looks at them
  extern __shared__ __align__(16) uint8_t smem[];
  typename F::Shared& sh = *reinterpret_cast<typename F::Shared*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(typename F::Shared));  // [competing pages, rounded up to 32]
  uint32_t* lives = keys + p.key_cap;  // a bit per key: it stays

  cg::cluster_group cluster = cg::this_cluster();
  const int C = WIDE ? (int)cluster.num_blocks() : 1, rank = WIDE ? (int)cluster.block_rank() : 0;
  const int unit = blockIdx.x / C;
  const int i = unit / p.num_kv_heads, h = unit - i * p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  pdl_wait();
  pdl_launch_dependents();
  const int4 rq = __ldg(reinterpret_cast<const int4*>(p.req + i));  // page_base, kv_len, q_begin, q_len
  // (a captured call's plan may have been made anew over pages that the bounds do not have: they count as the last one.
  // A flag from where the pages are read cost 0.3 us; one read beside the request's costs nothing)
  if (blockIdx.x == 0 && tid == 0 && __ldg(p.max_page) > (int)p.last_page) record_error(p.err, PKV_DEVERR_PAGE_RANGE);
  if (rq.w == 0) return;  // (the whole cluster)
  const int N = (int)p.by_page.div((uint32_t)rq.y + (uint32_t)p.page_size - 1u);
  const int K = p.num_blocks, S = p.num_sink, R = p.num_recent;
  int32_t* out = p.blocks + ((int64_t)rq.z * p.num_kv_heads + h) * K;
  const int m = K - S - R;  // pages to find
  const int nb = N - S - R;  // competing pages S .. N - R - 1
  if (N <= K || m == 0 || nb > p.key_cap) {  // (the whole cluster) nothing competes; or a captured call's plan was made anew
    if (rank == 0) {                         // for longer requests than it has room for
      const bool fits = N <= K || m == 0;
      if (!fits && tid == 0) record_error(p.err, PKV_DEVERR_CAPACITY);
      for (int j = tid; j < K; j += THREADS) out[j] = !fits ? -1 : N <= K ? (j < N ? j : -1) : (j < S ? j : N - K + j);
    }
    return;
  }
  if (rank == 0) {
    for (int k = tid; k < BINS; k += THREADS) sh.hist[k] = 0u;
    if (tid == 0) {
      sh.candidates = 0u;
      sh.least = 0xffffffffu;
      sh.most = 0u;
    }
  }
  if (C > 1) cluster.barrier_arrive();  // (every CTA of the cluster runs, and rank 0 is ready, before its memory is written to)

  // ---- the first bounds of this CTA's slice are on their way while the weights are formed ----
  const int slice = C > 1 ? ((nb + C - 1) / C + 31) / 32 * 32 : nb;
  const int lo = rank * slice, hi = min(nb, lo + slice);
  const int lc = lane % LANES, lp = lane / LANES;
  const int32_t* pages = p.kv_indices + rq.x + S;
  const int8_t* codes = p.codes + (int64_t)h * (2 * D) + lc * 16;
  const int64_t page_bytes = (int64_t)p.num_kv_heads * (2 * D);
  int b0 = lo + warp * PAGES + lp;  // this lane's first page
  int page[UNROLL];
  uint4 x[UNROLL][2];
  auto fetch_pages = [&](int b) {
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      page[u] = b + u * STEP < hi ? __ldg(pages + b + u * STEP) : 0;
      page[u] = (int)min((uint32_t)page[u], p.last_page);
    }
  };
  auto fetch_bounds = [&](int b) {
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      x[u][0] = x[u][1] = make_uint4(0u, 0u, 0u, 0u);
      if (b + u * STEP < hi) {
        const uint4* at = reinterpret_cast<const uint4*>(codes + page[u] * page_bytes);
        x[u][0] = ldg_once(at);
        x[u][1] = ldg_once(at + LANES);
      }
    }
  };
  fetch_pages(b0);

  // ---- whole-number weights ----
  const int G = p.group;
  const int d = tid % D, part = tid / D;
  const float scale = __ldg(p.scale + h * D + d);
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + ((int64_t)rq.z * p.num_kv_heads + h) * G * D + d;
  auto value = [&](uint16_t bits) -> float {
    const float a = __uint_as_float((uint32_t)bits << 16) * scale;
    return fabsf(a) <= 3.402823466e38f ? a : 0.f;  // an infinity or a NaN counts as 0
  };
  uint16_t held[HELD];
#pragma unroll
  for (int r = 0; r < HELD; ++r) held[r] = part + r * PARTS < G ? __ldg(q + (part + r * PARTS) * D) : (uint16_t)0;
  fetch_bounds(b0);
  float top = 0.f;
#pragma unroll
  for (int r = 0; r < HELD; ++r) top = fmaxf(top, fabsf(value(held[r])));
  for (int g = part + HELD * PARTS; g < G; g += PARTS) top = fmaxf(top, fabsf(value(__ldg(q + g * D))));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) sh.warp_max[warp] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < WARPS; ++k) top = fmaxf(top, sh.warp_max[k]);
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
      if (part + r * PARTS < G) add(value(held[r]));
    for (int g = part + HELD * PARTS; g < G; g += PARTS) add(value(__ldg(q + g * D)));
  }
  // two parts at a time (sums of whole numbers: in any order)
#pragma unroll
  for (int k = 0; k < PARTS; k += 2) {
    if ((part & ~1) == k) {
      int32_t(&w)[2][128] = sh.w[part & 1];
      w[0][d] = k ? w[0][d] + neg : neg;
      w[1][d] = k ? w[1][d] + pos : pos;
    }
    __syncthreads();
  }
  if (tid < D) {
    const int s = tid / (D / 2), c = tid % (D / 2) * 2;  // channels c, c + 1 of the lower or of the upper bounds
    const int a = sh.w[0][s][c] + sh.w[1][s][c], b = sh.w[0][s][c + 1] + sh.w[1][s][c + 1];
    sh.packed[s][c >> 3 & 1][c >> 4][c >> 1 & 3] = ((uint32_t)a & 0xffffu) | ((uint32_t)b << 16);
  }
  __syncthreads();
  // this lane's weights: channels 16 lc .. 16 lc + 15
  uint32_t w[2][8];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 x4 = *reinterpret_cast<const uint4*>(sh.packed[s][j][lc]);
      w[s][4 * j] = x4.x, w[s][4 * j + 1] = x4.y, w[s][4 * j + 2] = x4.z, w[s][4 * j + 3] = x4.w;
    }

  // ---- scores of the slice, to the first CTA ----
  if (C > 1) cluster.barrier_wait();
  uint32_t* to = C > 1 ? cluster.map_shared_rank(keys, 0) : keys;
  uint32_t least = 0xffffffffu, most = 0u;
  for (; b0 - lp < hi; b0 += UNROLL * STEP) {  // warp-uniform
    fetch_pages(b0 + UNROLL * STEP);
    uint32_t key[UNROLL];
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
      key[u] = (uint32_t)acc;
    }
    fetch_bounds(b0 + UNROLL * STEP);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
#pragma unroll
      for (int o = 1; o < LANES; o <<= 1) key[u] += __shfl_xor_sync(0xffffffffu, key[u], o);
      key[u] ^= 0x80000000u;  // in the order of the scores
      if (b0 + u * STEP < hi) {
        if (lc == 0) to[b0 + u * STEP] = key[u];
        least = min(least, key[u]);
        most = max(most, key[u]);
      }
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0 && least <= most) {
    atomicMin(C > 1 ? cluster.map_shared_rank(&sh.least, 0) : &sh.least, least);
    atomicMax(C > 1 ? cluster.map_shared_rank(&sh.most, 0) : &sh.most, most);
  }
  if (C > 1) {
    cluster.sync();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  // ---- the m largest of nb keys, equal ones from the front ----
  // Keys (less the least of them) whose digits from bit `shift` on are above `found` stay, and `rest` of the `count` at it.
  const int words = (nb + 31) / 32;
  uint32_t rest = (uint32_t)m, count = 0, found = 0;
  least = sh.least;
  int shift = max(0, 32 - __clz((int)(sh.most - least)) - BIN_BITS);
  int above = 32;  // keys whose digits from bit `above` on equal `found` compete (all of them in the first pass)
  while (true) {
    for (int b = tid; b < nb; b += READ * THREADS) {
      uint32_t k[READ];
#pragma unroll
      for (int r = 0; r < READ; ++r) k[r] = keys[min(b + r * THREADS, nb - 1)] - least;
#pragma unroll
      for (int r = 0; r < READ; ++r)
        if (b + r * THREADS < nb && (above == 32 || k[r] >> above == found))
          atomicAdd(&sh.hist[BINS - 1 - ((k[r] >> shift) & (BINS - 1))], 1u);
    }
    __syncthreads();
    // the digit at which the count from the top reaches `rest`
    constexpr int PER = BINS / THREADS;
    static_assert(PER == 1 || PER == 4, "one load per thread");
    uint32_t n[PER], mine = 0;
    if constexpr (PER == 4) {
      const uint4 x4 = *reinterpret_cast<const uint4*>(&sh.hist[4 * tid]);
      n[0] = x4.x, n[1] = x4.y, n[2] = x4.z, n[3] = x4.w;
    } else {
      n[0] = sh.hist[tid];
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) mine += n[k];
    uint32_t before = block_prefix<WARPS>(mine, sh.warp_sum);
    if (before < rest && before + mine >= rest) {
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        if (before < rest && before + n[k] >= rest) {
          sh.digit = (uint32_t)(BINS - 1 - (tid * PER + k));
          sh.rest = rest - before;
          sh.count = n[k];
        }
        before += n[k];
      }
    }
    __syncthreads();
    const int width = min(BIN_BITS, above - shift);
    found = above == 32 ? sh.digit : (found << width) | (sh.digit & ((1u << width) - 1u));
    rest = sh.rest;
    count = sh.count;
    if (rest == count || shift == 0 || count <= kCandidates) break;
    above = shift;
    shift = max(0, shift - BIN_BITS);
    for (int k = tid; k < BINS; k += THREADS) sh.hist[k] = 0u;
    __syncthreads();
  }
  const bool all = rest == count;                    // of the digit's keys
  const bool few = !all && count <= kCandidates;     // each is compared with all
  if (all || few) {
    const uint32_t stays = found + (all ? 0u : 1u);  // the lowest digit whose keys all do
    for (int w0 = warp; w0 < words; w0 += READ * WARPS) {
      uint32_t k[READ];
#pragma unroll
      for (int r = 0; r < READ; ++r) k[r] = keys[min((w0 + r * WARPS) * 32 + lane, nb - 1)] - least;
      uint32_t here = 0;  // a bit per key that is a candidate
#pragma unroll
      for (int r = 0; r < READ; ++r) {
        const int wd = w0 + r * WARPS;
        const bool in = wd * 32 + lane < nb;
        const uint32_t live = __ballot_sync(0xffffffffu, in && k[r] >> shift >= stays);
        if (lane == 0 && wd < words) lives[wd] = live;
        here |= (uint32_t)(few && in && k[r] >> shift == found) << r;
      }
      if (here) {
#pragma unroll
        for (int r = 0; r < READ; ++r)
          if (here >> r & 1u)
            sh.candidate[atomicAdd(&sh.candidates, 1u)] = make_uint2(k[r], (uint32_t)((w0 + r * WARPS) * 32 + lane));
      }
    }
    __syncthreads();
    if (few && tid < (int)count) {
      const uint2 own = sh.candidate[tid];
      uint32_t ahead = 0;
#pragma unroll 4
      for (uint32_t j = 0; j < count; ++j) {
        const uint2 c = sh.candidate[j];
        ahead += c.x > own.x || (c.x == own.x && c.y < own.y);
      }
      if (ahead < rest) atomicOr(&lives[own.y >> 5], 1u << (own.y & 31u));
    }
  } else if (warp == 0) {  // many equal keys: the first `rest` of them, counted by one warp (2 x 8 units of 8192 equal scores
                           // 30 us, unequal ones 14.3; 8 units of 49152: 150 and 60)
    for (int wd = 0; wd < words; ++wd) {
      const int b = wd * 32 + lane;
      const uint32_t k = b < nb ? keys[b] - least : 0u;  // (shift is 0)
      const uint32_t equal = __ballot_sync(0xffffffffu, b < nb && k == found);
      const bool first = __popc(equal & ((1u << lane) - 1u)) < rest;
      const uint32_t live = __ballot_sync(0xffffffffu, b < nb && (k > found || (k == found && first)));
      if (lane == 0) lives[wd] = live;
      rest -= min(rest, (uint32_t)__popc(equal));
    }
  }
  __syncthreads();

  // ---- the survivors, in order ----
  const int run = (words + WARPS - 1) / WARPS, first_word = warp * run, last_word = min(words, first_word + run);
  // a warp's survivors, and those before it
  uint32_t mine = 0;
  for (int wd = first_word + lane; wd < last_word; wd += 32) mine += __popc(lives[wd]);
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) sh.warp_sum[warp] = mine;
  __syncthreads();
  uint32_t at = S;
#pragma unroll
  for (int k = 0; k < WARPS; ++k) at += k < warp ? sh.warp_sum[k] : 0u;
  if (run < 8) {  // few words: a lane per bit
    for (int wd = first_word; wd < last_word; ++wd) {
      const uint32_t live = lives[wd];
      if (live >> lane & 1u) out[at + __popc(live & ((1u << lane) - 1u))] = S + wd * 32 + lane;
      at += __popc(live);
    }
  } else {  // a lane per word
    for (int w0 = first_word; w0 < last_word; w0 += 32) {
      const int wd = w0 + lane;
      uint32_t live = wd < last_word ? lives[wd] : 0u, inc = __popc(live);
      const uint32_t n = inc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      uint32_t to_at = at + inc - n;
      at += __shfl_sync(0xffffffffu, inc, 31);
      for (; live; live &= live - 1u) out[to_at++] = S + wd * 32 + __ffs(live) - 1;
    }
  }
  for (int j = tid; j < S; j += THREADS) out[j] = j;
  for (int j = tid; j < R; j += THREADS) out[K - R + j] = N - R + j;
}

template <int D, bool WIDE>
cudaError_t allow_shared_memory(int dev) {
  static bool done[64] = {false};
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(block_select_kernel<D, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

template <int D, bool WIDE>
void configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], const SelectParams& p, int64_t ctas, int C, cudaStream_t s) {
  cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(Form<WIDE>::THREADS);
  cfg.dynamicSmemBytes = sizeof(typename Form<WIDE>::Shared) + (size_t)p.key_cap * 4 + (size_t)p.key_cap / 32 * 4;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

// Clusters of c CTAs of the wide form that the device runs at once (fewer than its SMs alone would let it), for a
// request whose scores take a quarter of the shared memory; longer ones take all of an SM's either way.
template <int D>
cudaError_t clusters_at_once(int dev, int c, int64_t* out) {
  static std::atomic<int> known[64][kSelectMaxCluster + 1];  // 0: not asked yet, else the answer + 1
  int v = dev >= 0 && dev < 64 ? known[dev][c].load(std::memory_order_relaxed) : 0;
  if (v == 0) {
    SelectParams p{};
    p.key_cap = kSelectMaxBlocks / 4;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    configure<D, true>(cfg, attr, p, c, c, nullptr);
    cfg.numAttrs = 1;
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, block_select_kernel<D, true>, &cfg);
    if (e != cudaSuccess) return e;
    v = n + 1;
    if (dev >= 0 && dev < 64) known[dev][c].store(v, std::memory_order_relaxed);
  }
  *out = v - 1;
  return cudaSuccess;
}

template <int D>
cudaError_t launch_form(const SelectParams& p, int64_t units, int most, int num_sms, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // Narrow for few pages (128 units of up to 512 pages 6.8 us, wide 8.2; of 768 8.9, wide 9.8; of 1024 14.0, wide 11.0;
  // 8 units of 512 pages 6.6, wide 8.0; of 1024 9.1, wide 7.9), and where units outnumber the SMs, which hold one wide
  // CTA each (512 units of 400 to 512 pages 13.8 us, wide 32.6; 256 of 768 to 1024 pages 16.8, wide 23.3; 152 of as
  // many 14.8, wide 12.4; 192 of up to 4096 pages 49.6, wide 47.3).
  const bool wide = most > kFewPages && units <= num_sms;
  e = wide ? allow_shared_memory<D, true>(dev) : allow_shared_memory<D, false>(dev);
  if (e != cudaSuccess) return e;
  int C = 1;
  // clusters while all of them run at once and every warp of a slice has two loads to make
  for (int c = kSelectMaxCluster; wide && c > 1 && C == 1; --c) {
    if (most / c < 2 * Form<true>::WARPS * (512 / D)) continue;
    int64_t at_once = 0;
    e = clusters_at_once<D>(dev, c, &at_once);
    if (e != cudaSuccess) return e;
    if (units <= at_once) C = c;
  }
  if (units * C > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  if (!wide) {
    configure<D, false>(cfg, attr, p, units, 1, s);
    return cudaLaunchKernelEx(&cfg, block_select_kernel<D, false>, p);
  }
  configure<D, true>(cfg, attr, p, units * C, C, s);
  return cudaLaunchKernelEx(&cfg, block_select_kernel<D, true>, p);
}

static_assert(sizeof(Form<true>::Shared) + (size_t)kSelectMaxBlocks * 4 + (size_t)kSelectMaxBlocks / 32 * 4 <= 232448,
              "the scores of the longest request fit the shared memory of one CTA");

}  // namespace

cudaError_t launch_block_select(SelectParams p, int32_t batch, int32_t max_blocks, int num_sms, cudaStream_t s) {
  const int64_t units = (int64_t)batch * p.num_kv_heads;
  const int32_t most = std::max(1, max_blocks - p.num_sink - p.num_recent);
  p.key_cap = (most + 31) / 32 * 32;
  p.by_page = divider(p.page_size);
  p.err = device_error_ptr();
  if (!p.err) return cudaErrorInvalidDevice;
  return p.head_dim == 128 ? launch_form<128>(p, units, most, num_sms, s) : launch_form<64>(p, units, most, num_sms, s);
}

}  // namespace pkv
