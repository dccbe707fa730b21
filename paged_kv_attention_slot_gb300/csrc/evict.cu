// Eviction by accumulated attention weight, with the compaction of the pages in place (pkv_kv_evict).
//
// For one (request, KV head), a "unit", with L keys, a budget b < L, S first keys and R last keys that
// stay, the body [S, L - R) keeps the m = b - S - R keys with the largest scores (equal scores: the
// lower position).  Then, moving as few rows as the result allows,
//   hole t   = the t-th evicted position of the front [S, b - R), ascending,
//   mover t  = the t-th survivor beyond the front, in [b - R, L - R), ascending,
//   row[hole t] <- row[mover t]       (as many movers as holes: m = survivors in front + movers)
//   row[b - R + j] <- row[L - R + j]  (j < R, in order).
// Sources and destinations of the first kind are disjoint; the second kind overlaps itself when
// L - b < R and overwrites sources of the first, so it runs after them, tile by tile, every tile read
// before it is written.
//
// What bounds it: reading the scores once (4 bytes per key) and moving the rows; there is no
// arithmetic to speak of, but a chain of steps (scores, selection, prefix counts, moves).  One launch does
// them all, and nothing is read back: the new length is min(L, b).  A unit belongs to a thread-block
// cluster of C CTAs, in one of two forms:
//   * requests of up to kMaxWhole keys: every CTA of the cluster selects on its own, from its own copy of
//     the scores (C-fold reads, from L2), and moves its own columns of every row (C = 2: K and V).  The CTAs
//     exchange nothing; one cluster barrier, long passed when it is waited for, keeps the scores from
//     being rewritten before everyone has read them.
//   * longer ones: each CTA takes a contiguous slice of the positions; histograms, prefix counts and
//     the list of moves go through distributed shared memory.
//
// Selection: a radix select on the scores as order-preserving 32-bit keys, 11 + 11 + 10 bits from the
// top; each pass histograms the keys that share the digits found so far, and the passes end early when
// all of those survive.  It leaves the smallest surviving key and how many of the keys equal to it
// survive; those go by position.

#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pkv {

namespace {

constexpr int kBins = 2048;
constexpr int kUnroll = 4;         // 16-byte chunks in flight per thread
constexpr int kMaxWhole = 12288;   // longest request of the whole form (48 KB of scores)
constexpr int kMaxKeys = 32768;    // scores of a slice kept in shared memory (128 KB); longer slices re-read them
constexpr int kMaxSlice = 262144;  // positions per CTA at most (12 bytes of shared memory per 32 of them)
constexpr int kMaxCluster = 8;
static_assert((int64_t)kMaxSlice * kMaxCluster >= kEvictMaxLen, "a cluster covers the longest request");

template <bool SLICED>
struct Form {
  static constexpr int THREADS = SLICED ? 1024 : 256;
  static constexpr int CTAS = SLICED ? 1 : 5;     // resident per SM by registers (whole: by shared memory too, to 5700 keys)
  static constexpr int WARPS = THREADS / 32;
  static constexpr int LIST = SLICED ? 2048 : 512;  // moves one CTA holds at a time
  static constexpr int HISTS = SLICED ? 2 : 1;
  // groups of four scores in flight per thread (sliced: 4 is 0.1 us slower on 2 x 131072 keys)
  static constexpr int SCORES = SLICED ? 6 : 4;
  // keys read ahead per thread: whole, 8 x 1060 keys, 8.9 us with 4, 9.9 with 1 (a warp has little else to
  // do); sliced, where eight warps per scheduler hide the reads, 35.9 us with 1, 37 with 2
  static constexpr int KEYS = SLICED ? 1 : 4;
  // moves whose rows a thread looks up at once: whole, 64 x 512..4160 keys, 64 us with 1, 69 with 2 (spills)
  static constexpr int PLACES = SLICED ? 2 : 1;
  static_assert(THREADS <= LIST, "the list holds a tile of the last rows");
  static constexpr int GROUPS = SLICED ? kBins / 32 : 1;  // sliced: sums of 32 neighbouring bins
  struct alignas(16) Shared {
    uint32_t hist[HISTS][kBins];
    uint32_t group[HISTS][GROUPS];
    int2 move[LIST];         // (destination position, source position)
    longlong2 place[LIST];   // byte offsets of their rows in the pools: (destination, source)
    unsigned long long warp_sum[WARPS];
    uint32_t digit, rest, count;  // of the radix pass: the digit found, the keys to take inside it, its keys
    unsigned long long hm_total;  // sliced: this CTA's holes (high half) and movers (low half)
  };
};

// scores in an order-preserving unsigned form; a NaN is the lowest, -0 equals +0
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// exclusive prefix over the block's threads of `v`, and the total of the block
template <int WARPS, typename V>
__device__ __forceinline__ V block_prefix(V v, unsigned long long* warp_sum, V& total) {
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
  // every warp scans the warps' sums itself
  V s = lane < WARPS ? (V)warp_sum[lane] : (V)0;
#pragma unroll
  for (int o = 1; o < WARPS; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  total = __shfl_sync(0xffffffffu, s, WARPS - 1);
  const V before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : (V)0) + inc - v;
}

// bits [lo, hi) of the 32 positions that start at `first`
__device__ __forceinline__ uint32_t range_mask(int first, int lo, int hi) {
  const int a = max(lo - first, 0), b = min(hi - first, 32);
  if (b <= a) return 0u;
  return (b - a == 32 ? 0xffffffffu : ((1u << (b - a)) - 1u)) << a;
}

template <bool SLICED>
__global__ void __launch_bounds__(Form<SLICED>::THREADS, Form<SLICED>::CTAS) evict_kernel(const EvictParams p, int slice_cap,
                                                                                         int key_cap) {
  using F = Form<SLICED>;
  constexpr int THREADS = F::THREADS, WARPS = F::WARPS;
  extern __shared__ __align__(16) uint8_t smem[];
  typename F::Shared& sh = *reinterpret_cast<typename F::Shared*>(smem);
  const int word_cap = slice_cap / 32;
  // [key_cap] order-preserving scores of the slice (a multiple of 32, or 0: not kept; 16-byte aligned)
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(typename F::Shared));
  uint32_t* lives = keys + key_cap;  // survivors of the slice, a bit each
  uint32_t* eqw = lives + word_cap;  // keys equal to the threshold; later the holes before each word
  uint32_t* mov = eqw + word_cap;    // movers before each word

  cg::cluster_group cluster = cg::this_cluster();
  const int CN = (int)cluster.num_blocks(), CR = (int)cluster.block_rank();
  const int C = SLICED ? CN : 1, rank = SLICED ? CR : 0;  // how positions and rows are shared out
  auto unit_sync = [&]() {
    if constexpr (SLICED) cluster.sync();
    else __syncthreads();
  };
  const int unit = blockIdx.x / CN;
  const int h = unit % p.num_kv_heads, i = unit / p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  pdl_wait();
  const ReqInfo rq = p.req[i];
  const int L = rq.kv_len, b = p.budget, S = p.num_sink, R = p.num_recent;
  int32_t* kept = p.kept + (int64_t)unit * b;
  if (L <= b) {  // the whole cluster: nothing to evict
    for (int j = CR * THREADS + tid; j < b; j += CN * THREADS) kept[j] = j < L ? j : -1;
    return;
  }
  const int32_t* pages = p.kv_indices + rq.page_base;
  const int ps = p.page_size;
  const int ps_shift = (ps & (ps - 1)) == 0 ? __ffs(ps) - 1 : -1;
  auto place_of = [&](int pos, int& page, int& off) {
    const int q = ps_shift >= 0 ? pos >> ps_shift : pos / ps;
    page = __ldg(pages + q);
    off = pos - q * ps;
  };
  auto score_at = [&](int page, int off) -> float* {
    return p.scores + ((int64_t)page * p.num_kv_heads + h) * ps + off;
  };

  const int m = b - S - R;  // body keys that survive
  const int front = b - R, tail = L - R;
  const int slice = ((L + C - 1) / C + 31) / 32 * 32;  // <= slice_cap
  const int base = rank * slice;
  const int n = max(0, min(slice, L - base));  // positions of this slice
  const int nw = (n + 31) / 32;

  if (m > 0)
    for (int k = tid; k < F::HISTS * kBins; k += THREADS) (&sh.hist[0][0])[k] = 0u;

  // ---- the scores of the body ----
  auto key_from_memory = [&](int pos) -> uint32_t {
    int page, off;
    place_of(pos, page, off);
    return order_key(*score_at(page, off));
  };
  const bool cached = !SLICED || key_cap > 0;
  const int body_lo = min(max(S - base, 0), n), body_hi = min(max(tail - base, 0), n);
  if (cached) {
    // (positions outside the body get some key that no one looks at)
    if ((ps & 3) == 0 && (reinterpret_cast<uintptr_t>(p.scores) & 15) == 0) {
      // four positions of one page at a time; a last group may reach past L, but not past its page
      const int groups = (n + 3) / 4;
      for (int q0 = tid; q0 < groups; q0 += THREADS * F::SCORES) {
        float4 x[F::SCORES];
#pragma unroll
        for (int u = 0; u < F::SCORES; ++u) {
          const int q = q0 + u * THREADS;
          if (q < groups) {
            int page, off;
            place_of(base + 4 * q, page, off);
            x[u] = *reinterpret_cast<const float4*>(score_at(page, off));
          }
        }
#pragma unroll
        for (int u = 0; u < F::SCORES; ++u) {
          const int q = q0 + u * THREADS;
          if (q < groups)
            *reinterpret_cast<uint4*>(keys + 4 * q) =
                make_uint4(order_key(x[u].x), order_key(x[u].y), order_key(x[u].z), order_key(x[u].w));
        }
      }
    } else {
      for (int k0 = tid; k0 < n; k0 += THREADS * F::SCORES) {
        uint32_t x[F::SCORES];
#pragma unroll
        for (int u = 0; u < F::SCORES; ++u) {
          const int k = k0 + u * THREADS;
          if (k < n) x[u] = key_from_memory(base + k);
        }
#pragma unroll
        for (int u = 0; u < F::SCORES; ++u) {
          const int k = k0 + u * THREADS;
          if (k < n) keys[k] = x[u];
        }
      }
    }
  }
  auto key_at = [&](int k) -> uint32_t { return cached ? keys[k] : key_from_memory(base + k); };
  // whole form: this CTA has read every score it will read (waited for before scores are moved)
  if constexpr (!SLICED) cluster.barrier_arrive();

  // ---- the m-th largest key of the unit's body ----
  uint32_t T = 0xffffffffu;  // keys above T survive, and need_eq of those equal to it (m = 0: none is above)
  uint32_t need_eq = 0;
  uint32_t eq_before = 0;  // keys equal to T in the slices before this one
  __syncthreads();
  if (m > 0) {
    uint32_t prefix = 0, fixed = 0, rest = (uint32_t)m;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bits = pass == 2 ? 0x3ffu : 0x7ffu;
      uint32_t* hist = sh.hist[SLICED ? pass & 1 : 0];
      for (int k0 = body_lo + tid; k0 < body_hi; k0 += THREADS * F::KEYS) {
        uint32_t x[F::KEYS];
#pragma unroll
        for (int u = 0; u < F::KEYS; ++u)
          if (k0 + u * THREADS < body_hi) x[u] = key_at(k0 + u * THREADS);
#pragma unroll
        for (int u = 0; u < F::KEYS; ++u)
          if (k0 + u * THREADS < body_hi && (x[u] & fixed) == prefix) atomicAdd(&hist[(x[u] >> shift) & bits], 1u);
      }
      if constexpr (SLICED) {
        // the bin of the rest-th key from the top, over the cluster's slices: first its group of 32 bins,
        // then the bin, so that two short rounds of remote reads do (one warp) instead of whole histograms
        __syncthreads();
        uint32_t* group = sh.group[pass & 1];
        for (int g = tid / 16; g < F::GROUPS; g += THREADS / 16) {
          uint32_t v = hist[32 * g + 2 * (tid & 15)] + hist[32 * g + 2 * (tid & 15) + 1];
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if ((tid & 15) == 0) group[g] = v;
        }
        cluster.sync();
        if (warp == 0) {
          uint32_t hi = 0, lo = 0;  // groups 63 - lane and 31 - lane
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            if (r < C) {
              const uint32_t* gr = cluster.map_shared_rank(group, r);
              hi += gr[63 - lane];
              lo += gr[31 - lane];
            }
          uint32_t ihi = hi, ilo = lo;  // inclusive, from the top
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xffffffffu, ihi, o), c = __shfl_up_sync(0xffffffffu, ilo, o);
            if (lane >= o) {
              ihi += a;
              ilo += c;
            }
          }
          ilo += __shfl_sync(0xffffffffu, ihi, 31);
          const uint32_t bh = __ballot_sync(0xffffffffu, ihi >= rest), bl = __ballot_sync(0xffffffffu, ilo >= rest);
          const int src = __ffs(bh ? bh : bl) - 1;  // the body holds at least m keys, so one is set
          const uint32_t above_g = __shfl_sync(0xffffffffu, bh ? ihi - hi : ilo - lo, src);
          const int g = (bh ? 63 : 31) - src;
          uint32_t c = 0;
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            if (r < C) c += cluster.map_shared_rank(hist, r)[32 * g + 31 - lane];
          uint32_t inc = c;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += a;
          }
          inc += above_g;
          if (inc >= rest && inc - c < rest) {  // exactly one lane
            sh.digit = (uint32_t)(32 * g + 31 - lane);
            sh.rest = rest - (inc - c);
            sh.count = c;
          }
        }
      } else {
        __syncthreads();
        // this thread's bins, in descending order over the threads
        constexpr int BINS_PT = kBins / THREADS;
        const int bin0 = kBins - BINS_PT * (tid + 1);
        uint32_t cnt[BINS_PT];
#pragma unroll
        for (int k = 0; k < BINS_PT; k += 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(hist + bin0 + k);
          cnt[k] = x.x;
          cnt[k + 1] = x.y;
        }
        uint32_t mine = 0, total;
#pragma unroll
        for (int k = 0; k < BINS_PT; ++k) mine += cnt[k];
        uint32_t above = block_prefix<WARPS, uint32_t>(mine, sh.warp_sum, total);
#pragma unroll
        for (int k = BINS_PT - 1; k >= 0; --k) {
          if (above < rest && above + cnt[k] >= rest) {  // exactly one (thread, bin) of the block
            sh.digit = (uint32_t)(bin0 + k);
            sh.rest = rest - above;
            sh.count = cnt[k];
          }
          above += cnt[k];
        }
      }
      // Sliced: pass 2 uses hist[0] again; every CTA read it before the cluster barrier of pass 1.
      // Whole: every thread of this CTA has read it before the barriers of block_prefix.
      if (SLICED ? pass == 1 : pass < 2)
        for (int k = tid; k < kBins; k += THREADS) sh.hist[0][k] = 0u;
      __syncthreads();
      prefix |= sh.digit << shift;
      fixed |= bits << shift;
      rest = sh.rest;
      if (sh.count == rest && prefix > 0) {
        // every key with these digits survives: all keys from `prefix` up, none by position
        prefix -= 1;
        rest = 0;
        break;
      }
      if constexpr (SLICED)
        if (pass == 2) {
          // the last pass counted every slice's keys equal to T
          const uint32_t x = lane < rank ? cluster.map_shared_rank(hist, lane)[sh.digit] : 0u;
          eq_before = __reduce_add_sync(0xffffffffu, x);
        }
    }
    T = prefix;
    need_eq = rest;
  }

  // ---- survivors, a bit per position ----
  for (int wu = warp; wu < nw; wu += WARPS * F::KEYS) {
    uint32_t x[F::KEYS];
#pragma unroll
    for (int u = 0; u < F::KEYS; ++u) {
      const int k = (wu + u * WARPS) * 32 + lane;
      if (k >= body_lo && k < body_hi) x[u] = key_at(k);
    }
#pragma unroll
    for (int u = 0; u < F::KEYS; ++u) {
      const int w = wu + u * WARPS, k = w * 32 + lane;
      const bool body = k >= body_lo && k < body_hi;
      const uint32_t gt = __ballot_sync(0xffffffffu, body && x[u] > T);
      const uint32_t eq = __ballot_sync(0xffffffffu, body && x[u] == T);
      if (lane == 0 && w < nw) {
        lives[w] = gt;
        eqw[w] = eq;
      }
    }
  }
  __syncthreads();
  const int per_thread = (nw + THREADS - 1) / THREADS;  // consecutive words per thread
  const int w0 = min(tid * per_thread, nw), w1 = min(w0 + per_thread, nw);
  if (need_eq > 0) {
    uint32_t eq_mine = 0, total;
    for (int w = w0; w < w1; ++w) eq_mine += __popc(eqw[w]);
    eq_before += block_prefix<WARPS, uint32_t>(eq_mine, sh.warp_sum, total);
  }
  unsigned long long hm = 0;
  for (int w = w0; w < w1; ++w) {
    uint32_t e = need_eq > 0 ? eqw[w] : 0u;
    const uint32_t c = __popc(e);
    if (eq_before + c > need_eq) {  // only the lowest (need_eq - eq_before) of them
      uint32_t take = eq_before < need_eq ? need_eq - eq_before : 0u, out = 0u;
      for (; take > 0; --take) {
        out |= e & (0u - e);
        e &= e - 1;
      }
      e = out;
    }
    eq_before += c;
    const uint32_t alive = lives[w] | e;
    lives[w] = alive;
    const int first = base + w * 32;
    hm += (unsigned long long)__popc(~alive & range_mask(first, S, front)) << 32 | __popc(alive & range_mask(first, front, tail));
  }
  unsigned long long hm_all;
  unsigned long long hm_before = block_prefix<WARPS, unsigned long long>(hm, sh.warp_sum, hm_all);
  uint32_t holes = (uint32_t)(hm_all >> 32);  // of the unit (= its movers)
  if constexpr (SLICED) {
    if (tid == 0) sh.hm_total = hm_all;
    cluster.sync();
    const unsigned long long x = lane < C ? *cluster.map_shared_rank(&sh.hm_total, lane) : 0ull;
    holes = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 32));
    hm_before += (unsigned long long)__reduce_add_sync(0xffffffffu, lane < rank ? (uint32_t)(x >> 32) : 0u) << 32;
    hm_before += __reduce_add_sync(0xffffffffu, lane < rank ? (uint32_t)x : 0u);
  }
  for (int w = w0; w < w1; ++w) {
    const int first = base + w * 32;
    const uint32_t alive = lives[w];
    eqw[w] = (uint32_t)(hm_before >> 32);
    mov[w] = (uint32_t)hm_before;
    hm_before += (unsigned long long)__popc(~alive & range_mask(first, S, front)) << 32 | __popc(alive & range_mask(first, front, tail));
  }
  __syncthreads();

  // ---- fill the holes, C * LIST moves at a time ----
  // A CTA moves `cols` 16-byte chunks from chunk col0 on of every row pair it is given (K, then V).
  const int rc = p.row_chunks;  // a power of two
  const int cols = SLICED ? 2 * rc : 2 * rc / CN, col0 = SLICED ? 0 : CR * cols;
  const int item_shift = 31 - __clz(cols);
  // whole form: the first CTA moves scores, kept positions and K scales, the last one V scales
  const bool with_k = SLICED || CR == 0, with_v = SLICED || CR == CN - 1;
  const int64_t head_off = (int64_t)h * p.stride_head_b, sf_head = (int64_t)h * p.sf_head_b;
  auto row_off = [&](int page, int off) -> int64_t {
    return (int64_t)page * p.stride_page_b + (int64_t)off * p.stride_token_b + head_off;
  };
  // Each thread moves one column, of the rows row0, row0 + rows_at_once, ... of a list (THREADS is a
  // multiple of cols).
  const int col = col0 + (tid & (cols - 1)), row0 = tid >> item_shift, rows_at_once = THREADS >> item_shift;
  char* const column = (col < rc ? p.k_pool : p.v_pool) + (col & (rc - 1)) * 16;
  auto sf_off = [&](int page, int off) -> int64_t {
    return (int64_t)page * p.sf_page_b + (int64_t)off * p.sf_token_b + sf_head;
  };
  if constexpr (!SLICED) cluster.barrier_wait();  // all CTAs of the unit have read its scores
  const uint32_t lt = (1u << lane) - 1u;
  const int front_here = min(max(front - base, 0), n);  // positions of the slice that are in the front
  const int front_words = (front_here + 31) / 32, mover_word0 = front_here / 32;
  for (uint32_t t0 = 0, per = 0; t0 < holes || t0 == 0; t0 += per * C) {
    per = min((uint32_t)F::LIST, (holes - t0 + C - 1) / C);  // moves per CTA of this round
    const float inv_per = 1.f / (float)max(per, 1u);
    auto entry = [&](uint32_t t) -> int2* {  // of move t0 + t, in the list of the CTA that does it
      if constexpr (!SLICED) return sh.move + t;
      int r = (int)((float)t * inv_per);  // t / per, off by one at most (t < 2^14)
      r += (uint32_t)(r + 1) * per <= t;
      r -= (uint32_t)r * per > t;
      return cluster.map_shared_rank(sh.move, r) + (t - r * per);
    };
    // the front, a lane per position: holes take numbers, the others stay
    for (int w = warp; w < front_words; w += WARPS) {
      const int first = base + w * 32, pos = first + lane;
      const uint32_t hb = ~lives[w] & range_mask(first, S, front);
      const bool hole = (hb >> lane) & 1;
      if (with_k && t0 == 0 && pos < front && !hole) kept[pos] = pos;
      const uint32_t t = eqw[w] + __popc(hb & lt) - t0;  // wraps below t0
      if (hole && t < per * C) entry(t)->x = pos;
    }
    // the survivors behind it.  Sliced: a thread per word, since few of many positions survive (131072
    // keys to 8192: the lists take 4.6 us, with a lane per position 9.6); whole: a lane per position, where a
    // budget near the length leaves dense words (1088 keys to 1024: 1.1 us, a thread per word 2.1)
    if constexpr (SLICED) {
      for (int w = mover_word0 + tid; w < nw; w += THREADS) {
        const int first = base + w * 32;
        uint32_t mb = lives[w] & range_mask(first, front, tail);
        for (uint32_t t = mov[w] - t0; mb != 0; ++t, mb &= mb - 1)
          if (t < per * C) entry(t)->y = first + __ffs(mb) - 1;
      }
    } else {
      for (int w = mover_word0 + warp; w < nw; w += WARPS) {
        const int first = base + w * 32;
        const uint32_t mb = lives[w] & range_mask(first, front, tail);
        const uint32_t t = mov[w] + __popc(mb & lt) - t0;
        if (((mb >> lane) & 1) && t < per) entry(t)->y = first + lane;
      }
    }
    if (holes == 0) break;
    unit_sync();  // the lists are complete
    const int mine = (int)min((int64_t)per, max((int64_t)0, (int64_t)holes - t0 - (int64_t)rank * per));
    for (int e = tid; e < mine; e += THREADS * F::PLACES) {
      int2 mv[F::PLACES];
      int dp[F::PLACES], dof[F::PLACES], sp[F::PLACES], sof[F::PLACES];
      float sc[F::PLACES];
#pragma unroll
      for (int u = 0; u < F::PLACES; ++u)
        if (e + u * THREADS < mine) {
          mv[u] = sh.move[e + u * THREADS];
          place_of(mv[u].x, dp[u], dof[u]);
          place_of(mv[u].y, sp[u], sof[u]);
        }
#pragma unroll
      for (int u = 0; u < F::PLACES; ++u)
        if (e + u * THREADS < mine) {
          if (with_k) sc[u] = *score_at(sp[u], sof[u]);
          sh.place[e + u * THREADS] = make_longlong2(row_off(dp[u], dof[u]), row_off(sp[u], sof[u]));
        }
#pragma unroll
      for (int u = 0; u < F::PLACES; ++u)
        if (e + u * THREADS < mine) {
          if (p.k_sf) {
            const int64_t d = sf_off(dp[u], dof[u]), s = sf_off(sp[u], sof[u]);
            if (with_k) *reinterpret_cast<uint2*>(p.k_sf + d) = *reinterpret_cast<const uint2*>(p.k_sf + s);
            if (with_v) *reinterpret_cast<uint2*>(p.v_sf + d) = *reinterpret_cast<const uint2*>(p.v_sf + s);
          }
          if (with_k) {
            kept[mv[u].x] = mv[u].y;
            *score_at(dp[u], dof[u]) = sc[u];
          }
        }
    }
    __syncthreads();
    for (int e0 = row0; e0 < mine; e0 += rows_at_once * kUnroll) {
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int e = e0 + u * rows_at_once;
        if (e < mine) v[u] = *reinterpret_cast<const uint4*>(column + sh.place[e].y);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int e = e0 + u * rows_at_once;
        if (e < mine) *reinterpret_cast<uint4*>(column + sh.place[e].x) = v[u];
      }
    }
    unit_sync();  // the lists may be rewritten; sources in [front, tail) may be overwritten
  }

  // ---- the last R keys move down by L - b, in order ----
  const bool overlap = L - b < R;  // tiles are then read by all who share them before any is written
  const int rows = min(THREADS, rows_at_once * kUnroll);  // rows per CTA and tile
  for (int j0 = 0; j0 < R; j0 += C * rows) {
    const int first = j0 + rank * rows;
    const int mine = max(0, min(rows, R - first));
    float sc = 0.f;
    uint2 fk = make_uint2(0u, 0u), fv = fk;
    int dp = 0, dof = 0;
    if (tid < mine) {
      const int j = first + tid;
      int sp, sof;
      place_of(tail + j, sp, sof);
      place_of(front + j, dp, dof);
      sh.place[tid] = make_longlong2(row_off(dp, dof), row_off(sp, sof));
      if (with_k) {
        sc = *score_at(sp, sof);
        kept[front + j] = tail + j;
      }
      if (p.k_sf) {
        if (with_k) fk = *reinterpret_cast<const uint2*>(p.k_sf + sf_off(sp, sof));
        if (with_v) fv = *reinterpret_cast<const uint2*>(p.v_sf + sf_off(sp, sof));
      }
    }
    __syncthreads();
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int e = row0 + u * rows_at_once;
      if (e < mine) v[u] = *reinterpret_cast<const uint4*>(column + sh.place[e].y);
    }
    if (overlap) unit_sync();
    if (tid < mine) {
      if (with_k) *score_at(dp, dof) = sc;
      if (p.k_sf) {
        if (with_k) *reinterpret_cast<uint2*>(p.k_sf + sf_off(dp, dof)) = fk;
        if (with_v) *reinterpret_cast<uint2*>(p.v_sf + sf_off(dp, dof)) = fv;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int e = row0 + u * rows_at_once;
      if (e < mine) *reinterpret_cast<uint4*>(column + sh.place[e].x) = v[u];
    }
    __syncthreads();  // the list is rewritten by the next tile
  }
  if constexpr (SLICED) cluster.sync();  // no CTA leaves while another may still read its shared memory
}

// Clusters of c CTAs of the sliced form (one CTA per SM) that the device runs at once.  Not SMs / c: a
// cluster lives within one GPC (16 clusters of 8 were one too many for this part: the last one ran alone,
// 79 us instead of 41 for 2 x 131072 keys and 8 KV heads).
cudaError_t clusters_at_once(int dev, int c, int64_t* out) {
  static std::atomic<int> known[64][kMaxCluster + 1];  // 0: not asked yet, else the answer + 1
  int v = dev >= 0 && dev < 64 ? known[dev][c].load(std::memory_order_relaxed) : 0;
  if (v == 0) {
    cudaError_t e = cudaFuncSetAttribute(evict_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(Form<true>::THREADS);
    cfg.dynamicSmemBytes = sizeof(typename Form<true>::Shared) + (size_t)kMaxKeys * 4 + (size_t)kMaxKeys / 32 * 12;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, evict_kernel<true>, &cfg);
    if (e != cudaSuccess) return e;
    v = n + 1;
    if (dev >= 0 && dev < 64) known[dev][c].store(v, std::memory_order_relaxed);
  }
  *out = v - 1;
  return cudaSuccess;
}

template <bool SLICED>
cudaError_t launch_form(const EvictParams& p, int64_t units, int C, int slice_cap, int key_cap, cudaStream_t s) {
  using F = Form<SLICED>;
  if (units * C > INT32_MAX) return cudaErrorInvalidValue;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(evict_kernel<SLICED>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(F::THREADS);
  cfg.dynamicSmemBytes = sizeof(typename F::Shared) + (size_t)slice_cap / 32 * 12 + (size_t)key_cap * 4;
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
  return cudaLaunchKernelEx(&cfg, evict_kernel<SLICED>, p, slice_cap, key_cap);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int32_t batch, int32_t num_long, int32_t max_len, int num_sms, cudaStream_t s) {
  const int64_t units = (int64_t)batch * p.num_kv_heads, busy = (int64_t)num_long * p.num_kv_heads;
  int C = 1;
  if (max_len <= kMaxWhole) {
    // K and V to two CTAs while registers let these be resident at once: 64 requests of up to 4160 keys 67.6 us
    // (one CTA per unit 73.2), 320 units of 4000 keys 74.2 (78.3), 192 units of 8000 keys 112 (130), of 12288
    // keys 173 (200).  Beyond 5700 keys shared memory holds fewer than CTAS per SM (4 at 8192, 3 at 12288),
    // and where two per unit then no longer fit the bound errs: 320 units of 8000 keys 201 us (180), of
    // 12288 keys 302 (273).
    if (busy * 2 <= Form<false>::CTAS * (int64_t)num_sms) C = 2;
    const int cap = (max_len + 31) / 32 * 32;
    return launch_form<false>(p, units, C, cap, cap, s);
  }
  // slices: enough to cover the longest request, then as many as let all busy units run at once.  (The form is
  // the launch's: one request beyond kMaxWhole takes every unit here.  63 requests of up to 4160 keys and one of
  // 131072, to 2048 keys: 313 us; the 64 without it 66.)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  while ((max_len + C - 1) / C > kMaxSlice) ++C;
  for (int c = kMaxCluster; c > C; --c) {
    int64_t at_once = 0;
    e = clusters_at_once(dev, c, &at_once);
    if (e != cudaSuccess) return e;
    if (busy <= at_once) C = c;
  }
  const int slice_cap = ((max_len + C - 1) / C + 31) / 32 * 32;
  return launch_form<true>(p, units, C, slice_cap, slice_cap <= kMaxKeys ? slice_cap : 0, s);
}

}  // namespace pkv
