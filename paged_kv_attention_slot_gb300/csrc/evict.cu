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
// arithmetic to speak of.  With few units the work of one has to be spread, so a unit belongs to a
// thread-block cluster of C CTAs: each takes a contiguous slice of the positions, and histograms, prefix
// counts and the list of moves go through distributed shared memory.  One launch does it all, and
// nothing is read back: the new length is min(L, b).
//
// Selection: a radix select on the scores as order-preserving 32-bit keys, 11 + 11 + 10 bits from the
// top; each pass histograms the keys that share the digits found so far.  It leaves the m-th largest
// key and how many of the keys equal to it survive; those go by position.

#include <cooperative_groups.h>

#include <algorithm>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pkv {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;       // 4 per thread
constexpr int kListCap = 1024;    // moves one CTA holds at a time
constexpr int kUnroll = 4;        // 16-byte chunks in flight per thread
constexpr int kMaxKeys = 32768;   // scores of a slice kept in shared memory (128 KB); longer slices re-read them
constexpr int kMaxSlice = 262144; // positions per CTA at most (12 bytes of shared memory per 32 of them)
constexpr int kMaxCluster = 8;

static_assert(kBins == 4 * kThreads, "four bins per thread");
static_assert((int64_t)kMaxSlice * kMaxCluster >= kEvictMaxLen, "a cluster covers the longest request");

struct Shared {
  uint32_t hist[2][kBins];
  int2 move[kListCap];        // (destination position, source position)
  int4 place[kListCap];       // their (page, offset): dst page, dst offset, src page, src offset
  uint32_t warp_sum[kWarps];
  unsigned long long warp_sum2[kWarps];
  uint32_t digit, rest;       // of the radix pass: the digit found, how many keys to take inside it
  uint32_t eq_total;          // this CTA's keys equal to the threshold
  unsigned long long hm_total;  // this CTA's holes (high half) and movers (low half)
};

// scores in an order-preserving unsigned form; a NaN is the lowest, -0 equals +0
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// exclusive prefix over the threads of `v`, and the total of the block
template <typename V>
__device__ __forceinline__ V block_prefix(V v, V* warp_sum, V& total) {
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
  V before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const V s = warp_sum[k];
    before += k < warp ? s : 0;
    all += s;
  }
  total = all;
  return before + inc - v;
}

// bits [lo, hi) of the 32 positions that start at `first`
__device__ __forceinline__ uint32_t range_mask(int first, int lo, int hi) {
  const int a = max(lo - first, 0), b = min(hi - first, 32);
  if (b <= a) return 0u;
  return (b - a == 32 ? 0xffffffffu : ((1u << (b - a)) - 1u)) << a;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictParams p, int slice_cap, int key_cap) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int word_cap = slice_cap / 32;
  uint32_t* lives = reinterpret_cast<uint32_t*>(smem + sizeof(Shared));  // survivors of the slice, a bit each
  uint32_t* eqw = lives + word_cap;    // keys equal to the threshold; later the holes before each word
  uint32_t* mov = eqw + word_cap;      // movers before each word
  uint32_t* keys = mov + word_cap;     // [key_cap] order-preserving scores of the slice (key_cap = 0: not kept)

  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int unit = blockIdx.x / C;
  const int h = unit % p.num_kv_heads, i = unit / p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  pdl_wait();
  const ReqInfo rq = p.req[i];
  const int L = rq.kv_len, b = p.budget, S = p.num_sink, R = p.num_recent;
  int32_t* kept = p.kept + (int64_t)unit * b;
  if (L <= b) {  // the whole cluster: nothing to evict
    for (int j = rank * kThreads + tid; j < b; j += C * kThreads) kept[j] = j < L ? j : -1;
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

  const int m = b - S - R;          // body keys that survive
  const int front = b - R, tail = L - R;
  const int slice = ((L + C - 1) / C + 31) / 32 * 32;  // <= slice_cap
  const int base = rank * slice;
  const int n = max(0, min(slice, L - base));  // positions of this slice
  const int nw = (n + 31) / 32;

  // ---- the scores of the body ----
  auto key_from_memory = [&](int pos) -> uint32_t {
    int page, off;
    place_of(pos, page, off);
    return order_key(*score_at(page, off));
  };
  const bool cached = key_cap > 0;
  if (cached)
    for (int k = tid; k < n; k += kThreads) {
      const int pos = base + k;
      keys[k] = pos >= S && pos < tail ? key_from_memory(pos) : 0u;
    }
  auto key_at = [&](int k) -> uint32_t { return cached ? keys[k] : key_from_memory(base + k); };
  const int body_lo = min(max(S - base, 0), n), body_hi = min(max(tail - base, 0), n);

  // ---- the m-th largest key of the unit's body ----
  uint32_t T = 0xffffffffu;  // above every key: nothing survives
  uint32_t need_eq = 0;
  if (m > 0) {
    for (int k = tid; k < 2 * kBins; k += kThreads) (&sh.hist[0][0])[k] = 0u;
    __syncthreads();
    uint32_t prefix = 0, fixed = 0, rest = (uint32_t)m;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bits = pass == 2 ? 0x3ffu : 0x7ffu;
      uint32_t* hist = sh.hist[pass & 1];
      for (int k = body_lo + tid; k < body_hi; k += kThreads) {
        const uint32_t key = key_at(k);
        if ((key & fixed) == prefix) atomicAdd(&hist[(key >> shift) & bits], 1u);
      }
      cluster.sync();
      // this thread's four bins, over the cluster's slices; bins in descending order over the threads
      const int bin0 = kBins - 4 - 4 * tid;
      uint4 c = make_uint4(0u, 0u, 0u, 0u);
      for (int r = 0; r < C; ++r) {
        const uint4 x = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(hist, r) + bin0);
        c.x += x.x;
        c.y += x.y;
        c.z += x.z;
        c.w += x.w;
      }
      uint32_t total;
      uint32_t above = block_prefix<uint32_t>(c.x + c.y + c.z + c.w, sh.warp_sum, total);
      const uint32_t cnt[4] = {c.w, c.z, c.y, c.x};  // descending
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (above < rest && above + cnt[k] >= rest) {  // exactly one (thread, bin) of the block
          sh.digit = (uint32_t)(bin0 + 3 - k);
          sh.rest = rest - above;
        }
        above += cnt[k];
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      fixed |= bits << shift;
      rest = sh.rest;
      // pass 2 uses hist[0] again: every CTA read it before the cluster barrier of pass 1
      if (pass == 1)
        for (int k = tid; k < kBins; k += kThreads) sh.hist[0][k] = 0u;
      __syncthreads();
    }
    T = prefix;
    need_eq = rest;
  } else {
    __syncthreads();
  }

  // ---- survivors, a bit per position ----
  for (int w = warp; w < nw; w += kWarps) {
    const int k = w * 32 + lane;
    const bool body = k >= body_lo && k < body_hi;
    const uint32_t key = body ? key_at(k) : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, body && key > T);
    const uint32_t eq = __ballot_sync(0xffffffffu, body && key == T);
    if (lane == 0) {
      lives[w] = gt;
      eqw[w] = eq;
    }
  }
  __syncthreads();
  const int per_thread = (nw + kThreads - 1) / kThreads;  // consecutive words per thread
  const int w0 = min(tid * per_thread, nw), w1 = min(w0 + per_thread, nw);
  uint32_t eq_mine = 0;
  for (int w = w0; w < w1; ++w) eq_mine += __popc(eqw[w]);
  uint32_t total;
  uint32_t eq_before = block_prefix<uint32_t>(eq_mine, sh.warp_sum, total);
  if (tid == 0) sh.eq_total = total;
  cluster.sync();
  for (int r = 0; r < rank; ++r) eq_before += *cluster.map_shared_rank(&sh.eq_total, r);
  unsigned long long hm = 0;
  for (int w = w0; w < w1; ++w) {
    uint32_t e = eqw[w];
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
  unsigned long long hm_before = block_prefix<unsigned long long>(hm, sh.warp_sum2, hm_all);
  if (tid == 0) sh.hm_total = hm_all;
  cluster.sync();
  uint32_t holes = 0;  // of the unit (= its movers)
  for (int r = 0; r < C; ++r) {
    const unsigned long long x = *cluster.map_shared_rank(&sh.hm_total, r);
    if (r < rank) hm_before += x;
    holes += (uint32_t)(x >> 32);
  }
  for (int w = w0; w < w1; ++w) {
    const int first = base + w * 32;
    const uint32_t alive = lives[w];
    eqw[w] = (uint32_t)(hm_before >> 32);
    mov[w] = (uint32_t)hm_before;
    hm_before += (unsigned long long)__popc(~alive & range_mask(first, S, front)) << 32 | __popc(alive & range_mask(first, front, tail));
  }
  __syncthreads();

  // ---- fill the holes, C * kListCap moves at a time ----
  const int rc = p.row_chunks;                     // a power of two
  const int item_shift = 31 - __clz(2 * rc);       // 16-byte chunks of a K and a V row
  const int64_t head_off = (int64_t)h * p.stride_head_b, sf_head = (int64_t)h * p.sf_head_b;
  auto chunk_ptr = [&](int page, int off, int c) -> uint4* {
    char* pool = c < rc ? p.k_pool : p.v_pool;
    return reinterpret_cast<uint4*>(pool + (int64_t)page * p.stride_page_b + (int64_t)off * p.stride_token_b + head_off) +
           (c & (rc - 1));
  };
  auto sf_off = [&](int page, int off) -> int64_t {
    return (int64_t)page * p.sf_page_b + (int64_t)off * p.sf_token_b + sf_head;
  };
  const uint32_t lt = (1u << lane) - 1u;
  for (uint32_t t0 = 0, per = 0; t0 < holes || t0 == 0; t0 += per * C) {
    per = min((uint32_t)kListCap, (holes - t0 + C - 1) / C);  // moves per CTA of this round
    for (int w = warp; w < nw; w += kWarps) {
      const int first = base + w * 32, pos = first + lane;
      const uint32_t alive = lives[w];
      const uint32_t hb = ~alive & range_mask(first, S, front), mb = alive & range_mask(first, front, tail);
      if (t0 == 0 && pos < front && !((hb >> lane) & 1)) kept[pos] = pos;
      const bool hole = (hb >> lane) & 1, mover = (mb >> lane) & 1;
      if (hole || mover) {
        const uint32_t t = (hole ? eqw[w] + __popc(hb & lt) : mov[w] + __popc(mb & lt)) - t0;  // wraps below t0
        if (t < per * C) {
          int2* e = cluster.map_shared_rank(sh.move, t / per) + t % per;
          if (hole) e->x = pos;
          else e->y = pos;
        }
      }
    }
    if (holes == 0) break;
    cluster.sync();  // the lists are complete
    const int mine = (int)min((int64_t)per, max((int64_t)0, (int64_t)holes - t0 - (int64_t)rank * per));
    for (int e = tid; e < mine; e += kThreads) {
      const int2 mv = sh.move[e];
      int4 pl;
      place_of(mv.x, pl.x, pl.y);
      place_of(mv.y, pl.z, pl.w);
      sh.place[e] = pl;
      kept[mv.x] = mv.y;
      *score_at(pl.x, pl.y) = *score_at(pl.z, pl.w);
      if (p.k_sf) {
        const int64_t d = sf_off(pl.x, pl.y), s = sf_off(pl.z, pl.w);
        *reinterpret_cast<uint2*>(p.k_sf + d) = *reinterpret_cast<const uint2*>(p.k_sf + s);
        *reinterpret_cast<uint2*>(p.v_sf + d) = *reinterpret_cast<const uint2*>(p.v_sf + s);
      }
    }
    __syncthreads();
    const int items = mine << item_shift;
    for (int x0 = tid; x0 < items; x0 += kThreads * kUnroll) {
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int x = x0 + u * kThreads;
        if (x < items) {
          const int4 pl = sh.place[x >> item_shift];
          v[u] = *chunk_ptr(pl.z, pl.w, x & (2 * rc - 1));
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int x = x0 + u * kThreads;
        if (x < items) {
          const int4 pl = sh.place[x >> item_shift];
          *chunk_ptr(pl.x, pl.y, x & (2 * rc - 1)) = v[u];
        }
      }
    }
    cluster.sync();  // the lists may be rewritten; sources in [front, tail) may be overwritten
  }

  // ---- the last R keys move down by L - b, in order ----
  const bool overlap = L - b < R;  // tiles are then read by the whole cluster before any is written
  const int gtid = rank * kThreads + tid, gstride = C * kThreads;
  for (int j0 = 0; j0 < R; j0 += gstride) {
    const int j = j0 + gtid;
    float sc = 0.f;
    uint2 fk = make_uint2(0u, 0u), fv = fk;
    int dp = 0, dof = 0;
    if (j < R) {
      int sp, so;
      place_of(tail + j, sp, so);
      place_of(front + j, dp, dof);
      sc = *score_at(sp, so);
      if (p.k_sf) {
        fk = *reinterpret_cast<const uint2*>(p.k_sf + sf_off(sp, so));
        fv = *reinterpret_cast<const uint2*>(p.v_sf + sf_off(sp, so));
      }
      kept[front + j] = tail + j;
    }
    if (overlap) cluster.sync();
    if (j < R) {
      *score_at(dp, dof) = sc;
      if (p.k_sf) {
        *reinterpret_cast<uint2*>(p.k_sf + sf_off(dp, dof)) = fk;
        *reinterpret_cast<uint2*>(p.v_sf + sf_off(dp, dof)) = fv;
      }
    }
  }
  const int64_t items = (int64_t)R << item_shift;
  for (int64_t x0 = 0; x0 < items; x0 += (int64_t)gstride * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t x = x0 + gtid + (int64_t)u * gstride;
      if (x < items) {
        int page, off;
        place_of(tail + (int)(x >> item_shift), page, off);
        v[u] = *chunk_ptr(page, off, (int)(x & (2 * rc - 1)));
      }
    }
    if (overlap) cluster.sync();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t x = x0 + gtid + (int64_t)u * gstride;
      if (x < items) {
        int page, off;
        place_of(front + (int)(x >> item_shift), page, off);
        *chunk_ptr(page, off, (int)(x & (2 * rc - 1))) = v[u];
      }
    }
  }
  cluster.sync();  // no CTA leaves while another may still read its shared memory
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int32_t batch, int32_t max_len, int num_sms, cudaStream_t s) {
  const int64_t units = (int64_t)batch * p.num_kv_heads;
  // CTAs per unit: enough to cover the longest request, then doubled while there are SMs without a
  // CTA and slices longer than 1024 positions
  int C = 1;
  while (C < kMaxCluster && (max_len + C - 1) / C > kMaxSlice) C *= 2;
  while (C < kMaxCluster && units * C * 2 <= 2 * (int64_t)num_sms && max_len / C > 1024) C *= 2;
  if (units * C > INT32_MAX) return cudaErrorInvalidValue;
  const int slice_cap = ((max_len + C - 1) / C + 31) / 32 * 32;
  const int key_cap = slice_cap <= kMaxKeys ? slice_cap : 0;
  const size_t smem = sizeof(Shared) + (size_t)slice_cap / 32 * 12 + (size_t)key_cap * 4;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
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
  return cudaLaunchKernelEx(&cfg, evict_kernel, p, slice_cap, key_cap);
}

}  // namespace pkv
