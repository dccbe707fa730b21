// Batched paged decode (one new token per request) with the split-KV merge fused in.
//
// What it computes: for request i, KV head h and every query head of h's group, the softmax over
// the visible keys of the scaled scores q.k_j, applied to v_j, with K/V read through the CSR page
// table ("SGLang 源码完全拆解(八)：Attention Backend", sections «统一元数据的编译» and «其他后端的元数据»
// (split-KV: partial outputs and log-sum-exps per KV chunk, merged by a reduction); "手写 mini-sglang
// 阶段四 · GPU 注意力后端", section «FlashInfer：plan 与 run»: with a GQA group >= 4, decode is a chain of
// small matrix products and tensor cores pay).
//
// GB300 design.  Decode is HBM-bound (about G flops per byte of KV), so the kernel is built around
// streaming the pages at full bandwidth while keeping the per-key work short:
//  * one CTA = 4 warps = one work item (request, KV head, group of <= 16 query heads) with a key
//    range; a range short enough for one CTA is read by it alone (each warp takes every 4th tile of
//    16 keys, NVFP4: 32), a long one is shared by several CTAs whose warps claim groups of two tiles
//    from a per-range counter at run time, so the CTAs of a range finish together;
//  * every warp runs its own cp.async ring (a tile per stage, K and V rows gathered page by page
//    through kv_indices, 16-byte vectors, XOR-swizzled so ldmatrix reads are conflict-free), so no
//    CTA-wide barrier sits in the main loop;
//  * the products run on m16n8k16 tensor-core MMAs with the KEYS in M and the (<= 8 per n-block)
//    query heads of one KV head in N: S^T = K Q^T, then O^T += V^T P^T.  Each K/V row is read once
//    per KV head, a 16-key tile costs 8 MMAs per product (not 16 with heads in M), and the output
//    accumulator is 32 registers per 8 heads.  P^T goes from the accumulator layout of the first MMA
//    to the operand layout of the second with one movmatrix.trans per 8x8 block;
//  * the online softmax runs per head column: base-2 exponentials with the scale folded in, against a
//    reference that moves only when a key exceeds it by more than 2^8 (one vote per tile; only then is the
//    tile's maximum formed across lanes, 3 shuffles), running sums kept per lane and reduced at the end;
//  * scores, references, sums and outputs are float32; the probabilities enter the second product in the
//    type its MMA takes beside V: bf16 for bf16 pools, f16 for the others.  That is what the outputs are
//    off by beyond their own rounding: relative to a 64-bit result the bf16 outputs by 0.0023 and the NVFP4
//    and E4M3 ones by 0.0017, where 32 bits throughout, rounded once, are off by 0.0017 (batches of 64).
//    Keeping more would take a second product per tile for the rest of the bits;
//  * FP8 (E4M3) pages are widened to f16 in registers (exact); the K scale is folded into the score
//    scale and the V scale into the output; the head-dim order inside each 16-element block is
//    permuted identically for Q and K (a dot product does not depend on order) so one ldmatrix feeds
//    two code bytes per register half, and V's byte pairs are split into even/odd head-dim rows;
//  * NVFP4 pages (E2M1 codes, one E4M3 scale per 16) are widened to f16 in registers and multiplied by
//    their block scale there, which is exact (a 2-bit times a 4-bit significand; 2^-10 .. 2688); the
//    8-byte scale rows of a tile travel in the same ring stage;
//  * the 4 warps merge their softmax states through shared memory at the end; a CTA either writes
//    the final bf16 output (no split) or a normalised fp32 partial plus its log2-sum-exp; the last
//    CTA of a split unit to finish (an atomic count per unit, reset after use, no waiting) merges
//    the unit: m = max lse_s, o = sum_s 2^(lse_s - m) o_s / sum_s 2^(lse_s - m).

#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {

int32_t* device_error_ptr();

// The K/V rows are read once per launch: they are copied with an evict-first L2 policy, so the
// stream (hundreds of MB through a 129 MB L2) does not push out the lines that are read again -- the
// work list, the page table, the split partials and whatever the surrounding layers keep there.
__device__ __forceinline__ uint64_t l2_evict_first() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(pol));
  return pol;
}
// cp.async of 8 bytes through L1 (src_bytes == 0 writes zeros).
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// cp.async of 16 bytes (src_bytes < 16 zero-fills the rest) under an L2 cache policy.
__device__ __forceinline__ void cp_async16_pol(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t pol) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;\n" ::"r"(dst), "l"(src),
               "r"(src_bytes), "l"(pol)
               : "memory");
}

// ---- accumulated attention weights (scored runs) ----
// The weight of key j for KV head h, a_j = sum over its query heads g of 2^(x_gj - lse_g) (x: the scaled
// scores in log2 units, [key][query head] at lg0), is added to scores[slot(j), h] for the keys
// [lo, hi) of a unit.  The additions are reductions at L2, so no thread waits for a score's old value;
// every score gets one per launch, so their order does not matter.  A thread takes four neighbouring keys
// (of one page: one page id, one 16-byte reduction) where pages and scores allow it, UNROLL times in flight.
// The page ids may be read at once; `ready` is called before the first look at lg0 and lse.
template <int UNROLL, typename Ready>
__device__ __forceinline__ void add_weights(const RunParams& p, const WorkItem& w, const float* lg0, const float* lse, int lo,
                                            int hi, int tid, int threads, Ready ready) {
  const int G = p.group, ps = p.page_size;
  const int ps_shift = (ps & (ps - 1)) == 0 ? __ffs(ps) - 1 : -1;
  const int32_t* pages = p.kv_indices + w.page_base;
  auto score_at = [&](int page, int off) -> float* {
    return p.scores + ((int64_t)page * p.num_kv_heads + w.kv_head) * ps + off;
  };
  auto in_pool = [&](int page) {  // (a page outside was recorded where its rows were read)
    return (unsigned long long)(unsigned)page < (unsigned long long)p.num_pages;
  };
  bool waited = false;
  if ((ps & 3) == 0 && (reinterpret_cast<uintptr_t>(p.scores) & 15) == 0) {
    for (int base = lo & ~3; base < hi; base += 4 * UNROLL * threads) {  // block-uniform
      int page[UNROLL], off[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int key = base + 4 * (tid + u * threads);
        page[u] = -1;
        off[u] = 0;
        if (key < hi) {
          const int pg = ps_shift >= 0 ? key >> ps_shift : key / ps;
          page[u] = __ldg(pages + pg);
          off[u] = key - pg * ps;
        }
      }
      if (!waited) ready();
      waited = true;
      float a[UNROLL][4];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) a[u][0] = a[u][1] = a[u][2] = a[u][3] = 0.f;
      // (a score outside [lo, hi) was not computed and is not read)
      if ((G & 3) == 0) {
        for (int g = 0; g < G; g += 4) {
          float4 x[UNROLL][4];
#pragma unroll
          for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = base + 4 * (tid + u * threads) + k;
              x[u][k] = key >= lo && key < hi ? __ldcg(reinterpret_cast<const float4*>(lg0 + (int64_t)key * G + g))
                                              : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            }
          const float l0 = lse[g], l1 = lse[g + 1], l2 = lse[g + 2], l3 = lse[g + 3];
#pragma unroll
          for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              a[u][k] += (ex2(x[u][k].x - l0) + ex2(x[u][k].y - l1)) + (ex2(x[u][k].z - l2) + ex2(x[u][k].w - l3));
        }
      } else {
        for (int g = 0; g < G; ++g) {
          const float l0 = lse[g];
#pragma unroll
          for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = base + 4 * (tid + u * threads) + k;
              if (key >= lo && key < hi) a[u][k] += ex2(__ldcg(lg0 + (int64_t)key * G + g) - l0);
            }
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int key = base + 4 * (tid + u * threads);
        if (key >= hi || !in_pool(page[u])) continue;
        float* at = score_at(page[u], off[u]);
        if (key >= lo && key + 4 <= hi) {
          red_add_v4(at, a[u][0], a[u][1], a[u][2], a[u][3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (key + k >= lo && key + k < hi) red_add(at + k, a[u][k]);
        }
      }
    }
    return;
  }
  constexpr int KU = 4;  // odd page sizes: single keys, four in flight
  for (int base = lo; base < hi; base += KU * threads) {  // block-uniform
    int page[KU], off[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const int key = base + tid + u * threads;
      page[u] = -1;
      off[u] = 0;
      if (key < hi) {
        const int pg = ps_shift >= 0 ? key >> ps_shift : key / ps;
        page[u] = __ldg(pages + pg);
        off[u] = key - pg * ps;
      }
    }
    if (!waited) ready();
    waited = true;
    float a[KU] = {0.f, 0.f, 0.f, 0.f};
    for (int g = 0; g < G; ++g) {
      const float l0 = lse[g];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int key = base + tid + u * threads;
        if (key < hi) a[u] += ex2(__ldcg(lg0 + (int64_t)key * G + g) - l0);
      }
    }
#pragma unroll
    for (int u = 0; u < KU; ++u)
      if (base + tid + u * threads < hi && in_pool(page[u])) red_add(score_at(page[u], off[u]), a[u]);
  }
}
// Scores of the unit of work item w.
__device__ __forceinline__ float* unit_logits(const RunParams& p, const WorkItem& w) {
  return p.logits + (int64_t)w.page_base * p.page_size * p.num_qo_heads + (int64_t)w.kv_head * w.kv_end * p.group;
}

// KV: the pool's pkv_dtype; NB: 8-column n-blocks; HPB: query heads per n-block, 8 or, for NVFP4, 4 in
// "pair" form (every head in two neighbouring columns, see the V product in the kernel).
template <int D, int KV, int NB, int HPB = 8>
struct DecodeCfg {
  static constexpr bool FP4 = KV == PKV_NVFP4;
  static constexpr bool PAIR = HPB == 4;
  static constexpr int ROWB = FP4 ? D / 2 : KV == PKV_FP8_E4M3 ? D : 2 * D;  // bytes per key row of one head
  static constexpr int CH = ROWB / 16;          // 16-byte chunks per row
  static constexpr int KEYS = FP4 ? 32 : 16;    // keys per warp tile
  static constexpr int SUBS = KEYS / 16;        // 16-key MMA tiles in it
  static constexpr int TILE_B = KEYS * ROWB;    // bytes of one K (or V) tile
  static constexpr int SF_B = FP4 ? KEYS * D / 16 : 0;    // bytes of the block scales of one K (or V) tile
  static constexpr int STAGE_B = 2 * TILE_B + 2 * SF_B;  // K, V, K scales, V scales
  static constexpr int HEADS = HPB * NB;        // query heads per CTA (n dimension)
  static constexpr int STAGES = FP4 ? 2 : 3;   // (NVFP4: 2 x 131072 keys 57.8 us with 3, 56.6 to 57.4 with 2)
  static constexpr int WARPS = 4;
  // resident CTAs per SM: the 8-KB-per-stage bf16/D128 variant fits 2 (shared memory), the 4-KB
  // variants fit 4 when the accumulators are for 8 heads (registers)
  static constexpr int CTAS = (2 * TILE_B > 4096 || (NB > 1 && !PAIR)) ? 2 : 4;
  static constexpr int WARP_SMEM = STAGES * STAGE_B;
  static constexpr int PIPE_SMEM = WARPS * WARP_SMEM;
  static constexpr int MERGE_SMEM = (WARPS * HEADS * D + 3 * WARPS * HEADS) * 4;
  static constexpr int SMEM = PIPE_SMEM > MERGE_SMEM ? PIPE_SMEM : MERGE_SMEM;
  static constexpr int MB = PAIR ? D / 32 : D / 16;  // 16-row m-blocks of O^T (rows: dims, or pairs of dims)
  static_assert(!PAIR || FP4, "the pair form is for 4-bit codes");
  static constexpr int KS = D / 16;  // k-steps of S^T
  static_assert(CH >= 8 || CH == 4, "the XOR swizzles below are for rows of 4 or at least 8 chunks");
  static_assert(SMEM * CTAS <= 232448, "shared memory per SM");
  // Byte offset of 16-byte chunk c of a tile's row.  The 8 rows one ldmatrix phase reads at the same
  // chunk must fall in 8 different 16-byte columns of the 128-byte bank line: a row of 8 or more chunks
  // is XORed with its row number; of 4-chunk rows two share a line, so pairs of rows are XORed.
  static __device__ __forceinline__ int at(int row, int c) {
    return row * ROWB + ((CH == 4 ? c ^ ((row >> 1) & 3) : c ^ (row & 7)) << 4);
  }
};

// Head-dim index of accumulator element j (0..3) of O^T m-block mb, lane row g.
template <int KV>
__device__ __forceinline__ int o_dim(int mb, int j, int g) {
  if constexpr (KV == PKV_BF16) {
    return mb * 16 + g + 8 * (j >> 1);
  } else if constexpr (KV == PKV_NVFP4) {
    // m-block mb = 2 q + half of the 32-dim chunk q: rows g -> dims 32 q + 4 g + 2 half, rows g + 8 -> the next dim
    return (mb >> 1) * 32 + 4 * g + 2 * (mb & 1) + (j >> 1);
  } else {
    // m-block mb = 2 q + parity: rows g -> dims 32 q + 2 g + parity, rows g + 8 -> 32 q + 16 + 2 g + parity
    return (mb >> 1) * 32 + 16 * (j >> 1) + 2 * g + (mb & 1);
  }
}

// acc[k] += sum over the ns partials of weight(partial, row of column k) * partial[column k], for
// the NC float4 columns col[k] < n4 of this thread, U partial reads per column in flight.
template <int NC, int U, int HEADS, int NA>
__device__ __forceinline__ void merge_accumulate(float4 (&acc)[NA], const int (&col)[NA], const int (&crow)[NA], int n4,
                                                 const float4* base, int ns, const float* wgt, int slot4) {
  int sp = 0;
  for (; sp + U <= ns; sp += U) {
    float4 x[U][NC];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < NC; ++k)
        x[u][k] = col[k] < n4 ? __ldcg(base + (int64_t)(sp + u) * slot4 + col[k]) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const float wv = wgt[(sp + u) * HEADS + (col[k] < n4 ? crow[k] : 0)];
        acc[k].x += wv * x[u][k].x;
        acc[k].y += wv * x[u][k].y;
        acc[k].z += wv * x[u][k].z;
        acc[k].w += wv * x[u][k].w;
      }
  }
  for (; sp < ns; ++sp) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      if (col[k] < n4) {
        const float4 x = __ldcg(base + (int64_t)sp * slot4 + col[k]);
        const float wv = wgt[sp * HEADS + crow[k]];
        acc[k].x += wv * x.x;
        acc[k].y += wv * x.y;
        acc[k].z += wv * x.z;
        acc[k].w += wv * x.w;
      }
    }
  }
}

// SCORED: every visible key's scaled score (log2 units) goes to p.logits, each row's log2-sum-exp to
// p.lse2 (for the accumulated attention weights, decode_scored.cu).
template <int D, int KV, int NB, int HPB, bool SCORED>
__global__ void __launch_bounds__(128, DecodeCfg<D, KV, NB, HPB>::CTAS) decode_kernel(const RunParams p, int32_t* err) {
  using C = DecodeCfg<D, KV, NB, HPB>;
  constexpr bool FP4 = KV == PKV_NVFP4;
  constexpr bool PAIR = C::PAIR;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_stage_key[C::WARPS][C::STAGES];

  pdl_wait();  // the plan's metadata copy and the KV write before this run must be complete
  const WorkItem w = p.work[blockIdx.x];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2;
  const int t = lane & 3;
  const int qh0 = w.kv_head * p.group + w.head_group * kDecodeRows;
  const int rows = min(C::HEADS, p.group - w.head_group * kDecodeRows);

  // ---- Q^T fragments (B operand: k = head dim, n = query head g of each n-block) ----
  uint32_t qb[C::KS][NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int head = PAIR ? nb * 4 + (g >> 1) : nb * 8 + g;
    const bool valid = head < rows;
    const uint16_t* qr = static_cast<const uint16_t*>(p.q) + ((int64_t)w.q_row * p.num_qo_heads + qh0 + head) * D;
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
      if constexpr (KV == PKV_BF16) {
        qb[ks][nb][0] = valid ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * t) : 0u;
        qb[ks][nb][1] = valid ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 8 + 2 * t) : 0u;
      } else {
        // permuted order: logical k {2t, 2t+1} <- dims 16ks+4t+{0,1}; {2t+8, 2t+9} <- 16ks+4t+{2,3}
        // (raw bf16 pairs here; widened to f16 below)
        // (NVFP4: a lane's ldmatrix register holds 8 codes, so k-step 2c + h takes dims 32c + 8t + 4h + 0..3)
        const int d0 = FP4 ? (ks >> 1) * 32 + 8 * t + 4 * (ks & 1) : ks * 16 + 4 * t;
        const uint2 x = valid ? *reinterpret_cast<const uint2*>(qr + d0) : make_uint2(0, 0);
        qb[ks][nb][0] = x.x;
        qb[ks][nb][1] = x.y;
      }
    }
  }
  // ---- per-warp cp.async ring ----
  uint8_t* wsm = smem + warp * C::WARP_SMEM;
  const uint32_t wsm_u = smem_u32(wsm);
  const int lr = lane & (C::KEYS - 1);  // row whose page this lane resolves
  const int64_t head_off = (int64_t)w.kv_head * p.stride_head_b;
  const int64_t sf_head = FP4 ? (int64_t)w.kv_head * p.sf_head_b : 0;
  const uint64_t kv_policy = l2_evict_first();

  // Lane lr (0..15, NVFP4: 0..31) resolves the page of row lr of a tile; then every warp-wide cp.async covers
  // 32 / CH whole rows with consecutive lanes on consecutive 16-byte chunks (fully coalesced).
  constexpr int RPI = 32 / C::CH;  // rows per warp instruction
  const int lc = lane % C::CH;
  const int lsub = lane / C::CH;
  const int ps = p.page_size;
  const int ps_shift = (ps & (ps - 1)) == 0 ? __ffs(ps) - 1 : -1;  // page sizes are usually powers of 2
  auto page_of = [&](int key) -> int { return ps_shift >= 0 ? key >> ps_shift : key / ps; };
  // NVFP4: tiles start on multiples of 16, pages are a power of two and hold whole 16-key halves, and the
  // byte strides fit 32 bits; narrow: so do all offsets into the pools
  const bool halves_paged = FP4 && ps_shift >= 4 && (w.kv_begin & 15) == 0 &&
                            ((p.stride_page_b | p.stride_token_b | p.sf_page_b | p.sf_token_b) >> 32) == 0;
  const bool narrow =
      halves_paged && ((p.num_pages | p.stride_head_b | p.sf_head_b) >> 31) == 0 &&
      ((p.num_pages * p.stride_page_b + ps * p.stride_token_b + p.num_kv_heads * p.stride_head_b) >> 32) == 0 &&
      ((p.num_pages * p.sf_page_b + ps * p.sf_token_b + p.num_kv_heads * p.sf_head_b) >> 32) == 0;
  const unsigned pool_pages = (unsigned)min(p.num_pages, (int64_t)0x7fffffff);  // (a page id is a non-negative int)
  const int64_t lane_off = head_off + (int64_t)lsub * p.stride_token_b + lc * 16;
  const int lane_sw = C::at(lsub, lc);
  const int64_t row_step = (int64_t)RPI * p.stride_token_b;  // bytes between the rows of consecutive instructions

  // ---- the warp's tile sequence ----
  // Alone on its range (num_splits == 1) a warp takes every 4th 16-key tile.  When num_splits CTAs
  // share the range, it is cut into 32-key groups: warp w of split s starts on group 4 s + w and
  // then claims group 4 num_splits + atomicAdd(claim, 1), and so on, until the groups run out (so
  // the warps of all the CTAs end within about one group of each other).  The claim for the next
  // group is sent when the warp starts loading a group, 2 tiles before it is needed.  A key >=
  // kv_end ends the sequence.
  constexpr int GROUP_KEYS = 2 * C::KEYS;  // (NVFP4: 64-key groups of two 32-key tiles)
  const bool shared_range = w.num_splits > 1;
  const int claim_base = w.num_splits * C::WARPS;
  int pending = 0;  // lane 0: value returned by the outstanding claim
  if (shared_range && lane == 0) pending = atomicAdd(p.claim + w.unit * kClaimStride, 1);
  auto next_key = [&](int k) -> int {  // first key of the tile after the one starting at k (k < kv_end)
    if (!shared_range) return k + C::WARPS * C::KEYS;
    if (((k - w.kv_begin) & (GROUP_KEYS - 1)) != GROUP_KEYS - C::KEYS) return k + C::KEYS;
    const int grp = claim_base + __shfl_sync(0xffffffffu, pending, 0);
    const int nk = grp < (w.kv_end - w.kv_begin + GROUP_KEYS - 1) / GROUP_KEYS ? w.kv_begin + grp * GROUP_KEYS : w.kv_end;
    if (nk < w.kv_end && lane == 0) pending = atomicAdd(p.claim + w.unit * kClaimStride, 1);
    return nk;
  };
  int lkey = w.kv_begin + (shared_range ? (w.split * C::WARPS + warp) * GROUP_KEYS : warp * C::KEYS);
  lkey = min(lkey, w.kv_end);
  int nkey = lkey < w.kv_end ? next_key(lkey) : w.kv_end;
  int* key_of_stage = s_stage_key[warp];  // first key of the tile in each ring stage (kv_end: none)

  // The page id of the row this lane resolves is fetched one tile ahead, so the index load never
  // stalls the issue of the copies.
  auto fetch_page = [&](int key) -> int {
    return key < w.kv_end ? __ldg(p.kv_indices + w.page_base + page_of(key)) : 0;
  };
  int next_page = fetch_page(lkey + lr);
  // Load the tile starting at lkey into `stage` and advance the sequence.
  auto load_tile = [&](int stage) {
    const int key0 = lkey;
    const int key = key0 + lr;
    const int page = next_page;
    next_page = fetch_page(nkey + lr);
    lkey = nkey;
    nkey = nkey < w.kv_end ? next_key(nkey) : w.kv_end;
    const uint32_t dk = wsm_u + stage * C::STAGE_B;
    const uint32_t dv = dk + C::TILE_B;
    if constexpr (FP4) {
      // Common case: all 32 keys present and each half of them on one page (whole 16-key halves per page:
      // halves_paged), so the row addresses follow from two pages and a stride.
      const bool in_pool = (unsigned)page < pool_pages;
      if (halves_paged && key0 + C::KEYS <= w.kv_end && __all_sync(0xffffffffu, in_pool)) {
        auto issue = [&](auto zero) {
          using O = decltype(zero);  // of the offsets
          const unsigned off = (unsigned)(key0 + lr) & (unsigned)(ps - 1);  // of this lane's row
          const O srow = (O)(unsigned)page * (unsigned)p.sf_page_b + (O)off * (unsigned)p.sf_token_b + (O)sf_head;
          cp_async8(dv + C::TILE_B + lane * 8, p.k_sf + srow, 8u);
          cp_async8(dv + C::TILE_B + C::SF_B + lane * 8, p.v_sf + srow, 8u);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const unsigned hp = __shfl_sync(0xffffffffu, page, 16 * hf), ho = (unsigned)(key0 + 16 * hf) & (unsigned)(ps - 1);
            const O base = (O)hp * (unsigned)p.stride_page_b + (O)ho * (unsigned)p.stride_token_b + (O)lane_off;
#pragma unroll
            for (int j = 0; j < 16 / RPI; ++j) {
              const O at = base + (O)j * (O)row_step;  // (the step may pass 2^32 where a token's stride does not)
              cp_async16_pol(dk + lane_sw + (16 * hf + j * RPI) * C::ROWB, p.k_pool + at, 16u, kv_policy);
              cp_async16_pol(dv + lane_sw + (16 * hf + j * RPI) * C::ROWB, p.v_pool + at, 16u, kv_policy);
            }
          }
        };
        if (narrow) issue((uint32_t)0);
        else issue((uint64_t)0);
        return;
      }
    } else {
    // Common case: all 16 keys present and on one page (page size >= 16, chunk starts aligned), so
    // every lane has the same page id and the row addresses follow from one base and a stride.
    const bool one_page = key0 + C::KEYS <= w.kv_end && page_of(key0) == page_of(key0 + C::KEYS - 1) &&
                          (unsigned long long)(unsigned)page < (unsigned long long)p.num_pages;
    if (__all_sync(0xffffffffu, one_page)) {
      const int off0 = key0 - page_of(key0) * ps;
      const int64_t base = (int64_t)page * p.stride_page_b + (int64_t)(off0 + lsub) * p.stride_token_b + head_off + lc * 16;
      const char* ks = p.k_pool + base;
      const char* vs = p.v_pool + base;
#pragma unroll
      for (int j = 0; j < C::KEYS / RPI; ++j) {
        const int row = j * RPI + lsub;
        const uint32_t sw = C::at(row, lc);
        cp_async16_pol(dk + sw, ks + j * row_step, 16u, kv_policy);
        cp_async16_pol(dv + sw, vs + j * row_step, 16u, kv_policy);
      }
      return;
    }
    }
    int64_t roff = -1, soff = -1;
    if (key < w.kv_end) {
      const int off = key - page_of(key) * ps;
      if ((unsigned long long)(unsigned)page >= (unsigned long long)p.num_pages)
        record_error(err, PKV_DEVERR_PAGE_RANGE);
      else
        roff = (int64_t)page * p.stride_page_b + (int64_t)off * p.stride_token_b + head_off;
      if constexpr (FP4)
        if (roff >= 0) soff = (int64_t)page * p.sf_page_b + (int64_t)off * p.sf_token_b + sf_head;
    }
    if constexpr (FP4) {
      cp_async8(dv + C::TILE_B + lane * 8, soff >= 0 ? p.k_sf + soff : p.k_sf, soff >= 0 ? 8u : 0u);
      cp_async8(dv + C::TILE_B + C::SF_B + lane * 8, soff >= 0 ? p.v_sf + soff : p.v_sf, soff >= 0 ? 8u : 0u);
    }
#pragma unroll
    for (int j = 0; j < C::KEYS / RPI; ++j) {
      const int row = j * RPI + lsub;
      const int64_t o = __shfl_sync(0xffffffffu, roff, row);
      const uint32_t sw = C::at(row, lc);
      const bool ok = o >= 0;
      cp_async16_pol(dk + sw, ok ? p.k_pool + o + lc * 16 : p.k_pool, ok ? 16u : 0u, kv_policy);
      cp_async16_pol(dv + sw, ok ? p.v_pool + o + lc * 16 : p.v_pool, ok ? 16u : 0u, kv_policy);
    }
  };

  float m[NB][2], l[NB][2];  // per head column 2t, 2t+1: reference max (log2 units) and this lane's sum
  float o[C::MB][NB][4];     // O^T: rows = head dims, columns = heads
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb][0] = m[nb][1] = -INFINITY;
    l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb) o[mb][nb][0] = o[mb][nb][1] = o[mb][nb][2] = o[mb][nb][3] = 0.f;
  }

  int cur = 0;  // two stages (NVFP4): first key of the tile that was loaded last, in every lane
  static_assert(!FP4 || C::STAGES == 2, "`cur` holds one tile");
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) {
    if constexpr (FP4) cur = lkey;
    else if (lane == 0) key_of_stage[s] = lkey;
    if (lkey < w.kv_end) load_tile(s);
    cp_async_commit();
  }

  // (Done here, after the first tiles' copies are issued, so the Q loads overlap them.)
  // FP8 and NVFP4 KV run the products in f16, whose largest finite value is 65504: a larger |q| would become
  // inf.  The CTA's Q rows are scaled by 2^-e, with e the smallest power that brings max |q| below
  // 2^15, and the score scale is multiplied by 2^e.  The scaling is exact (a bf16 value inside the f16
  // normal range is an f16 value; down to 2^-28 of the CTA's max |q|; smaller ones are off by at most
  // 2^-39 of it), and for FP8 e = 0 whenever max |q| < 2^15.
  float sc = p.scale_log2;
  if constexpr (KV != PKV_BF16) {
    // largest finite |q| as bf16 magnitude bits (monotonic in the value); an infinity or a NaN counts as 0, so
    // that it does not cost the CTA's other heads their bits (a power per head would need a score scale
    // per column: 64 requests of 512-4096 keys 41.3 us against 39.5, NVFP4)
    uint32_t amax = 0;
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t r = qb[ks][nb][h];
          const uint32_t lo = r & 0x7fffu, hi = (r >> 16) & 0x7fffu;
          amax = max(amax, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
    amax = __reduce_max_sync(0xffffffffu, amax);  // every warp holds the CTA's whole Q
    // (NVFP4: small rows are scaled up too, so that a small q against a pool of large scale keeps its
    // bits; where the score scale underflows with it, the scores are 0 to float32 anyway)
    const int top = (int)(amax >> 7) - 127 - 14;    // bf16 exponent field -> floor(log2 max |q|), less 14
    const int e = FP4 ? max(-126, top) : max(0, top);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e (e <= 114: a normal float)
    sc *= __uint_as_float((uint32_t)(127 + e) << 23);              // 2^e
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t r = qb[ks][nb][h];
          qb[ks][nb][h] = pack_f16(__uint_as_float(r << 16) * down, __uint_as_float(r & 0xffff0000u) * down);
        }
  }

  // ldmatrix lane roles: K as the A operand (rows = keys), V^T as the A operand (.trans, rows = dims)
  const int mi = lane >> 3, rr = lane & 7;
  const int k_key = ((mi & 1) << 3) + rr;  // matrices: (keys 0-7, c), (keys 8-15, c), (keys 0-7, c+1), (8-15, c+1)
  const int v_key = ((mi >> 1) << 3) + rr; // matrices: (keys 0-7, c), (keys 0-7, c+1), (keys 8-15, c), (8-15, c+1)

  // SCORED: the unit's scores, [key][query head of the KV head], in a region of the request's pages' size
  float* logits = nullptr;
  const bool pair_rows = (p.group & 1) == 0;
  if constexpr (SCORED)
    logits = unit_logits(p, w) + w.head_group * kDecodeRows;

  int stage = 0, fill = C::STAGES - 1;  // ring slot of the tile computed now and of the one loaded now
  while (true) {
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();
    const int key0 = FP4 ? cur : key_of_stage[stage];
    if (key0 >= w.kv_end) break;
    // refill the stage the previous tile used before computing this one, so STAGES-1 tiles stay
    // in flight during the compute
    if constexpr (FP4) cur = lkey;
    else if (lane == 0) key_of_stage[fill] = lkey;
    if (lkey < w.kv_end) load_tile(fill);
    cp_async_commit();
    fill = fill + 1 == C::STAGES ? 0 : fill + 1;
    const uint32_t kb = wsm_u + stage * C::STAGE_B;
    const uint32_t vb = kb + C::TILE_B;
    const uint8_t* sfs = wsm + stage * C::STAGE_B + 2 * C::TILE_B;  // block scales of the K rows, then the V rows
    stage = stage + 1 == C::STAGES ? 0 : stage + 1;

    // ---- S^T = K Q^T for 16 keys (NVFP4: twice 16) ----
    float s[C::SUBS][NB][4];
#pragma unroll
    for (int su = 0; su < C::SUBS; ++su)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) s[su][nb][0] = s[su][nb][1] = s[su][nb][2] = s[su][nb][3] = 0.f;
    if constexpr (KV == PKV_BF16) {
#pragma unroll
      for (int ks = 0; ks < C::KS; ++ks) {
        uint32_t a[4];
        const int chunk = 2 * ks + (mi >> 1);
        ldsm_x4(a, kb + C::at(k_key, chunk));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_bf16(s[0][nb], a, qb[ks][nb][0], qb[ks][nb][1]);
      }
    } else if constexpr (FP4) {
      // This lane's codes of chunk c (8t .. 8t+7 of its 32) lie in block 2c + (t >> 1): one scale per
      // (key row, chunk), here for key rows g and g + 8
      const uint32_t sel = t < 2 ? 0x6420u : 0x7531u;
#pragma unroll
      for (int su = 0; su < C::SUBS; ++su) {
        const uint2 f0 = *reinterpret_cast<const uint2*>(sfs + (16 * su + g) * 8);
        const uint2 f1 = *reinterpret_cast<const uint2*>(sfs + (16 * su + g + 8) * 8);
        uint32_t sg[2][2];  // [key row][chunk pair], f16x2
        e4m3x4_to_f16x2x2(__byte_perm(f0.x, f0.y, sel), sg[0][0], sg[0][1]);
        e4m3x4_to_f16x2x2(__byte_perm(f1.x, f1.y, sel), sg[1][0], sg[1][1]);
#pragma unroll
        for (int c = 0; c < C::CH; c += 2) {
          uint32_t r[4];
          const int chunk = c + (mi >> 1);
          ldsm_x4(r, kb + C::at(16 * su + k_key, chunk));
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // r[2h]: key g, chunk c + h; r[2h + 1]: key g + 8
            uint32_t x[4], y[4];
            e2m1x8_to_f16x2x4(r[2 * h], x);
            e2m1x8_to_f16x2x4(r[2 * h + 1], y);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a[4] = {hmul2_by(x[2 * k], sg[0][c >> 1], h), hmul2_by(y[2 * k], sg[1][c >> 1], h),
                                     hmul2_by(x[2 * k + 1], sg[0][c >> 1], h), hmul2_by(y[2 * k + 1], sg[1][c >> 1], h)};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma_f16(s[su][nb], a, qb[2 * (c + h) + k][nb][0], qb[2 * (c + h) + k][nb][1]);
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < C::KS; c += 2) {
        uint32_t r[4];
        const int chunk = c + (mi >> 1);
        ldsm_x4(r, kb + C::at(k_key, chunk));
        // r[0]: keys 0-7 / chunk c, r[1]: keys 8-15 / chunk c, r[2], r[3]: chunk c + 1; the low
        // code pair of each register feeds k-step c + h's first half, the high pair its second
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a[4];
          e4m3x4_to_f16x2x2(r[2 * h], a[0], a[2]);
          e4m3x4_to_f16x2x2(r[2 * h + 1], a[1], a[3]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_f16(s[0][nb], a, qb[c + h][nb][0], qb[c + h][nb][1]);
        }
      }
    }

    // ---- online softmax per head column (log2 domain) ----
    // The reference max m moves only when a column's tile max exceeds it by more than 2^8 (one
    // warp-wide decision), so most tiles skip the O rescale; probabilities stay below 2^8.
    const bool full = key0 + C::KEYS <= w.kv_end;
    uint32_t pb[C::SUBS][NB][2];
    // per head column: scaled scores of keys 16 su + g, 16 su + g + 8 (NCOL = 1: columns 2t and 2t + 1 hold
    // the same head, one of them is enough)
    constexpr int NCOL = PAIR ? 1 : 2;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float x[C::SUBS][2][NCOL];
#pragma unroll
      for (int su = 0; su < C::SUBS; ++su) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int k = 0; k < NCOL; ++k) x[su][r][k] = s[su][nb][2 * r + k] * sc;
        const int kl = key0 + 16 * su + g;
        const bool lo_ok = full || kl < w.kv_end, hi_ok = full || kl + 8 < w.kv_end;
        if constexpr (SCORED) {
          // [key][query head of the group]
          const int head = PAIR ? nb * 4 + t : nb * 8 + 2 * t;
          float* lg = logits + (int64_t)kl * p.group + head;
          if (!PAIR && pair_rows) {  // two heads at once: every row of heads starts on 8 bytes
            if (head < rows) {
              if (lo_ok) *reinterpret_cast<float2*>(lg) = make_float2(x[su][0][0], x[su][0][NCOL - 1]);
              if (hi_ok) *reinterpret_cast<float2*>(lg + 8 * p.group) = make_float2(x[su][1][0], x[su][1][NCOL - 1]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < NCOL; ++k) {
              if (lo_ok && head + k < rows) lg[k] = x[su][0][k];
              if (hi_ok && head + k < rows) lg[8 * p.group + k] = x[su][1][k];
            }
          }
        }
        if (!full) {
#pragma unroll
          for (int k = 0; k < NCOL; ++k) {
            x[su][0][k] = lo_ok ? x[su][0][k] : -INFINITY;
            x[su][1][k] = hi_ok ? x[su][1][k] : -INFINITY;
          }
        }
      }
      float mx[NCOL];
#pragma unroll
      for (int k = 0; k < NCOL; ++k) {
        mx[k] = fmaxf(x[0][0][k], x[0][1][k]);
        if constexpr (C::SUBS == 2) mx[k] = fmax3(mx[k], x[1][0][k], x[1][1][k]);
      }
      // (A column's lanes hold the same m, so the vote over each lane's own keys decides for the column; its
      // maximum over the lanes is formed only where m moves.)
      if (__any_sync(0xffffffffu, mx[0] > m[nb][0] + 8.f || mx[NCOL - 1] > m[nb][NCOL - 1] + 8.f)) {
        // every tile holds at least one visible key, so the tile maxima are finite
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1)
#pragma unroll
          for (int k = 0; k < NCOL; ++k) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], sh));
        float cf[NCOL];
#pragma unroll
        for (int k = 0; k < NCOL; ++k) {
          const float mn = fmaxf(m[nb][k], mx[k]);
          cf[k] = ex2(m[nb][k] - mn);
          m[nb][k] = mn;
          l[nb][k] *= cf[k];
        }
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[mb][nb][j] *= cf[PAIR ? 0 : (j & 1)];
      }
#pragma unroll
      for (int su = 0; su < C::SUBS; ++su) {
#pragma unroll
        for (int k = 0; k < NCOL; ++k) {
          x[su][0][k] = ex2(x[su][0][k] - m[nb][k]);
          x[su][1][k] = ex2(x[su][1][k] - m[nb][k]);
          l[nb][k] += x[su][0][k] + x[su][1][k];
        }
        // P^T in accumulator layout (row = key, column pair = heads) -> B operand (k = keys, n = head)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (KV == PKV_BF16)
            pb[su][nb][r] = movmatrix_trans(pack_bf16(x[su][r][0], x[su][r][NCOL - 1]));
          else
            pb[su][nb][r] = movmatrix_trans(pack_f16(x[su][r][0], x[su][r][NCOL - 1]));
        }
      }
    }

    // ---- O^T += V^T P^T ----
    if constexpr (PAIR) {
      // A byte holds two neighbouring dims of one key, and an A operand register wants two values that are
      // neighbours in k.  So k runs over (key, parity of the dim): the A rows are pairs of dims, the 8
      // columns are (head, parity), and B[(key, parity), (head, parity')] is P where the parities agree and
      // 0 elsewhere.  One ldmatrix.trans register (key 2t: dims 4g .. 4g+3, key 2t + 1: the same) is then
      // the A fragment of a whole 8-key x 32-dim MMA, byte by byte, with no bit of it moved; half of the
      // tensor work is spent on zeros, which 4 heads in 8 columns would leave idle anyway.
      const uint32_t sel = g < 4 ? 0x6420u : 0x7531u;
#pragma unroll
      for (int su = 0; su < C::SUBS; ++su) {
        uint32_t sv[2][2][2];   // [keys 0-7 | 8-15][key 2t | 2t + 1][chunk pair], f16x2
        uint32_t bb[NB][2][2];  // [..][keys 0-7 | 8-15][key 2t | 2t + 1]: (P, 0) in even columns, (0, P) in odd ones
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 f = *reinterpret_cast<const uint4*>(sfs + C::SF_B + (16 * su + 2 * t + 8 * h) * 8);
          e4m3x4_to_f16x2x2(__byte_perm(f.x, f.y, sel), sv[h][0][0], sv[h][0][1]);
          e4m3x4_to_f16x2x2(__byte_perm(f.z, f.w, sel), sv[h][1][0], sv[h][1][1]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            bb[nb][h][0] = __byte_perm(pb[su][nb][h], 0, (g & 1) ? 0x1044u : 0x4410u);
            bb[nb][h][1] = __byte_perm(pb[su][nb][h], 0, (g & 1) ? 0x3244u : 0x4432u);
          }
        }
#pragma unroll
        for (int c = 0; c < C::CH; c += 2) {
          uint32_t r[4];
          const int chunk = c + (mi & 1);
          ldsm_x4_t(r, vb + C::at(16 * su + v_key, chunk));  // r[2h + u]: keys 8h + 0-7, chunk c + u
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t x[4];
              e2m1x8_to_f16x2x4(r[2 * h + u], x);
              const uint32_t s0 = sv[h][0][c >> 1], s1 = sv[h][1][c >> 1];
              const uint32_t a[4] = {hmul2_by(x[0], s0, u), hmul2_by(x[1], s0, u), hmul2_by(x[2], s1, u), hmul2_by(x[3], s1, u)};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_f16(o[c + u][nb], a, bb[nb][h][0], bb[nb][h][1]);
            }
        }
      }
    } else if constexpr (FP4) {
      // The codes of this lane's ldmatrix.trans register (dims 4g .. 4g+3 of a 32-dim chunk, keys 2t and
      // 2t + 1) lie in block 2 chunk + (g >> 2).  Its scale differs between the two keys, and so does the
      // f16x2 of one dim: the pair of scales multiplies the pair of values.
      const uint32_t sel = g < 4 ? 0x6420u : 0x7531u;
#pragma unroll
      for (int su = 0; su < C::SUBS; ++su) {
        uint32_t sv[2][C::CH];  // [keys 2t, 2t+1 | keys 2t+8, 2t+9][chunk], f16x2 (one key per half)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 f = *reinterpret_cast<const uint4*>(sfs + C::SF_B + (16 * su + 2 * t + 8 * h) * 8);
          const uint32_t fa = __byte_perm(f.x, f.y, sel), fb = __byte_perm(f.z, f.w, sel);
          e4m3x4_to_f16x2x2(__byte_perm(fa, fb, 0x5140u), sv[h][0], sv[h][1]);
          e4m3x4_to_f16x2x2(__byte_perm(fa, fb, 0x7362u), sv[h][2], sv[h][3]);
        }
#pragma unroll
        for (int c = 0; c < C::CH; c += 2) {
          uint32_t r[4];
          const int chunk = c + (mi & 1);
          ldsm_x4_t(r, vb + C::at(16 * su + v_key, chunk));
          // r[u]: keys 2t (low half), 2t + 1 (high half) x dims 4g .. 4g+3 of chunk c + u; r[2 + u]: keys + 8
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t x[4], y[4];
            e2m1_2x4_to_f16x2x4(r[u], x);
            e2m1_2x4_to_f16x2x4(r[2 + u], y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = hmul2(x[k], sv[0][c + u]);
              y[k] = hmul2(y[k], sv[1][c + u]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a[4] = {x[2 * k], x[2 * k + 1], y[2 * k], y[2 * k + 1]};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_f16(o[2 * (c + u) + k][nb], a, pb[su][nb][0], pb[su][nb][1]);
            }
          }
        }
      }
    } else if constexpr (KV == PKV_BF16) {
#pragma unroll
      for (int mb = 0; mb < C::MB; ++mb) {
        uint32_t a[4];
        const int chunk = 2 * mb + (mi & 1);
        ldsm_x4_t(a, vb + C::at(v_key, chunk));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_bf16(o[mb][nb], a, pb[0][nb][0], pb[0][nb][1]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < D / 16; c += 2) {
        uint32_t r[4];
        const int chunk = c + (mi & 1);
        ldsm_x4_t(r, vb + C::at(v_key, chunk));
        // r[0]: keys 0-7 x chunk c, r[1]: keys 0-7 x chunk c+1, r[2]: keys 8-15 x chunk c,
        // r[3]: keys 8-15 x chunk c+1.  Each register holds, for byte-pair column g:
        // (key 2t: d, d+1), (key 2t+1: d, d+1) with d = 16 chunk + 2g; bytes 0/2 are the even dim,
        // bytes 1/3 the odd one.  One byte permute puts the even pair in the low half and the odd
        // pair in the high half.
        uint32_t ev[4], od[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e4m3x4_to_f16x2x2(__byte_perm(r[k], 0, 0x3120u), ev[k], od[k]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          mma_f16(o[c][nb], ev, pb[0][nb][0], pb[0][nb][1]);
          mma_f16(o[c + 1][nb], od, pb[0][nb][0], pb[0][nb][1]);
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();

  // full per-head sums across the 8 key rows g of the warp
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
      l[nb][0] += __shfl_xor_sync(0xffffffffu, l[nb][0], sh);
      l[nb][1] += __shfl_xor_sync(0xffffffffu, l[nb][1], sh);
    }
  }

  // ---- merge the 4 warps' states through shared memory ----
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);   // [4][HEADS][D]
  float* sm = so + C::WARPS * C::HEADS * D;     // [4][HEADS]
  float* sl = sm + C::WARPS * C::HEADS;         // [4][HEADS]
  float* sf = sl + C::WARPS * C::HEADS;         // [4][HEADS] weights
  if (g == 0) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if constexpr (PAIR) {
        sm[warp * C::HEADS + nb * 4 + t] = m[nb][0];
        sl[warp * C::HEADS + nb * 4 + t] = l[nb][0];
      } else {
        sm[warp * C::HEADS + nb * 8 + 2 * t] = m[nb][0];
        sm[warp * C::HEADS + nb * 8 + 2 * t + 1] = m[nb][1];
        sl[warp * C::HEADS + nb * 8 + 2 * t] = l[nb][0];
        sl[warp * C::HEADS + nb * 8 + 2 * t + 1] = l[nb][1];
      }
    }
  }
#pragma unroll
  for (int mb = 0; mb < C::MB; ++mb) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if constexpr (PAIR) {  // rows g, g + 8 x columns 2t, 2t + 1: dims 4g .. 4g+3 of chunk mb, head t
        if (nb * 4 + t < rows)
          *reinterpret_cast<float4*>(so + (warp * C::HEADS + nb * 4 + t) * D + mb * 32 + 4 * g) =
              make_float4(o[mb][nb][0], o[mb][nb][1], o[mb][nb][2], o[mb][nb][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int head = nb * 8 + 2 * t + (j & 1);
          if (head < rows) so[(warp * C::HEADS + head) * D + o_dim<KV>(mb, j, g)] = o[mb][nb][j];
        }
      }
    }
  }
  __syncthreads();
  __shared__ float s_lse2[C::HEADS];
  if (threadIdx.x < C::HEADS) {
    const int r = threadIdx.x;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < C::WARPS; ++k) M = fmaxf(M, sm[k * C::HEADS + r]);
    float W = 0.f;
    float e[C::WARPS];
#pragma unroll
    for (int k = 0; k < C::WARPS; ++k) {
      e[k] = ex2(sm[k * C::HEADS + r] - M);  // a warp without tiles has m = -inf: weight 0
      W += e[k] * sl[k * C::HEADS + r];
    }
    const float inv = W > 0.f ? 1.f / W : 0.f;
#pragma unroll
    for (int k = 0; k < C::WARPS; ++k) sf[k * C::HEADS + r] = e[k] * inv;
    s_lse2[r] = M + __log2f(W);
  }
  __syncthreads();
  if (w.out_slot < 0) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + ((int64_t)w.q_row * p.num_qo_heads + qh0) * D;
    for (int idx = threadIdx.x; idx < rows * D; idx += blockDim.x) {
      const int r = idx / D, d = idx - r * D;
      float acc = 0.f;
#pragma unroll
      for (int k = 0; k < C::WARPS; ++k) acc += sf[k * C::HEADS + r] * so[(k * C::HEADS + r) * D + d];
      out[idx] = __float2bfloat16_rn(acc * p.out_scale);
    }
    if (p.lse && threadIdx.x < rows)
      p.lse[(int64_t)w.q_row * p.num_qo_heads + qh0 + threadIdx.x] = s_lse2[threadIdx.x] * 0.69314718055994531f;
    if constexpr (SCORED) {
      if (p.group > kDecodeRows) {  // other CTAs hold the other query heads' sums: score_add_kernel
        if (threadIdx.x < rows) p.lse2[(int64_t)w.q_row * p.num_qo_heads + qh0 + threadIdx.x] = s_lse2[threadIdx.x];
      } else {  // every score of this unit was written by this CTA
        add_weights<(C::CTAS >= 4 ? 2 : 4)>(p, w, unit_logits(p, w), s_lse2, w.kv_begin, w.kv_end, threadIdx.x, 128, [] {});
      }
    }
  } else {
    float* po = p.part_o + (int64_t)w.out_slot * kDecodeRows * D;
    for (int idx = threadIdx.x; idx < rows * D; idx += blockDim.x) {
      const int r = idx / D, d = idx - r * D;
      float acc = 0.f;
#pragma unroll
      for (int k = 0; k < C::WARPS; ++k) acc += sf[k * C::HEADS + r] * so[(k * C::HEADS + r) * D + d];
      po[idx] = acc;
    }
    if (threadIdx.x < rows) p.part_lse[(int64_t)w.out_slot * kDecodeRows + threadIdx.x] = s_lse2[threadIdx.x];
    // The last chunk of a (request, KV head, group) to finish merges all of its partials:
    // m = max lse_s, o = sum_s 2^(lse_s - m) o_s / sum_s 2^(lse_s - m).  No CTA waits for another.
    __shared__ int s_last;
    __threadfence();
    __syncthreads();
    const int unit = w.unit;
    const MergeItem mi_ = p.merge[unit];
    if (threadIdx.x == 0) {
      const int done = atomicAdd(p.unit_count + unit, 1);
      s_last = done == mi_.num_splits - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (rows * D <= 4 * 128) {
      // One float4 column per thread (up to 4 rows of 128 dims): an online merge.  Each thread loads
      // the log2-sum-exp of its row and its column of U partials at once (as many as its registers
      // hold: 20 with 4 resident CTAs, 32 with 2) and folds them in under a running maximum, so 38
      // partials cost two dependent L2 round trips and no shared-memory staging.
      constexpr int U = C::CTAS >= 4 ? 20 : 32;
      const int ns = mi_.num_splits;
      const int n4 = rows * D / 4;
      const int col = threadIdx.x;
      const bool active = col < n4;
      const int crow = active ? col * 4 / D : 0;
      const float* lse_g = p.part_lse + (int64_t)mi_.first_slot * kDecodeRows + crow;
      const float4* pm = reinterpret_cast<const float4*>(p.part_o + (int64_t)mi_.first_slot * kDecodeRows * D) + col;
      constexpr int SLOT4 = kDecodeRows * D / 4;
      float la[U];
      float4 oa[U];
      auto fetch = [&](float (&l)[U], float4 (&o)[U], int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool in = active && s0 + u < ns;
          l[u] = in ? __ldcg(lse_g + (int64_t)(s0 + u) * kDecodeRows) : -INFINITY;
          o[u] = in ? __ldcg(pm + (int64_t)(s0 + u) * SLOT4) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      };
      float m = -INFINITY, W = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      auto fold = [&](const float (&l)[U], const float4 (&o)[U]) {
        float mb = m;
#pragma unroll
        for (int u = 0; u < U; ++u) mb = fmaxf(mb, l[u]);
        if (mb == -INFINITY) return;  // a partial without keys has lse -inf and weight 0
        const float c = ex2(m - mb);  // 0 while nothing has been seen
        W *= c;
        acc.x *= c;
        acc.y *= c;
        acc.z *= c;
        acc.w *= c;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float wv = ex2(l[u] - mb);
          W += wv;
          acc.x = fmaf(wv, o[u].x, acc.x);
          acc.y = fmaf(wv, o[u].y, acc.y);
          acc.z = fmaf(wv, o[u].z, acc.z);
          acc.w = fmaf(wv, o[u].w, acc.w);
        }
        m = mb;
      };
      for (int s0 = 0; s0 < ns; s0 += U) {
        fetch(la, oa, s0);
        fold(la, oa);
      }
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + ((int64_t)mi_.q_row * p.num_qo_heads + qh0) * D;
      if (active) {
        const float f = W > 0.f ? p.out_scale / W : 0.f;
        __nv_bfloat162* o2 = reinterpret_cast<__nv_bfloat162*>(out + col * 4);
        o2[0] = __floats2bfloat162_rn(acc.x * f, acc.y * f);
        o2[1] = __floats2bfloat162_rn(acc.z * f, acc.w * f);
        if (p.lse && (col * 4) % D == 0)  // the row's first column writes its log-sum-exp
          p.lse[(int64_t)mi_.q_row * p.num_qo_heads + qh0 + crow] = (m + __log2f(W)) * 0.69314718055994531f;
        if constexpr (SCORED)
          if ((col * 4) % D == 0) p.lse2[(int64_t)mi_.q_row * p.num_qo_heads + qh0 + crow] = m + __log2f(W);
      }
      if (threadIdx.x == 0) {  // ready for the next run of this plan
        p.unit_count[unit] = 0;
        atomicExch(p.claim + unit * kClaimStride, 0);
      }
      return;
    }
    // Online merge over chunks of splits: the chunk's log2-sum-exps are staged in shared memory by
    // all threads and turned into per-row weights 2^(lse_s - M) once, one warp per row (lanes over
    // the splits, shuffle reductions); each thread owns float4 columns of the output and keeps 8-16
    // partial reads per column in flight.  With one column per thread and one chunk (the usual
    // case) the first 8-16 partials are read before the weights are known, so that round trip
    // overlaps the staging of the log2-sum-exps.
    constexpr int V4 = C::HEADS * D / 4;            // float4s of the (at most HEADS) output rows
    constexpr int PER_T = (V4 + 127) / 128;         // float4s per thread
    constexpr int SLOT4 = kDecodeRows * D / 4;      // float4s between consecutive partials
    const int n4 = rows * D / 4;
    const int cap = C::SMEM / (4 * C::HEADS) - 2;   // splits per chunk that fit the shared scratch
    float* wgt = reinterpret_cast<float*>(smem);    // [cap][HEADS] lse, then weights
    __shared__ float sM[C::HEADS], sScale[C::HEADS], sW[C::HEADS];
    if (threadIdx.x < C::HEADS) {
      sM[threadIdx.x] = -INFINITY;
      sW[threadIdx.x] = 0.f;
    }
    float4 acc[PER_T];
    int col[PER_T], crow[PER_T];
#pragma unroll
    for (int k = 0; k < PER_T; ++k) {
      acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      col[k] = threadIdx.x + k * 128;
      crow[k] = col[k] * 4 / D;
    }
    const float* lse_g = p.part_lse + (int64_t)mi_.first_slot * kDecodeRows;
    const float4* pm = reinterpret_cast<const float4*>(p.part_o + (int64_t)mi_.first_slot * kDecodeRows * D);
    constexpr int PRE = C::CTAS >= 4 ? 8 : 16;  // registers: 4 resident CTAs leave ~128 per thread
    const int npre = (n4 <= 128 && mi_.num_splits <= cap) ? min(PRE, mi_.num_splits) : 0;
    float4 pre[PRE];
#pragma unroll
    for (int u = 0; u < PRE; ++u)
      pre[u] = (u < npre && col[0] < n4) ? __ldcg(pm + (int64_t)u * SLOT4 + col[0]) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < mi_.num_splits; s0 += cap) {
      const int ns = min(cap, mi_.num_splits - s0);
      __syncthreads();
      for (int e = threadIdx.x; e < ns * C::HEADS; e += blockDim.x) {
        const int sp = e / C::HEADS, r = e - sp * C::HEADS;
        wgt[e] = r < rows ? __ldcg(lse_g + (int64_t)(s0 + sp) * kDecodeRows + r) : -INFINITY;
      }
      __syncthreads();
      for (int r = warp; r < rows; r += C::WARPS) {
        float m = -INFINITY;
        for (int sp = lane; sp < ns; sp += 32) m = fmaxf(m, wgt[sp * C::HEADS + r]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float m_prev = sM[r];
        const float Mc = fmaxf(m_prev, m);
        const bool none = Mc == -INFINITY;              // no key seen yet: keep every weight 0
        const float sc = none ? 1.f : ex2(m_prev - Mc);  // 0 on the first chunk
        float W = 0.f;
        for (int sp = lane; sp < ns; sp += 32) {
          const float e = none ? 0.f : ex2(wgt[sp * C::HEADS + r] - Mc);
          wgt[sp * C::HEADS + r] = e;
          W += e;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
        __syncwarp();  // every lane has read sM[r] before lane 0 rewrites it
        if (lane == 0) {
          sW[r] = sW[r] * sc + W;
          sM[r] = Mc;
          sScale[r] = sc;
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < PER_T; ++k) {
        if (col[k] < n4) {
          const float sc = sScale[crow[k]];
          acc[k].x *= sc;
          acc[k].y *= sc;
          acc[k].z *= sc;
          acc[k].w *= sc;
        }
      }
      const float4* base = pm + (int64_t)s0 * SLOT4;
      if (npre > 0) {  // one chunk: the first npre partials are already in registers
        if (col[0] < n4) {
#pragma unroll
          for (int u = 0; u < PRE; ++u) {
            const float wv = u < npre ? wgt[u * C::HEADS + crow[0]] : 0.f;
            acc[0].x += wv * pre[u].x;
            acc[0].y += wv * pre[u].y;
            acc[0].z += wv * pre[u].z;
            acc[0].w += wv * pre[u].w;
          }
        }
        merge_accumulate<1, 16, C::HEADS>(acc, col, crow, n4, base + (int64_t)npre * SLOT4, ns - npre,
                                          wgt + npre * C::HEADS, SLOT4);
      } else if (n4 <= 128)  // one column per thread (up to 4 rows of 128 dims): 16 reads in flight
        merge_accumulate<1, 16, C::HEADS>(acc, col, crow, n4, base, ns, wgt, SLOT4);
      else
        merge_accumulate<PER_T, 8, C::HEADS>(acc, col, crow, n4, base, ns, wgt, SLOT4);
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + ((int64_t)mi_.q_row * p.num_qo_heads + qh0) * D;
#pragma unroll
    for (int k = 0; k < PER_T; ++k) {
      if (col[k] < n4) {
        const float W = sW[crow[k]];
        const float f = W > 0.f ? p.out_scale / W : 0.f;
        __nv_bfloat162* o2 = reinterpret_cast<__nv_bfloat162*>(out + col[k] * 4);
        o2[0] = __floats2bfloat162_rn(acc[k].x * f, acc[k].y * f);
        o2[1] = __floats2bfloat162_rn(acc[k].z * f, acc[k].w * f);
      }
    }
    if (p.lse && threadIdx.x < rows)
      p.lse[(int64_t)mi_.q_row * p.num_qo_heads + qh0 + threadIdx.x] =
          (sM[threadIdx.x] + __log2f(sW[threadIdx.x])) * 0.69314718055994531f;
    if constexpr (SCORED)
      if (threadIdx.x < rows)
        p.lse2[(int64_t)mi_.q_row * p.num_qo_heads + qh0 + threadIdx.x] = sM[threadIdx.x] + __log2f(sW[threadIdx.x]);
    if (threadIdx.x == 0) {  // ready for the next run of this plan
      p.unit_count[unit] = 0;
      atomicExch(p.claim + unit * kClaimStride, 0);
    }
  }
}

template <int D, int KV, int NB, int HPB, bool SCORED>
static cudaError_t launch_decode_t(const RunParams& p, cudaStream_t s) {
  using C = DecodeCfg<D, KV, NB, HPB>;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, KV, NB, HPB, SCORED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  int32_t* err = device_error_ptr();
  if (!err) return cudaErrorInvalidDevice;
  return launch_pdl(decode_kernel<D, KV, NB, HPB, SCORED>, dim3((unsigned)p.num_work), dim3(128), (size_t)C::SMEM, s, p, err);
}

// The instance for the pool's type, head_dim and query heads per KV head.
template <bool SCORED>
static cudaError_t launch_decode_any(const RunParams& p, int kv_dtype, cudaStream_t s) {
  const bool nb2 = p.group > 8;
  if (kv_dtype == PKV_FP8_E4M3 || kv_dtype == PKV_NVFP4) {
    if (p.head_dim != 128) return cudaErrorInvalidValue;
    // NVFP4: up to 4 query heads the pair form fills the 8 columns (4 heads: 64 requests of 512-4096 keys
    // 39.4 us against 46.7 in the 8-head form, 2 x 131072 keys 54.9 against 64.9); for 5 to 8 heads it
    // needs a second n-block and loses (8 heads: 64 requests 53.0 against 48.9, 2 x 131072 keys 75.8
    // against 69.3, 256 ragged requests 112.5 against 100.0)
    if (kv_dtype == PKV_NVFP4)
      return p.group <= 4 ? launch_decode_t<128, PKV_NVFP4, 1, 4, SCORED>(p, s)
             : !nb2       ? launch_decode_t<128, PKV_NVFP4, 1, 8, SCORED>(p, s)
                          : launch_decode_t<128, PKV_NVFP4, 2, 8, SCORED>(p, s);
    return nb2 ? launch_decode_t<128, PKV_FP8_E4M3, 2, 8, SCORED>(p, s)
               : launch_decode_t<128, PKV_FP8_E4M3, 1, 8, SCORED>(p, s);
  }
  if (p.head_dim == 128)
    return nb2 ? launch_decode_t<128, PKV_BF16, 2, 8, SCORED>(p, s) : launch_decode_t<128, PKV_BF16, 1, 8, SCORED>(p, s);
  if (p.head_dim == 64)
    return nb2 ? launch_decode_t<64, PKV_BF16, 2, 8, SCORED>(p, s) : launch_decode_t<64, PKV_BF16, 1, 8, SCORED>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace pkv
