// 8-bit bounds of the keys of each page, per KV head and channel (pkv_key_bounds_update).
//
// For page p of a request, KV head h, channel d, over the page's valid keys j, in units of s = scale[h, d]:
//   lo = clamp(floor(min_j k_jd / s), -127, 127),  hi = clamp(ceil(max_j k_jd / s), -127, 127),
// the quotients in float32.  A NaN key element gives (-127, 127), so that its page is not passed over.
//
// What bounds it: reading the keys once.  A warp takes the page of one KV head: its lanes hold 16 bytes of a row each,
// several rows to an instruction, and keep the extremes in 16-bit pairs, which is exact (bf16 as they are; E4M3
// values and E2M1 values times their block scale are f16 values), so the two divisions come after the last key.
// A call for few large pages shares a page's rows among the four warps of a CTA.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_blocks.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr int kBoundWarps = 4;

template <int KV, int D>
struct BoundCfg {
  static constexpr int ROWB = KV == PKV_NVFP4 ? D / 2 : KV == PKV_FP8_E4M3 ? D : 2 * D;
  static constexpr int LANES = ROWB / 16;                                              // per row
  static constexpr int ROWS = 32 / LANES;                                              // per warp-wide load
  static constexpr int PAIRS = KV == PKV_NVFP4 ? 16 : KV == PKV_FP8_E4M3 ? 8 : 4;  // of elements per lane
  static constexpr int UNROLL = 8;  // loads in flight: a 16-token page of bf16 rows at once
};

// minimum and maximum of 16-bit float pairs; a NaN wins
template <int KV>
__device__ __forceinline__ uint32_t pair_min(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (KV == PKV_BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int KV>
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (KV == PKV_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// the pairs (element 2 j, 2 j + 1) of a 16-byte vector of a row; sf: the block scales of its two blocks (NVFP4)
template <int KV>
__device__ __forceinline__ void widen(const uint4& x, uint32_t sf, uint32_t (&out)[BoundCfg<KV, 128>::PAIRS]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (KV == PKV_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = w[j];
  } else if constexpr (KV == PKV_FP8_E4M3) {
#pragma unroll
    for (int j = 0; j < 4; ++j) e4m3x4_to_f16x2x2(w[j], out[2 * j], out[2 * j + 1]);
  } else {
    const uint32_t s = e4m3x2_to_f16x2(sf);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t v[4];
      e2m1x8_to_f16x2x4(w[j], v);
#pragma unroll
      for (int k = 0; k < 4; ++k) out[4 * j + k] = hmul2_by(v[k], s, j >= 2);
    }
  }
}

template <int KV, int D>
__global__ void __launch_bounds__(kBoundWarps * 32, KV == PKV_BF16 ? 8 : 4) key_bounds_kernel(const BoundsParams p) {
  using C = BoundCfg<KV, D>;
  constexpr uint32_t INF = KV == PKV_BF16 ? 0x7f807f80u : 0x7c007c00u, SIGNS = 0x80008000u;
  static_assert(C::ROWS >= 2, "the first row's lanes write the lower bounds, the second's the upper ones");
  __shared__ uint32_t s_part[kBoundWarps - 1][2 * C::PAIRS][C::LANES];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lane_c = lane % C::LANES, lane_r = lane / C::LANES;
  const int ps = p.page_size;
  const int stride = p.shared_page ? kBoundWarps * C::ROWS : C::ROWS;
  const int start = (p.shared_page ? warp * C::ROWS : 0) + lane_r;
  const int64_t unit = p.shared_page ? (int64_t)blockIdx.x : blockIdx.x * (int64_t)kBoundWarps + warp;
  const int64_t u = unit / p.num_kv_heads;
  const int h = (int)(unit - u * p.num_kv_heads);
  const bool upper = lane_r == 1;
  if (u >= p.pages) return;  // (whole CTAs where they share a page)
  const char* rows = nullptr;
  const char* sfs = nullptr;
  uint4 x[C::UNROLL];
  uint32_t sf[C::UNROLL];
  auto open_page = [&](int page) {
    rows = p.k_pool + (int64_t)page * p.stride_page_b + (int64_t)h * p.stride_head_b + lane_c * 16;
    if constexpr (KV == PKV_NVFP4) sfs = p.k_sf + (int64_t)page * p.sf_page_b + (int64_t)h * p.sf_head_b + lane_c * 2;
  };
  auto read = [&](int r0, int limit) {  // rows r0, r0 + stride, ... below the limit
#pragma unroll
    for (int k = 0; k < C::UNROLL; ++k) {
      const int r = r0 + k * stride;
      if (r < limit) {
        x[k] = ldg_once(rows + r * p.stride_token_b);
        if constexpr (KV == PKV_NVFP4) sf[k] = __ldg(reinterpret_cast<const unsigned short*>(sfs + r * p.sf_token_b));
      }
    }
  };

  // the request of the page, and the page's place in its list
  int i, page = 0;
  const bool early = !p.last_only && !p.new_only;  // every page is looked at: its first rows are read before its request is known
  if (p.last_only) {  // one page per request: its last one
    i = (int)u;
  } else {
    if (early) {
      page = __ldg(p.kv_indices + u);
      open_page(page);
      read(start, ps);
    }
    // the last request whose pages start at or before the entry, 32 probes at a time (requests without pages
    // share their successor's start)
    int lo = 0, n = p.batch;
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int at = lane * step;
      const bool below = at < n && __ldg(&p.req[lo + at].page_base) <= u;
      const int k = __popc(__ballot_sync(0xffffffffu, below)) - 1;  // (the first probe always is)
      lo += k * step;
      n = min(step, n - k * step);
    }
    i = lo;
  }
  const int4 rq = __ldg(reinterpret_cast<const int4*>(p.req + i));  // page_base, kv_len, q_begin, q_len
  const int L = rq.y;
  const int N = (int)p.by_page.div((uint32_t)L + (uint32_t)ps - 1u);
  const int block = p.last_only ? N - 1 : (int)(u - rq.x);
  if (p.last_only && (rq.w == 0 || N == 0)) return;
  const int valid = min(ps, L - block * ps);
  if (!early) {
    if (p.new_only && (rq.w == 0 || block * ps + valid <= L - rq.w)) return;  // no new token in it
    page = __ldg(p.kv_indices + rq.x + block);
    open_page(page);
    read(start, valid);
  }

  // largest values, and largest negated ones (floor(x) = -ceil(-x): both bounds are rounded up)
  uint32_t mn[C::PAIRS], mx[C::PAIRS];
#pragma unroll
  for (int j = 0; j < C::PAIRS; ++j) mn[j] = INF, mx[j] = INF | SIGNS;
  for (int r0 = start; r0 < valid;) {
#pragma unroll
    for (int k = 0; k < C::UNROLL; ++k) {
      if (r0 + k * stride < valid) {
        uint32_t v[C::PAIRS];
        widen<KV>(x[k], sf[k], v);
#pragma unroll
        for (int j = 0; j < C::PAIRS; ++j) {
          mn[j] = pair_min<KV>(mn[j], v[j]);
          mx[j] = pair_max<KV>(mx[j], v[j]);
        }
      }
    }
    r0 += C::UNROLL * stride;
    if (r0 < valid) read(r0, valid);
  }
  __syncwarp();
#pragma unroll
  for (int o = C::LANES; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < C::PAIRS; ++j) {
      mn[j] = pair_min<KV>(mn[j], __shfl_xor_sync(0xffffffffu, mn[j], o));
      mx[j] = pair_max<KV>(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], o));
    }
  if (p.shared_page) {
    if (warp > 0 && lane < C::LANES)
#pragma unroll
      for (int j = 0; j < C::PAIRS; ++j) {
        s_part[warp - 1][j][lane] = mn[j];
        s_part[warp - 1][C::PAIRS + j][lane] = mx[j];
      }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 0; k < kBoundWarps - 1; ++k)
#pragma unroll
      for (int j = 0; j < C::PAIRS; ++j) {
        mn[j] = pair_min<KV>(mn[j], s_part[k][j][lane_c]);
        mx[j] = pair_max<KV>(mx[j], s_part[k][C::PAIRS + j][lane_c]);
      }
  }
  if (lane_r > 1) return;
  const float sign = upper ? 1.f : -1.f;
  uint32_t out[C::PAIRS / 2];
#pragma unroll
  for (int j = 0; j < C::PAIRS; j += 2) {
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(p.scale + h * D + lane_c * 2 * C::PAIRS + 2 * j));
    const float scale[4] = {s4.x, s4.y, s4.z, s4.w};
    uint32_t code[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = upper ? mx[j + (e >> 1)] : mn[j + (e >> 1)] ^ SIGNS;
      float f;
      if constexpr (KV == PKV_BF16) f = __uint_as_float((e & 1) ? w & 0xffff0000u : w << 16);
      else f = __half2float(__ushort_as_half((unsigned short)((e & 1) ? w >> 16 : w & 0xffffu))) * p.k_scale;
      const float c = ceilf(__fdiv_rn(f, scale[e]));
      // (a NaN becomes 127; the code is the low byte of 1.5 * 2^23 + c)
      code[e] = __float_as_uint(fmaf(fmaxf(fminf(c, 127.f), -127.f), sign, 12582912.f));
    }
    out[j / 2] = __byte_perm(__byte_perm(code[0], code[1], 0x0040u), __byte_perm(code[2], code[3], 0x0040u), 0x5410u);
  }
  int8_t* dst = p.codes + (((int64_t)page * p.num_kv_heads + h) * 2 + (upper ? 1 : 0)) * D + lane_c * 2 * C::PAIRS;
  if constexpr (C::PAIRS == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  } else {
#pragma unroll
    for (int j = 0; j < C::PAIRS / 2; j += 4)
      *reinterpret_cast<uint4*>(dst + 4 * j) = make_uint4(out[j], out[j + 1], out[j + 2], out[j + 3]);
  }
}

template <int KV, int D>
cudaError_t launch_form(const BoundsParams& p, cudaStream_t s) {
  const int64_t units = p.pages * p.num_kv_heads, ctas = p.shared_page ? units : (units + kBoundWarps - 1) / kBoundWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(key_bounds_kernel<KV, D>, dim3((unsigned)ctas), dim3(kBoundWarps * 32), 0, s, p);
}

}  // namespace

cudaError_t launch_key_bounds(BoundsParams p, int dtype, int head_dim, int num_sms, cudaStream_t s) {
  // four warps to a page while that does not take more CTAs than run at once, and a page has rows for them
  p.shared_page = p.page_size >= 32 && p.pages * p.num_kv_heads <= (int64_t)num_sms * 4;
  p.by_page = divider(p.page_size);
  if (dtype == PKV_NVFP4) return launch_form<PKV_NVFP4, 128>(p, s);
  if (dtype == PKV_FP8_E4M3) return launch_form<PKV_FP8_E4M3, 128>(p, s);
  return head_dim == 128 ? launch_form<PKV_BF16, 128>(p, s) : launch_form<PKV_BF16, 64>(p, s);
}

}  // namespace pkv
