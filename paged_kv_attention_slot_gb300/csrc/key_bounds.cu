// 8-bit bounds of the keys of each page, per KV head and channel (pkv_key_bounds_update).
//
// For page p of a request, KV head h, channel d, over the page's valid keys j, in units of s = scale[h, d]:
//   lo = clamp(floor(min_j k_jd / s), -127, 127),  hi = clamp(ceil(max_j k_jd / s), -127, 127),
// the quotients in float32.  A NaN key element gives (-127, 127), so that its page is not passed over.
//
// What bounds it: reading the keys once.  A warp takes the page of one KV head: its lanes read 16 bytes (NVFP4: 8) of a
// row each, several rows to an instruction, past L1, and keep the extremes in 16-bit pairs, which is exact (bf16 as
// they are; E4M3 values and E2M1 values times their block scale are f16 values), so the divisions come after the
// last key.  The rows of every page are read before its request is known (which only says how many are valid).  At
// the end the channels are shared out over the lanes before they are divided and rounded: small pages are bound by
// those instructions, not by memory.  64 x 512 to 4096 keys x 8 heads, pages of 16: bf16 47 us for 287 MB, 91 % of the
// measured copy rate (kept in L1: 2.5 more; 66 registers instead of 64: 5); 64 x 2048 to 4096 keys: E4M3 62 us, 55 % (128-token
// pages 36), NVFP4 66 us, 31 % (32).  A decode step's one page per request: 2.6 us.  Not writing what a captured call's new
// plan lists beyond the pool, or behind its last request, is 0.8 of the 47 us.
// A call for few large pages shares a page's rows among the four warps of a CTA.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "decode_blocks.h"
#include "ptx.cuh"

namespace pkv {

int32_t* device_error_ptr();

namespace {

constexpr int kBoundWarps = 4;

template <int KV, int D>
struct BoundCfg {
  static constexpr int VECB = KV == PKV_NVFP4 ? 8 : 16;                                // bytes of a row that a lane reads
  static constexpr int LANES = (KV == PKV_NVFP4 ? D / 2 : KV == PKV_FP8_E4M3 ? D : 2 * D) / VECB;  // per row
  static constexpr int ROWS = 32 / LANES;                                              // per warp-wide load
  static constexpr int PAIRS = KV == PKV_BF16 ? 4 : 8;                                 // of elements per lane
  static constexpr int MINE = D / 16;                                                  // channels of one bound that a lane ends with
  static constexpr int UNROLL = 16 / ROWS;                                             // loads in flight: a 16-token page at once
  using Vec = typename std::conditional<KV == PKV_NVFP4, uint2, uint4>::type;
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

// the pairs (element 2 j, 2 j + 1) of a lane's part of a row; sf: its block scale (NVFP4)
__device__ __forceinline__ void widen(const uint4& x, uint32_t, uint32_t (&out)[4]) {  // bf16
  out[0] = x.x, out[1] = x.y, out[2] = x.z, out[3] = x.w;
}
__device__ __forceinline__ void widen(const uint4& x, uint32_t, uint32_t (&out)[8]) {  // E4M3
  e4m3x4_to_f16x2x2(x.x, out[0], out[1]);
  e4m3x4_to_f16x2x2(x.y, out[2], out[3]);
  e4m3x4_to_f16x2x2(x.z, out[4], out[5]);
  e4m3x4_to_f16x2x2(x.w, out[6], out[7]);
}
__device__ __forceinline__ void widen(const uint2& x, uint32_t sf, uint32_t (&out)[8]) {  // E2M1 times its block's scale
  const uint32_t s = e4m3x2_to_f16x2(sf);
  uint32_t v[4];
  e2m1x8_to_f16x2x4(x.x, v);
#pragma unroll
  for (int k = 0; k < 4; ++k) out[k] = hmul2_by(v[k], s, false);
  e2m1x8_to_f16x2x4(x.y, v);
#pragma unroll
  for (int k = 0; k < 4; ++k) out[4 + k] = hmul2_by(v[k], s, false);
}

template <int KV, int D>
__global__ void __launch_bounds__(kBoundWarps * 32, 8) key_bounds_kernel(const BoundsParams p) {
  using C = BoundCfg<KV, D>;
  constexpr uint32_t INF = KV == PKV_BF16 ? 0x7f807f80u : 0x7c007c00u, SIGNS = 0x80008000u;
  __shared__ uint32_t s_part[kBoundWarps - 1][C::MINE / 2][32];
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
  if (u >= p.pages) return;  // (whole CTAs where they share a page)
  const char* rows = nullptr;
  const char* sfs = nullptr;
  typename C::Vec x[C::UNROLL];
  uint32_t sf[C::UNROLL];
  auto open_page = [&](int page) {
    rows = p.k_pool + (int64_t)page * p.stride_page_b + (int64_t)h * p.stride_head_b + lane_c * C::VECB;
    if constexpr (KV == PKV_NVFP4) sfs = p.k_sf + (int64_t)page * p.sf_page_b + (int64_t)h * p.sf_head_b + lane_c;
  };
  auto read = [&](int r0, int limit) {  // rows r0, r0 + stride, ... below the limit
#pragma unroll
    for (int k = 0; k < C::UNROLL; ++k) {
      const int r = r0 + k * stride;
      if (r < limit) {
        if constexpr (KV == PKV_NVFP4) {
          x[k] = ldg_once8(rows + r * p.stride_token_b);
          sf[k] = __ldg(reinterpret_cast<const unsigned char*>(sfs + r * p.sf_token_b));
        } else {
          x[k] = ldg_once(rows + r * p.stride_token_b);
        }
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
      open_page((int)min((uint32_t)page, p.last_page));
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
  if (unit == 0 && lane == 0 && warp == 0 && __ldg(p.max_page) > (int)p.last_page) record_error(p.err, PKV_DEVERR_PAGE_RANGE);
  const int L = rq.y;
  const int N = (int)p.by_page.div((uint32_t)L + (uint32_t)ps - 1u);
  const int block = p.last_only ? N - 1 : (int)(u - rq.x);
  if (p.last_only && (rq.w == 0 || N == 0)) return;
  if (block >= N) return;  // (a captured call whose plan was made anew for fewer pages: an entry behind the last request)
  const int valid = min(ps, L - block * ps);
  if (!early) {
    if (p.new_only && (rq.w == 0 || block * ps + valid <= L - rq.w)) return;  // no new token in it
    page = __ldg(p.kv_indices + rq.x + block);
  }
  if ((uint32_t)page > p.last_page) return;  // (and over pages that the pool does not have: recorded above)
  if (!early) {
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
        widen(x[k], sf[k], v);
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
  // Across the warp's rows: the upper half of the lanes takes the largest values, the lower half the largest negated
  // ones, then each step halves the channels, so that every lane ends with C::MINE of one bound.
  const bool upper = lane & 16;
  uint32_t best[C::PAIRS];
#pragma unroll
  for (int j = 0; j < C::PAIRS; ++j) {
    mn[j] ^= SIGNS;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? mn[j] : mx[j], 16);
    best[j] = pair_max<KV>(upper ? mx[j] : mn[j], other);
  }
  int held = C::PAIRS, first = 0;  // pairs of this lane's 16 bytes of a row that it still holds
#pragma unroll
  for (int o = 8; o >= C::LANES; o >>= 1) {
    held >>= 1;
    const bool high = lane & o;
    if (high) first += held;
#pragma unroll
    for (int j = 0; j < C::PAIRS / 2; ++j)
      if (j < held) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, high ? best[j] : best[held + j], o);
        best[j] = pair_max<KV>(high ? best[held + j] : best[j], other);
      }
  }
  if (p.shared_page) {
    if (warp > 0)
#pragma unroll
      for (int j = 0; j < C::MINE / 2; ++j) s_part[warp - 1][j][lane] = best[j];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 0; k < kBoundWarps - 1; ++k)
#pragma unroll
      for (int j = 0; j < C::MINE / 2; ++j) best[j] = pair_max<KV>(best[j], s_part[k][j][lane]);
  }
  const int channel = lane_c * 2 * C::PAIRS + 2 * first;  // the first of this lane's
  const float sign = upper ? 1.f : -1.f;
  uint32_t out[C::MINE / 4];
#pragma unroll
  for (int j = 0; j < C::MINE / 4; ++j) {
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(p.scale + h * D + channel + 4 * j));
    const float scale[4] = {s4.x, s4.y, s4.z, s4.w};
    uint32_t code[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = best[2 * j + (e >> 1)];
      float f;
      if constexpr (KV == PKV_BF16) f = __uint_as_float((e & 1) ? w & 0xffff0000u : w << 16);
      else f = __half2float(__ushort_as_half((unsigned short)((e & 1) ? w >> 16 : w & 0xffffu))) * p.k_scale;
      const float c = ceilf(__fdiv_rn(f, scale[e]));
      // (a NaN becomes 127; the code is the low byte of 1.5 * 2^23 + c)
      code[e] = __float_as_uint(fmaf(fmaxf(fminf(c, 127.f), -127.f), sign, 12582912.f));
    }
    out[j] = __byte_perm(__byte_perm(code[0], code[1], 0x0040u), __byte_perm(code[2], code[3], 0x0040u), 0x5410u);
  }
  int8_t* dst = p.codes + (((int64_t)page * p.num_kv_heads + h) * 2 + (upper ? 1 : 0)) * D + channel;
  if constexpr (C::MINE == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else *reinterpret_cast<uint32_t*>(dst) = out[0];
}

template <int KV, int D>
cudaError_t launch_form(const BoundsParams& p, cudaStream_t s) {
  const int64_t units = p.pages * p.num_kv_heads, ctas = p.shared_page ? units : (units + kBoundWarps - 1) / kBoundWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(key_bounds_kernel<KV, D>, dim3((unsigned)ctas), dim3(kBoundWarps * 32), 0, s, p);
}

}  // namespace

cudaError_t launch_key_bounds(BoundsParams p, int dtype, int head_dim, int num_sms, cudaStream_t s) {
  // Four warps to a page where a page has rows for them and there are few pages for its size: 128 tokens, 1024 pages x heads
  // bf16 10.0 -> 6.0 us, 2048 11.0 -> 8.8, 4096 no change; 64 tokens, 1024 6.2 -> 4.1, 2048 5.9 -> 6.1; 32 tokens, 512 3.1 (a
  // warp each 3.0), 1024 3.4 -> 3.6, 2048 4.7 -> 6.2.
  p.shared_page = p.page_size >= 32 && p.pages * p.num_kv_heads <= (int64_t)num_sms * p.page_size / 8;
  p.by_page = divider(p.page_size);
  p.err = device_error_ptr();
  if (!p.err) return cudaErrorInvalidDevice;
  if (dtype == PKV_NVFP4) return launch_form<PKV_NVFP4, 128>(p, s);
  if (dtype == PKV_FP8_E4M3) return launch_form<PKV_FP8_E4M3, 128>(p, s);
  return head_dim == 128 ? launch_form<PKV_BF16, 128>(p, s) : launch_form<PKV_BF16, 64>(p, s);
}

}  // namespace pkv
