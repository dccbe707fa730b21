// The KV write: scatter this step's K/V rows into the paged pool through slot_mapping.
//
// "vLLM 源码完全拆解（六）：Attention Backend", sections «Runner 先构造公共事实» (slot =
// physical_page * page_size + offset_in_page) and «为什么 KV 写入在 Attention 之前» (the write runs
// before attention on the same stream so a query sees its own step's keys); "SGLang 源码完全拆解(八)：
// Attention Backend", section «层与后端的边界» (FP8 caches quantise on write with the same scale the
// read side uses).
//
// One thread moves one 16-byte chunk of one (token, head) row: for D = 128 bf16 a row is 16
// chunks, so a warp writes two full rows and every global access is a full 16-byte vector.  The
// kernel is a pure memory op; it is launched with enough CTAs to cover every chunk once.  An NVFP4 pool
// takes one thread per 16-element block instead (two chunks in, one scale and 8 code bytes out).
// kv_load is the way back: one thread per 8 elements of a row (one 16-byte vector out), widened and
// rounded to bf16.

#include <algorithm>

#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {

__device__ int32_t g_device_error;  // first error recorded by any kernel of this library

int32_t* device_error_ptr() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  static int32_t* cache[64] = {nullptr};
  if (dev < 0 || dev >= 64) return nullptr;
  if (!cache[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    cache[dev] = static_cast<int32_t*>(p);
  }
  return cache[dev];
}

cudaError_t read_device_error(int32_t* code, int reset, cudaStream_t s) {
  int32_t* p = device_error_ptr();
  if (!p) return cudaErrorInvalidDevice;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  e = cudaMemcpy(code, p, sizeof(int32_t), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return e;
  if (reset) e = cudaMemset(p, 0, sizeof(int32_t));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  return e;
}

struct StoreParams {
  const uint8_t* k;
  const uint8_t* v;
  const int64_t* slots;
  uint8_t* k_pool;
  uint8_t* v_pool;
  int64_t T;
  int64_t total_slots;
  int64_t sp_b, st_b, sh_b;  // strides in bytes
  int32_t page_size;
  int32_t heads;
  int32_t chunks;  // 16-byte source chunks per (token, head) row
  float inv_k, inv_v;
  float* scores;  // nullable: [num_pages, heads, page_size] accumulated weights, zeroed at the written slots
  int32_t* err;
};

template <bool FP8>
__global__ void __launch_bounds__(256) kv_store_kernel(const StoreParams p) {
  pdl_wait();
  pdl_launch_dependents();  // the attention run that follows may be scheduled now (it waits for us)
  const int64_t n = p.T * p.heads * p.chunks;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / p.chunks;  // token * heads + head
    const int c = (int)(i - row * p.chunks);
    const int64_t tok = row / p.heads;
    const int h = (int)(row - tok * p.heads);
    const int64_t slot = __ldg(p.slots + tok);
    if (slot < 0) continue;  // padding token
    if (slot >= p.total_slots) {
      record_error(p.err, PKV_DEVERR_SLOT_RANGE);
      continue;
    }
    const int64_t page = slot / p.page_size;
    const int64_t off = slot - page * p.page_size;
    if (p.scores && c == 0) p.scores[(page * p.heads + h) * p.page_size + off] = 0.f;
    const int64_t src = row * (int64_t)p.chunks * 16 + c * 16;
    const uint4 kx = __ldg(reinterpret_cast<const uint4*>(p.k + src));
    const uint4 vx = __ldg(reinterpret_cast<const uint4*>(p.v + src));
    if constexpr (!FP8) {
      const int64_t dst = page * p.sp_b + off * p.st_b + h * p.sh_b + c * 16;
      *reinterpret_cast<uint4*>(p.k_pool + dst) = kx;
      *reinterpret_cast<uint4*>(p.v_pool + dst) = vx;
    } else {
      // 8 bf16 -> 8 E4M3 codes: code = E4M3_RNE_satfinite(float(x) * inv_scale), product in fp32
      const int64_t dst = page * p.sp_b + off * p.st_b + h * p.sh_b + c * 8;
      auto quant = [](const uint4 x, float inv) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lo = __uint_as_float(w[j] << 16) * inv;
          const float hi = __uint_as_float(w[j] & 0xffff0000u) * inv;
          b[j] = f32x2_to_e4m3x2(lo, hi);
        }
        return make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
      };
      *reinterpret_cast<uint2*>(p.k_pool + dst) = quant(kx, p.inv_k);
      *reinterpret_cast<uint2*>(p.v_pool + dst) = quant(vx, p.inv_v);
    }
  }
}

// ---- NVFP4: codes and block scales ----
struct Fp4Pools {
  uint8_t* k_sf;
  uint8_t* v_sf;
  int64_t sp_b, st_b, sh_b;  // strides of the scale pools in bytes
};

// Quotients t / s rounded to nearest without a division: q = t r with r = 1 / s rounded, then one Newton step on
// the quotient (Markstein's correction), two quotients at a time.  It takes u = -t and -r: the step is then
// q - r (q s - t), whose sums keep the sign of t = -0 where t - q s would be +0.  The caller keeps t / s away
// from over- and underflow.
__device__ __forceinline__ uint64_t div2_rn(uint64_t u2, uint64_t s2, uint64_t minus_r2) {
  const uint64_t q2 = fmul2(u2, minus_r2);
  return ffma2(ffma2(q2, s2, u2), minus_r2, q2);
}

// The 16 codes of a block of bf16 pairs w under the block scale s (r = 1 / s rounded).  CLAMP: values may be
// beyond 2688 = 6 * 448, where the scale is 448 and the code 6, infinities included.
template <bool CLAMP>
__device__ __forceinline__ uint2 quant_codes(const uint32_t (&w)[8], float inv, float s, float r) {
  const uint64_t minus_inv2 = f2pack(-inv, -inv), minus_r2 = f2pack(-r, -r), s2 = f2pack(s, s);
  uint32_t c[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = w[4 * v + j];
      uint64_t u2 = fmul2(f2pack(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), minus_inv2);
      if constexpr (CLAMP) {
        float lo, hi;
        f2unpack(u2, lo, hi);
        u2 = f2pack(fminf(fmaxf(lo, -2688.f), 2688.f), fminf(fmaxf(hi, -2688.f), 2688.f));
      }
      f2unpack(div2_rn(u2, s2, minus_r2), q[2 * j], q[2 * j + 1]);
    }
    c[v] = f32x8_to_e2m1x8(q);
  }
  return make_uint2(c[0], c[1]);
}

// One block of 16 bf16 values (two 16-byte vectors) to its E4M3 scale code and 8 bytes of E2M1 codes.
// The largest magnitude is found on the bf16 bits (scaling is monotonic), two at a time; a NaN's are
// above infinity's.
__device__ __forceinline__ uint2 quant_block(const uint4 a, const uint4 b, float inv, uint32_t& sf) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __vmaxu2(top, w[j] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
  const float amax = fminf(__uint_as_float(top << 16) * inv, 1e30f);  // (above 2688 the scale is 448 in any case)
  const float sixth = 1.f / 6.f, q6 = amax * sixth;
  sf = f32x2_to_e4m3x2(fmaf(fmaf(-q6, 6.f, amax), sixth, q6), 0.f) & 0xffu;
  if (top > 0x7f80u) sf = 0x7fu;  // a NaN
  if (sf == 0 || sf == 0x7fu) return make_uint2(0u, 0u);
  // an E4M3 value's reciprocal is never near the middle of two floats, so one Newton step rounds it
  const float s = e4m3_to_f32(sf), r0 = rcp_approx(s), r = fmaf(fmaf(-s, r0, 1.f), r0, r0);
  if (amax > 1e6f) return quant_codes<true>(w, inv, s, r);
  return quant_codes<false>(w, inv, s, r);
}

// Quotients by a number that is usually a power of two.
struct Divider {
  int32_t d, shift;  // shift >= 0: d == 1 << shift
  __device__ __forceinline__ uint32_t div(uint32_t x) const { return shift >= 0 ? x >> shift : x / (uint32_t)d; }
  __device__ __forceinline__ uint32_t div64(int64_t x) const {  // x >= 0, quotient below 2^32
    if (shift >= 0) return (uint32_t)(x >> shift);
    return x >> 32 ? (uint32_t)(x / d) : (uint32_t)x / (uint32_t)d;
  }
};
Divider divider(int32_t d) {
  int s = 0;
  while ((1 << s) < d && s < 30) ++s;
  return Divider{d, (1 << s) == d ? s : -1};
}
constexpr int64_t kMaxRows = (int64_t)1 << 26;  // (token, head) rows per launch: 32-bit indices

// One thread per (token, head, block of 16): the 8 threads of a row write its 64 code bytes and, packed
// four to a word by shuffles, its 8 scale bytes.  The rows are read beside the slot, not after it.
__global__ void __launch_bounds__(256) kv_store_fp4_kernel(const StoreParams p, const Fp4Pools f, const Divider heads,
                                                           const Divider pages) {
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t n = (uint32_t)(p.T * p.heads) * 8;  // a multiple of 8: the threads of a row stay together
  const unsigned row_mask = 0xffu << (threadIdx.x & 24);
  const int c = threadIdx.x & 7;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
    const uint4* ks = reinterpret_cast<const uint4*>(p.k) + (int64_t)i * 2;
    const uint4* vs = reinterpret_cast<const uint4*>(p.v) + (int64_t)i * 2;
    const uint4 k0 = __ldg(ks), k1 = __ldg(ks + 1), v0 = __ldg(vs), v1 = __ldg(vs + 1);
    const uint32_t row = i >> 3, tok = heads.div(row), h = row - tok * p.heads;
    const int64_t slot = __ldg(p.slots + tok);
    if (slot < 0) continue;  // padding token (all 8 threads of the row)
    if (slot >= p.total_slots) {
      record_error(p.err, PKV_DEVERR_SLOT_RANGE);
      continue;
    }
    const uint32_t page = pages.div64(slot);
    const uint32_t off = (uint32_t)(slot - (int64_t)page * p.page_size);
    if (p.scores && c == 0) p.scores[((int64_t)page * p.heads + h) * p.page_size + off] = 0.f;
    const int64_t dst = page * p.sp_b + off * p.st_b + h * p.sh_b + c * 8;
    uint32_t fk, fv;
    *reinterpret_cast<uint2*>(p.k_pool + dst) = quant_block(k0, k1, p.inv_k, fk);
    *reinterpret_cast<uint2*>(p.v_pool + dst) = quant_block(v0, v1, p.inv_v, fv);
    fk <<= 8 * (c & 3);
    fv <<= 8 * (c & 3);
#pragma unroll
    for (int sh = 1; sh < 4; sh <<= 1) {
      fk |= __shfl_xor_sync(row_mask, fk, sh);
      fv |= __shfl_xor_sync(row_mask, fv, sh);
    }
    if ((c & 3) == 0) {
      const int64_t sd = page * f.sp_b + off * f.st_b + h * f.sh_b + c;
      *reinterpret_cast<uint32_t*>(f.k_sf + sd) = fk;
      *reinterpret_cast<uint32_t*>(f.v_sf + sd) = fv;
    }
  }
}

// ---- the read back ----
struct LoadParams {
  const int64_t* slots;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const uint8_t* k_sf;
  const uint8_t* v_sf;
  uint4* k;
  uint4* v;
  int64_t T, total_slots;
  int64_t sp_b, st_b, sh_b, fp_b, ft_b, fh_b;
  int32_t page_size, heads, unit_shift;  // 1 << unit_shift 16-byte vectors of a bf16 row
  float k_scale, v_scale;
  Divider by_heads, by_page;
  int32_t* err;
};

// Eight elements (unit c) of the row at byte offset `at` (block scales at `sat`) as one vector of bf16.
template <int KV>
__device__ __forceinline__ uint4 load_unit(const uint8_t* pool, const uint8_t* sf, int64_t at, int64_t sat, int c, float scale) {
  if constexpr (KV == PKV_BF16) {
    return __ldg(reinterpret_cast<const uint4*>(pool + at + c * 16));
  } else {
    uint32_t h[4];
    float s = 1.f;
    if constexpr (KV == PKV_NVFP4) {
      // code * block scale has 6 significant bits; the tensor's scale is the first rounding, bf16 the last
      s = e4m3_to_f32(__ldg(sf + sat + (c >> 1)));
      e2m1x8_to_f16x2x4(__ldg(reinterpret_cast<const uint32_t*>(pool + at + c * 4)), h);
    } else {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(pool + at + c * 8));
      e4m3x4_to_f16x2x2(x.x, h[0], h[1]);
      e4m3x4_to_f16x2x2(x.y, h[2], h[3]);
    }
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = f16x2_to_f32x2(h[j]);
      r[j] = KV == PKV_NVFP4 ? pack_bf16(y.x * s * scale, y.y * s * scale) : pack_bf16(y.x * scale, y.y * scale);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
}

template <int KV>
__global__ void __launch_bounds__(256) kv_load_kernel(const LoadParams p) {
  constexpr int U = 2;  // units in flight per thread
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t n = (uint32_t)(p.T * p.heads) << p.unit_shift, step = gridDim.x * 256;
  const int c = threadIdx.x & ((1 << p.unit_shift) - 1);
  for (uint32_t i0 = blockIdx.x * 256 + threadIdx.x; i0 < n; i0 += U * step) {
    int64_t slot[U];
    uint32_t h[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * step;
      slot[u] = -1;
      h[u] = 0;
      if (i < n) {
        const uint32_t row = i >> p.unit_shift, tok = p.by_heads.div(row);
        h[u] = row - tok * p.heads;
        slot[u] = __ldg(p.slots + tok);
      }
    }
    uint4 ko[U], vo[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ko[u] = vo[u] = make_uint4(0u, 0u, 0u, 0u);
      if (slot[u] >= p.total_slots) {
        record_error(p.err, PKV_DEVERR_SLOT_RANGE);
      } else if (slot[u] >= 0) {
        const uint32_t page = p.by_page.div64(slot[u]);
        const uint32_t off = (uint32_t)(slot[u] - (int64_t)page * p.page_size);
        const int64_t at = page * p.sp_b + off * p.st_b + h[u] * p.sh_b;
        const int64_t sat = KV == PKV_NVFP4 ? page * p.fp_b + off * p.ft_b + h[u] * p.fh_b : 0;
        ko[u] = load_unit<KV>(p.k_pool, p.k_sf, at, sat, c, p.k_scale);
        vo[u] = load_unit<KV>(p.v_pool, p.v_sf, at, sat, c, p.v_scale);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * step;
      if (i < n) {
        p.k[i] = ko[u];
        p.v[i] = vo[u];
      }
    }
  }
}

static cudaError_t launch_kv_load_rows(const LoadParams& p, int dtype, cudaStream_t s) {
  const int64_t blocks = std::min<int64_t>((((p.T * p.heads) << p.unit_shift) + 255) / 256, 152 * 8);
  const dim3 g((unsigned)blocks), b(256);
  if (dtype == PKV_NVFP4) return launch_pdl(kv_load_kernel<PKV_NVFP4>, g, b, 0, s, p);
  if (dtype == PKV_FP8_E4M3) return launch_pdl(kv_load_kernel<PKV_FP8_E4M3>, g, b, 0, s, p);
  return launch_pdl(kv_load_kernel<PKV_BF16>, g, b, 0, s, p);
}

cudaError_t launch_kv_load(const int64_t* slots, int64_t T, const pkv_cache& c, void* k, void* v, cudaStream_t s) {
  const bool fp4 = c.dtype == PKV_NVFP4;
  const int64_t esz = pool_elem_bytes(c.dtype);
  LoadParams p{};
  p.slots = slots;
  p.k_pool = static_cast<const uint8_t*>(c.k);
  p.v_pool = static_cast<const uint8_t*>(c.v);
  p.k = static_cast<uint4*>(k);
  p.v = static_cast<uint4*>(v);
  p.T = T;
  p.total_slots = c.num_pages * (int64_t)c.page_size;
  p.sp_b = c.stride_page * esz;
  p.st_b = c.stride_token * esz;
  p.sh_b = c.stride_head * esz;
  if (fp4) {
    p.k_sf = static_cast<const uint8_t*>(c.k_sf);
    p.v_sf = static_cast<const uint8_t*>(c.v_sf);
    p.fp_b = c.sf_stride_page;
    p.ft_b = c.sf_stride_token;
    p.fh_b = c.sf_stride_head;
  }
  p.page_size = c.page_size;
  p.heads = c.num_kv_heads;
  p.unit_shift = c.head_dim == 128 ? 4 : 3;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.by_heads = divider(p.heads);
  p.by_page = divider(p.page_size);
  p.err = device_error_ptr();
  if (!p.err) return cudaErrorInvalidDevice;
  const int64_t most = kMaxRows / p.heads;  // tokens per launch (check_indices: at least one)
  for (int64_t t0 = 0; t0 < T; t0 += most) {
    LoadParams q = p;
    q.slots = slots + t0;
    q.T = std::min(most, T - t0);
    q.k += (t0 * p.heads) << p.unit_shift;
    q.v += (t0 * p.heads) << p.unit_shift;
    const cudaError_t e = launch_kv_load_rows(q, c.dtype, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_kv_store(const void* k, const void* v, const int64_t* slots, int64_t T, const pkv_cache& c,
                            float inv_k, float inv_v, float* scores, cudaStream_t s) {
  const bool fp4 = c.dtype == PKV_NVFP4;
  const bool fp8 = c.dtype == PKV_FP8_E4M3;
  const int64_t esz = pool_elem_bytes(c.dtype);
  StoreParams p;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.slots = slots;
  p.k_pool = static_cast<uint8_t*>(c.k);
  p.v_pool = static_cast<uint8_t*>(c.v);
  p.T = T;
  p.total_slots = c.num_pages * (int64_t)c.page_size;
  p.sp_b = c.stride_page * esz;
  p.st_b = c.stride_token * esz;
  p.sh_b = c.stride_head * esz;
  p.page_size = c.page_size;
  p.heads = c.num_kv_heads;
  p.chunks = fp4 ? c.head_dim / 16 : c.head_dim * 2 / 16;
  p.scores = scores;
  p.inv_k = inv_k;
  p.inv_v = inv_v;
  p.err = device_error_ptr();
  if (!p.err) return cudaErrorInvalidDevice;
  const int64_t n = T * p.heads * p.chunks;
  int64_t blocks = (n + 255) / 256;
  if (blocks > 152 * 16) blocks = 152 * 16;
  if (fp4) {
    const Fp4Pools f{static_cast<uint8_t*>(c.k_sf), static_cast<uint8_t*>(c.v_sf), c.sf_stride_page, c.sf_stride_token,
                     c.sf_stride_head};
    const int64_t most = kMaxRows / p.heads;  // tokens per launch (check_indices: at least one)
    for (int64_t t0 = 0; t0 < T; t0 += most) {
      StoreParams q = p;
      q.slots = slots + t0;
      q.T = std::min(most, T - t0);
      q.k += t0 * p.heads * 256;
      q.v += t0 * p.heads * 256;
      const cudaError_t e = launch_pdl(kv_store_fp4_kernel, dim3((unsigned)blocks), dim3(256), 0, s, q, f, divider(p.heads),
                                       divider(p.page_size));
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  return fp8 ? launch_pdl(kv_store_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, s, p)
             : launch_pdl(kv_store_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, s, p);
}

}  // namespace pkv
