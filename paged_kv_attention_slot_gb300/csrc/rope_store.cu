// Rotary positions with the KV write (pkv_rope_kv_store): q and k turned by their positions' angles, q out, K and V
// into the paged pool, in one launch.
//
// For a token at position P and pair i of a head's first R elements, with angle P f_i, c = A cos, s = A sin:
//   (x1, x2) -> (x1 c - x2 s, x2 c + x1 s),
// the pair being elements (i, i + R / 2) or, interleaved, (2i, 2i + 1); elements R.. pass through.
//
// Angles: f_i / 2 pi arrives as a 64-bit binary fraction of a turn, so P times it modulo 2^64 is the phase, exactly
// (an integer multiplication that wraps), whatever the position; its top 32 bits as a float, at most 2^-25 of a
// half turn off, go to sincospi.  No table, whose rows would be read from memory, and no argument reduction.
// Rotation in float32, one rounding to bf16; an FP8 or NVFP4 pool gets what the KV write makes of that bf16 key.
//
// What bounds it: HBM (q in and out, k and v in, the pool's rows out).  One CTA takes one token: its first R / 2 threads
// compute the token's sines and cosines once for all heads, while every thread's row pieces are on their
// way.  A thread takes 16 elements of a row as two 16-byte vectors that hold both halves of 8 pairs.  8191 tokens of
// 32 + 8 + 8 heads, bf16 (201 MB): 31.8 us, 95 % of the measured copy rate; 2047 tokens of 64 + 8 + 8 heads into an E4M3
// pool (80 MB): 13.9 us, 86 %; 64 tokens: 1.9 us, one chain of dependent reads.  An NVFP4 pool takes 39.0 us for the 8191
// tokens (177 MB, 68 %) and 2.5 for the 64: its quantisation needs up to 64 registers, so fewer CTAs hide each other's chain.
// Many small CTAs hide each other's chain (position -> angle -> barrier): of up to 256 threads, at 40 registers, for more
// tokens than SMs (8191 tokens: 384 threads 38.2 us, at 50 registers 41.8, at 32 with spills 43.1); up to
// that many tokens all pieces in one round, where 512 threads do (64 tokens: 256 threads 2.2 us).

#include <algorithm>

#include "decode_blocks.h"
#include "kv_quant.cuh"
#include "ptx.cuh"

namespace pkv {

int32_t* device_error_ptr();

namespace {

constexpr int kRopeMaxThreads = 512;
constexpr int kRopeFewTokens = 152;    // a CTA per SM: latency counts, one round of row pieces where 512 threads allow it
constexpr int kRopeManyThreads = 256;  // at most, where there are more tokens than run at once

struct RopeParams {
  const char* q;
  const char* k;
  const char* v;
  int64_t qt, qh, kt, kh, vt, vh;  // strides of the inputs in bytes: token, head
  char* q_out;                     // [T, Hq, D]
  char* k_out;                     // [T, H, D], nullable
  const int64_t* positions;
  const int64_t* slots;
  const uint64_t* step;  // [R / 2] turns per position, in units of 2^-64
  float amplitude;
  char* k_pool;
  char* v_pool;
  char* k_sf;
  char* v_sf;
  int64_t sp_b, st_b, sh_b, fp_b, ft_b, fh_b;  // strides of the pools and block scales in bytes
  float* scores;  // nullable
  int64_t total_slots;
  int32_t page_size, q_heads, heads, half;  // half = R / 2
  Divider by_page;
  float inv_k, inv_v;
  int32_t* err;
};

// eight pairs (x1 in a, x2 in b) of bf16, turned
__device__ __forceinline__ void turn_halves(uint4& a, uint4& b, const float* cs, const float* sn) {
  uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float ya[2], yb[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x1 = __uint_as_float(e ? wa[j] & 0xffff0000u : wa[j] << 16);
      const float x2 = __uint_as_float(e ? wb[j] & 0xffff0000u : wb[j] << 16);
      const float c = cs[2 * j + e], s = sn[2 * j + e];
      ya[e] = fmaf(x1, c, -(x2 * s));
      yb[e] = fmaf(x2, c, x1 * s);
    }
    wa[j] = pack_bf16(ya[0], ya[1]);
    wb[j] = pack_bf16(yb[0], yb[1]);
  }
  a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}
// four pairs of neighbours, turned
__device__ __forceinline__ void turn_neighbours(uint4& a, const float* cs, const float* sn) {
  uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x1 = __uint_as_float(w[j] << 16), x2 = __uint_as_float(w[j] & 0xffff0000u);
    w[j] = pack_bf16(fmaf(x1, cs[j], -(x2 * sn[j])), fmaf(x2, cs[j], x1 * sn[j]));
  }
  a = make_uint4(w[0], w[1], w[2], w[3]);
}

// Vector v (8 elements) of a row whose 16-element pieces its 8 lanes hold as (a, b): piece c < pairs holds vectors
// c and c + pairs, the others 2c and 2c + 1.
__device__ __forceinline__ uint4 row_vector(const uint4& a, const uint4& b, int v, int pairs, unsigned mask) {
  const int own = v < 2 * pairs ? (v < pairs ? v : v - pairs) : v >> 1;
  const bool second = v < 2 * pairs ? v >= pairs : v & 1;
  uint4 x, y;
  x.x = __shfl_sync(mask, a.x, own, 8);
  x.y = __shfl_sync(mask, a.y, own, 8);
  x.z = __shfl_sync(mask, a.z, own, 8);
  x.w = __shfl_sync(mask, a.w, own, 8);
  y.x = __shfl_sync(mask, b.x, own, 8);
  y.y = __shfl_sync(mask, b.y, own, 8);
  y.z = __shfl_sync(mask, b.z, own, 8);
  y.w = __shfl_sync(mask, b.w, own, 8);
  return second ? y : x;
}

template <int KV, int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeMaxThreads, KV == PKV_NVFP4 ? 2 : 3) rope_store_kernel(const RopeParams p) {
  constexpr int PIECES = D / 16;  // threads per row
  __shared__ __align__(16) float s_cos[D / 2], s_sin[D / 2];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t tok = blockIdx.x;
  const int rows = p.q_heads + 2 * p.heads, tasks = rows * PIECES;
  const int c = threadIdx.x % PIECES;  // blockDim is a multiple of 32: the piece is the same in every round
  const int pairs = p.half >> 3;       // pieces that are turned
  const bool turned = c < pairs;
  // element offsets of the two vectors of a piece of q or k
  const int a_at = !NEIGHBOURS && turned ? 8 * c : 16 * c;
  const int b_at = !NEIGHBOURS && turned ? a_at + p.half : a_at + 8;

  auto row_of = [&](int r) -> const char* {
    if (r < p.q_heads) return p.q + tok * p.qt + r * p.qh;
    if (r < p.q_heads + p.heads) return p.k + tok * p.kt + (r - p.q_heads) * p.kh;
    return p.v + tok * p.vt + (r - p.q_heads - p.heads) * p.vh;
  };
  // (plain loads: q_out and k_out may be q and k themselves)
  auto load = [&](int task, uint4& a, uint4& b) {
    const int r = task / PIECES;
    const char* at = row_of(r);
    const bool is_v = r >= p.q_heads + p.heads;
    a = *reinterpret_cast<const uint4*>(at + 2 * (is_v ? 16 * c : a_at));
    b = *reinterpret_cast<const uint4*>(at + 2 * (is_v ? 16 * c + 8 : b_at));
  };

  uint4 a, b;
  if ((int)threadIdx.x < tasks) load(threadIdx.x, a, b);
  const int64_t slot = __ldg(p.slots + tok);
  for (int i = threadIdx.x; i < p.half; i += blockDim.x) {
    const uint64_t phase = (uint64_t)__ldg(p.positions + tok) * __ldg(p.step + i);
    float sn, cs;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: the phase in half turns
    s_cos[i] = cs * p.amplitude;
    s_sin[i] = sn * p.amplitude;
  }
  __syncthreads();
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    const int at = turned ? 8 * c + j : 0;
    const float4 x = *reinterpret_cast<const float4*>(s_cos + at), y = *reinterpret_cast<const float4*>(s_sin + at);
    cs[j] = x.x, cs[j + 1] = x.y, cs[j + 2] = x.z, cs[j + 3] = x.w;
    sn[j] = y.x, sn[j + 1] = y.y, sn[j + 2] = y.z, sn[j + 3] = y.w;
  }
  const bool stored = slot >= 0 && slot < p.total_slots;
  if (threadIdx.x == 0 && slot >= p.total_slots) record_error(p.err, PKV_DEVERR_SLOT_RANGE);
  const uint32_t page = stored ? p.by_page.div64(slot) : 0u;
  const uint32_t off = stored ? (uint32_t)(slot - (int64_t)page * p.page_size) : 0u;
  const int64_t pool_at = (int64_t)page * p.sp_b + (int64_t)off * p.st_b;
  const int64_t sf_at = KV == PKV_NVFP4 ? (int64_t)page * p.fp_b + (int64_t)off * p.ft_b : 0;

  for (int task = threadIdx.x; task < tasks; task += blockDim.x) {
    if (task != (int)threadIdx.x) load(task, a, b);
    const int r = task / PIECES;
    const bool is_v = r >= p.q_heads + p.heads;
    if (turned && !is_v) {
      if constexpr (NEIGHBOURS) {
        turn_neighbours(a, cs, sn);
        turn_neighbours(b, cs + 4, sn + 4);
      } else {
        turn_halves(a, b, cs, sn);
      }
    }
    if (r < p.q_heads) {
      char* at = p.q_out + (tok * p.q_heads + r) * (2 * D);
      *reinterpret_cast<uint4*>(at + 2 * a_at) = a;
      *reinterpret_cast<uint4*>(at + 2 * b_at) = b;
      continue;
    }
    const int h = r - p.q_heads - (is_v ? p.heads : 0);
    const int a_el = is_v ? 16 * c : a_at, b_el = is_v ? 16 * c + 8 : b_at;
    if (!is_v && p.k_out) {
      char* at = p.k_out + (tok * p.heads + h) * (2 * D);
      *reinterpret_cast<uint4*>(at + 2 * a_el) = a;
      *reinterpret_cast<uint4*>(at + 2 * b_el) = b;
    }
    if (!stored) continue;  // the whole CTA
    if (p.scores && !is_v && c == 0) p.scores[((int64_t)page * p.heads + h) * p.page_size + off] = 0.f;
    char* row = (is_v ? p.v_pool : p.k_pool) + pool_at + h * p.sh_b;
    if constexpr (KV == PKV_BF16) {
      *reinterpret_cast<uint4*>(row + 2 * a_el) = a;
      *reinterpret_cast<uint4*>(row + 2 * b_el) = b;
    } else if constexpr (KV == PKV_FP8_E4M3) {
      const float inv = is_v ? p.inv_v : p.inv_k;
      *reinterpret_cast<uint2*>(row + a_el) = quant_e4m3x8(a, inv);
      *reinterpret_cast<uint2*>(row + b_el) = quant_e4m3x8(b, inv);
    } else {
      // thread c quantises block c of the row, and packs the blocks' scales four to a word
      const unsigned mask = 0xffu << (threadIdx.x & 24);
      uint4 x = a, y = b;
      if (!NEIGHBOURS && !is_v) {  // (is_v is the row's)
        x = row_vector(a, b, 2 * c, pairs, mask);
        y = row_vector(a, b, 2 * c + 1, pairs, mask);
      }
      uint32_t sf;
      *reinterpret_cast<uint2*>(row + 8 * c) = quant_block(x, y, is_v ? p.inv_v : p.inv_k, sf);
      sf <<= 8 * (c & 3);
      sf |= __shfl_xor_sync(mask, sf, 1);
      sf |= __shfl_xor_sync(mask, sf, 2);
      if ((c & 3) == 0) *reinterpret_cast<uint32_t*>((is_v ? p.v_sf : p.k_sf) + sf_at + h * p.fh_b + c) = sf;
    }
  }
}

template <int KV, int D>
cudaError_t launch_form(const RopeParams& p, bool neighbours, int64_t tokens, cudaStream_t s) {
  const int tasks = (p.q_heads + 2 * p.heads) * (D / 16);
  const int cap = tokens > kRopeFewTokens ? kRopeManyThreads : kRopeMaxThreads;
  const int rounds = (tasks + cap - 1) / cap;
  const int threads = ((tasks + rounds - 1) / rounds + 31) / 32 * 32;
  const dim3 g((unsigned)tokens), b((unsigned)threads);
  return neighbours ? launch_pdl(rope_store_kernel<KV, D, true>, g, b, 0, s, p)
                    : launch_pdl(rope_store_kernel<KV, D, false>, g, b, 0, s, p);
}

}  // namespace

cudaError_t launch_rope_store(const pkv_rope_args& a, const pkv_cache& c, float inv_k, float inv_v, cudaStream_t s) {
  const int64_t esz = pool_elem_bytes(c.dtype);
  RopeParams p{};
  p.q = static_cast<const char*>(a.q);
  p.k = static_cast<const char*>(a.k);
  p.v = static_cast<const char*>(a.v);
  p.qt = a.q_stride_token * 2;
  p.qh = a.q_stride_head * 2;
  p.kt = a.k_stride_token * 2;
  p.kh = a.k_stride_head * 2;
  p.vt = a.v_stride_token * 2;
  p.vh = a.v_stride_head * 2;
  p.q_out = static_cast<char*>(a.q_out);
  p.k_out = static_cast<char*>(a.k_out);
  p.positions = a.positions;
  p.slots = a.slot_mapping;
  p.step = a.phase_step;
  p.amplitude = a.amplitude;
  p.k_pool = static_cast<char*>(c.k);
  p.v_pool = static_cast<char*>(c.v);
  p.sp_b = c.stride_page * esz;
  p.st_b = c.stride_token * esz;
  p.sh_b = c.stride_head * esz;
  if (c.dtype == PKV_NVFP4) {
    p.k_sf = static_cast<char*>(c.k_sf);
    p.v_sf = static_cast<char*>(c.v_sf);
    p.fp_b = c.sf_stride_page;
    p.ft_b = c.sf_stride_token;
    p.fh_b = c.sf_stride_head;
  }
  p.scores = a.scores;
  p.total_slots = c.num_pages * (int64_t)c.page_size;
  p.page_size = c.page_size;
  p.q_heads = a.num_qo_heads;
  p.heads = c.num_kv_heads;
  p.half = a.rotary_dim / 2;
  p.by_page = divider(c.page_size);
  p.inv_k = inv_k;
  p.inv_v = inv_v;
  p.err = device_error_ptr();
  if (!p.err) return cudaErrorInvalidDevice;
  const bool nb = a.interleaved != 0;
  if (c.dtype == PKV_NVFP4) return launch_form<PKV_NVFP4, 128>(p, nb, a.num_tokens, s);
  if (c.dtype == PKV_FP8_E4M3)
    return c.head_dim == 128 ? launch_form<PKV_FP8_E4M3, 128>(p, nb, a.num_tokens, s)
                             : launch_form<PKV_FP8_E4M3, 64>(p, nb, a.num_tokens, s);
  return c.head_dim == 128 ? launch_form<PKV_BF16, 128>(p, nb, a.num_tokens, s)
                           : launch_form<PKV_BF16, 64>(p, nb, a.num_tokens, s);
}

// ------------------------------------------------------------------------------------------------
// positions and slots of the planned new tokens (pkv_token_map)
// ------------------------------------------------------------------------------------------------
namespace {

// One thread per token row.  Token t of request i (the last request whose rows start at or before the token) sits
// at key P = L_i - n_i + t, in slot page(P / ps) ps + P % ps.
__global__ void __launch_bounds__(256) token_map_kernel(const ReqInfo* req, const int32_t* kv_indices, int32_t batch,
                                                        int64_t tokens, Divider by_page, int32_t ps, const int64_t* offsets,
                                                        int64_t* positions, int64_t* slots) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (row >= tokens) return;
  int lo = 0, hi = batch;  // q_begin[lo] <= row < q_begin[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(&req[mid].q_begin) <= row) lo = mid;
    else hi = mid;
  }
  const int4 r = __ldg(reinterpret_cast<const int4*>(req + lo));  // page_base, kv_len, q_begin, q_len
  if (row - r.z >= r.w) {  // (a captured call whose plan was made anew for fewer tokens: a row behind the last one)
    slots[row] = -1;
    positions[row] = 0;
    return;
  }
  const int32_t key = r.y - r.w + (int32_t)(row - r.z);
  const int32_t page = (int32_t)by_page.div((uint32_t)key);
  slots[row] = (int64_t)__ldg(kv_indices + r.x + page) * ps + (key - page * ps);
  positions[row] = key + (offsets ? __ldg(offsets + lo) : 0);
}

}  // namespace

cudaError_t launch_token_map(const ReqInfo* req, const int32_t* kv_indices, int32_t batch, int64_t tokens, int32_t page_size,
                             const int64_t* offsets, int64_t* positions, int64_t* slots, cudaStream_t s) {
  return launch_pdl(token_map_kernel, dim3((unsigned)((tokens + 255) / 256)), dim3(256), 0, s, req, kv_indices, batch, tokens,
                    divider(page_size), page_size, offsets, positions, slots);
}

}  // namespace pkv
