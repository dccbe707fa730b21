// Decode that accumulates every key's attention weight (pkv_attn_decode_run_scored).
//
// For a request with one new token, KV head h and visible key j the weight is
//   a_j = sum over the query heads g of h of exp(scale q_g.k_j - lse_g),
// and scores[slot(j), h] += a_j.  lse_g is known only after the last key, so the weights take a second
// look at every score.  Reading K again would add half of the decode's own traffic; instead the
// decode kernel leaves its scaled scores (log2 units, 4 bytes per key and query head: 16 bytes
// beside the 512 of a bf16 key row pair at 4 query heads per KV head) in a scratch that mostly stays in
// L2, and the kernel below turns them into weights and adds them.  It runs on the decode's own work
// list: a CTA takes the keys its decode CTA would take on an even split, one key per thread, so every
// score has one owner and needs no atomic.

#include "decode_kernel.cuh"

namespace pkv {

namespace {

constexpr int kScoreThreads = 256;

__global__ void __launch_bounds__(kScoreThreads) score_add_kernel(const RunParams p) {
  extern __shared__ float s_lse[];  // [group] log2-sum-exp of the KV head's query heads
  pdl_wait();                       // the decode run's scores
  const WorkItem w = p.work[blockIdx.x];
  if (w.head_group != 0) return;  // the first head group's CTA adds all of the KV head's query heads
  const int G = p.group;
  for (int g = threadIdx.x; g < G; g += kScoreThreads)
    s_lse[g] = p.lse2[(int64_t)w.q_row * p.num_qo_heads + w.kv_head * G + g];
  __syncthreads();
  const int share = (w.kv_end - w.kv_begin + w.num_splits - 1) / w.num_splits;
  const int lo = w.kv_begin + w.split * share, hi = min(w.kv_end, lo + share);
  const int ps = p.page_size;
  const float* lg0 = p.logits + (int64_t)w.page_base * ps * p.num_qo_heads + (int64_t)w.kv_head * w.kv_end * G;
  for (int key = lo + (int)threadIdx.x; key < hi; key += kScoreThreads) {
    const float* lg = lg0 + (int64_t)key * G;
    const int pg = key / ps;
    const int page = __ldg(p.kv_indices + w.page_base + pg);
    if ((unsigned long long)(unsigned)page >= (unsigned long long)p.num_pages) continue;  // recorded by the decode kernel
    float a = 0.f;
    if ((G & 3) == 0) {
      for (int g = 0; g < G; g += 4) {
        const float4 x = *reinterpret_cast<const float4*>(lg + g);
        a += (ex2(x.x - s_lse[g]) + ex2(x.y - s_lse[g + 1])) + (ex2(x.z - s_lse[g + 2]) + ex2(x.w - s_lse[g + 3]));
      }
    } else {
      for (int g = 0; g < G; ++g) a += ex2(lg[g] - s_lse[g]);
    }
    p.scores[((int64_t)page * p.num_kv_heads + w.kv_head) * ps + (key - pg * ps)] += a;
  }
}

}  // namespace

cudaError_t launch_decode_scored(const RunParams& p, int kv_dtype, cudaStream_t s) {
  cudaError_t e = launch_decode_any<true>(p, kv_dtype, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(score_add_kernel, dim3((unsigned)p.num_work), dim3(kScoreThreads), sizeof(float) * p.group, s, p);
}

}  // namespace pkv
