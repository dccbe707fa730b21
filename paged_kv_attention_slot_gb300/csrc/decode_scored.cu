// Decode that accumulates every key's attention weight (pkv_attn_decode_run_scored).
//
// For a request with one new token, KV head h and visible key j the weight is
//   a_j = sum over the query heads g of h of exp(scale q_g.k_j - lse_g),
// and scores[slot(j), h] += a_j.  lse_g is known only after the last key, so the weights take a second
// look at every score.  Reading K again would add half of the decode's own traffic; instead the
// decode kernel leaves its scaled scores (log2 units, 4 bytes per key and query head: 16 bytes
// beside the 512 of a bf16 key row pair at 4 query heads per KV head) in a scratch that mostly stays in
// L2.  A CTA that read a whole unit turns its scores into weights itself when it knows lse; for units
// shared by several CTAs the kernel below does it, on the decode's own work list: a CTA takes the keys
// its decode CTA would take on an even split.  Either way one thread makes one addition to a score per launch,
// so no order of additions matters; it is made at L2 (red.add), so that no thread waits for the old value.

#include "decode_kernel.cuh"

namespace pkv {

namespace {

constexpr int kScoreThreads = 256;
static_assert(kScoredMaxGroup * sizeof(float) <= 48 << 10, "s_lse fits the shared memory of a plain launch");
constexpr int kScoreUnroll = 2;  // groups of four keys in flight per thread

__global__ void __launch_bounds__(kScoreThreads) score_add_kernel(const RunParams p) {
  extern __shared__ float s_lse[];  // [group] log2-sum-exp of the KV head's query heads
  // The work list and the page table were written by kernels that the decode run had waited for before
  // this grid could start (which is when the decode's last CTA has left: it has no earlier trigger), so
  // they may be read before the wait for the decode's own writes.
  const WorkItem w = p.work[blockIdx.x];
  const int G = p.group;
  // the first head group's CTAs add all of the KV head's query heads; a unit that one decode CTA read
  // whole was done there
  if (w.head_group != 0 || (w.num_splits == 1 && G <= kDecodeRows)) return;
  const int share = (w.kv_end - w.kv_begin + w.num_splits - 1) / w.num_splits;
  const int lo = w.kv_begin + w.split * share, hi = min(w.kv_end, lo + share);
  add_weights<kScoreUnroll>(p, w, unit_logits(p, w), s_lse, lo, hi, threadIdx.x, kScoreThreads, [&] {
    pdl_wait();  // the decode run's scaled scores and log-sum-exps
    for (int g = threadIdx.x; g < G; g += kScoreThreads)
      s_lse[g] = __ldcg(p.lse2 + (int64_t)w.q_row * p.num_qo_heads + w.kv_head * G + g);
    __syncthreads();
  });
}

}  // namespace

cudaError_t launch_decode_scored(const RunParams& p, int kv_dtype, bool any_split, cudaStream_t s) {
  cudaError_t e = launch_decode_any<true>(p, kv_dtype, s);
  if (e != cudaSuccess || (!any_split && p.group <= kDecodeRows)) return e;
  return launch_pdl(score_add_kernel, dim3((unsigned)p.num_work), dim3(kScoreThreads), sizeof(float) * p.group, s, p);
}

}  // namespace pkv
