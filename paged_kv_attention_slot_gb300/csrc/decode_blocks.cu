// Decode over selected pages (pkv_attn_decode_run_blocks): instances of the decode kernel (decode_kernel.cuh) that look
// up their pages through the selection: page = kv_indices[blocks[key / page_size]], two dependent reads, made once per
// CTA for all of its unit's pages, into a table in shared memory (beyond 1024 pages, a tile ahead).  Before every
// tile they cost 64 requests of 1024 selected keys (260 MB) 44.5 us instead of 43.2 to 44.1 (39.1 at the measured
// copy rate; the rest is two waves of CTAs that each begin with a chain of reads), and 2 x 4096 keys of a 4-bit pool 11.4
// instead of 10.6, of which the merge of 16 parts of 8 rows takes 3.
// A plan over few selected keys is cut like any other (pieces of 128 keys: 13.4 us, 512: 11.4).

#include "decode_blocks.h"
#include "decode_kernel.cuh"

namespace pkv {

cudaError_t launch_decode_blocks(const RunParams& p, int kv_dtype, cudaStream_t s) {
  return launch_decode_any<false, true>(p, kv_dtype, s);
}

}  // namespace pkv
