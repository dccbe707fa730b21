// Decode over selected pages (pkv_attn_decode_run_blocks): instances of the decode kernel (decode_kernel.cuh) that look
// up their pages through the selection.  A list per KV head costs a second dependent look-up per tile, which is made a
// tile ahead like the first.

#include "decode_blocks.h"
#include "decode_kernel.cuh"

namespace pkv {

cudaError_t launch_decode_blocks(const RunParams& p, int kv_dtype, cudaStream_t s) {
  return launch_decode_any<false, true>(p, kv_dtype, s);
}

}  // namespace pkv
