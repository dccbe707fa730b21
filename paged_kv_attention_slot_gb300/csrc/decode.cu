// The decode runs: instances of the decode kernel (decode_kernel.cuh) without attention-weight scores.

#include "decode_kernel.cuh"

namespace pkv {

int decode_ctas_per_sm(int kv_dtype, int head_dim, int group) {
  const bool nb2 = group > 8;
  if (kv_dtype == PKV_NVFP4)
    return group <= 4 ? DecodeCfg<128, PKV_NVFP4, 1, 4>::CTAS
           : !nb2     ? DecodeCfg<128, PKV_NVFP4, 1, 8>::CTAS
                      : DecodeCfg<128, PKV_NVFP4, 2, 8>::CTAS;
  if (kv_dtype == PKV_FP8_E4M3)
    return nb2 ? DecodeCfg<128, PKV_FP8_E4M3, 2>::CTAS : DecodeCfg<128, PKV_FP8_E4M3, 1>::CTAS;
  if (head_dim == 64) return nb2 ? DecodeCfg<64, PKV_BF16, 2>::CTAS : DecodeCfg<64, PKV_BF16, 1>::CTAS;
  return nb2 ? DecodeCfg<128, PKV_BF16, 2>::CTAS : DecodeCfg<128, PKV_BF16, 1>::CTAS;
}

cudaError_t launch_decode(const RunParams& p, int kv_dtype, cudaStream_t s) {
  return launch_decode_any<false>(p, kv_dtype, s);
}

}  // namespace pkv
