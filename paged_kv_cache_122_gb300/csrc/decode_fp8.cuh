// Parameters and launchers of attention over the 8-bit paged cache.
#pragma once

#include "../../include/pagedkv_fp8.h"
#include "decode.cuh"

namespace pk {

// k_cache and v_cache of the base are unused: the caches are k8 and v8,
// [P, Hkv, B, D] e4m3, with scales [P, Hkv].
struct DecodeFp8Params : DecodeParams {
    const uint8_t *k8, *v8;
    const float *k_scales, *v_scales;
};

// Tensor cores (tcgen05, 8-bit operands): decode and, with cu_q_lens set,
// several query tokens per sequence (q_len a power of two, G * q_len <= 16).
cudaError_t launch_decode_fp8_tensor_core(const DecodeFp8Params &p, cudaStream_t stream);

}  // namespace pk
