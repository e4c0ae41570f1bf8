// Products with 4-bit weights in groups: what the kernels and the entry point share.
//
//   out[m, n] = s_m sum_g ( scale[n, g] sum_{k in g} (c - 8) x[m, k] + (bias[n, g] + 8 scale[n, g]) sum_{k in g} x[m, k] )
//
// with the second term left out without biases (a weight is then scale (c - 8)).  c - 8 is a whole
// number of at most 8, exact in bf16, and so is an activation in e4m3: the tensor cores multiply
// codes by activations exactly into fp32 sums, and scales and biases meet those sums in fp32.  No
// weight is rounded.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "kv_cache.cuh"
#include "trellis.h"
#include "trellis_device.cuh"

namespace trellis {

struct Q4Args {
    const void* x;                  // bf16 or e4m3 [M, K]
    const uint32_t* codes;          // [N, K / 8]
    const uint16_t* scales;         // bf16 [N, groups]
    const uint16_t* biases;         // the same, or NULL
    const float* x_scales;          // [M], with e4m3 activations
    uint16_t* out;                  // bf16 [M, N]
    int M, K, N, groups;
};

// The codes in the low bits of a word's halves as a bf16 pair of c - 8: a code in the low bits of 128's significand is
// 128 + c, and 136 comes off exactly.  (One logical instruction: left to itself the compiler takes one for the mask and
// one for the exponent.)
template <int kMinus>
__device__ __forceinline__ uint32_t code_pair(uint32_t v) {
    uint32_t c, r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(c) : "r"(v), "r"(0x000f000fu), "r"(0x43004300u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(c), "r"(kMinus == 136 ? 0x43084308u : 0x43004300u));
    return r;
}

// Codes 0 and 4, 1 and 5, 2 and 6, 3 and 7 of a word as such pairs.
__device__ __forceinline__ void q4_pairs(uint32_t w, uint32_t (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = code_pair<136>(w >> (4 * i));
}

// Eight activations, bf16 or e4m3, as bf16 pairs.
__device__ __forceinline__ uint4 q4_load_x(const void* x, bool eight, size_t at) {
    if (!eight) return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(x) + at));
    uint32_t f[4], r[4];
    e4m3x4_to_f16x2(v.x, f[0], f[1]);
    e4m3x4_to_f16x2(v.y, f[2], f[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 d = f16x2_to_f32(f[i]);
        r[i] = pack_bf16x2(d.x, d.y);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The kernels of group size 32, 64 and 128 are translation units of their own.
template <int G>
cudaError_t launch_q4_mma(const Q4Args& a, const DeviceInfo& dev, cudaStream_t stream);

// On the tensor cores, for more rows; workspace bytes: 0 where it takes none.
size_t q4_tc_workspace_bytes(int M, int K, bool eight);
cudaError_t launch_q4_tc(const Q4Args& a, int group, void* workspace, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace trellis
