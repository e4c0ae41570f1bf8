// What the two attention kernels over the paged cache share.
#pragma once

#include <cstddef>

#include "kv_cache.cuh"

namespace trellis {

struct AttendArgs {
    KvLayout l;
    const uint16_t* q;
    long long q_stride;          // elements between packed rows
    int group;                   // query heads of a key head
    int window;                  // tokens a row sees, itself included; 0: all before it
    float scale_log2;            // score factor times log2(e)
    const uint8_t *k_codes, *v_codes;
    const float *k_scales, *v_scales;
    uint16_t* out;               // [tokens, q_heads, D]
    unsigned int* counters;      // workspace: zero before and after every call
    float* partials;
};

// The workspace starts with the counters, in the region that the products' workspace
// reserves for theirs, so one buffer serves both.
constexpr size_t kKvCounterBytes = size_t(1) << 20;

// Exponent by which a query row is scaled to f16: the largest magnitude (bf16 bits)
// lands in [1, 2).  Clamped so that the factor and its inverse stay normal floats.
__device__ __forceinline__ int query_exponent(uint32_t most) {
    const int e = static_cast<int>(most >> 7) - 127;
    return min(max(e, -100), 126);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

// Row r of a sequence's rows to a key head (token r / group, query head r % group):
// values d .. d + 3 of the output.  A row that sees nothing (l == 0) is zero.
__device__ __forceinline__ void store_row4(const AttendArgs& a, int start, int head, int r, int D, int d, float4 acc,
                                           float l) {
    const size_t row = static_cast<size_t>(start) + r / a.group;
    const int h = head * a.group + r % a.group;
    const float inv = 1.0f / l;
    uint2 w = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (l == 0.0f) w = make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(a.out + (row * a.l.q_heads + h) * D + d) = w;
}

size_t kv_stream_workspace_bytes(int head_dim, int rows, const DeviceInfo& dev);
int launch_kv_stream(const AttendArgs& a, int head_dim, int rows, const DeviceInfo& dev, cudaStream_t stream);
size_t kv_tile_workspace_bytes(int tokens, int seqs, int q_heads, int kv_heads, int head_dim, const DeviceInfo& dev);
int launch_kv_tile(const AttendArgs& a, int head_dim, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace trellis
