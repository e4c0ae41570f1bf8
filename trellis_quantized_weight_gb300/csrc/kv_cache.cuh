// Shared pieces of the kernels around the paged 8-bit key/value cache.
//
// Cache: codes e4m3 [pages, kv_heads, page_size, D], one float scale per 16
// tokens of a page and head, [pages, kv_heads, page_size / 16].  A stored value
// is code * scale and every scale is a power of two: e4m3 is a floating type, so
// a power of two costs it no precision, scaling is exact, and a block whose
// scale grows keeps its codes' significands (only subnormals round again).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "trellis_device.cuh"

namespace trellis {

constexpr int kKvBlock = 16;             // tokens that share a scale

// What both cache operators read on the device to find their tokens.
struct KvLayout {
    const int* starts;      // [seqs + 1] rows of the packed tokens
    const int* kv_len;      // [seqs] tokens of each sequence, this call's included
    const int* pages;       // [seqs, page_cols]
    int tokens, seqs, page_cols, num_pages;
    int q_heads, kv_heads, page_size, page_shift;
};

// A sequence's rows and tokens.
struct Seq {
    int start, n, p0, total;      // packed rows; the first one's position; cached tokens
};

// n <= 0: it has no rows, or a range that is not inside the packed tokens (nothing of it
// is touched then).  Tokens past the page table are left out of `total`.  The three loads
// do not wait for one another.  (Ordinary loads, here and of the table: trellis_kv_grow may have written both just before,
// while this grid already lived beside it, so they are not read-only for as long as it lives.)
__device__ __forceinline__ Seq load_seq(const KvLayout& l, int s) {
    const int b = l.starts[s], e = l.starts[s + 1], len = l.kv_len[s];
    const long long most = static_cast<long long>(l.page_cols) << l.page_shift;
    Seq q;
    q.start = b;
    q.n = b >= 0 && e <= l.tokens ? e - b : 0;
    q.p0 = len - q.n;
    q.total = len < most ? len : static_cast<int>(most);
    return q;
}

// Page of column c of sequence s, clamped into the pool: a wrong id reads or
// writes a wrong page, never outside the cache.
__device__ __forceinline__ int kv_page_id(const KvLayout& l, int s, int c) {
    return l.pages[static_cast<size_t>(s) * l.page_cols + c];
}
__device__ __forceinline__ int kv_page_of_id(const KvLayout& l, int id) { return min(max(id, 0), l.num_pages - 1); }
__device__ __forceinline__ int kv_page(const KvLayout& l, int s, int c) { return kv_page_of_id(l, kv_page_id(l, s, c)); }

// ---- conversions ------------------------------------------------------------------
// Two e4m3 codes (low byte first) -> f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}
// Four codes of a word -> two f16x2.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    uint16_t a, b;
    asm("mov.b32 {%0, %1}, %2;" : "=h"(a), "=h"(b) : "r"(w));
    lo = e4m3x2_to_f16x2(a);
    hi = e4m3x2_to_f16x2(b);
}
// Two floats -> e4m3x2 (lo in the low byte), nearest even, saturating.
__device__ __forceinline__ uint16_t f32_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f32_to_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t v) {
    float2 r;
    asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
        : "=f"(r.x), "=f"(r.y) : "r"(v));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// log2 and reciprocal of a power of two 2^-60 .. 2^120 by its exponent field;
// a NaN scale (a block that took a NaN or infinite input) stays NaN.
__device__ __forceinline__ float pow2_log2(float s) {
    const int e = static_cast<int>(__float_as_uint(s) >> 23);
    return e < 255 ? static_cast<float>(e - 127) : s;
}
__device__ __forceinline__ float pow2_recip(float s) {
    const uint32_t e = __float_as_uint(s) >> 23;
    return e < 254u ? __uint_as_float((254u - e) << 23) : s;
}

// The same where the factor goes with weights: finite for a NaN scale (whose logarithm makes the
// weights that count NaN), so that a weight of 0 stays 0.
__device__ __forceinline__ float pow2_recip_finite(float s) {
    return __uint_as_float((254u - min(__float_as_uint(s) >> 23, 253u)) << 23);
}

// ---- asynchronous copies and small matrix products ----------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// d[16 x 8] += a[16 x 16] b[16 x 8], f16 operands, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit values held one row per four lanes.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

}  // namespace trellis
