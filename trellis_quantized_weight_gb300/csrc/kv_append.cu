// trellis_kv_append: rotates a step's queries and keys, quantizes its keys and
// values and writes them into the paged cache, in one launch.
//
//   rotation   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first
//              `rot` values of a head: (i, i + rot/2), or (2i, 2i + 1); cos and sin
//              of the token's position come from the caller's float table.  The
//              products and sums are single fp32 operations (no fused multiply-add),
//              so a key's code does not depend on how a compiler pairs them.
//   scale      of a block of 16 cached tokens and a head: the smallest power of two
//              s >= 2^-60 with max|x| <= 448 s, never below the scale the block has
//              if it holds tokens from before; NaN when an input is NaN or infinite.
//   codes      e4m3(x / s), nearest even.  When a block's scale grows, the codes from
//              before are multiplied by the (power of two) ratio and rounded again.
//
// One warp owns one (sequence, cache block, key or value head) or one (sequence,
// 16 new tokens, query head): it holds the block's values in registers between
// the maximum and the codes, so every input is read from HBM once.  A lane takes
// 8 consecutive values (16 bytes in, 8 bytes of codes out); a pair's other half in
// the half layout is read from the neighbour's 16 bytes, an L1 hit.
#include "kv_cache.cuh"
#include "trellis.h"

namespace trellis {

namespace {

constexpr int kWarps = 4;

struct AppendArgs {
    KvLayout l;
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;   // elements between packed rows
    const float* rope;                        // [rope_rows, rot]: cosines, then sines; or NULL
    int rope_rows, rot, interleaved;
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    uint16_t* q_out;                          // [tokens, q_heads, D]
};

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

// Values 8c .. 8c+7 of a head's row, rotated when they belong to its first `rot`
// values (rot is a multiple of 16, so a chunk lies in one half).
__device__ __forceinline__ void load_rotated(const uint16_t* __restrict__ row, int c, const float* __restrict__ table,
                                             int rot, int interleaved, float (&x)[8]) {
    const uint4* r4 = reinterpret_cast<const uint4*>(row);
    const uint4 own = __ldg(r4 + c);
    unpack8(own, x);
    if (table == nullptr || 8 * c >= rot) return;
    const int half = rot >> 1;
    if (interleaved) {
        const float4 co = __ldg(reinterpret_cast<const float4*>(table + 4 * c));
        const float4 si = __ldg(reinterpret_cast<const float4*>(table + half + 4 * c));
        const float cs[4] = {co.x, co.y, co.z, co.w}, sn[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a, cs[i]), __fmul_rn(b, sn[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(b, cs[i]), __fmul_rn(a, sn[i]));
        }
    } else {
        const bool low = 8 * c < half;
        const int i0 = low ? 8 * c : 8 * c - half;
        float y[8];
        unpack8(__ldg(r4 + (low ? c + half / 8 : c - half / 8)), y);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 co = __ldg(reinterpret_cast<const float4*>(table + i0) + h);
            const float4 si = __ldg(reinterpret_cast<const float4*>(table + half + i0) + h);
            const float cs[4] = {co.x, co.y, co.z, co.w}, sn[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float own_c = __fmul_rn(x[4 * h + i], cs[i]), other_s = __fmul_rn(y[4 * h + i], sn[i]);
                x[4 * h + i] = low ? __fsub_rn(own_c, other_s) : __fadd_rn(own_c, other_s);
            }
        }
    }
}

// The smallest power of two s >= 2^-60 with a <= 448 s, from a's bits: 448 is
// 1.75 * 2^8, so adding 0x1FFFFF carries into the exponent exactly when the
// significand is above 1.75.  NaN for a NaN or infinite a.
__device__ __forceinline__ float block_scale(uint32_t abits) {
    if (abits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    int e = static_cast<int>((abits + 0x1FFFFFu) >> 23) - 127 - 8;
    e = e < -60 ? -60 : e;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    griddep_wait();
    constexpr int kChunks = D / 8;                       // 16-byte chunks of a row
    constexpr int kPer = 32 / kChunks;                   // tokens a warp covers in a pass
    constexpr int kPasses = kKvBlock / kPer;
    const KvLayout& l = a.l;
    const int lane = threadIdx.x & 31;
    const int task = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int s = blockIdx.y;
    const int c = lane % kChunks, sub = lane / kChunks;
    int start, n;
    const int kv_tasks = 2 * l.kv_heads;
    const int tasks = kv_tasks + (a.q_out != nullptr ? l.q_heads : 0);
    if (task < tasks && kv_rows(l, s, &start, &n)) {
        const int total = kv_total(l, s);
        const int p0 = __ldg(l.kv_len + s) - n;          // position of the first new token
        if (task >= kv_tasks) {
            // ---- a query head: rotate and store
            const int h = task - kv_tasks;
            for (int b = blockIdx.z; b * kKvBlock < n; b += gridDim.z) {
#pragma unroll 4
                for (int i = 0; i < kPasses; ++i) {
                    const int tok = b * kKvBlock + i * kPer + sub;
                    if (tok >= n) continue;
                    const int pos = p0 + tok;
                    // a row before position 0 (an idle slot) is stored as it is
                    const float* table = a.rope == nullptr || pos < 0
                        ? nullptr : a.rope + static_cast<size_t>(min(pos, a.rope_rows - 1)) * a.rot;
                    const size_t row = static_cast<size_t>(start) + tok;
                    float x[8];
                    load_rotated(a.q + row * a.q_stride + h * D, c, table, a.rot, a.interleaved, x);
                    uint4 o;
                    o.x = pack_bf16x2(x[0], x[1]); o.y = pack_bf16x2(x[2], x[3]);
                    o.z = pack_bf16x2(x[4], x[5]); o.w = pack_bf16x2(x[6], x[7]);
                    reinterpret_cast<uint4*>(a.q_out + (row * l.q_heads + h) * D)[c] = o;
                }
            }
        } else {
            const bool key = task < l.kv_heads;
            const int h = key ? task : task - l.kv_heads;
            const uint16_t* src = key ? a.k : a.v;
            const long long stride = key ? a.k_stride : a.v_stride;
            uint8_t* codes = key ? a.k_codes : a.v_codes;
            float* scales = key ? a.k_scales : a.v_scales;
            const float* rope = key ? a.rope : nullptr;
            const int first = max(p0, 0);
            for (int b = first / kKvBlock + static_cast<int>(blockIdx.z); b * kKvBlock < total; b += gridDim.z) {
                const int lo = max(first, b * kKvBlock), hi = min(total, (b + 1) * kKvBlock);
                const int kept = lo - b * kKvBlock;       // tokens of the block from before
                const int slot0 = (b * kKvBlock) & (l.page_size - 1);
                const size_t unit = static_cast<size_t>(kv_page(l, s, (b * kKvBlock) >> l.page_shift)) * l.kv_heads + h;
                uint8_t* out = codes + (unit * l.page_size + slot0) * D;
                float* scale = scales + unit * (l.page_size / kKvBlock) + slot0 / kKvBlock;
                float x[kPasses][8];
                uint32_t most = 0u;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int pos = b * kKvBlock + i * kPer + sub;
                    if (pos < lo || pos >= hi) continue;
                    const float* table = rope == nullptr
                        ? nullptr : rope + static_cast<size_t>(min(pos, a.rope_rows - 1)) * a.rot;
                    const size_t row = static_cast<size_t>(start) + (pos - p0);
                    load_rotated(src + row * stride + h * D, c, table, a.rot, a.interleaved, x[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(x[i][j]) & 0x7fffffffu);
                }
                most = __reduce_max_sync(0xffffffffu, most);
                float sc = block_scale(most);
                if (kept > 0) {
                    const float had = *scale;
                    // NaN on either side stays NaN
                    const float now = (had != had || sc != sc) ? __uint_as_float(0x7fc00000u) : fmaxf(had, sc);
                    if (now != had) {
                        const float ratio = __fdiv_rn(had, now);
                        for (int t = sub; t < kept; t += kPer) {
                            uint2* p = reinterpret_cast<uint2*>(out + t * D) + c;
                            uint2 w = *p;
                            uint32_t* ww = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                uint32_t u0, u1;
                                e4m3x4_to_f16x2(ww[q], u0, u1);
                                const float2 f0 = f16x2_to_f32(u0), f1 = f16x2_to_f32(u1);
                                ww[q] = static_cast<uint32_t>(f32_to_e4m3x2(f0.x * ratio, f0.y * ratio)) |
                                        (static_cast<uint32_t>(f32_to_e4m3x2(f1.x * ratio, f1.y * ratio)) << 16);
                            }
                            *p = w;
                        }
                    }
                    sc = now;
                }
                const float inv = pow2_recip(sc);         // exact: the scale is a power of two
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int pos = b * kKvBlock + i * kPer + sub;
                    if (pos < lo || pos >= hi) continue;
                    uint2 w;
                    w.x = static_cast<uint32_t>(f32_to_e4m3x2(x[i][0] * inv, x[i][1] * inv)) |
                          (static_cast<uint32_t>(f32_to_e4m3x2(x[i][2] * inv, x[i][3] * inv)) << 16);
                    w.y = static_cast<uint32_t>(f32_to_e4m3x2(x[i][4] * inv, x[i][5] * inv)) |
                          (static_cast<uint32_t>(f32_to_e4m3x2(x[i][6] * inv, x[i][7] * inv)) << 16);
                    reinterpret_cast<uint2*>(out + (pos - b * kKvBlock) * D)[c] = w;
                }
                __syncwarp();                             // `had` was read by every lane
                if (lane == 0) *scale = sc;
            }
        }
    }
    griddep_launch_dependents();
}

template <int D>
cudaError_t launch(const AppendArgs& a, int blocks, cudaStream_t stream) {
    const int tasks = 2 * a.l.kv_heads + (a.q_out != nullptr ? a.l.q_heads : 0);
    return launch_programmatic_grid(kv_append_kernel<D>, dim3((tasks + kWarps - 1) / kWarps, a.l.seqs, blocks),
                                    kWarps * 32, 0, stream, a);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

// Checks shared by the cache operators, in this order: pointers, sizes, alignment.
int check_kv(const int* starts, const int* kv_len, const int* pages, int tokens, int seqs, int max_q, int page_cols,
             int num_pages, int q_heads, int kv_heads, int head_dim, int page_size, const void* k_codes,
             const void* v_codes, const float* k_scales, const float* v_scales) {
    if (starts == nullptr || kv_len == nullptr || pages == nullptr || k_codes == nullptr || v_codes == nullptr ||
        k_scales == nullptr || v_scales == nullptr)
        return TRELLIS_ERR_NULL;
    if (tokens < 0 || seqs < 1 || max_q < 1 || page_cols < 1 || num_pages < 1 || kv_heads < 1 || q_heads < kv_heads ||
        q_heads % kv_heads != 0)
        return TRELLIS_ERR_SHAPE;
    if (seqs > kKvMaxSeqs || q_heads > kKvMaxHeads) return TRELLIS_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return TRELLIS_ERR_UNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return TRELLIS_ERR_UNSUPPORTED;
    if (!aligned(starts, 4) || !aligned(kv_len, 4) || !aligned(pages, 4) || !aligned(k_scales, 4) ||
        !aligned(v_scales, 4) || !aligned(k_codes, 16) || !aligned(v_codes, 16))
        return TRELLIS_ERR_ALIGN;
    return TRELLIS_OK;
}

KvLayout kv_layout(const int* starts, const int* kv_len, const int* pages, int tokens, int seqs, int page_cols,
                   int num_pages, int q_heads, int kv_heads, int page_size) {
    KvLayout l;
    l.starts = starts; l.kv_len = kv_len; l.pages = pages;
    l.tokens = tokens; l.seqs = seqs; l.page_cols = page_cols; l.num_pages = num_pages;
    l.q_heads = q_heads; l.kv_heads = kv_heads; l.page_size = page_size;
    l.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    return l;
}

}  // namespace trellis

extern "C" int trellis_kv_append(const uint16_t* q, long long q_stride, const uint16_t* k, long long k_stride,
                                 const uint16_t* v, long long v_stride, const int* starts, const int* kv_len,
                                 const int* pages, int tokens, int seqs, int max_q, int page_cols, int num_pages,
                                 int q_heads, int kv_heads, int head_dim, int page_size, const float* rope,
                                 int rope_rows, int rot, int interleaved, uint8_t* k_codes, uint8_t* v_codes,
                                 float* k_scales, float* v_scales, uint16_t* q_out, cudaStream_t stream) {
    using namespace trellis;
    if (k == nullptr || v == nullptr || (q == nullptr) != (q_out == nullptr)) return TRELLIS_ERR_NULL;
    const int rc = check_kv(starts, kv_len, pages, tokens, seqs, max_q, page_cols, num_pages, q_heads, kv_heads,
                            head_dim, page_size, k_codes, v_codes, k_scales, v_scales);
    if (rc != TRELLIS_OK) return rc;
    const long long kv_row = static_cast<long long>(kv_heads) * head_dim;
    if (k_stride < kv_row || v_stride < kv_row ||
        (q != nullptr && q_stride < static_cast<long long>(q_heads) * head_dim))
        return TRELLIS_ERR_SHAPE;
    if (rope != nullptr) {
        if (rope_rows < 1) return TRELLIS_ERR_SHAPE;
        if (rot < 16 || rot > head_dim || rot % 16 != 0) return TRELLIS_ERR_UNSUPPORTED;
    }
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(rope, 16) ||
        k_stride % 8 != 0 || v_stride % 8 != 0 || (q != nullptr && q_stride % 8 != 0))
        return TRELLIS_ERR_ALIGN;
    if (tokens == 0) return TRELLIS_OK;
    AppendArgs a;
    a.l = kv_layout(starts, kv_len, pages, tokens, seqs, page_cols, num_pages, q_heads, kv_heads, page_size);
    a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.rope = rope; a.rope_rows = rope_rows; a.rot = rope != nullptr ? rot : 0; a.interleaved = interleaved != 0;
    a.k_codes = k_codes; a.v_codes = v_codes; a.k_scales = k_scales; a.v_scales = v_scales;
    a.q_out = q_out;
    // blocks of the longest sequence as the caller gives it, one more when it starts
    // inside a block (only the grid's depth: a longer sequence is looped over)
    int blocks = (max_q > tokens ? tokens : max_q) / kKvBlock + 1;
    if (max_q > 1 && max_q % kKvBlock != 0) blocks += 1;
    // and no deeper than eight times the blocks that the packed tokens can touch, so
    // that one long sequence among many short ones does not launch mostly empty CTAs
    const long long deep = 8ll * (tokens / kKvBlock + 2ll * seqs) / seqs;
    if (blocks > deep) blocks = static_cast<int>(deep);
    if (blocks > 16384) blocks = 16384;
    const cudaError_t e = head_dim == 64 ? launch<64>(a, blocks, stream)
                          : head_dim == 128 ? launch<128>(a, blocks, stream) : launch<256>(a, blocks, stream);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}
