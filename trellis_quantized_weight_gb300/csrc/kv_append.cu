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
// What bounds it: at prompts the bytes (2 in and 1 or 2 out a value) and the rotation's
// single operations; for a step of single tokens the latency of lengths -> page -> values.
// Measured (GPU time; the least bytes at 6.69 TB/s): prompts of 8k tokens 45.5 us (26.5),
// 128 single tokens 6.8 us (0.4), one 3.1 to 3.7 us.  A CTA takes one block of 16
// positions of a sequence and some of its heads ("tasks": a key head, a value head
// or a query head), a warp a task at a time.  The block's rows of the table are read once a
// CTA into shared memory.  A lane takes 8 consecutive values a token (16 bytes in, 8 of
// codes out).  A block's codes need its maximum first: its 16 tokens are read and rotated
// twice, the second time from L1.  In the half layout a pair's other half comes from another
// lane by shuffles.
#include "kv_cache.cuh"
#include "trellis.h"

namespace trellis {

namespace {

constexpr int kWarps = 4;
constexpr int kAppendCtas = 8;           // an SM: 32 warps at 64 registers

struct AppendArgs {
    KvLayout l;
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;   // elements between packed rows
    const float* rope;                        // [rope_rows, rot]: cosines, then sines; or NULL
    int rope_rows, rot, interleaved;          // rot = 0 without a table
    int per_warp;                             // tasks of a warp
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    uint16_t* q_out;                          // [tokens, q_heads, D]
};

__device__ __forceinline__ void unpack8(uint4 v, float2 (&x)[4]) {
    x[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
    x[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    x[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z));
    x[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
}

// (x c + y s) for two values: products and sums rounded one by one.  (Two-wide products
// would be fused into the two-wide sums by the assembler.)
__device__ __forceinline__ float2 turn2(float2 x, float2 y, float c0, float c1, float s0, float s1) {
    return make_float2(__fadd_rn(__fmul_rn(x.x, c0), __fmul_rn(y.x, s0)),
                       __fadd_rn(__fmul_rn(x.y, c1), __fmul_rn(y.y, s1)));
}

// Where float4 k (two of cosines, two of sines) of the 8 pairs cc of a table row stands in
// shared memory: 64 bytes for 8 pairs, turned so that the lanes of a quarter warp, which
// read the same k of neighbouring cc, hit different banks.
__device__ __forceinline__ int table_slot(int cc, int k) { return 4 * cc + (k ^ ((cc >> 1) & 3)); }

// The 8 values of chunk c of a head's row, rotated by the token's table row in shared
// memory when they belong to the first `rot` (a multiple of 16, so a chunk lies in one
// half).  Every lane of the warp calls it; in the half layout lane + `other` holds the
// chunk of the pairs' other halves.
__device__ __forceinline__ void rotated(uint4 raw, int c, const float* row, int rot, int interleaved, bool turn,
                                        float2 (&x)[4]) {
    unpack8(raw, x);
    if (rot == 0) return;
    const int half = rot >> 1, n = half / 8;
    const float4* row4 = reinterpret_cast<const float4*>(row);
    if (interleaved) {
        if (!turn || 8 * c >= rot) return;
        const float4 co = row4[table_slot(c >> 1, c & 1)], si = row4[table_slot(c >> 1, 2 + (c & 1))];
        const float cs[4] = {co.x, co.y, co.z, co.w}, sn[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = turn2(x[i], make_float2(x[i].y, x[i].x), cs[i], cs[i], -sn[i], sn[i]);
    } else {
        const int src = static_cast<int>(threadIdx.x & 31) + (c < n ? n : -n);
        const uint32_t minus = c < n ? 0x80008000u : 0u;       // a turns to a cos + (-b) sin
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, raw.x, src) ^ minus; o.y = __shfl_sync(0xffffffffu, raw.y, src) ^ minus;
        o.z = __shfl_sync(0xffffffffu, raw.z, src) ^ minus; o.w = __shfl_sync(0xffffffffu, raw.w, src) ^ minus;
        if (!turn || c >= 2 * n) return;
        float2 y[4];
        unpack8(o, y);
        const int cc = c < n ? c : c - n;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 co = row4[table_slot(cc, h)], si = row4[table_slot(cc, 2 + h)];
            x[2 * h] = turn2(x[2 * h], y[2 * h], co.x, co.y, si.x, si.y);
            x[2 * h + 1] = turn2(x[2 * h + 1], y[2 * h + 1], co.z, co.w, si.z, si.w);
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
__global__ void __launch_bounds__(kWarps * 32, kAppendCtas) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kChunks = D / 8;                       // 16-byte chunks of a row
    constexpr int kPer = 32 / kChunks;                   // tokens a warp covers in a pass
    constexpr int kGroup = 4;                            // passes loaded side by side
    __shared__ __align__(16) float table[kKvBlock * D];  // the block's rows of `rot` values
    const KvLayout& l = a.l;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane % kChunks, sub = lane / kChunks;
    const int kv_tasks = 2 * l.kv_heads, tasks = kv_tasks + (a.q_out != nullptr ? l.q_heads : 0);
    griddep_wait();
    const int s = blockIdx.y;
    const Seq q = load_seq(l, s);
    const int len = q.p0 + q.n;                          // tokens with these, past the table too
    // blocks of 16 positions (negative ones for rows before position 0), floor division
    const int b0 = q.p0 >> 4, b1 = (len - 1) >> 4;
    if (q.n > 0)
        for (int b = b0 + static_cast<int>(blockIdx.z); b <= b1; b += gridDim.z) {
            const int first = b * kKvBlock;
            const int lo = max(q.p0, first), hi = min(len, first + kKvBlock);
            if (b != b0 + static_cast<int>(blockIdx.z)) __syncthreads();     // the table is read no more
            for (int e = threadIdx.x; e < (hi - lo) * (a.rot / 4); e += kWarps * 32) {
                const int tok = e / (a.rot / 4), at = e % (a.rot / 4);
                const int pos = min(max(lo + tok, 0), a.rope_rows - 1);
                const bool sine = at >= a.rot / 8;
                const int f = sine ? at - a.rot / 8 : at;
                reinterpret_cast<float4*>(table + (lo + tok - first) * a.rot)[table_slot(f >> 1, (sine ? 2 : 0) + (f & 1))] =
                    __ldg(reinterpret_cast<const float4*>(a.rope + static_cast<size_t>(pos) * a.rot) + at);
            }
            if (a.rot > 0) __syncthreads();
            for (int i = 0; i < a.per_warp; ++i) {
                const int task = (blockIdx.x * a.per_warp + i) * kWarps + warp;
                if (task >= tasks) break;
                const bool query = task >= kv_tasks, key = task < l.kv_heads;
                const int h = query ? task - kv_tasks : key ? task : task - l.kv_heads;
                const uint16_t* src = query ? a.q : key ? a.k : a.v;
                const long long stride = query ? a.q_stride : key ? a.k_stride : a.v_stride;
                const int rot = query || key ? a.rot : 0;
                // this lane's chunk of the block's slot 0 (before the rows where the block starts earlier)
                const uint16_t* lane_src = src + (static_cast<long long>(q.start) + (first + sub - q.p0)) * stride + h * D + 8 * c;
                // kGroup passes' inputs are loaded side by side
                auto load = [&](int p0, uint4 (&raw)[kGroup]) {
                    const uint16_t* at = lane_src + p0 * kPer * stride;
#pragma unroll
                    for (int p = 0; p < kGroup; ++p) {
                        const int pos = first + (p0 + p) * kPer + sub;
                        raw[p] = make_uint4(0u, 0u, 0u, 0u);
                        if (pos >= lo && pos < hi) raw[p] = *reinterpret_cast<const uint4*>(at);
                        at += kPer * stride;
                    }
                };
                // passes that hold tokens [from, to) of the block
                auto passes = [&](int from, int to, auto&& body) {
#pragma unroll 1
                    for (int p0 = (from - first) / (kPer * kGroup) * kGroup; first + p0 * kPer < to; p0 += kGroup) {
                        uint4 raw[kGroup];
                        load(p0, raw);
#pragma unroll
                        for (int p = 0; p < kGroup; ++p) {
                            const int row = (p0 + p) * kPer + sub, pos = first + row;
                            float2 x[4];
                            // a query row before position 0 (an idle slot) is stored as it is
                            rotated(raw[p], c, table + row * a.rot, rot, a.interleaved, pos >= 0, x);
                            if (pos >= from && pos < to) body(pos, x);
                        }
                    }
                };
                if (query) {
                    uint16_t* lane_out = a.q_out + ((static_cast<long long>(q.start) + (first - q.p0)) * l.q_heads + h) * D + 8 * c;
                    const int out_stride = l.q_heads * D;
                    passes(lo, hi, [&](int pos, float2 (&x)[4]) {
                        *reinterpret_cast<uint4*>(lane_out + (pos - first) * out_stride) =
                            make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                                       pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
                    });
                    continue;
                }
                // tokens of the block that have a slot: from max(p0, 0) to the table's end
                const int from = max(lo, 0), to = min(hi, q.total);
                if (from >= to) continue;
                const int kept = from - first;            // tokens of the block from before
                const int slot0 = first & (l.page_size - 1);
                const size_t unit = static_cast<size_t>(kv_page(l, s, first >> l.page_shift)) * l.kv_heads + h;
                uint8_t* out = (key ? a.k_codes : a.v_codes) + (unit * l.page_size + slot0) * D;
                float* scale = (key ? a.k_scales : a.v_scales) + unit * (l.page_size / kKvBlock) + slot0 / kKvBlock;
                float had = 0.0f;
                if (kept > 0) had = *scale;
                uint32_t most = 0u;
                passes(from, to, [&](int, float2 (&x)[4]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        most = max(most, max(__float_as_uint(x[j].x) & 0x7fffffffu, __float_as_uint(x[j].y) & 0x7fffffffu));
                });
                most = __reduce_max_sync(0xffffffffu, most);
                float sc = block_scale(most);
                if (kept > 0) {
                    // NaN on either side stays NaN
                    const float now = (had != had || sc != sc) ? __uint_as_float(0x7fc00000u) : fmaxf(had, sc);
                    if (now != had) {
                        const float ratio = __fdiv_rn(had, now);
                        for (int tok = sub; tok < kept; tok += kPer) {
                            uint2* at = reinterpret_cast<uint2*>(out + tok * D) + c;
                            uint2 w = *at;
                            uint32_t ww[2] = {w.x, w.y};
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                uint32_t u0, u1;
                                e4m3x4_to_f16x2(ww[j], u0, u1);
                                const float2 f0 = f16x2_to_f32(u0), f1 = f16x2_to_f32(u1);
                                ww[j] = static_cast<uint32_t>(f32_to_e4m3x2(f0.x * ratio, f0.y * ratio)) |
                                        (static_cast<uint32_t>(f32_to_e4m3x2(f1.x * ratio, f1.y * ratio)) << 16);
                            }
                            *at = make_uint2(ww[0], ww[1]);
                        }
                    }
                    sc = now;
                }
                const float inv = pow2_recip(sc);         // exact: the scale is a power of two
                passes(from, to, [&](int pos, float2 (&x)[4]) {
                    uint2 w;
                    w.x = static_cast<uint32_t>(f32_to_e4m3x2(x[0].x * inv, x[0].y * inv)) |
                          (static_cast<uint32_t>(f32_to_e4m3x2(x[1].x * inv, x[1].y * inv)) << 16);
                    w.y = static_cast<uint32_t>(f32_to_e4m3x2(x[2].x * inv, x[2].y * inv)) |
                          (static_cast<uint32_t>(f32_to_e4m3x2(x[3].x * inv, x[3].y * inv)) << 16);
                    reinterpret_cast<uint2*>(out + (pos - first) * D)[c] = w;
                });
                __syncwarp();                             // `had` was read by every lane
                if (lane == 0) *scale = sc;
            }
        }
    griddep_launch_dependents();
}

template <int D>
cudaError_t launch(const AppendArgs& a, int blocks, cudaStream_t stream) {
    const int tasks = 2 * a.l.kv_heads + (a.q_out != nullptr ? a.l.q_heads : 0);
    const int warps = (tasks + a.per_warp - 1) / a.per_warp;
    return launch_programmatic_grid(kv_append_kernel<D>, dim3((warps + kWarps - 1) / kWarps, a.l.seqs, blocks),
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
    // tasks of a warp: two, so that fewer CTAs read the same table rows (8165 prompt tokens
    // and 48 heads: 45.5 us with 2, 46.9 with 1, 49.7 with 4, whose last wave is ragged);
    // one where that would leave fewer than 16 warps an SM
    const int tasks = 2 * kv_heads + (q != nullptr ? q_heads : 0);
    const long long units = (static_cast<long long>(tokens) + kKvBlock - 1) / kKvBlock * tasks;
    DeviceInfo dev;
    const int rc_dev = device_info(dev);
    if (rc_dev != TRELLIS_OK) return rc_dev;
    const long long per = units / (16ll * dev.num_sms);
    a.per_warp = static_cast<int>(per < 1 ? 1 : per > 2 ? 2 : per);
    const cudaError_t e = head_dim == 64 ? launch<64>(a, blocks, stream)
                          : head_dim == 128 ? launch<128>(a, blocks, stream) : launch<256>(a, blocks, stream);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}
