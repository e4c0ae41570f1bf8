// trellis_lora_add: the low-rank adapters of many requests, added to the output of
// a projection that they share.
//
//   out[m] = bf16( y[m] + s_a * B_a (A_a x[m]) ),  a = the adapter of row m's request
//
// Two launches: h = x A^T (sums over K, the long axis), then out = y + s h B^T (over
// the rank).  Both are skinny: at few rows they read A and B (2 R (K + N) bytes an
// adapter), at many rows x, y and out, and the tensor work is a few per cent of
// either time, so m16n8k16 with bf16 operands and fp32 sums is enough.
//
// * Fragments come straight from global memory: the order of a sum's terms is free,
//   so a lane's 8 consecutive elements (16 bytes) serve as its operands of two
//   products, in both factors alike.
// * h is summed over K by the warps of a CTA and over K splits by the second kernel,
//   always in the same order.  It stays fp32; the second product takes it as the
//   sum of two bf16 (16 significant bits), so that it rounds far below the one
//   rounding of the result.
// * Rows are cut into tiles inside each request's rows, 16 or 64 rows a CTA.
#include "kernels.h"
#include "kv_cache.cuh"
#include "trellis.h"

namespace trellis {

namespace {

constexpr int kLoraWarps = 8;
constexpr int kLoraThreads = kLoraWarps * 32;

struct LoraArgs {
    const uint16_t *y, *x, *a, *b;
    const float* scales;         // [adapters]
    const int* starts;           // [segments + 1] rows of each request
    const int* which;            // [segments] adapter, or none where outside 0 .. adapters - 1
    uint16_t* out;
    float* h;                    // [splits][M][R]
    int M, K, N, R, adapters, segments, splits;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Segment and rows [row, end) of row tile `tile` (tiles of kTileRows rows, counted
// segment by segment); false past the last one.  Every thread calls it.
template <int kTileRows>
__device__ bool find_tile(const LoraArgs& p, int tile, int* smem, int* seg, int* row, int* end) {
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        int base = 0, got = -1, r = 0, e = 0;
        for (int s0 = 0; s0 < p.segments && got < 0; s0 += 32) {
            const int s = s0 + lane;
            int a = 0, b = 0;
            if (s < p.segments) {
                a = max(0, __ldg(p.starts + s));
                b = min(p.M, __ldg(p.starts + s + 1));
            }
            const int n = b > a ? (b - a + kTileRows - 1) / kTileRows : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const int at = base + incl - n;
            const unsigned hit = __ballot_sync(0xffffffffu, tile >= at && tile < at + n);
            if (hit != 0u) {
                const int src = __ffs(hit) - 1;
                r = __shfl_sync(0xffffffffu, a + (tile - at) * kTileRows, src);
                e = __shfl_sync(0xffffffffu, b, src);
                got = s0 + src;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) { smem[0] = got; smem[1] = r; smem[2] = min(e, r + kTileRows); }
    }
    __syncthreads();
    *seg = smem[0]; *row = smem[1]; *end = smem[2];
    return *seg >= 0;
}

__device__ __forceinline__ int adapter_of(const LoraArgs& p, int seg) {
    const int w = __ldg(p.which + seg);
    return w >= 0 && w < p.adapters ? w : -1;
}

// h[split][row][r] = sum over the split's k of x[row][k] a[r][k].  kRowGroups groups of
// 16 rows; the other warps of the CTA, and the splits, share the sum over k in slabs of 32.
template <int NT, int kRowGroups>
__global__ void __launch_bounds__(kLoraThreads) lora_down_kernel(const __grid_constant__ LoraArgs p) {
    constexpr int kKGroups = kLoraWarps / kRowGroups;
    constexpr int kTileRows = 16 * kRowGroups;
    extern __shared__ __align__(16) float sums[];        // [kKGroups][kTileRows][R]
    __shared__ int found[4];
    griddep_wait();
    int seg, row0, end;
    const bool any = find_tile<kTileRows>(p, blockIdx.x, found, &seg, &row0, &end);
    const int w = any ? adapter_of(p, seg) : -1;
    if (w >= 0) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int rg = warp % kRowGroups, kg = warp / kRowGroups;
        const int r0 = row0 + rg * 16 + g, r1 = r0 + 8;
        const uint16_t* x0 = p.x + static_cast<size_t>(min(r0, end - 1)) * p.K;
        const uint16_t* x1 = p.x + static_cast<size_t>(min(r1, end - 1)) * p.K;
        const uint16_t* a = p.a + static_cast<size_t>(w) * p.R * p.K;
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
        const int slabs = (p.K + 31) / 32;
        for (int sl = blockIdx.y * kKGroups + kg; sl < slabs; sl += p.splits * kKGroups) {
            const int k = sl * 32 + t * 8;
            const bool in = k < p.K;
            uint4 u0 = make_uint4(0u, 0u, 0u, 0u), u1 = u0, b[NT];
            if (in) {
                u0 = __ldg(reinterpret_cast<const uint4*>(x0 + k));
                u1 = __ldg(reinterpret_cast<const uint4*>(x1 + k));
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                b[i] = make_uint4(0u, 0u, 0u, 0u);
                if (in && 8 * i + g < p.R)
                    b[i] = __ldg(reinterpret_cast<const uint4*>(a + static_cast<size_t>(8 * i + g) * p.K + k));
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                mma_bf16(acc[i], u0.x, u1.x, u0.y, u1.y, b[i].x, b[i].y);
                mma_bf16(acc[i], u0.z, u1.z, u0.w, u1.w, b[i].z, b[i].w);
            }
        }
        float* mine = sums + (kg * kTileRows + rg * 16) * p.R;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int c = 8 * i + 2 * t;
            if (c < p.R) {
                *reinterpret_cast<float2*>(mine + g * p.R + c) = make_float2(acc[i][0], acc[i][1]);
                *reinterpret_cast<float2*>(mine + (g + 8) * p.R + c) = make_float2(acc[i][2], acc[i][3]);
            }
        }
        __syncthreads();
        const int live = (end - row0) * p.R;
        float* h = p.h + (static_cast<size_t>(blockIdx.y) * p.M + row0) * p.R;
        for (int e = threadIdx.x; e < live; e += kLoraThreads) {
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < kKGroups; ++q) v += sums[q * kTileRows * p.R + e];
            h[e] = v;
        }
    }
    griddep_launch_dependents();
}

// out = y + s h B^T for a tile of rows and kCols columns a pass; NT slabs of 32 of the rank.
template <int NS, int kRowGroups, bool kVec>
__global__ void __launch_bounds__(kLoraThreads) lora_up_kernel(const __grid_constant__ LoraArgs p, int cols_per_cta) {
    constexpr int kColGroups = kLoraWarps / kRowGroups;
    constexpr int kTileRows = 16 * kRowGroups;
    __shared__ int found[4];
    griddep_wait();
    int seg, row0, end;
    const bool any = find_tile<kTileRows>(p, blockIdx.x, found, &seg, &row0, &end);
    if (any) {
        const int w = adapter_of(p, seg);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int rg = warp % kRowGroups, cg = warp / kRowGroups;
        const int ra = row0 + rg * 16 + g, rb = ra + 8;
        const bool la = ra < end, lb = rb < end;
        const float s = w >= 0 ? __ldg(p.scales + w) : 0.0f;
        // h as the sum of two bf16: fragments hi, lo of 2 products a slab
        uint32_t hi[NS][2][4], lo[NS][2][4];
#pragma unroll
        for (int sl = 0; sl < NS; ++sl) {
            const int r = sl * 32 + t * 8;
            float v[2][8];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
            if (w >= 0 && r < p.R) {
                for (int sp = 0; sp < p.splits; ++sp) {
                    const float* h = p.h + static_cast<size_t>(sp) * p.M * p.R + r;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (q == 0 ? la : lb) {
                            const float4* h4 = reinterpret_cast<const float4*>(h + static_cast<size_t>(q == 0 ? ra : rb) * p.R);
                            const float4 f0 = h4[0], f1 = h4[1];
                            v[q][0] += f0.x; v[q][1] += f0.y; v[q][2] += f0.z; v[q][3] += f0.w;
                            v[q][4] += f1.x; v[q][5] += f1.y; v[q][6] += f1.z; v[q][7] += f1.w;
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float v0 = s * v[q][2 * i], v1 = s * v[q][2 * i + 1];
                    const uint32_t h2 = pack_bf16x2(v0, v1);
                    // product i / 2; registers: row g then row g + 8, first pair then second.
                    // An infinite sum has no rest (inf - inf would make it NaN)
                    const float e0 = v0 - bf16_lo(h2), e1 = v1 - bf16_hi(h2);
                    hi[sl][i >> 1][(i & 1) * 2 + q] = h2;
                    lo[sl][i >> 1][(i & 1) * 2 + q] = pack_bf16x2(e0 == e0 ? e0 : 0.0f, e1 == e1 ? e1 : 0.0f);
                }
        }
        const uint16_t* B = p.b + (w >= 0 ? static_cast<size_t>(w) * p.N * p.R : 0);
        const int c_end = min(p.N, (static_cast<int>(blockIdx.y) + 1) * cols_per_cta);
        for (int c0 = blockIdx.y * cols_per_cta + cg * 32; c0 < c_end; c0 += kColGroups * 32) {
            float acc[4][4];
            // column c0 + 8 t + 2 i + e belongs to tile i, so a lane's columns are 8 neighbours
            uint4 b[4][NS];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
                const int n = min(c0 + 8 * (g >> 1) + 2 * i + (g & 1), p.N - 1);
#pragma unroll
                for (int sl = 0; sl < NS; ++sl) {
                    const int r = sl * 32 + t * 8;
                    b[i][sl] = make_uint4(0u, 0u, 0u, 0u);
                    if (w >= 0 && r < p.R)
                        b[i][sl] = __ldg(reinterpret_cast<const uint4*>(B + static_cast<size_t>(n) * p.R + r));
                }
            }
            const int col = c0 + 8 * t;
            uint4 ya = make_uint4(0u, 0u, 0u, 0u), yb = ya;
            const size_t ia = static_cast<size_t>(ra) * p.N + col, ib = static_cast<size_t>(rb) * p.N + col;
            if (kVec) {
                if (la && col < p.N) ya = *reinterpret_cast<const uint4*>(p.y + ia);
                if (lb && col < p.N) yb = *reinterpret_cast<const uint4*>(p.y + ib);
            }
            if (w >= 0) {
#pragma unroll
                for (int sl = 0; sl < NS; ++sl)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 q = b[i][sl];
                        mma_bf16(acc[i], lo[sl][0][0], lo[sl][0][1], lo[sl][0][2], lo[sl][0][3], q.x, q.y);
                        mma_bf16(acc[i], lo[sl][1][0], lo[sl][1][1], lo[sl][1][2], lo[sl][1][3], q.z, q.w);
                        mma_bf16(acc[i], hi[sl][0][0], hi[sl][0][1], hi[sl][0][2], hi[sl][0][3], q.x, q.y);
                        mma_bf16(acc[i], hi[sl][1][0], hi[sl][1][1], hi[sl][1][2], hi[sl][1][3], q.z, q.w);
                    }
            }
            if (kVec) {
                const uint32_t y0[4] = {ya.x, ya.y, ya.z, ya.w}, y1[4] = {yb.x, yb.y, yb.z, yb.w};
                uint32_t o0[4], o1[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // without an adapter y passes as it is, whatever its bits
                    o0[i] = w < 0 ? y0[i] : pack_bf16x2(bf16_lo(y0[i]) + acc[i][0], bf16_hi(y0[i]) + acc[i][1]);
                    o1[i] = w < 0 ? y1[i] : pack_bf16x2(bf16_lo(y1[i]) + acc[i][2], bf16_hi(y1[i]) + acc[i][3]);
                }
                if (la && col < p.N) *reinterpret_cast<uint4*>(p.out + ia) = make_uint4(o0[0], o0[1], o0[2], o0[3]);
                if (lb && col < p.N) *reinterpret_cast<uint4*>(p.out + ib) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = col + 2 * i + e;
                        if (c >= p.N) continue;
                        if (la) {
                            const size_t at = static_cast<size_t>(ra) * p.N + c;
                            const uint16_t v = p.y[at];
                            p.out[at] = w < 0 ? v : bf16_bits_rn(bf16_bits_to_f32(v) + acc[i][e]);
                        }
                        if (lb) {
                            const size_t at = static_cast<size_t>(rb) * p.N + c;
                            const uint16_t v = p.y[at];
                            p.out[at] = w < 0 ? v : bf16_bits_rn(bf16_bits_to_f32(v) + acc[i][2 + e]);
                        }
                    }
            }
        }
    }
    griddep_launch_dependents();
}

struct LoraShape {
    bool wide;          // 64-row tiles
    int tiles;          // upper bound: the segments' lengths are on the device
    int splits;
    int cols;           // columns of a CTA of the second kernel
};

LoraShape lora_shape(int M, int K, int N, int segments, const DeviceInfo& dev) {
    LoraShape s;
    // a tile of 64 rows reads its adapter once for four row groups (through L1); with
    // fewer than 64 rows a segment on average it would mostly hold padding
    s.wide = M / segments >= 64;
    const int rows = s.wide ? 64 : 16;
    // at most one partial tile a segment, and no tile without a row
    const long long bound = static_cast<long long>(M) / rows + segments;
    s.tiles = static_cast<int>(bound < M ? bound : M);
    const int slabs = (K + 31) / 32;
    const int groups = kLoraWarps / (rows / 16);
    int splits = (2 * dev.num_sms + s.tiles - 1) / s.tiles;
    const int most = slabs / (2 * groups) > 0 ? slabs / (2 * groups) : 1;
    splits = splits < most ? splits : most;
    s.splits = splits > 32 ? 32 : splits;
    const int unit = 32 * groups;
    int parts = (4 * dev.num_sms + s.tiles - 1) / s.tiles;
    const int col_units = (N + unit - 1) / unit;
    parts = parts < col_units ? parts : col_units;
    s.cols = (col_units + parts - 1) / parts * unit;
    return s;
}

template <int NT>
cudaError_t launch_down(const LoraArgs& p, const LoraShape& s, cudaStream_t stream) {
    const dim3 grid(s.tiles, s.splits);
    const size_t smem = static_cast<size_t>(kLoraWarps) * 16 * p.R * 4;
    if (s.wide) {
        static std::atomic<unsigned long long> opted{0};
        if (!smem_opt_in(lora_down_kernel<NT, 4>, kLoraWarps * 16 * 8 * NT * 4, opted)) return cudaErrorInvalidValue;
        return launch_programmatic_grid(lora_down_kernel<NT, 4>, grid, kLoraThreads, smem, stream, p);
    }
    static std::atomic<unsigned long long> opted{0};
    if (!smem_opt_in(lora_down_kernel<NT, 1>, kLoraWarps * 16 * 8 * NT * 4, opted)) return cudaErrorInvalidValue;
    return launch_programmatic_grid(lora_down_kernel<NT, 1>, grid, kLoraThreads, smem, stream, p);
}

template <int NS>
cudaError_t launch_up(const LoraArgs& p, const LoraShape& s, bool vec, cudaStream_t stream) {
    const dim3 grid(s.tiles, (p.N + s.cols - 1) / s.cols);
    if (s.wide)
        return vec ? launch_programmatic_grid(lora_up_kernel<NS, 4, true>, grid, kLoraThreads, 0, stream, p, s.cols)
                   : launch_programmatic_grid(lora_up_kernel<NS, 4, false>, grid, kLoraThreads, 0, stream, p, s.cols);
    return vec ? launch_programmatic_grid(lora_up_kernel<NS, 1, true>, grid, kLoraThreads, 0, stream, p, s.cols)
               : launch_programmatic_grid(lora_up_kernel<NS, 1, false>, grid, kLoraThreads, 0, stream, p, s.cols);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_lora_sizes(int M, int K, int N, int R, int adapters, int segments) {
    if (M < 0 || K < 1 || N < 1 || R < 1 || adapters < 1 || segments < 1 || K % 8 != 0 || R % 8 != 0)
        return TRELLIS_ERR_SHAPE;
    if (R > 128 || M > 65536 || segments > 65536) return TRELLIS_ERR_UNSUPPORTED;
    return TRELLIS_OK;
}

}  // namespace

}  // namespace trellis

extern "C" {

int trellis_lora_add_workspace_size(int M, int K, int N, int R, int adapters, int segments, size_t* bytes) {
    using namespace trellis;
    if (bytes == nullptr) return TRELLIS_ERR_NULL;
    int rc = check_lora_sizes(M, K, N, R, adapters, segments);
    if (rc != TRELLIS_OK) return rc;
    DeviceInfo dev;
    rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    const LoraShape s = lora_shape(M > 0 ? M : 1, K, N, segments, dev);
    // the products' counter region stays free (and zero) in front
    *bytes = (size_t(1) << 20) + static_cast<size_t>(s.splits) * M * R * 4;
    return TRELLIS_OK;
}

int trellis_lora_add(const uint16_t* y, const uint16_t* x, const uint16_t* a, const uint16_t* b, const float* scales,
                     const int* starts, const int* which, int M, int K, int N, int R, int adapters, int segments,
                     uint16_t* out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace trellis;
    if (y == nullptr || x == nullptr || a == nullptr || b == nullptr || scales == nullptr || starts == nullptr ||
        which == nullptr || out == nullptr)
        return TRELLIS_ERR_NULL;
    int rc = check_lora_sizes(M, K, N, R, adapters, segments);
    if (rc != TRELLIS_OK) return rc;
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(y, 2) || !aligned(out, 2) ||
        !aligned(scales, 4) || !aligned(starts, 4) || !aligned(which, 4))
        return TRELLIS_ERR_ALIGN;
    size_t need = 0;
    rc = trellis_lora_add_workspace_size(M, K, N, R, adapters, segments, &need);
    if (rc != TRELLIS_OK) return rc;
    if (workspace == nullptr || workspace_bytes < need) return TRELLIS_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return TRELLIS_ERR_ALIGN;
    if (M == 0) return TRELLIS_OK;
    DeviceInfo dev;
    rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    const LoraShape s = lora_shape(M, K, N, segments, dev);
    LoraArgs p;
    p.y = y; p.x = x; p.a = a; p.b = b; p.scales = scales; p.starts = starts; p.which = which; p.out = out;
    p.h = reinterpret_cast<float*>(static_cast<char*>(workspace) + (size_t(1) << 20));
    p.M = M; p.K = K; p.N = N; p.R = R; p.adapters = adapters; p.segments = segments; p.splits = s.splits;
    cudaError_t e = R <= 16 ? launch_down<2>(p, s, stream) : R <= 32 ? launch_down<4>(p, s, stream)
                    : R <= 64 ? launch_down<8>(p, s, stream) : launch_down<16>(p, s, stream);
    if (e != cudaSuccess) return TRELLIS_ERR_CUDA;
    // 16-byte accesses of y and out
    const bool vec = N % 8 == 0 && aligned(y, 16) && aligned(out, 16);
    e = R <= 32 ? launch_up<1>(p, s, vec, stream) : R <= 64 ? launch_up<2>(p, s, vec, stream)
                                                            : launch_up<4>(p, s, vec, stream);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

}  // extern "C"
