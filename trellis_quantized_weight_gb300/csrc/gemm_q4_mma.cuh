// Products with 4-bit weights for few activation rows: a warp's tile is 16 weight rows, its
// operands go from global memory to registers.
//
// mma.m16n8k16 takes 16 weight rows times 8 activation rows.  The sum over k does not depend on
// which k stands where, so a lane's word of eight codes is its part of two products: the pairs that
// a mask and a shift leave, codes (0, 4), (1, 5) and (2, 6), (3, 7).  The activations are brought
// into that order once, on their way to shared memory.  The four lanes of a row hold a whole group
// of it at a time, so each group's sum is complete in the accumulators and is scaled there.
//
// A CTA has kRows x 16 weight rows and 8 / kRows warps a row tile, which take steps of 128 k in
// turn; where there are few row tiles, a cluster of CTAs shares them further.  Parts are added in
// their order, so equal calls give equal bits.
#pragma once

#include <cooperative_groups.h>

#include "gemm_q4.cuh"

namespace trellis {

namespace {

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kQ4Warps = 8, kQ4Threads = 32 * kQ4Warps;
constexpr int kQ4Step = 128;                    // k of a warp's step
constexpr int kQ4Depth = 4;                     // steps whose codes are on their way, and the one at work

template <int G, int MT, int kTiles>
struct Q4Shape {
    static constexpr int kRows = 8 * MT;                            // activation rows of a CTA
    static constexpr int kSplit = kQ4Warps / kTiles;                // warps that share a row tile
    static constexpr int kChunk = MT == 1 ? 32 : MT == 2 ? 16 : MT == 4 ? 8 : 4;    // steps whose activations are staged at once
    static constexpr int kRowBytes = kChunk * kQ4Step * 2 + 64;     // 64 modulo 128: two rows' lanes hit different banks
    static constexpr int kSumBytes = kChunk * (kQ4Step / G) * kRows * 4;
    static constexpr int kRedBytes = kQ4Warps * 16 * kRows * 4, kTotalBytes = kTiles * 16 * kRows * 4;
    static_assert(kChunk % (kSplit * kQ4Depth) == 0, "a chunk's steps go round the warps and the ring evenly");
    static int smem(int rows) {
        const int staged = rows * kRowBytes + kSumBytes, ends = kRedBytes + kTotalBytes;
        return staged > ends ? staged : ends;
    }
};

template <int G>
struct Q4Step {
    uint32_t w[2][4];                           // rows gid and gid + 8: the words of this lane
    uint32_t s[2][kQ4Step / G];                 // scale of each group, its bias above
};

template <int G, int MT, int kTiles, bool kBias>
__global__ void __launch_bounds__(kQ4Threads, MT <= 2 ? 3 : 2)
q4_mma_kernel(const __grid_constant__ Q4Args a) {
    using S = Q4Shape<G, MT, kTiles>;
    constexpr int kSplit = S::kSplit, kPer = kQ4Step / G, kWords = G / 32;    // groups of a step, words a lane and group
    extern __shared__ __align__(16) unsigned char smem[];
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int part = blockIdx.y, parts = gridDim.y;       // the cluster lies along y
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = warp / kSplit, turn = warp % kSplit;
    const int gid = lane >> 2, tig = lane & 3;
    const int n0 = blockIdx.x * (16 * kTiles);
    const int m0 = blockIdx.z * S::kRows, rows = min(a.M - m0, S::kRows);
    float* const sums = reinterpret_cast<float*>(smem + rows * S::kRowBytes);     // [group of the chunk][activation row]
    const int steps = (a.K + kQ4Step - 1) / kQ4Step;
    const int begin = static_cast<int>(static_cast<long long>(steps) * part / parts);
    const int end = static_cast<int>(static_cast<long long>(steps) * (part + 1) / parts);
    // rows past the last read it again; their results are not stored
    const int row[2] = {min(n0 + 16 * tile + gid, a.N - 1), min(n0 + 16 * tile + gid + 8, a.N - 1)};
    const uint32_t* codes[2];
    const uint16_t *scales[2], *biases[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        codes[h] = a.codes + static_cast<size_t>(row[h]) * (a.K / 8) + tig * kWords;
        scales[h] = a.scales + static_cast<size_t>(row[h]) * a.groups;
        biases[h] = kBias ? a.biases + static_cast<size_t>(row[h]) * a.groups : nullptr;
    }
    auto load = [&](int step, Q4Step<G>& r) {
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const int g = step * kPer + q;
            const bool has = step < end && g < a.groups;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t* src = codes[h] + static_cast<size_t>(g) * (G / 8);
                uint32_t* dst = r.w[h] + q * kWords;
                if constexpr (kWords == 4) {
                    const uint4 v = has ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0u, 0u, 0u, 0u);
                    dst[0] = v.x; dst[1] = v.y; dst[2] = v.z; dst[3] = v.w;
                } else if constexpr (kWords == 2) {
                    const uint2 v = has ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0u, 0u);
                    dst[0] = v.x; dst[1] = v.y;
                } else {
                    dst[0] = has ? __ldg(src) : 0u;
                }
                r.s[h][q] = has ? __ldg(scales[h] + g) : 0u;
                if constexpr (kBias) r.s[h][q] |= has ? static_cast<uint32_t>(__ldg(biases[h] + g)) << 16 : 0u;
            }
        }
    };

    float o[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][j] = 0.0f;

    griddep_wait();
    Q4Step<G> ring[kQ4Depth];
#pragma unroll
    for (int d = 0; d < kQ4Depth - 1; ++d) load(begin + turn + d * kSplit, ring[d]);

    // activation row of a lane's operand in each row tile of 8: rows past the last repeat it
    uint32_t x_at[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) x_at[t] = static_cast<uint32_t>(min(8 * t + gid, rows - 1) * S::kRowBytes + tig * 16);

    for (int chunk = begin; chunk < end; chunk += S::kChunk) {
        if (chunk != begin) __syncthreads();
        // the chunk's activations, eight at a time
        for (int e = threadIdx.x; e < rows * (S::kChunk * 16); e += kQ4Threads) {
            const int m = e / (S::kChunk * 16), b = e % (S::kChunk * 16);        // block of eight
            const long long k = (static_cast<long long>(chunk) * 16 + b) * 8;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (k < a.K) v = q4_load_x(a.x, a.x_scales != nullptr, static_cast<size_t>(m0 + m) * a.K + k);
            // the block of lane tig and word j of a group stands at 4 j + tig
            const int in = b % (G / 8), slot = b - in + (in % kWords) * 4 + in / kWords;
            *reinterpret_cast<uint4*>(smem + m * S::kRowBytes + slot * 16) =
                make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                           __byte_perm(v.y, v.w, 0x7632));
            if constexpr (kBias) {
                float s = ((bf16_lo(v.x) + bf16_hi(v.x)) + (bf16_lo(v.y) + bf16_hi(v.y))) +
                          ((bf16_lo(v.z) + bf16_hi(v.z)) + (bf16_lo(v.w) + bf16_hi(v.w)));
#pragma unroll
                for (int d = G / 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                if (in == 0) sums[(b / (G / 8)) * S::kRows + m] = s;
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int i = turn; i < S::kChunk; i += kSplit * kQ4Depth) {
#pragma unroll
            for (int d = 0; d < kQ4Depth; ++d) {
                const int step = chunk + i + d * kSplit;
                load(step + (kQ4Depth - 1) * kSplit, ring[(d + kQ4Depth - 1) % kQ4Depth]);
                if (step >= end) continue;
                const Q4Step<G>& r = ring[d];
                const unsigned char* x = smem + (i + d * kSplit) * (kQ4Step * 2);
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    float acc[MT][4];
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[t][j] = 0.0f;
#pragma unroll
                    for (int j = 0; j < kWords; ++j) {
                        uint32_t lo[4], hi[4];
                        q4_pairs(r.w[0][q * kWords + j], lo);
                        q4_pairs(r.w[1][q * kWords + j], hi);
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const uint4 v = *reinterpret_cast<const uint4*>(x + x_at[t] + (q * (G / 8) + 4 * j) * 16);
                            mma_bf16(acc[t], lo[0], hi[0], lo[1], hi[1], v.x, v.y);
                            mma_bf16(acc[t], lo[2], hi[2], lo[3], hi[3], v.z, v.w);
                        }
                    }
                    const float s0 = __uint_as_float(r.s[0][q] << 16), s1 = __uint_as_float(r.s[1][q] << 16);
                    float b0 = 0.0f, b1 = 0.0f;
                    if constexpr (kBias) {
                        b0 = fmaf(8.0f, s0, __uint_as_float(r.s[0][q] & 0xffff0000u));
                        b1 = fmaf(8.0f, s1, __uint_as_float(r.s[1][q] & 0xffff0000u));
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        o[t][0] = fmaf(s0, acc[t][0], o[t][0]);
                        o[t][1] = fmaf(s0, acc[t][1], o[t][1]);
                        o[t][2] = fmaf(s1, acc[t][2], o[t][2]);
                        o[t][3] = fmaf(s1, acc[t][3], o[t][3]);
                        if constexpr (kBias) {
                            const float2 u = *reinterpret_cast<const float2*>(sums + ((i + d * kSplit) * kPer + q) * S::kRows + 8 * t + 2 * tig);
                            o[t][0] = fmaf(b0, u.x, o[t][0]);
                            o[t][1] = fmaf(b0, u.y, o[t][1]);
                            o[t][2] = fmaf(b1, u.x, o[t][2]);
                            o[t][3] = fmaf(b1, u.y, o[t][3]);
                        }
                    }
                }
            }
        }
    }

    // the warps' parts of a tile, then the cluster's, each in order
    __syncthreads();
    float* const red = reinterpret_cast<float*>(smem);                      // [warp][16 rows][kRows]
    float* const total = reinterpret_cast<float*>(smem + S::kRedBytes);     // [kRows][16 kTiles]
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(red + (warp * 16 + gid + 8 * h) * S::kRows + 8 * t + 2 * tig) = make_float2(o[t][2 * h], o[t][2 * h + 1]);
    __syncthreads();
    auto finish = [&](int m, int n, float y) {
        if (n0 + n < a.N) {
            if (a.x_scales != nullptr) y *= __ldg(a.x_scales + m0 + m);
            a.out[static_cast<size_t>(m0 + m) * a.N + n0 + n] = bf16_bits_rn(y);
        }
    };
    for (int e = threadIdx.x; e < rows * 16 * kTiles; e += kQ4Threads) {
        const int n = e % (16 * kTiles), m = e / (16 * kTiles);
        const float* from = red + ((n / 16) * kSplit * 16 + n % 16) * S::kRows + m;
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < kSplit; ++w) y += from[w * 16 * S::kRows];
        if (parts == 1) finish(m, n, y);
        else total[e] = y;
    }
    if (parts > 1) {
        cluster.sync();
        for (int e = part * kQ4Threads + threadIdx.x; e < rows * 16 * kTiles; e += parts * kQ4Threads) {
            float y = 0.0f;
            for (int r = 0; r < parts; ++r) y += cluster.map_shared_rank(total, r)[e];
            finish(e / (16 * kTiles), e % (16 * kTiles), y);
        }
        cluster.sync();                 // the others may still be reading this CTA's part
    }
    griddep_launch_dependents();
}

template <int G, int MT, int kTiles, bool kBias>
cudaError_t launch_as(const Q4Args& a, int parts, cudaStream_t stream) {
    using S = Q4Shape<G, MT, kTiles>;
    static std::atomic<unsigned long long> done{0};
    const int smem = S::smem(a.M < S::kRows ? a.M : S::kRows);
    if (!smem_opt_in(q4_mma_kernel<G, MT, kTiles, kBias>, S::smem(S::kRows), done)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.N + 16 * kTiles - 1) / (16 * kTiles), parts, (a.M + S::kRows - 1) / S::kRows);
    cfg.blockDim = dim3(kQ4Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1; attr[1].val.clusterDim.y = parts; attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q4_mma_kernel<G, MT, kTiles, kBias>, a);
}

template <int G, int MT, int kTiles>
cudaError_t launch_tiles(const Q4Args& a, const DeviceInfo& dev, cudaStream_t stream) {
    // CTAs of a cluster: enough for two an SM, as long as each has a step for every warp
    const long long tiles = (static_cast<long long>(a.N) + 16 * kTiles - 1) / (16 * kTiles) * ((a.M + 8 * MT - 1) / (8 * MT));
    const int steps = (a.K + kQ4Step - 1) / kQ4Step;
    int parts = 1;
    while (parts < 8 && tiles * parts < 2 * dev.num_sms && steps >= 2 * parts * Q4Shape<G, MT, kTiles>::kSplit) parts *= 2;
    return a.biases != nullptr ? launch_as<G, MT, kTiles, true>(a, parts, stream) : launch_as<G, MT, kTiles, false>(a, parts, stream);
}

}  // namespace

template <int G>
cudaError_t launch_q4_mma(const Q4Args& a, const DeviceInfo& dev, cudaStream_t stream) {
    if (a.M <= 8) return launch_tiles<G, 1, 1>(a, dev, stream);
    if (a.M <= 16) return launch_tiles<G, 2, 2>(a, dev, stream);
    if (a.M <= 32) return launch_tiles<G, 4, 8>(a, dev, stream);
    return launch_tiles<G, 8, 8>(a, dev, stream);
}

}  // namespace trellis
