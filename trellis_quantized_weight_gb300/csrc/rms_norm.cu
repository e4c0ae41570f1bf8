// trellis_rms_norm: the residual's addition, the root-mean-square norm and the
// rounding to bf16, or to e4m3 with a scale a row, in one pass.
//
//   h = x + residual                     fp32, exact to one rounding; residual_out = bf16(h)
//   y = h * rsqrt(mean(h^2) + eps) * w   from the unrounded h, sums in fp32
//   out = bf16(y), or codes = e4m3(y / s) with s = max(max|y| / 448, 2^-100)
//
// A row stays in registers between its two reductions (sum of squares and, for the
// 8-bit form, max|h w|, which are taken together: y's maximum is the product's times
// rsqrt) and its stores, so each value is read and written once.
#include "kernels.h"
#include "kv_cache.cuh"
#include "trellis.h"
#include "trellis_device.cuh"

namespace trellis {

namespace {

struct NormArgs {
    const uint16_t *x, *residual, *weight;
    long long x_stride;                 // elements between tokens
    long long rows;                     // tokens * heads
    int heads, width;
    float eps;
    uint16_t *out, *residual_out;
    uint8_t* codes;
    float* scales;
};

constexpr float kLeastScale = 7.888609052210118e-31f;    // 2^-100

__device__ __forceinline__ void bf16x8_to_f32(uint4 v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Magnitudes compare as their bits do, and NaN above all of them.
__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// The scale of a row whose largest |y| has these bits; NaN where it is not finite.
__device__ __forceinline__ float row_scale(uint32_t bits) {
    return bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : fmaxf(__fdiv_rn(__uint_as_float(bits), 448.0f), kLeastScale);
}

// Sum and maximum over the `threads` threads of a row (a warp, or the whole CTA).  part: two buffers, taken in
// turn from one row to the next, so that one barrier a row is enough.
template <bool kWarpRow>
__device__ __forceinline__ void reduce(float& sum, uint32_t& most, float2* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = __reduce_max_sync(0xffffffffu, most);
    if constexpr (!kWarpRow) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) part[warp] = make_float2(sum, __uint_as_float(most));
        __syncthreads();
        const float2 p = lane < warps ? part[lane] : make_float2(0.0f, 0.0f);
        sum = p.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        most = __reduce_max_sync(0xffffffffu, __float_as_uint(p.y));
    }
}

// kVec: 8 values by one 16-byte access; otherwise single values, a thread apart.
// kPer: units of 8 values that a thread holds.
template <int kPer, bool kVec, bool kWarpRow, bool kEight, int kThreads>
__global__ void __launch_bounds__(kThreads) rms_norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float2 part[2][32];
    const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x, threads = kWarpRow ? 32 : blockDim.x;
    const long long step = static_cast<long long>(gridDim.x) * (kWarpRow ? 8 : 1);
    long long row = static_cast<long long>(blockIdx.x) * (kWarpRow ? 8 : 1) + (kWarpRow ? threadIdx.x >> 5 : 0);
    // position of value j of unit i, and whether the row has it
    auto at = [&](int i, int j) { return kVec ? 8 * (t + i * threads) + j : t + (8 * i + j) * threads; };
    griddep_wait();
    griddep_launch_dependents();        // the next grid's start beside this one; it waits for the end before it reads
    uint4 w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (kVec) {
            if (at(i, 0) < a.width) w[i] = __ldg(reinterpret_cast<const uint4*>(a.weight + at(i, 0)));
        } else {
            uint32_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = at(i, j) < a.width ? __ldg(a.weight + at(i, j)) : 0u;
            w[i] = make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16));
        }
    }
    auto load = [&](const uint16_t* src, uint4 (&v)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (kVec) {
                if (at(i, 0) < a.width) v[i] = *reinterpret_cast<const uint4*>(src + at(i, 0));
            } else {
                uint32_t u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = at(i, j) < a.width ? src[at(i, j)] : 0u;
                v[i] = make_uint4(u[0] | (u[1] << 16), u[2] | (u[3] << 16), u[4] | (u[5] << 16), u[6] | (u[7] << 16));
            }
        }
    };
    auto store = [&](uint16_t* dst, int i, const float (&f)[8]) {
        if constexpr (kVec) {
            if (at(i, 0) < a.width) *reinterpret_cast<uint4*>(dst + at(i, 0)) = f32_to_bf16x8(f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at(i, j) < a.width) dst[at(i, j)] = bf16_bits_rn(f[j]);
        }
    };
    auto source = [&](long long r) {
        const long long token = a.heads == 1 ? r : r / a.heads;
        return a.x + token * a.x_stride + (r - token * a.heads) * a.width;
    };
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        uint4 x[kPer], r[kPer];
        load(source(row), x);
        const long long base = row * a.width;
        if (a.residual != nullptr) load(a.residual + base, r);
        float h[kPer][8];
        float sum = 0.0f;
        uint32_t most = 0u;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            bf16x8_to_f32(x[i], h[i]);
            if (a.residual != nullptr) {
                float f[8];
                bf16x8_to_f32(r[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] += f[j];
                store(a.residual_out + base, i, h[i]);
            }
            float g[8];
            bf16x8_to_f32(w[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum = fmaf(h[i][j], h[i][j], sum);
                if constexpr (kEight) {
                    h[i][j] *= g[j];
                    most = max(most, magnitude(h[i][j]));
                }
            }
        }
        reduce<kWarpRow>(sum, most, part[turn]);
        const float factor = rsqrtf(sum / static_cast<float>(a.width) + a.eps);
        if constexpr (kEight) {
            const float s = row_scale(magnitude(__uint_as_float(most) * factor));
            const float inv = factor / s;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                uint32_t c[2];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    c[q] = static_cast<uint32_t>(f32_to_e4m3x2(h[i][4 * q] * inv, h[i][4 * q + 1] * inv)) |
                           (static_cast<uint32_t>(f32_to_e4m3x2(h[i][4 * q + 2] * inv, h[i][4 * q + 3] * inv)) << 16);
                if constexpr (kVec) {
                    if (at(i, 0) < a.width) *reinterpret_cast<uint2*>(a.codes + base + at(i, 0)) = make_uint2(c[0], c[1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (at(i, j) < a.width) a.codes[base + at(i, j)] = static_cast<uint8_t>(c[j >> 2] >> (8 * (j & 3)));
                }
            }
            if (t == 0) a.scales[row] = s;
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                float g[8];
                bf16x8_to_f32(w[i], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = h[i][j] * factor * g[j];
                store(a.out + base, i, g);
            }
        }
    }
}

// Rows that do not fit a CTA's registers: read twice, the second time from L2.
template <bool kEight>
__global__ void __launch_bounds__(1024) rms_norm_wide_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float2 part[2][32];
    griddep_wait();
    griddep_launch_dependents();        // the next grid's start beside this one; it waits for the end before it reads
    int turn = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const long long token = row / a.heads, base = row * a.width;
        const uint16_t* x = a.x + token * a.x_stride + (row - token * a.heads) * a.width;
        auto value = [&](int c) {
            const float f = bf16_bits_to_f32(x[c]);
            return a.residual != nullptr ? f + bf16_bits_to_f32(a.residual[base + c]) : f;
        };
        float sum = 0.0f;
        uint32_t most = 0u;
        for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
            const float h = value(c);
            sum = fmaf(h, h, sum);
            if constexpr (kEight) most = max(most, magnitude(h * bf16_bits_to_f32(__ldg(a.weight + c))));
        }
        reduce<false>(sum, most, part[turn]);
        const float factor = rsqrtf(sum / static_cast<float>(a.width) + a.eps);
        const float s = kEight ? row_scale(magnitude(__uint_as_float(most) * factor)) : 1.0f;
        const float inv = kEight ? factor / s : factor;
        for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
            const float h = value(c), y = h * bf16_bits_to_f32(__ldg(a.weight + c));
            if (a.residual != nullptr) a.residual_out[base + c] = bf16_bits_rn(h);
            if constexpr (kEight)
                a.codes[base + c] = static_cast<uint8_t>(f32_to_e4m3x2(y * inv, 0.0f));
            else
                a.out[base + c] = bf16_bits_rn(y * inv);
        }
        if (kEight && threadIdx.x == 0) a.scales[row] = s;
    }
}

constexpr int kMostThreads = 1024, kMostPer = 4;

template <int kPer, bool kVec, bool kEight, bool kWarpRow, int kThreads>
cudaError_t launch(const NormArgs& a, int threads, const DeviceInfo& dev, cudaStream_t stream) {
    // as many CTAs as run at once, each with its weights in registers: the next row's CTA would load them again
    auto* kernel = rms_norm_kernel<kPer, kVec, kWarpRow, kEight, kThreads>;
    const int per_sm = 2048 / threads;
    const long long ctas = kWarpRow ? (a.rows + 7) / 8 : a.rows, most = static_cast<long long>(per_sm) * dev.num_sms;
    return launch_programmatic(kernel, static_cast<unsigned>(ctas < most ? ctas : most), static_cast<unsigned>(threads), 0, stream, a);
}

template <bool kVec, bool kEight>
cudaError_t launch_rows(const NormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
    const int units = (a.width + 7) / 8;
    auto threads = [&](int per) { return ((units + per - 1) / per + 31) / 32 * 32; };
    if (units > kMostThreads * kMostPer) {
        const long long most = 2ll * dev.num_sms;
        return launch_programmatic(rms_norm_wide_kernel<kEight>, static_cast<unsigned>(a.rows < most ? a.rows : most), 1024u, 0, stream, a);
    }
    if (units <= 32) return launch<1, kVec, kEight, true, 256>(a, 256, dev, stream);
    if (units <= 64) return launch<2, kVec, kEight, true, 256>(a, 256, dev, stream);
    // few rows: one unit a thread where that fits, for the shortest chain
    if (a.rows < dev.num_sms && units <= kMostThreads) return launch<1, kVec, kEight, false, 1024>(a, threads(1), dev, stream);
    // two units a thread: 8165 rows of 5120 with residual to 8 bits take 50 us, with one 64 to 68, four 59, five 54
    if (units <= 1024) return launch<2, kVec, kEight, false, 512>(a, threads(2), dev, stream);
    if (units <= 2048) return launch<2, kVec, kEight, false, 1024>(a, threads(2), dev, stream);
    return launch<4, kVec, kEight, false, 1024>(a, threads(4), dev, stream);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

}  // namespace trellis

extern "C" int trellis_rms_norm(const uint16_t* x, long long x_stride, const uint16_t* residual, const uint16_t* weight, int rows,
                                int heads, int width, float eps, uint16_t* out, uint8_t* codes, float* scales,
                                uint16_t* residual_out, cudaStream_t stream) {
    using namespace trellis;
    if (x == nullptr || weight == nullptr || (out == nullptr) == (codes == nullptr) || (codes == nullptr) != (scales == nullptr) ||
        (residual == nullptr) != (residual_out == nullptr))
        return TRELLIS_ERR_NULL;
    if (rows < 0 || heads < 1 || width < 1 || !(eps >= 0.0f) || eps > 3.0e38f ||
        x_stride < static_cast<long long>(heads) * width || (out != nullptr && out == residual_out))
        return TRELLIS_ERR_SHAPE;
    if (width > kNormMaxWidth || static_cast<long long>(rows) * heads > (1ll << 31) - 1) return TRELLIS_ERR_UNSUPPORTED;
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(weight, 2) || !aligned(out, 2) || !aligned(residual_out, 2) ||
        !aligned(scales, 4))
        return TRELLIS_ERR_ALIGN;
    if (rows == 0) return TRELLIS_OK;
    DeviceInfo dev;
    const int rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    NormArgs a;
    a.x = x; a.residual = residual; a.weight = weight; a.x_stride = x_stride;
    a.rows = static_cast<long long>(rows) * heads; a.heads = heads; a.width = width; a.eps = eps;
    a.out = out; a.residual_out = residual_out; a.codes = codes; a.scales = scales;
    // 16-byte accesses (8 of codes) everywhere
    const bool vec = width % 8 == 0 && x_stride % 8 == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) &&
                     aligned(out, 16) && aligned(residual_out, 16) && aligned(codes, 8);
    const cudaError_t e = codes != nullptr ? (vec ? launch_rows<true, true>(a, dev, stream) : launch_rows<false, true>(a, dev, stream))
                                           : (vec ? launch_rows<true, false>(a, dev, stream) : launch_rows<false, false>(a, dev, stream));
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}
