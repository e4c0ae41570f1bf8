// trellis_rms_norm: the residual's addition, the root-mean-square norm and the
// rounding to bf16, or to e4m3 with a scale a row, in one pass.
//
//   h = x + residual                     fp32, exact to one rounding; residual_out = bf16(h)
//   y = h * rsqrt(mean(h^2) + eps) * w   from the unrounded h of any size, sums in fp32
//   out = bf16(y), or codes = e4m3(y / s) with s = max(max|y| / 448, 2^-100)
//
// A row stays in registers between its two reductions (sum of squares and, for the
// 8-bit form, max|h w|, which are taken together: y's maximum is the product's times
// rsqrt) and its stores (the 8-bit form takes its products with w a second time there, so that h is at hand where a
// row's squares are past fp32), so each value is read and written once (rows past 32768 values twice, two bytes at a
// time: 2000 of 40000 to bf16 233 us).  Bound by HBM: 8165 rows of 5120 with a residual to 8 bits 46.5 us, 6.3 TB/s of
// the 6.7 that a copy reaches, to bf16 52.4 (6.4); without one 31.0 us (4.0 TB/s) to 8 bits and 32.5 (5.1) to bf16: the
// chain load, sum, store of a row, with as many rows in flight as there is room for.  2000 tokens of 40 heads of 128: 18.4
// us to bf16, 20.8 to 8 bits, by instructions (a warp a row).  One row of 5120: 2.5 us.
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

// Eight values as four pairs: sums, products and multiply-adds take two at a time.
__device__ __forceinline__ void bf16x8_to_f32(uint4 v, float2 (&f)[4]) {
    f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x)); f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z)); f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float2 (&f)[4]) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}
// The largest magnitude of a (already one) and two more values; NaN if one of them is.
__device__ __forceinline__ float most_of(float a, float2 v) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(v.x), "f"(v.y));
    return r;
}

// Magnitudes compare as their bits do, and NaN above all of them.
__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// The scale of a row whose largest |y| has these bits; NaN where it is not finite.
__device__ __forceinline__ float row_scale(uint32_t bits) {
    return bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : fmaxf(__fdiv_rn(__uint_as_float(bits), 448.0f), kLeastScale);
}

// factor / s of rows next to nothing and a small eps: taken in two steps there, since neither of them is.
__device__ __forceinline__ bool too_large(float inv) { return __float_as_uint(inv) == 0x7f800000u; }

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

// Squares of bf16 values reach from 2^-266 to 2^256, fp32 from 2^-149 to 2^128.  Where a row's sum is past that, or eps is next to
// nothing and the sum too (least), the squares are added again of the values times 2^-80 or 2^80, and those are what the factor is for.
constexpr float kDown = 8.271806125530277e-25f, kUp = 1.2089258196146292e24f;              // 2^-80, 2^80
constexpr float kTinyEps = 7.523163845262640e-37f;      // 2^-120: beside a larger one, what a sum of squares drops below 2^-149 is nothing
constexpr float kLeastSum = 7.888609052210118e-31f;     // 2^-100
__device__ __forceinline__ float least_sum(float eps) { return eps < kTinyEps ? kLeastSum : 0.0f; }
__device__ __forceinline__ bool fits(float sum, float least) { return sum >= least && sum <= 3.0e38f; }

// kVec: 8 values by one 16-byte access; otherwise single values, a thread apart.
// kPer: units of 8 values that a thread holds.  kRing: rows under way, the one at work included (0: loaded when their turn comes).
// Rows of a warp: five CTAs an SM (2000 x 40 heads of 128 to 8 bits 20.9 -> 20.6 us).
template <int kPer, bool kVec, bool kWarpRow, bool kEight, int kThreads, int kRing>
__global__ void __launch_bounds__(kThreads, kWarpRow && kPer == 1 ? 5 : 1) rms_norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float2 part[2][32];
    const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x, threads = kWarpRow ? 32 : blockDim.x;
    const long long step = static_cast<long long>(gridDim.x) * (kWarpRow ? 8 : 1);
    long long row = static_cast<long long>(blockIdx.x) * (kWarpRow ? 8 : 1) + (kWarpRow ? threadIdx.x >> 5 : 0);
    // position of value j of unit i, and whether the row has it
    auto at = [&](int i, int j) { return kVec ? 8 * (t + i * threads) + j : t + (8 * i + j) * threads; };
    griddep_wait();
    griddep_launch_dependents();        // the next grid's start beside this one; it waits for the end before it reads
    const float least = least_sum(a.eps);
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
    auto store = [&](uint16_t* dst, int i, const float2 (&f)[4]) {
        if constexpr (kVec) {
            if (at(i, 0) < a.width) *reinterpret_cast<uint4*>(dst + at(i, 0)) = f32_to_bf16x8(f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at(i, j) < a.width) dst[at(i, j)] = bf16_bits_rn(j & 1 ? f[j / 2].y : f[j / 2].x);
        }
    };
    auto source = [&](long long r) {
        const long long token = a.heads == 1 ? r : r / a.heads;
        return a.x + token * a.x_stride + (r - token * a.heads) * a.width;
    };
    // With a ring, a thread's units of the rows to come are on their way to shared memory, where only it reads them: no
    // thread waits for another's copies.
    extern __shared__ __align__(16) unsigned char ring[];
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + 16 * threadIdx.x;
    auto slot = [&](int stage, int which, int i) { return ring_at + ((stage * 2 + which) * kPer + i) * blockDim.x * 16; };
    auto ahead = [&](long long of, int stage) {
        if (of < a.rows) {
            const uint16_t* src = source(of);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (at(i, 0) < a.width) {
                    cp_async16(slot(stage, 0, i), src + at(i, 0));
                    if (a.residual != nullptr) cp_async16(slot(stage, 1, i), a.residual + of * a.width + at(i, 0));
                }
        }
        cp_async_commit();
    };
    if constexpr (kRing > 0) {
#pragma unroll
        for (int p = 0; p < kRing - 1; ++p) ahead(row + p * step, p);
    }
    int stage = 0;
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        uint4 x[kPer], r[kPer];
        const long long base = row * a.width;
        if constexpr (kRing > 0) {
            cp_async_wait<kRing - 2>();
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                x[i] = r[i] = make_uint4(0u, 0u, 0u, 0u);
                if (at(i, 0) < a.width) {
                    x[i] = *reinterpret_cast<const uint4*>(ring + 16 * threadIdx.x + (stage * 2 * kPer + i) * blockDim.x * 16);
                    if (a.residual != nullptr) r[i] = *reinterpret_cast<const uint4*>(ring + 16 * threadIdx.x + ((stage * 2 + 1) * kPer + i) * blockDim.x * 16);
                }
            }
            ahead(row + (kRing - 1) * step, (stage + kRing - 1) % kRing);
            stage = (stage + 1) % kRing;
        } else {
            load(source(row), x);
            if (a.residual != nullptr) load(a.residual + base, r);
        }
        float2 h[kPer][4], sum2 = make_float2(0.0f, 0.0f);
        float largest = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            bf16x8_to_f32(x[i], h[i]);
            if (a.residual != nullptr) {
                float2 f[4];
                bf16x8_to_f32(r[i], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[i][j] = __fadd2_rn(h[i][j], f[j]);
                store(a.residual_out + base, i, h[i]);
            }
            float2 g[4];
            if constexpr (kEight) bf16x8_to_f32(w[i], g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum2 = __ffma2_rn(h[i][j], h[i][j], sum2);
                if constexpr (kEight) largest = most_of(largest, __fmul2_rn(h[i][j], g[j]));
            }
        }
        float sum = sum2.x + sum2.y;
        uint32_t most = magnitude(largest);
        reduce<kWarpRow>(sum, most, part[turn]);
        // all threads of the row have the same sum
        float factor;
        if (__builtin_expect(fits(sum, least), 1)) {
            factor = rsqrtf(sum / static_cast<float>(a.width) + a.eps);
        } else {
            const float times = sum < least ? kUp : kDown;
            float2 again = make_float2(0.0f, 0.0f);
            largest = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                float2 g[4];
                if constexpr (kEight) bf16x8_to_f32(w[i], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[i][j] = __fmul2_rn(h[i][j], make_float2(times, times));
                    again = __ffma2_rn(h[i][j], h[i][j], again);
                    if constexpr (kEight) largest = most_of(largest, __fmul2_rn(h[i][j], g[j]));
                }
            }
            sum = again.x + again.y;
            most = magnitude(largest);
            if constexpr (!kWarpRow) __syncthreads();           // others may still be reading their parts
            reduce<kWarpRow>(sum, most, part[turn]);
            factor = rsqrtf(sum / static_cast<float>(a.width) + a.eps * times * times);
        }
        if constexpr (kEight) {
            const float s = row_scale(magnitude(__uint_as_float(most) * factor));
            float inv = factor / s;
            if (too_large(inv)) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[i][j] = __fmul2_rn(h[i][j], make_float2(factor, factor));
                inv = 1.0f / s;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                uint32_t c[2];
                float2 y[4];
                bf16x8_to_f32(w[i], y);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = __fmul2_rn(__fmul2_rn(h[i][j], y[j]), make_float2(inv, inv));
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    c[q] = static_cast<uint32_t>(f32_to_e4m3x2(y[2 * q].x, y[2 * q].y)) |
                           (static_cast<uint32_t>(f32_to_e4m3x2(y[2 * q + 1].x, y[2 * q + 1].y)) << 16);
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
                float2 g[4];
                bf16x8_to_f32(w[i], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) g[j] = __fmul2_rn(__fmul2_rn(h[i][j], make_float2(factor, factor)), g[j]);
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
    const float least = least_sum(a.eps);
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
        float factor, times = 1.0f;
        if (fits(sum, least)) {
            factor = rsqrtf(sum / static_cast<float>(a.width) + a.eps);
        } else {
            times = sum < least ? kUp : kDown;
            sum = 0.0f;
            most = 0u;
            for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
                const float h = value(c) * times;
                sum = fmaf(h, h, sum);
                if constexpr (kEight) most = max(most, magnitude(h * bf16_bits_to_f32(__ldg(a.weight + c))));
            }
            __syncthreads();                                    // others may still be reading their parts
            reduce<false>(sum, most, part[turn]);
            factor = rsqrtf(sum / static_cast<float>(a.width) + a.eps * times * times);
        }
        const float s = kEight ? row_scale(magnitude(__uint_as_float(most) * factor)) : 1.0f;
        float first = factor, inv = kEight ? factor / s : 1.0f;
        if (kEight) {
            if (too_large(inv))
                inv = 1.0f / s;
            else
                first = 1.0f;
        }
        for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
            const float h = value(c), t = h * times, w = bf16_bits_to_f32(__ldg(a.weight + c)), y = kEight ? t * w * first : t * first * w;
            if (a.residual != nullptr) a.residual_out[base + c] = bf16_bits_rn(h);
            if constexpr (kEight)
                a.codes[base + c] = static_cast<uint8_t>(f32_to_e4m3x2(y * inv, 0.0f));
            else
                a.out[base + c] = bf16_bits_rn(y);
        }
        if (kEight && threadIdx.x == 0) a.scales[row] = s;
    }
}

constexpr int kMostThreads = 1024, kMostPer = 4, kAheadThreads = 1024;

template <int kPer, bool kVec, bool kEight, bool kWarpRow, int kThreads, int kRing = 0>
cudaError_t launch(const NormArgs& a, int threads, const DeviceInfo& dev, cudaStream_t stream) {
    // as many CTAs as run at once (of the ring's, whose registers hold half as many, in two turns: 512 or 2048 threads an SM
    // take the same 45 to 46 us), each with its weights in registers: the next row's CTA would load them again
    auto* kernel = rms_norm_kernel<kPer, kVec, kWarpRow, kEight, kThreads, kRing>;
    const int per_sm = (kRing > 0 ? kAheadThreads : 2048) / threads, smem = kRing * 2 * kPer * 16 * threads;
    static std::atomic<unsigned long long> done{0};
    if (kRing > 0 && !smem_opt_in(kernel, kRing * 2 * kPer * 16 * kThreads, done)) return cudaErrorInvalidValue;
    const long long ctas = kWarpRow ? (a.rows + 7) / 8 : a.rows, most = static_cast<long long>(per_sm) * dev.num_sms;
    return launch_programmatic(kernel, static_cast<unsigned>(ctas < most ? ctas : most), static_cast<unsigned>(threads), smem, stream, a);
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
    // Rows enough for a second one to be on its way while a CTA's first is at work: four units a thread, 1024 threads an SM.
    // 8165 rows of 5120 with residual to 8 bits 46 us (50 without the second row, two units a thread; 59 with four); without
    // a residual 31 against 34; two rows ahead 46 to 53.
    if constexpr (kVec)
        if (units <= 2048 && a.rows >= 2ll * (kAheadThreads / threads(4)) * dev.num_sms)
            return launch<4, kVec, kEight, false, 512, 2>(a, threads(4), dev, stream);
    // fewer rows: two units a thread (8165 rows this way 50 us, with one unit 64 to 68, with five 54)
    if (units <= 1024) return launch<2, kVec, kEight, false, 512>(a, threads(2), dev, stream);
    if (units <= 2048) return launch<2, kVec, kEight, false, 1024>(a, threads(2), dev, stream);
    // a bound of fewer threads where that does: with 64 registers each more of the four units' values spill (2000 rows of 17408
    // to 8 bits 53 us, with 80 44; to bf16 46 and 41)
    if (threads(4) <= 768) return launch<4, kVec, kEight, false, 768>(a, threads(4), dev, stream);
    return launch<4, kVec, kEight, false, 1024>(a, threads(4), dev, stream);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Bytes of an array: `rows` pieces of `n`, `step` apart.
struct Span {
    uintptr_t at;
    unsigned long long n, step, rows;
    Span(const void* p, unsigned long long n_, unsigned long long step_ = 0, unsigned long long rows_ = 1)
        : at(reinterpret_cast<uintptr_t>(p)), n(p == nullptr ? 0 : n_), step(step_), rows(rows_) {}
};
// Whether the piece `one` and a piece of `of` share a byte.
bool overlap(const Span& one, const Span& of) {
    if (one.n == 0 || of.n == 0 || one.at + one.n <= of.at) return false;
    if (one.at < of.at + of.n) return true;
    // the last piece that begins before the end of `one`
    if (of.rows == 1 || of.step == 0) return false;
    const unsigned long long last = (one.at + one.n - 1 - of.at) / of.step, row = last < of.rows ? last : of.rows - 1;
    return one.at < of.at + row * of.step + of.n;
}

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
    // Outputs lie apart from each other and from the inputs; those of h's size may be x or residual, row on row.
    const unsigned long long count = static_cast<unsigned long long>(rows) * heads * width, token = 2ull * heads * width;
    const Span in[] = {{x, token, 2ull * x_stride, static_cast<unsigned long long>(rows)}, {residual, 2 * count}, {weight, 2ull * width}};
    const Span written[] = {{out, 2 * count}, {residual_out, 2 * count}, {codes, count}, {scales, 4ull * rows * heads}};
    const bool whole = rows == 1 || 2ull * x_stride == token;
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (overlap(written[i], written[j])) return TRELLIS_ERR_SHAPE;
        for (int j = 0; j < 3; ++j) {
            const bool in_place = i < 2 && written[i].at == in[j].at && (j == 0 ? whole : j == 1);
            if (!in_place && overlap(written[i], in[j])) return TRELLIS_ERR_SHAPE;
        }
    }
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
