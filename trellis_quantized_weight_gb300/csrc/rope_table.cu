// trellis_rope_table: cosines and sines of the rotary positions, built once by a
// program and read by trellis_kv_append.
//
// Pair i of `rot` / 2 turns by base^(-2i / rot) radians a position.  For contexts
// longer than the model was trained on (stretch > 1) pairs turn slower: all of them by
// 1 / stretch when original == 0; else by parts, after how many turns a pair makes over
// the original context: at `high` turns or more it keeps its speed, at `low` or fewer
// it is slowed fully, and the factor is linear in between.  Angles in fp64: at
// position 2^20 an fp32 angle would be off by 0.06 rad.
#include <cmath>

#include "kernels.h"
#include "trellis.h"
#include "trellis_device.cuh"

namespace trellis {

namespace {

__global__ void __launch_bounds__(256) rope_table_kernel(float* __restrict__ table, int rows, int rot, double base,
                                                         double stretch, double original, double low, double high,
                                                         double gain) {
    griddep_wait();
    const int half = rot / 2;
    const int i = blockIdx.y;
    const double f0 = pow(base, -2.0 * i / rot);
    double slow = 1.0 / stretch;
    if (original > 0.0) {
        const double turns = original * f0 / 6.283185307179586;
        const double w = turns >= high ? 1.0 : turns <= low ? 0.0 : (turns - low) / (high - low);
        slow = w + (1.0 - w) / stretch;
    }
    const double f = f0 * slow;
    for (int p = blockIdx.x * blockDim.x + threadIdx.x; p < rows; p += gridDim.x * blockDim.x) {
        double sn, cs;
        sincos(p * f, &sn, &cs);
        float* row = table + static_cast<size_t>(p) * rot;
        row[i] = static_cast<float>(gain * cs);
        row[half + i] = static_cast<float>(gain * sn);
    }
    griddep_launch_dependents();
}

}  // namespace

}  // namespace trellis

extern "C" int trellis_rope_table(float* table, int rows, int rot, double base, double stretch, double original,
                                  double low, double high, double gain, cudaStream_t stream) {
    using namespace trellis;
    if (table == nullptr) return TRELLIS_ERR_NULL;
    if (rows < 1 || rows > (1 << 30) || !(base > 0.0) || !(stretch >= 1.0) || !(original >= 0.0) ||
        !(gain > 0.0) || !std::isfinite(base * stretch * original * gain) ||
        (original > 0.0 && !(low >= 0.0 && high > low && std::isfinite(high))))
        return TRELLIS_ERR_SHAPE;
    if (rot < 16 || rot > 256 || rot % 16 != 0) return TRELLIS_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(table) & 15u) != 0) return TRELLIS_ERR_ALIGN;
    unsigned blocks = (static_cast<unsigned>(rows) + 255u) / 256u;
    if (blocks > 1024u) blocks = 1024u;
    const cudaError_t e = launch_programmatic_grid(rope_table_kernel, dim3(blocks, rot / 2), 256, 0, stream, table, rows,
                                                   rot, base, stretch, original, low, high, gain);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}
