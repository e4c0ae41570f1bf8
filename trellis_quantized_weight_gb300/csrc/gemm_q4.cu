// trellis_gemm_q4: the entry point of the products with 4-bit weights in groups.
#include "gemm_q4.cuh"

namespace trellis {

template <> cudaError_t launch_q4_mma<32>(const Q4Args&, const DeviceInfo&, cudaStream_t);
template <> cudaError_t launch_q4_mma<64>(const Q4Args&, const DeviceInfo&, cudaStream_t);
template <> cudaError_t launch_q4_mma<128>(const Q4Args&, const DeviceInfo&, cudaStream_t);

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// More rows than the register tiles' kernel takes at once go to the tensor cores' tiles.
bool on_tensor_cores(int M) { return M > 0; }

int check_sizes(int M, int K, int N, int group) {
    if (M < 0 || K < 1 || N < 1) return TRELLIS_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128) return TRELLIS_ERR_UNSUPPORTED;
    if (K % group != 0) return TRELLIS_ERR_SHAPE;
    if (M > 65536 || K > (1 << 20) || N > (1 << 20)) return TRELLIS_ERR_UNSUPPORTED;
    return TRELLIS_OK;
}

}  // namespace

}  // namespace trellis

extern "C" {

int trellis_gemm_q4_workspace_size(int M, int K, int N, int group, int eight, int bias, size_t* bytes) {
    using namespace trellis;
    if (bytes == nullptr) return TRELLIS_ERR_NULL;
    const int rc = check_sizes(M, K, N, group);
    if (rc != TRELLIS_OK) return rc;
    *bytes = on_tensor_cores(M) ? q4_tc_workspace_bytes(M, K, eight != 0) : 0;
    (void)bias;
    return TRELLIS_OK;
}

int trellis_gemm_q4(const void* x, const float* x_scales, const uint32_t* codes, const uint16_t* scales, const uint16_t* biases,
                    int M, int K, int N, int group, uint16_t* out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace trellis;
    if (x == nullptr || codes == nullptr || scales == nullptr || out == nullptr) return TRELLIS_ERR_NULL;
    int rc = check_sizes(M, K, N, group);
    if (rc != TRELLIS_OK) return rc;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(biases, 2) || !aligned(x_scales, 4) || !aligned(out, 2))
        return TRELLIS_ERR_ALIGN;
    if (M == 0) return TRELLIS_OK;
    const size_t need = on_tensor_cores(M) ? q4_tc_workspace_bytes(M, K, x_scales != nullptr) : 0;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return TRELLIS_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return TRELLIS_ERR_ALIGN;
    DeviceInfo dev;
    rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    Q4Args a;
    a.x = x; a.codes = codes; a.scales = scales; a.biases = biases; a.x_scales = x_scales; a.out = out;
    a.M = M; a.K = K; a.N = N; a.groups = K / group;
    const cudaError_t e = on_tensor_cores(M) ? launch_q4_tc(a, group, workspace, dev, stream)
                          : group == 32 ? launch_q4_mma<32>(a, dev, stream)
                          : group == 64 ? launch_q4_mma<64>(a, dev, stream) : launch_q4_mma<128>(a, dev, stream);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

}  // extern "C"
