// trellis_kv_attention: argument checks and the choice of kernel.
#include <cmath>

#include "kv_attention.cuh"
#include "trellis.h"

namespace {

using trellis::DeviceInfo;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Query rows to a key head of the longest sequence, as the caller gives it.
int rows_of(int tokens, int max_q, int q_heads, int kv_heads) {
    const long long n = max_q < tokens ? max_q : tokens;
    const long long r = n * (q_heads / kv_heads);
    return r > (1 << 30) ? 1 << 30 : static_cast<int>(r < 1 ? 1 : r);
}

// The tensor-core kernel where a sequence has more rows to a key head than one unit of the
// streaming kernel, whose time grows with every 8 or 16 rows while the other's does not.
// Measured, us streaming / tensor cores, 16 sequences of 300 to 9000 tokens and 8 key heads
// (4 at D = 256): D = 128, 16 rows 59 / 77, 18 to 24 98 / 78, 32 104 / 79, 64 197 / 83;
// D = 256, 8 rows 41 / 65, 16 72 / 67, 24 95 / 68, 40 154 / 71.  One sequence of 100000:
// D = 128, 16 rows 58 / 90, 24 93 / 94, 40 128 / 97; D = 256, 16 rows 79 / 74, 24 107 / 81.
// At D = 64 two units still take less: 16 sequences, 24 rows 69 / 68, 32 70 / 69, 40 98 / 70;
// one, 32 rows 64 / 83, 40 87 / 86.
bool on_tensor_cores(int head_dim, int rows) { return rows > (head_dim == 64 ? 32 : 16); }

size_t workspace_bytes_of(int tokens, int seqs, int rows, int q_heads, int kv_heads, int head_dim,
                          const DeviceInfo& dev) {
    return on_tensor_cores(head_dim, rows)
               ? trellis::kv_tile_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim, dev)
               : trellis::kv_stream_workspace_bytes(head_dim, rows, dev);
}

}  // namespace

extern "C" {

int trellis_kv_attention_workspace_size(int tokens, int seqs, int max_q, int q_heads, int kv_heads, int head_dim,
                                        size_t* bytes) {
    if (bytes == nullptr) return TRELLIS_ERR_NULL;
    if (tokens < 0 || seqs < 1 || max_q < 1 || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0)
        return TRELLIS_ERR_SHAPE;
    if (seqs > trellis::kKvMaxSeqs || q_heads > trellis::kKvMaxHeads) return TRELLIS_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return TRELLIS_ERR_UNSUPPORTED;
    DeviceInfo dev;
    const int rc = trellis::device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    *bytes = workspace_bytes_of(tokens, seqs, rows_of(tokens, max_q, q_heads, kv_heads), q_heads, kv_heads, head_dim, dev);
    return TRELLIS_OK;
}

int trellis_kv_attention(const uint16_t* q, long long q_stride, const int* starts, const int* kv_len, const int* pages,
                         int tokens, int seqs, int max_q, int page_cols, int num_pages, int q_heads, int kv_heads,
                         int head_dim, int page_size, float scale, int window, const uint8_t* k_codes,
                         const uint8_t* v_codes, const float* k_scales, const float* v_scales, uint16_t* out,
                         void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace trellis;
    if (q == nullptr || out == nullptr) return TRELLIS_ERR_NULL;
    int rc = check_kv(starts, kv_len, pages, tokens, seqs, max_q, page_cols, num_pages, q_heads, kv_heads, head_dim,
                      page_size, k_codes, v_codes, k_scales, v_scales);
    if (rc != TRELLIS_OK) return rc;
    if (q_stride < static_cast<long long>(q_heads) * head_dim || window < 0 || !std::isfinite(scale))
        return TRELLIS_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8 != 0) return TRELLIS_ERR_ALIGN;
    DeviceInfo dev;
    rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    const int rows = rows_of(tokens, max_q, q_heads, kv_heads);
    if (workspace == nullptr ||
        workspace_bytes < workspace_bytes_of(tokens, seqs, rows, q_heads, kv_heads, head_dim, dev))
        return TRELLIS_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return TRELLIS_ERR_ALIGN;
    if (tokens == 0) return TRELLIS_OK;
    AttendArgs a;
    a.l = kv_layout(starts, kv_len, pages, tokens, seqs, page_cols, num_pages, q_heads, kv_heads, page_size);
    a.q = q; a.q_stride = q_stride;
    a.group = q_heads / kv_heads;
    a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.k_codes = k_codes; a.v_codes = v_codes; a.k_scales = k_scales; a.v_scales = v_scales;
    a.out = out;
    a.counters = static_cast<unsigned int*>(workspace);
    a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + kKvCounterBytes);
    return on_tensor_cores(head_dim, rows) ? launch_kv_tile(a, head_dim, dev, stream)
                                           : launch_kv_stream(a, head_dim, rows, dev, stream);
}

}  // extern "C"
