// Pages of the paged cache, handed out and taken back on the device: trellis_kv_grow,
// trellis_kv_fork and trellis_kv_compact.
//
// refs[p] counts the places of the table that name page p; 0 is free.  A call hands out the
// lowest free pages, to sequences in their order, so the result is one function of the arrays
// and not of how threads meet.  The pages that a call gives back are free from the next call
// on: a page handed out is one that nothing named when the call began, so no copy of this call
// reads it, and the counts may be changed in any order.
//
//   need of a sequence = pages(new length) - pages(old length); its pages are the free ones of
//   ranks [sum of the needs before it, that + its need), by prefix sums over needs and over the
//   free flags.
//
// All three are bound by latency but for the bytes that fork and compact copy: a growth of 5 tokens 4 us, of 64 prompts of
// up to 16384 tokens 10.5 (one CTA: the scans need all needs and counts anyway, and more CTAs a barrier between them); a
// fork of 24 x 4 beams 9.9 us with 27 MB of copies; compaction of 8 short sequences 8.6 us, of
// 0.73 GB 220 us, 6.6 TB/s of the 6.7 that a copy reaches.
#include "kv_cache.cuh"
#include "trellis.h"

namespace trellis {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr size_t kCounters = size_t(1) << 20;      // the products' counters in front of a workspace stay zero

__device__ __forceinline__ long long pages_of(long long tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// Sum over the CTA and over the threads before this one.  part: kWarps values, free on entry.
template <class T>
__device__ __forceinline__ T scan(T v, T& total, T* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31) part[warp] = sum;
    __syncthreads();
    const T mine = part[lane];
    T upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
    }
    total = __shfl_sync(0xffffffffu, upto, 31);
    const T before = __shfl_sync(0xffffffffu, upto - mine, warp);
    __syncthreads();
    return before + sum - v;
}

// The first `want` free pages to list, in order; returns how many there are (at most `want`).
// A warp takes 32 * kRun counts at a time, a bit mask for each 32.
__device__ __forceinline__ int list_free(const int* refs, int num_pages, int want, int* list, int* part) {
    constexpr int kRun = 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int found = 0;
    for (long long first = 0; first < num_pages && found < want; first += kThreads * kRun) {
        const long long base = first + warp * (32 * kRun) + lane;
        uint32_t mask[kRun];
        int v[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) v[i] = base + 32 * i < num_pages ? refs[base + 32 * i] : 1;
        int count = 0;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            mask[i] = __ballot_sync(0xffffffffu, v[i] == 0);
            count += __popc(mask[i]);
        }
        int total;
        // a warp's count, at its first lane
        int at = found + scan(lane == 0 ? count : 0, total, part);
        at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int rank = at + __popc(mask[i] & ((1u << lane) - 1u));
            if (v[i] == 0 && rank < want) list[rank] = static_cast<int>(base + 32 * i);
            at += __popc(mask[i]);
        }
        found += total;
    }
    return found < want ? found : want;
}

// ---- grow -----------------------------------------------------------------------------
struct GrowArgs {
    int *refs, *kv_len, *pages;
    const int* grow;
    uint8_t* ok;
    int *upto, *list;                   // [seqs] needs before each sequence's; the free pages
    int seqs, cols, num_pages, shift;
};

struct Growth {
    long long now, have, want;          // tokens afterwards; pages before and afterwards
    int g;
};
__device__ __forceinline__ Growth growth(const GrowArgs& a, int s) {
    Growth r;
    const int old = max(a.kv_len[s], 0);
    r.g = a.grow[s];
    r.now = max(static_cast<long long>(old) + r.g, 0ll);
    r.have = min(pages_of(old, a.shift), static_cast<long long>(a.cols));
    r.want = pages_of(r.now, a.shift);
    return r;
}

// A warp's way through `count` page ids: eight loads a lane before the first use (one at a time, 64 prompts of up to 16384
// tokens in pages of 32 took 14.5 us).
template <class Load, class Use>
__device__ __forceinline__ void eight_at_once(long long count, int lane, Load load, Use use) {
    for (long long i0 = lane; i0 < count; i0 += 256) {
        int id[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) id[j] = i0 + 32 * j < count ? load(i0 + 32 * j) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i0 + 32 * j < count) use(i0 + 32 * j, id[j]);
    }
}

__global__ void __launch_bounds__(kThreads) kv_grow_kernel(const __grid_constant__ GrowArgs a) {
    __shared__ int part[kWarps];
    __shared__ long long part64[kWarps];
    griddep_wait();
    griddep_launch_dependents();        // the next grid's start beside this one; it waits for the end before it reads
    // needs, and the sequences that are not served whatever the pool holds
    long long before = 0;
    for (int s0 = 0; s0 < a.seqs; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        long long need = 0, total;
        if (s < a.seqs) {
            const Growth r = growth(a, s);
            bool ok = true;
            if (r.g > 0) {
                ok = r.want <= a.cols && r.now <= 0x7fffffffll;
                if (ok) need = r.want - r.have;
            } else if (r.g < 0 && (r.now & ((1 << a.shift) - 1)) != 0 && r.want <= a.cols) {
                // tokens to come would go to a page that another sequence names too
                const int id = a.pages[static_cast<size_t>(s) * a.cols + r.want - 1];
                ok = id < 0 || id >= a.num_pages || a.refs[id] <= 1;
            }
            a.ok[s] = ok;
        }
        const long long at = before + scan(need, total, part64);
        if (s < a.seqs) a.upto[s] = static_cast<int>(min(at, 0x7fffffffll));
        before += total;
    }
    const int wanted = static_cast<int>(min(before, static_cast<long long>(a.num_pages)));
    const int found = list_free(a.refs, a.num_pages, wanted, a.list, part);
    __syncthreads();                    // the list, `ok` and `upto` are written, the counts read
    const int lane = threadIdx.x & 31;
    for (int s = threadIdx.x >> 5; s < a.seqs; s += kWarps) {
        const Growth r = growth(a, s);
        bool ok = a.ok[s];
        __syncwarp();                   // lane 0 writes both below
        int* row = a.pages + static_cast<size_t>(s) * a.cols;
        if (ok && r.g > 0) {
            const long long need = r.want - r.have, at = a.upto[s];
            ok = need == 0 || at + need <= found;
            if (ok)
                eight_at_once(need, lane, [&](long long i) { return a.list[at + i]; }, [&](long long i, int id) {
                    row[r.have + i] = id;
                    a.refs[id] = 1;
                });
        } else if (ok && r.g < 0) {
            eight_at_once(r.have - r.want, lane, [&](long long i) { return row[r.want + i]; }, [&](long long, int id) {
                if (id >= 0 && id < a.num_pages) atomicSub(a.refs + id, 1);
            });
        }
        if (lane == 0) {
            if (ok && r.g != 0) a.kv_len[s] = static_cast<int>(r.now);
            a.ok[s] = ok;
        }
    }
}

// ---- fork -----------------------------------------------------------------------------
struct ForkArgs {
    int *refs, *kv_len, *pages;
    const int* parents;
    uint8_t* ok;
    int *old_len, *now, *fresh, *list, *rows;      // [seqs] lengths before and afterwards and pages for copies; list; rows before
    uint8_t* codes[2];
    float* scales[2];
    int seqs, cols, num_pages, shift, kv_heads, head_dim;
};

// The plan by one CTA; the others keep the rows that the second kernel changes and may have to read.
__global__ void __launch_bounds__(kThreads) kv_fork_plan_kernel(const __grid_constant__ ForkArgs a) {
    extern __shared__ int first[];                  // [seqs] the sequence that keeps a parent's last page
    __shared__ int part[kWarps];
    griddep_wait();
    griddep_launch_dependents();        // the next grid's start beside this one; it waits for the end before it reads
    if (blockIdx.x > 0) {
        for (int s = blockIdx.x - 1; s < a.seqs; s += gridDim.x - 1) {
            if (a.parents[s] == s) continue;
            const long long have = min(pages_of(max(a.kv_len[s], 0), a.shift), static_cast<long long>(a.cols));
            const size_t row = static_cast<size_t>(s) * a.cols;
            for (int c = threadIdx.x; c < have; c += kThreads) a.rows[row + c] = a.pages[row + c];
        }
        return;
    }
    for (int s = threadIdx.x; s < a.seqs; s += kThreads) first[s] = 0x7fffffff;
    __syncthreads();
    for (int s = threadIdx.x; s < a.seqs; s += kThreads) {
        const int p = a.parents[s];
        if (p >= 0 && p < a.seqs) atomicMin(first + p, p == s ? -1 : s);      // -1: the sequence itself
    }
    __syncthreads();
    int copies = 0;
    for (int s0 = 0; s0 < a.seqs; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        int copy = 0, total, len = 0;
        if (s < a.seqs) {
            const int p = a.parents[s];
            if (p >= 0 && p < a.seqs) {
                len = max(a.kv_len[p], 0);
                const bool keeps = p == s || first[p] == s;
                copy = !keeps && (len & ((1 << a.shift) - 1)) != 0 && (len >> a.shift) < a.cols;
            }
            a.old_len[s] = max(a.kv_len[s], 0);
            a.now[s] = len;
        }
        const int rank = copies + scan(copy, total, part);
        if (s < a.seqs) a.fresh[s] = copy ? rank : -1;
        copies += total;
    }
    const int found = list_free(a.refs, a.num_pages, min(copies, a.num_pages), a.list, part);
    __syncthreads();
    for (int s = threadIdx.x; s < a.seqs; s += kThreads) {
        const int rank = a.fresh[s];
        const bool lost = rank >= found;
        if (rank >= 0) a.fresh[s] = lost ? -1 : a.list[rank];
        if (lost) a.now[s] = 0;
        a.ok[s] = !lost && a.parents[s] < a.seqs;
    }
}

// Column y = 0: a sequence's row and its pages' counts.  The others: a head's keys or values of the page that it copies.
__global__ void __launch_bounds__(256) kv_fork_apply_kernel(const __grid_constant__ ForkArgs a) {
    griddep_wait();
    griddep_launch_dependents();        // the next grid's start beside this one; it waits for the end before it reads
    const int s = blockIdx.x, p = a.parents[s];
    if (p == s) return;
    const int now = a.now[s], fresh = a.fresh[s], whole = now >> a.shift;
    const bool alive = p >= 0 && p < a.seqs;
    const int from = alive ? p : s;
    // the parent's row as it was: rows that stay are where they were
    const int* of = (alive && a.parents[from] == from ? a.pages : a.rows) + static_cast<size_t>(from) * a.cols;
    if (blockIdx.y == 0) {
        int* row = a.pages + static_cast<size_t>(s) * a.cols;
        const int had = static_cast<int>(min(pages_of(a.old_len[s], a.shift), static_cast<long long>(a.cols)));
        const int has = static_cast<int>(min(pages_of(now, a.shift), static_cast<long long>(a.cols)));
        for (int c = threadIdx.x; c < max(had, has); c += 256) {
            const int old = c < had ? row[c] : -1;
            const int id = c >= has ? -1 : c == whole && fresh >= 0 ? fresh : of[c];
            if (old != id) {
                if (old >= 0 && old < a.num_pages) atomicSub(a.refs + old, 1);
                if (id >= 0 && id < a.num_pages) atomicAdd(a.refs + id, 1);
            }
            if (c < has) row[c] = id;
        }
        if (threadIdx.x == 0) a.kv_len[s] = now;
        return;
    }
    if (fresh < 0) return;
    const int h = (blockIdx.y - 1) >> 1, kv = (blockIdx.y - 1) & 1;
    const int src = min(max(of[whole], 0), a.num_pages - 1);
    const int blocks = ((now & ((1 << a.shift) - 1)) + kKvBlock - 1) / kKvBlock;
    const size_t src_unit = static_cast<size_t>(src) * a.kv_heads + h, dst_unit = static_cast<size_t>(fresh) * a.kv_heads + h;
    const size_t page_bytes = static_cast<size_t>(a.head_dim) << a.shift;
    const uint4* in = reinterpret_cast<const uint4*>(a.codes[kv] + src_unit * page_bytes);
    uint4* out = reinterpret_cast<uint4*>(a.codes[kv] + dst_unit * page_bytes);
    const int n = blocks * kKvBlock * a.head_dim / 16;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += 256) out[i] = in[i];
    const int per = 1 << (a.shift - 4);
    if (threadIdx.x < blocks) a.scales[kv][dst_unit * per + threadIdx.x] = a.scales[kv][src_unit * per + threadIdx.x];
}

// ---- compact --------------------------------------------------------------------------
constexpr int kRankChunk = 4096;        // pages of a CTA that ranks

struct CompactArgs {
    const int *refs, *kv_len, *pages;
    int *refs_out, *kv_len_out, *pages_out;
    int *local, *chunks;                // [num_pages] used pages before this one in its chunk; [chunks] used pages of each
    const uint8_t* codes[2];
    const float* scales[2];
    uint8_t* codes_out[2];
    float* scales_out[2];
    int seqs, cols, num_pages, room, shift;
    int code_vecs, page_scales;         // 16-byte pieces of a page's codes, floats of its scales
};

__global__ void __launch_bounds__(kThreads) kv_rank_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ int part[kWarps];
    griddep_wait();
    griddep_launch_dependents();        // the next grid's start beside this one; it waits for the end before it reads
    int before = 0;
    for (int i = 0; i < kRankChunk; i += kThreads) {
        const long long p = static_cast<long long>(blockIdx.x) * kRankChunk + i + threadIdx.x;
        int total;
        const int used = p < a.num_pages && a.refs[p] > 0;
        const int at = before + scan(used, total, part);
        if (p < a.num_pages) a.local[p] = used ? at : -1;
        before += total;
    }
    if (threadIdx.x == 0) a.chunks[blockIdx.x] = before;
    for (long long p = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; p < a.room; p += static_cast<long long>(gridDim.x) * kThreads)
        a.refs_out[p] = 0;
}

__global__ void __launch_bounds__(256) kv_compact_kernel(const __grid_constant__ CompactArgs a, int chunks) {
    extern __shared__ int base[];       // used pages before each chunk
    __shared__ int warp_sum[8];
    griddep_wait();
    griddep_launch_dependents();        // the next grid's start beside this one; it waits for the end before it reads
    // prefix sums of the chunks: a thread takes a run of them
    const int run = (chunks + 255) / 256, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = 0;
    for (int i = 0; i < run; ++i) {
        const int c = threadIdx.x * run + i;
        if (c < chunks) sum += a.chunks[c];
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int at = upto - sum;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    for (int i = 0; i < run; ++i) {
        const int c = threadIdx.x * run + i;
        if (c < chunks) {
            base[c] = at;
            at += a.chunks[c];
        }
    }
    __syncthreads();
    // where a page goes; -1 for one that is free or not of the pool
    auto place = [&](int p) {
        if (p < 0 || p >= a.num_pages) return -1;
        const int local = a.local[p];
        return local < 0 ? -1 : base[p / kRankChunk] + local;
    };
    for (int s = blockIdx.x; s < a.seqs; s += gridDim.x) {
        const int len = max(a.kv_len[s], 0);
        const int have = static_cast<int>(min(pages_of(len, a.shift), static_cast<long long>(a.cols)));
        const size_t row = static_cast<size_t>(s) * a.cols;
        // an entry that is no page in use has no place either: as page 0 it would be another sequence's
        int left = 0;
        for (int c = threadIdx.x; c < have; c += 256) left |= static_cast<unsigned>(place(a.pages[row + c])) >= static_cast<unsigned>(a.room);
        left = __syncthreads_or(left);
        for (int c = threadIdx.x; c < a.cols; c += 256) {
            const int to = c < have ? place(a.pages[row + c]) : -1;
            a.pages_out[row + c] = left ? 0 : max(to, 0);
            if (left && to >= 0 && to < a.room) atomicSub(a.refs_out + to, 1);
        }
        if (threadIdx.x == 0) a.kv_len_out[s] = left ? 0 : a.kv_len[s];
    }
    for (int p = blockIdx.x; p < a.num_pages; p += gridDim.x) {
        const int to = place(p);
        if (to < 0 || to >= a.room) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint4* in = reinterpret_cast<const uint4*>(a.codes[kv]) + static_cast<size_t>(p) * a.code_vecs;
            uint4* out = reinterpret_cast<uint4*>(a.codes_out[kv]) + static_cast<size_t>(to) * a.code_vecs;
            // eight loads before the first store (ordinary ones, which the compiler does not take past a store by itself: 249 us)
            for (int i0 = threadIdx.x; i0 < a.code_vecs; i0 += 8 * 256) {
                uint4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i0 + 256 * j < a.code_vecs) v[j] = in[i0 + 256 * j];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i0 + 256 * j < a.code_vecs) out[i0 + 256 * j] = v[j];
            }
            for (int i = threadIdx.x; i < a.page_scales; i += 256)
                a.scales_out[kv][static_cast<size_t>(to) * a.page_scales + i] = a.scales[kv][static_cast<size_t>(p) * a.page_scales + i];
        }
        if (threadIdx.x == 0) atomicAdd(a.refs_out + to, a.refs[p]);
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int page_shift(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : 0; }

// The checks that the three share, in this order: pointers, sizes, alignment.
int check_pages(const int* refs, const int* kv_len, const int* pages, int seqs, int page_cols, int num_pages, int page_size) {
    if (refs == nullptr || kv_len == nullptr || pages == nullptr) return TRELLIS_ERR_NULL;
    if (seqs < 1 || page_cols < 1 || num_pages < 1) return TRELLIS_ERR_SHAPE;
    if (seqs > kKvMaxSeqs || num_pages > kKvMaxPages || page_cols > kKvMaxPages || page_shift(page_size) == 0) return TRELLIS_ERR_UNSUPPORTED;
    if (!aligned(refs, 4) || !aligned(kv_len, 4) || !aligned(pages, 4)) return TRELLIS_ERR_ALIGN;
    return TRELLIS_OK;
}

int check_cache(int kv_heads, int head_dim, const void* k_codes, const void* v_codes, const float* k_scales, const float* v_scales) {
    if (k_codes == nullptr || v_codes == nullptr || k_scales == nullptr || v_scales == nullptr) return TRELLIS_ERR_NULL;
    if (kv_heads < 1) return TRELLIS_ERR_SHAPE;
    if (kv_heads > kKvMaxHeads || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return TRELLIS_ERR_UNSUPPORTED;
    if (!aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_scales, 4) || !aligned(v_scales, 4)) return TRELLIS_ERR_ALIGN;
    return TRELLIS_OK;
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (workspace == nullptr || bytes < need) return TRELLIS_ERR_WORKSPACE;
    return aligned(workspace, 256) ? TRELLIS_OK : TRELLIS_ERR_ALIGN;
}

size_t grow_bytes(int seqs, int num_pages) { return kCounters + 4 * (static_cast<size_t>(seqs) + num_pages); }
size_t fork_bytes(int seqs, int cols) { return kCounters + 4 * (static_cast<size_t>(seqs) * 4 + static_cast<size_t>(seqs) * cols); }
int rank_chunks(int num_pages) { return (num_pages + kRankChunk - 1) / kRankChunk; }
size_t compact_bytes(int num_pages) { return kCounters + 4 * (static_cast<size_t>(num_pages) + rank_chunks(num_pages)); }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace

}  // namespace trellis

extern "C" {

int trellis_kv_pages_workspace_size(int seqs, int page_cols, int num_pages, size_t* bytes) {
    using namespace trellis;
    if (bytes == nullptr) return TRELLIS_ERR_NULL;
    if (seqs < 1 || page_cols < 1 || num_pages < 1) return TRELLIS_ERR_SHAPE;
    if (seqs > kKvMaxSeqs || num_pages > kKvMaxPages || page_cols > kKvMaxPages) return TRELLIS_ERR_UNSUPPORTED;
    size_t n = grow_bytes(seqs, num_pages);
    if (fork_bytes(seqs, page_cols) > n) n = fork_bytes(seqs, page_cols);
    if (compact_bytes(num_pages) > n) n = compact_bytes(num_pages);
    *bytes = n;
    return TRELLIS_OK;
}

int trellis_kv_grow(int* refs, int* kv_len, int* pages, const int* grow, int seqs, int page_cols, int num_pages, int page_size,
                    uint8_t* ok, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace trellis;
    if (grow == nullptr || ok == nullptr) return TRELLIS_ERR_NULL;
    int rc = check_pages(refs, kv_len, pages, seqs, page_cols, num_pages, page_size);
    if (rc != TRELLIS_OK) return rc;
    if (!aligned(grow, 4)) return TRELLIS_ERR_ALIGN;
    rc = check_workspace(workspace, workspace_bytes, grow_bytes(seqs, num_pages));
    if (rc != TRELLIS_OK) return rc;
    GrowArgs a;
    a.refs = refs; a.kv_len = kv_len; a.pages = pages; a.grow = grow; a.ok = ok;
    a.upto = reinterpret_cast<int*>(static_cast<char*>(workspace) + kCounters);
    a.list = a.upto + seqs;
    a.seqs = seqs; a.cols = page_cols; a.num_pages = num_pages; a.shift = page_shift(page_size);
    return launch_programmatic(kv_grow_kernel, 1u, kThreads, 0, stream, a) == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

int trellis_kv_fork(int* refs, int* kv_len, int* pages, const int* parents, int seqs, int page_cols, int num_pages, int page_size,
                    int kv_heads, int head_dim, uint8_t* k_codes, uint8_t* v_codes, float* k_scales, float* v_scales, uint8_t* ok,
                    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace trellis;
    if (parents == nullptr || ok == nullptr) return TRELLIS_ERR_NULL;
    int rc = check_pages(refs, kv_len, pages, seqs, page_cols, num_pages, page_size);
    if (rc == TRELLIS_OK) rc = check_cache(kv_heads, head_dim, k_codes, v_codes, k_scales, v_scales);
    if (rc != TRELLIS_OK) return rc;
    if (!aligned(parents, 4)) return TRELLIS_ERR_ALIGN;
    rc = check_workspace(workspace, workspace_bytes, fork_bytes(seqs, page_cols));
    if (rc != TRELLIS_OK) return rc;
    DeviceInfo dev;
    rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    ForkArgs a;
    a.refs = refs; a.kv_len = kv_len; a.pages = pages; a.parents = parents; a.ok = ok;
    a.old_len = reinterpret_cast<int*>(static_cast<char*>(workspace) + kCounters);
    a.now = a.old_len + seqs; a.fresh = a.now + seqs; a.list = a.fresh + seqs; a.rows = a.list + seqs;
    a.codes[0] = k_codes; a.codes[1] = v_codes; a.scales[0] = k_scales; a.scales[1] = v_scales;
    a.seqs = seqs; a.cols = page_cols; a.num_pages = num_pages; a.shift = page_shift(page_size);
    a.kv_heads = kv_heads; a.head_dim = head_dim;
    static std::atomic<unsigned long long> done{0};
    const size_t smem = static_cast<size_t>(seqs) * 4;
    if (smem > 40 * 1024 && !smem_opt_in(kv_fork_plan_kernel, kKvMaxSeqs * 4, done)) return TRELLIS_ERR_CUDA;
    const int keepers = seqs < 2 * dev.num_sms ? seqs : 2 * dev.num_sms;
    cudaError_t e = launch_programmatic(kv_fork_plan_kernel, 1u + keepers, kThreads, smem, stream, a);
    if (e != cudaSuccess) return TRELLIS_ERR_CUDA;
    e = launch_programmatic_grid(kv_fork_apply_kernel, dim3(seqs, 1 + 2 * kv_heads), 256, 0, stream, a);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

int trellis_kv_compact(const int* refs, const int* kv_len, const int* pages, int seqs, int page_cols, int num_pages, int page_size,
                       int kv_heads, int head_dim, const uint8_t* k_codes, const uint8_t* v_codes, const float* k_scales,
                       const float* v_scales, int num_pages_out, uint8_t* k_codes_out, uint8_t* v_codes_out, float* k_scales_out,
                       float* v_scales_out, int* refs_out, int* kv_len_out, int* pages_out, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
    using namespace trellis;
    if (refs_out == nullptr || kv_len_out == nullptr || pages_out == nullptr) return TRELLIS_ERR_NULL;
    int rc = check_pages(refs, kv_len, pages, seqs, page_cols, num_pages, page_size);
    if (rc == TRELLIS_OK) rc = check_cache(kv_heads, head_dim, k_codes, v_codes, k_scales, v_scales);
    if (rc == TRELLIS_OK) rc = check_cache(kv_heads, head_dim, k_codes_out, v_codes_out, k_scales_out, v_scales_out);
    if (rc != TRELLIS_OK) return rc;
    if (num_pages_out < 1) return TRELLIS_ERR_SHAPE;
    if (num_pages_out > kKvMaxPages) return TRELLIS_ERR_UNSUPPORTED;
    if (!aligned(refs_out, 4) || !aligned(kv_len_out, 4) || !aligned(pages_out, 4)) return TRELLIS_ERR_ALIGN;
    const size_t code_bytes = static_cast<size_t>(kv_heads) * page_size * head_dim;
    const size_t scale_bytes = static_cast<size_t>(kv_heads) * (page_size / kKvBlock) * 4;
    const size_t lens = static_cast<size_t>(seqs) * 4, table = lens * page_cols;
    const struct { const void* p; size_t n; } in[] = {
        {k_codes, code_bytes * num_pages}, {v_codes, code_bytes * num_pages}, {k_scales, scale_bytes * num_pages},
        {v_scales, scale_bytes * num_pages}, {refs, 4ull * num_pages}, {kv_len, lens}, {pages, table}};
    const struct { const void* p; size_t n; } out[] = {
        {k_codes_out, code_bytes * num_pages_out}, {v_codes_out, code_bytes * num_pages_out}, {k_scales_out, scale_bytes * num_pages_out},
        {v_scales_out, scale_bytes * num_pages_out}, {refs_out, 4ull * num_pages_out}, {kv_len_out, lens}, {pages_out, table}};
    for (int i = 0; i < 7; ++i)
        for (int j = 0; j < 7; ++j)
            if (overlap(in[i].p, in[i].n, out[j].p, out[j].n) || (i < j && overlap(out[i].p, out[i].n, out[j].p, out[j].n)))
                return TRELLIS_ERR_SHAPE;
    rc = check_workspace(workspace, workspace_bytes, compact_bytes(num_pages));
    if (rc != TRELLIS_OK) return rc;
    DeviceInfo dev;
    rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    CompactArgs a;
    a.refs = refs; a.kv_len = kv_len; a.pages = pages;
    a.refs_out = refs_out; a.kv_len_out = kv_len_out; a.pages_out = pages_out;
    a.local = reinterpret_cast<int*>(static_cast<char*>(workspace) + kCounters);
    a.chunks = a.local + num_pages;
    a.codes[0] = k_codes; a.codes[1] = v_codes; a.scales[0] = k_scales; a.scales[1] = v_scales;
    a.codes_out[0] = k_codes_out; a.codes_out[1] = v_codes_out; a.scales_out[0] = k_scales_out; a.scales_out[1] = v_scales_out;
    a.seqs = seqs; a.cols = page_cols; a.num_pages = num_pages; a.room = num_pages_out; a.shift = page_shift(page_size);
    a.code_vecs = static_cast<int>(code_bytes / 16);
    a.page_scales = static_cast<int>(scale_bytes / 4);
    const int chunks = rank_chunks(num_pages);
    cudaError_t e = launch_programmatic(kv_rank_kernel, static_cast<unsigned>(chunks), kThreads, 0, stream, a);
    if (e != cudaSuccess) return TRELLIS_ERR_CUDA;
    // Many more CTAs than run at once (8 an SM): those that find free pages make room at once for others, and pages that are copied
    // at the same time lie near each other.  0.73 GB with 8 CTAs an SM 250 us, 16 235, 32 226, 48 221.5, 96 the same.
    const int most = num_pages > seqs ? num_pages : seqs, ctas = 48 * dev.num_sms;
    e = launch_programmatic(kv_compact_kernel, static_cast<unsigned>(most < ctas ? most : ctas), 256u, static_cast<size_t>(chunks) * 4,
                            stream, a, chunks);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

}  // extern "C"
