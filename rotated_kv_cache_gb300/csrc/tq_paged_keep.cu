// tq_paged_keep.cu -- the accepted rows of a verified step moved together.
//
//   row (len - n + path[k])  ->  row (len - n + k),   k < kept
//
// for the n new tokens of a sequence, all five planes, byte for byte.  A path
// grows strictly, so path[k] >= k: a row is never moved over one that a later k
// still needs, but over ones of its own group of rows; a CTA takes a (sequence,
// kv-head), reads a group of rows into registers, waits, and writes it.
//
// A few rows of 200 bytes for each of hundreds of CTAs: bound by the latency of
// three dependent loads (path, page, row).
// 32 sequences of up to 5 kept rows, 8 kv-heads: 3.4 us, of which a launch is 2; 256 of up
// to 12, 4 kv-heads at head_dim 256: 7.2 us.
#include "tq_common.cuh"
#include "tq_kernels.h"
#include "tq_paged.cuh"

namespace tq {
namespace {

constexpr int kpThreads = 128;
constexpr int kpWords = 8;   // of a thread, in flight
constexpr int kpRows = 32;   // of a group, at most

struct KeepParams {
    PagedView v;
    int64_t max_new;
    const int32_t *path, *kept;
    int64_t path_stride;
    int32_t *lens_out;
    uint32_t *plane[5];
    int words[5];   // 32-bit words of a row in each plane
    int row_words;  // of all planes
    int H;
};

__global__ void __launch_bounds__(kpThreads) paged_keep_kernel(const __grid_constant__ KeepParams p)
{
    __shared__ int64_t from[kpRows], to[kpRows];  // plane rows
    pdl_wait_primary();
    pdl_allow_dependents();
    const int s = blockIdx.x / p.H, h = blockIdx.x - s * p.H, tid = threadIdx.x;
    const int64_t n = paged_new(p.v, s), len = paged_len(p.v, s);
    const int32_t *path = p.path + s * p.path_stride;
    const int kept = p.kept[s];
    bool good = kept >= 0 && kept <= n && n <= p.max_new;
    if (good)
        for (int k = tid; k < kept; k += kpThreads) {
            const int i = path[k];
            good &= i >= k && i < n && (k == 0 || i > path[k - 1]);
        }
    good = __syncthreads_and(good);
    if (tid == 0 && h == 0) {
        const int64_t left = len - n + kept;
        p.lens_out[s] = (int)(!good ? len : left < 0 ? 0 : left);
        if (!good) atomicOr(p.v.err, kErrTree);
    }
    if (!good) return;
    const int group = kpThreads * kpWords / p.row_words < kpRows ? kpThreads * kpWords / p.row_words : kpRows;
    auto place = [&](int64_t pos) -> int64_t {
        if (pos < 0) return -1;  // stands before the sequence's first row
        uint32_t slot;
        const int page = paged_page(p.v, s, (uint32_t)pos, slot);
        return page < 0 ? -1 : ((int64_t)page * p.H + h) * p.v.page + slot;
    };
    for (int k0 = 0; k0 < kept; k0 += group) {
        const int rows = kept - k0 < group ? kept - k0 : group;
        __syncthreads();  // the previous group is written
        if (tid < rows) {
            const int i = path[k0 + tid];
            from[tid] = i == k0 + tid ? -1 : place(len - n + i);
            to[tid] = i == k0 + tid ? -1 : place(len - n + k0 + tid);
        }
        __syncthreads();
        uint32_t x[kpWords];
        uint32_t *dst[kpWords];
#pragma unroll
        for (int j = 0; j < kpWords; ++j) {
            const int it = tid + j * kpThreads, r = it / p.row_words;
            dst[j] = nullptr;
            if (r < rows && from[r] >= 0 && to[r] >= 0) {
                int w = it - r * p.row_words, k = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (k == q && w >= p.words[q]) {
                        w -= p.words[q];
                        k = q + 1;
                    }
                x[j] = p.plane[k][from[r] * p.words[k] + w];
                dst[j] = p.plane[k] + to[r] * p.words[k] + w;
            }
        }
        __syncthreads();  // every row of the group is read before the first is written
#pragma unroll
        for (int j = 0; j < kpWords; ++j)
            if (dst[j]) *dst[j] = x[j];
    }
}

}  // namespace

cudaError_t launch_paged_keep(const CacheView &c, const PagedView &v, int64_t max_new, const int32_t *path, int64_t path_stride,
                              const int32_t *kept, int32_t *lens_out, cudaStream_t s)
{
    KeepParams p{};
    p.v = v;
    p.max_new = max_new;
    p.path = path;
    p.kept = kept;
    p.path_stride = path_stride;
    p.lens_out = lens_out;
    const void *plane[5] = {c.k_codes, c.k_scale, c.k_zero, c.v_codes, c.v_scale};
    const int words[5] = {c.d * c.kb / 32, c.d / 64, c.d / 64, c.d * c.vb / 32, c.d / 64};  // (head_dims are multiples of 64)
    for (int k = 0; k < 5; ++k) {
        p.plane[k] = static_cast<uint32_t *>(const_cast<void *>(plane[k]));
        p.words[k] = words[k];
        p.row_words += words[k];
    }
    p.H = c.H;
    return launch_dependent(paged_keep_kernel, dim3((unsigned)(v.seqs * c.H)), dim3(kpThreads), 0, s, p);
}

}  // namespace tq
