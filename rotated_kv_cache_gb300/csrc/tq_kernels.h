// tq_kernels.h -- internal launch interface between the C ABI and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <atomic>
#include <functional>

namespace tq {

// Output i of SplitMix64 started at `seed` (Steele, Lea & Flood, OOPSLA 2014).
__host__ __device__ constexpr uint64_t splitmix64(uint64_t seed, uint64_t i)
{
    uint64_t z = seed + (i + 1u) * 0x9E3779B97F4A7C15ull;
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

// The value sign vector of one cache as bits (bit e % 32 of word e / 32 set
// when sign e is -1): sign e is -1 when the top bit of SplitMix64 output e of
// the cache's seed is set.  Built on the host once per call and passed to the
// kernels by value (head_dim <= 512).
struct SignBits {
    uint32_t w[16];
};

inline SignBits make_sign_bits(uint64_t seed, int d)
{
    SignBits s{};
    for (int e = 0; e < d; ++e)
        if (splitmix64(seed, (uint64_t)e) >> 63) s.w[e >> 5] |= 1u << (e & 31);
    return s;
}

__host__ __device__ __forceinline__ bool sign_negative(const SignBits &s, int e) { return (s.w[e >> 5] >> (e & 31)) & 1u; }

struct CacheView {
    int d, kb, vb, H, B;
    int64_t cap;
    uint8_t *k_codes;
    uint16_t *k_scale, *k_zero;
    uint8_t *v_codes;
    uint16_t *v_scale;
    SignBits signs;  // the cache's value sign vector
};

// Division by a run-time constant d >= 1 for dividends x < 2^31: q = (x * m) >> sh
// with sh = 31 + ceil(log2 d), m = ceil(2^sh / d) < 2^32 (Granlund & Montgomery,
// "Division by invariant integers using multiplication", PLDI 1994, Thm 4.2).
struct FastDiv {
    uint32_t m, sh;
};

inline FastDiv make_fastdiv(uint32_t d)
{
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    const uint32_t sh = 31 + l;
    return FastDiv{(uint32_t)(((1ull << sh) + d - 1) / d), sh};
}

// A page table and the ragged tokens of one call (tq_paged.cuh reads it).
struct PagedView {
    const int32_t *pages;   // [seqs][stride]
    const int32_t *lens;    // [seqs]
    const int32_t *starts;  // [seqs + 1]
    int64_t stride, max_len, total;
    int seqs, num_pages;
    uint32_t page;          // rows per page
    FastDiv div_page;
    uint32_t *err;
};

// The partials of a unit (sequence, kv-head, column block): slots first ..
// first + count - 1, written by the CTA of its first segment.
struct PagedUnit {
    int first, count;
};

// A paged attention call, for the split kernels (tq_paged.cuh).
struct PagedSplit {
    PagedView v;
    int64_t q_token, q_head;  // element strides of q
    PagedUnit *units;         // [seqs][H][blocks]: where a unit's partials are
    int64_t slots;            // partial slots of the workspace
    int blocks;               // column blocks of a sequence's kv-head, at most
    int64_t max_new;          // bound of a sequence's new tokens, which sized the workspace and picked the kernel
    int64_t wide;             // sequences with more new tokens than this are another kernel's
    const int32_t *spill;     // [seqs], or null: but for those marked here
    int nch, ru;              // chunks per stage, rows per chunk
};

__host__ __device__ constexpr int gcd_int(int a, int b) { return b == 0 ? a : gcd_int(b, a % b); }

// What the host knows of a paged attention call.
struct PagedBounds {
    int seqs;
    int64_t total, max_new, max_len, total_len;
    int64_t wide;  // more new tokens than this make a sequence wide (tq_paged_wide.cu); INT32_MAX: none is
};

// The chunks of a kernel with `stage` rows per stage: a chunk lies within a page.
inline void set_paged_chunks(PagedSplit &p, int stage, int page)
{
    p.ru = gcd_int(stage, page);
    p.nch = stage / p.ru;
}

// A split kernel's geometry for a paged batch: rows per stage, columns per
// block, CTAs of the launch.
struct PagedShape {
    int stage, block, ctas;
};

struct Tables {
    float centroids[256];
    float boundaries[255];
};

// Host-side tables (computed once per width; thread safe).
const Tables &codebook_tables(int vb);
float inv_sqrt_head_dim(int d);  // fl(1/sqrt(d)) rounded from binary64

uint32_t *device_error_word();  // per current device; nullptr on failure

// cuTensorMapEncodeTiled from the driver, or nullptr when unavailable.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

cudaError_t launch_encode(const CacheView &c, const uint16_t *k, const int64_t ks[3], const uint16_t *v,
                          const int64_t vs[3], int64_t t0, int64_t n, cudaStream_t s);

#define TQ_DECLARE_PER_D(D)                                                                                  \
    cudaError_t launch_encode_d##D(const CacheView &c, const uint16_t *k, const int64_t ks[3], const uint16_t *v, \
                                   const int64_t vs[3], int64_t t0, int64_t n, cudaStream_t s);                  \
    cudaError_t launch_decode_values_d##D(const CacheView &c, int64_t t0, int64_t n, bool f32, void *out,        \
                                          void *k_out, cudaStream_t s);                                          \
    cudaError_t launch_paged_append_d##D(const CacheView &c, const PagedView &v, const uint16_t *k,               \
                                         const int64_t ks[2], const uint16_t *vv, const int64_t vs[2],           \
                                         cudaStream_t s);                                                        \
    cudaError_t launch_paged_decode_values_d##D(const CacheView &c, const PagedView &v, bool f32, void *out,     \
                                                void *k_out, cudaStream_t s);
TQ_DECLARE_PER_D(64)
TQ_DECLARE_PER_D(128)
TQ_DECLARE_PER_D(256)
TQ_DECLARE_PER_D(512)
#undef TQ_DECLARE_PER_D

// Attention for every head_dim, bit pair and group size (the specialised
// kernel above covers d128, k8/k4, v3, groups of 8).
// M query rows per sequence (q and out [B][M][q_heads][d]); query row i sees
// cache rows [0, seq_len - M + i].  M = 1 is plain decode attention.
size_t attention_generic_workspace_bytes(const CacheView &c, int q_heads, int64_t m, int64_t seq_len);
cudaError_t launch_attention_generic(const CacheView &c, const uint16_t *q, int q_heads, int64_t m, int64_t seq_len,
                                     float scale, float *out, void *ws, size_t ws_bytes, cudaStream_t s);

// Merge split partials (o, m, l) laid out [B][H][hb][splits][cb][d] (+ [..][cb][2])
// into out [B][m][QH][d]: log-sum-exp over splits, then the inverse rotation.
cudaError_t launch_attention_combine_parts(int d, const float *part_o, const float *part_ml, float *out, int B, int H,
                                           int QH, int m, int hb, int cb, int splits, const SignBits &sg,
                                           cudaStream_t s);

// Multi-token attention on the tcgen05 tensor cores: head_dim 64 or 128 with
// at least 128 (query row, q-head) columns per kv-head.
bool attention_tc_applies(const CacheView &c, int q_heads, int64_t m);
size_t attention_tc_workspace_bytes(const CacheView &c, int q_heads, int64_t m, int64_t seq_len);
cudaError_t launch_attention_tc(const CacheView &c, const uint16_t *q, int q_heads, int64_t m, int64_t seq_len,
                                float scale, float *out, void *ws, size_t ws_bytes, cudaStream_t s);

// Deferred fetch, un-rotation and cache row copy / clear (src null: zeros).
cudaError_t launch_decode_rotated(const CacheView &c, int64_t t0, int64_t n, bool f32, void *out, cudaStream_t s);
cudaError_t launch_unrotate(int d, const SignBits &sg, bool in_f32, const void *x, int64_t rows, bool out_f32, void *out,
                            cudaStream_t s);
cudaError_t launch_copy_rows(const CacheView &dst, int64_t dst_t0, const CacheView *src, int64_t src_t0, int64_t n,
                             cudaStream_t s);

cudaError_t launch_decode(const CacheView &c, int64_t t0, int64_t n, bool f32, void *k_out, void *v_out,
                          cudaStream_t s);

bool attention_supported(int d, int kb, int vb, int group);
size_t attention_workspace_bytes(const CacheView &c, int q_heads, int64_t seq_len);
cudaError_t launch_attention(const CacheView &c, const uint16_t *q, int q_heads, int64_t seq_len, float scale,
                             float *out, void *ws, size_t ws_bytes, cudaStream_t s);

int num_sms();

constexpr int kMaxDevices = 64;
int current_device();  // in [0, kMaxDevices), or -1

// A kernel's shared-memory opt-in, a setting of the current device, and its
// resident CTAs per SM there (the same whichever thread asks first): once per
// device and shared-memory size.  A failure is not kept.
class KernelSetup {
public:
    // optin: dynamic shared memory to allow (0: the kernel needs no opt-in); ctas: as the query answers, 0 included
    template <typename Kernel>
    cudaError_t get(Kernel kern, int threads, size_t smem, size_t optin, int &ctas)
    {
        ctas = 0;
        const int dev = current_device();
        if (dev < 0) return cudaErrorInvalidDevice;
        std::atomic<uint64_t> &known = known_[dev];
        uint64_t k = known.load(std::memory_order_acquire);
        if (k == 0 || k >> 32 != (uint64_t)smem) {
            cudaError_t e = optin ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)optin) : cudaSuccess;
            if (e != cudaSuccess) return e;
            int n = 0;
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem);
            if (e != cudaSuccess) return e;
            k = (uint64_t)smem << 32 | (uint32_t)(n + 1);
            known.store(k, std::memory_order_release);
        }
        ctas = (int)(uint32_t)k - 1;
        return cudaSuccess;
    }

private:
    std::atomic<uint64_t> known_[kMaxDevices]{};  // smem << 32 | CTAs + 1; 0: not asked yet
};

// Paged caches: the view's pool is `c` (batch = pages, capacity = page size).
// K, V of ragged tokens -> their rows, and back ([total][H][d]; either output may be null).
cudaError_t launch_paged_append(const CacheView &c, const PagedView &v, const uint16_t *k, const int64_t ks[2],
                                const uint16_t *vv, const int64_t vs[2], cudaStream_t s);
cudaError_t launch_paged_decode(const CacheView &c, const PagedView &v, bool f32, void *k_out, void *v_out,
                                cudaStream_t s);
// Causal attention of ragged tokens q (strides {token, head}) -> out bf16 [total][QH][d];
// no sequence has more than max_new of them.  0 bytes: an occupancy query failed.
size_t paged_attention_workspace_bytes(const CacheView &c, const PagedBounds &b, int QH);
cudaError_t launch_paged_attention(const CacheView &c, const PagedView &v, const PagedBounds &b, const uint16_t *q,
                                   const int64_t qs[2], int QH, float scale, uint16_t *out, void *ws, size_t ws_bytes,
                                   cudaStream_t s);
// ... of the wide sequences, by tcgen05 (head_dim 64 and 128).
bool paged_wide_applies(const CacheView &c);
size_t paged_wide_workspace_bytes(const CacheView &c, const PagedBounds &b, int QH);
// The workspace holds tiles for a bounded number of rows: whether the bounds allow more, and the
// sequences whose chunks found no room, which the split kernels take (null: there are none).
bool paged_wide_spills(const CacheView &c, const PagedBounds &b, int QH);
int32_t *paged_wide_spill(const CacheView &c, const PagedBounds &b, int QH, void *ws);
// `split` launches the other sequences' split kernel, behind the expansion of the rows.
cudaError_t launch_paged_wide(const CacheView &c, const PagedSplit &pg, const PagedBounds &b, const uint16_t *q, int QH,
                              float scale, uint16_t *out, void *ws, cudaStream_t s,
                              const std::function<cudaError_t()> &split);

// Allocation-free decode attention: partials in a library-owned device array.
size_t noalloc_scratch_bytes();
bool noalloc_fits(const CacheView &c, int q_heads);
cudaError_t launch_attention_noalloc(const CacheView &c, const uint16_t *q, int q_heads, int64_t seq_len, float scale,
                                     float *out, cudaStream_t s);

}  // namespace tq
