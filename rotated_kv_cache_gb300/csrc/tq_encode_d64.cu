// tq_encode_d64.cu -- encode kernels instantiated for head_dim 64.
#include "tq_encode.cuh"

namespace tq {
cudaError_t launch_encode_d64(const CacheView &c, const uint16_t *k, const int64_t ks[3], const uint16_t *v,
                             const int64_t vs[3], int64_t t0, int64_t n, cudaStream_t s)
{
    return encode_d<64>(c, k, ks, v, vs, t0, n, s);
}

cudaError_t launch_paged_append_d64(const CacheView &c, const PagedView &v, const uint16_t *k, const int64_t ks[2],
                                    const uint16_t *vv, const int64_t vs[2], cudaStream_t s)
{
    return paged_encode_d<64>(c, v, k, ks, vv, vs, s);
}
}  // namespace tq
