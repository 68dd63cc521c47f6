// tq_decode_d64.cu -- value fetch kernels instantiated for head_dim 64.
#include "tq_decode.cuh"

namespace tq {
cudaError_t launch_decode_values_d64(const CacheView &c, int64_t t0, int64_t n, bool f32, void *out, void *k_out,
                                     cudaStream_t s)
{
    return f32 ? value_dispatch_vb<64, true>(c, t0, n, out, k_out, s)
               : value_dispatch_vb<64, false>(c, t0, n, out, k_out, s);
}

cudaError_t launch_paged_decode_values_d64(const CacheView &c, const PagedView &v, bool f32, void *out, void *k_out,
                                           cudaStream_t s)
{
    return f32 ? value_dispatch_vb<64, true, true>(c, 0, v.total, out, k_out, s, &v)
               : value_dispatch_vb<64, false, true>(c, 0, v.total, out, k_out, s, &v);
}
}  // namespace tq
