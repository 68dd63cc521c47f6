// tq_paged_split.cuh -- paged launches of the specialised split kernel
// (tq_attention.cuh) for one head_dim.
//
// A batch with at most one new token a sequence takes a kernel of its own (MODE
// 1): no limits per column to compare with (64 sequences of 2048 rows: 63.0 us,
// through the kernel for more, MODE 2, 65.5; 16 of 8192 rows at head_dim 256:
// 101.1 and 106.7).
#pragma once
#include "tq_attention.cuh"

namespace tq {
namespace {

// A block takes two column blocks of kG where a kv-head has more than kG
// columns and the registers allow it (head_dims up to 128), as in the
// contiguous launches: 16 sequences of 4096 rows with 16 columns take 50.0 us
// with two and 62.6 with one, 64 sequences of 2048 rows with 8 columns 63.0 us
// with one and 80.0 with two.
template <int D>
constexpr int paged_split_nbc(int64_t cols) { return D <= 128 && cols > kG ? 2 : 1; }

// f(kernel geometry) for the pool's widths and the block's columns.
template <int D, int NBC, typename F>
auto paged_split_widths(const CacheView &c, F &&f)
{
    using std::integral_constant;
    if (c.kb == 8)
        return c.vb == 2 ? f(integral_constant<int, 8>{}, integral_constant<int, 2>{})
               : c.vb == 4 ? f(integral_constant<int, 8>{}, integral_constant<int, 4>{})
                           : f(integral_constant<int, 8>{}, integral_constant<int, 3>{});
    return c.vb == 2 ? f(integral_constant<int, 4>{}, integral_constant<int, 2>{})
           : c.vb == 4 ? f(integral_constant<int, 4>{}, integral_constant<int, 4>{})
                       : f(integral_constant<int, 4>{}, integral_constant<int, 3>{});
}

template <int D, int NBC, int MODE>
PagedShape paged_split_shape_n(const CacheView &c)
{
    return paged_split_widths<D, NBC>(c, [](auto kb, auto vb) {
        return PagedShape{AGeo<kb.value, D, vb.value, NBC>::ST, kG * NBC,
                          ctas_per_sm_for<kb.value, D, vb.value, NBC, MODE>() * num_sms()};
    });
}

template <int D, int NBC, int MODE>
cudaError_t paged_split_run(const CacheView &c, const PagedSplit &pg, const PagedShape &sh, const uint16_t *q, int QH,
                            float scale, float *part_o, float *part_ml, cudaStream_t s)
{
    return paged_split_widths<D, NBC>(c, [&](auto kb, auto vb) {
        using A = AGeo<kb.value, D, vb.value, NBC>;
        AttnParams p{};
        if (!attn_params<kb.value, vb.value>(c, q, QH, scale, p)) return cudaErrorInvalidDevice;
        p.part_o = part_o;
        p.part_ml = part_ml;
        p.pg = pg;
        set_paged_chunks(p.pg, A::ST, (int)c.cap);
        CUtensorMap map;
        if (!split_key_map<A>(c, p.pg.ru, &map)) return cudaErrorInvalidValue;
        return launch_dependent(attn_split_kernel<kb.value, D, vb.value, NBC, MODE>, dim3((unsigned)sh.ctas), dim3(kThreads),
                                (size_t)A::SMEM, s, map, p);
    });
}

}  // namespace
}  // namespace tq

// The entry points of one head_dim's translation unit for MODE 1 or 2 (NAME d<head_dim>_one / _any).
#define TQ_PAGED_SPLIT_ENTRIES(D, MODE, NAME)                                                                          \
    namespace tq {                                                                                                     \
    PagedShape paged_split_shape_##NAME(const CacheView &c, int64_t cols)                                              \
    {                                                                                                                  \
        if constexpr (D <= 128)                                                                                        \
            if (paged_split_nbc<D>(cols) == 2) return paged_split_shape_n<D, 2, MODE>(c);                              \
        return paged_split_shape_n<D, 1, MODE>(c);                                                                     \
    }                                                                                                                  \
    cudaError_t launch_paged_split_##NAME(const CacheView &c, const PagedSplit &pg, const PagedShape &sh,              \
                                          const uint16_t *q, int QH, float scale, float *part_o, float *part_ml,       \
                                          cudaStream_t s)                                                              \
    {                                                                                                                  \
        if constexpr (D <= 128)                                                                                        \
            if (sh.block == 2 * kG) return paged_split_run<D, 2, MODE>(c, pg, sh, q, QH, scale, part_o, part_ml, s);   \
        return paged_split_run<D, 1, MODE>(c, pg, sh, q, QH, scale, part_o, part_ml, s);                               \
    }                                                                                                                  \
    }
