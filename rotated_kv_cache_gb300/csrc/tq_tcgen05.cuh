// tq_tcgen05.cuh -- fifth-generation tensor core helpers (sm_103a): descriptors,
// MMA, tensor-memory loads and stores, operand tile layouts, and the
// dequantisation of packed codes into them.
#pragma once
#include "tq_common.cuh"

namespace tq {
namespace {

// ---------------------------------------------------------------- tcgen05 / descriptor helpers
// Shared-memory matrix descriptor: 128-byte swizzle, descriptor version 1.
// lbo / sbo in bytes (K-major tiles: sbo = 1024 between 8-row groups, lbo
// unused; MN-major tiles: lbo between 64-element blocks of the M/N extent,
// sbo between 8-row groups of K).
__host__ __device__ constexpr uint64_t tc_desc_const(uint32_t lbo, uint32_t sbo)  // all but the address
{
    return (uint64_t)((lbo >> 4) & 0x3FFF) << 16 | (uint64_t)((sbo >> 4) & 0x3FFF) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ uint64_t tc_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((saddr >> 4) & 0x3FFF) | tc_desc_const(lbo, sbo);
}

// Instruction descriptor, kind::f16: f16 A and B, f32 accumulator, M x N,
// A K-major, B K-major (b_mn = 0) or MN-major (b_mn = 1).
__host__ __device__ constexpr uint32_t tc_idesc(int M, int N, int b_mn)
{
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

// A operand in tensor memory (M = 128 lanes, two f16 per 32-bit column, the
// even k in the low half), B from shared memory
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}

__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// The same, called by a whole warp with warp-uniform operands; the lane that
// tc_elect() chose (1 there, 0 elsewhere) issues.
__device__ __forceinline__ uint32_t tc_elect()
{
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e;
}

__device__ __forceinline__ void tc_mma_elected(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader));
}

__device__ __forceinline__ void tc_mma_ts_elected(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                                  uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc), "r"(leader));
}

__device__ __forceinline__ void tc_commit_elected(uint32_t leader, uint32_t bar)
{
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
        "r"(leader)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive 32-bit columns of this thread's tensor-memory lane
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// ... 16 of them
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// ... four of them, and their store
__device__ __forceinline__ void tc_ld4(uint32_t taddr, uint32_t (&r)[4])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
}

__device__ __forceinline__ void tc_st4(uint32_t taddr, const uint32_t (&r)[4])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// Keeps what uses loaded registers behind the wait for the load before it.
template <int N>
__device__ __forceinline__ void tc_pin(uint32_t (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// Barrier `id` of n threads; true when all of them say so.
__device__ __forceinline__ bool named_and(int id, int n, bool ok)
{
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n barrier.cta.red.and.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float tc_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t tc_pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t tc_lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// Byte offset of element (r, k) in a K-major tile of R rows (64-element K blocks
// of R * 128 bytes; 16-byte chunks XOR-swizzled by r % 8).
__host__ __device__ constexpr uint32_t kmaj_off(int R, int r, int k)
{
    return (uint32_t)((k / 64) * (R * 128) + (r / 8) * 1024 + (r % 8) * 128 + ((((k % 64) / 8) ^ (r % 8)) * 16) +
                      (k % 8) * 2);
}

// Byte offset of element (k = cache row, n = dim) of the MN-major value tile
// (N dims: 64-dim blocks 1024 bytes apart inside each group of 8 rows).
template <int N>
__host__ __device__ constexpr uint32_t mnmaj_off(int k, int n)
{
    return (uint32_t)((k / 8) * (N / 64) * 1024 + (n / 64) * 1024 + (k % 8) * 128 + ((((n % 64) / 8) ^ (k % 8)) * 16) +
                      (n % 8) * 2);
}

// power-of-two exponent e with bound * 2^e in [2^13, 2^14) (0 if the bound is
// zero or not finite), clamped to [-100, 100]
__device__ __forceinline__ int tile_exponent(float bound)
{
    if (!(bound > 0.0f) || !(bound < INFINITY)) return 0;
    const int e = 13 - (((int)(__float_as_uint(bound) >> 23) & 0xFF) - 127);
    return e < -100 ? -100 : (e > 100 ? 100 : e);
}

// ---------------------------------------------------------------- dequantisation of one 8-element item
// Keys: 8 codes from the 64-bit window (w1:w0) >> sh; kv = (code + zero) * scale * 2^e.
template <int KB>
__device__ __forceinline__ void key_values(uint32_t w0, uint32_t w1, int sh, int kb, float sc, float cz, float (&kv)[8])
{
    uint32_t m[8];
    if constexpr (KB == 8) {
        const uint32_t a = w0 ^ 0x80808080u, b = w1 ^ 0x80808080u;  // int8 -> code + 128
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = __byte_perm(a, 0x4B000000u, 0x7440 + i);
            m[4 + i] = __byte_perm(b, 0x4B000000u, 0x7440 + i);
        }
    } else if constexpr (KB == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = ((w0 >> (4 * i)) & 0xFu) | 0x4B000000u;
    } else {
        const uint64_t v = ((uint64_t)w1 << 32 | w0) >> sh;
        const uint32_t mask = (1u << kb) - 1u, flip = kb == 8 ? 0x80u : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = ((((uint32_t)(v >> (i * kb))) & mask) ^ flip) | 0x4B000000u;
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 f = __fmul2_rn(fsub2(make_float2(__uint_as_float(m[i]), __uint_as_float(m[i + 1])),
                                          make_float2(cz, cz)),
                                    make_float2(sc, sc));
        kv[i] = f.x;
        kv[i + 1] = f.y;
    }
}

// Values: 8 codes from (w1:w0) >> sh; vv = centroid * rms * 2^ev.
template <int VB>
__device__ __forceinline__ void value_values(uint32_t w0, uint32_t w1, int sh, int vb, float sv, uint32_t lut,
                                             float (&vv)[8])
{
    uint32_t c[8];
    if constexpr (VB == 3) {
        const uint32_t x = __funnelshift_r(w0, w1, sh);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = (x >> (3 * i)) & 7u;
    } else {
        const uint64_t v = ((uint64_t)w1 << 32 | w0) >> sh;
        const uint32_t mask = (1u << vb) - 1u;
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = (uint32_t)(v >> (i * vb)) & mask;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) vv[i] = __uint_as_float(tc_lds32(lut + 4 * c[i])) * sv;
}

}  // namespace
}  // namespace tq
