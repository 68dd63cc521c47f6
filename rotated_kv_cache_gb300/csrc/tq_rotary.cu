// tq_rotary.cu -- rotary positions of ragged queries and keys.
//
//   (a, b) -> m (a cos t - b sin t, a sin t + b cos t),   t = position * frequency
//
// for each pair of the first `rot` elements of a head: (2 i, 2 i + 1)
// interleaved, (i, i + rot / 2) in halves; the elements behind are copied.  A
// position times a frequency is taken in 64 bits and reduced to a turn there (a
// position of 10^6 in 32 bits would lose the angle's last four digits), the
// sine and cosine of what is left in 32, corrected by the part that 32 bits of
// it leave out; products and sums are 32-bit, and the result is rounded once.
//
// Every element is read and written once: bound by memory for many tokens, by
// latency for few.  A CTA takes a token (or some of its heads): a position's
// angles are worked out once for all of them, while their rows are on the way.
#include "tq_common.cuh"
#include "tq_kernels.h"

namespace tq {
namespace {

constexpr int roThreads = 256;

struct RotaryParams {
    RotaryCall r;
    int heads, per_block;  // heads of both tensors, of a block
    int turn, chunks;      // 16-byte accesses (pairs of them for halves) that turn; with those that copy
};

// cos and sin of angle i of a position, times the scale
__device__ __forceinline__ float2 rotary_angle(const RotaryCall &r, int pos, int i)
{
    const double t = (double)pos * r.freqs[i];
    const double k = rint(t * 0.15915494309189535);  // 1 / (2 pi)
    double y = fma(-k, 6.283185307179586, t);        // 2 pi in two parts
    y = fma(-k, 2.4492935982947064e-16, y) * 0.3183098861837907;  // in half turns
    const float h = (float)y, e = (float)((y - (double)h) * 3.141592653589793);
    float sn, cs;
    sincospif(h, &sn, &cs);
    return make_float2((cs - sn * e) * r.scale, (sn + cs * e) * r.scale);
}

template <typename T>
struct RotaryVec;  // a 16-byte access as floats

template <>
struct RotaryVec<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void get(const uint4 &v, float (&x)[4])
    {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

template <>
struct RotaryVec<uint16_t> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void get(const uint4 &v, float (&x)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8])
    {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
};

// A head of either tensor: its rows of the token in and out.
template <typename T>
__device__ __forceinline__ void rotary_head(const RotaryCall &r, int64_t t, int h, const T *&x, T *&out)
{
    const bool second = h >= r.t[0].heads;
    const RotaryTensor &a = r.t[second];
    const int hh = second ? h - r.t[0].heads : h;
    x = static_cast<const T *>(a.x) + t * a.x_token + hh * a.x_head;
    out = static_cast<T *>(a.out) + t * a.out_token + hh * a.out_head;
}

// Turned parts of whole 16-byte accesses: a thread keeps its place in the head
// and goes from head to head, so its cosines and sines stay in registers.
template <typename T, bool INTER>
__global__ void __launch_bounds__(roThreads) rotary_kernel(const __grid_constant__ RotaryParams p)
{
    using V = RotaryVec<T>;
    constexpr int E = V::E, NA = INTER ? E / 2 : E, U = 4;  // angles of a thread, heads under way
    __shared__ float2 cs[256];
    pdl_wait_primary();
    pdl_allow_dependents();
    const RotaryCall &r = p.r;
    const int64_t t = blockIdx.x;
    const int pos = r.pos[t];
    if (pos < 0) return;  // of no sequence: left as it was
    const int tid = threadIdx.x, hpp = roThreads / p.chunks, chunk = tid % p.chunks, hl = tid / p.chunks;
    const int h0 = blockIdx.y * p.per_block, h1 = h0 + p.per_block < p.heads ? h0 + p.per_block : p.heads;
    const bool turns = chunk < p.turn;
    const int at = turns ? chunk * E : r.rot + (chunk - p.turn) * E;  // first element
    uint4 a[U], b[U];
    T *out[U];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hu = h + u * hpp;
            out[u] = nullptr;
            if (hu >= h1 || hl >= hpp) continue;
            const T *x;
            rotary_head<T>(r, t, hu, x, out[u]);
            if (!turns && out[u] == x) {  // in place: nothing to copy
                out[u] = nullptr;
                continue;
            }
            a[u] = *reinterpret_cast<const uint4 *>(x + at);
            if (!INTER && turns) b[u] = *reinterpret_cast<const uint4 *>(x + at + r.rot / 2);
        }
    };
    load(h0 + hl);
    for (int i = tid; i < r.rot / 2; i += roThreads) cs[i] = rotary_angle(r, pos, i);
    __syncthreads();
    float2 c[NA];
    if (turns)
#pragma unroll
        for (int i = 0; i < NA; ++i) c[i] = cs[(INTER ? at / 2 : at) + i];
    for (int h = h0 + hl; h < h1; h += U * hpp) {
        if (h > h0 + hl) load(h);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!out[u]) continue;
            if (turns) {
                float x[E], y[E];
                V::get(a[u], x);
                if constexpr (INTER) {
#pragma unroll
                    for (int i = 0; i < NA; ++i) {
                        y[2 * i] = x[2 * i] * c[i].x - x[2 * i + 1] * c[i].y;
                        y[2 * i + 1] = x[2 * i] * c[i].y + x[2 * i + 1] * c[i].x;
                    }
                    a[u] = V::put(y);
                } else {
                    float z[E], w[E];
                    V::get(b[u], z);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        y[i] = x[i] * c[i].x - z[i] * c[i].y;
                        w[i] = x[i] * c[i].y + z[i] * c[i].x;
                    }
                    a[u] = V::put(y);
                    *reinterpret_cast<uint4 *>(out[u] + at + r.rot / 2) = V::put(w);
                }
            }
            *reinterpret_cast<uint4 *>(out[u] + at) = a[u];
        }
    }
}

// Any even rot: whole rows pass through shared memory in 16-byte accesses, and
// a thread takes its elements' partners from there.
template <typename T, bool INTER>
__global__ void __launch_bounds__(roThreads) rotary_any_kernel(const __grid_constant__ RotaryParams p)
{
    using V = RotaryVec<T>;
    constexpr int E = V::E;
    __shared__ float2 cs[256];
    __shared__ __align__(16) T rows[roThreads * E];
    pdl_wait_primary();
    pdl_allow_dependents();
    const RotaryCall &r = p.r;
    const int64_t t = blockIdx.x;
    const int pos = r.pos[t];
    if (pos < 0) return;
    const int tid = threadIdx.x, per = r.d / E, hpp = roThreads / per, chunk = tid % per, hl = tid / per;
    const int h0 = blockIdx.y * p.per_block, h1 = h0 + p.per_block < p.heads ? h0 + p.per_block : p.heads, half = r.rot / 2;
    for (int i = tid; i < half; i += roThreads) cs[i] = rotary_angle(r, pos, i);
    for (int h = h0; h < h1; h += hpp) {
        const bool live = h + hl < h1;
        const T *x = nullptr;
        T *out = nullptr;
        if (live) rotary_head<T>(r, t, h + hl, x, out);
        uint4 a = make_uint4(0u, 0u, 0u, 0u);
        if (live) a = *reinterpret_cast<const uint4 *>(x + chunk * E);
        __syncthreads();  // the previous rows have been used (and the angles are there)
        reinterpret_cast<uint4 *>(rows)[tid] = a;
        __syncthreads();
        if (!live) continue;
        float y[E];
        V::get(a, y);
        auto value = [&](int e) {  // of the row
            if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)rows[hl * r.d + e] << 16);
            else return rows[hl * r.d + e];
        };
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int e = chunk * E + i;
            if (e >= r.rot) continue;
            const bool upper = INTER ? e & 1 : e >= half;
            const float2 c = cs[INTER ? e >> 1 : upper ? e - half : e];
            const float o = value(INTER ? e ^ 1 : upper ? e - half : e + half);
            y[i] = upper ? o * c.y + y[i] * c.x : y[i] * c.x - o * c.y;
        }
        *reinterpret_cast<uint4 *>(out + chunk * E) = V::put(y);
    }
}

template <typename T>
cudaError_t rotary_run(RotaryParams &p, cudaStream_t s)
{
    constexpr int E = RotaryVec<T>::E;
    RotaryCall &r = p.r;
    const bool whole = r.interleaved ? r.rot % E == 0 : r.rot / 2 % E == 0;
    p.heads = r.t[0].heads + r.t[1].heads;
    bool copies = false;
    for (const RotaryTensor &t : r.t) copies |= t.heads > 0 && t.x != t.out;
    p.turn = r.interleaved ? r.rot / E : r.rot / 2 / E;
    p.chunks = whole ? p.turn + (copies ? (r.d - r.rot) / E : 0) : r.d / E;
    // few tokens: the heads of one over several blocks
    const int passes = (p.heads + roThreads / p.chunks - 1) / (roThreads / p.chunks);
    const int64_t want = (4 * (int64_t)num_sms() + r.tokens - 1) / r.tokens;
    const int blocks = (int)(want < passes ? want : passes);
    p.per_block = (p.heads + blocks - 1) / blocks;
    const dim3 grid((unsigned)r.tokens, (unsigned)((p.heads + p.per_block - 1) / p.per_block));
    const auto kern = whole ? (r.interleaved ? rotary_kernel<T, true> : rotary_kernel<T, false>)
                            : (r.interleaved ? rotary_any_kernel<T, true> : rotary_any_kernel<T, false>);
    return launch_dependent(kern, grid, dim3(roThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_rotary(const RotaryCall &r, cudaStream_t s)
{
    RotaryParams p{};
    p.r = r;
    return r.f32 ? rotary_run<float>(p, s) : rotary_run<uint16_t>(p, s);
}

}  // namespace tq
