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
// latency for few.  A CTA takes a token (or some of its heads), or four of them: a
// position's angles are worked out once for all heads, while their rows are on the way.
//
// 8191 tokens of 40 heads out of 48, head_dim 128, bf16: 33.0 us interleaved, half the
// head (5.1 TB/s, 0.75 of a copy; 35.6 with a token a block), 36.2 in halves, all of it
// (halves with 2 rows of a thread under way 39, interleaved with 2 of 4 33.2); 64
// tokens of 72 heads 2.9 us, of which a launch is 2.  rot 100: 70 us, bound by the
// instructions that take single elements from shared memory.
#include "tq_common.cuh"
#include "tq_kernels.h"

namespace tq {
namespace {

constexpr int roThreads = 256;
constexpr int roTokens = 4;      // of a block, where there are many
constexpr int kManyTokens = 16;  // per SM

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
// and goes from row (token, head) to row, U of them under way.  Blocks of several
// tokens work out all their angles side by side, while their first rows are on
// the way (a chain of a dozen 64-bit operations, 500 cycles).
template <typename T, bool INTER, int TK>
__global__ void __launch_bounds__(roThreads) rotary_kernel(const __grid_constant__ RotaryParams p)
{
    using V = RotaryVec<T>;
    constexpr int E = V::E, NA = INTER ? E / 2 : E, U = INTER ? 4 : 1;  // angles of an access, rows under way
    __shared__ __align__(16) float2 cs[TK][256];
    __shared__ int pos[TK];
    pdl_wait_primary();
    pdl_allow_dependents();
    const RotaryCall &r = p.r;
    const int tid = threadIdx.x, hpp = roThreads / p.chunks, chunk = tid % p.chunks, hl = tid / p.chunks;
    const int64_t t0 = (int64_t)blockIdx.x * TK;
    const int tokens = (int)imin64(TK, r.tokens - t0), half = r.rot / 2;
    if (tid < tokens) pos[tid] = r.pos[t0 + tid];
    const int h0 = blockIdx.y * p.per_block, h1 = h0 + p.per_block < p.heads ? h0 + p.per_block : p.heads;
    const bool turns = chunk < p.turn;
    const int at = turns ? chunk * E : r.rot + (chunk - p.turn) * E;  // first element
    // the thread's next row
    int tk = 0, h = h0 + hl;
    auto settle = [&] {
        while (h >= h1 && tk < tokens) {
            h -= h1 - h0;
            ++tk;
        }
    };
    settle();
    if (hl >= hpp) tk = tokens;  // (threads left over)
    uint4 a[U], b[U];
    T *out[U];
    int of[U];
    auto load = [&] {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            out[u] = nullptr;
            of[u] = tk;
            if (tk >= tokens) continue;
            const T *x;
            rotary_head<T>(r, t0 + tk, h, x, out[u]);
            h += hpp;
            settle();
            if (!turns && out[u] == x) {  // in place: nothing to copy
                out[u] = nullptr;
                continue;
            }
            a[u] = *reinterpret_cast<const uint4 *>(x + at);
            if (!INTER && turns) b[u] = *reinterpret_cast<const uint4 *>(x + at + half);
        }
    };
    load();
    __syncthreads();
    for (int i = tid; i < tokens * half; i += roThreads) {
        const int k = i / half, j = i - k * half;
        cs[k][j] = rotary_angle(r, pos[k], j);
    }
    __syncthreads();
    for (;;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!out[u] || pos[of[u]] < 0) continue;  // (below 0: of no sequence, left as it was)
            if (turns) {
                float2 c[NA];
                const float4 *src = reinterpret_cast<const float4 *>(&cs[of[u]][INTER ? at / 2 : at]);
#pragma unroll
                for (int i = 0; i < NA / 2; ++i) {
                    const float4 v = src[i];
                    c[2 * i] = make_float2(v.x, v.y);
                    c[2 * i + 1] = make_float2(v.z, v.w);
                }
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
                    *reinterpret_cast<uint4 *>(out[u] + at + half) = V::put(w);
                }
            }
            *reinterpret_cast<uint4 *>(out[u] + at) = a[u];
        }
        if (tk >= tokens) break;
        load();
    }
}

// Any even rot: whole rows pass through shared memory, and a thread takes its
// elements' partners from there.  Element e of a row (and of the angles) stands at
// (e % E) PS + e / E: lanes that read elements E apart, whatever offset they have in
// common, read neighbouring places (as the row stands, 4 to 8 lanes would share a
// bank: 8191 tokens of 40 heads, rot 100 of 128, 71 us so).
template <typename T, bool INTER>
__global__ void __launch_bounds__(roThreads) rotary_any_kernel(const __grid_constant__ RotaryParams p)
{
    using V = RotaryVec<T>;
    constexpr int E = V::E, U = 4;  // rows of a thread under way
    constexpr int CS = 256 / E + 1;
    __shared__ float2 cs[E * CS];
    __shared__ T rows[U][(roThreads + 64) * E];
    pdl_wait_primary();
    pdl_allow_dependents();
    const RotaryCall &r = p.r;
    const int64_t t = blockIdx.x;
    const int pos = r.pos[t];
    const int tid = threadIdx.x, per = r.d / E, hpp = roThreads / per, chunk = tid % per, hl = tid / per;
    const int h0 = blockIdx.y * p.per_block, h1 = h0 + p.per_block < p.heads ? h0 + p.per_block : p.heads, half = r.rot / 2;
    const int PS = per + 2, row0 = hl * E * PS;
    bool angles = false;
    for (int h = h0; h < h1; h += U * hpp) {
        uint4 a[U];
        T *out[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hu = h + u * hpp + hl;
            const T *x;
            out[u] = nullptr;
            a[u] = make_uint4(0u, 0u, 0u, 0u);
            if (hu < h1) {
                rotary_head<T>(r, t, hu, x, out[u]);
                a[u] = *reinterpret_cast<const uint4 *>(x + chunk * E);
            }
        }
        if (pos < 0) return;  // of no sequence: left as it was
        if (!angles)
            for (int i = tid; i < half; i += roThreads) cs[i % E * CS + i / E] = rotary_angle(r, pos, i);
        angles = true;
        __syncthreads();  // the previous rows have been used
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float y[E];
            V::get(a[u], y);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if constexpr (sizeof(T) == 2) rows[u][row0 + i * PS + chunk] = (T)(__float_as_uint(y[i]) >> 16);
                else rows[u][row0 + i * PS + chunk] = y[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!out[u]) continue;
            float y[E];
            V::get(a[u], y);
            auto value = [&](int e) {  // of the row
                const T x = rows[u][row0 + e % E * PS + e / E];
                if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)x << 16);
                else return x;
            };
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int e = chunk * E + i;
                if (e >= r.rot) continue;
                const bool upper = INTER ? e & 1 : e >= half;
                const int k = INTER ? e >> 1 : upper ? e - half : e;
                const float2 c = cs[k % E * CS + k / E];
                const float o = value(INTER ? e ^ 1 : upper ? e - half : e + half);
                y[i] = upper ? o * c.y + y[i] * c.x : y[i] * c.x - o * c.y;
            }
            *reinterpret_cast<uint4 *>(out[u] + chunk * E) = V::put(y);
        }
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
    const unsigned by = (unsigned)((p.heads + p.per_block - 1) / p.per_block);
    if (!whole)
        return launch_dependent(r.interleaved ? rotary_any_kernel<T, true> : rotary_any_kernel<T, false>, dim3((unsigned)r.tokens, by),
                                dim3(roThreads), 0, s, p);
    const bool many = r.tokens >= kManyTokens * (int64_t)num_sms();
    const auto kern = many ? (r.interleaved ? rotary_kernel<T, true, roTokens> : rotary_kernel<T, false, roTokens>)
                           : (r.interleaved ? rotary_kernel<T, true, 1> : rotary_kernel<T, false, 1>);
    const unsigned bx = (unsigned)(many ? (r.tokens + roTokens - 1) / roTokens : r.tokens);
    return launch_dependent(kern, dim3(bx, by), dim3(roThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_rotary(const RotaryCall &r, cudaStream_t s)
{
    RotaryParams p{};
    p.r = r;
    return r.f32 ? rotary_run<float>(p, s) : rotary_run<uint16_t>(p, s);
}

}  // namespace tq
