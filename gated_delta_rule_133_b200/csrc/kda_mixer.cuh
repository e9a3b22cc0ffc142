// Shared parts of the short convolution and the selective scan: element
// vectors, gate functions, packed-sequence lookup, internal launchers.
#pragma once

#include <type_traits>

#include "kda_common.cuh"

namespace kda {
namespace mixer {

// V consecutive elements as fp32 (V * sizeof(T) a multiple of 4; addresses
// aligned to the smaller of that and 16 bytes).
template <int V>
__device__ __forceinline__ void load_vec(const float* p, float (&x)[V])
{
    static_assert(V % 2 == 0, "vector width");
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(p + i);
            x[i] = a.x; x[i + 1] = a.y; x[i + 2] = a.z; x[i + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 a = *reinterpret_cast<const float2*>(p + i);
            x[i] = a.x; x[i + 1] = a.y;
        }
    }
}

__device__ __forceinline__ void unpack2(unsigned w, float& a, float& b)
{
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
}

template <int V>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&x)[V])
{
    static_assert(V % 2 == 0, "vector width");
    if constexpr (V % 8 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 8) {
            const uint4 a = *reinterpret_cast<const uint4*>(p + i);
            unpack2(a.x, x[i], x[i + 1]); unpack2(a.y, x[i + 2], x[i + 3]);
            unpack2(a.z, x[i + 4], x[i + 5]); unpack2(a.w, x[i + 6], x[i + 7]);
        }
    } else if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const uint2 a = *reinterpret_cast<const uint2*>(p + i);
            unpack2(a.x, x[i], x[i + 1]); unpack2(a.y, x[i + 2], x[i + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) unpack2(*reinterpret_cast<const unsigned*>(p + i), x[i], x[i + 1]);
    }
}

template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&x)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) *reinterpret_cast<float2*>(p + i) = make_float2(x[i], x[i + 1]);
    }
}

// Rounds to nearest even (the output type the caller asked for).
__device__ __forceinline__ unsigned pack2(float a, float b)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&r);
}

template <int V>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&x)[V])
{
    if constexpr (V % 8 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 8)
            *reinterpret_cast<uint4*>(p + i) = make_uint4(pack2(x[i], x[i + 1]), pack2(x[i + 2], x[i + 3]),
                                                          pack2(x[i + 4], x[i + 5]), pack2(x[i + 6], x[i + 7]));
    } else if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<uint2*>(p + i) = make_uint2(pack2(x[i], x[i + 1]), pack2(x[i + 2], x[i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) *reinterpret_cast<unsigned*>(p + i) = pack2(x[i], x[i + 1]);
    }
}

// 2^x (ex2.approx: at most 2 ulp; results below 2^-126 flush to zero, which
// for a decay factor is exact enough by far).
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x)   // 1 ulp
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(x) from one exponential and one reciprocal; 0 and 1 at the ends.
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + exp2_approx(-kLog2e * x)); }

__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// d silu(x) / dx = s + x s (1 - s), s = sigmoid(x)
__device__ __forceinline__ float silu_grad(float x)
{
    const float s = sigmoid(x);
    return fmaf(x * s, 1.f - s, s);
}

// Two fp32 values in one 64-bit register: the packed multiply-add does both in
// one issue slot.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack(float a, float b)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(f32x2 v, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ f32x2 silu2(float x, float y)
{
    const f32x2 v = pack(x, y);
    float a, b;
    unpack(mul2(v, pack(-kLog2e, -kLog2e)), a, b);
    unpack(add2(pack(exp2_approx(a), exp2_approx(b)), pack(1.f, 1.f)), a, b);
    return mul2(v, pack(rcp_approx(a), rcp_approx(b)));
}

// silu'(x) = s + x s (1 - s)
__device__ __forceinline__ f32x2 silu_grad2(float x, float y)
{
    const f32x2 v = pack(x, y), one = pack(1.f, 1.f);
    float a, b;
    unpack(mul2(v, pack(-kLog2e, -kLog2e)), a, b);
    unpack(add2(pack(exp2_approx(a), exp2_approx(b)), one), a, b);
    const f32x2 s = pack(rcp_approx(a), rcp_approx(b));
    return fma2(mul2(v, s), fma2(s, pack(-1.f, -1.f), one), s);
}

// Two or four consecutive elements as loaded, and as fp32.
template <typename T> struct Raw;
template <> struct Raw<float> { typedef float2 pair; typedef float4 quad; };
template <> struct Raw<__nv_bfloat16> { typedef unsigned pair; typedef uint2 quad; };
__device__ __forceinline__ float2 widen(float2 v) { return v; }
__device__ __forceinline__ float2 widen(unsigned v)
{
    float2 r;
    unpack2(v, r.x, r.y);
    return r;
}
__device__ __forceinline__ void widen(const float4& v, f32x2 (&x)[2])
{
    x[0] = pack(v.x, v.y);
    x[1] = pack(v.z, v.w);
}
__device__ __forceinline__ void widen(const uint2& v, f32x2 (&x)[2])
{
    const float2 a = widen(v.x), b = widen(v.y);
    x[0] = pack(a.x, a.y);
    x[1] = pack(b.x, b.y);
}

// The sequences of a call: nseq equal ones of T tokens (cu == nullptr), or
// packed ones given by cu over `tokens` tokens.
struct Seqs {
    const int32_t* cu;
    int n;
    int T;
    long long tokens;

    __device__ __forceinline__ long long begin(int i) const { return cu ? (long long)cu[i] : (long long)i * T; }
    // A sequence is used if its range lies in [0, tokens); an empty pair has no
    // tokens, a decreasing one none either (and is reported).
    __device__ __forceinline__ static bool inside(long long s, long long e, long long tokens)
    {
        return s >= 0 && e <= tokens;
    }
};

// Largest i in [0, n] with cu[i] <= t, or -1: a search by a whole warp, 32
// probes at a time (log32(n) dependent loads instead of log2(n)).
__device__ __forceinline__ int find_sequence(const Seqs& q, long long t)
{
    if (!q.cu) return (int)(t / q.T);
    const int lane = threadIdx.x & 31;
    int lo = 0, n = q.n + 1;   // entries [0, lo) are <= t, those from lo + n on are not
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int at = (lane + 1) * step - 1;
        const bool le = at < n && (long long)q.cu[lo + at] <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        lo += c * step;
        n = min(n - c * step, step - 1);
    }
    return lo - 1;
}

// Reports every packed sequence whose range leaves the token axis, and every
// decreasing pair of boundaries: the rows around it are found by a search that
// takes them in order (spread over the whole grid).
__device__ __forceinline__ void flag_bad_sequences(const Seqs& q)
{
    if (!q.cu) return;
    const long long nt = (long long)gridDim.x * gridDim.y * blockDim.x;
    long long i = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
    for (; i < q.n; i += nt) {
        const long long s = q.cu[i], e = q.cu[i + 1];
        if (e < s || (e > s && !Seqs::inside(s, e, q.tokens))) flag_bad_input();
    }
}

}  // namespace mixer

// Short causal depthwise convolution.  Arguments as the entry points of kda.h
// with the sequences given by (cu, nseq, T, tokens) as in chunk_fwd_simt.
struct ConvArgs {
    const void* x;
    long long ldx;
    const float* w;
    const float* bias;
    const int32_t* cu;
    int nseq, T;
    long long tokens;
    int D, W;
    bool silu;
    kda_dtype dtype;
};

cudaError_t conv_fwd(const ConvArgs& a, const void* s0, void* y, void* sT, kda_dtype o_dtype, cudaStream_t s);
cudaError_t conv_step(const ConvArgs& a, void* state, void* y, kda_dtype o_dtype, cudaStream_t s);
size_t conv_bwd_workspace(long long tokens, int D, int W);
cudaError_t conv_bwd(const ConvArgs& a, const void* s0, const float* gy, const float* gsT, float* gx, float* gw,
                     float* gb, float* gs0, void* ws, cudaStream_t s);

// Selective scan.
struct SsmArgs {
    const void *x, *dt, *b, *c, *z;
    long long ldx, lddt, ldb, ldc, ldz;
    const float *A, *skip, *dt_bias;
    const float* s0;
    const int32_t* cu;
    int nseq, T;
    long long tokens;
    int D, N, G;
    bool softplus;
    kda_dtype dtype;
};

cudaError_t ssm_fwd(const SsmArgs& a, void* y, float* sT, kda_dtype o_dtype, cudaStream_t s);
cudaError_t ssm_step(const SsmArgs& a, float* state, void* y, kda_dtype o_dtype, cudaStream_t s);

struct SsmGrads {
    const float *gy, *gsT;
    float *gx, *gdt, *gA, *gb, *gc, *gskip, *gz, *gdt_bias, *gs0;
};
size_t ssm_bwd_workspace(int nseq, int T, long long tokens, int D, int N, int G, bool varlen);
cudaError_t ssm_bwd(const SsmArgs& a, const SsmGrads& g, void* ws, cudaStream_t s);
size_t ssm_bwd_selftest_workspace();
cudaError_t ssm_bwd_selftest(long long limit_cycles, void* ws, cudaStream_t s);

}  // namespace kda
