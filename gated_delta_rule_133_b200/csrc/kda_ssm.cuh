// Device parts shared by the selective scan's forward and backward kernels.
#pragma once

#include "kda_mixer.cuh"

namespace kda {
namespace mixer {

// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// softplus(v) = max(v, 0) + log(1 + e), e = e^-|v|, of two values, to fp32 accuracy
// for every v.  e: 2^(-|v| log2 e) with the rounding error of the exponent put back
// (log2 e in two parts, as Cody and Waite reduce an argument).  log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3, without
// the cancellation of 1 + e; atanh(s) / s is a degree-4 polynomial in s^2 (largest
// relative error 7.8e-9, at s = 0.103, fitted by reweighted least squares).
__device__ __forceinline__ f32x2 softplus2(float v0, float v1)
{
    auto two = [](float x) { return pack(x, x); };
    // below e^-100 the result is zero; without the bound the rounding error of an
    // infinite exponent (a token masked by the lowest value or -inf) would be NaN
    const f32x2 t = pack(max_nan(-fabsf(v0), -100.f), max_nan(-fabsf(v1), -100.f));
    const f32x2 nhi = mul2(t, two(-kLog2e));
    const f32x2 lo = fma2(t, two(1.9259629e-8f), fma2(t, two(kLog2e), nhi));
    float h0, h1;
    unpack(nhi, h0, h1);
    f32x2 e = pack(exp2_approx(-h0), exp2_approx(-h1));
    e = fma2(mul2(e, lo), two(0.69314718f), e);
    unpack(fma2(e, two(1.f), two(2.f)), h0, h1);
    const f32x2 s = mul2(e, pack(rcp_approx(h0), rcp_approx(h1))), q = mul2(s, s);
    f32x2 p = fma2(q, two(0.14089163f), two(0.13980302f));
    p = fma2(q, p, two(0.20012455f));
    p = fma2(q, p, two(0.33333158f));
    p = fma2(q, p, two(1.f));
    return fma2(mul2(s, two(2.f)), p, pack(fmaxf(v0, 0.f), fmaxf(v1, 0.f)));
}
__device__ __forceinline__ float softplus(float v)
{
    float r, unused;
    unpack(softplus2(v, v), r, unused);
    return r;
}

// A, kept from infinity: a rate of -inf would make 0 * inf of a step size of zero (a
// masked token, or one that fills up a turn behind the last token), and a sum of
// w A beyond the largest number inf * 0 of its gradient.  Below -1e30 every step
// size above 1e-28 forgets everything.
__device__ __forceinline__ float bounded_decay(float a) { return max_nan(a, -1e30f); }

// Decays 2^(Delta A2) of two states.  ex2.approx is below the true value by 0.26 to
// 0.44 2^-24 on average over any factor of two to three of exponents in [-0.25, -0.003],
// which hundreds of slow decays in a row would add up; the exponent is moved by that
// much, at no cost in the multiply, which leaves -0.05 to +0.11 there.  Closer to zero
// ex2.approx is only 0.1 low, and the move leaves 0.2 to 0.3 2^-24 above.
constexpr float kDecayShift = 3.4e-8f;   // 0.4 2^-24 log2 e
__device__ __forceinline__ f32x2 decay2(f32x2 delta, f32x2 A2)
{
    float x, y;
    unpack(fma2(delta, A2, pack(kDecayShift, kDecayShift)), x, y);
    return pack(exp2_approx(x), exp2_approx(y));
}

// Sums p[j] over LANES lanes that lie STRIDE apart, for V >= LANES values at
// once: the lane with index i = (lane / STRIDE) % LANES gets the sums of values
// i V / LANES and on, in p[0 .. V / LANES).  V - V / LANES shuffles instead of
// V log2(LANES).
template <int V, int LANES, int STRIDE, int P>
__device__ __forceinline__ void reduce_transposed(float (&p)[P], int lane)
{
    static_assert(V <= P && V % LANES == 0, "values");
    if constexpr (LANES > 1) {
        const bool up = (lane & (STRIDE * LANES / 2)) != 0;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const float keep = up ? p[j + V / 2] : p[j];
            const float send = up ? p[j] : p[j + V / 2];
            p[j] = keep + __shfl_xor_sync(0xffffffffu, send, STRIDE * LANES / 2);
        }
        reduce_transposed<V / 2, LANES / 2, STRIDE>(p, lane);
    }
}

// Index of a sequence's first checkpoint; ceil(len / CK) of them follow.  For
// packed sequences floor(begin / CK) + seq leaves every sequence its room.
template <int CK>
__device__ __forceinline__ long long ckpt_base(const Seqs& q, int seq, long long begin)
{
    return q.cu ? begin / CK + seq : (long long)seq * ((q.T + CK - 1) / CK);
}

// Row t of an array with rows `bytes` apart: one wide multiply-add, and no pointer
// is kept in registers.
template <typename E>
__device__ __forceinline__ const E* row(const void* base, unsigned t, unsigned bytes)
{
    return reinterpret_cast<const E*>(static_cast<const char*>(base) + (unsigned long long)t * bytes);
}
template <typename E>
__device__ __forceinline__ E* row(void* base, unsigned t, unsigned bytes)
{
    return reinterpret_cast<E*>(static_cast<char*>(base) + (unsigned long long)t * bytes);
}

// 2 P consecutive elements in shared memory, in pairs.  bf16 stays bf16 there: the
// walk is bound by the words that shared memory returns, and widening is cheap.
template <int P>
__device__ __forceinline__ void read_states(const __nv_bfloat16* p, f32x2 (&v)[P])
{
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        const uint2 t = *reinterpret_cast<const uint2*>(p + 2 * i);
        v[i] = pack(__uint_as_float(t.x << 16), __uint_as_float(t.x & 0xffff0000u));
        v[i + 1] = pack(__uint_as_float(t.y << 16), __uint_as_float(t.y & 0xffff0000u));
    }
}
template <int P>
__device__ __forceinline__ void read_states(const float* p, f32x2 (&v)[P])
{
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p + 2 * i);
        v[i] = t.x;
        v[i + 1] = t.y;
    }
}
template <int P>
__device__ __forceinline__ void write_states(float* p, const f32x2 (&v)[P])
{
#pragma unroll
    for (int i = 0; i < P; i += 2) *reinterpret_cast<ulonglong2*>(p + 2 * i) = make_ulonglong2(v[i], v[i + 1]);
}

struct SsmDev {
    const void *x, *dt, *b, *c, *z;
    unsigned ldx, lddt, ldb, ldc, ldz;   // bytes from row to row
    const float *A, *skip, *dt_bias, *s0;
    void* y;
    float* sT;
    Seqs q;
    int D, G, tiles;   // tiles: channel tiles per group
    bool softplus, o_bf16;
};

}  // namespace mixer
}  // namespace kda
