// Selective state space scan: per channel d with N states
//   Delta_t = softplus(dt_t + dt_bias)  (or dt_t + dt_bias),
//   h_t[n] = exp(Delta_t A[d, n]) h_{t-1}[n] + Delta_t x_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + skip[d] x_t) silu(z_t)
// over dense or packed sequences, and as a step of one token per sequence.
//
// The decay depends on the channel and on the state index, so a chunk's
// interaction matrix has no low-rank factors: there is no tensor-core form, and
// the work is N exponentials and 3 N multiply-adds per (token, channel).  The
// floor of a prompt is the exponentials' rate (16 per SM and clock), that of a step
// the state's traffic.
#include "kda_ssm.cuh"

namespace kda {
namespace mixer {

// The walk's additions of the backward pass (CK = 0: none): the state before
// every CK-th token, and the gradient of z in the place of y.
struct WalkBwd {
    const float* gy;
    float *gz, *ckpt;
};

// Shape of a walk.  A block owns DT = 8 channels of a sequence.  A warp holds all
// states of the channels, a channel's N states on L = 4 lanes, NPT = N / 4 states
// each, and takes TK tokens at a time; W such warps take turns.
template <int N_>
struct Walk {
    static constexpr int N = N_, W = 4, L = 4, NPT = N / L, DT = 32 / L, THREADS = 32 * W;
    static constexpr int TK = 32 / NPT;                      // 32 decays in registers
    static constexpr int R = L < TK ? L : TK, VP = TK / R;   // lanes of a channel that finish tokens, tokens of each
    static constexpr int DUROW = DT + 2, YROW = DT;          // (Delta, u) of a token: rows on other banks
};

__device__ __forceinline__ void bar_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The recurrence is a chain of one multiply-add per token and state; everything
// else of a token is independent of it.  So the warps of a block take turns along
// the sequence: each computes the step sizes, decays and inputs of its TK tokens
// into registers, waits for the state of the warp before it, runs the chain (TK
// multiply-adds), hands the state on, and only then forms y, the gate and the
// output.  Every exponential is computed once, W warps per 8 channels are at work
// at any time, and the warps meet nowhere but at that hand-over (a named barrier
// of the two warps).
//
// Measured (bf16, N = 16, gated): 2 x 4096 tokens x 2048 channels in 172 us, 41 % of
// the exponentials' rate (72 us); four times the blocks, 45 %.  Per warp and 32
// (channel, state, token) 11.5 instructions are issued (62 % of the slots at full
// load) and 3.6 words per lane leave shared memory (76 % of its cycles), so no single
// unit is full but the two together are.  Four warps of 8 channels and 120 registers:
// with 96 (five blocks) the decays spill, 20 cycles for 18 (at 128, N = 64 spills 8 bytes
// in bf16 and 24 in fp32, the backward pass's form 16 and 64); W = 8 is 2 % faster at
// 512 blocks and 5 % slower at 2048, W = 3, 5, 6 slower at both; twice the states per
// lane save shared memory and wait at the hand-over (275 cycles), 20 to 22 cycles; two
// states per lane 197 us; B and C in fp32 8 % slower; the time split into groups with
// a second pass over the states 236 us; one warp that stages for the others 216.
template <typename T, int N, int CK>
__global__ void __launch_bounds__(Walk<N>::THREADS, 4)
ssm_walk_kernel(const SsmDev p, const WalkBwd wb)
{
    using K = Walk<N>;
    constexpr int TK = K::TK, DT = K::DT, L = K::L, W = K::W, NPT = K::NPT, R = K::R, VP = K::VP;
    __shared__ __align__(16) float2 sDU[W][TK * K::DUROW];   // [token][channel]: Delta, u
    __shared__ __align__(16) T sB[W][TK * N], sC[W][TK * N];  // [token][N]
    __shared__ float4 sState[W][DT * N / 4];                 // handed on by warp w: [lane][NPT]
    __shared__ __align__(16) float sY[W][TK * K::YROW];

    if (CK == 0) flag_bad_sequences(p.q);
    const int ntiles = p.tiles * p.G;
    const int tile = blockIdx.x % ntiles, seq = blockIdx.x / ntiles;
    const int Dg = p.D / p.G, g = tile / p.tiles, c0 = g * Dg + tile % p.tiles * DT;   // D / G is a multiple of 8
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = lane / L, l = lane % L;

    const long long s = p.q.begin(seq);
    long long e = p.q.begin(seq + 1);
    if (e < s || !Seqs::inside(s, e, p.q.tokens)) e = s;
    const int len = (int)(e - s);

    f32x2 A2[NPT / 2], h[NPT / 2];
    const long long srow = ((long long)seq * p.D + c0 + c) * N + l * NPT;
#pragma unroll
    for (int n = 0; n < NPT / 2; ++n) {
        const float2 a = *reinterpret_cast<const float2*>(p.A + (long long)(c0 + c) * N + l * NPT + 2 * n);
        A2[n] = pack(bounded_decay(a.x) * kLog2e, bounded_decay(a.y) * kLog2e);
        h[n] = p.s0 ? *reinterpret_cast<const f32x2*>(p.s0 + srow + 2 * n) : 0ull;
    }
    const bool gated = p.z != nullptr;

    // the lane's elements outside the chain: channels ec, ec + 1 of token et, and a
    // quad each of B and C
    const bool mine = lane < TK * DT / 2;
    const int et = lane / (DT / 2), ec = c0 + lane % (DT / 2) * 2, bt = lane / (N / 4), bn = g * N + lane % (N / 4) * 4;
    float2 bias = make_float2(0.f, 0.f), skip = bias;
    if (p.dt_bias) bias = *reinterpret_cast<const float2*>(p.dt_bias + ec);
    if (p.skip) skip = *reinterpret_cast<const float2*>(p.skip + ec);
    const int first = (int)s;

    typedef typename Raw<T>::pair Pair;
    typedef typename Raw<T>::quad Quad;
    Pair nx, ndt, nz;
    float2 ngy;
    Quad nb, nc;
    auto fetch = [&](int t0) {   // the lane's inputs of the TK tokens from t0 on; zero behind the end
        nx = ndt = nz = Pair{};
        nb = nc = Quad{};
        if (mine && t0 + et < len) {
            const unsigned t = first + t0 + et;
            nx = *reinterpret_cast<const Pair*>(row<T>(p.x, t, p.ldx) + ec);
            ndt = *reinterpret_cast<const Pair*>(row<T>(p.dt, t, p.lddt) + ec);
            if (gated) nz = *reinterpret_cast<const Pair*>(row<T>(p.z, t, p.ldz) + ec);
            if (CK > 0) ngy = *reinterpret_cast<const float2*>(row<float>(wb.gy, t, 4u * p.D) + ec);
        }
        if (t0 + bt < len) {
            const unsigned t = first + t0 + bt;
            nb = *reinterpret_cast<const Quad*>(row<T>(p.b, t, p.ldb) + bn);
            nc = *reinterpret_cast<const Quad*>(row<T>(p.c, t, p.ldc) + bn);
        }
    };
    fetch(w * TK);

    for (int t0 = w * TK; t0 < len; t0 += W * TK) {
        const float2 x = widen(nx), z = widen(nz), gy = ngy;
        __syncwarp();
        if (mine) {
            const float2 dt = widen(ndt);
            f32x2 d = add2(pack(dt.x, dt.y), pack(bias.x, bias.y));
            float d0, d1, u0, u1;
            unpack(d, d0, d1);
            if (p.softplus) unpack(softplus2(d0, d1), d0, d1);
            if (t0 + et >= len) d0 = d1 = 0.f;   // a token behind the end leaves the state as it is
            unpack(mul2(pack(d0, d1), pack(x.x, x.y)), u0, u1);
            *reinterpret_cast<float4*>(&sDU[w][et * K::DUROW + ec - c0]) = make_float4(d0, u0, d1, u1);
        }
        reinterpret_cast<Quad*>(sB[w])[lane] = nb;
        reinterpret_cast<Quad*>(sC[w])[lane] = nc;
        __syncwarp();
        fetch(t0 + W * TK);

        f32x2 a[TK][NPT / 2], b[TK][NPT / 2];
        const T* pB = sB[w] + l * NPT;
#pragma unroll
        for (int j = 0; j < TK; ++j) {
            const float2 d = sDU[w][j * K::DUROW + c];
            const f32x2 dd = pack(d.x, d.x), uu = pack(d.y, d.y);
            f32x2 B[NPT / 2];
            read_states(pB + j * N, B);
#pragma unroll
            for (int n = 0; n < NPT / 2; ++n) {
                a[j][n] = decay2(dd, A2[n]);
                b[j][n] = mul2(uu, B[n]);
            }
        }
        if (t0 > 0) {
            const int from = (w + W - 1) % W;
            bar_sync(1 + from, 64);
            read_states(reinterpret_cast<const float*>(sState[from]) + lane * NPT, h);
        }
        if constexpr (CK > 0) {
            if (t0 % CK == 0) {
                float* o = wb.ckpt + ((ckpt_base<CK>(p.q, seq, s) + t0 / CK) * p.D + c0 + c) * N + l * NPT;
#pragma unroll
                for (int n = 0; n < NPT / 2; ++n) *reinterpret_cast<f32x2*>(o + 2 * n) = h[n];
            }
        }
#pragma unroll
        for (int j = 0; j < TK; ++j)
#pragma unroll
            for (int n = 0; n < NPT / 2; ++n) b[j][n] = h[n] = fma2(a[j][n], h[n], b[j][n]);   // b: now the states
        if (t0 + TK < len) {
            write_states(reinterpret_cast<float*>(sState[w]) + lane * NPT, h);
            bar_arrive(1 + w, 64);
        } else if (CK == 0 && p.sT) {
#pragma unroll
            for (int n = 0; n < NPT / 2; ++n) *reinterpret_cast<f32x2*>(p.sT + srow + 2 * n) = h[n];
        }
        float y[TK];
        const T* pC = sC[w] + l * NPT;
#pragma unroll
        for (int j = 0; j < TK; ++j) {
            f32x2 C[NPT / 2], sum;
            read_states(pC + j * N, C);
            sum = mul2(C[0], b[j][0]);
#pragma unroll
            for (int n = 1; n < NPT / 2; ++n) sum = fma2(C[n], b[j][n], sum);
            float lo, hi;
            unpack(sum, lo, hi);
            y[j] = lo + hi;
        }
        reduce_transposed<TK, R, L / R>(y, lane);
#pragma unroll
        for (int v = 0; v < VP; ++v) {
#pragma unroll
            for (int m = L / R / 2; m >= 1; m >>= 1) y[v] += __shfl_xor_sync(0xffffffffu, y[v], m);
            if (l % (L / R) == 0) sY[w][(l / (L / R) * VP + v) * K::YROW + c] = y[v];
        }
        __syncwarp();
        if (mine && t0 + et < len && (CK == 0 || gated)) {
            const float2 r = *reinterpret_cast<const float2*>(&sY[w][et * K::YROW + ec - c0]);
            f32x2 out = fma2(pack(skip.x, skip.y), pack(x.x, x.y), pack(r.x, r.y));
            float o[2];
            const unsigned t = first + t0 + et;
            if constexpr (CK > 0) {
                unpack(out, o[0], o[1]);
                o[0] *= gy.x * silu_grad(z.x);
                o[1] *= gy.y * silu_grad(z.y);
                store_vec<2>(row<float>(wb.gz, t, 4u * p.D) + ec, o);
            } else {
                if (gated) out = mul2(out, silu2(z.x, z.y));
                unpack(out, o[0], o[1]);
                if (p.o_bf16)
                    store_vec<2>(row<__nv_bfloat16>(p.y, t, 2u * p.D) + ec, o);
                else
                    store_vec<2>(row<float>(p.y, t, 4u * p.D) + ec, o);
            }
        }
    }
    if (CK == 0 && p.sT && len == 0 && w == 0) {
#pragma unroll
        for (int n = 0; n < NPT / 2; ++n) *reinterpret_cast<f32x2*>(p.sT + srow + 2 * n) = h[n];
    }
}

// One token per sequence.  A lane owns 4 states (16 bytes) of a channel, a
// thread the same 4 states of RN sequences, so that A is read once for them and
// their states are in flight together; a state is read once and written once.
// With RN = 4, what is per (sequence, channel) -- the step size, the gate, the
// output -- is done by one lane for one of the four sequences instead of by
// every lane for all of them.  Bound by HBM: 256 x 4096 x 16 in 30 us, 143 MB, 4.8 TB/s
// (59 us with RN = 1; the state read through the caches and B, C held from the start
// 41); 2.2 us for one sequence, a launch.  The rate hardly climbs with the size (every
// tensor out of the L2: 4.5 TB/s with 256 sequences, 4.7 with 512, 4.9 with 2048).
template <typename T, int N, int RN>
__global__ void __launch_bounds__(256)
ssm_step_kernel(const SsmDev p, int n_seq)
{
    static_assert(RN == 1 || RN == 4, "a row per lane of the smallest group, or one row");
    constexpr int L = N / 4;
    const int f = blockIdx.x * 256 + threadIdx.x;   // 16-byte vector within one sequence's state (D N / 4 <= 2^24)
    const int d = f / L, l = f % L;
    if (d >= p.D) return;   // D is a multiple of 8 and 32 / L divides 8: whole warps leave
    const int lane = threadIdx.x & 31, group = lane / L * L;
    const int bn = d / (p.D / p.G) * N + 4 * l;
    float4 A = *reinterpret_cast<const float4*>(p.A + (long long)d * N + 4 * l);
    A.x = bounded_decay(A.x) * kLog2e;
    A.y = bounded_decay(A.y) * kLog2e;
    A.z = bounded_decay(A.z) * kLog2e;
    A.w = bounded_decay(A.w) * kLog2e;
    for (int i0 = blockIdx.y * RN; i0 < n_seq; i0 += gridDim.y * RN) {   // one round unless n_seq is beyond the grid
        float4* state = reinterpret_cast<float4*>(p.sT) + ((long long)i0 * p.D + d) * L + l;
        const long long next = (long long)p.D * L;      // 16-byte vectors from sequence to sequence
        const int rows = min(RN, n_seq - i0);
        float4 h[RN];
#pragma unroll
        for (int r = 0; r < RN; ++r) {
            if (r < rows) h[r] = __ldcs(state + r * next);
        }
        const int mine = RN == 1 ? 0 : l / (L / 4);     // the sequence whose elements are this lane's
        float x = 0.f, delta = 0.f, z = 0.f;
        if (mine < rows) {
            x = Elem<T>::load(row<T>(p.x, i0 + mine, p.ldx) + d);
            delta = Elem<T>::load(row<T>(p.dt, i0 + mine, p.lddt) + d);
            if (p.z) z = Elem<T>::load(row<T>(p.z, i0 + mine, p.ldz) + d);
        }
        if (p.dt_bias) delta += p.dt_bias[d];
        if (p.softplus) delta = softplus(delta);
        const float u = delta * x;
        float y[RN];
#pragma unroll
        for (int r = 0; r < RN; ++r) {
            const float dr = RN == 1 ? delta : __shfl_sync(0xffffffffu, delta, group + r * (L / 4));
            const float ur = RN == 1 ? u : __shfl_sync(0xffffffffu, u, group + r * (L / 4));
            y[r] = 0.f;
            if (r < rows) {
                float b[4], c[4];   // read here: held from the start they would halve the blocks per SM
                load_vec<4>(row<T>(p.b, i0 + r, p.ldb) + bn, b);
                load_vec<4>(row<T>(p.c, i0 + r, p.ldc) + bn, c);
                h[r].x = fmaf(exp2_approx(fmaf(dr, A.x, kDecayShift)), h[r].x, ur * b[0]);
                h[r].y = fmaf(exp2_approx(fmaf(dr, A.y, kDecayShift)), h[r].y, ur * b[1]);
                h[r].z = fmaf(exp2_approx(fmaf(dr, A.z, kDecayShift)), h[r].z, ur * b[2]);
                h[r].w = fmaf(exp2_approx(fmaf(dr, A.w, kDecayShift)), h[r].w, ur * b[3]);
                __stcs(state + r * next, h[r]);
                y[r] = fmaf(c[0], h[r].x, c[1] * h[r].y) + fmaf(c[2], h[r].z, c[3] * h[r].w);
            }
        }
        reduce_transposed<RN, RN, L / RN>(y, lane);
#pragma unroll
        for (int m = L / RN / 2; m >= 1; m >>= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], m);
        if (l % (L / RN) == 0 && mine < rows) {
            float out = p.skip ? fmaf(p.skip[d], x, y[0]) : y[0];
            if (p.z) out *= silu(z);
            if (p.o_bf16)
                row<__nv_bfloat16>(p.y, i0 + mine, 2u * p.D)[d] = __float2bfloat16_rn(out);
            else
                row<float>(p.y, i0 + mine, 4u * p.D)[d] = out;
        }
    }
}

static SsmDev ssm_dev(const SsmArgs& a, void* y, float* sT, kda_dtype o_dtype)
{
    SsmDev p;
    p.x = a.x; p.dt = a.dt; p.b = a.b; p.c = a.c; p.z = a.z;
    const unsigned es = a.dtype == KDA_BF16 ? 2 : 4;   // strides in bytes: below 2^32
    p.ldx = (unsigned)a.ldx * es; p.lddt = (unsigned)a.lddt * es; p.ldb = (unsigned)a.ldb * es;
    p.ldc = (unsigned)a.ldc * es; p.ldz = (unsigned)a.ldz * es;
    p.A = a.A; p.skip = a.skip; p.dt_bias = a.dt_bias; p.s0 = a.s0;
    p.y = y; p.sT = sT;
    p.q = Seqs{a.cu, a.nseq, a.T, a.tokens};
    p.D = a.D; p.G = a.G; p.tiles = 0;
    p.softplus = a.softplus; p.o_bf16 = o_dtype == KDA_BF16;
    return p;
}

template <typename T, int N, int CK = 0>
static cudaError_t launch_walk(const SsmArgs& a, SsmDev p, cudaStream_t s, const WalkBwd& w = WalkBwd{})
{
    using K = Walk<N>;
    p.tiles = a.D / a.G / K::DT;
    const long long blocks = (long long)a.nseq * p.tiles * a.G;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    ssm_walk_kernel<T, N, CK><<<(unsigned)blocks, K::THREADS, 0, s>>>(p, w);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t walk_dispatch(const SsmArgs& a, const SsmDev& p, cudaStream_t s)
{
    if (a.N == 16) return launch_walk<T, 16>(a, p, s);
    if (a.N == 32) return launch_walk<T, 32>(a, p, s);
    return launch_walk<T, 64>(a, p, s);
}

template <typename T, int N>
static cudaError_t launch_step(const SsmArgs& a, const SsmDev& p, cudaStream_t s)
{
    const unsigned gx = (unsigned)(((long long)a.D * (N / 4) + 255) / 256);
    // four sequences per thread once that leaves a block per SM, or where the grid's
    // second dimension would run out (D = 4096, N = 16, bf16, one against four: 4
    // sequences 2.46 / 3.17 us, 8 3.18 / 3.40, 12 4.34 / 3.76, 64 15.6 / 9.5, 256 59 / 30)
    if ((long long)gx * a.nseq / 4 >= 148LL || a.nseq > 65535) {
        const int blocks = (int)(((long long)a.nseq + 3) / 4);
        ssm_step_kernel<T, N, 4><<<dim3(gx, blocks < 65535 ? blocks : 65535), 256, 0, s>>>(p, a.nseq);
    } else {
        ssm_step_kernel<T, N, 1><<<dim3(gx, a.nseq), 256, 0, s>>>(p, a.nseq);
    }
    return cudaGetLastError();
}

template <typename T>
static cudaError_t step_dispatch(const SsmArgs& a, const SsmDev& p, cudaStream_t s)
{
    if (a.N == 16) return launch_step<T, 16>(a, p, s);
    if (a.N == 32) return launch_step<T, 32>(a, p, s);
    return launch_step<T, 64>(a, p, s);
}

}  // namespace mixer

cudaError_t ssm_fwd(const SsmArgs& a, void* y, float* sT, kda_dtype o_dtype, cudaStream_t s)
{
    const mixer::SsmDev p = mixer::ssm_dev(a, y, sT, o_dtype);
    return a.dtype == KDA_BF16 ? mixer::walk_dispatch<__nv_bfloat16>(a, p, s) : mixer::walk_dispatch<float>(a, p, s);
}

cudaError_t ssm_step(const SsmArgs& a, float* state, void* y, kda_dtype o_dtype, cudaStream_t s)
{
    const mixer::SsmDev p = mixer::ssm_dev(a, y, state, o_dtype);
    return a.dtype == KDA_BF16 ? mixer::step_dispatch<__nv_bfloat16>(a, p, s) : mixer::step_dispatch<float>(a, p, s);
}

}  // namespace kda
