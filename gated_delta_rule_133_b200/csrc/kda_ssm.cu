// Selective state space scan: per channel d with N states
//   Delta_t = softplus(dt_t + dt_bias)  (or dt_t + dt_bias),
//   h_t[n] = exp(Delta_t A[d, n]) h_{t-1}[n] + Delta_t x_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + skip[d] x_t) silu(z_t)
// over dense or packed sequences, and as a step of one token per sequence.
//
// The decay depends on the channel and on the state index, so a chunk's
// interaction matrix has no low-rank factors: there is no tensor-core form, and
// the work is N exponentials and 3 N multiply-adds per (token, channel).  The
// prompt kernel is bound by the exponentials' rate (16 per SM and clock), the
// step by the state's traffic.
#include "kda_ssm.cuh"

namespace kda {
namespace mixer {

// The walk's additions of the backward pass (CK = 0: none): the state before
// every CK-th token, and the gradient of z in the place of y.
struct WalkBwd {
    const float* gy;
    float *gz, *ckpt;
};

template <typename T, int N, int L, int CK>
__global__ void __launch_bounds__(128)
ssm_walk_kernel(const SsmDev p, const WalkBwd w)
{
    using K = Walk<T, N, L>;
    constexpr int TT = K::TT, DT = K::DT, NPT = K::NPT, EP = K::EP;
    extern __shared__ __align__(16) unsigned char smem[];
    float* sDU = reinterpret_cast<float*>(smem + 2 * K::STAGE);
    float* sB = sDU + TT * K::DUROW;
    float* sC = sB + TT * N;

    if (CK == 0) flag_bad_sequences(p.q);
    const int ntiles = p.tiles * p.G;
    const int tile = blockIdx.x % ntiles, seq = blockIdx.x / ntiles;
    const int Dg = p.D / p.G, g = tile / p.tiles, off = (tile % p.tiles) * DT;
    const int c0 = g * Dg + off, nvalid = min(DT, Dg - off);
    const int tid = threadIdx.x, l = tid % L, c = tid / L;
    const bool live = c < nvalid;

    long long s = p.q.begin(seq), e = p.q.begin(seq + 1);
    if (e < s || !Seqs::inside(s, e, p.q.tokens)) e = s;

    const T* x = static_cast<const T*>(p.x) + c0;
    const T* dt = static_cast<const T*>(p.dt) + c0;
    const T* z = p.z ? static_cast<const T*>(p.z) + c0 : nullptr;
    const T* b = static_cast<const T*>(p.b) + g * N;
    const T* cc = static_cast<const T*>(p.c) + g * N;

    float A2[NPT], h[NPT];
    const long long srow = ((long long)seq * p.D + c0 + c) * N + l * NPT;
#pragma unroll
    for (int n = 0; n < NPT; ++n) {
        A2[n] = live ? p.A[(long long)(c0 + c) * N + l * NPT + n] * kLog2e : 0.f;
        h[n] = live && p.s0 ? p.s0[srow + n] : 0.f;
    }
    // the thread's EP elements outside the walk: token rt, channels rc ..
    const int rt = tid * EP / DT, rc = tid * EP % DT;
    const bool rlive = rc < nvalid;
    float bias[EP], skip[EP];
#pragma unroll
    for (int k = 0; k < EP; ++k) {
        bias[k] = rlive && p.dt_bias ? p.dt_bias[c0 + rc + k] : 0.f;
        skip[k] = rlive && p.skip ? p.skip[c0 + rc + k] : 0.f;
    }

    auto fetch = [&](long long t0, int stage) {
        T* st = reinterpret_cast<T*>(smem + stage * K::STAGE);
        fetch_rows<T, TT, DT, 128>(st, x, p.ldx, t0, e, nvalid);
        fetch_rows<T, TT, DT, 128>(st + TT * DT, dt, p.lddt, t0, e, nvalid);
        if (z) fetch_rows<T, TT, DT, 128>(st + 2 * TT * DT, z, p.ldz, t0, e, nvalid);
        fetch_rows<T, TT, N, 128>(st + 3 * TT * DT, b, p.ldb, t0, e, N);
        fetch_rows<T, TT, N, 128>(st + 3 * TT * DT + TT * N, cc, p.ldc, t0, e, N);
    };
    int stage = 0;
    if (s < e) fetch(s, 0);
    cp_async_commit();
    for (long long t0 = s; t0 < e; t0 += TT, stage ^= 1) {
        if (t0 + TT < e) fetch(t0 + TT, stage ^ 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const T* st = reinterpret_cast<const T*>(smem + stage * K::STAGE);
        const bool rin = t0 + rt < e;
        float xv[EP];
        load_vec<EP>(st + rt * DT + rc, xv);
        {
            float dv[EP];
            load_vec<EP>(st + TT * DT + rt * DT + rc, dv);
#pragma unroll
            for (int k = 0; k < EP; ++k) {
                const float v = dv[k] + bias[k];
                const float delta = !rin || !rlive ? 0.f : p.softplus ? softplus(v) : v;
                *reinterpret_cast<float2*>(sDU + rt * K::DUROW + 2 * (rc + k)) = make_float2(delta, delta * xv[k]);
            }
        }
        for (int i = tid * 2; i < TT * N; i += 256) {
            float v[2];
            load_vec<2>(st + 3 * TT * DT + i, v);
            store_vec<2>(sB + i, v);
            load_vec<2>(st + 3 * TT * DT + TT * N + i, v);
            store_vec<2>(sC + i, v);
        }
        __syncthreads();

        const int steps = (int)min((long long)TT, e - t0);
        for (int tb = 0; tb < steps; tb += L) {
            float acc[L];
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int t = tb + j;
                if constexpr (CK > 0) {
                    if (j % (CK < L ? CK : L) == 0 && t % CK == 0 && t < steps && live) {
                        float* o = w.ckpt + (ckpt_base<CK>(p.q, seq, s) + (t0 - s + t) / CK) * ((long long)p.D * N) +
                                   (long long)(c0 + c) * N + l * NPT;
#pragma unroll
                        for (int n = 0; n < NPT; ++n) o[n] = h[n];
                    }
                }
                const float2 du = *reinterpret_cast<const float2*>(sDU + t * K::DUROW + 2 * c);
                acc[j] = 0.f;
#pragma unroll
                for (int n = 0; n < NPT; ++n) {
                    const float a = exp2_approx(du.x * A2[n]);
                    h[n] = fmaf(a, h[n], du.y * sB[t * N + l * NPT + n]);
                    acc[j] = fmaf(sC[t * N + l * NPT + n], h[n], acc[j]);
                }
            }
            reduce_transposed<L, L, 1>(acc, tid);
            __syncwarp();
            // every lane of the group has read its (Delta, u) of these L tokens
            sDU[(tb + l) * K::DUROW + 2 * c] = acc[0];
        }
        __syncthreads();
        if (CK > 0) {
            if (z && rin && rlive) {
                float zv[EP], g[EP];
                const long long o = (t0 + rt) * p.D + c0 + rc;
                load_vec<EP>(st + 2 * TT * DT + rt * DT + rc, zv);
                load_vec<EP>(w.gy + o, g);
#pragma unroll
                for (int k = 0; k < EP; ++k)
                    g[k] *= fmaf(skip[k], xv[k], sDU[rt * K::DUROW + 2 * (rc + k)]) * silu_grad(zv[k]);
                store_vec<EP>(w.gz + o, g);
            }
        } else if (rin && rlive) {
            float out[EP];
#pragma unroll
            for (int k = 0; k < EP; ++k) out[k] = fmaf(skip[k], xv[k], sDU[rt * K::DUROW + 2 * (rc + k)]);
            if (z) {
                float zv[EP];
                load_vec<EP>(st + 2 * TT * DT + rt * DT + rc, zv);
#pragma unroll
                for (int k = 0; k < EP; ++k) out[k] *= silu(zv[k]);
            }
            const long long o = (t0 + rt) * p.D + c0 + rc;
            if (p.o_bf16)
                store_vec<EP>(static_cast<__nv_bfloat16*>(p.y) + o, out);
            else
                store_vec<EP>(static_cast<float*>(p.y) + o, out);
        }
        __syncthreads();   // the stage and (Delta, u) are free
    }
    if (CK == 0 && p.sT && live) {
#pragma unroll
        for (int n = 0; n < NPT; ++n) p.sT[srow + n] = h[n];
    }
}

// One token per sequence.  A lane owns 4 states (16 bytes) of a channel, a
// thread the same 4 states of RN sequences, so that A is read once for them;
// the state is read once and written once.
template <typename T, int N>
__global__ void __launch_bounds__(256)
ssm_step_kernel(const SsmDev p, int n_seq, int RN)
{
    constexpr int L = N / 4;
    const long long f = ((long long)blockIdx.x * 256 + threadIdx.x);   // float4 index within one sequence's state
    const int d = (int)(f / L), l = (int)(f % L);
    if (d >= p.D) return;   // D is a multiple of 8: whole groups of L <= 16 lanes leave together
    const unsigned mask = __activemask();
    const int g = d / (p.D / p.G);
    const float4 A = *reinterpret_cast<const float4*>(p.A + (long long)d * N + 4 * l);
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = p.skip ? p.skip[d] : 0.f;
    const int i1 = min((int)(blockIdx.y + 1) * RN, n_seq);
    for (int i = blockIdx.y * RN; i < i1; ++i) {
        float4* sp = reinterpret_cast<float4*>(p.sT + ((long long)i * p.D + d) * N + 4 * l);
        float4 h = *sp;
        const float x = Elem<T>::load(static_cast<const T*>(p.x) + i * p.ldx + d);
        const float v = Elem<T>::load(static_cast<const T*>(p.dt) + i * p.lddt + d) + bias;
        float b[4], c[4];
        load_vec<4>(static_cast<const T*>(p.b) + i * p.ldb + g * N + 4 * l, b);
        load_vec<4>(static_cast<const T*>(p.c) + i * p.ldc + g * N + 4 * l, c);
        const float delta = p.softplus ? softplus(v) : v, u = delta * x, d2 = delta * kLog2e;
        h.x = fmaf(exp2_approx(d2 * A.x), h.x, u * b[0]);
        h.y = fmaf(exp2_approx(d2 * A.y), h.y, u * b[1]);
        h.z = fmaf(exp2_approx(d2 * A.z), h.z, u * b[2]);
        h.w = fmaf(exp2_approx(d2 * A.w), h.w, u * b[3]);
        *sp = h;
        float y = fmaf(c[0], h.x, c[1] * h.y) + fmaf(c[2], h.z, c[3] * h.w);
#pragma unroll
        for (int m = L / 2; m >= 1; m >>= 1) y += __shfl_xor_sync(mask, y, m);
        if (l == 0) {
            y = fmaf(skip, x, y);
            if (p.z) y *= silu(Elem<T>::load(static_cast<const T*>(p.z) + i * p.ldz + d));
            const long long o = (long long)i * p.D + d;
            if (p.o_bf16)
                static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(y);
            else
                static_cast<float*>(p.y)[o] = y;
        }
    }
}

static SsmDev ssm_dev(const SsmArgs& a, void* y, float* sT, kda_dtype o_dtype)
{
    SsmDev p;
    p.x = a.x; p.dt = a.dt; p.b = a.b; p.c = a.c; p.z = a.z;
    p.ldx = a.ldx; p.lddt = a.lddt; p.ldb = a.ldb; p.ldc = a.ldc; p.ldz = a.ldz;
    p.A = a.A; p.skip = a.skip; p.dt_bias = a.dt_bias; p.s0 = a.s0;
    p.y = y; p.sT = sT;
    p.q = Seqs{a.cu, a.nseq, a.T, a.tokens};
    p.D = a.D; p.G = a.G; p.tiles = 0;
    p.softplus = a.softplus; p.o_bf16 = o_dtype == KDA_BF16;
    return p;
}

template <typename T, int N, int L, int CK = 0>
static cudaError_t launch_walk(const SsmArgs& a, SsmDev p, cudaStream_t s, const WalkBwd& w = WalkBwd{})
{
    using K = Walk<T, N, L>;
    p.tiles = (a.D / a.G + K::DT - 1) / K::DT;
    const long long blocks = (long long)a.nseq * p.tiles * a.G;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const cudaError_t e = cudaFuncSetAttribute(
        ssm_walk_kernel<T, N, L, CK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::SMEM);
    if (e != cudaSuccess) return e;
    ssm_walk_kernel<T, N, L, CK><<<(unsigned)blocks, K::THREADS, K::SMEM, s>>>(p, w);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t walk_dispatch(const SsmArgs& a, const SsmDev& p, cudaStream_t s)
{
    // States per lane: 4 where that still gives every scheduler of the 148 SMs
    // about two warps, else fewer (more lanes per channel).
    const long long warps = (long long)a.nseq * a.D * (a.N / 4) / 32;
    const bool wide = warps >= 148LL * 8;
    if (a.N == 16) {
        if (wide) return launch_walk<T, 16, 4>(a, p, s);
        if (warps >= 148LL * 2) return launch_walk<T, 16, 8>(a, p, s);
        return launch_walk<T, 16, 16>(a, p, s);
    }
    if (a.N == 32) return wide ? launch_walk<T, 32, 8>(a, p, s) : launch_walk<T, 32, 16>(a, p, s);
    return launch_walk<T, 64, 16>(a, p, s);
}

template <typename T>
static cudaError_t launch_step(const SsmArgs& a, const SsmDev& p, cudaStream_t s)
{
    const long long vecs = (long long)a.D * (a.N / 4);
    const unsigned gx = (unsigned)((vecs + 255) / 256);
    int RN = 4;
    while (RN > 1 && (long long)gx * a.nseq / RN < 148LL * 6) RN /= 2;
    while ((a.nseq + RN - 1) / RN > 65535) RN *= 2;
    const dim3 grid(gx, (a.nseq + RN - 1) / RN);
    if (a.N == 16)
        ssm_step_kernel<T, 16><<<grid, 256, 0, s>>>(p, a.nseq, RN);
    else if (a.N == 32)
        ssm_step_kernel<T, 32><<<grid, 256, 0, s>>>(p, a.nseq, RN);
    else
        ssm_step_kernel<T, 64><<<grid, 256, 0, s>>>(p, a.nseq, RN);
    return cudaGetLastError();
}

}  // namespace mixer

size_t ssm_fwd_workspace(int, int, long long, int, int, int, bool) { return 0; }

cudaError_t ssm_fwd(const SsmArgs& a, void* y, float* sT, kda_dtype o_dtype, void*, cudaStream_t s)
{
    const mixer::SsmDev p = mixer::ssm_dev(a, y, sT, o_dtype);
    return a.dtype == KDA_BF16 ? mixer::walk_dispatch<__nv_bfloat16>(a, p, s) : mixer::walk_dispatch<float>(a, p, s);
}

cudaError_t ssm_step(const SsmArgs& a, float* state, void* y, kda_dtype o_dtype, cudaStream_t s)
{
    const mixer::SsmDev p = mixer::ssm_dev(a, y, state, o_dtype);
    return a.dtype == KDA_BF16 ? mixer::launch_step<__nv_bfloat16>(a, p, s) : mixer::launch_step<float>(a, p, s);
}

}  // namespace kda
