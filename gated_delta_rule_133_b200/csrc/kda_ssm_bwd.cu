// Gradients of the selective scan.  With dy0 = gy silu(z), a_t = exp(Delta_t A):
//   g_t = C_t dy0_t + a_{t+1} g_{t+1}                    (reverse recurrence)
//   dB_t = sum_d g_t Delta_t x_t,   dC_t = sum_d h_t dy0_t,   du_t = sum_n g_t B_t
//   w_t = g_t a_t h_{t-1},   dA = sum_t w_t Delta_t,   dDelta_t = sum_n w_t A + du_t x_t
//   dx_t = du_t Delta_t + skip dy0_t,   ddt_t = dDelta_t sigmoid(dt_t + bias)
//   dz_t = gy_t y0_t silu'(z_t),   dh_0 = a_0 g_0
// Four launches: the forward walk, which leaves the state before every CK-th
// token (and dz, as it has y0); the reverse walk, which recomputes CK states at
// a time into registers and runs the reverse recurrence over them; and two sums
// in a fixed order, of dB and dC over channel tiles and of dA, dskip and dbias
// over the blocks that share a channel.
#include "kda_ssm.cuh"

namespace kda {
namespace mixer {

struct BwdDev {
    SsmDev p;
    const float *gy, *gsT;
    float *gx, *gdt, *gz, *gs0;
    const float* ckpt;
    float *part;              // [tile of the group][token][G][2 N]: dB, dC
    float *partA, *partv;     // [slot][D][N]; [slot][2][D]: dskip, dbias
    int slots;
};

template <typename T, int N_, int L_, int CK_>
struct Rev {
    static constexpr int N = N_, L = L_, CK = CK_, NPT = N / L, DT = L == 4 ? 32 : 16, THREADS = DT * L;
    static constexpr int TT = N == 64 ? 32 : L == 4 ? 32 : 64, WARPS = THREADS / 32, CPW = 32 / L, GT = L / 2;
    static constexpr int EP = TT * DT / THREADS;
    static constexpr int DUROW = 2 * DT + 16, DYROW = DT + 4;
    static constexpr size_t RAW_X = (size_t)TT * DT * sizeof(T), RAW_B = (size_t)TT * N * sizeof(T);
    static constexpr size_t RAW_G = (size_t)TT * DT * 4;
    static constexpr size_t STAGE = 3 * RAW_X + 2 * RAW_B + RAW_G;
    static constexpr size_t WORK = ((size_t)TT * (DUROW + DYROW + 2 * N) + (size_t)WARPS * CK * 2 * N) * 4;
    static constexpr size_t SMEM = 2 * STAGE + WORK;
    static_assert(CK % GT == 0 && TT % CK == 0, "groups");
};

template <typename T, int N, int L, int CK>
__global__ void __launch_bounds__(Rev<T, N, L, CK>::THREADS)
ssm_reverse_kernel(const BwdDev b)
{
    using K = Rev<T, N, L, CK>;
    constexpr int TT = K::TT, DT = K::DT, NPT = K::NPT, EP = K::EP, NT = K::THREADS, GT = K::GT;
    const SsmDev& p = b.p;
    extern __shared__ __align__(16) unsigned char smem[];
    float* sDU = reinterpret_cast<float*>(smem + 2 * K::STAGE);
    float* sDY = sDU + TT * K::DUROW;
    float* sB = sDY + TT * K::DYROW;
    float* sC = sB + TT * N;
    float* sP = sC + TT * N;

    flag_bad_sequences(p.q);
    const int ntiles = p.tiles * p.G;
    const int tile = blockIdx.x % ntiles, slot = blockIdx.x / ntiles;
    const int Dg = p.D / p.G, g = tile / p.tiles, gt = tile % p.tiles, off = gt * DT;
    const int c0 = g * Dg + off, nvalid = min(DT, Dg - off);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, l = tid % L, c = tid / L;
    const bool live = c < nvalid;

    const T* x = static_cast<const T*>(p.x) + c0;
    const T* dt = static_cast<const T*>(p.dt) + c0;
    const T* z = p.z ? static_cast<const T*>(p.z) + c0 : nullptr;
    const T* bb = static_cast<const T*>(p.b) + g * N;
    const T* cc = static_cast<const T*>(p.c) + g * N;

    float A[NPT], gA[NPT];
#pragma unroll
    for (int n = 0; n < NPT; ++n) {
        A[n] = live ? p.A[(long long)(c0 + c) * N + l * NPT + n] : 0.f;
        gA[n] = 0.f;
    }
    const int rt = tid * EP / DT, rc = tid * EP % DT;
    const bool rlive = rc < nvalid;
    float bias[EP], skip[EP], gskip[EP], gbias[EP];
#pragma unroll
    for (int k = 0; k < EP; ++k) {
        bias[k] = rlive && p.dt_bias ? p.dt_bias[c0 + rc + k] : 0.f;
        skip[k] = rlive && p.skip ? p.skip[c0 + rc + k] : 0.f;
        gskip[k] = gbias[k] = 0.f;
    }

    for (int seq = slot; seq < p.q.n; seq += b.slots) {
        const long long s = p.q.begin(seq);
        long long e = p.q.begin(seq + 1);
        if (e < s || !Seqs::inside(s, e, p.q.tokens)) e = s;
        auto fetch = [&](long long t0, int stage) {
            T* st = reinterpret_cast<T*>(smem + stage * K::STAGE);
            fetch_rows<T, TT, DT, NT>(st, x, p.ldx / sizeof(T), t0, e, nvalid);
            fetch_rows<T, TT, DT, NT>(st + TT * DT, dt, p.lddt / sizeof(T), t0, e, nvalid);
            if (z) fetch_rows<T, TT, DT, NT>(st + 2 * TT * DT, z, p.ldz / sizeof(T), t0, e, nvalid);
            fetch_rows<T, TT, N, NT>(st + 3 * TT * DT, bb, p.ldb / sizeof(T), t0, e, N);
            fetch_rows<T, TT, N, NT>(st + 3 * TT * DT + TT * N, cc, p.ldc / sizeof(T), t0, e, N);
            fetch_rows<float, TT, DT, NT>(reinterpret_cast<float*>(st + 3 * TT * DT + 2 * TT * N), b.gy + c0, p.D, t0, e,
                                          nvalid);
        };
        const long long srow = ((long long)seq * p.D + c0 + c) * N + l * NPT;
        float carry[NPT];
#pragma unroll
        for (int n = 0; n < NPT; ++n) carry[n] = live && b.gsT ? b.gsT[srow + n] : 0.f;

        int stage = 0;
        long long t0 = s + (e - s - 1) / TT * TT;
        if (s < e) fetch(t0, 0);
        cp_async_commit();
        for (; s < e && t0 >= s; t0 -= TT, stage ^= 1) {
            if (t0 > s) fetch(t0 - TT, stage ^ 1);
            cp_async_commit();
            cp_async_wait<1>();
            __syncthreads();
            const T* st = reinterpret_cast<const T*>(smem + stage * K::STAGE);
            const float* sg = reinterpret_cast<const float*>(st + 3 * TT * DT + 2 * TT * N);
            const bool rin = rlive && t0 + rt < e;
            float xv[EP], delta[EP], dy[EP];
            load_vec<EP>(st + rt * DT + rc, xv);
            {
                float v[EP];
                load_vec<EP>(st + TT * DT + rt * DT + rc, v);
#pragma unroll
                for (int k = 0; k < EP; ++k) {
                    v[k] += bias[k];
                    delta[k] = !rin ? 0.f : p.softplus ? softplus(v[k]) : v[k];
                    *reinterpret_cast<float2*>(sDU + rt * K::DUROW + 2 * (rc + k)) =
                        make_float2(delta[k], delta[k] * xv[k]);
                }
                load_vec<EP>(sg + rt * DT + rc, dy);
                if (z) {
                    load_vec<EP>(st + 2 * TT * DT + rt * DT + rc, v);
#pragma unroll
                    for (int k = 0; k < EP; ++k) dy[k] *= silu(v[k]);
                }
#pragma unroll
                for (int k = 0; k < EP; ++k) {
                    dy[k] = rin ? dy[k] : 0.f;
                    sDY[rt * K::DYROW + rc + k] = dy[k];
                }
            }
            for (int i = tid * 2; i < TT * N; i += 2 * NT) {
                float v[2];
                load_vec<2>(st + 3 * TT * DT + i, v);
                store_vec<2>(sB + i, v);
                load_vec<2>(st + 3 * TT * DT + TT * N + i, v);
                store_vec<2>(sC + i, v);
            }
            __syncthreads();

            for (int tb = (int)(min((long long)TT, e - t0) - 1) / CK * CK; tb >= 0; tb -= CK) {
                float h0[NPT], a[CK][NPT], h[CK][NPT];
                const float* cp = b.ckpt + ((ckpt_base<CK>(p.q, seq, s) + (t0 - s + tb) / CK) * p.D + c0 + c) * N + l * NPT;
#pragma unroll
                for (int n = 0; n < NPT; ++n) h0[n] = live ? cp[n] : 0.f;
#pragma unroll
                for (int j = 0; j < CK; ++j) {
                    const float2 du = *reinterpret_cast<const float2*>(sDU + (tb + j) * K::DUROW + 2 * c);
#pragma unroll
                    for (int n = 0; n < NPT; ++n) {
                        a[j][n] = exp2_approx(fmaf(du.x, A[n] * kLog2e, kDecayShift));
                        h[j][n] = fmaf(a[j][n], j ? h[j - 1][n] : h0[n], du.y * sB[(tb + j) * N + l * NPT + n]);
                    }
                }
#pragma unroll
                for (int jg = CK - GT; jg >= 0; jg -= GT) {
                    float sums[2 * GT];
#pragma unroll
                    for (int jj = GT - 1; jj >= 0; --jj) {
                        const int j = jg + jj, t = tb + j;
                        const float2 du = *reinterpret_cast<const float2*>(sDU + t * K::DUROW + 2 * c);
                        const float d = sDY[t * K::DYROW + c];
                        float v[2 * NPT], s1 = 0.f, s2 = 0.f;
#pragma unroll
                        for (int n = 0; n < NPT; ++n) {
                            const float gh = fmaf(sC[t * N + l * NPT + n], d, carry[n]);
                            v[n] = gh * du.y;
                            v[NPT + n] = h[j][n] * d;
                            s1 = fmaf(gh, sB[t * N + l * NPT + n], s1);
                            carry[n] = gh * a[j][n];
                            const float w = carry[n] * (j ? h[j > 0 ? j - 1 : 0][n] : h0[n]);
                            gA[n] = fmaf(w, du.x, gA[n]);
                            s2 = fmaf(w, A[n], s2);
                        }
                        sums[2 * jj] = s1;
                        sums[2 * jj + 1] = s2;
                        // over the warp's channels: dB, dC of this token
                        reduce_transposed<2 * NPT, K::CPW, L>(v, lane);
                        constexpr int VPL = 2 * NPT / K::CPW;   // values this lane is left with
                        const int i0 = (lane / L) * VPL;
                        float* o = sP + (wid * CK + j) * 2 * N + (i0 / NPT) * N + l * NPT + i0 % NPT;
#pragma unroll
                        for (int k = 0; k < VPL; ++k) o[k] = v[k];
                    }
                    reduce_transposed<2 * GT, L, 1>(sums, lane);
                    __syncwarp();
                    // every lane of the channel has read (Delta, u) of these GT tokens
                    sDU[(tb + jg + l / 2) * K::DUROW + 2 * c + (l & 1)] = sums[0];
                }
                __syncthreads();
                for (int i = tid; i < CK * 2 * N; i += NT) {
                    const long long t = t0 + tb + i / (2 * N);
                    if (t < e) {
                        float acc = sP[i];
#pragma unroll
                        for (int w = 1; w < K::WARPS; ++w) acc += sP[w * CK * 2 * N + i];
                        b.part[(((long long)gt * p.q.tokens + t) * p.G + g) * 2 * N + i % (2 * N)] = acc;
                    }
                }
                __syncthreads();
            }
            if (rin) {
                const long long o = (t0 + rt) * p.D + c0 + rc;
                float gx[EP], gd[EP], v[EP];
                load_vec<EP>(st + TT * DT + rt * DT + rc, v);
#pragma unroll
                for (int k = 0; k < EP; ++k) {
                    const float2 ss = *reinterpret_cast<const float2*>(sDU + rt * K::DUROW + 2 * (rc + k));
                    gx[k] = fmaf(ss.x, delta[k], skip[k] * dy[k]);
                    gd[k] = fmaf(ss.x, xv[k], ss.y) * (p.softplus ? sigmoid(v[k] + bias[k]) : 1.f);
                    gskip[k] = fmaf(dy[k], xv[k], gskip[k]);
                    gbias[k] += gd[k];
                }
                store_vec<EP>(b.gx + o, gx);
                store_vec<EP>(b.gdt + o, gd);
            }
            __syncthreads();   // the stage and the work arrays are free
        }
        if (b.gs0 && live) {
#pragma unroll
            for (int n = 0; n < NPT; ++n) b.gs0[srow + n] = carry[n];
        }
    }

    // this block's sums over its tokens
    if (live) {
#pragma unroll
        for (int n = 0; n < NPT; ++n) b.partA[((long long)slot * p.D + c0 + c) * N + l * NPT + n] = gA[n];
    }
    __syncthreads();
    float* red = sDU;   // [TT][2 DT]: TT rows of threads share a channel vector
    static_assert(K::DUROW >= 2 * DT, "room");
#pragma unroll
    for (int k = 0; k < EP; ++k) {
        red[rt * 2 * DT + rc + k] = gskip[k];
        red[rt * 2 * DT + DT + rc + k] = gbias[k];
    }
    __syncthreads();
    for (int i = tid; i < 2 * DT; i += NT) {
        float acc = 0.f;
        for (int r = 0; r < TT; ++r) acc += red[r * 2 * DT + i];
        if (i % DT < nvalid) b.partv[((long long)slot * 2 + i / DT) * p.D + c0 + i % DT] = acc;
    }
}

// dB and dC of every token from the channel tiles' sums, a warp per (token,
// group, 32 values).  Rows of no sequence: zero, here and in gx, gdt, gz.
__global__ void __launch_bounds__(256)
ssm_bwd_bc_kernel(const BwdDev b, float* __restrict__ gb, float* __restrict__ gc, int N)
{
    const SsmDev& p = b.p;
    const long long t = (long long)blockIdx.x * 8 + threadIdx.x / 32;
    if (t >= p.q.tokens) return;
    const int lane = threadIdx.x & 31;
    bool covered = true;
    if (p.q.cu) {
        const int i = find_sequence(p.q, t);
        covered = i >= 0 && i < p.q.n && t < p.q.begin(i + 1) &&
                  Seqs::inside(p.q.begin(i), p.q.begin(i + 1), p.q.tokens);
    }
    if (!covered) {
        for (int d = lane; d < p.D; d += 32) {
            b.gx[t * p.D + d] = b.gdt[t * p.D + d] = 0.f;
            if (b.gz) b.gz[t * p.D + d] = 0.f;
        }
    }
    const int cols = p.G * 2 * N;
    for (int i = lane; i < cols; i += 32) {
        float acc = 0.f;
        if (covered) {
#pragma unroll 8
            for (int k = 0; k < p.tiles; ++k) acc += b.part[((long long)k * p.q.tokens + t) * cols + i];
        }
        const int g = i / (2 * N), j = i % (2 * N);
        (j < N ? gb : gc)[(t * p.G + g) * N + j % N] = acc;
    }
}

// dA, dskip, dbias over the slots.
__global__ void __launch_bounds__(256)
ssm_bwd_params_kernel(const BwdDev b, float* __restrict__ gA, float* __restrict__ gskip, float* __restrict__ gbias, int N)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, nA = (long long)b.p.D * N;
    float acc = 0.f;
    if (i < nA) {
        for (int k = 0; k < b.slots; ++k) acc += b.partA[k * nA + i];
        gA[i] = acc;
    } else if (i < nA + 2 * b.p.D) {
        for (int k = 0; k < b.slots; ++k) acc += b.partv[(long long)k * 2 * b.p.D + (i - nA)];
        const int d = (int)((i - nA) % b.p.D);
        float* o = i - nA < b.p.D ? gskip : gbias;
        if (o) o[d] = acc;
    }
}

// Sequences are dealt to this many blocks per channel tile: enough to fill the
// 148 SMs several times, few enough that the partial sums of dA stay small.
static int bwd_slots(int nseq, int ntiles)
{
    const int want = (148 * 8 + ntiles - 1) / ntiles;
    return nseq < want ? nseq : want;
}

template <int N>
struct BwdShape {
    static constexpr int L = N == 64 ? 16 : 8, CK = 8, DT = 16;
};

struct BwdWorkspace {
    size_t ckpt, part, partA, partv, total;
};

template <int N>
static BwdWorkspace bwd_layout(int nseq, int T, long long tokens, int D, int G, bool varlen)
{
    using S = BwdShape<N>;
    const int tiles = (D / G + S::DT - 1) / S::DT, slots = bwd_slots(nseq, tiles * G);
    const size_t blocks = varlen ? (size_t)(tokens / S::CK) + nseq : (size_t)nseq * ((T + S::CK - 1) / S::CK);
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    BwdWorkspace w;
    w.ckpt = 0;
    w.part = w.ckpt + up(blocks * D * N * 4);
    w.partA = w.part + up((size_t)tiles * tokens * G * 2 * N * 4);
    w.partv = w.partA + up((size_t)slots * D * N * 4);
    w.total = w.partv + up((size_t)slots * 2 * D * 4);
    return w;
}

template <typename T, int N>
static cudaError_t launch_bwd(const SsmArgs& a, const SsmGrads& g, void* ws, cudaStream_t s)
{
    using S = BwdShape<N>;
    using K = Rev<T, N, S::L, S::CK>;
    static_assert(K::DT == S::DT, "channel tile");
    const BwdWorkspace w = bwd_layout<N>(a.nseq, a.T, a.tokens, a.D, a.G, a.cu != nullptr);
    char* base = static_cast<char*>(ws);
    BwdDev b;
    b.p = ssm_dev(a, nullptr, nullptr, KDA_F32);
    b.gy = g.gy; b.gsT = g.gsT;
    b.gx = g.gx; b.gdt = g.gdt; b.gz = g.gz; b.gs0 = g.gs0;
    b.ckpt = reinterpret_cast<float*>(base + w.ckpt);
    b.part = reinterpret_cast<float*>(base + w.part);
    b.partA = reinterpret_cast<float*>(base + w.partA);
    b.partv = reinterpret_cast<float*>(base + w.partv);
    b.p.tiles = (a.D / a.G + S::DT - 1) / S::DT;
    b.slots = bwd_slots(a.nseq, b.p.tiles * a.G);
    cudaError_t e = launch_walk<T, N, S::CK>(a, b.p, s,
                                                    WalkBwd{g.gy, g.gz, reinterpret_cast<float*>(base + w.ckpt)});
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(ssm_reverse_kernel<T, N, S::L, S::CK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)K::SMEM);
    if (e != cudaSuccess) return e;
    ssm_reverse_kernel<T, N, S::L, S::CK><<<(unsigned)(b.slots * b.p.tiles * a.G), K::THREADS, K::SMEM, s>>>(b);
    ssm_bwd_bc_kernel<<<(unsigned)((a.tokens + 7) / 8), 256, 0, s>>>(b, g.gb, g.gc, N);
    ssm_bwd_params_kernel<<<(unsigned)(((long long)a.D * (N + 2) + 255) / 256), 256, 0, s>>>(b, g.gA, g.gskip,
                                                                                             g.gdt_bias, N);
    return cudaGetLastError();
}

}  // namespace mixer

size_t ssm_bwd_workspace(int nseq, int T, long long tokens, int D, int N, int G, bool varlen)
{
    using namespace mixer;
    return (N == 16 ? bwd_layout<16>(nseq, T, tokens, D, G, varlen)
                    : N == 32 ? bwd_layout<32>(nseq, T, tokens, D, G, varlen)
                              : bwd_layout<64>(nseq, T, tokens, D, G, varlen)).total;
}

cudaError_t ssm_bwd(const SsmArgs& a, const SsmGrads& g, void* ws, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    using namespace mixer;
    if (a.N == 16) return a.dtype == KDA_BF16 ? launch_bwd<bf, 16>(a, g, ws, s) : launch_bwd<float, 16>(a, g, ws, s);
    if (a.N == 32) return a.dtype == KDA_BF16 ? launch_bwd<bf, 32>(a, g, ws, s) : launch_bwd<float, 32>(a, g, ws, s);
    return a.dtype == KDA_BF16 ? launch_bwd<bf, 64>(a, g, ws, s) : launch_bwd<float, 64>(a, g, ws, s);
}

}  // namespace kda
