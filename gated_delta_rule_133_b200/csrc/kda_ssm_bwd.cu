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
#include "kda_sm100.cuh"
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
    long long timeout_cycles;
};

// Shape of the reverse walk.  A channel's N states lie on L lanes, NPT each, so a
// warp holds a set of DT channels; it takes TK tokens at a time and does so for
// the SETS sets of a tile of 32 channels one after the other, with the sums of dB
// and dC over the channels in registers.  W warps take turns along the sequence.
template <int N_>
struct Rev {
    static constexpr int N = N_, L = N == 16 ? 4 : 8, NPT = N / L, DT = 32 / L, TK = 32 / NPT, TILE = 32;
    static constexpr int SETS = TILE / DT, W = N == 64 ? 8 : 12, THREADS = 32 * W;
    static constexpr int V = 2 * NPT, VL = V / DT;          // values of dB, dC per token: of a lane, left to a lane
    static constexpr int EL = TK * DT / 2;                  // lanes with a pair of channels outside the walk
    static constexpr int DUROW = DT + 2, DYROW = DT + 2, BQ = TK * N / 128;
    // floats of shared memory: per warp, and in all
    template <typename T>
    static constexpr int warp_floats()
    {
        return TK * (2 * DUROW + DYROW + 2 * DT) + 2 * TK * N * (int)sizeof(T) / 4;
    }
    template <typename T>
    static constexpr size_t smem()
    {
        return 4 * ((size_t)W * warp_floats<T>() + SETS * 32 * NPT + 2 * (size_t)W * SETS * 32 * NPT +
                    (size_t)W * SETS * EL * 4) + 8 * W * SETS + 16;
    }
};

// As in the forward walk, the warps of a block take turns, backwards in time: a
// warp recomputes the states of its TK tokens from the checkpoint before them,
// waits for the state gradient of the warp behind it (an mbarrier per warp and
// set), runs the chain g = C dy0 + a g', hands it on, and then forms everything
// else.  Sums over a channel's lanes (dx, dDelta) and over a warp's channels (dB,
// dC) are transposed reductions, many values at a time.
template <typename T, int N>
__global__ void __launch_bounds__(Rev<N>::THREADS, 1)
ssm_reverse_kernel(const BwdDev b)
{
    using K = Rev<N>;
    constexpr int TK = K::TK, DT = K::DT, L = K::L, NPT = K::NPT, SETS = K::SETS, W = K::W, VL = K::VL, BQ = K::BQ;
    const SsmDev& p = b.p;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = lane / L, l = lane % L;
    float* base = reinterpret_cast<float*>(smem);
    float* sA = base + W * K::template warp_floats<T>();                 // [set][lane][NPT]
    float* sCarry = sA + SETS * 32 * NPT;                                // [warp][set][lane][NPT]
    float* sGA = sCarry + W * SETS * 32 * NPT;                           // the same: sums of dA
    float* sGP = sGA + W * SETS * 32 * NPT;                              // [warp][set][EL][4]: dskip, dbias of a pair
    uint64_t* bars = reinterpret_cast<uint64_t*>(sGP + W * SETS * K::EL * 4);   // [warp][set]
    int* aborted = reinterpret_cast<int*>(bars + W * SETS);
    float* mine = base + w * K::template warp_floats<T>();
    float2* sDU = reinterpret_cast<float2*>(mine);                       // [token][channel]: Delta, u
    float* sDY = mine + 2 * TK * K::DUROW;                               // [token][channel]: dy0
    float* sS = sDY + TK * K::DYROW;                                     // [token][channel][2]: sums of g B, w A
    T* sB = reinterpret_cast<T*>(sS + 2 * TK * DT);                      // [token][N]
    T* sC = sB + TK * N;

    flag_bad_sequences(p.q);
    const int ntiles = p.tiles * p.G;
    const int tile = blockIdx.x % ntiles, slot = blockIdx.x / ntiles;
    const int Dg = p.D / p.G, g = tile / p.tiles, gt = tile % p.tiles, off = gt * K::TILE, c00 = g * Dg + off;
    const int sets = min(SETS, (Dg - off) / DT);   // D / G is a multiple of 8: whole sets

    for (int i = threadIdx.x; i < SETS * 32 * NPT; i += K::THREADS) {
        const int ch = i / N;   // [set][channel][N] is the same order as [set][lane][NPT]
        sA[i] = ch < sets * DT ? p.A[(long long)(c00 + ch) * N + i % N] : 0.f;
    }
    for (int i = threadIdx.x; i < W * SETS * 32 * NPT; i += K::THREADS) sGA[i] = 0.f;
    for (int i = threadIdx.x; i < W * SETS * K::EL * 4; i += K::THREADS) sGP[i] = 0.f;
    if (threadIdx.x < W * SETS) sm100::mbar_init(bars + threadIdx.x, 1);
    if (threadIdx.x == 0) {
        *aborted = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    const bool gated = p.z != nullptr, el = lane < K::EL;
    const int et = lane / (DT / 2), ec = lane % (DT / 2) * 2;   // the lane's pair outside the walk: token, channel of the set
    const int from = (w + W - 1) % W;
    unsigned parity = 0;
    bool ok = true;   // no wait has run out
    typedef typename Raw<T>::pair Pair;
    typedef typename Raw<T>::quad Quad;

    for (int seq = slot; seq < p.q.n; seq += b.slots) {
        const long long s = p.q.begin(seq);
        long long e = p.q.begin(seq + 1);
        if (e < s || !Seqs::inside(s, e, p.q.tokens)) e = s;
        const int len = (int)(e - s), nb = (len + TK - 1) / TK, first = (int)s;
        const long long ckpt0 = ckpt_base<TK>(p.q, seq, s);
        const long long srow = ((long long)seq * p.D + c00) * N + lane * NPT;   // + set * 32 * NPT
        if (nb == 0 && b.gs0 && w == 0) {
            for (int o = 0; o < sets; ++o)
#pragma unroll
                for (int n = 0; n < NPT; ++n)
                    b.gs0[srow + o * 32 * NPT + n] = b.gsT ? b.gsT[srow + o * 32 * NPT + n] : 0.f;
        }

        Pair nx, ndt, nz;
        float2 ngy;
        f32x2 nh[NPT / 2];
        auto fetch = [&](int blk, int o) {   // set o of block blk (blk < 0: none left)
            nx = ndt = nz = Pair{};
            ngy = make_float2(0.f, 0.f);
            if (blk < 0) return;
            const int ch = c00 + o * DT + ec;
            if (el && blk * TK + et < len) {
                const unsigned t = first + blk * TK + et;
                nx = *reinterpret_cast<const Pair*>(row<T>(p.x, t, p.ldx) + ch);
                ndt = *reinterpret_cast<const Pair*>(row<T>(p.dt, t, p.lddt) + ch);
                if (gated) nz = *reinterpret_cast<const Pair*>(row<T>(p.z, t, p.ldz) + ch);
                ngy = *reinterpret_cast<const float2*>(row<float>(b.gy, t, 4u * p.D) + ch);
            }
            const float* cp = b.ckpt + ((ckpt0 + blk) * p.D + c00 + o * DT) * N + lane * NPT;
            read_states(cp, nh);
        };
        if (w < nb) fetch(nb - 1 - w, 0);

        for (int r = w; ok && r < nb; r += W) {
            const int blk = nb - 1 - r, t0 = blk * TK;
            __syncwarp();
#pragma unroll
            for (int q = 0; q < BQ; ++q) {
                const int i = q * 32 + lane, t = t0 + i / (N / 4), n = g * N + i % (N / 4) * 4;
                Quad vb{}, vc{};
                if (t < len) {
                    vb = *reinterpret_cast<const Quad*>(row<T>(p.b, first + t, p.ldb) + n);
                    vc = *reinterpret_cast<const Quad*>(row<T>(p.c, first + t, p.ldc) + n);
                }
                reinterpret_cast<Quad*>(sB)[i] = vb;
                reinterpret_cast<Quad*>(sC)[i] = vc;
            }
            float acc[TK][VL];
#pragma unroll
            for (int j = 0; j < TK; ++j)
#pragma unroll
                for (int v = 0; v < VL; ++v) acc[j][v] = 0.f;

            for (int o = 0; o < sets; ++o) {
                // the pair's elements
                const float2 x = widen(nx), z = widen(nz), raw = widen(ndt);
                float2 dy = ngy, v = raw, bias = make_float2(0.f, 0.f), delta;
                const int ch = c00 + o * DT + ec;
                if (p.dt_bias && el) bias = *reinterpret_cast<const float2*>(p.dt_bias + ch);
                v.x += bias.x;
                v.y += bias.y;
                delta = v;
                if (p.softplus) unpack(softplus2(v.x, v.y), delta.x, delta.y);
                if (t0 + et >= len) delta = make_float2(0.f, 0.f);   // (x and gy are zero there)
                if (gated) {
                    dy.x *= silu(z.x);
                    dy.y *= silu(z.y);
                }
                f32x2 h0[NPT / 2];
#pragma unroll
                for (int n = 0; n < NPT / 2; ++n) h0[n] = nh[n];
                if (el) {
                    *reinterpret_cast<float4*>(&sDU[et * K::DUROW + ec]) =
                        make_float4(delta.x, delta.x * x.x, delta.y, delta.y * x.y);
                    *reinterpret_cast<float2*>(&sDY[et * K::DYROW + ec]) = dy;
                }
                __syncwarp();
                fetch(o + 1 < sets ? blk : blk - W, o + 1 < sets ? o + 1 : 0);

                f32x2 A[NPT / 2], a[TK][NPT / 2], h[TK][NPT / 2], q[TK][NPT / 2];
                read_states(sA + (o * 32 + lane) * NPT, A);
#pragma unroll
                for (int j = 0; j < TK; ++j) {
                    const float2 du = sDU[j * K::DUROW + c];
                    const float d = sDY[j * K::DYROW + c];
                    f32x2 B[NPT / 2], C[NPT / 2];
                    read_states(sB + j * N + l * NPT, B);
                    read_states(sC + j * N + l * NPT, C);
#pragma unroll
                    for (int n = 0; n < NPT / 2; ++n) {
                        a[j][n] = decay2(pack(du.x, du.x), mul2(A[n], pack(kLog2e, kLog2e)));
                        h[j][n] = fma2(a[j][n], j ? h[j > 0 ? j - 1 : 0][n] : h0[n], mul2(pack(du.y, du.y), B[n]));
                        q[j][n] = mul2(C[n], pack(d, d));
                    }
                }
                f32x2 cr[NPT / 2];
                if (r > 0) {
                    ok = sm100::mbar_wait(bars + from * SETS + o, parity, aborted, b.timeout_cycles);
                    if (!ok) break;
                    read_states(sCarry + ((from * SETS + o) * 32 + lane) * NPT, cr);
                } else {
#pragma unroll
                    for (int n = 0; n < NPT / 2; ++n)
                        cr[n] = b.gsT ? *reinterpret_cast<const f32x2*>(b.gsT + srow + o * 32 * NPT + 2 * n) : 0ull;
                }
                // q becomes g, and a the gradient handed to the token before: a g
#pragma unroll
                for (int j = TK - 1; j >= 0; --j)
#pragma unroll
                    for (int n = 0; n < NPT / 2; ++n) {
                        q[j][n] = add2(q[j][n], cr[n]);
                        cr[n] = a[j][n] = mul2(a[j][n], q[j][n]);
                    }
                if (blk > 0) {
                    write_states(sCarry + ((w * SETS + o) * 32 + lane) * NPT, cr);
                    __syncwarp();
                    if (lane == 0) sm100::mbar_arrive(bars + w * SETS + o);
                } else if (b.gs0) {
#pragma unroll
                    for (int n = 0; n < NPT / 2; ++n) *reinterpret_cast<f32x2*>(b.gs0 + srow + o * 32 * NPT + 2 * n) = cr[n];
                }

                f32x2 gA[NPT / 2];
                read_states(sGA + ((w * SETS + o) * 32 + lane) * NPT, gA);
                constexpr int GT = L / 2;   // tokens whose two sums fill the channel's lanes
#pragma unroll
                for (int jg = 0; jg < TK; jg += GT) {
                    float sums[L];
#pragma unroll
                    for (int jj = 0; jj < GT; ++jj) {
                        const int j = jg + jj;
                        const float2 du = sDU[j * K::DUROW + c];
                        const float d = sDY[j * K::DYROW + c];
                        f32x2 B[NPT / 2], s1 = 0ull, s2 = 0ull;
                        read_states(sB + j * N + l * NPT, B);
                        float val[K::V];
#pragma unroll
                        for (int n = 0; n < NPT / 2; ++n) {
                            unpack(mul2(q[j][n], pack(du.y, du.y)), val[2 * n], val[2 * n + 1]);
                            unpack(mul2(h[j][n], pack(d, d)), val[NPT + 2 * n], val[NPT + 2 * n + 1]);
                            s1 = n ? fma2(q[j][n], B[n], s1) : mul2(q[j][n], B[n]);
                            const f32x2 wt = mul2(a[j][n], j ? h[j > 0 ? j - 1 : 0][n] : h0[n]);
                            gA[n] = fma2(wt, pack(du.x, du.x), gA[n]);
                            s2 = n ? fma2(wt, A[n], s2) : mul2(wt, A[n]);
                        }
                        reduce_transposed<K::V, DT, L>(val, lane);
#pragma unroll
                        for (int k = 0; k < VL; ++k) acc[j][k] += val[k];
                        float lo, hi;
                        unpack(s1, lo, hi);
                        sums[2 * jj] = lo + hi;
                        unpack(s2, lo, hi);
                        sums[2 * jj + 1] = lo + hi;
                    }
                    reduce_transposed<L, L, 1>(sums, lane);
                    sS[((jg + l / 2) * DT + c) * 2 + (l & 1)] = sums[0];
                }
                write_states(sGA + ((w * SETS + o) * 32 + lane) * NPT, gA);
                __syncwarp();
                if (el && t0 + et < len) {
                    const float4 ss = *reinterpret_cast<const float4*>(sS + (et * DT + ec) * 2);   // s1, s2 of both channels
                    float2 skip = make_float2(0.f, 0.f);
                    if (p.skip) skip = *reinterpret_cast<const float2*>(p.skip + ch);
                    const unsigned t = first + t0 + et;
                    float2 gx, gd;
                    gx.x = fmaf(ss.x, delta.x, skip.x * dy.x);
                    gx.y = fmaf(ss.z, delta.y, skip.y * dy.y);
                    gd.x = fmaf(ss.x, x.x, ss.y) * (p.softplus ? sigmoid(v.x) : 1.f);
                    gd.y = fmaf(ss.z, x.y, ss.w) * (p.softplus ? sigmoid(v.y) : 1.f);
                    *reinterpret_cast<float2*>(row<float>(b.gx, t, 4u * p.D) + ch) = gx;
                    *reinterpret_cast<float2*>(row<float>(b.gdt, t, 4u * p.D) + ch) = gd;
                    float4* gp = reinterpret_cast<float4*>(sGP + ((w * SETS + o) * K::EL + lane) * 4);
                    float4 f = *gp;
                    f.x = fmaf(dy.x, x.x, f.x);
                    f.y = fmaf(dy.y, x.y, f.y);
                    f.z += gd.x;
                    f.w += gd.y;
                    *gp = f;
                }
                __syncwarp();   // the warp's arrays are free
            }
            if (!ok) break;
            if (r > 0) parity ^= 1u;
            // dB, dC of the tile's channels: values i0 .. of (dB, dC) x NPT states
            const int i0 = lane / L * VL, col = i0 / NPT * N + l * NPT + i0 % NPT;
#pragma unroll
            for (int j = 0; j < TK; ++j) {
                if (t0 + j < len) {
                    float* o = b.part + (((long long)gt * p.q.tokens + first + t0 + j) * p.G + g) * 2 * N + col;
#pragma unroll
                    for (int k = 0; k < VL; ++k) o[k] = acc[j][k];
                }
            }
        }
        __syncthreads();   // the next sequence starts with every hand-over taken
    }

    // this block's sums over its tokens: the warps' sums in order
    for (int i = threadIdx.x; i < sets * 32 * NPT; i += K::THREADS) {
        float sum = 0.f;
        for (int v = 0; v < W; ++v) sum += sGA[v * SETS * 32 * NPT + i];
        b.partA[((long long)slot * p.D + c00) * N + i] = sum;
    }
    for (int i = threadIdx.x; i < sets * DT * 2; i += K::THREADS) {
        const int ch = i / 2, which = i % 2, o = ch / DT, cc = ch % DT;
        float sum = 0.f;
        for (int v = 0; v < W; ++v)
            for (int t = 0; t < TK; ++t)
                sum += sGP[((v * SETS + o) * K::EL + t * (DT / 2) + cc / 2) * 4 + which * 2 + cc % 2];
        b.partv[((long long)slot * 2 + which) * p.D + c00 + ch] = sum;
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

// Budget of a wait for the next warp's state, in SM clock cycles (about a second).
constexpr long long kBwdTimeoutCycles = 1LL << 31;

// Sequences are dealt to this many blocks per channel tile: enough to fill the
// 148 SMs several times, few enough that the partial sums of dA stay small.
static int bwd_slots(int nseq, int ntiles)
{
    const int want = (148 * 4 + ntiles - 1) / ntiles;
    return nseq < want ? nseq : want;
}

struct BwdWorkspace {
    size_t ckpt, part, partA, partv, total;
};

template <int N>
static BwdWorkspace bwd_layout(int nseq, int T, long long tokens, int D, int G, bool varlen)
{
    using K = Rev<N>;
    const int tiles = (D / G + K::TILE - 1) / K::TILE, slots = bwd_slots(nseq, tiles * G);
    const size_t blocks = varlen ? (size_t)(tokens / K::TK) + nseq : (size_t)nseq * ((T + K::TK - 1) / K::TK);
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
    using K = Rev<N>;
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
    b.p.tiles = (a.D / a.G + K::TILE - 1) / K::TILE;
    b.slots = bwd_slots(a.nseq, b.p.tiles * a.G);
    b.timeout_cycles = kBwdTimeoutCycles;
    cudaError_t e = launch_walk<T, N, K::TK>(a, b.p, s,
                                                    WalkBwd{g.gy, g.gz, reinterpret_cast<float*>(base + w.ckpt)});
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(ssm_reverse_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)K::template smem<T>());
    if (e != cudaSuccess) return e;
    ssm_reverse_kernel<T, N><<<(unsigned)(b.slots * b.p.tiles * a.G), K::THREADS, K::template smem<T>(), s>>>(b);
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
