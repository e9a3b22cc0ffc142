// Gradients of the selective scan.  With dy0 = gy silu(z), a_t = exp(Delta_t A):
//   g_t = C_t dy0_t + a_{t+1} g_{t+1}                    (reverse recurrence)
//   dB_t = sum_d g_t Delta_t x_t,   dC_t = sum_d h_t dy0_t,   du_t = sum_n g_t B_t
//   w_t = g_t a_t h_{t-1},   dA = sum_t w_t Delta_t,   dDelta_t = sum_n w_t A + du_t x_t
//   dx_t = du_t Delta_t + skip dy0_t,   ddt_t = dDelta_t sigmoid(dt_t + bias)
//   dz_t = gy_t y0_t silu'(z_t),   dh_0 = a_0 g_0
// Four launches: the forward walk, which leaves the state before every CK-th token
// and forms dz where it has y0 anyway; the reverse walk, which recomputes CK states
// at a time into registers and runs the reverse recurrence over them; and two sums
// in a fixed order, of dB and dC over channel tiles and of dA, dskip and dbias over
// the blocks that share a channel.
//
// 2 x 4096 tokens x 2048 channels, N = 16, bf16: 183 + 401 + 25 + 2 us.  The floor is
// the exponentials, twice 72 us.  (dz and y0 in the reverse walk instead of the
// forward one: 509 us for its 411 of that time.)
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
    int arrivals;             // that complete a hand-over: 1 (2 in the self-test: none ever completes)
    long long timeout_cycles;
};

// Shape of the reverse walk.  A channel's N states lie on L lanes, NPT each, so a
// warp holds a set of DT channels; it takes TK tokens at a time and does so for
// the SETS sets of a tile of 32 channels one after the other, with the sums of dB
// and dC over the channels in registers.  W warps take turns along the sequence.
template <int N_, int W_ = N_ == 16 ? 12 : 8>
struct Rev {
    static constexpr int N = N_, L = N == 16 ? 4 : 8, NPT = N / L, DT = 32 / L, TK = 32 / NPT, TILE = 32;
    static constexpr int SETS = TILE / DT, W = W_, THREADS = 32 * W;
    static constexpr int BLOCKS = (N == 16 ? 12 : 8) / W;   // per SM
    static constexpr int VL = 2 * NPT / DT;                 // values of dB, dC of a token left to a lane
    static constexpr int EL = TK * DT / 2;                  // lanes with a pair of channels outside the walk
    static constexpr int DUROW = DT + 2, DYROW = DT + 2, SROW = 2 * DT, BQ = TK * N / 128;
    static constexpr int COPY = TK * N + (N == 64 ? 0 : N);   // elements from order to order of B, C: on other banks
    // floats of shared memory: per warp, and in all
    template <typename T>
    static constexpr int warp_floats()
    {
        return TK * (2 * DUROW + DYROW + SROW) + 2 * 4 * COPY * (int)sizeof(T) / 4;
    }
    template <typename T>
    static constexpr size_t smem()
    {
        return 4 * ((size_t)W * warp_floats<T>() + SETS * 32 * NPT + 2 * (size_t)W * SETS * 32 * NPT +
                    (size_t)W * SETS * EL * 4 + 2 * TILE) + 8 * W * SETS + 16;
    }
};

// The order of a lane's states.  The sums of dB and dC over a warp's channels
// halve the values at every step: a lane sends one half and keeps the other, and
// which half depends on its channel.  So that no value has to be selected, a lane
// holds state i ^ X of its NPT in place i, X from the bits of its channel: what it
// keeps is always in front.  (B and C are staged in four orders for that.)
template <int N>
struct Order {
    using K = Rev<N>;
    static constexpr int HI = K::NPT / 2;                           // the step between lanes 16 apart swaps halves
    static constexpr int LO = K::NPT / 4 ? (N == 16 ? 1 : K::NPT / 4) : 1;
    static constexpr int LOBIT = N == 16 ? 2 : 3;                   // the last step's lane bit
    __device__ __forceinline__ static int copy(int lane) { return (lane >> 4 & 1) * 2 + (lane >> LOBIT & 1); }
    __device__ __forceinline__ static constexpr int x_of(int copy) { return (copy >> 1) * HI + (copy & 1) * LO; }
};

// A quad of B or C with its elements in places ^ X (X's two low bits).
__device__ __forceinline__ uint2 permuted(const uint2& v, int X)
{
    uint2 r = (X & 2) ? make_uint2(v.y, v.x) : v;
    if (X & 1) r = make_uint2(__byte_perm(r.x, 0u, 0x1032), __byte_perm(r.y, 0u, 0x1032));
    return r;
}
__device__ __forceinline__ float4 permuted(const float4& v, int X)
{
    float4 r = (X & 2) ? make_float4(v.z, v.w, v.x, v.y) : v;
    if (X & 1) r = make_float4(r.y, r.x, r.w, r.z);
    return r;
}

// A lane's states in global memory (natural order), in its own order.
template <int P>
__device__ __forceinline__ void read_permuted(const float* p, f32x2 (&v)[P], int X)
{
#pragma unroll
    for (int n = 0; n < P; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(p + 2 * (n ^ (X >> 1)));
        v[n] = (X & 1) ? pack(f.y, f.x) : pack(f.x, f.y);
    }
}
template <int P>
__device__ __forceinline__ void write_permuted(float* p, const f32x2 (&v)[P], int X)
{
#pragma unroll
    for (int n = 0; n < P; ++n) {
        float a, b;
        unpack(v[n], a, b);
        *reinterpret_cast<float2*>(p + 2 * (n ^ (X >> 1))) = (X & 1) ? make_float2(b, a) : make_float2(a, b);
    }
}

__device__ __forceinline__ f32x2 add_shuffled(f32x2 keep, f32x2 send, int mask)
{
    return add2(keep, __shfl_xor_sync(0xffffffffu, send, mask));
}

// One token's dB (vb) and dC (vc) summed over the warp's channels; acc gets what is
// left to the lane: N = 16: one state of dB or (lane bit 3) dC; N = 32: one state of
// both; N = 64: two states of both.
__device__ __forceinline__ void sum_channels(const f32x2 (&vb)[2], const f32x2 (&vc)[2], int lane, float (&acc)[1])
{
    const f32x2 kb = add_shuffled(vb[0], vb[1], 16), kc = add_shuffled(vc[0], vc[1], 16);
    const bool up = lane & 8;
    float lo, hi;
    unpack(add_shuffled(up ? kc : kb, up ? kb : kc, 8), lo, hi);
    acc[0] += lo + __shfl_xor_sync(0xffffffffu, hi, 4);
}
__device__ __forceinline__ void sum_channels(const f32x2 (&vb)[2], const f32x2 (&vc)[2], int, float (&acc)[2])
{
    float lo, hi;
    unpack(add_shuffled(vb[0], vb[1], 16), lo, hi);
    acc[0] += lo + __shfl_xor_sync(0xffffffffu, hi, 8);
    unpack(add_shuffled(vc[0], vc[1], 16), lo, hi);
    acc[1] += lo + __shfl_xor_sync(0xffffffffu, hi, 8);
}
__device__ __forceinline__ void sum_channels(const f32x2 (&vb)[4], const f32x2 (&vc)[4], int, float (&acc)[4])
{
    float lo, hi;
    unpack(add_shuffled(add_shuffled(vb[0], vb[2], 16), add_shuffled(vb[1], vb[3], 16), 8), lo, hi);
    acc[0] += lo;
    acc[1] += hi;
    unpack(add_shuffled(add_shuffled(vc[0], vc[2], 16), add_shuffled(vc[1], vc[3], 16), 8), lo, hi);
    acc[2] += lo;
    acc[3] += hi;
}

// As in the forward walk, the warps of a block take turns, backwards in time: a
// warp recomputes the states of its TK tokens from the checkpoint before them,
// waits for the state gradient of the warp behind it (an mbarrier per warp and
// set), runs the chain g = C dy0 + a g', hands it on, and then forms everything
// else.  Sums over a channel's lanes (dx, dDelta) and over a warp's channels (dB,
// dC) are transposed reductions, many values at a time.
//
// Bound by issue: 30 instructions per warp and 32 (channel, state, token) in 63 % of
// the slots, 8.8 words per lane of shared memory.  12 warps of 168 registers and 4
// sets of 8 channels per warp: sums of dB and dC stay in registers over the sets (one
// set per warp: 1115 us in all for 647), and are formed without selects (435 -> 411 us).
// The warps take turns along one sequence; kNarrowTurns is about short ones.  N = 16 spills
// 12 bytes in bf16 and 16 in fp32, with four warps 44 and 32; N = 32 and 64 none.
template <typename T, int N, int W_>
__global__ void __launch_bounds__(Rev<N, W_>::THREADS, Rev<N, W_>::BLOCKS)
ssm_reverse_kernel(const BwdDev b)
{
    using K = Rev<N, W_>;
    constexpr int TK = K::TK, DT = K::DT, L = K::L, NPT = K::NPT, SETS = K::SETS, W = K::W, VL = K::VL, BQ = K::BQ;
    const SsmDev& p = b.p;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = lane / L, l = lane % L;
    float* base = reinterpret_cast<float*>(smem);
    float* sA = base + W * K::template warp_floats<T>();                 // [set][lane][NPT]
    float* sCarry = sA + SETS * 32 * NPT;                                // [warp][set][lane][NPT]
    float* sGA = sCarry + W * SETS * 32 * NPT;                           // the same: sums of dA
    float* sGP = sGA + W * SETS * 32 * NPT;                              // [warp][set][EL][4]: dskip, dbias of a pair
    float* sBias = sGP + W * SETS * K::EL * 4;                           // [channel of the tile]
    float* sSkip = sBias + K::TILE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sSkip + K::TILE);       // [warp][set]
    int* aborted = reinterpret_cast<int*>(bars + W * SETS);
    float* mine = base + w * K::template warp_floats<T>();
    float2* sDU = reinterpret_cast<float2*>(mine);                       // [token][channel]: Delta, u
    float* sDY = mine + 2 * TK * K::DUROW;                               // [token][channel]: dy0
    float* sS = sDY + TK * K::DYROW;                                     // [token][channel][2]: sums of g B, w A
    T* sB = reinterpret_cast<T*>(sS + TK * K::SROW);                     // [order][token][N]
    T* sC = sB + 4 * K::COPY;
    const int copy = Order<N>::copy(lane), X = Order<N>::x_of(copy);

    flag_bad_sequences(p.q);
    const int ntiles = p.tiles * p.G;
    const int tile = blockIdx.x % ntiles, slot = blockIdx.x / ntiles;
    const int Dg = p.D / p.G, g = tile / p.tiles, gt = tile % p.tiles, off = gt * K::TILE, c00 = g * Dg + off;
    const int sets = min(SETS, (Dg - off) / DT);   // D / G is a multiple of 8: whole sets

    for (int i = threadIdx.x; i < SETS * 32 * NPT; i += K::THREADS) {
        // [set][lane][place]
        const int ch = i / N, of = i / NPT % 32, n = i % N ^ Order<N>::x_of(Order<N>::copy(of));
        sA[i] = ch < sets * DT ? bounded_decay(p.A[(long long)(c00 + ch) * N + n]) : 0.f;
    }
    for (int i = threadIdx.x; i < W * SETS * 32 * NPT; i += K::THREADS) sGA[i] = 0.f;
    for (int i = threadIdx.x; i < W * SETS * K::EL * 4; i += K::THREADS) sGP[i] = 0.f;
    if (threadIdx.x < K::TILE) {
        const bool in = (int)threadIdx.x < sets * DT;
        sBias[threadIdx.x] = in && p.dt_bias ? p.dt_bias[c00 + threadIdx.x] : 0.f;
        sSkip[threadIdx.x] = in && p.skip ? p.skip[c00 + threadIdx.x] : 0.f;
    }
    if (threadIdx.x < W * SETS) sm100::mbar_init(bars + threadIdx.x, b.arrivals);
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
        float2 nh[NPT / 2];
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
#pragma unroll
            for (int n = 0; n < NPT / 2; ++n) nh[n] = *reinterpret_cast<const float2*>(cp + 2 * (n ^ (X >> 1)));
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
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int Xk = Order<N>::x_of(k), at = k * (K::COPY / 4) + (i ^ (Xk >> 2));
                    reinterpret_cast<Quad*>(sB)[at] = permuted(vb, Xk);
                    reinterpret_cast<Quad*>(sC)[at] = permuted(vc, Xk);
                }
            }
            float acc[TK][VL];
#pragma unroll
            for (int j = 0; j < TK; ++j)
#pragma unroll
                for (int v = 0; v < VL; ++v) acc[j][v] = 0.f;

            for (int o = 0; o < sets; ++o) {
                // the pair's elements
                const float2 x = widen(nx), z = widen(nz), raw = widen(ndt);
                float2 dy = ngy, v = raw, delta;
                const float2 bias = *reinterpret_cast<const float2*>(sBias + o * DT + ec);
                const int ch = c00 + o * DT + ec;
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
                for (int n = 0; n < NPT / 2; ++n) h0[n] = (X & 1) ? pack(nh[n].y, nh[n].x) : pack(nh[n].x, nh[n].y);
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
                    read_states(sB + copy * K::COPY + j * N + l * NPT, B);
                    read_states(sC + copy * K::COPY + j * N + l * NPT, C);
#pragma unroll
                    for (int n = 0; n < NPT / 2; ++n) {
                        a[j][n] = decay2(pack(du.x, du.x), mul2(A[n], pack(kLog2e, kLog2e)));
                        h[j][n] = fma2(a[j][n], j ? h[j > 0 ? j - 1 : 0][n] : h0[n], mul2(pack(du.y, du.y), B[n]));
                        q[j][n] = mul2(C[n], pack(d, d));
                    }
                }
                f32x2 cr[NPT / 2];
                if (r > 0) {
                    ok = sm100::mbar_wait_warp(bars + from * SETS + o, parity, aborted, b.timeout_cycles);
                    if (!ok) break;
                    read_states(sCarry + ((from * SETS + o) * 32 + lane) * NPT, cr);
                } else {
#pragma unroll
                    for (int n = 0; n < NPT / 2; ++n) cr[n] = 0ull;
                    if (b.gsT) read_permuted(b.gsT + srow + o * 32 * NPT, cr, X);
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
                    write_permuted(b.gs0 + srow + o * 32 * NPT, cr, X);
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
                        f32x2 B[NPT / 2], vb[NPT / 2], vc[NPT / 2], s1 = 0ull, s2 = 0ull;
                        read_states(sB + copy * K::COPY + j * N + l * NPT, B);
#pragma unroll
                        for (int n = 0; n < NPT / 2; ++n) {
                            vb[n] = mul2(q[j][n], pack(du.y, du.y));
                            vc[n] = mul2(h[j][n], pack(d, d));
                            s1 = n ? fma2(q[j][n], B[n], s1) : mul2(q[j][n], B[n]);
                            const f32x2 wt = mul2(a[j][n], j ? h[j > 0 ? j - 1 : 0][n] : h0[n]);
                            gA[n] = fma2(wt, pack(du.x, du.x), gA[n]);
                            s2 = n ? fma2(wt, A[n], s2) : mul2(wt, A[n]);
                        }
                        sum_channels(vb, vc, lane, acc[j]);
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
                    const float4 ss = *reinterpret_cast<const float4*>(sS + (et * DT + ec) * 2);   // of both channels
                    const float2 skip = *reinterpret_cast<const float2*>(sSkip + o * DT + ec);
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
            // dB, dC of the tile's channels
            const int n = l * NPT + X;
#pragma unroll
            for (int j = 0; j < TK; ++j) {
                if (t0 + j < len) {
                    float* o = b.part + (((long long)gt * p.q.tokens + first + t0 + j) * p.G + g) * 2 * N + n;
                    if constexpr (N == 16) {
                        o[(lane >> 3 & 1) * N] = acc[j][0];
                    } else if constexpr (N == 32) {
                        o[0] = acc[j][0];
                        o[N] = acc[j][1];
                    } else {
                        *reinterpret_cast<float2*>(o) = make_float2(acc[j][0], acc[j][1]);
                        *reinterpret_cast<float2*>(o + N) = make_float2(acc[j][2], acc[j][3]);
                    }
                }
            }
        }
        __syncthreads();   // the next sequence starts with every hand-over taken
    }

    // this block's sums over its tokens: the warps' sums in order
    for (int i = threadIdx.x; i < sets * 32 * NPT; i += K::THREADS) {
        float sum = 0.f;
        for (int v = 0; v < W; ++v) sum += sGA[v * SETS * 32 * NPT + i];
        const int n = i % N ^ Order<N>::x_of(Order<N>::copy(i / NPT % 32));
        b.partA[((long long)slot * p.D + c00 + i / N) * N + n] = sum;
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

// dB and dC of every token from the channel tiles' sums, a warp per token.  Rows of
// no sequence: zero, here and in gx, gdt, gz.  Bound by HBM: 67 MB of sums in 24 us
// for 64 tiles of 8192 tokens (2.8 TB/s: 32 columns need only one load per tile and
// lane, eight of them in flight).
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

// dA, dskip, dbias over the slots: 2 us.
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

// Turns along one sequence leave warps idle where it has few of them.  So up to
// kNarrowTurns rounds of turns, where the sequences fill the SMs all the same, a block
// has four warps, and an SM three (N = 16) or two of these.  All four launches,
// D = 1024, bf16, 12 or 8 warps against 4, us: N = 16, 256 x 32 tokens 633 / 395,
// 64 x 96 279 / 247, 32 x 256 303 / 309, 16 x 1024 591 / 670; N = 32, 64 x 64 340 / 307,
// 32 x 256 552 / 572; N = 64, 64 x 64 791 / 728, 32 x 256 1368 / 1425.  The host knows
// the mean length only: with one long sequence among short ones four warps cost (512 x
// 16 tokens and one of 8192 last 2232 / 2270, one of 4096 in the middle 1234 / 1643).
constexpr int kNarrowTurns = 2;

// Sequences are dealt to `slots` blocks per channel tile: enough to fill the 148 SMs
// several times, few enough that the partial sums of dA stay small.  (64 x 64 tokens x
// 1024 channels with 2, 4, 16 times 148 blocks of 12 warps: 238, 221, 233 us.)
struct BwdShape {
    bool narrow;
    int slots;
};
static BwdShape bwd_shape(int nseq, long long tokens, int ntiles, int N)
{
    const int wide = N == 16 ? 12 : 8, per_sm = wide / 4, tk = N == 64 ? 4 : 8;
    BwdShape s;
    s.narrow = tokens / nseq <= kNarrowTurns * wide * tk && (long long)nseq * ntiles >= 148LL * per_sm;
    const int want = (148 * 4 * (s.narrow ? per_sm : 1) + ntiles - 1) / ntiles;
    s.slots = nseq < want ? nseq : want;
    return s;
}

struct BwdWorkspace {
    size_t ckpt, part, partA, partv, total;
};

template <int N>
static BwdWorkspace bwd_layout(int nseq, int T, long long tokens, int D, int G, bool varlen)
{
    using K = Rev<N>;
    const int tiles = (D / G + K::TILE - 1) / K::TILE, slots = bwd_shape(nseq, tokens, tiles * G, N).slots;
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

template <typename T, int N, int W>
static cudaError_t launch_reverse(const BwdDev& b, cudaStream_t s)
{
    using K = Rev<N, W>;
    constexpr size_t smem = K::template smem<T>();
    static_assert(smem <= 227 * 1024 && K::BLOCKS * (smem + 1024) <= 228 * 1024, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(ssm_reverse_kernel<T, N, W>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ssm_reverse_kernel<T, N, W><<<(unsigned)(b.slots * b.p.tiles * b.p.G), K::THREADS, smem, s>>>(b);
    return cudaGetLastError();
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
    const BwdShape shape = bwd_shape(a.nseq, a.tokens, b.p.tiles * a.G, N);
    b.slots = shape.slots;
    b.arrivals = 1;
    b.timeout_cycles = kBwdTimeoutCycles;
    cudaError_t e = launch_walk<T, N, K::TK>(a, b.p, s,
                                                    WalkBwd{g.gy, g.gz, reinterpret_cast<float*>(base + w.ckpt)});
    if (e != cudaSuccess) return e;
    e = shape.narrow ? launch_reverse<T, N, 4>(b, s) : launch_reverse<T, N, K::W>(b, s);
    if (e != cudaSuccess) return e;
    ssm_bwd_bc_kernel<<<(unsigned)((a.tokens + 7) / 8), 256, 0, s>>>(b, g.gb, g.gc, N);
    ssm_bwd_params_kernel<<<(unsigned)(((long long)a.D * (N + 2) + 255) / 256), 256, 0, s>>>(b, g.gA, g.gskip,
                                                                                             g.gdt_bias, N);
    return cudaGetLastError();
}

// The reverse walk over one sequence of kTestTokens tokens and one tile of channels,
// all zeros, with every hand-over withheld: each warp's wait runs out, and the block
// leaves through its common exit.
constexpr int kTestTokens = 100, kTestD = 32, kTestN = 16;
constexpr int kTestZeros = (kTestTokens / 8 + 1) * kTestD * kTestN;   // floats of any input, the states the longest

template <int W>
static cudaError_t launch_reverse_withheld(float* ws, long long limit_cycles, cudaStream_t s)
{
    BwdDev b{};
    float* out = ws + kTestZeros;
    b.p.x = b.p.dt = b.p.b = b.p.c = b.p.A = b.gy = b.ckpt = ws;
    b.p.ldx = b.p.lddt = 4 * kTestD;
    b.p.ldb = b.p.ldc = 4 * kTestN;
    b.p.q = Seqs{nullptr, 1, kTestTokens, kTestTokens};
    b.p.D = kTestD;
    b.p.G = b.p.tiles = b.slots = 1;
    b.gx = out; out += kTestTokens * kTestD;
    b.gdt = out; out += kTestTokens * kTestD;
    b.part = out; out += kTestTokens * 2 * kTestN;
    b.partA = out; out += kTestD * kTestN;
    b.partv = out;
    b.arrivals = 2;
    b.timeout_cycles = limit_cycles;
    return launch_reverse<float, kTestN, W>(b, s);
}

}  // namespace mixer

size_t ssm_bwd_selftest_workspace()
{
    using namespace mixer;
    return sizeof(float) * (kTestZeros + kTestTokens * 2 * (kTestD + kTestN) + kTestD * (kTestN + 2));
}

cudaError_t ssm_bwd_selftest(long long limit_cycles, void* ws, cudaStream_t s)
{
    float* f = static_cast<float*>(ws);
    cudaError_t e = cudaMemsetAsync(f, 0, mixer::kTestZeros * sizeof(float), s);
    if (e == cudaSuccess) e = mixer::launch_reverse_withheld<mixer::Rev<mixer::kTestN>::W>(f, limit_cycles, s);
    if (e == cudaSuccess) e = mixer::launch_reverse_withheld<4>(f, limit_cycles, s);
    return e;
}

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
