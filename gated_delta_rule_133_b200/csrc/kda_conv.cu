// Short causal depthwise convolution of W = 2..4 taps with an optional SiLU:
//   pre[t, d] = bias[d] + sum_j w[d, j] x[t - W + 1 + j, d],   y = pre or silu(pre)
// over dense or packed sequences, as a step of one token per sequence, and its
// gradients.  A sequence's tokens before its first one come from its state: the
// last W - 1 inputs, in the inputs' type (they are copies of inputs).
//
// Every path is bound by HBM: each input element is read once and each output
// element written once (plus a halo of W - 1 rows per token tile, which the L2
// holds).  A thread owns four channels and walks a tile of tokens with the last
// W - 1 rows and the weights in registers, so no shared memory or synchronisation
// is needed and the loads of the next tokens are in flight together.
//
// Measured (bf16 in and out, W = 4, SiLU; here and below calls in a captured graph over
// tensors of 600 MB in all, so out of the L2): 65536 x 2048 in 109 us, 4.9 TB/s of 6.55
// of a copy; 16384 x 2048 in 31.9 us, 8192 x 2048 in 19.1, 4096 x 2048 in 11.2: about
// 6 us and then 5.2 TB/s.  Eight channels per thread halve the requests but need 198
// registers and half the warps: 320 us where four take 209.  Blocks of one token tile in
// a row instead of one channel block: the same.
#include "kda_mixer.cuh"

namespace kda {
namespace mixer {

constexpr int kV = 4;   // channels per thread

template <int W, int V>
__device__ __forceinline__ void load_taps(const float* __restrict__ w, const float* __restrict__ bias, int c,
                                          float (&wt)[W][V], float (&bv)[V])
{
    float flat[V * W];
    load_vec<V * W>(w + (size_t)c * W, flat);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) wt[j][v] = flat[v * W + j];
        bv[v] = 0.f;
    }
    if (bias) load_vec<V>(bias + c, bv);
}

// Row `pos` (relative to the sequence's first token, >= -(W - 1)) of one
// sequence: a token, a row of its initial state, or zero.
template <typename T, int W, int V>
__device__ __forceinline__ void load_row(const T* __restrict__ x, long long ldx, const T* __restrict__ s0,
                                         long long begin, int seq, long long pos, int D, int c, float (&out)[V])
{
    if (pos >= 0) {
        load_vec<V>(x + (begin + pos) * ldx + c, out);
    } else if (s0) {
        load_vec<V>(s0 + ((long long)seq * (W - 1) + pos + W - 1) * D + c, out);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = 0.f;
    }
}

// Final state of sequence i: its last W - 1 inputs, of which the first come
// from its initial state when it has fewer tokens.  All rows are read before
// any is written, so the final state may be the initial one's memory.
template <typename T, int W>
__device__ __forceinline__ void write_state(const T* __restrict__ x, long long ldx, const T* s0, T* sT,
                                            const Seqs& q, int i, int D, int c)
{
    typedef typename Raw<T>::quad Quad;
    long long s = q.begin(i), e = q.begin(i + 1);
    if (e < s || !Seqs::inside(s, e, q.tokens)) e = s;
    Quad rows[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const long long pos = e - s - (W - 1) + j;
        rows[j] = Quad{};
        if (pos >= 0)
            rows[j] = *reinterpret_cast<const Quad*>(x + (s + pos) * ldx + c);
        else if (s0)
            rows[j] = *reinterpret_cast<const Quad*>(s0 + ((long long)i * (W - 1) + pos + W - 1) * D + c);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) *reinterpret_cast<Quad*>(sT + ((long long)i * (W - 1) + j) * D + c) = rows[j];
}

template <typename T, int W>
__global__ void __launch_bounds__(128)
conv_state_kernel(const T* __restrict__ x, long long ldx, const T* s0, T* sT, Seqs q, int D)
{
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * kV;
    if (c < D) write_state<T, W>(x, ldx, s0, sT, q, blockIdx.x, D, c);
}

// The taps as pairs of channels.
template <int W>
__device__ __forceinline__ void load_taps2(const float* __restrict__ w, const float* __restrict__ bias, int c,
                                           f32x2 (&wt)[W][2], f32x2 (&bv)[2])
{
    float f[W][kV], g[kV];
    load_taps<W, kV>(w, bias, c, f, g);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) wt[j][v] = pack(f[j][2 * v], f[j][2 * v + 1]);
        bv[v] = pack(g[2 * v], g[2 * v + 1]);
    }
}

template <bool SILU, typename TO>
__device__ __forceinline__ void put(TO* y, const f32x2 (&p)[2])
{
    float out[kV];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        unpack(p[v], out[2 * v], out[2 * v + 1]);
        if (SILU) unpack(silu2(out[2 * v], out[2 * v + 1]), out[2 * v], out[2 * v + 1]);
    }
    store_vec<kV>(y, out);
}

// Grid: x = token tiles of R tokens, then (if sT) one block per sequence for
// the final states; y = channel blocks.  A token is loaded U tokens before it is
// summed (16384 x 2048: 31.5 us; U loaded, then summed, six blocks per SM instead of
// five: 32.7; U = 8 with six or seven blocks 33.9, 35.8, U = 4 with eight 32.4, but
// 11.9 instead of 10.2 at 4096 x 2048).
template <typename T, typename TO, int W, bool SILU>
__global__ void __launch_bounds__(128, 5)
conv_fwd_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                const T* s0, TO* __restrict__ y, T* sT, Seqs q, int D, int R, int ntiles)
{
    // 16 registers; fp32 with 8: 65536 x 2048 206 us for 175 (spills).  bf16 with SiLU spills a
    // little at this bound: 4 bytes with 4 taps, 4, 20 and 32 with 2, 3 and 4 taps into fp32
    // (139 us, 5.8 TB/s).
    constexpr int U = sizeof(T) == 2 ? 8 : 4;
    typedef typename Raw<T>::quad Quad;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * kV;
    flag_bad_sequences(q);   // by every block: the sequences are dealt to the whole grid
    if ((int)blockIdx.x >= ntiles) {
        if (c < D) write_state<T, W>(x, ldx, s0, sT, q, blockIdx.x - ntiles, D, c);
        return;
    }
    long long t = (long long)blockIdx.x * R;
    const long long t1 = min(t + R, q.tokens);
    int i = max(find_sequence(q, t), 0);
    if (c >= D) return;

    f32x2 wt[W][2], bv[2];
    load_taps2<W>(w, bias, c, wt, bv);
    for (; i < q.n && t < t1; ++i) {
        const long long s = q.begin(i), e = q.begin(i + 1);
        if (e <= t || e <= s) continue;
        if (s > t) t = s;
        if (t >= t1) break;
        const long long stop = min(e, t1);
        if (!Seqs::inside(s, e, q.tokens)) {
            t = max(t, stop);
            continue;
        }
        f32x2 win[W - 1][2];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            float f[kV];
            load_row<T, W, kV>(x, ldx, s0, s, i, t - s - (W - 1) + j, D, c, f);
            win[j][0] = pack(f[0], f[1]);
            win[j][1] = pack(f[2], f[3]);
        }
        const T* px = x + t * ldx + c;
        TO* py = y + t * D + c;
        auto step = [&](const Quad& raw) {
            f32x2 xv[2], p[2];
            widen(raw, xv);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                p[v] = fma2(wt[W - 1][v], xv[v], bv[v]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) p[v] = fma2(wt[j][v], win[j][v], p[v]);
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
                win[W - 2][v] = xv[v];
            }
            put<SILU>(py, p);
            py += D;
        };
        int n = (int)(stop - t);
        if (n >= U) {
            Quad next[U];
#pragma unroll
            for (int u = 0; u < U; ++u, px += ldx) next[u] = *reinterpret_cast<const Quad*>(px);
#pragma unroll 1
            for (; n >= 2 * U; n -= U) {
#pragma unroll
                for (int u = 0; u < U; ++u, px += ldx) {
                    const Quad raw = next[u];
                    next[u] = *reinterpret_cast<const Quad*>(px);
                    step(raw);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) step(next[u]);
            n -= U;
        }
#pragma unroll 1
        for (; n > 0; --n, px += ldx) step(*reinterpret_cast<const Quad*>(px));
        t = stop;
    }
}

// One token per sequence: y from the state's rows and x; the state moves up by
// one row.  A thread owns a channel vector of RN sequences, so that the weights
// are read once for them and all their rows are in flight together.  bf16, W = 4: 1024 x
// 4096 in 13.2 us for 67.1 MB, 5.1 TB/s, 4096 x 4096 46.4 us, 5.8 TB/s; 16 sequences:
// 2.4 us, a launch.
template <typename T, typename TO, int W, bool SILU, int RN>
__global__ void __launch_bounds__(128)
conv_step_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                 T* __restrict__ state, TO* __restrict__ y, int n, int D)
{
    typedef typename Raw<T>::quad Quad;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * kV;
    if (c >= D) return;
    const int i0 = blockIdx.x * RN;
    Quad raw[RN][W];
#pragma unroll
    for (int r = 0; r < RN; ++r) {
        if (i0 + r < n) {
            const T* st = state + (long long)(i0 + r) * (W - 1) * D + c;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) raw[r][j] = *reinterpret_cast<const Quad*>(st + (long long)j * D);
            raw[r][W - 1] = *reinterpret_cast<const Quad*>(x + (i0 + r) * ldx + c);
        }
    }
    f32x2 wt[W][2], bv[2];
    load_taps2<W>(w, bias, c, wt, bv);
#pragma unroll
    for (int r = 0; r < RN; ++r) {
        if (i0 + r < n) {
            T* st = state + (long long)(i0 + r) * (W - 1) * D + c;
            f32x2 p[2] = {bv[0], bv[1]};
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                f32x2 xv[2];
                widen(raw[r][j], xv);
                p[0] = fma2(wt[j][0], xv[0], p[0]);
                p[1] = fma2(wt[j][1], xv[1], p[1]);
                if (j > 0) *reinterpret_cast<Quad*>(st + (long long)(j - 1) * D) = raw[r][j];
            }
            put<SILU>(y + (long long)(i0 + r) * D + c, p);
        }
    }
}

// ---------------------------------------------------------------- backward
// With dpre = gy silu'(pre):  gx[p] = sum_j w[j] dpre[p + W - 1 - j] (tokens of
// the same sequence), plus the final state's gradient for the last W - 1 rows;
// gw[j] = sum_t dpre[t] x[t - W + 1 + j];  gb = sum_t dpre[t].
// A tile walks its R tokens and the W - 1 after them (whose dpre it needs for
// its own gx but does not add to gw and gb).  gw and gb of a tile go to a
// partial sum of its own, part[tile][j][D] (j = W: the bias), which a second
// kernel adds in a fixed order: no atomics, the same result every time.
//
// Ten bytes per element (x in bf16, gy, gx in fp32), so HBM is the bound; what it
// reaches is set by the loads in flight: four blocks of 128 registers per SM, and
// every token's loads issued U tokens before they are used.  Both kernels: 8192 x 2048
// 44 us, 3.8 TB/s; 65536 x 2048 271 us, 4.9 TB/s (with loads and sums in turn 48 and
// 313; without the bound of 128 registers 56 and 280; five blocks 82 and 476).  At that
// bound 4 taps with SiLU spill 116 bytes in bf16 and 32 in fp32.  Two
// channels per thread, tiles staged in shared memory by cp.async, and channel blocks
// first in the grid measured slower.
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(128, 4)
conv_bwd_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                const T* __restrict__ s0, const float* __restrict__ gy, const float* __restrict__ gsT,
                float* __restrict__ gx, float* __restrict__ part, Seqs q, int D, int R)
{
    constexpr int U = sizeof(T) == 2 ? 4 : 2;   // tokens ahead; fp32 with 3: 8192 x 2048 54 us for 50 (spills)
    typedef typename Raw<T>::quad Quad;
    flag_bad_sequences(q);
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * kV;
    long long t = (long long)blockIdx.x * R;
    const long long t1 = min(t + R, q.tokens);
    int i = max(find_sequence(q, t), 0);
    if (c >= D) return;

    f32x2 wt[W][2], bv[2], gw[W + 1][2];
    load_taps2<W>(w, bias, c, wt, bv);
#pragma unroll
    for (int j = 0; j <= W; ++j) gw[j][0] = gw[j][1] = 0ull;
    const float zero[kV] = {0.f, 0.f, 0.f, 0.f};

    for (; t < t1; ++i) {
        long long s = q.tokens, e = q.tokens;   // behind the last sequence: rows of no sequence
        bool use = false;
        if (i < q.n) {
            s = q.begin(i);
            e = q.begin(i + 1);
            if (e <= t || e <= s) continue;
            use = Seqs::inside(s, e, q.tokens);
        }
        for (; t < min(s, t1); ++t) store_vec<kV>(gx + t * D + c, zero);
        if (t >= t1) break;
        if (i >= q.n) break;
        const long long a = t, b = min(e, t1);
        if (!use) {   // a skipped sequence: zero gradient
            for (; t < b; ++t) store_vec<kV>(gx + t * D + c, zero);
            continue;
        }
        f32x2 win[W - 1][2], dp[W - 1][2];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            float f[kV];
            load_row<T, W, kV>(x, ldx, s0, s, i, a - s - (W - 1) + j, D, c, f);
            win[j][0] = pack(f[0], f[1]);
            win[j][1] = pack(f[2], f[3]);
            dp[j][0] = dp[j][1] = 0ull;
        }
        const T* px = x + a * ldx + c;
        const float* pg = gy + a * D + c;
        // dpre of the next token (x, gy as loaded); `own`: it counts in gw and gb
        auto slope = [&](const Quad& raw, const float4& g, bool own, f32x2 (&d)[2]) {
            f32x2 xv[2];
            widen(raw, xv);
            d[0] = pack(g.x, g.y);
            d[1] = pack(g.z, g.w);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (SILU) {
                    f32x2 pre = fma2(wt[W - 1][v], xv[v], bv[v]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) pre = fma2(wt[j][v], win[j][v], pre);
                    float p0, p1;
                    unpack(pre, p0, p1);
                    d[v] = mul2(d[v], silu_grad2(p0, p1));
                }
                if (own) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) gw[j][v] = fma2(d[v], win[j][v], gw[j][v]);
                    gw[W - 1][v] = fma2(d[v], xv[v], gw[W - 1][v]);
                    gw[W][v] = add2(gw[W][v], d[v]);
                }
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
                win[W - 2][v] = xv[v];
            }
        };
        // gx of the token W - 1 before the one with slope d: dp[k] is the slope k
        // tokens after it
        auto input_grad = [&](const f32x2 (&d)[2], f32x2 (&o)[2]) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                o[v] = mul2(wt[0][v], d[v]);
#pragma unroll
                for (int j = 1; j < W; ++j) o[v] = fma2(wt[j][v], dp[W - 1 - j][v], o[v]);
            }
        };
        auto shift = [&](const f32x2 (&d)[2]) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) dp[j][v] = dp[j + 1][v];
                dp[W - 2][v] = d[v];
            }
        };
        float* po = gx + a * D + c;
        auto emit = [&](const f32x2 (&o)[2]) {
            *reinterpret_cast<ulonglong2*>(po) = make_ulonglong2(o[0], o[1]);
            po += D;
        };
        int n = (int)(b - a);
        f32x2 d[2], o[2];
        // the first W - 1 own tokens: their predecessors are another tile's
        for (int k = 0; k < W - 1 && n > 0; ++k, --n, px += ldx, pg += D) {
            slope(*reinterpret_cast<const Quad*>(px), *reinterpret_cast<const float4*>(pg), true, d);
            shift(d);
        }
        if (n >= U) {
            Quad raw[U];
            float4 g[U];
#pragma unroll
            for (int u = 0; u < U; ++u, px += ldx, pg += D) {
                raw[u] = *reinterpret_cast<const Quad*>(px);
                g[u] = *reinterpret_cast<const float4*>(pg);
            }
#pragma unroll 1
            for (; n >= 2 * U; n -= U) {
#pragma unroll
                for (int u = 0; u < U; ++u, px += ldx, pg += D) {
                    const Quad r0 = raw[u];
                    const float4 g0 = g[u];
                    raw[u] = *reinterpret_cast<const Quad*>(px);
                    g[u] = *reinterpret_cast<const float4*>(pg);
                    slope(r0, g0, true, d);
                    input_grad(d, o);
                    shift(d);
                    emit(o);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                slope(raw[u], g[u], true, d);
                input_grad(d, o);
                shift(d);
                emit(o);
            }
            n -= U;
        }
#pragma unroll 1
        for (; n > 0; --n, px += ldx, pg += D) {
            slope(*reinterpret_cast<const Quad*>(px), *reinterpret_cast<const float4*>(pg), true, d);
            input_grad(d, o);
            shift(d);
            emit(o);
        }
        // the W - 1 tokens after the last own one: the next tile's, or none and the
        // final state's gradient instead
#pragma unroll 1
        for (long long u = b; u < b + W - 1; ++u, px += ldx, pg += D) {
            d[0] = d[1] = 0ull;
            if (u < e) slope(*reinterpret_cast<const Quad*>(px), *reinterpret_cast<const float4*>(pg), false, d);
            if (u - (W - 1) >= a) {
                input_grad(d, o);
                if (u >= e && gsT) {
                    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(
                        gsT + ((long long)i * (W - 1) + (u - e)) * D + c);
                    o[0] = add2(o[0], f.x);
                    o[1] = add2(o[1], f.y);
                }
                emit(o);
            }
            shift(d);
        }
        t = b;
    }
    float* o = part + (long long)blockIdx.x * (W + 1) * D + c;
#pragma unroll
    for (int j = 0; j <= W; ++j)
        *reinterpret_cast<ulonglong2*>(o + (long long)j * D) = make_ulonglong2(gw[j][0], gw[j][1]);
}

// gw[d, j] and gb[d] from the tiles' partial sums: 32 columns per block, 32 rows
// of threads over the tiles, then a sum over those rows.  4 us for 128 tiles of
// 2048 channels (5.2 MB, from the L2).
__global__ void __launch_bounds__(1024)
conv_bwd_reduce_kernel(const float* __restrict__ part, int ntiles, float* __restrict__ gw, float* __restrict__ gb,
                       int D, int W)
{
    __shared__ float red[32][33];
    const int col = blockIdx.x * 32 + threadIdx.x;   // j * D + d
    const int ncol = (W + 1) * D;
    float acc = 0.f;
    if (col < ncol) {
#pragma unroll 4
        for (int r = threadIdx.y; r < ntiles; r += 32) acc += part[(long long)r * ncol + col];
    }
    red[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    acc = warp_sum(red[threadIdx.x][threadIdx.y]);   // a warp per column now
    const int mine = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && mine < ncol) {
        const int j = mine / D, d = mine % D;
        if (j < W)
            gw[(long long)d * W + j] = acc;
        else if (gb)
            gb[d] = acc;
    }
}

// Gradient of the initial states: row k of sequence i is the input at position
// k - (W - 1) before its first token, read by tokens m <= k; with len <= k
// tokens it is also row k - len of the final state.  W - 1 rows of 2 W - 2 inputs per
// sequence: a launch's time (5 us for two sequences of 2048 channels).
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(128)
conv_bwd_state_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w,
                      const float* __restrict__ bias, const T* __restrict__ s0, const float* __restrict__ gy,
                      const float* __restrict__ gsT, float* __restrict__ gs0, Seqs q, int D)
{
    constexpr int V = kV;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int i = blockIdx.x;
    if (c >= D) return;
    const long long s = q.begin(i);
    long long e = q.begin(i + 1);
    if (e < s || !Seqs::inside(s, e, q.tokens)) e = s;
    const int len = (int)min(e - s, (long long)W);
    float wt[W][V], bv[V], acc[W - 1][V];
    load_taps<W, V>(w, bias, c, wt, bv);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[k][v] = 0.f;
#pragma unroll
    for (int m = 0; m < W - 1; ++m) {
        if (m >= len) break;
        float g[V], pre[V];
        load_vec<V>(gy + (s + m) * D + c, g);
#pragma unroll
        for (int v = 0; v < V; ++v) pre[v] = bv[v];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float r[V];
            load_row<T, W, V>(x, ldx, s0, s, i, m - (W - 1) + j, D, c, r);
#pragma unroll
            for (int v = 0; v < V; ++v) pre[v] = fmaf(wt[j][v], r[v], pre[v]);
        }
#pragma unroll
        for (int k = m; k < W - 1; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
                acc[k][v] = fmaf(wt[k - m][v], SILU ? g[v] * silu_grad(pre[v]) : g[v], acc[k][v]);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        if (gsT && k >= len) {
            float g[V];
            load_vec<V>(gsT + ((long long)i * (W - 1) + k - len) * D + c, g);
#pragma unroll
            for (int v = 0; v < V; ++v) acc[k][v] += g[v];
        }
        store_vec<V>(gs0 + ((long long)i * (W - 1) + k) * D + c, acc[k]);
    }
}

// ---------------------------------------------------------------- launches
static int conv_threads(int vecs) { return vecs >= 128 ? 128 : (vecs + 31) / 32 * 32; }

// Tokens per tile of the backward pass: 128 where that leaves 256 threads per SM,
// less halo and fewer partial sums; else half, down to 8; at most about 4096 partial
// sums.  Both sides, D = 2048, bf16, us: T = 1024 with tiles of 8/16/32/128 15.3,
// 16.9, 19.2, 41.8; T = 4096 with 16/32/64 33.4, 28.6, 34.0; T = 8192 with 32/64/128
// 51.2, 44.4, 55.7; T = 16384 95.8, 82.3, 74.9; T = 65536 339, 288, 270.
static int conv_bwd_tile(long long tokens, int D)
{
    int r = 128;
    while (r > 8 && (tokens / r) * (D / kV) < 148LL * 256) r /= 2;
    while ((tokens + r - 1) / r > 4096) r *= 2;
    return r;
}

template <typename T, typename TO, int W, bool SILU>
static cudaError_t launch_conv_fwd(const ConvArgs& a, const void* s0, void* y, void* sT, cudaStream_t st)
{
    const Seqs q{a.cu, a.nseq, a.T, a.tokens};
    const int nt = conv_threads(a.D / kV);
    const unsigned cb = (a.D / kV + nt - 1) / nt;
    // Tokens per tile: long tiles re-read less halo, short ones give enough threads:
    // 32, halved to 8 until there are 256 threads per SM.  Both sides, D = 2048, bf16,
    // us: T = 1024 with tiles of 8/16/32 5.0, 5.6, 7.6; T = 2048 8.5, 7.3, 8.8; T = 4096
    // 13.1, 11.8, 11.3; T = 8192 with 16/32/64 19.3, 19.1, 18.8 (2.8, 1.4 and 0.7 waves
    // of blocks); T = 16384 34.3, 31.8, 34.0; T = 65536 121, 109, 106.
    int R = 32;
    while (R > 8 && (a.tokens / R) * cb * nt < 148LL * 256) R /= 2;
    const long long ntiles = (a.tokens + R - 1) / R;
    const bool apart = sT && sT == s0;   // in place: the states move after every tile has read them
    const long long gx = ntiles + (sT && !apart ? a.nseq : 0);
    if (gx > 0x7fffffffLL || cb > 65535u) return cudaErrorInvalidConfiguration;
    conv_fwd_kernel<T, TO, W, SILU><<<dim3((unsigned)gx, cb), nt, 0, st>>>(
        static_cast<const T*>(a.x), a.ldx, a.w, a.bias, static_cast<const T*>(s0), static_cast<TO*>(y),
        apart ? nullptr : static_cast<T*>(sT), q, a.D, R, (int)ntiles);
    if (apart)
        conv_state_kernel<T, W><<<dim3(a.nseq, cb), nt, 0, st>>>(static_cast<const T*>(a.x), a.ldx,
                                                                 static_cast<const T*>(s0), static_cast<T*>(sT), q, a.D);
    return cudaGetLastError();
}

template <typename T, typename TO, int W, bool SILU>
static cudaError_t launch_conv_step(const ConvArgs& a, void* state, void* y, cudaStream_t st)
{
    const int nt = conv_threads(a.D / kV);
    const unsigned cb = (a.D / kV + nt - 1) / nt;
    auto go = [&](auto rn) {
        constexpr int RN = decltype(rn)::value;
        conv_step_kernel<T, TO, W, SILU, RN><<<dim3((a.nseq + RN - 1) / RN, cb), nt, 0, st>>>(
            static_cast<const T*>(a.x), a.ldx, a.w, a.bias, static_cast<T*>(state), static_cast<TO*>(y), a.nseq, a.D);
    };
    // four sequences per thread share its weights once that leaves 128 threads per SM
    // (D = 4096, bf16, one against four, some of the state from the L2: 16 sequences
    // 1.85 / 2.18 us, 128 3.24 / 2.84, 1024 13.9 / 11.5)
    if ((long long)a.nseq / 4 * cb * nt >= 148LL * 128)
        go(std::integral_constant<int, 4>{});
    else
        go(std::integral_constant<int, 1>{});
    return cudaGetLastError();
}

template <typename T, int W, bool SILU>
static cudaError_t launch_conv_bwd(const ConvArgs& a, const void* s0, const float* gy, const float* gsT, float* gx,
                                   float* gw, float* gb, float* gs0, float* part, cudaStream_t st)
{
    const Seqs q{a.cu, a.nseq, a.T, a.tokens};
    const int nt = conv_threads(a.D / kV);
    const unsigned cb = (a.D / kV + nt - 1) / nt;
    const int R = conv_bwd_tile(a.tokens, a.D);
    const long long ntiles = (a.tokens + R - 1) / R;
    if (cb > 65535u) return cudaErrorInvalidConfiguration;
    conv_bwd_kernel<T, W, SILU><<<dim3((unsigned)ntiles, cb), nt, 0, st>>>(
        static_cast<const T*>(a.x), a.ldx, a.w, a.bias, static_cast<const T*>(s0), gy, gsT, gx, part, q, a.D, R);
    conv_bwd_reduce_kernel<<<((W + 1) * a.D + 31) / 32, dim3(32, 32), 0, st>>>(part, (int)ntiles, gw, gb, a.D, W);
    if (gs0)
        conv_bwd_state_kernel<T, W, SILU><<<dim3(a.nseq, cb), nt, 0, st>>>(
            static_cast<const T*>(a.x), a.ldx, a.w, a.bias, static_cast<const T*>(s0), gy, gsT, gs0, q, a.D);
    return cudaGetLastError();
}

// Calls f with the number of taps and whether there is a SiLU, as integral constants.
template <typename F>
static cudaError_t conv_dispatch_w(const ConvArgs& a, F&& f)
{
    if (a.silu) {
        if (a.W == 2) return f(std::integral_constant<int, 2>{}, std::true_type{});
        if (a.W == 3) return f(std::integral_constant<int, 3>{}, std::true_type{});
        return f(std::integral_constant<int, 4>{}, std::true_type{});
    }
    if (a.W == 2) return f(std::integral_constant<int, 2>{}, std::false_type{});
    if (a.W == 3) return f(std::integral_constant<int, 3>{}, std::false_type{});
    return f(std::integral_constant<int, 4>{}, std::false_type{});
}

}  // namespace mixer

cudaError_t conv_fwd(const ConvArgs& a, const void* s0, void* y, void* sT, kda_dtype o_dtype, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    return mixer::conv_dispatch_w(a, [&](auto w, auto act) {
        constexpr int W = decltype(w)::value;
        constexpr bool SILU = decltype(act)::value;
        if (a.dtype == KDA_BF16)
            return o_dtype == KDA_BF16 ? mixer::launch_conv_fwd<bf, bf, W, SILU>(a, s0, y, sT, s)
                                       : mixer::launch_conv_fwd<bf, float, W, SILU>(a, s0, y, sT, s);
        return o_dtype == KDA_BF16 ? mixer::launch_conv_fwd<float, bf, W, SILU>(a, s0, y, sT, s)
                                   : mixer::launch_conv_fwd<float, float, W, SILU>(a, s0, y, sT, s);
    });
}

cudaError_t conv_step(const ConvArgs& a, void* state, void* y, kda_dtype o_dtype, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    return mixer::conv_dispatch_w(a, [&](auto w, auto act) {
        constexpr int W = decltype(w)::value;
        constexpr bool SILU = decltype(act)::value;
        if (a.dtype == KDA_BF16)
            return o_dtype == KDA_BF16 ? mixer::launch_conv_step<bf, bf, W, SILU>(a, state, y, s)
                                       : mixer::launch_conv_step<bf, float, W, SILU>(a, state, y, s);
        return o_dtype == KDA_BF16 ? mixer::launch_conv_step<float, bf, W, SILU>(a, state, y, s)
                                   : mixer::launch_conv_step<float, float, W, SILU>(a, state, y, s);
    });
}

size_t conv_bwd_workspace(long long tokens, int D, int W)
{
    const int R = mixer::conv_bwd_tile(tokens, D);
    return (size_t)((tokens + R - 1) / R) * (W + 1) * D * sizeof(float);
}

cudaError_t conv_bwd(const ConvArgs& a, const void* s0, const float* gy, const float* gsT, float* gx, float* gw,
                     float* gb, float* gs0, void* ws, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    float* part = static_cast<float*>(ws);
    return mixer::conv_dispatch_w(a, [&](auto w, auto act) {
        constexpr int W = decltype(w)::value;
        constexpr bool SILU = decltype(act)::value;
        return a.dtype == KDA_BF16 ? mixer::launch_conv_bwd<bf, W, SILU>(a, s0, gy, gsT, gx, gw, gb, gs0, part, s)
                                   : mixer::launch_conv_bwd<float, W, SILU>(a, s0, gy, gsT, gx, gw, gb, gs0, part, s);
    });
}

}  // namespace kda
