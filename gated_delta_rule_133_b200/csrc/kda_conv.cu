// Short causal depthwise convolution of W = 2..4 taps with an optional SiLU:
//   pre[t, d] = bias[d] + sum_j w[d, j] x[t - W + 1 + j, d],   y = pre or silu(pre)
// over dense or packed sequences, as a step of one token per sequence, and its
// gradients.  A sequence's tokens before its first one come from its state: the
// last W - 1 inputs, in the inputs' type (they are copies of inputs).
//
// Every path is bound by HBM: each input element is read once and each output
// element written once (plus a halo of W - 1 rows per token tile, which the L2
// holds).  A thread owns a 16-byte vector of channels and walks a tile of
// tokens with the last W - 1 rows and the weights in registers, so no shared
// memory or synchronisation is needed and the loads of the next tokens are in
// flight together.
#include "kda_mixer.cuh"

namespace kda {
namespace mixer {

// 16 bytes of T as fp32.
template <typename T, int V>
__device__ __forceinline__ void raw_to_float(const uint4& r, float (&x)[V])
{
    if constexpr (sizeof(T) == 2) {
        static_assert(V == 8, "vector width");
        unpack2(r.x, x[0], x[1]); unpack2(r.y, x[2], x[3]); unpack2(r.z, x[4], x[5]); unpack2(r.w, x[6], x[7]);
    } else {
        static_assert(V == 4, "vector width");
        x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
    }
}

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
    long long s = q.begin(i), e = q.begin(i + 1);
    if (e < s || !Seqs::inside(s, e, q.tokens)) e = s;
    uint4 rows[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const long long pos = e - s - (W - 1) + j;
        if (pos >= 0)
            rows[j] = *reinterpret_cast<const uint4*>(x + (s + pos) * ldx + c);
        else if (s0)
            rows[j] = *reinterpret_cast<const uint4*>(s0 + ((long long)i * (W - 1) + pos + W - 1) * D + c);
        else
            rows[j] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        *reinterpret_cast<uint4*>(sT + ((long long)i * (W - 1) + j) * D + c) = rows[j];
}

template <typename T, int W>
__global__ void __launch_bounds__(128)
conv_state_kernel(const T* __restrict__ x, long long ldx, const T* s0, T* sT, Seqs q, int D)
{
    constexpr int V = 16 / sizeof(T);
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c < D) write_state<T, W>(x, ldx, s0, sT, q, blockIdx.x, D, c);
}

// Grid: x = token tiles of R tokens, then (if sT) one block per sequence for
// the final states; y = channel blocks.  U tokens are loaded ahead.
template <typename T, typename TO, int W, bool SILU>
__global__ void __launch_bounds__(128)
conv_fwd_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                const T* s0, TO* __restrict__ y, T* sT, Seqs q, int D, int R, int ntiles)
{
    constexpr int V = 16 / sizeof(T), U = 8;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if ((int)blockIdx.x >= ntiles) {
        if (c < D) write_state<T, W>(x, ldx, s0, sT, q, blockIdx.x - ntiles, D, c);
        return;
    }
    flag_bad_sequences(q);
    long long t = (long long)blockIdx.x * R;
    const long long t1 = min(t + R, q.tokens);
    int i = max(find_sequence(q, t), 0);
    if (c >= D) return;

    float wt[W][V], bv[V];
    load_taps<W, V>(w, bias, c, wt, bv);
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
        float win[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_row<T, W, V>(x, ldx, s0, s, i, t - s - (W - 1) + j, D, c, win[j]);
        for (; t < stop; t += U) {
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < stop) raw[u] = *reinterpret_cast<const uint4*>(x + (t + u) * ldx + c);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u < stop) {
                    float xv[V], out[V];
                    raw_to_float<T, V>(raw[u], xv);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float p = fmaf(wt[W - 1][v], xv[v], bv[v]);
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) p = fmaf(wt[j][v], win[j][v], p);
                        out[v] = SILU ? silu(p) : p;
#pragma unroll
                        for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
                        win[W - 2][v] = xv[v];
                    }
                    store_vec<V>(y + (t + u) * D + c, out);
                }
            }
        }
        t = stop;
    }
}

// One token per sequence: y from the state's rows and x; the state moves up by
// one row.  A thread owns a channel vector of RN sequences, so that the
// weights are read once for them.
template <typename T, typename TO, int W, bool SILU>
__global__ void __launch_bounds__(128)
conv_step_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                 T* __restrict__ state, TO* __restrict__ y, int n, int D, int RN)
{
    constexpr int V = 16 / sizeof(T);
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c >= D) return;
    float wt[W][V], bv[V];
    load_taps<W, V>(w, bias, c, wt, bv);
    const int i1 = min((int)(blockIdx.x + 1) * RN, n);
    for (int i = blockIdx.x * RN; i < i1; ++i) {
        T* st = state + (long long)i * (W - 1) * D + c;
        uint4 raw[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) raw[j] = *reinterpret_cast<const uint4*>(st + (long long)j * D);
        raw[W - 1] = *reinterpret_cast<const uint4*>(x + i * ldx + c);
        float out[V];
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = bv[v];
#pragma unroll
        for (int j = W - 1; j >= 0; --j) {
            float xv[V];
            raw_to_float<T, V>(raw[j], xv);
#pragma unroll
            for (int v = 0; v < V; ++v) out[v] = fmaf(wt[j][v], xv[v], out[v]);
            if (j > 0) *reinterpret_cast<uint4*>(st + (long long)(j - 1) * D) = raw[j];
        }
        if (SILU) {
#pragma unroll
            for (int v = 0; v < V; ++v) out[v] = silu(out[v]);
        }
        store_vec<V>(y + (long long)i * D + c, out);
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
constexpr int kBwdV = 4;   // channels per thread: 16-byte vectors of the fp32 gradients

template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(128)
conv_bwd_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                const T* __restrict__ s0, const float* __restrict__ gy, const float* __restrict__ gsT,
                float* __restrict__ gx, float* __restrict__ part, Seqs q, int D, int R)
{
    constexpr int V = kBwdV, U = 4;
    flag_bad_sequences(q);
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    long long t = (long long)blockIdx.x * R;
    const long long t1 = min(t + R, q.tokens);
    int i = max(find_sequence(q, t), 0);
    if (c >= D) return;

    float wt[W][V], bv[V], gw[W + 1][V];
    load_taps<W, V>(w, bias, c, wt, bv);
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) gw[j][v] = 0.f;
    const float zero[V] = {0.f, 0.f, 0.f, 0.f};

    for (; t < t1; ++i) {
        long long s = q.tokens, e = q.tokens;   // behind the last sequence: rows of no sequence
        bool use = false;
        if (i < q.n) {
            s = q.begin(i);
            e = q.begin(i + 1);
            if (e <= t || e <= s) continue;
            use = Seqs::inside(s, e, q.tokens);
        }
        for (; t < min(s, t1); ++t) store_vec<V>(gx + t * D + c, zero);
        if (t >= t1) break;
        if (i >= q.n) break;
        const long long a = t, b = min(e, t1);
        if (!use) {   // a skipped sequence: zero gradient
            for (; t < b; ++t) store_vec<V>(gx + t * D + c, zero);
            continue;
        }
        float win[W - 1][V], dp[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            load_row<T, W, V>(x, ldx, s0, s, i, a - s - (W - 1) + j, D, c, win[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) dp[j][v] = 0.f;
        }
        const long long load_end = min(b + W - 1, e);
        for (; t < b + W - 1; t += U) {
            float xs[U][V], gs[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u < load_end) {
                    load_vec<V>(x + (t + u) * ldx + c, xs[u]);
                    load_vec<V>(gy + (t + u) * D + c, gs[u]);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) xs[u][v] = gs[u][v] = 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long p = t + u - (W - 1);
                const bool own = t + u < b, emit = p >= a && p < b;
                float out[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float pre = fmaf(wt[W - 1][v], xs[u][v], bv[v]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) pre = fmaf(wt[j][v], win[j][v], pre);
                    const float d = t + u >= load_end ? 0.f : SILU ? gs[u][v] * silu_grad(pre) : gs[u][v];
                    if (own) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) gw[j][v] = fmaf(d, win[j][v], gw[j][v]);
                        gw[W - 1][v] = fmaf(d, xs[u][v], gw[W - 1][v]);
                        gw[W][v] += d;
                    }
                    // dp[0] = dpre[p], ..., dp[W - 2] = dpre[p + W - 2], d = dpre[p + W - 1]
                    float o = wt[0][v] * d;
#pragma unroll
                    for (int j = 1; j < W; ++j) o = fmaf(wt[j][v], dp[W - 1 - j][v], o);
                    out[v] = o;
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) {
                        win[j][v] = win[j + 1][v];
                        dp[j][v] = dp[j + 1][v];
                    }
                    win[W - 2][v] = xs[u][v];
                    dp[W - 2][v] = d;
                }
                if (emit) {
                    if (gsT && e - p <= W - 1) {
                        float g[V];
                        load_vec<V>(gsT + ((long long)i * (W - 1) + (W - 1) - (e - p)) * D + c, g);
#pragma unroll
                        for (int v = 0; v < V; ++v) out[v] += g[v];
                    }
                    store_vec<V>(gx + p * D + c, out);
                }
            }
        }
        t = b;
    }
    float* o = part + (long long)blockIdx.x * (W + 1) * D + c;
#pragma unroll
    for (int j = 0; j <= W; ++j) store_vec<V>(o + (long long)j * D, gw[j]);
}

// gw[d, j] and gb[d] from the tiles' partial sums: 32 columns per block, 8 rows
// of threads over the tiles, then a sum over those rows.
__global__ void __launch_bounds__(256)
conv_bwd_reduce_kernel(const float* __restrict__ part, int ntiles, float* __restrict__ gw, float* __restrict__ gb,
                       int D, int W)
{
    __shared__ float red[8][33];
    const int col = blockIdx.x * 32 + threadIdx.x;   // j * D + d
    const int ncol = (W + 1) * D;
    float acc = 0.f;
    if (col < ncol)
        for (int r = threadIdx.y; r < ntiles; r += 8) acc += part[(long long)r * ncol + col];
    red[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.y == 0 && col < ncol) {
#pragma unroll
        for (int r = 1; r < 8; ++r) acc += red[r][threadIdx.x];
        const int j = col / D, d = col % D;
        if (j < W)
            gw[(long long)d * W + j] = acc;
        else if (gb)
            gb[d] = acc;
    }
}

// Gradient of the initial states: row k of sequence i is the input at position
// k - (W - 1) before its first token, read by tokens m <= k; with len <= k
// tokens it is also row k - len of the final state.
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(128)
conv_bwd_state_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w,
                      const float* __restrict__ bias, const T* __restrict__ s0, const float* __restrict__ gy,
                      const float* __restrict__ gsT, float* __restrict__ gs0, Seqs q, int D)
{
    constexpr int V = kBwdV;
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

static int conv_bwd_tile(long long tokens)
{
    const long long r = (tokens + 4095) / 4096;   // at most about 4096 partial sums
    return (int)(r < 64 ? 64 : r);
}

template <typename T, typename TO, int W, bool SILU>
static cudaError_t launch_conv_fwd(const ConvArgs& a, const void* s0, void* y, void* sT, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const Seqs q{a.cu, a.nseq, a.T, a.tokens};
    const int nt = conv_threads(a.D / V);
    const unsigned cb = (a.D / V + nt - 1) / nt;
    // Tokens per tile: long tiles re-read less halo, short ones give enough
    // threads; at least ~1024 threads per SM while a tile keeps 16 tokens.
    int R = 64;
    while (R > 16 && (a.tokens / R) * cb * nt < 148LL * 1024) R /= 2;
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
    constexpr int V = 16 / sizeof(T);
    const int nt = conv_threads(a.D / V);
    const unsigned cb = (a.D / V + nt - 1) / nt;
    int RN = 4;
    while (RN > 1 && (long long)a.nseq / RN * cb * nt < 148LL * 256) RN /= 2;
    conv_step_kernel<T, TO, W, SILU><<<dim3((a.nseq + RN - 1) / RN, cb), nt, 0, st>>>(
        static_cast<const T*>(a.x), a.ldx, a.w, a.bias, static_cast<T*>(state), static_cast<TO*>(y), a.nseq, a.D, RN);
    return cudaGetLastError();
}

template <typename T, int W, bool SILU>
static cudaError_t launch_conv_bwd(const ConvArgs& a, const void* s0, const float* gy, const float* gsT, float* gx,
                                   float* gw, float* gb, float* gs0, float* part, cudaStream_t st)
{
    const Seqs q{a.cu, a.nseq, a.T, a.tokens};
    const int nt = conv_threads(a.D / kBwdV);
    const unsigned cb = (a.D / kBwdV + nt - 1) / nt;
    const int R = conv_bwd_tile(a.tokens);
    const long long ntiles = (a.tokens + R - 1) / R;
    if (cb > 65535u) return cudaErrorInvalidConfiguration;
    conv_bwd_kernel<T, W, SILU><<<dim3((unsigned)ntiles, cb), nt, 0, st>>>(
        static_cast<const T*>(a.x), a.ldx, a.w, a.bias, static_cast<const T*>(s0), gy, gsT, gx, part, q, a.D, R);
    conv_bwd_reduce_kernel<<<((W + 1) * a.D + 31) / 32, dim3(32, 8), 0, st>>>(part, (int)ntiles, gw, gb, a.D, W);
    if (gs0)
        conv_bwd_state_kernel<T, W, SILU><<<dim3(a.nseq, cb), nt, 0, st>>>(
            static_cast<const T*>(a.x), a.ldx, a.w, a.bias, static_cast<const T*>(s0), gy, gsT, gs0, q, a.D);
    return cudaGetLastError();
}

// Calls f.template operator()<T, TO, W, SILU>() for the call's types.
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
    const int R = mixer::conv_bwd_tile(tokens);
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
