// C ABI of the short convolution and the selective scan: argument validation
// and the calls without tokens.  Contract: include/kda.h.
#include "kda_mixer.cuh"

namespace {

constexpr int kMaxChannels = 1 << 20;
constexpr long long kMaxTokens = 0x7fff0000LL;   // token indices and a tile beyond them stay below 2^31

// Row stride of a token-major input: whole 16-byte vectors, rows that do not
// overlap, below 4 GiB.
bool valid_ld(long long ld, long long row, kda_dtype dtype)
{
    const long long per16 = dtype == KDA_BF16 ? 8 : 4;
    return ld >= row && ld % per16 == 0 && ld < 1LL << 30;
}

bool opt_aligned16(const void* p) { return !p || aligned16(p); }

// Memory that a call reads or writes.
struct Span {
    const void* p;
    size_t bytes;
};

size_t elem_size(kda_dtype dtype) { return dtype == KDA_BF16 ? 2 : 4; }

// `tokens` rows of `row` elements, `ld` apart (what lies between them counts).
Span rows(const void* p, long long ld, long long row, long long tokens, kda_dtype dtype)
{
    return Span{p, tokens > 0 ? (size_t)((tokens - 1) * ld + row) * elem_size(dtype) : 0};
}

Span floats(const float* p, long long n) { return Span{p, (size_t)n * sizeof(float)}; }

bool overlap(const Span& a, const Span& b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

// Whether an output shares memory with an input or with another output: blocks
// write it while others still read.
template <int NO, int NI>
bool any_overlap(const Span (&out)[NO], const Span (&in)[NI])
{
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i], in[j])) return true;
    }
    return false;
}

Span bounds(const int32_t* cu, int nseq) { return Span{cu, cu ? (size_t)(nseq + 1LL) * sizeof(int32_t) : 0}; }

kda_status check_conv(const kda::ConvArgs& a, const void* y, const void* s0, const void* sT, int mode)
{
    if (a.tokens < 0 || a.nseq < 0 || a.D <= 0 || a.W <= 0 || !valid_dtype(a.dtype) || (mode & ~KDA_CONV_SILU))
        return KDA_ERR_INVALID_ARG;
    if (!a.w || !aligned16(a.w) || !opt_aligned16(a.bias) || !opt_aligned16(s0) || !opt_aligned16(sT))
        return KDA_ERR_INVALID_ARG;
    if (a.tokens > 0 && (!a.x || !y || !aligned16(a.x) || !aligned16(y) || !valid_ld(a.ldx, a.D, a.dtype)))
        return KDA_ERR_INVALID_ARG;
    if (a.W < 2 || a.W > 4 || a.D % 8 != 0 || a.D > kMaxChannels || a.tokens > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda::ConvArgs conv_args(const void* x, long long ldx, const float* w, const float* bias, const int32_t* cu, int nseq,
                        int T, long long tokens, int D, int W, kda_dtype dtype, int mode)
{
    return kda::ConvArgs{x, ldx, w, bias, cu, nseq, T, tokens, D, W, (mode & KDA_CONV_SILU) != 0, dtype};
}

// final = initial (or zeros) for the states of sequences without tokens
kda_status copy_bytes(const void* from, void* to, size_t bytes, cudaStream_t s)
{
    if (!to || bytes == 0 || from == to) return KDA_OK;
    if (from) return from_cuda(cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s));
    return from_cuda(cudaMemsetAsync(to, 0, bytes, s));
}

kda_status check_cu(const int32_t* cu, int N, int T)
{
    if (N < 0 || N > 65535 || T < 0) return KDA_ERR_INVALID_ARG;
    if (N == 0 && T > 0) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (!cu || !aligned4(cu))) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// The state may be updated in place: s0 == sT counts as the output alone.
bool conv_overlap(const kda::ConvArgs& a, const void* s0, const void* y, const void* sT, kda_dtype o_dtype)
{
    const size_t state = (size_t)a.nseq * (a.W - 1) * a.D * elem_size(a.dtype);
    const Span out[] = {rows(y, a.D, a.D, a.tokens, o_dtype), {sT, state}};
    const Span in[] = {rows(a.x, a.ldx, a.D, a.tokens, a.dtype), floats(a.w, (long long)a.D * a.W),
                       floats(a.bias, a.D), bounds(a.cu, a.nseq), {s0 == sT ? nullptr : s0, state}};
    return any_overlap(out, in);
}

kda_status conv_fwd_call(const kda::ConvArgs& a, const void* s0, void* y, void* sT, kda_dtype o_dtype, int mode,
                         void* stream)
{
    const kda_status st = check_conv(a, y, s0, sT, mode);
    if (st != KDA_OK) return st;
    if (!valid_dtype(o_dtype) || conv_overlap(a, s0, y, sT, o_dtype)) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.tokens == 0) return copy_bytes(s0, sT, (size_t)a.nseq * (a.W - 1) * a.D * elem_size(a.dtype), s);
    return from_cuda(kda::conv_fwd(a, s0, y, sT, o_dtype, s));
}

kda_status conv_bwd_call(const kda::ConvArgs& a, const void* s0, const float* gy, const float* gsT, float* gx,
                         float* gw, float* gb, float* gs0, int mode, void* ws, size_t ws_bytes, void* stream)
{
    kda_status st = check_conv(a, gx, s0, gsT, mode);
    if (st != KDA_OK) return st;
    if (!gw || !aligned16(gw) || !opt_aligned16(gb) || !opt_aligned16(gs0)) return KDA_ERR_INVALID_ARG;
    if (a.tokens > 0 && (!gy || !aligned16(gy))) return KDA_ERR_INVALID_ARG;
    const size_t need = a.tokens == 0 ? 0 : kda::conv_bwd_workspace(a.tokens, a.D, a.W);
    st = check_workspace(ws, ws_bytes, need);
    if (st != KDA_OK) return st;
    const long long act = a.tokens * a.D, state = (long long)a.nseq * (a.W - 1) * a.D;
    const Span out[] = {floats(gx, act), floats(gw, (long long)a.D * a.W), floats(gb, a.D), floats(gs0, state),
                        {ws, need}};
    const Span in[] = {rows(a.x, a.ldx, a.D, a.tokens, a.dtype), floats(a.w, (long long)a.D * a.W),
                       floats(a.bias, a.D), bounds(a.cu, a.nseq), {s0, (size_t)state * elem_size(a.dtype)},
                       floats(gy, act), floats(gsT, state)};
    if (any_overlap(out, in)) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.tokens == 0) {
        st = copy_bytes(nullptr, gw, (size_t)a.D * a.W * 4, s);
        if (st == KDA_OK) st = copy_bytes(nullptr, gb, (size_t)a.D * 4, s);
        if (st == KDA_OK) st = copy_bytes(gsT, gs0, (size_t)a.nseq * (a.W - 1) * a.D * 4, s);
        return st;
    }
    return from_cuda(kda::conv_bwd(a, s0, gy, gsT, gx, gw, gb, gs0, ws, s));
}

kda_status check_ssm_sizes(int D, int S, int G, kda_dtype dtype)
{
    if (D <= 0 || S <= 0 || G <= 0 || !valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if (D % G != 0 || (D / G) % 8 != 0 || D > kMaxChannels || (S != 16 && S != 32 && S != 64))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_ssm(const kda::SsmArgs& a, const void* y, int mode)
{
    if (a.tokens < 0 || a.nseq < 0 || (mode & ~KDA_SSM_SOFTPLUS)) return KDA_ERR_INVALID_ARG;
    if (a.D <= 0 || a.N <= 0 || a.G <= 0 || !valid_dtype(a.dtype)) return KDA_ERR_INVALID_ARG;
    if (!a.A || !aligned16(a.A) || !opt_aligned16(a.skip) || !opt_aligned16(a.dt_bias) || !opt_aligned16(a.s0))
        return KDA_ERR_INVALID_ARG;
    if (a.tokens > 0) {
        if (!a.x || !a.dt || !a.b || !a.c || !y) return KDA_ERR_INVALID_ARG;
        if (!aligned16(a.x) || !aligned16(a.dt) || !aligned16(a.b) || !aligned16(a.c) || !opt_aligned16(a.z) ||
            !aligned16(y))
            return KDA_ERR_INVALID_ARG;
        const long long gs = (long long)a.G * a.N;
        if (!valid_ld(a.ldx, a.D, a.dtype) || !valid_ld(a.lddt, a.D, a.dtype) || !valid_ld(a.ldb, gs, a.dtype) ||
            !valid_ld(a.ldc, gs, a.dtype) || (a.z && !valid_ld(a.ldz, a.D, a.dtype)))
            return KDA_ERR_INVALID_ARG;
    }
    const kda_status st = check_ssm_sizes(a.D, a.N, a.G, a.dtype);
    if (st != KDA_OK) return st;
    return a.tokens > kMaxTokens ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

// The inputs of a scan; `s0` where it is read and not also written.
struct SsmSpans {
    Span in[10];
};
SsmSpans ssm_inputs(const kda::SsmArgs& a, const float* s0)
{
    const long long gs = (long long)a.G * a.N;
    return SsmSpans{{rows(a.x, a.ldx, a.D, a.tokens, a.dtype), rows(a.dt, a.lddt, a.D, a.tokens, a.dtype),
                     rows(a.b, a.ldb, gs, a.tokens, a.dtype), rows(a.c, a.ldc, gs, a.tokens, a.dtype),
                     rows(a.z, a.ldz, a.D, a.tokens, a.dtype), floats(a.A, (long long)a.D * a.N), floats(a.skip, a.D),
                     floats(a.dt_bias, a.D), bounds(a.cu, a.nseq), floats(s0, (long long)a.nseq * a.D * a.N)}};
}

// The state may be updated in place: s0 == sT counts as the output alone.
bool ssm_overlap(const kda::SsmArgs& a, const void* y, const float* sT, kda_dtype o_dtype)
{
    const Span out[] = {rows(y, a.D, a.D, a.tokens, o_dtype), floats(sT, (long long)a.nseq * a.D * a.N)};
    return any_overlap(out, ssm_inputs(a, a.s0 == sT ? nullptr : a.s0).in);
}

kda_status ssm_fwd_call(const kda::SsmArgs& a, void* y, float* sT, kda_dtype o_dtype, int mode, void* stream)
{
    const kda_status st = check_ssm(a, y, mode);
    if (st != KDA_OK) return st;
    if (!valid_dtype(o_dtype) || !opt_aligned16(sT) || ssm_overlap(a, y, sT, o_dtype)) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.tokens == 0) return copy_state(a.s0, sT, (size_t)a.nseq * a.D * a.N, s);
    return from_cuda(kda::ssm_fwd(a, y, sT, o_dtype, s));
}

kda_status ssm_bwd_call(const kda::SsmArgs& a, const kda::SsmGrads& g, int mode, bool varlen, void* ws, size_t ws_bytes,
                        void* stream)
{
    kda_status st = check_ssm(a, g.gx, mode);
    if (st != KDA_OK) return st;
    if (!g.gA || !aligned16(g.gA) || !opt_aligned16(g.gsT) || !opt_aligned16(g.gs0)) return KDA_ERR_INVALID_ARG;
    if ((a.skip != nullptr) != (g.gskip != nullptr) || (a.dt_bias != nullptr) != (g.gdt_bias != nullptr) ||
        !opt_aligned16(g.gskip) || !opt_aligned16(g.gdt_bias))
        return KDA_ERR_INVALID_ARG;
    if (a.tokens > 0) {
        if (!g.gy || !g.gdt || !g.gb || !g.gc || (a.z != nullptr) != (g.gz != nullptr)) return KDA_ERR_INVALID_ARG;
        if (!aligned16(g.gy) || !aligned16(g.gdt) || !aligned16(g.gb) || !aligned16(g.gc) || !opt_aligned16(g.gz))
            return KDA_ERR_INVALID_ARG;
    }
    const size_t need =
        a.tokens == 0 ? 0 : kda::ssm_bwd_workspace(a.nseq, a.T, a.tokens, a.D, a.N, a.G, varlen);
    st = check_workspace(ws, ws_bytes, need);
    if (st != KDA_OK) return st;
    const long long act = a.tokens * a.D, bc = a.tokens * a.G * a.N, state = (long long)a.nseq * a.D * a.N;
    const Span out[] = {floats(g.gx, act), floats(g.gdt, act), floats(g.gA, (long long)a.D * a.N), floats(g.gb, bc),
                        floats(g.gc, bc), floats(g.gskip, a.D), floats(g.gz, act), floats(g.gdt_bias, a.D),
                        floats(g.gs0, state), {ws, need}};
    const Span grads[] = {floats(g.gy, act), floats(g.gsT, state)};
    if (any_overlap(out, ssm_inputs(a, a.s0).in) || any_overlap(out, grads)) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.tokens == 0) {
        st = copy_bytes(nullptr, g.gA, (size_t)a.D * a.N * 4, s);
        if (st == KDA_OK) st = copy_bytes(nullptr, g.gskip, (size_t)a.D * 4, s);
        if (st == KDA_OK) st = copy_bytes(nullptr, g.gdt_bias, (size_t)a.D * 4, s);
        if (st == KDA_OK) st = copy_state(g.gsT, g.gs0, (size_t)a.nseq * a.D * a.N, s);
        return st;
    }
    return from_cuda(kda::ssm_bwd(a, g, ws, s));
}

}  // namespace

extern "C" {

kda_status kda_conv_fwd(const void* x, long long ldx, const float* weight, const float* bias,
                        const void* initial_state, void* y, void* final_state, int B, int T, int D, int W,
                        kda_dtype dtype, kda_dtype o_dtype, int mode, void* stream)
{
    if (B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
    return conv_fwd_call(conv_args(x, ldx, weight, bias, nullptr, B, T, (long long)B * T, D, W, dtype, mode),
                         initial_state, y, final_state, o_dtype, mode, stream);
}

kda_status kda_conv_varlen_fwd(const void* x, long long ldx, const float* weight, const float* bias,
                               const int32_t* cu_seqlens, int N, const void* initial_state, void* y,
                               void* final_state, int T, int D, int W, kda_dtype dtype, kda_dtype o_dtype, int mode,
                               void* stream)
{
    const kda_status st = check_cu(cu_seqlens, N, T);
    if (st != KDA_OK) return st;
    return conv_fwd_call(conv_args(x, ldx, weight, bias, cu_seqlens, N, T, T, D, W, dtype, mode), initial_state, y,
                         final_state, o_dtype, mode, stream);
}

kda_status kda_conv_step(const void* x, long long ldx, const float* weight, const float* bias, void* state, void* y,
                         int N, int D, int W, kda_dtype dtype, kda_dtype o_dtype, int mode, void* stream)
{
    if (N < 0) return KDA_ERR_INVALID_ARG;
    const kda::ConvArgs a = conv_args(x, ldx, weight, bias, nullptr, N, 1, N, D, W, dtype, mode);
    const kda_status st = check_conv(a, y, state, nullptr, mode);
    if (st != KDA_OK) return st;
    if (!valid_dtype(o_dtype) || (N > 0 && !state) || conv_overlap(a, nullptr, y, state, o_dtype))
        return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    return from_cuda(kda::conv_step(a, state, y, o_dtype, static_cast<cudaStream_t>(stream)));
}

kda_status kda_conv_bwd(const void* x, long long ldx, const float* weight, const float* bias,
                        const void* initial_state, const float* grad_y, const float* grad_final_state, float* grad_x,
                        float* grad_weight, float* grad_bias, float* grad_initial_state, int B, int T, int D, int W,
                        kda_dtype dtype, int mode, void* workspace, size_t workspace_bytes_, void* stream)
{
    if (B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
    return conv_bwd_call(conv_args(x, ldx, weight, bias, nullptr, B, T, (long long)B * T, D, W, dtype, mode),
                         initial_state, grad_y, grad_final_state, grad_x, grad_weight, grad_bias, grad_initial_state,
                         mode, workspace, workspace_bytes_, stream);
}

kda_status kda_conv_varlen_bwd(const void* x, long long ldx, const float* weight, const float* bias,
                               const int32_t* cu_seqlens, int N, const void* initial_state, const float* grad_y,
                               const float* grad_final_state, float* grad_x, float* grad_weight, float* grad_bias,
                               float* grad_initial_state, int T, int D, int W, kda_dtype dtype, int mode,
                               void* workspace, size_t workspace_bytes_, void* stream)
{
    const kda_status st = check_cu(cu_seqlens, N, T);
    if (st != KDA_OK) return st;
    return conv_bwd_call(conv_args(x, ldx, weight, bias, cu_seqlens, N, T, T, D, W, dtype, mode), initial_state,
                         grad_y, grad_final_state, grad_x, grad_weight, grad_bias, grad_initial_state, mode, workspace,
                         workspace_bytes_, stream);
}

kda_status kda_conv_bwd_workspace_size(long long tokens, int D, int W, size_t* bytes)
{
    if (!bytes || tokens < 0 || D <= 0 || W <= 0) return KDA_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || D % 8 != 0 || D > kMaxChannels || tokens > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    *bytes = tokens == 0 ? 0 : kda::conv_bwd_workspace(tokens, D, W);
    return KDA_OK;
}

kda_status kda_ssm_fwd(const void* x, long long ldx, const void* dt, long long lddt, const float* A, const void* B_,
                       long long ldb, const void* C_, long long ldc, const float* skip, const void* z, long long ldz,
                       const float* dt_bias, const float* initial_state, void* y, float* final_state, int B, int T,
                       int D, int S, int G, kda_dtype dtype, kda_dtype o_dtype, int mode, void* stream)
{
    if (B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
    const kda::SsmArgs a{x, dt, B_, C_, z, ldx, lddt, ldb, ldc, ldz, A, skip, dt_bias, initial_state, nullptr, B, T,
                         (long long)B * T, D, S, G, (mode & KDA_SSM_SOFTPLUS) != 0, dtype};
    return ssm_fwd_call(a, y, final_state, o_dtype, mode, stream);
}

kda_status kda_ssm_varlen_fwd(const void* x, long long ldx, const void* dt, long long lddt, const float* A,
                              const void* B_, long long ldb, const void* C_, long long ldc, const float* skip,
                              const void* z, long long ldz, const float* dt_bias, const int32_t* cu_seqlens, int N,
                              const float* initial_state, void* y, float* final_state, int T, int D, int S, int G,
                              kda_dtype dtype, kda_dtype o_dtype, int mode, void* stream)
{
    const kda_status st = check_cu(cu_seqlens, N, T);
    if (st != KDA_OK) return st;
    const kda::SsmArgs a{x, dt, B_, C_, z, ldx, lddt, ldb, ldc, ldz, A, skip, dt_bias, initial_state, cu_seqlens, N, T,
                         T, D, S, G, (mode & KDA_SSM_SOFTPLUS) != 0, dtype};
    return ssm_fwd_call(a, y, final_state, o_dtype, mode, stream);
}

kda_status kda_ssm_step(const void* x, long long ldx, const void* dt, long long lddt, const float* A, const void* B_,
                        long long ldb, const void* C_, long long ldc, const float* skip, const void* z, long long ldz,
                        const float* dt_bias, float* state, void* y, int N, int D, int S, int G, kda_dtype dtype,
                        kda_dtype o_dtype, int mode, void* stream)
{
    if (N < 0) return KDA_ERR_INVALID_ARG;
    const kda::SsmArgs a{x, dt, B_, C_, z, ldx, lddt, ldb, ldc, ldz, A, skip, dt_bias, nullptr, nullptr, N, 1,
                         N, D, S, G, (mode & KDA_SSM_SOFTPLUS) != 0, dtype};
    const kda_status st = check_ssm(a, y, mode);
    if (st != KDA_OK) return st;
    if (!valid_dtype(o_dtype) || (N > 0 && (!state || !aligned16(state))) || ssm_overlap(a, y, state, o_dtype))
        return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    return from_cuda(kda::ssm_step(a, state, y, o_dtype, static_cast<cudaStream_t>(stream)));
}

kda_status kda_ssm_bwd(const void* x, long long ldx, const void* dt, long long lddt, const float* A, const void* B_,
                       long long ldb, const void* C_, long long ldc, const float* skip, const void* z, long long ldz,
                       const float* dt_bias, const float* initial_state, const float* grad_y,
                       const float* grad_final_state, float* grad_x, float* grad_dt, float* grad_A, float* grad_B,
                       float* grad_C, float* grad_skip, float* grad_z, float* grad_dt_bias, float* grad_initial_state,
                       int B, int T, int D, int S, int G, kda_dtype dtype, int mode, void* workspace,
                       size_t workspace_bytes_, void* stream)
{
    if (B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
    const kda::SsmArgs a{x, dt, B_, C_, z, ldx, lddt, ldb, ldc, ldz, A, skip, dt_bias, initial_state, nullptr, B, T,
                         (long long)B * T, D, S, G, (mode & KDA_SSM_SOFTPLUS) != 0, dtype};
    const kda::SsmGrads g{grad_y, grad_final_state, grad_x, grad_dt, grad_A, grad_B, grad_C, grad_skip, grad_z,
                          grad_dt_bias, grad_initial_state};
    return ssm_bwd_call(a, g, mode, false, workspace, workspace_bytes_, stream);
}

kda_status kda_ssm_bwd_workspace_size(int B, int T, int D, int S, int G, kda_dtype dtype, size_t* bytes)
{
    if (!bytes || B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
    const kda_status st = check_ssm_sizes(D, S, G, dtype);
    if (st != KDA_OK) return st;
    const long long tokens = (long long)B * T;
    if (tokens > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    *bytes = tokens == 0 ? 0 : kda::ssm_bwd_workspace(B, T, tokens, D, S, G, false);
    return KDA_OK;
}

kda_status kda_ssm_varlen_bwd(const void* x, long long ldx, const void* dt, long long lddt, const float* A,
                              const void* B_, long long ldb, const void* C_, long long ldc, const float* skip,
                              const void* z, long long ldz, const float* dt_bias, const int32_t* cu_seqlens, int N,
                              const float* initial_state, const float* grad_y, const float* grad_final_state,
                              float* grad_x, float* grad_dt, float* grad_A, float* grad_B, float* grad_C,
                              float* grad_skip, float* grad_z, float* grad_dt_bias, float* grad_initial_state, int T,
                              int D, int S, int G, kda_dtype dtype, int mode, void* workspace,
                              size_t workspace_bytes_, void* stream)
{
    const kda_status st = check_cu(cu_seqlens, N, T);
    if (st != KDA_OK) return st;
    const kda::SsmArgs a{x, dt, B_, C_, z, ldx, lddt, ldb, ldc, ldz, A, skip, dt_bias, initial_state, cu_seqlens, N, T,
                         T, D, S, G, (mode & KDA_SSM_SOFTPLUS) != 0, dtype};
    const kda::SsmGrads g{grad_y, grad_final_state, grad_x, grad_dt, grad_A, grad_B, grad_C, grad_skip, grad_z,
                          grad_dt_bias, grad_initial_state};
    return ssm_bwd_call(a, g, mode, true, workspace, workspace_bytes_, stream);
}

kda_status kda_ssm_varlen_bwd_workspace_size(int N, int T, int D, int S, int G, kda_dtype dtype, size_t* bytes)
{
    if (!bytes || N < 0 || N > 65535 || T < 0) return KDA_ERR_INVALID_ARG;
    const kda_status st = check_ssm_sizes(D, S, G, dtype);
    if (st != KDA_OK) return st;
    if (T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    *bytes = (N == 0 || T == 0) ? 0 : kda::ssm_bwd_workspace(N, T, T, D, S, G, true);
    return KDA_OK;
}

kda_status kda_selftest_scan_timeout(long long limit_cycles, void* workspace, size_t workspace_bytes_, void* stream)
{
    if (limit_cycles < 1 || limit_cycles > (1LL << 32)) return KDA_ERR_INVALID_ARG;
    const kda_status st = check_workspace(workspace, workspace_bytes_, kda::ssm_bwd_selftest_workspace());
    if (st != KDA_OK) return st;
    return from_cuda(kda::ssm_bwd_selftest(limit_cycles, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
