// Device parts shared by the selective scan's forward and backward kernels.
#pragma once

#include "kda_mixer.cuh"

namespace kda {
namespace mixer {

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool valid)
{
    const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
    const int bytes = valid ? 16 : 0;   // 0: the 16 bytes are zero-filled and src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int K>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(K) : "memory");
}

// softplus(v) = max(v, 0) + log(1 + e^-|v|), to fp32 accuracy for every v.
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

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

struct SsmDev {
    const void *x, *dt, *b, *c, *z;
    long long ldx, lddt, ldb, ldc, ldz;
    const float *A, *skip, *dt_bias, *s0;
    void* y;
    float* sT;
    Seqs q;
    int D, G, tiles;   // tiles: channel tiles per group
    bool softplus, o_bf16;
};

// Shape of a walk: 128 threads; a channel's N states lie on L lanes (NPT states
// each), so a block owns DT = 128 / L channels and walks its sequence in tiles
// of TT tokens.
template <typename T, int N_, int L_>
struct Walk {
    static constexpr int N = N_, L = L_, NPT = N / L, THREADS = 128, DT = THREADS / L;
    static constexpr int TT = L == 4 ? 32 : N == 64 ? 32 : 64;
    static constexpr int EP = TT * DT / THREADS;          // elements per thread outside the walk
    static constexpr int DUROW = 2 * DT + 16;             // floats per token of (Delta, u); rows 16 banks apart
    static constexpr size_t RAW_X = (size_t)TT * DT * sizeof(T), RAW_B = (size_t)TT * N * sizeof(T);
    static constexpr size_t STAGE = 3 * RAW_X + 2 * RAW_B;
    static constexpr size_t SMEM = 2 * STAGE + (size_t)TT * DUROW * 4 + 2 * (size_t)TT * N * 4;
};

// One tile of rows [t0, t0 + TT) of a token-major array into shared memory, 16
// bytes at a time; rows from `stop` on and channels from `nvalid` on are zero.
template <typename T, int TT, int COLS, int THREADS>
__device__ __forceinline__ void fetch_rows(T* dst, const T* src, long long ld, long long t0, long long stop, int nvalid)
{
    constexpr int VE = 16 / sizeof(T), VPR = COLS / VE;
    static_assert(COLS % VE == 0, "row of whole 16-byte vectors");
    for (int i = threadIdx.x; i < TT * VPR; i += THREADS) {
        const int r = i / VPR, v = (i % VPR) * VE;
        const bool ok = t0 + r < stop && v < nvalid;
        cp_async16(dst + r * COLS + v, ok ? src + (t0 + r) * ld + v : src, ok);
    }
}

}  // namespace mixer
}  // namespace kda
