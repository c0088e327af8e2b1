// Shared definitions of the paged-cache kernels: the cache and the step as the kernels see
// them, the placement of a sequence's tokens, and the workspace layout.
#pragma once

#include "common.cuh"

namespace path {
namespace paged {

// Status word: a sequence's lengths or page numbers do not fit the cache.
constexpr uint32_t kStatusCache = 10u;

// Element strides of a per-token tensor: (token, head, ...) with the head's d values contiguous.
struct Stride {
    long long tok, head;
};

struct Cache {
    void *k_pages, *v_pages;  // (pages, Hkv, page, d)
    float *g_pages;           // (K pages, Hq, page), PaTH-FoX
    int *k_table, *v_table;   // (seqs, max_pages)
    int *k_ref, *v_ref;       // (pages)
    int *lens;                // (seqs)
    int seqs, max_pages, page, page_shift, nk, nv, Hq, Hkv, G;
};

struct Step {
    Cache c;
    const void *q, *k, *v, *w;
    const float *beta, *log_f;
    void *out;
    Stride sq, sk, sv, sw, sb, sf, so;
    const int *cu;
    int N, max_chunk;
    float scale_log2;
    uint32_t *status;
};

// Sequence b's tokens: first .. first + T - 1 of the packed step, behind n cached ones.
struct Seq {
    int first, T, n;
};

// T = 0 (and the status word set) where the lengths do not fit the step or the cache.
__device__ __forceinline__ Seq seq_of(const Step &a, int b) {
    const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), n = __ldg(a.c.lens + b);
    Seq s{c0, c1 - c0, n};
    const bool ok = c0 >= 0 && c1 >= c0 && c1 <= a.N && s.T <= a.max_chunk && n >= 0 &&
                    (long long)n + s.T <= ((long long)a.c.max_pages << a.c.page_shift);
    if (!ok) {
        report_status(a.status, kStatusCache);
        s.T = 0;
    }
    return s;
}

// Page number of a sequence's slot, -1 (and the status word set) if it is outside the pool.
__device__ __forceinline__ int page_of(const Step &a, const int *table, int b, int slot, int npool) {
    const int id = __ldg(table + (size_t)b * a.c.max_pages + slot);
    if ((unsigned)id < (unsigned)npool) return id;
    report_status(a.status, kStatusCache);
    return -1;
}

// Blocks of 64 tokens of all sequences share one numbering: block c of sequence b is slot
// cu[b] / 64 + b + c. A sequence's blocks end below the next one's first, because
// ceil(T / 64) <= cu[b+1] / 64 - cu[b] / 64 + 1, so N / 64 + seqs slots hold them all and no
// prefix sum over the sequences is needed.
__host__ __device__ __forceinline__ int slots_of(int N, int seqs) { return N / kC + seqs; }
__device__ __forceinline__ int slot_of(const Seq &s, int b, int c) { return s.first / kC + b + c; }

// The (sequence, block) of a slot; false for a slot that no block has. The first slots of
// the sequences rise with b, so a binary search finds the last one at or below the slot.
__device__ __forceinline__ bool block_of(const Step &a, int slot, int &b, int &c, Seq &s) {
    int lo = 0, hi = a.c.seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(a.cu + mid) / kC + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    b = lo;
    s = seq_of(a, b);
    c = slot - (s.first / kC + b);
    return c >= 0 && c * kC < s.T;
}

// PaTH-FoX: sums of a block's 64 gates, formed by one warp in fp64; lane t holds those of tokens t
// and t + 32.
//   before  f_0 + ... + f_t
//   behind  f_{t+1} + ... + f_63
//   pair    as `before`, but fit for differences: pair_i - pair_j is the sum of the gates behind j up
//           to i
// A difference loses what lies below 2^-53 of the sums, so a gate that closes for good (-1e30, the
// type's lowest value) would take the block's other gates with it. Where a gate is as large as
// kClosed, it counts as kClosed in `pair`: the sums then stay within 2^30 and a difference is right to
// 2^-22, and a key behind such a gate has no weight either way (logits in fp32 are whole numbers
// apart there). `behind` is then summed from the end; else it is the block's sum less `before`.
struct GateSums {
    double before[2], behind[2], pair[2], all;
};
constexpr double kClosed = 16777216.0;  // 2^24

// (UNROLL 1 for the rare form: what a CTA seldom runs stays short; unrolled it cost first chunks 1 us)
template <int UNROLL>
__device__ __forceinline__ void gate_prefix(double (&x)[2], int lane) {
#pragma unroll UNROLL
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const double z = __shfl_up_sync(0xffffffffu, x[half], o);
            if (lane >= o) x[half] += z;
        }
    x[1] += __shfl_sync(0xffffffffu, x[0], 31);
}

__device__ __forceinline__ GateSums gate_sums(double f0, double f1, int lane) {
    GateSums g;
    g.before[0] = f0;
    g.before[1] = f1;
    gate_prefix<5>(g.before, lane);
    g.all = __shfl_sync(0xffffffffu, g.before[1], 31);
    if (!__any_sync(0xffffffffu, fmax(fabs(f0), fabs(f1)) >= kClosed)) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            g.pair[half] = g.before[half];
            g.behind[half] = g.all - g.before[half];
        }
        return g;
    }
    g.pair[0] = fmin(fmax(f0, -kClosed), kClosed);
    g.pair[1] = fmin(fmax(f1, -kClosed), kClosed);
    gate_prefix<1>(g.pair, lane);
    double s[2] = {f0, f1};  // sums of a half from its lane on
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const double z = __shfl_down_sync(0xffffffffu, s[half], o);
            if (lane + o < 32) s[half] += z;
        }
    const double upper = __shfl_sync(0xffffffffu, s[1], 0);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const double z = __shfl_down_sync(0xffffffffu, s[half], 1);
        g.behind[half] = lane < 31 ? z : 0.0;
    }
    g.behind[0] += upper;
    return g;
}

// The four 16 x 16 diagonal blocks of (I + E)^{-1} for a strictly lower triangular E (64 x 64,
// shared, stride LD), by substitution (one column per thread of the first 64), in place.
template <int LD>
__device__ __forceinline__ void diagonal_inverses(float *E, int tid) {
    const int b0 = (tid >> 4) << 4, lu = tid & 15;
    float x[16];
    if (tid < kC) {
#pragma unroll
        for (int l = 0; l < 16; ++l) x[l] = l == lu ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 15; ++m)
#pragma unroll
            for (int l = m + 1; l < 16; ++l) x[l] = fmaf(-E[(b0 + l) * LD + b0 + m], x[m], x[l]);
    }
    __syncthreads();
    if (tid < kC)
#pragma unroll
        for (int l = 0; l < 16; ++l) E[(b0 + l) * LD + tid] = x[l];
    __syncthreads();
}

// (I + E)^{-1} in fp32: the diagonal blocks, then X21 = -X22 E21 X11 for the 16- and the
// 32-blocks; every factor is bounded (products of contractions), so nothing grows.
// 256 threads. `Y`: 32 x 36 floats of scratch; nt: the 16-row tiles in use (the others are the identity).
template <int LD>
__device__ __forceinline__ void unit_lower_inverse(float *E, float *Y, int tid, int nt) {
    constexpr int YL = 36, kThr = 256;
    diagonal_inverses<LD>(E, tid);
    if (nt <= 1) return;
    // level 1: two 32-blocks at o, X21 (16 x 16)
    for (int pass = 0; pass < 2; ++pass) {
        float v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = tid + i * kThr, o = 32 * (e >> 8), r = (e >> 4) & 15, c = e & 15;
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                t = pass == 0 ? fmaf(E[(o + 16 + r) * LD + o + k], E[(o + k) * LD + o + c], t)
                              : fmaf(E[(o + 16 + r) * LD + o + 16 + k], Y[((o >> 1) + k) * YL + c], t);
            v[i] = t;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = tid + i * kThr, o = 32 * (e >> 8), r = (e >> 4) & 15, c = e & 15;
            if (pass == 0) Y[((o >> 1) + r) * YL + c] = v[i];
            else E[(o + 16 + r) * LD + o + c] = -v[i];
        }
        __syncthreads();
    }
    if (nt <= 2) return;
    // level 2: X21 (32 x 32)
    for (int pass = 0; pass < 2; ++pass) {
        float v[4];
        const int r = tid >> 3, c0 = (tid & 7) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = 0.f;
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float l = pass == 0 ? E[(32 + r) * LD + k] : E[(32 + r) * LD + 32 + k];
            const float4 q = *reinterpret_cast<const float4 *>(pass == 0 ? E + k * LD + c0 : Y + k * YL + c0);
            v[0] = fmaf(l, q.x, v[0]);
            v[1] = fmaf(l, q.y, v[1]);
            v[2] = fmaf(l, q.z, v[2]);
            v[3] = fmaf(l, q.w, v[3]);
        }
        __syncthreads();
        float *dst = pass == 0 ? Y + r * YL + c0 : E + (32 + r) * LD + c0;
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = pass == 0 ? v[i] : -v[i];
        __syncthreads();
    }
}

// The kernels of one call follow each other as programmatic dependents: the next one's CTAs
// may come up while the last ones of the one before still run, and look up there which sequence and
// block they have; the kernels with barriers and tensor memory set these up behind grid_wait. Up to
// grid_wait they read only what the caller gave (cu_tokens, lengths, tables, the step's own
// tensors: complete since before the call's first kernel, which is launched as any other) and
// write nothing that an earlier kernel of the call reads or writes. What a kernel of the call writes
// is read by plain loads (not __ldg, no __restrict__, which promise that nobody writes it while the
// reader lives). Every CTA waits, also those without work, so a kernel's end implies the ends of all
// before it.
__device__ __forceinline__ void grid_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch behind another kernel of the same call (first: behind whatever the stream holds).
template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, bool first,
                   A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = first ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace paged
}  // namespace path
