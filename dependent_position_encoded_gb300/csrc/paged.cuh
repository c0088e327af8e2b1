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

// The kernels of one call follow each other as programmatic dependents: the next one's CTAs
// may come up (barriers, tensor memory) while the last ones of the one before still run, and
// wait here before they touch memory. Every CTA waits before anything else that counts, so a
// kernel's end implies the ends of all before it.
__device__ __forceinline__ void grid_wait() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

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
