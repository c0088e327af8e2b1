// Helpers of the fp32 kernels of a step over a paged cache, and their pass over cached keys, which
// paged_f32.cu and paged_prefix_f32.cu share.
#pragma once

#include <climits>

#include "paged.cuh"

namespace path {
namespace paged {

namespace {

constexpr int LD = 68;             // padded row stride (floats) of a 64 x 64 shared tile
constexpr int TILE = kC * LD;
constexpr int kThr = 256;          // thread (ty, tx) = (tid / 16, tid % 16)

using Acc = float[4][4];

__device__ __forceinline__ void zero(Acc &c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
}

// c[i][j] += sum_k A[ty + 16 i][k] B[tx + 16 j][k]
__device__ __forceinline__ void mm_nt(const float *A, const float *B, Acc &c) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 4
    for (int k = 0; k < kC; k += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * LD + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * LD + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float t = c[i][j];
                t = fmaf(a[i].x, b[j].x, t);
                t = fmaf(a[i].y, b[j].y, t);
                t = fmaf(a[i].z, b[j].z, t);
                c[i][j] = fmaf(a[i].w, b[j].w, t);
            }
    }
}

// c[i][j] += sum_k A[ty + 16 i][k] B[k][4 tx + j]
__device__ __forceinline__ void mm_nn(const float *A, const float *B, Acc &c) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 4
    for (int k = 0; k < kC; k += 4) {
        float4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * LD + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const float4 b = *reinterpret_cast<const float4 *>(B + (k + kk) * LD + 4 * tx);
            const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float av = kk == 0 ? a[i].x : kk == 1 ? a[i].y : kk == 2 ? a[i].z : a[i].w;
#pragma unroll
                for (int j = 0; j < 4; ++j) c[i][j] = fmaf(av, bv[j], c[i][j]);
            }
        }
    }
}

// c[i][j] += sum_k A[k][ty + 16 i] B[k][4 tx + j]
__device__ __forceinline__ void mm_tn(const float *A, const float *B, Acc &c) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 8
    for (int k = 0; k < kC; ++k) {
        const float4 b = *reinterpret_cast<const float4 *>(B + k * LD + 4 * tx);
        const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float av = A[k * LD + ty + 16 * i];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i][j] = fmaf(av, bv[j], c[i][j]);
        }
    }
}

// an mm_nt tile into shared memory
__device__ __forceinline__ void put_nt(float *dst, const Acc &c) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[(ty + 16 * i) * LD + tx + 16 * j] = c[i][j];
}
// an mm_nn / mm_tn tile into shared memory
__device__ __forceinline__ void put_nn(float *dst, const Acc &c) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(dst + (ty + 16 * i) * LD + 4 * tx) =
            make_float4(c[i][0], c[i][1], c[i][2], c[i][3]);
}

// 64 rows of D contiguous fp32 in global memory into D / 64 shared tiles
template <int D>
__device__ __forceinline__ void load_rows(float *dst, const float *src) {
    for (int e = threadIdx.x; e < kC * D / 4; e += kThr) {
        const int r = 4 * e / D, c = 4 * e % D;
        *reinterpret_cast<float4 *>(dst + (c >> 6) * TILE + r * LD + (c & 63)) =
            *reinterpret_cast<const float4 *>(src + (size_t)r * D + c);
    }
}

__device__ __forceinline__ float4 get4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void set4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }

// tokens i0 .. of one head (rows past `rows` zero) into D / 64 shared tiles
template <int D>
__device__ __forceinline__ void load_tokens(float *dst, const void *src, Stride st, long long first,
                                            int head, int rows) {
    for (int e = threadIdx.x; e < kC * D / 4; e += kThr) {
        const int r = 4 * e / D, c = 4 * e % D;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows)
            x = get4(static_cast<const float *>(src) + (first + r) * st.tok + head * st.head + c);
        *reinterpret_cast<float4 *>(dst + (c >> 6) * TILE + r * LD + (c & 63)) = x;
    }
}

// The page numbers of the slots of 64 cached positions from j0 (-1: bad, or nothing there is in
// sight); returns the first slot.
template <typename A>
__device__ __forceinline__ int find_pages(const A &a, int *ids, const int *table, int pool, int b, int j0, int n,
                                          const Sight &seen) {
    const int slot0 = j0 >> a.c.page_shift, last = (min(j0 + kC, n) - 1) >> a.c.page_shift, i = threadIdx.x;
    if (i <= last - slot0)
        ids[i] = seen.any((slot0 + i) << a.c.page_shift, a.c.page) ? page_of(a, table, b, slot0 + i, pool) : -1;
    return slot0;
}

// 64 cached positions from j0 of one key head into shared tiles; positions at or past n, out of sight
// and those of bad pages are zero. ids: page numbers of the positions' slots from slot0.
template <int D>
__device__ __forceinline__ void load_cached(float *dst, const void *pages, const Cache &c, const int *ids,
                                            int slot0, int h, int j0, int n, const Sight &seen) {
    for (int e = threadIdx.x; e < kC * D / 4; e += kThr) {
        const int r = 4 * e / D, col = 4 * e % D, j = j0 + r;
        const int id = j < n && seen.sees(j) ? ids[(j >> c.page_shift) - slot0] : -1;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (id >= 0)
            x = get4(static_cast<const float *>(pages) +
                     ((((size_t)id * c.Hkv + h) << c.page_shift) + (j & (c.page - 1))) * D + col);
        *reinterpret_cast<float4 *>(dst + (col >> 6) * TILE + r * LD + (col & 63)) = x;
    }
}

// The online softmax of a 64 x 64 tile of log2-unit logits in shared memory (masked entries
// -inf): replaces the logits by their weights and updates the rows' maximum and sum; alpha[r]
// is the factor of what the row had before. A row that has nothing yet keeps -inf and 0.
__device__ __forceinline__ void softmax_rows(float *S, float *m, float *l, float *alpha) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < kC; r += kThr / 32) {
        const float x0 = S[r * LD + lane], x1 = S[r * LD + lane + 32];
        float mx = fmaxf(x0, x1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mo = m[r], mn = fmaxf(mo, mx);
        const float use = mn == -INFINITY ? 0.f : mn;
        const float p0 = exp2f(x0 - use), p1 = exp2f(x1 - use);
        float sum = p0 + p1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        S[r * LD + lane] = p0;
        S[r * LD + lane + 32] = p1;
        __syncwarp();
        if (lane == 0) {
            const float al = exp2f(mo - use);
            alpha[r] = al;
            m[r] = mn;
            l[r] = l[r] * al + sum;
        }
    }
}

template <int NH>
__device__ __forceinline__ void scale_rows(Acc (&o)[NH], const float *alpha) {
    const int ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float al = alpha[ty + 16 * i];
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[h][i][j] *= al;
    }
}

// one softmax part: rows of D values, then the rows' maxima and sums
template <int D>
__device__ __forceinline__ void store_part(float *p, const Acc (&o)[D / 64], const float *m, const float *l) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(p + (ty + 16 * i) * D + 64 * h + 4 * tx) =
                make_float4(o[h][i][0], o[h][i][1], o[h][i][2], o[h][i][3]);
    if (threadIdx.x < kC) {
        p[kC * D + threadIdx.x] = m[threadIdx.x];
        p[kC * D + kC + threadIdx.x] = l[threadIdx.x];
    }
}

struct Ws {
    float *qt, *kt, *pb, *part, *gq, *gt, *ptot;
    double *gtot;
    int splits;
    bool singles;  // sequences of one token go to the one-pass kernels
    __device__ __forceinline__ bool takes(const Seq &s) const { return !(singles && s.T == 1); }
};
template <int D> constexpr size_t kPart = (size_t)kC * (D + 2);

// ---------------------------------------------------------------- cached keys
// Tiles of 64 positions of split sp of so many in sight.
__device__ __forceinline__ void split_range(int tiles, int splits, int sp, int &t0, int &t1) {
    const int per = (tiles + splits - 1) / splits;
    t0 = min(tiles, sp * per);
    t1 = min(tiles, t0 + per);
}

template <int D>
constexpr size_t cached_smem() { return ((size_t)(3 * (D / 64) + 1) * TILE + 4 * kC) * 4 + 16 * 4; }

// SHARED: over the keys of prefixes (paged_prefix.cuh), whose rows are placed by a kernel of this call.
template <int D, bool SHARED, typename A>
__global__ void __launch_bounds__(kThr) f32_cached_kernel(const A a, const Ws y) {
    constexpr int NH = D / 64;
    extern __shared__ float sm[];
    float *X = sm, *K = X + NH * TILE, *V = K + NH * TILE, *S = V + NH * TILE, *m = S + TILE,
          *l = m + kC, *alpha = l + kC, *gj = alpha + kC;
    int *kid = reinterpret_cast<int *>(gj + kC), *vid = kid + 8;
    const int slot = blockIdx.x, hq = blockIdx.y, sp = blockIdx.z, h = hq / a.c.G, tid = threadIdx.x;
    const int ty = tid >> 4, tx = tid & 15;
    int b, c, t0, t1;
    Seq s;
    grid_begin();
    if (SHARED) grid_wait();
    const bool mine = block_of(a, slot, b, c, s) && y.takes(s);
    if (!SHARED) grid_wait();
    if (!mine) return;
    const Sight seen = sight_of(a, s);
    split_range(seen.tiles(s.n, kC), y.splits, sp, t0, t1);
    if (t0 >= t1) return;
    const size_t bq = (size_t)slot * a.c.Hq + hq;
    load_rows<D>(X, y.qt + bq * kC * D);
    if (tid < kC) {
        m[tid] = -INFINITY;
        l[tid] = 0.f;
    }
    float gq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) gq[i] = a.log_f != nullptr ? y.gq[bq * kC + ty + 16 * i] : 0.f;
    Acc o[NH];
#pragma unroll
    for (int x = 0; x < NH; ++x) zero(o[x]);
    // a window: row i of the block sees the positions from `from` + i on, and the sinks
    const int from = s.n + c * kC + 1 - window_of(a), past = window_of(a) > 0 ? sinks_of(a) : INT_MAX;
    for (int t = t0; t < t1; ++t) {
        const int j = kC * seen.tile(t, s.n, kC);
        __syncthreads();
        const int slot0 = find_pages(a, kid, a.c.k_table, a.c.nk, b, j, s.n, seen);
        find_pages(a, vid, a.c.v_table, a.c.nv, b, j, s.n, seen);
        __syncthreads();
        load_cached<D>(K, a.c.k_pages, a.c, kid, slot0, h, j, s.n, seen);
        load_cached<D>(V, a.c.v_pages, a.c, vid, slot0, h, j, s.n, seen);
        if (tid < kC) {
            // the key's gate sum; -inf where there is no such key
            const int jj = j + tid, sl = (jj >> a.c.page_shift) - slot0;
            const bool in = jj < s.n && kid[sl] >= 0 && vid[sl] >= 0;
            float g = in ? 0.f : -INFINITY;
            if (in && a.log_f != nullptr)
                g = a.c.g_pages[(((size_t)kid[sl] * a.c.Hq + hq) << a.c.page_shift) + (jj & (a.c.page - 1))];
            gj[tid] = g;
        }
        __syncthreads();
        Acc c0;
        zero(c0);
#pragma unroll
        for (int x = 0; x < NH; ++x) mm_nt(X + x * TILE, K + x * TILE, c0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                S[(ty + 16 * i) * LD + tx + 16 * q] =
                    j + tx + 16 * q >= past && j + tx + 16 * q < from + ty + 16 * i
                        ? -INFINITY
                        : fmaf(gq[i] + gj[tx + 16 * q], kLog2e, c0[i][q] * a.scale_log2);
        __syncthreads();
        softmax_rows(S, m, l, alpha);
        __syncthreads();
        scale_rows<NH>(o, alpha);
#pragma unroll
        for (int x = 0; x < NH; ++x) mm_nn(S, V + x * TILE, o[x]);
    }
    __syncthreads();
    store_part<D>(y.part + (bq * (1 + y.splits) + 1 + sp) * kPart<D>, o, m, l);
}

template <typename K>
cudaError_t big_smem(K kern, size_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

}  // namespace paged
}  // namespace path
