// The bf16 block path of a step over a paged cache: workspace and warp-level product helpers.
//
// Rows. The Hq / Hkv = G query heads of a key head are taken together: row t G + g of a
// sequence is query head g of its new token t, so that 128 consecutive rows (one tensor-core
// tile) hold as many tokens as share the cached keys. All sequences' rows of a key head stand
// one behind the other, R = N G of them.
#pragma once

#include <climits>
#include <type_traits>

#include "paged.cuh"

namespace path {
namespace paged {

// Work on cached keys. A unit is one tile of 128 NT rows against one tile of 128 cached
// positions; an item is a row tile with all its key tiles. Items are ordered by sequence, key
// head and row tile, and their units numbered through; each of `ctas` resident CTAs takes `per`
// consecutive units, whatever the sequences' lengths, so the load is even and only items that
// reach over a border have several parts. Sequences whose rows fit one tile go with NT = 1, the
// others with NT = 2 (one_tile).
struct Plan {
    long long *units, *items;  // (seqs + 1): units and items before each sequence
    int ctas;
};

// What a pass over cached keys does: that of a step over its own cache, the same seen through a
// window, that of single tokens (a window or none), or one over keys that several sequences share,
// which stay as they are.
enum class Pass { step, window, one, shared };

// Whether a carried query enters the cached keys' logits as a high and a low bf16 part. Rounded
// once to bf16 it adds as much error to the output as the weights' and the output's own rounding
// do: 2.9e-3 of the norm against 2.3e-3 with the second part and 1.7e-3 for the output's rounding
// alone, for single tokens. The second product costs 4 to 6% where the cache's bytes bound the pass (NT = 1: 207 ->
// 215 us for 32 sequences of 8192 at D = 64) and little beside the exponentials at D = 64; at
// D = 128 with several row tiles shared memory has no room for the parts.
__host__ __device__ constexpr bool keeps_low(int NT, int D) { return NT == 1 || D == 64; }

// Workspace of the bf16 block path, behind the 256-byte status header:
//   qt   (Hkv, R, D) bf16       queries carried to the chunk's start, times scale log2(e)
//   ql   (Hkv, R, D) bf16       what that rounding left, where keeps_low
//   po   (Hkv, R, D) fp32, pml (Hkv, R) fp32 pairs: the step's own tokens' unnormalised softmax
//        part and its (maximum in log2 units, sum)
//   so, sml per NT: (ctas + items, 128 NT, D) fp32 and (.., 128 NT) pairs, the parts of the
//        cached keys: the part that CTA c has of item i is number c + i
//   gq   (Hkv, R) fp32          PaTH-FoX: gate sum of a row from the chunk's start
//   gt   (slots, Hq, 64) fp32   PaTH-FoX: gate sum behind a key to its block's end
//   gtot (slots, Hq) fp64       PaTH-FoX: gate sum of a block
//   gblk (slots, Hq, 2) fp32    PaTH-FoX: the same rounded, and the largest of the block's gt
//   mt   (min(seqs, N), Hkv, 2, D, D) bf16 high and low parts of (H_1 ... H_T) - I of the chunk
// and, where a chunk may have several blocks of 64 tokens:
//   kh, kl (slots, Hkv, 64 + D, D) bf16 high and low parts of [k~; P_b - I]
//   vb   (slots, Hkv, 64, D) bf16 the block's values, zero past its tokens
// and, where it may have several groups of blocks (paged_prep_tc.cuh):
//   ch, cl (slots, Hkv, 64, D) bf16 high and low parts of the new keys at their group's end
//   gp   (groups, Hkv, 2, D, D) bf16 high and low parts of the groups' products less I
struct TcWs {
    __nv_bfloat16 *qt, *ql, *mt, *kh, *kl, *vb, *ch, *cl, *gp;
    float *po;
    float2 *pml;
    float *so[2];
    float2 *sml[2];
    Plan plan[2];
    float *gq, *gt;
    double *gtot;
    float2 *gblk;
    long long R;
};

// A sequence's row of mt: with more sequences than tokens (most of them idle) its first token.
__device__ __forceinline__ size_t mt_row(const Step &a, const Seq &s, int b) {
    return a.N < a.c.seqs ? s.first : b;
}

// Whether a sequence goes with NT = 1. At D = 64 without gates one of several blocks does not: its
// queries have been through the scan's roundings, and there only the pass of NT = 2 makes up for
// that with the weights' second part (low_weights).
__host__ __device__ __forceinline__ bool one_tile(int T, int G, int D, bool fox) {
    return (T <= kC || D == 128 || fox) && (long long)T * G <= 128;
}

// Rows of a prefix's queries up to which they go by one row tile at a time (NT = 1).
// At D = 64 all of them: two CTAs on an SM, each with a tile, are ahead of one CTA with two (one token each
// of G = 4 behind 16,384 keys, 384 rows 54 us against 66, 16,384 rows 1,219 against 1,380; with gates 90 and
// 97, 2,172 and 2,288), but that queries of several blocks need the weights' second part (low_weights),
// unless there are gates.
// At D = 128 a key slot is worth two tiles (1,536 rows: 319 us by one, 309 by two; 10,000 rows of chunks of
// up to 512: 1,259 and 1,121), but two leave no room for the queries' second part (keeps_low), whose
// rounding is behind a prefix of thousands the largest. Errors of the output by one and by two, in
// chunks of 7: 2.27e-3 and 2.55e-3 of the norm, 64: 2.35 and 2.54, 100: 2.31 and 2.47, 200: 2.33 and 2.42,
// 500: 2.33 and 2.29, whose chunks' own roundings are the most by then. With gates few keys count: 1.9e-3.
inline int prefix_one_rows(int D, int max_chunk, bool fox) {
    return (D == 64 ? max_chunk <= kC || fox : max_chunk <= 4 * kC && !fox) ? INT_MAX : 128;
}

// Whether queries carried to the chunk's start are left in two parts: for the cached keys' pass, or to
// be carried on to a prefix.
__device__ __forceinline__ bool low_queries(const Step &a, int T, int D) {
    return keeps_low(one_tile(T, a.c.G, D, a.log_f != nullptr) ? 1 : 2, D);
}
__device__ __forceinline__ bool low_queries(const StepMore &a, int T, int D) {
    return a.prefix_of != nullptr || keeps_low(one_tile(T, a.c.G, D, a.log_f != nullptr) ? 1 : 2, D);
}

__host__ __device__ constexpr int rows_by_one(const Step &) { return 0; }  // (a plain step has no prefixes)
__host__ __device__ inline int rows_by_one(const StepMore &a) { return a.one_rows; }

// Row tiles and key tiles of a sequence in the plan of NT (0 where it goes with the other).
template <typename A>
__device__ __forceinline__ void plan_of(const A &a, const Seq &s, int D, int NT, int &tiles, int &ktiles) {
    const int G = a.c.G, rows = s.T * G;  // T G <= N G, which the host keeps within an int
    ktiles = sight_of(a, s).tiles(s.n, 128);
    const bool one = enters(a) ? one_tile(s.T, G, D, a.log_f != nullptr) : rows <= rows_by_one(a);
    tiles = one == (NT == 1) ? (rows + 128 * NT - 1) / (128 * NT) : 0;
}

// Units per CTA: at least two, so that a part is worth its join.
__device__ __forceinline__ long long plan_per(const Plan &p, int seqs) {
    const long long all = p.units[seqs], per = (all + p.ctas - 1) / p.ctas;
    return per < 2 ? 2 : per;
}

// The stretch of units from u on that lies in one item and below `end`.
struct Stretch {
    Seq s;
    int b, h, tile, k0, steps, kt;  // kt: key tiles of the item
    long long item;  // over all sequences
};
// One after the other: the sequence of the last one is kept, since its next key head or row tile mostly
// comes next, and a look-up is half a dozen loads that wait for each other. (Walk().at(): looked up anew.)
struct Walk {
    long long u0 = 0, u1 = -1, items = 0;  // the sequence's units and its first item
    Seq s;
    int b, tiles, kt;
    template <typename A>
    __device__ __forceinline__ Stretch at(const A &a, const Plan &p, int D, int NT, long long u, long long end) {
        if (u >= u1) {
            int lo = 0, hi = a.c.seqs - 1;  // the last sequence with units[b] <= u: it has units
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.units[mid] <= u) lo = mid;
                else hi = mid - 1;
            }
            b = lo;
            s = seq_of(a, lo);
            plan_of(a, s, D, NT, tiles, kt);
            u0 = p.units[lo];
            u1 = p.units[lo + 1];
            items = p.items[lo];
        }
        Stretch t;
        t.b = b;
        t.s = s;
        const long long rem = u - u0;
        const int it = (int)(rem / kt);
        t.k0 = (int)(rem - (long long)it * kt);
        t.kt = kt;
        t.h = it / tiles;
        t.tile = it - t.h * tiles;
        t.item = items + it;
        const long long left = end - u;
        t.steps = kt - t.k0 < left ? kt - t.k0 : (int)left;
        return t;
    }
};

constexpr int kThr = 256;  // threads of a CTA of the kernels beside the attention's

// Units and items of cached-key work before each sequence (one CTA, both plans). The parts'
// buffers hold what sequences without common tokens can need, so one that begins before an
// earlier one's begin or end (cu_tokens falls somewhere, which the falling sequence reports) gets
// no work: with m the largest cu_tokens so far, a sequence counts where cu_tokens = m.
template <int D, typename A>
__device__ __forceinline__ void make_plans(const A &a, const TcWs &y, long long *sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *const tops = reinterpret_cast<int *>(sums + kThr / 32);
    long long run[4] = {0, 0, 0, 0};
    int top = 0;
    for (int base = 0; base <= a.c.seqs; base += kThr) {
        const int b = base + tid;
        const int begin = b < a.c.seqs ? cu_at(a, b) : 0;
        int m = begin;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o) m = max(m, t);
        }
        __syncthreads();
        if (lane == 31) tops[warp] = m;
        __syncthreads();
        m = max(m, top);
#pragma unroll
        for (int i = 0; i < kThr / 32; ++i) {
            if (i < warp) m = max(m, tops[i]);
            top = max(top, tops[i]);
        }
        long long v[4] = {0, 0, 0, 0};
        if (b < a.c.seqs && begin == m) {
            const Seq s = seq_of(a, b);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                int tiles, kt;
                plan_of(a, s, D, p + 1, tiles, kt);
                v[2 * p + 1] = kt > 0 ? (long long)tiles * a.c.Hkv : 0;
                v[2 * p] = v[2 * p + 1] * kt;
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            long long x = v[q];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += t;
            }
            __syncthreads();
            if (lane == 31) sums[warp] = x;
            __syncthreads();
            long long before = run[q], all = 0;
#pragma unroll
            for (int i = 0; i < kThr / 32; ++i) {
                if (i < warp) before += sums[i];
                all += sums[i];
            }
            if (b <= a.c.seqs) (q & 1 ? y.plan[q >> 1].items : y.plan[q >> 1].units)[b] = before + x - v[q];
            run[q] += all;
        }
    }
}

// A sequence's only token: H = I - beta w w^T, q~ = q - beta (w . q) w, and the token's own key
// and value enter the cache as they are. A warp per query head in turns.
template <int D, typename A>
__device__ __forceinline__ void enter_single(const A &a, const TcWs &y, const Seq &s, int b, int slot, int h) {
    using bf = __nv_bfloat16;
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.c.G, kw = kThr / 32;
    const float beta = a.beta[(long long)s.first * a.sb.tok + h * a.sb.head];
    auto row = [&](const void *p, Stride st, int head) {
        return static_cast<const bf *>(p) + (long long)s.first * st.tok + (long long)head * st.head + lane * E;
    };
    const bf *const wp = row(a.w, a.sw, h), *const kp = row(a.k, a.sk, h), *const vp = row(a.v, a.sv, h);
    float w[E], k[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        w[e] = __bfloat162float(wp[e]);
        k[e] = __bfloat162float(kp[e]);
    }
    const int pos = s.n, sl = pos >> a.c.page_shift, off = pos & (a.c.page - 1);
    const int kid = page_of(a, a.c.k_table, b, sl, a.c.nk), vid = page_of(a, a.c.v_table, b, sl, a.c.nv);
    if (warp == kw - 1) {
        if (kid >= 0)
#pragma unroll
            for (int e = 0; e < E; ++e)
                static_cast<bf *>(a.c.k_pages)[((((size_t)kid * a.c.Hkv + h) << a.c.page_shift) + off) * D + lane * E +
                                               e] = kp[e];
        if (vid >= 0)
#pragma unroll
            for (int e = 0; e < E; ++e)
                static_cast<bf *>(a.c.v_pages)[((((size_t)vid * a.c.Hkv + h) << a.c.page_shift) + off) * D + lane * E +
                                               e] = vp[e];
    }
    for (int g = warp; g < G; g += kw) {
        const int hq = h * G + g;
        const bf *const qp = row(a.q, a.sq, hq);
        float q[E], wq = 0.f, kq = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            q[e] = __bfloat162float(qp[e]);
            wq = fmaf(w[e], q[e], wq);
            kq = fmaf(k[e], q[e], kq);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            wq += __shfl_xor_sync(0xffffffffu, wq, o);
            kq += __shfl_xor_sync(0xffffffffu, kq, o);
        }
        const size_t r = (size_t)h * y.R + (size_t)s.first * G + g;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float x = fmaf(-beta * wq, w[e], q[e]) * a.scale_log2;
            const bf xh = __float2bfloat16_rn(x);
            y.qt[r * D + lane * E + e] = xh;
            if (low_queries(a, 1, D))
                y.ql[r * D + lane * E + e] = __float2bfloat16_rn(x - __bfloat162float(xh));
            y.po[r * D + lane * E + e] = __bfloat162float(vp[e]);
        }
        if (lane == 0) {
            y.pml[r] = make_float2(kq * a.scale_log2, 1.f);
            if (a.log_f != nullptr) {
                const float f = a.log_f[(long long)s.first * a.sf.tok + (long long)hq * a.sf.head];
                y.gq[r] = f;
                y.gtot[(size_t)slot * a.c.Hq + hq] = f;
                if (kid >= 0) a.c.g_pages[(((size_t)kid * a.c.Hq + hq) << a.c.page_shift) + off] = 0.f;
            }
        }
    }
}

// The parts of the prefixes' pass (paged_prefix.cuh), for the step's joining; of: null where the step has
// none.
struct Behind {
    const int *of, *cu, *start;
    float *so[2];
    float2 *sml[2];
    Plan plan[2];
};

// The parts of a row, row `r` of sequence b's and key head h's, that the pass over cached keys left: number
// of the first, how many, and where they begin (part q at `first` + (q >> copies) * tile + (q & ..) * (128 >> copies)).
struct RowParts {
    long long first;
    int number, copies, tile;
    const float *so;
    const float2 *sml;
    __device__ __forceinline__ size_t at(int q) const {
        return first + (size_t)(q >> copies) * tile + (q & ((1 << copies) - 1)) * (128 >> copies);
    }
};
// rows: those of the sequence and key head; kt: its key tiles; one: whether it goes with NT = 1.
template <typename Y>
__device__ __forceinline__ RowParts parts_of(const Y &y, int seqs, int rows, int kt, bool one, int b, int h, int r) {
    const Plan &p = one ? y.plan[0] : y.plan[1];
    const int tile = one ? 128 : 256, tiles = (rows + tile - 1) / tile, it = h * tiles + r / tile;
    RowParts x{0, 0, !one ? 0 : rows <= 32 ? 2 : rows <= 64 ? 1 : 0, tile, one ? y.so[0] : y.so[1],
               one ? y.sml[0] : y.sml[1]};
    // (none where the sequence has no work)
    if (kt > 0 && p.items[b + 1] > p.items[b]) {
        const long long per = plan_per(p, seqs), u = p.units[b] + (long long)it * kt, c0 = u / per;
        x.first = (c0 + p.items[b] + it) * tile + r % tile;
        x.number = ((int)((u + kt - 1) / per - c0) + 1) << x.copies;
    }
    return x;
}
// The parts of sequence b's row of new token t and query head g of key head h with its prefix.
template <typename A>
__device__ __forceinline__ RowParts parts_behind(const A &a, const Behind &x, int b, int h, int t, int g) {
    const int start = x.start[b];
    if (start < 0) return RowParts{};
    const int p = __ldg(x.of + b), first = x.cu[p], rows = (x.cu[p + 1] - first) * a.c.G;
    return parts_of(x, a.c.seqs, rows, (__ldg(a.c.lens + p) + 127) / 128, rows <= rows_by_one(a), p, h,
                    (start - first + t) * a.c.G + g);
}

// Rows of `rows` per tile over all sequences: tile i of sequence b is slot
// cu[b] G / rows + b + i (as slots_of).
__host__ __device__ __forceinline__ int tile_slots(int N, int G, int seqs, int rows) {
    return (int)((long long)N * G / rows) + seqs;
}
template <typename A>
__device__ __forceinline__ bool tile_of(const A &a, int slot, int rows, int &b, int &i, Seq &s) {
    const int G = a.c.G;
    int lo = 0, hi = a.c.seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int)((long long)__ldg(a.cu + mid) * G / rows) + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    b = lo;
    s = seq_of(a, b);
    i = slot - ((int)((long long)s.first * G / rows) + b);
    return i >= 0 && (long long)i * rows < (long long)s.T * G;
}

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Fragments of a 16 x 16 piece at (r0, k0) of a row-major bf16 shared tile (ld elements per
// row): A rows r0.., as stored ([m][k]) or from [k][m].
__device__ __forceinline__ void frag_a(uint32_t (&r)[4], const __nv_bfloat16 *t, int ld, int m0, int k0) {
    const int lane = threadIdx.x & 31;
    ldm4(r, smem_u32(t + (m0 + (lane & 15)) * ld + k0 + (lane >> 4) * 8));
}
__device__ __forceinline__ void frag_at(uint32_t (&r)[4], const __nv_bfloat16 *t, int ld, int m0, int k0) {
    const int lane = threadIdx.x & 31, i = lane >> 3;
    ldm4t(r, smem_u32(t + (k0 + (lane & 7) + (i >> 1) * 8) * ld + m0 + (i & 1) * 8));
}
// Two n-tiles (n0, n0 + 8) of B from [n][k] or [k][n]: b0, b1 of the first, then of the second.
__device__ __forceinline__ void frag_bt(uint32_t (&r)[4], const __nv_bfloat16 *t, int ld, int n0, int k0) {
    const int lane = threadIdx.x & 31, i = lane >> 3;
    ldm4(r, smem_u32(t + (n0 + (lane & 7) + (i >> 1) * 8) * ld + k0 + (i & 1) * 8));
}
__device__ __forceinline__ void frag_b(uint32_t (&r)[4], const __nv_bfloat16 *t, int ld, int n0, int k0) {
    const int lane = threadIdx.x & 31, i = lane >> 3;
    ldm4t(r, smem_u32(t + (k0 + (lane & 7) + (i & 1) * 8) * ld + n0 + (i >> 1) * 8));
}

// One warp: acc (16 rows from m0, 8 NT columns from n0) += A B over K, K = 16 ksteps. AT: A is
// stored [k][m]; BN: B is stored [k][n] (else [n][k]). acc[n][0..1]: row lane / 4, columns
// 2 (lane % 4), + 1; acc[n][2..3]: row + 8.
template <int NT, bool AT, bool BN>
__device__ __forceinline__ void warp_mma(float (&acc)[NT][4], const __nv_bfloat16 *A, int lda, int m0,
                                         const __nv_bfloat16 *B, int ldb, int n0, int ksteps,
                                         int k0 = 0) {
#pragma unroll 2
    for (int k = k0; k < ksteps; ++k) {
        uint32_t a[4];
        if (AT) frag_at(a, A, lda, m0, 16 * k);
        else frag_a(a, A, lda, m0, 16 * k);
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            if (BN) frag_b(b, B, ldb, n0 + 8 * n, 16 * k);
            else frag_bt(b, B, ldb, n0 + 8 * n, 16 * k);
            mma_bf16(acc[n], a, b[0], b[1]);
            mma_bf16(acc[n + 1], a, b[2], b[3]);
        }
    }
}

// As warp_mma with split operands, fragments shared between the products: A = Ah + Al with B as
// it is, or with B = Bh + Bl (low x low left out).
template <int NT, bool AT, bool BN>
__device__ __forceinline__ void warp_mma_a2(float (&acc)[NT][4], const __nv_bfloat16 *Ah, const __nv_bfloat16 *Al,
                                            int lda, int m0, const __nv_bfloat16 *B, int ldb, int n0, int ksteps,
                                         int k0 = 0) {
#pragma unroll 2
    for (int k = k0; k < ksteps; ++k) {
        uint32_t a[4], c[4];
        if (AT) {
            frag_at(a, Ah, lda, m0, 16 * k);
            frag_at(c, Al, lda, m0, 16 * k);
        } else {
            frag_a(a, Ah, lda, m0, 16 * k);
            frag_a(c, Al, lda, m0, 16 * k);
        }
#pragma unroll
        for (int n = 0; n < NT; n += 4) {  // products of one accumulator four apart
            uint32_t b[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (BN) frag_b(b[i], B, ldb, n0 + 8 * n + 16 * i, 16 * k);
                else frag_bt(b[i], B, ldb, n0 + 8 * n + 16 * i, 16 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16(acc[n + i], a, b[i >> 1][2 * (i & 1)], b[i >> 1][2 * (i & 1) + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16(acc[n + i], c, b[i >> 1][2 * (i & 1)], b[i >> 1][2 * (i & 1) + 1]);
        }
    }
}
template <int NT, bool BN>
__device__ __forceinline__ void warp_mma_3(float (&acc)[NT][4], const __nv_bfloat16 *Ah, const __nv_bfloat16 *Al,
                                           int lda, int m0, const __nv_bfloat16 *Bh, const __nv_bfloat16 *Bl,
                                           int ldb, int n0, int ksteps,
                                         int k0 = 0) {
#pragma unroll 1
    for (int k = k0; k < ksteps; ++k) {
        uint32_t a[4], c[4];
        frag_a(a, Ah, lda, m0, 16 * k);
        frag_a(c, Al, lda, m0, 16 * k);
#pragma unroll
        for (int n = 0; n < NT; n += 4) {  // products of one accumulator four apart
            uint32_t b[2][4], l[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (BN) {
                    frag_b(b[i], Bh, ldb, n0 + 8 * n + 16 * i, 16 * k);
                    frag_b(l[i], Bl, ldb, n0 + 8 * n + 16 * i, 16 * k);
                } else {
                    frag_bt(b[i], Bh, ldb, n0 + 8 * n + 16 * i, 16 * k);
                    frag_bt(l[i], Bl, ldb, n0 + 8 * n + 16 * i, 16 * k);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16(acc[n + i], a, b[i >> 1][2 * (i & 1)], b[i >> 1][2 * (i & 1) + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16(acc[n + i], c, b[i >> 1][2 * (i & 1)], b[i >> 1][2 * (i & 1) + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16(acc[n + i], a, l[i >> 1][2 * (i & 1)], l[i >> 1][2 * (i & 1) + 1]);
        }
    }
}

template <int NT>
__device__ __forceinline__ void zero_acc(float (&acc)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
}

// x as a high and a low bf16 part: together 16 bits of significand, so a product of split
// operands (three MMAs, low x low left out) is off by 2^-16 of its terms
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(x, y);
    const float2 h = unpack_bf16x2(hi);
    lo = pack_bf16x2(x - h.x, y - h.y);
}

// Lane t of a quad holds v[n] of four things n; afterwards those of thing t by all four lanes.
__device__ __forceinline__ void quad_turn(uint32_t (&v)[4]) {
    const int t = threadIdx.x & 3;
    uint32_t a = __shfl_xor_sync(0xffffffffu, t & 1 ? v[0] : v[1], 1);
    uint32_t b = __shfl_xor_sync(0xffffffffu, t & 1 ? v[2] : v[3], 1);
    if (t & 1) {
        v[0] = a;
        v[2] = b;
    } else {
        v[1] = a;
        v[3] = b;
    }
    a = __shfl_xor_sync(0xffffffffu, t & 2 ? v[0] : v[2], 2);
    b = __shfl_xor_sync(0xffffffffu, t & 2 ? v[1] : v[3], 2);
    if (t & 2) {
        v[0] = a;
        v[1] = b;
    } else {
        v[2] = a;
        v[3] = b;
    }
}

__device__ __forceinline__ void turn_quad_rows(uint4 (&v)[4]) {
    uint32_t a[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[0][i] = v[i].x;
        a[1][i] = v[i].y;
        a[2][i] = v[i].z;
        a[3][i] = v[i].w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) quad_turn(a[e]);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_uint4(a[0][i], a[1][i], a[2][i], a[3][i]);
}

// 64 bytes of each row, a row per lane: a quad's lanes load (store) 16 bytes each of one of its four
// rows after the other, so that a load touches eight lines instead of 32. `at(i)`: where lane i of
// the quad has its bytes, null to leave the row out (zeros). All lanes of the warp take part.
template <typename F>
__device__ __forceinline__ void load_quad_rows(uint4 (&v)[4], F at) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 *p = reinterpret_cast<const uint4 *>(at(i));
        v[i] = p != nullptr ? p[t] : make_uint4(0u, 0u, 0u, 0u);
    }
    turn_quad_rows(v);
}
template <typename F>
__device__ __forceinline__ void store_quad_rows(uint4 (&v)[4], F at) {
    const int t = threadIdx.x & 3;
    turn_quad_rows(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 *p = reinterpret_cast<uint4 *>(at(i));
        if (p != nullptr) p[t] = v[i];
    }
}

// A warp's accumulator tile to global memory, eight consecutive columns a lane (a store of a lane's
// pair of columns instead touches as many lines for a quarter of the bytes, which bounded the
// preparation): value(row, column, x, y) changes a pair in place, put(row, column, high, low) takes
// eight columns as split2 gives them. All lanes of the warp take part.
template <int NT, typename V, typename P>
__device__ __forceinline__ void each_eight(const float (&acc)[NT][4], int m0, int n0, V value, P put) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = m0 + (lane >> 2) + 8 * half;
#pragma unroll
        for (int n = 0; n < NT; n += 4) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = acc[n + i][2 * half], y = acc[n + i][2 * half + 1];
                value(r, n0 + 8 * (n + i) + 2 * t, x, y);
                split2(x, y, h[i], l[i]);
            }
            quad_turn(h);
            quad_turn(l);
            put(r, n0 + 8 * (n + t), make_uint4(h[0], h[1], h[2], h[3]), make_uint4(l[0], l[1], l[2], l[3]));
        }
    }
}

// fn(row, column, value, value of the next column) over a warp's accumulator tile
template <int NT, typename F>
__device__ __forceinline__ void each_pair(float (&acc)[NT][4], int m0, int n0, F fn) {
    const int lane = threadIdx.x & 31, r = m0 + (lane >> 2), c = n0 + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        fn(r, c + 8 * n, acc[n][0], acc[n][1]);
        fn(r + 8, c + 8 * n, acc[n][2], acc[n][3]);
    }
}

// (paged_cached_tc.cuh)
template <Pass M>
using StepOf = std::conditional_t<M == Pass::step, Step, StepMore>;
template <int NT, int D, bool FOX, Pass M>
cudaError_t launch_cached(const StepOf<M> &a, const TcWs &y, uint64_t limit_ns, cudaStream_t stream);

}  // namespace paged
}  // namespace path
