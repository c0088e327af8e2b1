// The bf16 block path of a step over a paged cache: workspace and warp-level product helpers.
//
// Rows. The Hq / Hkv = G query heads of a key head are taken together: row t G + g of a
// sequence is query head g of its new token t, so that 128 consecutive rows (one tensor-core
// tile) hold as many tokens as share the cached keys. All sequences' rows of a key head stand
// one behind the other, R = N G of them.
#pragma once

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
// and, where it may have several groups of blocks (paged_prep_tc.cu):
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

// Row tiles and key tiles of a sequence in the plan of NT (0 where it goes with the other).
__device__ __forceinline__ void plan_of(const Step &a, const Seq &s, int D, int NT, int &tiles, int &ktiles) {
    const int G = a.c.G, rows = s.T * G;  // T G <= N G, which the host keeps within an int
    ktiles = (s.n + 127) / 128;
    tiles = one_tile(s.T, G, D, a.log_f != nullptr) == (NT == 1) ? (rows + 128 * NT - 1) / (128 * NT) : 0;
}

// Units per CTA: at least two, so that a part is worth its join.
__device__ __forceinline__ long long plan_per(const Plan &p, int seqs) {
    const long long all = p.units[seqs], per = (all + p.ctas - 1) / p.ctas;
    return per < 2 ? 2 : per;
}

// The stretch of units from u on that lies in one item and below `end`.
struct Stretch {
    Seq s;
    int b, h, tile, k0, steps;
    long long item;  // over all sequences
};
__device__ __forceinline__ Stretch stretch_at(const Step &a, const Plan &p, int D, int NT, long long u,
                                              long long end) {
    int lo = 0, hi = a.c.seqs - 1;  // the last sequence with units[b] <= u: it has units
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.units[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    Stretch t;
    t.b = lo;
    t.s = seq_of(a, lo);
    int tiles, kt;
    plan_of(a, t.s, D, NT, tiles, kt);
    const long long rem = u - p.units[lo];
    const int it = (int)(rem / kt);
    t.k0 = (int)(rem - (long long)it * kt);
    t.h = it / tiles;
    t.tile = it - t.h * tiles;
    t.item = p.items[lo] + it;
    const long long left = end - u;
    t.steps = kt - t.k0 < left ? kt - t.k0 : (int)left;
    return t;
}

// Rows of `rows` per tile over all sequences: tile i of sequence b is slot
// cu[b] G / rows + b + i (as slots_of).
__host__ __device__ __forceinline__ int tile_slots(int N, int G, int seqs, int rows) {
    return (int)((long long)N * G / rows) + seqs;
}
__device__ __forceinline__ bool tile_of(const Step &a, int slot, int rows, int &b, int &i, Seq &s) {
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

}  // namespace paged
}  // namespace path
