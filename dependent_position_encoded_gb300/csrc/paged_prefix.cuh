// Steps of sequences that continue a prefix: a row of the cache whose keys stay as they were when
// its last token came, however many sequences continue it.
//
// A sequence's carry C (D x D fp32 per key head) is the product of the transitions of its own cached
// tokens, c (per query head) the sum of their gates. New token i's logit with key j of the prefix is
//     scale k_j . (C H_1 ... H_i q_i)  (+ g_j + c + sum_{s<=i} log f_s),
// so all sequences of a prefix ask the same keys, with queries carried to the prefix's end:
//     plan    counts each prefix's new tokens and gives every sequence its place among them, so that
//             the queries of one prefix stand one behind the other;
//     query   C q~_i (q~_i = H_1 ... H_i q_i, from the step's own kernels; a single token's is formed
//             here, with the carry's update, C - beta (C w) w^T);
//     pass    the attention of a prefix's queries over its keys, as if it were one sequence with that
//             many new tokens (Step::shared), each key read once for all of them; the step's own joining
//             takes up its parts (fp32: joined into one here);
//     carry   C <- C H_1 ... H_T, c <- c + sum log f, of sequences with several tokens.
#pragma once

#include "paged.cuh"

namespace path {
namespace paged {

struct Prefix {
    const int *of;  // (seqs) the row that a sequence continues, below 0: none
    float *carry;   // (seqs, Hkv, D, D)
    float *gates;   // (seqs, Hq), PaTH-FoX
    int *cu;        // (seqs + 1) where each prefix's new tokens begin in their own order
    int *start;     // (seqs) where a sequence's tokens begin in that order, -1: nowhere
    float *px;      // fp32: (Hkv, N G, D) and pairs, the rows' softmax parts in the step's order
    float2 *pxml;
};

constexpr int kPrefixThr = 256;

// Sequences take their places in their order, so that no result depends on timing; those with
// tokens of an earlier one (cu_tokens falls somewhere, which the falling sequence reports) get none,
// so that no more than N tokens are placed. visit(b, p, T): what thread b % kPrefixThr finds of sequence b,
// p < 0 where it has no place; every thread of the CTA calls it in each round.
template <typename V>
__device__ __forceinline__ void each_sequence(const StepMore &a, const int *of, int *sums, V visit) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, S = a.c.seqs;
    int top = 0;
    for (int base = 0; base < S; base += kPrefixThr) {
        const int b = base + tid, begin = b < S ? __ldg(a.cu + b) : 0;
        int m = begin;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o) m = max(m, t);
        }
        __syncthreads();
        if (lane == 31) sums[warp] = m;
        __syncthreads();
        m = max(m, top);
#pragma unroll
        for (int i = 0; i < kPrefixThr / 32; ++i) {
            if (i < warp) m = max(m, sums[i]);
            top = max(top, sums[i]);
        }
        int p = -1, T = 0;
        if (b < S && begin == m) {
            T = seq_of(a, b).T;
            if (T > 0) p = __ldg(of + b);
        }
        visit(b, p, T);
    }
}

// The plan, by one CTA: x.cu and x.start.
__device__ __forceinline__ void place_tokens(const StepMore &a, const Prefix &x) {
    __shared__ int row[kPrefixThr], tokens[kPrefixThr], sums[kPrefixThr / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, S = a.c.seqs;
    for (int p = tid; p <= S; p += kPrefixThr) x.cu[p] = 0;
    each_sequence(a, x.of, sums, [&](int b, int p, int T) {
        row[tid] = p;
        tokens[tid] = T;
        __syncthreads();
        // the tokens of the prefix's earlier sequences: of the rounds before, and of this one
        int before = p >= 0 ? x.cu[p] : 0;
        if (p >= 0)
            for (int i = 0; i < tid; ++i) before += row[i] == p ? tokens[i] : 0;
        __syncthreads();
        if (p >= 0) atomicAdd(x.cu + p, T);
        if (b < S) x.start[b] = p >= 0 ? before : -1;
        __syncthreads();
    });
    // counts to where they begin
    int run = 0;
    for (int base = 0; base <= S; base += kPrefixThr) {
        const int p = base + tid, v = p <= S ? x.cu[p] : 0;
        int t = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += u;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = t;
        __syncthreads();
        int before = run;
#pragma unroll
        for (int i = 0; i < kPrefixThr / 32; ++i) {
            if (i < warp) before += sums[i];
            run += sums[i];
        }
        if (p <= S) x.cu[p] = before + t - v;
    }
    __syncthreads();
    for (int b = tid; b < S; b += kPrefixThr)
        if (x.start[b] >= 0) x.start[b] += x.cu[__ldg(x.of + b)];
    __syncthreads();
}

// What the plan gives sequence b, by a CTA of its own: the tokens of the prefixes before its own, and of the
// sequences before it. -1: it has no place.
__device__ __forceinline__ int place_one(const StepMore &a, const Prefix &x, int mine) {
    __shared__ int sums[kPrefixThr / 32], total, found;
    const int tid = threadIdx.x, of = __ldg(x.of + mine);
    int before = 0;
    if (tid == 0) total = 0, found = -1;
    each_sequence(a, x.of, sums, [&](int b, int p, int T) {
        if (p >= 0 && (p < of || (p == of && b < mine))) before += T;
        if (b == mine) found = p;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    __syncthreads();
    if ((tid & 31) == 0 && before > 0) atomicAdd(&total, before);
    __syncthreads();
    return found >= 0 ? total : -1;
}

// The step whose sequences are the prefixes.
inline StepMore shared_step(const StepMore &a, const Prefix &x) {
    StepMore v = a;
    v.cu = x.cu;
    v.max_chunk = a.N;
    v.window = v.sinks = 0;
    v.prefix_of = nullptr;
    v.pstart = nullptr;
    v.px = nullptr;
    v.pxml = nullptr;
    v.shared = true;
    return v;
}

// A sequence's only token and a key head: its queries carried to the prefix's end and the carry's
// update from one read of the carry, all in fp32, by a CTA for `R` rows of C from `row0` on (they do not
// meet; that of row 0 sees to the gates). Eight lanes share a row, 16 bytes each at a time; bound by the
// carry's bytes, there and back (22.5 us for 64 tokens of 8 key heads at D = 128, 67 MB: 3.0 TB/s, beside
// the look for a place). put(g, i, x):
// entry i of query head g's carried query; gate(g, x): its gates.
template <typename T, int D, int R, typename P, typename F>
__device__ __forceinline__ void prefix_single(const StepMore &a, const Prefix &x, const Seq &s, int b, int h, int row0,
                                              P put, F gate) {
    constexpr int NC = D / 32, NR = R / 32, kHeads = 16;  // columns / 32 of a row, rows / 32
    __shared__ __align__(16) float ws[D], qs[kHeads][D], os[kHeads][R];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = a.c.G;
    const int sub = lane & 7, r0 = tid >> 3;
    float4 *const C = reinterpret_cast<float4 *>(x.carry + (((size_t)b * a.c.Hkv + h) * D + row0) * D);
    float4 c[NR][NC];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int k = 0; k < NC; ++k) c[i][k] = C[(r0 + 32 * i) * (D / 4) + 8 * k + sub];
    const float beta = a.beta[(long long)s.first * a.sb.tok + h * a.sb.head];
    const T *const wp = static_cast<const T *>(a.w) + (long long)s.first * a.sw.tok + h * a.sw.head;
    if (tid < D) ws[tid] = Elt<T>::to_f(wp[tid]);
    __syncthreads();
    auto dot = [&](const float4 (&u)[NC], const float *v) {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const float4 f = *reinterpret_cast<const float4 *>(v + 32 * k + 4 * sub);
            t[0] = fmaf(u[k].x, f.x, t[0]);
            t[1] = fmaf(u[k].y, f.y, t[1]);
            t[2] = fmaf(u[k].z, f.z, t[2]);
            t[3] = fmaf(u[k].w, f.w, t[3]);
        }
        float z = (t[0] + t[1]) + (t[2] + t[3]);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        return z;
    };
    for (int g0 = 0; g0 < G; g0 += kHeads) {
        const int some = min(kHeads, G - g0);
        // q~ = q - beta (w . q) w, a warp per head
        for (int g = warp; g < some; g += kPrefixThr / 32) {
            const T *const qp = static_cast<const T *>(a.q) + (long long)s.first * a.sq.tok +
                                (long long)(h * G + g0 + g) * a.sq.head;
            float q[D / 32], wq = 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                q[e] = Elt<T>::to_f(qp[lane + 32 * e]);
                wq = fmaf(ws[lane + 32 * e], q[e], wq);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) wq += __shfl_xor_sync(0xffffffffu, wq, o);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) qs[g][lane + 32 * e] = fmaf(-beta * wq, ws[lane + 32 * e], q[e]);
        }
        __syncthreads();
        for (int g = 0; g < some; ++g)
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const float z = dot(c[i], qs[g]);
                if (sub == 0) os[g][r0 + 32 * i] = z;
            }
        __syncthreads();
        for (int e = tid; e < some * R; e += kPrefixThr) put(g0 + e / R, row0 + e % R, os[e / R][e % R]);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const float z = beta * dot(c[i], ws);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const float4 f = *reinterpret_cast<const float4 *>(ws + 32 * k + 4 * sub);
            C[(r0 + 32 * i) * (D / 4) + 8 * k + sub] =
                make_float4(fmaf(-z, f.x, c[i][k].x), fmaf(-z, f.y, c[i][k].y), fmaf(-z, f.z, c[i][k].z),
                            fmaf(-z, f.w, c[i][k].w));
        }
    }
    if (a.log_f != nullptr && row0 == 0)
        for (int g = tid; g < G; g += kPrefixThr) {
            float *const p = x.gates + (size_t)b * a.c.Hq + h * G + g;
            const float t = *p + a.log_f[(long long)s.first * a.sf.tok + (long long)(h * G + g) * a.sf.head];
            *p = t;
            gate(g, t);
        }
}

// The carries of sequences with several tokens, in fp32, eight tokens at a time: with y_t = C w_t and the
// 8 x 8 factor A = (I + D N)^{-1} D of the tokens (the UT form, as for a block of 64: N the strictly lower
// part of W W^T, D = diag(beta)), C <- C - sum_t (A y)_t w_t^T. The rows of C do not meet: a CTA takes 64
// of them, eight lanes to four rows (the tokens' w come from shared memory, whose reads bound the kernel
// with fewer), and forms the factors of 32 tokens by itself. In fp32 because a carry outlives its step:
// bf16 parts would leave 2^-17 of it with every chunk. Bound by that chain, whose CTAs are few: 100 us for 8
// sequences of up to 512 tokens and 8 heads at D = 128, 128 CTAs, each at a third of its SM's fp32 rate
// (token by token 198, with one row of C to eight lanes 136).
constexpr int kCarryThr = 128, kCarryPer = 4, kCarryRows = kCarryThr / 8 * kCarryPer;
constexpr int kCarryTokens = 32, kCarryBlock = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kCarryThr) prefix_carry_kernel(const StepMore a, const Prefix x) {
    constexpr int NC = D / 32, B = kCarryBlock, NB = kCarryTokens / B;
    constexpr int E = 16 / sizeof(T), PER = D / E, IT = kCarryTokens * PER / kCarryThr, LD = D + 4;
    __shared__ __align__(16) float ws[kCarryTokens][LD];  // (rows begin in different banks)
    __shared__ __align__(16) float As[NB][B][B], Gs[NB][B][B];  // A, by rows; W W^T
    __shared__ float bs[kCarryTokens];
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, sub = tid & 7;
    const int r = blockIdx.x * kCarryRows + (tid >> 3) * kCarryPer;
    grid_begin();
    const Seq s = seq_of(a, b);
    const bool mine = s.T > 1 && __ldg(x.of + b) >= 0;
    grid_wait();
    if (!mine || x.start[b] < 0) return;  // (no place among the prefix's tokens: left as it was)
    float4 *const C = reinterpret_cast<float4 *>(x.carry + (((size_t)b * a.c.Hkv + h) * D + r) * D);
    float4 c[kCarryPer][NC];
#pragma unroll
    for (int i = 0; i < kCarryPer; ++i)
#pragma unroll
        for (int k = 0; k < NC; ++k) c[i][k] = C[i * (D / 4) + 8 * k + sub];
    // the next tokens' w and beta are on their way while those before are used
    uint4 next[IT];
    float beta = 0.f;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int e = tid + i * kCarryThr, t = t0 + e / PER;
            next[i] = t < s.T ? *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.w) + h * a.sw.head +
                                                                 (long long)(s.first + t) * a.sw.tok + e % PER * E)
                              : make_uint4(0u, 0u, 0u, 0u);
        }
        if (tid < kCarryTokens)
            beta = t0 + tid < s.T ? a.beta[(long long)(s.first + t0 + tid) * a.sb.tok + h * a.sb.head] : 0.f;
    };
    fetch(0);
    for (int t0 = 0; t0 < s.T; t0 += kCarryTokens) {
        const int blocks = (min(kCarryTokens, s.T - t0) + B - 1) / B;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int e = tid + i * kCarryThr;
            const T *const v = reinterpret_cast<const T *>(&next[i]);
#pragma unroll
            for (int q = 0; q < E; q += 4)
                *reinterpret_cast<float4 *>(&ws[e / PER][e % PER * E + q]) =
                    make_float4(Elt<T>::to_f(v[q]), Elt<T>::to_f(v[q + 1]), Elt<T>::to_f(v[q + 2]),
                                Elt<T>::to_f(v[q + 3]));
        }
        if (tid < kCarryTokens) bs[tid] = beta;
        __syncthreads();
        if (t0 + kCarryTokens < s.T) fetch(t0 + kCarryTokens);
        // w_i . w_j, j < i: four lanes to each
        for (int e = tid >> 2; e < blocks * 28; e += kCarryThr / 4) {
            const int n = e / 28;
            int i = 1, j = e % 28;
            while (j >= i) j -= i++;
            float z = 0.f;
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
                const float4 u = *reinterpret_cast<const float4 *>(&ws[n * B + i][16 * q + 4 * (tid & 3)]);
                const float4 v = *reinterpret_cast<const float4 *>(&ws[n * B + j][16 * q + 4 * (tid & 3)]);
                z = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, z))));
            }
            const unsigned quad = 0xfu << (tid & 28);
            z += __shfl_xor_sync(quad, z, 1);
            z += __shfl_xor_sync(quad, z, 2);
            if ((tid & 3) == 0) Gs[n][i][j] = z;
        }
        __syncthreads();
        // column j of A by forward substitution: a_ij = beta_i ([i = j] - sum_{l<i} g_il a_lj)
        if (tid < blocks * B) {
            const int n = tid / B, j = tid % B;
            float col[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                float z = i == j ? 1.f : 0.f;
#pragma unroll
                for (int l = 0; l < i; ++l) z = fmaf(-Gs[n][i][l], col[l], z);
                col[i] = i < j ? 0.f : bs[n * B + i] * z;
                As[n][i][j] = col[i];
            }
        }
        __syncthreads();
        for (int n = 0; n < blocks; ++n) {
            float y[kCarryPer][B];
#pragma unroll
            for (int t = 0; t < B; ++t) {
                float2 z[kCarryPer];
#pragma unroll
                for (int i = 0; i < kCarryPer; ++i) z[i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const float4 w = *reinterpret_cast<const float4 *>(&ws[n * B + t][32 * k + 4 * sub]);
#pragma unroll
                    for (int i = 0; i < kCarryPer; ++i) {
                        z[i] = ffma2(make_float2(c[i][k].x, c[i][k].y), make_float2(w.x, w.y), z[i]);
                        z[i] = ffma2(make_float2(c[i][k].z, c[i][k].w), make_float2(w.z, w.w), z[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < kCarryPer; ++i) y[i][t] = z[i].x + z[i].y;
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
#pragma unroll
                for (int i = 0; i < kCarryPer; ++i)
#pragma unroll
                    for (int t = 0; t < B; ++t) y[i][t] += __shfl_xor_sync(0xffffffffu, y[i][t], o);
#pragma unroll
            for (int t = 0; t < B; ++t) {
                float u[B], z[kCarryPer];
                *reinterpret_cast<float4 *>(u) = *reinterpret_cast<const float4 *>(&As[n][t][0]);
                if (t >= 4) *reinterpret_cast<float4 *>(u + 4) = *reinterpret_cast<const float4 *>(&As[n][t][4]);
#pragma unroll
                for (int i = 0; i < kCarryPer; ++i) {
                    z[i] = 0.f;
#pragma unroll
                    for (int l = 0; l <= t; ++l) z[i] = fmaf(-u[l], y[i][l], z[i]);
                }
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const float4 w = *reinterpret_cast<const float4 *>(&ws[n * B + t][32 * k + 4 * sub]);
#pragma unroll
                    for (int i = 0; i < kCarryPer; ++i) {
                        const float2 zz = make_float2(z[i], z[i]);
                        const float2 lo = ffma2(zz, make_float2(w.x, w.y), make_float2(c[i][k].x, c[i][k].y));
                        const float2 hi = ffma2(zz, make_float2(w.z, w.w), make_float2(c[i][k].z, c[i][k].w));
                        c[i][k] = make_float4(lo.x, lo.y, hi.x, hi.y);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kCarryPer; ++i)
#pragma unroll
        for (int k = 0; k < NC; ++k) C[i * (D / 4) + 8 * k + sub] = c[i][k];
    if (a.log_f != nullptr && blockIdx.x == 0)
        for (int g = tid >> 5; g < a.c.G; g += kCarryThr / 32) {
            float *const p = x.gates + (size_t)b * a.c.Hq + h * a.c.G + g;
            double sum = 0.0;
            for (int t = tid & 31; t < s.T; t += 32)
                sum += a.log_f[(long long)(s.first + t) * a.sf.tok + (long long)(h * a.c.G + g) * a.sf.head];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if ((tid & 31) == 0) *p = (float)(*p + sum);
        }
}

template <typename T, int D>
cudaError_t launch_prefix_carry(const StepMore &a, const Prefix &x, cudaStream_t stream) {
    if (a.max_chunk <= 1) return cudaSuccess;
    return launch(prefix_carry_kernel<T, D>, dim3(D / kCarryRows, a.c.Hkv, a.c.seqs), kCarryThr, 0, stream, false, a,
                  x);
}

}  // namespace paged
}  // namespace path
