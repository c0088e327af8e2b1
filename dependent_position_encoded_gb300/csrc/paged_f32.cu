// A step of several new tokens per sequence over a paged cache, on the CUDA cores: fp32
// inputs, every product and sum in fp32 (gate sums in fp64).
//
// With u_t = beta_t (w_t - sum_{s<t} (w_s . w_t) u_s) a product of transitions is
// H_1 ... H_i = I - sum_{s<=i} u_s w_s^T (the UT form; technical summary "技術要約: PaTH
// Attention" §3 "UT変換による表現"), per block of 64 tokens with A = (I + D N)^{-1} D,
// N the strictly lower part of W W^T, D = diag(beta) and U = A W:
//   prep       per block: P_b = I - U^T W; queries carried to the block's start,
//              q~ = Q - (Lq A) W with Lq = tril(Q W^T); keys carried to its end,
//              k~ = K - (R A^T) W with R the part t > j of K W^T; the block's own logits
//              Q K^T - (Lq A) R^T and their softmax part; the new values into their pages;
//   scan       chunks of several blocks: a query block visits the earlier blocks of its
//              chunk right to left, logits X k~_b^T, X <- X P_b^T, and so arrives at the
//              chunk's start;
//   cached     the carried queries against the cached keys as they are (a cached key's
//              logit with the chunk's transitions is k_j . (H_1 ... H_i q_i)), in splits;
//   combine    the softmax parts of a row joined;
//   carry      the new keys, k~_b P_{b+1} ... P_last, into their pages, and the whole chunk's
//              product P = P_1 ... P_last;
//   transform  the cached keys in place, K <- K P, after the cached pass has read them.
// For results in full precision, not for speed: at two chunks of up to 130 tokens on 1,000
// cached, 4 heads, D = 64, too few blocks to fill the machine, it is bound by the latency of
// each kernel's chain of products (prep 37 us, scan 32, cached 21, combine 9, carry 14,
// transform 11).
#include "paged_f32.cuh"

namespace path {
namespace paged {

namespace {

// ---------------------------------------------------------------- prep
template <int D>
constexpr size_t prep_smem() { return ((size_t)(4 * (D / 64) + 4) * TILE + 6 * kC) * 4 + 2 * kC * 8; }

template <int D, typename AnyStep>
__global__ void __launch_bounds__(kThr) f32_prep_kernel(const AnyStep a, const Ws y) {
    constexpr int NH = D / 64;
    extern __shared__ float sm[];
    float *W = sm, *K = W + NH * TILE, *U = K + NH * TILE, *Q = U + NH * TILE, *A = Q + NH * TILE,
          *R = A + TILE, *S = R + TILE, *L = S + TILE, *beta = L + TILE, *m = beta + kC, *l = m + kC,
          *alpha = l + kC;
    double *cum = reinterpret_cast<double *>(alpha + 3 * kC);
    const int slot = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int ty = tid >> 4, tx = tid & 15;
    int b, c;
    Seq s;
    grid_begin();  // the first of the call: nothing to wait for
    if (!block_of(a, slot, b, c, s) || !y.takes(s)) return;
    const int i0 = c * kC, rows = min(kC, s.T - i0);
    const long long first = s.first + i0;
    // what this CTA forms: the keys' factors, and its query heads' part; one of them, where the
    // blocks are too few for the machine
    const int parts = gridDim.z - 1, z = blockIdx.z - 1;
    const bool keys = blockIdx.z == 0;
    const int g0 = parts == 0 ? 0 : keys ? 0 : a.c.G * z / parts,
              g1 = parts == 0 ? a.c.G : keys ? 0 : a.c.G * (z + 1) / parts;
    load_tokens<D>(W, a.w, a.sw, first, h, rows);
    load_tokens<D>(K, a.k, a.sk, first, h, rows);
    if (tid < kC) beta[tid] = tid < rows ? a.beta[(first + tid) * a.sb.tok + h * a.sb.head] : 0.f;
    __syncthreads();
    Acc c0;
    zero(c0);
#pragma unroll
    for (int x = 0; x < NH; ++x) mm_nt(W + x * TILE, W + x * TILE, c0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = ty + 16 * i, q = tx + 16 * j;
            A[r * LD + q] = q < r ? beta[r] * c0[i][j] : 0.f;
        }
    zero(c0);
#pragma unroll
    for (int x = 0; x < NH; ++x) mm_nt(K + x * TILE, W + x * TILE, c0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = ty + 16 * i, q = tx + 16 * j;
            R[r * LD + q] = q > r ? c0[i][j] : 0.f;
        }
    __syncthreads();
    // A = (I + E)^{-1} D
    unit_lower_inverse<LD>(A, L, tid, 4);
    for (int e = tid; e < kC * kC; e += kThr) A[(e >> 6) * LD + (e & 63)] *= beta[e & 63];
    __syncthreads();
    const size_t bh = (size_t)slot * a.c.Hkv + h;
    if (keys) {
        // the values go to their pages here: nothing reads the step's own tensors behind the kernel that
        // writes `out`, which may be one of them
        for (int e = tid; e < rows * D / 4; e += kThr) {
            const int r = 4 * e / D, q = 4 * e % D, pos = s.n + i0 + r;
            const int vid = page_of(a, a.c.v_table, b, pos >> a.c.page_shift, a.c.nv);
            if (vid >= 0)
                set4(static_cast<float *>(a.c.v_pages) +
                         ((((size_t)vid * a.c.Hkv + h) << a.c.page_shift) + (pos & (a.c.page - 1))) * D + q,
                     get4(static_cast<const float *>(a.v) + (first + r) * a.sv.tok + h * a.sv.head + q));
        }
#pragma unroll 1
        for (int x2 = 0; x2 < NH; ++x2) {
            zero(c0);
            mm_nn(A, W + x2 * TILE, c0);
            put_nn(U + x2 * TILE, c0);
        }
        zero(c0);
        mm_nt(R, A, c0);
        put_nt(S, c0);
        __syncthreads();
    }
#pragma unroll 1
    for (int x2 = 0; x2 < (keys ? NH : 0); ++x2) {
        zero(c0);
        mm_nn(S, W + x2 * TILE, c0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            const float *kr = K + x2 * TILE + r * LD + 4 * tx;
            *reinterpret_cast<float4 *>(y.kt + (bh * kC + r) * D + 64 * x2 + 4 * tx) =
                make_float4(kr[0] - c0[i][0], kr[1] - c0[i][1], kr[2] - c0[i][2], kr[3] - c0[i][3]);
        }
#pragma unroll 1
        for (int x1 = 0; x1 < NH; ++x1) {
            zero(c0);
            mm_tn(U + x1 * TILE, W + x2 * TILE, c0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 64 * x1 + ty + 16 * i, q = 64 * x2 + 4 * tx;
                *reinterpret_cast<float4 *>(y.pb + (bh * D + r) * D + q) =
                    make_float4((r == q) - c0[i][0], (r == q + 1) - c0[i][1],
                                (r == q + 2) - c0[i][2], (r == q + 3) - c0[i][3]);
            }
        }
    }
    if (g0 == g1) return;
    __syncthreads();
    float *V = U;
    load_tokens<D>(V, a.v, a.sv, first, h, rows);
    for (int g = g0; g < g1; ++g) {
        const int hq = h * a.c.G + g;
        const size_t bq = (size_t)slot * a.c.Hq + hq;
        __syncthreads();
        load_tokens<D>(Q, a.q, a.sq, first, hq, rows);
        if (a.log_f != nullptr && tid < 32) {
            double f[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = 32 * half + tid;
                f[half] = i < rows ? (double)a.log_f[(first + i) * a.sf.tok + hq * a.sf.head] : 0.0;
            }
            const GateSums sums = gate_sums(f[0], f[1], tid);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = 32 * half + tid;
                cum[i] = sums.pair[half];
                y.gq[bq * kC + i] = (float)sums.before[half];
                y.gt[bq * kC + i] = (float)sums.behind[half];
            }
            if (tid == 0) y.gtot[bq] = sums.all;
        }
        if (tid < kC) {
            m[tid] = -INFINITY;
            l[tid] = 0.f;
        }
        __syncthreads();
        zero(c0);
#pragma unroll
        for (int x2 = 0; x2 < NH; ++x2) mm_nt(Q + x2 * TILE, W + x2 * TILE, c0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty + 16 * i, q = tx + 16 * j;
                S[r * LD + q] = q <= r ? c0[i][j] : 0.f;
            }
        __syncthreads();
        zero(c0);
        mm_nn(S, A, c0);
        put_nn(L, c0);
        __syncthreads();
#pragma unroll 1
        for (int x2 = 0; x2 < NH; ++x2) {
            zero(c0);
            mm_nn(L, W + x2 * TILE, c0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ty + 16 * i;
                const float *qr = Q + x2 * TILE + r * LD + 4 * tx;
                *reinterpret_cast<float4 *>(y.qt + (bq * kC + r) * D + 64 * x2 + 4 * tx) =
                    make_float4(qr[0] - c0[i][0], qr[1] - c0[i][1], qr[2] - c0[i][2], qr[3] - c0[i][3]);
            }
        }
        Acc c1;
        zero(c0);
        zero(c1);
#pragma unroll
        for (int x2 = 0; x2 < NH; ++x2) mm_nt(Q + x2 * TILE, K + x2 * TILE, c0);
        mm_nt(L, R, c1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty + 16 * i, q = tx + 16 * j;
                float v = (c0[i][j] - c1[i][j]) * a.scale_log2;
                if (a.log_f != nullptr && q < r) v = fmaf((float)(cum[r] - cum[q]), kLog2e, v);
                S[r * LD + q] = q <= r ? v : -INFINITY;
            }
        __syncthreads();
        softmax_rows(S, m, l, alpha);
        __syncthreads();
        Acc o[NH];
#pragma unroll
        for (int x2 = 0; x2 < NH; ++x2) {
            zero(o[x2]);
            mm_nn(S, V + x2 * TILE, o[x2]);
        }
        store_part<D>(y.part + bq * (1 + y.splits) * kPart<D>, o, m, l);
    }
}

// ---------------------------------------------------------------- scan
template <int D>
constexpr size_t scan_smem() {
    return ((size_t)(3 * (D / 64) + (D / 64) * (D / 64) + 1) * TILE + 5 * kC) * 4;
}

template <int D, typename AnyStep>
__global__ void __launch_bounds__(kThr) f32_scan_kernel(const AnyStep a, const Ws y) {
    constexpr int NH = D / 64;
    extern __shared__ float sm[];
    float *X = sm, *K = X + NH * TILE, *V = K + NH * TILE, *P = V + NH * TILE, *S = P + NH * NH * TILE,
          *m = S + TILE, *l = m + kC, *alpha = l + kC, *gt = alpha + kC;
    const int slot = blockIdx.x, hq = blockIdx.y, h = hq / a.c.G, tid = threadIdx.x;
    const int ty = tid >> 4, tx = tid & 15;
    int b, c;
    Seq s;
    grid_begin();
    const bool mine = block_of(a, slot, b, c, s) && c > 0;
    grid_wait();
    if (!mine) return;
    const size_t bq = (size_t)slot * a.c.Hq + hq;
    float *const part = y.part + bq * (1 + y.splits) * kPart<D>;
    load_rows<D>(X, y.qt + bq * kC * D);
    Acc o[NH];
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 t = *reinterpret_cast<const float4 *>(part + (ty + 16 * i) * D + 64 * x + 4 * tx);
            o[x][i][0] = t.x; o[x][i][1] = t.y; o[x][i][2] = t.z; o[x][i][3] = t.w;
        }
    if (tid < kC) {
        m[tid] = part[kC * D + tid];
        l[tid] = part[kC * D + kC + tid];
    }
    float gq[4];
    double between = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) gq[i] = a.log_f != nullptr ? y.gq[bq * kC + ty + 16 * i] : 0.f;
    for (int kb = c - 1; kb >= 0; --kb) {
        const int ks = slot_of(s, b, kb);
        const size_t kh = (size_t)ks * a.c.Hkv + h;
        __syncthreads();
        load_rows<D>(K, y.kt + kh * kC * D);
        load_tokens<D>(V, a.v, a.sv, (long long)s.first + kb * kC, h, kC);
#pragma unroll
        for (int x = 0; x < NH; ++x) load_rows<D>(P + x * NH * TILE, y.pb + (kh * D + 64 * x) * D);
        if (a.log_f != nullptr && tid < kC) gt[tid] = y.gt[((size_t)ks * a.c.Hq + hq) * kC + tid];
        __syncthreads();
        Acc c0;
        zero(c0);
#pragma unroll
        for (int x = 0; x < NH; ++x) mm_nt(X + x * TILE, K + x * TILE, c0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float bi = (float)((double)gq[i] + between);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v = c0[i][j] * a.scale_log2;
                if (a.log_f != nullptr) v = fmaf(bi + gt[tx + 16 * j], kLog2e, v);
                S[(ty + 16 * i) * LD + tx + 16 * j] = v;
            }
        }
        Acc xn[NH];
#pragma unroll
        for (int x1 = 0; x1 < NH; ++x1) {
            zero(xn[x1]);
#pragma unroll
            for (int x2 = 0; x2 < NH; ++x2) mm_nt(X + x2 * TILE, P + (x1 * NH + x2) * TILE, xn[x1]);
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < NH; ++x) put_nt(X + x * TILE, xn[x]);
        softmax_rows(S, m, l, alpha);
        __syncthreads();
        scale_rows<NH>(o, alpha);
#pragma unroll
        for (int x = 0; x < NH; ++x) mm_nn(S, V + x * TILE, o[x]);
        if (a.log_f != nullptr) between += y.gtot[(size_t)ks * a.c.Hq + hq];
    }
    __syncthreads();
    store_part<D>(part, o, m, l);
    for (int e = tid; e < kC * D / 4; e += kThr) {
        const int r = 4 * e / D, q = 4 * e % D;
        *reinterpret_cast<float4 *>(y.qt + (bq * kC + r) * D + q) =
            *reinterpret_cast<const float4 *>(X + (q >> 6) * TILE + r * LD + (q & 63));
    }
    if (a.log_f != nullptr && tx == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) y.gq[bq * kC + ty + 16 * i] = (float)((double)gq[i] + between);
}

// ---------------------------------------------------------------- combine
// One warp per row, eight parts' rows in flight at a time; grid (slots, Hq, 8).
template <int D, typename AnyStep>
__global__ void __launch_bounds__(kThr) f32_combine_kernel(const AnyStep a, const Ws y) {
    constexpr int E = D / 32;
    const int slot = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x & 31;
    const int r = blockIdx.z * 8 + (threadIdx.x >> 5);
    int b, c;
    Seq s;
    grid_begin();
    const bool mine = block_of(a, slot, b, c, s) && r < s.T - c * kC && y.takes(s);
    grid_wait();
    if (!mine) return;
    const int tiles = sight_of(a, s).tiles(s.n, kC), per = (tiles + y.splits - 1) / y.splits;
    const int used = 1 + (per > 0 ? (tiles + per - 1) / per : 0);
    const float *p0 = y.part + ((size_t)slot * a.c.Hq + hq) * (1 + y.splits) * kPart<D>;
    float M = -INFINITY, L = 0.f, O[E];
#pragma unroll
    for (int e = 0; e < E; ++e) O[e] = 0.f;
    for (int i0 = 0; i0 < used; i0 += 8) {
        float m[8], l[8], v[8][E], top = M;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] = 0.f;
            if (i0 + i < used) {
                const float *p = p0 + (i0 + i) * kPart<D>;
                m[i] = p[kC * D + r];
                l[i] = p[kC * D + kC + r];
#pragma unroll
                for (int e = 0; e < E; ++e) v[i][e] = p[r * D + lane * E + e];
            }
            top = fmaxf(top, m[i]);
        }
        const float f0 = exp2f(M - top);  // 0 at first; part 0 holds the row's own key
        M = top;
        L *= f0;
#pragma unroll
        for (int e = 0; e < E; ++e) O[e] *= f0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = exp2f(m[i] - top);
            L = fmaf(l[i], f, L);
#pragma unroll
            for (int e = 0; e < E; ++e) O[e] = fmaf(v[i][e], f, O[e]);
        }
    }
    if constexpr (std::is_same<AnyStep, StepMore>::value)
        if (a.px != nullptr && __ldg(a.prefix_of + b) >= 0 && a.pstart[b] >= 0) {  // the keys of the sequence's prefix
            const size_t at = ((size_t)(hq / a.c.G) * a.N + s.first + c * kC + r) * a.c.G + hq % a.c.G;
            const float2 ml = a.pxml[at];
            const float top = fmaxf(M, ml.x), f0 = exp2f(M - top), f1 = exp2f(ml.x - top);
            L = fmaf(ml.y, f1, L * f0);
#pragma unroll
            for (int e = 0; e < E; ++e) O[e] = fmaf(a.px[at * D + lane * E + e], f1, O[e] * f0);
        }
    float *dst = static_cast<float *>(a.out) + (long long)(s.first + c * kC + r) * a.so.tok + hq * a.so.head + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = O[e] / L;
}

// ---------------------------------------------------------------- carry
template <int D>
constexpr size_t carry_smem() { return (size_t)(D / 64 + (D / 64) * (D / 64)) * TILE * 4; }

// Items of a key head: the slots, then D / 64 row tiles of the identity per sequence.
template <int D, typename AnyStep>
__global__ void __launch_bounds__(kThr) f32_carry_kernel(const AnyStep a, const Ws y, int nslots) {
    constexpr int NH = D / 64;
    extern __shared__ float sm[];
    float *Y = sm, *P = Y + NH * TILE;
    const int h = blockIdx.y, tid = threadIdx.x;
    const bool ident = (int)blockIdx.x >= nslots;
    int b, c = -1;
    Seq s;
    grid_begin();
    grid_wait();
    int tile = 0;
    if (ident) {
        b = ((int)blockIdx.x - nslots) / NH;
        tile = ((int)blockIdx.x - nslots) % NH;
        s = seq_of(a, b);
        if (s.T == 0 || s.n == 0 || !y.takes(s)) return;
        for (int e = tid; e < kC * D; e += kThr) {
            const int r = e / D, q = e % D;
            Y[(q >> 6) * TILE + r * LD + (q & 63)] = (q == 64 * tile + r) ? 1.f : 0.f;
        }
    } else {
        if (!block_of(a, blockIdx.x, b, c, s) || !y.takes(s)) return;
        load_rows<D>(Y, y.kt + ((size_t)blockIdx.x * a.c.Hkv + h) * kC * D);
    }
    const int nb = (s.T + kC - 1) / kC;
    for (int kb = c + 1; kb < nb; ++kb) {
        const size_t kh = (size_t)slot_of(s, b, kb) * a.c.Hkv + h;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < NH; ++x) load_rows<D>(P + x * NH * TILE, y.pb + (kh * D + 64 * x) * D);
        __syncthreads();
        Acc yn[NH];
#pragma unroll
        for (int x1 = 0; x1 < NH; ++x1) {
            zero(yn[x1]);
#pragma unroll
            for (int x2 = 0; x2 < NH; ++x2) mm_nn(Y + x2 * TILE, P + (x2 * NH + x1) * TILE, yn[x1]);
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < NH; ++x) put_nn(Y + x * TILE, yn[x]);
    }
    __syncthreads();
    if (ident) {
        float *dst = y.ptot + (((size_t)b * a.c.Hkv + h) * D + 64 * tile) * D;
        for (int e = tid; e < kC * D; e += kThr) {
            const int r = e / D, q = e % D;
            dst[(size_t)r * D + q] = Y[(q >> 6) * TILE + r * LD + (q & 63)];
        }
        return;
    }
    // the block's keys into their pages, and the keys' gate sums
    const int rows = min(kC, s.T - c * kC);
    for (int e = tid; e < rows * D / 4; e += kThr) {
        const int r = 4 * e / D, q = 4 * e % D, pos = s.n + c * kC + r;
        const int kid = page_of(a, a.c.k_table, b, pos >> a.c.page_shift, a.c.nk);
        if (kid >= 0)
            set4(static_cast<float *>(a.c.k_pages) +
                     ((((size_t)kid * a.c.Hkv + h) << a.c.page_shift) + (pos & (a.c.page - 1))) * D + q,
                 *reinterpret_cast<const float4 *>(Y + (q >> 6) * TILE + r * LD + (q & 63)));
    }
    if (a.log_f != nullptr)
        for (int e = tid; e < rows * a.c.G; e += kThr) {
            const int r = e % rows, hq = h * a.c.G + e / rows, pos = s.n + c * kC + r;
            double g = y.gt[((size_t)blockIdx.x * a.c.Hq + hq) * kC + r];
            for (int kb = c + 1; kb < nb; ++kb) g += y.gtot[(size_t)slot_of(s, b, kb) * a.c.Hq + hq];
            const int kid = page_of(a, a.c.k_table, b, pos >> a.c.page_shift, a.c.nk);
            if (kid >= 0)
                a.c.g_pages[(((size_t)kid * a.c.Hq + hq) << a.c.page_shift) + (pos & (a.c.page - 1))] = (float)g;
        }
}

// ---------------------------------------------------------------- transform
template <int D>
constexpr size_t transform_smem() { return (size_t)(D / 64 + (D / 64) * (D / 64)) * TILE * 4 + 8 * 4; }

// grid (parts, key heads, sequences): a CTA keeps P in shared memory and takes every parts-th
// tile of 64 cached keys.
template <int D, typename AnyStep>
__global__ void __launch_bounds__(kThr) f32_transform_kernel(const AnyStep a, const Ws y) {
    constexpr int NH = D / 64;
    extern __shared__ float sm[];
    float *K = sm, *P = K + NH * TILE;
    int *kid = reinterpret_cast<int *>(P + NH * NH * TILE);
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    grid_begin();
    const Seq s = seq_of(a, b);
    grid_wait();
    const Sight seen = sight_of(a, s);
    const int tiles = seen.tiles(s.n, kC);
    if (s.T == 0 || (int)blockIdx.x >= tiles || !y.takes(s)) return;
    const int nb = (s.T + kC - 1) / kC;
#pragma unroll
    for (int x = 0; x < NH; ++x)
        load_rows<D>(P + x * NH * TILE, y.ptot + (((size_t)b * a.c.Hkv + h) * D + 64 * x) * D);
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int j = kC * seen.tile(t, s.n, kC), jend = min(j + kC, s.n);
        __syncthreads();
        const int slot0 = find_pages(a, kid, a.c.k_table, a.c.nk, b, j, s.n, seen);
        __syncthreads();
        load_cached<D>(K, a.c.k_pages, a.c, kid, slot0, h, j, s.n, seen);
        __syncthreads();
#pragma unroll
        for (int x1 = 0; x1 < NH; ++x1) {
            Acc c0;
            zero(c0);
#pragma unroll
            for (int x2 = 0; x2 < NH; ++x2) mm_nn(K + x2 * TILE, P + (x2 * NH + x1) * TILE, c0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int jj = j + ty + 16 * i;
                const int id = jj < jend && seen.sees(jj) ? kid[(jj >> a.c.page_shift) - slot0] : -1;
                if (id >= 0)
                    set4(static_cast<float *>(a.c.k_pages) + ((((size_t)id * a.c.Hkv + h) << a.c.page_shift) +
                                                          (jj & (a.c.page - 1))) * D + 64 * x1 + 4 * tx,
                         make_float4(c0[i][0], c0[i][1], c0[i][2], c0[i][3]));
            }
        }
        if (a.log_f != nullptr)
            for (int e = tid; e < kC * a.c.G; e += kThr) {
                const int jj = j + e % kC, hq = h * a.c.G + e / kC;
                const int id = jj < jend && seen.sees(jj) ? kid[(jj >> a.c.page_shift) - slot0] : -1;
                if (id < 0) continue;
                double t = 0.0;
                for (int kb = 0; kb < nb; ++kb) t += y.gtot[(size_t)slot_of(s, b, kb) * a.c.Hq + hq];
                float *g = a.c.g_pages + (((size_t)id * a.c.Hq + hq) << a.c.page_shift) + (jj & (a.c.page - 1));
                *g = (float)((double)*g + t);
            }
    }
}

// What a step's own tokens give: the blocks' factors, and the queries carried to the chunk's start.
template <int D, typename AnyStep>
cudaError_t launch_blocks(const AnyStep &a, const Ws &y, cudaStream_t stream) {
    const int nslots = slots_of(a.N, a.c.seqs), Hq = a.c.Hq, Hkv = a.c.Hkv;
    cudaError_t e;
    if ((e = big_smem(f32_prep_kernel<D, AnyStep>, prep_smem<D>())) != cudaSuccess ||
        (e = big_smem(f32_scan_kernel<D, AnyStep>, scan_smem<D>())) != cudaSuccess)
        return e;
    // while half of the SMs would be idle, a CTA for the keys and others for the query heads
    const int room = 152 / (nslots * Hkv), z = room < 2 ? 1 : 1 + (room - 1 < a.c.G ? room - 1 : a.c.G);
    e = launch(f32_prep_kernel<D, AnyStep>, dim3(nslots, Hkv, z), kThr, prep_smem<D>(), stream, true, a, y);
    if (e == cudaSuccess && a.max_chunk > kC)
        e = launch(f32_scan_kernel<D, AnyStep>, dim3(nslots, Hq), kThr, scan_smem<D>(), stream, false, a, y);
    return e;
}

// The cached keys, the outputs and the cache.
template <int D, typename AnyStep>
cudaError_t launch_cache(const AnyStep &a, const Ws &y, cudaStream_t stream) {
    const int nslots = slots_of(a.N, a.c.seqs), Hq = a.c.Hq, Hkv = a.c.Hkv;
    cudaError_t e;
    if ((e = big_smem(f32_cached_kernel<D, false, AnyStep>, cached_smem<D>())) != cudaSuccess ||
        (e = big_smem(f32_carry_kernel<D, AnyStep>, carry_smem<D>())) != cudaSuccess ||
        (e = big_smem(f32_transform_kernel<D, AnyStep>, transform_smem<D>())) != cudaSuccess)
        return e;
    const long long cap = most_seen(a);
    e = launch(f32_cached_kernel<D, false, AnyStep>, dim3(nslots, Hq, y.splits), kThr, cached_smem<D>(), stream, false, a,
               y);
    if (e == cudaSuccess)
        e = launch(f32_combine_kernel<D, AnyStep>, dim3(nslots, Hq, kC / 8), kThr, 0, stream, false, a, y);
    if (e == cudaSuccess)
        e = launch(f32_carry_kernel<D, AnyStep>, dim3(nslots + a.c.seqs * (D / 64), Hkv), kThr, carry_smem<D>(), stream,
                   false, a, y, nslots);
    // CTAs of 64 cached keys, or of several where that makes more than four to an SM
    long long parts = 4 * 152 / ((long long)Hkv * a.c.seqs) + 1;
    if (parts > (cap + kC - 1) / kC) parts = (cap + kC - 1) / kC;
    if (e == cudaSuccess && parts > 0)
        e = launch(f32_transform_kernel<D, AnyStep>, dim3((unsigned)parts, Hkv, a.c.seqs), kThr, transform_smem<D>(),
                   stream, false, a, y);
    return e;
}

struct F32Layout {
    int splits;
    size_t qt, kt, pb, part, gq, gt, gtot, ptot, total;
};

// Splits of the cached keys: enough CTAs for every SM four times, none below 64 positions.
F32Layout f32_layout(const Cache &c, int N, int d, bool fox) {
    F32Layout y;
    const size_t slots = slots_of(N, c.seqs);
    const long long cap = (long long)c.max_pages << c.page_shift;
    const long long want = 608 / (long long)(slots * c.Hq) + 1, most = (cap + 63) / 64;
    y.splits = (int)(want < most ? want : most);
    if (y.splits < 1) y.splits = 1;
    size_t off = 256;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    y.qt = take(slots * c.Hq * kC * d * 4);
    y.kt = take(slots * c.Hkv * kC * d * 4);
    y.pb = take(slots * c.Hkv * d * d * 4);
    // parts: (1 + splits) per row block, taken as a bound that does not fall as slots rises, so
    // that a workspace for many tokens serves steps of fewer
    const size_t blocks = slots * c.Hq, by_want = 2 * blocks + 608, by_most = blocks * (1 + (size_t)most);
    const size_t parts = most < 1 ? 2 * blocks : (by_want < by_most ? by_want : by_most);
    y.part = take(parts * kC * (d + 2) * 4);
    y.gq = take(fox ? slots * c.Hq * kC * 4 : 0);
    y.gt = take(fox ? slots * c.Hq * kC * 4 : 0);
    y.gtot = take(fox ? slots * c.Hq * 8 : 0);
    y.ptot = take((size_t)c.seqs * c.Hkv * d * d * 4);
    y.total = off;
    return y;
}

}  // namespace

bool decode_takes(int G);
size_t decode_part_bytes(const Cache &c, int d);
struct Behind;
template <typename A>
cudaError_t launch_decode(const A &a, int d, bool bf16, const Behind *behind, float *part, cudaStream_t stream);

cudaError_t launch_prefix_f32(StepMore &a, int d, float *carry, float *gates, float *y_qt, float *y_gq, void *ws,
                              bool first, cudaStream_t stream);

size_t f32_ws_bytes(const Cache &c, int N, int d, bool fox) {
    return f32_layout(c, N, d, fox).total + (decode_takes(c.G) ? align256(decode_part_bytes(c, d)) : 0);
}

// carry: of a step with prefixes (gates, and pws, the workspace's part for them, likewise)
template <typename A>
cudaError_t launch_f32(A a, int d, void *ws, float *carry, float *gates, void *pws, cudaStream_t stream) {
    const F32Layout f = f32_layout(a.c, a.N, d, a.log_f != nullptr);
    char *w = static_cast<char *>(ws);
    auto at = [&](size_t off) { return reinterpret_cast<float *>(w + off); };
    // A sequence of one token takes a whole block of 64 rows here. Where all but the longest chunk bring
    // under four tokens on average, those of one go to the one-pass kernels first, which is two
    // launches more (8 us where there are none): one chunk of 3 tokens among 35 single ones behind
    // 1,050, 32 / 8 heads, D = 128: 2,202 us without, 639 with.
    const bool singles = decode_takes(a.c.G) && a.c.seqs > 1 && a.N - a.max_chunk < 4 * (a.c.seqs - 1);
    const Ws y{at(f.qt), at(f.kt), at(f.pb), at(f.part), at(f.gq), at(f.gt), at(f.ptot),
               reinterpret_cast<double *>(w + f.gtot), f.splits, singles};
    auto blocks = [&]() { return d == 64 ? launch_blocks<64>(a, y, stream) : launch_blocks<128>(a, y, stream); };
    cudaError_t e = cudaSuccess;
    if (carry != nullptr) {  // before any joining
        e = blocks();
        if constexpr (std::is_same<A, StepMore>::value)
            if (e == cudaSuccess) e = launch_prefix_f32(a, d, carry, gates, y.qt, y.gq, pws, false, stream);
    }
    if (e == cudaSuccess && singles) e = launch_decode(a, d, false, nullptr, at(f.total), stream);
    if (e == cudaSuccess && carry == nullptr) e = blocks();
    if (e != cudaSuccess) return e;
    return d == 64 ? launch_cache<64>(a, y, stream) : launch_cache<128>(a, y, stream);
}

template cudaError_t launch_f32(Step, int, void *, float *, float *, void *, cudaStream_t);
template cudaError_t launch_f32(StepMore, int, void *, float *, float *, void *, cudaStream_t);

}  // namespace paged
}  // namespace path
