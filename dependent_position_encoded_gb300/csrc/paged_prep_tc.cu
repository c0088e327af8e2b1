// The bf16 block path of a step over a paged cache, except its attention: per-block factors,
// the new keys' way into the cache, the cached keys' update and the joining of the softmax
// parts. Warp-level MMAs (mma.sync, bf16 operands, fp32 accumulators): every product here is
// 64 x 64 x d or the pass is bound by memory, and none of them is worth a tensor-memory
// pipeline; the attention itself is in paged_attn_tc.cu.
//
// Precision. The inputs are bf16; what is computed from them (A, U, Lq, R A^T, P_b) enters
// further products as a high and a low bf16 part (16 bits of significand, see split2), so
// carried keys and transitions are exact to 2^-16 before the cache rounds the keys to bf16.
// The 16 x 16 diagonal blocks of A = (I + D N)^{-1} D are solved in fp32. Rounded to bf16 are the
// softmax weights, in the scan over a chunk's blocks keys, state and transitions, and the carried
// queries (low_weights, scan_low and keeps_low say where these have a second part).
#include "paged_tc.cuh"

namespace path {
namespace paged {

namespace {

constexpr int kThr = 256;
using bf = __nv_bfloat16;

// ---------------------------------------------------------------- prep
// One CTA per 64-token block and key head. With the block's tokens in `nt` tiles of 16 rows,
// every product is cut to those (a step of a few tokens costs a few tiles), and triangular
// factors to their tiles.
//   A = (I + D N)^{-1} D, U = A W, S = R A^T with R the part t > j of K W^T;
//   P_b - I = -U^T W, k~ = K - S W; per query head, with Lq = tril(Q W^T):
//   q~ = Q - Lq U and the block's own logits Q K^T - Lq S^T.
// Bound by the latency of that chain of small products between barriers, each of them run for the
// first time by most CTAs (the warp-level tensor path is busy an eighth to a quarter of the time):
// 69 us for four first chunks of up to 1,500 tokens, 8 key heads of two query heads, D = 64 (two
// CTAs per SM, 1.7 waves; 88 with the products (Lq A) W and (Lq A) R^T in place of those with U and
// S, the gates in line, the inverse on the CUDA cores and stores of a lane's pairs), 76 us for
// 2,048 tokens of 8 key heads of four, D = 128 (84), 9 us for 32 single tokens of 16 heads, D = 64.
template <int D>
struct PrepSmem {
    static constexpr int LDD = D + 8, LDS = 72, LDF = 72;  // row strides: 16-byte phases differ
    static constexpr size_t big = (size_t)kC * LDD * 2, sml = (size_t)kC * LDS * 2;
    // pairs (hi, lo): U; S = R A^T; A, in its place Lq and then P; R in the places of Q and V
    static constexpr size_t W = 0, K = big, Q = 2 * big, V = 3 * big, Uh = 4 * big, Ul = 5 * big, Ah = 6 * big,
                            Al = Ah + sml, Sh = Al + sml, Sl = Sh + sml, Rh = Q, Rl = V;
    static constexpr size_t F = Sl + sml;  // fp32 64 x 72: E and its inverse, then the logits
    // beta, row maxima and sums: 64 floats each; 16 pages; the gates' prefix sums of kHeads query
    // heads as float pairs
    static constexpr int kHeads = 8;
    static constexpr size_t vec = F + kC * LDF * 4, cum = vec + 3 * kC * 4 + 16 * 4, bytes = cum + kHeads * kC * 8;
};
static_assert(PrepSmem<64>::kHeads == kThr / 32, "a warp per head");
static_assert(2 * (PrepSmem<64>::bytes + 1024) <= 228 * 1024 && PrepSmem<128>::bytes <= 227 * 1024, "shared memory");

// 64 tokens (rows past `rows` zero) of one head into registers, and from there into a shared
// tile: the loads of several tiles are in flight together
template <int D>
struct Block {
    static constexpr int LDD = D + 8, PER = D / 8, IT = kC * PER / kThr;
    uint4 x[IT];
    __device__ __forceinline__ void load(const void *src, Stride st, long long first, int head, int rows) {
        const bf *p = static_cast<const bf *>(src) + head * st.head;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int e = threadIdx.x + i * kThr, r = e / PER, c = e % PER * 8;
            x[i] = r < rows ? *reinterpret_cast<const uint4 *>(p + (first + r) * st.tok + c)
                            : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __device__ __forceinline__ void put(bf *dst) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int e = threadIdx.x + i * kThr, r = e / PER, c = e % PER * 8;
            *reinterpret_cast<uint4 *>(dst + r * LDD + c) = x[i];
        }
    }
};

__device__ __forceinline__ void put2(bf *t, int ld, int r, int c, uint32_t v) {
    *reinterpret_cast<uint32_t *>(t + r * ld + c) = v;
}

// Units and items of cached-key work before each sequence (one CTA, both plans). The parts'
// buffers hold what sequences without common tokens can need, so one that begins before an
// earlier one's begin or end (cu_tokens falls somewhere, which the falling sequence reports) gets
// no work: with m the largest cu_tokens so far, a sequence counts where cu_tokens = m.
template <int D>
__device__ __forceinline__ void make_plans(const Step &a, const TcWs &y, long long *sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *const tops = reinterpret_cast<int *>(sums + kThr / 32);
    long long run[4] = {0, 0, 0, 0};
    int top = 0;
    for (int base = 0; base <= a.c.seqs; base += kThr) {
        const int b = base + tid;
        const int begin = b < a.c.seqs ? __ldg(a.cu + b) : 0;
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
// and value enter the cache as they are. A warp per query head in turns; all threads form the
// product less I, -beta w w^T.
template <int D>
__device__ __forceinline__ void prep_single(const Step &a, const TcWs &y, const Seq &s, int b, int slot, int h,
                                            float *buf) {
    constexpr int E = D / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = a.c.G, kw = kThr / 32;
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
    if (warp == 0)
#pragma unroll
        for (int e = 0; e < E; ++e) buf[lane * E + e] = w[e];
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
            if (keeps_low(one_tile(1, G, D, a.log_f != nullptr) ? 1 : 2, D))
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
    if (s.n == 0) return;  // no cached key takes the product
    __syncthreads();
    bf *const mh = y.mt + (mt_row(a, s, b) * a.c.Hkv + h) * 2 * D * D, *const ml = mh + (size_t)D * D;
    for (int e = tid; e < D * D / 8; e += kThr) {
        const int i = e / (D / 8), j = e % (D / 8) * 8;
        const float f = -beta * buf[i];
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) split2(f * buf[j + 2 * q], f * buf[j + 2 * q + 1], hi[q], lo[q]);
        *reinterpret_cast<uint4 *>(mh + (size_t)i * D + j) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(ml + (size_t)i * D + j) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// (I + E)^{-1} as unit_lower_inverse forms it, but with the products behind the diagonal blocks on
// the warp-level tensor path, their factors as two bf16 parts (what A enters further products
// with has no more): a factor of the shared fp32 matrix is split as it is loaded, and the first
// product's sums are the second one's A operand as they lie in registers.
template <int LD>
__device__ __forceinline__ void unit_lower_inverse_mma(float *E, int tid, int nt) {
    diagonal_inverses<LD>(E, tid);
    if (nt <= 1) return;
    const int warp = tid >> 5, g = (tid & 31) >> 2, t2 = 2 * (tid & 3);
    struct A {
        uint32_t h[4], l[4];
    };
    auto a_of = [&](int r0, int k0) {  // 16 x 16 from (r0, k0)
        A f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v =
                *reinterpret_cast<const float2 *>(E + (r0 + g + 8 * (i & 1)) * LD + k0 + t2 + 8 * (i >> 1));
            split2(v.x, v.y, f.h[i], f.l[i]);
        }
        return f;
    };
    // acc (16 x 8) += a E[k0 .. k0 + 15][n0 .. n0 + 7]
    auto product = [&](float (&acc)[4], const A &a, int k0, int n0) {
        uint32_t h[2], l[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float *const p = E + (k0 + t2 + 8 * i) * LD + n0 + g;
            split2(p[0], p[LD], h[i], l[i]);
        }
        mma_bf16(acc, a.h, h[0], h[1]);
        mma_bf16(acc, a.l, h[0], h[1]);
        mma_bf16(acc, a.h, l[0], l[1]);
    };
    auto a_from = [&](const float (&x)[4], const float (&y)[4]) {  // two 16 x 8 sums side by side
        A f;
        split2(x[0], x[1], f.h[0], f.l[0]);
        split2(x[2], x[3], f.h[1], f.l[1]);
        split2(y[0], y[1], f.h[2], f.l[2]);
        split2(y[2], y[3], f.h[3], f.l[3]);
        return f;
    };
    auto put_minus = [&](const float (&x)[4], int r0, int n0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2 *>(E + (r0 + g + 8 * i) * LD + n0 + t2) = make_float2(-x[2 * i], -x[2 * i + 1]);
    };
    if (warp < 2) {  // a warp for the 16-blocks of each 32-block, at o
        const int o = 32 * warp;
        const A x22 = a_of(o + 16, o + 16);
        float t[2][4], x[2][4];
        zero_acc(t);
        zero_acc(x);
#pragma unroll
        for (int n = 0; n < 2; ++n) product(t[n], x22, o + 16, o + 8 * n);
        const A ta = a_from(t[0], t[1]);
#pragma unroll
        for (int n = 0; n < 2; ++n) product(x[n], ta, o, o + 8 * n);
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 2; ++n) put_minus(x[n], o + 16, o + 8 * n);
    }
    __syncthreads();
    if (nt <= 2) return;
    // the 32-blocks: a warp for 16 rows and 16 columns
    const int i0 = 16 * (warp & 1), j0 = 16 * (warp >> 1);
    float x[2][4];
    zero_acc(x);
    if (warp < 4) {
        float t[4][4];
        zero_acc(t);
#pragma unroll 1
        for (int k = 0; k <= i0; k += 16) {  // X22 is lower triangular
            const A x22 = a_of(32 + i0, 32 + k);
#pragma unroll
            for (int n = 0; n < 4; ++n) product(t[n], x22, 32 + k, 8 * n);
        }
        for (int k = j0; k < 32; k += 16) {  // and so is X11
            const A ta = k == 0 ? a_from(t[0], t[1]) : a_from(t[2], t[3]);
#pragma unroll
            for (int n = 0; n < 2; ++n) product(x[n], ta, k, j0 + 8 * n);
        }
    }
    __syncthreads();
    if (warp < 4)
#pragma unroll
        for (int n = 0; n < 2; ++n) put_minus(x[n], 32 + i0, j0 + 8 * n);
    __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kThr, D == 64 ? 2 : 1) tc_prep_kernel(const Step a, const TcWs y) {
    using S = PrepSmem<D>;
    constexpr int LDD = S::LDD, LDS = S::LDS, LDF = S::LDF, NH = D / 64;
    extern __shared__ __align__(16) uint8_t smem[];
    auto tile = [&](size_t at) { return reinterpret_cast<bf *>(smem + at); };
    bf *const W = tile(S::W), *const K = tile(S::K), *const Q = tile(S::Q), *const V = tile(S::V),
       *const Uh = tile(S::Uh), *const Ul = tile(S::Ul), *const Ah = tile(S::Ah), *const Al = tile(S::Al),
       *const Sh = tile(S::Sh), *const Sl = tile(S::Sl), *const Rh = tile(S::Rh), *const Rl = tile(S::Rl),
       *const Lh = Ah, *const Ll = Al, *const P = Ah;
    float *const F = reinterpret_cast<float *>(smem + S::F);
    float *const beta = reinterpret_cast<float *>(smem + S::vec), *const rm = beta + kC, *const rl = rm + kC;
    int *const kpage = reinterpret_cast<int *>(rl + kC), *const vpage = kpage + 8;
    float2 *const cums = reinterpret_cast<float2 *>(smem + S::cum);
    const int slot = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.c.G;
    int b, c;
    Seq s;
    grid_begin();  // the first of the call: nothing to wait for
    if ((int)blockIdx.x == gridDim.x - 1) {  // the CTA behind the slots
        if (h == 0 && blockIdx.z == 0) make_plans<D>(a, y, reinterpret_cast<long long *>(smem));
        return;
    }
    if (!block_of(a, slot, b, c, s)) return;
    if (s.T == 1) {
        if (blockIdx.z == 0) prep_single<D>(a, y, s, b, slot, h, reinterpret_cast<float *>(smem));
        return;
    }
    const int rows = min(kC, s.T - c * kC), nt = (rows + 15) >> 4;
    const bool single = s.T <= kC;
    const long long first = s.first + c * kC;
    const size_t bh = (size_t)slot * a.c.Hkv + h;
    // this CTA's query heads of the key head; the first CTA writes what they share
    const int g0 = G * (int)blockIdx.z / (int)gridDim.z, g1 = G * ((int)blockIdx.z + 1) / (int)gridDim.z;
    const bool lead = blockIdx.z == 0;
    const int pos0 = s.n + c * kC, slot0 = pos0 >> a.c.page_shift;  // where the block goes in the cache
    Block<D> vb, qb;
    {
        Block<D> wb, kb;
        wb.load(a.w, a.sw, first, h, rows);
        kb.load(a.k, a.sk, first, h, rows);
        qb.load(a.q, a.sq, first, h * G + g0, rows);
        vb.load(a.v, a.sv, first, h, rows);
        wb.put(W);
        kb.put(K);
    }
    if (tid < 8 && tid <= ((pos0 + rows - 1) >> a.c.page_shift) - slot0) {
        kpage[tid] = page_of(a, a.c.k_table, b, slot0 + tid, a.c.nk);
        vpage[tid] = page_of(a, a.c.v_table, b, slot0 + tid, a.c.nv);
    }
    // the place of the block's row i on its page (-1: the page is bad)
    auto place = [&](const int *pages, int i, int heads, int head) -> long long {
        const int pos = pos0 + i, id = pages[(pos >> a.c.page_shift) - slot0];
        return id < 0 ? -1 : (((long long)id * heads + head) << a.c.page_shift) + (pos & (a.c.page - 1));
    };
    if (tid < kC) beta[tid] = tid < rows ? a.beta[(first + tid) * a.sb.tok + h * a.sb.head] : 0.f;
    __syncthreads();
    // a warp's 16 x 32 piece of a 64 x 64 product
    const int m0 = 16 * (warp & 3), n0 = 32 * (warp >> 2);
    const bool live = (warp & 3) < nt && n0 < 16 * nt;  // the piece has rows and columns
    // and entries at or below the diagonal, or above it. A lower triangle's rows m0 .. m0 + 15 end in
    // column tile m_end - 1, an upper one's begin in column tile m0 / 16
    const bool lower = live && n0 <= m0, upper = live && m0 < n0 + 32;
    const int m_end = min(nt, (warp & 3) + 1);
    {
        float e[4][4], r[4][4];
        zero_acc(e);
        zero_acc(r);
        if (lower) warp_mma<4, false, false>(e, W, LDD, m0, W, LDD, n0, D / 16);
        if (upper) warp_mma<4, false, false>(r, K, LDD, m0, W, LDD, n0, D / 16);
        each_pair(e, m0, n0, [&](int i, int j, float x, float z) {
            *reinterpret_cast<float2 *>(F + i * LDF + j) =
                make_float2(j < i ? beta[i] * x : 0.f, j + 1 < i ? beta[i] * z : 0.f);
        });
        each_pair(r, m0, n0, [&](int i, int j, float x, float z) {
            uint32_t hi, lo;
            split2(j > i ? x : 0.f, j + 1 > i ? z : 0.f, hi, lo);
            put2(Rh, LDS, i, j, hi);
            put2(Rl, LDS, i, j, lo);
        });
    }
    __syncthreads();
    // PaTH-FoX, a warp per query head: sums of the block's 64 gates (gate_sums), lane t those of tokens
    // t and t + 32. Those for differences are shared as two floats each: a difference of two is
    // right to 2^-47 of the sums
    auto gates = [&](int g, float2 *cum) {
        const int hq = h * G + g;
        const size_t bq = (size_t)slot * a.c.Hq + hq;
        double f[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 32 * half + lane;
            f[half] = t < rows ? (double)a.log_f[(first + t) * a.sf.tok + hq * a.sf.head] : 0.0;
        }
        const GateSums sums = gate_sums(f[0], f[1], lane);
        float most = -INFINITY;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 32 * half + lane;
            const float hi = (float)sums.pair[half], behind = (float)sums.behind[half];
            cum[t] = make_float2(hi, (float)(sums.pair[half] - (double)hi));
            y.gt[bq * kC + t] = behind;
            most = fmaxf(most, behind);
            if (t < rows) {
                y.gq[(size_t)h * y.R + (first + t) * G + g] = (float)sums.before[half];
                const long long at = single ? place(kpage, t, a.c.Hq, hq) : -1;
                if (at >= 0) a.c.g_pages[at] = behind;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (lane == 0) {
            y.gtot[bq] = sums.all;
            y.gblk[bq] = make_float2((float)sums.all, most);
        }
    };
    // those of the first heads, by the warps that the inverse's first part leaves idle
    if (a.log_f != nullptr && warp >= 2)
        for (int g = g0 + warp - 2; g < min(g1, g0 + S::kHeads); g += kThr / 32 - 2) gates(g, cums + (g - g0) * kC);
    unit_lower_inverse_mma<LDF>(F, tid, nt);
    for (int e = tid; e < kC * kC / 2; e += kThr) {
        const int i = e / 32, j = 2 * (e % 32);
        uint32_t hi, lo;
        split2(j <= i ? F[i * LDF + j] * beta[j] : 0.f, j + 1 <= i ? F[i * LDF + j + 1] * beta[j + 1] : 0.f,
               hi, lo);
        put2(Ah, LDS, i, j, hi);
        put2(Al, LDS, i, j, lo);
    }
    __syncthreads();
    // U = A W (64 x D) and S = R A^T (64 x 64, strictly upper)
#pragma unroll
    for (int x = 0; x < NH; ++x) {
        float u[4][4];
        zero_acc(u);
        if ((warp & 3) < nt) warp_mma_a2<4, false, true>(u, Ah, Al, LDS, m0, W, LDD, 64 * x + n0, m_end);
        each_pair(u, m0, 64 * x + n0, [&](int i, int j, float p, float q) {
            uint32_t hi, lo;
            split2(p, q, hi, lo);
            put2(Uh, LDD, i, j, hi);
            put2(Ul, LDD, i, j, lo);
        });
    }
    {
        float r[4][4];
        zero_acc(r);
        if (upper) warp_mma_3<4, false>(r, Rh, Rl, LDS, m0, Ah, Al, LDS, n0, min(nt, n0 / 16 + 2), m0 / 16);
        each_pair(r, m0, n0, [&](int i, int j, float p, float q) {
            uint32_t hi, lo;
            split2(p, q, hi, lo);
            put2(Sh, LDS, i, j, hi);
            put2(Sl, LDS, i, j, lo);
        });
    }
    __syncthreads();
    // P_b - I = -U^T W (D x D): to the chunk's product or the block's factors
    if (lead) {
        bf *const mh = single ? y.mt + (mt_row(a, s, b) * a.c.Hkv + h) * 2 * D * D : y.kh + (bh * (kC + D) + kC) * D;
        bf *const ml = single ? mh + (size_t)D * D : y.kl + (bh * (kC + D) + kC) * D;
#pragma unroll 1
        for (int t = warp; t < D / 16 * (D / 32); t += kThr / 32) {
            const int r0 = 16 * (t % (D / 16)), c0 = 32 * (t / (D / 16));
            float u[4][4];
            zero_acc(u);
            warp_mma_a2<4, true, true>(u, Uh, Ul, LDD, r0, W, LDD, c0, nt);
            each_eight(
                u, r0, c0,
                [](int, int, float &p, float &q) {
                    p = -p;
                    q = -q;
                },
                [&](int i, int j, uint4 hi, uint4 lo) {
                    *reinterpret_cast<uint4 *>(mh + (size_t)i * D + j) = hi;
                    *reinterpret_cast<uint4 *>(ml + (size_t)i * D + j) = lo;
                });
        }
    }
    // k~ = K - S W: into the pages (the chunk's only block) or the block's factors
#pragma unroll
    for (int x = 0; x < NH; ++x) {
        if (!lead || (single && (warp & 3) >= nt)) break;
        float u[4][4];
        zero_acc(u);
        warp_mma_a2<4, false, true>(u, Sh, Sl, LDS, m0, W, LDD, 64 * x + n0, nt, m0 / 16);
        each_eight(
            u, m0, 64 * x + n0,
            [&](int i, int j, float &p, float &q) {
                const float2 k2 = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(K + i * LDD + j));
                p = k2.x - p;
                q = k2.y - q;
            },
            [&](int i, int j, uint4 hi, uint4 lo) {
                if (single) {
                    const long long at = i < rows ? place(kpage, i, a.c.Hkv, h) : -1;
                    if (at >= 0) *reinterpret_cast<uint4 *>(static_cast<bf *>(a.c.k_pages) + at * D + j) = hi;
                } else {
                    *reinterpret_cast<uint4 *>(y.kh + (bh * (kC + D) + i) * D + j) = hi;
                    *reinterpret_cast<uint4 *>(y.kl + (bh * (kC + D) + i) * D + j) = lo;
                }
            });
    }
    // the block's values: into the pages, and beside the factors for the scan
    if (lead)
#pragma unroll
        for (int i = 0; i < Block<D>::IT; ++i) {
            const int e = tid + i * kThr, r = e / Block<D>::PER, q = e % Block<D>::PER * 8;
            if (!single) *reinterpret_cast<uint4 *>(y.vb + (bh * kC + r) * D + q) = vb.x[i];
            const long long at = r < rows ? place(vpage, r, a.c.Hkv, h) : -1;
            if (at >= 0) *reinterpret_cast<uint4 *>(static_cast<bf *>(a.c.v_pages) + at * D + q) = vb.x[i];
        }
    vb.put(V);  // R has been read
    for (int g = g0; g < g1; ++g) {
        const int hq = h * G + g;
        // the row of token t: its place in the step's packed rows
        auto row_of = [&](int t) { return (size_t)h * y.R + (first + t) * G + g; };
        const float2 *const cum = cums + (g - g0) % S::kHeads * kC;
        qb.put(Q);
        if (g + 1 < g1) qb.load(a.q, a.sq, first, hq + 1, rows);
        if (a.log_f != nullptr && g > g0 && (g - g0) % S::kHeads == 0 && g + warp < g1)
            gates(g + warp, cums + warp * kC);  // the next heads'
        __syncthreads();
        float u[4][4];
        zero_acc(u);
        {  // Lq = tril(Q W^T), and Q K^T
            float z[4][4];
            zero_acc(z);
            if (lower) {
                warp_mma<4, false, false>(z, Q, LDD, m0, W, LDD, n0, D / 16);
                warp_mma<4, false, false>(u, Q, LDD, m0, K, LDD, n0, D / 16);
            }
            each_pair(z, m0, n0, [&](int i, int j, float p, float q) {
                uint32_t hi, lo;
                split2(j <= i ? p : 0.f, j + 1 <= i ? q : 0.f, hi, lo);
                put2(Lh, LDS, i, j, hi);
                put2(Ll, LDS, i, j, lo);
            });
        }
        __syncthreads();
        {  // the block's logits Q K^T - Lq S^T
            float z[4][4];
            zero_acc(z);
            if (lower) warp_mma_3<4, false>(z, Lh, Ll, LDS, m0, Sh, Sl, LDS, n0, m_end, n0 / 16);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) u[n][i] = (u[n][i] - z[n][i]) * a.scale_log2;
            each_pair(u, m0, n0, [&](int i, int j, float p, float q) {
                if (a.log_f != nullptr) {
                    const float2 ci = cum[i];
                    const float4 cj = *reinterpret_cast<const float4 *>(cum + j);
                    if (j < i) p = fmaf((ci.x - cj.x) + (ci.y - cj.y), kLog2e, p);
                    if (j + 1 < i) q = fmaf((ci.x - cj.z) + (ci.y - cj.w), kLog2e, q);
                }
                *reinterpret_cast<float2 *>(F + i * LDF + j) =
                    make_float2(j <= i ? p : -INFINITY, j + 1 <= i ? q : -INFINITY);
            });
        }
        // q~ = Q - Lq U
#pragma unroll
        for (int x = 0; x < NH; ++x) {
            if ((warp & 3) >= nt) break;
            float v[4][4];
            zero_acc(v);
            warp_mma_3<4, true>(v, Lh, Ll, LDS, m0, Uh, Ul, LDD, 64 * x + n0, m_end);
            // the scan starts from both parts
            const bool low = !single || keeps_low(one_tile(s.T, G, D, a.log_f != nullptr) ? 1 : 2, D);
            each_eight(
                v, m0, 64 * x + n0,
                [&](int i, int j, float &p, float &q) {  // scaled here once: the attention's logits need no factor
                    const float2 q2 = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(Q + i * LDD + j));
                    p = (q2.x - p) * a.scale_log2;
                    q = (q2.y - q) * a.scale_log2;
                },
                [&](int i, int j, uint4 hi, uint4 lo) {
                    if (i >= rows) return;
                    *reinterpret_cast<uint4 *>(y.qt + row_of(i) * D + j) = hi;
                    if (low) *reinterpret_cast<uint4 *>(y.ql + row_of(i) * D + j) = lo;
                });
        }
        __syncthreads();
        // row maxima and sums; the weights, rounded to bf16, for the product with the values: eight
        // lanes per row, eight columns each. (One part: 64 keys of a row at most, and with nothing else
        // the output's error is 2.05e-3 of its norm, its own rounding alone 1.65e-3.)
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            const int i = 8 * warp + 4 * pass + (lane >> 3), j = 8 * (lane & 7);
            const float4 u = *reinterpret_cast<const float4 *>(F + i * LDF + j);
            const float4 v = *reinterpret_cast<const float4 *>(F + i * LDF + j + 4);
            float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
            float m = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) m = fmaxf(m, x[e]);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            float l = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = exp2f(x[e] - m);  // the row's own key is never masked
                l += x[e];
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            *reinterpret_cast<uint4 *>(P + i * LDS + j) =
                make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                           pack_bf16x2(x[6], x[7]));
            if ((lane & 7) == 0) {
                rm[i] = m;
                rl[i] = l;
            }
        }
        __syncthreads();
        if (tid < rows) y.pml[row_of(tid)] = make_float2(rm[tid], rl[tid]);
#pragma unroll
        for (int x = 0; x < NH; ++x) {
            if ((warp & 3) >= nt) break;
            float v[4][4];
            zero_acc(v);
            warp_mma<4, false, true>(v, P, LDS, m0, V, LDD, 64 * x + n0, m_end);
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // eight consecutive columns a lane, as each_eight
                uint32_t p[4], q[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    p[n] = __float_as_uint(v[n][2 * half]);
                    q[n] = __float_as_uint(v[n][2 * half + 1]);
                }
                quad_turn(p);
                quad_turn(q);
                const int i = m0 + (lane >> 2) + 8 * half;
                if (i >= rows) continue;
                uint4 *const dst = reinterpret_cast<uint4 *>(y.po + row_of(i) * D + 64 * x + n0 + 8 * (lane & 3));
                dst[0] = make_uint4(p[0], q[0], p[1], q[1]);
                dst[1] = make_uint4(p[2], q[2], p[3], q[3]);
            }
        }
    }
}

// ---------------------------------------------------------------- carry
// Chunks of several blocks: the new keys of a block through the later ones, Y <- Y P_b for
// b = c + 1 .. last, into their pages; and the identity through all blocks, which gives the
// chunk's own product. Y is split into 16-bit pairs at every step, its sum stays in fp32
// registers (Y + Y (P_b - I)), eight warps of 16 rows and half of the columns each. A chain of all blocks would be as
// long as the chunk, so it goes in two passes over groups of kGroup blocks: to the group's
// end (and the group's product), then over the later groups' products. Each step waits for
// 2 D^2 bf16 from L2 and for its MMAs, two CTAs to an SM: 44 + 19 us for 2,048 tokens of 8 key
// heads at D = 128, 23 + 14 us for four chunks of up to 1,500 at D = 64.
constexpr int kGroup = 8;

template <int D>
struct CarrySmem {
    static constexpr int LDD = D + 8;
    static constexpr size_t Mh = 0, Ml = (size_t)D * LDD * 2, Yh = 2 * Ml, Yl = Yh + (size_t)kC * LDD * 2,
                            bytes = Yl + (size_t)kC * LDD * 2;
};

// Groups of all sequences share one numbering: group i of a sequence whose first block is slot
// f is number f / kGroup + b + i.
__device__ __forceinline__ int group_of(const Seq &s, int b, int i) { return slot_of(s, b, 0) / kGroup + b + i; }
// The (sequence, group) of a number, as block_of.
__device__ __forceinline__ bool group_at(const Step &a, int number, int &b, int &i, Seq &s) {
    int lo = 0, hi = a.c.seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((__ldg(a.cu + mid) / kC + mid) / kGroup + mid <= number) lo = mid;
        else hi = mid - 1;
    }
    b = lo;
    s = seq_of(a, b);
    i = number - group_of(s, b, 0);
    return i >= 0 && i * kGroup * kC < s.T;
}

__device__ __forceinline__ void cp16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// PASS 1: within the group; PASS 2: over the groups behind. The grid, key heads within: D / 64 row
// tiles of the identity for each of `idents` groups (pass 2: sequences), the longest chains, then
// the slots. A chunk of one group is done after pass 1.
template <int D, int PASS>
__global__ void __launch_bounds__(kThr) tc_carry_kernel(const Step a, const TcWs y, int idents) {
    using S = CarrySmem<D>;
    constexpr int LDD = S::LDD, NT = D / 16, PER = D / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    bf *const Mh = reinterpret_cast<bf *>(smem + S::Mh), *const Ml = reinterpret_cast<bf *>(smem + S::Ml),
       *const Yh = reinterpret_cast<bf *>(smem + S::Yh), *const Yl = reinterpret_cast<bf *>(smem + S::Yl);
    const int h = blockIdx.x % a.c.Hkv, at = blockIdx.x / a.c.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int m0 = 16 * (warp & 3), n0 = D / 2 * (warp >> 2);  // the warp's 16 rows and half of the columns
    const bool ident = at < idents * (D / 64);
    int b, c = 0, tile = 0, grp = 0, slot = 0;
    Seq s;
    bool mine = true;
    grid_begin();
    float acc[NT][4];
    zero_acc(acc);
    if (ident) {
        tile = at % (D / 64);
        if (PASS == 1) {
            mine = group_at(a, at / (D / 64), b, grp, s);
        } else {
            b = at / (D / 64);
            s = seq_of(a, b);
        }
    } else {
        slot = at - idents * (D / 64);
        mine = block_of(a, slot, b, c, s);
        grp = c / kGroup;
    }
    grid_wait();
    if (!mine) return;
    const int nb = (s.T + kC - 1) / kC, ng = (nb + kGroup - 1) / kGroup;
    if (s.T <= kC || grp >= ng || (PASS == 2 && ng == 1)) return;
    if (ident) {
        // the chunk's product is for the cached keys, a group's for the groups before it too
        if (s.n == 0 && (ng == 1 || PASS == 2 || grp == 0)) return;
        const int r = 64 * tile + m0 + (lane >> 2), q = 2 * (lane & 3);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = (n0 + 8 * n + q + (i & 1) == r + 8 * (i >> 1)) ? 1.f : 0.f;
    } else {
        const size_t bh = (size_t)slot * a.c.Hkv + h, base = PASS == 1 ? bh * (kC + D) : bh * kC;
        const bf *const ph = PASS == 1 ? y.kh : y.ch, *const pl = PASS == 1 ? y.kl : y.cl;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const size_t at = (base + m0 + (lane >> 2) + 8 * i) * D + n0 + 8 * n + 2 * (lane & 3);
                const float2 p = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(ph + at));
                const float2 q = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(pl + at));
                acc[n][2 * i] = p.x + q.x;
                acc[n][2 * i + 1] = p.y + q.y;
            }
    }
    // the factors: blocks of the group, or groups
    const int from = PASS == 1 ? (ident ? grp * kGroup : c + 1) : (ident ? 0 : grp + 1);
    const int to = PASS == 1 ? min(nb, (grp + 1) * kGroup) : ng;
    for (int k = from; k < to; ++k) {
        const size_t at = PASS == 1 ? (((size_t)slot_of(s, b, k) * a.c.Hkv + h) * (kC + D) + kC) * D
                                    : ((size_t)group_of(s, b, k) * a.c.Hkv + h) * 2 * D * D;
        const bf *const ph = PASS == 1 ? y.kh + at : y.gp + at, *const pl = PASS == 1 ? y.kl + at : ph + D * D;
        __syncthreads();
#pragma unroll 4
        for (int e = tid; e < D * PER; e += kThr) {
            const int r = e / PER, q = e % PER * 8;
            cp16(Mh + r * LDD + q, ph + (size_t)r * D + q);
            cp16(Ml + r * LDD + q, pl + (size_t)r * D + q);
        }
        each_pair(acc, m0, n0, [&](int i, int j, float p, float q) {
            uint32_t hi, lo;
            split2(p, q, hi, lo);
            put2(Yh, LDD, i, j, hi);
            put2(Yl, LDD, i, j, lo);
        });
        cp_wait_all();
        __syncthreads();
        warp_mma_3<NT, true>(acc, Yh, Yl, LDD, m0, Mh, Ml, LDD, n0, D / 16);
    }
    const bool done = PASS == 2 || ng == 1;
    if (ident) {
        bf *const mh = done ? y.mt + (mt_row(a, s, b) * a.c.Hkv + h) * 2 * D * D
                            : y.gp + ((size_t)group_of(s, b, grp) * a.c.Hkv + h) * 2 * D * D;
        bf *const ml = mh + (size_t)D * D;
        each_eight(
            acc, 64 * tile + m0, n0,
            [](int i, int j, float &p, float &q) {
                p -= i == j;
                q -= i == j + 1;
            },
            [&](int i, int j, uint4 hi, uint4 lo) {
                *reinterpret_cast<uint4 *>(mh + (size_t)i * D + j) = hi;
                *reinterpret_cast<uint4 *>(ml + (size_t)i * D + j) = lo;
            });
        return;
    }
    if (!done && grp + 1 < ng) {
        const size_t base = ((size_t)slot * a.c.Hkv + h) * kC;
        each_eight(
            acc, m0, n0, [](int, int, float &, float &) {},
            [&](int i, int j, uint4 hi, uint4 lo) {
                *reinterpret_cast<uint4 *>(y.ch + (base + i) * D + j) = hi;
                *reinterpret_cast<uint4 *>(y.cl + (base + i) * D + j) = lo;
            });
        return;
    }
    if (PASS == 2 && grp + 1 == ng) return;  // the last group's keys went to the pages in pass 1
    const int rows = min(kC, s.T - c * kC);
    each_eight(
        acc, m0, n0, [](int, int, float &, float &) {},
        [&](int i, int j, uint4 hi, uint4) {
            if (i >= rows) return;
            const int pos = s.n + c * kC + i, id = page_of(a, a.c.k_table, b, pos >> a.c.page_shift, a.c.nk);
            if (id >= 0)
                *reinterpret_cast<uint4 *>(static_cast<bf *>(a.c.k_pages) +
                                           ((((size_t)id * a.c.Hkv + h) << a.c.page_shift) + (pos & (a.c.page - 1))) *
                                               D +
                                           j) = hi;
        });
    if (a.log_f != nullptr)
        for (int e = tid; e < rows * a.c.G; e += kThr) {
            const int r = e % rows, hq = h * a.c.G + e / rows, pos = s.n + c * kC + r;
            double g = y.gt[((size_t)slot * a.c.Hq + hq) * kC + r];
            for (int kb = c + 1; kb < nb; ++kb) g += y.gtot[(size_t)slot_of(s, b, kb) * a.c.Hq + hq];
            const int id = page_of(a, a.c.k_table, b, pos >> a.c.page_shift, a.c.nk);
            if (id >= 0)
                a.c.g_pages[(((size_t)id * a.c.Hq + hq) << a.c.page_shift) + (pos & (a.c.page - 1))] = (float)g;
        }
}

// ---------------------------------------------------------------- transform
// K <- K + K (P - I) in place for sequences whose rows fill several tiles (with one tile the
// attention pass does it on the keys that it has loaded). A key is read and written once; the
// two products of P - I's parts keep the warp-level tensor path busy for longer than HBM at
// D = 128. A warp takes 32 positions at a time, so that a fragment of P - I serves two row
// tiles, and loads the next 32 meanwhile. grid (parts, key heads, sequences), a CTA keeps
// P - I in shared memory. 51 us for 32,768 positions of 8 heads at D = 128: 2.6 TB/s of keys,
// 0.33 PFLOP/s.
template <int D>
struct TransformSmem {
    static constexpr int LDD = D + 8;
    static constexpr size_t Mh = 0, Ml = (size_t)D * LDD * 2, K = 2 * Ml, strip = (size_t)32 * LDD * 2,
                            bytes = K + 8 * 2 * strip;
};

template <int D>
__global__ void __launch_bounds__(kThr, 1) tc_transform_kernel(const Step a, const TcWs y) {
    using S = TransformSmem<D>;
    constexpr int LDD = S::LDD, NT = D / 8, PER = D / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    bf *const Mh = reinterpret_cast<bf *>(smem + S::Mh), *const Ml = reinterpret_cast<bf *>(smem + S::Ml);
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_begin();
    const Seq s = seq_of(a, b);
    grid_wait();
    const int strips = (s.n + 31) / 32, per = (strips + (int)gridDim.x - 1) / (int)gridDim.x;
    const int first = (int)blockIdx.x * per, last = min(strips, first + per);
    if (one_tile(s.T, a.c.G, D, a.log_f != nullptr) || first >= last) return;
    const bf *const m = y.mt + (mt_row(a, s, b) * a.c.Hkv + h) * 2 * D * D;
#pragma unroll 4
    for (int e = tid; e < D * PER; e += kThr) {
        const int r = e / PER, q = e % PER * 8;
        cp16(Mh + r * LDD + q, m + (size_t)r * D + q);
        cp16(Ml + r * LDD + q, m + (size_t)(D + r) * D + q);
    }
    bf *const pool = static_cast<bf *>(a.c.k_pages);
    bf *const mine = reinterpret_cast<bf *>(smem + S::K + warp * 2 * S::strip);
    // where 16 positions from j lie (pages are multiples of 16); null past the end or on a bad page
    auto rows_at = [&](int j) -> bf * {
        if (j >= s.n) return nullptr;
        const int id = page_of(a, a.c.k_table, b, j >> a.c.page_shift, a.c.nk);
        return id < 0 ? nullptr
                      : pool + ((((size_t)id * a.c.Hkv + h) << a.c.page_shift) + (j & (a.c.page - 1))) * D;
    };
    auto fetch = [&](int strip, int buf) {
        bf *const dst = mine + buf * 32 * LDD;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const bf *src = rows_at(32 * strip + 16 * half);
#pragma unroll
            for (int e = lane; e < 16 * PER; e += 32) {
                const int r = e / PER, q = e % PER * 8;
                if (src != nullptr) cp16(dst + (16 * half + r) * LDD + q, src + (size_t)r * D + q);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int buf = 0;
    if (first + warp < last) fetch(first + warp, 0);
    cp_wait_all();
    __syncthreads();
    for (int strip = first + warp; strip < last; strip += 8, buf ^= 1) {
        if (strip + 8 < last) {
            fetch(strip + 8, buf ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            cp_wait_all();
        }
        __syncwarp();
        bf *const k = mine + buf * 32 * LDD;
        float acc[2][NT][4];
        zero_acc(acc[0]);
        zero_acc(acc[1]);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            const bf *const M = part == 0 ? Mh : Ml;
#pragma unroll 2
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t a0[4], a1[4];
                frag_a(a0, k, LDD, 0, 16 * kk);
                frag_a(a1, k, LDD, 16, 16 * kk);
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t f[4];
                    frag_b(f, M, LDD, 8 * n, 16 * kk);
                    mma_bf16(acc[0][n], a0, f[0], f[1]);
                    mma_bf16(acc[0][n + 1], a0, f[2], f[3]);
                    mma_bf16(acc[1][n], a1, f[0], f[1]);
                    mma_bf16(acc[1][n + 1], a1, f[2], f[3]);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int half = 0; half < 2; ++half)
            each_pair(acc[half], 16 * half, 0, [&](int i, int j, float p, float q) {
                uint32_t *at = reinterpret_cast<uint32_t *>(k + i * LDD + j);
                const float2 k2 = unpack_bf16x2(*at);
                *at = pack_bf16x2(k2.x + p, k2.y + q);
            });
        __syncwarp();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int j = 32 * strip + 16 * half, left = min(16, s.n - j);
            bf *const dst = rows_at(j);
#pragma unroll
            for (int e = lane; e < 16 * PER; e += 32) {
                const int r = e / PER, q = e % PER * 8;
                if (dst != nullptr && r < left)
                    *reinterpret_cast<uint4 *>(dst + (size_t)r * D + q) =
                        *reinterpret_cast<const uint4 *>(k + (16 * half + r) * LDD + q);
            }
        }
        __syncwarp();
    }
}

// PaTH-FoX: every cached key's gate sums advance by the chunk's, four positions a thread (the
// pool's rows of 16 or more positions are 16-byte aligned). grid (parts, Hq, seqs). 15 us for 16
// sequences of 16,384 positions and 32 heads (67 MB: 4.4 TB/s).
__global__ void __launch_bounds__(kThr) tc_gates_kernel(const Step a, const TcWs y) {
    const int hq = blockIdx.y, b = blockIdx.z;
    grid_begin();
    const Seq s = seq_of(a, b);
    grid_wait();
    if (s.T == 0 || (int)blockIdx.x * kThr * 4 >= s.n) return;
    const int nb = (s.T + kC - 1) / kC;
    double sum = 0.0;
    for (int kb = 0; kb < nb; ++kb) sum += y.gtot[(size_t)slot_of(s, b, kb) * a.c.Hq + hq];
    const float t = (float)sum;
    for (int j = (blockIdx.x * kThr + threadIdx.x) * 4; j < s.n; j += gridDim.x * kThr * 4) {
        const int id = page_of(a, a.c.k_table, b, j >> a.c.page_shift, a.c.nk);
        if (id < 0) continue;
        float *g = a.c.g_pages + (((size_t)id * a.c.Hq + hq) << a.c.page_shift) + (j & (a.c.page - 1));
        if (j + 4 <= s.n) {
            float4 v = *reinterpret_cast<const float4 *>(g);
            v.x += t;
            v.y += t;
            v.z += t;
            v.w += t;
            *reinterpret_cast<float4 *>(g) = v;
        } else {
            for (int i = 0; j + i < s.n; ++i) g[i] += t;
        }
    }
}

// ---------------------------------------------------------------- combine
// A warp joins `rows` consecutive rows of a key head, each the part of the step's own tokens and
// those of the cached keys, P of them at a time. What the rows of a tile share (their sequence
// and the numbers of their parts) is looked up once. Bound by the latency of the look-up and of
// the parts' rows: two or four rows joined together, sixteen a warp, or own parts loaded before
// the look-up took longer. 19 us for 79,000 rows without parts at D = 64 (1.6 TB/s, most of it
// from L2), 7 us for 512 rows of ten parts or so.
template <int D, int P>
__global__ void __launch_bounds__(kThr) tc_combine_kernel(const Step a, const TcWs y, int rows) {
    constexpr int E = D / 32;
    const int G = a.c.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
    const int r0 = (blockIdx.x * (kThr / 32) + warp) * rows, r1 = min(r0 + rows, (int)y.R);  // R <= INT_MAX / 2
    grid_begin();
    // the last sequence that begins at or before a token
    int lo = 0;
    auto find = [&](int tok) {
        lo = 0;
        for (int hi = a.c.seqs - 1; lo < hi;) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(a.cu + mid) <= tok) lo = mid;
            else hi = mid - 1;
        }
        return seq_of(a, lo);
    };
    Seq s = find(r0 / G);
    grid_wait();
    auto load = [&](const float *p, float (&v)[E]) {
        if (E == 2) {
            const float2 t = *reinterpret_cast<const float2 *>(p + lane * E);
            v[0] = t.x;
            v[1] = t.y;
        } else {
            const float4 t = *reinterpret_cast<const float4 *>(p + lane * E);
            v[0] = t.x;
            v[1] = t.y;
            v[E - 2] = t.z;
            v[E - 1] = t.w;
        }
    };
    // of the row looked up last: rows below `known` are of the same tile
    long long first = 0;
    int known = -1, start = 0, number = 0, cp = 0, tile = 128;
    for (int r = r0; r < r1; ++r) {
        const int tok = r / G, hq = h * G + (r - tok * G);
        if (r >= known) {
            if (r > r0) s = find(tok);
            if (tok < s.first || tok >= s.first + s.T) continue;
            const int rows_all = s.T * G;
            start = s.first * G;
            int NT = 1, tiles, kt;
            plan_of(a, s, D, 1, tiles, kt);
            if (tiles == 0) {
                NT = 2;
                plan_of(a, s, D, 2, tiles, kt);
            }
            tile = 128 * NT;
            const Plan &p = NT == 1 ? y.plan[0] : y.plan[1];
            const int ti = (r - start) / tile, it = h * tiles + ti;
            // the first part's number and how many there are (none where the sequence has no work)
            first = number = 0;
            if (kt > 0 && p.items[lo + 1] > p.items[lo]) {
                const long long per = plan_per(p, a.c.seqs), u = p.units[lo] + (long long)it * kt, c0 = u / per;
                first = c0 + p.items[lo] + it;
                number = (int)((u + kt - 1) / per - c0) + 1;
            }
            // short sequences' tiles hold copies of their rows, each a part of its own
            cp = NT == 2 ? 0 : rows_all <= 32 ? 2 : rows_all <= 64 ? 1 : 0;
            number <<= cp;
            known = start + min(rows_all, (ti + 1) * tile);
        }
        const size_t row = (size_t)h * y.R + r;
        const long long at0 = first * tile + (r - start) % tile;
        const float *const so = tile == 128 ? y.so[0] : y.so[1];
        const float2 *const sml = tile == 128 ? y.sml[0] : y.sml[1];
        const float2 z = y.pml[row];
        float M = z.x, L = z.y, O[E];  // M is never -inf: a row has its own key
        load(y.po + row * D, O);
        for (int p0 = 0; p0 < number; p0 += P) {
            float2 ml[P];
            float v[P][E];
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int q = p0 + j;
                ml[j] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int e = 0; e < E; ++e) v[j][e] = 0.f;
                if (q < number) {
                    const size_t at = at0 + (size_t)(q >> cp) * tile + (q & ((1 << cp) - 1)) * (128 >> cp);
                    ml[j] = sml[at];
                    load(so + at * D, v[j]);
                }
            }
            float m = M;
#pragma unroll
            for (int j = 0; j < P; ++j) m = fmaxf(m, ml[j].x);
            const float f0 = exp2f(M - m);
            M = m;
            L *= f0;
#pragma unroll
            for (int e = 0; e < E; ++e) O[e] *= f0;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float f = exp2f(ml[j].x - m);  // absent keys alone: 0, and their row 0
                L = fmaf(ml[j].y, f, L);
#pragma unroll
                for (int e = 0; e < E; ++e) O[e] = fmaf(v[j][e], f, O[e]);
            }
        }
        bf *dst = static_cast<bf *>(a.out) + (long long)tok * a.so.tok + hq * a.so.head + lane * E;
        const float inv = 1.f / L;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(dst + e) = pack_bf16x2(O[e] * inv, O[e + 1] * inv);
    }
}

template <typename K>
cudaError_t big_smem(K kern, size_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

template <int D>
cudaError_t launch_tc_prep(const Step &a, const TcWs &y, cudaStream_t stream) {
    const cudaError_t e = big_smem(tc_prep_kernel<D>, PrepSmem<D>::bytes);
    if (e != cudaSuccess) return e;
    // a CTA takes all query heads of a key head, or fewer while CTAs would be idle (what they
    // share is then formed by each: the step waits for the slowest CTA, not for the sum)
    const int slots = slots_of(a.N, a.c.seqs), room = 152 * (D == 64 ? 2 : 1) / (slots * a.c.Hkv);
    const int z = room < 1 ? 1 : room < a.c.G ? room : a.c.G;
    return launch(tc_prep_kernel<D>, dim3(slots + 1, a.c.Hkv, z), kThr, PrepSmem<D>::bytes, stream, true, a, y);
}

// Chunks of several blocks: new keys into the pages and the chunks' products (before the
// attention, which takes those of short sequences).
template <int D>
cudaError_t launch_tc_carry(const Step &a, const TcWs &y, cudaStream_t stream) {
    cudaError_t e;
    if ((e = big_smem(tc_carry_kernel<D, 1>, CarrySmem<D>::bytes)) != cudaSuccess ||
        (e = big_smem(tc_carry_kernel<D, 2>, CarrySmem<D>::bytes)) != cudaSuccess)
        return e;
    const int slots = slots_of(a.N, a.c.seqs), groups = slots / kGroup + a.c.seqs;
    e = launch(tc_carry_kernel<D, 1>, dim3((groups * (D / 64) + slots) * a.c.Hkv), kThr, CarrySmem<D>::bytes, stream,
               false, a, y, groups);
    if (e == cudaSuccess && a.max_chunk > kC * kGroup)
        e = launch(tc_carry_kernel<D, 2>, dim3((a.c.seqs * (D / 64) + slots) * a.c.Hkv), kThr, CarrySmem<D>::bytes,
                   stream, false, a, y, a.c.seqs);
    return e;
}

// The rest of a step after its attention: outputs, the cached keys of sequences of more than one
// tile, the gate sums.
template <int D>
cudaError_t launch_tc_finish(const Step &a, const TcWs &y, cudaStream_t stream) {
    const long long cap = (long long)a.c.max_pages << a.c.page_shift;
    // few rows: a warp for each, its parts eight at a time; many (whose sequences have few parts):
    // four a warp
    const bool few = y.R * a.c.Hkv < 8 * 152 * 24;
    const int rows = few ? 1 : 4, per = kThr / 32 * rows;
    cudaError_t e = launch(few ? tc_combine_kernel<D, 8> : tc_combine_kernel<D, 2>,
                           dim3((unsigned)((y.R + per - 1) / per), a.c.Hkv), kThr, 0, stream, false, a, y, rows);
    if (e != cudaSuccess || cap == 0) return e;  // no sequence has room for a token
    if (!one_tile(a.max_chunk, a.c.G, D, a.log_f != nullptr)) {
        const size_t bytes = TransformSmem<D>::bytes;
        if ((e = big_smem(tc_transform_kernel<D>, bytes)) != cudaSuccess) return e;
        // one wave for one long sequence, at least 256 positions a CTA (further long sequences take
        // further waves, the others' CTAs leave at once)
        long long parts = (152 + a.c.Hkv - 1) / a.c.Hkv;
        if (parts > (cap + 255) / 256) parts = (cap + 255) / 256;
        e = launch(tc_transform_kernel<D>, dim3((unsigned)parts, a.c.Hkv, a.c.seqs), kThr, bytes, stream, false, a, y);
        if (e != cudaSuccess) return e;
    }
    if (a.log_f != nullptr)
        e = launch(tc_gates_kernel, dim3((unsigned)((cap + 4 * kThr - 1) / (4 * kThr)), a.c.Hq, a.c.seqs), kThr, 0,
                   stream, false, a, y);
    return e;
}

template cudaError_t launch_tc_prep<64>(const Step &, const TcWs &, cudaStream_t);
template cudaError_t launch_tc_prep<128>(const Step &, const TcWs &, cudaStream_t);
template cudaError_t launch_tc_carry<64>(const Step &, const TcWs &, cudaStream_t);
template cudaError_t launch_tc_carry<128>(const Step &, const TcWs &, cudaStream_t);
template cudaError_t launch_tc_finish<64>(const Step &, const TcWs &, cudaStream_t);
template cudaError_t launch_tc_finish<128>(const Step &, const TcWs &, cudaStream_t);

}  // namespace paged
}  // namespace path
