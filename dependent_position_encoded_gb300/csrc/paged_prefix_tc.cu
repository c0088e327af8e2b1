// The prefixes of a bf16 step (paged_prefix.cuh): plan, queries, the pass over the shared keys on
// tcgen05 tensor cores (paged_cached_tc.cuh) and its joining.
#include "paged_cached_tc.cuh"
#include "paged_prefix.cuh"

namespace path {
namespace paged {

EACH_PASS(PASS, Pass::shared)

namespace {

static_assert(kThr == kPrefixThr, "make_plans");

template <int D>
__global__ void __launch_bounds__(kThr) prefix_plan_kernel(const Step a, const Step v, const Prefix x, const TcWs y) {
    __shared__ long long sums[2 * kThr / 32];
    grid_begin();
    place_tokens(a, x);
    make_plans<D>(v, y, sums);
    grid_wait();  // what it writes is this call's alone
}

// ---------------------------------------------------------------- queries
template <int D>
struct QuerySmem {
    static constexpr int LDD = D + 8;
    static constexpr size_t Ch = 0, Cl = (size_t)D * LDD * 2, Xh = 2 * Cl, Xl = Xh + (size_t)kC * LDD * 2,
                            bytes = Xl + (size_t)kC * LDD * 2;
};

// 64 rows of a sequence and key head, X C^T with both in two bf16 parts (16 bits of significand), or
// its only token's. y: the step's, whose queries have been carried to the chunk's start; z: those of the
// shared step.
template <int D>
__global__ void __launch_bounds__(kThr) prefix_query_kernel(const Step a, const Prefix x, const TcWs y, const TcWs z) {
    using S = QuerySmem<D>;
    constexpr int LDD = S::LDD, NT = D / 16, PER = D / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    const int h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, G = a.c.G;
    int b, tile;
    Seq s;
    grid_begin();
    const bool mine = tile_of(a, blockIdx.x, kC, b, tile, s);
    grid_wait();
    if (!mine || x.start[b] < 0) return;
    const size_t from = (size_t)h * y.R + (size_t)s.first * G, to = (size_t)h * y.R + (size_t)x.start[b] * G;
    if (s.T == 1) {
        if (tile > 0) return;
        prefix_single<bf, D>(
            a, x, s, b, h,
            [&](int g, int i, float q) {
                q *= a.scale_log2;
                const bf hi = __float2bfloat16_rn(q);
                z.qt[(to + g) * D + i] = hi;
                z.ql[(to + g) * D + i] = __float2bfloat16_rn(q - __bfloat162float(hi));
            },
            [&](int g, float t) { z.gq[to + g] = t; });
        return;
    }
    bf *const Ch = reinterpret_cast<bf *>(smem + S::Ch), *const Cl = reinterpret_cast<bf *>(smem + S::Cl),
       *const Xh = reinterpret_cast<bf *>(smem + S::Xh), *const Xl = reinterpret_cast<bf *>(smem + S::Xl);
    const int row0 = kC * tile, rows = min(kC, s.T * G - row0);
    for (int e = tid; e < kC * PER; e += kThr) {
        const int r = e / PER, q = e % PER * 8;
        const size_t at = (from + row0 + r) * D + q;
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(Xh + r * LDD + q) = r < rows ? *reinterpret_cast<const uint4 *>(y.qt + at) : none;
        *reinterpret_cast<uint4 *>(Xl + r * LDD + q) = r < rows ? *reinterpret_cast<const uint4 *>(y.ql + at) : none;
    }
    const float4 *const C = reinterpret_cast<const float4 *>(x.carry + ((size_t)b * a.c.Hkv + h) * D * D);
#pragma unroll 4
    for (int e = tid; e < D * D / 4; e += kThr) {
        const int r = e / (D / 4), q = e % (D / 4) * 4;
        const float4 c = C[e];
        uint2 hi, lo;
        split2(c.x, c.y, hi.x, lo.x);
        split2(c.z, c.w, hi.y, lo.y);
        *reinterpret_cast<uint2 *>(Ch + r * LDD + q) = hi;
        *reinterpret_cast<uint2 *>(Cl + r * LDD + q) = lo;
    }
    __syncthreads();
    const int m0 = 16 * (warp & 3), n0 = D / 2 * (warp >> 2);
    float acc[NT][4];
    zero_acc(acc);
    warp_mma_3<NT, false>(acc, Xh, Xl, LDD, m0, Ch, Cl, LDD, n0, D / 16);
    each_eight(
        acc, m0, n0, [](int, int, float &, float &) {},
        [&](int i, int j, uint4 hi, uint4 lo) {
            if (i >= rows) return;
            *reinterpret_cast<uint4 *>(z.qt + (to + row0 + i) * D + j) = hi;
            *reinterpret_cast<uint4 *>(z.ql + (to + row0 + i) * D + j) = lo;
        });
    if (a.log_f != nullptr && tid < rows)
        z.gq[to + row0 + tid] = y.gq[from + row0 + tid] + x.gates[(size_t)b * a.c.Hq + h * G + (row0 + tid) % G];
}

// ---------------------------------------------------------------- join
// A warp per row: the parts of its prefix's keys into one, four at a time.
template <int D>
__global__ void __launch_bounds__(kThr) prefix_join_kernel(const Step a, const Step v, const Prefix x, const TcWs z) {
    constexpr int E = D / 32, P = 4;
    const int G = a.c.G, h = blockIdx.y, lane = threadIdx.x & 31;
    const long long r = blockIdx.x * (long long)(kThr / 32) + (threadIdx.x >> 5);
    grid_begin();
    // the sequence of the row: the last that begins at or before its token
    int b = 0;
    Seq s{0, 0, 0};
    const int tok = (int)(r / G);
    if (r < z.R) {
        for (int hi = a.c.seqs - 1; b < hi;) {
            const int mid = (b + hi + 1) >> 1;
            if (__ldg(a.cu + mid) <= tok) b = mid;
            else hi = mid - 1;
        }
        s = seq_of(a, b);
    }
    grid_wait();
    if (r >= z.R || tok < s.first || tok >= s.first + s.T || x.start[b] < 0) return;
    const int p = __ldg(x.of + b);
    const Seq g = seq_of(v, p);
    const int row = (x.start[b] - g.first + tok - s.first) * G + (int)(r - (long long)tok * G);
    const RowParts parts = parts_of(v, z, g, p, h, row, D);
    float M = -INFINITY, L = 0.f, O[E];
#pragma unroll
    for (int e = 0; e < E; ++e) O[e] = 0.f;
    for (int q0 = 0; q0 < parts.number; q0 += P) {
        float2 ml[P];
        float w[P][E], m = M;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            ml[j] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) w[j][e] = 0.f;
            if (q0 + j < parts.number) {
                const size_t at = parts.at(q0 + j);
                ml[j] = parts.sml[at];
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 t = *reinterpret_cast<const float2 *>(parts.so + at * D + lane * E + e);
                    w[j][e] = t.x;
                    w[j][e + 1] = t.y;
                }
            }
            m = fmaxf(m, ml[j].x);
        }
        const float use = m == -INFINITY ? 0.f : m, f0 = exp2f(M - use);
        M = m;
        L *= f0;
#pragma unroll
        for (int e = 0; e < E; ++e) O[e] *= f0;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float f = exp2f(ml[j].x - use);  // absent keys alone: 0, and their row 0
            L = fmaf(ml[j].y, f, L);
#pragma unroll
            for (int e = 0; e < E; ++e) O[e] = fmaf(w[j][e], f, O[e]);
        }
    }
    const size_t at = (size_t)h * z.R + r;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<float2 *>(x.px + at * D + lane * E + e) = make_float2(O[e], O[e + 1]);
    if (lane == 0) x.pxml[at] = make_float2(M, L);
}

template <int D, bool FOX>
cudaError_t launch_all(const Step &a, const Prefix &x, const TcWs &y, const TcWs &z, bool first, uint64_t limit_ns,
                       cudaStream_t stream) {
    const Step v = shared_step(a, x);
    cudaError_t e = launch(prefix_plan_kernel<D>, dim3(1), kThr, 0, stream, first, a, v, x, z);
    if (e == cudaSuccess) e = big_smem(prefix_query_kernel<D>, QuerySmem<D>::bytes);
    if (e == cudaSuccess)
        e = launch(prefix_query_kernel<D>, dim3(tile_slots(a.N, a.c.G, a.c.seqs, kC), a.c.Hkv), kThr,
                   QuerySmem<D>::bytes, stream, false, a, x, y, z);
    if (e == cudaSuccess) e = launch_cached<1, D, FOX, Pass::shared>(v, z, limit_ns, stream);
    if (e == cudaSuccess && (long long)a.N * a.c.G > 128) e = launch_cached<2, D, FOX, Pass::shared>(v, z, limit_ns, stream);
    if (e == cudaSuccess)
        e = launch(prefix_join_kernel<D>, dim3((unsigned)((z.R + kThr / 32 - 1) / (kThr / 32)), a.c.Hkv), kThr, 0,
                   stream, false, a, v, x, z);
    if (e == cudaSuccess) e = launch_prefix_carry<bf, D>(a, x, stream);
    return e;
}

// The workspace's part for prefixes, from the byte `off` on: plan, queries, parts of the shared step.
size_t layout(const Step &a, int d, char *w, Prefix *x, TcWs *z) {
    const Cache &c = a.c;
    const size_t rows = (size_t)a.N * c.G * c.Hkv;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *const at = w + off;
        off = align256(off + bytes);
        return at;
    };
    x->cu = reinterpret_cast<int *>(take(((size_t)c.seqs + 1) * 4));
    x->start = reinterpret_cast<int *>(take((size_t)c.seqs * 4));
    x->px = reinterpret_cast<float *>(take(rows * d * 4));
    x->pxml = reinterpret_cast<float2 *>(take(rows * 8));
    z->qt = reinterpret_cast<bf *>(take(rows * d * 2));
    z->ql = reinterpret_cast<bf *>(take(rows * d * 2));
    z->gq = reinterpret_cast<float *>(take(rows * 4));
    for (int p = 0; p < 2; ++p) {
        const int ctas = 152 * (p == 0 && d == 64 ? CachedCfg<1, 64, Pass::shared>::ctas_per_sm : 1);
        const size_t tile = 128 * (p + 1);
        // (both plans in any case: the sizes must not fall as the step grows)
        const size_t parts = ctas + (size_t)tile_slots(a.N, c.G, c.seqs < a.N ? c.seqs : a.N, (int)tile) * c.Hkv;
        z->so[p] = reinterpret_cast<float *>(take(parts * tile * d * 4));
        z->sml[p] = reinterpret_cast<float2 *>(take(parts * tile * 8));
        long long *const units = reinterpret_cast<long long *>(take(((size_t)c.seqs + 1) * 8));
        z->plan[p] = Plan{units, reinterpret_cast<long long *>(take(((size_t)c.seqs + 1) * 8)), ctas};
    }
    z->mt = z->qt;  // no keys are advanced
    z->R = (long long)a.N * c.G;
    return off;
}

}  // namespace

size_t prefix_tc_bytes(const Step &a, int d) {
    Prefix x;
    TcWs z;
    return layout(a, d, nullptr, &x, &z);
}

cudaError_t launch_prefix_tc(Step &a, int d, float *carry, float *gates, const TcWs *y, void *ws, bool first,
                             uint64_t limit_ns, cudaStream_t stream) {
    Prefix x;
    TcWs z = {};
    layout(a, d, static_cast<char *>(ws), &x, &z);
    x.of = a.prefix_of;
    x.carry = carry;
    x.gates = gates;
    a.px = x.px;
    a.pxml = x.pxml;
    TcWs from = y != nullptr ? *y : z;  // (single tokens alone: their queries are formed from the inputs)
    from.R = z.R;
    const bool fox = a.log_f != nullptr;
    if (d == 64)
        return fox ? launch_all<64, true>(a, x, from, z, first, limit_ns, stream)
                   : launch_all<64, false>(a, x, from, z, first, limit_ns, stream);
    return fox ? launch_all<128, true>(a, x, from, z, first, limit_ns, stream)
               : launch_all<128, false>(a, x, from, z, first, limit_ns, stream);
}

}  // namespace paged
}  // namespace path
