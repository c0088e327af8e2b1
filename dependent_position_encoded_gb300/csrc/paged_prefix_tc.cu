// The prefixes of a bf16 step (paged_prefix.cuh): plan, queries and the pass over the shared keys on
// tcgen05 tensor cores (paged_cached_tc.cuh); and steps of single tokens behind them or through a window.
#include "paged_cached_tc.cuh"
#include "paged_prefix.cuh"

namespace path {
namespace paged {

SHARED_PASS(PASS)

namespace {

static_assert(kThr == kPrefixThr, "make_plans");

// ---------------------------------------------------------------- plans and single tokens
// Grid (plans and sequences, key heads). The first CTA makes the plan of the prefixes, the next one (OWN)
// that of the step, the others take the single tokens, a sequence and key head each (BEHIND: and 64 rows
// of its carry): OWN, of a step that has no others, enter them into the cache and leave their queries and
// parts; BEHIND, carry their queries to the prefix's end, as a high and a low bf16 part (16 bits of
// significand: keeps_low says what one part costs). With few sequences and heads these find their places
// by themselves beside the plan, each CTA reading all sequences' lengths, else in one made before, by a
// launch of this kernel without sequences. Steps of single tokens behind 500 keys, us, beside / before:
//   2 heads, d = 64:   30 sequences 21/25, 500 64/70, 1,000 105/113, 2,000 225/226, 4,000 501/428
//   8 heads, d = 128:  30 sequences 28/32, 250 152/153, 500 281/269, 1,000 567/502, 4,000 3,613/1,968
constexpr long long kFused = 1 << 20;  // lengths read by all CTAs, at most

template <int D, bool OWN, bool BEHIND>
__global__ void __launch_bounds__(kThr) tc_single_kernel(const StepMore a, const StepMore v, const Prefix x,
                                                         const TcWs y, const TcWs z, int plans, bool fused) {
    __shared__ long long sums[2 * kThr / 32];
    const int G = a.c.G;
    grid_begin();
    // (no kernel before reads or writes what this one does, but for a plan made before)
    if ((int)blockIdx.x < plans) {
        if (blockIdx.y == 0) {
            if (BEHIND && blockIdx.x == 0) {
                place_tokens(a, x);
                make_plans<D>(v, z, sums);
            } else if (OWN) {
                make_plans<D>(a, y, sums);
            }
        }
        grid_wait();
        return;
    }
    constexpr int kParts = BEHIND ? D / 64 : 1;
    const int b = (blockIdx.x - plans) / kParts, part = (blockIdx.x - plans) % kParts, h = blockIdx.y;
    if (!fused) grid_wait();
    const Seq s = seq_of(a, b);
    if (s.T == 1) {
        int start = -1;
        // the carry's rows are on their way while the place is looked for
        if (BEHIND && (int)threadIdx.x < 64 * D * 4 / 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(x.carry + (((size_t)b * a.c.Hkv + h) * D + 64 * part) * D +
                                                          threadIdx.x * 32));
        if (BEHIND && __ldg(x.of + b) >= 0) start = fused ? place_one(a, x, b) : x.start[b];
        if (OWN && part == 0) enter_single<D>(a, y, s, b, slot_of(s, b, 0), h);
        if (BEHIND && start >= 0) {
            const size_t to = (size_t)h * z.R + (size_t)start * G;
            prefix_single<bf, D, 64>(
                a, x, s, b, h, 64 * part,
                [&](int g, int i, float q) {
                    q *= a.scale_log2;
                    const bf hi = __float2bfloat16_rn(q);
                    z.qt[(to + g) * D + i] = hi;
                    z.ql[(to + g) * D + i] = __float2bfloat16_rn(q - __bfloat162float(hi));
                },
                [&](int g, float t) { z.gq[to + g] = t; });
        }
    }
    if (fused) grid_wait();
}

template <int D, bool OWN, bool BEHIND>
cudaError_t launch_tokens(const StepMore &a, const Prefix &x, const TcWs &y, const TcWs &z, bool first,
                          cudaStream_t stream) {
    const StepMore v = BEHIND ? shared_step(a, x) : a;
    const int items = a.c.seqs * (BEHIND ? D / 64 : 1), plans = (OWN ? 1 : 0) + (BEHIND ? 1 : 0);
    const auto kern = tc_single_kernel<D, OWN, BEHIND>;
    if (!BEHIND || (long long)items * a.c.Hkv * a.c.seqs <= kFused)
        return launch(kern, dim3(plans + items, a.c.Hkv), kThr, 0, stream, first, a, v, x, y, z, plans, true);
    const cudaError_t e = launch(kern, dim3(plans), kThr, 0, stream, first, a, v, x, y, z, plans, true);
    return e != cudaSuccess ? e : launch(kern, dim3(items, a.c.Hkv), kThr, 0, stream, false, a, v, x, y, z, 0, false);
}

// ---------------------------------------------------------------- queries of several tokens
// X C^T over tiles of 64 rows of a sequence and key head, kTiles of them on one load of C, both factors
// in two bf16 parts (16 bits of significand; 3 of the 4 products, mma.sync: the rows' bytes bound it). 51 us
// for 80,000 rows at D = 128, 82 MB of them: 1.6 TB/s, two CTAs an SM. y: the step's, whose queries have been
// carried to the chunk's start; z: those of the shared step.
constexpr int kTiles = 4;

template <int D>
struct QuerySmem {
    static constexpr int LDD = D + 8;
    static constexpr size_t Ch = 0, Cl = (size_t)D * LDD * 2, Xh = 2 * Cl, Xl = Xh + (size_t)kC * LDD * 2,
                            bytes = Xl + (size_t)kC * LDD * 2;
};

template <int D>
__global__ void __launch_bounds__(kThr, 2)
prefix_query_kernel(const StepMore a, const Prefix x, const TcWs y, const TcWs z) {
    using S = QuerySmem<D>;
    constexpr int LDD = S::LDD, NT = D / 16, PER = D / 8, IT = kC * PER / kThr;
    extern __shared__ __align__(16) uint8_t smem[];
    const int h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, G = a.c.G;
    int b, part;
    Seq s;
    grid_begin();
    const bool mine = tile_of(a, blockIdx.x, kC * kTiles, b, part, s) && s.T > 1;
    bf *const Ch = reinterpret_cast<bf *>(smem + S::Ch), *const Cl = reinterpret_cast<bf *>(smem + S::Cl),
       *const Xh = reinterpret_cast<bf *>(smem + S::Xh), *const Xl = reinterpret_cast<bf *>(smem + S::Xl);
    const bool behind = mine && __ldg(x.of + b) >= 0;
    if (behind) {
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
    }
    grid_wait();
    if (!behind || x.start[b] < 0) return;
    const size_t from = (size_t)h * y.R + (size_t)s.first * G, to = (size_t)h * y.R + (size_t)x.start[b] * G;
    const int rows_all = s.T * G, m0 = 16 * (warp & 3), n0 = D / 2 * (warp >> 2);
    uint4 xh[IT], xl[IT];
    auto fetch = [&](int row0) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int e = tid + i * kThr, r = row0 + e / PER;
            const size_t at = (from + r) * D + e % PER * 8;
            xh[i] = r < rows_all ? *reinterpret_cast<const uint4 *>(y.qt + at) : make_uint4(0u, 0u, 0u, 0u);
            xl[i] = r < rows_all ? *reinterpret_cast<const uint4 *>(y.ql + at) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    const int first = kC * kTiles * part, last = min(rows_all, first + kC * kTiles);
    fetch(first);
    for (int row0 = first; row0 < last; row0 += kC) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int e = tid + i * kThr, at = e / PER * LDD + e % PER * 8;
            *reinterpret_cast<uint4 *>(Xh + at) = xh[i];
            *reinterpret_cast<uint4 *>(Xl + at) = xl[i];
        }
        if (row0 + kC < last) fetch(row0 + kC);
        __syncthreads();
        float acc[NT][4];
        zero_acc(acc);
        warp_mma_3<NT, false>(acc, Xh, Xl, LDD, m0, Ch, Cl, LDD, n0, D / 16);
        each_eight(
            acc, m0, n0, [](int, int, float &, float &) {},
            [&](int i, int j, uint4 hi, uint4 lo) {
                if (row0 + i >= rows_all) return;
                *reinterpret_cast<uint4 *>(z.qt + (to + row0 + i) * D + j) = hi;
                *reinterpret_cast<uint4 *>(z.ql + (to + row0 + i) * D + j) = lo;
            });
        if (a.log_f != nullptr && tid < kC && row0 + tid < rows_all)
            z.gq[to + row0 + tid] = y.gq[from + row0 + tid] + x.gates[(size_t)b * a.c.Hq + h * G + (row0 + tid) % G];
    }
}

// The attention of the prefixes' sequences, behind their queries.
template <int D, bool FOX>
cudaError_t launch_shared(const StepMore &a, const Prefix &x, const TcWs &z, uint64_t limit_ns, cudaStream_t stream) {
    const StepMore v = shared_step(a, x);
    const cudaError_t e = launch_cached<1, D, FOX, Pass::shared>(v, z, limit_ns, stream);
    if (e != cudaSuccess || (long long)a.N * a.c.G <= a.one_rows) return e;
    if constexpr (D == 64 && FOX) return cudaErrorInvalidValue;  // (prefix_one_rows: all go with NT = 1)
    else return launch_cached<2, D, FOX, Pass::shared>(v, z, limit_ns, stream);
}

template <int D, bool FOX>
cudaError_t launch_all(const StepMore &a, const Prefix &x, const TcWs *y, const TcWs &z, bool first, uint64_t limit_ns,
                       cudaStream_t stream) {
    cudaError_t e = launch_tokens<D, false, true>(a, x, z, z, first, stream);
    if (a.max_chunk > 1) {
        if (e == cudaSuccess) e = big_smem(prefix_query_kernel<D>, QuerySmem<D>::bytes);
        if (e == cudaSuccess)
            e = launch(prefix_query_kernel<D>, dim3(tile_slots(a.N, a.c.G, a.c.seqs, kC * kTiles), a.c.Hkv), kThr,
                       QuerySmem<D>::bytes, stream, false, a, x, *y, z);
    }
    if (e == cudaSuccess) e = launch_shared<D, FOX>(a, x, z, limit_ns, stream);
    if (e == cudaSuccess) e = launch_prefix_carry<bf, D>(a, x, stream);
    return e;
}

// A step of single tokens, through a window or behind prefixes, up to its joining.
template <int D, bool FOX>
cudaError_t launch_ones(const StepMore &a, const Prefix *x, const TcWs &y, const TcWs &z, uint64_t limit_ns,
                        cudaStream_t stream) {
    cudaError_t e = x != nullptr ? launch_tokens<D, true, true>(a, *x, y, z, true, stream)
                                 : launch_tokens<D, true, false>(a, Prefix{}, y, z, true, stream);
    if (e == cudaSuccess && a.c.max_pages > 0) e = launch_cached<1, D, FOX, Pass::one>(a, y, limit_ns, stream);
    if (e == cudaSuccess && x != nullptr) e = launch_shared<D, FOX>(a, *x, z, limit_ns, stream);
    return e;
}

// The workspace's part for prefixes, from the byte `off` on: plan, queries, parts of the shared step.
size_t layout(const StepMore &a, int d, char *w, Prefix *x, TcWs *z) {
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
    z->qt = reinterpret_cast<bf *>(take(rows * d * 2));
    z->ql = reinterpret_cast<bf *>(take(rows * d * 2));
    z->gq = reinterpret_cast<float *>(take(rows * 4));
    for (int p = 0; p < 2; ++p) {
        const int ctas = 152 * (p == 0 && d == 64 ? CachedCfg<1, 64, Pass::shared, false>::ctas_per_sm : 1);
        const size_t tile = 128 * (p + 1);
        // (both plans in any case: the sizes must not fall as the step grows)
        const size_t parts = ctas + (size_t)tile_slots(a.N, c.G, c.seqs < a.N ? c.seqs : a.N, (int)tile) * c.Hkv;
        z->so[p] = reinterpret_cast<float *>(take(parts * tile * d * 4));
        z->sml[p] = reinterpret_cast<float2 *>(take(parts * tile * 8));
        long long *const units = reinterpret_cast<long long *>(take(((size_t)c.seqs + 1) * 8));
        z->plan[p] = Plan{units, reinterpret_cast<long long *>(take(((size_t)c.seqs + 1) * 8)), ctas};
    }
    z->R = (long long)a.N * c.G;
    return off;
}

}  // namespace

size_t prefix_tc_bytes(const StepMore &a, int d) {
    Prefix x;
    TcWs z;
    return layout(a, d, nullptr, &x, &z);
}

namespace {

Prefix prefix_at(const StepMore &a, int d, float *carry, float *gates, void *ws, TcWs *z, Behind *behind) {
    Prefix x = {};
    layout(a, d, static_cast<char *>(ws), &x, z);
    x.of = a.prefix_of;
    x.carry = carry;
    x.gates = gates;
    *behind = Behind{x.of, x.cu, x.start, {z->so[0], z->so[1]}, {z->sml[0], z->sml[1]}, {z->plan[0], z->plan[1]}};
    return x;
}

}  // namespace

// y: the step's workspace, null for single tokens alone, whose queries are formed from the inputs;
// behind: what the step's joining takes up
cudaError_t launch_prefix_tc(const StepMore &a, int d, float *carry, float *gates, const TcWs *y, void *ws, bool first,
                             uint64_t limit_ns, Behind *behind, cudaStream_t stream) {
    TcWs z = {};
    const Prefix x = prefix_at(a, d, carry, gates, ws, &z, behind);
    const bool fox = a.log_f != nullptr;
    auto all = [&](auto run) { return run(a, x, y, z, first, limit_ns, stream); };
    if (d == 64) return fox ? all(launch_all<64, true>) : all(launch_all<64, false>);
    return fox ? all(launch_all<128, true>) : all(launch_all<128, false>);
}

cudaError_t launch_singles(const StepMore &a, int d, const TcWs &y, float *carry, float *gates, void *ws,
                           uint64_t limit_ns, Behind *behind, cudaStream_t stream) {
    TcWs z = {};
    Prefix x = {};
    if (carry != nullptr) x = prefix_at(a, d, carry, gates, ws, &z, behind);
    const bool fox = a.log_f != nullptr;
    auto all = [&](auto run) { return run(a, carry != nullptr ? &x : nullptr, y, z, limit_ns, stream); };
    if (d == 64) return fox ? all(launch_ones<64, true>) : all(launch_ones<64, false>);
    return fox ? all(launch_ones<128, true>) : all(launch_ones<128, false>);
}

}  // namespace paged
}  // namespace path
