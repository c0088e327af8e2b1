// The prefixes of an fp32 step (paged_prefix.cuh), on the CUDA cores: plan, queries, the pass over the
// shared keys (paged_f32.cuh) and its joining.
#include "paged_f32.cuh"
#include "paged_prefix.cuh"

namespace path {
namespace paged {

namespace {

static_assert(kThr == kPrefixThr, "place_tokens");

__global__ void __launch_bounds__(kThr) prefix_plan_f32_kernel(const StepMore a, const Prefix x) {
    grid_begin();
    place_tokens(a, x);
    grid_wait();  // what it writes is this call's alone
}

// Where token t of sequence b, which continues p, stands in the shared step's blocks of 64: the row over
// all blocks of a query head is slot * 64 + ..
__device__ __forceinline__ size_t place_of(const Prefix &x, int b, int p, int t) {
    const int first = x.cu[p], i = x.start[b] - first + t;
    return (size_t)(first / kC + p + i / kC) * kC + i % kC;
}
// that row's place in a (slots, Hq, 64) array
__device__ __forceinline__ size_t row_of(size_t place, int Hq, int hq) {
    return (place / kC * Hq + hq) * kC + place % kC;
}

// ---------------------------------------------------------------- queries
template <int D>
constexpr size_t query_smem() { return (size_t)2 * (D / 64) * TILE * 4; }

// 64 tokens of a query head, X C^T, or all heads of a key head of a sequence's only token; y: the step's,
// z: those of the shared step.
template <int D>
__global__ void __launch_bounds__(kThr)
prefix_query_f32_kernel(const StepMore a, const Prefix x, const Ws y, const Ws z) {
    constexpr int NH = D / 64;
    extern __shared__ float sm[];
    float *const X = sm, *const C = X + NH * TILE;
    const int slot = blockIdx.x, hq = blockIdx.y, h = hq / a.c.G, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    int b, c;
    Seq s;
    grid_begin();
    const bool mine = block_of(a, slot, b, c, s);
    grid_wait();
    if (!mine || x.start[b] < 0) return;
    const int p = __ldg(x.of + b);
    if (s.T == 1) {
        if (hq % a.c.G != 0) return;
        const size_t at = place_of(x, b, p, 0);
        prefix_single<float, D, D>(
            a, x, s, b, h, 0, [&](int g, int i, float q) { z.qt[row_of(at, a.c.Hq, h * a.c.G + g) * D + i] = q; },
            [&](int g, float t) { z.gq[row_of(at, a.c.Hq, h * a.c.G + g)] = t; });
        return;
    }
    const int rows = min(kC, s.T - c * kC);
    const size_t bq = (size_t)slot * a.c.Hq + hq;
    load_rows<D>(X, y.qt + bq * kC * D);
    for (int x1 = 0; x1 < NH; ++x1) {
        __syncthreads();
        load_rows<D>(C, x.carry + (((size_t)b * a.c.Hkv + h) * D + 64 * x1) * D);
        __syncthreads();
        Acc q;
        zero(q);
#pragma unroll
        for (int x2 = 0; x2 < NH; ++x2) mm_nt(X + x2 * TILE, C + x2 * TILE, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            if (r >= rows) continue;
            float *const dst = z.qt + row_of(place_of(x, b, p, c * kC + r), a.c.Hq, hq) * D + 64 * x1;
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[tx + 16 * j] = q[i][j];
        }
    }
    if (a.log_f != nullptr && tid < rows)
        z.gq[row_of(place_of(x, b, p, c * kC + tid), a.c.Hq, hq)] =
            y.gq[bq * kC + tid] + x.gates[(size_t)b * a.c.Hq + hq];
}

// ---------------------------------------------------------------- join
// A warp per row: the parts of its prefix's keys into one; grid (slots, Hq, 8).
template <int D>
__global__ void __launch_bounds__(kThr)
prefix_join_f32_kernel(const StepMore a, const StepMore v, const Prefix x, const Ws z) {
    constexpr int E = D / 32;
    const int slot = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x & 31, r = blockIdx.z * 8 + (threadIdx.x >> 5);
    int b, c;
    Seq s;
    grid_begin();
    const bool mine = block_of(a, slot, b, c, s) && r < s.T - c * kC;
    grid_wait();
    if (!mine || x.start[b] < 0) return;
    const int p = __ldg(x.of + b), t = c * kC + r;
    const size_t place = place_of(x, b, p, t);
    const int tiles = (seq_of(v, p).n + kC - 1) / kC, per = (tiles + z.splits - 1) / z.splits;
    const int used = per > 0 ? (tiles + per - 1) / per : 0;
    const float *const first = z.part + ((place / kC * a.c.Hq + hq) * (1 + z.splits) + 1) * kPart<D>;
    const int row = (int)(place % kC);
    float M = -INFINITY, L = 0.f, O[E];
#pragma unroll
    for (int e = 0; e < E; ++e) O[e] = 0.f;
    for (int i = 0; i < used; ++i) {
        const float *const q = first + i * kPart<D>;
        const float m = q[kC * D + row], top = fmaxf(M, m), use = top == -INFINITY ? 0.f : top;
        const float f0 = exp2f(M - use), f1 = exp2f(m - use);
        M = top;
        L = fmaf(q[kC * D + kC + row], f1, L * f0);
#pragma unroll
        for (int e = 0; e < E; ++e) O[e] = fmaf(q[row * D + lane * E + e], f1, O[e] * f0);
    }
    const size_t at = ((size_t)(hq / a.c.G) * a.N + s.first + t) * a.c.G + hq % a.c.G;
#pragma unroll
    for (int e = 0; e < E; ++e) x.px[at * D + lane * E + e] = O[e];
    if (lane == 0) x.pxml[at] = make_float2(M, L);
}

template <int D>
cudaError_t launch_all(const StepMore &a, const Prefix &x, const Ws &y, const Ws &z, bool first, cudaStream_t stream) {
    const StepMore v = shared_step(a, x);
    const int nslots = slots_of(a.N, a.c.seqs);
    cudaError_t e;
    if ((e = big_smem(prefix_query_f32_kernel<D>, query_smem<D>())) != cudaSuccess ||
        (e = big_smem(f32_cached_kernel<D, true, StepMore>, cached_smem<D>())) != cudaSuccess)
        return e;
    e = launch(prefix_plan_f32_kernel, dim3(1), kThr, 0, stream, first, a, x);
    if (e == cudaSuccess)
        e = launch(prefix_query_f32_kernel<D>, dim3(nslots, a.c.Hq), kThr, query_smem<D>(), stream, false, a, x, y, z);
    if (e == cudaSuccess)
        e = launch(f32_cached_kernel<D, true, StepMore>, dim3(nslots, a.c.Hq, z.splits), kThr, cached_smem<D>(), stream,
                   false, v, z);
    if (e == cudaSuccess)
        e = launch(prefix_join_f32_kernel<D>, dim3(nslots, a.c.Hq, kC / 8), kThr, 0, stream, false, a, v, x, z);
    if (e == cudaSuccess) e = launch_prefix_carry<float, D>(a, x, stream);
    return e;
}

// The workspace's part for prefixes, from `w` on.
size_t layout(const StepMore &a, int d, char *w, Prefix *x, Ws *z) {
    const Cache &c = a.c;
    const size_t rows = (size_t)a.N * c.G * c.Hkv, slots = slots_of(a.N, c.seqs), blocks = slots * c.Hq;
    const long long cap = (long long)c.max_pages << c.page_shift, most = (cap + 63) / 64,
                    want = 608 / (long long)blocks + 1;
    z->splits = (int)(want < most ? want : most > 0 ? most : 1);
    z->singles = false;
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
    z->qt = reinterpret_cast<float *>(take(blocks * kC * d * 4));
    z->gq = reinterpret_cast<float *>(take(blocks * kC * 4));
    // (1 + splits) parts a block, by a bound that does not fall as the blocks rise
    z->part = reinterpret_cast<float *>(take((2 * blocks + 608) * kC * (d + 2) * 4));
    return off;
}

}  // namespace

size_t prefix_f32_bytes(const StepMore &a, int d) {
    Prefix x;
    Ws z;
    return layout(a, d, nullptr, &x, &z);
}

// y_qt, y_gq: the step's queries carried to the chunk's start and their gates, null where it has single
// tokens alone (theirs are formed from the inputs).
cudaError_t launch_prefix_f32(StepMore &a, int d, float *carry, float *gates, float *y_qt, float *y_gq, void *ws,
                              bool first, cudaStream_t stream) {
    Prefix x;
    Ws z = {};
    layout(a, d, static_cast<char *>(ws), &x, &z);
    x.of = a.prefix_of;
    x.carry = carry;
    x.gates = gates;
    a.pstart = x.start;
    a.px = x.px;
    a.pxml = x.pxml;
    Ws y = z;
    y.qt = y_qt;
    y.gq = y_gq;
    return d == 64 ? launch_all<64>(a, x, y, z, first, stream) : launch_all<128>(a, x, y, z, first, stream);
}

}  // namespace paged
}  // namespace path
