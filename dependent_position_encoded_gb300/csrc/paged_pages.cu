// The pages of a paged cache: reserving, forking, freeing and compacting, on the device, so
// that a captured step can grow its sequences without the host.
//
// Every decode step rewrites every cached key of a sequence (review "거리에서 경로로, PaTH
// Attention" §9), so no two sequences can share a key page; values never change, so a fork
// shares the full value pages of its source and counts them. The counts (one per page) are
// the allocator's whole state: a page is free where its count is 0, and the lowest free
// pages are handed out first, in the order of the requests, so that the result does not
// depend on timing.
//
// Planning (counts, page numbers, tables) is one CTA per call, half of it for the key pool and
// half for the value pool, whose loops run over 8192 counts at a time; both pools are
// checked before either changes, so a call that does not fit changes nothing. The copies
// are a second launch over whole pages, bound by HBM (each byte read and written once): 16 forks
// of up to 12,000 positions, 8 heads, D = 128, 112 us for 0.66 GB (5.9 TB/s); compacting 9,000
// pages of 64 positions 174 us for 1.13 GB (6.5 TB/s). The plans are bound by the latency of their
// rounds: 9 us (fork of 3 rows), 13 (16 rows), 7 to 12 (reserve), 10 (compact, 300 pages), 20
// (9,000).
#include <climits>

#include "paged.cuh"
#include "paged_pages.cuh"

namespace path {
namespace paged {

namespace {

constexpr uint32_t kStatusCapacity = 6u;
constexpr int kPlanThr = 1024, kHalf = 512, kHalfWarps = kHalf / 32;
constexpr int kItems = 16;

struct Pool {
    int *table, *ref, *list, *list2, *cnt;
    int pages;
};

struct PagesWs {
    uint32_t *status;
    int *go;          // [0] whether the plan holds, [1 + pool] moves of a compaction
    int *list[2];     // per pool: free pages, or the holes of a compaction
    int *list2[2];    // per pool: the pages that move
    int *to[2];       // per pool: new number of a page that moves
    int *cnt[2];      // per pool and sequence
};

// Exclusive prefix sum over the 512 threads of a half; `total` is the half's sum. sums: 32
// ints of shared memory, one per warp of the CTA. Every thread of the CTA calls it.
__device__ __forceinline__ int half_scan(int v, int *sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half0 = warp & ~(kHalfWarps - 1);
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += t;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kHalfWarps; ++i) {
        const int t = sums[half0 + i];
        if (half0 + i < warp) before += t;
        total += t;
    }
    return before + x - v;
}

// kItems counts from index i (past the pool: -1, neither free nor live)
__device__ __forceinline__ void load_counts(const Pool &p, long long i, int (&r)[kItems]) {
#pragma unroll
    for (int q = 0; q < kItems; q += 4) {
        if (i + q + 3 < p.pages) {
            const int4 t = *reinterpret_cast<const int4 *>(p.ref + i + q);
            r[q] = t.x; r[q + 1] = t.y; r[q + 2] = t.z; r[q + 3] = t.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) r[q + e] = i + q + e < p.pages ? p.ref[i + q + e] : -1;
        }
    }
}

// The first `want` free pages of the half's pool into p.list, lowest first; returns how many
// there are (at most want). Every thread of the CTA calls it.
__device__ __forceinline__ int find_free(const Pool &p, int want, int most_pages, int *sums) {
    const int t = threadIdx.x & (kHalf - 1);
    int found = 0;
    for (long long base = 0; base < most_pages; base += kHalf * kItems) {
        int r[kItems], n = 0;
        load_counts(p, base + t * kItems, r);
#pragma unroll
        for (int q = 0; q < kItems; ++q) n += r[q] == 0;
        int total, at = found + half_scan(n, sums, total);
#pragma unroll
        for (int q = 0; q < kItems; ++q)
            if (r[q] == 0) {
                if (at < want) p.list[at] = (int)(base + t * kItems + q);
                ++at;
            }
        found += total;
        // both halves have what they want
        if (__syncthreads_and(found >= want)) break;
    }
    return min(found, want);
}

__device__ __forceinline__ Pool pool_of(const Cache &c, const PagesWs &y, int half) {
    return half == 0 ? Pool{c.k_table, c.k_ref, y.list[0], y.list2[0], y.cnt[0], c.nk}
                     : Pool{c.v_table, c.v_ref, y.list[1], y.list2[1], y.cnt[1], c.nv};
}

// Where the wanted pages of item i begin in the half's list: exclusive sums of cnt[0 .. n)
// in place. Returns the sum, INT_MAX where it is larger (65,535 sequences of 2^18 slots pass an int; no
// pool has as many pages, so the places are not used then). Every thread of the CTA calls it.
__device__ __forceinline__ int scan_counts(int *cnt, int n, int *sums) {
    const int t = threadIdx.x & (kHalf - 1);
    long long run = 0;
    for (int base = 0; base < n; base += kHalf) {
        const int v = base + t < n ? cnt[base + t] : 0;
        int total;
        const long long at = run + half_scan(v, sums, total);
        if (base + t < n) cnt[base + t] = (int)at;
        run += total;
    }
    __syncthreads();
    return run < INT_MAX ? (int)run : INT_MAX;
}

// ---------------------------------------------------------------- reserve
__global__ void __launch_bounds__(kPlanThr) reserve_kernel(const Cache c, const int *extra, const PagesWs y) {
    __shared__ int sums[32];
    const int half = threadIdx.x / kHalf, warp = (threadIdx.x & (kHalf - 1)) >> 5, lane = threadIdx.x & 31;
    const Pool p = pool_of(c, y, half);
    bool bad = false;
    auto upto = [&](int s) {
        const int n = c.lens[s], e = extra[s];
        const long long t = ((long long)n + e + c.page - 1) >> c.page_shift;
        if (n < 0 || e < 0 || t > c.max_pages) {
            bad = true;
            return 0;
        }
        return (int)t;
    };
    for (int s = warp; s < c.seqs; s += kHalfWarps) {
        const int up = upto(s);
        int n = 0;
        for (int i = lane; i < up; i += 32) n += p.table[(size_t)s * c.max_pages + i] < 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        if (lane == 0) p.cnt[s] = n;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) report_status(y.status, kStatusCapacity);
        return;
    }
    const int want = scan_counts(p.cnt, c.seqs, sums);
    const int found = find_free(p, want, max(c.nk, c.nv), sums);
    if (__syncthreads_or(found < want)) {
        if (threadIdx.x == 0) report_status(y.status, kStatusCapacity);
        return;
    }
    for (int s = warp; s < c.seqs; s += kHalfWarps) {
        const int up = upto(s);
        int at = p.cnt[s];
        for (int i0 = 0; i0 < up; i0 += 32) {
            const int i = i0 + lane;
            int *e = p.table + (size_t)s * c.max_pages + i;
            const bool w = i < up && *e < 0;
            const unsigned m = __ballot_sync(0xffffffffu, w);
            if (w) {
                const int id = p.list[at + __popc(m & ((1u << lane) - 1u))];
                *e = id;
                p.ref[id] = 1;
            }
            at += __popc(m);
        }
    }
}

// ---------------------------------------------------------------- fork
template <int N>
__global__ void __launch_bounds__(kPlanThr) fork_plan_kernel(const Cache c, const Rows<N> src, const Rows<N> dst,
                                                             const PagesWs y) {
    __shared__ int sums[32];
    const int tid = threadIdx.x, half = tid / kHalf, t = tid & (kHalf - 1), warp = t >> 5, lane = tid & 31;
    const Pool p = pool_of(c, y, half);
    const int pairs = src.n;
    bool bad = false;
    grid_begin();  // the first of the call: nothing to wait for
    if (tid == 0) y.go[0] = 0;
    for (int i = warp; i < pairs; i += kHalfWarps) {
        const int n = c.lens[src.row[i]];
        const long long used = ((long long)n + c.page - 1) >> c.page_shift;
        if (n < 0 || used > c.max_pages || c.lens[dst.row[i]] != 0) {
            bad = true;
            continue;
        }
        // the source's pages lie in the pool, the destination has none
        for (int s = lane; s < (int)used; s += 32)
            bad |= (unsigned)p.table[(size_t)src.row[i] * c.max_pages + s] >= (unsigned)p.pages;
        for (int s = lane; s < c.max_pages; s += 32)
            bad |= p.table[(size_t)dst.row[i] * c.max_pages + s] >= 0;
        if (lane == 0) p.cnt[i] = half == 0 ? (int)used : (n & (c.page - 1)) != 0;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) report_status(y.status, kStatusCache);
        return;
    }
    const int want = scan_counts(p.cnt, pairs, sums);
    const int found = find_free(p, want, max(c.nk, c.nv), sums);
    if (__syncthreads_or(found < want)) {
        if (tid == 0) report_status(y.status, kStatusCapacity);
        return;
    }
    for (int i = warp; i < pairs; i += kHalfWarps) {
        const int n = c.lens[src.row[i]], used = (n + c.page - 1) >> c.page_shift, full = n >> c.page_shift;
        const int *from = p.table + (size_t)src.row[i] * c.max_pages;
        int *to = p.table + (size_t)dst.row[i] * c.max_pages;
        for (int s = lane; s < used; s += 32) {
            if (half == 1 && s < full) {  // shared
                const int id = from[s];
                to[s] = id;
                atomicAdd(p.ref + id, 1);
            } else {
                const int id = p.list[p.cnt[i] + (half == 0 ? s : 0)];
                to[s] = id;
                p.ref[id] = 1;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += kPlanThr) c.lens[dst.row[i]] = c.lens[src.row[i]];
    if (tid == 0) y.go[0] = 1;
}

// n 16-byte words by the CTA's threads, eight loads in flight per thread
__device__ __forceinline__ void copy16(uint4 *dst, const uint4 *src, int n) {
    const int nt = blockDim.x;
    int i = threadIdx.x;
    for (; i + 7 * nt < n; i += 8 * nt) {
        uint4 r[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] = __ldcs(src + i + q * nt);
#pragma unroll
        for (int q = 0; q < 8; ++q) __stcs(dst + i + q * nt, r[q]);
    }
    for (; i < n; i += nt) __stcs(dst + i, __ldcs(src + i));
}

// The first `rows` token rows of every head of a page; row_bytes = d * element size.
__device__ __forceinline__ void copy_page(char *dst, const char *src, int heads, int page, int rows,
                                          int row_bytes) {
    // in 16-byte words: a page's bytes may pass an int, its words do not (65,535 heads of 256 rows)
    const int per = rows * row_bytes / 16, pitch = page * row_bytes / 16;
    if (rows == page) {
        copy16(reinterpret_cast<uint4 *>(dst), reinterpret_cast<const uint4 *>(src), heads * pitch);
        return;
    }
    for (int i = threadIdx.x; i < heads * per; i += blockDim.x) {
        const int h = i / per, e = h * pitch + i % per;
        __stcs(reinterpret_cast<uint4 *>(dst) + e, __ldcs(reinterpret_cast<const uint4 *>(src) + e));
    }
}

// grid (slots, pairs): the key page (and its gate sums) of a slot, or the value page that is
// not shared
template <int N>
__global__ void __launch_bounds__(256) fork_copy_kernel(const Cache c, const Rows<N> src, const Rows<N> dst,
                                                        int row_bytes, const PagesWs y) {
    grid_begin();
    grid_wait();
    if (y.go[0] == 0) return;
    const int s = blockIdx.x, i = blockIdx.y;
    const int n = c.lens[src.row[i]], rows = min(c.page, n - (s << c.page_shift));
    if (rows <= 0) return;
    const size_t from = (size_t)src.row[i] * c.max_pages + s, to = (size_t)dst.row[i] * c.max_pages + s;
    const size_t page_bytes = (size_t)c.Hkv * c.page * row_bytes;
    const int ks = c.k_table[from], kd = c.k_table[to];
    copy_page(static_cast<char *>(c.k_pages) + kd * page_bytes,
              static_cast<const char *>(c.k_pages) + ks * page_bytes, c.Hkv, c.page, rows, row_bytes);
    if (c.g_pages != nullptr) {
        const size_t per = (size_t)c.Hq * c.page;
        for (int e = threadIdx.x; e < c.Hq * rows; e += blockDim.x) {
            const size_t at = (size_t)(e / rows) * c.page + e % rows;
            c.g_pages[kd * per + at] = c.g_pages[ks * per + at];
        }
    }
    if (rows < c.page)
        copy_page(static_cast<char *>(c.v_pages) + c.v_table[to] * page_bytes,
                  static_cast<const char *>(c.v_pages) + c.v_table[from] * page_bytes, c.Hkv, c.page,
                  rows, row_bytes);
}

// ---------------------------------------------------------------- free
// grid (rows, pools)
template <int N>
__global__ void __launch_bounds__(256) free_kernel(const Cache c, const Rows<N> rows, const PagesWs y) {
    const int s = rows.row[blockIdx.x];
    const Pool p = pool_of(c, y, blockIdx.y);
    for (int i = threadIdx.x; i < c.max_pages; i += 256) {
        int *e = p.table + (size_t)s * c.max_pages + i;
        const int id = *e;
        if (id == -1) continue;
        *e = -1;
        if ((unsigned)id < (unsigned)p.pages) atomicSub(p.ref + id, 1);
        else report_status(y.status, kStatusCache);
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) c.lens[s] = 0;
}

// ---------------------------------------------------------------- compact
// With L live pages, the k-th free page below L takes the k-th live page at or above L: the
// two sets are as large as each other and disjoint, so the copies may run in any order.
__global__ void __launch_bounds__(kPlanThr) compact_plan_kernel(const Cache c, const PagesWs y) {
    __shared__ int sums[32];
    const int tid = threadIdx.x, half = tid / kHalf, t = tid & (kHalf - 1);
    const Pool p = pool_of(c, y, half);
    const int most = max(c.nk, c.nv);
    int live = 0;
    grid_begin();  // the first of the call: nothing to wait for
    for (long long base = 0; base < most; base += kHalf * kItems) {
        int r[kItems];
        load_counts(p, base + t * kItems, r);
#pragma unroll
        for (int q = 0; q < kItems; ++q) live += r[q] > 0;
    }
    int L;
    half_scan(live, sums, L);
    int holes = 0, moves = 0;
    for (long long base = 0; base < most; base += kHalf * kItems) {
        const long long i0 = base + t * kItems;
        int r[kItems], nh = 0, nm = 0;
        load_counts(p, i0, r);
#pragma unroll
        for (int q = 0; q < kItems; ++q) {
            nh += i0 + q < L && r[q] <= 0;
            nm += i0 + q >= L && r[q] > 0;
        }
        int th, tm;
        int ah = holes + half_scan(nh, sums, th), am = moves + half_scan(nm, sums, tm);
#pragma unroll
        for (int q = 0; q < kItems; ++q) {
            if (i0 + q < L && r[q] <= 0) p.list[ah++] = (int)i0 + q;
            if (i0 + q >= L && r[q] > 0) p.list2[am++] = (int)i0 + q;
            if (i0 + q >= L && i0 + q < p.pages && r[q] <= 0) y.to[half][i0 + q] = -1;
        }
        holes += th;
        moves += tm;
    }
    __syncthreads();
    for (int k = t; k < moves; k += kHalf) {
        const int from = p.list2[k], to = p.list[k];
        y.to[half][from] = to;
        p.ref[to] = p.ref[from];
        p.ref[from] = 0;
    }
    if (t == 0) {
        y.go[1 + half] = moves;
        y.go[3 + half] = L;
    }
}

// CTAs below `table_ctas` renumber the tables' entries, the others move pages.
__global__ void __launch_bounds__(256) compact_move_kernel(const Cache c, int row_bytes, int table_ctas,
                                                           const PagesWs y) {
    grid_begin();
    grid_wait();
    if ((int)blockIdx.x < table_ctas) {
        const long long per = (long long)c.seqs * c.max_pages;
        for (long long i = blockIdx.x * 256ll + threadIdx.x; i < 2 * per; i += table_ctas * 256ll) {
            const int pool = i >= per;
            int *e = (pool ? c.v_table : c.k_table) + (i - pool * per);
            const int id = *e, L = y.go[3 + pool], pages = pool ? c.nv : c.nk;
            if (id < L) continue;
            // an entry outside the pool, or of a page that nobody holds, stays as it is
            const int to = id < pages ? y.to[pool][id] : -1;
            if (to < 0) {
                report_status(y.status, kStatusCache);
                continue;
            }
            *e = to;
        }
        return;
    }
    const size_t page_bytes = (size_t)c.Hkv * c.page * row_bytes;
    const int nk = y.go[1], nv = y.go[2], step = gridDim.x - table_ctas;
    for (int i = blockIdx.x - table_ctas; i < nk + nv; i += step) {
        const int pool = i >= nk, k = i - pool * nk;
        const size_t from = y.list2[pool][k], to = y.list[pool][k];
        char *base = static_cast<char *>(pool ? c.v_pages : c.k_pages);
        copy16(reinterpret_cast<uint4 *>(base + to * page_bytes),
               reinterpret_cast<const uint4 *>(base + from * page_bytes), (int)(page_bytes / 16));
        if (!pool && c.g_pages != nullptr) {
            const size_t per = (size_t)c.Hq * c.page;  // a multiple of 16 floats
            copy16(reinterpret_cast<uint4 *>(c.g_pages + to * per),
                   reinterpret_cast<const uint4 *>(c.g_pages + from * per), (int)(per / 4));
        }
    }
}

PagesWs pages_ws(const Cache &c, void *ws, size_t *total) {
    PagesWs y;
    char *base = static_cast<char *>(ws);
    size_t off = 256;
    auto take = [&](size_t n) {
        int *p = reinterpret_cast<int *>(base + off);
        off = align256(off + n * 4);
        return p;
    };
    y.status = reinterpret_cast<uint32_t *>(base);
    y.go = take(8);
    const int rows = c.seqs > kMaxRows ? c.seqs : kMaxRows;
    for (int p = 0; p < 2; ++p) {
        const int n = p ? c.nv : c.nk;
        y.list[p] = take(n);
        y.list2[p] = take(n);
        y.to[p] = take(n);
        y.cnt[p] = take(rows);
    }
    if (total) *total = off;
    return y;
}

}  // namespace

size_t pages_ws_bytes(const Cache &c) {
    size_t n;
    pages_ws(c, nullptr, &n);
    return n;
}

cudaError_t launch_reserve(const Cache &c, const int *extra, void *ws, cudaStream_t stream) {
    reserve_kernel<<<1, kPlanThr, 0, stream>>>(c, extra, pages_ws(c, ws, nullptr));
    return cudaGetLastError();
}

// A list as a smaller one: most calls name a few rows, and a launch copies its parameters.
constexpr int kFewRows = 32;
Rows<kFewRows> few_rows(const Rows<kMaxRows> &a) {
    Rows<kFewRows> r;
    r.n = a.n;
    for (int i = 0; i < a.n; ++i) r.row[i] = a.row[i];
    return r;
}

template <int N>
cudaError_t launch_fork_n(const Cache &c, const Rows<N> &src, const Rows<N> &dst, int row_bytes, const PagesWs &y,
                          cudaStream_t stream) {
    const cudaError_t e = launch(fork_plan_kernel<N>, dim3(1), kPlanThr, 0, stream, true, c, src, dst, y);
    if (e != cudaSuccess) return e;
    return launch(fork_copy_kernel<N>, dim3(c.max_pages, src.n), 256, 0, stream, false, c, src, dst, row_bytes, y);
}

cudaError_t launch_fork(const Cache &c, const Rows<kMaxRows> &src, const Rows<kMaxRows> &dst, int row_bytes,
                        void *ws, cudaStream_t stream) {
    const PagesWs y = pages_ws(c, ws, nullptr);
    return src.n <= kFewRows ? launch_fork_n(c, few_rows(src), few_rows(dst), row_bytes, y, stream)
                             : launch_fork_n(c, src, dst, row_bytes, y, stream);
}

cudaError_t launch_free(const Cache &c, const Rows<kMaxRows> &rows, void *ws, cudaStream_t stream) {
    const PagesWs y = pages_ws(c, ws, nullptr);
    return rows.n <= kFewRows
               ? launch(free_kernel<kFewRows>, dim3(rows.n, 2), 256, 0, stream, true, c, few_rows(rows), y)
               : launch(free_kernel<kMaxRows>, dim3(rows.n, 2), 256, 0, stream, true, c, rows, y);
}

cudaError_t launch_compact(const Cache &c, int row_bytes, void *ws, cudaStream_t stream) {
    const PagesWs y = pages_ws(c, ws, nullptr);
    const cudaError_t e = launch(compact_plan_kernel, dim3(1), kPlanThr, 0, stream, true, c, y);
    if (e != cudaSuccess) return e;
    const long long entries = 2ll * c.seqs * c.max_pages;
    const int table_ctas = (int)(entries / 2048 < 64 ? entries / 2048 + 1 : 64);
    // at most min(nk, nv) + ... / 2 pages move; eight CTAs per SM keep the copies in flight
    const long long most = ((long long)c.nk + c.nv) / 2 + 1;
    const int movers = (int)(most < 8 * 152 ? most : 8 * 152);
    return launch(compact_move_kernel, dim3(table_ctas + movers), 256, 0, stream, false, c, row_bytes, table_ctas, y);
}

}  // namespace paged
}  // namespace path
