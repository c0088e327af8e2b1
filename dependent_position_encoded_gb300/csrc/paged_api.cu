// Host side of the paged-cache entry points of include/path_attn.h: argument checks
// (synchronous, before any launch), workspace sizes and kernel dispatch.
#include <climits>
#include <cmath>

#include "paged_tc.cuh"
#include "paged_pages.cuh"
#include "path_attn.h"

namespace path {
namespace paged {
bool decode_takes(int G);
size_t decode_part_bytes(const Cache &c, int d);
template <typename A>
cudaError_t launch_decode(const A &a, int d, bool bf16, const Behind *behind, float *part, cudaStream_t stream);
size_t f32_ws_bytes(const Cache &c, int N, int d, bool fox);
template <typename A>
cudaError_t launch_f32(A a, int d, void *ws, float *carry, float *gates, void *pws, cudaStream_t stream);
size_t tc_ws_bytes(const Cache &c, int N, int max_chunk, int d, bool fox);
template <typename A>
cudaError_t launch_tc(const A &a, int d, void *ws, float *carry, float *gates, void *pws, uint64_t limit_ns,
                      cudaStream_t stream);
size_t prefix_tc_bytes(const StepMore &a, int d);
size_t prefix_f32_bytes(const StepMore &a, int d);
cudaError_t launch_prefix_tc(const StepMore &a, int d, float *carry, float *gates, const TcWs *y, void *ws, bool first,
                             uint64_t limit_ns, Behind *behind, cudaStream_t stream);
cudaError_t launch_prefix_f32(StepMore &a, int d, float *carry, float *gates, float *y_qt, float *y_gq, void *ws,
                              bool first, cudaStream_t stream);
size_t pages_ws_bytes(const Cache &c);
cudaError_t launch_reserve(const Cache &c, const int *extra, void *ws, cudaStream_t stream);
cudaError_t launch_fork(const Cache &c, const Rows<kMaxRows> &src, const Rows<kMaxRows> &dst, int row_bytes,
                        void *ws, cudaStream_t stream);
cudaError_t launch_free(const Cache &c, const Rows<kMaxRows> &rows, void *ws, cudaStream_t stream);
cudaError_t launch_compact(const Cache &c, int row_bytes, void *ws, cudaStream_t stream);
cudaError_t launch_trim(const Cache &c, const Rows<kMaxRows> &rows, int window, int sinks, void *ws,
                        cudaStream_t stream);
}  // namespace paged
}  // namespace path

namespace {

using namespace path;
using paged::Cache;
using Rows = paged::Rows<paged::kMaxRows>;

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // bounded waits of the tensor-core kernels

bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Sizes of a cache (no pointer is looked at): the workspace sizes go by them alone.
path_status check_cache_sizes(const path_paged_cache *p) {
    if (p == nullptr) return PATH_ERR_NULL;
    if (p->dtype != PATH_F32 && p->dtype != PATH_BF16) return PATH_ERR_DTYPE;
    if (p->d != 64 && p->d != 128) return PATH_ERR_SHAPE;
    if (p->page < 16 || p->page > 256 || (p->page & (p->page - 1)) != 0) return PATH_ERR_SHAPE;
    if (p->seqs < 0 || p->seqs > PATH_MAX_HEADS || p->max_pages < 0 || p->num_k_pages < 0 ||
        p->num_v_pages < 0 || p->Hq < 1 || p->Hkv < 1 || p->Hq > PATH_MAX_HEADS || p->Hq % p->Hkv != 0)
        return PATH_ERR_SHAPE;
    if ((long long)p->max_pages * p->page > PATH_MAX_LEN) return PATH_ERR_SHAPE;
    // a page of one head is one index of the kernels' tensor maps
    if ((long long)p->num_k_pages * p->Hkv > INT_MAX || (long long)p->num_v_pages * p->Hkv > INT_MAX)
        return PATH_ERR_SHAPE;
    return PATH_OK;
}

path_status check_cache(const path_paged_cache *p, bool counts) {
    const path_status st = check_cache_sizes(p);
    if (st != PATH_OK) return st;
    const void *need[] = {p->k_pages, p->v_pages, p->k_table, p->v_table, p->lens};
    for (const void *x : need)
        if (x == nullptr) return PATH_ERR_NULL;
    if (counts && (!p->k_ref || !p->v_ref)) return PATH_ERR_NULL;
    if (!is_aligned(p->k_pages, 16) || !is_aligned(p->v_pages, 16) || !is_aligned(p->g_pages, 16) ||
        !is_aligned(p->k_table, 4) || !is_aligned(p->v_table, 4) || !is_aligned(p->lens, 4) ||
        (counts && (!is_aligned(p->k_ref, 16) || !is_aligned(p->v_ref, 16))))
        return PATH_ERR_ALIGN;
    return PATH_OK;
}

Cache to_cache(const path_paged_cache *p) {
    int shift = 0;
    while ((1 << shift) < p->page) ++shift;
    return Cache{p->k_pages, p->v_pages, p->g_pages, p->k_table, p->v_table, p->k_ref, p->v_ref,
                 p->lens, p->seqs, p->max_pages, p->page, shift, p->num_k_pages, p->num_v_pages,
                 p->Hq, p->Hkv, p->Hq / p->Hkv};
}

int elt_size(const path_paged_cache *p) { return p->dtype == PATH_BF16 ? 2 : 4; }

path_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PATH_OK : PATH_ERR_CUDA; }

path_status check_workspace(const void *ws, size_t bytes, size_t need) {
    if (ws == nullptr) return PATH_ERR_NULL;
    if (!is_aligned(ws, 256)) return PATH_ERR_ALIGN;
    return bytes < need ? PATH_ERR_WORKSPACE : PATH_OK;
}

// The step's kernels. One token per sequence at most, and a few query heads per key head: the
// one-pass kernel on the CUDA cores scores them from registers and needs one launch more for
// the join, where the block kernels need three; but it does G products per key on the CUDA cores.
// The rule goes by what the tables can hold (query heads x positions of the whole cache, or of the
// window and the sinks), not by the lengths, which only the device knows. Measured for bf16 plain steps
// with tables that are full (us, one-pass / block kernels; 8 key heads, 1 to 8 sequences):
//                        2^14       2^15       2^16       2^17       2^18       2^19       2^20      2^22
//   G = 1, d =  64    12.5/18.5  18.6/22.6  29.7/28.5  26.0/28.7  32.8/35.5  44.3/47.5  78/73   248/210
//              128    14.5/23.1  22.6/28.8  34.9/34.4  34.4/38.5  61.4/57.6  79.6/79.9  141/128 468/412
//   G = 2, d =  64    10.3/16.5  14.4/18.5  20.6/20.9  23.1/23.3  30.7/28.7  30.9/30.9  53/49   159/114
//              128    12.3/21.9  16.3/24.2  24.7/28.7  28.7/30.8  41.5/37.4  53.4/52.6  95/80   298/214
//   G = 4, d =  64    10.4/16.5  10.4/18.1  14.5/18.6  18.5/20.6  29.2/24.6  32.6/26.9  43/31   122/73
//              128    12.3/21.3  12.4/22.6  16.5/24.8  22.4/26.8  34.9/32.3  43.1/36.9  72/53   223/127
// with gates
//   G = 1, d =  64    16.4/22.6  26.3/24.7  39.0/32.4  32.8/32.9  34.8/43.1  38.5/55.4  72/82   242/235
//              128    22.6/26.7  35.0/32.9  53.4/39.0  47.2/44.0  53.6/67.0  81.3/92.4  147/142 503/457
//   G = 2, d =  64    14.9/20.5  19.6/22.5  29.6/24.7  34.3/28.8  41.2/34.9  37.5/39.0  60/59   203/132
//              128    22.6/24.8  26.8/27.0  43.1/32.8  48.3/35.0  61.8/45.1  62.3/63.9  127/94  413/245
//   G = 4, d =  64    16.5/20.5  18.5/22.0  22.6/22.6  28.7/24.6  43.3/29.0  43.0/33.0  47/39   143/88
//              128    24.6/24.7  26.5/26.5  30.8/28.8  43.2/30.8  64.5/38.1  67.3/42.1  79/61   294/151
// With gates and G = 1 the one-pass kernel leaves most value rows unread and takes every size: behind at
// 2^16 and from 2^21 on, ahead between. Its weights are fp32 where the block kernels' are bf16, so
// equal times go to it. fp32 inputs have no tensor path: one-pass wherever it takes G.
// A window counts by what it can have in sight. Behind prefixes the positions are those of the tables still,
// which are as wide as the prefix, while these kernels go over the sequences' own tails, and each tail is
// cut into splits by that width. Whole steps there, with 8 key heads, pages of 64 and one prefix (us,
// one-pass / block kernels; sequences, prefix, tails):
//                         4, 2,000, 64  32, 2,000, 64  4, 16,384, 64  32, 16,384, 64  8, 16,384, 2,000
//   gates, G = 1, d =  64    30.2/32.4      37.1/39.7      49.9/39.5       63.0/51.7        68.5/48.3
//                    128     37.6/36.5      50.0/47.6      54.8/47.4       86.6/70.2       105.5/79.9
// so from tables of 2^19 on the rule takes the slower side there. Without gates, G = 1, it takes the one-pass
// kernels in the first column alone (25.0/27.6, 27.3/31.5).
bool one_pass(const Cache &c, long long seen, int max_chunk, bool bf16, bool fox) {
    if (max_chunk != 1 || !paged::decode_takes(c.G)) return false;
    if (!bf16 || (fox && c.G == 1)) return true;
    const long long positions = seen * c.seqs * c.Hq;
    return positions <= (c.G == 1 ? 1 << 19 : fox ? 1 << 15 : 1 << 17);
}

// seen: the positions that a sequence's step can have in sight (most_seen)
size_t step_ws_bytes(const path_paged_cache *p, long long seen, int N, int max_chunk, bool fox) {
    const Cache c = to_cache(p);
    if (one_pass(c, seen, max_chunk, p->dtype == PATH_BF16, fox))
        return 256 + align256(paged::decode_part_bytes(c, p->d));
    if (p->dtype == PATH_BF16) return paged::tc_ws_bytes(c, N, max_chunk, p->d, fox);
    return paged::f32_ws_bytes(c, N, p->d, fox);
}

path_status check_step_sizes(const path_paged_cache *p, int N, int max_chunk) {
    if (N < 0 || N > PATH_MAX_LEN || max_chunk < 0 || max_chunk > N) return PATH_ERR_SHAPE;
    if (N > 0 && max_chunk < 1) return PATH_ERR_SHAPE;
    // rows of a key head (query heads that share it, taken together) are counted in an int
    if ((long long)N * (p->Hq / p->Hkv) > INT_MAX / 2) return PATH_ERR_SHAPE;
    return PATH_OK;
}

// (token, head) strides of a (N, H, inner) tensor: packed where st is null. The stride of an axis
// of one element says nothing.
paged::Stride stride_of(const int64_t *st, int N, int H, int inner) {
    if (!st) return paged::Stride{(long long)H * inner, inner};
    return paged::Stride{N > 1 ? st[0] : 0, H > 1 ? st[1] : 0};
}
bool bad_stride(const paged::Stride &s, int bytes) {
    return s.tok < 0 || s.head < 0 || s.tok * bytes % 16 != 0 || s.head * bytes % 16 != 0;
}

// What a step has beyond its own tokens and cache: a window (0: none) and its sinks, or prefixes.
struct More {
    int window = 0, sinks = 0;
    const int *prefix_of = nullptr;
    float *carry = nullptr, *gates = nullptr;
};

size_t prefix_bytes(const path_paged_cache *p, int N) {
    paged::StepMore a{};
    a.c = to_cache(p);
    a.N = N;
    return p->dtype == PATH_BF16 ? paged::prefix_tc_bytes(a, p->d) : paged::prefix_f32_bytes(a, p->d);
}

path_status extend(const path_paged_cache *p, const void *q, const void *k, const void *v,
                   const void *w, const float *beta, const float *log_f, bool fox,
                   const int *cu_tokens, int N, int max_chunk, float scale, void *out,
                   const path_paged_strides *strides, void *ws, size_t ws_bytes, void *stream,
                   const More &more = More{}) {
    path_status st = check_cache_sizes(p);
    if (st == PATH_OK) st = check_step_sizes(p, N, max_chunk);
    if (st != PATH_OK) return st;
    if (!std::isfinite(scale)) return PATH_ERR_ARG;
    if (p->seqs == 0 || N == 0) return PATH_OK;
    if ((st = check_cache(p, false)) != PATH_OK) return st;
    if (!q || !k || !v || !w || !beta || !out || !cu_tokens || (fox && (!log_f || !p->g_pages)))
        return PATH_ERR_NULL;
    const void *al16[] = {q, k, v, w, out};
    for (const void *x : al16)
        if (!is_aligned(x, 16)) return PATH_ERR_ALIGN;
    if (!is_aligned(beta, 4) || !is_aligned(log_f, 4) || !is_aligned(cu_tokens, 4)) return PATH_ERR_ALIGN;
    const paged::Stride sq = stride_of(strides ? strides->q : nullptr, N, p->Hq, p->d),
                        sk = stride_of(strides ? strides->k : nullptr, N, p->Hkv, p->d),
                        sv = stride_of(strides ? strides->v : nullptr, N, p->Hkv, p->d),
                        sw = stride_of(strides ? strides->w : nullptr, N, p->Hkv, p->d),
                        sb = stride_of(strides ? strides->beta : nullptr, N, p->Hkv, 1),
                        sf = stride_of(strides ? strides->log_f : nullptr, N, p->Hq, 1),
                        so = stride_of(strides ? strides->out : nullptr, N, p->Hq, p->d);
    for (const paged::Stride &r : {sq, sk, sv, sw, so})
        if (bad_stride(r, elt_size(p))) return PATH_ERR_ALIGN;
    for (const paged::Stride &r : {sb, sf})
        if (r.tok < 0 || r.head < 0) return PATH_ERR_ALIGN;
    const Cache c = to_cache(p);
    const paged::Step plain{c, q, k, v, w, beta, fox ? log_f : nullptr, out,
                            sq, sk, sv, sw, sb, sf, so,
                            cu_tokens, N, max_chunk, scale * kLog2e, static_cast<uint32_t *>(ws)};
    paged::StepMore a{plain, more.window, more.sinks, more.prefix_of, nullptr, nullptr, nullptr,
                      paged::prefix_one_rows(p->d, max_chunk, fox), false};
    const bool bf16 = p->dtype == PATH_BF16, prefix = more.prefix_of != nullptr, is_plain = !prefix && more.window == 0;
    const long long seen = paged::most_seen(a);
    const size_t own = align256(step_ws_bytes(p, seen, N, max_chunk, fox));
    if ((st = check_workspace(ws, ws_bytes, own + (prefix ? prefix_bytes(p, N) : 0))) != PATH_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char *const pws = static_cast<char *>(ws) + own;
    if (one_pass(c, seen, max_chunk, bf16, fox)) {
        float *const part = reinterpret_cast<float *>(static_cast<char *>(ws) + 256);
        if (is_plain) return cuda_status(paged::launch_decode(plain, p->d, bf16, nullptr, part, s));
        cudaError_t e = cudaSuccess;
        paged::Behind behind = {};
        if (prefix)
            e = bf16 ? paged::launch_prefix_tc(a, p->d, more.carry, more.gates, nullptr, pws, true, kWaitLimitNs,
                                               &behind, s)
                     : paged::launch_prefix_f32(a, p->d, more.carry, more.gates, nullptr, nullptr, pws, true, s);
        return cuda_status(e == cudaSuccess ? paged::launch_decode(a, p->d, bf16, &behind, part, s) : e);
    }
    if (bf16)
        return cuda_status(is_plain
                               ? paged::launch_tc(plain, p->d, ws, nullptr, nullptr, nullptr, kWaitLimitNs, s)
                               : paged::launch_tc(a, p->d, ws, more.carry, more.gates, pws, kWaitLimitNs, s));
    return cuda_status(is_plain ? paged::launch_f32(plain, p->d, ws, nullptr, nullptr, nullptr, s)
                                : paged::launch_f32(a, p->d, ws, more.carry, more.gates, pws, s));
}

path_status check_window(int window, int sinks) {
    return window < 1 || window > PATH_MAX_LEN || sinks < 0 || sinks > PATH_MAX_LEN ? PATH_ERR_ARG : PATH_OK;
}

path_status window_extend(const path_paged_cache *p, const void *q, const void *k, const void *v,
                          const void *w, const float *beta, const float *log_f, bool fox,
                          const int *cu_tokens, int N, int max_chunk, int window, int sinks,
                          float scale, void *out, const path_paged_strides *strides, void *ws,
                          size_t ws_bytes, void *stream) {
    // with longer chunks the new tokens would hide one another
    if (check_window(window, sinks) != PATH_OK || max_chunk > window) return PATH_ERR_ARG;
    return extend(p, q, k, v, w, beta, log_f, fox, cu_tokens, N, max_chunk, scale, out, strides, ws,
                  ws_bytes, stream, More{window, sinks});
}

path_status prefix_extend(const path_paged_cache *p, const void *q, const void *k, const void *v,
                          const void *w, const float *beta, const float *log_f, bool fox,
                          const int *cu_tokens, int N, int max_chunk, const int *prefix_of, float *carry,
                          float *gate_carry, float scale, void *out, const path_paged_strides *strides,
                          void *ws, size_t ws_bytes, void *stream) {
    path_status st = check_cache_sizes(p);
    if (st == PATH_OK) st = check_step_sizes(p, N, max_chunk);
    if (st != PATH_OK) return st;
    if (!std::isfinite(scale)) return PATH_ERR_ARG;
    if (p->seqs == 0 || N == 0) return PATH_OK;
    if (!prefix_of || !carry || (fox && !gate_carry)) return PATH_ERR_NULL;
    if (!is_aligned(prefix_of, 4) || !is_aligned(carry, 16) || !is_aligned(gate_carry, 4)) return PATH_ERR_ALIGN;
    return extend(p, q, k, v, w, beta, log_f, fox, cu_tokens, N, max_chunk, scale, out, strides, ws,
                  ws_bytes, stream, More{0, 0, prefix_of, carry, fox ? gate_carry : nullptr});
}

// A list of sequence rows from the host: in range, none twice.
path_status check_rows(const path_paged_cache *p, const int *rows, int n, Rows *out) {
    if (n < 0 || n > paged::kMaxRows) return PATH_ERR_SHAPE;
    if (n > 0 && rows == nullptr) return PATH_ERR_NULL;
    out->n = n;
    for (int i = 0; i < n; ++i) {
        if (rows[i] < 0 || rows[i] >= p->seqs) return PATH_ERR_ARG;
        out->row[i] = rows[i];
    }
    return PATH_OK;
}

bool repeats(const Rows &a) {
    for (int i = 0; i < a.n; ++i)
        for (int j = 0; j < i; ++j)
            if (a.row[i] == a.row[j]) return true;
    return false;
}

path_status trim(const path_paged_cache *p, const Rows &rows, int window, int sinks, void *ws, size_t ws_bytes,
                 void *stream) {
    path_status st = check_cache(p, true);
    if (st != PATH_OK) return st;
    const Cache c = to_cache(p);
    if ((st = check_workspace(ws, ws_bytes, paged::pages_ws_bytes(c))) != PATH_OK) return st;
    if (c.max_pages == 0) return PATH_OK;
    return cuda_status(paged::launch_trim(c, rows, window, sinks, ws, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t path_paged_workspace_bytes(const path_paged_cache *cache, int num_tokens, int max_chunk) {
    if (check_cache_sizes(cache) != PATH_OK || check_step_sizes(cache, num_tokens, max_chunk) != PATH_OK)
        return 0;
    const Cache c = to_cache(cache);
    size_t n = paged::pages_ws_bytes(c);
    if (num_tokens > 0) {
        // with and without gates, a step of single tokens too, so that a workspace for chunks serves the
        // steps between them, and one that sees the least, which may go with the one-pass kernels where
        // the others do not
        for (int chunk : {max_chunk, 1})
            for (bool fox : {false, true})
                for (long long seen : {(long long)c.max_pages << c.page_shift, 0ll}) {
                    const size_t s = step_ws_bytes(cache, seen, num_tokens, chunk, fox);
                    n = s > n ? s : n;
                }
    }
    return n;
}

path_status path_paged_extend(const path_paged_cache *cache, const void *q, const void *k,
                              const void *v, const void *w, const float *beta,
                              const int *cu_tokens, int num_tokens, int max_chunk, float scale,
                              void *out, const path_paged_strides *strides, void *ws,
                              size_t ws_bytes, void *stream) {
    return extend(cache, q, k, v, w, beta, nullptr, false, cu_tokens, num_tokens, max_chunk, scale,
                  out, strides, ws, ws_bytes, stream);
}

path_status path_fox_paged_extend(const path_paged_cache *cache, const void *q, const void *k,
                                  const void *v, const void *w, const float *beta,
                                  const float *log_f, const int *cu_tokens, int num_tokens,
                                  int max_chunk, float scale, void *out,
                                  const path_paged_strides *strides, void *ws, size_t ws_bytes,
                                  void *stream) {
    return extend(cache, q, k, v, w, beta, log_f, true, cu_tokens, num_tokens, max_chunk, scale, out,
                  strides, ws, ws_bytes, stream);
}

path_status path_paged_window_extend(const path_paged_cache *cache, const void *q, const void *k,
                                     const void *v, const void *w, const float *beta,
                                     const int *cu_tokens, int num_tokens, int max_chunk, int window,
                                     int sinks, float scale, void *out,
                                     const path_paged_strides *strides, void *ws, size_t ws_bytes,
                                     void *stream) {
    return window_extend(cache, q, k, v, w, beta, nullptr, false, cu_tokens, num_tokens, max_chunk,
                         window, sinks, scale, out, strides, ws, ws_bytes, stream);
}

path_status path_fox_paged_window_extend(const path_paged_cache *cache, const void *q, const void *k,
                                         const void *v, const void *w, const float *beta,
                                         const float *log_f, const int *cu_tokens, int num_tokens,
                                         int max_chunk, int window, int sinks, float scale, void *out,
                                         const path_paged_strides *strides, void *ws, size_t ws_bytes,
                                         void *stream) {
    return window_extend(cache, q, k, v, w, beta, log_f, true, cu_tokens, num_tokens, max_chunk, window,
                         sinks, scale, out, strides, ws, ws_bytes, stream);
}

size_t path_paged_prefix_workspace_bytes(const path_paged_cache *cache, int num_tokens, int max_chunk) {
    const size_t n = path_paged_workspace_bytes(cache, num_tokens, max_chunk);
    return n == 0 || num_tokens == 0 ? n : align256(n) + prefix_bytes(cache, num_tokens);
}

path_status path_paged_prefix_extend(const path_paged_cache *cache, const void *q, const void *k,
                                     const void *v, const void *w, const float *beta,
                                     const int *cu_tokens, int num_tokens, int max_chunk,
                                     const int *prefix_of, float *carry, float scale, void *out,
                                     const path_paged_strides *strides, void *ws, size_t ws_bytes,
                                     void *stream) {
    return prefix_extend(cache, q, k, v, w, beta, nullptr, false, cu_tokens, num_tokens, max_chunk,
                         prefix_of, carry, nullptr, scale, out, strides, ws, ws_bytes, stream);
}

path_status path_fox_paged_prefix_extend(const path_paged_cache *cache, const void *q, const void *k,
                                         const void *v, const void *w, const float *beta,
                                         const float *log_f, const int *cu_tokens, int num_tokens,
                                         int max_chunk, const int *prefix_of, float *carry,
                                         float *gate_carry, float scale, void *out,
                                         const path_paged_strides *strides, void *ws, size_t ws_bytes,
                                         void *stream) {
    return prefix_extend(cache, q, k, v, w, beta, log_f, true, cu_tokens, num_tokens, max_chunk,
                         prefix_of, carry, gate_carry, scale, out, strides, ws, ws_bytes, stream);
}

path_status path_paged_trim(const path_paged_cache *cache, int window, int sinks, void *ws,
                            size_t ws_bytes, void *stream) {
    path_status st = check_cache_sizes(cache);
    if (st != PATH_OK) return st;
    if ((st = check_window(window, sinks)) != PATH_OK) return st;
    if (cache->seqs == 0) return PATH_OK;
    return trim(cache, Rows{}, window, sinks, ws, ws_bytes, stream);
}

path_status path_paged_trim_rows(const path_paged_cache *cache, const int *rows, int num_rows, int window,
                                 int sinks, void *ws, size_t ws_bytes, void *stream) {
    path_status st = check_cache_sizes(cache);
    if (st != PATH_OK) return st;
    Rows a;
    if ((st = check_rows(cache, rows, num_rows, &a)) != PATH_OK) return st;
    if (repeats(a)) return PATH_ERR_ARG;
    if ((st = check_window(window, sinks)) != PATH_OK) return st;
    if (num_rows == 0) return PATH_OK;
    return trim(cache, a, window, sinks, ws, ws_bytes, stream);
}

path_status path_paged_reserve(const path_paged_cache *cache, const int *extra, void *ws,
                               size_t ws_bytes, void *stream) {
    path_status st = check_cache_sizes(cache);
    if (st != PATH_OK) return st;
    if (cache->seqs == 0) return PATH_OK;
    if ((st = check_cache(cache, true)) != PATH_OK) return st;
    if (extra == nullptr) return PATH_ERR_NULL;
    if (!is_aligned(extra, 4)) return PATH_ERR_ALIGN;
    const Cache c = to_cache(cache);
    if ((st = check_workspace(ws, ws_bytes, paged::pages_ws_bytes(c))) != PATH_OK) return st;
    return cuda_status(paged::launch_reserve(c, extra, ws, static_cast<cudaStream_t>(stream)));
}

path_status path_paged_fork(const path_paged_cache *cache, const int *src, const int *dst, int pairs,
                            void *ws, size_t ws_bytes, void *stream) {
    path_status st = check_cache_sizes(cache);
    if (st != PATH_OK) return st;
    Rows a, b;
    if ((st = check_rows(cache, src, pairs, &a)) != PATH_OK) return st;
    if ((st = check_rows(cache, dst, pairs, &b)) != PATH_OK) return st;
    if (repeats(b)) return PATH_ERR_ARG;
    for (int i = 0; i < pairs; ++i)
        for (int j = 0; j < pairs; ++j)
            if (a.row[i] == b.row[j]) return PATH_ERR_ARG;
    if (pairs == 0) return PATH_OK;
    if ((st = check_cache(cache, true)) != PATH_OK) return st;
    const Cache c = to_cache(cache);
    if ((st = check_workspace(ws, ws_bytes, paged::pages_ws_bytes(c))) != PATH_OK) return st;
    if (c.max_pages == 0) return PATH_OK;
    return cuda_status(paged::launch_fork(c, a, b, cache->d * elt_size(cache), ws,
                                          static_cast<cudaStream_t>(stream)));
}

path_status path_paged_free(const path_paged_cache *cache, const int *rows, int num_rows, void *ws,
                            size_t ws_bytes, void *stream) {
    path_status st = check_cache_sizes(cache);
    if (st != PATH_OK) return st;
    Rows a;
    if ((st = check_rows(cache, rows, num_rows, &a)) != PATH_OK) return st;
    if (repeats(a)) return PATH_ERR_ARG;
    if (num_rows == 0) return PATH_OK;
    if ((st = check_cache(cache, true)) != PATH_OK) return st;
    const Cache c = to_cache(cache);
    if ((st = check_workspace(ws, ws_bytes, paged::pages_ws_bytes(c))) != PATH_OK) return st;
    return cuda_status(paged::launch_free(c, a, ws, static_cast<cudaStream_t>(stream)));
}

path_status path_paged_compact(const path_paged_cache *cache, void *ws, size_t ws_bytes,
                               void *stream) {
    path_status st = check_cache_sizes(cache);
    if (st != PATH_OK) return st;
    if (cache->num_k_pages == 0 && cache->num_v_pages == 0) return PATH_OK;
    if ((st = check_cache(cache, true)) != PATH_OK) return st;
    const Cache c = to_cache(cache);
    if ((st = check_workspace(ws, ws_bytes, paged::pages_ws_bytes(c))) != PATH_OK) return st;
    return cuda_status(paged::launch_compact(c, cache->d * elt_size(cache), ws,
                                             static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
