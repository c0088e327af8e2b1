// One new token per sequence over a paged cache (PaTH and PaTH-FoX), in one pass over it;
// sequences with none or several are left out.
//
// The new token's transition H = I - beta w w^T is applied to every cached key in place,
// k <- k - beta (w . k) w, and the attention of the token's query runs over the updated keys
// (review "거리에서 경로로, PaTH Attention" §9; technical summary "技術要約: PaTH Attention"
// §3 "推論"). Each cached key is read once, written once and its value read once:
// 6 d bytes per key in bf16, which is what bounds the step where the cache is large; the small
// ones that come here (paged_api.cu) are bound by latency: 6 + 7 us for both kernels at one
// sequence of 300, 8 heads, D = 64, bf16.
//
// Split-K layout: grid (splits, key heads, sequences); a CTA takes `chunk` cached positions of
// one key head, whose page numbers it stages (and checks) in shared memory. A key row is
// D * sizeof(T) bytes over TPK = D / E lanes with one 16-byte load each. The G query heads
// that share the key head are scored on the same registers, so the row is read once for all
// of them. The logit is formed from the updated key before its rounding. A second kernel
// appends the new key and value, scores it and merges the splits.
//
// PaTH-FoX: the gate sum of every cached key (per query head) is advanced in place, and a
// value row is read only if one of its G logits comes within 2^-64 of the head's own token
// (a lower bound of the row's maximum): 2^22 keys below that move the sum by less than
// 2^-42 of itself.
#include "paged.cuh"

namespace path {
namespace paged {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunk = 1024;
constexpr int kMaxIds = kMaxChunk / 16 + 1;

template <typename T> struct Row;
template <> struct Row<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_bf16x2(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};
template <> struct Row<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};

template <typename T>
__device__ __forceinline__ uint4 ld16(const T *p) {
    return *reinterpret_cast<const uint4 *>(p);
}

template <typename T, bool FOX, int D, int G>
__global__ void __launch_bounds__(kThreads, G == 4 ? 2 : 3)
paged_decode_split(const Step a, int chunk, int nsplit, float *__restrict__ part) {
    constexpr int E = Row<T>::E;
    constexpr int TPK = D / E;     // lanes per key
    constexpr int KPW = 32 / TPK;  // keys per warp pass
    constexpr int SLOTS = kWarps * KPW;
    __shared__ int kid[kMaxIds], vid[kMaxIds];
    __shared__ float sm_m[G][SLOTS], sm_l[G][SLOTS];
    __shared__ float sm_o[G][SLOTS][D];

    const int sp = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    grid_begin();  // the first of the call: nothing to wait for
    const Seq s = seq_of(a, b);
    const int j0 = sp * chunk, j1 = min(j0 + chunk, s.n);
    if (s.T != 1 || j0 >= j1) return;  // the merge skips the splits past n
    const int shift = a.c.page_shift, pmask = a.c.page - 1;
    const int slot0 = j0 >> shift;
    for (int i = threadIdx.x; i <= ((j1 - 1) >> shift) - slot0; i += kThreads) {
        kid[i] = page_of(a, a.c.k_table, b, slot0 + i, a.c.nk);
        vid[i] = page_of(a, a.c.v_table, b, slot0 + i, a.c.nv);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = lane / TPK, e0 = (lane % TPK) * E;
    float qv[G][E], wv[E], thr[G], m[G], l[G], o[G][E];
    Row<T>::unpack(ld16(static_cast<const T *>(a.w) + s.first * a.sw.tok + h * a.sw.head + e0), wv);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        Row<T>::unpack(ld16(static_cast<const T *>(a.q) + s.first * a.sq.tok +
                            (h * G + g) * a.sq.head + e0), qv[g]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            qv[g][e] *= a.scale_log2;
            o[g][e] = 0.f;
        }
        m[g] = -INFINITY;
        l[g] = 0.f;
        thr[g] = -INFINITY;
    }
    const float bt = __ldg(a.beta + s.first * a.sb.tok + h * a.sb.head);
    float lf[G];
    if (FOX) {
        float kn[E];
        Row<T>::unpack(ld16(static_cast<const T *>(a.k) + s.first * a.sk.tok + h * a.sk.head + e0), kn);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float dn = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) dn = fmaf(qv[g][e], kn[e], dn);
#pragma unroll
            for (int off = 1; off < TPK; off <<= 1) dn += __shfl_xor_sync(0xffffffffu, dn, off);
            thr[g] = dn - 64.f;
            lf[g] = __ldg(a.log_f + s.first * a.sf.tok + (h * G + g) * a.sf.head);
        }
    }
    __syncthreads();

    T *const kp = static_cast<T *>(a.c.k_pages);
    const T *const vp = static_cast<const T *>(a.c.v_pages);
    // row of position j in its page, or -1 past the split's end or where the page is bad
    auto place = [&](int j, const int *ids) -> long long {
        if (j >= j1) return -1;
        const int id = ids[(j >> shift) - slot0];
        if (id < 0) return -1;
        return ((((long long)id * a.c.Hkv + h) << shift) + (j & pmask)) * D;
    };
    // One cached key whose row is in registers: update it in place, score it for the G heads
    // and fold it into their softmax. Every lane calls it (the shuffles are warp-wide).
    auto key_math = [&](long long row, long long vrow, const float (&gj)[G], float (&kv)[E],
                        uint4 vraw) {
        float dw = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) dw = fmaf(wv[e], kv[e], dw);
#pragma unroll
        for (int off = 1; off < TPK; off <<= 1) dw += __shfl_xor_sync(0xffffffffu, dw, off);
        const float al = bt * dw;
#pragma unroll
        for (int e = 0; e < E; ++e) kv[e] = fmaf(-al, wv[e], kv[e]);
        if (row >= 0) *reinterpret_cast<uint4 *>(kp + row + e0) = Row<T>::pack(kv);
        float x[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float dq = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) dq = fmaf(qv[g][e], kv[e], dq);
#pragma unroll
            for (int off = 1; off < TPK; off <<= 1) dq += __shfl_xor_sync(0xffffffffu, dq, off);
            x[g] = FOX ? fmaf(gj[g], kLog2e, dq) : dq;
        }
        if (row < 0 || vrow < 0) return;
        if (FOX) {
            bool any = false;
#pragma unroll
            for (int g = 0; g < G; ++g) any |= !(x[g] < thr[g]);  // NaN counts
            if (!any) return;  // the same for all lanes of the key
            vraw = ld16(vp + vrow + e0);
        }
        float vv[E];
        Row<T>::unpack(vraw, vv);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (x[g] > m[g]) {  // the same for all lanes of the key
                const float sc = exp2f(m[g] - x[g]);  // 0 while m is -inf
                m[g] = x[g];
                l[g] *= sc;
#pragma unroll
                for (int e = 0; e < E; ++e) o[g][e] *= sc;
            }
            const float p = (x[g] == -INFINITY) ? 0.f : exp2f(x[g] - m[g]);
            l[g] += p;
#pragma unroll
            for (int e = 0; e < E; ++e) o[g][e] = fmaf(p, vv[e], o[g][e]);
        }
    };
    const float zero[G] = {};
    if (!FOX) {
        // two passes' key and value rows are loaded together, so each warp keeps twice the
        // bytes in flight
        constexpr int kStride = kWarps * KPW;
        for (int jb = j0 + warp * KPW; jb < j1; jb += 2 * kStride) {
            uint4 kr[2], vr[2];
            long long rk[2], rv[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int j = jb + p * kStride + grp;
                rk[p] = place(j, kid);
                rv[p] = place(j, vid);
                kr[p] = rk[p] >= 0 ? ld16(kp + rk[p] + e0) : make_uint4(0u, 0u, 0u, 0u);
                vr[p] = rv[p] >= 0 ? ld16(vp + rv[p] + e0) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float kv[E];
                Row<T>::unpack(kr[p], kv);
                key_math(rk[p], rv[p], zero, kv, vr[p]);
            }
        }
    } else {
        // each warp owns runs of 32 positions: lane i advances the gate sums of position
        // run + i, and the key's lanes fetch them by shuffle
        constexpr int kPasses = 32 / KPW;
        constexpr int kBatch = kPasses < 4 ? kPasses : 4;
        for (int rb = j0 + warp * 32; rb < j1; rb += kWarps * 32) {
            const int jl = rb + lane;
            float gl[G];
            const int id = jl < j1 ? kid[(jl >> shift) - slot0] : -1;
            float *gp = a.c.g_pages + ((((long long)id * a.c.Hq + h * G)) << shift) + (jl & pmask);
#pragma unroll
            for (int g = 0; g < G; ++g) gl[g] = id >= 0 ? gp[(long long)g << shift] : 0.f;
#pragma unroll
            for (int b0 = 0; b0 < kPasses; b0 += kBatch) {
                uint4 kr[kBatch];
                long long rk[kBatch];
#pragma unroll
                for (int p = 0; p < kBatch; ++p) {
                    rk[p] = place(rb + (b0 + p) * KPW + grp, kid);
                    kr[p] = rk[p] >= 0 ? ld16(kp + rk[p] + e0) : make_uint4(0u, 0u, 0u, 0u);
                }
                if (b0 == 0) {
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        gl[g] += lf[g];
                        if (id >= 0) gp[(long long)g << shift] = gl[g];
                    }
                }
#pragma unroll
                for (int p = 0; p < kBatch; ++p) {
                    const int src = (b0 + p) * KPW + grp;
                    float gj[G], kv[E];
#pragma unroll
                    for (int g = 0; g < G; ++g) gj[g] = __shfl_sync(0xffffffffu, gl[g], src);
                    Row<T>::unpack(kr[p], kv);
                    key_math(rk[p], place(rb + src, vid), gj, kv, make_uint4(0u, 0u, 0u, 0u));
                }
            }
        }
    }
    // merge the CTA's SLOTS partial states of every head
    const int slot = warp * KPW + grp;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        if ((lane % TPK) == 0) {
            sm_m[g][slot] = m[g];
            sm_l[g][slot] = l[g];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[g][slot][e0 + e] = o[g][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += kThreads) {
        const int g = i / D, c = i % D;
        float M = -INFINITY, Ls = 0.f, Oc = 0.f;
        for (int t = 0; t < SLOTS; ++t) M = fmaxf(M, sm_m[g][t]);
        // a slot without a key has a sum of 0 under its -inf, one whose keys are NaN a sum of NaN
        const float use = M == -INFINITY ? 0.f : M;
        for (int t = 0; t < SLOTS; ++t) {
            const float f = exp2f(sm_m[g][t] - use);
            Ls += sm_l[g][t] * f;
            Oc += sm_o[g][t][c] * f;
        }
        float *dst = part + (((size_t)b * a.c.Hq + h * G + g) * nsplit + sp) * (D + 2);
        dst[2 + c] = Oc;
        if (c == 0) {
            dst[0] = M;
            dst[1] = Ls;
        }
    }
}

// D threads per (query head, sequence): score the new token, merge the splits and, for the
// first query head of a key head, append the new key and value.
template <typename T, bool FOX, int D>
__global__ void __launch_bounds__(D)
paged_decode_merge(const Step a, int chunk, int nsplit, const float *part) {
    __shared__ float red[D / 32];
    const int hq = blockIdx.x, b = blockIdx.y, c = threadIdx.x;
    grid_begin();
    const Seq s = seq_of(a, b);
    if (s.T != 1) {
        grid_wait();
        return;
    }
    // the new token's own part, while the splits still run (they read nothing from position n on)
    const int h = hq / a.c.G;
    const T kt = static_cast<const T *>(a.k)[s.first * a.sk.tok + h * a.sk.head + c];
    const T vt = static_cast<const T *>(a.v)[s.first * a.sv.tok + h * a.sv.head + c];
    const int slot = s.n >> a.c.page_shift, off = s.n & (a.c.page - 1);
    const int kid = page_of(a, a.c.k_table, b, slot, a.c.nk);
    if (hq % a.c.G == 0) {
        const int vid = page_of(a, a.c.v_table, b, slot, a.c.nv);
        if (kid >= 0)
            static_cast<T *>(a.c.k_pages)[((((size_t)kid * a.c.Hkv + h) << a.c.page_shift) + off) * D + c] = kt;
        if (vid >= 0)
            static_cast<T *>(a.c.v_pages)[((((size_t)vid * a.c.Hkv + h) << a.c.page_shift) + off) * D + c] = vt;
    }
    if (FOX && c == 0 && kid >= 0)
        a.c.g_pages[(((size_t)kid * a.c.Hq + hq) << a.c.page_shift) + off] = 0.f;
    float d = Elt<T>::to_f(static_cast<const T *>(a.q)[s.first * a.sq.tok + hq * a.sq.head + c]) *
              Elt<T>::to_f(kt);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((c & 31) == 0) red[c >> 5] = d;
    __syncthreads();
    float dsum = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) dsum += red[i];
    const float x_new = dsum * a.scale_log2;
    grid_wait();
    const int used = (s.n + chunk - 1) / chunk;
    const float *pp = part + ((size_t)b * a.c.Hq + hq) * nsplit * (D + 2);
    float M = x_new;
    for (int i = 0; i < used; ++i) M = fmaxf(M, pp[i * (D + 2)]);
    const float f_new = exp2f(x_new - M);
    float Ls = f_new, Oc = f_new * Elt<T>::to_f(vt);
    for (int i = 0; i < used; ++i) {
        const float f = exp2f(pp[i * (D + 2)] - M);  // M is at least the new token's logit
        Ls += pp[i * (D + 2) + 1] * f;
        Oc += pp[i * (D + 2) + 2 + c] * f;
    }
    static_cast<T *>(a.out)[s.first * a.so.tok + hq * a.so.head + c] = Elt<T>::from_f(Oc / Ls);
}

template <typename T, bool FOX, int D, int G>
cudaError_t launch_g(const Step &a, int chunk, int nsplit, float *part, cudaStream_t stream) {
    if (nsplit > 0) {
        const cudaError_t e = launch(paged_decode_split<T, FOX, D, G>, dim3(nsplit, a.c.Hkv, a.c.seqs), kThreads, 0,
                                     stream, true, a, chunk, nsplit, part);
        if (e != cudaSuccess) return e;
    }
    return launch(paged_decode_merge<T, FOX, D>, dim3(a.c.Hq, a.c.seqs), D, 0, stream, nsplit == 0, a, chunk, nsplit,
                  part);
}

template <typename T, bool FOX, int D>
cudaError_t launch_d(const Step &a, int chunk, int nsplit, float *part, cudaStream_t stream) {
    switch (a.c.G) {
        case 1: return launch_g<T, FOX, D, 1>(a, chunk, nsplit, part, stream);
        case 2: return launch_g<T, FOX, D, 2>(a, chunk, nsplit, part, stream);
        default: return launch_g<T, FOX, D, 4>(a, chunk, nsplit, part, stream);
    }
}

}  // namespace

// The query heads per key head that the kernel scores on one read of the key.
bool decode_takes(int G) { return G == 1 || G == 2 || G == 4; }

// Cached positions per CTA: the most that still gives every SM six CTAs (two rounds of the
// three that are resident), so that short caches spread over the machine and long ones have
// few parts to merge.
int decode_chunk(const Cache &c) {
    const long long cap = (long long)c.max_pages << c.page_shift;
    int chunk = kMaxChunk;
    while (chunk > 64 && (cap + chunk - 1) / chunk * c.Hkv * c.seqs < 6 * 152) chunk >>= 1;
    return chunk;
}

size_t decode_part_bytes(const Cache &c, int d) {
    const long long cap = (long long)c.max_pages << c.page_shift;
    const int chunk = decode_chunk(c);
    return (size_t)c.seqs * c.Hq * ((cap + chunk - 1) / chunk) * (d + 2) * sizeof(float);
}

cudaError_t launch_decode(const Step &a, int d, bool bf16, float *part, cudaStream_t stream) {
    const long long cap = (long long)a.c.max_pages << a.c.page_shift;
    const int chunk = decode_chunk(a.c), nsplit = (int)((cap + chunk - 1) / chunk);
    const bool fox = a.log_f != nullptr;
    auto pick = [&](auto t) {
        using T = decltype(t);
        if (d == 64)
            return fox ? launch_d<T, true, 64>(a, chunk, nsplit, part, stream)
                       : launch_d<T, false, 64>(a, chunk, nsplit, part, stream);
        return fox ? launch_d<T, true, 128>(a, chunk, nsplit, part, stream)
                   : launch_d<T, false, 128>(a, chunk, nsplit, part, stream);
    };
    return bf16 ? pick(__nv_bfloat16{}) : pick(0.f);
}

}  // namespace paged
}  // namespace path
