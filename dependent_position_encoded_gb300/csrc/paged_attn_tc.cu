// The attention of a step over a paged cache, bf16, on tcgen05 tensor cores: the carried
// queries against the cached keys (`cached`, with the keys' in-place update where a sequence
// has one tile of rows) and, for chunks of several blocks, the walk of the queries through
// the chunk's earlier blocks (`scan`).
//
// A cached key keeps the basis of the last cached token, so its logit with query i of the
// chunk is k_j . q~_i, q~_i = H_1 ... H_i q_i: one pass of ordinary softmax attention over
// the pages, for whatever number of new tokens. Only the keys' own update needs the chunk's
// product, K <- K + K (P - I) (review "거리에서 경로로, PaTH Attention" §9; technical summary
// "技術要約: PaTH Attention" §3 "推論").
#include "paged_tc.cuh"

namespace path {
namespace paged {

namespace {

using bf = __nv_bfloat16;

__host__ __device__ constexpr uint32_t idesc_b16(int M, int N, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// tcgen05.mma with the A operand in tensor memory (lane = row, a 32-bit column = two
// consecutive K elements, eight columns per K = 16 instruction).
__device__ __forceinline__ void umma_tA(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Bounded wait: after limit_ns it records PATH_ERR_TIMEOUT and raises the CTA's abort flag,
// which ends every other wait of the CTA.
struct Wait {
    volatile uint32_t *abort;
    uint32_t *status;
    uint64_t limit_ns;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = cycles_now(), lim = ns_to_cycles(limit_ns);
        for (;;) {
            if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
            if (*abort) return false;
            if (cycles_now() - t0 > lim) {
                report_status(status, kStatusTimeout);
                *abort = 1u;
                return false;
            }
        }
    }
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, (*this)(bar, parity)) != 0;
    }
};

__device__ __forceinline__ void tld32(uint32_t taddr, float *x) {
    uint32_t u[32];
    tmem_ld32(taddr, u);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(u[j]);
}

__device__ __forceinline__ void tst32(uint32_t taddr, const float *x) {
    uint32_t u[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(x[j]);
    tmem_st32(taddr, u);
}

// multiplies N fp32 columns of the thread's row by f
template <int N>
__device__ __forceinline__ void tmem_scale(uint32_t taddr, float f) {
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
        uint32_t u[32];
        tmem_ld32(taddr + c, u);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * f);
        tmem_st32(taddr + c, u);
    }
    tmem_st_wait();
}

constexpr float kRescale = 8.f;  // the running maximum may lag by 2^8 before O is rescaled

// ================================================================ cached keys
// A CTA takes NT tiles of 128 rows of one sequence and key head and a range of key tiles of
// 128 positions. Keys and values stream through one ring of shared-memory slots (TMA, one
// box per page; a slot holds 128 rows of D bf16 in 128-byte-swizzled atoms of 64 columns).
// Per key tile and row tile: S = X K^T (N = 128) into TMEM, softmax by the 128 threads of a
// warpgroup, one row each, which write the weights as bf16 over S, and O += P V with the
// weights as the A operand in TMEM. With NT = 2 the two row tiles share every slot and take
// turns on the tensor core, one in its softmax while the other multiplies.
//
// NT = 1 is for sequences whose rows fit one tile (a few tokens: bound by the cache's bytes)
// and updates the keys too: a second MMA forms K (P - I) with the loaded keys as the A operand
// (P - I split into two bf16 parts), and the second warpgroup adds it to the keys in shared
// memory and stores them back, so each key is read once and written once.
//
// Warps: 0-3 softmax of tile 0; 4-7 softmax of tile 1 (NT = 2) or the keys' update (NT = 1); 8
// allocates TMEM and issues the MMAs; 9 streams the pages.
// Positions past the sequence's n and those on bad pages: the streaming warp zeroes their rows
// after the copy, and the softmax masks them.
template <int NT, int D>
struct CachedSmem {
    static constexpr uint32_t tile = 128 * D * 2, atom = 128 * 128;
    static constexpr uint32_t X = 0, M = X + NT * tile, mbytes = NT == 1 ? 2 * D * D * 2 : 0;
    // slots: what fits beside; for NT = 1 and D = 64 so that two CTAs share an SM
    static constexpr int slots = NT == 1 ? 4 : (D == 64 ? 8 : 5);
    static constexpr uint32_t ring = M + mbytes, bars = ring + slots * tile;
    static constexpr int FULL = 0, EMPTY = slots, XF = 2 * slots, SF = XF + 1, PR = SF + 2, FIN = PR + 2,
                         DF = FIN + 1, DE = DF + 1, TMP = DE + 1, count = TMP + 1;
    static constexpr uint32_t bytes = bars + count * 8 + 16, alloc = bytes + 1024;
};

template <int NT, int D>
struct CachedTmem {
    static constexpr uint32_t S = 0, O = 128, per_tile = 256, Dt = O + D;  // Dt: NT = 1 only
    static constexpr uint32_t cols = NT == 2 ? 512 : (D == 64 ? 256 : 512);
};

constexpr int kCachedThr = 320;

template <int NT, int D, bool FOX>
__global__ void __launch_bounds__(kCachedThr, (NT == 1 && D == 64) ? 2 : 1)
tc_cached_kernel(const Step a, const TcWs y, const __grid_constant__ CUtensorMap tm_x,
                 const __grid_constant__ CUtensorMap tm_m, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, uint64_t limit_ns) {
    using L = CachedSmem<NT, D>;
    using C = CachedTmem<NT, D>;
    constexpr int NA = D / 64, NS = L::slots;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const sm = smem_raw + (base - raw);
    auto bar = [&](int i) { return base + L::bars + 8u * (uint32_t)i; };
    uint32_t *const tslot = reinterpret_cast<uint32_t *>(sm + L::bars + 8 * L::count);
    volatile uint32_t *const abort_f = tslot + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y, G = a.c.G;
    int b, ti;
    Seq s;
    if (!tile_of(a, blockIdx.x, 128 * NT, b, ti, s)) return;
    const int rows_all = s.T * G;
    if ((rows_all <= 128) != (NT == 1)) return;  // the other kernel's
    const int ktiles = (s.n + 127) / 128, per = (ktiles + y.splits - 1) / y.splits;
    const int k0 = blockIdx.z * per, k1 = min(ktiles, k0 + per), steps = k1 - k0;
    if (steps <= 0) return;
    const int row0 = 128 * NT * ti;                                // first row within the sequence
    const bool two = NT == 2 && row0 + 128 < rows_all;             // the second tile has rows
    const Wait wait{abort_f, a.status, limit_ns};

    if (tid == 0) {
        *abort_f = 0u;
        for (int i = 0; i < L::count; ++i) mbar_init(bar(i), (i >= L::PR && i < L::FIN) || i == L::DE ? 4u : 1u);
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tslot), C::cols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    auto slot_at = [&](int u) { return base + L::ring + (uint32_t)(u % NS) * L::tile; };
    // Ring use u: keys of step j at u = 2 j, its values at u = 2 j + 1.

    if (warp == 9) {
        // ============================================================ pages into the ring
        int issued = 0;
        bool ok = true;
        if (lane == 0) {
            const int xr = (int)((long long)s.first * G) + row0;
            mbar_arrive_expect_tx(bar(L::XF), (two ? 2 : 1) * L::tile + L::mbytes);
            for (int t = 0; t < (two ? 2 : 1); ++t)
                for (int x = 0; x < NA; ++x)
                    tma_load_3d(base + L::X + t * L::tile + x * L::atom, &tm_x, bar(L::XF), 64 * x, xr + 128 * t, h);
            if (NT == 1)
                for (int p = 0; p < 2; ++p)
                    for (int x = 0; x < NA; ++x)
                        tma_load_3d(base + L::M + (uint32_t)(p * NA + x) * D * 128, &tm_m, bar(L::XF), 64 * x, 0,
                                    (b * a.c.Hkv + h) * 2 + p);
        }
        const int page = a.c.page, box_shift = min(a.c.page_shift, 7), box = 1 << box_shift, nbox = 128 / box;
        uint32_t tmp_phase = 0;
        for (int u = 0; ok && u < 2 * steps; ++u) {
            const bool keys = (u & 1) == 0;
            const int pos0 = (k0 + (u >> 1)) * 128;
            // lane i < nbox: the page of box i, -1 past the end or where it is bad
            int id = -1;
            if (lane < nbox && pos0 + lane * box < s.n)
                id = page_of(a, keys ? a.c.k_table : a.c.v_table, b, (pos0 + lane * box) >> a.c.page_shift,
                             keys ? a.c.nk : a.c.nv);
            const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
            const int valid = min(128, s.n - pos0);
            const bool whole = valid == 128 && have == (1u << nbox) - 1u;
            if (u >= NS && !(ok = wait.warp(bar(L::EMPTY + u % NS), ((u / NS) & 1) ^ 1))) break;
            const uint32_t dst = slot_at(u);
            const uint32_t full = bar(L::FULL + u % NS), target = whole ? full : bar(L::TMP);
            if (lane == 0) mbar_arrive_expect_tx(target, (uint32_t)__popc(have) * box * D * 2);
            __syncwarp();
            if (id >= 0)
#pragma unroll
                for (int x = 0; x < NA; ++x)
                    tma_load_3d(dst + x * L::atom + lane * box * 128, keys ? &tm_k : &tm_v, target, 64 * x,
                                (pos0 + lane * box) & (page - 1), id * a.c.Hkv + h);
            if (!whole) {
                // zero the rows that hold no cached position, then hand the slot on
                if (!(ok = wait.warp(bar(L::TMP), tmp_phase))) break;
                tmp_phase ^= 1;
                uint8_t *const rowp = sm + (dst - base);
                for (int r = 0; r < 128; ++r) {
                    if (r < valid && ((have >> (r >> box_shift)) & 1u)) continue;
                    if (lane < NA * 8)
                        *reinterpret_cast<uint4 *>(rowp + (lane >> 3) * L::atom + r * 128 + (lane & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
            }
            issued = u + 1;
        }
        // on an abort: no copy may land after the CTA is gone
        if (!ok) {
            const int from = issued > NS ? issued - NS : 0;
            for (int u = from; u < issued; ++u) mbar_wait(bar(L::FULL + u % NS), (u / NS) & 1, limit_ns);
            mbar_wait(bar(L::XF), 0, limit_ns);
        }
    } else if (warp == 8) {
        // ============================================================ MMA issue
        if (lane == 0) {
            constexpr uint32_t ID_S = idesc_b16(128, 128, false), ID_O = idesc_b16(128, D, true);
            bool ok = wait(bar(L::XF), 0);
            auto issue_s = [&](int t, int j) {
                const uint32_t kb = slot_at(2 * j);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16(tmem + C::per_tile * t + C::S,
                              sdesc_sw128(base + L::X + t * L::tile + (kk >> 2) * L::atom, 16, 1024) + 2 * (kk & 3),
                              sdesc_sw128(kb + (kk >> 2) * L::atom, 16, 1024) + 2 * (kk & 3), ID_S, kk > 0);
                umma_commit(bar(L::SF + t));
            };
            auto issue_pv = [&](int t, int j) {
                const uint64_t v = sdesc_sw128(slot_at(2 * j + 1), L::atom, 1024);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    umma_tA(tmem + C::per_tile * t + C::O, tmem + C::per_tile * t + C::S + 8 * kk, v + 128 * kk, ID_O,
                            j > 0 || kk > 0);
            };
            auto keys_ready = [&](int j) { return wait(bar(L::FULL + (2 * j) % NS), ((2 * j) / NS) & 1); };
            auto issue_update = [&](int j) {  // K (P - I): the keys are the A operand
                if (j > 0 && !wait(bar(L::DE), (j - 1) & 1)) return false;
                tc_fence_after();
                const uint32_t kb = slot_at(2 * j);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint64_t m = sdesc_sw128(base + L::M + p * NA * D * 128, D * 128, 1024);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_bf16(tmem + C::Dt, sdesc_sw128(kb + (kk >> 2) * L::atom, 16, 1024) + 2 * (kk & 3),
                                  m + 128 * kk, ID_O, p > 0 || kk > 0);
                }
                umma_commit(bar(L::DF));
                return true;
            };
            if (ok && (ok = keys_ready(0))) {
                tc_fence_after();
                issue_s(0, 0);
                if (two) issue_s(1, 0);
                if (NT == 1) ok = issue_update(0);
                else umma_commit(bar(L::EMPTY + 0));
            }
            for (int j = 0; ok && j < steps; ++j) {
                const int vs = (2 * j + 1) % NS;
                if (!(ok = wait(bar(L::FULL + vs), ((2 * j + 1) / NS) & 1))) break;
                for (int t = 0; t < (two ? 2 : 1); ++t) {
                    if (!(ok = wait(bar(L::PR + t), j & 1))) break;
                    tc_fence_after();
                    issue_pv(t, j);
                    if (t == (two ? 1 : 0)) umma_commit(bar(L::EMPTY + vs));
                    if (j + 1 < steps) {
                        if (t == 0 && !(ok = keys_ready(j + 1))) break;
                        if (t == 0) tc_fence_after();
                        issue_s(t, j + 1);
                    }
                }
                if (!ok) break;
                if (j + 1 < steps) {
                    if (NT == 1) ok = issue_update(j + 1);
                    else umma_commit(bar(L::EMPTY + (2 * j + 2) % NS));
                }
            }
            umma_commit(bar(L::FIN));
            mbar_wait(bar(L::FIN), 0, limit_ns);
        }
    } else if (NT == 1 && warp >= 4) {
        // ============================================================ the keys' update
        const int r = tid - 128;
        const uint32_t tm = tmem + ((uint32_t)(32 * (warp - 4)) << 16) + C::Dt;
        const int page = a.c.page, box_shift = min(a.c.page_shift, 7), box = 1 << box_shift, nbox = 128 / box;
        bool ok = true;
        for (int j = 0; j < steps; ++j) {
            const int pos0 = (k0 + j) * 128;
            int id = -1;
            if (lane < nbox && pos0 + lane * box < s.n)
                id = page_of(a, a.c.k_table, b, (pos0 + lane * box) >> a.c.page_shift, a.c.nk);
            const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
            const bool whole = pos0 + 128 <= s.n && have == (1u << nbox) - 1u;
            const int mine = __shfl_sync(0xffffffffu, id, r >> box_shift);
            if (!(ok = wait.warp(bar(L::DF), j & 1))) break;
            tc_fence_after();
            uint8_t *const kt = sm + (slot_at(2 * j) - base);
            bf *const dst = mine >= 0 && pos0 + r < s.n
                                ? static_cast<bf *>(a.c.k_pages) +
                                      ((((size_t)mine * a.c.Hkv + h) << a.c.page_shift) + ((pos0 + r) & (page - 1))) * D
                                : nullptr;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float x[32];
                tld32(tm + c, x);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint4 *at = reinterpret_cast<uint4 *>(kt + (c >> 6) * L::atom + sw128_offset(r, ((c & 63) >> 3) + q));
                    const uint4 k4 = *at;
                    const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 k2 = unpack_bf16x2(w[e]);
                        o[e] = pack_bf16x2(k2.x + x[8 * q + 2 * e], k2.y + x[8 * q + 2 * e + 1]);
                    }
                    const uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
                    if (whole) *at = v;
                    else if (dst) *reinterpret_cast<uint4 *>(dst + c + 8 * q) = v;
                }
            }
            tc_fence_before();
            mbar_arrive_warp(bar(L::DE));
            fence_proxy_async_smem();
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (warp == 4) {
                if (whole && id >= 0) {
#pragma unroll
                    for (int x = 0; x < NA; ++x)
                        tma_store_3d(&tm_k, slot_at(2 * j) + x * L::atom + lane * box * 128, 64 * x,
                                     (pos0 + lane * box) & (page - 1), id * a.c.Hkv + h);
                    bulk_wait_read();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::EMPTY + (2 * j) % NS));
            }
        }
        if (warp == 4) bulk_wait_all();
    } else if (warp < 4 || two) {
        // ============================================================ softmax
        const int t = warp >> 2, r = 128 * t + (tid & 127);
        const uint32_t tm = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C::per_tile * t;
        const bool live = row0 + r < rows_all;
        const bool warp_live = row0 + 128 * t + 32 * (warp & 3) < rows_all;
        const size_t row = (size_t)h * y.R + (size_t)s.first * G + row0 + r;
        const int hq = h * G + (live ? (row0 + r) % G : 0);
        const float gq = FOX && live ? y.gq[row] * kLog2e : 0.f;
        constexpr bool kTwice = NT == 1 || FOX;
        const int page = a.c.page, box_shift = min(a.c.page_shift, 7), box = 1 << box_shift, nbox = 128 / box;
        float m_run = -INFINITY, l_run = 0.f;
        bool ok = true;
        for (int j = 0; j < steps; ++j) {
            const int pos0 = (k0 + j) * 128;
            int id = -1;
            bool good = false;
            if (lane < nbox && pos0 + lane * box < s.n) {
                const int sl = (pos0 + lane * box) >> a.c.page_shift;
                const size_t at = (size_t)b * a.c.max_pages + sl;
                id = __ldg(a.c.k_table + at);
                good = (unsigned)id < (unsigned)a.c.nk && (unsigned)__ldg(a.c.v_table + at) < (unsigned)a.c.nv;
            }
            const unsigned have = __ballot_sync(0xffffffffu, good);
            const int valid = min(128, s.n - pos0);
            const bool whole = valid == 128 && have == (1u << nbox) - 1u;
            if (!(ok = wait.warp(bar(L::SF + t), j & 1))) break;
            tc_fence_after();
            if (warp_live) {
                // 32 logits of the row from column c: scaled, gated and masked
                auto logits = [&](int c, float *x) {
                    uint32_t u[32];
                    tmem_ld32(tm + C::S + c, u);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(u[e]) * a.scale_log2;
                    if (FOX) {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {  // 16 positions lie in one page
                            const int bx = (c + e) >> box_shift;
                            const int pid = __shfl_sync(0xffffffffu, id, bx);
                            const bool in = (have >> bx) & 1u;
                            const float4 *gp = reinterpret_cast<const float4 *>(
                                a.c.g_pages + (((size_t)(in ? pid : 0) * a.c.Hq + hq) << a.c.page_shift) +
                                ((pos0 + c + e) & (page - 1)));
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float4 g4 = in ? __ldg(gp + q) : make_float4(0.f, 0.f, 0.f, 0.f);
                                float *v = x + e + 4 * q;
                                v[0] = fmaf(g4.x, kLog2e, v[0] + gq);
                                v[1] = fmaf(g4.y, kLog2e, v[1] + gq);
                                v[2] = fmaf(g4.z, kLog2e, v[2] + gq);
                                v[3] = fmaf(g4.w, kLog2e, v[3] + gq);
                            }
                        }
                    }
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            const int last = ((have >> ((c + e) >> box_shift)) & 1u) ? valid - c - e : 0;
#pragma unroll
                            for (int q = 0; q < 16; ++q) x[e + q] = q < last ? x[e + q] : -INFINITY;
                        }
                    }
                };
                // the logits once in registers, or (where registers are short) read twice
                float x[kTwice ? 32 : 128];
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    float *v = x + (kTwice ? 0 : c);
                    logits(c, v);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) mx = fmax3(mx, v[e], v[e + 1]);
                }
                float alpha = 1.f;
                if (mx > m_run + kRescale || (m_run == -INFINITY && mx > -INFINITY)) {
                    alpha = m_run == -INFINITY ? 0.f : ex2_approx(m_run - mx);
                    m_run = mx;
                }
                // S of this step is complete, so the previous P V is too: O may be rescaled
                const bool resc = alpha != 1.f && l_run > 0.f;
                if (__any_sync(0xffffffffu, resc)) tmem_scale<D>(tm + C::O, resc ? alpha : 1.f);
                l_run *= alpha;
                const float use = m_run == -INFINITY ? 0.f : m_run;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 128; c += 64) {
                    uint32_t p[32];
#pragma unroll
                    for (int half = 0; half < 64; half += 32) {
                        float *v = x + (kTwice ? 0 : c + half);
                        if (kTwice) logits(c + half, v);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float p0 = ex2_approx(v[e] - use), p1 = ex2_approx(v[e + 1] - use);
                            sum += p0 + p1;
                            p[(half + e) / 2] = pack_bf16x2(p0, p1);
                        }
                    }
                    // the weights of columns c .. c + 63 take 32 columns of S that have been read
                    tmem_st32(tm + C::S + c / 2, p);
                }
                l_run += sum;
                tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive_warp(bar(L::PR + t));
        }
        if (ok) ok = wait.warp(bar(L::FIN), 0);
        if (ok && warp_live) {
            tc_fence_after();
            const size_t at = (size_t)(1 + blockIdx.z) * a.c.Hkv * y.R + row;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tld32(tm + C::O + c, o);
                if (live) {
                    // a row whose keys were all absent has weights of nothing: its sum is 0
                    float4 *dst = reinterpret_cast<float4 *>(y.po + at * D + c);
#pragma unroll
                    for (int q = 0; q < 8; ++q) dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
            }
            if (live) y.pml[at] = make_float2(m_run, l_run);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, C::cols);
    }
}

// ================================================================ scan
// Chunks of several blocks of 64 tokens. A CTA takes 128 rows of a sequence and key head,
// which span blocks lo .. hi of the chunk, and visits the key blocks hi - 1, ..., 0. A row of
// block c takes part from block c - 1 on: its logits are x . k~_j (N = 64), its softmax goes
// on from the part that the preparation left, and its state moves on by x += x (P_b - I)^T.
// The state is the fp32 accumulator itself in TMEM; each step's products take a bf16 copy
// of it (rows that do not take part yet have a zero copy and so keep their state). At the
// end the state is the query carried to the chunk's start.
// Warps: 0-3 softmax, one row per thread; 4-7 the bf16 copy of the state; 8 allocates TMEM,
// issues the MMAs and streams [k~_b; P_b - I] and V_b.
template <int D>
struct ScanSmem {
    static constexpr int NR = 3, NV = 2;
    static constexpr uint32_t xtile = 128 * D * 2, xatom = 128 * 128, ratom = (64 + D) * 128, rtile = ratom * (D / 64),
                              vatom = 64 * 128, vtile = vatom * (D / 64);
    static constexpr uint32_t X = 0, R = X + xtile, V = R + NR * rtile, bars = V + NV * vtile;
    static constexpr int RF = 0, RE = RF + NR, VF = RE + NR, VE = VF + NV, SX = VE + NV, XR = SX + 1, SFREE = XR + 1,
                         PR = SFREE + 1, PV = PR + 1, FIN = PV + 1, count = FIN + 1;
    static constexpr uint32_t bytes = bars + count * 8 + 16, alloc = bytes + 1024;
    // TMEM columns
    static constexpr uint32_t cS = 0, cP = 64, cX = 128, cO = 128 + D, cols = D == 64 ? 256 : 512;
};

constexpr int kScanThr = 288;

template <int D, bool FOX>
__global__ void __launch_bounds__(kScanThr, D == 64 ? 2 : 1)
tc_scan_kernel(const Step a, const TcWs y, const __grid_constant__ CUtensorMap tm_r,
               const __grid_constant__ CUtensorMap tm_v, uint64_t limit_ns) {
    using L = ScanSmem<D>;
    constexpr int NA = D / 64;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const sm = smem_raw + (base - raw);
    auto bar = [&](int i) { return base + L::bars + 8u * (uint32_t)i; };
    uint32_t *const tslot = reinterpret_cast<uint32_t *>(sm + L::bars + 8 * L::count);
    volatile uint32_t *const abort_f = tslot + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y, G = a.c.G;
    int b, ti;
    Seq s;
    // later rows walk further: the last tiles first
    if (!tile_of(a, gridDim.x - 1 - blockIdx.x, 128, b, ti, s)) return;
    const int row0 = 128 * ti, rows_all = s.T * G, per_block = kC * G;
    const int hi = (min(row0 + 128, rows_all) - 1) / per_block, steps = hi;
    if (steps <= 0) return;
    const Wait wait{abort_f, a.status, limit_ns};
    if (tid == 0) {
        *abort_f = 0u;
        for (int i = 0; i < L::count; ++i)
            mbar_init(bar(i), i == L::XR || i == L::SFREE || i == L::PR ? 4u : 1u);
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tslot), L::cols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    // the row of a thread of warps 0-3 or 4-7 and its block (one per warp: 64 G is a multiple of 32)
    const int r = tid & 127;
    const bool live = row0 + r < rows_all;
    const int own = min(row0 + (r & ~31), rows_all - 1) / per_block;
    const size_t row = (size_t)h * y.R + (size_t)s.first * G + row0 + r;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;

    if (warp == 8) {
        if (lane == 0) {
            int r_iss = 0, v_iss = 0, r_done = 0, v_done = 0;
            auto load_r = [&](int st) {
                const int kb = hi - 1 - st, i = st % L::NR, head = slot_of(s, b, kb) * a.c.Hkv + h;
                mbar_arrive_expect_tx(bar(L::RF + i), L::rtile);
                for (int x = 0; x < NA; ++x)
                    tma_load_3d(base + L::R + i * L::rtile + x * L::ratom, &tm_r, bar(L::RF + i), 64 * x, 0, head);
                ++r_iss;
            };
            auto load_v = [&](int st) {
                const int kb = hi - 1 - st, i = st % L::NV, head = slot_of(s, b, kb) * a.c.Hkv + h;
                mbar_arrive_expect_tx(bar(L::VF + i), L::vtile);
                for (int x = 0; x < NA; ++x)
                    tma_load_3d(base + L::V + i * L::vtile + x * L::vatom, &tm_v, bar(L::VF + i), 64 * x, 0, head);
                ++v_iss;
            };
            for (int st = 0; st < steps && st < L::NR; ++st) load_r(st);
            for (int st = 0; st < steps && st < L::NV; ++st) load_v(st);
            constexpr uint32_t ID_S = idesc_b16(128, 64, false), ID_X = idesc_b16(128, D, false),
                               ID_O = idesc_b16(128, D, true);
            bool ok = true;
            auto issue_pv = [&](int st) -> bool {
                const int i = st % L::NV;
                if (!wait(bar(L::VF + i), (st / L::NV) & 1)) return false;
                ++v_done;
                if (!wait(bar(L::PR), st & 1)) return false;
                tc_fence_after();
                const uint64_t v = sdesc_sw128(base + L::V + i * L::vtile, L::vatom, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) umma_tA(tmem + L::cO, tmem + L::cP + 8 * kk, v + 128 * kk, ID_O, 1);
                umma_commit(bar(L::PV));
                umma_commit(bar(L::VE + i));
                if (st + L::NV < steps) {
                    if (!wait(bar(L::VE + i), (st / L::NV) & 1)) return false;
                    load_v(st + L::NV);
                }
                return true;
            };
            for (int st = 0; ok && st < steps; ++st) {
                const int i = st % L::NR;
                if (!(ok = wait(bar(L::RF + i), (st / L::NR) & 1))) break;
                ++r_done;
                if (!(ok = wait(bar(L::XR), st & 1))) break;                       // the copy of the state
                if (st > 0 && !(ok = wait(bar(L::SFREE), (st - 1) & 1))) break;    // the last logits read
                tc_fence_after();
                const uint32_t rs = base + L::R + i * L::rtile;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16(tmem + L::cS, sdesc_sw128(base + L::X + (kk >> 2) * L::xatom, 16, 1024) + 2 * (kk & 3),
                              sdesc_sw128(rs + (kk >> 2) * L::ratom, 16, 1024) + 2 * (kk & 3), ID_S, kk > 0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16(tmem + L::cX, sdesc_sw128(base + L::X + (kk >> 2) * L::xatom, 16, 1024) + 2 * (kk & 3),
                              sdesc_sw128(rs + 64 * 128 + (kk >> 2) * L::ratom, 16, 1024) + 2 * (kk & 3), ID_X, 1);
                umma_commit(bar(L::SX));
                umma_commit(bar(L::RE + i));
                // P V of the previous step behind this step's products; then the slot of the step
                // before refills
                if (st > 0 && !(ok = issue_pv(st - 1))) break;
                if (st > 0 && st - 1 + L::NR < steps) {
                    const int pi = (st - 1) % L::NR;
                    if (!(ok = wait(bar(L::RE + pi), ((st - 1) / L::NR) & 1))) break;
                    load_r(st - 1 + L::NR);
                }
            }
            if (ok) ok = issue_pv(steps - 1);
            umma_commit(bar(L::FIN));
            mbar_wait(bar(L::FIN), 0, limit_ns);
            for (; r_done < r_iss; ++r_done) mbar_wait(bar(L::RF + r_done % L::NR), (r_done / L::NR) & 1, limit_ns);
            for (; v_done < v_iss; ++v_done) mbar_wait(bar(L::VF + v_done % L::NV), (v_done / L::NV) & 1, limit_ns);
        }
    } else if (warp < 4) {
        // ============================================================ softmax
        const int hq = h * G + (live ? (row0 + r) % G : 0);
        float m_run = -INFINITY, l_run = 0.f;
        if (live) {
            const float2 ml = y.pml[row];
            m_run = ml.x;
            l_run = ml.y;
        }
        const float gq = FOX && live ? y.gq[row] : 0.f;
        double between = 0.0;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            float o[32];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 v = live ? *reinterpret_cast<const float4 *>(y.po + row * D + c + 4 * q)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                o[4 * q] = v.x; o[4 * q + 1] = v.y; o[4 * q + 2] = v.z; o[4 * q + 3] = v.w;
            }
            tst32(tmem + lane_off + L::cO + c, o);
        }
        tmem_st_wait();
        bool ok = true;
        for (int st = 0; st < steps; ++st) {
            const int kb = hi - 1 - st;
            const bool part = kb < own;  // the same for the warp
            if (!(ok = wait.warp(bar(L::SX), st & 1))) break;
            tc_fence_after();
            float x[64];
            if (part) {
                tld32(tmem + lane_off + L::cS, x);
                tld32(tmem + lane_off + L::cS + 32, x + 32);
            }
            tc_fence_before();
            mbar_arrive_warp(bar(L::SFREE));
            if (part) {
                const int ks = slot_of(s, b, kb);
                if (FOX) {
                    const float bias = (float)((double)gq + between) * kLog2e;
                    const float4 *gt = reinterpret_cast<const float4 *>(y.gt + ((size_t)ks * a.c.Hq + hq) * kC);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const float4 g4 = __ldg(gt + q);
                        x[4 * q] = fmaf(g4.x, kLog2e, fmaf(x[4 * q], a.scale_log2, bias));
                        x[4 * q + 1] = fmaf(g4.y, kLog2e, fmaf(x[4 * q + 1], a.scale_log2, bias));
                        x[4 * q + 2] = fmaf(g4.z, kLog2e, fmaf(x[4 * q + 2], a.scale_log2, bias));
                        x[4 * q + 3] = fmaf(g4.w, kLog2e, fmaf(x[4 * q + 3], a.scale_log2, bias));
                    }
                    between += y.gtot[(size_t)ks * a.c.Hq + hq];
                } else {
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c] *= a.scale_log2;
                }
            }
            // P and O are free once the previous P V has completed
            if (st > 0 && !(ok = wait.warp(bar(L::PV), (st - 1) & 1))) break;
            tc_fence_after();
            uint32_t p[32];
            if (part) {
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 64; c += 2) mx = fmax3(mx, x[c], x[c + 1]);
                float alpha = 1.f;
                if (mx > m_run + kRescale) {
                    alpha = ex2_approx(m_run - mx);
                    m_run = mx;
                }
                if (!live) alpha = 1.f;
                if (__any_sync(0xffffffffu, alpha != 1.f)) tmem_scale<D>(tmem + lane_off + L::cO, alpha);
                l_run *= alpha;
                const float use = m_run == -INFINITY ? 0.f : m_run;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    const float p0 = live ? ex2_approx(x[c] - use) : 0.f, p1 = live ? ex2_approx(x[c + 1] - use) : 0.f;
                    sum += p0 + p1;
                    p[c / 2] = pack_bf16x2(p0, p1);
                }
                l_run += sum;
            } else {
#pragma unroll
                for (int c = 0; c < 32; ++c) p[c] = 0u;
            }
            tmem_st32(tmem + lane_off + L::cP, p);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(bar(L::PR));
        }
        if (ok) ok = wait.warp(bar(L::FIN), 0);
        if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tld32(tmem + lane_off + L::cO + c, o);
                if (live) {
                    float4 *dst = reinterpret_cast<float4 *>(y.po + row * D + c);
#pragma unroll
                    for (int q = 0; q < 8; ++q) dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
            }
            if (live) {
                y.pml[row] = make_float2(m_run, l_run);
                if (FOX) y.gq[row] = (float)((double)gq + between);
            }
        }
    } else {
        // ============================================================ the state's bf16 copy
        bool ok = true;
        uint8_t *const xs = sm + L::X;
        auto put = [&](int c, const float *x, bool take) {  // 32 columns from c
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float *v = x + 8 * q;
                *reinterpret_cast<uint4 *>(xs + (c >> 6) * L::xatom + sw128_offset(r, ((c & 63) >> 3) + q)) =
                    take ? make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                      pack_bf16x2(v[6], v[7]))
                         : make_uint4(0u, 0u, 0u, 0u);
            }
        };
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            float x[32];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 u = live ? *reinterpret_cast<const uint4 *>(y.qt + row * D + c + 8 * q)
                                     : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack_bf16x2(w[e]);
                    x[8 * q + 2 * e] = f.x;
                    x[8 * q + 2 * e + 1] = f.y;
                }
            }
            tst32(tmem + lane_off + L::cX + c, x);
            put(c, x, hi - 1 < own);
        }
        tmem_st_wait();
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive_warp(bar(L::XR));
        for (int st = 1; st < steps; ++st) {
            if (!(ok = wait.warp(bar(L::SX), (st - 1) & 1))) break;
            tc_fence_after();
            const bool take = hi - 1 - st < own;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float x[32];
                if (take) tld32(tmem + lane_off + L::cX + c, x);
                put(c, x, take);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive_warp(bar(L::XR));
        }
        if (ok) ok = wait.warp(bar(L::FIN), 0);
        if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float x[32];
                tld32(tmem + lane_off + L::cX + c, x);
                if (live) {
                    uint4 *dst = reinterpret_cast<uint4 *>(y.qt + row * D + c);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        dst[q] = make_uint4(pack_bf16x2(x[8 * q], x[8 * q + 1]), pack_bf16x2(x[8 * q + 2], x[8 * q + 3]),
                                            pack_bf16x2(x[8 * q + 4], x[8 * q + 5]),
                                            pack_bf16x2(x[8 * q + 6], x[8 * q + 7]));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, L::cols);
    }
}

// (heads, rows, D columns) bf16 with (64 columns, box_rows) boxes, 128-byte swizzle
bool make_map(CUtensorMap *m, const void *ptr, int D, long long rows, long long heads, int box_rows) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)rows * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t big_smem(K kern, size_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int NT, int D, bool FOX>
cudaError_t launch_cached(const Step &a, const TcWs &y, uint64_t limit_ns, cudaStream_t stream) {
    CUtensorMap tx, tm, tk, tv;
    if (!make_map(&tx, y.qt, D, y.R, a.c.Hkv, 128) ||
        !make_map(&tm, y.mt, D, D, (long long)a.c.seqs * a.c.Hkv * 2, D) ||
        !make_map(&tk, a.c.k_pages, D, a.c.page, (long long)a.c.nk * a.c.Hkv, a.c.page < 128 ? a.c.page : 128) ||
        !make_map(&tv, a.c.v_pages, D, a.c.page, (long long)a.c.nv * a.c.Hkv, a.c.page < 128 ? a.c.page : 128))
        return cudaErrorInvalidValue;
    auto kern = tc_cached_kernel<NT, D, FOX>;
    const cudaError_t e = big_smem(kern, CachedSmem<NT, D>::alloc);
    if (e != cudaSuccess) return e;
    kern<<<dim3(tile_slots(a.N, a.c.G, a.c.seqs, 128 * NT), a.c.Hkv, y.splits), kCachedThr, CachedSmem<NT, D>::alloc,
           stream>>>(a, y, tx, tm, tk, tv, limit_ns);
    return cudaGetLastError();
}

template <int D, bool FOX>
cudaError_t launch_scan(const Step &a, const TcWs &y, uint64_t limit_ns, cudaStream_t stream) {
    CUtensorMap tr, tv;
    const long long heads = (long long)slots_of(a.N, a.c.seqs) * a.c.Hkv;
    if (!make_map(&tr, y.kh, D, 64 + D, heads, 64 + D) || !make_map(&tv, y.vb, D, 64, heads, 64))
        return cudaErrorInvalidValue;
    auto kern = tc_scan_kernel<D, FOX>;
    const cudaError_t e = big_smem(kern, ScanSmem<D>::alloc);
    if (e != cudaSuccess) return e;
    kern<<<dim3(tile_slots(a.N, a.c.G, a.c.seqs, 128), a.c.Hkv), kScanThr, ScanSmem<D>::alloc, stream>>>(a, y, tr, tv,
                                                                                                        limit_ns);
    return cudaGetLastError();
}

}  // namespace

template <int D>
cudaError_t launch_tc_prep(const Step &a, const TcWs &y, cudaStream_t stream);
template <int D>
cudaError_t launch_tc_carry(const Step &a, const TcWs &y, cudaStream_t stream);
template <int D>
cudaError_t launch_tc_finish(const Step &a, const TcWs &y, int tile_rows, cudaStream_t stream);

namespace {

template <int D, bool FOX>
cudaError_t launch_all(const Step &a, const TcWs &y, uint64_t limit_ns, cudaStream_t stream) {
    cudaError_t e = launch_tc_prep<D>(a, y, stream);
    if (a.max_chunk > kC) {
        if (e == cudaSuccess) e = launch_tc_carry<D>(a, y, stream);
        if (e == cudaSuccess) e = launch_scan<D, FOX>(a, y, limit_ns, stream);
    }
    if (a.c.max_pages > 0 && a.c.nk > 0 && a.c.nv > 0) {
        if (e == cudaSuccess) e = launch_cached<1, D, FOX>(a, y, limit_ns, stream);
        if (e == cudaSuccess && (long long)a.max_chunk * a.c.G > 128) e = launch_cached<2, D, FOX>(a, y, limit_ns, stream);
    }
    if (e == cudaSuccess) e = launch_tc_finish<D>(a, y, 128, stream);
    return e;
}

struct TcLayout {
    int splits;
    size_t qt, po, pml, gq, gt, gtot, mt, kh, kl, vb, total;
};

// Splits of the cached keys, for two CTAs per SM. The parts are sized by a bound that does not
// fall as the step grows, so that a workspace for many tokens serves smaller steps.
TcLayout tc_layout(const Cache &c, int N, int max_chunk, int d, bool fox) {
    TcLayout y;
    const size_t slots = slots_of(N, c.seqs), R = (size_t)N * c.G;
    const long long cap = (long long)c.max_pages << c.page_shift;
    const long long tiles = (long long)tile_slots(N, c.G, c.seqs, 128) * c.Hkv;
    const long long want = 2 * 152 / tiles + 1, most = (cap + 511) / 512;
    y.splits = (int)(want < most ? want : most);
    if (y.splits < 1) y.splits = 1;
    size_t off = 256;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    const size_t rows = R * c.Hkv;
    // (1 + splits) rows <= 2 rows + 304 / tiles * rows, and rows <= 128 tiles
    const size_t by_want = 2 * rows + 304 * 128, by_most = rows * (1 + (size_t)(most < 1 ? 1 : most));
    const size_t parts = by_want < by_most ? by_want : by_most;
    y.qt = take(rows * d * 2);
    y.po = take(parts * d * 4);
    y.pml = take(parts * 8);
    y.gq = take(fox ? rows * 4 : 0);
    y.gt = take(fox ? slots * c.Hq * kC * 4 : 0);
    y.gtot = take(fox ? slots * c.Hq * 8 : 0);
    y.mt = take((size_t)c.seqs * c.Hkv * 2 * d * d * 2);
    const bool blocks = max_chunk > kC;
    y.kh = take(blocks ? slots * c.Hkv * (kC + d) * d * 2 : 0);
    y.kl = take(blocks ? slots * c.Hkv * (kC + d) * d * 2 : 0);
    y.vb = take(blocks ? slots * c.Hkv * kC * d * 2 : 0);
    y.total = off;
    return y;
}

}  // namespace

size_t tc_ws_bytes(const Cache &c, int N, int max_chunk, int d, bool fox) {
    return tc_layout(c, N, max_chunk, d, fox).total;
}

cudaError_t launch_tc(const Step &a, int d, void *ws, uint64_t limit_ns, cudaStream_t stream) {
    const bool fox = a.log_f != nullptr;
    const TcLayout f = tc_layout(a.c, a.N, a.max_chunk, d, fox);
    char *w = static_cast<char *>(ws);
    auto b16 = [&](size_t off) { return reinterpret_cast<bf *>(w + off); };
    auto f32 = [&](size_t off) { return reinterpret_cast<float *>(w + off); };
    const TcWs y{b16(f.qt), b16(f.mt), b16(f.kh), b16(f.kl), b16(f.vb), f32(f.po),
                 reinterpret_cast<float2 *>(w + f.pml), f32(f.gq), f32(f.gt),
                 reinterpret_cast<double *>(w + f.gtot), f.splits, (long long)a.N * a.c.G};
    if (d == 64)
        return fox ? launch_all<64, true>(a, y, limit_ns, stream) : launch_all<64, false>(a, y, limit_ns, stream);
    return fox ? launch_all<128, true>(a, y, limit_ns, stream) : launch_all<128, false>(a, y, limit_ns, stream);
}

}  // namespace paged
}  // namespace path
