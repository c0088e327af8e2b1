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
#pragma once

#include "paged_cached_tc.cuh"

namespace path {
namespace paged {

namespace {

// ================================================================ scan
// Chunks of several blocks of 64 tokens. A CTA takes 128 rows of a sequence and key head,
// which span blocks lo .. hi of the chunk, and visits the key blocks hi - 1, ..., 0. A row of
// block c takes part from block c - 1 on: its logits are x . k~_j (N = 64), its softmax goes
// on from the part that the preparation left, and its state moves on by x += x (P_b - I)^T.
// The state is the fp32 accumulator itself in TMEM; each step's products take a bf16 copy
// of it (rows that do not take part yet have a zero copy and so keep their state). At the
// end the state is the query carried to the chunk's start.
// Per step the logits go first, so that the softmax runs beside the state's product and copy,
// which are the chain from step to step. Bound by that chain and the softmax (3,000 cycles a step
// with gates at D = 64): 176 us for 2,048 tokens of 32 heads at
// D = 128 (94 with one part of the state), 57 us for four chunks of up to 1,500 tokens, 16 heads,
// D = 64, gates (91 before the blocks whose gates have closed were left out, 70 with the tiles of
// one key head after the other's, 65 with a row's loads by one lane).
// Warps: 0-3 softmax, one row per thread; 4-7 the bf16 copy of the state; 8 allocates TMEM and
// issues the MMAs; 9 streams [k~_b; P_b - I] and V_b.
//
// LOW: the copy of the state and its own product's factor P_b - I have a second bf16 part. Their
// roundings gather from step to step in the queries that go on to the cached keys; without gates
// and at D = 128, where these then are rounded once more, an output's error behind 1,000 cached
// keys is 2.91e-3 of its norm without, 2.59e-3 with (T = 300; the plain 1.66e-3 is the output's own
// rounding). The scan takes 94 us without and 180 with for 2,048 tokens of 32 heads. At D = 64 the
// weights' second part (low_weights) does more for less. The scan's own weights and keys are rounded
// once: where the chunk is all there is, an output's error is 2.05e-3 of its norm (T = 300, both head
// sizes; 1.95e-3 to 1.98e-3 with gates), and a second part of the weights would lengthen the chain
// that bounds the scan.
template <int D, bool LOW>
struct ScanSmem {
    // slots of [k~_b; P_b - I], of P_b - I's low part and of values
    static constexpr int NR = LOW ? 2 : 3, NL = LOW ? 1 : 0, NV = 2;
    static constexpr uint32_t xtile = 128 * D * 2, xatom = 128 * 128, ratom = (64 + D) * 128, rtile = ratom * (D / 64),
                              latom = D * 128, ltile = latom * (D / 64), vatom = 64 * 128, vtile = vatom * (D / 64);
    static constexpr uint32_t X = 0, R = X + (LOW ? 2 : 1) * xtile, P = R + NR * rtile, V = P + NL * ltile,
                              bars = V + NV * vtile;
    static constexpr int RF = 0, RE = RF + NR, LF = RE + NR, LE = LF + NL, VF = LE + NL, VE = VF + NV, SD = VE + NV,
                         XD = SD + 1, XR = XD + 1, SFREE = XR + 1, PR = SFREE + 1, PV = PR + 1, FIN = PV + 1,
                         count = FIN + 1;
    // behind the barriers: TMEM's address, the abort flag, the last step whose values count (need)
    static constexpr int need = 2;
    static constexpr uint32_t bytes = bars + count * 8 + 16, alloc = bytes + 1024;
    // TMEM columns
    static constexpr uint32_t cS = 0, cP = 64, cX = 128, cO = 128 + D, cols = D == 64 ? 256 : 512;
};

static_assert(ScanSmem<128, true>::alloc <= 227 * 1024, "shared memory");
__host__ __device__ constexpr bool scan_low(int D, bool fox) { return D == 128 && !fox; }
constexpr int kScanThr = 320;

template <int D, bool FOX, typename A>
__global__ void __launch_bounds__(kScanThr, D == 64 ? 2 : 1)
tc_scan_kernel(const A a, const TcWs y, const __grid_constant__ CUtensorMap tm_r,
               const __grid_constant__ CUtensorMap tm_l, const __grid_constant__ CUtensorMap tm_v, uint64_t limit_ns) {
    constexpr bool LOW = scan_low(D, FOX);
    using L = ScanSmem<D, LOW>;
    constexpr int NA = D / 64;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const sm = smem_raw + (base - raw);
    auto bar = [&](int i) { return base + L::bars + 8u * (uint32_t)i; };
    uint32_t *const tslot = reinterpret_cast<uint32_t *>(sm + L::bars + 8 * L::count);
    volatile uint32_t *const abort_f = tslot + 1, *const need = tslot + L::need;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.x % a.c.Hkv, G = a.c.G;
    int b, ti;
    Seq s;
    grid_begin();
    // later rows walk further: the last tiles first, those of all key heads
    const bool mine = tile_of(a, (int)((gridDim.x - 1 - blockIdx.x) / a.c.Hkv), 128, b, ti, s);
    grid_wait();
    if (!mine) return;
    const int row0 = 128 * ti, rows_all = s.T * G, per_block = kC * G;
    const int hi = (min(row0 + 128, rows_all) - 1) / per_block, steps = hi;
    if (steps <= 0) return;
    const Wait wait{abort_f, a.status, limit_ns};
    if (tid == 0) {
        *abort_f = *need = 0u;
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
    // the four rows of this thread's quad in (Hkv, R, D): null past the sequence's end
    auto quad = [&](auto *p, int c) {
        return [=](int i) { return row0 + (r & ~3) + i < rows_all ? p + (row - (r & 3) + i) * D + c : nullptr; };
    };

    if (warp == 9) {
        // ============================================================ factors and values
        if (lane == 0) {
            int r = 0, l = 0, v = 0;
            bool ok = true;
            for (int st = 0; ok && st < steps; ++st) {
                const int head = slot_of(s, b, hi - 1 - st) * a.c.Hkv + h, i = st % L::NR, q = st % L::NV;
                if (st >= L::NR && !(ok = wait(bar(L::RE + i), (st / L::NR - 1) & 1))) break;
                mbar_arrive_expect_tx(bar(L::RF + i), L::rtile);
                for (int x = 0; x < NA; ++x)
                    tma_load_3d(base + L::R + i * L::rtile + x * L::ratom, &tm_r, bar(L::RF + i), 64 * x, 0, head);
                ++r;
                if (LOW) {
                    if (st >= L::NL && !(ok = wait(bar(L::LE), (st - 1) & 1))) break;
                    mbar_arrive_expect_tx(bar(L::LF), L::ltile);
                    for (int x = 0; x < NA; ++x)
                        tma_load_3d(base + L::P + x * L::latom, &tm_l, bar(L::LF), 64 * x, 64, head);
                    ++l;
                }
                if (st >= L::NV && !(ok = wait(bar(L::VE + q), (st / L::NV - 1) & 1))) break;
                mbar_arrive_expect_tx(bar(L::VF + q), L::vtile);
                for (int x = 0; x < NA; ++x)
                    tma_load_3d(base + L::V + q * L::vtile + x * L::vatom, &tm_v, bar(L::VF + q), 64 * x, 0, head);
                ++v;
            }
            if (!ok) {  // an abort: no copy may land after the CTA is gone
                for (int st = r > L::NR ? r - L::NR : 0; st < r; ++st)
                    mbar_wait(bar(L::RF + st % L::NR), (st / L::NR) & 1, limit_ns);
                if (l > 0) mbar_wait(bar(L::LF), (l - 1) & 1, limit_ns);
                for (int st = v > L::NV ? v - L::NV : 0; st < v; ++st)
                    mbar_wait(bar(L::VF + st % L::NV), (st / L::NV) & 1, limit_ns);
            }
        }
    } else if (warp == 8) {
        // ============================================================ MMA issue
        if (lane == 0) {
            constexpr uint32_t ID_S = idesc_b16(128, 64, false), ID_X = idesc_b16(128, D, false),
                               ID_O = idesc_b16(128, D, true);
            bool ok = true;
            auto issue_pv = [&](int st) -> bool {
                const int i = st % L::NV;
                if (!wait(bar(L::VF + i), (st / L::NV) & 1) || !wait(bar(L::PR), st & 1)) return false;
                tc_fence_after();
                const uint64_t v = sdesc_sw128(base + L::V + i * L::vtile, L::vatom, 1024);
                if (!FOX || *need == st + 1u)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) umma_tA(tmem + L::cO, tmem + L::cP + 8 * kk, v + 128 * kk, ID_O, 1);
                umma_commit(bar(L::PV));
                umma_commit(bar(L::VE + i));
                return true;
            };
            for (int st = 0; ok && st < steps; ++st) {
                const int i = st % L::NR;
                if (!(ok = wait(bar(L::RF + i), (st / L::NR) & 1))) break;
                if (!(ok = wait(bar(L::XR), st & 1))) break;                       // the copy of the state
                if (st > 0 && !(ok = wait(bar(L::SFREE), (st - 1) & 1))) break;    // the last logits read
                tc_fence_after();
                const uint32_t rs = base + L::R + i * L::rtile;
                // a part of the state with a factor's tile
                auto product = [&](uint32_t d, int part, uint32_t b, uint32_t batom, uint32_t id, bool first) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_bf16(d,
                                  sdesc_sw128(base + L::X + part * L::xtile + (kk >> 2) * L::xatom, 16, 1024) +
                                      2 * (kk & 3),
                                  sdesc_sw128(b + (kk >> 2) * batom, 16, 1024) + 2 * (kk & 3), id, !first || kk > 0);
                };
                product(tmem + L::cS, 0, rs, L::ratom, ID_S, true);
                if (LOW) product(tmem + L::cS, 1, rs, L::ratom, ID_S, false);
                umma_commit(bar(L::SD));
                product(tmem + L::cX, 0, rs + 64 * 128, L::ratom, ID_X, false);
                if (LOW) {
                    product(tmem + L::cX, 1, rs + 64 * 128, L::ratom, ID_X, false);
                    if (!(ok = wait(bar(L::LF), st & 1))) break;
                    tc_fence_after();
                    product(tmem + L::cX, 0, base + L::P, L::latom, ID_X, false);
                    umma_commit(bar(L::LE));
                }
                umma_commit(bar(L::XD));
                umma_commit(bar(L::RE + i));
                // P V of the previous step behind this step's products
                if (st > 0 && !(ok = issue_pv(st - 1))) break;
            }
            if (ok) ok = issue_pv(steps - 1);
            umma_commit(bar(L::FIN));
            mbar_wait(bar(L::FIN), 0, limit_ns);
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
        float between = 0.f;  // gates of the blocks passed (where they matter the sum is small: fp32 will do)
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint4 u[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) load_quad_rows(u[q], quad(y.po, c + 16 * q));
            tmem_st32(tmem + lane_off + L::cO + c, reinterpret_cast<uint32_t(&)[32]>(u));
        }
        tmem_st_wait();
        bool ok = true;
        for (int st = 0; st < steps; ++st) {
            const int kb = hi - 1 - st;
            const bool part = kb < own;  // the same for the warp
            const int ks = slot_of(s, b, kb);
            const float4 *const gt =
                FOX ? reinterpret_cast<const float4 *>(y.gt + ((size_t)ks * a.c.Hq + hq) * kC) : nullptr;
            // the block's gates: their sum, and the largest sum behind a key
            float2 block = make_float2(0.f, 0.f);
            float bias = 0.f;
            if (FOX && part) {
                block = y.gblk[(size_t)ks * a.c.Hq + hq];
                bias = (gq + between) * kLog2e;
                if (bias > m_run - kNothing - kGuess) {  // on their way while the product runs
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(gt));
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(gt + 8));
                }
            }
            if (!(ok = wait.warp(bar(L::SD), st & 1))) break;
            tc_fence_after();
            float x[64];
            {
                uint32_t(*u)[32] = reinterpret_cast<uint32_t(*)[32]>(x);
                tmem_ld32(tmem + lane_off + L::cS, u[0]);
                tmem_ld32(tmem + lane_off + L::cS + 32, u[1]);
                tmem_ld_wait();
            }
            tc_fence_before();
            mbar_arrive_warp(bar(L::SFREE));
            // NaN if one of them is, which then counts below and makes its row's sums NaN
            auto top64 = [&]() {
                float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c < 60; c += 8)
#pragma unroll
                    for (int q = 0; q < 4; ++q) m4[q] = fmax3_nan(m4[q], x[c + 2 * q], x[c + 2 * q + 1]);
                return fmax3_nan(fmax3_nan(m4[0], m4[1], m4[2]), fmax3_nan(m4[3], x[60], x[61]),
                                 fmax3_nan(x[62], x[63], x[63]));
            };
            // PaTH-FoX: a block whose logits all lie below 2^-64 of what a row has is left out (2^22 keys
            // of those move a sum by less than 2^-42 of itself), its values' product too if that
            // holds for all rows
            bool counts = part;
            if (FOX && part)
                counts = __any_sync(0xffffffffu,
                                    live && !(top64() + fmaf(block.y, kLog2e, bias) < m_run - kNothing)) != 0;
            if (FOX && counts) {
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const float4 g4 = gt[q];
                    x[4 * q] = fmaf(g4.x, kLog2e, x[4 * q] + bias);
                    x[4 * q + 1] = fmaf(g4.y, kLog2e, x[4 * q + 1] + bias);
                    x[4 * q + 2] = fmaf(g4.z, kLog2e, x[4 * q + 2] + bias);
                    x[4 * q + 3] = fmaf(g4.w, kLog2e, x[4 * q + 3] + bias);
                }
            }
            if (FOX) between += block.x;
            // P and O are free once the previous P V has completed
            if (st > 0 && !(ok = wait.warp(bar(L::PV), (st - 1) & 1))) break;
            tc_fence_after();
            if (FOX && counts && lane == 0) *need = st + 1;  // the last step's has been read
            uint32_t p[16];
            if (counts) {
                const float mx = top64();
                float alpha = 1.f;
                if (mx > m_run + kRescale) {
                    alpha = ex2_approx(m_run - mx);
                    m_run = mx;
                }
                if (!live) alpha = 1.f;
                if (__any_sync(0xffffffffu, alpha != 1.f)) tmem_scale<D>(tmem + lane_off + L::cO, alpha);
                l_run *= alpha;
                // rows past the sequence's end weigh as they will: nobody reads their sums
                const float use = m_run == -INFINITY ? 0.f : -m_run;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int half = 0; half < 64; half += 32) {
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float2 z = fadd2(make_float2(x[half + c], x[half + c + 1]), make_float2(use, use));
                        const float2 q = make_float2(ex2_approx(z.x), ex2_approx(z.y));
                        sum[(c >> 1) & 1] = fadd2(sum[(c >> 1) & 1], q);
                        p[c / 2] = pack_bf16x2(q.x, q.y);
                    }
                    tmem_st16(tmem + lane_off + L::cP + half / 2, p);
                }
                l_run += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            } else {
#pragma unroll
                for (int c = 0; c < 16; ++c) p[c] = 0u;
                tmem_st16(tmem + lane_off + L::cP, p);
                tmem_st16(tmem + lane_off + L::cP + 16, p);
            }
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
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint4 u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        u[e] = make_uint4(__float_as_uint(o[16 * q + 4 * e]), __float_as_uint(o[16 * q + 4 * e + 1]),
                                          __float_as_uint(o[16 * q + 4 * e + 2]), __float_as_uint(o[16 * q + 4 * e + 3]));
                    store_quad_rows(u, quad(y.po, c + 16 * q));
                }
            }
            if (live) {
                y.pml[row] = make_float2(m_run, l_run);
                if (FOX) y.gq[row] = gq + between;
            }
        }
    } else if (warp < 8) {
        // ============================================================ the state's bf16 copy
        bool ok = true;
        const bool low = low_queries(a, s.T, D);  // of what goes on to the cached keys
        uint8_t *const xs = sm + L::X;
        auto put = [&](int c, const float *x, bool take) {  // 32 columns from c
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t hi[4] = {}, lo[4] = {};
                if (take)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (LOW) split2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1], hi[e], lo[e]);
                        else hi[e] = pack_bf16x2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1]);
                uint4 *const at =
                    reinterpret_cast<uint4 *>(xs + (c >> 6) * L::xatom + sw128_offset(r, ((c & 63) >> 3) + q));
                at[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if (LOW) at[L::xtile / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        };
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            float x[32];
            uint4 u[4], z[4];
            load_quad_rows(u, quad(y.qt, c));
            load_quad_rows(z, quad(y.ql, c));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t w[4] = {u[q].x, u[q].y, u[q].z, u[q].w}, wl[4] = {z[q].x, z[q].y, z[q].z, z[q].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack_bf16x2(w[e]), g = unpack_bf16x2(wl[e]);
                    x[8 * q + 2 * e] = f.x + g.x;
                    x[8 * q + 2 * e + 1] = f.y + g.y;
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
            if (!(ok = wait.warp(bar(L::XD), (st - 1) & 1))) break;
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
                uint4 u[4], z[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1], hi[e], lo[e]);
                    u[q] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    z[q] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                store_quad_rows(u, quad(y.qt, c));
                if (low) store_quad_rows(z, quad(y.ql, c));
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

template <int D, bool FOX, typename A>
cudaError_t launch_scan(const A &a, const TcWs &y, uint64_t limit_ns, cudaStream_t stream) {
    CUtensorMap tr, tl, tv;
    const long long heads = (long long)slots_of(a.N, a.c.seqs) * a.c.Hkv;
    if (!make_map(&tr, y.kh, D, 64 + D, heads, 64 + D) || !make_map(&tl, y.kl, D, 64 + D, heads, D) ||
        !make_map(&tv, y.vb, D, 64, heads, 64))
        return cudaErrorInvalidValue;
    using L = ScanSmem<D, scan_low(D, FOX)>;
    auto kern = tc_scan_kernel<D, FOX, A>;
    const cudaError_t e = big_smem(kern, L::alloc);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3(tile_slots(a.N, a.c.G, a.c.seqs, 128) * a.c.Hkv), kScanThr, L::alloc, stream, false, a, y,
                  tr, tl, tv, limit_ns);
}

}  // namespace

template <int D, typename A>
cudaError_t launch_tc_prep(const A &a, const TcWs &y, cudaStream_t stream);
template <int D, typename A>
cudaError_t launch_tc_carry(const A &a, const TcWs &y, cudaStream_t stream);
template <int D, typename A>
cudaError_t launch_tc_finish(const A &a, const TcWs &y, const Behind &x, cudaStream_t stream);
cudaError_t launch_prefix_tc(const StepMore &a, int d, float *carry, float *gates, const TcWs *y, void *ws, bool first,
                             uint64_t limit_ns, Behind *behind, cudaStream_t stream);
cudaError_t launch_singles(const StepMore &a, int d, const TcWs &y, float *carry, float *gates, void *ws,
                           uint64_t limit_ns, Behind *behind, cudaStream_t stream);

namespace {

// What a step has of prefixes: the carries (and gates) and the workspace's part for them; null where none.
struct PrefixArgs {
    float *carry, *gates;
    void *ws;
};

template <int D, bool FOX, typename A>
cudaError_t launch_all(const A &a, const TcWs &y, const PrefixArgs &x, uint64_t limit_ns, cudaStream_t stream) {
    constexpr bool more = std::is_same<A, StepMore>::value;
    constexpr Pass M = more ? Pass::window : Pass::step;
    Behind behind = {};
    cudaError_t e;
    // single tokens, unless more query heads share a key head than a tile has rows
    if constexpr (more)
        if (a.max_chunk == 1 && a.c.G <= 128) {
            TcWs one = y;
            one.plan[0].ctas = 152 * CachedCfg<1, D, Pass::one, FOX>::ctas_per_sm;
            e = launch_singles(a, D, one, x.carry, x.gates, x.ws, limit_ns, &behind, stream);
            return e != cudaSuccess ? e : launch_tc_finish<D>(a, one, behind, stream);
        }
    e = launch_tc_prep<D>(a, y, stream);
    if (a.max_chunk > kC) {
        if (e == cudaSuccess) e = launch_tc_carry<D>(a, y, stream);
        if (e == cudaSuccess) e = launch_scan<D, FOX>(a, y, limit_ns, stream);
    }
    if constexpr (more)
        if (e == cudaSuccess && x.carry != nullptr)
            e = launch_prefix_tc(a, D, x.carry, x.gates, &y, x.ws, false, limit_ns, &behind, stream);
    if (a.c.max_pages > 0) {
        if (e == cudaSuccess) e = launch_cached<1, D, FOX, M>(a, y, limit_ns, stream);
        if (e == cudaSuccess && !one_tile(a.max_chunk, a.c.G, D, FOX))
            e = launch_cached<2, D, FOX, M>(a, y, limit_ns, stream);
    }
    if (e == cudaSuccess) e = launch_tc_finish<D>(a, y, behind, stream);
    return e;
}

struct TcLayout {
    int ctas[2];
    size_t qt, ql, po, pml, so[2], sml[2], units[2], items[2], gq, gt, gtot, gblk, mt, kh, kl, vb, ch, cl, gp, total;
};

// The regions depend on the sizes in ways that do not fall as the step grows, so that a workspace
// for many tokens serves smaller steps.
TcLayout tc_layout(const Cache &c, int N, int max_chunk, int d, bool fox) {
    TcLayout y;
    const size_t slots = slots_of(N, c.seqs), rows = (size_t)N * c.G * c.Hkv;
    size_t off = 256;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    y.qt = take(rows * d * 2);
    y.ql = take(rows * d * 2);
    y.po = take(rows * d * 4);
    y.pml = take(rows * 8);
    for (int p = 0; p < 2; ++p) {
        // one CTA per SM, or two: every SM of the part (152) has its share of the units
        y.ctas[p] = 152 * (p == 0 && d == 64 ? CachedCfg<1, 64, Pass::step, false>::ctas_per_sm : 1);
        const bool used = p == 0 || !one_tile(max_chunk, c.G, d, fox);
        const size_t tile = 128 * (p + 1);
        const size_t parts =
            used ? y.ctas[p] + (size_t)tile_slots(N, c.G, std::min(c.seqs, N), (int)tile) * c.Hkv : 0;
        y.so[p] = take(parts * tile * d * 4);
        y.sml[p] = take(parts * tile * 8);
        y.units[p] = take(((size_t)c.seqs + 1) * 8);
        y.items[p] = take(((size_t)c.seqs + 1) * 8);
    }
    y.gq = take(fox ? rows * 4 : 0);
    y.gt = take(fox ? slots * c.Hq * kC * 4 : 0);
    y.gtot = take(fox ? slots * c.Hq * 8 : 0);
    y.gblk = take(fox ? slots * c.Hq * 8 : 0);
    y.mt = take((size_t)std::min(c.seqs, N) * c.Hkv * 2 * d * d * 2);
    const bool blocks = max_chunk > kC;
    y.kh = take(blocks ? slots * c.Hkv * (kC + d) * d * 2 : 0);
    y.kl = take(blocks ? slots * c.Hkv * (kC + d) * d * 2 : 0);
    y.vb = take(blocks ? slots * c.Hkv * kC * d * 2 : 0);
    const bool groups = max_chunk > kC * 8;  // kGroup blocks
    y.ch = take(groups ? slots * c.Hkv * kC * d * 2 : 0);
    y.cl = take(groups ? slots * c.Hkv * kC * d * 2 : 0);
    y.gp = take(groups ? (slots / 8 + c.seqs) * c.Hkv * 2 * d * d * 2 : 0);
    y.total = off;
    return y;
}

}  // namespace

template <typename A>
cudaError_t launch_tc(const A &a, int d, void *ws, float *carry, float *gates, void *pws, uint64_t limit_ns,
                      cudaStream_t stream) {
    const bool fox = a.log_f != nullptr;
    const TcLayout f = tc_layout(a.c, a.N, a.max_chunk, d, fox);
    char *w = static_cast<char *>(ws);
    auto b16 = [&](size_t off) { return reinterpret_cast<bf *>(w + off); };
    auto f32 = [&](size_t off) { return reinterpret_cast<float *>(w + off); };
    TcWs y;
    y.qt = b16(f.qt);
    y.ql = b16(f.ql);
    y.mt = b16(f.mt);
    y.kh = b16(f.kh);
    y.kl = b16(f.kl);
    y.vb = b16(f.vb);
    y.ch = b16(f.ch);
    y.cl = b16(f.cl);
    y.gp = b16(f.gp);
    y.po = f32(f.po);
    y.pml = reinterpret_cast<float2 *>(w + f.pml);
    for (int p = 0; p < 2; ++p) {
        y.so[p] = f32(f.so[p]);
        y.sml[p] = reinterpret_cast<float2 *>(w + f.sml[p]);
        y.plan[p] = Plan{reinterpret_cast<long long *>(w + f.units[p]),
                         reinterpret_cast<long long *>(w + f.items[p]), f.ctas[p]};
    }
    y.gq = f32(f.gq);
    y.gt = f32(f.gt);
    y.gtot = reinterpret_cast<double *>(w + f.gtot);
    y.gblk = reinterpret_cast<float2 *>(w + f.gblk);
    y.R = (long long)a.N * a.c.G;
    auto all = [&](auto run) { return run(a, y, PrefixArgs{carry, gates, pws}, limit_ns, stream); };
    if (d == 64) return fox ? all(launch_all<64, true, A>) : all(launch_all<64, false, A>);
    return fox ? all(launch_all<128, true, A>) : all(launch_all<128, false, A>);
}

}  // namespace paged
}  // namespace path
