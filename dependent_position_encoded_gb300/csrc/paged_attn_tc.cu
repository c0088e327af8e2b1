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
#include <algorithm>

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

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// multiplies N fp32 columns of the thread's row by f (16 at a time: the row's logits are in
// registers beside it)
template <int N>
__device__ __forceinline__ void tmem_scale(uint32_t taddr, float f) {
#pragma unroll 1
    for (int c = 0; c < N; c += 16) {
        uint32_t u[16];
        tmem_ld16(taddr + c, u);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * f);
        tmem_st16(taddr + c, u);
    }
    tmem_st_wait();
}

// as fmax3, but NaN where an operand is
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

constexpr float kRescale = 8.f;  // the running maximum may lag by 2^8 before O is rescaled
// PaTH-FoX: how far (a power of two) below a row's maximum a weight counts for nothing, and how far
// above its gates a logit is not expected (only what is fetched early goes by that)
constexpr float kNothing = 64.f, kGuess = 32.f;

// ================================================================ cached keys
// Persistent: a CTA walks its stretches of units (paged_tc.cuh), each of them one item: NT tiles
// of 128 rows of one sequence and key head against consecutive key tiles of 128 positions. Keys
// and values stream through two rings of shared-memory slots (TMA, one box per page; a slot
// holds 128 rows of D bf16 in 128-byte-swizzled atoms of 64 columns), which run on from
// stretch to stretch, as every barrier's phase does. Per key tile and row tile: S = X K^T (N =
// 128) into TMEM, softmax by the 128 threads of a warpgroup, one row each, which write the
// weights as bf16 over S, and O += P V with the weights as the A operand in TMEM. With NT = 2
// the two row tiles share every slot and take turns on the tensor core, one in its softmax
// while the other multiplies.
//
// NT = 1 is for sequences whose rows fit one tile (a few tokens: bound by the cache's bytes)
// and updates the keys too: a second MMA forms K (P - I) with the loaded keys as the A operand
// (P - I split into two bf16 parts), and the second warpgroup adds it to the keys in shared
// memory and stores them back, so each key is read once and written once.
//
// With NT = 1 and at most 64 (32) rows, the tile holds two (four) copies of them and each copy's
// softmax takes a half (quarter) of the key tile's columns, with weights of 0 in the others: the
// warps share the row's softmax, and the copies' sums are parts to join like any others.
//
// Warps: 0-3 softmax of tile 0; 4-7 softmax of tile 1 (NT = 2) or the keys' update (NT = 1); 8
// allocates TMEM and issues the MMAs of S and P V; 11 those of the update (NT = 1); 9 and 10
// stream the key and the value pages. One thread issues both row tiles' MMAs: two of them, whose
// products mix on the tensor core, were a sixth slower (n = 32768, T = 2048, D = 128: 1,420 us a
// step against 1,200), and so were weights handed over in two halves (1,243).
// Positions past the sequence's n and those on bad pages: the streaming warp zeroes their rows
// after the copy, and the softmax masks them.
//
// NT = 1 is bound by the bytes of keys (read and written) and values: 194 us for 1.17 GB of them
// (32 sequences of up to 8,192, 16 heads, D = 64, one token each: 6.0 TB/s), 226 us for 1.2 GB (16
// of up to 16,384, 8 key heads of four query heads, D = 128, gates: 5.4 TB/s). NT = 2 by the
// tensor core: 976 us for 2,048 tokens of 32 heads against 32,768 keys at D = 128, a quarter of it
// the weights' second part (755 us and 1.46 PFLOP/s without; instructions take 77 to 85 cycles of the
// 64 that they need alone).
template <int NT, int D>
struct CachedCfg {
    static constexpr uint32_t tile = 128 * D * 2, atom = 128 * 128;
    // The rows' tiles, their high parts and then (keeps_low) their low ones; for NT = 1 at D = 128,
    // where the update's product takes 64 KB, they lie in tensor memory instead.
    static constexpr bool rows_in_tmem = NT == 1 && D == 128, low = keeps_low(NT, D);
    static constexpr uint32_t X = 0, xbytes = rows_in_tmem ? 0 : NT * (low ? 2 : 1) * tile;
    static constexpr uint32_t M = X + xbytes, mbytes = NT == 1 ? 2 * D * D * 2 : 0;
    // slots of keys and of values: what fits beside; for NT = 1 and D = 64 so that two CTAs share
    // an SM. With NT = 1 a key slot is held until the updated keys have left it.
    static constexpr int NK = NT == 1 ? (D == 64 ? 2 : 3) : (D == 64 ? 4 : 3);
    static constexpr int NV = NT == 1 ? 2 : (D == 64 ? 4 : 2);
    static constexpr uint32_t K = M + mbytes, V = K + NK * tile, bars = V + NV * tile;
    static constexpr int KF = 0, KE = NK, VF = 2 * NK, VE = VF + NV, XF = VE + NV, XE = XF + 1, SF = XE + 1,
                         PR = SF + 2, FIN = PR + 2, DF = FIN + 2, DE = DF + NK, TMP = DE + 1, END = TMP + 2,
                         XT = END + 2, count = XT + 1;
    static constexpr uint32_t bytes = bars + count * 8 + 16;  // from a 1024-byte boundary
    static constexpr int threads = 384;
    static constexpr int ctas_per_sm = NT == 1 && D == 64 ? 2 : 1;
    // registers after the split of what the CTA is launched with (NT = 2: 168 for each thread; NT = 1
    // with two CTAs per SM: 80): the softmax's warpgroups, the update's and the last one
    static constexpr bool split = NT == 2 || D == 64;
    static constexpr int reg_row = NT == 2 ? 200 : 104, reg_update = 72, reg_other = NT == 2 ? 104 : 64;
    // TMEM columns: per row tile S 128 (the weights over it) and O; NT = 1: the update's product
    static constexpr uint32_t cS = 0, cO = 128, per_tile = 256, cD = 128 + D, cX = 384;
    static constexpr uint32_t cols = NT == 1 && D == 64 ? 256 : 512;
};
static_assert(CachedCfg<1, 128>::bytes <= 227 * 1024 && CachedCfg<2, 128>::bytes <= 227 * 1024 &&
                  2 * (CachedCfg<1, 64>::bytes + 1024) <= 228 * 1024,
              "shared memory");
static_assert(256 * CachedCfg<2, 64>::reg_row + 128 * CachedCfg<2, 64>::reg_other <= 384 * 168, "registers");
static_assert(128 * (CachedCfg<1, 64>::reg_row + CachedCfg<1, 64>::reg_update + CachedCfg<1, 64>::reg_other) <= 384 * 80,
              "registers");

template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// A ring's running slot and the parity of its use.
template <int N>
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// How many of a key tile's 128 columns have the weights' second bf16 part (in the columns of the
// logits that the first leaves free): a weight's rounding is the largest error of an output, 1.4e-3 of
// the norm beside 1.66e-3 for the output's own, and for longer chunks the carried queries' and the
// scan's come to it. Behind 1,000 cached keys with T = 300, without and with the second part: D = 64
// 2.66e-3 and 2.18e-3; D = 128, where the tensor core bounds the pass, so that only half of the columns
// have it, 2.59e-3 and 2.37e-3 (a quarter: 2.48e-3). It costs 6% at D = 64 (one chunk of 512 in a
// batch of 32: 232 -> 246 us a step) and 20% of a long chunk at D = 128 (2,048 behind 32,768: 1,143 ->
// 1,370 us). NT = 1, whose queries have fewer steps behind them, stays at 2.2e-3 without; with
// gates few keys count: below 2.0e-3.
__host__ __device__ constexpr int low_weights(int NT, int D, bool fox) {
    return NT == 1 || fox ? 0 : D == 64 ? 128 : 64;
}

// Whether all boxes of a key tile lie on good pages below n: `have` one bit per box of
// 1 << box_shift rows.
__device__ __forceinline__ bool tile_whole(int pos0, int n, unsigned have, int box_shift) {
    return pos0 + 128 <= n && have == (1u << (128 >> box_shift)) - 1u;
}

template <int NT, int D, bool FOX>
__global__ void __launch_bounds__(CachedCfg<NT, D>::threads, CachedCfg<NT, D>::ctas_per_sm)
tc_cached_kernel(const Step a, const TcWs y, const __grid_constant__ CUtensorMap tm_x,
                 const __grid_constant__ CUtensorMap tm_l, const __grid_constant__ CUtensorMap tm_m,
                 const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, uint64_t limit_ns) {
    using L = CachedCfg<NT, D>;
    constexpr int NA = D / 64, NK = L::NK, NV = L::NV, kLow = low_weights(NT, D, FOX);
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t base = smem_u32(sm);
    auto bar = [&](int i) { return base + L::bars + 8u * (uint32_t)i; };
    uint32_t *const tslot = reinterpret_cast<uint32_t *>(sm + L::bars + 8 * L::count);
    volatile uint32_t *const abort_f = tslot + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = a.c.G;
    grid_begin();
    grid_wait();
    if (base & 1023u) {  // the swizzle's atoms need it; the kernel has no other shared memory
        report_status(a.status, kStatusTimeout);
        return;
    }
    const Plan plan = y.plan[NT - 1];
    const long long all = plan.units[a.c.seqs], per = plan_per(plan, a.c.seqs);
    const long long u_begin = (long long)blockIdx.x * per, u_end = u_begin + per < all ? u_begin + per : all;
    if (u_begin >= u_end) return;
    const Wait wait{abort_f, a.status, limit_ns};

    if (tid == 0) {
        *abort_f = 0u;
        // four warps: weights written, update's product read; both issuing threads (NT = 1): rows' tile
        // free, keys read by their products; both row tiles (NT = 2): keys and values read
        for (int i = 0; i < L::count; ++i) {
            const bool four = (i >= L::PR && i < L::FIN) || i == L::DE || i == L::XT;
            const bool both = NT == 1 ? (i == L::XE && !L::rows_in_tmem) || (i >= L::DF && i < L::DE)
                                      : (i >= L::KE && i < L::VF) || (i >= L::VE && i < L::XF);
            mbar_init(bar(i), four ? 4u : both ? 2u : 1u);
        }
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
    // Step j of the CTA (counted over all its stretches) uses key slot j % NK and value slot j % NV;
    // each ring has one producing warp, which waits for every release of its slots in turn.
    auto key_slot = [&](uint32_t j) { return base + L::K + (j % NK) * L::tile; };
    auto value_slot = [&](uint32_t j) { return base + L::V + (j % NV) * L::tile; };
    auto second = [&](const Stretch &t) { return NT == 2 && t.tile * 256 + 128 < t.s.T * G; };
    // log2 of the copies of the rows
    auto copies = [&](const Stretch &t) { return NT == 2 ? 0 : t.s.T * G <= 32 ? 2 : t.s.T * G <= 64 ? 1 : 0; };
    const int page = a.c.page, box_shift = min(a.c.page_shift, 7), box = 1 << box_shift, nbox = 128 >> box_shift;

    if (warp >= 8) {
        if (L::split) reg_dec<L::reg_other>();
        if (warp == 9 || warp == 10) {
            // ======================================================== pages into the ring
            const bool keys = warp == 9;
            const int *const table = keys ? a.c.k_table : a.c.v_table;
            const int npool = keys ? a.c.nk : a.c.nv;
            const uint32_t tmp = bar(L::TMP + (keys ? 0 : 1));
            const uint32_t ring = keys ? NK : NV, full0 = keys ? L::KF : L::VF, empty0 = keys ? L::KE : L::VE;
            uint32_t j = 0, seg = 0, tmp_phase = 0;
            bool ok = true;
            for (long long at = u_begin; ok && at < u_end; ++seg) {
                const Stretch t = stretch_at(a, plan, D, NT, at, u_end);
                at += t.steps;
                if (keys) {
                    // the rows' tile (and the update's product) once the last stretch's are read
                    if (seg > 0 && !(ok = wait.warp(bar(L::XE), (seg - 1) & 1))) break;
                    if (lane == 0) {
                        const int xr = t.s.first * G + 128 * NT * t.tile;
                        // boxes of 32 rows
                        const int nx = L::rows_in_tmem ? 0 : second(t) ? 8 : 4, parts = L::low ? 2 : 1;
                        const int mask = (128 * NT >> copies(t)) - 1;
                        mbar_arrive_expect_tx(bar(L::XF), nx * parts * (L::tile / 4) + L::mbytes);
                        for (int part = 0; part < parts; ++part)
                            for (int i = 0; i < nx; ++i)
                                for (int x = 0; x < NA; ++x)
                                    tma_load_3d(base + L::X + (part * NT + (i >> 2)) * L::tile + x * L::atom +
                                                    (i & 3) * 32 * 128,
                                                part ? &tm_l : &tm_x, bar(L::XF), 64 * x, xr + ((32 * i) & mask), t.h);
                        if (NT == 1)
                            for (int p = 0; p < 2; ++p)
                                for (int x = 0; x < NA; ++x)
                                    tma_load_3d(base + L::M + (uint32_t)(p * NA + x) * D * 128, &tm_m, bar(L::XF),
                                                64 * x, 0, ((int)mt_row(a, t.s, t.b) * a.c.Hkv + t.h) * 2 + p);
                    }
                }
                // lane i < nbox: the page of box i of a key tile, -1 past the end or where it is bad;
                // looked up one tile ahead
                int next;
                auto look_up = [&](int pos0) {
                    next = -1;
                    if (lane < nbox && pos0 + lane * box < t.s.n)
                        next = page_of(a, table, t.b, (pos0 + lane * box) >> a.c.page_shift, npool);
                };
                look_up(t.k0 * 128);
                for (int i = 0; ok && i < t.steps; ++i, ++j) {
                    const int pos0 = (t.k0 + i) * 128, id = next;
                    if (i + 1 < t.steps) look_up(pos0 + 128);
                    const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
                    const int valid = min(128, t.s.n - pos0);
                    const bool whole = tile_whole(pos0, t.s.n, have, box_shift);
                    const uint32_t sl = j % ring, turn = j / ring;
                    if (turn > 0 && !(ok = wait.warp(bar(empty0 + sl), (turn - 1) & 1))) break;
                    const uint32_t dst = keys ? key_slot(j) : value_slot(j);
                    const uint32_t full = bar(full0 + sl), target = whole ? full : tmp;
                    if (lane == 0) mbar_arrive_expect_tx(target, (uint32_t)__popc(have) * box * D * 2);
                    __syncwarp();
                    if (id >= 0)
#pragma unroll
                        for (int x = 0; x < NA; ++x)
                            tma_load_3d(dst + x * L::atom + lane * box * 128, keys ? &tm_k : &tm_v, target, 64 * x,
                                        (pos0 + lane * box) & (page - 1), id * a.c.Hkv + t.h);
                    if (!whole) {
                        // zero the rows that hold no cached position, then hand the slot on
                        if (!(ok = wait.warp(tmp, tmp_phase))) break;
                        tmp_phase ^= 1;
                        uint8_t *const rowp = sm + (dst - base);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int r = 32 * q + lane;
                            if (r < valid && ((have >> (r >> box_shift)) & 1u)) continue;
#pragma unroll
                            for (int x = 0; x < NA; ++x)
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    *reinterpret_cast<uint4 *>(rowp + x * L::atom + sw128_offset(r, c)) =
                                        make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full);
                    }
                }
            }
            // on an abort: no copy may land after the CTA is gone (those that may still be on their way
            // are the last ones of the ring's slots)
            if (!ok) {
                for (uint32_t v = j > ring ? j - ring : 0; v < j; ++v)
                    mbar_wait(bar(full0 + v % ring), (v / ring) & 1, limit_ns);
                if (keys) mbar_wait(bar(L::XF), seg & 1, limit_ns);
            }
        } else if (lane == 0 && warp == 8) {
            // ======================================================== S and P V
            // A lone thread's instructions follow each other slowly, and two tiles' MMAs keep the
            // tensor core busy only if little stands between them: slots and phases run along,
            // descriptors are sums.
            constexpr uint32_t ID_S = idesc_b16(128, 128, false), ID_O = idesc_b16(128, D, true);
            constexpr uint64_t kAtom = L::atom >> 4, kTile = L::tile >> 4;
            const uint64_t x_desc = sdesc_sw128(base + L::X, 16, 1024), k_desc = sdesc_sw128(base + L::K, 16, 1024),
                           v_desc = sdesc_sw128(base + L::V, L::atom, 1024);
            Ring<NK> k;
            Ring<NV> v;
            uint32_t seg = 0, parity[2] = {0, 0};
            bool ok = true;
            auto issue_s = [&](int q) {
                const uint64_t xd = x_desc + q * kTile, kd = k_desc + k.slot * kTile;
#pragma unroll
                for (int part = 0; part < (L::low ? 2 : 1); ++part)  // the rows' high and low parts
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t b = kd + (kk >> 2) * kAtom + 2 * (kk & 3);
                        if (L::rows_in_tmem)
                            umma_tA(tmem + L::cS, tmem + L::cX + part * (D / 2) + 8 * kk, b, ID_S, part > 0 || kk > 0);
                        else
                            umma_bf16(tmem + L::per_tile * q + L::cS,
                                      xd + part * NT * kTile + (kk >> 2) * kAtom + 2 * (kk & 3), b, ID_S,
                                      part > 0 || kk > 0);
                    }
                umma_commit(bar(L::SF + q));
            };
            auto issue_pv = [&](int q, bool first) {
                const uint64_t vd = v_desc + v.slot * kTile;
                const uint32_t tm = tmem + L::per_tile * q;
                umma_tA(tm + L::cO, tm + L::cS, vd, ID_O, !first);
#pragma unroll
                for (int kk = 1; kk < 8; ++kk) umma_tA(tm + L::cO, tm + L::cS + 8 * kk, vd + 128 * kk, ID_O, 1);
                if (kLow > 0)
#pragma unroll
                    for (int kk = 0; kk < kLow / 16; ++kk)
                        umma_tA(tm + L::cO, tm + L::cS + 64 + 8 * kk, vd + 128 * kk, ID_O, 1);
            };
            // behind the products of the ring's keys; last of a stretch: the rows' tile is free. (Slots are
            // handed back by the softmax's warps, which learn of the products' ends anyway.)
            auto after_s = [&](bool last) {
                if (NT == 1) umma_commit(bar(L::DF + k.slot));
                if (last && !L::rows_in_tmem) umma_commit(bar(L::XE));
                k.next();
            };
            for (long long at = u_begin; ok && at < u_end; ++seg) {
                const Stretch t = stretch_at(a, plan, D, NT, at, u_end);
                at += t.steps;
                const bool two = second(t);
                if (!(ok = wait(bar(L::rows_in_tmem ? L::XT : L::XF), seg & 1))) break;
                if (!(ok = wait(bar(L::KF + k.slot), k.phase))) break;
                tc_fence_after();
                issue_s(0);
                if (two) issue_s(1);
                after_s(t.steps == 1);
                for (int i = 0; i < t.steps; ++i) {
                    const bool more = i + 1 < t.steps;
                    if (!(ok = wait(bar(L::VF + v.slot), v.phase))) break;
                    if (!(ok = wait(bar(L::PR), parity[0]))) break;
                    tc_fence_after();
                    issue_pv(0, i == 0);
                    if (more) {
                        if (!(ok = wait(bar(L::KF + k.slot), k.phase))) break;
                        issue_s(0);
                    }
                    parity[0] ^= 1;
                    if (NT == 2 && two) {
                        if (!(ok = wait(bar(L::PR + 1), parity[1]))) break;
                        tc_fence_after();
                        issue_pv(1, i == 0);
                        if (more) issue_s(1);
                        parity[1] ^= 1;
                    }
                    v.next();
                    if (more) after_s(i + 2 == t.steps);
                }
                // a barrier per row tile: the second has a phase only where it has rows, so neither
                // can run ahead of the warps that wait for it
                umma_commit(bar(L::FIN));
                if (two) umma_commit(bar(L::FIN + 1));
            }
            // every product has completed before TMEM is freed
            umma_commit(bar(L::END));
            mbar_wait(bar(L::END), 0, limit_ns);
        } else if (NT == 1 && lane == 0 && warp == 11) {
            // ======================================================== K (P - I), NT = 1
            constexpr uint32_t ID_D = idesc_b16(128, D, true);
            constexpr uint64_t kAtom = L::atom >> 4, kTile = L::tile >> 4, kPart = (NA * D * 128) >> 4;
            const uint64_t k_desc = sdesc_sw128(base + L::K, 16, 1024), m_desc = sdesc_sw128(base + L::M, D * 128, 1024);
            Ring<NK> k;
            uint32_t j = 0, seg = 0;
            bool ok = true;
            for (long long at = u_begin; ok && at < u_end; ++seg) {
                const Stretch t = stretch_at(a, plan, D, NT, at, u_end);
                at += t.steps;
                if (!(ok = wait(bar(L::XF), seg & 1))) break;
                for (int i = 0; i < t.steps; ++i, ++j) {
                    if (!(ok = wait(bar(L::KF + k.slot), k.phase))) break;
                    if (j > 0 && !(ok = wait(bar(L::DE), (j - 1) & 1))) break;
                    tc_fence_after();
                    const uint64_t kd = k_desc + k.slot * kTile;  // the keys are the A operand
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            umma_bf16(tmem + L::cD, kd + (kk >> 2) * kAtom + 2 * (kk & 3), m_desc + p * kPart + 128 * kk,
                                      ID_D, p > 0 || kk > 0);
                    umma_commit(bar(L::DF + k.slot));
                    if (i + 1 == t.steps) umma_commit(bar(L::XE));
                    k.next();
                }
            }
            umma_commit(bar(L::END + 1));
            mbar_wait(bar(L::END + 1), 0, limit_ns);
        }
    } else if (NT == 1 && warp >= 4) {
        // ============================================================ the keys' update
        if (L::split) reg_dec<L::reg_update>();
        const int r = tid - 128;
        const uint32_t tm = tmem + ((uint32_t)(32 * (warp - 4)) << 16) + L::cD;
        bool ok = true;
        uint32_t j = 0;
        for (long long at = u_begin; ok && at < u_end;) {
            const Stretch t = stretch_at(a, plan, D, NT, at, u_end);
            at += t.steps;
            int next;  // the key pages of the next tile's boxes
            auto look_up = [&](int pos0) {
                next = -1;
                if (lane < nbox && pos0 + lane * box < t.s.n)
                    next = page_of(a, a.c.k_table, t.b, (pos0 + lane * box) >> a.c.page_shift, a.c.nk);
            };
            look_up(t.k0 * 128);
            for (int i = 0; i < t.steps; ++i, ++j) {
                const int pos0 = (t.k0 + i) * 128, id = next;
                if (i + 1 < t.steps) look_up(pos0 + 128);
                const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
                const bool whole = tile_whole(pos0, t.s.n, have, box_shift);
                const int mine = __shfl_sync(0xffffffffu, id, r >> box_shift);
                // the product is there, and the logits' product has read the keys too
                if (!(ok = wait.warp(bar(L::DF + j % NK), (j / NK) & 1))) break;
                tc_fence_after();
                uint8_t *const kt = sm + (key_slot(j) - base);
                bf *const dst = mine >= 0 && pos0 + r < t.s.n
                                    ? static_cast<bf *>(a.c.k_pages) +
                                          ((((size_t)mine * a.c.Hkv + t.h) << a.c.page_shift) +
                                           ((pos0 + r) & (page - 1))) * D
                                    : nullptr;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float x[32];
                    tld32(tm + c, x);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint4 *p4 =
                            reinterpret_cast<uint4 *>(kt + (c >> 6) * L::atom + sw128_offset(r, ((c & 63) >> 3) + q));
                        const uint4 k4 = *p4;
                        const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 k2 = unpack_bf16x2(w[e]);
                            o[e] = pack_bf16x2(k2.x + x[8 * q + 2 * e], k2.y + x[8 * q + 2 * e + 1]);
                        }
                        const uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
                        if (whole) *p4 = v;
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
                            tma_store_3d(&tm_k, key_slot(j) + x * L::atom + lane * box * 128, 64 * x,
                                         (pos0 + lane * box) & (page - 1), id * a.c.Hkv + t.h);
                        bulk_wait_read();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::KE + j % NK));
                }
            }
        }
        if (warp == 4) bulk_wait_all();
    } else {
        // ============================================================ softmax
        if (L::split) reg_inc<L::reg_row>();
        constexpr bool kTwice = NT == 1 || FOX;
        const int w = warp >> 2, r = tid & 127;  // row tile and row in it
        const uint32_t tm = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + L::per_tile * w;
        bool ok = true;
        // One thread of a row tile hands slots back: the logits' product of step j has read its keys, and
        // it ends behind the values' product of step j - 1. (NT = 1: the update's warps release keys.)
        const bool releases = (warp & 3) == 0 && lane == 0;
        uint32_t j = 0, seg = 0, step = 0;  // steps and stretches with rows in this tile; steps of the CTA
        for (long long at = u_begin; ok && at < u_end;) {
            const Stretch t = stretch_at(a, plan, D, NT, at, u_end);
            at += t.steps;
            if (w == 1 && !second(t)) {
                step += t.steps;
                continue;
            }
            const bool alone = NT == 2 && !second(t);  // no other tile: its part of the releases too
            // the row of this thread, and the columns of the key tiles that its copy takes
            const int rows_all = t.s.T * G, cp = copies(t), rw = r & ((128 >> cp) - 1);
            const int row0 = 128 * (NT * t.tile + w), cols = 128 >> cp, c_begin = (r >> (7 - cp)) * cols;
            const bool live = row0 + rw < rows_all, warp_live = row0 + (rw & ~31) < rows_all;
            const int hq = t.h * G + (live ? (row0 + rw) % G : 0);
            const float gq =
                FOX && live ? y.gq[(size_t)t.h * y.R + (size_t)t.s.first * G + row0 + rw] * kLog2e : 0.f;
            if (L::rows_in_tmem) {
                // the row's two parts (the last stretch's products have ended)
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int c = 0; c < D / 2; c += 32) {  // 32 columns of two elements
                        const uint4 *src = reinterpret_cast<const uint4 *>(
                            (part ? y.ql : y.qt) +
                            ((size_t)t.h * y.R + (size_t)t.s.first * G + row0 + (live ? rw : 0)) * D + 2 * c);
                        uint32_t u[32];
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint4 v = live ? src[q] : make_uint4(0u, 0u, 0u, 0u);
                            u[4 * q] = v.x;
                            u[4 * q + 1] = v.y;
                            u[4 * q + 2] = v.z;
                            u[4 * q + 3] = v.w;
                        }
                        tmem_st32(tm + L::cX + part * (D / 2) + c, u);
                    }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive_warp(bar(L::XT));
            }
            float m_run = -INFINITY, l_run = 0.f;
            int kid1, vid1;  // the pages of the next tile's boxes
            auto look_up = [&](int pos0) {
                kid1 = vid1 = -1;
                if (lane < nbox && pos0 + lane * box < t.s.n) {
                    const size_t e = (size_t)t.b * a.c.max_pages + ((pos0 + lane * box) >> a.c.page_shift);
                    kid1 = __ldg(a.c.k_table + e);
                    vid1 = __ldg(a.c.v_table + e);
                }
            };
            look_up(t.k0 * 128);
            auto release = [&](int empty, uint32_t slot) {
                mbar_arrive(bar(empty + slot));
                if (alone) mbar_arrive(bar(empty + slot));
            };
            for (int i = 0; i < t.steps; ++i, ++j, ++step) {
                const int pos0 = (t.k0 + i) * 128, id = kid1;
                const bool good = (unsigned)id < (unsigned)a.c.nk && (unsigned)vid1 < (unsigned)a.c.nv;
                if (i + 1 < t.steps) look_up(pos0 + 128);
                const unsigned have = __ballot_sync(0xffffffffu, good);
                const int valid = min(128, t.s.n - pos0);
                const bool whole = tile_whole(pos0, t.s.n, have, box_shift);
                // gate sums of 32 keys from column c for the row's query head
                auto gates_of = [&](int c, float4 *v) {
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {  // 16 positions lie in one page
                        const int bx = (c + 4 * e) >> box_shift;
                        const int pid = __shfl_sync(0xffffffffu, id, bx);
                        const bool in = (have >> bx) & 1u;
                        const float4 *gp = reinterpret_cast<const float4 *>(
                            a.c.g_pages + (((size_t)(in ? pid : 0) * a.c.Hq + hq) << a.c.page_shift) +
                            ((pos0 + c + 4 * e) & (page - 1)));
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[e + q] = in ? gp[q] : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                };
                // on their way while the product runs: in registers where there are enough for the 32
                // columns of a copy, else into L1
                constexpr bool kAhead = FOX && NT == 1 && D == 128;
                float4 ahead[kAhead ? 8 : 1];
                const bool early = kAhead && cols == 32;
                if (early) {
                    gates_of(c_begin, ahead);
                } else if (FOX) {
#pragma unroll 1
                    for (int c = c_begin; c < c_begin + cols; c += 16) {
                        const int bx = c >> box_shift, pid = __shfl_sync(0xffffffffu, id, bx);
                        if ((have >> bx) & 1u)
                            asm volatile("prefetch.global.L1 [%0];" ::"l"(
                                a.c.g_pages + (((size_t)pid * a.c.Hq + hq) << a.c.page_shift) +
                                ((pos0 + c) & (page - 1))));
                    }
                }
                if (!(ok = wait.warp(bar(L::SF + w), j & 1))) break;
                tc_fence_after();
                if (releases) {
                    if (NT == 2) release(L::KE, step % NK);
                    if (i > 0) release(L::VE, (step - 1) % NV);
                }
                if (warp_live) {
                    // gates and mask of 32 logits of the row from column c
                    auto gate = [&](int c, float *x) {
                        if (FOX) {
                            float4 own[8];
                            if (!early) gates_of(c, own);
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float4 g4 = early ? ahead[kAhead ? q : 0] : own[q];
                                float *v = x + 4 * q;
                                v[0] = fmaf(g4.x, kLog2e, v[0] + gq);
                                v[1] = fmaf(g4.y, kLog2e, v[1] + gq);
                                v[2] = fmaf(g4.z, kLog2e, v[2] + gq);
                                v[3] = fmaf(g4.w, kLog2e, v[3] + gq);
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
                    float top;
                    auto max32 = [&](const float *v) {
                        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                        for (int e = 4; e < 28; e += 8)
#pragma unroll
                            for (int q = 0; q < 4; ++q) mx[q] = fmax3(mx[q], v[e + 2 * q], v[e + 2 * q + 1]);
                        return fmax3(fmax3(mx[0], mx[1], mx[2]), mx[3], fmax3(fmaxf(v[28], v[29]), v[30], v[31]));
                    };
                    // the running maximum of the row; O follows it when it has risen by 2^8. (S of this
                    // step is complete, so the previous P V is too.)
                    float use;
                    auto raise = [&]() {
                        float alpha = 1.f;
                        if (top > m_run + kRescale || (m_run == -INFINITY && top > -INFINITY)) {
                            alpha = m_run == -INFINITY ? 0.f : ex2_approx(m_run - top);
                            m_run = top;
                        }
                        const bool resc = alpha != 1.f && l_run > 0.f;
                        if (__any_sync(0xffffffffu, resc)) tmem_scale<D>(tm + L::cO, resc ? alpha : 1.f);
                        l_run *= alpha;
                        use = m_run == -INFINITY ? 0.f : -m_run;
                    };
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    // 32 weights as 16 bf16 pairs, and what the rounding left as others
                    auto weigh = [&](const float *v, uint32_t *p, uint32_t *low, bool both) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 z = fadd2(make_float2(v[e], v[e + 1]), make_float2(use, use));
                            const float2 q = make_float2(ex2_approx(z.x), ex2_approx(z.y));
                            sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], q);
                            if (both) split2(q.x, q.y, p[e / 2], low[e / 2]);
                            else p[e / 2] = pack_bf16x2(q.x, q.y);
                        }
                    };
                    if (kTwice) {
                        // registers are short: the logits of more than 32 columns are read twice. The
                        // weights of columns c .. c + 31 take the 16 columns from c / 2, whose logits
                        // have been read or are another copy's
                        float x[32];
                        top = -INFINITY;
#pragma unroll 1
                        for (int c = c_begin; c < c_begin + cols; c += 32) {
                            tld32(tm + L::cS + c, x);
                            gate(c, x);
                            top = fmaxf(top, max32(x));
                        }
                        raise();
                        uint32_t p[16];
#pragma unroll 1
                        for (int c = c_begin; c < c_begin + cols; c += 32) {
                            if (cols > 32) {
                                tld32(tm + L::cS + c, x);
                                gate(c, x);
                            }
                            weigh(x, p, p, false);
                            tmem_st16(tm + L::cS + c / 2, p);
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) p[e] = 0u;
#pragma unroll 1
                        for (int c = 0; c < 128; c += 32)
                            if (c < c_begin || c >= c_begin + cols) tmem_st16(tm + L::cS + c / 2, p);
                    } else {
                        float x[128];
                        uint32_t(*u)[32] = reinterpret_cast<uint32_t(*)[32]>(x);
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld32(tm + L::cS + 32 * c, u[c]);
                        tmem_ld_wait();
                        float mx[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            gate(32 * c, x + 32 * c);
                            mx[c] = max32(x + 32 * c);
                        }
                        top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        raise();
#pragma unroll
                        for (int c = 0; c < 128; c += 32) {
                            uint32_t p[16], l[16];
                            weigh(x + c, p, l, c < kLow);
                            tmem_st16(tm + L::cS + c / 2, p);
                            if (c < kLow) tmem_st16(tm + L::cS + 64 + c / 2, l);
                        }
                    }
                    l_run += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tmem_st_wait();
                }
                tc_fence_before();
                mbar_arrive_warp(bar(L::PR + w));
            }
            if (!ok || !(ok = wait.warp(bar(L::FIN + w), seg & 1))) break;
            ++seg;
            tc_fence_after();
            if (releases) release(L::VE, (step - 1) % NV);
            if (warp_live) {
                // the part's place: its CTA and item; a row whose keys were all absent leaves a sum of 0
                const size_t e = ((size_t)(blockIdx.x + t.item) * NT + w) * 128 + r;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tld32(tm + L::cO + c, o);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint4 u[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            u[i] = make_uint4(__float_as_uint(o[16 * q + 4 * i]), __float_as_uint(o[16 * q + 4 * i + 1]),
                                              __float_as_uint(o[16 * q + 4 * i + 2]),
                                              __float_as_uint(o[16 * q + 4 * i + 3]));
                        store_quad_rows(u, [&](int i) {
                            return row0 + (rw & ~3) + i < rows_all
                                       ? y.so[NT - 1] + (e - (r & 3) + i) * D + c + 16 * q
                                       : nullptr;
                        });
                    }
                }
                if (live) y.sml[NT - 1][e] = make_float2(m_run, l_run);
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, L::cols);
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

template <int D, bool FOX>
__global__ void __launch_bounds__(kScanThr, D == 64 ? 2 : 1)
tc_scan_kernel(const Step a, const TcWs y, const __grid_constant__ CUtensorMap tm_r,
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
        const bool low = keeps_low(one_tile(s.T, G, D, FOX) ? 1 : 2, D);  // of what goes on to the cached keys
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
    CUtensorMap tx, tl, tm, tk, tv;
    // a map has no empty axis; of an empty pool nothing is loaded, every page number is outside it
    auto heads = [&](int pages) { return (long long)std::max(pages, 1) * a.c.Hkv; };
    if (!make_map(&tx, y.qt, D, y.R, a.c.Hkv, 32) || !make_map(&tl, y.ql, D, y.R, a.c.Hkv, 32) ||
        !make_map(&tm, y.mt, D, D, (long long)std::min(a.c.seqs, a.N) * a.c.Hkv * 2, D) ||
        !make_map(&tk, a.c.k_pages, D, a.c.page, heads(a.c.nk), a.c.page < 128 ? a.c.page : 128) ||
        !make_map(&tv, a.c.v_pages, D, a.c.page, heads(a.c.nv), a.c.page < 128 ? a.c.page : 128))
        return cudaErrorInvalidValue;
    using L = CachedCfg<NT, D>;
    auto kern = tc_cached_kernel<NT, D, FOX>;
    const cudaError_t e = big_smem(kern, L::bytes);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3(y.plan[NT - 1].ctas), L::threads, L::bytes, stream, false, a, y, tx, tl, tm, tk, tv,
                  limit_ns);
}

template <int D, bool FOX>
cudaError_t launch_scan(const Step &a, const TcWs &y, uint64_t limit_ns, cudaStream_t stream) {
    CUtensorMap tr, tl, tv;
    const long long heads = (long long)slots_of(a.N, a.c.seqs) * a.c.Hkv;
    if (!make_map(&tr, y.kh, D, 64 + D, heads, 64 + D) || !make_map(&tl, y.kl, D, 64 + D, heads, D) ||
        !make_map(&tv, y.vb, D, 64, heads, 64))
        return cudaErrorInvalidValue;
    using L = ScanSmem<D, scan_low(D, FOX)>;
    auto kern = tc_scan_kernel<D, FOX>;
    const cudaError_t e = big_smem(kern, L::alloc);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3(tile_slots(a.N, a.c.G, a.c.seqs, 128) * a.c.Hkv), kScanThr, L::alloc, stream, false, a, y,
                  tr, tl, tv, limit_ns);
}

}  // namespace

template <int D>
cudaError_t launch_tc_prep(const Step &a, const TcWs &y, cudaStream_t stream);
template <int D>
cudaError_t launch_tc_carry(const Step &a, const TcWs &y, cudaStream_t stream);
template <int D>
cudaError_t launch_tc_finish(const Step &a, const TcWs &y, cudaStream_t stream);

namespace {

template <int D, bool FOX>
cudaError_t launch_all(const Step &a, const TcWs &y, uint64_t limit_ns, cudaStream_t stream) {
    cudaError_t e = launch_tc_prep<D>(a, y, stream);
    if (a.max_chunk > kC) {
        if (e == cudaSuccess) e = launch_tc_carry<D>(a, y, stream);
        if (e == cudaSuccess) e = launch_scan<D, FOX>(a, y, limit_ns, stream);
    }
    if (a.c.max_pages > 0) {
        if (e == cudaSuccess) e = launch_cached<1, D, FOX>(a, y, limit_ns, stream);
        if (e == cudaSuccess && !one_tile(a.max_chunk, a.c.G, D, FOX))
            e = launch_cached<2, D, FOX>(a, y, limit_ns, stream);
    }
    if (e == cudaSuccess) e = launch_tc_finish<D>(a, y, stream);
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
        y.ctas[p] = 152 * (p == 0 && d == 64 ? CachedCfg<1, 64>::ctas_per_sm : 1);
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

size_t tc_ws_bytes(const Cache &c, int N, int max_chunk, int d, bool fox) {
    return tc_layout(c, N, max_chunk, d, fox).total;
}

cudaError_t launch_tc(const Step &a, int d, void *ws, uint64_t limit_ns, cudaStream_t stream) {
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
    if (d == 64)
        return fox ? launch_all<64, true>(a, y, limit_ns, stream) : launch_all<64, false>(a, y, limit_ns, stream);
    return fox ? launch_all<128, true>(a, y, limit_ns, stream) : launch_all<128, false>(a, y, limit_ns, stream);
}

}  // namespace paged
}  // namespace path
