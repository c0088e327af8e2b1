// Helpers of the kernels of paged_attn_tc.cuh, and the pass of carried queries over cached keys, whose
// forms (paged_tc.cuh, Pass) are compiled in files of their own.
#pragma once

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

// `bytes` (a multiple of 16) of global memory into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Waits until all committed stores but the last N have finished reading shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read_but() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
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
// query heads of a key head whose gates come through a ring in shared memory; of more they are read in place
constexpr int kGateHeads = 8;

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
// memory and stores them back, so each key is read once and written once. That is the pass of a
// plain step and, over the key tiles in sight, of one through a window (Pass::step, window). Two more
// have an NT = 1 of their own, whose rows lie in TMEM and come while the stretch before ends:
//
// Pass::one, steps of single tokens through a window or behind prefixes. P - I is -beta w w^T, so the
// second warpgroup forms -beta (w . k) w itself, a thread to a key: no product in TMEM and no P - I in
// shared memory. The room goes to a second place for S, so that a tile's logits wait for the softmax and
// not it for them, and (D = 64) to rings of eight and five slots; a key slot is given back a step after
// its store was issued. 64 sequences, W = 4,096, 16 heads, D = 64: 219 us, 5.8 TB/s (with the product, two
// CTAs an SM: 234, and 15 to prepare it where this takes 7); 16, W = 2,048, 8 key heads of four query heads,
// D = 128, gates: the whole step 69 (with the product 81). Plain steps keep the product, and with it their
// results to the bit.
//
// Pass::shared, the read-only pass over a prefix's keys. At D = 64 two CTAs share an SM; at D = 128, where
// the slots leave room for one, two warpgroups share a row tile's softmax, half the columns each (they meet
// once for the row's maximum and once before a half's weights cover the other's logits), with two places
// for S: 4 prefixes of up to 16,384, 8 key heads of four query heads, gates, D = 128, 16 single tokens
// behind each: 61 us, 3.6 TB/s (one warpgroup and one place: 78, this then 64); at D = 64 the halves' meetings cost more
// than they give (32 tokens behind 8,192 keys of 16 heads: 18 us, with halves 19).
//
// With gates these two take them from a ring in shared memory that a warp fills (183 us -> 176 for the
// whole step of the 4 prefixes); where more than kGateHeads query heads share a key head, kernels
// compiled apart read them in place. The softmax is then bound not by bytes but by its instructions' way to
// the SM, which four roles of straight code do not hold near (no instruction there: the largest stall, 1.9
// cycles an issue): 325 us where the same pass without gates takes 218 (64 sequences, W = 4,096, 16 key
// heads of four query heads, D = 64). So less code is faster code: one way of reading gates in a kernel and
// the update's loops unrolled twice (four times without gates) took the whole step from 72 us to 69 (16
// sequences, W = 2,048, D = 128) and the 4 prefixes from 165 to 162.5. Deeper rings, gates a tile ahead
// and rows padded against bank conflicts changed nothing.
//
// With NT = 1 and at most 64 (32) rows, the tile holds two (four) copies of them and each copy's
// softmax takes a half (quarter) of the key tile's columns, with weights of 0 in the others: the
// warps share the row's softmax, and the copies' sums are parts to join like any others.
//
// Warps: 0-3 softmax of tile 0; 4-7 softmax of tile 1 (NT = 2), the keys' update (NT = 1) or the
// softmax's second half (shared keys at D = 128; at D = 64 they have none, and the others follow from
// 4); 8 allocates TMEM and issues the MMAs of S and P V; 11 those of the update, or fills the ring
// of gates; 9 and 10 stream the key and the value pages. One thread issues both row tiles' MMAs: two
// of them, whose products mix on the tensor core, were a sixth slower (n = 32768, T = 2048, D = 128:
// 1,420 us a step against 1,200), and so were weights handed over in two halves (1,243).
// Positions past the sequence's n and those on bad pages: the streaming warp zeroes their rows
// after the copy, and the softmax masks them.
//
// NT = 1 of a plain step is bound by the bytes of keys (read and written) and values: 194 us for
// 1.17 GB of them (32 sequences of up to 8,192, 16 heads, D = 64, one token each: 6.0 TB/s), 226 us
// for 1.2 GB (16 of up to 16,384, 8 key heads of four query heads, D = 128, gates: 5.4 TB/s). NT = 2 by the
// tensor core: 976 us for 2,048 tokens of 32 heads against 32,768 keys at D = 128, a quarter of it
// the weights' second part (755 us and 1.46 PFLOP/s without; instructions take 77 to 85 cycles of the
// 64 that they need alone).
template <int NT, int D, Pass M, bool FOX, bool RING = FOX && NT == 1 && (M == Pass::one || M == Pass::shared)>
struct CachedCfg {
    static constexpr uint32_t tile = 128 * D * 2, atom = 128 * 128;
    // the keys' update in this pass: by a product with P - I, or (single tokens) on the CUDA cores
    static constexpr bool update = NT == 1 && M != Pass::shared, single = NT == 1 && M == Pass::one,
                          matrix = update && !single;
    // shared keys at D = 128: two warpgroups for the softmax of one row tile; and, as for single tokens, two
    // places for its logits, so that the next step's product runs beside it. (Else at D = 64 two CTAs run
    // beside each other instead.)
    static constexpr bool duo = NT == 1 && D == 128 && M == Pass::shared, two_s = duo || single;
    // the next stretch is looked up, and its rows fetched, before the last one's end
    static constexpr bool ahead = NT == 1 && !matrix;
    // single tokens at D = 64: the thread's key stays in registers between its product with w and its update.
    // At D = 128 and with gates it is read from its slot again: the softmax's threads have no more registers
    // than these. (64 sequences, W = 4,096, 16 heads, D = 64: 228 us a step held, 272 read again; with gates
    // and four query heads to a key head: 441 and 375. 16 sequences, W = 2,048, 8 key heads of four query
    // heads, D = 128: 60 and 56, with gates 81 and 71.)
    static constexpr bool held = single && D == 64 && !FOX;
    // gates come through a ring of their own, of up to kGateHeads query heads
    static constexpr bool ring = RING;
    static_assert(!RING || (FOX && ahead), "a ring of gates");
    // The rows' tiles, their high parts and then (keeps_low) their low ones, in shared memory, or in tensor
    // memory: where the update's product takes 64 KB (D = 128), and where they come ahead.
    static constexpr bool rows_in_tmem = ahead || (update && D == 128), low = keeps_low(NT, D);
    static constexpr uint32_t X = 0, xbytes = rows_in_tmem ? 0 : NT * (low ? 2 : 1) * tile;
    static constexpr uint32_t P = X + xbytes, pbytes = matrix ? 2 * D * D * 2 : 0;
    // slots of keys and of values: what fits beside; for NT = 1 and D = 64 (but for single tokens) so that
    // two CTAs share an SM. A key slot is held until the updated keys have left it.
    static constexpr int NK = matrix ? (D == 64 ? 2 : 3)
                              : NT == 2 ? (D == 64 ? 4 : 3)
                                        : (single && D == 64 ? 8 : 4) - (ring ? 1 : 0);
    static constexpr int NV = matrix ? 2 : NT == 2 ? (D == 64 ? 4 : 2) : single && D == 64 ? 5 : 3;
    static constexpr int NG = ring ? (single || D == 128 ? 4 : 3) : 0, NG_ = ring ? NG : 1;
    static constexpr uint32_t K = P + pbytes, V = K + NK * tile, bars = V + NV * tile;
    static constexpr int KF = 0, KE = NK, VF = 2 * NK, VE = VF + NV, XF = VE + NV, XE = XF + 1, SF = XE + 1,
                         PR = SF + 2, FIN = PR + 2, DF = FIN + 2, DE = DF + NK, TMP = DE + 1, END = TMP + 2,
                         XT = END + 2, EX = XT + 1, PD = EX + 1, GF = PD + 1, GE = GF + NG, count = GE + NG;
    // behind the barriers: TMEM's address and the abort flag; single: the token's w, two of them; duo: what the
    // halves of a row tell each other, two turns of it; the ring of gates
    static constexpr uint32_t W = (bars + count * 8 + 16 + 15) / 16 * 16;  // read 16 bytes at a time
    static constexpr uint32_t gates = W + (single ? 2 * D * 4 : duo ? 2 * 256 * 4 : 0), gslot = kGateHeads * 128 * 4;
    static constexpr uint32_t bytes = gates + NG * gslot;  // from a 1024-byte boundary
    // warps: those of the rows, the update's, then the others from `other` on
    static constexpr int other = update || duo || NT == 2 ? 8 : 4, threads = 32 * (other + 4);
    static constexpr int ctas_per_sm = NT == 1 && D == 64 && !single ? 2 : 1;
    // registers after the split of what the CTA is launched with (NT = 2: 168 for each thread; NT = 1
    // with two CTAs per SM: 80): the softmax's warpgroups, the update's and the last one. A window's pass of
    // NT = 1 goes without: a form of it that held more across its steps raised an illegal address whose cause
    // nobody found, and so had one of the plain step's, both with this split. Its softmax spills instead (64
    // streams of 4 tokens, W = 4,096, 16 heads: 361 -> 367 us a step; 32 with gates and four query heads to a
    // key head 148 -> 182).
    static constexpr bool split = NT == 2 || (matrix && D == 64 && M == Pass::step);
    static constexpr int reg_row = NT == 2 ? 200 : 104, reg_update = 72, reg_other = NT == 2 ? 104 : 64;
    // TMEM columns: per row tile S 128 (the weights over it) and O; NT = 1: the update's product, or the
    // rows' two parts
    static constexpr uint32_t cS = 0, cO = 128, per_tile = 256, cD = 128 + D, cX = D == 64 ? 192 : 384;
    static constexpr uint32_t cS2 = 256;  // two_s: the odd steps' logits and weights
    static constexpr uint32_t cols = NT == 1 && D == 64 && !single ? 256 : 512;
};
template <Pass M, bool FOX, bool RING = FOX>
struct CachedFits {
    using A = CachedCfg<1, 64, M, FOX, RING>;
    using B = CachedCfg<2, 64, M, FOX>;
    static_assert(CachedCfg<1, 128, M, FOX, RING>::bytes <= 227 * 1024 && CachedCfg<2, 128, M, FOX>::bytes <= 227 * 1024 &&
                      A::bytes <= 227 * 1024 && A::ctas_per_sm * (A::bytes + 1024) <= 228 * 1024,
                  "shared memory");
    static_assert(256 * B::reg_row + 128 * B::reg_other <= 384 * 168, "registers");
    static_assert(128 * (A::reg_row + A::reg_update + A::reg_other) <= 384 * 80, "registers");
};
template struct CachedFits<Pass::step, false>;
template struct CachedFits<Pass::one, false>;
template struct CachedFits<Pass::one, true>;
template struct CachedFits<Pass::one, true, false>;
template struct CachedFits<Pass::shared, false>;
template struct CachedFits<Pass::shared, true>;
template struct CachedFits<Pass::shared, true, false>;

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
// A window's pass at D = 128 has it for three quarters: behind a window of thousands a half leaves 2.51e-3
// in chunks of 64 and of 100 tokens (W = 12,000), three quarters 2.40e-3 (two chunks of up to 1,024, W = 4,096: the
// whole step 396 -> 406 us).
__host__ __device__ constexpr int low_weights(int NT, int D, bool fox, Pass M) {
    return NT == 1 || fox ? 0 : D == 64 ? 128 : M == Pass::window ? 96 : 64;
}

// Whether all boxes of a key tile lie on good pages below n: `have` one bit per box of
// 1 << box_shift rows.
__device__ __forceinline__ bool tile_whole(int pos0, int n, unsigned have, int box_shift) {
    return pos0 + 128 <= n && have == (1u << (128 >> box_shift)) - 1u;
}

template <int NT, int D, bool FOX, Pass M, bool RING>
__global__ void __launch_bounds__(CachedCfg<NT, D, M, FOX, RING>::threads, CachedCfg<NT, D, M, FOX, RING>::ctas_per_sm)
tc_cached_kernel(const StepOf<M> a, const TcWs y, const __grid_constant__ CUtensorMap tm_x,
                 const __grid_constant__ CUtensorMap tm_l, const __grid_constant__ CUtensorMap tm_m,
                 const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, uint64_t limit_ns) {
    using L = CachedCfg<NT, D, M, FOX, RING>;
    constexpr bool WIN = M == Pass::window || M == Pass::one;
    constexpr int NA = D / 64, NK = L::NK, NV = L::NV, kLow = low_weights(NT, D, FOX, M);
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
        // four warps (duo: eight): weights written, update's product read; both issuing threads (NT = 1):
        // rows' tile free, keys read by their products; both row tiles (NT = 2): keys and values read
        for (int i = 0; i < L::count; ++i) {
            const bool four = (i >= L::PR && i < L::FIN) || i == L::DE || i == L::XT || i == L::EX || i >= L::GE;
            const bool both = NT == 1 ? L::matrix && ((i == L::XE && !L::rows_in_tmem) || (i >= L::DF && i < L::DE))
                                      : (i >= L::KE && i < L::VF) || (i >= L::VE && i < L::XF);
            mbar_init(bar(i), four ? (L::duo && i != L::XT ? 8u : 4u) : both ? 2u : 1u);
        }
        fence_mbar_init();
    }
    if (warp == L::other) {
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
    auto stretch_of = [&](Walk &walk, long long at) {
        return L::ahead ? walk.at(a, plan, D, NT, at, u_end) : Walk().at(a, plan, D, NT, at, u_end);
    };
    const int window = window_of(a), sinks = sinks_of(a);
    // what the first new token sees, the first position of a stretch's step i, and whether the page of
    // the lane's box at j is wanted
    auto sight = [&](const Stretch &t) { return sight_of(a, t.s); };
    // (gates, but for a plain step: from the last tile to the first, since a row's maximum then comes early
    // and its sums seldom have to follow it)
    auto pos_of = [&](const Stretch &t, const Sight &seen, int i) {
        const int tile = FOX && M != Pass::step ? t.kt - 1 - t.k0 - i : t.k0 + i;
        return 128 * (WIN ? seen.tile(tile, t.s.n, 128) : tile);
    };
    auto box_in = [&](const Stretch &t, const Sight &seen, int j) {
        return lane < nbox && j < t.s.n && (!WIN || seen.any(j, box));
    };

    if (warp >= L::other) {
        if (L::split) reg_dec<L::reg_other>();
        if (warp == L::other + 1 || warp == L::other + 2) {
            // ======================================================== pages into the ring
            const bool keys = warp == L::other + 1;
            const int *const table = keys ? a.c.k_table : a.c.v_table;
            const int npool = keys ? a.c.nk : a.c.nv;
            const uint32_t tmp = bar(L::TMP + (keys ? 0 : 1));
            const uint32_t ring = keys ? NK : NV, full0 = keys ? L::KF : L::VF, empty0 = keys ? L::KE : L::VE;
            uint32_t j = 0, seg = 0, tmp_phase = 0;
            bool ok = true;
            Walk walk;
            for (long long at = u_begin; ok && at < u_end; ++seg) {
                const Stretch t = stretch_of(walk, at);
                at += t.steps;
                if (keys && !L::ahead) {
                    // the rows' tile (and the update's product) once the last stretch's are read
                    if (seg > 0 && !(ok = wait.warp(bar(L::XE), (seg - 1) & 1))) break;
                    if (lane == 0) {
                        const int xr = t.s.first * G + 128 * NT * t.tile;
                        // boxes of 32 rows
                        const int nx = L::rows_in_tmem ? 0 : second(t) ? 8 : 4, parts = L::low ? 2 : 1;
                        const int mask = (128 * NT >> copies(t)) - 1;
                        mbar_arrive_expect_tx(bar(L::XF), nx * parts * (L::tile / 4) + L::pbytes);
                        for (int part = 0; part < parts; ++part)
                            for (int i = 0; i < nx; ++i)
                                for (int x = 0; x < NA; ++x)
                                    tma_load_3d(base + L::X + (part * NT + (i >> 2)) * L::tile + x * L::atom +
                                                    (i & 3) * 32 * 128,
                                                part ? &tm_l : &tm_x, bar(L::XF), 64 * x, xr + ((32 * i) & mask), t.h);
                        if (L::matrix)
                            for (int p = 0; p < 2; ++p)
                                for (int x = 0; x < NA; ++x)
                                    tma_load_3d(base + L::P + (uint32_t)(p * NA + x) * D * 128, &tm_m, bar(L::XF),
                                                64 * x, 0, ((int)mt_row(a, t.s, t.b) * a.c.Hkv + t.h) * 2 + p);
                    }
                }
                // lane i < nbox: the page of box i of a key tile, -1 past the end or where it is bad;
                // looked up one tile ahead
                const Sight seen = sight(t);
                int next;
                auto look_up = [&](int pos0) {
                    next = -1;
                    if (box_in(t, seen, pos0 + lane * box))
                        next = page_of(a, table, t.b, (pos0 + lane * box) >> a.c.page_shift, npool);
                };
                look_up(pos_of(t, seen, 0));
                for (int i = 0; ok && i < t.steps; ++i, ++j) {
                    const int pos0 = pos_of(t, seen, i), id = next;
                    if (i + 1 < t.steps) look_up(pos_of(t, seen, i + 1));
                    const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
                    const int valid = min(128, t.s.n - pos0);
                    const bool whole = tile_whole(pos0, t.s.n, have, box_shift) && (!WIN || seen.all(pos0, 128));
                    const uint32_t sl = j % ring, turn = j / ring;
                    if (turn > 0 && !(ok = wait.warp(bar(empty0 + sl), (turn - 1) & 1))) break;
                    const uint32_t dst = keys ? key_slot(j) : value_slot(j);
                    // (ahead: keys that are none need not be zero, their logits are masked and nothing of them
                    // is written)
                    const bool direct = whole || (L::ahead && keys);
                    const uint32_t full = bar(full0 + sl), target = direct ? full : tmp;
                    if (lane == 0) mbar_arrive_expect_tx(target, (uint32_t)__popc(have) * box * D * 2);
                    __syncwarp();
                    if (id >= 0)
#pragma unroll
                        for (int x = 0; x < NA; ++x)
                            tma_load_3d(dst + x * L::atom + lane * box * 128, keys ? &tm_k : &tm_v, target, 64 * x,
                                        (pos0 + lane * box) & (page - 1), id * a.c.Hkv + t.h);
                    if (!direct) {
                        // zero the rows that hold no cached position or one that no new token sees, then
                        // hand the slot on
                        if (!(ok = wait.warp(tmp, tmp_phase))) break;
                        tmp_phase ^= 1;
                        uint8_t *const rowp = sm + (dst - base);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int r = 32 * q + lane;
                            if (r < valid && ((have >> (r >> box_shift)) & 1u) && (!WIN || seen.sees(pos0 + r)))
                                continue;
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
                if (keys && !L::ahead) mbar_wait(bar(L::XF), seg & 1, limit_ns);
            }
        } else if (lane == 0 && warp == L::other) {
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
            uint32_t seg = 0, parity[2] = {0, 0}, turns = 0;  // (turns: the same bits, by place)
            bool ok = true;
            auto issue_s = [&](int q) {  // of row tile q (two_s: into place q)
                const uint64_t xd = x_desc + (L::two_s ? 0 : q) * kTile, kd = k_desc + k.slot * kTile;
#pragma unroll
                for (int part = 0; part < (L::low ? 2 : 1); ++part)  // the rows' high and low parts
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t b = kd + (kk >> 2) * kAtom + 2 * (kk & 3);
                        if (L::rows_in_tmem)
                            umma_tA(tmem + L::cS + (L::two_s ? L::cS2 * q : 0), tmem + L::cX + part * (D / 2) + 8 * kk,
                                    b, ID_S, part > 0 || kk > 0);
                        else
                            umma_bf16(tmem + (L::two_s ? L::cS2 : L::per_tile) * q + L::cS,
                                      xd + part * NT * kTile + (kk >> 2) * kAtom + 2 * (kk & 3), b, ID_S,
                                      part > 0 || kk > 0);
                    }
                umma_commit(bar(L::SF + q));
            };
            auto issue_pv = [&](int q, bool first) {
                const uint64_t vd = v_desc + v.slot * kTile;
                const uint32_t tm = tmem + (L::two_s ? 0 : L::per_tile * q);
                const uint32_t p = tm + L::cS + (L::two_s ? L::cS2 * q : 0);
                umma_tA(tm + L::cO, p, vd, ID_O, !first);
#pragma unroll
                for (int kk = 1; kk < 8; ++kk) umma_tA(tm + L::cO, p + 8 * kk, vd + 128 * kk, ID_O, 1);
                if (kLow > 0)
#pragma unroll
                    for (int kk = 0; kk < kLow / 16; ++kk)
                        umma_tA(tm + L::cO, tm + L::cS + 64 + 8 * kk, vd + 128 * kk, ID_O, 1);
            };
            // behind the products of the ring's keys; last of a stretch: the rows' tile is free. (Slots are
            // handed back by the softmax's warps, which learn of the products' ends anyway.)
            auto after_s = [&](bool last) {
                if (L::update) umma_commit(bar(L::DF + k.slot));
                if (L::duo) umma_commit(bar(L::KE + k.slot));
                if (last && !L::rows_in_tmem) umma_commit(bar(L::XE));
                k.next();
            };
            Walk walk;
            for (long long at = u_begin; ok && at < u_end; ++seg) {
                const Stretch t = stretch_of(walk, at);
                at += t.steps;
                const bool two = second(t);
                if (!(ok = wait(bar(L::rows_in_tmem ? L::XT : L::XF), seg & 1))) break;
                if (!(ok = wait(bar(L::KF + k.slot), k.phase))) break;
                tc_fence_after();
                issue_s(0);
                if (two) issue_s(1);
                after_s(t.steps == 1);
                if (L::two_s) {
                    // the logits run a step ahead of the weights
                    if (t.steps > 1) {
                        if (!(ok = wait(bar(L::KF + k.slot), k.phase))) break;
                        issue_s(1);
                        after_s(t.steps == 2);
                    }
                    for (int i = 0; i < t.steps; ++i) {
                        const int q = i & 1;
                        if (!(ok = wait(bar(L::VF + v.slot), v.phase))) break;
                        if (!(ok = wait(bar(L::PR + q), (turns >> q) & 1))) break;
                        turns ^= 1u << q;
                        tc_fence_after();
                        issue_pv(q, i == 0);
                        umma_commit(bar(L::VE + v.slot));
                        umma_commit(bar(L::PD));
                        v.next();
                        if (i + 2 < t.steps) {
                            if (!(ok = wait(bar(L::KF + k.slot), k.phase))) break;
                            issue_s(q);
                            after_s(i + 3 == t.steps);
                        }
                    }
                }
                for (int i = 0; !L::two_s && i < t.steps; ++i) {
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
        } else if (RING && warp == L::other + 3) {
            // ======================================================== gates into their ring
            uint32_t j = 0;
            bool ok = true;
            Walk walk;
            for (long long at = u_begin; ok && at < u_end;) {
                const Stretch t = stretch_of(walk, at);
                at += t.steps;
                const Sight seen = sight(t);
                for (int i = 0; i < t.steps; ++i, ++j) {
                    const int pos0 = pos_of(t, seen, i);
                    int id = -1;
                    if (box_in(t, seen, pos0 + lane * box))
                        id = page_of(a, a.c.k_table, t.b, (pos0 + lane * box) >> a.c.page_shift, a.c.nk);
                    const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
                    const uint32_t sl = j % L::NG_, turn = j / L::NG_;
                    if (turn > 0 && !(ok = wait.warp(bar(L::GE + sl), (turn - 1) & 1))) break;
                    if (lane == 0) mbar_arrive_expect_tx(bar(L::GF + sl), (uint32_t)__popc(have) * box * G * 4);
                    __syncwarp();
                    if (id >= 0)
                        for (int g = 0; g < G; ++g)
                            bulk_load(base + L::gates + sl * L::gslot + (g * 128 + lane * box) * 4,
                                      a.c.g_pages + (((size_t)id * a.c.Hq + t.h * G + g) << a.c.page_shift) +
                                          ((pos0 + lane * box) & (page - 1)),
                                      box * 4, bar(L::GF + sl));
                }
            }
            if (!ok)  // on an abort: as above
                for (uint32_t v = j > L::NG_ ? j - L::NG_ : 0; v < j; ++v)
                    mbar_wait(bar(L::GF + v % L::NG_), (v / L::NG_) & 1, limit_ns);
        } else if (L::matrix && lane == 0 && warp == L::other + 3) {
            // ======================================================== K (P - I), NT = 1
            constexpr uint32_t ID_D = idesc_b16(128, D, true);
            constexpr uint64_t kAtom = L::atom >> 4, kTile = L::tile >> 4, kPart = (NA * D * 128) >> 4;
            const uint64_t k_desc = sdesc_sw128(base + L::K, 16, 1024), m_desc = sdesc_sw128(base + L::P, D * 128, 1024);
            Ring<NK> k;
            uint32_t j = 0, seg = 0;
            bool ok = true;
            Walk walk;
            for (long long at = u_begin; ok && at < u_end; ++seg) {
                const Stretch t = stretch_of(walk, at);
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
    } else if (L::update && warp >= 4) {
        // ============================================================ the keys' update
        if (L::split) reg_dec<L::reg_update>();
        const int r = tid - 128;
        const uint32_t tm = tmem + ((uint32_t)(32 * (warp - 4)) << 16) + L::cD;
        bool ok = true;
        uint32_t j = 0, seg = 0;
        bool held = false;
        Walk walk;
        for (long long at = u_begin; ok && at < u_end; ++seg) {
            const Stretch t = stretch_of(walk, at);
            at += t.steps;
            // single: the token's w and beta. (A stretch's first step has a barrier behind which nobody reads
            // the w of the stretch before the last.)
            float *const wv = reinterpret_cast<float *>(sm + L::W) + (seg & 1) * D;
            float beta = 0.f;
            if (L::single) {
                if (r < D)
                    wv[r] = __bfloat162float(
                        static_cast<const bf *>(a.w)[(long long)t.s.first * a.sw.tok + t.h * a.sw.head + r]);
                beta = a.beta[(long long)t.s.first * a.sb.tok + t.h * a.sb.head];
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            const Sight seen = sight(t);
            int next;  // the key pages of the next tile's boxes
            auto look_up = [&](int pos0) {
                next = -1;
                if (box_in(t, seen, pos0 + lane * box))
                    next = page_of(a, a.c.k_table, t.b, (pos0 + lane * box) >> a.c.page_shift, a.c.nk);
            };
            look_up(pos_of(t, seen, 0));
            for (int i = 0; i < t.steps; ++i, ++j) {
                const int pos0 = pos_of(t, seen, i), id = next;
                if (i + 1 < t.steps) look_up(pos_of(t, seen, i + 1));
                const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
                const bool whole = tile_whole(pos0, t.s.n, have, box_shift) && (!WIN || seen.all(pos0, 128));
                const int mine = __shfl_sync(0xffffffffu, id, r >> box_shift);
                uint8_t *const kt = sm + (key_slot(j) - base);
                auto key_at = [&](int c) {
                    return reinterpret_cast<uint4 *>(kt + (c >> 3) * L::atom + sw128_offset(r, c & 7));
                };
                uint4 key[L::held ? D / 8 : 1];
                float al = 0.f;  // -beta (w . k) of the thread's key
                if (L::single) {
                    if (!(ok = wait.warp(bar(L::KF + j % NK), (j / NK) & 1))) break;
                    float2 dot[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll(L::held ? D / 8 : FOX ? 2 : 4)
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 k8 = *key_at(c);
                        if (L::held) key[c] = k8;
                        const uint32_t k4[4] = {k8.x, k8.y, k8.z, k8.w};
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float4 w4 = *reinterpret_cast<const float4 *>(wv + 8 * c + 2 * e);
                            dot[0] = ffma2(unpack_bf16x2(k4[e]), make_float2(w4.x, w4.y), dot[0]);
                            dot[1] = ffma2(unpack_bf16x2(k4[e + 1]), make_float2(w4.z, w4.w), dot[1]);
                        }
                    }
                    al = -beta * ((dot[0].x + dot[0].y) + (dot[1].x + dot[1].y));
                }
                // the product is there, and the logits' product has read the keys too
                if (!(ok = wait.warp(bar(L::DF + j % NK), (j / NK) & 1))) break;
                tc_fence_after();
                bf *const dst = mine >= 0 && pos0 + r < t.s.n && (!WIN || seen.sees(pos0 + r))
                                    ? static_cast<bf *>(a.c.k_pages) +
                                          ((((size_t)mine * a.c.Hkv + t.h) << a.c.page_shift) +
                                           ((pos0 + r) & (page - 1))) * D
                                    : nullptr;
                if (L::single) {
#pragma unroll(L::held ? D / 8 : FOX ? 2 : 4)
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 k8 = L::held ? key[c] : *key_at(c);
                        const uint32_t k4[4] = {k8.x, k8.y, k8.z, k8.w};
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float4 w4 = *reinterpret_cast<const float4 *>(wv + 8 * c + 2 * e);
                            const float2 lo = ffma2(make_float2(al, al), make_float2(w4.x, w4.y), unpack_bf16x2(k4[e]));
                            const float2 hi =
                                ffma2(make_float2(al, al), make_float2(w4.z, w4.w), unpack_bf16x2(k4[e + 1]));
                            o[e] = pack_bf16x2(lo.x, lo.y);
                            o[e + 1] = pack_bf16x2(hi.x, hi.y);
                        }
                        const uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
                        if (whole) *key_at(c) = v;
                        else if (dst) *reinterpret_cast<uint4 *>(dst + 8 * c) = v;
                    }
                }
#pragma unroll 1
                for (int c = 0; c < (L::single ? 0 : D); c += 32) {
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
                if (!L::single) mbar_arrive_warp(bar(L::DE));
                fence_proxy_async_smem();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (warp == 4) {
                    if (whole && id >= 0) {
#pragma unroll
                        for (int x = 0; x < NA; ++x)
                            tma_store_3d(&tm_k, key_slot(j) + x * L::atom + lane * box * 128, 64 * x,
                                         (pos0 + lane * box) & (page - 1), id * a.c.Hkv + t.h);
                        if (!L::single) bulk_wait_read();
                    }
                    // single: a slot is released a step later, while the next step's keys leave
                    if (L::single) {
                        if (whole) bulk_wait_read_but<NA>();
                        else bulk_wait_read();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if (L::single && held) mbar_arrive(bar(L::KE + (j - 1) % NK));
                        if (!L::single || !whole) mbar_arrive(bar(L::KE + j % NK));
                    }
                    held = whole;
                }
            }
        }
        if (warp == 4) bulk_wait_all();
    } else {
        // ============================================================ softmax
        if (L::split) reg_inc<L::reg_row>();
        constexpr bool kTwice = (NT == 1 && !L::duo) || FOX;
        // row tile and row in it; duo: which half of the columns that the row takes
        const int w = NT == 1 ? 0 : warp >> 2, r = tid & 127, half = L::duo ? warp >> 2 : 0;
        const uint32_t tm = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + L::per_tile * w;
        bool ok = true;
        // One thread of a row tile hands slots back: the logits' product of step j has read its keys, and
        // it ends behind the values' product of step j - 1. (Keys that the pass updates: its warps do.)
        const bool releases = (warp & 3) == 0 && lane == 0 && half == 0;
        uint32_t j = 0, seg = 0, step = 0;  // steps and stretches with rows in this tile; steps of the CTA
        Walk walk;
        // duo: the other half's x of the row (a step later its column is written again at the earliest), or
        // (of nothing) until it has read its logits
        uint32_t turn = 0, phases = 0;  // (two_s: bits of the two places' logits)
        auto meet = [&]() {
            tc_fence_before();
            mbar_arrive_warp(bar(L::EX));
            ok = wait.warp(bar(L::EX), turn++ & 1);
            tc_fence_after();
        };
        auto exchange = [&](float x) {
            float *const at = reinterpret_cast<float *>(sm + L::W) + (turn & 1) * 256 + r;
            at[128 * half] = x;
            meet();
            return at[128 * (1 - half)];
        };
        // the row's two parts into tensor memory (the last products of the stretch before have ended)
        auto load_rows = [&](const Stretch &t) {
            const int row = 128 * NT * t.tile + (r & ((128 >> copies(t)) - 1));
            const bool live = row < t.s.T * G;
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {  // 32 columns of two elements
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        (part ? y.ql : y.qt) +
                        ((size_t)t.h * y.R + (size_t)t.s.first * G + (live ? row : 0)) * D + 2 * c);
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
        };
        Stretch next;
        if (L::ahead) next = stretch_of(walk, u_begin);
        if (L::ahead && half == 0) load_rows(next);
        for (long long at = u_begin; ok && at < u_end;) {
            const Stretch t = L::ahead ? next : stretch_of(walk, at);
            at += t.steps;
            if (w == 1 && !second(t)) {
                step += t.steps;
                continue;
            }
            const bool alone = NT == 2 && !second(t);  // no other tile: its part of the releases too
            // the row of this thread, and the columns of the key tiles that its copy takes (duo: that
            // this half of it takes, none of the second where a copy has 32)
            const int rows_all = t.s.T * G, cp = copies(t), rw = r & ((128 >> cp) - 1);
            const int row0 = 128 * (NT * t.tile + w), c_copy = (r >> (7 - cp)) * (128 >> cp);
            const bool halves = L::duo && cp < 2, idle = L::duo && cp == 2 && half == 1;
            const int cols = 128 >> (cp + (halves ? 1 : 0)), c_begin = c_copy + (halves ? half * cols : 0);
            const bool live = row0 + rw < rows_all, warp_live = row0 + (rw & ~31) < rows_all;
            const int head = live ? (row0 + rw) % G : 0, hq = t.h * G + head;
            const float gq =
                FOX && live ? y.gq[(size_t)t.h * y.R + (size_t)t.s.first * G + row0 + rw] * kLog2e : 0.f;
            if (L::rows_in_tmem && !L::ahead) load_rows(t);
            // a window: the row sees the keys from `from` on (and the sinks); from `edge` on all rows of the
            // tile do
            const Sight seen = sight(t);
            const int from = WIN ? t.s.n + 1 - window + (live && M != Pass::one ? (row0 + rw) / G : 0) : 0;
            const int last = M != Pass::one ? (min(rows_all, row0 + 128) - 1) / G : 0;  // the tile's last token
            const int edge = WIN && window > 0 ? t.s.n + 1 - window + last : 0;
            float m_run = -INFINITY, l_run = 0.f;
            int kid1, vid1;  // the pages of the next tile's boxes
            auto look_up = [&](int pos0) {
                kid1 = vid1 = -1;
                if (box_in(t, seen, pos0 + lane * box)) {
                    const size_t e = (size_t)t.b * a.c.max_pages + ((pos0 + lane * box) >> a.c.page_shift);
                    kid1 = __ldg(a.c.k_table + e);
                    vid1 = __ldg(a.c.v_table + e);
                }
            };
            look_up(pos_of(t, seen, 0));
            auto release = [&](int empty, uint32_t slot) {
                mbar_arrive(bar(empty + slot));
                if (alone) mbar_arrive(bar(empty + slot));
            };
            for (int i = 0; i < t.steps; ++i, ++j, ++step) {
                const int pos0 = pos_of(t, seen, i), id = kid1;
                const bool good = (unsigned)id < (unsigned)a.c.nk && (unsigned)vid1 < (unsigned)a.c.nv;
                if (i + 1 < t.steps) look_up(pos_of(t, seen, i + 1));
                const unsigned have = __ballot_sync(0xffffffffu, good);
                const int valid = min(128, t.s.n - pos0);
                const bool whole = tile_whole(pos0, t.s.n, have, box_shift);
                // gate sums of 32 keys from column c for the row's query head
                auto gates_of = [&](int c, float4 *v) {
                    if (RING) {
                        const float4 *const gp = reinterpret_cast<const float4 *>(
                            sm + L::gates + (j % L::NG_) * L::gslot + (head * 128 + c) * 4);
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] = gp[q];
                        return;
                    }
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
                constexpr bool kAhead = FOX && NT == 1 && D == 128 && !L::ahead;
                float4 ahead[kAhead ? 8 : 1];
                const bool early = kAhead && cols == 32;
                if (early) {
                    gates_of(c_begin, ahead);
                } else if (FOX && !RING) {
#pragma unroll 1
                    for (int c = c_begin; c < c_begin + cols; c += 16) {
                        const int bx = c >> box_shift, pid = __shfl_sync(0xffffffffu, id, bx);
                        if ((have >> bx) & 1u)
                            asm volatile("prefetch.global.L1 [%0];" ::"l"(
                                a.c.g_pages + (((size_t)pid * a.c.Hq + hq) << a.c.page_shift) +
                                ((pos0 + c) & (page - 1))));
                    }
                }
                const int place = L::two_s ? i & 1 : w;
                const uint32_t cS = L::cS + (L::two_s ? place * L::cS2 : 0);
                if (!(ok = wait.warp(bar(L::SF + place), (L::two_s ? phases >> place : j) & 1))) break;
                if (L::two_s) phases ^= 1u << place;
                if (RING && !(ok = wait.warp(bar(L::GF + j % L::NG_), (j / L::NG_) & 1))) break;
                tc_fence_after();
                if (releases && !L::two_s) {
                    if (!L::update) release(L::KE, step % NK);
                    if (i > 0) release(L::VE, (step - 1) % NV);
                }
                // (duo: every warp meets the other half's)
                if (warp_live || halves) {
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
                        if (WIN && pos0 + c < edge) {
                            const int over = sinks - pos0 - c, under = from - pos0 - c;
#pragma unroll
                            for (int q = 0; q < 32; ++q) x[q] = q < over || q >= under ? x[q] : -INFINITY;
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
                    // step is complete, so the previous P V is too, but with two places for S.)
                    float use;
                    auto raise = [&]() {
                        float alpha = 1.f;
                        const bool had = L::duo ? m_run > -INFINITY : l_run > 0.f;  // (duo: the same for both halves)
                        if (top > m_run + kRescale || (m_run == -INFINITY && top > -INFINITY)) {
                            alpha = m_run == -INFINITY ? 0.f : ex2_approx(m_run - top);
                            m_run = top;
                        }
                        const bool resc = alpha != 1.f && had;
                        if (__any_sync(0xffffffffu, resc)) {
                            if (L::two_s) {  // that product may still run
                                ok = wait.warp(bar(L::PD), (j - 1) & 1);
                                tc_fence_after();
                            }
                            if (halves) tmem_scale<D / 2>(tm + L::cO + half * (D / 2), resc ? alpha : 1.f);
                            else tmem_scale<D>(tm + L::cO, resc ? alpha : 1.f);
                        }
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
                    if (L::duo) {
                        // Both halves of a row have the same maximum. A half's weights take columns that may
                        // hold logits of the other: none is written before both have been read.
                        float x[32];
                        top = -INFINITY;
                        if (warp_live && !idle)
#pragma unroll 1
                            for (int c = c_begin; c < c_begin + cols; c += 32) {
                                tld32(tm + cS + c, x);
                                gate(c, x);
                                top = fmaxf(top, max32(x));
                            }
                        if (halves) top = fmaxf(top, exchange(top));
                        if (!ok) break;
                        uint32_t p[16], p2[16];
                        if (warp_live && !idle) {
                            raise();
                            if (cols > 32) {
                                tld32(tm + cS + c_begin, x);
                                gate(c_begin, x);
                            }
                            weigh(x, p, p, false);
                            if (cols > 32) {
                                tld32(tm + cS + c_begin + 32, x);
                                gate(c_begin + 32, x);
                                weigh(x, p2, p2, false);
                            }
                        }
                        if (halves && cols > 32) meet();
                        if (!ok) break;
                        if (warp_live && !idle) {
                            tmem_st16(tm + cS + c_begin / 2, p);
                            if (cols > 32) tmem_st16(tm + cS + c_begin / 2 + 16, p2);
#pragma unroll
                            for (int e = 0; e < 16; ++e) p[e] = 0u;
#pragma unroll 1
                            for (int c = 0; c < 128; c += 32)
                                if (half == 0 && (c < c_copy || c >= c_copy + (128 >> cp)))
                                    tmem_st16(tm + cS + c / 2, p);
                        }
                    } else if (kTwice) {
                        // registers are short: the logits of more than 32 columns are read twice. The
                        // weights of columns c .. c + 31 take the 16 columns from c / 2, whose logits
                        // have been read or are another copy's
                        float x[32];
                        top = -INFINITY;
#pragma unroll 1
                        for (int c = c_begin; c < c_begin + cols; c += 32) {
                            tld32(tm + cS + c, x);
                            gate(c, x);
                            top = fmaxf(top, max32(x));
                        }
                        raise();
                        uint32_t p[16];
#pragma unroll 1
                        for (int c = c_begin; c < c_begin + cols; c += 32) {
                            if (cols > 32) {
                                tld32(tm + cS + c, x);
                                gate(c, x);
                            }
                            weigh(x, p, p, false);
                            tmem_st16(tm + cS + c / 2, p);
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) p[e] = 0u;
#pragma unroll 1
                        for (int c = 0; c < 128; c += 32)
                            if (c < c_begin || c >= c_begin + cols) tmem_st16(tm + cS + c / 2, p);
                    } else {
                        float x[128];
                        uint32_t(*u)[32] = reinterpret_cast<uint32_t(*)[32]>(x);
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld32(tm + cS + 32 * c, u[c]);
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
                            tmem_st16(tm + cS + c / 2, p);
                            if (c < kLow) tmem_st16(tm + cS + 64 + c / 2, l);
                        }
                    }
                    if (!idle) l_run += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tmem_st_wait();
                }
                tc_fence_before();
                mbar_arrive_warp(bar(L::PR + place));
                if (RING) mbar_arrive_warp(bar(L::GE + j % L::NG_));
            }
            // the next stretch's rows while the last product of values runs
            if (L::ahead && ok && at < u_end) {
                next = stretch_of(walk, at);
                if (half == 0) load_rows(next);
            }
            if (!ok || !(ok = wait.warp(bar(L::FIN + w), seg & 1))) break;
            ++seg;
            tc_fence_after();
            if (releases && !L::two_s) release(L::VE, (step - 1) % NV);
            if (halves) {  // the row's sum
                l_run += exchange(l_run);
                if (!ok) break;
            }
            if (warp_live) {
                // the part's place: its CTA and item; a row whose keys were all absent leaves a sum of 0
                const size_t e = ((size_t)(blockIdx.x + t.item) * NT + w) * 128 + r;
#pragma unroll 1
                for (int c = L::duo ? half * (D / 2) : 0; c < (L::duo ? (half + 1) * (D / 2) : D); c += 32) {
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
                if (live && half == 0) y.sml[NT - 1][e] = make_float2(m_run, l_run);
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == L::other) {
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

}  // namespace

template <int NT, int D, bool FOX, Pass M, bool RING>
cudaError_t launch_cached_as(const StepOf<M> &a, const TcWs &y, uint64_t limit_ns, cudaStream_t stream) {
    using L = CachedCfg<NT, D, M, FOX, RING>;
    CUtensorMap tx{}, tl{}, tm{}, tk, tv;  // (rows that come ahead, and no P - I, need no map)
    // a map has no empty axis; of an empty pool nothing is loaded, every page number is outside it
    auto heads = [&](int pages) { return (long long)std::max(pages, 1) * a.c.Hkv; };
    if ((!L::ahead && (!make_map(&tx, y.qt, D, y.R, a.c.Hkv, 32) || !make_map(&tl, y.ql, D, y.R, a.c.Hkv, 32))) ||
        (L::matrix && !make_map(&tm, y.mt, D, D, (long long)std::min(a.c.seqs, a.N) * a.c.Hkv * 2, D)) ||
        !make_map(&tk, a.c.k_pages, D, a.c.page, heads(a.c.nk), a.c.page < 128 ? a.c.page : 128) ||
        !make_map(&tv, a.c.v_pages, D, a.c.page, heads(a.c.nv), a.c.page < 128 ? a.c.page : 128))
        return cudaErrorInvalidValue;
    auto kern = tc_cached_kernel<NT, D, FOX, M, RING>;
    const cudaError_t e = big_smem(kern, L::bytes);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3(y.plan[NT - 1].ctas), L::threads, L::bytes, stream, false, a, y, tx, tl, tm, tk, tv,
                  limit_ns);
}

template <int NT, int D, bool FOX, Pass M>
cudaError_t launch_cached(const StepOf<M> &a, const TcWs &y, uint64_t limit_ns, cudaStream_t stream) {
    if constexpr (CachedCfg<NT, D, M, FOX>::ring)
        if (a.c.G > kGateHeads) return launch_cached_as<NT, D, FOX, M, false>(a, y, limit_ns, stream);
    return launch_cached_as<NT, D, FOX, M, CachedCfg<NT, D, M, FOX>::ring>(a, y, limit_ns, stream);
}

#define EACH_PASS(WHAT, M)                                                                      \
    WHAT(1, 64, false, M) WHAT(2, 64, false, M) WHAT(1, 128, false, M) WHAT(2, 128, false, M)   \
    WHAT(1, 64, true, M) WHAT(2, 64, true, M) WHAT(1, 128, true, M) WHAT(2, 128, true, M)
#define SHARED_PASS(WHAT)                                                                       \
    WHAT(1, 64, false, Pass::shared) WHAT(2, 64, false, Pass::shared)                           \
    WHAT(1, 128, false, Pass::shared) WHAT(2, 128, false, Pass::shared)                         \
    WHAT(1, 64, true, Pass::shared) WHAT(1, 128, true, Pass::shared) WHAT(2, 128, true, Pass::shared)
#define PASS(NT, D, FOX, M) \
    template cudaError_t launch_cached<NT, D, FOX, M>(const StepMore &, const TcWs &, uint64_t, cudaStream_t);
#define EXTERN_PASS(NT, D, FOX, M) extern PASS(NT, D, FOX, M)
#define ONE_PASS(WHAT)                                                                          \
    WHAT(1, 64, false, Pass::one) WHAT(1, 128, false, Pass::one)                                \
    WHAT(1, 64, true, Pass::one) WHAT(1, 128, true, Pass::one)
EACH_PASS(EXTERN_PASS, Pass::window)
SHARED_PASS(EXTERN_PASS)
ONE_PASS(EXTERN_PASS)

}  // namespace paged
}  // namespace path
