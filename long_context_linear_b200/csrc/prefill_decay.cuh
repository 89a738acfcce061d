// Chunked causal linear attention with a decay per head on tcgen05 tensor
// cores (bf16 in, fp32 state).
//
// Per chunk of up to C = 128 tokens (R of them valid), local rows l, lam =
// exp(log_decay[head]) (decay.cuh):
//
//   P         = Q_c K_c^T                    8 x N=128, fp32 in TMEM (two buffers)
//   P[l][m]  <- lam^(l-m) P[l][m], m <= l    fp32 factor, then bf16, in place
//   Opv       = P V_c                        8 x N=64, A = P from TMEM, into P's upper columns
//   Oqs       = Q_c bf16(S)                  8 x N=64
//   O[l]      = Opv[l] + lam^(l+1) Oqs[l]    joined in fp32 on the way out
//   dS        = K_c^T [V1 | V2 | V3]         8 x N=192; V1 + V2 + V3 = lam^(R-1-m) V
//   S        <- lam^R S + dS1 + (dS2 + dS3)  fp32 registers
//
// The decay enters where a factor can be fp32.  The one place where it must
// multiply a tensor-core operand is the state update, whose weights run along
// the contraction: lam^(R-1-m) v_m is split into three bf16 terms (24 bits), so
// that the fp32 state keeps fp32 accuracy (one bf16 term: 2e-3 off, two: 2.6e-6,
// three: the rounding of the fp32 sums, 2e-7).  (Of an infinite v the second and
// third term are NaN, and an infinite key times a term that is zero is: the state
// entries that they reach are then NaN where one product would have infinity.
// Taking the NaN out of the small products as dS is read, one fmaxf per value,
// cost 7 to 25 % of the dense passes.)  The terms sit side by side as
// 3 x 64 value columns: K is read once for the three.  The two halves of an
// output have accumulators of their own because they take different factors
// per row: scaling Q's rows instead would round them once more.
//
// Work item = (unit or sequence and head, 64 value columns), persistent CTAs,
// as in prefill_tc.cuh, whose items, segments, reverse order and packed batches
// it shares; dense items that are not a multiple of the SMs are shared out by
// chunks (piece()).  In reverse order rows take lam^(m-l) and lam^(R-1-l), the update
// lam^(m+1) (the state is held already decayed).
//
// Shared memory (217 KB): Q 2 x 32 KB, K 2 x 32 KB, V 2 x 16 KB, the three V
// terms of 32 rows at a time 2 x 12 KB (written while the product of the 32 rows
// before runs), bf16(S) 16 KB, key dims as rows: each state thread writes its
// row in 16-byte vectors, and 16 KB to stage O.  (All 128 rows of the terms at
// once leave no room for that; O staged in its chunk's V slot held the slot for
// too long: 2.5 us a chunk against 2.3.)
// TMEM (512 columns): two P buffers of 128 (bf16 P in the first 64 of each,
// Opv in the others once they have been read), Oqs 64, dS 192.
//
// Warp roles (16 warps):
//   w0 lane 0  : TMA producer
//   w1 lane 0  : MMA thread A: Q K^T
//   w14 lane 0 : MMA thread B: dS
//   w15 lane 0 : MMA thread C: P V, Q S
//   w2..w5     : P warps (V terms of rows 0 .. 63, then masked and decayed P)
//   w6..w9     : state warps (V terms of rows 64 .. 127, publish bf16(S), absorb dS)
//   w10..w13   : output warps
// Q K^T, P and P V need no state and run ahead; the chain from chunk to chunk
// is terms -> dS -> S -> Q S.  Every wait is bounded (wait_bounded); a timeout
// stops the CTA cleanly.
//
// Measured at B=1 H=64 N=16K, d = 128 (128 CTAs): 0.29 ms, 2.26 us per chunk of
// 128 tokens (without a decay 1.64, the bytes at the copy rate 1.28); B=4 H=32
// N=8K: 0.28 to 0.29 ms = 3.7 TB/s, 0.56 of the copy rate, for some tens of calls
// in a row, 0.34 to 0.35 ms between other work (cold L2, lower clock).
// What bounds it: neither the bytes (38 % of DRAM's rate) nor the tensor pipe
// (42 % busy).  Its code size matters: with everything unrolled a chunk took 5.4
// us, the cache of instructions that SMs share is still 70 % busy, and 64 more
// instructions in the state warps cost 7 to 25 %.  But few stalls are for a
// missing instruction (0.5 per issue, against 3.1 for long scoreboards): how
// much of a chunk is the chain of its steps is not measured.  128 registers a
// thread spill 100 to 180 bytes.
#pragma once
#include "decay.cuh"
#include "f32x2.cuh"
#include "prefill_tc.cuh"

namespace lcl {
namespace tcd {

using tc::C;
using tc::DVS;
using tc::PANEL;

struct Params : tc::Params {
    const float* log_decay;  // [H] log of the decay per head, or null (prefill_tc.cuh's kernels); dense: head u % H
    // dense whole sequences: chunks per CTA of the wrapped schedule (0: items in
    // turn), the states handed on from CTA to CTA [grid][DK][DVS] and how many
    // warps have written each (zero at launch)
    int wrap;
    float* wrap_state;
    int* wrap_ready;
};

constexpr int SLOTS = 2;                    // Q, K, V ring depth
constexpr int TERMS = 3;                    // bf16 terms of the weighted V
constexpr int TILE = 2 * PANEL;             // Q, K: two 64-column panels
constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + SLOTS * TILE;
constexpr int OFF_V = OFF_K + SLOTS * TILE;
constexpr int OFF_VT = OFF_V + SLOTS * PANEL;
constexpr int QROWS = 32;                   // rows of a quarter of the chunk
constexpr int VT_PANEL = QROWS * 128;       // one term of a quarter
constexpr int VT_BUF = TERMS * VT_PANEL;
constexpr int OFF_S = OFF_VT + 2 * VT_BUF;
constexpr int OFF_OST = OFF_S + PANEL;
constexpr int OFF_BAR = OFF_OST + PANEL;
static_assert(OFF_VT % 1024 == 0 && OFF_S % 1024 == 0 && VT_PANEL % 1024 == 0, "swizzled tiles need 1024-byte alignment");
// mbarriers (8 bytes each) at OFF_BAR, then the TMEM base.  A wait knows a phase
// by its parity alone, so no barrier may complete a second phase while a warp has
// yet to see the first: whoever waits on one also takes part in its next phase
// (directly, or in a step that its arrivals wait for).  With [2] the next phase is
// that of chunk g + 2; a single o_empty would break the rule, as thread A comes to
// it only two chunks later and chunk g + 1 goes on without A once its Q K^T is
// issued.  [4] are once per chunk each, like the single ones.
constexpr int BAR_Q_FULL = 0;                      // [2] TMA -> A, C
constexpr int BAR_Q_EMPTY = BAR_Q_FULL + SLOTS;    // [2] A (Q K^T) + C (Q S) -> TMA
constexpr int BAR_K_FULL = BAR_Q_EMPTY + SLOTS;    // [2] TMA -> A, B, P warps (ragged tail)
constexpr int BAR_K_EMPTY = BAR_K_FULL + SLOTS;    // [2] A (Q K^T) + B (dS) -> TMA
constexpr int BAR_V_FULL = BAR_K_EMPTY + SLOTS;    // [2] TMA -> P warps, state warps
constexpr int BAR_V_EMPTY = BAR_V_FULL + SLOTS;    // [2] P warps, state warps (V read) + C (P V) -> TMA
constexpr int BAR_VT_FULL = BAR_V_EMPTY + SLOTS;   // [4] by quarter of the rows: P warps (0, 1), state warps (2, 3) -> B
constexpr int BAR_VT_EMPTY = BAR_VT_FULL + 4;      // [4] by quarter: B (its product done) -> state warps (0, 1), P warps (2, 3)
constexpr int BAR_P_FULL = BAR_VT_EMPTY + 4;       // [2] A (Q K^T) -> P warps
constexpr int BAR_P_READY = BAR_P_FULL + 2;        // [2] P warps (bf16 P written, V landed) -> C
constexpr int BAR_O_FULL = BAR_P_READY + 2;        // C (P V, Q S) -> output warps, state warps
constexpr int BAR_O_EMPTY = BAR_O_FULL + 1;        // [2] output warps (Opv, Oqs read) -> A (two chunks later), C (the next)
constexpr int BAR_DS_FULL = BAR_O_EMPTY + 2;       // B -> state warps
constexpr int BAR_DS_EMPTY = BAR_DS_FULL + 1;      // state warps -> B
constexpr int BAR_S_FULL = BAR_DS_EMPTY + 1;       // state warps (bf16(S) written) -> C
constexpr int BAR_TAB = BAR_S_FULL + 1;            // P warps (decay table of an item written) -> P warps
constexpr int BAR_DRAIN = BAR_TAB + 1;             // [3] A, B, C
constexpr int BAR_COUNT = BAR_DRAIN + 3;
constexpr int BAR_BYTES = 320;
static_assert((BAR_COUNT + 1) * 8 <= BAR_BYTES, "barrier area too small");
constexpr int OFF_TAB = OFF_BAR + BAR_BYTES;       // lam^n, n = 0 .. C, by item parity
constexpr int TAB_PAD = 32;                        // entries in front of lam^0
constexpr int TAB = TAB_PAD + C + 4;
constexpr int SMEM_BYTES = OFF_TAB + 2 * TAB * 4 + 1024;
static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KB per-block shared memory limit");
constexpr int NUM_THREADS = 512;
constexpr int WARP_MMA_A = 1;
constexpr int WARP_MMA_B = 14;
constexpr int WARP_MMA_C = 15;

constexpr uint32_t TM_P = 0;       // P buffer b at 128 b; bf16 P in its first 64 columns
constexpr uint32_t TM_OPV = 64;    // Opv of buffer b at 64 + 128 b
constexpr uint32_t TM_OQS = 256;
constexpr uint32_t TM_DS = 320;    // three terms of 64 columns
constexpr uint32_t TMEM_COLS = 512;

// One 16-byte vector (8 values of a row of V) times the row's weight, cut into
// three runs of 8 bits: each term is the upper half of what is left, so no
// conversion is needed and the three hold all 24 bits of the fp32 product.
__device__ __forceinline__ void v_split(uint32_t vt, const uint4& r, float w) {
    const uint32_t in[4] = {r.x, r.y, r.z, r.w};
    const uint64_t w2 = f32x2(w, w), minus = f32x2(-1.f, -1.f);
    uint32_t out[TERMS][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t x = mul2(f32x2(in[i] << 16, in[i] & 0xffff0000u), w2);
#pragma unroll
        for (int n = 0; n < TERMS; ++n) {
            float lo, hi;
            f32x2_split(x, lo, hi);
            const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
            out[n][i] = __byte_perm(a, b, 0x7632);
            // the remainder: the bits cut off, exact
            if (n + 1 < TERMS) x = fma2(f32x2(a & 0xffff0000u, b & 0xffff0000u), minus, x);
        }
    }
#pragma unroll
    for (int n = 0; n < TERMS; ++n) st_shared_v4(vt + n * VT_PANEL, out[n][0], out[n][1], out[n][2], out[n][3]);
}

// A group of 128 threads forms the terms of 64 rows of V, a quarter of 32 rows
// at a time: thread t takes the vectors at places t + 128 j of the (swizzled)
// tile, rows r0 + 16 j; a vector's place in V is its place in every term.
struct Weights {
    float w[4];
    // of rows r0 + 16 j of a chunk of `rows`, from the smallest exponent up (rows
    // past the end are zero, whatever their weight)
    template <bool kRev, typename F>
    __device__ __forceinline__ void set(const F& power, double lam16, int r0, int rows) {
        const int left = rows - 1 - r0;  // in order: exponent left - 16 j
        const float2 first = power(kRev ? r0 + 1 : left >= 48 ? left - 48 : left & 15);
        double x = static_cast<double>(first.x) + first.y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = kRev ? i : 3 - i;
            w[j] = static_cast<float>(x);
            if (kRev || 16 * j <= left) x *= lam16;
        }
    }
};
// Quarter h (0, 1) of the group's 64 rows, whose places in V start at v.
// (rolled: see piece())
__device__ __forceinline__ void v_terms(uint32_t v, uint32_t vt, const Weights& w, int h, int r0, int rows, bool tail) {
    float wa = h ? w.w[2] : w.w[0];
    const float wb = h ? w.w[3] : w.w[1];
    r0 += 32 * h;
    v += static_cast<uint32_t>(h) * VT_PANEL;
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
        uint4 x = ld_shared_v4(v);
        if (tail && r0 >= rows) x = make_uint4(0u, 0u, 0u, 0u);
        v_split(vt, x, wa);
        wa = wb;
        r0 += 16;
        v += 2048u;
        vt += 2048u;
    }
    fence_proxy_async_smem();
}

// Rows rows .. C - 1 of a tile of 128-byte rows set to zero, by 128 threads t.
__device__ __noinline__ void clear_rows(uint32_t tile, int rows, int t) {
    for (int e = rows * 8 + t; e < C * 8; e += 128) st_shared_v4(tile + static_cast<uint32_t>(e) * 16u, 0u, 0u, 0u, 0u);
}

// Bounded wait for the phase of the given parity, in few instructions (see
// piece()): up to 100,000 tries, each of which sleeps for up to 20 us or until
// the phase completes; two seconds in all at most.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 100000;\n\t"
        "W: mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@p bra D;\n\tsub.u32 n, n, 1;\n\tsetp.ne.u32 q, n, 0;\n\t@q bra W;\n\t"
        "D: selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}

// Out of line, one copy for all roles: they run once per item, and the
// kernel's instruction footprint counts (all roles of all
// SMs run at once; with these inlined and everything unrolled it was 112 KB and
// took 10,000 cycles per chunk).
//
// What CTA `cta` of `G` does in turn r: an item, or part of one; len < 0 when
// it has no more.  With more items than CTAs whole items in turn leave CTAs idle
// in the last turn (150 items take twice as long as 148).  The wrapped schedule
// instead lays the chunks of all units of a value slice end to end and cuts the
// row into equal shares, p.wrap chunks each.  A unit that a cut divides is begun
// by the CTA below the cut, as the first thing it does, and finished by the one
// above, as the last: with a share no shorter than a unit the state to go on
// from has long been written (wait_state).  A CTA waits for a lower one's first
// piece, which waits for nothing, and all are resident (cooperative launch).
// The two slices of a unit share Q and K: their CTAs, neighbours, keep step.
struct Piece : tc::Item {
    const float* init;  // initial state of this value slice, rows init_ld apart, or null
    float* out;         // where the state goes, or null
    int init_ld, out_ld;
    int from, to;       // CTA whose state is continued, own slot written for the next one (or -1)
};
template <int KD, bool kRev, bool kLean>
__device__ __noinline__ Piece piece(const Params& p, int r, int cta, int G) {
    constexpr int NV = KD / DVS;
    constexpr long SLOT = (long)KD * DVS;
    Piece it;
    it.from = it.to = -1;
    int idx = tc::item_index(r, cta, G), from = 0, to = 0;
    const int n = (p.N + C - 1) / C;
    const bool wrapped = kLean && p.wrap > 0;
    if (wrapped) {
        const long lo = (long)(cta / NV) * p.wrap, hi = min(lo + p.wrap, (long)(p.n_items / NV) * n);
        const long u = (hi - 1) / n - r;
        if (hi <= lo || (u + 1) * n <= lo) idx = p.n_items;
        else {
            idx = (int)u * NV + cta % NV;
            from = (int)(max(lo, u * n) - u * n);
            to = (int)(min(hi, (u + 1) * n) - u * n);
        }
    }
    if (idx >= p.n_items) {
        it.len = -1;
        return it;
    }
    static_cast<tc::Item&>(it) = tc::decode_item<true, KD>(p, idx);
    it.init = static_cast<const tc::Item&>(it).init;
    if (it.init) it.init += p.init_transposed ? (long)DVS * it.vs * KD : DVS * it.vs;
    it.init_ld = p.dv;
    it.out = p.s_out && it.write_state ? p.s_out + it.state * KD * p.dv + DVS * it.vs : nullptr;
    it.out_ld = p.dv;
    if (wrapped) {
        // chunks [from, to) in visiting order
        it.t0 = (kRev ? n - to : from) * C;
        it.len = min(p.N, (kRev ? n - from : to) * C) - it.t0;
        if (from > 0) {
            it.from = cta - NV;
            it.init = p.wrap_state + it.from * SLOT;
            it.init_ld = DVS;
        }
        if (to < n) {
            it.to = cta;
            it.out = p.wrap_state + cta * SLOT;
            it.out_ld = DVS;
        }
    }
    return it;
}
// Waits until the state warps of another CTA have all written their rows of its
// slot; a second at most.
__device__ __noinline__ bool wait_state(const int* ready) {
    for (int i = 0; i < 500000; ++i) {
        int n;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(n) : "l"(ready) : "memory");
        if (n >= 4) return true;
        __nanosleep(1000);
    }
    return false;
}
// lam^n as two fp32 values, for the head of `it`
__device__ __noinline__ float2 item_power(const Params& p, int c1, int c2, int n) {
    float2 f;
    decay::power2(p.log_decay[p.mode == 0 ? c2 % p.H : c1], n, f.x, f.y);
    return f;
}

// kRev: chunks visited last to first (the backward's reverse passes).  kLean:
// dense, with outputs; the other instance adds packed batches and the states
// alone (kept in one instance they took 12 % of the dense passes).
template <int KD, bool kRev, bool kLean>
__global__ void __launch_bounds__(NUM_THREADS, 1)
prefill_decay_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                     const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    uint64_t* q_full = bars + BAR_Q_FULL;
    uint64_t* q_empty = bars + BAR_Q_EMPTY;
    uint64_t* k_full = bars + BAR_K_FULL;
    uint64_t* k_empty = bars + BAR_K_EMPTY;
    uint64_t* v_full = bars + BAR_V_FULL;
    uint64_t* v_empty = bars + BAR_V_EMPTY;
    uint64_t* vt_full = bars + BAR_VT_FULL;
    uint64_t* vt_empty = bars + BAR_VT_EMPTY;
    uint64_t* p_full = bars + BAR_P_FULL;
    uint64_t* p_ready = bars + BAR_P_READY;
    uint64_t* o_full = bars + BAR_O_FULL;
    uint64_t* o_empty = bars + BAR_O_EMPTY;
    uint64_t* ds_full = bars + BAR_DS_FULL;
    uint64_t* ds_empty = bars + BAR_DS_EMPTY;
    uint64_t* s_full = bars + BAR_S_FULL;
    uint64_t* tab_full = bars + BAR_TAB;
    uint64_t* drain = bars + BAR_DRAIN;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + BAR_COUNT);
    // a wait that runs out ends its role; the others, which then wait for what
    // it would have done, end the same way
    bool late = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = wait_bounded(bar, parity);
        late |= !ok;
        return ok;
    };
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = gridDim.x;
    const int cta = blockIdx.x;
    const bool state_only = !kLean && p.state_only;
    const bool packed = !kLean && p.mode == 1;
    constexpr bool rev = kRev;
    constexpr int NP = KD / 64;  // 64-column panels per Q / K tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 2);
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], state_only ? 1 : 2);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], state_only ? 8 : 9);
            mbar_init(&p_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&o_empty[i], 4);
        }
        mbar_init(o_full, 1);
        mbar_init(ds_full, 1);
        mbar_init(ds_empty, 4);
        mbar_init(s_full, 4);
        mbar_init(tab_full, 4);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&vt_full[i], 4);
            mbar_init(&vt_empty[i], 1);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&drain[i], 1);
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&map_q);
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
        prefetch_tmap(&map_o);
    }
    if (warp == WARP_MMA_A) {
        tmem_alloc(tmem_holder, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_holder;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            int g = 0;      // chunks whose copies are all issued
            int kg = 0, vg = 0, qg = 0;  // copies of K, V and Q issued
            bool stop = false;
            for (int r = 0; !stop; ++r) {
                const Piece it = piece<KD, kRev, kLean>(p, r, cta, G);
                if (it.len < 0) break;
                const int nc = (it.len + C - 1) / C;
                for (int c = 0; c < nc; ++c, ++g) {
                    const int t = it.t0 + tc::chunk_row(rev, c, nc);
                    const int y = !packed ? t : it.c1, z = !packed ? it.c2 : t;
                    const int s = g & 1, n = g >> 1;
                    if (n > 0 && !wait(&k_empty[s], (n - 1) & 1)) { stop = true; break; }
                    mbar_arrive_expect_tx(&k_full[s], NP * PANEL);
#pragma unroll
                    for (int pn = 0; pn < NP; ++pn)
                        tma_load_3d(sm + OFF_K + s * TILE + pn * PANEL, &map_k, &k_full[s], 64 * pn, y, z);
                    ++kg;
                    if (n > 0 && !wait(&v_empty[s], (n - 1) & 1)) { stop = true; break; }
                    mbar_arrive_expect_tx(&v_full[s], PANEL);
                    tma_load_3d(sm + OFF_V + s * PANEL, &map_v, &v_full[s], DVS * it.vs, y, z);
                    ++vg;
                    // (Q last: its slot is the one held longest)
                    if (!state_only) {
                        if (n > 0 && !wait(&q_empty[s], (n - 1) & 1)) { stop = true; break; }
                        mbar_arrive_expect_tx(&q_full[s], NP * PANEL);
#pragma unroll
                        for (int pn = 0; pn < NP; ++pn)
                            tma_load_3d(sm + OFF_Q + s * TILE + pn * PANEL, &map_q, &q_full[s], 64 * pn, y, z);
                        ++qg;
                    }
                }
            }
            // no copy into shared memory may still be in flight at exit
            for (int x = max(kg - 2, 0); x < kg; ++x) tc::drain_wait(&k_full[x & 1], (x >> 1) & 1);
            for (int x = max(qg - 2, 0); x < qg; ++x) tc::drain_wait(&q_full[x & 1], (x >> 1) & 1);
            for (int x = max(vg - 2, 0); x < vg; ++x) tc::drain_wait(&v_full[x & 1], (x >> 1) & 1);
        }
    } else if (warp == WARP_MMA_A || warp == WARP_MMA_B || warp == WARP_MMA_C) {
        // ------------------------------------------------------ MMA threads
        if (lane == 0 && (warp == WARP_MMA_B || !state_only)) {
            const uint32_t sq = smem_u32(sm + OFF_Q), sk = smem_u32(sm + OFF_K), sv = smem_u32(sm + OFF_V);
            int total = 0;  // this CTA's chunks
            for (int r = 0;; ++r) {
                const int len = piece<KD, kRev, kLean>(p, r, cta, G).len;
                if (len < 0) break;
                total += (len + C - 1) / C;
            }
            uint64_t* done = &drain[warp == WARP_MMA_A ? 0 : warp - WARP_MMA_B + 1];
            if (warp == WARP_MMA_A) {
                constexpr uint32_t id_qk = idesc_bf16(128, 128, 0, 0);  // Q K^T
                for (int g = 0; g < total; ++g) {
                    // once O of chunk g-2 has been read out of the buffer
                    const int s = g & 1;
                    if (g > 1 && !wait(&o_empty[s], ((g - 2) >> 1) & 1)) break;
                    if (!wait(&q_full[s], (g >> 1) & 1)) break;
                    if (!wait(&k_full[s], (g >> 1) & 1)) break;
                    tc_fence_after();
                    const uint64_t da = tc::kmaj_desc(sq + s * TILE, 0, PANEL), db = tc::kmaj_desc(sk + s * TILE, 0, PANEL);
#pragma unroll
                    for (int kk = 0; kk < KD / 16; ++kk)
                        mma_ss(tbase + TM_P + 128u * s, da + tc::kmaj_step(kk, PANEL), db + tc::kmaj_step(kk, PANEL), id_qk, kk > 0);
                    mma_commit(&p_full[s]);
                    mma_commit(&q_empty[s]);
                    mma_commit(&k_empty[s]);
                }
            } else if (warp == WARP_MMA_B) {
                constexpr uint32_t id_ds = idesc_bf16(128, TERMS * DVS, 1, 1);  // K^T [V1 | V2 | V3]
                const uint64_t dv = tc::mnmaj_desc(smem_u32(sm + OFF_VT), 0, VT_PANEL);
                for (int g = 0; g < total; ++g) {
                    const int s = g & 1;
                    bool ok = wait(&k_full[s], (g >> 1) & 1);
                    ok = ok && (g == 0 || wait(ds_empty, (g - 1) & 1));
                    // at d = 64 both 64-row halves of K^T read the same panel (rows 64 .. 127 are ignored)
                    const uint64_t dk = tc::mnmaj_desc(sk + s * TILE, 0, KD == 128 ? PANEL : 0);
#pragma unroll
                    for (int qd = 0; qd < 4; ++qd) {
                        ok = ok && wait(&vt_full[qd], g & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk)
                            mma_ss(tbase + TM_DS, dk + tc::mnmaj_step(2 * qd + kk), dv + (qd & 1) * (VT_BUF >> 4) + tc::mnmaj_step(kk),
                                   id_ds, qd + kk > 0);
                        mma_commit(&vt_empty[qd]);
                    }
                    if (!ok) break;
                    mma_commit(ds_full);
                    mma_commit(&k_empty[s]);
                }
            } else {
                constexpr uint32_t id_pv = idesc_bf16(128, DVS, 0, 1);  // P V (P from TMEM)
                constexpr uint32_t id_qs = idesc_bf16(128, DVS, 0, 1);  // Q S
                const uint64_t ds = tc::mnmaj_desc(smem_u32(sm + OFF_S), 0, PANEL);
                for (int g = 0; g < total; ++g) {
                    const int s = g & 1;
                    if (!wait(&p_ready[s], (g >> 1) & 1)) break;
                    tc_fence_after();
                    const uint64_t dv = tc::mnmaj_desc(sv + s * PANEL, 0, PANEL);
                    const uint32_t tp = tbase + TM_P + 128u * s;
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_ts(tp + TM_OPV, tp + kk * 8, dv + tc::mnmaj_step(kk), id_pv, kk > 0);
                    mma_commit(&v_empty[s]);
                    // (Q has landed: Q K^T has read it)
                    if (g > 0 && !wait(&o_empty[s ^ 1], ((g - 1) >> 1) & 1)) break;
                    if (!wait(s_full, g & 1)) break;
                    tc_fence_after();
                    const uint64_t da = tc::kmaj_desc(sq + s * TILE, 0, PANEL);
#pragma unroll
                    for (int kk = 0; kk < KD / 16; ++kk)
                        mma_ss(tbase + TM_OQS, da + tc::kmaj_step(kk, PANEL), ds + tc::mnmaj_step(kk), id_qs, kk > 0);
                    mma_commit(o_full);
                    mma_commit(&q_empty[s]);
                }
            }
            // every MMA issued by this thread must be finished before TMEM is freed
            mma_commit(done);
            tc::drain_wait(done, 0);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ------------------------------------------------------ P warps
        const int q4 = warp & 3;
        const int t = (warp - 2) * 32 + lane;  // 0 .. 127, for the table and the clearing
        const int row = q4 * 32 + lane;        // row of P
        const uint32_t tlane = tbase + (static_cast<uint32_t>(q4 * 32) << 16);
        const int r0 = t >> 3;                 // first row of its V terms
        int g = 0;
        bool stop = false;
        for (int r = 0; !stop; ++r) {
            const Piece it = piece<KD, kRev, kLean>(p, r, cta, G);
            if (it.len < 0) break;
            auto power = [&](int n) { return item_power(p, it.c1, it.c2, n); };
            const float2 step = power(16);
            const double lam16 = static_cast<double>(step.x) + step.y;
            Weights w;
            w.set<rev>(power, lam16, r0, C);
            // the item's table; the other one may still be read by a warp at the
            // item before, and nobody is two items behind (each waits here)
            float* tab = reinterpret_cast<float*>(sm + OFF_TAB) + (r & 1) * TAB + TAB_PAD;
            const float2 f1 = power(t + 1);
            tab[t + 1] = f1.x + f1.y;
            if (t == 0) tab[0] = 1.f;
            __syncwarp();
            if (lane == 0) mbar_arrive(tab_full);
            if (!warp_wait(tab_full, r & 1)) break;
            const int nc = (it.len + C - 1) / C;
            for (int c = 0; c < nc; ++c, ++g) {
                const int rows = min(C, it.len - tc::chunk_row(rev, c, nc));
                const int s = g & 1;
                const bool tail = packed && rows < C;
                const uint32_t v = smem_u32(sm + OFF_V + s * PANEL);
                if (!warp_wait(&v_full[s], (g >> 1) & 1)) { stop = true; break; }
                if (tail) {
                    // rows past the end of a packed sequence hold another one's tokens,
                    // or anything: cleared in V and K, since 0 x NaN is not 0 (Q K^T may
                    // read them either way: those columns of P are masked)
                    if (!warp_wait(&k_full[s], (g >> 1) & 1)) { stop = true; break; }
                    clear_rows(v, rows, t);
#pragma unroll 1
                    for (int pn = 0; pn < NP; ++pn) clear_rows(smem_u32(sm + OFF_K + s * TILE + pn * PANEL), rows, t);
                }
                // --- V terms of the first half of the rows, each quarter into the buffer of the one two before it
                if (!rev && rows < C) w.set<rev>(power, lam16, r0, rows);
#pragma unroll 1
                for (int h = 0; h < 2 && !stop; ++h) {
                    if (g > 0 && !warp_wait(&vt_empty[2 + h], (g - 1) & 1)) stop = true;
                    if (stop) break;
                    v_terms(v + static_cast<uint32_t>(t) * 16u, smem_u32(sm + OFF_VT + h * VT_BUF) + static_cast<uint32_t>(t) * 16u, w, h,
                            r0, rows, tail);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&vt_full[h]);
                }
                if (stop) break;
                if (lane == 0) mbar_arrive(&v_empty[s]);
                if (state_only) continue;
                const uint32_t tp = tlane + TM_P + 128u * s;
                if (!warp_wait(&p_full[s], (g >> 1) & 1)) { stop = true; break; }
                tc_fence_after();
                // 32-column pieces on the kept side of the diagonal piece take
                // lam^|l-m| as (factor of the row) x (factor of the column), both
                // exponents >= 0; the diagonal piece looks its factors up
#pragma unroll 1
                for (int pc = 0; pc < 4; ++pc) {
                    uint32_t pk[16];
                    if (rev ? pc < q4 : pc > q4) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = 0u;
                    } else {
                        uint32_t v[32];
                        tmem_ld32(tp + 32 * pc, v);
                        tmem_wait_ld();
                        if (pc == q4) {
                            // (the entries in front of lam^0 are read for masked places only)
                            const uint32_t keep = rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
                            const float* f = rev ? tab - lane : tab + lane;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float a = f[rev ? 2 * i : -2 * i], b = f[rev ? 2 * i + 1 : -2 * i - 1];
                                pk[i] = pack_bf16x2((keep & (1u << (2 * i))) ? __uint_as_float(v[2 * i]) * a : 0.f,
                                                    (keep & (2u << (2 * i))) ? __uint_as_float(v[2 * i + 1]) * b : 0.f);
                            }
                        } else {
                            const float rf = tab[rev ? 32 * pc - row : row - 32 * pc - 31];
                            const uint64_t rf2 = f32x2(rf, rf);
                            const float4* col = reinterpret_cast<const float4*>(tab);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                // lam^(4 i) .. lam^(4 i + 3) for columns 4 i .. in reverse order, 31 - 4 i .. in order
                                const float4 f = col[rev ? i : 7 - i];
                                const uint64_t f0 = rev ? f32x2(f.x, f.y) : f32x2(f.w, f.z);
                                const uint64_t f1 = rev ? f32x2(f.z, f.w) : f32x2(f.y, f.x);
                                pk[2 * i] = pack_bf16x2(mul2(f32x2(v[4 * i], v[4 * i + 1]), mul2(rf2, f0)));
                                pk[2 * i + 1] = pack_bf16x2(mul2(f32x2(v[4 * i + 2], v[4 * i + 3]), mul2(rf2, f1)));
                            }
                        }
                    }
                    tmem_st16(tp + 16 * pc, pk);  // over fp32 pieces that have been read
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[s]);
            }
        }
    } else if (warp < 10) {
        // ------------------------------------------------------ state warps
        const int q4 = warp & 3;
        const int i = q4 * 32 + lane;  // key-dim row of S owned by this thread
        const bool own = KD == 128 || q4 < KD / 32;  // warp-uniform; at d = 64 warps 6, 7 (q4 = 2, 3) only follow along
        const uint32_t tds = tbase + (static_cast<uint32_t>(q4 * 32) << 16) + TM_DS;
        const uint32_t srow = smem_u32(sm + OFF_S) + static_cast<uint32_t>(i) * 128u;
        const int t = (warp - 6) * 32 + lane;
        const int r0 = 64 + (t >> 3);  // first row of its V terms
        int g = 0;
        bool stop = false;
        for (int r = 0; !stop; ++r) {
            const Piece it = piece<KD, kRev, kLean>(p, r, cta, G);
            if (it.len < 0) break;
            uint64_t S[DVS / 2];  // pairs of value columns
            if (kLean && it.from >= 0) {
                const bool ok = wait_state(p.wrap_ready + it.from);
                late |= !ok;
                if (!__all_sync(0xffffffffu, ok)) break;
            }
            if (it.init && p.init_transposed && it.from < 0 && own) {
                const float* src = it.init + i;
#pragma unroll
                for (int j = 0; j < DVS; j += 2) S[j / 2] = f32x2(src[j * KD], src[(j + 1) * KD]);
            } else if (it.init && own) {
                const float4* src = reinterpret_cast<const float4*>(it.init + (long)i * it.init_ld);
#pragma unroll
                for (int j = 0; j < DVS / 4; ++j) {
                    const float4 x = src[j];
                    S[2 * j] = f32x2(x.x, x.y);
                    S[2 * j + 1] = f32x2(x.z, x.w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < DVS / 2; ++j) S[j] = 0ull;
            }
            auto power = [&](int n) { return item_power(p, it.c1, it.c2, n); };
            const float2 step = power(16);
            const double lam16 = static_cast<double>(step.x) + step.y;
            Weights w;
            w.set<rev>(power, lam16, r0, C);
            float2 lam = power(C);  // lam^R
            const int nc = (it.len + C - 1) / C;
            // a sequence's one chunk of other than C rows: its last (in reverse
            // order the first visited)
            const int odd = it.len % C, odd_at = odd ? (rev ? 0 : nc - 1) : -1;
            for (int c = 0; c < nc; ++c, ++g) {
                const int rows = c == odd_at ? odd : C;
                const int s = g & 1;
                // --- V terms of the second half of the rows
                if (!rev && rows < C) w.set<rev>(power, lam16, r0, rows);
                if (!warp_wait(&v_full[s], (g >> 1) & 1)) { stop = true; break; }
#pragma unroll 1
                for (int h = 0; h < 2 && !stop; ++h) {
                    if (!warp_wait(&vt_empty[h], g & 1)) stop = true;
                    if (stop) break;
                    v_terms(smem_u32(sm + OFF_V + s * PANEL) + static_cast<uint32_t>(512 + t) * 16u,
                            smem_u32(sm + OFF_VT + h * VT_BUF) + static_cast<uint32_t>(t) * 16u, w, h, r0, rows, packed && rows < C);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&vt_full[2 + h]);
                }
                if (stop) break;
                if (lane == 0) mbar_arrive(&v_empty[s]);
                if (!state_only) {
                    // publish bf16(S) once Q S of the chunk before has read the old one
                    if (g > 0 && !warp_wait(o_full, (g - 1) & 1)) { stop = true; break; }
                    if (own) {
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch)
                            st_shared_v4(srow + ((static_cast<uint32_t>(ch) ^ (i & 7)) << 4), pack_bf16x2(S[4 * ch]),
                                         pack_bf16x2(S[4 * ch + 1]), pack_bf16x2(S[4 * ch + 2]), pack_bf16x2(S[4 * ch + 3]));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_full);
                }
                if (c == odd_at) lam = power(odd);
                const uint64_t fh = f32x2(lam.x, lam.x), fl = f32x2(lam.y, lam.y);
                if (!warp_wait(ds_full, g & 1)) { stop = true; break; }
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t a[16], b[16], d[16];
                    tmem_ld16(tds + 16 * h, a);
                    tmem_ld16(tds + DVS + 16 * h, b);
                    tmem_ld16(tds + 2 * DVS + 16 * h, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        uint64_t& x = S[8 * h + j / 2];
                        const uint64_t low = add2(f32x2(b[j], b[j + 1]), f32x2(d[j], d[j + 1]));
                        x = add2(fma2(x, fh, f32x2(a[j], a[j + 1])), fma2(x, fl, low));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_empty);
                if (rev && c == odd_at) lam = power(C);
            }
            if (stop) break;
            if (it.out && own) {
                float4* dst = reinterpret_cast<float4*>(it.out + (long)i * it.out_ld);
#pragma unroll
                for (int j = 0; j < DVS / 4; ++j) {
                    float4 x;
                    f32x2_split(S[2 * j], x.x, x.y);
                    f32x2_split(S[2 * j + 1], x.z, x.w);
                    dst[j] = x;
                }
            }
            if (kLean && it.to >= 0) {
                __threadfence();
                __syncwarp();
                if (lane == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p.wrap_ready + it.to) : "memory");
            }
        }
    } else {
        // ------------------------------------------------------ output warps
        const int q4 = warp & 3;
        const int row = q4 * 32 + lane;
        const uint32_t tlane = tbase + (static_cast<uint32_t>(q4 * 32) << 16);
        int g = 0;
        bool stop = state_only;
        for (int r = 0; !stop; ++r) {
            const Piece it = piece<KD, kRev, kLean>(p, r, cta, G);
            if (it.len < 0) break;
            const int nc = (it.len + C - 1) / C;
            const float g2 = p.log_decay[!packed ? it.c2 % p.H : it.c1] * 1.4426950408889634f;
            for (int c = 0; c < nc; ++c, ++g) {
                const int c0 = tc::chunk_row(rev, c, nc);
                const int rows = min(C, it.len - c0);
                const int s = g & 1;
                // the chunk before has been stored from the staging rows
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
                // lam^n of this row (rounded to bf16 with the output: a plain fp32
                // power will do)
                const int n = rev ? max(rows - 1 - row, 0) : row + 1;
                const float fac = n == 0 ? 1.f : exp2f(static_cast<float>(n) * g2);
                const uint64_t f2 = f32x2(fac, fac);
                // where the row goes: through staging rows with TMA (a dense
                // tensor clips rows past N itself), row by row on the ragged tail of
                // a packed sequence, whose next rows belong to another one, or nowhere
                const int how = q4 * 32 >= rows ? 0 : (!packed || q4 * 32 + 32 <= rows) ? 1 : row < rows ? 2 : 0;
                uint8_t* stg = sm + OFF_OST + q4 * 4096;
                const uint32_t sa = smem_u32(stg) + static_cast<uint32_t>(lane) * 128u;
                uint4* dst = reinterpret_cast<uint4*>(p.o + ((long)(it.t0 + c0 + row) * p.H + it.c1) * p.dv + DVS * it.vs);
                if (!warp_wait(o_full, g & 1)) { stop = true; break; }
                tc_fence_after();
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t x[32], y[32], hp[16];
                    tmem_ld32(tlane + TM_P + 128u * s + TM_OPV + 32 * h, x);
                    tmem_ld32(tlane + TM_OQS + 32 * h, y);
                    tmem_wait_ld();
                    if (h == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&o_empty[s]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        hp[i] = pack_bf16x2(fma2(f32x2(y[2 * i], y[2 * i + 1]), f2, f32x2(x[2 * i], x[2 * i + 1])));
                    if (how == 1) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            st_shared_v4(sa + ((static_cast<uint32_t>(4 * h + e) ^ (row & 7)) << 4), hp[4 * e], hp[4 * e + 1],
                                         hp[4 * e + 2], hp[4 * e + 3]);
                    } else if (how == 2) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[4 * h + e] = make_uint4(hp[4 * e], hp[4 * e + 1], hp[4 * e + 2], hp[4 * e + 3]);
                    }
                }
                if (how == 1) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (!packed) tma_store_3d(&map_o, stg, DVS * it.vs, it.t0 + c0 + q4 * 32, it.c2);
                        else tma_store_3d(&map_o, stg, DVS * it.vs, it.c1, it.t0 + c0 + q4 * 32);
                        bulk_commit();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait<0>();
        __syncwarp();
    }

    if (late) atomicExch(p.status, kStatusTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA_A) {
        tc_fence_after();
        tmem_dealloc(tbase, TMEM_COLS);
    }
}

}  // namespace tcd
}  // namespace lcl
