// Chunked causal linear attention with a decay per head on tcgen05 tensor
// cores (bf16 in, fp32 state).
//
// Per chunk of up to C = 128 tokens (R of them valid), local rows l, lam =
// exp(log_decay[head]) (decay.cuh):
//
//   [P | Oqs] = Q_c [K_c ; bf16(S)^T]^T     one N = 192 product, fp32 in TMEM
//   P[l][m]  <- lam^(l-m) P[l][m], m <= l    fp32 factor, then bf16, in place
//   Opv       = P V_c                        A = P from TMEM
//   O[l]      = Opv[l] + lam^(l+1) Oqs[l]    joined in fp32 on the way out
//   dS        = K_c^T [V1 | V2 | V3]         one N = 192 product; V1 + V2 + V3 = lam^(R-1-m) V
//   S        <- lam^R S + dS1 + (dS2 + dS3)  fp32 registers
//
// The decay enters where a factor can be fp32.  The one place where it must
// multiply a tensor-core operand is the state update, whose weights run along
// the contraction: lam^(R-1-m) v_m is split into three bf16 terms (24 bits), so
// that the fp32 state keeps fp32 accuracy (one bf16 term: 2e-3 off, two: 2.6e-6,
// three: the rounding of the fp32 sums, 2e-7).  The terms sit side by side as
// 3 x 64 value columns: K is read once for the three.  The two halves of an
// output have accumulators of their own because they take different factors
// per row: scaling Q's rows instead would round them once more.
//
// Work item = (unit or sequence and head, 64 value columns), persistent CTAs,
// as in prefill_tc.cuh, whose items, segments, reverse order and packed batches
// it shares.  In reverse order rows take lam^(m-l) and lam^(R-1-l), the update
// lam^(m+1) (the state is held already decayed).
//
// Shared memory (225 KB): Q 2 x 32 KB; K 2 x 32 KB and one S^T of 16 KB in
// between, [K slot 0 | S^T | K slot 1] per 64-column panel, so that either slot
// and S^T form one run of rows (in slot 1 S^T comes first and the accumulator's
// columns swap); V 2 x 16 KB; the three V terms 48 KB.  O is staged in its
// chunk's V slot, whose last readers are the products that made it.
// TMEM (of 512 columns): [P | Oqs] 192, Opv 64, dS 192.
//
// Warp roles (16 warps):
//   w0 lane 0  : TMA producer for Q and K
//   w15 lane 0 : TMA producer for V
//   w1 lane 0  : MMA thread A: [P | Oqs], then P V
//   w14 lane 0 : MMA thread B: dS
//   w2..w5     : V terms of a chunk, then its masked and decayed P
//   w6..w9     : state warps (publish bf16(S)^T, absorb dS)
//   w10..w13   : output warps
// Every wait is bounded (mbar_wait); a timeout stops the CTA cleanly.
#pragma once
#include "decay.cuh"
#include "prefill_tc.cuh"

namespace lcl {
namespace tcd {

using tc::C;
using tc::DVS;
using tc::PANEL;
constexpr int SLOTS = 2;                    // Q, K, V ring depth
constexpr int TERMS = 3;                    // bf16 terms of the weighted V
constexpr int TILE_Q = 2 * PANEL;
constexpr int ST_BYTES = DVS * 128;         // S^T rows of one 64-column panel
constexpr int KPAN = 2 * PANEL + ST_BYTES;  // [K slot 0 | S^T | K slot 1]
constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + SLOTS * TILE_Q;
constexpr int OFF_V = OFF_K + 2 * KPAN;
constexpr int OFF_VT = OFF_V + SLOTS * PANEL;
constexpr int OFF_BAR = OFF_VT + TERMS * PANEL;
static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0 && OFF_VT % 1024 == 0 && ST_BYTES % 1024 == 0,
              "swizzled tiles need 1024-byte alignment");
// mbarriers (8 bytes each) at OFF_BAR, then the TMEM base and the abort flag
constexpr int BAR_Q_FULL = 0;                      // [2] TMA -> A
constexpr int BAR_Q_EMPTY = BAR_Q_FULL + SLOTS;    // [2] A ([P|Oqs]) -> TMA
constexpr int BAR_K_FULL = BAR_Q_EMPTY + SLOTS;    // [2] TMA -> A, B, P warps (ragged tail)
constexpr int BAR_K_EMPTY = BAR_K_FULL + SLOTS;    // [2] A ([P|Oqs]) + B (dS) -> TMA
constexpr int BAR_V_FULL = BAR_K_EMPTY + SLOTS;    // [2] TMA -> P warps
constexpr int BAR_V_EMPTY = BAR_V_FULL + SLOTS;    // [2] output warps (O stored from the slot) -> TMA
constexpr int BAR_VT_FULL = BAR_V_EMPTY + SLOTS;   // [2] by chunk parity: P warps (terms written) -> B
constexpr int BAR_VT_EMPTY = BAR_VT_FULL + SLOTS;  // B (dS) -> P warps
constexpr int BAR_F_FULL = BAR_VT_EMPTY + 1;       // A ([P|Oqs]) -> P warps, output warps
constexpr int BAR_F_FREE = BAR_F_FULL + 1;         // output warps (Oqs read) -> A
constexpr int BAR_P_READY = BAR_F_FREE + 1;        // P warps (bf16 P written) -> A
constexpr int BAR_O_FULL = BAR_P_READY + 1;        // A (P V) -> output warps, A
constexpr int BAR_O_EMPTY = BAR_O_FULL + 1;        // output warps (Opv read) -> A
constexpr int BAR_DS_FULL = BAR_O_EMPTY + 1;       // B -> state warps
constexpr int BAR_DS_EMPTY = BAR_DS_FULL + 1;      // state warps -> B
constexpr int BAR_S_FULL = BAR_DS_EMPTY + 1;       // state warps (S^T written) -> A
constexpr int BAR_ST_FREE = BAR_S_FULL + 1;        // A ([P|Oqs]) -> state warps: S^T may be rewritten
constexpr int BAR_TAB = BAR_ST_FREE + 1;           // P warps (decay table of an item written) -> P warps
constexpr int BAR_DRAIN_A = BAR_TAB + 1;
constexpr int BAR_DRAIN_B = BAR_DRAIN_A + 1;
constexpr int BAR_COUNT = BAR_DRAIN_B + 1;
constexpr int BAR_BYTES = 256;
static_assert((BAR_COUNT + 2) * 8 <= BAR_BYTES, "barrier area too small");
constexpr int OFF_TAB = OFF_BAR + BAR_BYTES;       // lam^n, n = 0 .. C, by item parity
constexpr int TAB_PAD = 32;                        // entries in front of lam^0
constexpr int TAB = TAB_PAD + C + 4;
constexpr int SMEM_BYTES = OFF_TAB + 2 * TAB * 4 + 1024;
static_assert(SMEM_BYTES <= 232448, "exceeds the 227 KB per-block shared memory limit");
constexpr int NUM_THREADS = 512;
constexpr int WARP_MMA_A = 1;
constexpr int WARP_MMA_B = 14;
constexpr int WARP_LOAD_V = 15;

constexpr uint32_t TM_F = 0;       // [P | Oqs]; [Oqs | P] in slot 1
constexpr uint32_t TM_OPV = 192;
constexpr uint32_t TM_DS = 256;    // three terms of 64 columns
constexpr uint32_t TMEM_COLS = 512;

// Shared-memory offsets of K slot s and of S^T inside a panel.
__device__ __forceinline__ constexpr int k_off(int s) { return s ? PANEL + ST_BYTES : 0; }

// The weighted V terms of a chunk (fp32 cut into three runs of 8 bits: each
// term is the upper half of what is left, so no conversion is needed and the
// three hold all 24 bits), by the 128 threads t of the P warps: 16-byte
// vectors of 8 values; a vector's place in the (swizzled) tile is the same in
// all four tiles, its row is place / 8.  Rows from `rows` on become zero; with
// `clear` (packed batch: they hold another sequence's tokens, or anything) they
// are cleared in the V and K slots too, since 0 x NaN is not 0.
template <int NP>
__device__ __forceinline__ void v_terms(uint32_t v, uint32_t vt, uint32_t k, const float* tab, int t, int rows, bool rev,
                                        bool clear) {
#pragma unroll 1
    for (int j = 0; j < PANEL / 16 / 128; ++j) {
        const int e = t + j * 128, row = e >> 3;
        const uint32_t off = static_cast<uint32_t>(e) * 16u;
        if (row >= rows) {
#pragma unroll
            for (int n = 0; n < TERMS; ++n) st_shared_v4(vt + n * PANEL + off, 0u, 0u, 0u, 0u);
            if (clear) {
                st_shared_v4(v + off, 0u, 0u, 0u, 0u);
#pragma unroll
                for (int pn = 0; pn < NP; ++pn) st_shared_v4(k + pn * KPAN + off, 0u, 0u, 0u, 0u);
            }
            continue;
        }
        const float w = tab[rev ? row + 1 : rows - 1 - row];
        const uint4 r = ld_shared_v4(v + off);
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
        for (int n = 0; n < TERMS; ++n) st_shared_v4(vt + n * PANEL + off, out[n][0], out[n][1], out[n][2], out[n][3]);
    }
}

// Out of line, one copy for all roles: they run once per item, and the
// kernel's instruction footprint is what its loops wait for (all roles of all
// SMs run at once; 112 KB with these inlined, P and the V terms unrolled and
// both orders in one instance took 10,000 cycles per chunk).
template <int KD>
__device__ __noinline__ tc::Item item(const tc::Params& p, int idx) {
    return tc::decode_item<true, KD>(p, idx);
}
// lam^n as two fp32 values, for the head of `it`
__device__ __noinline__ float2 item_power(const tc::Params& p, int c1, int c2, int n) {
    float2 f;
    decay::power2(p.log_decay[p.mode == 0 ? c2 % p.H : c1], n, f.x, f.y);
    return f;
}

// kRev: chunks visited last to first (the backward's reverse passes).
template <int KD, bool kRev>
__global__ void __launch_bounds__(NUM_THREADS, 1)
prefill_decay_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                     const __grid_constant__ tc::Params p) {
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
    uint64_t* f_full = bars + BAR_F_FULL;
    uint64_t* f_free = bars + BAR_F_FREE;
    uint64_t* p_ready = bars + BAR_P_READY;
    uint64_t* o_full = bars + BAR_O_FULL;
    uint64_t* o_empty = bars + BAR_O_EMPTY;
    uint64_t* ds_full = bars + BAR_DS_FULL;
    uint64_t* ds_empty = bars + BAR_DS_EMPTY;
    uint64_t* s_full = bars + BAR_S_FULL;
    uint64_t* st_free = bars + BAR_ST_FREE;
    uint64_t* tab_full = bars + BAR_TAB;
    uint64_t* drain_a = bars + BAR_DRAIN_A;
    uint64_t* drain_b = bars + BAR_DRAIN_B;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + BAR_COUNT);
    volatile int* abort = reinterpret_cast<volatile int*>(bars + BAR_COUNT + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = gridDim.x;
    const int cta = blockIdx.x;
    const bool state_only = p.state_only;
    constexpr bool rev = kRev;
    constexpr int NP = KD / 64;  // 64-column panels per Q / K tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], state_only ? 1 : 2);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 4);
            mbar_init(&vt_full[i], 4);
        }
        mbar_init(vt_empty, 1);
        mbar_init(f_full, 1);
        mbar_init(f_free, 4);
        mbar_init(p_ready, 4);
        mbar_init(o_full, 1);
        mbar_init(o_empty, 4);
        mbar_init(ds_full, 1);
        mbar_init(ds_empty, 4);
        mbar_init(s_full, 4);
        mbar_init(st_free, 1);
        mbar_init(tab_full, 4);
        mbar_init(drain_a, 1);
        mbar_init(drain_b, 1);
        *abort = 0;
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
        // ------------------------------------------------------ TMA producer: Q, K
        if (lane == 0) {
            int g = 0;
            bool stop = false;
            for (int r = 0; !stop; ++r) {
                const int idx = tc::item_index(r, cta, G);
                if (idx >= p.n_items) break;
                const tc::Item it = item<KD>(p, idx);
                const int nc = (it.len + C - 1) / C;
                for (int c = 0; c < nc; ++c) {
                    const int t = it.t0 + tc::chunk_row(rev, c, nc);
                    const int y = p.mode == 0 ? t : it.c1, z = p.mode == 0 ? it.c2 : t;
                    const int s = g % SLOTS, n = g / SLOTS;
                    if (!state_only) {
                        if (n > 0 && !mbar_wait(&q_empty[s], (n - 1) & 1, abort, p.status)) { stop = true; break; }
                        uint8_t* qb = sm + OFF_Q + s * TILE_Q;
                        mbar_arrive_expect_tx(&q_full[s], NP * PANEL);
#pragma unroll
                        for (int pn = 0; pn < NP; ++pn) tma_load_3d(qb + pn * PANEL, &map_q, &q_full[s], 64 * pn, y, z);
                    }
                    if (n > 0 && !mbar_wait(&k_empty[s], (n - 1) & 1, abort, p.status)) {
                        if (!state_only) tc::drain_wait(&q_full[s], n & 1);  // the Q copy just issued
                        stop = true;
                        break;
                    }
                    uint8_t* kb = sm + OFF_K + k_off(s);
                    mbar_arrive_expect_tx(&k_full[s], NP * PANEL);
#pragma unroll
                    for (int pn = 0; pn < NP; ++pn) tma_load_3d(kb + pn * KPAN, &map_k, &k_full[s], 64 * pn, y, z);
                    ++g;
                }
            }
            // no copy into shared memory may still be in flight at exit
            for (int x = (g >= SLOTS ? g - SLOTS : 0); x < g; ++x) {
                if (!state_only) tc::drain_wait(&q_full[x % SLOTS], (x / SLOTS) & 1);
                tc::drain_wait(&k_full[x % SLOTS], (x / SLOTS) & 1);
            }
        }
    } else if (warp == WARP_LOAD_V) {
        // ------------------------------------------------------ TMA producer: V
        if (lane == 0) {
            int g = 0;
            bool stop = false;
            for (int r = 0; !stop; ++r) {
                const int idx = tc::item_index(r, cta, G);
                if (idx >= p.n_items) break;
                const tc::Item it = item<KD>(p, idx);
                const int nc = (it.len + C - 1) / C;
                for (int c = 0; c < nc; ++c, ++g) {
                    const int t = it.t0 + tc::chunk_row(rev, c, nc);
                    const int y = p.mode == 0 ? t : it.c1, z = p.mode == 0 ? it.c2 : t;
                    const int s = g % SLOTS, n = g / SLOTS;
                    if (n > 0 && !mbar_wait(&v_empty[s], (n - 1) & 1, abort, p.status)) { stop = true; break; }
                    mbar_arrive_expect_tx(&v_full[s], PANEL);
                    tma_load_3d(sm + OFF_V + s * PANEL, &map_v, &v_full[s], DVS * it.vs, y, z);
                }
            }
            for (int x = (g >= SLOTS ? g - SLOTS : 0); x < g; ++x) tc::drain_wait(&v_full[x % SLOTS], (x / SLOTS) & 1);
        }
    } else if (warp == WARP_MMA_A) {
        // ------------------------------------------------------ MMA thread A
        if (lane == 0 && !state_only) {
            constexpr uint32_t id_f = idesc_bf16(128, C + DVS, 0, 0);  // Q [K ; S^T]^T
            constexpr uint32_t id_pv = idesc_bf16(128, DVS, 0, 1);     // P V (P from TMEM)
            const uint32_t sq = smem_u32(sm + OFF_Q), sk = smem_u32(sm + OFF_K), sv = smem_u32(sm + OFF_V);
            int total = 0;  // this CTA's chunks
            for (int r = 0;; ++r) {
                const int idx = tc::item_index(r, cta, G);
                if (idx >= p.n_items) break;
                total += (item<KD>(p, idx).len + C - 1) / C;
            }
            for (int g = 0; g < total; ++g) {
                // [P | Oqs], once Q, K and S^T are there, the output warps have read
                // Oqs of the chunk before and its P V (of another shape, so not
                // ordered before this product by itself) has read P
                const int s = g % SLOTS;
                if (!mbar_wait(s_full, g & 1, abort, p.status)) break;
                if (!mbar_wait(&q_full[s], (g / SLOTS) & 1, abort, p.status)) break;
                if (!mbar_wait(&k_full[s], (g / SLOTS) & 1, abort, p.status)) break;
                if (g > 0 && !mbar_wait(f_free, (g - 1) & 1, abort, p.status)) break;
                if (g > 0 && !mbar_wait(o_full, (g - 1) & 1, abort, p.status)) break;
                tc_fence_after();
                const uint64_t da = tc::kmaj_desc(sq + s * TILE_Q, 0, PANEL);
                const uint64_t db = tc::kmaj_desc(sk + (s ? PANEL : 0), 0, KPAN);
#pragma unroll
                for (int kk = 0; kk < KD / 16; ++kk)
                    mma_ss(tbase + TM_F, da + tc::kmaj_step(kk, PANEL), db + tc::kmaj_step(kk, KPAN), id_f, kk > 0);
                mma_commit(f_full);
                mma_commit(&q_empty[s]);
                mma_commit(&k_empty[s]);
                mma_commit(st_free);
                // P V
                if (!mbar_wait(p_ready, g & 1, abort, p.status)) break;
                if (g > 0 && !mbar_wait(o_empty, (g - 1) & 1, abort, p.status)) break;
                tc_fence_after();
                const uint32_t tp = tbase + TM_F + (s ? DVS : 0);
                const uint64_t dv = tc::mnmaj_desc(sv + s * PANEL, 0, PANEL);
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    mma_ts(tbase + TM_OPV, tp + kk * 8, dv + tc::mnmaj_step(kk), id_pv, kk > 0);
                mma_commit(o_full);
            }
            // every MMA issued by this thread must be finished before TMEM is freed
            mma_commit(drain_a);
            tc::drain_wait(drain_a, 0);
        }
        __syncwarp();
    } else if (warp == WARP_MMA_B) {
        // ------------------------------------------------------ MMA thread B
        if (lane == 0) {
            constexpr uint32_t id_ds = idesc_bf16(128, TERMS * DVS, 1, 1);  // K^T [V1 | V2 | V3]
            const uint32_t sk = smem_u32(sm + OFF_K);
            const uint64_t dv = tc::mnmaj_desc(smem_u32(sm + OFF_VT), 0, PANEL);
            int g = 0;
            bool stop = false;
            for (int r = 0; !stop; ++r) {
                const int idx = tc::item_index(r, cta, G);
                if (idx >= p.n_items) break;
                const int len = item<KD>(p, idx).len;
                for (int c0 = 0; c0 < len; c0 += C, ++g) {
                    const int s = g % SLOTS;
                    if (!mbar_wait(&k_full[s], (g / SLOTS) & 1, abort, p.status)) { stop = true; break; }
                    if (!mbar_wait(&vt_full[s], (g / SLOTS) & 1, abort, p.status)) { stop = true; break; }
                    if (g > 0 && !mbar_wait(ds_empty, (g - 1) & 1, abort, p.status)) { stop = true; break; }
                    tc_fence_after();
                    // at d = 64 both 64-row halves of K^T read the same panel (rows 64 .. 127 are ignored)
                    const uint64_t dk = tc::mnmaj_desc(sk + k_off(s), 0, KD == 128 ? KPAN : 0);
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_ss(tbase + TM_DS, dk + tc::mnmaj_step(kk), dv + tc::mnmaj_step(kk), id_ds, kk > 0);
                    mma_commit(ds_full);
                    mma_commit(vt_empty);
                    mma_commit(&k_empty[s]);
                }
            }
            mma_commit(drain_b);
            tc::drain_wait(drain_b, 0);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ------------------------------------------------------ P warps
        const int q4 = warp & 3;
        const int t = (warp - 2) * 32 + lane;  // 0 .. 127, for the table and the V terms
        const int row = q4 * 32 + lane;        // row of P
        const uint32_t tlane = tbase + (static_cast<uint32_t>(q4 * 32) << 16);
        int g = 0;
        bool stop = false;
        for (int r = 0; !stop; ++r) {
            const int idx = tc::item_index(r, cta, G);
            if (idx >= p.n_items) break;
            const tc::Item it = item<KD>(p, idx);
            // the item's table; the other one may still be read by a warp at the
            // item before, and nobody is two items behind (each waits here)
            float* tab = reinterpret_cast<float*>(sm + OFF_TAB) + (r & 1) * TAB + TAB_PAD;
            tab[t + 1] = item_power(p, it.c1, it.c2, t + 1).x;
            if (t == 0) tab[0] = 1.f;
            __syncwarp();
            if (lane == 0) mbar_arrive(tab_full);
            if (!tc::warp_wait(tab_full, r & 1, abort, p.status)) break;
            const int nc = (it.len + C - 1) / C;
            for (int c = 0; c < nc; ++c, ++g) {
                const int rows = min(C, it.len - tc::chunk_row(rev, c, nc));
                const int s = g % SLOTS;
                // --- V terms, once dS of the chunk before has read the old ones
                if (!tc::warp_wait(&v_full[s], (g / SLOTS) & 1, abort, p.status)) { stop = true; break; }
                const bool clear = p.mode == 1 && rows < C;
                if (clear && !tc::warp_wait(&k_full[s], (g / SLOTS) & 1, abort, p.status)) { stop = true; break; }
                if (g > 0 && !tc::warp_wait(vt_empty, (g - 1) & 1, abort, p.status)) { stop = true; break; }
                v_terms<NP>(smem_u32(sm + OFF_V + s * PANEL), smem_u32(sm + OFF_VT), smem_u32(sm + OFF_K + k_off(s)), tab, t,
                            rows, rev, clear);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&vt_full[s]);
                if (state_only) {
                    if (lane == 0) mbar_arrive(&v_empty[s]);
                    continue;
                }
                // --- P: 32-column pieces on the kept side of the diagonal piece
                // take lam^|l-m| as (factor of the row) x (factor of the column),
                // both exponents >= 0; the diagonal piece looks its factors up
                if (!tc::warp_wait(f_full, g & 1, abort, p.status)) { stop = true; break; }
                tc_fence_after();
                const uint32_t tp = tlane + TM_F + (s ? DVS : 0);
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
                    // over fp32 pieces that have been read
                    tmem_st16(tp + 16 * pc, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready);
            }
        }
    } else if (warp < 10) {
        // ------------------------------------------------------ state warps
        const int q4 = warp & 3;
        const int i = q4 * 32 + lane;  // key-dim row of S owned by this thread
        const bool own = KD == 128 || q4 < KD / 32;  // warp-uniform; at d = 64 warps 8, 9 only follow along
        const uint32_t tds = tbase + (static_cast<uint32_t>(q4 * 32) << 16) + TM_DS;
        // bf16(S[i][j]) goes to row j of S^T, key dim i
        const uint32_t colchunk = static_cast<uint32_t>((i & 63) >> 3);
        const uint32_t st_base = smem_u32(sm + OFF_K + (i >> 6) * KPAN + PANEL) + (i & 7) * 2;
        int g = 0;
        bool stop = false;
        for (int r = 0; !stop; ++r) {
            const int idx = tc::item_index(r, cta, G);
            if (idx >= p.n_items) break;
            const tc::Item it = item<KD>(p, idx);
            uint64_t S[DVS / 2];  // pairs of value columns
            if (it.init && p.init_transposed && own) {
                const float* src = it.init + (long)DVS * it.vs * KD + i;
#pragma unroll
                for (int j = 0; j < DVS; j += 2) S[j / 2] = f32x2(src[j * KD], src[(j + 1) * KD]);
            } else if (it.init && own) {
                const float4* src = reinterpret_cast<const float4*>(it.init + (long)i * p.dv + DVS * it.vs);
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
            const float2 lam_c = item_power(p, it.c1, it.c2, C);
            const int nc = (it.len + C - 1) / C;
            for (int c = 0; c < nc; ++c, ++g) {
                const int rows = min(C, it.len - tc::chunk_row(rev, c, nc));
                if (!state_only) {
                    // publish bf16(S)^T once the product of the chunk before has read the old one
                    if (g > 0 && !tc::warp_wait(st_free, (g - 1) & 1, abort, p.status)) { stop = true; break; }
                    if (own) {
#pragma unroll
                        for (int j = 0; j < DVS; j += 2) {
                            const uint32_t x = pack_bf16x2(S[j / 2]);
                            st_shared_b16(st_base + j * 128 + ((colchunk ^ (j & 7)) << 4), static_cast<unsigned short>(x));
                            st_shared_b16(st_base + (j + 1) * 128 + ((colchunk ^ ((j + 1) & 7)) << 4),
                                          static_cast<unsigned short>(x >> 16));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_full);
                }
                float2 lam = lam_c;  // lam^rows
                if (rows < C) lam = item_power(p, it.c1, it.c2, rows);
                if (!tc::warp_wait(ds_full, g & 1, abort, p.status)) { stop = true; break; }
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t a[16], b[16], d[16];
                    tmem_ld16(tds + 16 * h, a);
                    tmem_ld16(tds + DVS + 16 * h, b);
                    tmem_ld16(tds + 2 * DVS + 16 * h, d);
                    tmem_wait_ld();
                    const uint64_t fh = f32x2(lam.x, lam.x), fl = f32x2(lam.y, lam.y);
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
            }
            if (stop) break;
            if (p.s_out && it.write_state && own) {
                float4* dst = reinterpret_cast<float4*>(p.s_out + (it.state * KD + i) * p.dv + DVS * it.vs);
#pragma unroll
                for (int j = 0; j < DVS / 4; ++j) {
                    float4 x;
                    f32x2_split(S[2 * j], x.x, x.y);
                    f32x2_split(S[2 * j + 1], x.z, x.w);
                    dst[j] = x;
                }
            }
        }
    } else if (warp < 14) {
        if (!state_only) {
            // ------------------------------------------------------ output warps
            const int q4 = warp & 3;
            const int row = q4 * 32 + lane;
            const uint32_t tlane = tbase + (static_cast<uint32_t>(q4 * 32) << 16);
            int g = 0;
            int pending = -1;  // V slot whose O store may still be reading it
            bool stop = false;
            for (int r = 0; !stop; ++r) {
                const int idx = tc::item_index(r, cta, G);
                if (idx >= p.n_items) break;
                const tc::Item it = item<KD>(p, idx);
                const float g2 = p.log_decay[p.mode == 0 ? it.c2 % p.H : it.c1] * 1.4426950408889634f;
                const int nc = (it.len + C - 1) / C;
                for (int c = 0; c < nc; ++c, ++g) {
                    const int c0 = tc::chunk_row(rev, c, nc);
                    const int rows = it.len - c0;
                    const int s = g % SLOTS;
                    // lam^n of this row (rounded to bf16 with the output: a plain fp32 power will do)
                    const int n = rev ? max(min(rows, C) - 1 - row, 0) : row + 1;
                    const float fac = n == 0 ? 1.f : exp2f(static_cast<float>(n) * g2);
                    // --- Oqs, read out early: the next chunk's product overwrites it
                    if (!tc::warp_wait(f_full, g & 1, abort, p.status)) { stop = true; break; }
                    tc_fence_after();
                    uint32_t q0[32], q1[32];
                    tmem_ld32(tlane + TM_F + (s ? 0 : C), q0);
                    tmem_ld32(tlane + TM_F + (s ? 0 : C) + 32, q1);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(f_free);
                        if (pending >= 0) {
                            bulk_wait_read<0>();
                            mbar_arrive(&v_empty[pending]);
                        }
                    }
                    __syncwarp();
                    // --- Opv, joined with it
                    if (!tc::warp_wait(o_full, g & 1, abort, p.status)) { stop = true; break; }
                    tc_fence_after();
                    uint32_t hp[32];
                    const uint64_t f2 = f32x2(fac, fac);
                    auto join = [&](int h, const uint32_t (&qs)[32]) {
                        uint32_t x[32];
                        tmem_ld32(tlane + TM_OPV + 32 * h, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            hp[16 * h + i] = pack_bf16x2(fma2(f32x2(qs[2 * i], qs[2 * i + 1]), f2, f32x2(x[2 * i], x[2 * i + 1])));
                    };
                    join(0, q0);
                    join(1, q1);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_empty);
                    // --- out: through the chunk's V slot with TMA (a dense tensor clips
                    // rows past N itself), row by row on the ragged tail of a packed
                    // sequence, whose next rows belong to another one
                    if (q4 * 32 >= rows) {
                        // this warp's rows all lie past the end of the sequence
                    } else if (p.mode == 0 || q4 * 32 + 32 <= rows) {
                        uint8_t* stg = sm + OFF_V + s * PANEL + q4 * 4096;
                        const uint32_t sa = smem_u32(stg) + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch)
                            st_shared_v4(sa + ((static_cast<uint32_t>(ch) ^ (row & 7)) << 4), hp[4 * ch], hp[4 * ch + 1],
                                         hp[4 * ch + 2], hp[4 * ch + 3]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (p.mode == 0) tma_store_3d(&map_o, stg, DVS * it.vs, it.t0 + c0 + q4 * 32, it.c2);
                            else tma_store_3d(&map_o, stg, DVS * it.vs, it.c1, it.t0 + c0 + q4 * 32);
                            bulk_commit();
                        }
                    } else if (row < rows) {
                        uint4* dst = reinterpret_cast<uint4*>(
                            p.o + ((long)(it.t0 + c0 + row) * p.H + it.c1) * p.dv + DVS * it.vs);
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch)
                            dst[ch] = make_uint4(hp[4 * ch], hp[4 * ch + 1], hp[4 * ch + 2], hp[4 * ch + 3]);
                    }
                    pending = s;
                }
            }
            if (lane == 0) bulk_wait<0>();
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA_A) {
        tc_fence_after();
        tmem_dealloc(tbase, TMEM_COLS);
    }
}

}  // namespace tcd
}  // namespace lcl
