// diff_fwd.cu -- forward pass of differential attention for sm_103a (tcgen05 + TMA + TMEM).
//
// Per head, with two maps m = 1, 2 that share one value head of width 2d:
//     S_m = scale Q_m K_m^T + mask,  P_m = softmax(S_m),  O = (P_1 - lam P_2) V,
// and the log-sum-exp of both maps' rows; on request O_2 = P_2 V too, which the backward pass
// needs.  "FlashAttention V3：优化框架吞吐量的关键技术实践" §1.2 fuses mask, softmax and both
// products of one map; here the pair of maps is one kernel, so that V is read once for both
// and neither O_1 nor O_2 leaves the SM.
//
// Roles, ring and online softmax are those of attn_fwd.cuh, whose two query tiles of 128 rows
// become the two maps of the same 128 rows: one softmax warpgroup a map, ping-ponging on the
// tensor core, each with S (128 columns of TMEM, P over it) and its own accumulator of 128 value
// columns, since the maps' sums are known only at the end.  Both accumulators and both score
// tiles fill TMEM's 512 columns.  At the end each warpgroup combines 64 of the columns of both.
//
// At d = 64 that is a whole head.  At d = 128 the value head is 256 wide, twice what fits, so a
// unit takes one half of its columns and the scores are computed for each half: 16 d products
// per pair of tokens instead of 12 d.  (Each half reads the same q and k from L2.)
//
// Several heads may read one pair of key heads (H / Hkv): their units are handed out together
// (diff_units.cuh), so they share its tiles in L2.
//
// Measured, one sequence of 16384 tokens, 8 heads over 4 of d = 64, causal, with O_2: 650 us = 1269 TFLOP/s of 12 d;
// a step of both maps takes about 2900 cycles for 1536 of products, which the softmax warps need for its 32768 scores.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_fwd.cuh"
#include "diff_params.h"
#include "diff_units.cuh"

namespace gb300 {

template <int D, bool PK>
struct DiffFwdCfg {
    static constexpr bool PACKED = PK;
    static constexpr int BM = 128, NQ = 1, BN = 128;     // a unit: 128 rows of a head, both maps
    static constexpr int HEAD_DIM = D, CLUSTER = 1;
    static constexpr int VH = D / 64;                    // parts of 128 columns of a value head
    static constexpr int DV = 128;                       // value columns of a unit
    static constexpr int CB = 128 * 128;                 // 64 columns of a 128-row tile
    static constexpr int Q_BYTES = 2 * (D / 64) * CB;    // both maps' queries
    static constexpr int SLOT = 2 * CB;                  // 32 KB: both maps' keys (d 64) or one's, or V
    static constexpr int KSLOTS = D / 64;                // ring slots of a step's keys
    static constexpr int BAR_BYTES = 5120;
    static constexpr int SMEM_CAP = 227 * 1024;
    static constexpr int NSLOT = (SMEM_CAP - BAR_BYTES - 1024 - Q_BYTES) / SLOT;
    static constexpr int SMEM_BYTES = 1024 + Q_BYTES + NSLOT * SLOT + BAR_BYTES;
    static constexpr int S_COL0 = 0, O_COL0 = 256;
    static constexpr int NUM_SOFTMAX_WARPS = 8;
    static constexpr int PRODUCER_WARP = 8, MMA_WARP = 9, NUM_THREADS = 384;
    static constexpr int REG_SOFTMAX = 208, REG_CONTROL = 88;
    static constexpr int REG_POOL = 256 * REG_SOFTMAX + 128 * REG_CONTROL;
    // the running maximum moves when a score passes it by more than 2^TAU: P <= 2^8 meanwhile,
    // which bf16 holds with the same relative rounding
    static constexpr float TAU = 8.0f;
    static_assert(D == 64 || D == 128, "head dim");
    static_assert(NSLOT >= 4, "ring too small");
};

struct alignas(16) DiffFwdBars {
    uint64_t q_full, q_empty;
    uint64_t kv_full[8], kv_empty[8];
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t o_empty, sums_full;
    DiffHand hand;
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    float inv[2][2][128];    // 1 / sum of the maps' rows, by the parity of the unit: one map's warps may be a
                             // unit ahead of the other's
};
constexpr int kDiffTabOffset = 2816;
static_assert(sizeof(DiffFwdBars) <= kDiffTabOffset, "barrier block");
static_assert(kDiffTabOffset + sizeof(SortTab) <= 5120, "schedule table");

// Where a unit's rows live.
struct DiffAt {
    int h;                   // head
    int part;                // which 128 of the value columns
    int zq, zk, zv;          // head coordinates of q (map 1), k (map 1) and v
    size_t out_row;          // output row of the sequence's first token
    size_t out_step;         // output rows between two tokens
    size_t lse;              // LSE index of map 1 at the sequence's first token
    size_t lse_step;         // from map 1 to map 2
};

template <class C>
__device__ __forceinline__ DiffAt diff_at(const DiffFwdParams& p, const Unit& w)
{
    DiffAt a;
    const int z = w.z / C::VH, G = p.H / p.Hkv;
    a.part = w.z - z * C::VH;
    if constexpr (C::PACKED) {
        a.h = z;
        a.zq = 2 * z;
        a.zv = z / G;
        a.out_row = (size_t)w.y0 * p.H + z;
        a.out_step = (size_t)p.H;
        a.lse = (size_t)(2 * z) * p.f.T + w.y0;
        a.lse_step = (size_t)p.f.T;
    } else {
        const int b = z / p.H;
        a.h = z - b * p.H;
        a.zq = 2 * z;
        a.zv = b * p.Hkv + a.h / G;
        a.out_row = (size_t)z * p.f.N;
        a.out_step = 1;
        a.lse = (size_t)(2 * z) * p.f.N;
        a.lse_step = (size_t)p.f.N;
    }
    a.zk = 2 * a.zv;
    return a;
}

template <int D, bool PK>
__global__ void __launch_bounds__(DiffFwdCfg<D, PK>::NUM_THREADS, 1)
    diff_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const DiffFwdParams dp)
{
    using C = DiffFwdCfg<D, PK>;
    const FwdParams& p = dp.f;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* q_smem = smem;
    uint8_t* ring_smem = smem + C::Q_BYTES;
    DiffFwdBars* bars = reinterpret_cast<DiffFwdBars*>(ring_smem + C::NSLOT * C::SLOT);
    const volatile int* abort_flag = &bars->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const SortTab* tab = nullptr;
    if constexpr (C::PACKED) {
        if (p.num_seqs <= kSortMaxSeqs) {
            SortTab* t = reinterpret_cast<SortTab*>(reinterpret_cast<uint8_t*>(bars) + kDiffTabOffset);
            build_diff_tab<C>(p, t);
            tab = t;
        }
    }
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 1);
        mbar_init(smem_u32(&bars->q_empty), 1);
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), 1);
            mbar_init(smem_u32(&bars->kv_empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars->s_full[i]), 1);
            mbar_init(smem_u32(&bars->p_full[i]), 4);
            mbar_init(smem_u32(&bars->pv_done[i]), 1);
        }
        bars->hand.init(C::NUM_SOFTMAX_WARPS + 1);
        mbar_init(smem_u32(&bars->o_empty), 8);
        mbar_init(smem_u32(&bars->sums_full), 8);
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::PRODUCER_WARP && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == C::MMA_WARP) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    auto timed_out = [&]() {
        atomicExch(p.status, kStatusTimeout);
        *reinterpret_cast<volatile int*>(&bars->abort_flag) = 1;
    };

    DiffUnits<C> units(dp, tab, &bars->hand, abort_flag);

    if (warp == C::PRODUCER_WARP) {
        // ------------------------------------------------------------ TMA producer
        regs_decrease<C::REG_CONTROL>();
        if (lane == 0) {
            const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
            uint32_t ring = 0, uc = 0;
            bool ok = true;
            // the next ring slot, free and armed; false: stop, or (withheld) not armed
            auto slot_ready = [&](bool& issue) -> uint32_t {
                const uint32_t slot = ring % C::NSLOT;
                issue = false;
                if (!mbar_wait(smem_u32(&bars->kv_empty[slot]), ((ring / C::NSLOT) & 1) ^ 1, abort_flag,
                               p.timeout_ns)) {
                    ok = false;
                    return 0;
                }
                issue = ring + 1 != (uint32_t)p.withhold_kv;   // test hook: never arrives
                if (issue) mbar_arrive_expect_tx(smem_u32(&bars->kv_full[slot]), C::SLOT);
                ++ring;
                return slot;
            };
            Unit w;
            while (ok && units.give(w, ok)) {
                const DiffAt at = diff_at<C>(dp, w);
                if (!mbar_wait(smem_u32(&bars->q_empty), (uc & 1) ^ 1, abort_flag, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t qb = smem_u32(&bars->q_full);
                mbar_arrive_expect_tx(qb, C::Q_BYTES);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int cb = 0; cb < D / 64; ++cb)
                        tma_load_3d(smem_u32(q_smem + (i * (D / 64) + cb) * C::CB), &tmQ, qb, cb * 64, w.y0 + w.q0,
                                    at.zq + i, pol_q);
                ++uc;
                for (int jj = 0; jj < w.n && ok; ++jj) {
                    const int row = w.y0 + (w.t0 + jj) * C::BN;
                    bool issue;
#pragma unroll
                    for (int s = 0; s < C::KSLOTS && ok; ++s) {
                        const uint32_t slot = slot_ready(issue);
                        if (!issue) continue;
                        const uint32_t fb = smem_u32(&bars->kv_full[slot]);
                        const uint32_t dst = smem_u32(ring_smem + slot * C::SLOT);
                        // a slot: both maps' 64 columns (d 64), or one map's 128
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            tma_load_3d(dst + c * C::CB, &tmK, fb, D == 64 ? 0 : c * 64, row,
                                        at.zk + (D == 64 ? c : s), pol_kv);
                    }
                    if (!ok) break;
                    const uint32_t slot = slot_ready(issue);
                    if (!issue) continue;
                    const uint32_t fb = smem_u32(&bars->kv_full[slot]);
                    const uint32_t dst = smem_u32(ring_smem + slot * C::SLOT);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_3d(dst + c * C::CB, &tmV, fb, at.part * C::DV + c * 64, row, at.zv, pol_kv);
                }
            }
            if (!ok) timed_out();
            units.finish(ok);
            // every copy issued lands before shared memory is released
            const uint32_t armed = ring < C::NSLOT ? ring : C::NSLOT;
            for (uint32_t k = ring - armed; k < ring; ++k) {
                if (k + 1 == (uint32_t)p.withhold_kv) continue;
                mbar_wait(smem_u32(&bars->kv_full[k % C::NSLOT]), (k / C::NSLOT) & 1, nullptr, kCleanupTimeoutNs);
            }
            if (uc > 0) mbar_wait(smem_u32(&bars->q_full), (uc - 1) & 1, nullptr, kCleanupTimeoutNs);
        }
    } else if (warp == C::MMA_WARP) {
        // ------------------------------------------------------------ MMA issuer
        regs_decrease<C::REG_CONTROL>();
        constexpr uint32_t idesc_s = idesc_f32acc(1, 0, C::BM, C::BN);
        constexpr uint32_t idesc_o = idesc_f32acc(1, 1, C::BM, C::DV);
        const uint64_t q_desc = sdesc_sw128(smem_u32(q_smem), 16, 1024);
        const uint64_t k_desc = sdesc_sw128(smem_u32(ring_smem), 16, 1024);
        const uint64_t v_desc = sdesc_sw128(smem_u32(ring_smem), C::CB, 1024);
        uint32_t ring = 0, uc = 0, p_phase = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            bool r = ok && mbar_wait(smem_u32(bar), parity, abort_flag, p.timeout_ns);
            r = __all_sync(0xffffffffu, r);
            if (!r) ok = false;
            return r;
        };
        auto commit = [&](uint64_t* bar) { mma_commit_warp(smem_u32(bar)); };
        auto full = [&](uint32_t n) -> bool { return wait(&bars->kv_full[n % C::NSLOT], (n / C::NSLOT) & 1); };
        auto slot_of = [&](uint32_t n) { return n % C::NSLOT; };
        // S_i = Q_i K_i^T; the step's keys start at ring position nk
        auto issue_s = [&](int i, uint32_t nk) {
            const uint64_t a = q_desc + (uint64_t)((i * (D / 64) * C::CB) >> 4);
            const uint64_t b = k_desc + (uint64_t)((slot_of(D == 64 ? nk : nk + i) * C::SLOT + (D == 64 ? i * C::CB : 0)) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk / 4) * C::CB + (kk % 4) * 32) >> 4;
                mma_ss_warp<false>(tmem + C::S_COL0 + i * C::BN, a + off, b + off, idesc_s, kk > 0 ? 1u : 0u);
            }
        };
        // O_i (+)= P_i V
        auto issue_pv = [&](int i, uint32_t nv, bool accumulate) {
            const uint64_t b = v_desc + (uint64_t)((slot_of(nv) * C::SLOT) >> 4);
#pragma unroll
            for (int kk = 0; kk < C::BN / 16; ++kk)
                mma_ts_warp<false>(tmem + C::O_COL0 + i * C::DV, tmem + C::S_COL0 + i * C::BN + kk * 8,
                                   b + (uint64_t)((kk * 16 * 128) >> 4), idesc_o, (kk > 0 || accumulate) ? 1u : 0u);
        };
        // Packed rows behind the sequence are the next one's, or nobody's, and may hold anything: a
        // masked key has P = 0, but 0 times a NaN would be one.  They become 0 before the product.
        auto clear_tail = [&](const Unit& w, int jj, uint32_t nv) {
            if constexpr (C::PACKED) {
                const int live = w.N - (w.t0 + jj) * C::BN;
                if (live >= C::BN) return;
                uint8_t* v = ring_smem + slot_of(nv) * C::SLOT;
                for (int o = live * 128 + lane * 16; o < C::CB; o += 512) {
                    *reinterpret_cast<uint4*>(v + o) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(v + C::CB + o) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
        };
        Unit w;
        while (ok && units.take(w, ok)) {
            if (!wait(&bars->q_full, uc & 1)) break;
            for (int jj = 0; jj <= w.n && ok; ++jj) {
                // ring positions: V of step jj - 1, keys of step jj behind it
                const uint32_t nv = ring, nk = jj > 0 ? ring + 1 : ring;
                if (jj > 0) {
                    if (!full(nv)) break;
                    clear_tail(w, jj - 1, nv);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (jj > 0) {
                        if (!wait(&bars->p_full[i], (p_phase >> i) & 1)) break;
                        p_phase ^= 1u << i;
                        if (jj == 1 && i == 0 && !wait(&bars->o_empty, (uc & 1) ^ 1)) break;
                        tc_fence_after_sync();
                        issue_pv(i, nv, jj > 1);
                        if (jj == w.n) commit(&bars->pv_done[i]);
                        if (i == 1) commit(&bars->kv_empty[slot_of(nv)]);
                    }
                    if (jj < w.n) {
                        if ((i == 0 || C::KSLOTS == 2) && !full(nk + (C::KSLOTS == 2 ? i : 0))) break;
                        tc_fence_after_sync();
                        issue_s(i, nk);
                        commit(&bars->s_full[i]);
                        if (C::KSLOTS == 2 || i == 1) commit(&bars->kv_empty[slot_of(nk + (C::KSLOTS == 2 ? i : 0))]);
                        if (jj == w.n - 1 && i == 1) commit(&bars->q_empty);
                    }
                }
                ring = jj < w.n ? nk + C::KSLOTS : nv + 1;
            }
            ++uc;
        }
        if (!ok && lane == 0) timed_out();
        commit(&bars->drain);
        mbar_wait(smem_u32(&bars->drain), 0, nullptr, kCleanupTimeoutNs);
        __syncwarp();
    } else if (warp < C::NUM_SOFTMAX_WARPS) {
        // ------------------------------------------------------------ softmax, one warpgroup a map
        regs_increase<C::REG_SOFTMAX>();
        const int grp = warp >> 2, wq = warp & 3;
        const int row_in_tile = wq * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(wq * 32) << 16;
        const float NEG_INF = -__int_as_float(0x7f800000);
        const uint32_t s_addr = tmem + lane_addr + C::S_COL0 + grp * C::BN;
        uint32_t s_phase = 0, uc = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
            bool r = ok && mbar_wait(smem_u32(bar), parity, abort_flag, p.timeout_ns);
            r = __all_sync(0xffffffffu, r);
            if (!r) ok = false;
            return r;
        };
        Unit w;
        while (ok && units.take(w, ok)) {
            const int a = w.q0, row = a + row_in_tile;
            // keys allowed for row r: [lo, hi]; both grow with r
            auto key_bounds = [&](int r, int& lo, int& hi) {
                lo = 0;
                hi = w.N - 1;
                if (p.causal) hi = min(hi, r);
                if (p.window > 0) {
                    lo = r - p.window;
                    if (!p.causal) hi = min(hi, r + p.window);
                }
            };
            int jlo, jhi;
            key_bounds(row, jlo, jhi);
            float m_used = NEG_INF, l = 0.0f;
            const float c = p.c_log2;
            for (int jj = 0; jj < w.n; ++jj) {
                const int c0 = (w.t0 + jj) * C::BN;
                if (!wait_all(&bars->s_full[grp], s_phase)) break;
                s_phase ^= 1;
                tc_fence_after_sync();
                uint32_t sr[C::BN];
#pragma unroll
                for (int ch = 0; ch < C::BN / 32; ++ch) tmem_ld32p(s_addr + ch * 32, sr + ch * 32);
                tmem_wait_ld_only();
#pragma unroll
                for (int ch = 0; ch < C::BN / 32; ++ch) reg_fence32(sr + ch * 32);
                float* s = reinterpret_cast<float*>(sr);
                // mask only on tiles that cross a boundary of some row's allowed keys
                const bool edge = (c0 + C::BN > w.N) || (p.causal && c0 + C::BN - 1 > a) ||
                                  (p.window > 0 && (c0 < a + C::BM - 1 - p.window ||
                                                    (!p.causal && c0 + C::BN - 1 > a + p.window)));
                if (edge) {
                    int lo_min, hi_min, lo_max, hi_max;
                    key_bounds(a + wq * 32, lo_min, hi_min);
                    key_bounds(a + wq * 32 + 31, lo_max, hi_max);
                    const uint32_t span = (uint32_t)(jhi - jlo);
#pragma unroll
                    for (int ch = 0; ch < C::BN / 32; ++ch) {
                        const int x0 = c0 + ch * 32, x1 = x0 + 31;
                        if (!(x0 >= lo_max && x1 <= hi_min)) {
                            const int base = (x1 < lo_min || x0 > hi_max) ? -(1 << 30) : x0 - jlo;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if ((uint32_t)(base + e) > span) s[ch * 32 + e] = NEG_INF;
                        }
                    }
                }
                float mx[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float m = s[k];
#pragma unroll
                    for (int u = 1; u + 1 < C::BN / 8; u += 2) m = fmax3(m, s[k + 8 * u], s[k + 8 * u + 8]);
                    mx[k] = fmaxf(m, s[k + 8 * (C::BN / 8 - 1)]);
                }
                const float m_cand = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                           fmaxf(mx[6], mx[7])) * c;
                const bool resc = m_cand > m_used + C::TAU;
                const float alpha = resc ? ex2(m_used - m_cand) : 1.0f;   // ex2(-inf) = 0
                if (resc) {
                    l *= alpha;
                    m_used = m_cand;
                }
                const float mb = (m_used == NEG_INF) ? 0.0f : m_used;
                const float2 c2 = make_float2(c, c), b2 = make_float2(-mb, -mb);
                float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                 make_float2(0.f, 0.f)};
#pragma unroll
                for (int ch = 0; ch < C::BN / 64; ++ch) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int i0 = ch * 64 + 2 * e;
                        const float2 x = __ffma2_rn(make_float2(s[i0], s[i0 + 1]), c2, b2);
                        const float2 pp = make_float2(ex2(x.x), ex2(x.y));
                        acc[e & 3] = __fadd2_rn(acc[e & 3], pp);
                        pk[e] = pack_bf16x2(pp.x, pp.y);
                    }
                    tmem_st32p(s_addr + ch * 32, pk);
                }
                const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
                l += (a01.x + a01.y) + (a23.x + a23.y);
                // s_full of this step came behind the product of the one before
                if (jj > 0 && __any_sync(0xffffffffu, resc)) {
                    tc_fence_after_sync();
                    const float2 f2 = make_float2(alpha, alpha);
                    const uint32_t o_addr = tmem + lane_addr + C::O_COL0 + grp * C::DV;
                    uint32_t r[C::DV];
#pragma unroll
                    for (int ch = 0; ch < C::DV / 32; ++ch) tmem_ld32p(o_addr + ch * 32, r + ch * 32);
                    tmem_wait_ld_only();
#pragma unroll
                    for (int ch = 0; ch < C::DV / 32; ++ch) reg_fence32(r + ch * 32);
#pragma unroll
                    for (int e = 0; e < C::DV / 2; ++e) {
                        const float2 v2 = __fmul2_rn(
                            make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), f2);
                        r[2 * e] = __float_as_uint(v2.x);
                        r[2 * e + 1] = __float_as_uint(v2.y);
                    }
#pragma unroll
                    for (int ch = 0; ch < C::DV / 32; ++ch) tmem_st32p(o_addr + ch * 32, r + ch * 32);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[grp]));
            }
            if (!ok) break;
            // ---- the maps' sums change hands, then each warpgroup writes 64 columns of the difference
            const DiffAt at = diff_at<C>(dp, w);
            bars->inv[uc & 1][grp][row_in_tile] = l > 0.0f ? 1.0f / l : 0.0f;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->sums_full));
            if (!wait_all(&bars->sums_full, uc & 1)) break;
            if (!wait_all(&bars->pv_done[0], uc & 1)) break;
            if (!wait_all(&bars->pv_done[1], uc & 1)) break;
            tc_fence_after_sync();
            const float inv1 = bars->inv[uc & 1][0][row_in_tile], inv2 = bars->inv[uc & 1][1][row_in_tile];
            const float lam = __ldg(dp.lam + at.h);
            const size_t orow = at.out_row + (size_t)row * at.out_step;
            const size_t ocol = orow * (2 * D) + at.part * C::DV + grp * 64;
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                const uint32_t o_addr = tmem + lane_addr + C::O_COL0 + grp * 64 + ch * 32;
                uint32_t r1[32], r2[32];
                tmem_ld32p(o_addr, r1);
                tmem_ld32p(o_addr + C::DV, r2);
                tmem_wait_ld_only();
                reg_fence32(r1);
                reg_fence32(r2);
                uint32_t pk[16], pk2[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x2 = __uint_as_float(r2[2 * e]) * inv2, y2 = __uint_as_float(r2[2 * e + 1]) * inv2;
                    pk2[e] = pack_bf16x2(x2, y2);
                    pk[e] = pack_bf16x2(fmaf(__uint_as_float(r1[2 * e]), inv1, -(lam * x2)),
                                        fmaf(__uint_as_float(r1[2 * e + 1]), inv1, -(lam * y2)));
                }
                if (row < w.N) {
                    uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + ocol + ch * 32);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        o[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
                    if (dp.o2 != nullptr) {
                        uint4* o2 = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dp.o2) + ocol + ch * 32);
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            o2[v] = make_uint4(pk2[4 * v], pk2[4 * v + 1], pk2[4 * v + 2], pk2[4 * v + 3]);
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->o_empty));
            if (row < w.N && at.part == 0)
                p.lse[at.lse + grp * at.lse_step + row] =
                    (l == 0.0f ? NEG_INF : m_used + __log2f(l)) * 0.69314718055994531f;   // NaN stays one
            ++uc;
        }
        if (!ok) timed_out();
        tmem_wait_st();
    } else {
        regs_decrease<C::REG_CONTROL>();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == C::MMA_WARP) tmem_dealloc(tmem, 512);
}

template <int D, bool PK>
static cudaError_t launch_diff_fwd_t(const DiffFwdMaps& m, const DiffFwdParams& given, int sm_count,
                                     cudaStream_t stream)
{
    using C = DiffFwdCfg<D, PK>;
    auto kernel = diff_fwd_kernel<D, PK>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc would wait forever if the launch pool were smaller than the split
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
    if (attr.numRegs * C::NUM_THREADS < C::REG_POOL) return cudaErrorInvalidConfiguration;
    DiffFwdParams p = given;
    const int grid = diff_grid<C>(p, sm_count);
    if (grid < 1) return cudaErrorInvalidConfiguration;
    kernel<<<grid, C::NUM_THREADS, C::SMEM_BYTES, stream>>>(m.q, m.k, m.v, p);
    return cudaGetLastError();
}

cudaError_t launch_diff_fwd(const DiffFwdMaps& m, const DiffFwdParams& p, int d, int sm_count, cudaStream_t stream)
{
    const bool packed = p.f.cu_seqlens != nullptr;
    if (d == 64) return packed ? launch_diff_fwd_t<64, true>(m, p, sm_count, stream)
                               : launch_diff_fwd_t<64, false>(m, p, sm_count, stream);
    if (d == 128) return packed ? launch_diff_fwd_t<128, true>(m, p, sm_count, stream)
                                : launch_diff_fwd_t<128, false>(m, p, sm_count, stream);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
