// diff_fwd_wide.cu -- forward pass of differential attention at d = 128 in two launches: the rows'
// largest scores and sums of weights (and the log-sum-exps), then one product with both maps' weights.
//
//     S_m = scale Q_m K_m^T + mask,  M_m = max S_m,  l_m = sum exp(S_m - M_m),
//     O = (exp(S_1 - M_1) - lam l_1 / l_2 exp(S_2 - M_2)) V / l_1
//
// A value head of 256 columns leaves no room in TMEM for the two accumulators of diff_fwd.cu, which
// therefore takes each half of it with scores of its own: 16 d products per pair of tokens (two scores of
// 2 d and two products of 2 d for each half).  With the sums known the maps' weights are subtracted before the
// product, and one accumulator of 256 columns takes it: 4 d products for the sums, 4 d for the scores
// again, 4 d for O: 12 d, with as many exponentials, and no rescaling in the second launch.
//
// What passes from the first launch to the second is M_m and l_m, not the log-sum-exp M_m + log l_m: that one is
// rounded by half a step of its own size, an error of all of a row's weights (3 % where scores are some 2^18), while
// M_m, whatever its rounding, is the same number in l_m and in the weights.  The four floats of a row and head lie
// at the start of its output row, which the second launch overwrites when it has used them.
// Measured, 16 heads over 4 key pairs, 16384 tokens, causal: 3020 us in one launch, 2035 in two
// (1620 TFLOP/s of 12 d).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "attn_fwd.cuh"
#include "diff_params.h"
#include "diff_units.cuh"

namespace gb300 {

// ------------------------------------------------------------------ largest scores and sums
// A unit is 256 query rows of one map, as two tiles that share the stream of key tiles.  A step is 256 keys: a
// 128 x 256 x 16 product of two shared-memory operands reads 12 KB in its 128 cycles, one of 128 x 128 the 8 KB
// that shared memory has for its 64, with nothing left for TMA.  A tile's scores fill half of TMEM; the
// tensor pipe works on one tile's while the warps load the other's, two warpgroups a tile with half of the keys
// each, which join their sums at the end (one warpgroup a tile left the schedulers two warps, and half of their
// slots empty).
template <bool PK>
struct DiffLseCfg {
    static constexpr bool PACKED = PK;
    static constexpr int BM = 128, NQ = 2, BN = 256, D = 128, HEAD_DIM = D, CLUSTER = 1;
    static constexpr int CB = 128 * 128;                 // 64 columns of 128 rows
    static constexpr int Q_BYTES = 2 * NQ * CB, SLOT = 4 * CB;
    static constexpr int NSLOT = 2;
    static constexpr int TAB_OFF = 2560, BAR_BYTES = TAB_OFF + 2048;
    static constexpr int SMEM_BYTES = 1024 + Q_BYTES + NSLOT * SLOT + BAR_BYTES;
    static constexpr int COMPUTE_WARPS = 16, PRODUCER_WARP = 16, MMA_WARP = 17, NUM_THREADS = 640;
    static constexpr int REG_SOFTMAX = 104, REG_CONTROL = 64;
    static constexpr int REG_POOL = 512 * REG_SOFTMAX + 128 * REG_CONTROL;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static_assert(TAB_OFF + sizeof(SortTab) <= BAR_BYTES, "schedule table");
};

struct alignas(16) DiffLseBars {
    uint64_t q_full, q_empty;
    uint64_t k_full[2], k_empty[2];
    uint64_t s_full[2], s_free[2];                       // tile
    uint64_t half_full[2], half_free[2];                 // tile
    DiffHand hand;
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    float2 half[2][128];                                 // maximum and sum of the second half's keys
};
static_assert(sizeof(DiffLseBars) <= 2560, "barrier block");

// Keys [lo, hi] that row r may use; both grow with r.
__device__ __forceinline__ void diff_key_bounds(const FwdParams& p, int N, int r, int& lo, int& hi)
{
    lo = 0;
    hi = N - 1;
    if (p.causal) hi = min(hi, r);
    if (p.window > 0) {
        lo = r - p.window;
        if (!p.causal) hi = min(hi, r + p.window);
    }
}

// Some row of [a, a + 128) may not use some key of [c0, c0 + keys).
template <int keys>
__device__ __forceinline__ bool diff_edge(const FwdParams& p, int N, int a, int c0)
{
    return (c0 + keys > N) || (p.causal && c0 + keys - 1 > a) ||
           (p.window > 0 && (c0 < a + 127 - p.window || (!p.causal && c0 + keys - 1 > a + p.window)));
}

template <bool PK>
__global__ void __launch_bounds__(DiffLseCfg<PK>::NUM_THREADS, 1)
    diff_lse_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const DiffFwdParams dp)
{
    using C = DiffLseCfg<PK>;
    constexpr int D = C::D;
    const FwdParams& p = dp.f;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* q_smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring_smem = q_smem + C::Q_BYTES;
    DiffLseBars* bars = reinterpret_cast<DiffLseBars*>(ring_smem + C::NSLOT * C::SLOT);
    const volatile int* abort_flag = &bars->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const SortTab* tab = nullptr;
    if constexpr (C::PACKED) {
        if (p.num_seqs <= kSortMaxSeqs) {
            SortTab* t = reinterpret_cast<SortTab*>(reinterpret_cast<uint8_t*>(bars) + C::TAB_OFF);
            build_diff_tab<C>(p, t);
            tab = t;
        }
    }
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 1);
        mbar_init(smem_u32(&bars->q_empty), 1);
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(smem_u32(&bars->k_full[s]), 1);
            mbar_init(smem_u32(&bars->k_empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars->s_full[i]), 1);
            mbar_init(smem_u32(&bars->s_free[i]), 8);
            mbar_init(smem_u32(&bars->half_full[i]), 4);
            mbar_init(smem_u32(&bars->half_free[i]), 4);
        }
        bars->hand.init(C::COMPUTE_WARPS + 1);
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort_flag = 0;
        fence_mbar_init();
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
    // all lanes try once, which is the usual case; else they poll until the limit
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        const uint32_t a = smem_u32(bar);
        if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
        return __all_sync(0xffffffffu, mbar_wait(a, parity, abort_flag, p.timeout_ns));
    };

    DiffUnits<C> units(dp, tab, &bars->hand, abort_flag);

    if (warp == C::PRODUCER_WARP) {
        regs_decrease<C::REG_CONTROL>();
        if (lane == 0) {
            const uint64_t pol_q = l2_policy_evict_first(), pol_k = l2_policy_evict_last();
            uint32_t ring = 0, uc = 0;
            bool ok = true;
            Unit w;
            while (ok && units.give(w, ok)) {
                if (!mbar_wait(smem_u32(&bars->q_empty), (uc & 1) ^ 1, abort_flag, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t qb = smem_u32(&bars->q_full);
                mbar_arrive_expect_tx(qb, C::Q_BYTES);
#pragma unroll
                for (int i = 0; i < 2 * C::NQ; ++i)
                    tma_load_3d(smem_u32(q_smem + i * C::CB), &tmQ, qb, (i & 1) * 64, w.y0 + w.q0 + (i >> 1) * C::BM, w.z,
                                pol_q);
                ++uc;
                // map z = 2 h + m (behind 2 H b) reads the keys 2 (h / G) + m (behind 2 Hkv b)
                const int G = dp.H / dp.Hkv, b = C::PACKED ? 0 : w.z / (2 * dp.H), zz = w.z - b * 2 * dp.H;
                const int zk = 2 * (b * dp.Hkv + (zz >> 1) / G) + (zz & 1);
                for (int jj = 0; jj < w.n; ++jj) {
                    const uint32_t slot = ring % C::NSLOT;
                    if (!mbar_wait(smem_u32(&bars->k_empty[slot]), ((ring / C::NSLOT) & 1) ^ 1, abort_flag, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    if (++ring == (uint32_t)p.withhold_kv) continue;      // test hook: never arrives
                    const uint32_t fb = smem_u32(&bars->k_full[slot]);
                    mbar_arrive_expect_tx(fb, C::SLOT);
#pragma unroll
                    for (int c = 0; c < 4; ++c)            // 64 columns of 256 keys, then the other 64
                        tma_load_3d(smem_u32(ring_smem + slot * C::SLOT + c * C::CB), &tmK, fb, (c >> 1) * 64,
                                    w.y0 + (w.t0 + jj) * C::BN + (c & 1) * 128, zk, pol_k);
                }
            }
            if (!ok) timed_out();
            units.finish(ok);
            // every copy issued lands before shared memory is released
            for (uint32_t k = ring < C::NSLOT ? 0 : ring - C::NSLOT; k < ring; ++k)
                if (k + 1 != (uint32_t)p.withhold_kv)
                    mbar_wait(smem_u32(&bars->k_full[k % C::NSLOT]), (k / C::NSLOT) & 1, nullptr, kCleanupTimeoutNs);
            if (uc > 0) mbar_wait(smem_u32(&bars->q_full), (uc - 1) & 1, nullptr, kCleanupTimeoutNs);
        }
    } else if (warp == C::MMA_WARP) {
        regs_decrease<C::REG_CONTROL>();
        constexpr uint32_t idesc = idesc_f32acc(1, 0, C::BM, C::BN);
        const uint64_t q_desc = sdesc_sw128(smem_u32(q_smem), 16, 1024), k_desc = sdesc_sw128(smem_u32(ring_smem), 16, 1024);
        uint32_t ring = 0, uc = 0, count[2] = {0, 0};
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            ok = ok && warp_wait(bar, parity);
            return ok;
        };
        Unit w;
        while (ok && units.take(w, ok)) {
            int L[2], R[2];
            tile_steps<C>(w, 0, p, L[0], R[0]);
            tile_steps<C>(w, 1, p, L[1], R[1]);
            if (!wait(&bars->q_full, uc & 1)) break;
            for (int jj = 0; jj < w.n && ok; ++jj, ++ring) {
                const uint32_t slot = ring % C::NSLOT;
                if (!wait(&bars->k_full[slot], (ring / C::NSLOT) & 1)) break;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (jj < L[i] || jj >= R[i]) continue;
                    if (count[i] > 0 && !wait(&bars->s_free[i], (count[i] - 1) & 1)) break;
                    ++count[i];
                    tc_fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss_warp<false>(tmem + i * C::BN, q_desc + (((2 * i + kk / 4) * C::CB + (kk % 4) * 32) >> 4),
                                           k_desc + ((slot * C::SLOT + (kk / 4) * 2 * C::CB + (kk % 4) * 32) >> 4), idesc,
                                           kk > 0 ? 1u : 0u);
                    mma_commit_warp(smem_u32(&bars->s_full[i]));
                }
                if (!ok) break;
                mma_commit_warp(smem_u32(&bars->k_empty[slot]));
            }
            if (!ok) break;
            mma_commit_warp(smem_u32(&bars->q_empty));
            ++uc;
        }
        if (!ok && lane == 0) timed_out();
        mma_commit_warp(smem_u32(&bars->drain));
        mbar_wait(smem_u32(&bars->drain), 0, nullptr, kCleanupTimeoutNs);
        __syncwarp();
    } else if (warp < C::COMPUTE_WARPS) {
        regs_increase<C::REG_SOFTMAX>();
        constexpr int HC = C::BN / 2, CH = 64;           // keys of a warpgroup, loaded at once
        const int tile = warp >> 3, half = (warp >> 2) & 1, wq = warp & 3, trow = wq * 32 + lane;
        const uint32_t s_addr = tmem + ((uint32_t)(wq * 32) << 16) + tile * C::BN + half * HC;
        const float NEG_INF = -__int_as_float(0x7f800000), c = p.c_log2;
        uint32_t count = 0, uc = 0;
        bool ok = true;
        Unit w;
        while (ok && units.take(w, ok)) {
            int L, R;
            tile_steps<C>(w, tile, p, L, R);
            const int a = w.q0 + tile * C::BM, row = a + trow;
            int jlo, jhi;
            diff_key_bounds(p, w.N, row, jlo, jhi);
            if (jlo > jhi) jlo = jhi;                     // a row behind the sequence, which is not stored
            const uint32_t span = (uint32_t)(jhi - jlo);
            float m_used = NEG_INF;
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            for (int jj = L; jj < R; ++jj) {
                const int c0 = (w.t0 + jj) * C::BN + half * HC;
                ok = warp_wait(&bars->s_full[tile], count & 1);
                ++count;
                if (!ok) break;
                tc_fence_after_sync();
                const bool edge = diff_edge<HC>(p, w.N, a, c0);
#pragma unroll
                for (int part = 0; part < HC / CH; ++part) {
                    uint32_t sr[CH];
#pragma unroll
                    for (int ch = 0; ch < CH; ch += 32) tmem_ld32p(s_addr + part * CH + ch, sr + ch);
                    tmem_wait_ld_only();
#pragma unroll
                    for (int ch = 0; ch < CH; ch += 32) reg_fence32(sr + ch);
                    if (part == HC / CH - 1) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&bars->s_free[tile]));
                    }
                    float* s = reinterpret_cast<float*>(sr);
                    if (edge) {
                        const uint32_t first = (uint32_t)(c0 + part * CH - jlo);
#pragma unroll
                        for (int e = 0; e < CH; ++e)
                            if (first + (uint32_t)e > span) s[e] = NEG_INF;
                    }
                    float mx[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float m = s[k];
#pragma unroll
                        for (int u = 1; u + 1 < CH / 4; u += 2) m = fmax3(m, s[k + 4 * u], s[k + 4 * u + 4]);
                        mx[k] = fmaxf(m, s[k + 4 * (CH / 4 - 1)]);
                    }
                    const float m_cand = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * c;
                    if (m_cand > m_used) {                // a thread's own sums are all there is to rescale
                        const float alpha = ex2(m_used - m_cand);    // ex2(-inf) = 0
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[k] = __fmul2_rn(acc[k], make_float2(alpha, alpha));
                        m_used = m_cand;
                    }
                    const float mb = m_used == NEG_INF ? 0.0f : m_used;
                    const float2 c2 = make_float2(c, c), b2 = make_float2(-mb, -mb);
#pragma unroll
                    for (int e = 0; e < CH / 2; ++e) {
                        const float2 x = __ffma2_rn(make_float2(s[2 * e], s[2 * e + 1]), c2, b2);
                        acc[e & 3] = __fadd2_rn(acc[e & 3], make_float2(ex2(x.x), ex2(x.y)));
                    }
                }
            }
            if (!ok) break;
            const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
            float l = (a01.x + a01.y) + (a23.x + a23.y);
            if (half == 1) {
                ok = warp_wait(&bars->half_free[tile], (uc & 1) ^ 1);
                if (!ok) break;
                bars->half[tile][trow] = make_float2(m_used, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->half_full[tile]));
            } else {
                ok = warp_wait(&bars->half_full[tile], uc & 1);
                if (!ok) break;
                const float2 o = bars->half[tile][trow];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->half_free[tile]));
                const float top = fmaxf(m_used, o.x), mb = top == NEG_INF ? 0.0f : top;
                l = fmaf(l, ex2(m_used - mb), o.y * ex2(o.x - mb));
                if (row < w.N) {
                    const size_t at = C::PACKED ? (size_t)w.z * p.T + w.y0 : (size_t)w.z * p.N;
                    // a sum that is NaN stays one
                    p.lse[at + row] = (l == 0.0f ? NEG_INF : top + __log2f(l)) * 0.69314718055994531f;
                    // for the second launch: 16 bytes at the start of the head's output row, 8 of them a map's
                    const size_t orow = C::PACKED ? (size_t)(w.y0 + row) * dp.H + (w.z >> 1) : (size_t)(w.z >> 1) * p.N + row;
                    reinterpret_cast<float2*>(static_cast<__nv_bfloat16*>(p.o) + orow * (2 * D))[w.z & 1] = make_float2(mb, l);
                }
            }
            ++uc;
        }
        if (!ok) timed_out();
    } else {
        regs_decrease<C::REG_CONTROL>();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == C::MMA_WARP) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ the output
// A unit is 256 query rows of a head for a cluster of two CTAs: each has 128 of them, in its registers and TMEM,
// and half of every tile of K (64 keys) and V (128 columns), which the paired products (cta_group::2) of both
// read.  A step's scores of both maps (128 keys) fill 256 TMEM columns, which the compute warps load at once and
// give back; they take half of the keys of both maps each and put the difference of the weights, rounded once, into
// shared memory.  CTA 0's MMA warp issues the next step's scores before the product with it, so the tensor pipes
// work on both while the weights are made; CTA 1's tells it what has landed there.
//
// By itself a CTA would move 384 KB of shared memory a step (operands of 16 128 x 128 and 8 128 x 256 products of 16,
// what TMA and the compute warps write), at 128 bytes a cycle half as long again as the 2048 cycles of products.  A pair's CTA
// moves 256 KB.
template <bool PK>
struct DiffOutCfg {
    static constexpr bool PACKED = PK;
    static constexpr int BM = 128, NQ = 2, BN = 128, D = 128, HEAD_DIM = D, CLUSTER = 2;
    static constexpr int CB = 128 * 128, HB = 64 * 128;              // 64 columns of 128 rows, of 64
    static constexpr int Q_BYTES = 4 * CB, W_BYTES = 2 * CB, SLOT = 2 * HB, NSLOT = 8;
    static constexpr int TAB_OFF = 384, BAR_BYTES = 384 + 1792;
    static constexpr int SMEM_BYTES = Q_BYTES + W_BYTES + NSLOT * SLOT + BAR_BYTES;   // no room for alignment
    static constexpr int O_COL = 256;
    static constexpr int PRODUCER_WARP = 8, MMA_WARP = 9, NUM_THREADS = 384;
    static constexpr int REG_COMPUTE = 208, REG_CONTROL = 88;
    static constexpr int REG_POOL = 256 * REG_COMPUTE + 128 * REG_CONTROL;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static_assert(TAB_OFF + sizeof(SortTab) <= BAR_BYTES, "schedule table");
};

struct alignas(16) DiffOutBars {
    uint64_t q_full, q_empty;
    uint64_t kv_full[8], kv_empty[8];
    uint64_t s_full, s_free, w_full, w_free, o_full, o_empty;      // s_free, w_full and o_empty: CTA 0's count both
    DiffHand hand;
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(DiffOutBars) <= 384, "barrier block");

__device__ __forceinline__ void pair_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_mma_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
// One arrival on the barrier at this place in both CTAs when the products issued so far are done.
__device__ __forceinline__ void pair_commit_warp(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

template <bool PK>
__global__ void __launch_bounds__(DiffOutCfg<PK>::NUM_THREADS, 1)
    diff_out_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const DiffFwdParams dp)
{
    using C = DiffOutCfg<PK>;
    const FwdParams& p = dp.f;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* q_smem = smem;
    uint8_t* w_smem = smem + C::Q_BYTES;
    uint8_t* ring_smem = w_smem + C::W_BYTES;
    DiffOutBars* bars = reinterpret_cast<DiffOutBars*>(ring_smem + C::NSLOT * C::SLOT);
    const volatile int* abort_flag = &bars->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)pair_rank();
    if ((smem_u32(smem) & 1023) != 0) {                    // no kernel of this file has static shared memory
        if (threadIdx.x == 0) atomicExch(p.status, kStatusTimeout);
        return;
    }

    const SortTab* tab = nullptr;
    if constexpr (C::PACKED) {
        if (p.num_seqs <= kSortMaxSeqs) {
            SortTab* t = reinterpret_cast<SortTab*>(reinterpret_cast<uint8_t*>(bars) + C::TAB_OFF);
            build_diff_tab<C>(p, t);
            tab = t;
        }
    }
    if (threadIdx.x == 0) {
        // CTA 0's full barriers count its own copies and CTA 1's word that its have landed
        const uint32_t sides = rank == 0 ? 2 : 1;
        mbar_init(smem_u32(&bars->q_full), sides);
        mbar_init(smem_u32(&bars->q_empty), 1);
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), sides);
            mbar_init(smem_u32(&bars->kv_empty[s]), 1);
        }
        mbar_init(smem_u32(&bars->s_full), 1);
        mbar_init(smem_u32(&bars->s_free), 16);
        mbar_init(smem_u32(&bars->w_full), 16);
        mbar_init(smem_u32(&bars->w_free), 1);
        mbar_init(smem_u32(&bars->o_full), 1);
        mbar_init(smem_u32(&bars->o_empty), 16);
        bars->hand.init(9);                                // the MMA warp and the compute warps
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bars->tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before_sync();
    __syncthreads();
    pair_sync();                                           // both CTAs' barriers are there
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    const int G = dp.H / dp.Hkv;
    auto timed_out = [&]() {
        atomicExch(p.status, kStatusTimeout);
        *reinterpret_cast<volatile int*>(&bars->abort_flag) = 1;
    };
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        const uint32_t a = smem_u32(bar);
        if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
        return __all_sync(0xffffffffu, mbar_wait(a, parity, abort_flag, p.timeout_ns));
    };

    DiffUnits<C> units(dp, tab, &bars->hand, abort_flag);

    if (warp == C::PRODUCER_WARP) {
        regs_decrease<C::REG_CONTROL>();
        if (lane == 0) {
            const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
            uint32_t ring = 0, uc = 0;
            bool ok = true;
            // the next slot, free and armed; false: stop, or (withheld) not armed
            auto ready = [&](uint32_t& slot) -> bool {
                slot = ring % C::NSLOT;
                if (!ok) return false;
                if (!mbar_wait(smem_u32(&bars->kv_empty[slot]), ((ring / C::NSLOT) & 1) ^ 1, abort_flag, p.timeout_ns)) {
                    ok = false;
                    return false;
                }
                if (++ring == (uint32_t)p.withhold_kv) return false;      // test hook: never arrives
                mbar_arrive_expect_tx(smem_u32(&bars->kv_full[slot]), C::SLOT);
                return true;
            };
            Unit w;
            while (ok && units.give(w, ok)) {
                // heads of q (map 1), of V, of k (map 1)
                const int b = C::PACKED ? 0 : w.z / dp.H, zv = b * dp.Hkv + (w.z - b * dp.H) / G, zk = 2 * zv;
                if (!mbar_wait(smem_u32(&bars->q_empty), (uc & 1) ^ 1, abort_flag, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t qb = smem_u32(&bars->q_full);
                mbar_arrive_expect_tx(qb, C::Q_BYTES);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tma_load_3d(smem_u32(q_smem + i * C::CB), &tmQ, qb, (i & 1) * 64, w.y0 + w.q0 + rank * C::BM,
                                2 * w.z + (i >> 1), pol_q);
                ++uc;
                // in the order of their use: K of a step (a slot a map) before V of the step before (64 keys a slot)
                for (int x = -1; x < w.n && ok; ++x) {
                    uint32_t slot;
                    if (x + 1 < w.n)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (ready(slot))
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    tma_load_3d(smem_u32(ring_smem + slot * C::SLOT + c * C::HB), &tmK,
                                                smem_u32(&bars->kv_full[slot]), c * 64,
                                                w.y0 + (w.t0 + x + 1) * C::BN + rank * 64, zk + i, pol_kv);
                    if (x >= 0)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (ready(slot))
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    tma_load_3d(smem_u32(ring_smem + slot * C::SLOT + c * C::HB), &tmV,
                                                smem_u32(&bars->kv_full[slot]), rank * 128 + c * 64,
                                                w.y0 + (w.t0 + x) * C::BN + i * 64, zv, pol_kv);
                }
            }
            // CTA 0's commits reach this CTA by themselves, ordered by no barrier of the pair: the last of each has to be
            // here before shared memory is released (after an abort, the one that the MMA warp waits for)
            for (uint32_t k = ring < C::NSLOT ? 0 : ring - C::NSLOT; k < ring && ok; ++k)
                ok = mbar_wait(smem_u32(&bars->kv_empty[k % C::NSLOT]), (k / C::NSLOT) & 1, abort_flag, p.timeout_ns);
            if (ok && uc > 0) ok = mbar_wait(smem_u32(&bars->q_empty), (uc - 1) & 1, abort_flag, p.timeout_ns);
            if (!ok) timed_out();
            units.finish(ok);
            // every copy issued lands before shared memory is released (after an abort the other CTA's word may not
            // come: a millisecond is enough for the copies)
            const unsigned long long limit = ok ? kCleanupTimeoutNs : 1000000ull;
            for (uint32_t k = ring < C::NSLOT ? 0 : ring - C::NSLOT; k < ring; ++k)
                if (k + 1 != (uint32_t)p.withhold_kv)
                    mbar_wait(smem_u32(&bars->kv_full[k % C::NSLOT]), (k / C::NSLOT) & 1, nullptr, limit);
            if (uc > 0) mbar_wait(smem_u32(&bars->q_full), (uc - 1) & 1, nullptr, limit);
        }
    } else if (warp == C::MMA_WARP) {
        regs_decrease<C::REG_CONTROL>();
        constexpr uint32_t idesc_s = idesc_f32acc(1, 0, 2 * C::BM, C::BN), idesc_o = idesc_f32acc(1, 1, 2 * C::BM, 2 * C::D);
        const uint64_t q_desc = sdesc_sw128(smem_u32(q_smem), 16, 1024), w_desc = sdesc_sw128(smem_u32(w_smem), 16, 1024);
        const uint64_t k_desc = sdesc_sw128(smem_u32(ring_smem), 16, 1024);
        const uint64_t v_desc = sdesc_sw128(smem_u32(ring_smem), C::HB, 1024);
        uint32_t ring = 0, uc = 0, scores = 0, products = 0;       // steps whose S and whose product were issued
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            ok = ok && warp_wait(bar, parity);
            return ok;
        };
        auto full = [&](uint32_t n) -> bool { return wait(&bars->kv_full[n % C::NSLOT], (n / C::NSLOT) & 1); };
        // packed rows behind the sequence become 0: a weight of 0 times a NaN would be one
        auto clear_tail = [&](int live, uint8_t* v) {
            if constexpr (C::PACKED) {
                if (live >= 64) return;
                for (int o = max(live, 0) * 128 + lane * 16; o < C::HB; o += 512)
#pragma unroll
                    for (int c = 0; c < 2; ++c) *reinterpret_cast<uint4*>(v + c * C::HB + o) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            }
        };
        auto issue_s = [&]() -> bool {
            if (scores > 0 && !wait(&bars->s_free, (scores - 1) & 1)) return false;
#pragma unroll
            for (int i = 0; i < 2; ++i, ++ring) {
                const uint32_t slot = ring % C::NSLOT;
                if (!full(ring)) return false;
                tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < C::D / 16; ++kk)
                    pair_mma_warp(tmem + i * C::BN, q_desc + (((2 * i + kk / 4) * C::CB + (kk % 4) * 32) >> 4),
                                  k_desc + ((slot * C::SLOT + (kk / 4) * C::HB + (kk % 4) * 32) >> 4), idesc_s,
                                  kk > 0 ? 1u : 0u);
                pair_commit_warp(&bars->kv_empty[slot]);
            }
            pair_commit_warp(&bars->s_full);
            ++scores;
            return true;
        };
        auto issue_product = [&](const Unit& w, int x) -> bool {
            if (x == 0 && !wait(&bars->o_empty, (uc & 1) ^ 1)) return false;
            if (!wait(&bars->w_full, products & 1)) return false;
#pragma unroll
            for (int i = 0; i < 2; ++i, ++ring) {
                const uint32_t slot = ring % C::NSLOT;
                if (!full(ring)) return false;
                clear_tail(w.N - (w.t0 + x) * C::BN - i * 64, ring_smem + slot * C::SLOT);
                tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    pair_mma_warp(tmem + C::O_COL, w_desc + ((i * C::CB + kk * 32) >> 4),
                                  v_desc + ((slot * C::SLOT + kk * 16 * 128) >> 4), idesc_o, x > 0 || i > 0 || kk > 0 ? 1u : 0u);
                pair_commit_warp(&bars->kv_empty[slot]);
            }
            pair_commit_warp(&bars->w_free);
            ++products;
            return true;
        };
        // CTA 1: a slot that has landed
        auto pass_on = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) pair_arrive(bar);
        };
        Unit w;
        while (ok && units.take(w, ok)) {
            if (!wait(&bars->q_full, uc & 1)) break;
            if (rank == 0) {
                if (!issue_s()) break;
                for (int x = 0; x < w.n; ++x) {
                    if (x + 1 < w.n && !issue_s()) break;
                    if (x + 2 == w.n || w.n == 1) pair_commit_warp(&bars->q_empty);   // behind the unit's last scores
                    if (!issue_product(w, x)) break;
                }
                if (!ok) break;
                pair_commit_warp(&bars->o_full);
            } else {
                pass_on(&bars->q_full);
                for (int x = -1; x < w.n && ok; ++x) {
                    if (x + 1 < w.n)
                        for (int i = 0; i < 2 && ok; ++i, ++ring)
                            if (full(ring)) pass_on(&bars->kv_full[ring % C::NSLOT]);
                    if (x >= 0)
                        for (int i = 0; i < 2 && ok; ++i, ++ring)
                            if (full(ring)) {
                                clear_tail(w.N - (w.t0 + x) * C::BN - i * 64, ring_smem + (ring % C::NSLOT) * C::SLOT);
                                pass_on(&bars->kv_full[ring % C::NSLOT]);
                            }
                }
            }
            ++uc;
        }
        if (!ok && lane == 0) timed_out();
        if (rank == 0) pair_commit_warp(&bars->drain);
        // CTA 1 may have given up first: CTA 0 does when its own waits run out
        mbar_wait(smem_u32(&bars->drain), 0, nullptr, rank == 0 ? kCleanupTimeoutNs : p.timeout_ns + kCleanupTimeoutNs);
        __syncwarp();
    } else if (warp < 8) {
        // both warpgroups work on every step, warpgroup wg on its half of the keys, a thread one row
        regs_increase<C::REG_COMPUTE>();
        constexpr int HC = C::BN / 2;
        const int wg = warp >> 2, trow = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const float2 c2 = make_float2(p.c_log2, p.c_log2);
        uint8_t* w_row = w_smem + wg * C::CB + trow * 128;
        uint32_t h = 0, uc = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
            ok = ok && warp_wait(bar, parity);
            return ok;
        };
        Unit w;
        while (ok && units.take(w, ok)) {
            const int a0 = w.q0 + rank * C::BM, row = a0 + trow, head = C::PACKED ? w.z : w.z % dp.H;
            const bool valid = row < w.N;
            int jlo, jhi;
            diff_key_bounds(p, w.N, row, jlo, jhi);
            if (jlo > jhi) jlo = jhi;                     // a row behind the sequence, which is not stored
            const uint32_t span = (uint32_t)(jhi - jlo);
            // Each warpgroup writes half of the head's columns of this row, behind both warpgroups' last weights, so no
            // sooner than both have read what the first launch left there.
            const size_t orow = C::PACKED ? (size_t)(w.y0 + row) * p.H + w.z : (size_t)w.z * p.N + row;
            __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(p.o) + orow * (2 * C::D);
            const float4 sums = valid ? __ldcg(reinterpret_cast<const float4*>(out)) : make_float4(0.0f, 1.0f, 0.0f, 1.0f);
            // M_1, l_1, M_2, l_2 (log2 units).  A map whose every score is -inf has weights and a sum of 0, and the
            // other map is left.
            const float2 m1 = make_float2(-sums.x, -sums.x), m2 = make_float2(-sums.z, -sums.z);
            const float l1 = sums.y == 0.0f ? 1.0f : sums.y, inv1 = 1.0f / l1;
            const float f = sums.w == 0.0f ? 0.0f : -__ldg(dp.lam + head) * (l1 / sums.w);
            const float2 f2 = make_float2(f, f);
            for (int x = 0; x < w.n; ++x, ++h) {
                const int c0 = (w.t0 + x) * C::BN;
                if (!wait_all(&bars->s_full, h & 1)) break;
                tc_fence_after_sync();
                uint32_t a[HC], b[HC];
#pragma unroll
                for (int ch = 0; ch < HC; ch += 32) {
                    tmem_ld32p(tmem + lane_addr + wg * HC + ch, a + ch);
                    tmem_ld32p(tmem + lane_addr + C::BN + wg * HC + ch, b + ch);
                }
                tmem_wait_ld_only();
#pragma unroll
                for (int ch = 0; ch < HC; ch += 32) {
                    reg_fence32(a + ch);
                    reg_fence32(b + ch);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) pair_arrive(&bars->s_free);
                uint32_t pk[HC / 2];
                auto weigh = [&](auto masked_tag) {
                    constexpr bool kMasked = decltype(masked_tag)::value;
                    const uint32_t first = (uint32_t)(c0 + wg * HC - jlo);
#pragma unroll
                    for (int e = 0; e < HC; e += 2) {
                        const float2 x1 = __ffma2_rn(make_float2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])), c2, m1);
                        const float2 x2 = __ffma2_rn(make_float2(__uint_as_float(b[e]), __uint_as_float(b[e + 1])), c2, m2);
                        float2 r = __ffma2_rn(make_float2(ex2(x2.x), ex2(x2.y)), f2, make_float2(ex2(x1.x), ex2(x1.y)));
                        if constexpr (kMasked) {
                            r.x = first + (uint32_t)e <= span ? r.x : 0.0f;
                            r.y = first + (uint32_t)e + 1u <= span ? r.y : 0.0f;
                        }
                        pk[e / 2] = pack_bf16x2(r.x, r.y);
                    }
                };
                if (diff_edge<C::BN>(p, w.N, a0, c0)) weigh(std::true_type{});
                else weigh(std::false_type{});
                // the product of the step before has read the weights
                if (h > 0 && !wait_all(&bars->w_free, (h - 1) & 1)) break;
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    *reinterpret_cast<uint4*>(w_row + ((v ^ (trow & 7)) << 4)) =
                        make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) pair_arrive(&bars->w_full);
            }
            if (!ok) break;
            if (!wait_all(&bars->o_full, uc & 1)) break;
            tc_fence_after_sync();
#pragma unroll
            for (int ch = 0; ch < C::D / 32; ++ch) {
                uint32_t r[32];
                tmem_ld32(tmem + lane_addr + C::O_COL + wg * C::D + ch * 32, r);
                tmem_wait_ld(r);
                if (!valid) continue;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint32_t pk[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        pk[e] = pack_bf16x2(__uint_as_float(r[8 * v + 2 * e]) * inv1,
                                            __uint_as_float(r[8 * v + 2 * e + 1]) * inv1);
                    reinterpret_cast<uint4*>(out + wg * C::D + ch * 32)[v] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) pair_arrive(&bars->o_empty);
            ++uc;
        }
        if (ok && h > 0) wait_all(&bars->w_free, (h - 1) & 1);     // CTA 0's last word on the weights
        if (!ok) timed_out();
    } else {
        regs_decrease<C::REG_CONTROL>();
    }
    tc_fence_before_sync();
    __syncthreads();
    // The arrivals of the other CTA's threads are behind this barrier, its commits were waited for above, and its
    // requests for units are awaited here.
    pair_sync();
    if (threadIdx.x == 0) bars->hand.last_answer();
    tc_fence_after_sync();
    if (warp == C::MMA_WARP)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <class C, class Kernel, class... Args>
static cudaError_t launch_one(Kernel kernel, int grid, int cluster, cudaStream_t stream, const Args&... args)
{
    if (grid < 1) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc would wait forever if the launch pool were smaller than the split
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
    if (attr.numRegs * C::NUM_THREADS < C::REG_POOL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute pair[1];
    pair[0].id = cudaLaunchAttributeClusterDimension;
    pair[0].val.clusterDim.x = cluster;
    pair[0].val.clusterDim.y = pair[0].val.clusterDim.z = 1;
    cfg.attrs = pair;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    cfg.stream = stream;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(C::NUM_THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool PK>
static cudaError_t launch_wide(const DiffFwdMaps& m, DiffFwdParams& lse, DiffFwdParams& out, int sm_count, cudaStream_t stream)
{
    const int grid = diff_grid<DiffLseCfg<PK>>(lse, sm_count);
    const cudaError_t e = launch_one<DiffLseCfg<PK>>(diff_lse_kernel<PK>, grid, 1, stream, m.q, m.k, lse);
    if (e != cudaSuccess) return e;
    const int pairs = diff_grid<DiffOutCfg<PK>>(out, sm_count);
    return launch_one<DiffOutCfg<PK>>(diff_out_kernel<PK>, pairs, 2, stream, m.q, m.k64, m.v64, out);
}

cudaError_t launch_diff_fwd_wide(const DiffFwdMaps& m, DiffFwdParams lse, DiffFwdParams out, int sm_count,
                                 cudaStream_t stream)
{
    return out.f.cu_seqlens != nullptr ? launch_wide<true>(m, lse, out, sm_count, stream)
                                       : launch_wide<false>(m, lse, out, sm_count, stream);
}

}  // namespace gb300
