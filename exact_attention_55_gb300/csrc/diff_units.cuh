// diff_units.cuh -- how the forward kernels of differential attention share their units out.
//
// A unit is NQ x BM query rows of one head (a head's value part, a map).  The grid has a block for each,
// and blocks that run take over the work of blocks that were not launched yet
// (clusterlaunchcontrol.try_cancel), so costs even out by themselves, with no counter in memory: pairs of
// equal causal cost dealt out in advance left the busiest SM 15 % above the mean at nine documents of
// 200 to 5600 tokens x 8 heads (210 us against 193), and half a round idle where there are 3.4 (one
// sequence of 16384 x 8 heads: 780 us against 658).
//
// Order: the longest sequence first; within it groups of heads whose keys and values fit in L2 together; in a
// group the costliest rows first under a causal mask, of all its heads, so that the last units are short.
// Packed calls with more sequences than the sorted table holds walk pairs as attn_fwd.cuh does.
//
// With CLUSTER = 2 a unit is a cluster's: CTA 0 asks for both, and the answer lands in both.
#pragma once

#include "attn_fwd.cuh"
#include "diff_params.h"

namespace gb300 {

// The hand-over of units from a block's producer, in shared memory.
struct alignas(16) DiffHand {
    uint4 stolen;
    uint64_t full[2], empty[2], steal, ready;              // ready: CTA 1 can take an answer
    int unit[2];
    int owed;                                              // CTA 1: 1 + the parity of an answer that may still come

    __device__ __forceinline__ void init(int consumer_warps)
    {
        owed = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), consumer_warps);
        }
        mbar_init(smem_u32(&steal), 1);
        mbar_init(smem_u32(&ready), 1);
    }

    // CTA 1, once CTA 0 sends no more requests (behind a barrier of both): an answer on its way lands.  One thread; it
    // comes only after an abort, and a millisecond is enough for it.
    __device__ __forceinline__ void last_answer()
    {
        if (owed != 0) mbar_wait(smem_u32(&steal), (uint32_t)(owed - 1), nullptr, 1000000ull);
    }
};

// The table counts tiles of one head.
template <class C>
__device__ __forceinline__ void build_diff_tab(const FwdParams& p, SortTab* tab)
{
    build_sort_tab<C::NQ * C::BM / 2>(p.cu_seqlens, p.num_seqs, p.T, 1, tab);     // pairs of half a unit's rows
}

// Unit u; false: the grid, laid out for the most units there can be, has no unit u.
template <class C>
__device__ __forceinline__ bool diff_unit(int u, const DiffFwdParams& dp, Unit& w, const SortTab* tab)
{
    constexpr int ROWS = C::NQ * C::BM;
    const FwdParams& p = dp.f;
    int nt, rem;                                          // tiles of the sequence's heads, unit among its units
    if constexpr (C::PACKED) {
        const int tile = u / p.H;
        if (tile >= tab->total) return false;
        int seq, first, a, b;
        sorted_pair(tab, p.num_seqs, tile, seq, first);
        seq_span(p.cu_seqlens, seq, p.T, a, b);
        w.z = 0;
        w.y0 = a;
        w.N = b - a;
        nt = (w.N + ROWS - 1) / ROWS;
        rem = first * p.H + (u - tile * p.H);
    } else {
        nt = p.num_qblk;
        const int per = nt * p.H, b = u / per;
        w.z = b * p.H;
        w.y0 = 0;
        w.N = p.N;
        rem = u - b * per;
    }
    const int group = rem / (nt * dp.group), first = group * dp.group, heads = min(dp.group, p.H - first);
    rem -= first * nt;
    const int rank = rem / heads;
    w.z += first + (rem - rank * heads);
    w.q0 = (nt - 1 - rank) * ROWS;
    const int last = min(w.N, w.q0 + ROWS) - 1;
    int lo = 0, hi = w.N;                                 // keys [lo, hi) that some row of the unit may use
    if (p.window > 0) lo = max(0, w.q0 - p.window);
    if (p.causal) hi = last + 1;
    else if (p.window > 0) hi = min(w.N, last + p.window + 1);
    w.t0 = lo / C::BN;
    w.n = (hi + C::BN - 1) / C::BN - w.t0;
    return true;
}

__device__ __forceinline__ uint32_t pair_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// One arrival on CTA 0's barrier at this place.  No thread reads what the other CTA's threads wrote: operands pass from
// TMA, or behind their writers' proxy fences, to the tensor cores, and TMEM behind its fences.  So the order within
// the CTA is enough (a release to the cluster took the compute warps a memory barrier at each: 1440 us became 2130).
__device__ __forceinline__ void pair_arrive(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar)) : "memory");
}
// Asks for a block (cluster) that was not launched; the answer lands in `to`, with kBoth of both CTAs, and counts 16
// bytes on `bar`.
template <bool kBoth>
__device__ __forceinline__ void steal_request(uint4* to, uint64_t* bar)
{
    if constexpr (kBoth)
        asm volatile(
            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 "
            "[%0], [%1];" ::"r"(smem_u32(to)),
            "r"(smem_u32(bar))
            : "memory");
    else
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                         smem_u32(to)),
                     "r"(smem_u32(bar))
                     : "memory");
}
// The number of the block (cluster), or -1: there are no more, and none may be asked for again.
template <int kCluster>
__device__ __forceinline__ int steal_answer(const uint4* from)
{
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=&r"(got), "=&r"(x) : "r"(smem_u32(from)) : "memory");
    return got ? (int)x / kCluster : -1;
}

// One role's way through the units of its block.
template <class C>
struct DiffUnits {
    const DiffFwdParams& dp;
    const SortTab* tab;
    DiffHand* hand;
    const volatile int* abort_flag;
    bool walks;                     // pairs dealt out in advance
    int su = 0, mine;
    uint32_t units = 0, asked = 0, answered = 0;
    static constexpr bool kPair = C::CLUSTER == 2;

    __device__ __forceinline__ DiffUnits(const DiffFwdParams& dp, const SortTab* tab, DiffHand* hand,
                                         const volatile int* abort_flag)
        : dp(dp), tab(tab), hand(hand), abort_flag(abort_flag), walks(C::PACKED && tab == nullptr), mine((int)blockIdx.x / C::CLUSTER)
    {
    }

    __device__ __forceinline__ bool walk(Unit& w)
    {
        if constexpr (C::PACKED) {
            const int c = (int)blockIdx.x / C::CLUSTER, G = (int)gridDim.x / C::CLUSTER;
            while (true) {
                su = units++ == 0 ? 2 * c : (su & 1) ? su + 2 * G - 1 : su + 1;
                if (su >= num_subs(dp.f, nullptr)) return false;
                if (unit_of<C>(su, dp.f, w, nullptr)) return true;
            }
        }
        return false;
    }

    // A consumer warp's next unit (all lanes).
    __device__ __forceinline__ bool take(Unit& w, bool& ok)
    {
        if (walks) return walk(w);
        const uint32_t b = units & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&hand->full[b]), (units >> 1) & 1, abort_flag, dp.f.timeout_ns));
        if (!ok) return false;
        const int u = *reinterpret_cast<const volatile int*>(&hand->unit[b]);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&hand->empty[b]));
        ++units;
        return u >= 0 && diff_unit<C>(u, dp, w, tab);
    }

    __device__ __forceinline__ bool ask(bool& ok)
    {
        fence_proxy_async_smem();                         // the last answer was read
        mbar_arrive_expect_tx(smem_u32(&hand->steal), 16);
        ++asked;
        if constexpr (kPair) {
            if (pair_rank() != 0) {
                pair_arrive(&hand->ready);
                return true;
            }
            if (!mbar_wait(smem_u32(&hand->ready), (asked - 1) & 1, abort_flag, dp.f.timeout_ns)) {
                --asked;                                  // was not sent
                ok = false;
                mine = -1;
                return false;
            }
        }
        steal_request<kPair>(&hand->stolen, &hand->steal);
        return true;
    }

    // The producer's (one lane): this block's own, then those of blocks that were not launched.  It asks for one when
    // the loads of the last are issued (asked for before them, a block with a long unit took a second at once, which
    // others would have come to sooner).
    __device__ __forceinline__ bool give(Unit& w, bool& ok)
    {
        if (walks) return walk(w);
        bool there = false;
        for (bool first = units == 0; !there; first = false) {
            if (!first) {
                if (!ask(ok)) return false;
                if (!mbar_wait(smem_u32(&hand->steal), answered & 1, abort_flag, dp.f.timeout_ns)) {
                    ok = false;
                    return false;
                }
                ++answered;
                mine = steal_answer<C::CLUSTER>(&hand->stolen);
            }
            if (mine < 0) break;
            there = diff_unit<C>(mine, dp, w, tab);
        }
        const uint32_t b = units & 1;
        if (!mbar_wait(smem_u32(&hand->empty[b]), ((units >> 1) & 1) ^ 1, abort_flag, dp.f.timeout_ns)) {
            ok = false;
            return false;
        }
        *reinterpret_cast<volatile int*>(&hand->unit[b]) = mine;
        mbar_arrive(smem_u32(&hand->full[b]));
        ++units;
        return there;
    }

    // The producer's end: what was asked for lands, and after an abort the blocks that were not launched are not
    // needed either.  CTA 0 may send the request that CTA 1 made ready for after CTA 1 gave up: see last_answer.
    __device__ __forceinline__ void finish(bool ok)
    {
        if (walks || ok) return;
        if (kPair && pair_rank() != 0) {
            if (asked > answered) hand->owed = 1 + (int)(answered & 1);
            return;
        }
        while (mine >= 0) {
            if (asked == answered) {
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(smem_u32(&hand->steal), 16);
                steal_request<false>(&hand->stolen, &hand->steal);
                ++asked;
            }
            if (!mbar_wait(smem_u32(&hand->steal), answered & 1, nullptr, kCleanupTimeoutNs)) return;
            ++answered;
            mine = steal_answer<C::CLUSTER>(&hand->stolen);
        }
    }
};

// The launch's grid, and the heads of a group; 0: too many units.
template <class C>
inline int diff_grid(DiffFwdParams& dp, int sm_count)
{
    FwdParams& p = dp.f;
    constexpr long long kGroupBytes = 64 << 20;           // of the 126 MB of L2
    const long long per_token = 8LL * C::HEAD_DIM;        // bytes of a key pair and its value head
    const long long fit = kGroupBytes / (per_token * p.N), pairs = fit < 1 ? 1 : fit > dp.Hkv ? dp.Hkv : fit;
    dp.group = (int)pairs * (p.H / dp.Hkv);               // heads (maps, parts) of so many key pairs
    if (C::PACKED && p.num_seqs > kSortMaxSeqs) return fwd_grid(p, sm_count / C::CLUSTER) * C::CLUSTER;
    constexpr int ROWS = C::NQ * C::BM;
    const long long units =
        C::PACKED ? ((long long)p.T / ROWS + p.num_seqs) * p.H : (long long)(p.BH / p.H) * p.num_qblk * p.H;
    return units * C::CLUSTER <= 0x7fffffffLL ? (int)units * C::CLUSTER : 0;
}

}  // namespace gb300
