// diff_bwd.cu -- backward pass of differential attention: dQ, dK, dV and d lam.
//
// With P_m = exp(scale Q_m K_m^T + mask - LSE_m) of the two maps (m = 1, 2), O = (P_1 - lam P_2) V,
// f_1 = 1, f_2 = -lam and the upstream gradient dO (the chain rule through the forward pass):
//     D_m = dO . O_m per row (O_1 = O + lam O_2),    dP = dO V^T  (one for both maps),
//     dS_m = f_m P_m * (dP - D_m),
//     dQ_m = scale dS_m K_m,  dK_m = scale dS_m^T Q_m,  dV = (f_1 P_1 + f_2 P_2)^T dO,
//     d lam = - sum over the head's rows of D_2.
// Heads that share a key pair and value head add up in its dK and dV.
//
// Four launches, no floating-point atomics:
//   diff_dot_kernel              D_1 and D_2 of every row, one warp a row;
//   diff_bwd_kernel<D, kPassDK>  a unit is 128 keys of one map: in steps of 128 queries, over every
//                                head that reads them, S^T = K Q_i^T and dP^T = V dO_i^T into TMEM,
//                                the compute warps turn them into dS^T (bf16, over S^T), then
//                                dK += dS^T Q_i;
//   diff_bwd_kernel<D, kPassDV>  a unit is 128 keys of a pair: both maps' S^T, of which the compute
//                                warps make (P_1 - lam P_2)^T, rounded once, then dV += it dO_i;
//   diff_bwd_kernel<D, kPassDQ>  a unit is 128 query rows of one map: in steps of 128 keys, S = Q K_j^T
//                                and dP = dO V_j^T, then dQ += dS K_j.
// (The dV pass takes 64 queries a step at d = 128.)
// 40 d products per pair of tokens where 20 d would do: dP is computed for each map and again for dQ,
// the scores three times.  dK and dV of both maps in one unit want 640 columns of TMEM (d = 64: scores and
// dP 384, accumulators 256), of which there are 512.  dK, or dQ, of both maps in one unit would share dP
// and fit in TMEM (32 d in all); that form was not built.
//
// A step has two products of its own, S (Q K^T of the map; dV: of map 1) and X (dP; dV: map 2's
// scores), and one accumulation that waits for the compute warps.  S has two TMEM buffers and X one, which
// the compute warps release as soon as they have loaded it, so the MMA warp issues X(j), the
// accumulation of step j - 1, then S(j + 1), and the tensor pipe works on X(j) and S(j + 1) while both
// compute warpgroups (half of the columns each) turn steps j - 1 and j.
//
// Measured, 4 x 8 heads x 4096 tokens of d = 64, causal: 590 us = 582 TFLOP/s of 20 d (1164 executed); a step takes
// 1630 to 1740 cycles for 1024 of products.  Packed, 8 heads over 2, 8192 tokens of d = 128, window 2047: 375 us.
//
// What this was measured against, on 4 x 8 heads x 4096 tokens of d = 64, causal, all passes:
// steps of 64 columns with three TMEM buffers and a warpgroup each 1140 us, with quick waits 894.
// The tensor pipe was busy for a quarter of it: its queue holds about 8 MMAs, and a wait, even for what
// has long happened, took the issuing warp 150-200 cycles (one lane or all polling in a loop; 60-120
// with one attempt by all lanes first), so few large MMAs and few waits a column are what counts.
// A 128 x 64 x 16 product of two shared-memory operands takes 48 cycles instead of 32: it reads
// 6 KB of the 128 bytes a cycle there are.
//
// The three passes do not depend on one another, and each is launched as a dependent that starts
// when all CTAs of the one before have started: its CTAs take the SMs that run out of units.  Against
// launches one after another: 566 us to 574 (4 x 8 heads x 4096 tokens), 347 to 468 (packed, d = 128, where
// shared heads leave few units), 14.2 to 24.9 (2 x 4 heads x 300).
// Each waits for the one before at its end, so that the last one's end is the end of all.
// Units are handed out by a counter, the costliest first: shared heads leave few of them (128 key
// tiles for 152 SMs in an 8192-token step with two key pairs).
//
// What lies behind a packed sequence never enters a product: masked entries are selected away
// before dP can make them NaN, and the rows of the operands become 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "attn_params.h"
#include "diff_params.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace gb300 {

enum : int { kPassDK = 0, kPassDV = 1, kPassDQ = 2 };   // in the order of their launches

template <int D, int kPass>
struct DiffBwdCfg {
    static constexpr bool DQ = kPass == kPassDQ, DV = kPass == kPassDV;
    static constexpr int BT = 128;                 // rows of a unit's tile
    static constexpr int BC = DV && D == 128 ? 64 : 128, HC = BC / 2;   // columns of a step, of a warpgroup
    static constexpr int NCB = D / 64;             // 64-column blocks of a row of d
    static constexpr int FIX_CB = BT * 128;        // bytes of one, fixed tiles
    static constexpr int RING_CB = BC * 128;       // and ring tiles
    static constexpr int FIX_PARTS = DV ? 2 : 3;   // of d columns: K_1 and K_2; Q or K, then dO or V
    static constexpr int FIX_BYTES = FIX_PARTS * NCB * FIX_CB;
    // Three rings.  S: Q or K of the map (dV: Q_1), which the accumulation reads too.  X: dO or V in parts of
    // d columns (dV: Q_2).  dV alone: A, dO for the accumulation.
    static constexpr int S_BYTES = NCB * RING_CB, X_BYTES = NCB * RING_CB, A_BYTES = DV ? 2 * NCB * RING_CB : 0;
    static constexpr int X_PARTS = DV ? 1 : 2;
    static constexpr int NS = D == 64 ? 3 : DV ? 3 : 2, NX = D == 64 ? (DV ? 2 : 6) : 2, NACC = DV ? 2 : 1;   // slots
    // TMEM: S of step h at (h & 1) BC (then dS or the weights, packed), X behind both, the accumulator
    static constexpr int ACC = DV ? 2 * D : D;
    static constexpr int X_COL = 2 * BC, ACC_COL = 512 - (ACC > 128 ? 256 : 128);
    static constexpr int COMPUTE_WARPS = 8, PRODUCER_WARP = 8, MMA_WARP = 9, SUM_WARP = 10, NUM_THREADS = 384;
    static constexpr int REG_COMPUTE = 208, REG_CONTROL = 88;
    static constexpr int REG_POOL = 256 * REG_COMPUTE + 128 * REG_CONTROL;
    // Shared memory: fixed tiles, rings, barriers, two steps' column values (LSE, D, factor).  At d = 128 it
    // is full to 600 bytes, so there is none to spend on alignment: the tiles start where it starts.
    static constexpr int RING_BYTES = NS * S_BYTES + NX * X_BYTES + (DV ? NACC * A_BYTES : 0);
    static constexpr int COL_OFF = 384, COL_FLOATS = 2 * BC + 4;
    static constexpr int SMEM_BYTES = FIX_BYTES + RING_BYTES + COL_OFF + (DQ ? 0 : 2 * COL_FLOATS * 4);
    static constexpr int COLUMN_WARP = 11;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static_assert(D == 64 || D == 128, "head dim");
    static_assert(X_COL + BC <= ACC_COL && ACC_COL + ACC <= 512, "TMEM");
};

// One unit: tile t (128 rows) of a head, or of a key pair, of one sequence.
struct DiffBwdUnit {
    int t, N, y0;      // tile, rows of the sequence, its first token (packed)
    int b, z;          // batch entry (packed: 0); 2 h + map, 2 g + map, or (dV) the key pair g
    int lo, n;         // its steps: from column block lo on, n of them
    int more;          // 0: there is none
};

struct alignas(16) DiffBwdBars {
    uint64_t fix_full, fix_empty;
    uint64_t s_in_full[3], s_in_empty[3], x_in_full[6], x_in_empty[6], a_in_full[2], a_in_empty[2];   // rings
    uint64_t s_full, p_full, x_free;               // one phase a step
    uint64_t acc_done, acc_empty;
    uint64_t unit_full[2], unit_empty[2];
    uint64_t col_full[2], col_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(DiffBwdBars) + 2 * sizeof(DiffBwdUnit) <= 384, "barrier block");
constexpr int kDiffBwdUnitOff = 320;               // the two units handed out
static_assert(sizeof(DiffBwdBars) <= kDiffBwdUnitOff, "barrier block");

// Units of a pass over `heads` heads (of q, of k, or key pairs).
__device__ __forceinline__ int diff_bwd_units(const DiffBwdParams& p, int heads)
{
    if (p.tab == nullptr) return p.nt * p.B * heads;
    return __ldcg(&p.tab->total) * heads;
}

// Unit u, costliest first under a causal mask: a query tile t meets t + 1 key tiles, a key tile nt - t
// query tiles.  Batched: rank by rank over all heads; packed, from the table of sorted sequences that
// the first kernel left: the longest sequence first.  More sequences than the table holds: slots laid out
// for the longest one; false where a sequence is shorter.
template <bool kDQ, bool kPacked>
__device__ __forceinline__ bool diff_bwd_unit(const DiffBwdParams& p, int u, int heads, DiffBwdUnit& w)
{
    int rank, seq;
    if (kPacked && p.tab != nullptr) {
        const int tile = u / heads;                // over all sequences, in the table's order
        w.z = u - tile * heads;
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldcg(p.tab->prefix + mid) <= tile) lo = mid;
            else hi = mid - 1;
        }
        seq = __ldcg(p.tab->seq + lo);
        rank = tile - __ldcg(p.tab->prefix + lo);
    } else {
        rank = u / (p.B * heads);
        const int rem = u - rank * (p.B * heads);
        seq = rem / heads;
        w.z = rem - seq * heads;
    }
    w.b = 0;
    w.y0 = 0;
    w.N = p.N;
    if constexpr (kPacked) {
        int a, b;
        seq_span(p.cu_seqlens, seq, p.T, a, b);
        w.y0 = a;
        w.N = b - a;
    } else {
        w.b = seq;
    }
    const int nt = (w.N + 127) / 128;
    if (rank >= nt) return false;
    w.t = kDQ ? nt - 1 - rank : rank;
    return true;
}

// Steps [lo, hi) of a unit: the blocks of BC keys that a query tile meets, or of BC queries that a key
// tile meets.
template <bool kDQ, int BC>
__device__ __forceinline__ void diff_bwd_steps(const DiffBwdParams& p, const DiffBwdUnit& w, int& lo, int& hi)
{
    const int a = w.t * 128, last = min(w.N, a + 128) - 1;
    lo = 0;
    hi = (w.N + BC - 1) / BC;
    if (kDQ && p.causal) hi = min(hi, last / BC + 1);
    if (!kDQ && p.causal) lo = a / BC;
    if (p.window > 0) {
        if (kDQ || !p.causal) lo = max(0, (a - p.window) / BC);
        if (!kDQ || !p.causal) hi = min(hi, (last + p.window) / BC + 1);
    }
}

// Every pair of queries [q0, q0 + nq) and keys [k0, k0 + nk) is inside the sequence and allowed.
__device__ __forceinline__ bool diff_bwd_full(const DiffBwdParams& p, int N, int q0, int nq, int k0, int nk)
{
    if (q0 + nq > N || k0 + nk > N) return false;
    if (p.causal && k0 + nk - 1 > q0) return false;
    if (p.window > 0) {
        if (k0 < q0 + nq - 1 - p.window) return false;
        if (!p.causal && k0 + nk - 1 > q0 + p.window) return false;
    }
    return true;
}

// LSE / D index of row 0 of the unit's sequence in map z = 2 h + m.
template <bool kPacked>
__device__ __forceinline__ size_t diff_bwd_vec(const DiffBwdParams& p, const DiffBwdUnit& w, int z)
{
    return kPacked ? (size_t)z * p.T + w.y0 : ((size_t)w.b * 2 * p.H + z) * p.N;
}

// Output row r of head z of `heads`.
template <bool kPacked>
__device__ __forceinline__ size_t diff_bwd_row(const DiffBwdParams& p, const DiffBwdUnit& w, int heads, int z, int r)
{
    return kPacked ? (size_t)(w.y0 + r) * heads + z : ((size_t)w.b * heads + z) * p.N + r;
}

// A value that all lanes share, by a reduction, whose result the compiler knows to be uniform: what an
// MMA's descriptors are computed from then stays in uniform registers.
__device__ __forceinline__ int diff_uniform(int v) { return (int)__reduce_or_sync(0xffffffffu, (unsigned)v); }

// What the kernel ahead wrote, and what may still be in a cache of an SM that ran before: from L2.
__device__ __forceinline__ float diff_ld(const float* p) { return __ldcg(p); }

// D_1 and D_2 in fp32, one warp a row; the units' counters start at 0, and the table of packed sequences
// is sorted (tiles of 128 rows before each sequence).
template <int D>
__global__ void __launch_bounds__(256) diff_dot_kernel(const DiffBwdParams p)
{
    constexpr int E = 2 * D / 32;
    __shared__ SortTab tab;
    if (blockIdx.x == 0) {
        if (threadIdx.x < 3) p.next[threadIdx.x] = 0;
        if (p.tab != nullptr) {
            build_sort_tab<64>(p.cu_seqlens, p.B, p.T, 1, &tab);      // pairs of 64 rows: tiles
            for (int i = threadIdx.x; i < (int)(sizeof(SortTab) / 4); i += 256)
                reinterpret_cast<int*>(p.tab)[i] = reinterpret_cast<const int*>(&tab)[i];
        }
    }
    const bool packed = p.cu_seqlens != nullptr;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long rows = packed ? (long long)p.T * p.H : (long long)p.B * p.H * p.N;
    if (row >= rows) return;
    const int lane = threadIdx.x & 31;
    int h;
    size_t at, step;
    if (packed) {
        const long long t = row / p.H;
        h = (int)(row - t * p.H);
        if (t < __ldcg(p.cu_seqlens) || t >= __ldcg(p.cu_seqlens + p.B)) return;   // outside every sequence
        at = (size_t)(2 * h) * p.T + t;
        step = (size_t)p.T;
    } else {
        const long long bh = row / p.N;
        h = (int)(bh % p.H);
        at = (size_t)(2 * bh) * p.N + (size_t)(row - bh * p.N);
        step = (size_t)p.N;
    }
    const size_t off = (size_t)row * (2 * D) + lane * E;
    uint32_t o[E / 2], o2[E / 2], g[E / 2];
    auto load = [&](const void* src, uint32_t* x) {
        const __nv_bfloat16* s = static_cast<const __nv_bfloat16*>(src) + off;
        if constexpr (E == 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(s);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(s);
            x[0] = v.x, x[1] = v.y;
        }
    };
    load(p.o, o);
    load(p.o2, o2);
    load(p.dout, g);
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
        auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
        auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
        a = fmaf(lo(o[e]), lo(g[e]), fmaf(hi(o[e]), hi(g[e]), a));
        b = fmaf(lo(o2[e]), lo(g[e]), fmaf(hi(o2[e]), hi(g[e]), b));
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, s);
        b += __shfl_xor_sync(0xffffffffu, b, s);
    }
    if (lane == 0) {
        p.delta[at] = fmaf(__ldcg(p.lam + h), b, a);
        p.delta[at + step] = b;
    }
}

// d lam of the heads blockIdx.x, blockIdx.x + gridDim.x, ...: one warp adds up a head's D_2 in a fixed
// order (32 lanes of eight sums each).
__device__ __forceinline__ void diff_dlam(const DiffBwdParams& p, int lane)
{
    for (int h = blockIdx.x; h < p.H; h += gridDim.x) {
        float acc[8] = {};
        const int parts = p.cu_seqlens ? 1 : p.B;
        for (int b = 0; b < parts; ++b) {
            const float* d;
            long long n;
            if (p.cu_seqlens) {
                const int t0 = min(max(__ldcg(p.cu_seqlens), 0), p.T);
                n = min(max(__ldcg(p.cu_seqlens + p.B), t0), p.T) - t0;
                d = p.delta + (size_t)(2 * h + 1) * p.T + t0;
            } else {
                n = p.N;
                d = p.delta + ((size_t)b * 2 * p.H + 2 * h + 1) * p.N;
            }
            for (long long i = lane; i < n; i += 256) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (i + 32 * k < n) acc[k] += diff_ld(d + i + 32 * k);
            }
        }
        float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (lane == 0) p.dlam[h] = -sum;
    }
}

// One pass.  Maps: dK pass fixed K and V, ring Q and dO; dV pass fixed K, ring Q and dO; dQ pass fixed Q
// and dO, ring K and V.
template <int D, int kPass, bool kPacked>
__global__ void __launch_bounds__(DiffBwdCfg<D, kPass>::NUM_THREADS, 1)
    diff_bwd_kernel(const __grid_constant__ CUtensorMap tmFixA, const __grid_constant__ CUtensorMap tmFixB,
                    const __grid_constant__ CUtensorMap tmRingA, const __grid_constant__ CUtensorMap tmRingB,
                    const DiffBwdParams p)
{
    using C = DiffBwdCfg<D, kPass>;
    constexpr bool kDQ = C::DQ, kDV = C::DV;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* fix = smem;
    uint8_t* ring_s = smem + C::FIX_BYTES;
    uint8_t* ring_x = ring_s + C::NS * C::S_BYTES;
    uint8_t* ring_a = ring_x + C::NX * C::X_BYTES;         // dV only
    uint8_t* tail = smem + C::FIX_BYTES + C::RING_BYTES;
    DiffBwdBars* bars = reinterpret_cast<DiffBwdBars*>(tail);
    DiffBwdUnit* handed = reinterpret_cast<DiffBwdUnit*>(tail + kDiffBwdUnitOff);
    float* columns = reinterpret_cast<float*>(tail + C::COL_OFF);
    const volatile int* abort_flag = &bars->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = kDQ ? 2 * p.H : kDV ? p.Hkv : 2 * p.Hkv, G = p.H / p.Hkv;
    if ((smem_u32(smem) & 1023) != 0) {                    // no kernel of this file has static shared memory
        if (threadIdx.x == 0) atomicExch(p.status, kStatusTimeout);
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->fix_full), 1);
        mbar_init(smem_u32(&bars->fix_empty), 1);
        for (int s = 0; s < C::NS; ++s) mbar_init(smem_u32(&bars->s_in_full[s]), 1), mbar_init(smem_u32(&bars->s_in_empty[s]), 1);
        for (int s = 0; s < C::NX; ++s) mbar_init(smem_u32(&bars->x_in_full[s]), 1), mbar_init(smem_u32(&bars->x_in_empty[s]), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars->a_in_full[s]), 1);
            mbar_init(smem_u32(&bars->a_in_empty[s]), 1);
            mbar_init(smem_u32(&bars->unit_full[s]), 1);
            mbar_init(smem_u32(&bars->unit_empty[s]), C::COMPUTE_WARPS + (kDQ ? 1 : 2));
            mbar_init(smem_u32(&bars->col_full[s]), 1);
            mbar_init(smem_u32(&bars->col_empty[s]), C::COMPUTE_WARPS);
        }
        mbar_init(smem_u32(&bars->s_full), 1);
        mbar_init(smem_u32(&bars->p_full), C::COMPUTE_WARPS);
        mbar_init(smem_u32(&bars->x_free), C::COMPUTE_WARPS);
        mbar_init(smem_u32(&bars->acc_done), 1);
        mbar_init(smem_u32(&bars->acc_empty), C::COMPUTE_WARPS);
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::MMA_WARP) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    // The first pass waits for the dot products and the counters; the others' CTAs start when every CTA
    // of the pass before has come this far, and find them written.
    if constexpr (kPass == kPassDK) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    auto timed_out = [&]() {
        atomicExch(p.status, kStatusTimeout);
        *reinterpret_cast<volatile int*>(&bars->abort_flag) = 1;
    };
    // A warp's wait: all lanes try once, which is the usual case; else they poll until the limit.
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        const uint32_t a = smem_u32(bar);
        if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
        return __all_sync(0xffffffffu, mbar_wait(a, parity, abort_flag, p.timeout_ns));
    };
    // A consumer warp's next unit (all lanes); false at the end or after an abort.
    auto take_unit = [&](uint32_t& n, bool& ok, DiffBwdUnit& w) -> bool {
        const uint32_t b = n & 1;
        if (!warp_wait(&bars->unit_full[b], (n >> 1) & 1)) {
            ok = false;
            return false;
        }
        const volatile DiffBwdUnit* u = handed + b;
        w.t = diff_uniform(u->t), w.N = diff_uniform(u->N), w.y0 = diff_uniform(u->y0), w.b = diff_uniform(u->b);
        w.z = diff_uniform(u->z), w.lo = diff_uniform(u->lo), w.n = diff_uniform(u->n), w.more = diff_uniform(u->more);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->unit_empty[b]));
        ++n;
        return w.more != 0;
    };

    if (warp == C::PRODUCER_WARP) {
        regs_decrease<C::REG_CONTROL>();
        if (lane == 0) {
            const uint64_t pol_fix = l2_policy_evict_first(), pol_ring = l2_policy_evict_last();
            uint32_t ns = 0, nx = 0, na = 0, issued = 0, lost_s = 0, lost_x = 0, lost_a = 0, fixed = 0, given = 0;
            const int total = diff_bwd_units(p, heads);
            int walk = (int)blockIdx.x;
            bool ok = true;
            // the next slot of a ring: `blocks` blocks of 64 columns from `col` on of heads `head`, ...; a withheld
            // one is neither armed nor loaded (test hook)
            auto load = [&](uint8_t* base, uint64_t* full, uint64_t* empty, uint32_t slots, uint32_t& n, uint32_t& lost,
                            const CUtensorMap* map, auto blocks_tag, int col, int row, int head) {
                constexpr int blocks = decltype(blocks_tag)::value;
                if (!ok) return;
                const uint32_t slot = n % slots;
                if (!mbar_wait(smem_u32(&empty[slot]), ((n / slots) & 1) ^ 1, abort_flag, p.timeout_ns)) {
                    ok = false;
                    return;
                }
                ++n;
                if (++issued == (uint32_t)p.withhold) {
                    lost = n;
                    return;
                }
                const uint32_t fb = smem_u32(&full[slot]);
                mbar_arrive_expect_tx(fb, blocks * C::RING_CB);
#pragma unroll
                for (int i = 0; i < blocks; ++i)
                    tma_load_3d(smem_u32(base + (slot * blocks + i) * C::RING_CB), map, fb, col + i * 64, row, head, pol_ring);
            };
            using One = std::integral_constant<int, C::NCB>;
            using Two = std::integral_constant<int, 2 * C::NCB>;
            while (ok) {
                DiffBwdUnit w;
                int u;
                if (!kPacked || p.tab != nullptr) {
                    u = atomicAdd(p.next + kPass, 1);
                } else {                       // slots with gaps: walked without the counter
                    u = walk;
                    walk += gridDim.x;
                }
                w.more = u < total ? 1 : 0;
                if (w.more && !diff_bwd_unit<kDQ, kPacked>(p, u, heads, w)) continue;
                int hi = 0;
                w.lo = 0;
                if (w.more) diff_bwd_steps<kDQ, C::BC>(p, w, w.lo, hi);
                const int per = hi - w.lo, group = kDQ ? 1 : G;       // steps of a head, heads
                w.n = group * per;
                const uint32_t b = given & 1;
                if (!mbar_wait(smem_u32(&bars->unit_empty[b]), ((given >> 1) & 1) ^ 1, abort_flag, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                volatile DiffBwdUnit* v = handed + b;
                v->t = w.t, v->N = w.N, v->y0 = w.y0, v->b = w.b, v->z = w.z, v->lo = w.lo, v->n = w.n, v->more = w.more;
                mbar_arrive(smem_u32(&bars->unit_full[b]));
                ++given;
                if (!w.more) break;
                if (!mbar_wait(smem_u32(&bars->fix_empty), (fixed & 1) ^ 1, abort_flag, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = smem_u32(&bars->fix_full);
                mbar_arrive_expect_tx(fb, C::FIX_BYTES);
                ++fixed;
                // parts of d columns: Q, K or K_1; then dO, V, or K_2
                const int row = w.y0 + w.t * 128;
                const int za = w.b * heads * (kDV ? 2 : 1) + w.z * (kDV ? 2 : 1);
                const int zb = kDV ? za + 1 : kDQ ? w.b * p.H + (w.z >> 1) : w.b * p.Hkv + (w.z >> 1);
#pragma unroll
                for (int cb = 0; cb < C::FIX_PARTS * C::NCB; ++cb) {
                    const bool first = cb < C::NCB;
                    tma_load_3d(smem_u32(fix + cb * C::FIX_CB), first || kDV ? &tmFixA : &tmFixB, fb,
                                (first ? cb : cb - C::NCB) * 64, row, first ? za : zb, pol_fix);
                }
                for (int i = 0; i < group; ++i) {
                    int zs, zx;                // heads of S's operand, and of X's (dV: of dO)
                    if constexpr (kDQ) {
                        const int g = (w.z >> 1) / G;
                        zs = w.b * 2 * p.Hkv + 2 * g + (w.z & 1);
                        zx = w.b * p.Hkv + g;
                    } else {
                        const int h = (kDV ? w.z : w.z >> 1) * G + i;
                        zs = w.b * 2 * p.H + 2 * h + (kDV ? 0 : w.z & 1);
                        zx = w.b * p.H + h;
                    }
                    for (int s = w.lo; s < hi && ok; ++s) {
                        const int r = w.y0 + s * C::BC;
                        load(ring_s, bars->s_in_full, bars->s_in_empty, C::NS, ns, lost_s, &tmRingA, One{}, 0, r, zs);
                        if constexpr (kDV) {
                            load(ring_x, bars->x_in_full, bars->x_in_empty, C::NX, nx, lost_x, &tmRingA, One{}, 0, r, zs + 1);
                            load(ring_a, bars->a_in_full, bars->a_in_empty, C::NACC, na, lost_a, &tmRingB, Two{}, 0, r, zx);
                        } else {
                            load(ring_x, bars->x_in_full, bars->x_in_empty, C::NX, nx, lost_x, &tmRingB, One{}, 0, r, zx);
                            load(ring_x, bars->x_in_full, bars->x_in_empty, C::NX, nx, lost_x, &tmRingB, One{}, D, r, zx);
                        }
                    }
                }
            }
            if (!ok) timed_out();
            // every copy issued lands before shared memory is released
            auto landed = [&](uint64_t* full, uint32_t slots, uint32_t n, uint32_t lost) {
                for (uint32_t k = n < slots ? 0 : n - slots; k < n; ++k)
                    if (k + 1 != lost)
                        mbar_wait(smem_u32(&full[k % slots]), (k / slots) & 1, nullptr, kCleanupTimeoutNs);
            };
            landed(bars->s_in_full, C::NS, ns, lost_s);
            landed(bars->x_in_full, C::NX, nx, lost_x);
            if constexpr (kDV) landed(bars->a_in_full, C::NACC, na, lost_a);
            if (fixed > 0) mbar_wait(smem_u32(&bars->fix_full), (fixed - 1) & 1, nullptr, kCleanupTimeoutNs);
        }
    } else if (warp == C::MMA_WARP) {
        regs_decrease<C::REG_CONTROL>();
        constexpr uint32_t idesc_kk = idesc_f32acc(1, 0, 128, C::BC);      // both K-major
        constexpr uint32_t idesc_acc = idesc_f32acc(1, 1, 128, C::ACC);    // B MN-major
        const uint64_t fix_k = sdesc_sw128(smem_u32(fix), 16, 1024);
        const uint64_t s_k = sdesc_sw128(smem_u32(ring_s), 16, 1024), x_k = sdesc_sw128(smem_u32(ring_x), 16, 1024);
        const uint64_t acc_mn = sdesc_sw128(smem_u32(kDV ? ring_a : ring_s), C::RING_CB, 1024);
        uint32_t units_done = 0, h = 0, units = 0;      // h: steps so far
        uint32_t xs = 0;                                // slots of X's ring so far
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            ok = ok && warp_wait(bar, parity);
            return ok;
        };
        auto commit = [&](uint64_t* bar) { mma_commit_warp(smem_u32(bar)); };
        // d_col (+)= A B^T over d columns: fixed tiles from part `part` on, ring tile b0
        auto mm_kk = [&](uint32_t d_col, int part, uint64_t b0, bool accumulate) {
            const uint64_t a0 = fix_k + (uint64_t)((part * C::NCB * C::FIX_CB) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int byte = kk * 32;
                mma_ss_warp<false>(tmem + d_col, a0 + (uint64_t)(((byte / 128) * C::FIX_CB + byte % 128) >> 4),
                                   b0 + (uint64_t)(((byte / 128) * C::RING_CB + byte % 128) >> 4), idesc_kk,
                                   (kk > 0 || accumulate) ? 1u : 0u);
            }
        };
        // packed rows behind the sequence become 0 in a slot that starts at column `c` of the unit's columns
        auto clear_tail = [&](const DiffBwdUnit& w, int c, uint8_t* t, int blocks) {
            if constexpr (kPacked) {
                const int live = w.N - c;
                if (live >= C::BC) return;
                for (int o = live * 128 + lane * 16; o < C::RING_CB; o += 512)
                    for (int i = 0; i < blocks; ++i)
                        *reinterpret_cast<uint4*>(t + i * C::RING_CB + o) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            }
        };
        DiffBwdUnit w;
        while (take_unit(units, ok, w)) {
            const int per = kDQ ? w.n : w.n / G;
            if (!wait(&bars->fix_full, units_done & 1)) break;
            const uint32_t h0 = h;
            auto column = [&](int x) { return (w.lo + x % per) * C::BC; };
            // S of step x (number h): buffer h & 1 was last read by the accumulation of step h - 2
            auto issue_s = [&](int x) -> bool {
                const uint32_t hx = h0 + (uint32_t)x, slot = hx % C::NS;
                if (!wait(&bars->s_in_full[slot], (hx / C::NS) & 1)) return false;
                clear_tail(w, column(x), ring_s + slot * C::S_BYTES, C::NCB);
                tc_fence_after_sync();
                mm_kk((hx & 1) * C::BC, 0, s_k + (uint64_t)((slot * C::S_BYTES) >> 4), false);
                if (kDV) commit(&bars->s_in_empty[slot]);
                return true;
            };
            // the accumulation of step x: dS or the weights from TMEM, packed by both warpgroups over the first
            // half of their columns of S
            auto issue_acc = [&](int x) -> bool {
                const uint32_t hx = h0 + (uint32_t)x, slot = hx % (kDV ? C::NACC : C::NS);
                if (x == 0 && !wait(&bars->acc_empty, (units_done & 1) ^ 1)) return false;
                if constexpr (kDV) {
                    if (!wait(&bars->a_in_full[slot], (hx / C::NACC) & 1)) return false;
                    clear_tail(w, column(x), ring_a + slot * C::A_BYTES, 2 * C::NCB);
                    tc_fence_after_sync();
                }
                const uint64_t t = acc_mn + (uint64_t)((slot * (kDV ? C::A_BYTES : C::S_BYTES)) >> 4);
                constexpr int PER = C::HC / 16;         // k-steps of a warpgroup
#pragma unroll
                for (int kk = 0; kk < C::BC / 16; ++kk)
                    mma_ts_warp<false>(tmem + C::ACC_COL, tmem + (hx & 1) * C::BC + (kk / PER) * C::HC + (kk % PER) * 8,
                                       t + (uint64_t)((kk * 16 * 128) >> 4), idesc_acc, (kk > 0 || x > 0) ? 1u : 0u);
                commit(kDV ? &bars->a_in_empty[slot] : &bars->s_in_empty[slot]);
                return true;
            };
            if (!issue_s(0)) break;
            for (int x = 0; x < w.n && ok; ++x) {
                const uint32_t hx = h0 + (uint32_t)x;
                // X of this step, in parts of d columns, once the compute warps have read the last one
                if (hx > 0 && !wait(&bars->x_free, (hx - 1) & 1)) break;
                bool there = true;
#pragma unroll
                for (int part = 0; part < C::X_PARTS; ++part, ++xs) {
                    const uint32_t slot = xs % C::NX;
                    there = there && wait(&bars->x_in_full[slot], (xs / C::NX) & 1);
                    if (!there) break;
                    tc_fence_after_sync();
                    mm_kk(C::X_COL, 1 + part, x_k + (uint64_t)((slot * C::X_BYTES) >> 4), part > 0);
                    commit(&bars->x_in_empty[slot]);
                }
                if (!there) break;
                if (x == w.n - 1) commit(&bars->fix_empty);     // S of this step was issued before
                // s_full of this step before the accumulation of the last, and only when that one's p_full was
                // seen: no barrier runs a phase ahead
                if (x > 0) {
                    if (!wait(&bars->p_full, (hx - 1) & 1)) break;
                    commit(&bars->s_full);
                    tc_fence_after_sync();
                    if (!issue_acc(x - 1)) break;
                } else {
                    commit(&bars->s_full);
                }
                if (x + 1 < w.n && !issue_s(x + 1)) break;
            }
            if (!ok) break;
            h = h0 + (uint32_t)w.n;
            if (!wait(&bars->p_full, (h - 1) & 1)) break;
            tc_fence_after_sync();
            if (!issue_acc(w.n - 1)) break;
            commit(&bars->acc_done);
            ++units_done;
        }
        if (!ok && lane == 0) timed_out();
        commit(&bars->drain);
        mbar_wait(smem_u32(&bars->drain), 0, nullptr, kCleanupTimeoutNs);
        __syncwarp();
    } else if (warp < C::COMPUTE_WARPS) {
        // both warpgroups work on every step, warpgroup wg on its half of the columns, a thread one row
        regs_increase<C::REG_COMPUTE>();
        const int wg = warp >> 2, trow = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        constexpr float LOG2E = 1.4426950408889634f;
        const float2 c2 = make_float2(p.c_log2, p.c_log2);
        uint32_t h = 0, units = 0, units_done = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
            ok = ok && warp_wait(bar, parity);
            return ok;
        };
        DiffBwdUnit w;
        while (take_unit(units, ok, w)) {
            const int my = w.t * 128 + trow;            // this thread's row (query or key)
            const bool valid = my < w.N;
            // The columns that the mask allows for this row are [m_lo, m_hi]; a row behind the sequence
            // gets some interval, and what it computes is never stored.
            int m_lo, m_hi;
            if constexpr (kDQ) {
                m_lo = p.window > 0 ? my - p.window : 0;
                m_hi = p.causal ? my : (p.window > 0 ? my + p.window : w.N - 1);
            } else {
                m_lo = p.causal ? my : (p.window > 0 ? my - p.window : 0);
                m_hi = p.window > 0 ? my + p.window : w.N - 1;
            }
            m_hi = min(m_hi, w.N - 1);
            m_lo = min(m_lo, m_hi);
            const uint32_t m_span = (uint32_t)(m_hi - m_lo);
            const int per = kDQ ? w.n : w.n / G;
            // what this row needs (dQ): minus its LSE (log2 units) and minus its D
            float2 row_l = make_float2(0.0f, 0.0f), row_d = row_l;
            if constexpr (kDQ) {
                const size_t at = diff_bwd_vec<kPacked>(p, w, w.z) + (valid ? my : 0);
                row_l.x = row_l.y = -diff_ld(p.lse + at) * LOG2E;
                row_d.x = row_d.y = -diff_ld(p.delta + at);
            }
            int s = w.lo;
            for (int x = 0; x < w.n; ++x) {
                const uint32_t hx = h++;
                const int c0 = s * C::BC;
                if (++s == w.lo + per) s = w.lo;
                const float* col = columns + (hx & 1) * C::COL_FLOATS;
                if (!kDQ && !wait_all(&bars->col_full[hx & 1], (hx >> 1) & 1)) break;
                if (!wait_all(&bars->s_full, hx & 1)) break;
                tc_fence_after_sync();
                const uint32_t sb = tmem + lane_addr + (hx & 1) * C::BC + (uint32_t)(wg * C::HC);
                const uint32_t xb = tmem + lane_addr + C::X_COL + (uint32_t)(wg * C::HC);
                uint32_t a[C::HC], b[C::HC];
#pragma unroll
                for (int ch = 0; ch < C::HC; ch += 32) {
                    tmem_ld32p(xb + ch, b + ch);
                    tmem_ld32p(sb + ch, a + ch);
                }
                tmem_wait_ld_only();
#pragma unroll
                for (int ch = 0; ch < C::HC; ch += 32) {
                    reg_fence32(b + ch);
                    reg_fence32(a + ch);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->x_free));
                auto step = [&](auto masked_tag) {
                    constexpr bool kMasked = decltype(masked_tag)::value;
                    float2 f2 = make_float2(1.0f, 1.0f);
                    if constexpr (!kDQ) f2.x = f2.y = col[2 * C::BC];
#pragma unroll
                    for (int ch = 0; ch < C::HC / 32; ++ch) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e4 = 0; e4 < 8; ++e4) {
                            float4 l4, d4;
                            if constexpr (!kDQ) {
                                l4 = *reinterpret_cast<const float4*>(col + wg * C::HC + ch * 32 + 4 * e4);
                                d4 = *reinterpret_cast<const float4*>(col + C::BC + wg * C::HC + ch * 32 + 4 * e4);
                            }
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int e = ch * 32 + 4 * e4 + 2 * k;
                                const float2 l = kDQ ? row_l : k ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
                                const float2 d = kDQ ? row_d : k ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y);
                                const float2 va = make_float2(__uint_as_float(a[e]), __uint_as_float(a[e + 1]));
                                const float2 vb = make_float2(__uint_as_float(b[e]), __uint_as_float(b[e + 1]));
                                const float2 xa = __ffma2_rn(va, c2, l);
                                float2 pa = make_float2(ex2(xa.x), ex2(xa.y)), r;
                                if constexpr (kDV) {
                                    const float2 xv = __ffma2_rn(vb, c2, d);
                                    r = __ffma2_rn(make_float2(ex2(xv.x), ex2(xv.y)), f2, pa);
                                } else {
                                    if constexpr (!kDQ) pa = __fmul2_rn(pa, f2);
                                    r = __fmul2_rn(pa, __fadd2_rn(vb, d));
                                }
                                if constexpr (kMasked) {
                                    const uint32_t off = (uint32_t)(c0 + wg * C::HC - m_lo) + (uint32_t)e;
                                    r.x = off <= m_span ? r.x : 0.0f;
                                    r.y = off + 1u <= m_span ? r.y : 0.0f;
                                }
                                pk[2 * e4 + k] = pack_bf16x2(r.x, r.y);
                            }
                        }
                        tmem_st16p(sb + ch * 16, pk);           // over S, already loaded
                    }
                };
                if (diff_bwd_full(p, w.N, kDQ ? w.t * 128 : c0, kDQ ? 128 : C::BC, kDQ ? c0 : w.t * 128, kDQ ? C::BC : 128))
                    step(std::false_type{});
                else
                    step(std::true_type{});
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&bars->p_full));
                    if (!kDQ) mbar_arrive(smem_u32(&bars->col_empty[hx & 1]));
                }
            }
            if (!ok) break;
            if (!wait_all(&bars->acc_done, units_done & 1)) break;
            tc_fence_after_sync();
            // each warpgroup writes half of the accumulator's columns
            float f = kDV ? 1.0f : p.scale;
            __nv_bfloat16* out;
            if constexpr (kDQ) {
                if (w.z & 1) f *= -diff_ld(p.lam + (w.z >> 1));
                out = static_cast<__nv_bfloat16*>(p.dq);
            } else {
                out = static_cast<__nv_bfloat16*>(kDV ? p.dv : p.dk);
            }
            out += diff_bwd_row<kPacked>(p, w, heads, w.z, my) * C::ACC + wg * (C::ACC / 2);
#pragma unroll
            for (int ch = 0; ch < C::ACC / 64; ++ch) {
                uint32_t r[32];
                tmem_ld32(tmem + lane_addr + C::ACC_COL + wg * (C::ACC / 2) + ch * 32, r);
                tmem_wait_ld(r);
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    pk[e] = pack_bf16x2(__uint_as_float(r[2 * e]) * f, __uint_as_float(r[2 * e + 1]) * f);
                if (valid) {
                    uint4* dst = reinterpret_cast<uint4*>(out + ch * 32);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        dst[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->acc_empty));
            ++units_done;
        }
        if (!ok) timed_out();
        tmem_wait_st();
    } else {
        regs_decrease<C::REG_CONTROL>();
        if (!kDQ && warp == C::COLUMN_WARP) {
            // what the columns of a step need: minus the LSE (log2 units) of the map and minus D, or minus both
            // maps' LSE (dV), and the factor of the weights (of map 2), a step ahead of the compute warps
            constexpr int PER = C::BC / 32;             // columns of a lane
            constexpr float LOG2E = 1.4426950408889634f;
            uint32_t h = 0, units = 0;
            bool ok = true;
            DiffBwdUnit w;
            while (take_unit(units, ok, w)) {
                const int per = w.n / G;
                int head = 0, s = w.lo;
                for (int x = 0; x < w.n && ok; ++x, ++h) {
                    const int hq = (kDV ? w.z : w.z >> 1) * G + head;
                    const size_t at = diff_bwd_vec<kPacked>(p, w, 2 * hq + (kDV ? 0 : w.z & 1));
                    const size_t other = kPacked ? (size_t)p.T : (size_t)p.N;     // from map 1 to map 2
                    float l[PER], d[PER];
#pragma unroll
                    for (int k = 0; k < PER; ++k) {
                        const int q = min(s * C::BC + k * 32 + lane, w.N - 1);
                        l[k] = -diff_ld(p.lse + at + q) * LOG2E;
                        d[k] = kDV ? -diff_ld(p.lse + at + other + q) * LOG2E : -diff_ld(p.delta + at + q);
                    }
                    const float f = kDV || (w.z & 1) ? -diff_ld(p.lam + hq) : 1.0f;
                    if (++s == w.lo + per) {
                        s = w.lo;
                        ++head;
                    }
                    ok = warp_wait(&bars->col_empty[h & 1], ((h >> 1) & 1) ^ 1);
                    if (!ok) break;
                    float* col = columns + (h & 1) * C::COL_FLOATS;
#pragma unroll
                    for (int k = 0; k < PER; ++k) {
                        col[k * 32 + lane] = l[k];
                        col[C::BC + k * 32 + lane] = d[k];
                    }
                    if (lane == 0) col[2 * C::BC] = f;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->col_full[h & 1]));
                }
            }
            if (!ok) timed_out();
        }
        if (kPass == kPassDK && warp == C::SUM_WARP) diff_dlam(p, lane);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == C::MMA_WARP) tmem_dealloc(tmem, 512);
    // the last pass's end is the end of all
    if constexpr (kPass != kPassDK) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One pass, as a dependent of what was launched before it.
template <int D, int kPass, bool kPacked>
static cudaError_t launch_diff_bwd_pass(const DiffBwdMaps& m, const DiffBwdParams& p, int heads, int sm_count,
                                        cudaStream_t stream)
{
    using C = DiffBwdCfg<D, kPass>;
    auto kernel = diff_bwd_kernel<D, kPass, kPacked>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc would wait forever if the launch pool were smaller than the split
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
    if (attr.numRegs * C::NUM_THREADS < C::REG_POOL) return cudaErrorInvalidConfiguration;
    const long long units = (long long)p.nt * p.B * heads;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute dep[1];
    dep[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dep[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = dep;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3((unsigned)(units < sm_count ? units : sm_count));
    cfg.blockDim = dim3(C::NUM_THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    if constexpr (C::DQ) return cudaLaunchKernelEx(&cfg, kernel, m.q, m.dout, m.k, m.v, p);
    else if constexpr (C::BC == 64) return cudaLaunchKernelEx(&cfg, kernel, m.k, m.v, m.q64, m.dout64, p);
    else return cudaLaunchKernelEx(&cfg, kernel, m.k, m.v, m.q, m.dout, p);
}

template <int D, bool kPacked>
static cudaError_t launch_diff_bwd_t(const DiffBwdMaps& m, const DiffBwdParams& p, int sm_count, cudaStream_t stream)
{
    const long long rows = kPacked ? (long long)p.T * p.H : (long long)p.B * p.H * p.N;
    diff_dot_kernel<D><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if ((e = launch_diff_bwd_pass<D, kPassDK, kPacked>(m, p, 2 * p.Hkv, sm_count, stream)) != cudaSuccess) return e;
    if ((e = launch_diff_bwd_pass<D, kPassDV, kPacked>(m, p, p.Hkv, sm_count, stream)) != cudaSuccess) return e;
    return launch_diff_bwd_pass<D, kPassDQ, kPacked>(m, p, 2 * p.H, sm_count, stream);
}

cudaError_t launch_diff_bwd(const DiffBwdMaps& m, const DiffBwdParams& p, int d, int sm_count, cudaStream_t stream)
{
    const bool packed = p.cu_seqlens != nullptr;
    if (d == 64) return packed ? launch_diff_bwd_t<64, true>(m, p, sm_count, stream)
                               : launch_diff_bwd_t<64, false>(m, p, sm_count, stream);
    if (d == 128) return packed ? launch_diff_bwd_t<128, true>(m, p, sm_count, stream)
                                : launch_diff_bwd_t<128, false>(m, p, sm_count, stream);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
