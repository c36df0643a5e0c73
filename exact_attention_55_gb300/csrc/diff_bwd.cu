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
// Three launches, no floating-point atomics:
//   diff_dot_kernel            D_1 and D_2 of every row, one warp a row;
//   diff_bwd_kernel<D, true>   (dQ pass) a unit is 128 query rows of one map: in steps of 128 keys
//                              (64 at d = 128), S = Q K_j^T and dP = dO V_j^T into TMEM, the compute warps turn
//                              them into dS (bf16, over S), then dQ += dS K_j;
//   diff_bwd_kernel<D, false>  (dK/dV pass) a unit is 128 keys of a key pair, taken as two items, one
//                              a map: in steps of 64 queries over every head that reads it, the
//                              transposed products, then dV += P^T dO_i and dK += dS^T Q_i.  dV
//                              stays in TMEM from the first item to the second.
// dP is computed for each map: 28 d products per pair of tokens where 20 d would do if both maps'
// scores, dP and accumulators fitted TMEM at once (640 and 704 columns of 512 in the dK/dV pass).
// The structure of each pass, its roles and its waits are those of attn_bwd.cu, with two
// differences.  Units are handed out by a counter, the costliest first, because shared heads
// leave few of them (128 key tiles for 152 SMs in an 8192-token step with two key pairs).
// And what lies behind a packed sequence never enters a product: masked entries are selected
// away before dP can make them NaN, and the rows of the operands become 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "attn_params.h"
#include "diff_params.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace gb300 {

template <int D, bool kDQ>
struct DiffBwdCfg {
    static constexpr int BT = 128;                 // rows of a unit's tile
    // Columns of a step.  dQ pass at d = 128: a step of 128 keys would want K_{j-1}, K_j and V_j (128 KB)
    // beside Q and dO (96 KB), which leaves no room to load ahead.
    static constexpr int BC = kDQ && D == 64 ? 128 : 64;
    static constexpr int NCB = D / 64;             // 64-column blocks of a row of d
    static constexpr int FIX_CB = BT * 128;        // bytes of one, fixed tiles
    static constexpr int RING_CB = BC * 128;       // and ring tiles
    static constexpr int FIX_BYTES = 3 * NCB * FIX_CB;      // d columns (Q or K), then 2d (dO or V)
    static constexpr int SLOT = NCB * RING_CB;              // d columns of a step
    static constexpr int STEP_SLOTS = 3;                    // K and V's halves, or Q and dO's
    static constexpr int SMEM_CAP = 227 * 1024;
    // after the barriers, dK/dV: the warps' LSE and D, float [8][2][32]; then the schedule table
    static constexpr int MAX_SLOTS = 12;
    static constexpr int COL_OFF = 512;
    static constexpr int TAB_OFF = kDQ ? COL_OFF : COL_OFF + 2048;
    static constexpr int BAR_BYTES = (TAB_OFF + (int)sizeof(SortTab) + 15) / 16 * 16;
    static constexpr int NSLOT_FIT = (SMEM_CAP - BAR_BYTES - 1024 - FIX_BYTES) / SLOT;
    static constexpr int NSLOT = NSLOT_FIT < MAX_SLOTS ? NSLOT_FIT : MAX_SLOTS;
    static constexpr int SMEM_BYTES = 1024 + FIX_BYTES + NSLOT * SLOT + BAR_BYTES;
    // TMEM.  dQ pass: S of step h at 128 (h & 1), dP at 256, dQ at 384.  dK/dV pass: step buffers of
    // S^T (64 columns) and dP^T (64), two at d = 64 and one at d = 128, dV at 256, dK behind it
    // or (d = 128) before it.
    static constexpr int NB = kDQ || D == 64 ? 2 : 1;
    static constexpr int DP_OFF = kDQ ? 256 : 64;
    static constexpr int DQ_COL = 384, DV_COL = 256, DK_COL = D == 64 ? 384 : 128;
    static constexpr int COMPUTE_WARPS = 8, NUM_THREADS = 384, PRODUCER_WARP = 8, MMA_WARP = 9, SUM_WARP = 10;
    static constexpr int REG_COMPUTE = 208, REG_CONTROL = 88;
    static constexpr int REG_POOL = 256 * REG_COMPUTE + 128 * REG_CONTROL;
    static_assert(D == 64 || D == 128, "head dim");
    // dQ pass: V_j's second half waits for a slot while K_{j-1}, five before it, is still held
    static_assert(NSLOT >= (kDQ ? 6 : 3), "ring too small");
    static_assert(SMEM_BYTES <= SMEM_CAP, "shared memory");
};

struct alignas(16) DiffBwdBars {
    uint64_t fix_full, fix_empty;
    uint64_t ring_full[12], ring_empty[12];
    uint64_t s_full[2], p_full[2];
    uint64_t dp_free;
    uint64_t acc_done, acc_empty;
    uint64_t unit_full[2], unit_empty[2];
    uint64_t drain;
    int unit[2];                                   // the units handed out, -1 at the end
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(DiffBwdBars) <= 512, "barrier block");

// One unit: tile t (128 rows) of a head, or of a key pair, of one sequence.
struct DiffBwdUnit {
    int t, N, y0;      // tile, rows of the sequence, its first token (packed)
    int b, z;          // batch entry (packed: 0); dQ pass: 2 h + map, dK/dV pass: key pair
};

__device__ __forceinline__ int diff_bwd_units(const DiffBwdParams& p, int heads, const SortTab* tab)
{
    return tab != nullptr ? tab->total : p.nt * p.B * heads;
}

// Unit u, costliest first under a causal mask: a query tile t meets t + 1 key tiles, a key tile nt - t
// query tiles.  Batched: rank by rank over all heads; packed, from the table: the longest sequence
// first.  More sequences than the table holds: slots laid out for the longest one; false where
// a sequence is shorter.
template <bool kDQ, bool kPacked>
__device__ __forceinline__ bool diff_bwd_unit(const DiffBwdParams& p, int u, int heads, const SortTab* tab, DiffBwdUnit& w)
{
    int rank, seq;
    if (kPacked && tab != nullptr) {
        int rem;
        sorted_pair(tab, p.B, u, seq, rem);
        rank = rem / heads;
        w.z = rem - rank * heads;
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

// D_1 and D_2 in fp32, one warp a row; the units' counters start at 0.
template <int D>
__global__ void __launch_bounds__(256) diff_dot_kernel(const DiffBwdParams p)
{
    constexpr int E = 2 * D / 32;
    if (blockIdx.x == 0 && threadIdx.x < 2) p.next[threadIdx.x] = 0;
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
        if (t < __ldg(p.cu_seqlens) || t >= __ldg(p.cu_seqlens + p.B)) return;   // outside every sequence
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
        p.delta[at] = fmaf(__ldg(p.lam + h), b, a);
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
                const int t0 = min(max(__ldg(p.cu_seqlens), 0), p.T);
                n = min(max(__ldg(p.cu_seqlens + p.B), t0), p.T) - t0;
                d = p.delta + (size_t)(2 * h + 1) * p.T + t0;
            } else {
                n = p.N;
                d = p.delta + ((size_t)b * 2 * p.H + 2 * h + 1) * p.N;
            }
            for (long long i = lane; i < n; i += 256) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (i + 32 * k < n) acc[k] += d[i + 32 * k];
            }
        }
        float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (lane == 0) p.dlam[h] = -sum;
    }
}

// One pass.  Maps: dQ pass fixed Q and dO, ring K and V; dK/dV pass fixed K and V, ring Q and dO.
template <int D, bool kDQ, bool kPacked>
__global__ void __launch_bounds__(DiffBwdCfg<D, kDQ>::NUM_THREADS, 1)
    diff_bwd_kernel(const __grid_constant__ CUtensorMap tmFixA, const __grid_constant__ CUtensorMap tmFixB,
                    const __grid_constant__ CUtensorMap tmRingA, const __grid_constant__ CUtensorMap tmRingB,
                    const DiffBwdParams p)
{
    using C = DiffBwdCfg<D, kDQ>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* fix = smem;
    uint8_t* ring = smem + C::FIX_BYTES;
    auto* bars = reinterpret_cast<DiffBwdBars*>(ring + C::NSLOT * C::SLOT);
    const volatile int* abort_flag = &bars->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = kDQ ? 2 * p.H : p.Hkv, G = p.H / p.Hkv;
    const int items = kDQ ? 1 : 2;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->fix_full), 1);
        mbar_init(smem_u32(&bars->fix_empty), 1);
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(smem_u32(&bars->ring_full[s]), 1);
            mbar_init(smem_u32(&bars->ring_empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bars->s_full[b]), 1);
            mbar_init(smem_u32(&bars->p_full[b]), C::COMPUTE_WARPS);
            mbar_init(smem_u32(&bars->unit_full[b]), 1);
            mbar_init(smem_u32(&bars->unit_empty[b]), C::COMPUTE_WARPS + 1);
        }
        mbar_init(smem_u32(&bars->dp_free), C::COMPUTE_WARPS);
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
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    const SortTab* tab = nullptr;
    if constexpr (kPacked) {
        if (p.B <= kSortMaxSeqs) {
            SortTab* t = reinterpret_cast<SortTab*>(reinterpret_cast<uint8_t*>(bars) + C::TAB_OFF);
            build_sort_tab<64>(p.cu_seqlens, p.B, p.T, heads, t);   // pairs of 64 rows: tiles
            tab = t;
        }
    }
    const int total = diff_bwd_units(p, heads, tab);
    auto timed_out = [&]() {
        atomicExch(p.status, kStatusTimeout);
        *reinterpret_cast<volatile int*>(&bars->abort_flag) = 1;
    };
    // A consumer warp's next unit (all lanes); -1 at the end or after an abort.
    auto take_unit = [&](uint32_t& n, bool& ok) -> int {
        const uint32_t b = n & 1;
        const bool r = mbar_wait(smem_u32(&bars->unit_full[b]), (n >> 1) & 1, abort_flag, p.timeout_ns);
        if (!__all_sync(0xffffffffu, r)) {
            ok = false;
            return -1;
        }
        const int u = *reinterpret_cast<volatile int*>(&bars->unit[b]);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->unit_empty[b]));
        ++n;
        return u;
    };

    if (warp == C::PRODUCER_WARP) {
        regs_decrease<C::REG_CONTROL>();
        if (lane == 0) {
            const uint64_t pol_fix = l2_policy_evict_first(), pol_ring = l2_policy_evict_last();
            uint32_t rc = 0, fixed = 0, given = 0;
            int walk = (int)blockIdx.x;
            bool ok = true;
            // the next ring slot gets d columns from `col` on of `row` of a map
            auto load = [&](const CUtensorMap* map, int col, int row, int head) {
                if (!ok) return;
                const uint32_t slot = rc % C::NSLOT;
                if (!mbar_wait(smem_u32(&bars->ring_empty[slot]), ((rc / C::NSLOT) & 1) ^ 1, abort_flag, p.timeout_ns)) {
                    ok = false;
                    return;
                }
                if (++rc == (uint32_t)p.withhold) return;      // test hook: never arrives
                const uint32_t rb = smem_u32(&bars->ring_full[slot]);
                mbar_arrive_expect_tx(rb, C::SLOT);
#pragma unroll
                for (int cb = 0; cb < C::NCB; ++cb)
                    tma_load_3d(smem_u32(ring + slot * C::SLOT + cb * C::RING_CB), map, rb, col + cb * 64, row, head,
                                pol_ring);
            };
            while (ok) {
                DiffBwdUnit w;
                int u;
                if (!kPacked || tab != nullptr) {
                    u = atomicAdd(p.next + (kDQ ? 0 : 1), 1);
                } else {                       // slots with gaps: walked without the counter
                    u = walk;
                    walk += gridDim.x;
                }
                const bool more = u < total;
                if (more && !diff_bwd_unit<kDQ, kPacked>(p, u, heads, tab, w)) continue;
                const uint32_t b = given & 1;
                if (!mbar_wait(smem_u32(&bars->unit_empty[b]), ((given >> 1) & 1) ^ 1, abort_flag, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                *reinterpret_cast<volatile int*>(&bars->unit[b]) = more ? u : -1;
                mbar_arrive(smem_u32(&bars->unit_full[b]));
                ++given;
                if (!more) break;
                int lo, hi;
                diff_bwd_steps<kDQ, C::BC>(p, w, lo, hi);
                for (int m = 0; m < items && ok; ++m) {
                    if (!mbar_wait(smem_u32(&bars->fix_empty), (fixed & 1) ^ 1, abort_flag, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&bars->fix_full);
                    mbar_arrive_expect_tx(fb, C::FIX_BYTES);
                    ++fixed;
                    const int row = w.y0 + w.t * 128;
                    const int za = kDQ ? w.b * 2 * p.H + w.z : w.b * 2 * p.Hkv + 2 * w.z + m;
                    const int zb = kDQ ? w.b * p.H + (w.z >> 1) : w.b * p.Hkv + w.z;
#pragma unroll
                    for (int cb = 0; cb < 3 * C::NCB; ++cb) {
                        const bool first = cb < C::NCB;
                        tma_load_3d(smem_u32(fix + cb * C::FIX_CB), first ? &tmFixA : &tmFixB, fb,
                                    (first ? cb : cb - C::NCB) * 64, row, first ? za : zb, pol_fix);
                    }
                    if constexpr (kDQ) {
                        const int g = (w.z >> 1) / G, zk = w.b * 2 * p.Hkv + 2 * g + (w.z & 1), zv = w.b * p.Hkv + g;
                        for (int j = lo; j < hi && ok; ++j) {
                            load(&tmRingA, 0, w.y0 + j * C::BC, zk);
                            load(&tmRingB, 0, w.y0 + j * C::BC, zv);
                            load(&tmRingB, D, w.y0 + j * C::BC, zv);
                        }
                    } else {
                        for (int i = 0; i < G; ++i) {
                            const int h = w.z * G + i, zq = w.b * 2 * p.H + 2 * h + m, zo = w.b * p.H + h;
                            for (int s = lo; s < hi && ok; ++s) {
                                load(&tmRingA, 0, w.y0 + s * C::BC, zq);
                                load(&tmRingB, 0, w.y0 + s * C::BC, zo);
                                load(&tmRingB, D, w.y0 + s * C::BC, zo);
                            }
                        }
                    }
                }
            }
            if (!ok) timed_out();
            // every copy issued lands before shared memory is released
            const uint32_t n = rc < C::NSLOT ? rc : C::NSLOT;
            for (uint32_t k = rc - n; k < rc; ++k) {
                if (k + 1 == (uint32_t)p.withhold) continue;
                mbar_wait(smem_u32(&bars->ring_full[k % C::NSLOT]), (k / C::NSLOT) & 1, nullptr, kCleanupTimeoutNs);
            }
            if (fixed > 0) mbar_wait(smem_u32(&bars->fix_full), (fixed - 1) & 1, nullptr, kCleanupTimeoutNs);
        }
    } else if (warp == C::MMA_WARP) {
        regs_decrease<C::REG_CONTROL>();
        constexpr uint32_t idesc_kk = idesc_f32acc(1, 0, 128, C::BC);  // both K-major
        constexpr uint32_t idesc_acc = idesc_f32acc(1, 1, 128, D);     // B MN-major
        const uint64_t fix_k = sdesc_sw128(smem_u32(fix), 16, 1024);
        const uint64_t ring_k = sdesc_sw128(smem_u32(ring), 16, 1024);
        const uint64_t ring_mn = sdesc_sw128(smem_u32(ring), C::RING_CB, 1024);
        uint32_t rc = 0, items_done = 0, hs = 0, units = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            bool r = ok && mbar_wait(smem_u32(bar), parity, abort_flag, p.timeout_ns);
            r = __all_sync(0xffffffffu, r);
            if (!r) ok = false;
            return r;
        };
        auto commit = [&](uint64_t* bar) { mma_commit_warp(smem_u32(bar)); };
        auto slot = [&](uint32_t n) { return n % C::NSLOT; };
        auto full = [&](uint32_t n) -> bool { return wait(&bars->ring_full[slot(n)], (n / C::NSLOT) & 1); };
        // d_col (+)= A B^T over d columns: fixed part `part` (0: Q or K; 1, 2: halves of dO or V), ring tile n
        auto mm_kk = [&](uint32_t d_col, int part, uint32_t n, bool accumulate) {
            const uint64_t a0 = fix_k + (uint64_t)((part * C::NCB * C::FIX_CB) >> 4);
            const uint64_t b0 = ring_k + (uint64_t)((slot(n) * C::SLOT) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int byte = kk * 32;
                mma_ss_warp<false>(tmem + d_col, a0 + (uint64_t)(((byte / 128) * C::FIX_CB + byte % 128) >> 4),
                                   b0 + (uint64_t)(((byte / 128) * C::RING_CB + byte % 128) >> 4), idesc_kk,
                                   (kk > 0 || accumulate) ? 1u : 0u);
            }
        };
        // acc_col (+)= A (TMEM, packed to bf16 by both warpgroups, each over the first half of its
        // columns) times ring tile n as MN-major
        auto mm_acc = [&](uint32_t acc_col, uint32_t a_col, uint32_t n, bool accumulate) {
            const uint64_t b0 = ring_mn + (uint64_t)((slot(n) * C::SLOT) >> 4);
            constexpr int PER = C::BC / 32;                            // k-steps of a warpgroup
#pragma unroll
            for (int kk = 0; kk < C::BC / 16; ++kk)
                mma_ts_warp<false>(tmem + acc_col, tmem + a_col + (kk / PER) * (C::BC / 2) + (kk % PER) * 8,
                                   b0 + (uint64_t)((kk * 16 * 128) >> 4), idesc_acc, (kk > 0 || accumulate) ? 1u : 0u);
        };
        // packed rows behind the sequence become 0 in ring tile n, whose first row is `row`
        auto clear_tail = [&](const DiffBwdUnit& w, int row, uint32_t n) {
            if constexpr (kPacked) {
                const int live = w.N - row;
                if (live >= C::BC) return;
                uint8_t* t = ring + slot(n) * C::SLOT;
                for (int o = live * 128 + lane * 16; o < C::RING_CB; o += 512)
#pragma unroll
                    for (int cb = 0; cb < C::NCB; ++cb)
                        *reinterpret_cast<uint4*>(t + cb * C::RING_CB + o) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            }
        };
        while (ok) {
            const int u = take_unit(units, ok);
            if (u < 0) break;
            DiffBwdUnit w;
            diff_bwd_unit<kDQ, kPacked>(p, u, heads, tab, w);
            int lo, hi;
            diff_bwd_steps<kDQ, C::BC>(p, w, lo, hi);
            if constexpr (kDQ) {
                // Step j: dP(j) once the compute warps have read dP(j-1), the accumulation of step
                // j-1, S(j+1) into the other buffer.  Ring: K_j, V_j's halves, K_{j+1}, ...
                const uint32_t r0 = rc, h0 = hs;
                auto nk = [&](int j) { return r0 + 3u * (uint32_t)(j - lo); };
                if (!wait(&bars->fix_full, items_done & 1)) break;
                if (!full(nk(lo))) break;
                clear_tail(w, lo * C::BC, nk(lo));
                tc_fence_after_sync();
                mm_kk((h0 & 1) * 128, 0, nk(lo), false);
                bool started = false;
                for (int j = lo; j < hi && ok; ++j) {
                    const uint32_t hj = h0 + (uint32_t)(j - lo), nv = nk(j) + 1;
                    if (!full(nv) || !full(nv + 1)) break;
                    if (hj > 0 && !wait(&bars->dp_free, (hj - 1) & 1)) break;
                    tc_fence_after_sync();
                    mm_kk(C::DP_OFF, 1, nv, false);
                    commit(&bars->ring_empty[slot(nv)]);
                    mm_kk(C::DP_OFF, 2, nv + 1, true);
                    commit(&bars->ring_empty[slot(nv + 1)]);
                    if (j == hi - 1) commit(&bars->fix_empty);
                    if (j > lo) {
                        // s_full of this step before the accumulation of the last, and only when that
                        // one's p_full was seen: no barrier runs a phase ahead
                        if (!wait(&bars->p_full[0], (hj - 1) & 1)) break;
                        commit(&bars->s_full[0]);
                        if (!started && !wait(&bars->acc_empty, (items_done & 1) ^ 1)) break;
                        tc_fence_after_sync();
                        mm_acc(C::DQ_COL, ((hj - 1) & 1) * 128, nk(j - 1), started);
                        started = true;
                        commit(&bars->ring_empty[slot(nk(j - 1))]);
                    } else {
                        commit(&bars->s_full[0]);
                    }
                    if (j + 1 < hi) {
                        if (!full(nk(j + 1))) break;
                        clear_tail(w, (j + 1) * C::BC, nk(j + 1));
                        tc_fence_after_sync();
                        mm_kk(((hj + 1) & 1) * 128, 0, nk(j + 1), false);
                    }
                }
                if (!ok) break;
                const uint32_t hl = h0 + (uint32_t)(hi - 1 - lo);
                if (!wait(&bars->p_full[0], hl & 1)) break;
                if (!started && !wait(&bars->acc_empty, (items_done & 1) ^ 1)) break;
                tc_fence_after_sync();
                mm_acc(C::DQ_COL, (hl & 1) * 128, nk(hi - 1), started);
                commit(&bars->ring_empty[slot(nk(hi - 1))]);
                commit(&bars->acc_done);
                rc = nk(hi);
                hs = h0 + (uint32_t)(hi - lo);
                ++items_done;
            } else {
                const int ns = hi - lo, n = G * ns;
                for (int m = 0; m < 2 && ok; ++m) {
                    if (!wait(&bars->fix_full, items_done & 1)) break;
                    // the accumulations of step h of this item (number x), from ring position r on
                    auto issue_acc = [&](uint32_t h, uint32_t r, int x) -> bool {
                        const uint32_t buf = (h % C::NB) * 128;
                        if (!wait(&bars->p_full[h % C::NB], (h / C::NB) & 1)) return false;
                        if (x == 0 && !wait(&bars->acc_empty, (items_done & 1) ^ 1)) return false;
                        tc_fence_after_sync();
                        mm_acc(C::DV_COL, buf, r + 1, m > 0 || x > 0);                   // dV += P^T dO
                        mm_acc(C::DV_COL + D, buf, r + 2, m > 0 || x > 0);
                        commit(&bars->ring_empty[slot(r + 1)]);
                        commit(&bars->ring_empty[slot(r + 2)]);
                        mm_acc(C::DK_COL, buf + C::DP_OFF, r, x > 0);                    // dK += dS^T Q
                        commit(&bars->ring_empty[slot(r)]);
                        return true;
                    };
                    for (int x = 0; x < n; ++x) {
                        if (C::NB == 1 && x > 0 && !issue_acc(hs - 1, rc - 3, x - 1)) break;
                        if (!full(rc) || !full(rc + 1) || !full(rc + 2)) break;
                        const int row = (lo + x % ns) * C::BC;
                        clear_tail(w, row, rc);
                        clear_tail(w, row, rc + 1);
                        clear_tail(w, row, rc + 2);
                        tc_fence_after_sync();
                        const uint32_t buf = (hs % C::NB) * 128;
                        mm_kk(buf, 0, rc, false);                                        // S^T
                        mm_kk(buf + C::DP_OFF, 1, rc + 1, false);                        // dP^T
                        mm_kk(buf + C::DP_OFF, 2, rc + 2, true);
                        commit(&bars->s_full[hs % C::NB]);
                        if (x == n - 1) commit(&bars->fix_empty);
                        if (C::NB == 2 && x > 0 && !issue_acc(hs - 1, rc - 3, x - 1)) break;
                        ++hs;
                        rc += 3;
                    }
                    if (!ok) break;
                    if (!issue_acc(hs - 1, rc - 3, n - 1)) break;
                    commit(&bars->acc_done);
                    ++items_done;
                }
            }
        }
        if (!ok && lane == 0) timed_out();
        commit(&bars->drain);
        mbar_wait(smem_u32(&bars->drain), 0, nullptr, kCleanupTimeoutNs);
        __syncwarp();
    } else if (warp < C::COMPUTE_WARPS) {
        // both warpgroups work on every step, warpgroup wg on its half of the columns
        regs_increase<C::REG_COMPUTE>();
        const int wg = warp >> 2, trow = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const float LOG2E = 1.4426950408889634f;
        uint32_t h = 0, units = 0, items_done = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
            bool r = ok && mbar_wait(smem_u32(bar), parity, abort_flag, p.timeout_ns);
            r = __all_sync(0xffffffffu, r);
            if (!r) ok = false;
            return r;
        };
        // `cols` accumulator columns from `col` on, times f, to a row of bf16
        auto write = [&](auto cols_tag, uint32_t col, float f, __nv_bfloat16* out, bool valid) {
            constexpr int cols = decltype(cols_tag)::value;
#pragma unroll
            for (int ch = 0; ch < cols / 32; ++ch) {
                uint32_t r[32];
                tmem_ld32(tmem + lane_addr + col + ch * 32, r);
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
        };
        while (ok) {
            const int u = take_unit(units, ok);
            if (u < 0) break;
            DiffBwdUnit w;
            diff_bwd_unit<kDQ, kPacked>(p, u, heads, tab, w);
            int lo, hi;
            diff_bwd_steps<kDQ, C::BC>(p, w, lo, hi);
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
            if constexpr (kDQ) {
                const size_t vec = diff_bwd_vec<kPacked>(p, w, w.z);
                const float lse2 = valid ? __ldg(p.lse + vec + my) * LOG2E : 0.0f;
                const float dlt = valid ? __ldg(p.delta + vec + my) : 0.0f;
                const uint32_t h0 = h;
                h = h0 + (uint32_t)(hi - lo);
                for (int j = lo; j < hi; ++j) {
                    const uint32_t hj = h0 + (uint32_t)(j - lo);
                    constexpr int HC = C::BC / 2;       // this warpgroup's keys
                    const int c0 = j * C::BC + wg * HC;
                    if (!wait_all(&bars->s_full[0], hj & 1)) break;
                    tc_fence_after_sync();
                    const uint32_t sb = tmem + lane_addr + (hj & 1) * 128 + (uint32_t)(wg * HC);
                    const uint32_t db = tmem + lane_addr + C::DP_OFF + (uint32_t)(wg * HC);
                    uint32_t sra[HC], dra[HC];
#pragma unroll
                    for (int ch = 0; ch < HC; ch += 32) {
                        tmem_ld32p(sb + ch, sra + ch);
                        tmem_ld32p(db + ch, dra + ch);
                    }
                    tmem_wait_ld_only();
#pragma unroll
                    for (int ch = 0; ch < HC; ch += 32) {
                        reg_fence32(sra + ch);
                        reg_fence32(dra + ch);
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->dp_free));
                    auto step = [&](auto masked_tag) {
                        constexpr bool kMasked = decltype(masked_tag)::value;
#pragma unroll
                        for (int ch = 0; ch < HC / 32; ++ch) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float ds[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int i = ch * 32 + 2 * e + k;
                                    const float pr = ex2(fmaf(__uint_as_float(sra[i]), p.c_log2, -lse2));
                                    ds[k] = pr * (__uint_as_float(dra[i]) - dlt);
                                    if constexpr (kMasked) {
                                        const uint32_t off = (uint32_t)(c0 - m_lo) + (uint32_t)i;
                                        ds[k] = off <= m_span ? ds[k] : 0.0f;
                                    }
                                }
                                pk[e] = pack_bf16x2(ds[0], ds[1]);
                            }
                            tmem_st16p(sb + ch * 16, pk);
                        }
                    };
                    if (diff_bwd_full(p, w.N, w.t * 128, 128, j * C::BC, C::BC)) step(std::false_type{});
                    else step(std::true_type{});
                    tmem_wait_st();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[0]));
                }
                if (!ok) break;
                if (!wait_all(&bars->acc_done, items_done & 1)) break;
                tc_fence_after_sync();
                const float f = (w.z & 1) ? -p.scale * __ldg(p.lam + (w.z >> 1)) : p.scale;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.dq) +
                                     diff_bwd_row<kPacked>(p, w, 2 * p.H, w.z, my) * D + wg * (D / 2);
                write(std::integral_constant<int, D / 2>{}, C::DQ_COL + wg * (D / 2), f, out, valid);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->acc_empty));
                ++items_done;
            } else {
                float* my_lse2 = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + C::COL_OFF) + warp * 64;
                float* my_delta = my_lse2 + 32;
                const int ns = hi - lo, n = G * ns;
                for (int m = 0; m < 2 && ok; ++m) {
                    // this lane's column of the next step: LSE (log2 units) and D
                    float nl = 0.0f, nd = 0.0f;
                    auto col_load = [&](int head, int s) {
                        const size_t at = diff_bwd_vec<kPacked>(p, w, 2 * (w.z * G + head) + m) +
                                          min(s * C::BC + wg * 32 + lane, w.N - 1);
                        nl = __ldg(p.lse + at) * LOG2E;
                        nd = __ldg(p.delta + at);
                    };
                    col_load(0, lo);
                    int head = 0, s = lo;
                    float f = m ? -__ldg(p.lam + w.z * G) : 1.0f;
                    for (int x = 0; x < n; ++x) {
                        __syncwarp();                   // the last step's values have been read
                        my_lse2[lane] = nl;
                        my_delta[lane] = nd;
                        __syncwarp();
                        const int c0 = s * C::BC + wg * 32;
                        const float fx = f;
                        const bool open = diff_bwd_full(p, w.N, s * C::BC, C::BC, w.t * 128, 128);
                        if (++s == hi) {
                            s = lo;
                            ++head;
                            if (m && head < G) f = -__ldg(p.lam + w.z * G + head);
                        }
                        if (head < G) col_load(head, s);
                        const uint32_t hx = h++;
                        if (!wait_all(&bars->s_full[hx % C::NB], (hx / C::NB) & 1)) break;
                        tc_fence_after_sync();
                        const uint32_t sb = tmem + lane_addr + (hx % C::NB) * 128 + (uint32_t)wg * 32;
                        uint32_t sr[32], dr[32];
                        tmem_ld32p(sb, sr);
                        tmem_ld32p(sb + C::DP_OFF, dr);
                        tmem_wait_ld_only();
                        reg_fence32(sr);
                        reg_fence32(dr);
                        auto step = [&](auto masked_tag) {
                            constexpr bool kMasked = decltype(masked_tag)::value;
                            uint32_t pp[16], pd[16];
#pragma unroll
                            for (int e4 = 0; e4 < 8; ++e4) {
                                const float4 l4 = *reinterpret_cast<const float4*>(my_lse2 + 4 * e4);
                                const float4 d4 = *reinterpret_cast<const float4*>(my_delta + 4 * e4);
                                const float l[4] = {l4.x, l4.y, l4.z, l4.w}, d[4] = {d4.x, d4.y, d4.z, d4.w};
                                float pv[4], ds[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int i = 4 * e4 + k;
                                    pv[k] = fx * ex2(fmaf(__uint_as_float(sr[i]), p.c_log2, -l[k]));
                                    ds[k] = pv[k] * (__uint_as_float(dr[i]) - d[k]);
                                    if constexpr (kMasked) {
                                        const uint32_t off = (uint32_t)(c0 - m_lo) + (uint32_t)i;
                                        pv[k] = off <= m_span ? pv[k] : 0.0f;
                                        ds[k] = off <= m_span ? ds[k] : 0.0f;
                                    }
                                }
                                pp[2 * e4] = pack_bf16x2(pv[0], pv[1]);
                                pp[2 * e4 + 1] = pack_bf16x2(pv[2], pv[3]);
                                pd[2 * e4] = pack_bf16x2(ds[0], ds[1]);
                                pd[2 * e4 + 1] = pack_bf16x2(ds[2], ds[3]);
                            }
                            tmem_st16p(sb, pp);                 // P^T over S^T
                            tmem_st16p(sb + C::DP_OFF, pd);     // dS^T over dP^T
                        };
                        if (open) step(std::false_type{});
                        else step(std::true_type{});
                        tmem_wait_st();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[hx % C::NB]));
                    }
                    if (!ok) break;
                    if (!wait_all(&bars->acc_done, items_done & 1)) break;
                    tc_fence_after_sync();
                    __nv_bfloat16* dk = static_cast<__nv_bfloat16*>(p.dk) +
                                        diff_bwd_row<kPacked>(p, w, 2 * p.Hkv, 2 * w.z + m, my) * D + wg * (D / 2);
                    write(std::integral_constant<int, D / 2>{}, C::DK_COL + wg * (D / 2), p.scale, dk, valid);
                    if (m == 1) {
                        __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(p.dv) +
                                            diff_bwd_row<kPacked>(p, w, p.Hkv, w.z, my) * (2 * D) + wg * D;
                        write(std::integral_constant<int, D>{}, C::DV_COL + wg * D, 1.0f, dv, valid);
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->acc_empty));
                    ++items_done;
                }
            }
        }
        if (!ok) timed_out();
        tmem_wait_st();
    } else {
        regs_decrease<C::REG_CONTROL>();
        if (!kDQ && warp == C::SUM_WARP) diff_dlam(p, lane);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == C::MMA_WARP) tmem_dealloc(tmem, 512);
}

template <int D, bool kPacked>
static cudaError_t launch_diff_bwd_t(const DiffBwdMaps& m, const DiffBwdParams& p, int sm_count, cudaStream_t stream)
{
    using CQ = DiffBwdCfg<D, true>;
    using CK = DiffBwdCfg<D, false>;
    const long long rows = kPacked ? (long long)p.T * p.H : (long long)p.B * p.H * p.N;
    diff_dot_kernel<D><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    auto kq = diff_bwd_kernel<D, true, kPacked>;
    auto kk = diff_bwd_kernel<D, false, kPacked>;
    if ((e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, CQ::SMEM_BYTES)) != cudaSuccess)
        return e;
    if ((e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, CK::SMEM_BYTES)) != cudaSuccess)
        return e;
    // setmaxnreg.inc would wait forever if the launch pool were smaller than the split
    for (const void* f : {reinterpret_cast<const void*>(kq), reinterpret_cast<const void*>(kk)}) {
        cudaFuncAttributes attr;
        if ((e = cudaFuncGetAttributes(&attr, f)) != cudaSuccess) return e;
        if (attr.numRegs * CQ::NUM_THREADS < CQ::REG_POOL) return cudaErrorInvalidConfiguration;
    }
    const long long tiles = (long long)p.nt * p.B;
    auto grid = [&](int heads) { return (int)(tiles * heads < sm_count ? tiles * heads : sm_count); };
    kq<<<grid(2 * p.H), CQ::NUM_THREADS, CQ::SMEM_BYTES, stream>>>(m.q, m.dout, CQ::BC == 64 ? m.k64 : m.k,
                                                                       CQ::BC == 64 ? m.v64 : m.v, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    kk<<<grid(p.Hkv), CK::NUM_THREADS, CK::SMEM_BYTES, stream>>>(m.k, m.v, m.q64, m.dout64, p);
    return cudaGetLastError();
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
