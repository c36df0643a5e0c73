// diff_decode.cu -- one decoding step of differential attention over a paged bf16 cache.
//
// "大模型加速-核心网络算子-Flash Attention V3" §3 总结 (decoding over cached K and V); "Warp Group
// Cluster 优化：Flash Attention V3 在 H100 上的 FP8 融合计算实践", 局限性与后续方向 item 2
// (PagedAttention).  Head h has the query heads 2h, 2h + 1 and reads key pair g = h / (H / Hkv); the
// cache's heads 2g and 2g + 1 hold the pair's keys in K, and the two halves of value head g in V.
//     S_m = scale q_m K_m^T,  O = (softmax(S_1) - lam softmax(S_2)) V
// Row r = (h - g H / Hkv) nq + i of a map is query i of head h, at position L - nq + i; it sees keys
// max(0, position - window) .. position (window 0: all of them).
//
// HBM-bound: 8 d bytes of the cache a key and pair, each used by 2 to 4 products per row.
//   * Work is cut, walked and joined as in decode_fp8.cuh: equal ranges of 64-key tiles, one a
//     resident CTA; parts of a split pair meet in the workspace and a dependent launch joins them,
//     takes the two maps' quotients and subtracts.
//   * Warp 4 streams the tiles: TMA boxes (one per page or 64 rows) of both keys and both value
//     halves into a ring, and the next unit's queries by cp.async.
//   * Warps 0-3 take 16 keys of each tile: S^T = K Q^T and O^T += V^T P^T as mma.m16n8k16, with 16
//     keys (or value columns) by eight query rows.  With up to four rows of a map both maps share
//     one product's eight columns, map 1 in 0-3 and map 2 in 4-7: K_1 meets (q_1 | 0) and K_2
//     (0 | q_2), each column takes its own map's sum, and V is multiplied once for both.  Otherwise the
//     columns of a product are one map's, and V's fragments are used for both.
//     A tcgen05 tile would be at least 64 rows high, mostly empty.
// Measured, 16 sequences x 8 heads x 8192 keys of d = 128 (1.07 GB): 158.8 us = 6.76 TB/s.
// Scores, weights' sums and O are fp32.  A weight, relative to a running maximum that it may pass by
// 2^8, enters as two bf16 numbers, what it rounds to and the rest, off by 2^-17 of it (one of them
// would double O's error, 0.0017 to 0.0026 relative at 16 x 8 heads x 8192 keys; the second product
// hides behind the loads).  Keys that a row does not see have weight 0, value rows outside every
// row's range become 0, and a NaN or infinite value at a key that only some rows see is taken out
// of the product and reaches those rows as NaN (keep_nan).
#include <cmath>

#include "decode_fp8.cuh"
#include "diff_params.h"

namespace gb300 {

constexpr int kDdWarps = 4, kDdThreads = (kDdWarps + 1) * 32, kDdTile = 64;
constexpr float kDdTau = 8.0f;

template <int D, int NT>
struct DdCfg {
    static constexpr int RC = 4 * NT;                     // rows of a map
    static constexpr int COLS = 8 * NT;                   // both maps
    static constexpr int CB = kDdTile * 128;              // 64 columns of a tile
    static constexpr int PART = (D / 64) * CB;            // one cache head of a tile
    static constexpr int STAGE = 4 * PART;                // K_1, K_2 and V's halves
    static constexpr int STAGES = 3;
    static constexpr int QS = D + 8;                      // elements between two query rows
    static constexpr int Q_BYTES = COLS * QS * 2;
    static constexpr int SMEM = 1024 + STAGES * STAGE + 2 * Q_BYTES + 1024;
    static constexpr int CTAS = diff_decode_ctas(D);
    static_assert(SMEM <= (CTAS == 2 ? 113 : 227) * 1024, "shared memory");
    static_assert(STAGE >= kDdWarps * 8 * 2 * D * 4, "a unit's last stage holds the warps' O for joining");
};

template <int D, int NT>
struct alignas(16) DdShared {
    using C = DdCfg<D, NT>;
    uint64_t full[C::STAGES], empty[C::STAGES];
    uint64_t q_full[2], q_empty[2];
    uint64_t meet;
    float m[kDdWarps][8], l[kDdWarps][8];                 // eight columns at a time
    Dec8Setup<kDdThreads> setup;
    int abort_flag;
};

__device__ __forceinline__ void dd_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool kTrans>
__device__ __forceinline__ void dd_ldmatrix(uint32_t (&r)[4], uint32_t addr)
{
    if constexpr (kTrans)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t dd_transpose(uint32_t x)   // 8x8 of 16-bit across the warp
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// 0xFFFF in each half of w whose bf16 is not finite.
__device__ __forceinline__ uint32_t dd_nonfinite(uint32_t w)
{
    const uint32_t top = ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;   // the exponent is all ones
    return (top >> 15) * 0xFFFFu;
}

// Index of query (or LSE) row `row` of map m: row = (b Hkv + g) rows + r, heads x queries in order.
__device__ __forceinline__ size_t dd_qrow(size_t row, int nq, int m)
{
    const size_t bh = row / (unsigned)nq;
    return (2 * bh + m) * nq + (row - bh * nq);
}

__device__ __forceinline__ float dd_lse(float m, float l)
{
    if (l == 0.0f) return -__int_as_float(0x7f800000);
    return ((m == -__int_as_float(0x7f800000) ? 0.0f : m) + __log2f(l)) * 0.69314718055994531f;
}

__device__ __forceinline__ float dd_lam(const DiffDecodeParams& p, size_t row)   // of output row `row`
{
    float v;                                              // plain, behind the grid's wait (decode_fp8.cuh)
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p.lam + (row / (unsigned)p.w.nq) % (unsigned)p.H));
    return v;
}

// Four columns of an output row from both maps' sums.
__device__ __forceinline__ uint2 dd_out(float4 a, float l1, float4 b, float l2, float lam)
{
    const float i1 = l1 == 0.0f ? 0.0f : 1.0f / l1, i2 = l2 == 0.0f ? 0.0f : lam / l2;
    return make_uint2(pack_bf16x2(fmaf(a.x, i1, -(b.x * i2)), fmaf(a.y, i1, -(b.y * i2))),
                      pack_bf16x2(fmaf(a.z, i1, -(b.z * i2)), fmaf(a.w, i1, -(b.w * i2))));
}

// Sequences without a key: O = 0, LSE = -inf.  The CTAs share them.
template <int D>
__device__ __forceinline__ void dd_write_empty(const DiffDecodeParams& p, int threads)
{
    for (int b = blockIdx.x; b < p.w.B; b += gridDim.x) {
        if (dec8_seq<kDdTile>(p.w, b).n > 0) continue;
        const size_t rows = (size_t)p.w.Hkv * p.w.rows, r0 = (size_t)b * rows;
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.w.o) + r0 * 2 * D);
        for (size_t i = threadIdx.x; i < rows * (2 * D / 8); i += threads) o[i] = make_uint4(0, 0, 0, 0);
        for (size_t i = threadIdx.x; i < 2 * rows; i += threads) p.w.lse[2 * r0 + i] = -__int_as_float(0x7f800000);
        if (dec8_per_unit(p.w))
            for (int i = threadIdx.x; i < p.w.Hkv * p.w.row_groups; i += threads)
                reinterpret_cast<int4*>(p.w.ws)[b * p.w.Hkv * p.w.row_groups + i] = make_int4(-1, 0, 0, 0);
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(kDdThreads, DdCfg<D, NT>::CTAS)
    diff_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const DiffDecodeParams p)
{
    using C = DdCfg<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __nv_bfloat16* qs = reinterpret_cast<__nv_bfloat16*>(smem + C::STAGES * C::STAGE);   // [2][COLS][QS]
    auto* sh = reinterpret_cast<DdShared<D, NT>*>(reinterpret_cast<uint8_t*>(qs) + 2 * C::Q_BYTES);
    static_assert(sizeof(DdShared<D, NT>) <= 1024, "shared memory");
    const volatile int* abort_flag = &sh->abort_flag;
    const DecodeFp8Params& pw = p.w;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float NEG_INF = -__int_as_float(0x7f800000);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&sh->full[s]), 1);
            mbar_init(smem_u32(&sh->empty[s]), kDdWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sh->q_full[s]), 32);       // every lane's copies
            mbar_init(smem_u32(&sh->q_empty[s]), kDdWarps);
        }
        mbar_init(smem_u32(&sh->meet), kDdWarps);
        sh->abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what ran before has written its results
    if (threadIdx.x == 0 && !dec8_per_unit(pw)) reinterpret_cast<int4*>(pw.ws)[blockIdx.x] = make_int4(-1, 0, 0, 0);
    const int x = blockIdx.x / pw.row_groups, rg = blockIdx.x - x * pw.row_groups, row0 = rg * C::RC;
    const Dec8Line line = dec8_line<kDdTile>(pw, sh->setup, x);
    if (x >= line.X) {
        dd_write_empty<D>(p, kDdThreads);
        return;
    }
    Dec8Walk<kDdTile> w(pw, line, sh->setup, x);
    auto timed_out = [&]() {
        atomicExch(pw.status, kStatusTimeout);
        *reinterpret_cast<volatile int*>(&sh->abort_flag) = 1;
    };

    if (warp == kDdWarps) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = l2_policy_evict_first();
        const int log2_r = pw.log2_ps < 6 ? pw.log2_ps : 6;     // rows per TMA box: a page, or 64
        const int nbox = kDdTile >> log2_r;
        const int ps_mask = (1 << pw.log2_ps) - 1;
        int stage = 0, q_slot = 0;
        uint32_t filled = 0, parity = 1, q_parity = 1;
        bool ok = true;
        auto wait_lane0 = [&](uint64_t* bar, uint32_t par) {
            int r = 1;
            if (lane == 0) r = mbar_wait(smem_u32(bar), par, abort_flag, pw.timeout_ns);
            ok = __shfl_sync(0xffffffffu, r, 0) != 0;
            return ok;
        };
        while (w.more && ok) {
            // the unit's queries, a 16-byte piece at a time; rows that do not exist become 0
            if (!wait_lane0(&sh->q_empty[q_slot], q_parity)) break;
            const size_t unit_row = ((size_t)w.b * pw.Hkv + w.hk) * pw.rows;
            for (int i = lane; i < C::COLS * (D / 8); i += 32) {
                const int col = i / (D / 8), piece = i - col * (D / 8), r = row0 + col % C::RC;
                const bool real = r < pw.rows;
                const size_t src = dd_qrow(unit_row + (real ? r : 0), pw.nq, col / C::RC);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 smem_u32(qs + (q_slot * C::COLS + col) * C::QS + piece * 8)),
                             "l"(static_cast<const __nv_bfloat16*>(pw.q) + src * D + piece * 8), "r"(real ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh->q_full[q_slot]))
                         : "memory");
            if (++q_slot == 2) {
                q_slot = 0;
                q_parity ^= 1;
            }
            const int* ptab = pw.page_table + (size_t)w.b * pw.max_pages;
            int held = 0, pg = 0;                                // 32 boxes' pages from box `held` on
            for (int k = w.k0; k < w.k1 && ok; ++k) {
                const int key0 = (w.seq.t0 + k) * kDdTile, box0 = key0 >> log2_r;
                if (k == w.k0 || box0 + nbox - held > 32) {
                    held = box0;
                    const long long key = (long long)(box0 + lane) << log2_r;
                    const int pi = (int)min(key >> pw.log2_ps, (long long)pw.max_pages - 1);
                    pg = min(max(dec8_ld(ptab + pi), 0), pw.num_pages - 1);
                }
                if (!wait_lane0(&sh->empty[stage], parity)) break;
                const uint32_t fb = smem_u32(&sh->full[stage]);
                const bool issue = ++filled != pw.withhold;      // test hook: never arrives
                if (lane == 0 && issue) mbar_arrive_expect_tx(fb, C::STAGE);
                __syncwarp();
                // 4 parts (K_1, K_2, V's halves) x D / 64 column boxes x nbox row boxes: 32 lanes at most
                const int box = lane & (nbox - 1), rest = lane / nbox;
                const int pg_box = __shfl_sync(0xffffffffu, pg, box0 - held + box);
                if (rest < 4 * (D / 64) && issue) {
                    const int part = rest / (D / 64), c = rest - part * (D / 64);
                    const uint32_t dst = smem_u32(smem + stage * C::STAGE) + part * C::PART + c * C::CB +
                                         (box << log2_r) * 128;
                    tma_load_3d(dst, part < 2 ? &tmK : &tmV, fb, c * 64, (key0 + (box << log2_r)) & ps_mask,
                                (pg_box * pw.Hkv + w.hk) * 2 + (part & 1), pol);
                }
                if (++stage == C::STAGES) {
                    stage = 0;
                    parity ^= 1;
                }
            }
            if (ok) w.next(pw);
        }
        if (!ok && lane == 0) timed_out();
        // every copy issued lands before shared memory is released
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (lane == 0)
            for (uint32_t k = filled < C::STAGES ? 0 : filled - C::STAGES; k < filled; ++k)
                if (k + 1 != pw.withhold)
                    mbar_wait(smem_u32(&sh->full[k % C::STAGES]), (k / C::STAGES) & 1, nullptr, kCleanupTimeoutNs);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ consumers
        const int g = lane >> 2, t = lane & 3;
        int stage = 0, q_slot = 0;
        uint32_t parity = 0, q_parity = 0, meet_parity = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t* bar, uint32_t par) {
            const bool r = mbar_wait(smem_u32(bar), par, abort_flag, pw.timeout_ns);
            ok = __all_sync(0xffffffffu, r);
            return ok;
        };
        auto meet = [&]() {     // all consumer warps, bounded
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->meet));
            const bool r = wait_all(&sh->meet, meet_parity);
            meet_parity ^= 1;
            return r;
        };
        // Fragments of 16 keys by 16 columns, column block i of part `part`: K's as stored, V's transposed.
        const int k_row = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), k_ch = lane >> 4;
        const int v_row = warp * 16 + (lane >> 4) * 8 + (lane & 7), v_ch = (lane >> 3) & 1;
        auto frag_at = [&](uint32_t base, int part, int i, int row, int ch) {
            return base + part * C::PART + (i / 4) * C::CB + row * 128 + ((((i % 4) * 2 + ch) ^ (row & 7)) << 4);
        };
        while (w.more) {
            const size_t unit_row = ((size_t)w.b * pw.Hkv + w.hk) * pw.rows + row0;
            if (!wait_all(&sh->q_full[q_slot], q_parity)) break;
            // queries as B fragments; with one product for both maps, [0] is (q_1 | 0) and [1] (0 | q_2)
            constexpr int QT = NT == 1 ? 2 : NT;
            uint32_t qf[QT][D / 16][2];
#pragma unroll
            for (int nt = 0; nt < QT; ++nt) {
                const int col = NT == 1 ? g : nt * 8 + g;
                const uint32_t* row = reinterpret_cast<const uint32_t*>(qs + (q_slot * C::COLS + col) * C::QS);
                const bool mine = NT > 1 || (g >= 4) == (nt == 1);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qf[nt][ks][0] = mine ? row[ks * 8 + t] : 0u;
                    qf[nt][ks][1] = mine ? row[ks * 8 + 4 + t] : 0u;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->q_empty[q_slot]));
            if (++q_slot == 2) {
                q_slot = 0;
                q_parity ^= 1;
            }
            float acc[NT][2 * D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 2 * D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.0f;
                m[nt][0] = m[nt][1] = NEG_INF;
                l[nt][0] = l[nt][1] = 0.0f;
            }
            for (int k = w.k0; k < w.k1; ++k) {
                const int key0 = (w.seq.t0 + k) * kDdTile + warp * 16;
                if (!wait_all(&sh->full[stage], parity)) break;
                // this warp's keys: some row sees one of them; not all rows see all of them
                const bool any = key0 < w.seq.L && key0 + 15 >= w.seq.lo;
                const bool edge = key0 + 15 > w.seq.L - pw.nq || (pw.window > 0 && key0 < w.seq.L - 1 - pw.window);
                const uint32_t base = smem_u32(smem + stage * C::STAGE);
                if (any) {
                    float xs[NT][4];
                    {
                        float s[NT][2][4];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[nt][0][e] = s[nt][1][e] = 0.0f;
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                            for (int mp = 0; mp < 2; ++mp) {
                                uint32_t a[4];
                                dd_ldmatrix<false>(a, frag_at(base, mp, ks, k_row, k_ch));
                                if constexpr (NT == 1) {
                                    dd_mma(s[0][mp], a, qf[mp][ks][0], qf[mp][ks][1]);
                                } else {
#pragma unroll
                                    for (int j = 0; j < NT / 2; ++j) {
                                        const int nt = mp * (NT / 2) + j;
                                        dd_mma(s[nt][ks & 1], a, qf[nt][ks][0], qf[nt][ks][1]);
                                    }
                                }
                            }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                // one product for both maps: the other map's sums in this column are 0 times its keys, NaN
                                // where one is not finite
                                if constexpr (NT == 1) xs[nt][e] = (t >= 2 ? s[0][1][e] : s[0][0][e]) * pw.c_log2;
                                else xs[nt][e] = (s[nt][0][e] + s[nt][1][e]) * pw.c_log2;
                            }
                    }
                    if (edge) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = key0 + g + (e & 2) * 4;
                                const int r = row0 + (nt * 8 + 2 * t + (e & 1)) % C::RC;
                                const int last = w.seq.L - pw.nq + r % pw.nq;
                                if (key > last || (pw.window > 0 && key < last - pw.window)) xs[nt][e] = NEG_INF;
                            }
                    }
                    bool raise = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) raise |= fmaxf(xs[nt][e], xs[nt][e + 2]) > m[nt][e] + kDdTau;
                    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float al[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float mx = fmaxf(xs[nt][e], xs[nt][e + 2]);
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                                mx = fmaxf(mx, m[nt][e]);
                                al[e] = mx == NEG_INF ? 1.0f : ex2(m[nt][e] - mx);
                                m[nt][e] = mx;
                                l[nt][e] *= al[e];
                            }
#pragma unroll
                            for (int i = 0; i < 2 * D / 16; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[nt][i][e] *= al[e & 1];
                        }
                    }
                    uint32_t pb[NT][2], pl[NT][2];                 // the weights in bf16, and what that leaves
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float wt[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float mm = m[nt][e & 1];
                            wt[e] = ex2(xs[nt][e] - (mm == NEG_INF ? 0.0f : mm));
                        }
                        l[nt][0] += wt[0] + wt[2];
                        l[nt][1] += wt[1] + wt[3];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t hi = pack_bf16x2(wt[2 * h], wt[2 * h + 1]);
                            pb[nt][h] = dd_transpose(hi);
                            pl[nt][h] = dd_transpose(pack_bf16x2(wt[2 * h] - __uint_as_float(hi << 16),
                                                                 wt[2 * h + 1] - __uint_as_float(hi & 0xFFFF0000u)));
                        }
                    }
                    // ---- O^T += V^T P^T, this lane's keys 2t, 2t+1 and 2t+8, 2t+9 of 16
                    if (!edge) {
#pragma unroll
                        for (int i = 0; i < 2 * D / 16; ++i) {
                            uint32_t a[4];
                            dd_ldmatrix<true>(a, frag_at(base, 2 + i / (D / 16), i % (D / 16), v_row, v_ch));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                dd_mma(acc[nt][i], a, pb[nt][0], pb[nt][1]);
                                dd_mma(acc[nt][i], a, pl[nt][0], pl[nt][1]);
                            }
                        }
                    } else {
                        uint32_t live[2], seen[NT][2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = key0 + 2 * t + 8 * h;
                            auto in = [&](int j) { return j < w.seq.L && j >= w.seq.lo; };
                            live[h] = (in(key) ? 0xFFFFu : 0u) | (in(key + 1) ? 0xFFFF0000u : 0u);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                seen[nt][h] = dd_transpose(pack_bf16x2(xs[nt][2 * h] == NEG_INF ? 0.0f : 1.0f,
                                                                       xs[nt][2 * h + 1] == NEG_INF ? 0.0f : 1.0f));
#pragma unroll
                        for (int i = 0; i < 2 * D / 16; ++i) {
                            uint32_t a[4], odd[4];
                            dd_ldmatrix<true>(a, frag_at(base, 2 + i / (D / 16), i % (D / 16), v_row, v_ch));
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                a[e] &= live[e >> 1];
                                odd[e] = dd_nonfinite(a[e]);
                                a[e] &= ~odd[e];
                                odd[e] &= 0x3F803F80u;                       // 1 where it was not finite
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                dd_mma(acc[nt][i], a, pb[nt][0], pb[nt][1]);
                                dd_mma(acc[nt][i], a, pl[nt][0], pl[nt][1]);
                            }
                            if (__any_sync(0xffffffffu, (odd[0] | odd[1] | odd[2] | odd[3]) != 0)) {
                                // keep_nan: O becomes NaN where a row sees such a value
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                    dd_mma(hit, odd, seen[nt][0], seen[nt][1]);
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (hit[e] > 0.0f) acc[nt][i][e] = __int_as_float(0x7fc00000);
                                }
                            }
                        }
                    }
                }
                if (k == w.k1 - 1) break;                          // the last stage is kept for the joining
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh->empty[stage]));
                if (++stage == C::STAGES) {
                    stage = 0;
                    parity ^= 1;
                }
            }
            if (!ok) break;

            // ---- join the four warps, eight columns at a time, in the last tile's stage.  Column c's float v
            // of warp x lies at (8 x + c) 2D + (v ^ (c / 2) 8): no bank twice.
            const bool whole = w.whole();
            float* part = dec8_my_part<C::COLS, 2 * D>(pw, w.k0 == 0);
            float* area = reinterpret_cast<float*>(smem + stage * C::STAGE);
            constexpr int VEC = 2 * D / 4;                         // float4s of a row
            auto publish = [&](int nt) {
#pragma unroll
                for (int i = 0; i < 2 * D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        area[(warp * 8 + 2 * t + (e & 1)) * (2 * D) + ((16 * i + g + (e & 2) * 4) ^ (t << 3))] =
                            acc[nt][i][e];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float sum = l[nt][h];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (g == 0) {
                        sh->m[warp][2 * t + h] = m[nt][h];
                        sh->l[warp][2 * t + h] = sum;
                    }
                }
            };
            auto joined = [&](int c, int v4, float& M, float& sum) -> float4 {
                M = fmaxf(fmaxf(sh->m[0][c], sh->m[1][c]), fmaxf(sh->m[2][c], sh->m[3][c]));
                const float mb = M == NEG_INF ? 0.0f : M;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                sum = 0.0f;
#pragma unroll
                for (int x = 0; x < kDdWarps; ++x) {
                    const float fac = ex2(sh->m[x][c] - mb);        // ex2(-inf) = 0
                    const float4 u = *reinterpret_cast<const float4*>(area + (x * 8 + c) * (2 * D) +
                                                                      ((v4 ^ ((c >> 1) << 1)) * 4));
                    sum = fmaf(sh->l[x][c], fac, sum);
                    v.x = fmaf(u.x, fac, v.x), v.y = fmaf(u.y, fac, v.y);
                    v.z = fmaf(u.z, fac, v.z), v.w = fmaf(u.w, fac, v.w);
                }
                return v;
            };
            // column `col` of the CTA's: its part, or (both maps of row r known) the output
            auto keep = [&](int col, int v4, float4 v, float M, float sum) {
                *reinterpret_cast<float4*>(part + col * (2 * D) + v4 * 4) = v;
                if (v4 == 0) {
                    part[C::COLS * 2 * D + col] = M;
                    part[C::COLS * 2 * D + C::COLS + col] = sum;
                }
            };
            auto finish = [&](int r, int v4, float4 a, float m1, float l1, float4 b, float m2, float l2) {
                const size_t row = unit_row + r;
                reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(pw.o) + row * (2 * D))[v4] =
                    dd_out(a, l1, b, l2, dd_lam(p, row));
                if (v4 == 0) {
                    pw.lse[dd_qrow(row, pw.nq, 0)] = dd_lse(m1, l1);
                    pw.lse[dd_qrow(row, pw.nq, 1)] = dd_lse(m2, l2);
                }
            };
            if constexpr (NT == 1) {
                if (!meet()) break;                                // the tile has been read
                publish(0);
                if (!meet()) break;
                for (int idx = threadIdx.x; idx < 4 * VEC; idx += kDdWarps * 32) {
                    const int r = idx / VEC, v4 = idx - r * VEC;
                    if (row0 + r >= pw.rows) break;
                    float m1, l1, m2, l2;
                    const float4 a = joined(r, v4, m1, l1), b = joined(4 + r, v4, m2, l2);
                    if (whole) {
                        finish(r, v4, a, m1, l1, b, m2, l2);
                    } else {
                        keep(r, v4, a, m1, l1);
                        keep(4 + r, v4, b, m2, l2);
                    }
                }
            } else {
                constexpr int PER = 8 * VEC / (kDdWarps * 32);     // a thread's float4s of eight rows
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    float4 a[PER];
                    float m1[PER], l1[PER];
                    if (!meet()) break;
                    publish(j);
                    if (!meet()) break;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int idx = threadIdx.x + i * kDdWarps * 32, c = idx / VEC;
                        a[i] = joined(c, idx - c * VEC, m1[i], l1[i]);
                    }
                    if (!meet()) break;
                    publish(NT / 2 + j);
                    if (!meet()) break;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int idx = threadIdx.x + i * kDdWarps * 32, c = idx / VEC, v4 = idx - c * VEC;
                        float m2, l2;
                        const float4 b = joined(c, v4, m2, l2);
                        if (row0 + j * 8 + c >= pw.rows) continue;
                        if (whole) {
                            finish(j * 8 + c, v4, a[i], m1[i], l1[i], b, m2, l2);
                        } else {
                            keep(j * 8 + c, v4, a[i], m1[i], l1[i]);
                            keep(C::RC + j * 8 + c, v4, b, m2, l2);
                        }
                    }
                }
            }
            if (!ok) break;
            fence_proxy_async_smem();                              // TMA writes the stage next
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->empty[stage]));
            if (++stage == C::STAGES) {
                stage = 0;
                parity ^= 1;
            }
            if (threadIdx.x == 0)
                dec8_name_parts(pw, w, line, x, rg, (size_t)w.b * pw.Hkv + w.hk);
            w.next(pw);
        }
        if (!ok) timed_out();
        else dd_write_empty<D>(p, kDdWarps * 32);
    }
}

// Joins the parts of a unit that several ranges shared and subtracts the maps.  grid.x: the units, or
// where there are more of them the CTAs (each leaves at most one unit to its successors); grid.y shares a
// unit's rows and columns.  Up to eight parts, the usual batch: a thread joins a float4 of both maps from
// all of them, with their loads in flight together.  More, one long sequence: sixteen threads take every
// sixteenth part, then one adds them up in order.
constexpr int kDdJoinThreads = 128, kDdFew = 8;

struct DdSum {
    float m, l;
    float4 v;

    __device__ __forceinline__ DdSum() : m(-INFINITY), l(0.0f), v(make_float4(0.0f, 0.0f, 0.0f, 0.0f)) {}

    // Adds kParts parts (m, l, v) at once; absent ones have m = -inf and zeros.
    template <int kParts>
    __device__ __forceinline__ void add(const float (&pm)[kParts], const float (&pl)[kParts], const float4 (&pv)[kParts])
    {
        float top = m;
#pragma unroll
        for (int k = 0; k < kParts; ++k) top = fmaxf(top, pm[k]);
        const float mb = top == -__int_as_float(0x7f800000) ? 0.0f : top, f = ex2(m - mb);
        m = top;
        l *= f;
        v.x *= f, v.y *= f, v.z *= f, v.w *= f;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            const float fac = ex2(pm[k] - mb);
            l = fmaf(fac, pl[k], l);
            v.x = fmaf(fac, pv[k].x, v.x), v.y = fmaf(fac, pv[k].y, v.y);
            v.z = fmaf(fac, pv[k].z, v.z), v.w = fmaf(fac, pv[k].w, v.w);
        }
    }
};

template <int D, int COLS>
__global__ void __launch_bounds__(kDdJoinThreads) diff_decode_join_kernel(const DiffDecodeParams p)
{
    constexpr int RC = COLS / 2, PART = dec8_part(COLS, 2 * D), SLICES = 2 * D / 32, VEC = 2 * D / 4;
    constexpr int VECS = 8, GROUPS = kDdJoinThreads / VECS, FLY = 5;
    __shared__ float4 sm_v[2][GROUPS][VECS];
    __shared__ float2 sm_ml[2][GROUPS];
    const DecodeFp8Params& pw = p.w;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int tid = threadIdx.x, ctas = pw.ranges * pw.row_groups, grp = tid / VECS, vec = tid % VECS;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 todo = reinterpret_cast<const int4*>(pw.ws)[blockIdx.x];
    const int x0 = todo.x, x1 = min(todo.y, pw.ranges - 1), rg = todo.z;
    // a main grid that gave up on a wait leaves entries unwritten: whatever they hold, stay inside
    if (x0 < 0 || rg < 0 || rg >= pw.row_groups || todo.w < 0 || todo.w >= (long long)pw.B * pw.Hkv) return;
    const int rows = min(RC, pw.rows - rg * RC);
    const size_t row0 = (size_t)todo.w * pw.rows + rg * RC;
    // up to kParts parts x, x + step, ... of row r's map mp and float4 v4
    auto gather = [&](auto parts_tag, int x, int step, int r, int v4, DdSum (&sum)[2]) {
        constexpr int kParts = decltype(parts_tag)::value;
        float m[2][kParts], l[2][kParts];
        float4 v[2][kParts];
#pragma unroll
        for (int k = 0; k < kParts; ++k)
#pragma unroll
            for (int mp = 0; mp < 2; ++mp) {
                m[mp][k] = NEG_INF;
                l[mp][k] = 0.0f;
                v[mp][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                const int at = x + k * step, col = mp * RC + r;
                if (at > x1) continue;
                const float* w = pw.ws + 4 * ctas + (size_t)(2 * (at * pw.row_groups + rg) + (at == x0 ? 1 : 0)) * PART;
                m[mp][k] = w[COLS * 2 * D + col];
                l[mp][k] = w[COLS * 2 * D + COLS + col];
                v[mp][k] = *reinterpret_cast<const float4*>(w + col * (2 * D) + v4 * 4);
            }
        sum[0].add(m[0], l[0], v[0]);
        sum[1].add(m[1], l[1], v[1]);
    };
    auto finish = [&](int r, int v4, const DdSum (&sum)[2]) {
        const size_t row = row0 + r;
        reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(pw.o) + row * (2 * D))[v4] =
            dd_out(sum[0].v, sum[0].l, sum[1].v, sum[1].l, dd_lam(p, row));
        if (v4 == 0) {
            pw.lse[dd_qrow(row, pw.nq, 0)] = dd_lse(sum[0].m, sum[0].l);
            pw.lse[dd_qrow(row, pw.nq, 1)] = dd_lse(sum[1].m, sum[1].l);
        }
    };
    if (x1 - x0 < kDdFew) {
        for (int i = blockIdx.y * kDdJoinThreads + tid; i < rows * VEC; i += gridDim.y * kDdJoinThreads) {
            DdSum sum[2];
            const int r = i / VEC;
            gather(std::integral_constant<int, kDdFew>{}, x0, 1, r, i - r * VEC, sum);
            finish(r, i - r * VEC, sum);
        }
        return;
    }
    for (int item = blockIdx.y; item < rows * SLICES; item += gridDim.y) {
        const int r = item / SLICES, v4 = (item - r * SLICES) * VECS + vec;
        DdSum sum[2];
        for (int x = x0 + grp; x <= x1; x += FLY * GROUPS)
            gather(std::integral_constant<int, FLY>{}, x, GROUPS, r, v4, sum);
#pragma unroll
        for (int mp = 0; mp < 2; ++mp) {
            sm_v[mp][grp][vec] = sum[mp].v;
            if (vec == 0) sm_ml[mp][grp] = make_float2(sum[mp].m, sum[mp].l);
        }
        __syncthreads();
        if (tid < VECS) {
            DdSum all[2];
#pragma unroll
            for (int mp = 0; mp < 2; ++mp) {
                float m[GROUPS], l[GROUPS];
                float4 v[GROUPS];
#pragma unroll
                for (int k = 0; k < GROUPS; ++k) {
                    m[k] = sm_ml[mp][k].x, l[k] = sm_ml[mp][k].y;
                    v[k] = sm_v[mp][k][tid];
                }
                all[mp].add(m, l, v);
            }
            finish(r, v4, all);
        }
        __syncthreads();
    }
}

template <int D, int NT>
static cudaError_t launch_diff_decode_n(const CUtensorMap& mk, const CUtensorMap& mv, const DiffDecodeParams& p,
                                        cudaStream_t stream)
{
    using C = DdCfg<D, NT>;
    auto kernel = diff_decode_kernel<D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(p.w.ranges * p.w.row_groups);
    cfg.blockDim = dim3(kDdThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, mk, mv, p)) != cudaSuccess) return e;
    if (p.w.whole) return cudaSuccess;
    const long long units = (long long)p.w.B * p.w.Hkv * p.w.row_groups, ctas = (long long)p.w.ranges * p.w.row_groups;
    // a unit's float4s over its CTAs, and four CTAs a part of the average unit while that is more, up to one
    // for 32 columns of a row
    const int rows = p.w.rows < C::RC ? p.w.rows : C::RC, items = rows * (2 * D / 32);
    const int least = (rows * (2 * D / 4) + kDdJoinThreads - 1) / kDdJoinThreads;
    long long share = units < ctas ? 4 * ctas / units : least;
    share = share > items ? items : share < least ? least : share;
    cfg.gridDim = dim3((unsigned)(units < ctas ? units : ctas), (unsigned)share);
    cfg.blockDim = dim3(kDdJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, diff_decode_join_kernel<D, C::COLS>, p);
}

cudaError_t launch_diff_decode(const CUtensorMap& mk, const CUtensorMap& mv, const DiffDecodeParams& p, int d,
                               int cta_rows, cudaStream_t stream)
{
    if (d == 64) {
        if (cta_rows == 4) return launch_diff_decode_n<64, 1>(mk, mv, p, stream);
        if (cta_rows == 8) return launch_diff_decode_n<64, 2>(mk, mv, p, stream);
        return launch_diff_decode_n<64, 4>(mk, mv, p, stream);
    }
    if (cta_rows == 4) return launch_diff_decode_n<128, 1>(mk, mv, p, stream);
    return launch_diff_decode_n<128, 2>(mk, mv, p, stream);
}

}  // namespace gb300
