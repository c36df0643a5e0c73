// decode_fp8.cu -- one decoding step of attention over a paged cache of 8-bit codes with one
// scale per block of tokens and head, query heads sharing key heads.
//
// "大模型加速-核心网络算子-Flash Attention V3" §3 总结 (decoding over cached K and V) and §1.5
// (E4M3, E5M2); "Warp Group Cluster 优化：Flash Attention V3 在 H100 上的 FP8 融合计算实践",
// 局限性与后续方向 item 2 (PagedAttention) and §3 (a scale per block).
//
// Row r = g * nq + i of key head hk is query i of head hk * G + g, at position L - nq + i;
// it sees keys max(0, position - window) .. position (window 0: all of them).  With key
// scales ks and value scales vs = f 2^e (1 <= f < 2), in log2 units:
//   s_j = c ks_j (q . k8_j),   w_j = 2^(s_j + e_j - M),   M = running max of s_j + e_j, less 6,
//   l = sum w_j 2^-e_j,   a = sum (w_j f_j) v8_j,   O = a / l,   LSE = ln2 (M + log2 l).
// Taking the maximum over what a key adds to O, not over its score alone, keeps the fp16
// weights w f below 2^15 whatever the blocks' scales are; the 6 keeps those of light keys above
// fp16's smallest step (kD8Room).
//
// This kernel takes up to 16 query rows per key head (8 at d = 256) in one pass over the
// cache, and more in several; decode_fp8_wide.cu takes many rows of a large step.  HBM-bound:
// a byte of the cache is used by 2 * rows FLOP and half a conversion.  The design is about
// keeping the loads in flight and the work even:
//   * The work is cut into equal ranges, one per resident CTA (decode_fp8.cuh).  Up to 8 rows
//     three CTAs fit an SM (two: 85.5 for 84.7 us at B16 H16 L8192 d128, 36.3 for 35.3 on
//     a ragged batch of 48).
//   * Warp 4 walks the range ahead of the others: TMA boxes (one per page or 64 rows) into a
//     ring of stages, the blocks' scales beside them by cp.async on the same barrier, and the
//     next head's queries as product fragments.
//   * Warps 0-3 take 16 keys of each tile (32 at d = 64, where 16 are too little work per
//     barrier: 29.4 for 25.6 us, 8 rows, 16 x 8 heads x 8192 keys).  The codes are exact in
//     fp16 and a query row scaled by a power of two is too, so S^T = K Q^T and O^T += V^T P^T
//     run as mma.m16n8k16 fp16 with fp32 sums: 16 keys (or 16 values of d) by 8 query rows,
//     operands straight from registers.  A tcgen05 tile would be at least 64 rows high and
//     want converted tiles in shared memory; up to 16 rows that costs more than it saves
//     (53.8 here, 63.8 us there at 16 rows, d 128).
//   * The order of d inside a product is free, so a lane takes 16 consecutive bytes of a row
//     (no bank conflicts under TMA's swizzle) and uses them as four k-steps; for V, byte
//     permutes pair two keys before the conversion.
// Keys a row does not see get the weight 0; value rows outside every row's range are zeroed
// before the product, and a NaN value at a key that only some rows see is replaced by 0
// there and added back as NaN to the rows that do (keep_nan), so what stale rows and pages
// hold never reaches O.
//
// Measured: B16 H16 L8192 d128, one new token: 84.5 us = 6.35 TB/s, 93 % of the measured copy
// rate; what is left is the start (lengths, table, first boxes: the first tile is there after 4
// us) and the spread of the CTAs' ends (equal ranges end within 13 us of each other: HBM does
// not serve all SMs alike).  48 sequences of 37 to 9000 keys, 32 over 8 heads: 32.6 us = 5.2
// TB/s; beside the same start, 1 us to join a CTA's warps and 2-3 us for the joining launch.
// The common path is 264 instructions per warp and 16 keys (with masks and NaN handling inside
// it 485, and 109.5 us for the first case), which keeps the issue slots 43 % busy.
#include "decode_fp8.cuh"

namespace gb300 {

constexpr int kD8Warps = 4;            // consumer warps
constexpr int kD8Threads = (kD8Warps + 1) * 32;

template <int D, int NT>
struct Dec8Cfg {
    static constexpr int ROWS = 8 * NT;                   // query rows of a CTA
    static constexpr int CB = D < 128 ? D : 128;          // bytes of a row in one TMA box
    static constexpr int NCB = D / CB;                    // column boxes of a row
    static constexpr int G = D == 64 ? 2 : 1;             // 16-key groups of a warp in a tile
    static constexpr int TILE = 64 * G;                   // keys of a tile
    static constexpr int HALF = TILE * D;                 // K or V of a tile
    static constexpr int STAGE = 2 * HALF;
    static constexpr bool Q_REGS = NT * D <= 128;         // query fragments held in registers
    static constexpr int Q_FRAGS = NT * (D / 16) * 32;    // 8 bytes each, two heads' worth
    static constexpr int CTAS = NT == 1 && D <= 128 ? 3 : 2;   // per SM
    static constexpr int CAP = (CTAS == 3 ? 74 : 112) * 1024;
    static constexpr int FIXED = 1024 + 2 * Q_FRAGS * 8 + 2048;   // 1024: alignment
    static constexpr int FIT = (CAP - FIXED) / STAGE;
    static constexpr int STAGES = FIT < 8 ? FIT : 8;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static_assert(STAGES >= 2, "ring");
    static_assert(STAGE >= kD8Warps * 8 * D * 4, "a head's last stage holds the warps' O for joining");
};

template <int D, int NT>
struct alignas(16) Dec8Shared {
    using C = Dec8Cfg<D, NT>;
    uint64_t full[C::STAGES], empty[C::STAGES];
    uint64_t q_full[2], q_empty[2];
    uint64_t meet;                     // the consumer warps' barrier
    float scale[C::STAGES][8 * C::G];  // K scales of the tile's 16-key parts, then V's
    float rowc[2][C::ROWS];            // per query row: softmax scale over its fragments' factor
    float m[kD8Warps][C::ROWS], l[kD8Warps][C::ROWS];
    Dec8Setup<kD8Threads> setup;
    int abort_flag;
};

__device__ __forceinline__ void dec8_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t dec8_transpose(uint32_t x)   // 8x8 of 16-bit across the warp
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, bool kE5M2, int NT>
__global__ void __launch_bounds__(kD8Threads, Dec8Cfg<D, NT>::CTAS)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const DecodeFp8Params p)
{
    using C = Dec8Cfg<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint2* qs = reinterpret_cast<uint2*>(smem + C::STAGES * C::STAGE);       // [2][Q_FRAGS]
    auto* sh = reinterpret_cast<Dec8Shared<D, NT>*>(qs + 2 * C::Q_FRAGS);
    static_assert(sizeof(Dec8Shared<D, NT>) <= 2048, "shared memory");
    const volatile int* abort_flag = &sh->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float NEG_INF = -__int_as_float(0x7f800000);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&sh->full[s]), 1 + 8 * C::G);   // lane 0's bytes, lanes' scales
            mbar_init(smem_u32(&sh->empty[s]), kD8Warps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sh->q_full[s]), 1);
            mbar_init(smem_u32(&sh->q_empty[s]), kD8Warps);
        }
        mbar_init(smem_u32(&sh->meet), kD8Warps);
        sh->abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what ran before has written its results
    if (threadIdx.x == 0 && !dec8_per_unit(p)) reinterpret_cast<int4*>(p.ws)[blockIdx.x] = make_int4(-1, 0, 0, 0);
    const int x = blockIdx.x / p.row_groups, rg = blockIdx.x - x * p.row_groups, row0 = rg * C::ROWS;
    const Dec8Line line = dec8_line<C::TILE>(p, sh->setup, x);
    if (x >= line.X) {
        dec8_write_empty<C::TILE, D>(p, kD8Threads);
        return;
    }
    Dec8Walk<C::TILE> w(p, line, sh->setup, x);

    if (warp == kD8Warps) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = l2_policy_evict_first();
        const int g = lane >> 2, t = lane & 3;
        const int log2_r = p.log2_ps < 6 ? p.log2_ps : 6;       // rows per TMA box: a page, or 64
        const int nbox = C::TILE >> log2_r;
        const int ps_mask = (1 << p.log2_ps) - 1;
        int stage = 0, q_slot = 0;
        uint32_t filled = 0, parity = 1, q_parity = 1;
        bool ok = true;
        auto wait_lane0 = [&](uint64_t* bar, uint32_t par) {
            int r = 1;
            if (lane == 0) r = mbar_wait(smem_u32(bar), par, abort_flag, p.timeout_ns);
            ok = __shfl_sync(0xffffffffu, r, 0) != 0;
            return ok;
        };
        while (w.more && ok) {
            // this head's queries: lane (g, t) holds row 8 nt + g, 16-byte pieces of its share of d
            constexpr int PER = D / 8;                           // words of a row in a lane
            uint32_t qw[NT][PER];
            const size_t unit_row = ((size_t)w.b * p.Hkv + w.hk) * p.rows + row0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < C::NCB; ++c)
#pragma unroll
                    for (int v = 0; v < C::CB / 32; ++v) {
                        const int r = nt * 8 + g, o = (c * (C::CB / 32) + v) * 4;
                        uint4 u = make_uint4(0, 0, 0, 0);
                        if (row0 + r < p.rows)
                            u = dec8_ld(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (unit_row + r) * D +
                                                                       c * C::CB + t * (C::CB / 4) + v * 8));
                        qw[nt][o] = u.x, qw[nt][o + 1] = u.y, qw[nt][o + 2] = u.z, qw[nt][o + 3] = u.w;
                    }
            const int* ptab = p.page_table + (size_t)w.b * p.max_pages;
            int held = 0, pg = 0;                                // 32 boxes' pages from box `held` on
            for (int k = w.k0; k < w.k1 && ok; ++k) {
                const int key0 = (w.seq.t0 + k) * C::TILE, box0 = key0 >> log2_r;
                if (k == w.k0 || box0 - held >= 32) {
                    held = box0;
                    const long long key = (long long)(box0 + lane) << log2_r;
                    const int pi = (int)min(key >> p.log2_ps, (long long)p.max_pages - 1);
                    pg = min(max(dec8_ld(ptab + pi), 0), p.num_pages - 1);
                }
                if (!wait_lane0(&sh->empty[stage], parity)) break;
                const uint32_t fb = smem_u32(&sh->full[stage]);
                const bool issue = ++filled != p.withhold;
                if (lane == 0 && issue) mbar_arrive_expect_tx(fb, C::STAGE);
                __syncwarp();
                const int pg_box = __shfl_sync(0xffffffffu, pg, box0 - held + (lane & (nbox - 1)));
                const int pg_part = __shfl_sync(0xffffffffu, pg, ((key0 + (lane & (4 * C::G - 1)) * 16) >> log2_r) - held);
                if (lane < 2 * nbox && issue) {
                    const bool is_v = lane >= nbox;
                    const int box = lane & (nbox - 1);
                    const uint32_t dst = smem_u32(smem + stage * C::STAGE + (is_v ? C::HALF : 0)) + (box << log2_r) * C::CB;
#pragma unroll
                    for (int c = 0; c < C::NCB; ++c)
                        tma_load_3d(dst + c * C::TILE * C::CB, is_v ? &tmV : &tmK, fb, c * C::CB,
                                    (key0 + (box << log2_r)) & ps_mask, pg_box * p.Hkv + w.hk, pol);
                }
                if (lane < 8 * C::G && issue) {
                    const int key = key0 + (lane & (4 * C::G - 1)) * 16;
                    const size_t at = (((size_t)pg_part * p.Hkv + w.hk) << (p.log2_ps - p.log2_blk)) +
                                      ((key & ps_mask) >> p.log2_blk);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n\t"
                                 "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%2];" ::"r"(
                                     smem_u32(&sh->scale[stage][lane])),
                                 "l"((lane < 4 * C::G ? p.ks : p.vs) + at), "r"(fb)
                                 : "memory");
                }
                if (++stage == C::STAGES) {
                    stage = 0;
                    parity ^= 1;
                }
                if (k > w.k0) continue;
                // fragments: a row scaled by a power of two so that its largest value is just
                // below 2^15 in fp16; what is 2^-38 of that and less is rounded
                if (!wait_lane0(&sh->q_empty[q_slot], q_parity)) break;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t big = 0;
#pragma unroll
                    for (int i = 0; i < PER; ++i) big = max(big, max((qw[nt][i] << 16) & 0x7FFF0000u, qw[nt][i] & 0x7FFF0000u));
                    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    const int ex = max((int)(big >> 23), 15) - 14;   // biased exponent of the factor's inverse
                    const float down = __int_as_float((254 - ex) << 23);
                    if (t == 0) sh->rowc[q_slot][nt * 8 + g] = __int_as_float(ex << 23) * p.c_log2;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t u = qw[nt][2 * i], v = qw[nt][2 * i + 1];
                        qs[q_slot * C::Q_FRAGS + (nt * (D / 16) + i) * 32 + lane] = make_uint2(
                            dec8_pack_half2(__uint_as_float(u << 16) * down, __uint_as_float(u & 0xFFFF0000u) * down),
                            dec8_pack_half2(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xFFFF0000u) * down));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh->q_full[q_slot]));
                if (++q_slot == 2) {
                    q_slot = 0;
                    q_parity ^= 1;
                }
            }
            if (ok) w.next(p);
        }
        if (!ok && lane == 0) dec8_timeout(p, &sh->abort_flag);
        // every copy issued lands before shared memory is released
        if (lane == 0)
            for (uint32_t k = filled < C::STAGES ? 0 : filled - C::STAGES; k < filled; ++k)
                if (k + 1 != p.withhold)
                    mbar_wait(smem_u32(&sh->full[k % C::STAGES]), (k / C::STAGES) & 1, nullptr, kCleanupTimeoutNs);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ consumers
        const int g = lane >> 2, t = lane & 3;
        int stage = 0, q_slot = 0;
        uint32_t parity = 0, q_parity = 0, meet_parity = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t* bar, uint32_t par) {
            const bool r = mbar_wait(smem_u32(bar), par, abort_flag, p.timeout_ns);
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
        while (w.more) {
            const size_t unit_row = ((size_t)w.b * p.Hkv + w.hk) * p.rows + row0;
            if (!wait_all(&sh->q_full[q_slot], q_parity)) break;
            const uint2* frag = qs + q_slot * C::Q_FRAGS + lane;
            uint2 qf[C::Q_REGS ? NT * (D / 16) : 1];
            if constexpr (C::Q_REGS) {
#pragma unroll
                for (int i = 0; i < NT * (D / 16); ++i) qf[i] = frag[i * 32];
            }
            float rowc[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) rowc[nt][h] = sh->rowc[q_slot][nt * 8 + 2 * t + h];

            float acc[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int h = 0; h < 4; ++h) acc[nt][i][h] = 0.0f;
                m[nt][0] = m[nt][1] = NEG_INF;
                l[nt][0] = l[nt][1] = 0.0f;
            }
            int v_top = 0;                                       // largest value exponent so far
            // Non-finite values of column box c at keys that only some rows see: O becomes NaN
            // where a row sees one (a product of two indicators), and the codes become 0.
            constexpr int VW = C::CB / 32;                       // words of a key in this lane
            auto keep_nan = [&](int c, uint32_t (&v)[4][VW], const float (&xs)[NT][4]) {
                constexpr uint32_t one = kE5M2 ? 0x3C : 0x38;
                uint32_t seen[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        seen[nt][h] = dec8_transpose(dec8_pack_half2(xs[nt][2 * h] == NEG_INF ? 0.0f : 1.0f,
                                                                     xs[nt][2 * h + 1] == NEG_INF ? 0.0f : 1.0f));
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    uint32_t n[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        n[k] = dec8_nonfinite<kE5M2>(v[k][i]) >> 7;
                        v[k][i] &= ~(n[k] * 0xFFu);
                        n[k] *= one;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t sel = h ? 0x7362 : 0x5140;
                        const uint32_t a = __byte_perm(n[0], n[1], sel), d = __byte_perm(n[2], n[3], sel);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            dec8_mma(hit, dec8_half2<kE5M2>(a & 0xFFFF), dec8_half2<kE5M2>(a >> 16),
                                     dec8_half2<kE5M2>(d & 0xFFFF), dec8_half2<kE5M2>(d >> 16), seen[nt][0], seen[nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (hit[e] > 0.0f) acc[nt][(c * VW + i) * 2 + h][e] = __int_as_float(0x7fc00000);
                        }
                    }
                }
            };

            for (int k = w.k0; k < w.k1; ++k) {
                const int key0 = (w.seq.t0 + k) * C::TILE + warp * 16 * C::G;
                if (!wait_all(&sh->full[stage], parity)) break;
                // this warp's keys: some row sees one of them; all rows see all of them
                const bool any = key0 < w.seq.L && key0 + 16 * C::G - 1 >= w.seq.lo;
                const bool edge = key0 + 16 * C::G - 1 > w.seq.L - p.nq ||
                                  (p.window > 0 && key0 < w.seq.L - 1 - p.window);
                const uint32_t kb = smem_u32(smem + stage * C::STAGE) + warp * 16 * C::G * C::CB, vb = kb + C::HALF;
                if (any) {
                    // ---- S^T = K Q^T: keys key0 + 16 u + g (+ 8) by rows 8 nt + 2 t (+ 1)
                    float s[C::G][NT][2][4];
                    constexpr int KW = C::CB / 16;               // k-steps (words of a lane) per column box
#pragma unroll
                    for (int u = 0; u < C::G; ++u) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[u][nt][0][e] = s[u][nt][1][e] = 0.0f;
#pragma unroll
                        for (int c = 0; c < C::NCB; ++c) {
                            uint32_t lo[KW], hi[KW];
                            const uint32_t ra = kb + c * C::TILE * C::CB + (u * 16 + g) * C::CB, rb = ra + 8 * C::CB;
#pragma unroll
                            for (int v = 0; v < KW / 4; ++v) {
                                const int ch = C::CB == 128 ? ((2 * t + v) ^ g) : (t ^ ((g >> 1) & 3));
                                const uint4 a = dec8_lds128(ra + ch * 16), d = dec8_lds128(rb + ch * 16);
                                lo[4 * v] = a.x, lo[4 * v + 1] = a.y, lo[4 * v + 2] = a.z, lo[4 * v + 3] = a.w;
                                hi[4 * v] = d.x, hi[4 * v + 1] = d.y, hi[4 * v + 2] = d.z, hi[4 * v + 3] = d.w;
                            }
#pragma unroll
                            for (int i = 0; i < KW; ++i) {
                                const uint32_t a0 = dec8_half2<kE5M2>(lo[i] & 0xFFFF), a2 = dec8_half2<kE5M2>(lo[i] >> 16);
                                const uint32_t a1 = dec8_half2<kE5M2>(hi[i] & 0xFFFF), a3 = dec8_half2<kE5M2>(hi[i] >> 16);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    const int at = nt * (D / 16) + c * KW + i;
                                    const uint2 q2 = C::Q_REGS ? qf[C::Q_REGS ? at : 0] : frag[at * 32];
                                    dec8_mma(s[u][nt][i & 1], a0, a1, a2, a3, q2.x, q2.y);
                                }
                            }
                        }
                    }
                    // ---- scales, mask, running base, weights
                    float vf[C::G], vinv[C::G], xs[C::G][NT][4];
                    bool raise = false;
#pragma unroll
                    for (int u = 0; u < C::G; ++u) {
                        float ksc = sh->scale[stage][warp * C::G + u], vsc = sh->scale[stage][(4 + warp) * C::G + u];
                        if (C::G > 1 && edge && (key0 + u * 16 >= w.seq.L || key0 + u * 16 + 15 < w.seq.lo))
                            ksc = vsc = 0.0f;                    // nobody's keys: whatever their scales are
                        const Dec8ValueScale vs(vsc, v_top);
                        vf[u] = vs.f;
                        vinv[u] = vs.inv;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float k0 = ksc * rowc[nt][0], k1 = ksc * rowc[nt][1];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                xs[u][nt][e] = fmaf(s[u][nt][0][e] + s[u][nt][1][e], (e & 1) ? k1 : k0, vs.e);
                        }
                    }
                    if (edge) {
#pragma unroll
                        for (int u = 0; u < C::G; ++u)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int key = key0 + u * 16 + g + (e & 2) * 4;
                                    const int last = w.seq.L - p.nq + (row0 + nt * 8 + 2 * t + (e & 1)) % p.nq;
                                    if (key > last || (p.window > 0 && key < last - p.window)) xs[u][nt][e] = NEG_INF;
                                }
                    }
                    float top[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            top[nt][e] = fmaxf(xs[0][nt][e], xs[0][nt][e + 2]);
#pragma unroll
                            for (int u = 1; u < C::G; ++u) top[nt][e] = fmax3(top[nt][e], xs[u][nt][e], xs[u][nt][e + 2]);
                            raise |= top[nt][e] > m[nt][e] + (kD8Room + kD8Tau);
                        }
                    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float al[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float mx = top[nt][e];
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                                mx = fmaxf(mx - kD8Room, m[nt][e]);
                                al[e] = mx == NEG_INF ? 1.0f : ex2(m[nt][e] - mx);
                                m[nt][e] = mx;
                                l[nt][e] *= al[e];
                            }
#pragma unroll
                            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[nt][i][e] *= al[e & 1];
                        }
                    }
                    uint32_t pb[C::G][NT][2];
#pragma unroll
                    for (int u = 0; u < C::G; ++u)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float wt[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float mm = m[nt][e & 1];
                                wt[e] = ex2(xs[u][nt][e] - (mm == NEG_INF ? 0.0f : mm));
                            }
                            l[nt][0] = fmaf(wt[0] + wt[2], vinv[u], l[nt][0]);
                            l[nt][1] = fmaf(wt[1] + wt[3], vinv[u], l[nt][1]);
                            pb[u][nt][0] = dec8_transpose(dec8_pack_half2(wt[0] * vf[u], wt[1] * vf[u]));
                            pb[u][nt][1] = dec8_transpose(dec8_pack_half2(wt[2] * vf[u], wt[3] * vf[u]));
                        }
                    // ---- O^T += V^T P^T: this lane's keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
                    for (int uc = 0; uc < C::G * C::NCB; ++uc) {
                        const int u = uc / C::NCB, c = uc % C::NCB;
                        uint32_t v[4][VW];
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            const int kr = 2 * t + (k4 & 1) + (k4 & 2) * 4;
                            const uint32_t ra = vb + c * C::TILE * C::CB + (u * 16 + kr) * C::CB;
                            if constexpr (C::CB == 128) {
                                const uint4 r = dec8_lds128(ra + ((g ^ (kr & 7)) * 16));
                                v[k4][0] = r.x, v[k4][1] = r.y, v[k4][2] = r.z, v[k4][3] = r.w;
                            } else {
                                const uint2 r = dec8_lds64(ra + (((g >> 1) ^ ((kr >> 1) & 3)) * 16) + (g & 1) * 8);
                                v[k4][0] = r.x, v[k4][1] = r.y;
                            }
                        }
                        if (edge) {
                            uint32_t odd = 0;                    // non-finite codes among this lane's
#pragma unroll
                            for (int k4 = 0; k4 < 4; ++k4) {
                                const int key = key0 + u * 16 + 2 * t + (k4 & 1) + (k4 & 2) * 4;
                                const bool out = key >= w.seq.L || key < w.seq.lo;
#pragma unroll
                                for (int i = 0; i < VW; ++i) {
                                    v[k4][i] = out ? 0u : v[k4][i];
                                    odd |= dec8_nonfinite<kE5M2>(v[k4][i]);
                                }
                            }
                            if (__any_sync(0xffffffffu, odd != 0)) keep_nan(c, v, xs[u]);
                        }
#pragma unroll
                        for (int i = 0; i < VW; ++i) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {        // two values of d per product
                                const uint32_t sel = h ? 0x7362 : 0x5140;
                                const uint32_t a = __byte_perm(v[0][i], v[1][i], sel), d = __byte_perm(v[2][i], v[3][i], sel);
                                const uint32_t a0 = dec8_half2<kE5M2>(a & 0xFFFF), a1 = dec8_half2<kE5M2>(a >> 16);
                                const uint32_t a2 = dec8_half2<kE5M2>(d & 0xFFFF), a3 = dec8_half2<kE5M2>(d >> 16);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    dec8_mma(acc[nt][(c * VW + i) * 2 + h], a0, a1, a2, a3, pb[u][nt][0], pb[u][nt][1]);
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

            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->q_empty[q_slot]));
            if (++q_slot == 2) {
                q_slot = 0;
                q_parity ^= 1;
            }

            // ---- join the four warps, eight rows at a time, in the last tile's stage: warp w's
            // row r, float4 c at ((w * 8 + r) * D / 4 + (c ^ (r / 2 & 3))), which keeps the
            // writes below to two lanes a bank
            const bool whole = w.whole();
            float* part = dec8_my_part<C::ROWS, D>(p, w.k0 == 0);
            float4* area = reinterpret_cast<float4*>(smem + stage * C::STAGE);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (!meet()) break;                              // the tile, or the rows before, have been read
                // value d of acc[..][i][h]: group g holds CB/8 consecutive ones of a column box
                constexpr int VT = C::CB / 16;                   // products per column box
#pragma unroll
                for (int i = 0; i < D / 16; i += 2)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        area[(warp * 8 + 2 * t + h) * (D / 4) +
                             (((i / VT) * (C::CB / 4) + g * (C::CB / 32) + (i % VT) / 2) ^ t)] =
                            make_float4(acc[nt][i][h], acc[nt][i][h + 2], acc[nt][i + 1][h], acc[nt][i + 1][h + 2]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], o);
                    if (g == 0) {
                        sh->m[warp][nt * 8 + 2 * t + h] = m[nt][h];
                        sh->l[warp][nt * 8 + 2 * t + h] = l[nt][h];
                    }
                }
                if (!meet()) break;
                for (int idx = threadIdx.x; idx < 8 * (D / 4); idx += kD8Warps * 32) {
                    const int r8 = idx / (D / 4), d4 = idx - r8 * (D / 4), r = nt * 8 + r8;
                    if (row0 + r >= p.rows) break;
                    const float M = fmaxf(fmaxf(sh->m[0][r], sh->m[1][r]), fmaxf(sh->m[2][r], sh->m[3][r]));
                    const float mb = M == NEG_INF ? 0.0f : M;
                    float sum = 0.0f;
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < kD8Warps; ++w) {
                        const float fac = ex2(sh->m[w][r] - mb);     // ex2(-inf) = 0
                        const float4 u = area[(w * 8 + r8) * (D / 4) + (d4 ^ (r8 >> 1))];
                        sum = fmaf(sh->l[w][r], fac, sum);
                        v.x = fmaf(u.x, fac, v.x), v.y = fmaf(u.y, fac, v.y);
                        v.z = fmaf(u.z, fac, v.z), v.w = fmaf(u.w, fac, v.w);
                    }
                    if (whole) {
                        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (unit_row + r) * D + d4 * 4) =
                            make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                        if (d4 == 0) p.lse[unit_row + r] = dec8_lse(M, sum);
                    } else {
                        *reinterpret_cast<float4*>(part + r * D + d4 * 4) = v;
                        if (d4 == 0) {
                            part[C::ROWS * D + r] = M;
                            part[C::ROWS * D + C::ROWS + r] = sum;
                        }
                    }
                }
            }
            if (!ok) break;
            fence_proxy_async_smem();                            // TMA writes the stage next
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->empty[stage]));
            if (++stage == C::STAGES) {
                stage = 0;
                parity ^= 1;
            }
            if (threadIdx.x == 0) dec8_name_parts(p, w, line, x, rg, unit_row);
            w.next(p);
        }
        if (!ok) dec8_timeout(p, &sh->abort_flag);
        else dec8_write_empty<C::TILE, D>(p, kD8Warps * 32);
    }
}

template <int D, bool kE5M2, int NT>
static cudaError_t launch_decode_fp8_n(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeFp8Params& p,
                                       cudaStream_t stream)
{
    using C = Dec8Cfg<D, NT>;
    auto kernel = decode_fp8_kernel<D, kE5M2, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(p.ranges * p.row_groups);
    cfg.blockDim = dim3(kD8Threads);
    cfg.dynamicSmemBytes = C::SMEM;
    e = cudaLaunchKernelEx(&cfg, kernel, mk, mv, p);
    if (e != cudaSuccess) return e;
    return launch_decode_fp8_combine<D, C::ROWS>(p, cfg);
}

template <int D, bool kE5M2>
static cudaError_t launch_decode_fp8_d(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeFp8Params& p,
                                       int cta_rows, cudaStream_t stream)
{
    if constexpr (D < 256)
        if (cta_rows == 16) return launch_decode_fp8_n<D, kE5M2, 2>(mk, mv, p, stream);
    return launch_decode_fp8_n<D, kE5M2, 1>(mk, mv, p, stream);
}

cudaError_t launch_decode_fp8(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeFp8Params& p, int d,
                              bool e5m2, int cta_rows, cudaStream_t stream)
{
    switch (d) {
    case 64:
        return e5m2 ? launch_decode_fp8_d<64, true>(mk, mv, p, cta_rows, stream)
                    : launch_decode_fp8_d<64, false>(mk, mv, p, cta_rows, stream);
    case 128:
        return e5m2 ? launch_decode_fp8_d<128, true>(mk, mv, p, cta_rows, stream)
                    : launch_decode_fp8_d<128, false>(mk, mv, p, cta_rows, stream);
    case 256:
        return e5m2 ? launch_decode_fp8_d<256, true>(mk, mv, p, cta_rows, stream)
                    : launch_decode_fp8_d<256, false>(mk, mv, p, cta_rows, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gb300
