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
//   s_j = c ks_j (q . k8_j),   w_j = 2^(s_j + e_j - M),   M = running max of s_j + e_j,
//   l = sum w_j 2^-e_j,   a = sum (w_j f_j) v8_j,   O = a / l,   LSE = ln2 (M + log2 l).
// Taking the maximum over what a key adds to O, not over its score alone, keeps the fp16
// weights w f at or below a small constant whatever the blocks' scales are.
//
// HBM-bound: a byte of the cache is used by 2 * rows FLOP and half the rows' weight of a
// conversion.  The design is about keeping the loads in flight and the work even:
//   * The tiles (64 keys of one head) of all sequences form one line that is cut into equal
//     ranges, one per resident CTA (two per SM), so a ragged batch and a single long sequence
//     both keep every SM busy to the end; a range may end inside a sequence, and then its
//     part goes to the workspace and decode_fp8_combine_kernel joins the parts.  It is
//     launched as a dependent of the main grid, its set-up hidden behind it.
//   * Warp 4 walks the range ahead of the others: TMA boxes (one per page or 64 rows) into a
//     ring of stages, the blocks' scales beside them by cp.async on the same barrier.
//   * Warps 0-3 take 16 keys of each tile.  The codes are exact in fp16 and a query row
//     scaled by a power of two is too, so S^T = K Q^T and O^T += V^T P^T run as
//     mma.m16n8k16 fp16 with fp32 sums: 16 keys (or 16 values of d) by 8 query rows, which
//     wastes nothing down to 8 rows and needs no per-row padding to 128.  An m64+ tcgen05
//     tile would want its operands in one type (the queries split into two E4M3 parts) and
//     the probabilities through shared memory for a product that HBM bounds anyway.
//   * The order of d inside a product is free, so a lane takes 16 consecutive bytes of a row
//     (no bank conflicts under TMA's swizzle) and uses them as four k-steps; for V, byte
//     permutes pair two keys before the conversion.
// Keys a row does not see get the weight 0; value rows outside every row's range are zeroed
// before the product, and a NaN value at a key that only some rows see is replaced by 0
// there and added back as NaN to the rows that do (keep_nan), so what stale rows and pages
// hold never reaches O.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_params.h"
#include "paged_params.h"
#include "ptx.cuh"

namespace gb300 {

constexpr int kD8Tile = 64;            // keys of a tile, 16 per consumer warp
constexpr int kD8Warps = 4;            // consumer warps
constexpr int kD8Threads = (kD8Warps + 1) * 32;
constexpr float kD8Tau = 8.0f;         // the running maximum is raised when passed by this (log2)
constexpr int kD8CombineThreads = 256;

template <int D, int NT>
struct Dec8Cfg {
    static constexpr int ROWS = 8 * NT;                   // query rows of a CTA
    static constexpr int CB = D < 128 ? D : 128;          // bytes of a row in one TMA box
    static constexpr int NCB = D / CB;                    // column boxes of a row
    static constexpr int HALF = kD8Tile * D;              // K or V of a tile
    static constexpr int STAGE = 2 * HALF;
    static constexpr bool Q_REGS = NT * D <= 256;         // query fragments in registers
    static constexpr int Q_BYTES = Q_REGS ? 0 : NT * (D / 16) * 32 * 8;
    static constexpr int PAD = 4;
    static constexpr int MERGE = 2 * ROWS * (D + PAD) * 4;
    static constexpr int CAP = 112 * 1024;                // two CTAs per SM
    static constexpr int FIXED = 1024 + Q_BYTES + MERGE + 4096;   // alignment, barriers, statistics
    static constexpr int FIT = (CAP - FIXED) / STAGE;
    static constexpr int STAGES = FIT < 8 ? FIT : 8;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static_assert(STAGES >= 2, "ring");
};

template <int STAGES>
struct alignas(16) Dec8Shared {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t meet;                     // the consumer warps' barrier
    float scale[STAGES][8];            // K scales of the tile's four 16-key parts, then V's
    float m[kD8Warps][64], l[kD8Warps][64];
    long long sum[kD8Threads / 32];    // set-up: tiles per warp's sequences
    long long first;                   // tiles before sequence b0
    int b0;
    int abort_flag;
};

// Tiles of sequence b: [t0, t0 + n) of 64 keys, of which keys lo .. L-1 may be seen.
struct Dec8Seq {
    int L, lo, t0, n;
};

__device__ __forceinline__ Dec8Seq dec8_seq(const DecodeFp8Params& p, int b)
{
    Dec8Seq s;
    s.L = min(max(__ldg(p.seq_lens + b), 0), p.max_pages << p.log2_ps);
    s.lo = p.window > 0 ? max(0, s.L - p.nq - p.window) : 0;
    s.t0 = s.lo / kD8Tile;
    s.n = (int)(((unsigned)s.L + kD8Tile - 1) / kD8Tile) - s.t0;
    return s;
}

// Set-up of main and combine kernel: the sum of all sequences' tiles, and the tiles before
// the sequence that `pick` chooses from (tiles before it, its own).  All threads call it.
template <int kThreads, class Pick>
__device__ __forceinline__ long long dec8_scan(const DecodeFp8Params& p, long long* warp_sum, Pick pick)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += dec8_seq(p, b).n;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    long long before = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    for (int b = b0; b < b1; ++b) {
        const int n = dec8_seq(p, b).n;
        pick(b, before, n, total);
        before += n;
    }
    return total;
}

template <bool kE5M2>
__device__ __forceinline__ uint32_t dec8_half2(uint32_t two)   // codes in bits 0-15 -> f16x2, exact
{
    uint32_t h;
    if constexpr (kE5M2) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

// 0x80 in every byte of w whose code is not finite (E5M2: infinities too).
template <bool kE5M2>
__device__ __forceinline__ uint32_t dec8_nonfinite(uint32_t w)
{
    return (kE5M2 ? (w & 0x7C7C7C7Cu) + 0x04040404u : (w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

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

__device__ __forceinline__ uint32_t dec8_pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 dec8_lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 dec8_lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ void dec8_timeout(const DecodeFp8Params& p, int* abort_flag)
{
    atomicExch(p.status, kStatusTimeout);
    *reinterpret_cast<volatile int*>(abort_flag) = 1;
}

template <int D, bool kE5M2, int NT>
__global__ void __launch_bounds__(kD8Threads, 2)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const DecodeFp8Params p)
{
    using C = Dec8Cfg<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* q_smem = smem + C::STAGES * C::STAGE;
    float* merge = reinterpret_cast<float*>(q_smem + C::Q_BYTES);
    auto* sh = reinterpret_cast<Dec8Shared<C::STAGES>*>(q_smem + C::Q_BYTES + C::MERGE);
    static_assert(sizeof(Dec8Shared<C::STAGES>) <= 3072, "shared memory");
    const volatile int* abort_flag = &sh->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&sh->full[s]), 9);        // lane 0's bytes, eight lanes' scales
            mbar_init(smem_u32(&sh->empty[s]), kD8Warps);
        }
        mbar_init(smem_u32(&sh->meet), kD8Warps);
        sh->abort_flag = 0;
        fence_mbar_init();
    }
    // this CTA's range [f0, f_end) of the line of tiles (sequence, key head, tile)
    const int x = blockIdx.x / p.row_groups, rg = blockIdx.x - x * p.row_groups;
    const long long total = p.Hkv * dec8_scan<kD8Threads>(
        p, sh->sum, [&](int b, long long before, int n, long long all) {
            const long long T = all * p.Hkv, X = T < p.ranges ? T : p.ranges;
            if (x >= X) return;
            const long long f = x * T / X;
            if (n > 0 && before * p.Hkv <= f && f < (before + n) * p.Hkv) {
                sh->b0 = b;
                sh->first = before;
            }
        });
    __syncthreads();
    const long long X = total < p.ranges ? total : p.ranges;
    if (x >= X) return;
    long long f = x * total / X;
    const long long f_end = (x + 1) * total / X;
    int b = sh->b0;
    Dec8Seq seq = dec8_seq(p, b);
    const long long in_seq = f - sh->first * p.Hkv;
    int hk = (int)(in_seq / seq.n), j = (int)(in_seq - (long long)hk * seq.n);
    // to the next unit (sequence, key head) of the line
    auto next_unit = [&]() {
        j = 0;
        if (++hk == p.Hkv) {
            hk = 0;
            do seq = dec8_seq(p, ++b);
            while (seq.n == 0);
        }
    };

    if (warp == kD8Warps) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        const uint64_t pol = l2_policy_evict_first();
        const int log2_r = p.log2_ps < 6 ? p.log2_ps : 6;       // rows per TMA box: a page, or 64
        const int nbox = kD8Tile >> log2_r;
        const int ps_mask = (1 << p.log2_ps) - 1;
        int stage = 0, filled = 0;
        uint32_t parity = 1;
        bool ok = true;
        while (f < f_end && ok) {
            const int part = (int)min((long long)(seq.n - j), f_end - f);
            const int* ptab = p.page_table + (size_t)b * p.max_pages;
            int held = 0, pg = 0;                                // 32 boxes' pages from box `held` on
            for (int jj = 0; jj < part && ok; ++jj) {
                const int key0 = (seq.t0 + j + jj) * kD8Tile, box0 = key0 >> log2_r;
                if (jj == 0 || box0 - held >= 32) {
                    held = box0;
                    const long long key = (long long)(box0 + lane) << log2_r;
                    const int pi = (int)min(key >> p.log2_ps, (long long)p.max_pages - 1);
                    pg = min(max(__ldg(ptab + pi), 0), p.num_pages - 1);
                }
                int r = 1;
                if (lane == 0) r = mbar_wait(smem_u32(&sh->empty[stage]), parity, abort_flag, p.timeout_ns);
                ok = __shfl_sync(0xffffffffu, r, 0) != 0;
                if (!ok) break;
                const uint32_t fb = smem_u32(&sh->full[stage]);
                if (lane == 0) mbar_arrive_expect_tx(fb, C::STAGE);
                __syncwarp();
                const int pg_box = __shfl_sync(0xffffffffu, pg, box0 - held + (lane & (nbox - 1)));
                const int pg_part = __shfl_sync(0xffffffffu, pg, ((key0 + (lane & 3) * 16) >> log2_r) - held);
                if (lane < 2 * nbox) {
                    const bool is_v = lane >= nbox;
                    const int box = lane & (nbox - 1);
                    const uint32_t dst = smem_u32(smem + stage * C::STAGE + (is_v ? C::HALF : 0)) + (box << log2_r) * C::CB;
#pragma unroll
                    for (int c = 0; c < C::NCB; ++c)
                        tma_load_3d(dst + c * kD8Tile * C::CB, is_v ? &tmV : &tmK, fb, c * C::CB,
                                    (key0 + (box << log2_r)) & ps_mask, pg_box * p.Hkv + hk, pol);
                }
                if (lane < 8) {
                    const int key = key0 + (lane & 3) * 16;
                    const size_t at = (((size_t)pg_part * p.Hkv + hk) << (p.log2_ps - p.log2_blk)) +
                                      ((key & ps_mask) >> p.log2_blk);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n\t"
                                 "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%2];" ::"r"(
                                     smem_u32(&sh->scale[stage][lane])),
                                 "l"((lane < 4 ? p.ks : p.vs) + at), "r"(fb)
                                 : "memory");
                }
                ++filled;
                if (++stage == C::STAGES) {
                    stage = 0;
                    parity ^= 1;
                }
            }
            f += part;
            if (ok && f < f_end) next_unit();
        }
        if (!ok && lane == 0) dec8_timeout(p, &sh->abort_flag);
        // every copy issued lands before shared memory is released
        if (lane == 0)
            for (int k = filled < C::STAGES ? 0 : filled - C::STAGES; k < filled; ++k)
                mbar_wait(smem_u32(&sh->full[k % C::STAGES]), (k / C::STAGES) & 1, nullptr, kCleanupTimeoutNs);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ consumers
        const int g = lane >> 2, t = lane & 3;
        const float NEG_INF = -__int_as_float(0x7f800000);
        const int row0 = rg * C::ROWS;
        int stage = 0;
        uint32_t parity = 0, meet_parity = 0;
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
        while (f < f_end && ok) {
            const int part = (int)min((long long)(seq.n - j), f_end - f);
            const size_t unit_row = ((size_t)b * p.Hkv + hk) * p.rows + row0;

            // query fragments: row 8 nt + g, scaled by a power of two so that its largest
            // value is just below 2^15; what is 2^-38 of that and less rounds in fp16
            uint2 qf[C::Q_REGS ? NT : 1][C::Q_REGS ? D / 16 : 1];
            float rowc[NT][2];
            uint2* qs = reinterpret_cast<uint2*>(q_smem);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = nt * 8 + g;
                constexpr int PER = D / 4;                       // values of a lane: D/4 in NCB pieces
                uint32_t w[PER / 2];
                uint32_t big = 0;
#pragma unroll
                for (int c = 0; c < C::NCB; ++c)
#pragma unroll
                    for (int v = 0; v < C::CB / 32; ++v) {       // 8 values each
                        uint4 u = make_uint4(0, 0, 0, 0);
                        if (row0 + r < p.rows)
                            u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                                     (unit_row + r) * D + c * C::CB + t * (C::CB / 4) + v * 8));
                        const int o = (c * (C::CB / 32) + v) * 4;
                        w[o] = u.x, w[o + 1] = u.y, w[o + 2] = u.z, w[o + 3] = u.w;
                    }
#pragma unroll
                for (int i = 0; i < PER / 2; ++i) big = max(big, max((w[i] << 16) & 0x7FFF0000u, w[i] & 0x7FFF0000u));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const int e = max((int)(big >> 23), 15) - 14;    // biased exponent of the factor's inverse
                const float down = __int_as_float((254 - e) << 23), up = __int_as_float(e << 23);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t a = w[2 * i], d = w[2 * i + 1];
                    const uint2 fr = make_uint2(
                        dec8_pack_half2(__uint_as_float(a << 16) * down, __uint_as_float(a & 0xFFFF0000u) * down),
                        dec8_pack_half2(__uint_as_float(d << 16) * down, __uint_as_float(d & 0xFFFF0000u) * down));
                    if constexpr (C::Q_REGS) qf[nt][i] = fr;
                    else if (warp == (nt & 3)) qs[(nt * (D / 16) + i) * 32 + lane] = fr;
                }
                rowc[nt][0] = __shfl_sync(0xffffffffu, up, (2 * t) * 4) * p.c_log2;
                rowc[nt][1] = __shfl_sync(0xffffffffu, up, (2 * t + 1) * 4) * p.c_log2;
            }
            if constexpr (!C::Q_REGS) {
                if (!meet()) break;
            }
            float acc[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.0f;
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

            for (int jj = 0; jj < part; ++jj) {
                const int key0 = (seq.t0 + j + jj) * kD8Tile + warp * 16;
                if (!wait_all(&sh->full[stage], parity)) break;
                // this warp's keys: some row sees one of them; all rows see all of them
                const bool any = key0 < seq.L && key0 + 15 >= seq.lo;
                const bool edge = key0 + 15 > seq.L - p.nq ||
                                  (p.window > 0 && key0 < seq.L - 1 - p.window);
                const uint32_t kb = smem_u32(smem + stage * C::STAGE), vb = kb + C::HALF;
                if (any) {
                    // ---- S^T = K Q^T: keys key0 + g (+ 8) by rows 8 nt + 2 t (+ 1)
                    float s[NT][2][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[nt][0][e] = s[nt][1][e] = 0.0f;
                    constexpr int KW = C::CB / 16;               // k-steps (words of a lane) per column box
#pragma unroll
                    for (int c = 0; c < C::NCB; ++c) {
                        uint32_t lo[KW], hi[KW];
                        const uint32_t ra = kb + c * kD8Tile * C::CB + (warp * 16 + g) * C::CB, rb = ra + 8 * C::CB;
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
                                const uint2 q2 = C::Q_REGS ? qf[C::Q_REGS ? nt : 0][C::Q_REGS ? c * KW + i : 0]
                                                           : qs[(nt * (D / 16) + c * KW + i) * 32 + lane];
                                dec8_mma(s[nt][i & 1], a0, a1, a2, a3, q2.x, q2.y);
                            }
                        }
                    }
                    // ---- scales, mask, running maximum, weights
                    const float ksc = sh->scale[stage][warp], vsc = sh->scale[stage][4 + warp];
                    // vs = f 2^e with e at most 60 below the largest so far (a scale of 0 has
                    // f = 0): 2^-e stays in range and every key counts in l
                    const int ve = min(max((int)((__float_as_uint(vsc) >> 23) & 0xFF) - 127, v_top - 60), 126);
                    v_top = max(v_top, ve);
                    const float vf = vsc * __int_as_float((127 - ve) << 23), vinv = __int_as_float((127 - ve) << 23);
                    const float vef = (float)ve;
                    float xs[NT][4];
                    bool raise = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float k0 = ksc * rowc[nt][0], k1 = ksc * rowc[nt][1];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            xs[nt][e] = fmaf(s[nt][0][e] + s[nt][1][e], (e & 1) ? k1 : k0, vef);
                        }
                    }
                    if (edge) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = key0 + g + (e & 2) * 4;
                                const int last = seq.L - p.nq + (row0 + nt * 8 + 2 * t + (e & 1)) % p.nq;
                                if (key > last || (p.window > 0 && key < last - p.window)) xs[nt][e] = NEG_INF;
                            }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        raise |= fmaxf(xs[nt][0], xs[nt][2]) > m[nt][0] + kD8Tau ||
                                 fmaxf(xs[nt][1], xs[nt][3]) > m[nt][1] + kD8Tau;
                    }
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
                            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[nt][i][e] *= al[e & 1];
                        }
                    }
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float mm = m[nt][e & 1];
                            w[e] = ex2(xs[nt][e] - (mm == NEG_INF ? 0.0f : mm));
                        }
                        l[nt][0] = fmaf(w[0] + w[2], vinv, l[nt][0]);
                        l[nt][1] = fmaf(w[1] + w[3], vinv, l[nt][1]);
                        pb[nt][0] = dec8_transpose(dec8_pack_half2(w[0] * vf, w[1] * vf));
                        pb[nt][1] = dec8_transpose(dec8_pack_half2(w[2] * vf, w[3] * vf));
                    }
                    // ---- O^T += V^T P^T: this lane's keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
                    for (int c = 0; c < C::NCB; ++c) {
                        uint32_t v[4][VW];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int kr = 2 * t + (k & 1) + (k & 2) * 4;
                            const uint32_t ra = vb + c * kD8Tile * C::CB + (warp * 16 + kr) * C::CB;
                            if constexpr (C::CB == 128) {
                                const uint4 u = dec8_lds128(ra + ((g ^ (kr & 7)) * 16));
                                v[k][0] = u.x, v[k][1] = u.y, v[k][2] = u.z, v[k][3] = u.w;
                            } else {
                                const uint2 u = dec8_lds64(ra + (((g >> 1) ^ ((kr >> 1) & 3)) * 16) + (g & 1) * 8);
                                v[k][0] = u.x, v[k][1] = u.y;
                            }
                        }
                        if (edge) {
                            uint32_t odd = 0;                    // non-finite codes among this lane's
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int key = key0 + 2 * t + (k & 1) + (k & 2) * 4;
                                const bool out = key >= seq.L || key < seq.lo;
#pragma unroll
                                for (int i = 0; i < VW; ++i) {
                                    v[k][i] = out ? 0u : v[k][i];
                                    odd |= dec8_nonfinite<kE5M2>(v[k][i]);
                                }
                            }
                            if (__any_sync(0xffffffffu, odd != 0)) keep_nan(c, v, xs);
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
                                    dec8_mma(acc[nt][(c * VW + i) * 2 + h], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh->empty[stage]));
                if (++stage == C::STAGES) {
                    stage = 0;
                    parity ^= 1;
                }
            }
            if (!ok) break;

            // ---- join the four warps: statistics, then O in two steps
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], o);
                    if (g == 0) {
                        sh->m[warp][nt * 8 + 2 * t + e] = m[nt][e];
                        sh->l[warp][nt * 8 + 2 * t + e] = l[nt][e];
                    }
                }
            if (!meet()) break;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = nt * 8 + 2 * t + e;
                    const float M = fmaxf(fmaxf(sh->m[0][r], sh->m[1][r]), fmaxf(sh->m[2][r], sh->m[3][r]));
                    const float fac = ex2(m[nt][e] - (M == NEG_INF ? 0.0f : M));   // ex2(-inf) = 0
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        acc[nt][i][e] *= fac;
                        acc[nt][i][e + 2] *= fac;
                    }
                }
            // value d of acc[..][i][e]: lane group g holds CB/8 consecutive ones of a column box
            constexpr int VT = C::CB / 16;                       // products per column box
            float* area = merge + (warp & 1) * C::ROWS * (D + C::PAD);
            auto place = [&](int nt, int i, int e) {             // float4 over i, i + 1
                return area + (nt * 8 + 2 * t + e) * (D + C::PAD) + (i / VT) * C::CB + g * (C::CB / 8) + (i % VT) * 2;
            };
            if (warp >= 2) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < D / 16; i += 2)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float4*>(place(nt, i, e)) =
                                make_float4(acc[nt][i][e], acc[nt][i][e + 2], acc[nt][i + 1][e], acc[nt][i + 1][e + 2]);
            }
            if (!meet()) break;
            if (warp < 2) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < D / 16; i += 2)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float4* at = reinterpret_cast<float4*>(place(nt, i, e));
                            float4 v = *at;
                            v.x += acc[nt][i][e], v.y += acc[nt][i][e + 2];
                            v.z += acc[nt][i + 1][e], v.w += acc[nt][i + 1][e + 2];
                            *at = v;
                        }
            }
            if (!meet()) break;
            const bool whole = part == seq.n;
            const int slot = 2 * blockIdx.x + (j == 0 ? 1 : 0);
            float* ws = p.ws + (size_t)slot * C::ROWS * (D + 2);
            for (int idx = threadIdx.x; idx < C::ROWS * (D / 4); idx += kD8Warps * 32) {
                const int r = idx / (D / 4), d4 = idx - r * (D / 4);
                if (row0 + r >= p.rows) break;
                const float4 a = *reinterpret_cast<const float4*>(merge + r * (D + C::PAD) + d4 * 4);
                const float4 d = *reinterpret_cast<const float4*>(merge + (C::ROWS + r) * (D + C::PAD) + d4 * 4);
                float4 v = make_float4(a.x + d.x, a.y + d.y, a.z + d.z, a.w + d.w);
                const float M = fmaxf(fmaxf(sh->m[0][r], sh->m[1][r]), fmaxf(sh->m[2][r], sh->m[3][r]));
                const float mb = M == NEG_INF ? 0.0f : M;
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kD8Warps; ++w) sum = fmaf(sh->l[w][r], ex2(sh->m[w][r] - mb), sum);
                if (whole) {
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (unit_row + r) * D + d4 * 4) =
                        make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                    if (d4 == 0)
                        p.lse[unit_row + r] = sum == 0.0f ? NEG_INF : (mb + __log2f(sum)) * 0.69314718055994531f;
                } else {
                    *reinterpret_cast<float4*>(ws + r * D + d4 * 4) = v;
                    if (d4 == 0) {
                        ws[C::ROWS * D + r] = M;
                        ws[C::ROWS * D + C::ROWS + r] = sum;
                    }
                }
            }
            f += part;
            if (f < f_end) {
                next_unit();
                if (!meet()) break;      // the statistics and areas have been read
            }
        }
        if (!ok) dec8_timeout(p, &sh->abort_flag);
    }
}

// Joins the parts of the units that several CTAs shared, one CTA per query row: with M the
// largest part maximum, O = sum_x 2^(M_x - M) a_x / sum_x 2^(M_x - M) l_x.  Units of one CTA
// are done already; rows of an empty sequence get O = 0, LSE = -inf here.
template <int D, int NT>
__global__ void __launch_bounds__(kD8CombineThreads) decode_fp8_combine_kernel(const DecodeFp8Params p)
{
    constexpr int ROWS = 8 * NT, COLS = D / 4, GROUPS = kD8CombineThreads / COLS;
    __shared__ long long warp_sum[kD8CombineThreads / 32], first;
    __shared__ float4 sm_a[GROUPS][COLS];
    __shared__ float sm_m[kD8CombineThreads / 32], sm_l[GROUPS];
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int tid = threadIdx.x;
    const long long row = blockIdx.x;
    const int r = (int)(row % p.rows);
    const long long bh = row / p.rows;
    const int my_b = (int)(bh / p.Hkv), hk = (int)(bh - (long long)my_b * p.Hkv);
    const long long T = p.Hkv * dec8_scan<kD8CombineThreads>(p, warp_sum, [&](int b, long long before, int, long long) {
        if (b == my_b) first = before;
    });
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = dec8_seq(p, my_b).n;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + row * D;
    if (n == 0) {
        if (tid < D / 8) reinterpret_cast<uint4*>(o)[tid] = make_uint4(0, 0, 0, 0);
        if (tid == 0) p.lse[row] = NEG_INF;
        return;
    }
    const long long X = T < p.ranges ? T : p.ranges, s0 = first * p.Hkv + (long long)hk * n;
    const int x0 = (int)(((s0 + 1) * X - 1) / T), x1 = (int)(((s0 + n) * X - 1) / T);
    if (x0 == x1) return;
    const int rg = r / ROWS, rr = r - rg * ROWS;
    auto part_of = [&](int x) {
        return p.ws + (size_t)(2 * (x * p.row_groups + rg) + (x == x0 ? 1 : 0)) * ROWS * (D + 2);
    };
    float M = NEG_INF;
    for (int x = x0 + tid; x <= x1; x += kD8CombineThreads) M = fmaxf(M, part_of(x)[ROWS * D + rr]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
    if ((tid & 31) == 0) sm_m[tid >> 5] = M;
    __syncthreads();
    M = sm_m[0];
#pragma unroll
    for (int w = 1; w < kD8CombineThreads / 32; ++w) M = fmaxf(M, sm_m[w]);
    const float mb = M == NEG_INF ? 0.0f : M;
    const int grp = tid / COLS, col = tid - grp * COLS;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
#pragma unroll 4
    for (int x = x0 + grp; x <= x1; x += GROUPS) {
        const float* w = part_of(x);
        const float fac = ex2(w[ROWS * D + rr] - mb);
        const float4 v = *reinterpret_cast<const float4*>(w + rr * D + col * 4);
        l = fmaf(fac, w[ROWS * D + ROWS + rr], l);
        a.x = fmaf(fac, v.x, a.x), a.y = fmaf(fac, v.y, a.y);
        a.z = fmaf(fac, v.z, a.z), a.w = fmaf(fac, v.w, a.w);
    }
    sm_a[grp][col] = a;
    if (col == 0) sm_l[grp] = l;
    __syncthreads();
    if (tid < COLS) {
        float sum = 0.0f;
        a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
            const float4 v = sm_a[k][tid];
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
            sum += sm_l[k];
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        reinterpret_cast<uint2*>(o)[tid] =
            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        if (tid == 0) p.lse[row] = sum == 0.0f ? NEG_INF : (mb + __log2f(sum)) * 0.69314718055994531f;
    }
}

// Query rows of a CTA, in eights: as many as the accumulators allow (128 registers of them),
// so that a key head under up to 32 rows (16 at d = 256) is read once.
int decode_fp8_row_tiles(int rows, int d)
{
    const int most = d == 256 ? 2 : 4;
    const int want = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    return want < most ? want : most;
}

template <int D, bool kE5M2, int NT>
static cudaError_t launch_decode_fp8_n(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeFp8Params& p,
                                       cudaStream_t stream)
{
    using C = Dec8Cfg<D, NT>;
    auto kernel = decode_fp8_kernel<D, kE5M2, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    kernel<<<p.ranges * p.row_groups, kD8Threads, C::SMEM, stream>>>(mk, mv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)p.B * p.Hkv * p.rows));
    cfg.blockDim = dim3(kD8CombineThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_fp8_combine_kernel<D, NT>, p);
}

template <int D, bool kE5M2>
static cudaError_t launch_decode_fp8_d(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeFp8Params& p,
                                       cudaStream_t stream)
{
    switch (decode_fp8_row_tiles(p.rows, D)) {
    case 1: return launch_decode_fp8_n<D, kE5M2, 1>(mk, mv, p, stream);
    case 2: return launch_decode_fp8_n<D, kE5M2, 2>(mk, mv, p, stream);
    default:
        if constexpr (D < 256) return launch_decode_fp8_n<D, kE5M2, 4>(mk, mv, p, stream);
        return cudaErrorInvalidValue;
    }
}

cudaError_t launch_decode_fp8(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeFp8Params& p, int d,
                              bool e5m2, cudaStream_t stream)
{
    switch (d) {
    case 64: return e5m2 ? launch_decode_fp8_d<64, true>(mk, mv, p, stream) : launch_decode_fp8_d<64, false>(mk, mv, p, stream);
    case 128: return e5m2 ? launch_decode_fp8_d<128, true>(mk, mv, p, stream) : launch_decode_fp8_d<128, false>(mk, mv, p, stream);
    case 256: return e5m2 ? launch_decode_fp8_d<256, true>(mk, mv, p, stream) : launch_decode_fp8_d<256, false>(mk, mv, p, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gb300
