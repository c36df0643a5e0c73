// decode_fp8_wide.cu -- the decoding step over an 8-bit paged cache (decode_fp8.cu) for many
// query rows under one key head: wide groups, several new tokens, or both.
//
// Same definition and scales as decode_fp8.cu:
//   s_j = c ks_j (q . k8_j),   vs = f 2^e,   w_j = 2^(s_j + e_j - M),   M = running max less 6,
//   l = sum w_j 2^-e_j,   a = sum (w_j f_j) v8_j,   O = a / l,   LSE = ln2 (M + log2 l).
// From about 16 rows on the register products of that kernel, not the cache's bytes, set the
// time (each 16 rows take the conversions and the tile's read again).  Here both products are
// tcgen05.mma with M = 128 rows, so up to 128 rows cost one pass over the cache:
//   * warp 12 streams K and V halves of a tile (128 keys; 64 at d = 256) through a TMA ring,
//     the blocks' scales beside them by cp.async;
//   * warps 4-7 (K) and 8-11 (V) convert a half's codes to fp16 (exact) into the K-major (K)
//     or MN-major (V) swizzled operand, with zeros for V outside the sequence and the window;
//   * warps 13 and 14 issue S = Q K^T and O += P V (neither waits for the other's operands),
//     with Q and P (fp16) read from tensor memory, so
//     the products' shared-memory traffic is the tile alone: per 32 KB of codes 32 + 64 + 64 KB
//     are read, written and read again, under the time that HBM takes to deliver them;
//   * warps 0-3 own 32 rows each: softmax, P, rescaling of O when a maximum is passed by 2^7.
// With 64 rows or fewer the rows are copied to the other warps' lanes and each copy takes its
// share of the tile's keys (its P is zero elsewhere), so all four warps work; the copies'
// results are joined through shared memory at the end of a unit.
// A NaN value at a key that only some rows see (the newest keys, the oldest of a window) is
// converted as 0 and noted; the rows that see it get their NaN when the unit is written.
//
// Measured, 16 sequences x 8 key heads x 8192 keys, d 128 (39.5 us at the copy rate): 32 rows
// 68 us, 64 rows 77, 128 rows 160 (102, 187 and 364 in passes of 16 rows); d 256, 128 rows 154
// (842).  Neither HBM (46 %) nor the tensor pipe (45 %) bounds it, but the chain of a softmax
// warp per tile (S arrives, maximum, weights, P leaves), whose warps share the issue slots with
// the eight that convert; at 128 rows each of its threads has all of a tile's 128 keys.  Loading and
// converting in one warpgroup each for K and V, and S and P V issued by two warps, each cut
// that chain (32 rows: 112.6, 84.5, 73.0 us).
#include "decode_fp8.cuh"

namespace gb300 {

constexpr int kD8WideThreads = 512;    // warpgroups: softmax, K converters, V converters, and the warps below
constexpr int kD8WideProducer = 12, kD8WideMmaS = 13, kD8WideMmaPV = 14;
// registers of a thread after the split; the block starts with 512 x 128 = 65536
constexpr int kD8WideSoftmaxRegs = 208, kD8WideConvertRegs = 96, kD8WideControlRegs = 112;
static_assert(128 * (kD8WideSoftmaxRegs + 2 * kD8WideConvertRegs + kD8WideControlRegs) <= 512 * 128,
              "the split draws on the registers the block was launched with");

template <int D, int COPIES>
struct Dec8WideCfg {
    static constexpr int ROWS = 128 / COPIES;             // query rows of a CTA
    static constexpr int TILE = D == 256 ? 64 : 128;      // keys of a tile
    static constexpr int KEYS = TILE / COPIES;            // keys of a softmax warp
    static constexpr int CB = D < 128 ? D : 128;          // bytes of a row in one TMA box
    static constexpr int NCB = D / CB;
    static constexpr int HALF = TILE * D;                 // bytes of K or V of a tile
    static constexpr int RING = D == 64 ? 8 : 5;          // halves in flight
    static constexpr int F16 = 2 * HALF;                  // a half as fp16
    static constexpr int CBW = TILE * 128;                // 128-byte column block of an fp16 half
    static constexpr int PARTS = TILE / 16;               // 16-key parts, one scale each
    static constexpr int SC_RING = 8;                     // tiles whose scales are held (see the producer)
    static constexpr int S_BUFS = D == 256 ? 1 : 2;
    static constexpr int Q_COL = S_BUFS * TILE;           // tensor memory: S, Q, P, O
    static constexpr int P_COL = Q_COL + D / 2;
    static constexpr int O_COL = P_COL + TILE / 2;
    static constexpr int TMEM_COLS = 512;
    static constexpr int MERGE = COPIES > 1 ? 128 * 32 * 4 : 0;
    static constexpr int SMEM = 1024 + RING * HALF + 4 * F16 + MERGE + 2048;
    static_assert(O_COL + D <= TMEM_COLS, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D, int COPIES>
struct alignas(16) Dec8WideShared {
    using C = Dec8WideCfg<D, COPIES>;
    uint64_t kv_full[C::RING], kv_empty[C::RING];
    uint64_t k16_full[2], k16_empty[2], v16_full[2], v16_empty[2];
    uint64_t s_full[2], s_empty[2];
    uint64_t q_full, q_empty, p_full, pv_done, o_empty, meet, drain[2];
    float scale[C::SC_RING][2 * C::PARTS];
    float m[128], l[128];
    uint32_t nan_keys[4];              // per unit in flight: partly seen keys with a NaN value
    Dec8Setup<kD8WideThreads> setup;
    uint32_t tmem_base;
    int abort_flag;
};

// The partly seen keys of a unit by number: 0-6 the newest (from L - nq + 1 on), 7-13 the
// oldest of the window (from lo on).
__device__ __forceinline__ int dec8_partly(const DecodeFp8Params& p, const Dec8Seq& s, int key)
{
    if (key > s.L - p.nq) return key - (s.L - p.nq + 1);
    return p.window > 0 && key < s.lo + p.nq - 1 ? 7 + key - s.lo : -1;
}

template <int D, int COPIES>
__global__ void __launch_bounds__(kD8WideThreads, 1)
    decode_fp8_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const DecodeFp8Params p, const int e5m2)
{
    using C = Dec8WideCfg<D, COPIES>;
    using Walk = Dec8Walk<C::TILE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* k16 = ring + C::RING * C::HALF;
    uint8_t* v16 = k16 + 2 * C::F16;
    float4* area = reinterpret_cast<float4*>(v16 + 2 * C::F16);
    auto* sh = reinterpret_cast<Dec8WideShared<D, COPIES>*>(v16 + 2 * C::F16 + C::MERGE);
    static_assert(sizeof(Dec8WideShared<D, COPIES>) <= 2048, "shared memory");
    const volatile int* abort_flag = &sh->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float NEG_INF = -__int_as_float(0x7f800000);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::RING; ++s) {
            mbar_init(smem_u32(&sh->kv_full[s]), 1 + 2 * C::PARTS);   // the bytes, lanes' scales
            mbar_init(smem_u32(&sh->kv_empty[s]), 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sh->k16_full[s]), 4);
            mbar_init(smem_u32(&sh->k16_empty[s]), 1);
            mbar_init(smem_u32(&sh->v16_full[s]), 4);
            mbar_init(smem_u32(&sh->v16_empty[s]), 1);
            mbar_init(smem_u32(&sh->s_full[s]), 1);
            mbar_init(smem_u32(&sh->s_empty[s]), 4);
        }
        mbar_init(smem_u32(&sh->q_full), 4);
        mbar_init(smem_u32(&sh->q_empty), 1);
        mbar_init(smem_u32(&sh->p_full), 4);
        mbar_init(smem_u32(&sh->pv_done), 1);
        mbar_init(smem_u32(&sh->o_empty), 4);
        mbar_init(smem_u32(&sh->meet), 4);
        mbar_init(smem_u32(&sh->drain[0]), 1);
        mbar_init(smem_u32(&sh->drain[1]), 1);
        for (int s = 0; s < 4; ++s) sh->nan_keys[s] = 0;
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
        dec8_write_empty<C::TILE, D>(p, kD8WideThreads);
        return;
    }
    Walk w(p, line, sh->setup, x);
    if (warp == kD8WideMmaS) {
        tmem_alloc(smem_u32(&sh->tmem_base), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh->tmem_base;
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool r = ok && mbar_wait(smem_u32(bar), parity, abort_flag, p.timeout_ns);
        ok = __all_sync(0xffffffffu, r);
        return ok;
    };
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(bar));
    };

    if (warp >= kD8WideProducer) regs_decrease<kD8WideControlRegs>();
    if (warp == kD8WideProducer) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = l2_policy_evict_first();
        const int log2_r = p.log2_ps < 6 ? p.log2_ps : 6;       // rows per TMA box: a page, or 64
        const int nbox = C::TILE >> log2_r;                     // 1 .. 8
        const int ps_mask = (1 << p.log2_ps) - 1;
        uint32_t h = 0, t = 0;                                  // halves and tiles issued
        auto wait_lane0 = [&](uint64_t* bar, uint32_t parity) {
            int r = 1;
            if (lane == 0) r = mbar_wait(smem_u32(bar), parity, abort_flag, p.timeout_ns);
            ok = __shfl_sync(0xffffffffu, r, 0) != 0;
            return ok;
        };
        while (w.more && ok) {
            const int* ptab = p.page_table + (size_t)w.b * p.max_pages;
            int held = 0, pg = 0;                                // 32 boxes' pages from box `held` on
            for (int k = w.k0; k < w.k1 && ok; ++k, ++t) {
                const int key0 = (w.seq.t0 + k) * C::TILE, box0 = key0 >> log2_r;
                if (k == w.k0 || box0 - held >= 32) {
                    held = box0;
                    const long long key = (long long)(box0 + lane) << log2_r;
                    const int pi = (int)min(key >> p.log2_ps, (long long)p.max_pages - 1);
                    pg = min(max(dec8_ld(ptab + pi), 0), p.num_pages - 1);
                }
                const int pg_box = __shfl_sync(0xffffffffu, pg, box0 - held + (lane & (nbox - 1)));
                const int part_key = key0 + (lane & (C::PARTS - 1)) * 16;
                const int pg_part = __shfl_sync(0xffffffffu, pg, (part_key >> log2_r) - held);
#pragma unroll
                for (int which = 0; which < 2; ++which) {        // K, then V
                    const uint32_t s = h % C::RING;
                    if (!wait_lane0(&sh->kv_empty[s], ((h / C::RING) & 1) ^ 1)) break;
                    const uint32_t fb = smem_u32(&sh->kv_full[s]);
                    const bool issue = ++h != p.withhold;
                    if (lane == 0 && issue) mbar_arrive_expect_tx(fb, C::HALF);
                    __syncwarp();
                    // The tile's scales complete on the barrier of its K half, so whoever has seen
                    // S of the tile may read them.  Their place is free: the half that makes room
                    // for this one was converted, so S two tiles after the one whose scales it
                    // held (eight tiles back) has begun, and the softmax reads a tile's scales
                    // before it gives up that tile's S.
                    const size_t at = (((size_t)pg_part * p.Hkv + w.hk) << (p.log2_ps - p.log2_blk)) +
                                      ((part_key & ps_mask) >> p.log2_blk);
                    if (which == 0 && lane < 2 * C::PARTS && issue)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                         smem_u32(&sh->scale[t % C::SC_RING][lane])),
                                     "l"((lane < C::PARTS ? p.ks : p.vs) + at) : "memory");
                    if (lane < 2 * C::PARTS && issue)
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(fb) : "memory");
                    if (lane < nbox && issue) {
                        const uint32_t dst = smem_u32(ring + s * C::HALF) + (lane << log2_r) * C::CB;
#pragma unroll
                        for (int c = 0; c < C::NCB; ++c)
                            tma_load_3d(dst + c * C::TILE * C::CB, which ? &tmV : &tmK, fb, c * C::CB,
                                        (key0 + (lane << log2_r)) & ps_mask, pg_box * p.Hkv + w.hk, pol);
                    }
                }
            }
            if (ok) w.next(p);
        }
        if (!ok && lane == 0) dec8_timeout(p, &sh->abort_flag);
        // every copy issued lands before shared memory is released
        if (lane == 0) {
            for (uint32_t k = h < C::RING ? 0 : h - C::RING; k < h; ++k)
                if (k + 1 != p.withhold)
                    mbar_wait(smem_u32(&sh->kv_full[k % C::RING]), (k / C::RING) & 1, nullptr, kCleanupTimeoutNs);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    } else if (warp == kD8WideMmaS) {
        // ------------------------------------------------------------ S(t) = Q K(t)^T
        constexpr uint32_t idesc = idesc_f32acc(0, 0, 128, C::TILE);     // fp16, K-major B
        const uint64_t k_desc = sdesc_sw128(smem_u32(k16), 16, 1024);
        uint32_t t = 0, uc = 0;
        while (w.more && ok) {
            if (!wait_all(&sh->q_full, uc & 1)) break;
            for (int k = w.k0; k < w.k1; ++k, ++t) {
                const uint32_t slot = t & 1, sb = C::S_BUFS == 2 ? slot : 0;
                if (!wait_all(&sh->k16_full[slot], (t >> 1) & 1)) break;
                if (!wait_all(&sh->s_empty[sb], ((t / C::S_BUFS) & 1) ^ 1)) break;
                tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (slot * C::F16 + ((kk * 32) / 128) * C::CBW + (kk * 32) % 128) >> 4;
                    mma_ts_warp<false>(tmem + sb * C::TILE, tmem + C::Q_COL + kk * 8, k_desc + off, idesc, kk > 0);
                }
                mma_commit_warp(smem_u32(&sh->s_full[sb]));
                mma_commit_warp(smem_u32(&sh->k16_empty[slot]));
            }
            if (!ok) break;
            mma_commit_warp(smem_u32(&sh->q_empty));
            ++uc;
            w.next(p);
        }
        if (!ok && lane == 0) dec8_timeout(p, &sh->abort_flag);
        mma_commit_warp(smem_u32(&sh->drain[0]));
        mbar_wait(smem_u32(&sh->drain[0]), 0, nullptr, kCleanupTimeoutNs);
        __syncwarp();
    } else if (warp == kD8WideMmaPV) {
        // ------------------------------------------------------------ O (+)= P(t) V(t)
        constexpr uint32_t idesc = idesc_f32acc(0, 1, 128, D);           // fp16, MN-major B
        const uint64_t v_desc = sdesc_sw128(smem_u32(v16), C::CBW, 1024);
        uint32_t t = 0, uc = 0;
        while (w.more && ok) {
            if (!wait_all(&sh->o_empty, (uc & 1) ^ 1)) break;            // the unit before has been read
            for (int k = w.k0; k < w.k1; ++k, ++t) {
                const uint32_t slot = t & 1;
                if (!wait_all(&sh->v16_full[slot], (t >> 1) & 1)) break;
                if (!wait_all(&sh->p_full, t & 1)) break;
                tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < C::TILE / 16; ++kk)
                    mma_ts_warp<false>(tmem + C::O_COL, tmem + C::P_COL + kk * 8,
                                       v_desc + ((slot * C::F16 + kk * 16 * 128) >> 4), idesc, kk > 0 || k > w.k0);
                mma_commit_warp(smem_u32(&sh->pv_done));
                mma_commit_warp(smem_u32(&sh->v16_empty[slot]));
            }
            if (!ok) break;
            ++uc;
            w.next(p);
        }
        if (!ok && lane == 0) dec8_timeout(p, &sh->abort_flag);
        mma_commit_warp(smem_u32(&sh->drain[1]));
        mbar_wait(smem_u32(&sh->drain[1]), 0, nullptr, kCleanupTimeoutNs);
        __syncwarp();
    } else if (warp >= 4 && warp < kD8WideProducer) {
        // ------------------------------------------------------------ converters
        regs_decrease<kD8WideConvertRegs>();
        const bool is_v = warp >= 8;                             // K halves, or V halves
        const int ct = threadIdx.x & 127;
        uint64_t* full16 = is_v ? sh->v16_full : sh->k16_full;
        uint64_t* empty16 = is_v ? sh->v16_empty : sh->k16_empty;
        const uint32_t to0 = smem_u32(is_v ? v16 : k16);
        uint32_t h = is_v ? 1 : 0, t = 0, uc = 0;
        // One half: chunks of 16 codes to two chunks of 8 fp16.  Eight lanes take four chunks of
        // two rows, r and r ^ 5 (r and r + 1 at d = 64): under the 128-byte swizzles of both
        // sides (64-byte at d = 64) they read and write all banks once.
        auto convert = [&](auto fmt, uint32_t from, uint32_t to, int key0) {
            constexpr bool kE5M2 = decltype(fmt)::value;
            constexpr int N = C::HALF / 16 / 128;                // chunks of a thread
            const bool edge = is_v && (key0 + (C::TILE - 1) > w.seq.L - p.nq || key0 < w.seq.lo + p.nq - 1);
            // chunk i of the thread: quad i % Q of four chunks in row first + (i / Q) * 32
            constexpr int Q = D / 64;
            const int l5 = ct & 31, c = l5 & 3;
            const int first = (ct >> 5) * 8 + (C::CB == 128 ? (l5 >> 3) ^ ((l5 & 4) ? 5 : 0) : l5 >> 2);
            uint4 u[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int quad = i % Q, row = first + (i / Q) * 32;
                const int ch = C::CB == 128 ? ((quad & 1) * 4 + c) ^ (first & 7) : c ^ ((first >> 1) & 3);
                u[i] = dec8_lds128(from + (quad >> 1) * C::TILE * C::CB + row * C::CB + ch * 16);
            }
            if (edge) {
#pragma unroll 1
                for (int i = 0; i < N; ++i) {
                    const int key = key0 + first + (i / Q) * 32;
                    uint4 v = u[0];
#pragma unroll
                    for (int k = 1; k < N; ++k)
                        if (k == i) v = u[k];
                    if (key >= w.seq.L || key < w.seq.lo) v = make_uint4(0, 0, 0, 0);
                    const int partly = dec8_partly(p, w.seq, key);
                    if (partly >= 0 && (dec8_nonfinite<kE5M2>(v.x) | dec8_nonfinite<kE5M2>(v.y) |
                                        dec8_nonfinite<kE5M2>(v.z) | dec8_nonfinite<kE5M2>(v.w))) {
                        atomicOr(&sh->nan_keys[uc & 3], 1u << partly);
                        v.x &= ~((dec8_nonfinite<kE5M2>(v.x) >> 7) * 0xFFu);
                        v.y &= ~((dec8_nonfinite<kE5M2>(v.y) >> 7) * 0xFFu);
                        v.z &= ~((dec8_nonfinite<kE5M2>(v.z) >> 7) * 0xFFu);
                        v.w &= ~((dec8_nonfinite<kE5M2>(v.w) >> 7) * 0xFFu);
                    }
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        if (k == i) u[k] = v;
                }
            }
            // quad q of a row is the 128-byte fp16 block q, chunk c of it the chunks 2c and 2c + 1
            const uint32_t out0 = to + first * 128 + (((2 * c) ^ (first & 7)) * 16);
            const uint32_t out1 = to + first * 128 + (((2 * c + 1) ^ (first & 7)) * 16);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t at = (i % Q) * C::CBW + (i / Q) * 32 * 128;
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(out0 + at),
                             "r"(dec8_half2<kE5M2>(u[i].x & 0xFFFF)), "r"(dec8_half2<kE5M2>(u[i].x >> 16)),
                             "r"(dec8_half2<kE5M2>(u[i].y & 0xFFFF)), "r"(dec8_half2<kE5M2>(u[i].y >> 16)) : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(out1 + at),
                             "r"(dec8_half2<kE5M2>(u[i].z & 0xFFFF)), "r"(dec8_half2<kE5M2>(u[i].z >> 16)),
                             "r"(dec8_half2<kE5M2>(u[i].w & 0xFFFF)), "r"(dec8_half2<kE5M2>(u[i].w >> 16)) : "memory");
            }
        };
        while (w.more && ok) {
            for (int k = w.k0; k < w.k1; ++k, ++t, h += 2) {
                const uint32_t slot = t & 1, s = h % C::RING;
                if (!wait_all(&sh->kv_full[s], (h / C::RING) & 1)) break;
                if (!wait_all(&empty16[slot], ((t >> 1) & 1) ^ 1)) break;
                const uint32_t from = smem_u32(ring + s * C::HALF), to = to0 + slot * C::F16;
                const int key0 = (w.seq.t0 + k) * C::TILE;
                if (e5m2) convert(std::true_type{}, from, to, key0);
                else convert(std::false_type{}, from, to, key0);
                fence_proxy_async_smem();
                arrive(&sh->kv_empty[s]);
                arrive(&full16[slot]);
            }
            if (!ok) break;
            ++uc;
            w.next(p);
        }
        if (!ok && lane == 0) dec8_timeout(p, &sh->abort_flag);
    } else if (warp < 4) {
        // ------------------------------------------------------------ softmax, 32 rows a warp
        regs_increase<kD8WideSoftmaxRegs>();
        constexpr int GROUPS = 4 / COPIES;                       // warps that hold the rows once
        const int copy = warp / GROUPS, row = (warp % GROUPS) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const bool live = row0 + row < p.rows;
        const int query = (row0 + row) % p.nq;
        uint32_t t = 0, uc = 0, meet_parity = 0;
        auto meet = [&]() {
            arrive(&sh->meet);
            const bool r = wait_all(&sh->meet, meet_parity);
            meet_parity ^= 1;
            return r;
        };
        // The unit's query row into tensor memory as fp16, scaled by a power of two so that its
        // largest value is just below 2^15; returns the softmax scale over that factor.
        // Held in registers between the two (HOLD) the row costs one latency instead of D / 32; us, held
        // and read twice: 32 rows d 128 68.0 / 70.1, d 256 124.9 / 128.2, 64 rows d 256 135.5 / 142.4, but
        // 64 rows d 128 91 / 76, 128 rows d 128 179 / 156, d 256 173 / 151 (the loop's registers).
        auto put_q = [&](uint32_t unit) -> float {
            constexpr bool HOLD = COPIES == 4 || (COPIES == 2 && D == 256);
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                            (((size_t)w.b * p.Hkv + w.hk) * p.rows + row0 + (live ? row : 0)) * D);
            uint32_t big = 0;
            auto largest = [&](const uint4& u) {
                big = max(max(big, max((u.x << 16) & 0x7FFF0000u, u.x & 0x7FFF0000u)),
                          max(max((u.y << 16) & 0x7FFF0000u, u.y & 0x7FFF0000u),
                              max(max((u.z << 16) & 0x7FFF0000u, u.z & 0x7FFF0000u),
                                  max((u.w << 16) & 0x7FFF0000u, u.w & 0x7FFF0000u))));
            };
            uint4 held[HOLD ? D / 8 : 1];
            if constexpr (HOLD) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) held[i] = dec8_ld(q + i);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) largest(held[i]);
            } else {
#pragma unroll 8
                for (int i = 0; i < D / 8; ++i) largest(dec8_ld(q + i));
            }
            const int ex = max((int)(big >> 23), 15) - 14;       // biased exponent of the factor's inverse
            const float down = live ? __int_as_float((254 - ex) << 23) : 0.0f;
            if (!wait_all(&sh->q_empty, (unit & 1) ^ 1)) return 0.0f;
            tc_fence_after_sync();
            auto put = [&](int c) {                              // 64 of the row's values
                uint32_t f[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 u = HOLD ? held[HOLD ? c * 8 + i : 0] : dec8_ld(q + c * 8 + i);
                    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        f[4 * i + k] = live ? dec8_pack_half2(__uint_as_float(v[k] << 16) * down,
                                                              __uint_as_float(v[k] & 0xFFFF0000u) * down)
                                            : 0u;
                }
                tmem_st32p(lanes + C::Q_COL + c * 32, f);
            };
            if constexpr (HOLD) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c) put(c);
            } else {
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) put(c);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            arrive(&sh->q_full);
            return __int_as_float(ex << 23) * p.c_log2;
        };
        if constexpr (COPIES > 1) {                              // the other copies' keys: P = 0 for good
            uint32_t z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = 0;
#pragma unroll
            for (int c = 0; c < C::TILE / 32; ++c) tmem_st16p(lanes + C::P_COL + c * 16, z);
        }
        float rowc = put_q(0);
        while (w.more && ok) {
            const size_t unit_row = ((size_t)w.b * p.Hkv + w.hk) * p.rows + row0;
            const int last = w.seq.L - p.nq + query;             // this row's newest key
            const int oldest = p.window > 0 ? last - p.window : 0;
            float m = NEG_INF, l = 0.0f;
            int v_top = 0;
            for (int k = w.k0; k < w.k1; ++k, ++t) {
                const int key0 = (w.seq.t0 + k) * C::TILE + copy * C::KEYS;
                const uint32_t sb = C::S_BUFS == 2 ? t & 1 : 0, sc = t % C::SC_RING;
                if (!wait_all(&sh->s_full[sb], (t / C::S_BUFS) & 1)) break;
                tc_fence_after_sync();
                const uint32_t from = lanes + sb * C::TILE + copy * C::KEYS, to = lanes + C::P_COL + copy * (C::KEYS / 2);
                // scores in pieces of at most 64 keys; with 128 they are read once for the maximum
                // and again for the weights
                constexpr int PIECE = C::KEYS < 64 ? C::KEYS : 64, BLOCKS = C::KEYS / 16;
                uint32_t sr[PIECE];
                float* s = reinterpret_cast<float*>(sr);
                auto load = [&](int at) {
                    if constexpr (PIECE >= 32) {
#pragma unroll
                        for (int c = 0; c < PIECE / 32; ++c) tmem_ld32p(from + at + c * 32, sr + c * 32);
                        tmem_wait_ld_only();
#pragma unroll
                        for (int c = 0; c < PIECE / 32; ++c) reg_fence32(sr + c * 32);
                    } else {
                        tmem_ld16(from + at, sr);
                        tmem_wait_ld16(sr);
                    }
                };
                load(0);
                const bool edge = key0 + C::KEYS - 1 > w.seq.L - p.nq ||
                                  (p.window > 0 && key0 < w.seq.L - 1 - p.window);
                float kf[BLOCKS], ve[BLOCKS], vf[BLOCKS];
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    kf[b] = sh->scale[sc][copy * BLOCKS + b] * rowc;
                    float vsc = sh->scale[sc][C::PARTS + copy * BLOCKS + b];
                    if (edge) {
                        const int kb = key0 + b * 16;
                        if (kb >= w.seq.L || kb + 15 < w.seq.lo) kf[b] = vsc = 0.0f;   // nobody's: whatever its scales are
                    }
                    const Dec8ValueScale vs(vsc, v_top);
                    ve[b] = vs.e;
                    vf[b] = vs.f;
                }
                if constexpr (C::KEYS == PIECE) {
                    tc_fence_before_sync();
                    arrive(&sh->s_empty[sb]);
                }
                auto scale_and_mask = [&](int at) {
#pragma unroll
                    for (int i = 0; i < PIECE; i += 2) {
                        const int b = (at + i) / 16;
                        const float2 v = __ffma2_rn(make_float2(s[i], s[i + 1]), make_float2(kf[b], kf[b]), make_float2(ve[b], ve[b]));
                        s[i] = v.x, s[i + 1] = v.y;
                    }
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < PIECE; ++i)
                            if (key0 + at + i > last || key0 + at + i < oldest) s[i] = NEG_INF;
                    }
                };
                float mx = NEG_INF;
#pragma unroll
                for (int at = 0; at < C::KEYS; at += PIECE) {
                    if (at > 0) load(at);
                    scale_and_mask(at);
#pragma unroll
                    for (int i = 0; i < PIECE; i += 2) mx = fmax3(mx, s[i], s[i + 1]);
                }
                const bool raise = mx > m + (kD8Room + kD8Tau);
                const float al = raise ? ex2(m - (mx - kD8Room)) : 1.0f;     // ex2(-inf) = 0
                if (raise) {
                    l *= al;
                    m = mx - kD8Room;
                }
                const float mb = m == NEG_INF ? 0.0f : m;
                if (k > w.k0) {
                    // P may be written, and O rescaled, once P(k-1) V(k-1) is done
                    if (!wait_all(&sh->pv_done, (t - 1) & 1)) break;
                    tc_fence_after_sync();
                    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(lanes + C::O_COL + c * 32, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                            tmem_st32p(lanes + C::O_COL + c * 32, o);
                        }
                    }
                }
#pragma unroll
                for (int at = 0; at < C::KEYS; at += PIECE) {
                    if constexpr (C::KEYS > PIECE) {
                        load(at);
                        scale_and_mask(at);
                    }
#pragma unroll
                    for (int b = 0; b < PIECE / 16; ++b) {
                        float2 sum = make_float2(0.0f, 0.0f);
                        const float2 down = make_float2(-mb, -mb), f = make_float2(vf[at / 16 + b], vf[at / 16 + b]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 d = __fadd2_rn(make_float2(s[b * 16 + 2 * i], s[b * 16 + 2 * i + 1]), down);
                            const float2 e = make_float2(ex2(d.x), ex2(d.y));
                            sum = __fadd2_rn(sum, e);
                            const float2 g = __fmul2_rn(e, f);
                            sr[b * 8 + i] = dec8_pack_half2(g.x, g.y);
                        }
                        l = fmaf(sum.x + sum.y, __int_as_float((127 - (int)ve[at / 16 + b]) << 23), l);
                    }
                    if constexpr (PIECE == 64) {
                        tmem_st32p(to + at / 2, sr);
                    } else if constexpr (PIECE == 32) {
                        tmem_st16p(to, sr);
                    } else {
                        uint32_t f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = sr[i];
                        tmem_st8(to, f);
                    }
                }
                if constexpr (C::KEYS > PIECE) {
                    tc_fence_before_sync();
                    arrive(&sh->s_empty[sb]);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                arrive(&sh->p_full);
            }
            if (!ok) break;

            // the next unit's queries first, so that its S can start while this one is written
            const Walk u = w;
            w.next(p);
            float next_rowc = 0.0f;
            if (w.more) {
                next_rowc = put_q(uc + 1);
                if (!ok) break;
            }
            if (!wait_all(&sh->pv_done, (t - 1) & 1)) break;
            tc_fence_after_sync();
            const bool whole = u.whole();
            float* part = dec8_my_part<C::ROWS, D>(p, u.k0 == 0);
            const uint32_t nan_keys = *reinterpret_cast<volatile uint32_t*>(&sh->nan_keys[uc & 3]);
            // four columns of row r: NaN where a noted key that the row sees has one
            auto put_nan = [&](int r, int d4, float4& v) {
                const int newest = u.seq.L - p.nq + (row0 + r) % p.nq;
                for (uint32_t left = nan_keys; left; left &= left - 1) {
                    const int i = __ffs(left) - 1, key = i < 7 ? u.seq.L - p.nq + 1 + i : u.seq.lo + i - 7;
                    if (key > newest || (p.window > 0 && key < newest - p.window)) continue;
                    const int page = min(max(dec8_ld(p.page_table + (size_t)u.b * p.max_pages + (key >> p.log2_ps)), 0),
                                         p.num_pages - 1);
                    const uint8_t* at = p.vc + (((((size_t)page * p.Hkv + u.hk) << p.log2_ps) +
                                                 (key & ((1 << p.log2_ps) - 1))) * D + d4 * 4);
                    const uint32_t codes = (uint32_t)dec8_ld(reinterpret_cast<const int*>(at));
                    const uint32_t bad = e5m2 ? dec8_nonfinite<true>(codes) : dec8_nonfinite<false>(codes);
                    const float nan = __int_as_float(0x7fc00000);
                    if (bad & 0x80u) v.x = nan;
                    if (bad & 0x8000u) v.y = nan;
                    if (bad & 0x800000u) v.z = nan;
                    if (bad & 0x80000000u) v.w = nan;
                }
            };
            auto put = [&](int r, int d4, float4 v, float top, float sum) {
                if (nan_keys) put_nan(r, d4, v);
                if (whole) {
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (unit_row + r) * D + d4 * 4) =
                        make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                    if (d4 == 0) p.lse[unit_row + r] = dec8_lse(top, sum);
                } else {
                    *reinterpret_cast<float4*>(part + r * D + d4 * 4) = v;
                    if (d4 == 0) {
                        part[C::ROWS * D + r] = top;
                        part[C::ROWS * D + C::ROWS + r] = sum;
                    }
                }
            };
            if constexpr (COPIES > 1) {
                sh->m[threadIdx.x] = m;
                sh->l[threadIdx.x] = l;
            }
#pragma unroll 1
            for (int c = 0; c < D / 32 && ok; ++c) {
                uint32_t o[32];
                tmem_ld32(lanes + C::O_COL + c * 32, o);
                tmem_wait_ld(o);
                const float* of = reinterpret_cast<const float*>(o);
                if constexpr (COPIES == 1) {
                    if (live) {
#pragma unroll
                        for (int q4 = 0; q4 < 8; ++q4)
                            put(row, c * 8 + q4, make_float4(of[4 * q4], of[4 * q4 + 1], of[4 * q4 + 2], of[4 * q4 + 3]), m, l);
                    }
                } else {
                    const int me = threadIdx.x;
#pragma unroll
                    for (int q4 = 0; q4 < 8; ++q4)
                        area[me * 8 + (q4 ^ (me & 7))] = make_float4(of[4 * q4], of[4 * q4 + 1], of[4 * q4 + 2], of[4 * q4 + 3]);
                    if (!meet()) break;
                    for (int idx = me; idx < C::ROWS * 8; idx += 128) {
                        const int r = idx >> 3, q4 = idx & 7;
                        if (row0 + r >= p.rows) break;
                        float top = NEG_INF, sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < COPIES; ++i) top = fmaxf(top, sh->m[i * C::ROWS + r]);
                        const float base = top == NEG_INF ? 0.0f : top;
                        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                        for (int i = 0; i < COPIES; ++i) {
                            const int from = i * C::ROWS + r;
                            const float fac = ex2(sh->m[from] - base);
                            const float4 a = area[from * 8 + (q4 ^ (from & 7))];
                            sum = fmaf(sh->l[from], fac, sum);
                            v.x = fmaf(a.x, fac, v.x), v.y = fmaf(a.y, fac, v.y);
                            v.z = fmaf(a.z, fac, v.z), v.w = fmaf(a.w, fac, v.w);
                        }
                        put(r, c * 8 + q4, v, top, sum);
                    }
                    if (!meet()) break;
                }
            }
            if (!ok) break;
            if (nan_keys) {                                      // for the unit after the next three
                __syncwarp();
                if constexpr (COPIES == 1) {
                    if (!meet()) break;
                }
                if (threadIdx.x == 0) sh->nan_keys[uc & 3] = 0;
            }
            tc_fence_before_sync();
            arrive(&sh->o_empty);
            if (threadIdx.x == 0) dec8_name_parts(p, u, line, x, rg, unit_row);
            rowc = next_rowc;
            ++uc;
        }
        if (!ok && lane == 0) dec8_timeout(p, &sh->abort_flag);
        tmem_wait_st();
        if (ok) dec8_write_empty<C::TILE, D>(p, 128);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kD8WideMmaS) tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int D, int COPIES>
static cudaError_t launch_wide_n(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeFp8Params& p, bool e5m2,
                                 cudaStream_t stream)
{
    using C = Dec8WideCfg<D, COPIES>;
    auto kernel = decode_fp8_wide_kernel<D, COPIES>;
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
    cfg.blockDim = dim3(kD8WideThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    e = cudaLaunchKernelEx(&cfg, kernel, mk, mv, p, e5m2 ? 1 : 0);
    if (e != cudaSuccess) return e;
    return launch_decode_fp8_combine<D, C::ROWS>(p, cfg);
}

template <int D>
static cudaError_t launch_wide_d(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeFp8Params& p, bool e5m2,
                                 int cta_rows, cudaStream_t stream)
{
    if (cta_rows == 32) return launch_wide_n<D, 4>(mk, mv, p, e5m2, stream);
    if (cta_rows == 64) return launch_wide_n<D, 2>(mk, mv, p, e5m2, stream);
    return launch_wide_n<D, 1>(mk, mv, p, e5m2, stream);
}

cudaError_t launch_decode_fp8_wide(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeFp8Params& p, int d,
                                   bool e5m2, int cta_rows, cudaStream_t stream)
{
    switch (d) {
    case 64: return launch_wide_d<64>(mk, mv, p, e5m2, cta_rows, stream);
    case 128: return launch_wide_d<128>(mk, mv, p, e5m2, cta_rows, stream);
    case 256: return launch_wide_d<256>(mk, mv, p, e5m2, cta_rows, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gb300
