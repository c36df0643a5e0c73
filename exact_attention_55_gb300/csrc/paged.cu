// paged.cu -- what a serving step needs around attention over a paged cache: the step's
// pages, slots and positions from the requests' lengths (attn_paged_plan), and the new
// keys and values written to their slots (attn_cache_append_bf16, attn_cache_append_fp8).
//
// "Warp Group Cluster 优化：Flash Attention V3 在 H100 上的 FP8 融合计算实践",
// 局限性与后续方向 item 2: KV-cache management with PagedAttention; its §3 FP8 量化与精度保持
// and "大模型加速-核心网络算子-Flash Attention V3" §1 item 3 (块量化): one scale per block.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_scale.cuh"
#include "paged_params.h"
#include "ptx.cuh"

namespace gb300 {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ the plan of a step
//
// With n_b new tokens (a negative count is 0) and L_b cached ones (clamped to the table):
//   end_b  = n_0 + ... + n_b                       (rows of the packed new tokens)
//   fits_b = L_b + n_b <= max_pages * ps and end_b <= num_tokens
//   need_b = ceil((L_b + n_b) / ps) - ceil(L_b / ps), 0 unless fits_b
//   base_b = need_0 + ... + need_{b-1}
//   served_b = fits_b and (need_b == 0 or base_b + need_b <= free)
// and the k-th page taken is free_pages[free - 1 - k], page ceil(L_b / ps) + k - base_b of
// the request with base_b <= k < base_b + need_b.  Once a request does not fit into the
// free pages no later one that needs a page does, so the pages taken are the first ones.
//
// Latency-bound (a step of 16 requests moves under 1 KB): one launch of one cluster.
// Every CTA scans all requests for itself into shared memory, the cluster meets once (the
// lengths and the free count may be overwritten in place after that), and then its
// threads share the tokens, pages and requests.  A token finds its request by bisection
// of the ends, four tokens at a time; a page that the step takes is read from the free stack,
// never from the table entry another thread writes.  Measured: 16 requests of one token 3.3
// us, 1024 requests with 29 thousand tokens 8.4 us (11.7 with a third scan and lookups one by
// one), of which a launch is about 2 and the dependent reads of lengths and pages 2.
constexpr int kPlanMaxThreads = 1024;

// Exclusive sum over the block's threads and the total; every thread calls it.  `sums` is a
// scan's own, one per warp.
__device__ __forceinline__ long long plan_block_scan(long long x, long long* sums, long long* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    long long all = lane < warps ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += y;
    }
    *total = __shfl_sync(0xffffffffu, all, 31);
    const long long before = __shfl_sync(0xffffffffu, all, (warp + 31) & 31);
    return (warp ? before : 0) + inc - x;
}

// For each x[k] the last index i in [0, n) with a[i] <= x[k], for a non-decreasing from
// a[0] <= x[k] on; `top` is the largest power of two below n (0 for n = 1).
template <int K>
__device__ __forceinline__ void last_not_above(const int* a, int n, int top, const int (&x)[K], int (&at)[K])
{
#pragma unroll
    for (int k = 0; k < K; ++k) at[k] = 0;
    for (int step = top; step > 0; step >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int next = at[k] + step;
            if (next < n && a[next] <= x[k]) at[k] = next;
        }
}

__global__ void __launch_bounds__(kPlanMaxThreads) paged_plan_kernel(const PlanParams p)
{
    extern __shared__ int sm_plan[];
    __shared__ long long sums[2][kPlanMaxThreads / 32];
    __shared__ int taken_s;
    int* start = sm_plan;               // first packed row of the request, at most num_tokens
    int* base = sm_plan + p.B;          // pages taken before it
    int* len = sm_plan + 2 * p.B;       // cached length, or its complement when not served
    const cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, nt = blockDim.x;
    const int ps = 1 << p.log2_ps;
    const long long cap = (long long)p.max_pages << p.log2_ps;   // fits an int
    const int free = min(max(*p.free_count, 0), p.free_capacity);
    const int per = (p.B + nt - 1) / nt, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    if (tid == 0) taken_s = 0;

    // the thread's own requests: their counts in start and lengths in len until they are replaced
    long long tokens = 0, total, all;
    for (int b = b0; b < b1; ++b) {
        const int n = max(p.new_lens[b], 0);
        start[b] = n;
        len[b] = (int)min((long long)max(p.seq_lens[b], 0), cap);
        tokens += n;
    }
    const long long first = plan_block_scan(tokens, sums[0], &total);
    auto pages_needed = [&](long long end, long long n, long long L) -> long long {
        if (L + n > cap || end > p.num_tokens) return -1;        // does not fit
        return ((L + n + ps - 1) >> p.log2_ps) - ((L + ps - 1) >> p.log2_ps);
    };
    long long need_sum = 0, end = first;
    for (int b = b0; b < b1; ++b) {
        end += start[b];
        const long long need = pages_needed(end, start[b], len[b]);
        need_sum += need > 0 ? need : 0;
    }
    long long at = plan_block_scan(need_sum, sums[1], &all);
    int taken = 0;
    end = first;
    for (int b = b0; b < b1; ++b) {
        const int n = start[b], L = len[b];
        start[b] = (int)min(end, (long long)p.num_tokens);
        end += n;
        const long long need = pages_needed(end, n, L);
        const bool ok = need == 0 || (need > 0 && at + need <= free);
        base[b] = (int)min(at, 0x7fffffffLL);
        len[b] = ok ? L : ~L;
        if (need > 0) {
            at += need;
            if (ok) taken = (int)at;              // the pages served are the first ones
        }
    }
    taken = (int)__reduce_max_sync(0xffffffffu, (unsigned)taken);
    if ((tid & 31) == 0 && taken > 0) atomicMax(&taken_s, taken);
    __syncthreads();
    cluster.sync();                               // every CTA has read the lengths
    taken = taken_s;

    const int rank = (int)cluster.block_rank() * nt + tid, threads = (int)cluster.num_blocks() * nt;
    const int rows = (int)min(total, (long long)p.num_tokens);   // packed rows in use
    const int top = p.B > 1 ? 1 << (31 - __clz(p.B - 1)) : 0;
    constexpr int K = 4;                          // tokens a thread looks up together
    for (long long t0 = rank; t0 < p.num_tokens; t0 += (long long)K * threads) {
        int t[K], b[K];
#pragma unroll
        for (int k = 0; k < K; ++k) t[k] = (int)min(t0 + (long long)k * threads, 0x7fffffffLL);
        last_not_above(start, p.B, top, t, b);
        int pos[K], id[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int L = len[b[k]];
            pos[k] = -1;
            id[k] = -1;
            if (t[k] < rows && L >= 0) {
                pos[k] = L + t[k] - start[b[k]];
                const int page = pos[k] >> p.log2_ps, old = (L + ps - 1) >> p.log2_ps;
                id[k] = page < old ? p.page_table[(size_t)b[k] * p.max_pages + page]
                                   : p.free_pages[free - 1 - (base[b[k]] + page - old)];
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t[k] < p.num_tokens) {
                p.slot_map[t[k]] = id[k] < 0 ? -1 : ((long long)id[k] << p.log2_ps) + (pos[k] & (ps - 1));
                p.positions[t[k]] = pos[k];
            }
    }
    for (int b = rank; b < p.B; b += threads) {
        const int next = b + 1 < p.B ? start[b + 1] : rows;
        const bool ok = len[b] >= 0;
        p.cu_new[b] = start[b];
        if (b == p.B - 1) p.cu_new[p.B] = rows;
        p.served[b] = ok ? 1 : 0;
        p.seq_lens_out[b] = ok ? len[b] + (next - start[b]) : ~len[b];
    }
    if (rank == 0) *p.free_count_out = free - taken;
    for (int k = rank; k < taken; k += threads) {
        const int x[1] = {k};
        int b[1];
        last_not_above(base, p.B, top, x, b);
        const int page = ((len[b[0]] + ps - 1) >> p.log2_ps) + k - base[b[0]];
        p.page_table[(size_t)b[0] * p.max_pages + page] = p.free_pages[free - 1 - k];
    }
}

cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t stream)
{
    const int smem = 3 * p.B * (int)sizeof(int);
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   200 * 1024);
        if (e != cudaSuccess) return e;
    }
    const int items = p.num_tokens > p.B ? p.num_tokens : p.B;
    int ctas = (items + 4095) / 4096;
    ctas = ctas >= 8 ? 8 : ctas >= 4 ? 4 : ctas >= 2 ? 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(items <= 128 ? 128 : items <= 512 ? 512 : kPlanMaxThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, p);
}

// ------------------------------------------------------------------ bf16 append
//
// cache[slot / ps][h][slot % ps] = row (t, h); slots outside the cache (padding) are
// skipped.  HBM-bound: each row is read once and written once.  A CTA takes kTokens tokens of
// K or V, all heads; a token's heads are one run of memory on the input side, so a thread
// copies the same 16-byte piece of each token, the loads of its tokens in flight together.
// Measured: 16006 tokens of 16 heads, d 128, as columns of a wider matrix 41.7 us = 6.3 TB/s
// read and written (54.0 with a 16-byte piece a thread and divisions for its place); a step
// of 16 tokens 1.7 us.
template <int kTokens>
__global__ void __launch_bounds__(256) cache_append_bf16_kernel(const AppendParams p)
{
    const bool is_v = blockIdx.y != 0;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k);
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.vc : p.kc);
    const long long stride = is_v ? p.v_stride : p.k_stride;
    const int t0 = blockIdx.x * kTokens, ps_mask = (1 << p.log2_ps) - 1;
    const int log2_d = p.d == 64 ? 6 : p.d == 128 ? 7 : 8;
    long long at[kTokens];                         // row of (page, head 0, slot % ps), or -1
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const long long slot = t0 + i < p.T ? __ldg(p.slot_map + t0 + i) : -1;
        at[i] = slot < 0 || slot >= p.num_slots
                    ? -1 : (((slot >> p.log2_ps) * p.H) << p.log2_ps) + (slot & ps_mask);
    }
    for (int e = threadIdx.x * 8; e < p.H << log2_d; e += 256 * 8) {
        const long long head = (long long)(e >> log2_d) << p.log2_ps;
        uint4 x[kTokens];
#pragma unroll
        for (int i = 0; i < kTokens; ++i)
            if (at[i] >= 0) x[i] = __ldcs(reinterpret_cast<const uint4*>(src + (t0 + i) * stride + e));
#pragma unroll
        for (int i = 0; i < kTokens; ++i)
            if (at[i] >= 0)
                *reinterpret_cast<uint4*>(dst + ((at[i] + head) << log2_d) + (e & (p.d - 1))) = x[i];
    }
}

cudaError_t launch_cache_append_bf16(const AppendParams& p, cudaStream_t stream)
{
    // one token a CTA while that is what spreads the work, else four (one against four, us: 16
    // tokens 1.5 / 1.8, 256 1.7 / 1.8, 1024 of 16 heads 3.2 / 3.4, 2048 4.9 / 4.5, 8192 20.2 / 15.9)
    if (p.T <= 1024) cache_append_bf16_kernel<1><<<dim3(p.T, 2), 256, 0, stream>>>(p);
    else cache_append_bf16_kernel<4><<<dim3((unsigned)(((long long)p.T + 3) / 4), 2), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ 8-bit append
//
// A block is `block` consecutive slots of one page and head, with one scale.  A run is the
// call's tokens of one block (consecutive rows with consecutive slots); o is its first row
// inside the block.  Per run, head and tensor, with a = the largest finite |x| of the run:
//   need = a / top (IEEE fp32; the power-of-two format takes the next power of two)
//   old  = the block's scale if o > 0, else 0;   s = max(old, need)
//   o > 0 and s > old: rows 0 .. o-1 become  code((code * old) / s)
//   the run's rows become  code(x / s)           (a scale of 0 divides by 1: all zeros)
// where code() rounds to nearest even and saturates.  All divisions are IEEE fp32, so the
// bytes are a pure function of the inputs.
//
// A CTA takes the runs whose first token lies in its tile of packed tokens, for some of the
// heads of K and V, one after the other: a run is at most one block long, so the runs of a tile
// span at most tile + block - 1 tokens.  Row maxima are joined per run in shared memory (a
// maximum does not depend on the order), one thread per run settles the scale, and the rows
// are converted.  HBM-bound when it prefills: the rows stay in registers in between, 128 of
// them (what a tile holds unless short runs and one of a whole block meet in it; rows past
// that are read again).  The quotient is formed from the reciprocal with one residual
// correction, as in the block quantiser; values that this cannot take (infinities, scales
// near fp32's limits) go through the division itself.  A tile that is one run, as in a
// prefill, takes a path without per-row bookkeeping.  Measured: 31826 tokens of 16 heads,
// d 128, blocks of 128: 73.5 us = 5.3 TB/s read and written (the rows read twice and divided
// one by one 143, the bookkeeping of several runs for every tile 142).  The issue slots are 68 %
// busy (100 instructions per warp and 8 values a lane, half of them the quotients) and HBM 60
// %, in turns: a tile's loads, its maximum and its codes follow one another, four CTAs an SM.
// A step of 61 tokens takes 3.3 us, three dependent reads (slots, rows or scale, launch) long, and 6
// where one block in ten grows.
constexpr int kAppendWindow = 256;     // tokens a CTA looks at: tile + block - 1 < 256
constexpr int kAppendHeld = 128;       // rows held in registers

template <bool kE5M2>
__device__ __forceinline__ uint32_t pack4_fp8(float a, float b, float c, float d)
{
    const uint32_t lo = kE5M2 ? pack_e5m2x2(a, b) : pack_e4m3x2(a, b);
    const uint32_t hi = kE5M2 ? pack_e5m2x2(c, d) : pack_e4m3x2(c, d);
    return lo | (hi << 16);
}

// Two codes to two floats (exact).
template <bool kE5M2>
__device__ __forceinline__ float2 unpack2_fp8(uint32_t two)
{
    uint32_t h;
    if constexpr (kE5M2) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi) : "r"(h));
    return make_float2(lo, hi);
}

// Per half: the larger of two bf16 magnitudes (its sign is of no use), NaN if one is NaN.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// RN(x / s) of four values as codes, from their bf16 words, s and RN(1 / s).  The residual
// correction loses the sign of a zero; it is put back on the codes.
template <bool kE5M2>
__device__ __forceinline__ uint32_t quotient4(uint32_t a, uint32_t b, float s, float inv)
{
    const float2 neg = make_float2(-s, -s), y = make_float2(inv, inv);
    const float2 xa = make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
    const float2 xb = make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
    const float2 qa = __fmul2_rn(xa, y), qb = __fmul2_rn(xb, y);
    const float2 ca = __ffma2_rn(__ffma2_rn(qa, neg, xa), y, qa), cb = __ffma2_rn(__ffma2_rn(qb, neg, xb), y, qb);
    return pack4_fp8<kE5M2>(ca.x, ca.y, cb.x, cb.y) | (__byte_perm(a, b, 0x7531) & 0x80808080u);
}

// Eight codes by division, out of line: the rare runs that the reciprocal cannot take.
template <bool kE5M2>
__device__ __noinline__ uint2 divide8(uint4 w, float s)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        out[k] = pack4_fp8<kE5M2>(__fdiv_rn(__uint_as_float(u[2 * k] << 16), s),
                                  __fdiv_rn(__uint_as_float(u[2 * k] & 0xFFFF0000u), s),
                                  __fdiv_rn(__uint_as_float(u[2 * k + 1] << 16), s),
                                  __fdiv_rn(__uint_as_float(u[2 * k + 1] & 0xFFFF0000u), s));
    return make_uint2(out[0], out[1]);
}

// Codes of (code * old) / s, products and quotients IEEE fp32, for four codes.  The quotient by
// the reciprocal, corrected by its residual twice: after the first time it is within one ulp,
// where the residual is exact, and with y = RN(1 / s) the second correction rounds to the
// quotient itself (Markstein 1990).  Finite codes; 1e-24 < s < 1e30 keeps the residual of every
// quotient that is not rounded to 0 above fp32's smallest step.
template <bool kE5M2>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float old, float s, float y)
{
    const float2 o = make_float2(old, old), n = make_float2(-s, -s), y2 = make_float2(y, y);
    const float2 a = __fmul2_rn(unpack2_fp8<kE5M2>(w & 0xFFFFu), o), b = __fmul2_rn(unpack2_fp8<kE5M2>(w >> 16), o);
    float2 qa = __fmul2_rn(a, y2), qb = __fmul2_rn(b, y2);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        qa = __ffma2_rn(__ffma2_rn(qa, n, a), y2, qa);
        qb = __ffma2_rn(__ffma2_rn(qb, n, b), y2, qb);
    }
    return pack4_fp8<kE5M2>(qa.x, qa.y, qb.x, qb.y) | (w & 0x80808080u);
}

// Four codes by division: scales near fp32's limits, codes that are not finite.
template <bool kE5M2>
__device__ __noinline__ uint32_t redivide4(uint32_t w, float old, float s)
{
    const float2 a = unpack2_fp8<kE5M2>(w & 0xFFFFu), b = unpack2_fp8<kE5M2>(w >> 16);
    return pack4_fp8<kE5M2>(__fdiv_rn(a.x * old, s), __fdiv_rn(a.y * old, s), __fdiv_rn(b.x * old, s),
                            __fdiv_rn(b.y * old, s));
}

// The earlier rows (n pieces of 16 codes) of a block whose scale grew from old to s, by the
// CTA; out of line: few blocks grow.  (A warp a block, four codes a lane and IEEE divisions, took
// 346 us where every block of 64 tokens and 8 heads grew under 60 rows; a code of 0 alone sends a
// division down its long path.)
template <bool kE5M2>
__device__ __noinline__ void requantise(uint4* codes, int n, float old, float s)
{
    const float y = s > 1e-24f && s < 1e30f ? __frcp_rn(s) : 0.0f;
    for (int at = threadIdx.x; at < n; at += blockDim.x) {
        const uint4 u = codes[at];
        uint32_t w[4] = {u.x, u.y, u.z, u.w}, odd = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            odd |= kE5M2 ? (w[k] & 0x7C7C7C7Cu) + 0x04040404u : (w[k] & 0x7F7F7F7Fu) + 0x01010101u;
        if (y == 0.0f || (odd & 0x80808080u)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = redivide4<kE5M2>(w[k], old, s);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = rescale4<kE5M2>(w[k], old, s, y);
        }
        codes[at] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int D> struct AppendCfg {
    static constexpr int LPR = D / 8;                       // lanes of a row, 8 values each
    static constexpr int THREADS = D == 256 ? 512 : 256;
    static constexpr int RPP = THREADS / LPR;               // rows of a pass
    static constexpr int HELD = kAppendHeld / RPP;          // passes whose rows stay in registers
};

template <int D, bool kE5M2>
__global__ void __launch_bounds__(AppendCfg<D>::THREADS, D == 256 ? 2 : 4)
    cache_append_fp8_kernel(const AppendParams p)
{
    using C = AppendCfg<D>;
    __shared__ long long slots[kAppendWindow];
    __shared__ int run_of[kAppendWindow];            // window index of the token's run, or -1
    __shared__ unsigned run_max[kAppendWindow];      // bits of the run's largest finite |x|
    __shared__ float run_scale[kAppendWindow], run_old[kAppendWindow];
    __shared__ float run_inv[kAppendWindow];         // 1 / scale, or 0: divide
    __shared__ int run_odd[kAppendWindow];           // the run has a value that is not finite
    __shared__ int grown[kAppendWindow];
    __shared__ int num_grown[2], warp_last[kAppendWindow / 32], first_row, end_row;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int block = 1 << p.log2_blk, tile = p.tile, ps_mask = (1 << p.log2_ps) - 1;
    const long long t0 = (long long)blockIdx.x * tile;
    const int window = (int)min((long long)(tile + block - 1), p.T - t0);

    auto slot_at = [&](long long t) -> long long {
        const long long s = __ldg(p.slot_map + t);
        return s >= 0 && s < p.num_slots ? s : -1;
    };
    // heads of runs, then the nearest head at or before each token
    int last = -1;
    long long slot = -1;
    if (tid < kAppendWindow) {
        long long before = -1;
        if (tid < window) {
            slot = slot_at(t0 + tid);
            if (t0 + tid > 0) before = slot_at(t0 + tid - 1);
        }
        const bool head = slot >= 0 && (before < 0 || slot != before + 1 || (slot & (block - 1)) == 0);
        last = head ? tid : -1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, last, o);
            if (lane >= o) last = max(last, y);
        }
        if (lane == 31) warp_last[warp] = last;
        if (tid == 0) {
            first_row = kAppendWindow;
            end_row = 0;
        }
        slots[tid] = slot;
    }
    __syncthreads();
    if (tid < kAppendWindow) {
        for (int w = 0; w < warp; ++w) last = max(last, warp_last[w]);
        const int run = slot >= 0 && last < tile ? last : -1;
        run_of[tid] = run;
        run_max[tid] = 0;
        run_odd[tid] = 0;
        const unsigned mine = __ballot_sync(0xffffffffu, run >= 0);
        if (lane == 0 && mine) {
            atomicMin(&first_row, tid + __ffs(mine) - 1);
            atomicMax(&end_row, tid + 32 - __clz(mine));
        }
    }
    if (tid == 0) num_grown[0] = 0;
    __syncthreads();
    const int begin = first_row, end = end_row;
    if (end <= begin) return;
    const int c = tid % C::LPR, row_in_pass = tid / C::LPR;
    // eight values' largest magnitude as bf16 bits, and the largest finite one
    auto largest = [](const uint4& w) -> uint32_t {
        const uint32_t m2 = max_abs_bf16x2(max_abs_bf16x2(w.x, w.y), max_abs_bf16x2(w.z, w.w));
        return max(m2 & 0x7FFFu, (m2 >> 16) & 0x7FFFu);
    };
    auto largest_finite = [](const uint4& w) -> uint32_t {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if ((u[i] & 0x7FFFu) < 0x7F80u) m = max(m, u[i] & 0x7FFFu);
            if (((u[i] >> 16) & 0x7FFFu) < 0x7F80u) m = max(m, (u[i] >> 16) & 0x7FFFu);
        }
        return m;
    };
    const bool single = run_of[begin] == run_of[end - 1] && end - begin <= kAppendHeld;   // one run: a prefill's tile

    for (int item = blockIdx.y, odd = 0; item < 2 * p.H; item += gridDim.y, odd ^= 1) {
        const int h = item >> 1, z = item & 1;
        auto row_address = [&](long long s) {
            return ((((s >> p.log2_ps) * p.H + h) << p.log2_ps) + (s & ps_mask)) * D;
        };
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(z ? p.v : p.k) + h * D + c * 8;
        const long long stride = z ? p.v_stride : p.k_stride;
        uint8_t* cache = static_cast<uint8_t*>(z ? p.vc : p.kc);
        float* scales = z ? p.vs : p.ks;
        auto load = [&](int i) { return __ldg(reinterpret_cast<const uint4*>(src + (t0 + i) * stride)); };
        auto run_at = [&](int i) { return i < end ? run_of[i] : -1; };
        auto join = [&](int run, const uint4& w) {
            uint32_t a = run >= 0 ? largest(w) : 0u;
            if (a >= 0x7F80u) {
                a = largest_finite(w);
                run_odd[run] = 1;
            }
            const unsigned row_lanes = C::LPR == 32 ? 0xffffffffu : ((1u << C::LPR) - 1) << (lane & ~(C::LPR - 1));
            a = __reduce_max_sync(row_lanes, a);
            if (run >= 0 && c == 0) atomicMax(&run_max[run], a << 16);
        };
        // a run's first thread: where its scale is, read while the rows arrive
        float* sc = nullptr;
        float old = 0.0f;
        if (tid < tile && run_of[tid] == tid) {
            const long long s0 = slots[tid];
            sc = scales + ((((s0 >> p.log2_ps) * p.H + h) << (p.log2_ps - p.log2_blk)) +
                           ((s0 & ps_mask) >> p.log2_blk));
            if ((s0 & (block - 1)) > 0) old = *sc;
        }
        uint4 x[C::HELD];
        auto load_rows = [&](int from) {             // 128 rows, their loads in flight together
#pragma unroll
            for (int k = 0; k < C::HELD; ++k) {
                if (from - row_in_pass + k * C::RPP >= end) break;   // a small step's few rows: one pass
                const int i = from + k * C::RPP;
                x[k] = make_uint4(0, 0, 0, 0);
                if (run_at(i) >= 0) x[k] = load(i);
            }
        };
        const int row0 = begin + row_in_pass;
        if (single) {
            const __nv_bfloat16* from = src + (t0 + row0) * stride;
            const long long step = C::RPP * stride;
#pragma unroll
            for (int k = 0; k < C::HELD; ++k) {
                x[k] = make_uint4(0, 0, 0, 0);
                if (row0 + k * C::RPP < end) x[k] = __ldcs(reinterpret_cast<const uint4*>(from + k * step));
            }
            uint32_t m2 = 0;
#pragma unroll
            for (int k = 0; k < C::HELD; ++k)
                m2 = max_abs_bf16x2(m2, max_abs_bf16x2(max_abs_bf16x2(x[k].x, x[k].y), max_abs_bf16x2(x[k].z, x[k].w)));
            uint32_t a = max(m2 & 0x7FFFu, (m2 >> 16) & 0x7FFFu);
            if (a >= 0x7F80u) {
                a = 0;
#pragma unroll
                for (int k = 0; k < C::HELD; ++k) a = max(a, largest_finite(x[k]));
                run_odd[run_of[begin]] = 1;
            }
            a = __reduce_max_sync(0xffffffffu, a);
            if (lane == 0) atomicMax(&run_max[run_of[begin]], a << 16);
        } else {
            for (int from = row0; from - row_in_pass < end; from += kAppendHeld) {
                load_rows(from);
#pragma unroll
                for (int k = 0; k < C::HELD; ++k) {
                    if (from - row_in_pass + k * C::RPP >= end) break;
                    join(run_at(from + k * C::RPP), x[k]);
                }
            }
        }
        __syncthreads();
        if (sc) {
            const int row = (int)(slots[tid] & (block - 1));
            const bool finite = run_odd[tid] == 0;
            float need = __fdiv_rn(__uint_as_float(run_max[tid]), kE5M2 ? 57344.0f : 448.0f);
            if (p.pow2) need = pow2_at_least(need);
            const float s = fmaxf(old, need);
            run_old[tid] = old;
            run_scale[tid] = s > 0.0f ? s : 1.0f;
            run_inv[tid] = finite && s > 1e-30f && s < 1e30f ? __frcp_rn(s) : 0.0f;
            if (row == 0 || s > old) *sc = s;
            if (row > 0 && s > old) grown[atomicAdd(&num_grown[odd], 1)] = tid;
            run_max[tid] = 0;                        // for the next head
            run_odd[tid] = 0;
        }
        __syncthreads();
        if (tid == 0) num_grown[odd ^ 1] = 0;
        auto write = [&](uint8_t* to, float s, float inv, const uint4& w) {
            if (inv == 0.0f) {
                *reinterpret_cast<uint2*>(to) = divide8<kE5M2>(w, s);
                return;
            }
            *reinterpret_cast<uint2*>(to) =
                make_uint2(quotient4<kE5M2>(w.x, w.y, s, inv), quotient4<kE5M2>(w.z, w.w, s, inv));
        };
        if (single) {                                // the run's rows follow one another in the cache
            const int run = run_of[begin];
            const float s = run_scale[run], inv = run_inv[run];
            uint8_t* to = cache + row_address(slots[run]) + row_in_pass * D + c * 8;
#pragma unroll
            for (int k = 0; k < C::HELD; ++k)
                if (row0 + k * C::RPP < end) write(to + k * C::RPP * D, s, inv, x[k]);
        } else {
            const int held = (end - begin - 1) / kAppendHeld * kAppendHeld;   // the rows loaded last
            for (int from = held; from >= 0; from -= kAppendHeld) {
                if (from != held) load_rows(row0 + from);
#pragma unroll
                for (int k = 0; k < C::HELD; ++k) {
                    if (begin + from + k * C::RPP >= end) break;
                    const int i = row0 + from + k * C::RPP, run = run_at(i);
                    if (run >= 0) write(cache + row_address(slots[i]) + c * 8, run_scale[run], run_inv[run], x[k]);
                }
            }
        }
        // blocks whose scale grew: their earlier rows
        for (int k = 0; k < num_grown[odd]; ++k) {
            const int run = grown[k];
            const int row = (int)(slots[run] & (block - 1));
            requantise<kE5M2>(reinterpret_cast<uint4*>(cache + row_address(slots[run] - row)), row * (D / 16),
                              run_old[run], run_scale[run]);
        }
    }
}

template <int D>
static cudaError_t launch_append_fp8_d(AppendParams p, bool e5m2, cudaStream_t stream)
{
    const int block = 1 << p.log2_blk;
    // small steps take small tiles while the grid is one wave: a tile's tokens are mostly runs of
    // their own, whose blocks may each have earlier rows to requantise (64 tokens of 8 heads, every
    // block growing under 60 rows: 64 tokens a tile 27, 8 11.8, 4 9.0 us; one in ten 15, 7.3, 6.8;
    // none 5.1, 4.1, 4.2)
    int tile = 8;
    while (tile < 64 && ((long long)p.T + tile - 1) / tile * 2 * p.H > 4LL * p.sm_count) tile *= 2;
    if (tile == 64 && block > 64) tile = block;
    p.tile = tile;
    const long long tiles = ((long long)p.T + tile - 1) / tile;
    // a head of K or V per CTA while there are few, else about 36 CTAs per SM, each with
    // several of its tile's heads (31826 tokens of 16 heads, d 128: 8 per SM 103.0 us, 12 90.6,
    // 24 78.1, 36 73.2, 60 76.5)
    const long long groups = (36LL * p.sm_count + tiles - 1) / tiles;
    const dim3 grid((unsigned)tiles, groups < 2 * p.H ? (unsigned)groups : 2 * p.H);
    constexpr int threads = AppendCfg<D>::THREADS;
    if (e5m2) cache_append_fp8_kernel<D, true><<<grid, threads, 0, stream>>>(p);
    else cache_append_fp8_kernel<D, false><<<grid, threads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_cache_append_fp8(const AppendParams& p, bool e5m2, cudaStream_t stream)
{
    switch (p.d) {
    case 64: return launch_append_fp8_d<64>(p, e5m2, stream);
    case 128: return launch_append_fp8_d<128>(p, e5m2, stream);
    case 256: return launch_append_fp8_d<256>(p, e5m2, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gb300
