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
// of the ends; a page that the step takes is read from the free stack, never from the
// table entry another thread writes.
constexpr int kPlanMaxThreads = 1024;

__device__ __forceinline__ long long plan_block_scan(long long x, long long* warp_sum, long long* total)
{
    // exclusive sum over the block's threads; every thread calls it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();   // the previous scan's warp sums have been read
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
        const long long s = warp_sum[w];
        if (w < warp) before += s;
        all += s;
    }
    *total = all;
    return before + inc - x;
}

// The last index i in [0, n) with a[i] <= x, for a non-decreasing with a[0] <= x.
__device__ __forceinline__ int last_not_above(const int* a, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanMaxThreads) paged_plan_kernel(const PlanParams p)
{
    extern __shared__ int sm_plan[];
    __shared__ long long warp_sum[kPlanMaxThreads / 32];
    int* start = sm_plan;               // first packed row of the request, at most num_tokens
    int* base = sm_plan + p.B;          // pages taken before it
    int* len = sm_plan + 2 * p.B;       // cached length, or its complement when not served
    const cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, nt = blockDim.x;
    const int ps = 1 << p.log2_ps;
    const long long cap = (long long)p.max_pages << p.log2_ps;   // fits an int
    const int free = min(max(*p.free_count, 0), p.free_capacity);
    const int per = (p.B + nt - 1) / nt, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);

    auto request = [&](int b, long long& n, int& L) {
        n = max(p.new_lens[b], 0);
        L = (int)min((long long)max(p.seq_lens[b], 0), cap);
    };
    long long n, tokens = 0, total, taken_all;
    int L;
    for (int b = b0; b < b1; ++b) {
        request(b, n, L);
        tokens += n;
    }
    const long long first = plan_block_scan(tokens, warp_sum, &total);
    auto pages_needed = [&](long long end, long long nn, int LL) -> long long {
        if (LL + nn > cap || end > p.num_tokens) return -1;      // does not fit
        return ((LL + nn + ps - 1) >> p.log2_ps) - ((LL + ps - 1) >> p.log2_ps);
    };
    long long need_sum = 0, end = first;
    for (int b = b0; b < b1; ++b) {
        request(b, n, L);
        end += n;
        const long long need = pages_needed(end, n, L);
        need_sum += need > 0 ? need : 0;
    }
    const long long need_first = plan_block_scan(need_sum, warp_sum, &taken_all);
    long long at = need_first, granted = 0;
    end = first;
    for (int b = b0; b < b1; ++b) {
        request(b, n, L);
        start[b] = (int)min(end, (long long)p.num_tokens);
        end += n;
        const long long need = pages_needed(end, n, L);
        const bool ok = need == 0 || (need > 0 && at + need <= free);
        base[b] = (int)min(at, 0x7fffffffLL);
        len[b] = ok ? L : ~L;
        if (need > 0) {
            at += need;
            if (ok) granted += need;
        }
    }
    long long taken;
    plan_block_scan(granted, warp_sum, &taken);   // also: every thread's entries are written
    __syncthreads();
    cluster.sync();                               // every CTA has read the lengths

    const int rank = (int)cluster.block_rank() * nt + tid, threads = (int)cluster.num_blocks() * nt;
    const int rows = (int)min(total, (long long)p.num_tokens);   // packed rows in use
    for (int b = rank; b < p.B; b += threads) {
        const int next = b + 1 < p.B ? start[b + 1] : rows;
        const bool ok = len[b] >= 0;
        p.cu_new[b] = start[b];
        if (b == p.B - 1) p.cu_new[p.B] = rows;
        p.served[b] = ok ? 1 : 0;
        p.seq_lens_out[b] = ok ? len[b] + (next - start[b]) : ~len[b];
    }
    if (rank == 0) *p.free_count_out = free - (int)taken;
    for (int k = rank; k < (int)taken; k += threads) {
        const int b = last_not_above(base, p.B, k);
        const int page = ((len[b] + ps - 1) >> p.log2_ps) + k - base[b];
        p.page_table[(size_t)b * p.max_pages + page] = p.free_pages[free - 1 - k];
    }
    for (int t = rank; t < p.num_tokens; t += threads) {
        long long slot = -1;
        int pos = -1;
        if (t < rows) {
            const int b = last_not_above(start, p.B, t);
            if (len[b] >= 0) {
                pos = len[b] + t - start[b];
                const int page = pos >> p.log2_ps, old = (len[b] + ps - 1) >> p.log2_ps;
                const int id = page < old ? p.page_table[(size_t)b * p.max_pages + page]
                                          : p.free_pages[free - 1 - (base[b] + page - old)];
                slot = id < 0 ? -1 : ((long long)id << p.log2_ps) + (pos & (ps - 1));
            }
        }
        p.slot_map[t] = slot;
        p.positions[t] = pos;
    }
}

cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t stream)
{
    const int smem = 3 * p.B * (int)sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         200 * 1024);
    if (e != cudaSuccess) return e;
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
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, p);
}

// ------------------------------------------------------------------ bf16 append
//
// cache[slot / ps][h][slot % ps] = row (t, h), 16 bytes a thread; slots outside the cache
// (padding) are skipped.  HBM-bound: each row is read once and written once.
__global__ void __launch_bounds__(256) cache_append_bf16_kernel(const AppendParams p)
{
    const int chunks = p.d / 8;                    // 16-byte pieces of a row
    const long long total = (long long)p.T * p.H * chunks;
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= total) return;
    const int c = (int)(idx % chunks);
    const long long row = idx / chunks;
    const int t = (int)(row / p.H), h = (int)(row - (long long)t * p.H);
    const long long slot = p.slot_map[t];
    if (slot < 0 || slot >= p.num_slots) return;
    const bool is_v = blockIdx.y != 0;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) +
                               (long long)t * (is_v ? p.v_stride : p.k_stride) + h * p.d + c * 8;
    const long long to = ((((slot >> p.log2_ps) * p.H + h) << p.log2_ps) + (slot & ((1 << p.log2_ps) - 1))) * p.d;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.vc : p.kc) + to + c * 8) =
        *reinterpret_cast<const uint4*>(src);
}

cudaError_t launch_cache_append_bf16(const AppendParams& p, cudaStream_t stream)
{
    const long long total = (long long)p.T * p.H * (p.d / 8);
    cache_append_bf16_kernel<<<dim3((unsigned)((total + 255) / 256), 2), 256, 0, stream>>>(p);
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
// A CTA takes the runs whose first token lies in its tile of packed tokens, for one head
// of K or V: a run is at most one block long, so it reads at most tile + block - 1 tokens.
// First pass: row maxima, joined per run in shared memory (a maximum does not depend on
// the order).  Then one thread per run settles the scale, and the second pass reads the
// rows again (from L1 or L2) and writes the codes.
constexpr int kAppendThreads = 256;
constexpr int kAppendWindow = 256;     // tokens a CTA looks at: tile + block - 1 < 256

__device__ __forceinline__ float append_pow2_at_least(float s)
{
    const uint32_t b = __float_as_uint(s);
    if ((b & 0x7F800000u) == 0) {      // zero or subnormal
        const uint32_t m = b & 0x7FFFFFu;
        return __uint_as_float((m & (m - 1)) == 0 ? m : (1u << (32 - __clz(m))));
    }
    return (b & 0x7FFFFFu) == 0 ? s : __uint_as_float((b & 0x7F800000u) + 0x00800000u);
}

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

template <int D, bool kE5M2>
__global__ void __launch_bounds__(kAppendThreads) cache_append_fp8_kernel(const AppendParams p)
{
    constexpr int LPR = D / 8;                       // lanes of a row, 8 values each
    constexpr int RPP = kAppendThreads / LPR;        // rows of a pass
    __shared__ long long slots[kAppendWindow];
    __shared__ int run_of[kAppendWindow];            // window index of the token's run, or -1
    __shared__ unsigned run_max[kAppendWindow];      // bits of the run's largest |x|
    __shared__ float run_scale[kAppendWindow], run_old[kAppendWindow];
    __shared__ int grown[kAppendWindow];
    __shared__ int num_grown, warp_last[kAppendThreads / 32], num_rows;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int block = 1 << p.log2_blk, tile = block < 64 ? 64 : block;
    const int h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const long long t0 = (long long)blockIdx.x * tile;
    const int window = (int)min((long long)(tile + block - 1), p.T - t0);

    auto slot_at = [&](long long t) -> long long {
        const long long s = p.slot_map[t];
        return s >= 0 && s < p.num_slots ? s : -1;
    };
    // heads of runs, then the nearest head at or before each token
    {
        const int i = tid;
        long long s = -1, before = -1;
        if (i < window) {
            s = slot_at(t0 + i);
            if (t0 + i > 0) before = slot_at(t0 + i - 1);
        }
        const bool head = s >= 0 && (before < 0 || s != before + 1 || (s & (block - 1)) == 0);
        int last = head ? i : -1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, last, o);
            if (lane >= o) last = max(last, y);
        }
        if (lane == 31) warp_last[warp] = last;
        if (tid == 0) {
            num_grown = 0;
            num_rows = 0;
        }
        run_max[i] = 0;
        slots[i] = s;
        __syncthreads();
        for (int w = 0; w < warp; ++w) last = max(last, warp_last[w]);
        const int run = s >= 0 && last < tile ? last : -1;
        run_of[i] = run;
        if (run >= 0) atomicMax(&num_rows, i + 1);
        __syncthreads();
    }
    const int rows = num_rows;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) + h * D;
    const long long stride = is_v ? p.v_stride : p.k_stride;
    uint8_t* cache = static_cast<uint8_t*>(is_v ? p.vc : p.kc);
    float* scales = is_v ? p.vs : p.ks;
    const int c = tid % LPR;
    auto load = [&](int i, float (&x)[8]) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + (t0 + i) * stride + c * 8);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(u[e] << 16);
            x[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
        }
    };
    auto row_address = [&](long long slot) {
        return ((((slot >> p.log2_ps) * p.H + h) << p.log2_ps) + (slot & ((1 << p.log2_ps) - 1))) * D;
    };
    for (int i0 = 0; i0 < rows; i0 += RPP) {
        const int i = i0 + tid / LPR;
        const int run = i < rows ? run_of[i] : -1;
        float a = 0.0f;
        if (run >= 0) {
            float x[8];
            load(i, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float m = fabsf(x[e]);
                a = fmaxf(a, m < __int_as_float(0x7f800000) ? m : 0.0f);   // finite values only
            }
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        if (run >= 0 && c == 0) atomicMax(&run_max[run], __float_as_uint(a));
    }
    __syncthreads();
    if (tid < tile && run_of[tid] == tid) {
        const long long slot = slots[tid];
        const int row = (int)(slot & (block - 1));
        float* sc = scales + ((((slot >> p.log2_ps) * p.H + h) << (p.log2_ps - p.log2_blk)) +
                              ((slot & ((1 << p.log2_ps) - 1)) >> p.log2_blk));
        float need = __fdiv_rn(__uint_as_float(run_max[tid]), kE5M2 ? 57344.0f : 448.0f);
        if (p.pow2) need = append_pow2_at_least(need);
        const float old = row > 0 ? *sc : 0.0f;
        const float s = fmaxf(old, need);
        run_old[tid] = old;
        run_scale[tid] = s;
        if (row == 0 || s > old) *sc = s;
        if (row > 0 && s > old) grown[atomicAdd(&num_grown, 1)] = tid;
    }
    __syncthreads();
    for (int i0 = 0; i0 < rows; i0 += RPP) {
        const int i = i0 + tid / LPR;
        const int run = i < rows ? run_of[i] : -1;
        if (run < 0) continue;
        float x[8];
        load(i, x);
        const float s = run_scale[run] > 0.0f ? run_scale[run] : 1.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(x[e], s);
        *reinterpret_cast<uint2*>(cache + row_address(slots[i]) + c * 8) =
            make_uint2(pack4_fp8<kE5M2>(x[0], x[1], x[2], x[3]), pack4_fp8<kE5M2>(x[4], x[5], x[6], x[7]));
    }
    // blocks whose scale grew: their earlier rows, one warp a block
    for (int g = warp; g < num_grown; g += kAppendThreads / 32) {
        const int run = grown[g];
        const long long slot = slots[run];
        const int row = (int)(slot & (block - 1));
        const float old = run_old[run], s = run_scale[run];
        uint32_t* base = reinterpret_cast<uint32_t*>(cache + row_address(slot - row));
        for (int w = lane; w < row * (D / 4); w += 32) {
            const uint32_t codes = base[w];
            const float2 a = unpack2_fp8<kE5M2>(codes & 0xFFFFu), b = unpack2_fp8<kE5M2>(codes >> 16);
            base[w] = pack4_fp8<kE5M2>(__fdiv_rn(a.x * old, s), __fdiv_rn(a.y * old, s),
                                       __fdiv_rn(b.x * old, s), __fdiv_rn(b.y * old, s));
        }
    }
}

template <int D>
static cudaError_t launch_append_fp8_d(const AppendParams& p, bool e5m2, cudaStream_t stream)
{
    const int block = 1 << p.log2_blk, tile = block < 64 ? 64 : block;
    const dim3 grid((unsigned)((p.T + tile - 1) / tile), p.H, 2);
    if (e5m2) cache_append_fp8_kernel<D, true><<<grid, kAppendThreads, 0, stream>>>(p);
    else cache_append_fp8_kernel<D, false><<<grid, kAppendThreads, 0, stream>>>(p);
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
