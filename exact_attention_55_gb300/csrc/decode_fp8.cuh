// decode_fp8.cuh -- what the two decoding kernels over an 8-bit paged cache share: how the
// work is cut into ranges, how a CTA walks its range, conversions, and the joining of parts.
//
// The tiles (TILE keys of one key head) of all sequences form one line that is cut into
// equal ranges, one per resident CTA, so a ragged batch and a single long sequence both keep
// every SM busy to the end.  A unit (sequence, key head) counts a few tiles more than it has,
// what starting and ending it costs.  A range may end inside a unit; its part (O not yet
// divided, the weights' bases, sums) then goes to the workspace, and decode_fp8_combine_kernel,
// launched as a dependent of the main grid, joins a unit's parts.
//
// Both grids may start before the one ahead of them has ended, and what that one writes (the
// queries, a cache, lengths, parts) is theirs to read after griddepcontrol.wait.  Such data changes
// while the grid runs, which the non-coherent path (__ldg, ld.global.nc) does not allow: all
// their loads are plain ones, behind the wait (dec8_ld).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "attn_params.h"
#include "paged_params.h"
#include "ptx.cuh"

namespace gb300 {

// Tiles a unit's start and end are worth (48 ragged sequences of 8 key heads: 1 36.1, 2 34.6,
// 4 35.3, 6 35.7, 10 37.7 us; 32 windowed heads 23.8, 22.9, 21.2, 22.3, 23.0).
constexpr int kD8UnitCost = 4;
constexpr int kD8CombineThreads = 128, kD8CombineFew = 8;

// Weights are stored in fp16 relative to a base that lies kD8Room (log2) under the row's largest
// when it is set, and is set again when a key passes that largest by more than kD8Tau: a stored
// weight w f is below 2^(6 + 7) * 4 = 2^15, and fp16's smallest step lies 2^-30 under the
// largest weight.  (With the base at the largest itself, 2^-24: beside one heavy key without a
// value, 131072 light ones of 2^-25 each, 0.4 % of O, were lost, at 2^-24.4 they counted a third too much.)
constexpr float kD8Room = 6.0f, kD8Tau = 7.0f;

// Floats of a part: O [rows][d], bases [rows], sums [rows].
__host__ __device__ constexpr int dec8_part(int rows, int d) { return rows * (d + 2); }

// A plain load that stays behind the waits written before it and, unlike a dereference, is not
// ordered with the stores and barriers around it (32 rows, d 128: 74.1 us by dereferences, 67.8 so).
__device__ __forceinline__ int dec8_ld(const int* a)
{
    int v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(a));
    return v;
}

__device__ __forceinline__ uint4 dec8_ld(const uint4* a)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(a));
    return v;
}

// Tiles of a sequence: [t0, t0 + n), of whose keys lo .. L-1 may be seen.
struct Dec8Seq {
    int L, lo, t0, n;
};

template <int TILE>
__device__ __forceinline__ Dec8Seq dec8_seq(const DecodeFp8Params& p, int b)
{
    Dec8Seq s;
    s.L = min(max(dec8_ld(p.seq_lens + b), 0), p.max_pages << p.log2_ps);
    s.lo = p.window > 0 ? max(0, s.L - p.nq - p.window) : 0;
    s.t0 = s.lo / TILE;
    s.n = (int)(((unsigned)s.L + TILE - 1) / TILE) - s.t0;
    return s;
}

// a / b for a >= 0 and 0 < b < 2^32, in 32 bits where a fits (the usual case, a third of the time).
__device__ __forceinline__ long long dec8_div(long long a, long long b)
{
    if ((a >> 32) == 0) return (unsigned)a / (unsigned)b;
    return a / b;
}

// The line: `tiles` in all, `cost` long; a unit of n tiles covers n + unit_cost of it, its
// tiles at the end; range x is [cut(x), cut(x + 1)) of X.  Where units are not split
// (p.whole) each counts as one tile.
struct Dec8Line {
    long long tiles, cost, X;
    int unit_cost;

    __device__ __forceinline__ Dec8Line(const DecodeFp8Params& p, long long seq_tiles, long long seqs)
    {
        tiles = seq_tiles * p.Hkv;
        unit_cost = tiles <= p.ranges ? 0 : kD8UnitCost;   // few tiles: one per range
        cost = tiles + seqs * p.Hkv * unit_cost;
        X = tiles < p.ranges ? tiles : p.ranges;
    }
    __device__ __forceinline__ long long cut(int x) const { return dec8_div(x * cost, X); }
    __device__ __forceinline__ int owner(long long at) const { return (int)(((at + 1) * X - 1) / cost); }
};

__device__ __forceinline__ int dec8_span(const DecodeFp8Params& p, int n) { return p.whole ? min(n, 1) : n; }

// What the set-up leaves in shared memory.
template <int THREADS>
struct Dec8Setup {
    long long sum[THREADS / 32];       // tiles and sequences of each warp's share
    long long first;                   // cost before sequence b0
    int b0;                            // the sequence that the range starts in
};

// The line, and the sequence that range x starts in.  All threads call it.
template <int TILE, int THREADS>
__device__ __forceinline__ Dec8Line dec8_line(const DecodeFp8Params& p, Dec8Setup<THREADS>& sh, int x)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    if (tid == 0) {                    // lengths that change under the call find no start: stay inside
        sh.b0 = 0;
        sh.first = 0;
    }
    // tiles in the lower 44 bits (at most 2^25 a sequence), sequences that have any above
    constexpr int shift = 44;
    constexpr long long mask = (1LL << shift) - 1;
    long long both = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = dec8_span(p, dec8_seq<TILE>(p, b).n);
        both += n + ((long long)(n > 0) << shift);
    }
    long long inc = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sh.sum[warp] = inc;
    __syncthreads();
    long long before2 = inc - both, total2 = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before2 += sh.sum[w];
        total2 += sh.sum[w];
    }
    const long long mine = both & mask, seqs = both >> shift, before = before2 & mask, before_s = before2 >> shift;
    const Dec8Line line(p, total2 & mask, total2 >> shift);
    if (x < line.X) {
        const long long at = line.cut(x);
        long long s0 = (before + before_s * line.unit_cost) * p.Hkv;
        if (s0 <= at && at < s0 + (mine + seqs * line.unit_cost) * p.Hkv)
            for (int b = b0; b < b1; ++b) {
                const int n = dec8_span(p, dec8_seq<TILE>(p, b).n);
                const long long len = n > 0 ? (long long)(n + line.unit_cost) * p.Hkv : 0;
                if (s0 <= at && at < s0 + len) {
                    sh.b0 = b;
                    sh.first = s0;
                }
                s0 += len;
            }
    }
    __syncthreads();
    return line;
}

// A CTA's walk over its range: unit (b, hk), which starts `at` behind the range's start (or
// before it: negative), and the unit's tiles that are this range's, [k0, k1).  A range is
// taken as at most 2^30 long (2^36 keys).  Lengths that change under the call can lead it
// astray, but not out of the tensors.
template <int TILE>
struct Dec8Walk {
    Dec8Seq seq;
    int len, at, b, hk, span, unit_cost, k0, k1;
    bool more;

    template <int THREADS>
    __device__ __forceinline__ Dec8Walk(const DecodeFp8Params& p, const Dec8Line& line, const Dec8Setup<THREADS>& sh, int x)
        : b(sh.b0), unit_cost(line.unit_cost)
    {
        const long long a = line.cut(x);
        len = (int)min(line.cut(x + 1) - a, 1LL << 30);
        seq = dec8_seq<TILE>(p, b);
        span = dec8_span(p, seq.n);
        hk = (int)min((unsigned)dec8_div(a - sh.first, span + unit_cost), (unsigned)(p.Hkv - 1));
        at = (int)(sh.first + (long long)hk * (span + unit_cost) - a);
        take(p);
        more = k1 > k0 || next(p);
    }
    __device__ __forceinline__ void take(const DecodeFp8Params& p)
    {
        k0 = max(0, -at - unit_cost);
        k1 = max(k0, min(span, len - at - unit_cost));
        if (p.whole && k1 > k0) k1 = seq.n;
    }
    // to the next unit with tiles of this range; false, and the end of the walk, if there is none
    __device__ __forceinline__ bool next(const DecodeFp8Params& p)
    {
        do {
            at += span + unit_cost;
            if (at + unit_cost >= len) return more = false;
            if (++hk == p.Hkv) {
                hk = 0;
                do {
                    b = min(b + 1, p.B - 1);
                    seq = dec8_seq<TILE>(p, b);
                } while (seq.n == 0 && b < p.B - 1);
                span = dec8_span(p, seq.n);
            }
            take(p);
        } while (k1 <= k0 && span > 0);
        return more = k1 > k0;
    }
    __device__ __forceinline__ bool whole() const { return k1 - k0 == seq.n; }
    // the range that has the unit's last tile, as range x sees it
    __device__ __forceinline__ int last_owner(const Dec8Line& line, int x) const
    {
        return line.owner(line.cut(x) + at + unit_cost + seq.n - 1);
    }
};

// What the combine kernel finds at the workspace's start: an entry per unit (and row group),
// or where there are more units than CTAs one per CTA, for the one unit that it may begin and
// not end.  (first range, last range, row group, first row), or a negative first range.
__device__ __forceinline__ bool dec8_per_unit(const DecodeFp8Params& p)
{
    return (long long)p.B * p.Hkv * p.row_groups <= p.ranges * p.row_groups;
}

template <int TILE>
__device__ __forceinline__ void dec8_name_parts(const DecodeFp8Params& p, const Dec8Walk<TILE>& w, const Dec8Line& line,
                                                int x, int rg, size_t unit_row)
{
    if (w.k0 != 0 || p.whole) return;
    const bool per_unit = dec8_per_unit(p);
    if (!per_unit && w.whole()) return;
    reinterpret_cast<int4*>(p.ws)[per_unit ? (w.b * p.Hkv + w.hk) * p.row_groups + rg : blockIdx.x] =
        w.whole() ? make_int4(-1, 0, 0, 0) : make_int4(x, w.last_owner(line, x), rg, (int)unit_row);
}

// This CTA's part of the unit it is on.
template <int ROWS, int D>
__device__ __forceinline__ float* dec8_my_part(const DecodeFp8Params& p, bool first)
{
    return p.ws + 4 * (size_t)(p.ranges * p.row_groups) + (size_t)(2 * blockIdx.x + (first ? 1 : 0)) * dec8_part(ROWS, D);
}

// Sequences without a key: O = 0, LSE = -inf, nothing to join.  The CTAs share them.
template <int TILE, int D>
__device__ __forceinline__ void dec8_write_empty(const DecodeFp8Params& p, int threads)
{
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (dec8_seq<TILE>(p, b).n > 0) continue;
        const size_t r0 = (size_t)b * p.Hkv * p.rows, rows = (size_t)p.Hkv * p.rows;
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + r0 * D);
        for (size_t i = threadIdx.x; i < rows * (D / 8); i += threads) o[i] = make_uint4(0, 0, 0, 0);
        for (size_t i = threadIdx.x; i < rows; i += threads) p.lse[r0 + i] = -__int_as_float(0x7f800000);
        if (dec8_per_unit(p))
            for (int i = threadIdx.x; i < p.Hkv * p.row_groups; i += threads)
                reinterpret_cast<int4*>(p.ws)[b * p.Hkv * p.row_groups + i] = make_int4(-1, 0, 0, 0);
    }
}

// The value scale of 16 keys as f 2^e with e at most 60 below the largest so far (a scale of 0
// has f = 0): 2^-e stays in range, and every key counts in the sum of weights.
struct Dec8ValueScale {
    float e, f, inv;   // exponent, factor, 2^-e
    __device__ __forceinline__ Dec8ValueScale(float s, int& top)
    {
        const int x = min(max((int)((__float_as_uint(s) >> 23) & 0xFF) - 127, top - 60), 126);
        top = max(top, x);
        inv = __int_as_float((127 - x) << 23);
        f = s * inv;
        e = (float)x;
    }
};

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

// LSE from the base of a row's weights and their sum; the logarithm is taken of the sum relative
// to the largest weight, near 1 for few keys.
__device__ __forceinline__ float dec8_lse(float base, float sum)
{
    constexpr float down = 1.0f / (1 << (int)kD8Room);
    if (sum == 0.0f) return -__int_as_float(0x7f800000);
    const float m = base == -__int_as_float(0x7f800000) ? 0.0f : base;
    return (m + kD8Room + __log2f(sum * down)) * 0.69314718055994531f;
}

// Joins the parts of a unit that several ranges shared: with M the largest part base,
// O = sum_x 2^(M_x - M) a_x / sum_x 2^(M_x - M) l_x.  grid.x: the units, or where there are
// more of them the ranges (each leaves at most one unit to its successors); grid.y shares
// a unit's rows and columns.  Latency-bound: a thread has all its parts' loads in flight
// together.  Up to few_max parts (the usual batch) a thread joins one float4 of one row;
// more (one long sequence), 32 columns of a row at a time, sixteen threads a float4.  few_max
// is eight, or with the wide kernel's many rows, eight parts at a time, where both ways take
// the same number of rounds (8 x 8000 keys under 64 heads, d 256: 34.3 for 29.6 us without;
// with up to 16 rows the rounds' loop only cost 0.4 us of 20).
template <int D, int ROWS>
__global__ void __launch_bounds__(kD8CombineThreads) decode_fp8_combine_kernel(const DecodeFp8Params p, const int few_max)
{
    constexpr int PART = dec8_part(ROWS, D);
    constexpr int FEW = kD8CombineFew, MANY = 10;            // parts of a thread at a time
    constexpr int COLS = 8, GROUPS = kD8CombineThreads / COLS, SLICES = D / 32;
    __shared__ float4 sm_a[GROUPS][COLS];
    __shared__ float2 sm_ml[GROUPS];
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int tid = threadIdx.x, ctas = p.ranges * p.row_groups;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 todo = reinterpret_cast<const int4*>(p.ws)[blockIdx.x];
    const int x0 = todo.x, x1 = min(todo.y, p.ranges - 1), rg = todo.z;
    // a main grid that gave up on a wait leaves entries unwritten: whatever they hold, stay inside
    if (x0 < 0 || rg < 0 || rg >= p.row_groups || todo.w < 0) return;
    const size_t row0 = (size_t)todo.w;
    const int rows = min(ROWS, p.rows - rg * ROWS);
    if (row0 + rows > (size_t)p.B * p.Hkv * p.rows) return;
    auto part_of = [&](int x) {
        return p.ws + 4 * ctas + (size_t)(2 * (x * p.row_groups + rg) + (x == x0 ? 1 : 0)) * PART;
    };
    auto finish = [&](int r, int col, float4 a, float sum, float M) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + (row0 + r) * D)[col] =
            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        if (col == 0) p.lse[row0 + r] = dec8_lse(M, sum);
    };
    // (M, l, a) += K parts x, x + step, ... up to x1, of row r
    auto join = [&](auto K, int x, int step, int r, int col, float& M, float& l, float4& a) {
        constexpr int k_parts = decltype(K)::value;
        float m[k_parts], sum[k_parts];
        float4 v[k_parts];
#pragma unroll
        for (int k = 0; k < k_parts; ++k) {
            m[k] = NEG_INF;
            if (x + k * step > x1) continue;
            const float* w = part_of(x + k * step);
            m[k] = w[ROWS * D + r];
            sum[k] = w[ROWS * D + ROWS + r];
            v[k] = *reinterpret_cast<const float4*>(w + r * D + col * 4);
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < k_parts; ++k) top = fmaxf(top, m[k]);
        const float mb = top == NEG_INF ? 0.0f : top, f = ex2(M - mb);
        M = top;
        l *= f;
        a.x *= f, a.y *= f, a.z *= f, a.w *= f;
#pragma unroll
        for (int k = 0; k < k_parts; ++k) {
            if (x + k * step > x1) continue;
            const float fac = ex2(m[k] - mb);
            l = fmaf(fac, sum[k], l);
            a.x = fmaf(fac, v[k].x, a.x), a.y = fmaf(fac, v[k].y, a.y);
            a.z = fmaf(fac, v[k].z, a.z), a.w = fmaf(fac, v[k].w, a.w);
        }
    };
    if (x1 - x0 < (ROWS > 16 ? few_max : FEW)) {
        for (int i = blockIdx.y * kD8CombineThreads + tid; i < rows * (D / 4); i += gridDim.y * kD8CombineThreads) {
            const int r = i / (D / 4), col = i - r * (D / 4);
            float M = NEG_INF, l = 0.0f;
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if constexpr (ROWS > 16)
                for (int x = x0; x <= x1; x += FEW) join(std::integral_constant<int, FEW>{}, x, 1, r, col, M, l, a);
            else
                join(std::integral_constant<int, FEW>{}, x0, 1, r, col, M, l, a);
            finish(r, col, a, l, M);
        }
        return;
    }
    const int grp = tid / COLS;
    for (int i = blockIdx.y; i < rows * SLICES; i += gridDim.y) {
        const int r = i / SLICES, col = (i - r * SLICES) * COLS + tid % COLS;
        float M = NEG_INF, l = 0.0f;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int x = x0 + grp; x <= x1; x += GROUPS * MANY)
            join(std::integral_constant<int, MANY>{}, x, GROUPS, r, col, M, l, a);
        sm_a[grp][tid % COLS] = a;
        if (tid % COLS == 0) sm_ml[grp] = make_float2(M, l);
        __syncthreads();
        if (tid < COLS) {
            float top = NEG_INF, sum = 0.0f;
            a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < GROUPS; ++k) top = fmaxf(top, sm_ml[k].x);
            const float mb = top == NEG_INF ? 0.0f : top;
#pragma unroll
            for (int k = 0; k < GROUPS; ++k) {
                const float4 v = sm_a[k][tid];
                const float fac = ex2(sm_ml[k].x - mb);
                sum = fmaf(fac, sm_ml[k].y, sum);
                a.x = fmaf(fac, v.x, a.x), a.y = fmaf(fac, v.y, a.y);
                a.z = fmaf(fac, v.z, a.z), a.w = fmaf(fac, v.w, a.w);
            }
            finish(r, col, a, sum, top);
        }
        __syncthreads();
    }
}

// The joining launch of a main grid whose CTAs take ROWS rows.
template <int D, int ROWS>
cudaError_t launch_decode_fp8_combine(const DecodeFp8Params& p, cudaLaunchConfig_t& cfg)
{
    if (p.whole) return cudaSuccess;
    // a unit's float4s over its CTAs, and four CTAs a part of the average unit while that is
    // more, up to one for 32 columns of a row
    const long long units = (long long)p.B * p.Hkv * p.row_groups, ctas = p.ranges * p.row_groups;
    const int rows = p.rows < ROWS ? p.rows : ROWS, items = rows * (D / 32);
    const int least = (rows * (D / 4) + kD8CombineThreads - 1) / kD8CombineThreads;
    int share = units < ctas ? (int)(4 * ctas / units) : least;
    share = share > items ? items : share < least ? least : share;
    cfg.gridDim = dim3((unsigned)(units < ctas ? units : ctas), share);
    cfg.blockDim = dim3(kD8CombineThreads);
    cfg.dynamicSmemBytes = 0;
    const int few_rounds = (least + share - 1) / share, many_rounds = (items + share - 1) / share;
    const int few_max = kD8CombineFew * (many_rounds > few_rounds ? many_rounds / few_rounds : 1);   // used above 16 rows
    return cudaLaunchKernelEx(&cfg, decode_fp8_combine_kernel<D, ROWS>, p, few_max);
}

}  // namespace gb300
