// decode_fp8.cu -- one decoding step of attention over a paged cache of 8-bit codes with one
// scale per block of tokens and head, query heads sharing key heads.
//
// "大模型加速-核心网络算子-Flash Attention V3" §3 总结 (decoding over cached K and V) and §1.5
// (E4M3, E5M2); "Warp Group Cluster 优化：Flash Attention V3 在 H100 上的 FP8 融合计算实践",
// 局限性与后续方向 item 2 (PagedAttention) and §3 (a scale per block).
//
// Row r = g * nq + i of key head hk is query i of head hk * G + g, at position
// L - nq + i; it sees keys max(0, position - window) .. position (window 0: all of them):
//   s_j = scale * ks(j) * q . k8_j,   O = sum_j softmax(s)_j vs(j) v8_j,   LSE = log sum exp s
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_params.h"
#include "ptx.cuh"

namespace gb300 {

constexpr int kDec8Warps = 8;

template <bool kE5M2>
__device__ __forceinline__ float2 dec8_unpack2(uint32_t two)
{
    uint32_t h;
    if constexpr (kE5M2) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi) : "r"(h));
    return make_float2(lo, hi);
}

// One CTA per query row; its warps take the row's keys in turn, a lane holds D/32 values.
template <int D, bool kE5M2>
__global__ void __launch_bounds__(kDec8Warps * 32) decode_fp8_kernel(const DecodeFp8Params p)
{
    constexpr int E = D / 32;
    __shared__ float sm_m[kDec8Warps], sm_l[kDec8Warps], sm_acc[kDec8Warps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = blockIdx.x;
    const int r = (int)(row % p.rows);
    const long long bh = row / p.rows;
    const int b = (int)(bh / p.Hkv), hk = (int)(bh - (long long)b * p.Hkv), i = r % p.nq;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int L = min(max(p.seq_lens[b], 0), p.max_pages << p.log2_ps);
    const int last = L - p.nq + i, first = p.window > 0 ? max(0, last - p.window) : 0;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row * D + lane * E;
    float qv[E], acc[E], m = NEG_INF, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = __bfloat162float(q[e]) * p.c_log2;
        acc[e] = 0.0f;
    }
    for (int t = first + warp; t <= last; t += kDec8Warps) {
        const int page = min(max(p.page_table[(size_t)b * p.max_pages + (t >> p.log2_ps)], 0), p.num_pages - 1);
        const size_t head = (size_t)page * p.Hkv + hk;
        const int in_page = t & ((1 << p.log2_ps) - 1);
        const size_t at = ((head << p.log2_ps) + in_page) * D + lane * E;
        const size_t sc = (head << (p.log2_ps - p.log2_blk)) + (in_page >> p.log2_blk);
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 k = dec8_unpack2<kE5M2>(*reinterpret_cast<const uint16_t*>(p.kc + at + e));
            s = fmaf(qv[e], k.x, fmaf(qv[e + 1], k.y, s));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= p.ks[sc];
        if (s > m) {
            const float alpha = ex2(m - s);
            l *= alpha;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= alpha;
            m = s;
        }
        const float w = ex2(s - m);
        l += w;
        const float wv = w * p.vs[sc];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 v = dec8_unpack2<kE5M2>(*reinterpret_cast<const uint16_t*>(p.vc + at + e));
            acc[e] = fmaf(wv, v.x, acc[e]);
            acc[e + 1] = fmaf(wv, v.y, acc[e + 1]);
        }
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_acc[warp][lane * E + e] = acc[e];
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += kDec8Warps * 32) {
        float M = sm_m[0];
        for (int w = 1; w < kDec8Warps; ++w) M = fmaxf(M, sm_m[w]);
        float sum = 0.0f, o = 0.0f;
        for (int w = 0; w < kDec8Warps; ++w) {
            const float f = M == NEG_INF ? 0.0f : ex2(sm_m[w] - M);
            sum = fmaf(sm_l[w], f, sum);
            o = fmaf(sm_acc[w][e], f, o);
        }
        static_cast<__nv_bfloat16*>(p.o)[row * D + e] = __float2bfloat16_rn(last < 0 ? 0.0f : o / sum);
        if (e == 0) p.lse[row] = last < 0 ? NEG_INF : (M + __log2f(sum)) * 0.69314718055994531f;
    }
}

template <int D>
static cudaError_t launch_decode_fp8_d(const DecodeFp8Params& p, bool e5m2, cudaStream_t stream)
{
    const unsigned grid = (unsigned)((long long)p.B * p.Hkv * p.rows);
    if (e5m2) decode_fp8_kernel<D, true><<<grid, kDec8Warps * 32, 0, stream>>>(p);
    else decode_fp8_kernel<D, false><<<grid, kDec8Warps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_decode_fp8(const DecodeFp8Params& p, int d, bool e5m2, cudaStream_t stream)
{
    switch (d) {
    case 64: return launch_decode_fp8_d<64>(p, e5m2, stream);
    case 128: return launch_decode_fp8_d<128>(p, e5m2, stream);
    case 256: return launch_decode_fp8_d<256>(p, e5m2, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gb300
