// rope.cu -- rotary positions of queries and keys on one or several axes (attn_rope_bf16).
//
// Pair i of a row (elements i and rot/2 + i, or 2i and 2i + 1) turns by the angle
//     a_i = position[axis_i] * inv_freq_i:   (x, y) -> (x cos a - y sin a, x sin a + y cos a),
// and by -a_i for the inverse, which is the gradient: the rotation is orthogonal.
//
// A far position times a frequency of 1 is many turns, of which fp32 would keep few digits of
// the last one (2^20 radians: 0.06).  The frequency is therefore taken in turns as a 64-bit
// fraction, f = inv_freq / 2 pi mod 1, from the product of its 24-bit mantissa and 2/pi to
// 64 bits; position * f in 64-bit integers then wraps to whole turns by itself, and its upper
// 32 bits are the angle, off by at most 2^-32 of a turn plus |position| 2^-63 (inv_freq <= 1).
// The nearest quarter of a turn comes from the fraction's top bits, sine and cosine of the rest, at
// most pi/4, from their Taylor series (to x^9 and x^8: off by less than 3e-8); they, products and sums
// are fp32, rounded once to bf16.
//
// Bound by memory: 4 bytes of traffic an element against half a multiplication.  A thread turns the
// same eight pairs (two 16-byte pieces of a row) of up to eight heads of its token, so an angle's
// instructions are shared by them; neighbouring threads take neighbouring pieces and heads.  Measured,
// 8191 tokens of 32 + 8 heads of d 128 on three axes: 33.2 us = 5.05 TB/s (36.8 with sincospif, 38.9
// with a block's angles shared through shared memory, 41 with several tokens a thread and their
// frequencies kept); blocks of 64 threads end more evenly than of 128 (34.8) or 256 (36.7).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "diff_params.h"
#include "ptx.cuh"

namespace gb300 {

constexpr int kRopeThreads = 64;

// inv_freq / 2 pi mod 1 turns, as a fraction of 2^64 (0 below 2^-64).
__device__ __forceinline__ unsigned long long rope_turns(float inv_freq)
{
    constexpr unsigned long long kTwoOverPi = 0xA2F9836E4E44152Aull;   // 2/pi * 2^64
    const uint32_t bits = __float_as_uint(inv_freq);
    const int ex = (int)((bits >> 23) & 0xFF);
    const uint32_t man = (bits & 0x7FFFFF) | (ex ? 0x800000u : 0u);
    // inv_freq = man 2^(ex - 150); times (2/pi) 2^64 / 4
    const unsigned __int128 prod = (unsigned __int128)kTwoOverPi * man;
    const int left = max(ex, 1) - 152;
    unsigned long long f = 0;
    if (left < 0 && left > -128) f = (unsigned long long)(prod >> -left);
    else if (left >= 0 && left < 64) f = (unsigned long long)prod << left;
    return (bits >> 31) ? 0ull - f : f;
}

// Sine and cosine of an angle in turns, a 64-bit fraction.
__device__ __forceinline__ void rope_sincos(unsigned long long a, float& sn, float& cs)
{
    const uint32_t top = (uint32_t)(a >> 32), quarter = (top + 0x20000000u) >> 30;
    const float x = (float)(int)(top - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi 2^-32
    const float z = x * x;
    float s = fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f), c = fmaf(z, 1.0f / 40320.0f, -1.0f / 720.0f);
    s = fmaf(z, s, 1.0f / 120.0f);
    c = fmaf(z, c, 1.0f / 24.0f);
    s = fmaf(z, s, -1.0f / 6.0f);
    c = fmaf(z, c, -0.5f);
    s = fmaf(x * z, s, x);
    c = fmaf(z, c, 1.0f);
    const bool odd = quarter & 1;
    sn = odd ? c : s;
    cs = odd ? s : c;
    if (quarter & 2) sn = -sn;
    if ((quarter + 1) & 2) cs = -cs;
}

template <int U>
__global__ void __launch_bounds__(kRopeThreads, 10) rope_kernel(const RopeParams p)
{
    const unsigned chunks = (unsigned)p.d / 16, i = blockIdx.x * kRopeThreads + threadIdx.x;
    const unsigned r = i / chunks, chunk = i - r * chunks;
    const unsigned tok = r / (unsigned)p.slots, slot = r - tok * (unsigned)p.slots;
    if (tok >= (unsigned)p.tokens) return;
    const unsigned b = tok / (unsigned)p.N, n = tok - b * (unsigned)p.N;
    // rows of padding (a negative first position) and what lies behind the pairs are copied
    const int first = __ldg(p.positions + tok);
    const bool paired = chunk < (unsigned)p.rot / 16, turned = paired && first >= 0;
    int c0, c1;                                     // this thread's two pieces of a row
    if (!paired || p.interleaved) c0 = chunk * 16, c1 = c0 + 8;
    else c0 = chunk * 8, c1 = c0 + p.rot / 2;
    const __nv_bfloat16* qi = static_cast<const __nv_bfloat16*>(p.q.in) + b * p.q.in_batch + n * p.q.in_token;
    const __nv_bfloat16* ki = static_cast<const __nv_bfloat16*>(p.k.in) + b * p.k.in_batch + n * p.k.in_token;
    __nv_bfloat16* qo = static_cast<__nv_bfloat16*>(p.q.out) + b * p.q.out_batch + n * p.q.out_token;
    __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(p.k.out) + b * p.k.out_batch + n * p.k.out_token;
    const int heads = p.Hq + p.Hk;

    float cs[8], sn[8];
    auto angles = [&]() {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int pair = chunk * 8 + e;
            const float f = __ldg(p.inv_freq + pair);
            int pos = first;
            if (p.axis != nullptr) {
                const int ax = min(max(__ldg(p.axis + pair), 0), p.axes - 1);
                pos = __ldg(p.positions + (size_t)ax * p.tokens + tok);
            }
            unsigned long long a = rope_turns(f) * (unsigned long long)(long long)pos;
            if (p.inverse) a = 0ull - a;
            rope_sincos(a, sn[e], cs[e]);
            if (!(fabsf(f) <= 3.402823466e38f)) cs[e] = sn[e] = __int_as_float(0x7fc00000);
        }
    };
    bool ready = false;
    for (int h0 = slot; h0 < heads; h0 += U * p.slots) {
        uint4 x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * p.slots;
            if (h >= heads) continue;
            const __nv_bfloat16* row = h < p.Hq ? qi + h * p.q.in_head : ki + (h - p.Hq) * p.k.in_head;
            x[u] = *reinterpret_cast<const uint4*>(row + c0);
            y[u] = *reinterpret_cast<const uint4*>(row + c1);
        }
        if (turned && !ready) {                     // the loads are in flight meanwhile
            angles();
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * p.slots;
            if (h >= heads) continue;
            uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, yw[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
            auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
            auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
            auto real = [&](float a, float c, int e) { return fmaf(a, cs[e], -(c * sn[e])); };
            auto imag = [&](float a, float c, int e) { return fmaf(a, sn[e], c * cs[e]); };
            if (turned && !p.interleaved) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float x0 = lo(xw[w]), x1 = hi(xw[w]), y0 = lo(yw[w]), y1 = hi(yw[w]);
                    xw[w] = pack_bf16x2(real(x0, y0, 2 * w), real(x1, y1, 2 * w + 1));
                    yw[w] = pack_bf16x2(imag(x0, y0, 2 * w), imag(x1, y1, 2 * w + 1));
                }
            } else if (turned) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float a0 = lo(xw[w]), b0 = hi(xw[w]), a1 = lo(yw[w]), b1 = hi(yw[w]);
                    xw[w] = pack_bf16x2(real(a0, b0, w), imag(a0, b0, w));
                    yw[w] = pack_bf16x2(real(a1, b1, 4 + w), imag(a1, b1, 4 + w));
                }
            }
            __nv_bfloat16* row = h < p.Hq ? qo + h * p.q.out_head : ko + (h - p.Hq) * p.k.out_head;
            *reinterpret_cast<uint4*>(row + c0) = make_uint4(xw[0], xw[1], xw[2], xw[3]);
            *reinterpret_cast<uint4*>(row + c1) = make_uint4(yw[0], yw[1], yw[2], yw[3]);
        }
    }
}

cudaError_t launch_rope(const RopeParams& given, int sm_count, cudaStream_t stream)
{
    RopeParams p = given;
    const int heads = p.Hq + p.Hk, chunks = p.d / 16;
    // threads enough to fill the card come first, heads that share a thread's angles second
    const long long room = (long long)sm_count * 1024;
    long long share = (long long)p.tokens * heads * chunks / room;
    share = share < 1 ? 1 : share > 8 ? 8 : share;
    if (share > heads) share = heads;
    p.slots = (int)((heads + share - 1) / share);
    const long long threads = (long long)p.tokens * p.slots * chunks;
    const long long grid = (threads + kRopeThreads - 1) / kRopeThreads;
    if (grid * kRopeThreads > 0xffffffffLL) return cudaErrorInvalidValue;
    if (share >= 4) rope_kernel<4><<<(unsigned)grid, kRopeThreads, 0, stream>>>(p);
    else rope_kernel<1><<<(unsigned)grid, kRopeThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gb300
