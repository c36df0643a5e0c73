// diff_params.h -- launch parameters of rotary positions (rope.cu) and of differential attention
// (diff_fwd.cu, diff_bwd.cu, diff_decode.cu).
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_params.h"
#include "paged_params.h"
#include "sched.cuh"

namespace gb300 {

// Rows of one tensor: element (b, n, h, i) at p + b * batch + n * token + h * head + i.
struct RopeRows {
    const void* in;
    void* out;
    long long in_batch, in_token, in_head;
    long long out_batch, out_token, out_head;
};

struct RopeParams {
    RopeRows q, k;
    const int* positions;   // int32 [axes, B * N]
    const float* inv_freq;  // fp32 [rot / 2], radians per position
    const int* axis;        // int32 [rot / 2], or null: all on axis 0
    int tokens, N;          // B * N, N
    int Hq, Hk, d, rot, axes;
    int interleaved, inverse;
    int slots;              // threads that share a token's heads: thread s takes heads s, s + slots, ...
};

// Differential attention: H heads, each of two maps.  f holds what the masks, the walk and the packed
// layout need, with f.BH (batched) or f.H (packed) counting heads times value parts.
struct DiffFwdParams {
    FwdParams f;            // f.o: bf16 [B, H, N, 2d] or [T, H, 2d]; f.lse: [B, 2H, N] or [2H, T]
    void* o2;               // the second map's output, laid out as o, or null
    const float* lam;       // fp32 [H]
    int H, Hkv;
    int group;              // heads (f's) whose units are handed out together, set at launch
};

struct DiffFwdMaps {
    CUtensorMap q, k, v;    // 128-row boxes of 64 columns
    CUtensorMap k64, v64;   // 64-row boxes (launch_diff_fwd_wide)
};

// Backward pass of differential attention.  Packed layout: B sequences' offsets in cu_seqlens, N the
// longest.
struct DiffBwdParams {
    const void* o;          // bf16 [B, H, N, 2d] or [T, H, 2d], as the forward pass wrote them
    const void* o2;
    const void* dout;
    const float* lse;       // fp32 [B, 2H, N] or [2H, T]
    const float* lam;       // fp32 [H]
    float* delta;           // fp32, laid out as lse: dO . O_1 and dO . O_2 of every row
    float* dlam;            // fp32 [H]
    void* dq;               // bf16 [B, 2H, N, d] or [T, 2H, d]
    void* dk;               // bf16 [B, 2Hkv, N, d] or [T, 2Hkv, d]
    void* dv;               // bf16 [B, Hkv, N, 2d] or [T, Hkv, 2d]
    int* next;              // [3]: the next unit of each pass, 0 before the first
    SortTab* tab;           // packed: the sequences by length, with the 128-row tiles before each; or null
    int* status;
    int B, H, Hkv, N;
    int nt;                 // 128-row tiles of N rows
    int causal, window;
    float c_log2, scale;
    unsigned long long timeout_ns;
    int withhold;           // 0, or n: each CTA's n-th ring load is never issued (failure tests)
    const int* cu_seqlens;  // int32 [B + 1], or null: batched
    int T;
};

struct DiffBwdMaps {
    CUtensorMap q, k, v, dout;      // 128-row boxes of 64 columns
    CUtensorMap q64, dout64;        // 64-row boxes
};

// One decoding step of differential attention over a paged bf16 cache.  w holds what the cut of the work
// needs (decode_fp8.cuh), with w.Hkv key pairs and w.rows = H / Hkv * nq query rows of each map; its
// scales and 8-bit caches are not used.
struct DiffDecodeParams {
    DecodeFp8Params w;      // w.q: bf16 [B, 2H, nq, d]; w.o: [B, H, nq, 2d]; w.lse: [B, 2H, nq]
    const float* lam;       // fp32 [H]
    int H;
};

// Rows of each map that a CTA takes, and CTAs of an SM.
constexpr int diff_decode_rows(int rows, int d) { return rows <= 4 ? 4 : rows <= 8 || d == 128 ? 8 : 16; }
constexpr int diff_decode_ctas(int d) { return d == 64 ? 2 : 1; }

cudaError_t launch_rope(const RopeParams& p, int sm_count, cudaStream_t stream);
cudaError_t launch_diff_fwd(const DiffFwdMaps& m, const DiffFwdParams& p, int d, int sm_count,
                            cudaStream_t stream);
// d = 128 without O_2: two launches with query blocks of 256 rows; lse.f counts maps as heads.
cudaError_t launch_diff_fwd_wide(const DiffFwdMaps& m, DiffFwdParams lse, DiffFwdParams out, int sm_count,
                                 cudaStream_t stream);
cudaError_t launch_diff_bwd(const DiffBwdMaps& m, const DiffBwdParams& p, int d, int sm_count,
                            cudaStream_t stream);
cudaError_t launch_diff_decode(const CUtensorMap& mk, const CUtensorMap& mv, const DiffDecodeParams& p, int d,
                               int cta_rows, cudaStream_t stream);

}  // namespace gb300
