// diff_params.h -- launch parameters of rotary positions (rope.cu) and of differential attention
// (diff_fwd.cu, diff_bwd.cu, diff_decode.cu).
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_params.h"

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
};

struct DiffFwdMaps {
    CUtensorMap q, k, v;    // 128-row boxes of 64 columns
};

cudaError_t launch_rope(const RopeParams& p, int sm_count, cudaStream_t stream);
cudaError_t launch_diff_fwd(const DiffFwdMaps& m, const DiffFwdParams& p, int d, int sm_count,
                            cudaStream_t stream);

}  // namespace gb300
