// paged_params.h -- launch parameters of the paged-cache operators (paged.cu, decode_fp8.cu).
#pragma once

#include <cstdint>

namespace gb300 {

// Pages, slots, positions and lengths of one serving step.
struct PlanParams {
    const int* new_lens;    // int32 [B]
    const int* seq_lens;    // int32 [B]
    int* page_table;        // int32 [B, max_pages], entries of the pages taken are written
    const int* free_pages;  // int32 [free_capacity], a stack of page numbers
    const int* free_count;  // int32 [1]
    int* seq_lens_out;      // int32 [B], may be seq_lens
    int* free_count_out;    // int32 [1], may be free_count
    int* cu_new;            // int32 [B + 1]
    long long* slot_map;    // int64 [num_tokens]
    int* positions;         // int32 [num_tokens]
    int* served;            // int32 [B]
    int B, log2_ps, max_pages, free_capacity, num_tokens;
};

// New rows into a cache: k and v [T, H, d] with token strides, caches [num_pages, H, ps, d].
struct AppendParams {
    const void* k;          // bf16, row (t, h) at k + t * k_stride + h * d
    const void* v;
    void* kc;               // bf16 or 8-bit codes
    void* vc;
    float* ks;              // fp32 [num_pages, H, ps / block] (8-bit caches only)
    float* vs;
    const long long* slot_map;  // int64 [T]
    long long k_stride, v_stride;  // elements
    long long num_slots;    // num_pages << log2_ps
    int T, H, d;
    int tile;               // tokens whose runs a CTA takes (8-bit caches; the launcher's)
    int log2_ps, log2_blk;
    int pow2;               // scales are rounded up to powers of two
    int sm_count;
};

// One decoding step over an 8-bit paged cache.
struct DecodeFp8Params {
    const void* q;          // bf16 [B, H, nq, d]
    const uint8_t* kc;      // codes [num_pages, Hkv, ps, d]
    const uint8_t* vc;
    const float* ks;        // fp32 [num_pages, Hkv, ps / block]
    const float* vs;
    const int* page_table;  // int32 [B, max_pages]
    const int* seq_lens;    // int32 [B]
    void* o;                // bf16 [B, H, nq, d]
    float* lse;             // fp32 [B, H, nq], natural log
    int B, Hkv, nq;
    int rows;               // query rows of one K/V head: H / Hkv * nq
    int log2_ps, log2_blk;
    int num_pages, max_pages;
    int window;
    float c_log2;           // softmax scale * log2(e)
    float* ws;              // per CTA: int4 for the joining kernel; then two parts per CTA
    int whole;              // 1: no unit is split over ranges (short tables), nothing to join
    int ranges;             // CTAs of one row group: at most this many ranges of tiles
    int row_groups;         // groups of query rows, each a CTA's share
    int* status;            // device status word (bounded waits)
    unsigned long long timeout_ns;
    unsigned withhold;      // 0, or n: each CTA's n-th load is never issued (failure tests)
};

}  // namespace gb300
