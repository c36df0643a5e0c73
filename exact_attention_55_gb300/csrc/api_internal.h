// api_internal.h -- what the files of the C ABI share: per-device facts, tensor maps and
// argument checks.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>

#include "../../include/attn.h"

namespace gb300 {

constexpr unsigned long long kWaitTimeoutNs = 4000000000ull;  // 4 s per mbarrier wait

struct DeviceInfo {
    bool ready = false;
    int sm_count = 0;
    int* status = nullptr;
    float* decode_scratch = nullptr;
};

// Facts of the current device, looked up once with that device current.
attn_status_t device_info(DeviceInfo** out);

// 3-D bf16 map over rows of `cols` elements: dims (cols, rows, heads) with the given strides in
// elements, 128-byte swizzled boxes of 64 columns x box_rows x 1 head.  Rows outside read as zero.
bool encode_rows(CUtensorMap* m, const void* base, int cols, long long rows, long long row_stride,
                 long long heads, long long head_stride, int box_rows);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace gb300
