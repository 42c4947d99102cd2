// context.h — the current device as the entry points outside moe_api.cu need it.
#pragma once

#include "internal.h"

namespace moe {

struct DeviceContext {
    int num_sms;
    WaitCfg wait;  // the limit of moe_set_wait_limit_ns and the library's device error word
};

// Fills `out` for the current device; a moe_status_t.
int device_context(DeviceContext &out);

// 16-bit floating-point tensor map of a stack [n, rows, cols] with a row pitch and a matrix
// pitch in elements (128-byte swizzle, boxes of 64 columns x box_rows rows of one matrix,
// elements outside a matrix read as zero). False if the driver rejects it.
bool map_stack_f16(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t n, int64_t pitch,
                   int64_t mat_pitch, uint32_t box_rows);

}  // namespace moe
