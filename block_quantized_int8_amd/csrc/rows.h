// rows.h - the plan of rows grouped by adapter or expert: its layout, and the launchers that make
// and use it (rows.hip, lora.hip, lora_grad.hip; api.cpp).
#pragma once

#include "mmq_internal.h"

namespace mmq {

constexpr int GROUP_UNIT = 64;      // rows of a unit at most

// Byte offsets of the plan's regions (mmq.h, mmq_group_rows); P = T * top_k pairs.
struct PlanLayout {
    int64_t nunits;
    int64_t offs_off, order_off, pos_off, units_off, scratch_off, bytes;
};
PlanLayout plan_layout(int64_t E, int64_t P);

// f32 -> bf16 bits, round to nearest even, NaN kept a NaN (v_cvt_pk_bf16_f32)
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ inline uint32_t bf16_pair(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ inline uint16_t bf16_rne(float x) { return (uint16_t)bf16_pair(x, x); }

hipError_t launch_group_rows(const int32_t* ids, int64_t E, int64_t P, void* plan, hipStream_t s);
hipError_t launch_moe_gather(mmq_otype o, const void* x, int64_t ldx, const void* plan, int64_t E,
                             int64_t T, int64_t top_k, int64_t N, void* rows, int64_t ldr, hipStream_t s);
hipError_t launch_moe_combine(mmq_otype o, const void* z, int64_t ldz, bool sorted, const float* w,
                              const void* plan, int64_t E, int64_t T, int64_t top_k, int64_t N, void* y,
                              int64_t ldy, hipStream_t s);
hipError_t launch_moe_combine_grad(mmq_otype o, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                                   bool sorted, const float* w, const void* plan, int64_t E, int64_t T,
                                   int64_t top_k, int64_t N, void* dz, int64_t lddz, float* dw, hipStream_t s);

}  // namespace mmq
