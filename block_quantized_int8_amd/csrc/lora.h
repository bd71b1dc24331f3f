// lora.h - what the adapters' forward and backward kernels share (lora.hip, lora_grad.hip): the
// matrix-core operands, the exact split of f32 values into bf16 terms, and the launchers.
//
// Operands of v_mfma_f32_16x16x32_{bf16,f16}, lane L = 16g + c (g < 4, c < 16): the A operand
// holds row c's and the B operand column c's values k = 8g .. 8g+7 of the 32-deep step; the
// accumulator holds rows 4g .. 4g+3 of column c.
//
// Products keep f32: an f32 value is exactly the sum of three bf16 terms of 8 significand bits
// each (an f16 value of two), so a product of terms is exact in f32 and only the accumulation
// rounds. Terms are cut off, not rounded, so that the rest is exact and of the same sign. Pairs
// of terms below 2^-23 of the product are left out.
#pragma once

#include "mmq_internal.h"
#include "rows.h"

namespace mmq {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
// 16 or 8 bytes at any address a value of the row's type may have (global memory only)
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

__device__ inline f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ inline f32x4 mfma_f16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ inline uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ inline float as_f(uint32_t x) { return __builtin_bit_cast(float, x); }
// the upper halves of two f32 (lo in the low half)
__device__ inline uint32_t pack_hi(float lo, float hi) { return __builtin_amdgcn_perm(bits(hi), bits(lo), 0x07060302u); }
__device__ inline float cut(float x) { return as_f(bits(x) & 0xFFFF0000u); }

// eight f32 values as three bf16 operands, the largest terms first
__device__ inline void split3(const float* x, u32x4* t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        const float a1 = a - cut(a), b1 = b - cut(b);
        const float a2 = a1 - cut(a1), b2 = b1 - cut(b1);
        t[0][i] = pack_hi(a, b);
        t[1][i] = pack_hi(a1, b1);
        t[2][i] = pack_hi(a2, b2);
    }
}

// eight f16 values (raw bits) as two bf16 operands
__device__ inline void split_f16(u32x4 h, u32x4* t) {
    const f16x8 v = __builtin_bit_cast(f16x8, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = (float)v[2 * i], b = (float)v[2 * i + 1];
        t[0][i] = pack_hi(a, b);
        t[1][i] = pack_hi(a - cut(a), b - cut(b));
    }
}

// An adapter's operand: one bf16 term, or an f16 value's two.
template <bool F16> struct Weights {
    static constexpr int T = F16 ? 2 : 1;
    u32x4 t[T];
    __device__ void set(u32x4 raw) {
        if constexpr (F16) split_f16(raw, t);
        else t[0] = raw;
    }
};

// acc += a weight operand (A) times f32 values given as three terms (B), small products first
template <bool F16>
__device__ inline f32x4 mfma_terms(const Weights<F16>& w, const u32x4* x, f32x4 acc) {
    if constexpr (F16) {
        acc = mfma_bf16(w.t[1], x[1], acc);
        acc = mfma_bf16(w.t[0], x[2], acc);
        acc = mfma_bf16(w.t[1], x[0], acc);
    } else {
        acc = mfma_bf16(w.t[0], x[2], acc);
    }
    acc = mfma_bf16(w.t[0], x[1], acc);
    return mfma_bf16(w.t[0], x[0], acc);
}

// eight int8 values as a bf16 or f16 operand (exact: 8 bits)
template <bool F16> __device__ inline u32x4 int8_operand(u32x2 q) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = q[i / 2] >> (16 * (i & 1));
        const float a = (float)(int8_t)w, b = (float)(int8_t)(w >> 8);
        if constexpr (F16) r[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
        else r[i] = pack_hi(a, b);
    }
    return r;
}

// Four values of a row of the output's type from column n on, as f32 (columns past N read 0).
template <bool BF16> __device__ inline f32x4 load4(const void* p, int64_t at, int left) {
    f32x4 r = 0;
    if constexpr (BF16) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + at;
        if (left >= 4) {
            const u32x2 w = *reinterpret_cast<const u32x2_any*>(q);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = as_f(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < left) r[j] = as_f((uint32_t)q[j] << 16);
        }
    } else {
        const float* q = static_cast<const float*>(p) + at;
        if (left >= 4) r = *reinterpret_cast<const f32x4_any*>(q);
        else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < left) r[j] = q[j];
        }
    }
    return r;
}

template <bool BF16> __device__ inline void store4(void* p, int64_t at, f32x4 v, int left) {
    if constexpr (BF16) {
        uint16_t* q = static_cast<uint16_t*>(p) + at;
        if (left >= 4) {
            u32x2 w;
#pragma unroll
            for (int j = 0; j < 2; ++j) w[j] = (uint32_t)bf16_rne(v[2 * j]) | ((uint32_t)bf16_rne(v[2 * j + 1]) << 16);
            *reinterpret_cast<u32x2_any*>(q) = w;
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < left) q[j] = bf16_rne(v[j]);
        }
    } else {
        float* q = static_cast<float*>(p) + at;
        if (left >= 4) *reinterpret_cast<f32x4_any*>(q) = v;
        else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < left) q[j] = v[j];
        }
    }
}

struct LoraArgs {
    const int8_t* xq;           // act region 0
    const uint32_t* xs2;        // q8_1 region 1 (xs as an f16 pair)
    const float* sa;            // i8_token region 1
    int KB, KBp;
    const uint16_t *A, *B;      // [E][R][K], [E][N][R] raw bf16 or f16
    const float* scale;         // [E]
    const int32_t* order;
    const int4* units;
    int E, R, M, N, K, nunits;
    float* part;                // partial sums [S][M][R] by sorted position
    int S;
    // forward
    const void* base;
    int64_t ldb;
    void* out;
    int64_t ldo;
    float* v;                   // [M][R]
    // backward
    const int32_t* offs;
    const void* dy;
    int64_t lddy;
    const float* dxb;
    int64_t lddxb;
    float* dx;
    int64_t lddx;
    float *dA, *dB, *u;         // u: [M][R] by sorted position
};

// The arguments both calls share.
inline LoraArgs lora_args(mmq_atype t, const void* act, const void* A, const void* B, const float* scale, int64_t E,
                          int64_t R, const void* plan, int64_t M, int64_t N, int64_t K) {
    const PlanLayout L = plan_layout(E, M);
    const uint8_t* p = static_cast<const uint8_t*>(plan);
    const uint8_t* x = static_cast<const uint8_t*>(act);
    LoraArgs a = {};
    if (t == MMQ_ACT_Q8_1) {
        const ActQ81Layout l = act_q8_1_layout(M, K);
        a.xq = reinterpret_cast<const int8_t*>(x + l.xq_off);
        a.xs2 = reinterpret_cast<const uint32_t*>(x + l.xs2_off);
        a.KBp = (int)l.KBp;
    } else {
        const ActI8Layout l = act_i8_layout(M, K);
        a.xq = reinterpret_cast<const int8_t*>(x + l.a_off);
        a.sa = reinterpret_cast<const float*>(x + l.sa_off);
        a.KBp = (int)l.KBp;
    }
    a.KB = (int)(K / QK);
    a.A = static_cast<const uint16_t*>(A);
    a.B = static_cast<const uint16_t*>(B);
    a.scale = scale;
    a.offs = reinterpret_cast<const int32_t*>(p + L.offs_off);
    a.order = reinterpret_cast<const int32_t*>(p + L.order_off);
    a.units = reinterpret_cast<const int4*>(p + L.units_off);
    a.E = (int)E;
    a.R = (int)R;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.nunits = (int)L.nunits;
    return a;
}

constexpr int LT = 256;             // threads of a workgroup
constexpr int UP_COLS = 256;        // columns of an up workgroup: 64 per wave
constexpr int LORA_RC = 64;        // ranks of a pass
constexpr int64_t LORA_MAX_R = 256;

size_t lora_workspace_bytes(int64_t E, int64_t M, int64_t K, int64_t R);
bool lora_grid_ok(int64_t E, int64_t M, int64_t N, int64_t K);
hipError_t launch_lora(mmq_atype t, bool f16, const void* act, const void* A, const void* B, const float* scale,
                       int64_t E, int64_t R, const void* plan, int64_t M, int64_t N, int64_t K, const void* base,
                       int64_t ldb, void* out, int64_t ldo, float* v, void* ws, hipStream_t s);
size_t lora_grad_workspace_bytes(int64_t E, int64_t M, int64_t N, int64_t R);
hipError_t launch_lora_grad(mmq_atype t, bool f16, const void* act, const void* A, const void* B, const float* scale,
                            int64_t E, int64_t R, const void* plan, int64_t M, int64_t N, int64_t K, const float* v,
                            const void* dy, int64_t lddy, const float* dxb, int64_t lddxb, float* dx, int64_t lddx,
                            float* dA, float* dB, void* ws, hipStream_t s);

}  // namespace mmq
