// cache.hip - rows of keys and values into the block-quantised cache, and back.
//
// Quantisation, per 32 values of a token's head (the act buffer's rule, mmq.h):
//   q8_0: d = max|x| / 127 in f32, di = 1/d, q = clamp(round-half-even(x di), -128, 127);
//   q4_0: d = peak / -8, peak the first value of largest magnitude, nib = clamp(round-half-even(x di)
//         + 8, 0, 15);
// the stored scale is d rounded to f16. Division is IEEE-correct and nothing is contracted, so the
// bits are those of the definition.
//
// Two lanes share a block, 16 values each.
#include <algorithm>

#include "cache.h"

namespace mmq {
namespace {

constexpr int THREADS = 256;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// 16 consecutive values of a row of f32 (uint32_t) or bf16 (uint16_t)
template <typename T> __device__ inline void load16(const void* row, int64_t at, float (&x)[16]) {
    const u32x4_any* p = reinterpret_cast<const u32x4_any*>(static_cast<const T*>(row) + at);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const u32x4 r = p[c];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * c + i] = __builtin_bit_cast(float, (uint32_t)r[i]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const u32x4 r = p[c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[8 * c + 2 * i] = __builtin_bit_cast(float, r[i] << 16);
                x[8 * c + 2 * i + 1] = __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
            }
        }
    }
}
template <typename T> __device__ inline void store16(void* row, int64_t at, const float (&x)[16]) {
    u32x4_any* p = reinterpret_cast<u32x4_any*>(static_cast<T*>(row) + at);
#pragma unroll
    for (int c = 0; c < (int)sizeof(T); ++c) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) r[i] = __builtin_bit_cast(uint32_t, x[4 * c + i]);
            else r[i] = bf16_pair(x[8 * c + 2 * i], x[8 * c + 2 * i + 1]);
        }
        p[c] = r;
    }
}

// 1/d, 0 for d = 0, and the largest finite f32 (with d's sign) where 1/d overflows
__device__ inline float inverse_scale(float d) {
    return d != 0.0f ? fminf(fmaxf(1.0f / d, -3.40282347e38f), 3.40282347e38f) : 0.0f;
}

// One lane's half of a block (values 16h.. of it; the other half is in lane ^ 1): the stored whole
// numbers (q + 128, or q + 8), and the block's scale.
template <bool Q8> __device__ inline float quantize16(const float (&x)[16], int h, int (&q)[16]) {
    float d;
    if constexpr (Q8) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
        d = fmaxf(amax, __shfl_xor(amax, 1)) / 127.0f;
    } else {
        float peak = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) peak = fabsf(x[i]) > fabsf(peak) ? x[i] : peak;
        const float other = __shfl_xor(peak, 1);
        // the lower half's value where both are as large
        const bool take = h ? fabsf(other) >= fabsf(peak) : fabsf(other) > fabsf(peak);
        d = (take ? other : peak) / -8.0f;
    }
    const float di = inverse_scale(d);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float r = __builtin_rintf(x[i] * di);
        q[i] = Q8 ? (int)fminf(fmaxf(r, -128.f), 127.f) + 128 : (int)fminf(fmaxf(r, -8.f), 7.f) + 8;
    }
    return d;
}

struct RowsArgs {
    const void *k, *v;              // write: the rows
    void *ko, *vo;                  // read: the rows
    uint8_t *kc, *vc;
    const int32_t* slots;
    int64_t ldk, ldv, items;        // items: rows * heads * D / 16
    CacheShape c;
};

// Where the item's 16 values lie: false for a row without a slot.
struct Item {
    int64_t row, at;                // at: the values' place in the row
    uint64_t rec;                   // the record's number
    int t, b, h;                    // token in the record, block, half
};
__device__ inline bool item_of(const RowsArgs& a, int64_t i, Item& m) {
    const int halves = a.c.D / 16;
    const int64_t rh = i / halves;
    const int half = (int)(i - rh * halves);
    m.row = rh / a.c.heads;
    const int head = (int)(rh - m.row * a.c.heads);
    m.at = (int64_t)head * a.c.D + half * 16;
    m.b = half >> 1;
    m.h = half & 1;
    const uint32_t slot = (uint32_t)a.slots[m.row];
    const uint32_t page = slot / (uint32_t)(a.c.tiles * CACHE_TILE);
    if (page >= (uint32_t)a.c.pages) return false;          // a negative slot is a large number here
    m.rec = ((uint64_t)page * a.c.heads + head) * a.c.tiles + (slot / CACHE_TILE) % (uint32_t)a.c.tiles;
    m.t = (int)(slot % CACHE_TILE);
    return true;
}

template <typename T, bool Q8> __device__ inline void write_item(const RowsArgs& a, const Item& m, bool live, bool value) {
    float x[16] = {};
    if (live) load16<T>(value ? a.v : a.k, m.row * (value ? a.ldv : a.ldk) + m.at, x);
    int q[16];
    const float d = quantize16<Q8>(x, m.h, q);
    int other[16];
    if constexpr (!Q8) {
        if (value) {
#pragma unroll
            for (int i = 0; i < 16; ++i) other[i] = __shfl_xor(q[i], 1);
        }
    }
    if (!live) return;
    uint8_t* rec = (value ? a.vc : a.kc) + m.rec * cache_record(Q8, a.c.D);
    if (!value) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (Q8) w[j / 4] |= (uint32_t)q[8 * p + j] << (8 * (j % 4));
                else w[0] |= (uint32_t)q[8 * p + j] << (4 * key_nibble(j));
            }
            uint8_t* to = rec + key_at(Q8, a.c.D, m.t, m.b, 2 * m.h + p);
            if constexpr (Q8) *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[1]};
            else *reinterpret_cast<uint32_t*>(to) = w[0];
        }
    } else if constexpr (Q8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) rec[value_at(true, m.t, m.b, 16 * m.h + i)] = (uint8_t)q[i];
    } else {
        // the lane pair's bytes: eight each
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int v = m.h ? (other[8 + i] | q[8 + i] << 4) : (q[i] | other[i] << 4);
            rec[value_at(false, m.t, m.b, 8 * m.h + i)] = (uint8_t)v;
        }
    }
    if (m.h == 0) {
        *reinterpret_cast<_Float16*>(rec + cache_values(Q8, a.c.D) + scale_at(a.c.D, m.t, m.b)) = (_Float16)d;
    }
}

template <typename T, bool K8, bool V8> __global__ __launch_bounds__(THREADS) void cache_write_kernel(RowsArgs a) {
    const int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    Item m = {};
    const bool live = i < a.items && item_of(a, i, m);
    write_item<T, K8>(a, m, live, false);
    write_item<T, V8>(a, m, live, true);
}

template <typename T, bool Q8> __device__ inline void read_item(const RowsArgs& a, const Item& m, bool value) {
    const uint8_t* rec = (value ? a.vc : a.kc) + m.rec * cache_record(Q8, a.c.D);
    const float d =
        (float)*reinterpret_cast<const _Float16*>(rec + cache_values(Q8, a.c.D) + scale_at(a.c.D, m.t, m.b));
    float x[16];
    if (!value) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint8_t* from = rec + key_at(Q8, a.c.D, m.t, m.b, 2 * m.h + p);
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(from);
            const uint32_t w1 = Q8 ? *reinterpret_cast<const uint32_t*>(from + 4) : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int q = Q8 ? (int)(((j < 4 ? w0 : w1) >> (8 * (j % 4))) & 255) - 128
                                 : (int)((w0 >> (4 * key_nibble(j))) & 15) - 8;
                x[8 * p + j] = d * (float)q;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int w = rec[value_at(Q8, m.t, m.b, Q8 ? 16 * m.h + i : i)];
            x[i] = d * (float)(Q8 ? w - 128 : ((m.h ? w >> 4 : w) & 15) - 8);
        }
    }
    store16<T>(value ? a.vo : a.ko, m.row * (value ? a.ldv : a.ldk) + m.at, x);
}

template <typename T, bool K8, bool V8> __global__ __launch_bounds__(THREADS) void cache_read_kernel(RowsArgs a) {
    const int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    Item m;
    if (i >= a.items || !item_of(a, i, m)) return;
    read_item<T, K8>(a, m, false);
    read_item<T, V8>(a, m, true);
}

// f(type of the rows, K8, V8) for the call's types
template <typename F> void by_types(mmq_otype o, mmq_wtype tk, mmq_wtype tv, F f) {
    const auto k = [&](auto t) {
        const auto v = [&](auto k8) {
            if (tv == MMQ_Q8_0) f(t, k8, std::true_type());
            else f(t, k8, std::false_type());
        };
        if (tk == MMQ_Q8_0) v(std::true_type());
        else v(std::false_type());
    };
    if (o == MMQ_OUT_F32) k(uint32_t());
    else k(uint16_t());
}

}  // namespace

hipError_t launch_cache_write(mmq_otype o, const void* k, int64_t ldk, const void* v, int64_t ldv, const int32_t* slots,
                              int64_t rows, mmq_wtype tk, void* kcache, mmq_wtype tv, void* vcache, CacheShape c,
                              hipStream_t s) {
    RowsArgs a = {};
    a.k = k;
    a.v = v;
    a.ldk = ldk;
    a.ldv = ldv;
    a.slots = slots;
    a.kc = static_cast<uint8_t*>(kcache);
    a.vc = static_cast<uint8_t*>(vcache);
    a.items = rows * c.heads * (c.D / 16);
    a.c = c;
    by_types(o, tk, tv, [&](auto t, auto k8, auto v8) {
        hipLaunchKernelGGL((cache_write_kernel<decltype(t), decltype(k8)::value, decltype(v8)::value>),
                           dim3((unsigned)ceil_div(a.items, THREADS)), dim3(THREADS), 0, s, a);
    });
    return hipGetLastError();
}

hipError_t launch_cache_read(mmq_otype o, const int32_t* slots, int64_t rows, mmq_wtype tk, const void* kcache,
                             mmq_wtype tv, const void* vcache, CacheShape c, void* k, int64_t ldk, void* v, int64_t ldv,
                             hipStream_t s) {
    RowsArgs a = {};
    a.ko = k;
    a.vo = v;
    a.ldk = ldk;
    a.ldv = ldv;
    a.slots = slots;
    a.kc = static_cast<uint8_t*>(const_cast<void*>(kcache));
    a.vc = static_cast<uint8_t*>(const_cast<void*>(vcache));
    a.items = rows * c.heads * (c.D / 16);
    a.c = c;
    by_types(o, tk, tv, [&](auto t, auto k8, auto v8) {
        hipLaunchKernelGGL((cache_read_kernel<decltype(t), decltype(k8)::value, decltype(v8)::value>),
                           dim3((unsigned)ceil_div(a.items, THREADS)), dim3(THREADS), 0, s, a);
    });
    return hipGetLastError();
}

}  // namespace mmq
