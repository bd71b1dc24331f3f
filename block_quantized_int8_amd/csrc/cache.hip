// cache.hip - rows of keys and values into the block-quantised cache, and back.
//
// Quantisation, per 32 values of a token's head (the act buffer's rule, mmq.h):
//   q8_0: d = max|x| / 127 in f32, di = 1/d, q = clamp(round-half-even(x di), -128, 127);
//   q4_0: d = peak / -8, peak the first value of largest magnitude, nib = clamp(round-half-even(x di)
//         + 8, 0, 15);
// the stored scale is d rounded to f16. Division is IEEE-correct and nothing is contracted, so the
// bits are those of the definition.
//
// Two lanes share a block, 16 values each. Few rows, or rows that lie anywhere, go one by one: a
// token's keys as 8-byte pieces, its values byte by byte (a record holds 8 tokens' values side by side).
// Many rows go by windows of 32 or 64 through LDS images of the two or three tiles that consecutive
// slots can touch, so that memory sees whole 16-byte pieces there; rows of other tiles go one by one.
//
// Memory bounds many rows: 32768 of 8 heads of 128 values are read from q8_0 as bf16 in 35 us (5.9 TB/s of both
// sides), written from f32 in 70 us (4.9 TB/s); 8192 of them written in 19.5 us (4.4), 2048 in 8.4 us (2.5 TB/s, and a
// launch). Few rows are a launch: one 2.8 us. Rows that lie anywhere cost several times that: 32768 written in 226 us and
// read as f32 in 99 (in order 72 and 55), where one by one would be 182 and 128; the host does not know the slots.
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
    int64_t ldk, ldv, rows;
    CacheShape c;
    int page_bits;                  // tokens of a page: 2^page_bits
};

// The record of a slot's token: its number for a head.
__device__ inline int page_of(const RowsArgs& a, int slot) { return slot >> a.page_bits; }
__device__ inline uint64_t record_of(const RowsArgs& a, int slot, int head) {
    return ((uint64_t)page_of(a, slot) * a.c.heads + head) * a.c.tiles + (uint32_t)((slot >> 5) & (a.c.tiles - 1));
}
// A row's slot, -1 if it has none.
__device__ inline int slot_of(const RowsArgs& a, int64_t row) {
    const int s = a.slots[row];
    return s >= 0 && page_of(a, s) < a.c.pages ? s : -1;
}

// 16 values of a row: half h of block b of a head, of a token t of its record.
struct Item {
    int64_t row, at;                // at: the values' place in the row
    int t, b, h;
};
__device__ inline Item item_of(int64_t row, int head, int half, int D, int slot) {
    return {row, (int64_t)head * D + half * 16, slot & (CACHE_TILE - 1), half >> 1, half & 1};
}

// Where a record's byte lies in an image in LDS: a row's lanes take bytes 8, 128 and 1024 apart, which would
// all be in a few banks (8 lanes a bank), so every 128 bytes are followed by 16 more and every 1024 by 32.
__host__ __device__ constexpr int in_image(int at) { return at + (at >> 7) * 16 + (at >> 10) * 32; }
template <bool IMAGE> __device__ inline int place(int at) { return IMAGE ? in_image(at) : at; }

// An item quantised; `other`: the whole numbers of the block's other half, where values of q4_0 need them.
template <typename T, bool Q8, bool VALUE>
__device__ inline float take_item(const RowsArgs& a, const Item& m, bool live, int (&q)[16], int (&other)[16]) {
    float x[16] = {};
    if (live) load16<T>(VALUE ? a.v : a.k, m.row * (VALUE ? a.ldv : a.ldk) + m.at, x);
    const float d = quantize16<Q8>(x, m.h, q);
    if constexpr (!Q8 && VALUE) {
#pragma unroll
        for (int i = 0; i < 16; ++i) other[i] = __shfl_xor(q[i], 1);
    }
    return d;
}
// And put into its token's record, or an image of it.
template <bool Q8, bool VALUE, bool IMAGE>
__device__ inline void put_item(const RowsArgs& a, const Item& m, const int (&q)[16], const int (&other)[16], float d, uint8_t* rec) {
    if constexpr (!VALUE) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (Q8) w[j / 4] |= (uint32_t)q[8 * p + j] << (8 * (j % 4));
                else w[0] |= (uint32_t)q[8 * p + j] << (4 * key_nibble(j));
            }
            uint8_t* to = rec + place<IMAGE>(key_at(Q8, a.c.D, m.t, m.b, 2 * m.h + p));
            if constexpr (Q8) *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[1]};
            else *reinterpret_cast<uint32_t*>(to) = w[0];
        }
    } else if constexpr (Q8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) rec[place<IMAGE>(value_at(true, m.t, m.b, 16 * m.h + i))] = (uint8_t)q[i];
    } else {
        // the lane pair's bytes: eight each
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int v = m.h ? (other[8 + i] | q[8 + i] << 4) : (q[i] | other[i] << 4);
            rec[place<IMAGE>(value_at(false, m.t, m.b, 8 * m.h + i))] = (uint8_t)v;
        }
    }
    if (m.h == 0) {
        *reinterpret_cast<_Float16*>(rec + place<IMAGE>(cache_values(Q8, a.c.D) + scale_at(a.c.D, m.t, m.b))) = (_Float16)d;
    }
}

// One lane an item of keys and of values
template <typename T, bool K8, bool V8> __global__ __launch_bounds__(THREADS) void cache_write_kernel(RowsArgs a) {
    const uint32_t i = blockIdx.x * THREADS + threadIdx.x, halves = (uint32_t)a.c.D / 16, rh = i / halves;
    const uint32_t row = rh / (uint32_t)a.c.heads, head = rh % (uint32_t)a.c.heads;
    const int slot = row < a.rows ? slot_of(a, row) : -1;
    const Item m = item_of(row, (int)head, (int)(i % halves), a.c.D, slot);
    const uint64_t rec = slot < 0 ? 0 : record_of(a, slot, (int)head);
    int q[16], other[16];
    const float dk = take_item<T, K8, false>(a, m, slot >= 0, q, other);
    if (slot >= 0) put_item<K8, false, false>(a, m, q, other, dk, a.kc + rec * cache_record(K8, a.c.D));
    const float dv = take_item<T, V8, true>(a, m, slot >= 0, q, other);
    if (slot >= 0) put_item<V8, true, false>(a, m, q, other, dv, a.vc + rec * cache_record(V8, a.c.D));
}

// 16 bytes of a row that is read: N values from i0 on of block b of a token's record, or an image of it.
template <typename T> constexpr int READ_N = 16 / (int)sizeof(T);
template <typename T, bool Q8, bool VALUE, bool IMAGE>
__device__ inline u32x4 read_piece(const uint8_t* rec, int D, int t, int b, int i0) {
    constexpr int N = READ_N<T>;
    const float d = (float)*reinterpret_cast<const _Float16*>(rec + place<IMAGE>(cache_values(Q8, D) + scale_at(D, t, b)));
    float x[N];
    if constexpr (!VALUE) {
        const uint8_t* from = rec + place<IMAGE>(key_at(Q8, D, t, b, i0 >> 3));
        uint32_t w[2];
        if constexpr (!Q8) w[0] = *reinterpret_cast<const uint32_t*>(from);
        else if constexpr (N == 4) w[0] = *reinterpret_cast<const uint32_t*>(from + (i0 & 4));
        else {
            const u32x2 v = *reinterpret_cast<const u32x2*>(from);
            w[0] = v[0];
            w[1] = v[1];
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            // (q4_0: values 4.. of a piece lie 8 bits on from values 0..)
            const int q = Q8 ? (int)((w[j / 4] >> (8 * (j % 4))) & 255) - 128
                             : (int)((w[0] >> (4 * key_nibble(j) + (N == 4 ? (i0 & 4) * 2 : 0))) & 15) - 8;
            x[j] = d * (float)q;
        }
    } else {
        // (the N values' 16-byte pieces lie in one run of 128 bytes)
        const uint8_t* from = rec + place<IMAGE>(value_at(Q8, t, b, Q8 ? i0 : i0 & 15));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int w = from[16 * j];
            x[j] = d * (float)(Q8 ? w - 128 : ((i0 & 16 ? w >> 4 : w) & 15) - 8);
        }
    }
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (N == 4) r[i] = __builtin_bit_cast(uint32_t, x[i]);
        else r[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
    }
    return r;
}

template <typename T, bool K8, bool V8> __global__ __launch_bounds__(THREADS) void cache_read_kernel(RowsArgs a) {
    constexpr int N = READ_N<T>;
    const uint32_t i = blockIdx.x * THREADS + threadIdx.x, pieces = (uint32_t)a.c.D / N, rh = i / pieces;
    const uint32_t row = rh / (uint32_t)a.c.heads, head = rh % (uint32_t)a.c.heads;
    const int slot = row < a.rows ? slot_of(a, row) : -1, v = (int)(i % pieces) * N;
    if (slot < 0) return;
    const uint64_t rec = record_of(a, slot, (int)head);
    const int64_t at = (int64_t)head * a.c.D + v;
    const int t = slot & (CACHE_TILE - 1);
    const u32x4 k = read_piece<T, K8, false, false>(a.kc + rec * cache_record(K8, a.c.D), a.c.D, t, v >> 5, v & 31);
    const u32x4 w = read_piece<T, V8, true, false>(a.vc + rec * cache_record(V8, a.c.D), a.c.D, t, v >> 5, v & 31);
    *reinterpret_cast<u32x4_any*>(static_cast<T*>(a.ko) + row * a.ldk + at) = k;
    *reinterpret_cast<u32x4_any*>(static_cast<T*>(a.vo) + row * a.ldv + at) = w;
}

// ------------------------------------------------------------------ windows of rows
// A workgroup has R rows of one head's keys or values.
template <int R> struct Window {
    static constexpr int IMAGES = R / CACHE_TILE + 1;       // tiles that consecutive slots can touch
    int tile[IMAGES];                                       // slot / 32, -1 for none or one that is there already
    int64_t row0;
    int rows, head;
    bool value;
    // The image that a slot's tile has, -1 if none
    __device__ int image(int slot) const {
        int at = -1;
#pragma unroll
        for (int j = 0; j < IMAGES; ++j)
            if (slot >= 0 && tile[j] == slot >> 5) at = j;
        return at;
    }
    __device__ uint64_t record(const RowsArgs& a, int j) const { return record_of(a, tile[j] * CACHE_TILE, head); }
    __device__ int slot(const RowsArgs& a, int r) const { return r < rows ? slot_of(a, row0 + r) : -1; }
    __device__ Window(const RowsArgs& a) {
        uint32_t b = blockIdx.x;
        value = b & 1;
        b >>= 1;
        head = (int)(b % (uint32_t)a.c.heads);
        row0 = (int64_t)(b / (uint32_t)a.c.heads) * R;
        rows = a.rows - row0 < R ? (int)(a.rows - row0) : R;
        // consecutive slots touch the tiles of the first row, of every 32nd from it and of the last
#pragma unroll
        for (int j = 0; j < IMAGES; ++j) {
            const int s = slot_of(a, row0 + (j * CACHE_TILE < rows ? j * CACHE_TILE : rows - 1));
            tile[j] = s < 0 ? -1 : s >> 5;
#pragma unroll
            for (int i = 0; i < j; ++i)
                if (tile[i] == tile[j]) tile[j] = -1;
        }
    }
};

// the 8 tokens of group g, in the order of a record's pieces, as bits
__device__ inline uint32_t group_bits(uint32_t covered, int g) {
    return (covered >> (4 * g) & 15) | (covered >> (16 + 4 * g) & 15) << 4;
}

template <typename T, bool Q8, bool VALUE, int R>
__device__ inline void write_window(const RowsArgs& a, const Window<R>& w, uint32_t* covered, uint8_t* images) {
    constexpr int IMAGES = Window<R>::IMAGES;
    const int D = a.c.D, rec = cache_record(Q8, D), halves = D / 16, n = R * halves;
    uint8_t* cache = VALUE ? a.vc : a.kc;
    if (threadIdx.x < IMAGES) covered[threadIdx.x] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += THREADS) {               // every thread: lanes exchange
        const int i = i0 + (int)threadIdx.x;
        const int r = i / halves, half = i % halves;
        const int slot = i < n ? w.slot(a, r) : -1, j = w.image(slot);
        const Item m = item_of(w.row0 + r, w.head, half, D, slot);
        if (j >= 0 && half == 0) atomicOr(&covered[j], 1u << m.t);
        int q[16], other[16];
        const float d = take_item<T, Q8, VALUE>(a, m, slot >= 0, q, other);
        // (two calls: one pointer to either would make its stores ones that do not know which memory)
        if (j >= 0) put_item<Q8, VALUE, true>(a, m, q, other, d, images + j * in_image(rec));
        else if (slot >= 0) put_item<Q8, VALUE, false>(a, m, q, other, d, cache + record_of(a, slot, w.head) * rec);
    }
    __syncthreads();
    const int pieces = rec / 16, values = cache_values(Q8, D) / 16;
#pragma unroll
    for (int j = 0; j < IMAGES; ++j) {
        if (w.tile[j] < 0) continue;
        const uint32_t cover = covered[j];
        uint8_t* there = cache + w.record(a, j) * rec;
        for (int p = (int)threadIdx.x; p < pieces; p += THREADS) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(images + j * in_image(rec) + in_image(p * 16));
            uint8_t* to = there + p * 16;
            const int lane = p % 64, r = lane % 16, g = lane / 16;
            if (p < values && !VALUE) {
                if constexpr (Q8) {                         // one token's
                    if (cover >> (p / 64 / (D / 64) * 16 + r) & 1) *reinterpret_cast<u32x4*>(to) = v;
                } else {                                    // 8 bytes of tokens r and 16 + r
                    if (cover >> r & 1) *reinterpret_cast<u32x2*>(to) = u32x2{v[0], v[1]};
                    if (cover >> (16 + r) & 1) *reinterpret_cast<u32x2*>(to + 8) = u32x2{v[2], v[3]};
                }
                continue;
            }
            // values: two runs of 8 tokens, a byte each; scales: one, two bytes each
            const bool scales = p >= values;
            const uint32_t bits = group_bits(cover, scales ? (p - values) / (D / 32) : g);
            if (bits == 0xFF) {
                *reinterpret_cast<u32x4*>(to) = v;
            } else if (scales) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (bits >> s & 1) reinterpret_cast<uint16_t*>(to)[s] = (uint16_t)(v[s / 2] >> (16 * (s & 1)));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {               // four tokens: of the lower 16, of the upper, twice
                    const uint32_t four = bits >> (4 * (k & 1)) & 15;
                    if (four == 15) {
                        reinterpret_cast<uint32_t*>(to)[k] = v[k];
                    } else {
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            // q4_0 holds the tokens of a run of four in the order 0, 2, 1, 3
                            const int tok = Q8 ? s : (s >> 1) + (s & 1) * 2;
                            if (four >> tok & 1) to[4 * k + s] = (uint8_t)(v[k] >> (8 * s));
                        }
                    }
                }
            }
        }
    }
}

template <typename T, bool K8, bool V8, int R>
__global__ __launch_bounds__(THREADS) void cache_write_window_kernel(RowsArgs a) {
    __shared__ uint32_t covered[Window<R>::IMAGES];         // tokens of an image that rows have
    extern __shared__ __attribute__((aligned(16))) uint8_t images[];
    const Window<R> w(a);
    if (w.value) write_window<T, V8, true>(a, w, covered, images);
    else write_window<T, K8, false>(a, w, covered, images);
}

template <typename T, bool Q8, bool VALUE, int R>
__device__ inline void read_window(const RowsArgs& a, const Window<R>& w, uint8_t* images) {
    const int D = a.c.D, rec = cache_record(Q8, D), pieces = rec / 16;
    const uint8_t* cache = VALUE ? a.vc : a.kc;
#pragma unroll
    for (int j = 0; j < Window<R>::IMAGES; ++j) {
        if (w.tile[j] < 0) continue;
        const uint8_t* there = cache + w.record(a, j) * rec;
        for (int p = (int)threadIdx.x; p < pieces; p += THREADS)
            *reinterpret_cast<u32x4*>(images + j * in_image(rec) + in_image(p * 16)) = *reinterpret_cast<const u32x4*>(there + p * 16);
    }
    __syncthreads();
    // a thread keeps its place in the row (for D = 192 some have none)
    constexpr int N = READ_N<T>;
    const int places = D / N, at_once = THREADS / places, place = (int)threadIdx.x % places, r0 = (int)threadIdx.x / places;
    const int v = place * N;
    T* out = static_cast<T*>(VALUE ? a.vo : a.ko) + w.head * D + v;
    const int64_t ld = VALUE ? a.ldv : a.ldk;
    if (r0 >= at_once) return;
    for (int r = r0; r < R; r += at_once) {
        const int slot = w.slot(a, r), j = w.image(slot), t = slot & (CACHE_TILE - 1);
        if (slot < 0) continue;
        u32x4 x;
        // (two calls: one pointer to either would make its loads ones that do not know which memory)
        if (j >= 0) x = read_piece<T, Q8, VALUE, true>(images + j * in_image(rec), D, t, v >> 5, v & 31);
        else x = read_piece<T, Q8, VALUE, false>(cache + record_of(a, slot, w.head) * rec, D, t, v >> 5, v & 31);
        // Past the caches: 32768 rows of 8 x 128 values in bf16 56 us, and 35.5 so, in f32 79 and 55. With a kernel behind it
        // that reads the rows, 103 and 99, and 173 and 169.5; fewer rows are found in the caches then: 8192 in f32 45 and 48.5.
        __builtin_nontemporal_store(x, reinterpret_cast<u32x4_any*>(out + (w.row0 + r) * ld));
    }
}

template <typename T, bool K8, bool V8, int R>
__global__ __launch_bounds__(THREADS) void cache_read_window_kernel(RowsArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t images[];
    const Window<R> w(a);
    if (w.value) read_window<T, V8, true>(a, w, images);
    else read_window<T, K8, false>(a, w, images);
}

// Values up to which rows go one by one. Measured, one by one against windows: 1003 rows of 4 x 256 (2^20)
// read 4.7 against 6.8 us, 1517 of 3 x 192, a quarter of them kept, written 4.8 against 6.7; 2048 of 8 x 128
// (2^21) written 11.7 against 8.6, read 8.9 against 7.0.
constexpr int64_t FEW = int64_t(3) << 19;
// Windows of 64 rows from which they are taken instead of 32 (which read two tiles for 32 rows, not
// three for 64): 4096 of them 58.3 against 63 us, 256 written 10.0 against 8.6.
constexpr int64_t WIDE = 2048;

// f(the window's rows, workgroups, bytes of the images)
template <typename F> void by_window(int64_t rows, const CacheShape& c, bool k8, bool v8, F f) {
    const auto go = [&](auto r) {
        constexpr int R = decltype(r)::value;
        f(r, dim3((unsigned)(2 * ceil_div(rows, R) * c.heads)),
          (size_t)Window<R>::IMAGES * in_image(std::max(cache_record(k8, c.D), cache_record(v8, c.D))));
    };
    if (rows / 64 * c.heads >= WIDE) go(std::integral_constant<int, 64>());
    else go(std::integral_constant<int, 32>());
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
    a.rows = rows;
    a.c = c;
    a.page_bits = __builtin_ctz(c.tiles * CACHE_TILE);
    by_types(o, tk, tv, [&](auto t, auto k8, auto v8) {
        constexpr bool K = decltype(k8)::value, V = decltype(v8)::value;
        if (rows * c.heads * c.D <= FEW) {
            const int64_t items = rows * c.heads * (c.D / 16);
            hipLaunchKernelGGL((cache_write_kernel<decltype(t), K, V>), dim3((unsigned)ceil_div(items, THREADS)), dim3(THREADS), 0, s,
                               a);
        } else {
            by_window(rows, c, K, V, [&](auto r, dim3 grid, size_t lds) {
                hipLaunchKernelGGL((cache_write_window_kernel<decltype(t), K, V, decltype(r)::value>), grid, dim3(THREADS), lds, s,
                                   a);
            });
        }
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
    a.rows = rows;
    a.c = c;
    a.page_bits = __builtin_ctz(c.tiles * CACHE_TILE);
    by_types(o, tk, tv, [&](auto t, auto k8, auto v8) {
        constexpr bool K = decltype(k8)::value, V = decltype(v8)::value;
        if (rows * c.heads * c.D <= FEW) {
            const int64_t items = rows * c.heads * (c.D / READ_N<decltype(t)>);
            hipLaunchKernelGGL((cache_read_kernel<decltype(t), K, V>), dim3((unsigned)ceil_div(items, THREADS)), dim3(THREADS), 0, s,
                               a);
        } else {
            by_window(rows, c, K, V, [&](auto r, dim3 grid, size_t lds) {
                hipLaunchKernelGGL((cache_read_window_kernel<decltype(t), K, V, decltype(r)::value>), grid, dim3(THREADS), lds, s,
                                   a);
            });
        }
    });
    return hipGetLastError();
}

}  // namespace mmq
