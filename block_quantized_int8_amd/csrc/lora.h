// lora.h - what the adapters' forward and backward kernels share (lora.hip, lora_grad.hip): the
// matrix-core operands, the exact split of f32 values into bf16 terms, and the launchers.
//
// Operands of v_mfma_f32_16x16x32_{bf16,f16}, lane L = 16g + c (g < 4, c < 16): the A operand
// holds row c's and the B operand column c's values k = 8g .. 8g+7 of the 32-deep step; the
// accumulator holds rows 4g .. 4g+3 of column c.
//
// Products keep f32: an f32 value is exactly the sum of three bf16 terms of 8 significand bits
// each (an f16 value of two), so a product of terms is exact in f32 and only the accumulation
// rounds. Terms are cut off, not rounded, so that the rest is exact and of the same sign: the second
// is below 2^-7 of the value, the third below 2^-15. Only the pair of two third terms, below
// 2^-30 of the product, is left out; without the pairs of a second and a third too, a product
// would be up to 2^-21 of itself too small.
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

// four f32 values to three planes of bf16 terms, `plane` values apart
__device__ inline void store_terms(uint16_t* at, int64_t plane, f32x4 d) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        u32x2 w;
        w[0] = pack_hi(d[0], d[1]);
        w[1] = pack_hi(d[2], d[3]);
        *reinterpret_cast<u32x2*>(at + k * plane) = w;
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] -= cut(d[j]);
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

// Rows of 16-byte pieces are loaded with four consecutive lanes on a row's 64 bytes (lane 4c + g:
// row c, piece g), one cache access for each four lanes; an operand wants lane 16g + c there. In
// the operand's own order every lane is an access of its own (49 of them for a load of 64 lanes),
// and the adapters' loads then bound the forward kernels: 17.5 us against 11.7 for the down
// kernel at 2048 x 4096, rank 64. The pieces turn in a wave's own 1 KB of LDS.
__device__ inline int piece_row(int lane) { return lane >> 2; }
__device__ inline int piece_of(int lane) { return lane & 3; }
__device__ inline int piece_at(int lane) { return 4 * (lane & 15) + (lane >> 4); }   // the operand's piece
// An operand from a row-major LDS tile with the operand's k along the rows (k = 8g .. 8g+7, 16
// columns from `tile` on): lane i of 16 gives the address of four values of row i / 4 and gets
// column i of the four rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ inline u32x4 turned_operand(const uint16_t* tile, int ld, int lane) {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const uint16_t* p = tile + (8 * (lane >> 4) + (lane & 15) / 4) * ld + 4 * (lane & 3);
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * ld)));
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
}
// LDS written by a wave's lanes is read by its other lanes (no other wave is concerned)
__device__ inline void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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
        acc = mfma_bf16(w.t[1], x[2], acc);
        acc = mfma_bf16(w.t[1], x[1], acc);
        acc = mfma_bf16(w.t[0], x[2], acc);
        acc = mfma_bf16(w.t[1], x[0], acc);
    } else {
        acc = mfma_bf16(w.t[0], x[2], acc);
    }
    acc = mfma_bf16(w.t[0], x[1], acc);
    return mfma_bf16(w.t[0], x[0], acc);
}

// the same with the f32 values as A: their rows are the accumulator's
template <bool F16>
__device__ inline f32x4 terms_mfma(const u32x4* x, const Weights<F16>& w, f32x4 acc) {
    if constexpr (F16) {
        acc = mfma_bf16(x[2], w.t[1], acc);
        acc = mfma_bf16(x[1], w.t[1], acc);
        acc = mfma_bf16(x[2], w.t[0], acc);
        acc = mfma_bf16(x[0], w.t[1], acc);
    } else {
        acc = mfma_bf16(x[2], w.t[0], acc);
    }
    acc = mfma_bf16(x[1], w.t[0], acc);
    return mfma_bf16(x[0], w.t[0], acc);
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

// Four values of an f32 or bf16 row, as they lie in memory: a load that is turned into f32 at once
// has to be waited for at once.
template <bool BF16> struct Quad { typedef f32x4 Raw; };
template <> struct Quad<true> { typedef u32x2 Raw; };
template <bool BF16> __device__ inline typename Quad<BF16>::Raw load_quad(const void* p, int64_t at) {
    if constexpr (BF16) return *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(p) + at);
    else return *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + at);
}
// At a row's end a quad is loaded from the last place that is whole, n - off, and what lies before n
// is dropped once it is used (zeros come in behind it): no lane takes a branch of its own, in which
// it would wait for its load. Rows of less than four values are loaded value by value.
struct QuadEnd {
    int at, off;
    __device__ QuadEnd(int n, int N) : at(N < 4 ? n : min(n, N - 4)), off(n - at) {}
};
template <bool BF16> __device__ inline typename Quad<BF16>::Raw load_quad_end(const void* p, int64_t row, QuadEnd q, int N) {
    if (N >= 4) return load_quad<BF16>(p, row + q.at);
    typename Quad<BF16>::Raw r = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (q.at + j < N) {
            if constexpr (BF16) r[j / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[row + q.at + j] << (16 * (j & 1));
            else r[j] = static_cast<const float*>(p)[row + q.at + j];
        }
    return r;
}
__device__ inline u32x2 drop_quad(u32x2 r, int off) {
    const uint64_t v = off < 4 ? __builtin_bit_cast(uint64_t, r) >> (16 * off) : 0;
    return __builtin_bit_cast(u32x2, v);
}
__device__ inline f32x4 drop_quad(f32x4 r, int off) {
    if (off & 1) r = f32x4{r[1], r[2], r[3], 0.f};
    if (off & 2) r = f32x4{r[2], r[3], 0.f, 0.f};
    return off < 4 ? r : f32x4(0);
}
__device__ inline f32x4 quad_f32(f32x4 r) { return r; }
__device__ inline f32x4 quad_f32(u32x2 r) {
    return f32x4{as_f(r[0] << 16), as_f(r[0] & 0xFFFF0000u), as_f(r[1] << 16), as_f(r[1] & 0xFFFF0000u)};
}

template <bool BF16> __device__ inline void store4(void* p, int64_t at, f32x4 v, int left) {
    if constexpr (BF16) {
        uint16_t* q = static_cast<uint16_t*>(p) + at;
        if (left >= 4) {
            u32x2 w;
#pragma unroll
            for (int j = 0; j < 2; ++j) w[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
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
    uint16_t* planes;           // three bf16 terms of s_e v or u: [3][R/8][M][8] by sorted position
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

// The plan's entries, held inside the buffers: a plan that was made for another batch gives
// meaningless results, but no access outside them and no endless loop.
__device__ inline int4 unit_at(const LoraArgs& a, int u) {
    int4 v = a.units[u];
    v.x = v.x < 0 ? a.E : v.x;
    v.y = min(max(v.y, 0), a.M);
    v.z = min(max(v.z, 0), min(GROUP_UNIT, a.M - v.y));
    return v;
}
__device__ inline int row_at(const LoraArgs& a, int pos) { return (int)min((uint32_t)a.order[pos], (uint32_t)a.M - 1u); }
__device__ inline int2 rows_of_group(const LoraArgs& a, int e) {
    const int p0 = min(max(a.offs[e], 0), a.M);
    return make_int2(p0, min(max(a.offs[e + 1], p0), a.M));
}

// The planes' values of ranks r .. of a position: eight ranks of consecutive positions lie side by
// side, so that a matrix-core operand of 16 positions is loaded in whole cache lines.
__device__ inline uint16_t* plane_at(const LoraArgs& a, int pos, int r) {
    return a.planes + (((int64_t)(r >> 3) * a.M + pos) * 8 + (r & 7));
}

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

// out = base + the rows' planes (s_e v, or u) times a weight matrix, for 16 rows x 64 columns a wave:
// waves 0-3 of a workgroup of W waves have the row tiles of a unit, each further four the next 64
// columns. The weights of up to 64 ranks go through LDS as bf16 terms, once for the four row
// tiles: rows of ranks for each column (B_e, TR false) or of columns for each rank (A_e, TR true).
// Operand mapping: A = the rows' planes, B = the columns; a lane ends with four rows, of four
// consecutive columns (TR false: column 4c + i of tile i) or of one (TR true: column 16i + c).
template <bool TR, bool F16, int W> struct ExpandLds {
    static constexpr int T = Weights<F16>::T, COLS = 16 * W;       // columns of the workgroup
    static constexpr int ROWS = TR ? LORA_RC : COLS, LD = (TR ? COLS : LORA_RC) + 8;
    uint16_t w[T][ROWS][LD];
};

template <bool TR, bool F16, bool BF16, bool TAIL, int W>
__device__ inline void expand_body(const LoraArgs& a, const uint16_t* weights, int C, const void* base_, int64_t ldb,
                                   void* out, int64_t ldo, int4 unit, int tile, ExpandLds<TR, F16, W>& lds) {
    using L = ExpandLds<TR, F16, W>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4, t = wave & 3;
    const int c0 = tile * L::COLS, n0 = c0 + 64 * (wave >> 2), n = n0 + (TR ? c : 4 * c);
    const bool none = unit.x >= a.E, live = 16 * t < unit.z && n0 < C;
    const uint16_t* w0 = weights + (none ? 0 : (int64_t)unit.x * C * a.R);

    int m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = row_at(a, unit.y + min(16 * t + 4 * g + j, unit.z - 1));
    f32x4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f32x4(none ? -0.f : 0.f);     // base + -0 is the base, -0 too
    typename Quad<BF16>::Raw base[4];
#pragma unroll 1
    for (int r0 = 0; r0 < a.R; r0 += LORA_RC) {
        const int rc = min(a.R - r0, LORA_RC);
        // pieces of eight values: eight of 64 ranks for each column, or COLS / 8 for each rank
        constexpr int PER = TR ? L::COLS / 8 : LORA_RC / 8, PIECES = L::ROWS * PER / (64 * W);
        u32x4 raw[PIECES];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int idx = i * 64 * W + (int)threadIdx.x, row = idx / PER, p = 8 * (idx % PER);
            raw[i] = 0;                                    // zeros past R and past the columns
            if constexpr (TR) {
                if (row < rc && c0 + p < C && !none) raw[i] = *reinterpret_cast<const u32x4*>(w0 + (int64_t)(r0 + row) * C + c0 + p);
            } else {
                if (p < rc && c0 + row < C && !none) raw[i] = *reinterpret_cast<const u32x4*>(w0 + (int64_t)(c0 + row) * a.R + r0 + p);
            }
        }
        // the row tile's planes: row c, ranks 8g .. of both steps; zeros past the unit and past R
        u32x4 x[2][3];
        const int at = 16 * t + c;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = r0 + 32 * k + 8 * g;
            const bool ok = live && !none && at < unit.z && r < a.R;
            const uint16_t* p = plane_at(a, unit.y + at, r);
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                x[k][j] = 0;
                if (ok) x[k][j] = *reinterpret_cast<const u32x4*>(p + (int64_t)j * a.M * a.R);
            }
        }
        if (r0 == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                base[j] = 0;
                if (!base_ || !live) continue;
                if constexpr (TR) {
                    const float* p = static_cast<const float*>(base_) + m[j] * ldb + n;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n0 + 16 * i < C) base[j][i] = p[16 * i];
                } else {
                    if constexpr (TAIL) base[j] = load_quad_end<BF16>(base_, m[j] * ldb, QuadEnd(n, C), C);
                    else if (n < C) base[j] = load_quad<BF16>(base_, m[j] * ldb + n);
                }
            }
        } else {
            __syncthreads();
        }
        __builtin_amdgcn_sched_barrier(0);                 // every load is issued before the first wait
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int idx = i * 64 * W + (int)threadIdx.x, row = idx / PER, p = 8 * (idx % PER);
            Weights<F16> w;
            w.set(raw[i]);
            const int to = TR ? row : (row & ~63) + 16 * (row & 3) + ((row & 63) >> 2);
#pragma unroll
            for (int j = 0; j < L::T; ++j) *reinterpret_cast<u32x4*>(&lds.w[j][to][p]) = w.t[j];
        }
        __syncthreads();
        if (!live || none) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (32 * k >= rc) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Weights<F16> w;
#pragma unroll
                for (int j = 0; j < L::T; ++j)
                    w.t[j] = TR ? turned_operand(&lds.w[j][32 * k][n0 - c0 + 16 * i], L::LD, lane)
                                : *reinterpret_cast<const u32x4*>(&lds.w[j][n0 - c0 + 16 * i + c][32 * k + 8 * g]);
                acc[i] = terms_mfma<F16>(x[k], w, acc[i]);
            }
        }
    }
    if (!live) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (16 * t + 4 * g + j >= unit.z) continue;
        if constexpr (TR) {
            float* p = static_cast<float*>(out) + m[j] * ldo + n;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n0 + 16 * i < C) p[16 * i] = base[j][i] + acc[i][j];
        } else if (n < C) {
            f32x4 o = quad_f32(TAIL ? drop_quad(base[j], QuadEnd(n, C).off) : base[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] += acc[i][j];
            store4<BF16>(out, m[j] * ldo + n, o, TAIL ? C - n : 4);
        }
    }
}

size_t lora_workspace_bytes(int64_t E, int64_t M, int64_t N, int64_t K, int64_t R);
bool lora_grid_ok(int64_t E, int64_t M, int64_t N, int64_t K);
hipError_t launch_lora(mmq_atype t, bool f16, const void* act, const void* A, const void* B, const float* scale,
                       int64_t E, int64_t R, const void* plan, int64_t M, int64_t N, int64_t K, const void* base,
                       int64_t ldb, void* out, int64_t ldo, float* v, void* ws, hipStream_t s);
size_t lora_grad_workspace_bytes(int64_t E, int64_t M, int64_t N, int64_t R);
bool lora_grad_grid_ok(int64_t E, int64_t M, int64_t N, int64_t K);
hipError_t launch_lora_grad(mmq_atype t, bool f16, const void* act, const void* A, const void* B, const float* scale,
                            int64_t E, int64_t R, const void* plan, int64_t M, int64_t N, int64_t K, const float* v,
                            const void* dy, int64_t lddy, const float* dxb, int64_t lddxb, float* dx, int64_t lddx,
                            float* dA, float* dB, void* ws, hipStream_t s);

}  // namespace mmq
