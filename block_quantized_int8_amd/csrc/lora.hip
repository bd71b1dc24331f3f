// lora.hip - low-rank adapters of many requests beside a shared projection:
//     v[m] = A_e x^[m],   out[m] = base[m] + s_e B_e v[m],   e the row's adapter (or none)
// on the act buffer that the projection reads and the output that it wrote.
//
// Two launches over the plan's units (up to 64 rows of one adapter):
//   1. lora_down_kernel: v. A workgroup has 16 of a unit's rows and one of S parts of K; its
//      eight waves take consecutive blocks of the part and join in LDS. The int8 values enter
//      the matrix core as they are (exact in bf16 and f16), each block's product is scaled by
//      its f32 scale; the per-token form accumulates on the matrix core.
//   2. s_e B_e v added to the base: lora_expand_kernel where K is not split (rows enough to fill the
//      chip), from the terms of s_e v that the first launch leaves; lora_up_kernel otherwise, which
//      sums the S parts in order and makes the terms itself.
// For few rows lora_small_kernel does both in one launch.
// Loops over rows stay loops: a launch fetches its code cold, and with the four row tiles
// unrolled (25 KB of code) the second launch took 13.8 us on 517 x 1536 instead of 5.4.
#include <algorithm>

#include "lora.h"

namespace mmq {
namespace {

constexpr int DW = 8;               // waves of a down workgroup
constexpr int MAX_PARTS = 8;

// acc += the adapter's rows (pieces at A + aoff) times one lane's activations over the blocks
// [b0, b1), turned in the wave's own LDS.
// Operand mapping: A = the adapter's rows r (lane c: rank 16i + c of tile i), B = the
// activations (lane c: row c of the 16), so a lane ends with four consecutive ranks of a row.
// NB blocks are loaded before the first is used.
template <int RT, int NB, bool F16, bool Q81>
__device__ inline void down_blocks(const uint16_t* A, const uint32_t (&aoff)[RT], const int8_t* xrow, const uint16_t* srow,
                                   int b0, int b1, u32x4 (*lds)[64], int lane, f32x4 (&acc)[RT]) {
#pragma unroll 1
    for (int b = b0; b < b1; b += NB) {
        u32x4 w[NB][RT];
        u32x2 q[NB];
        uint16_t xs[NB];
#pragma unroll
        for (int i = 0; i < RT; ++i)                       // a row's bytes in a row: whole cache lines
#pragma unroll
            for (int k = 0; k < NB; ++k)
                w[k][i] = *reinterpret_cast<const u32x4*>(A + (aoff[i] + (uint32_t)min(b + k, b1 - 1) * 32u));
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const uint32_t bk = (uint32_t)min(b + k, b1 - 1);
            q[k] = *reinterpret_cast<const u32x2*>(xrow + (uint64_t)bk * 1024);
            if constexpr (Q81) xs[k] = srow[bk * 64u];
        }
        __builtin_amdgcn_sched_barrier(0);                 // every load is issued before the first use
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int i = 0; i < RT; ++i) lds[k * RT + i][lane] = w[k][i];
        wave_lds_fence();
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            if (b + k >= b1) q[k] = 0;                     // the last block's repeat adds nothing
            const u32x4 x = int8_operand<F16>(q[k]);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const u32x4 ww = lds[k * RT + i][piece_at(lane)];
                const f32x4 from = Q81 ? f32x4(0) : acc[i];
                const f32x4 d = F16 ? mfma_f16(ww, x, from) : mfma_bf16(ww, x, from);
                if constexpr (Q81) {
                    const float f = (float)__builtin_bit_cast(_Float16, xs[k]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(f, d[j], acc[i][j]);
                } else {
                    acc[i] = d;
                }
            }
        }
        wave_lds_fence();
    }
}

// 2048 rows of 8 adapters, K = 4096, rank 64: 12.6 us. Bound by what the CUs' L1s take: the rows' A is
// read again for each 16 rows, 81 MB in all (the same with 16 waves, with the ranks split over
// two or four workgroups, or with half the L2 misses by keeping an adapter's rows on one XCD: 12.8
// to 15.5 us; 64 rows a workgroup need 216 registers: 15.5 us).
template <int RT, bool F16, bool Q81>
__global__ __launch_bounds__(DW * 64) void lora_down_kernel(LoraArgs a) {
    constexpr int NB = RT == 1 ? 4 : 2;
    __shared__ u32x4 lds[DW][NB * RT][64];      // each wave's pieces; the waves' sums at the end
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    // a unit's first 16 rows come first in the grid (units of few rows have no others); the part
    // turns with the unit, so that no XCD's L2 gets the same columns of every row of the adapters
    // (those are a few of its channels only: 14 us against 6.5 for 64 rows of 32 adapters)
    const int at = (int)blockIdx.x / a.S, s = ((int)blockIdx.x + at) % a.S;
    const int sub = at / a.nunits;
    const int4 unit = unit_at(a, at - sub * a.nunits);
    const int rows = min(unit.z - 16 * sub, 16);
    if (rows <= 0 || unit.x >= a.E) return;
    const int p0 = unit.y + 16 * sub, r0 = (int)blockIdx.y * 16 * RT;

    const int parts = a.S * DW, per = (a.KB + parts - 1) / parts;      // blocks of a wave
    const int b0 = (s * DW + wave) * per, b1 = min(b0 + per, a.KB);
    // rows past the unit's last repeat it; their columns are not stored. Ranks past R likewise.
    const int m = row_at(a, p0 + min(c, rows - 1));
    const uint16_t* A = a.A + (int64_t)unit.x * a.R * a.K;
    uint32_t aoff[RT];                          // R * K is 2^31 values at most
#pragma unroll
    for (int i = 0; i < RT; ++i)
        aoff[i] = (uint32_t)min(r0 + 16 * i + piece_row(lane), a.R - 1) * (uint32_t)a.K + 8u * piece_of(lane);
    const int64_t tile = (int64_t)(m >> 5) * a.KBp;
    const int8_t* xrow = a.xq + tile * 1024 + ((g >> 1) * 32 + (m & 31)) * 16 + (g & 1) * 8;
    const uint16_t* srow = reinterpret_cast<const uint16_t*>(a.xs2 + tile * 32 + (m & 31));

    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = 0;
    down_blocks<RT, NB, F16, Q81>(A, aoff, xrow, srow, b0, b1, lds[wave], lane, acc);
    // the waves' sums: wave i joins and stores tile i
#pragma unroll
    for (int i = 0; i < RT; ++i) lds[wave][i][lane] = __builtin_bit_cast(u32x4, acc[i]);
    __syncthreads();
    if (wave >= RT) return;
    f32x4 d = 0;
#pragma unroll
    for (int w = 0; w < DW; ++w) d += __builtin_bit_cast(f32x4, lds[w][wave][lane]);
    const int r = r0 + 16 * wave + 4 * g;
    if (c >= rows || r >= a.R) return;
    if constexpr (!Q81) d *= a.sa[m];
    const int64_t to = (int64_t)(p0 + c) * a.R + r;
    if (a.S > 1) {
        *reinterpret_cast<f32x4*>(a.part + (int64_t)s * a.M * a.R + to) = d;
    } else {
        *reinterpret_cast<f32x4*>(a.v + (int64_t)m * a.R + r) = d;
        store_terms(plane_at(a, p0 + c, r), (int64_t)a.M * a.R, d * a.scale[unit.x]);
    }
}

// 2048 rows x 4096 columns, rank 64: 14.5 us for 67 MB of base and output (4.6 TB/s; an elementwise
// kernel on as much takes 10.5 to 13). Without the planes, each wave making its rows' terms
// (lora_up_kernel): 19.3 us.
template <bool F16, bool BF16, bool TAIL>
__global__ __launch_bounds__(LT) void lora_expand_kernel(LoraArgs a, int ntiles) {
    __shared__ __attribute__((aligned(16))) ExpandLds<false, F16, 4> lds;
    const int u = (int)blockIdx.x / ntiles, tile = (int)blockIdx.x % ntiles;
    const int4 unit = unit_at(a, u);
    if (unit.z == 0) return;
    if (unit.x >= a.E && tile == 0)                         // rows without an adapter: v = 0
        for (int i = 8 * threadIdx.x; i < unit.z * a.R; i += 8 * LT) {
            float* to = a.v + (int64_t)row_at(a, unit.y + i / a.R) * a.R + i % a.R;
            *reinterpret_cast<f32x4*>(to) = *reinterpret_cast<f32x4*>(to + 4) = 0;
        }
    expand_body<false, F16, BF16, TAIL, 4>(a, a.B, a.N, a.base, a.ldb, a.out, a.ldo, unit, tile, lds);
}

// Operand mapping: A = the rows' v (lane c: row c of 16), B = the adapter's columns (lane c:
// column n + i of tile i, n = 4c), so a lane ends with four consecutive columns of each of its four
// rows and 16 lanes write 256 contiguous bytes. A wave has 64 columns of 16 rows (`tall`: the
// workgroup's four waves the unit's rows; else 256 columns, rows past 16 in a loop) and works
// alone: its loads depend on the unit, and the base on its rows, and on nothing else. RK: steps of
// 32 ranks, their operands held; 0 for any number, loaded step by step. TAIL: N % 4 != 0.
// 64 rows of 32 adapters, N = 14336, rank 32, f16: 11.5 us for 36 MB (3.2 TB/s). Half of it is
// vector instructions (464 a wave, of which about 130 split f16 weights, each of them once; 3450 a
// SIMD); the rest are latencies, as a wave has one strip of columns and no other's loads in flight.
template <int RK, bool F16, bool BF16, bool TAIL>
__global__ __launch_bounds__(LT) void lora_up_kernel(LoraArgs a, int ntiles, int tall) {
    constexpr int H = RK ? RK : 1;                          // steps held
    __shared__ u32x4 turn[LT / 64][4 * H][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int u = (int)blockIdx.x / ntiles, tile = (int)blockIdx.x % ntiles;
    const int4 unit = unit_at(a, u);
    const int nt = (unit.z + 15) >> 4;
    const int t0 = tall ? wave : 0, group = tall ? tile : 4 * tile + wave;
    const int n0 = 64 * group, n = n0 + 4 * c, left = a.N - n;
    if (t0 >= nt || n0 >= a.N) return;
    const bool none = unit.x >= a.E;
    const uint16_t* B = a.B + ((int64_t)(none ? 0 : unit.x) * a.N + n0) * a.R;
    const uint32_t col = 4u * piece_row(lane), last = (uint32_t)(a.N - 1 - n0);

    // the columns' pieces of rank step k, zeros past R
    auto pieces = [&](int k, int at) {
        const uint32_t r = 32u * k + 8u * piece_of(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u32x4 raw = 0;
            if (r < (uint32_t)a.R) raw = *reinterpret_cast<const u32x4*>(B + min(col + i, last) * (uint32_t)a.R + r);
            turn[wave][at + i][lane] = raw;
        }
    };
    // the rows' v of rank step k (the parts in order) as three terms; zeros past the unit and R.
    // The first columns' wave keeps it
    auto v_of = [&](int t, int k, u32x4* x) {
        const int at = 16 * t + c, r = 32 * k + 8 * g;
        f32x4 d[2] = {0, 0};
        if (at < unit.z && r < a.R) {
            if (!none) {
                const float* p = a.part + ((int64_t)unit.y + at) * a.R + r;
#pragma unroll 1
                for (int s = 0; s < a.S; s += 4) {
                    f32x4 q[4][2];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (s + j < a.S) {
                            q[j][0] = *reinterpret_cast<const f32x4*>(p);
                            q[j][1] = *reinterpret_cast<const f32x4*>(p + 4);
                            p += (int64_t)a.M * a.R;
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (s + j < a.S) {
                            d[0] += q[j][0];
                            d[1] += q[j][1];
                        }
                }
            }
            if (group == 0) {
                float* to = a.v + (int64_t)row_at(a, unit.y + at) * a.R + r;
                *reinterpret_cast<f32x4*>(to) = d[0];
                *reinterpret_cast<f32x4*>(to + 4) = d[1];
            }
        }
        const float f[8] = {d[0][0], d[0][1], d[0][2], d[0][3], d[1][0], d[1][1], d[1][2], d[1][3]};
        split3(f, x);
    };
    int m[4];
    auto rows_of = [&](int t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = row_at(a, unit.y + min(16 * t + 4 * g + j, unit.z - 1));
    };

    rows_of(t0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (RK != 0)
        if (!none)
#pragma unroll
            for (int k = 0; k < RK; ++k) pieces(k, 4 * k);
    const float scale = none ? 0.f : a.scale[unit.x];
#pragma unroll 1
    for (int t = t0; t < nt; t += tall ? 4 : 1) {
        typename Quad<BF16>::Raw base[4];
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] = 0;
            base[j] = 0;
            if (!a.base) continue;
            if constexpr (TAIL) base[j] = load_quad_end<BF16>(a.base, m[j] * a.ldb, QuadEnd(n, a.N), a.N);
            else if (left > 0) base[j] = load_quad<BF16>(a.base, m[j] * a.ldb + n);
        }
        __builtin_amdgcn_sched_barrier(0);
        wave_lds_fence();
        if constexpr (RK != 0) {
#pragma unroll
            for (int k = 0; k < RK; ++k) {
                u32x4 x[3];
                v_of(t, k, x);
                if (none) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Weights<F16> w;
                    w.set(turn[wave][4 * k + i][piece_at(lane)]);
                    acc[i] = terms_mfma<F16>(x, w, acc[i]);
                }
            }
        } else {
#pragma unroll 1
            for (int k = 0; 32 * k < a.R; ++k) {
                u32x4 x[3];
                v_of(t, k, x);
                if (none) continue;
                wave_lds_fence();
                pieces(k, 0);
                wave_lds_fence();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Weights<F16> w;
                    w.set(turn[wave][i][piece_at(lane)]);
                    acc[i] = terms_mfma<F16>(x, w, acc[i]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (left > 0 && 16 * t + 4 * g + j < unit.z) {
                f32x4 o = quad_f32(TAIL ? drop_quad(base[j], QuadEnd(n, a.N).off) : base[j]);
                if (!none)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = fmaf(scale, acc[i][j], o[i]);
                store4<BF16>(a.out, m[j] * a.ldo + n, o, TAIL ? left : 4);
            }
        if (!tall && t + 1 < nt) rows_of(t + 1);
    }
}

// Both steps in one launch, for few rows: a workgroup has 16 of a unit's rows and 1024 columns, makes
// v for itself (its sixteen waves share K) and multiplies. The adapters' A is read again for each
// 1024 columns; a second launch and the parts' way through memory are saved.
constexpr int SW = 16;              // waves
constexpr int SMALL_COLS = 64 * SW;

template <int RT, bool F16, bool Q81, bool TAIL>
__global__ __launch_bounds__(SW * 64) void lora_small_kernel(LoraArgs a, int ntiles, int subs) {
    constexpr int NB = RT == 1 ? 4 : 2, RK = RT == 4 ? 2 : 1, LD = 32 * RK + 8;
    static_assert(NB * RT >= 4 * RK, "the columns' pieces use the blocks' memory");
    constexpr bool BF16 = !Q81;
    __shared__ u32x4 lds[SW][NB * RT][64];
    __shared__ __attribute__((aligned(16))) uint16_t vt[3][16][LD];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int tile = (int)blockIdx.x % ntiles, us = (int)blockIdx.x / ntiles, u = us / subs, sub = us - u * subs;
    const int4 unit = unit_at(a, u);
    const bool none = unit.x >= a.E;
    const int64_t e = none ? 0 : unit.x;
    const int n0 = tile * SMALL_COLS + 64 * wave, n = n0 + 4 * c, left = a.N - n;
    // Sixteen rows of the unit, whose `subs` workgroups a tile of columns take them all (one where the
    // batch has no more): the loop ends after one turn. It stays one for its schedule: straight code
    // took 12.8 us on 300 rows, 2048 x 2048, rank 40, bf16 (12.3 so), 7.4 on one row (7.3), and 12.1
    // on 517 rows, 1536 x 4096, rank 24, f16 (12.3).
#pragma unroll 1
    for (int s0 = sub; 16 * s0 < unit.z; s0 += subs) {
        const int rows = min(unit.z - 16 * s0, 16), p0 = unit.y + 16 * s0;
        f32x4 acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = 0;
        const int m = row_at(a, p0 + min(c, rows - 1));
        if (!none) {
            const int per = (a.KB + SW - 1) / SW, b0 = wave * per, b1 = min(b0 + per, a.KB);
            const uint16_t* A = a.A + e * a.R * a.K;
            uint32_t aoff[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i)
                aoff[i] = (uint32_t)min(16 * i + piece_row(lane), a.R - 1) * (uint32_t)a.K + 8u * piece_of(lane);
            const int64_t cell = (int64_t)(m >> 5) * a.KBp;
            const int8_t* xrow = a.xq + cell * 1024 + ((g >> 1) * 32 + (m & 31)) * 16 + (g & 1) * 8;
            const uint16_t* srow = reinterpret_cast<const uint16_t*>(a.xs2 + cell * 32 + (m & 31));
            down_blocks<RT, NB, F16, Q81>(A, aoff, xrow, srow, b0, b1, lds[wave], lane, acc);
        }
        // the columns' pieces and the base are on their way while the waves join
        u32x4 raw[RK][4];
        typename Quad<BF16>::Raw base[4];
        int to[4];
        const uint16_t* B = a.B + (e * a.N + n0) * a.R;
        const uint32_t col = 4u * piece_row(lane), last = (uint32_t)max(a.N - 1 - n0, 0);
#pragma unroll
        for (int k = 0; k < RK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t r = 32u * k + 8u * piece_of(lane);
                raw[k][i] = 0;
                if (r < (uint32_t)a.R && n0 < a.N && !none)
                    raw[k][i] = *reinterpret_cast<const u32x4*>(B + min(col + i, last) * (uint32_t)a.R + r);
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = row_at(a, p0 + min(4 * g + j, rows - 1));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            base[j] = 0;
            if (!a.base) continue;
            if constexpr (TAIL) base[j] = load_quad_end<BF16>(a.base, to[j] * a.ldb, QuadEnd(n, a.N), a.N);
            else if (left > 0) base[j] = load_quad<BF16>(a.base, to[j] * a.ldb + n);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < RT; ++i) lds[wave][i][lane] = __builtin_bit_cast(u32x4, acc[i]);
        __syncthreads();
        if (wave < 2 * RK) {                               // wave i: ranks 16i .., zeros past R
            f32x4 d = 0;
            const int r = 16 * wave + 4 * g;
            if (wave < RT && r < a.R) {
#pragma unroll
                for (int w = 0; w < SW; ++w) d += __builtin_bit_cast(f32x4, lds[w][wave][lane]);
                if constexpr (!Q81)
                    if (!none) d *= a.sa[m];           // 0 without an adapter, whatever the row's scale is
                if (tile == 0 && c < rows) *reinterpret_cast<f32x4*>(a.v + (int64_t)m * a.R + r) = d;
            }
            store_terms(&vt[0][c][r], 16 * LD, d);
        }
        __syncthreads();
        if (n0 < a.N) {
            const float scale = none ? 0.f : a.scale[e];
            f32x4 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = 0;
#pragma unroll
            for (int k = 0; k < RK; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) lds[wave][4 * k + i][lane] = raw[k][i];
            wave_lds_fence();
            if (!none)
#pragma unroll
                for (int k = 0; k < RK; ++k) {
                    u32x4 x[3];
#pragma unroll
                    for (int j = 0; j < 3; ++j) x[j] = *reinterpret_cast<const u32x4*>(&vt[j][c][32 * k + 8 * g]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        Weights<F16> w;
                        w.set(lds[wave][4 * k + i][piece_at(lane)]);
                        o[i] = terms_mfma<F16>(x, w, o[i]);
                    }
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (left > 0 && 4 * g + j < rows) {
                    f32x4 d = quad_f32(TAIL ? drop_quad(base[j], QuadEnd(n, a.N).off) : base[j]);
                    if (!none)
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[i] = fmaf(scale, o[i][j], d[i]);
                    store4<BF16>(a.out, to[j] * a.ldo + n, d, TAIL ? left : 4);
                }
        }
        __syncthreads();
    }
}

// One launch while the adapters' A, read again for each 1024 columns of each 16 rows, come to 32 MB at
// most: it saves the host 4 us a call. Measured: one row 4096 x 4096, rank 16: 7.1 us against 4.2 +
// 4.9 in two launches; 517 rows of 6 adapters 1536 x 4096, rank 24 (15 MB): 10.4 against 4.8 + 5.4;
// 64 rows of 32 adapters 14336 x 4096, rank 32 (132 MB): 34 against 6.0 + 11.7.
bool small_call(int64_t E, int64_t M, int64_t N, int64_t K, int64_t R) {
    const int64_t tiles = ceil_div(M, 16) + std::min(E, M);
    return R <= 64 && K * R <= (int64_t(1) << 18) && tiles * ceil_div(N, SMALL_COLS) * K * R <= (int64_t(1) << 24);
}

// Parts that K is split into: a power of two that gives up to 128 workgroups of the first launch, a
// block a wave at least. Each part is read again by every workgroup of the second. Measured (us a
// call) with up to 64, 128, 256 and 512 workgroups: 64 rows of 32 adapters, N = 14336, K = 4096, rank
// 32: 25.0, 15.7, 15.5, 17.5; 200 rows of 4, 8192 x 8192, rank 64: 18.4, 16.3, 17.3, 17.5; 600 rows
// of 8, 8192 x 4096, rank 64: 22.8, 23.0, 29.3, 39.6; 300 rows of 2, 4096 x 11008, rank 128: 24.3,
// 25.4, 32.6, 32.5.
int64_t down_parts(int64_t E, int64_t M, int64_t K) {
    const int64_t tiles = ceil_div(M, 16) + std::min(E, M);
    int64_t S = 1;
    while (S < MAX_PARTS && 2 * S * tiles <= 128 && 2 * S * DW <= K / QK) S *= 2;
    return S;
}

template <bool F16, bool Q81>
void launch_down(const LoraArgs& a, hipStream_t s) {
    const int rt = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4;
    const dim3 grid((unsigned)a.nunits * 4 * a.S, (unsigned)ceil_div(a.R, 16 * rt));
    if (rt == 1) hipLaunchKernelGGL((lora_down_kernel<1, F16, Q81>), grid, dim3(DW * 64), 0, s, a);
    else if (rt == 2) hipLaunchKernelGGL((lora_down_kernel<2, F16, Q81>), grid, dim3(DW * 64), 0, s, a);
    else hipLaunchKernelGGL((lora_down_kernel<4, F16, Q81>), grid, dim3(DW * 64), 0, s, a);
}

template <bool F16, bool Q81, bool TAIL>
void launch_small(const LoraArgs& a, hipStream_t s) {
    const int ntiles = (int)ceil_div(a.N, SMALL_COLS), subs = a.M > 16 ? 4 : 1;
    const dim3 grid((unsigned)(a.nunits * subs * ntiles)), th(SW * 64);
    if (a.R <= 16) hipLaunchKernelGGL((lora_small_kernel<1, F16, Q81, TAIL>), grid, th, 0, s, a, ntiles, subs);
    else if (a.R <= 32) hipLaunchKernelGGL((lora_small_kernel<2, F16, Q81, TAIL>), grid, th, 0, s, a, ntiles, subs);
    else hipLaunchKernelGGL((lora_small_kernel<4, F16, Q81, TAIL>), grid, th, 0, s, a, ntiles, subs);
}
template <bool F16, bool Q81>
void launch_small(const LoraArgs& a, hipStream_t s) {
    if (a.N % 4) launch_small<F16, Q81, true>(a, s);
    else launch_small<F16, Q81, false>(a, s);
}

template <bool F16, bool BF16, bool TAIL>
void launch_up(const LoraArgs& a, hipStream_t s) {
    // Units of more than 16 rows on average: their row tiles side by side, 64 columns a workgroup.
    // 200 rows of 4 adapters, 8192 x 8192, rank 64: 17.6 us a call so, 26.9 with 256 columns; 64 rows
    // of 32, N = 14336, rank 32: 16.4 and 15.7.
    const int tall = a.M > 16 * std::min(a.E, a.M);
    const int ntiles = (int)ceil_div(a.N, tall ? 64 : UP_COLS);
    const dim3 grid((unsigned)a.nunits * (unsigned)ntiles);
    if (a.R <= 32) hipLaunchKernelGGL((lora_up_kernel<1, F16, BF16, TAIL>), grid, dim3(LT), 0, s, a, ntiles, tall);
    else if (a.R <= 64) hipLaunchKernelGGL((lora_up_kernel<2, F16, BF16, TAIL>), grid, dim3(LT), 0, s, a, ntiles, tall);
    else hipLaunchKernelGGL((lora_up_kernel<0, F16, BF16, TAIL>), grid, dim3(LT), 0, s, a, ntiles, tall);
}
template <bool F16, bool BF16>
void launch_up(const LoraArgs& a, hipStream_t s) {
    if (a.S == 1) {
        const int ntiles = (int)ceil_div(a.N, 64);
        const dim3 grid((unsigned)a.nunits * (unsigned)ntiles);
        if (a.N % 4) hipLaunchKernelGGL((lora_expand_kernel<F16, BF16, true>), grid, dim3(LT), 0, s, a, ntiles);
        else hipLaunchKernelGGL((lora_expand_kernel<F16, BF16, false>), grid, dim3(LT), 0, s, a, ntiles);
        return;
    }
    if (a.N % 4) launch_up<F16, BF16, true>(a, s);
    else launch_up<F16, BF16, false>(a, s);
}

}  // namespace

size_t lora_workspace_bytes(int64_t E, int64_t M, int64_t N, int64_t K, int64_t R) {
    if (small_call(E, M, N, K, R)) return 0;
    const int64_t S = down_parts(E, M, K);
    return (size_t)round_up(M * R * (S > 1 ? 4 * S : 6), REGION_ALIGN);      // f32 parts, or three bf16 planes
}

// both launches' grids stay below 2^32 threads (the down kernel has nunits * 4 * S workgroups, S > 1
// only for few units)
bool lora_grid_ok(int64_t E, int64_t M, int64_t N, int64_t K) {
    const int64_t units = plan_layout(E, M).nunits;
    return units * std::max<int64_t>({ceil_div(N, 64), ceil_div(K, 64), 8}) < (int64_t(1) << 32) / LT;
}

hipError_t launch_lora(mmq_atype t, bool f16, const void* act, const void* A, const void* B, const float* scale,
                       int64_t E, int64_t R, const void* plan, int64_t M, int64_t N, int64_t K, const void* base,
                       int64_t ldb, void* out, int64_t ldo, float* v, void* ws, hipStream_t s) {
    LoraArgs a = lora_args(t, act, A, B, scale, E, R, plan, M, N, K);
    a.part = static_cast<float*>(ws);
    a.planes = static_cast<uint16_t*>(ws);
    a.S = (int)down_parts(E, M, K);
    a.base = base;
    a.ldb = ldb;
    a.out = out;
    a.ldo = ldo;
    a.v = v;
    const bool q81 = t == MMQ_ACT_Q8_1;
    if (small_call(E, M, N, K, R)) {
        if (f16) q81 ? launch_small<true, true>(a, s) : launch_small<true, false>(a, s);
        else q81 ? launch_small<false, true>(a, s) : launch_small<false, false>(a, s);
        return hipGetLastError();
    }
    if (f16) q81 ? launch_down<true, true>(a, s) : launch_down<true, false>(a, s);
    else q81 ? launch_down<false, true>(a, s) : launch_down<false, false>(a, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (f16) q81 ? launch_up<true, false>(a, s) : launch_up<true, true>(a, s);
    else q81 ? launch_up<false, false>(a, s) : launch_up<false, true>(a, s);
    return hipGetLastError();
}

}  // namespace mmq
