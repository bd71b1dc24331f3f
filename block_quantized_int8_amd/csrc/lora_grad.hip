// lora_grad.hip - the adapters' gradients, from the 8-bit activations kept as the checkpoint:
//     u[m] = s_e B_e^T dy[m]        dB_e = s_e sum over the rows of e of dy[m] v[m]^T
//     dx[m] = dxb[m] + A_e^T u[m]   dA_e = sum over the rows of e of u[m] x^[m]^T
// The act buffer is read as it is: its int8 values enter the matrix core exactly and each block's
// scale goes to u's side, so no activation is ever restored to f32 in memory.
//
// Two launches, each of two kinds of workgroups that need nothing of each other:
//   1. u (16 rows, its eight waves share N) and dB_e (64 columns of N a workgroup or a wave);
//      u is left in f32 and as bf16 terms in operand order;
//   2. dA_e (one block of K a workgroup or a wave) and dx (expand_body).
// 2048 rows of 4 adapters 4096 x 4096, rank 16: 17.8 + 19.4 us. The first launch reads dy twice (71 MB
// of L2 misses, 4.0 TB/s); the second moves 84 MB (4.3 TB/s), most of it dx's base and dx.
// The workgroups that sum over rows own their output tile, so nothing is added across
// workgroups and the sums have one order.
#include <algorithm>

#include "lora.h"

namespace mmq {
namespace {

// f32 or bf16 gradients as matrix-core operands: three terms or one
template <bool BF16> struct Grad {
    static constexpr int T = BF16 ? 1 : 3;
    u32x4 t[T];
    __device__ void set(const float* x) {
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[0][i] = pack_hi(x[2 * i], x[2 * i + 1]);
        } else {
            split3(x, t);
        }
    }
};

template <bool F16, bool BF16>
__device__ inline f32x4 mfma_grad(const Weights<F16>& w, const Grad<BF16>& x, f32x4 acc) {
    if constexpr (!BF16) return mfma_terms<F16>(w, x.t, acc);
    else {
        if constexpr (F16) acc = mfma_bf16(w.t[1], x.t[0], acc);
        return mfma_bf16(w.t[0], x.t[0], acc);
    }
}

// acc += a (three terms) times b, small products first
template <int T> __device__ inline f32x4 mfma_3(const u32x4* a, const u32x4* b, f32x4 acc) {
    if constexpr (T == 3) {
        acc = mfma_bf16(a[1], b[2], acc);
        acc = mfma_bf16(a[2], b[1], acc);
        acc = mfma_bf16(a[0], b[2], acc);
        acc = mfma_bf16(a[1], b[1], acc);
        acc = mfma_bf16(a[2], b[0], acc);
        acc = mfma_bf16(a[0], b[1], acc);
    } else {
        acc = mfma_bf16(a[2], b[0], acc);
    }
    acc = mfma_bf16(a[1], b[0], acc);
    return mfma_bf16(a[0], b[0], acc);
}

constexpr int GW = 8;               // waves of a workgroup of either launch

template <int RT> struct RankVec;
template <> struct RankVec<1> { typedef float V; };
template <> struct RankVec<2> { typedef f32x2 V; };
template <> struct RankVec<4> { typedef f32x4 V; };

// RT values of consecutive ranks of eight rows as operands (tile i: the i-th of them)
template <int RT> __device__ inline void rank_operands(const typename RankVec<RT>::V* v, u32x4 (*t)[3]) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (RT == 1) x[j] = v[j];
            else x[j] = v[j][i];
        }
        split3(x, t[i]);
    }
}

// Joins the waves' NT accumulators; wave w is left with the tiles w, w + GW, ... .
template <int NT> using JoinLds = f32x4[GW / 2][NT][64];
template <int NT> __device__ inline void join_waves(JoinLds<NT>& red, f32x4* acc, int wave, int lane) {
    __syncthreads();                                       // the memory may have had another use
    if (wave >= GW / 2)
#pragma unroll
        for (int i = 0; i < NT; ++i) red[wave - GW / 2][i][lane] = acc[i];
    __syncthreads();
    if (wave < GW / 2)
#pragma unroll
        for (int i = 0; i < NT; ++i) red[wave][i][lane] += acc[i];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < (NT + GW - 1) / GW; ++k) {
        const int i = wave + GW * k;
        if (i >= NT) break;
        f32x4 d = red[0][i][lane];
#pragma unroll
        for (int w = 1; w < GW / 2; ++w) d += red[w][i][lane];
        acc[k] = d;
    }
}

// ------------------------------------------------------------------------------ launch 1
constexpr int MAX_U_PARTS = 8;
// Rows of an adapter that one wave sums alone (each_sum): 64, or 256 where the adapters in use have
// blocks enough for the chip. Measured, all alone against all shared (us a call): 41 rows of 4
// adapters, N = 10342, rank 64: first launch 11.8, 27.4; 800 rows of 8, 4096 x 4096, rank 64: 31.4,
// 42.8; 200 rows of 2: 26.8, 23.8; 1200 rows of 8: 42.2, 52.0; 4096 rows of 8, rank 16: 94.6, 69.4.
// Enough are FULL_B of dB's blocks and FULL_A of dA's. Measured by the launch (us; 100, 160 and 240 rows
// an adapter, several adapters of N = K): sharing against alone. dB, rank 64, 256 blocks: 18.7 20.6 21.4
// against 21.2 24.1 33.2; 512: 27.7 30.2 31.3, 23.0 26.3 35.5; 1024: 46.6 55.0 61.4, 31.9 36.7
// 53.1; rank 16, 512: 15.0 16.4 17.8, 14.7 17.1 22.7; 1792: 27.7 39.4 47.7, 30.7 39.0 51.4. dA, rank 64,
// 1024: 9.1 10.9 11.6, 10.0 11.9 16.3; 1792: 14.0 16.2 17.7, 11.1 13.0 17.3; rank 16, 1024: 6.0 6.7
// 7.0, 6.4 7.5 10.1; 1792: 9.1 9.7 10.3, 7.1 7.8 10.5. (So at rank 16 dB, and at 1024 blocks dA, the
// sharing would still be the faster.)
constexpr int FEW = 64, FEW_FULL = 256;
constexpr int FULL_B = 512, FULL_A = 1024;
constexpr int MANY_MAX = 512;       // workgroups that share rows, where the plan has such adapters

// four ranks of a row's u, in f32 and as terms
__device__ inline void keep_u(const LoraArgs& a, int pos, int r, f32x4 d) {
    *reinterpret_cast<f32x4*>(a.u + (int64_t)pos * a.R + r) = d;
    store_terms(plane_at(a, pos, r), (int64_t)a.M * a.R, d);
}

// u of 16 rows, over one of S parts of N. Each wave turns its blocks of 32 columns in LDS of its own: dy's rows (as terms)
// into the B operand, B_e's rows of ranks into the A operand.
template <int RT, bool F16, bool BF16> struct ULds {
    uint16_t dy[Grad<BF16>::T][16][40];
    uint16_t w[Weights<F16>::T][32][16 * RT + 8];
};

template <int RT, bool F16, bool BF16>
__device__ inline void u_body(const LoraArgs& a, int block, int r0, ULds<RT, F16, BF16>* turn, JoinLds<RT>& red) {
    constexpr int NB = 2, T = Weights<F16>::T;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int at = block / a.S, s = block - at * a.S, sub = at / a.nunits;     // a unit's first 16 rows come first
    const int4 unit = unit_at(a, at - sub * a.nunits);
    const int rows = min(unit.z - 16 * sub, 16);
    if (rows <= 0 || unit.x >= a.E) return;
    const int p0 = unit.y + 16 * sub, per_row = min(a.R - r0, LORA_RC) / 8;     // pieces of a row of B_e

    const int64_t row = (int64_t)row_at(a, p0 + min(piece_row(lane), rows - 1)) * a.lddy;
    const uint16_t* B = a.B + (int64_t)unit.x * a.N * a.R + r0;
    uint32_t brow[RT], bcol[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int idx = min(lane + 64 * i, 32 * per_row - 1);                   // the last piece again past them
        brow[i] = idx / per_row;
        bcol[i] = 8 * (idx % per_row);
    }
    ULds<RT, F16, BF16>& mine = turn[wave];
    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = 0;
    const int blocks = (a.N + 31) / 32, per = (blocks + GW * a.S - 1) / (GW * a.S);
    const int b0 = (s * GW + wave) * per, b1 = min(b0 + per, blocks);
#pragma unroll 1
    for (int b = b0; b < b1; b += NB) {
        u32x4 x[NB][BF16 ? 1 : 2], w[NB][RT];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int n = 32 * min(b + k, b1 - 1);
#pragma unroll
            for (int i = 0; i < RT; ++i)
                w[k][i] = *reinterpret_cast<const u32x4*>(B + (int64_t)min(n + (int)brow[i], a.N - 1) * a.R + bcol[i]);
            // (bf16: values 8p .. 8p+7 of piece p; f32: 4p .. and 16 + 4p ..)
            if (n + 32 <= a.N) {
                if constexpr (BF16) {
                    x[k][0] = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(a.dy) + row + n + 8 * piece_of(lane));
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        x[k][h] = __builtin_bit_cast(u32x4, load_quad<false>(a.dy, row + n + 16 * h + 4 * piece_of(lane)));
                }
            } else {
                typename Quad<BF16>::Raw q[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const QuadEnd at(n + (BF16 ? 8 * piece_of(lane) + 4 * h : 16 * h + 4 * piece_of(lane)), a.N);
                    q[h] = drop_quad(load_quad_end<BF16>(a.dy, row, at, a.N), at.off);
                }
                if constexpr (BF16) {
                    x[k][0] = u32x4{q[0][0], q[0][1], q[1][0], q[1][1]};
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) x[k][h] = __builtin_bit_cast(u32x4, q[h]);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);                 // every load is issued before the first use
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            if (b + k >= b1) break;
            wave_lds_fence();
            if constexpr (BF16) {
                *reinterpret_cast<u32x4*>(&mine.dy[0][piece_row(lane)][8 * piece_of(lane)]) = x[k][0];
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    store_terms(&mine.dy[0][piece_row(lane)][16 * h + 4 * piece_of(lane)], 16 * 40, __builtin_bit_cast(f32x4, x[k][h]));
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                Weights<F16> ww;
                ww.set(w[k][i]);
#pragma unroll
                for (int j = 0; j < T; ++j) *reinterpret_cast<u32x4*>(&mine.w[j][brow[i]][bcol[i]]) = ww.t[j];
            }
            wave_lds_fence();
            Grad<BF16> d;
#pragma unroll
            for (int j = 0; j < Grad<BF16>::T; ++j) d.t[j] = *reinterpret_cast<const u32x4*>(&mine.dy[j][c][8 * g]);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                Weights<F16> ww;
#pragma unroll
                for (int j = 0; j < T; ++j) ww.t[j] = turned_operand(&mine.w[j][0][16 * i], 16 * RT + 8, lane);
                acc[i] = mfma_grad<F16, BF16>(ww, d, acc[i]);
            }
        }
    }
    join_waves<RT>(red, acc, wave, lane);
    const int r = r0 + 16 * wave + 4 * g;
    if (wave >= RT || c >= rows || r >= a.R) return;
    if (a.S > 1) *reinterpret_cast<f32x4*>(a.part + ((int64_t)s * a.M + p0 + c) * a.R + r) = acc[0];
    else keep_u(a, p0 + c, r, acc[0] * a.scale[unit.x]);
}

// u from its parts, in order: a workgroup per unit.
__global__ __launch_bounds__(LT) void lora_join_kernel(LoraArgs a) {
    const int4 unit = unit_at(a, blockIdx.x);
    if (unit.z == 0 || unit.x >= a.E) return;
    const float scale = a.scale[unit.x];
    for (int i = 4 * threadIdx.x; i < unit.z * a.R; i += 4 * LT) {
        const float* p = a.part + (int64_t)unit.y * a.R + i;
        f32x4 v[MAX_U_PARTS], d = 0;
#pragma unroll
        for (int s = 0; s < MAX_U_PARTS; ++s)
            if (s < a.S) v[s] = *reinterpret_cast<const f32x4*>(p + (int64_t)s * a.M * a.R);
#pragma unroll
        for (int s = 0; s < MAX_U_PARTS; ++s)
            if (s < a.S) d += v[s];
        keep_u(a, unit.y + i / a.R, i % a.R, d * scale);
    }
}

// The sums over an adapter's rows (dB, dA) are dealt out by the rows that it has, which only the
// device knows. An adapter's output is cut into `blocks`. With few rows a wave takes one of them and
// all rows, eight blocks a workgroup, nothing to join (`alone`); else the eight waves share the rows
// of a block. The first `many` workgroups deal out the blocks of the adapters of many rows, the rest
// are one for each eight blocks of every adapter and end at once where it has many. (By the rows
// an adapter has on average, 2048 rows that all went to one of 32 adapters took 293 us, now 67;
// spread evenly 76 and 78.)
struct SumGrid {
    int blocks, one, many, full;                           // one: workgroups of an adapter of few rows
};

template <typename Body> __device__ inline void each_sum(const LoraArgs& a, const SumGrid& s, int w, Body body) {
    auto rows_of = [&](int e) {
        if (e >= a.E) return 0;
        const int2 r = rows_of_group(a, e);
        return r.y - r.x;
    };
    // `few` is chosen by the adapters in use among the first 64: one load, while all of 4096 would be
    // 64 one after another in every workgroup. Where only later ones are in use it is FEW.
    int e0 = 0, few;
    uint64_t big;                                          // which of 64 adapters from e0 on have many rows
    {
        const int rows = rows_of(threadIdx.x & 63);
        few = __popcll(__ballot(rows > 0)) * s.blocks >= s.full ? FEW_FULL : FEW;
        big = __ballot(rows > few);
    }
    const bool alone = w >= s.many;
    int i = alone ? w - s.many : w;
#pragma unroll 1
    for (;;) {
        int e, block;
        if (alone) {
            e = i / s.one;
            block = i - e * s.one;
            if (rows_of(e) > few) return;
        } else {
            while (i >= __popcll(big) * s.blocks) {
                i -= __popcll(big) * s.blocks;
                e0 += 64;
                if (e0 >= a.E) return;
                big = __ballot(rows_of(e0 + (int)(threadIdx.x & 63)) > few);
            }
            const int q = i / s.blocks;
            uint64_t left = big;
            for (int k = 0; k < q; ++k) left &= left - 1;
            e = e0 + __builtin_ctzll(left);
            block = i - q * s.blocks;
        }
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));                      // nothing of the body is held across the loop
        body(e, block, alone, tid);
        if (alone) return;
        __syncthreads();                                   // the join's memory is free again
        i += s.many;
    }
}

// dB_e[n][r] over all rows of adapter e: 64 columns n (eight times that if alone) and up to 64 ranks.
// Both operands come straight from memory: a lane loads four consecutive columns (RT consecutive
// ranks) of eight rows, which are its k.
template <int RT, bool BF16>
__device__ inline void dB_body(const LoraArgs& a, int e, int tile0, int r0, bool alone, int tid, JoinLds<4 * RT>& red) {
    typedef typename RankVec<RT>::V V;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int n0 = 64 * (alone ? GW * tile0 + wave : tile0), n = n0 + 4 * c;
    const int2 range = rows_of_group(a, e);
    const int p0 = range.x, p1 = range.y, step = alone ? 32 : 32 * GW;
    if (alone && n0 >= a.N) return;
    const float* vr = a.v + min(r0 + RT * c, a.R - RT);
    f32x4 acc[4 * RT];
#pragma unroll
    for (int i = 0; i < 4 * RT; ++i) acc[i] = 0;
#pragma unroll 1
    for (int p = p0 + (alone ? 0 : 32 * wave); p < p1; p += step) {
        int m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = row_at(a, min(p + 8 * g + j, p1 - 1));
        typename Quad<BF16>::Raw x[8];
        V v[8];
        if (n0 + 64 <= a.N) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = load_quad<BF16>(a.dy, m[j] * a.lddy + n);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = load_quad_end<BF16>(a.dy, m[j] * a.lddy, QuadEnd(n, a.N), a.N);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const V*>(vr + (int64_t)m[j] * a.R);
        __builtin_amdgcn_sched_barrier(0);
        if (n0 + 64 > a.N)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = drop_quad(x[j], QuadEnd(n, a.N).off);
        u32x4 t[RT][3];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (p + 8 * g + j >= p1) v[j] = V(0);          // the last row's repeats add nothing
        rank_operands<RT>(v, t);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = quad_f32(x[j])[k];
            Grad<BF16> d;
            d.set(f);
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[k * RT + i] = mfma_3<Grad<BF16>::T>(t[i], d.t, acc[k * RT + i]);
        }
    }
    // rows of the accumulators: ranks r0 + RT (4g + j) + i; column: n0 + 4c + k
    const float scale = a.scale[e];
    if (alone) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = r0 + RT * (4 * g + j);
                V d;
                if constexpr (RT == 1) d = acc[k][j] * scale;
                else
#pragma unroll
                    for (int i = 0; i < RT; ++i) d[i] = acc[k * RT + i][j] * scale;
                if (n + k < a.N && r < a.R) *reinterpret_cast<V*>(a.dB + ((int64_t)e * a.N + n + k) * a.R + r) = d;
            }
        return;
    }
    join_waves<4 * RT>(red, acc, wave, lane);
#pragma unroll
    for (int q = 0; q < (4 * RT + GW - 1) / GW; ++q) {
        const int tile = wave + GW * q, k = tile / RT, i = tile % RT;
        if (tile >= 4 * RT || n + k >= a.N) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + RT * (4 * g + j) + i;
            if (r < a.R) a.dB[((int64_t)e * a.N + n + k) * a.R + r] = acc[q][j] * scale;
        }
    }
}

template <int RT, bool F16, bool BF16>
__global__ __launch_bounds__(GW * 64) void lora_grad1_kernel(LoraArgs a, SumGrid sums) {
    __shared__ __attribute__((aligned(16))) union {
        struct { ULds<RT, F16, BF16> turn[GW]; } u;
        JoinLds<RT> ju;
        JoinLds<4 * RT> jb;
    } lds;
    const int r0 = (int)blockIdx.y * LORA_RC, nu = 4 * a.nunits * a.S;
    if ((int)blockIdx.x < nu) u_body<RT, F16, BF16>(a, (int)blockIdx.x, r0, lds.u.turn, lds.ju);
    else
        each_sum(a, sums, (int)blockIdx.x - nu,
                 [&](int e, int block, bool alone, int tid) { dB_body<RT, BF16>(a, e, block, r0, alone, tid, lds.jb); });
}

// ------------------------------------------------------------------------------ launch 2
// dA_e[r][k] over all rows of adapter e: one block of K (eight if alone) and up to 64 ranks. A wave
// loads the 32 rows' 1 KB of the block (16 bytes a lane), turns them in LDS as bf16, and scales u by
// the rows' block scales.
struct ALds {
    uint16_t x[32][40];
    float xs[32];
};

template <int RT, bool Q81>
__device__ inline void dA_body(const LoraArgs& a, int e, int block, int r0, bool alone, int tid, ALds* turn,
                               JoinLds<2 * RT>& red) {
    typedef typename RankVec<RT>::V V;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int b = alone ? GW * block + wave : block;
    const int2 range = rows_of_group(a, e);
    const int p0 = range.x, p1 = range.y, step = alone ? 32 : 32 * GW;
    if (alone && b >= a.KB) return;
    const float* ur = a.u + min(r0 + RT * c, a.R - RT);
    ALds& mine = turn[wave];
    f32x4 acc[2 * RT];
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) acc[i] = 0;
#pragma unroll 1
    for (int p = p0 + (alone ? 0 : 32 * wave); p < p1; p += step) {
        const int row = lane & 31, m = row_at(a, min(p + row, p1 - 1));
        V u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = *reinterpret_cast<const V*>(ur + (int64_t)min(p + 8 * g + j, p1 - 1) * a.R);
        const int64_t cell = (int64_t)(m >> 5) * a.KBp + b;
        const u32x4 q = *reinterpret_cast<const u32x4*>(a.xq + cell * 1024 + ((lane >> 5) * 32 + (m & 31)) * 16);
        float xs;
        if constexpr (Q81) xs = (float)__builtin_bit_cast(_Float16, (uint16_t)a.xs2[cell * 32 + (m & 31)]);
        else xs = a.sa[m];
        __builtin_amdgcn_sched_barrier(0);
        wave_lds_fence();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<u32x4*>(&mine.x[row][16 * (lane >> 5) + 8 * h]) = int8_operand<false>(u32x2{q[2 * h], q[2 * h + 1]});
        if (lane < 32) mine.xs[row] = p + row < p1 ? xs : 0.f;     // the last row's repeats add nothing
        wave_lds_fence();
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] *= mine.xs[8 * g + j];
        u32x4 t[RT][3], x[2];
        rank_operands<RT>(u, t);
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h] = turned_operand(&mine.x[0][16 * h], 40, lane);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4& s = acc[h * RT + i];
                s = mfma_bf16(t[i][2], x[h], s);
                s = mfma_bf16(t[i][1], x[h], s);
                s = mfma_bf16(t[i][0], x[h], s);
            }
    }
    // rows of the accumulators: ranks r0 + RT (4g + j) + i; column: k = 32b + 16h + c
    float* to = a.dA + (int64_t)e * a.R * a.K + 32 * b + c;
    if (alone) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = r0 + RT * (4 * g + j) + i;
                if (r >= a.R) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) to[(int64_t)r * a.K + 16 * h] = acc[h * RT + i][j];
            }
        return;
    }
    join_waves<2 * RT>(red, acc, wave, lane);
    if (wave >= 2 * RT) return;
    const int h = wave / RT, i = wave % RT;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = r0 + RT * (4 * g + j) + i;
        if (r < a.R) to[(int64_t)r * a.K + 16 * h] = acc[0][j];
    }
}

template <int RT, bool F16, bool Q81>
__global__ __launch_bounds__(GW * 64) void lora_grad2_kernel(LoraArgs a, int ktiles, SumGrid sums) {
    __shared__ __attribute__((aligned(16))) union {
        ALds turn[GW];
        JoinLds<2 * RT> ja;
        ExpandLds<true, F16, GW> x;
    } lds;
    const int na = sums.many + a.E * sums.one;
    if ((int)blockIdx.x < na) {
        each_sum(a, sums, (int)blockIdx.x, [&](int e, int block, bool alone, int tid) {
            dA_body<RT, Q81>(a, e, block, (int)blockIdx.y * LORA_RC, alone, tid, lds.turn, lds.ja);
        });
        return;
    }
    if (blockIdx.y) return;
    const int block = (int)blockIdx.x - na, u = block / ktiles;
    const int4 unit = unit_at(a, u);
    if (unit.z == 0) return;
    // the columns turn with the unit, so that an XCD's L2 sees all of its channels
    expand_body<true, F16, false, false, GW>(a, a.A, a.K, a.dxb, a.lddxb, a.dx, a.lddx, unit,
                                             (block - u * ktiles + u) % ktiles, lds.x);
}

constexpr int DX_COLS = 16 * GW;                           // columns of a dx workgroup

// `blocks` of an adapter's output, and how many of all adapters in use are enough for the chip
SumGrid sum_grid(const LoraArgs& a, int64_t blocks, int full) {
    const int64_t big = std::min<int64_t>(a.E, a.M / (FEW + 1));       // adapters of many rows at most
    return SumGrid{(int)blocks, (int)ceil_div(blocks, GW), (int)std::min<int64_t>(MANY_MAX, big * blocks), full};
}

template <int RT>
void launch_grads(const LoraArgs& a, bool f16, bool q81, hipStream_t s) {
    const unsigned rc = (unsigned)ceil_div(a.R, LORA_RC);
    const SumGrid sb = sum_grid(a, ceil_div(a.N, 64), FULL_B), sa = sum_grid(a, a.KB, FULL_A);
    const int kt = (int)ceil_div(a.K, DX_COLS);
    const dim3 g1((unsigned)(4 * a.nunits * a.S + sb.many + a.E * sb.one), rc);
    const dim3 g2((unsigned)(sa.many + a.E * sa.one + (a.dx ? a.nunits * kt : 0)), rc);
    const dim3 th(GW * 64);
    const auto join = [&] {
        if (a.S > 1) hipLaunchKernelGGL(lora_join_kernel, dim3((unsigned)a.nunits), dim3(LT), 0, s, a);
    };
    if (f16) {
        if (q81) {
            hipLaunchKernelGGL((lora_grad1_kernel<RT, true, false>), g1, th, 0, s, a, sb);
            join();
            hipLaunchKernelGGL((lora_grad2_kernel<RT, true, true>), g2, th, 0, s, a, kt, sa);
        } else {
            hipLaunchKernelGGL((lora_grad1_kernel<RT, true, true>), g1, th, 0, s, a, sb);
            join();
            hipLaunchKernelGGL((lora_grad2_kernel<RT, true, false>), g2, th, 0, s, a, kt, sa);
        }
    } else {
        if (q81) {
            hipLaunchKernelGGL((lora_grad1_kernel<RT, false, false>), g1, th, 0, s, a, sb);
            join();
            hipLaunchKernelGGL((lora_grad2_kernel<RT, false, true>), g2, th, 0, s, a, kt, sa);
        } else {
            hipLaunchKernelGGL((lora_grad1_kernel<RT, false, true>), g1, th, 0, s, a, sb);
            join();
            hipLaunchKernelGGL((lora_grad2_kernel<RT, false, false>), g2, th, 0, s, a, kt, sa);
        }
    }
}

// Parts of N for u: one while a wave has twelve steps of two blocks at most (N <= 6144); else as many
// as give it four, within 512 workgroups. Their sum is a launch of its own, 3 us of the host and 4
// of the card (64 rows of 32 adapters, N = 4096, rank 16: 17.1 us in one part, 13.8 + 4.2 in two;
// 37 rows of one adapter, N = 5221, rank 64: 20.4 us a call in one, 23.3 in two).
int64_t u_parts(int64_t E, int64_t M, int64_t N) {
    const int64_t blocks = ceil_div(N, 32), tiles = ceil_div(M, 16) + std::min(E, M);
    if (blocks <= 24 * GW) return 1;
    return std::max<int64_t>(1, std::min<int64_t>({512 / tiles, ceil_div(blocks, 8 * GW), MAX_U_PARTS}));
}

}  // namespace

// f32 u, its three bf16 planes, and its parts
size_t lora_grad_workspace_bytes(int64_t E, int64_t M, int64_t N, int64_t R) {
    const int64_t S = u_parts(E, M, N);
    return (size_t)(round_up(M * R * 4, REGION_ALIGN) + round_up(M * R * 6, REGION_ALIGN) +
                    (S > 1 ? round_up(S * M * R * 4, REGION_ALIGN) : 0));
}

// both launches' grids stay below 2^32 threads (u's parts are split for few units only)
bool lora_grad_grid_ok(int64_t E, int64_t M, int64_t N, int64_t K) {
    const int64_t units = plan_layout(E, M).nunits;
    return 4 * units * u_parts(E, M, N) + E * ceil_div(N, 64) < (int64_t(1) << 32) / (GW * 64) - MANY_MAX &&
           E * (K / QK) + units * ceil_div(K, DX_COLS) < (int64_t(1) << 32) / (GW * 64) - MANY_MAX;
}

hipError_t launch_lora_grad(mmq_atype t, bool f16, const void* act, const void* A, const void* B, const float* scale,
                            int64_t E, int64_t R, const void* plan, int64_t M, int64_t N, int64_t K, const float* v,
                            const void* dy, int64_t lddy, const float* dxb, int64_t lddxb, float* dx, int64_t lddx,
                            float* dA, float* dB, void* ws, hipStream_t s) {
    LoraArgs a = lora_args(t, act, A, B, scale, E, R, plan, M, N, K);
    a.v = const_cast<float*>(v);                       // only read here
    a.dy = dy;
    a.lddy = lddy;
    a.dxb = dxb;
    a.lddxb = lddxb;
    a.dx = dx;
    a.lddx = lddx;
    a.dA = dA;
    a.dB = dB;
    a.u = static_cast<float*>(ws);
    a.planes = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + round_up(M * R * 4, REGION_ALIGN));
    a.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.planes) + round_up(M * R * 6, REGION_ALIGN));
    a.S = (int)u_parts(E, M, N);
    const bool q81 = t == MMQ_ACT_Q8_1;
    if (R <= 16) launch_grads<1>(a, f16, q81, s);
    else if (R <= 32) launch_grads<2>(a, f16, q81, s);
    else launch_grads<4>(a, f16, q81, s);
    return hipGetLastError();
}

}  // namespace mmq
