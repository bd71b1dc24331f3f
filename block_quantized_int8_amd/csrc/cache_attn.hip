// cache_attn.hip - attention over the block-quantised cache, for one new token a sequence, chains of
// them and trees of drafted ones.
//
// Rows are (new token, query head) pairs that share a head of the cache; a workgroup has 16 of them
// and a chunk of the sequence's tiles of 32 tokens, its waves take the tiles in turn. Per tile:
//   1. scores, transposed: S^T = K q^T on the matrix core. int8 or 4-bit whole numbers are exact in
//      f16; a block of 32 values is one product, whose four sums a lane are scaled by their tokens'
//      f32 scales. q is held as f16 terms of q 2^e (e: the row's exponent), two for f32 rows, one
//      for bf16 rows (8 significand bits, exact).
//   2. p = 2^(score - m), m the running maximum; 2^10 of headroom keeps small p away from f16's
//      subnormals.
//   3. O^T += V^T P^T. The scale of a token's block of values lies along the sum, so it goes into P:
//      p d_v 2^k, in two f16 terms for f32 rows, one for bf16 rows. k, the wave's running exponent,
//      keeps the largest d_v 2^k in [1, 2).
// A lane holds the tokens of S^T's rows that it needs as P^T's k: the cache's order of tokens makes
// them the same (cache.h).
// The waves' sums are joined in LDS. A sequence of several chunks leaves its parts in the workspace,
// and a second launch joins them.
#include <algorithm>

#include "cache.h"

namespace mmq {
namespace {

constexpr int WAVES = 4, THREADS = WAVES * 64;
constexpr int CHUNK_MIN = 4;                // tiles of a chunk at least
constexpr int TARGET = 1024;                // workgroups aimed at
constexpr float P_BITS = 10.f;              // p is held times 2^10,
constexpr float P_SLACK = 4.f;              // and the maximum may rise by 4 before it is taken anew

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

struct AttnArgs {
    const void* q;
    void* out;
    const uint8_t *kc, *vc;
    const int32_t *table, *lens, *starts;
    const uint64_t* mask;
    float *part_o, *part_m, *part_l;        // parts: [part][rows][D], [part][rows] twice
    int4* list;                             // split sequences: their number, then (first row, rows, chunks, first part)
    int64_t ldq, ldo, ldt;
    CacheShape c;
    float scale;
    int rows, B, max_q, G, QG, cap, units, splits;        // cap: tokens a table row can hold
};

__device__ inline h2 as_h2(uint32_t x) { return __builtin_bit_cast(h2, x); }
__device__ inline u16x2 as_u16(uint32_t x) { return __builtin_bit_cast(u16x2, x); }
__device__ inline uint32_t as_u32(h2 x) { return __builtin_bit_cast(uint32_t, x); }

// A value that is the same in every lane, in a scalar register: what comes from LDS or an integer
// division would be kept, with all that follows from it (loop counts, buffer descriptors), in lanes.
__device__ inline int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Sequence b: its new tokens (0 if its rows are not in the batch) and its tokens in the cache.
struct Seq {
    int first, n, len;
};
__device__ inline Seq seq_of(const AttnArgs& a, int b) {
    Seq s;
    s.first = a.starts[b];
    const int end = a.starts[b + 1];
    const bool ok = s.first >= 0 && end >= s.first && end <= a.rows;
    s.n = ok ? end - s.first : 0;
    s.len = max(a.lens[b], 0);
    return s;
}
__device__ inline int seq_tiles(const AttnArgs& a, const Seq& s) {
    return s.n == 0 ? 0 : max(1, (min(s.len, a.cap) + CACHE_TILE - 1) / CACHE_TILE);
}

// What a unit (a chunk of one sequence's tiles) is, found by every workgroup from the sequences'
// lengths: chunks are as long as keeps the launch at TARGET workgroups.
struct Unit {
    int b, chunk, chunks, tiles, split, part;     // tiles of a chunk; split: number among split sequences
};
__device__ inline int64_t wave_total(int64_t v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor((long long)v, o);
    return v;
}
__device__ inline int wave_scan(int v, int lane) {          // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}
__device__ inline bool find_unit(const AttnArgs& a, int unit, int tid, Unit& u, int* splits) {
    __shared__ int64_t total[WAVES];
    __shared__ int sums[3][WAVES];
    __shared__ Unit found;
    __shared__ int any;
    const int lane = tid & 63, wave = tid >> 6;
    const int per = (a.B + THREADS - 1) / THREADS;
    if (tid == 0) any = 0;
    int64_t tiles = 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < a.B) tiles += seq_tiles(a, seq_of(a, b));
    }
    tiles = wave_total(tiles);
    if (lane == 0) total[wave] = tiles;
    __syncthreads();
    int64_t work = 0;
    for (int i = 0; i < WAVES; ++i) work += total[i];
    const int aim = max(1, TARGET / (a.c.heads * a.QG));
    // (a sequence has fewer than 2^26 tiles)
    const int chunk = max(CHUNK_MIN, (int)min((work + aim - 1) / aim, (int64_t)1 << 26));
    int mine[3] = {0, 0, 0};                                // units, parts of split sequences, those
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= a.B) break;
        const int n = (seq_tiles(a, seq_of(a, b)) + chunk - 1) / chunk;
        mine[0] += n;
        mine[1] += n > 1 ? n : 0;
        mine[2] += n > 1;
    }
    int before[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int s = wave_scan(mine[j], lane);
        if (lane == 63) sums[j][wave] = s;
        before[j] = s - mine[j];
    }
    __syncthreads();
    *splits = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        for (int i = 0; i < WAVES; ++i) {
            if (i < wave) before[j] += sums[j][i];
            if (j == 2) *splits += sums[j][i];
        }
    if (unit >= before[0] && unit < before[0] + mine[0]) {  // one thread's
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            const int n = (seq_tiles(a, seq_of(a, b)) + chunk - 1) / chunk;
            if (unit < before[0] + n) {
                found = {b, unit - before[0], n, chunk, before[2], before[1]};
                any = 1;
                break;
            }
            before[0] += n;
            before[1] += n > 1 ? n : 0;
            before[2] += n > 1;
        }
    }
    __syncthreads();
    u = {scalar(found.b), scalar(found.chunk), scalar(found.chunks), scalar(found.tiles), scalar(found.split), scalar(found.part)};
    return scalar(any) != 0;
}

// Eight whole numbers of the cache as f16
__device__ inline h8 join(h2 a, h2 b, h2 c, h2 d) {
    const u32x4 r = {as_u32(a), as_u32(b), as_u32(c), as_u32(d)};
    return __builtin_bit_cast(h8, r);
}
// q8_0: bytes q + 128 become 1024 + (q + 128) by their place in an f16 significand
__device__ inline h8 from_bytes(uint32_t x, uint32_t y) {
    const h2 off = {(_Float16)1152.f, (_Float16)1152.f};
    const uint32_t e = 0x64646464u;
    return join(as_h2(__builtin_amdgcn_perm(e, x, 0x04010400u)) - off, as_h2(__builtin_amdgcn_perm(e, x, 0x04030402u)) - off,
                as_h2(__builtin_amdgcn_perm(e, y, 0x04010400u)) - off, as_h2(__builtin_amdgcn_perm(e, y, 0x04030402u)) - off);
}
// q4_0: nibbles q + 8, 16 bits apart in x >> s
__device__ inline h2 from_nibbles(uint32_t x, int s) {
    const h2 off = {(_Float16)1032.f, (_Float16)1032.f};
    return as_h2(((x >> s) & 0x000F000Fu) | 0x64006400u) - off;
}

// A record as a buffer: of no bytes where there is none to load, which loads nothing and returns zeros.
// (Without a branch: where paths with and without loads meet, the compiler waits for all of them.)
struct Record {
    __amdgpu_buffer_rsrc_t r;
    __device__ Record(const uint8_t* base, uint64_t n, int bytes, bool there)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base + n * (uint64_t)bytes), 0, there ? bytes : 0, 0x00020000)) {}
    __device__ u32x4 at(int offset) const { return __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0); }
};

template <bool Q8, int NB> struct Keys {
    u32x4 w[Q8 ? NB : NB / 2];
    u32x4 d[NB];                                            // the scales of the lane's 8 tokens
    __device__ void load(const Record& r, int lane) {
#pragma unroll
        for (int i = 0; i < (Q8 ? NB : NB / 2); ++i) w[i] = r.at(lane * 16 + i * 1024);
#pragma unroll
        for (int b = 0; b < NB; ++b) d[b] = r.at((lane >> 4) * (NB * 16) + cache_values(Q8, NB * 32) + b * 16);
    }
    __device__ h8 get(int h, int b) const {                 // 8 values of block b of tokens 16h..
        if constexpr (Q8) {
            const u32x4 r = w[h * (NB / 2) + b / 2];
            return from_bytes(r[(b & 1) * 2], r[(b & 1) * 2 + 1]);
        } else {
            const uint32_t x = w[b / 2][h * 2 + (b & 1)];
            return join(from_nibbles(x, 0), from_nibbles(x, 4), from_nibbles(x, 8), from_nibbles(x, 12));
        }
    }
};
template <bool Q8, int NB> struct Values {
    u32x4 w[Q8 ? NB : NB / 2];
    u32x4 d[NB];
    __device__ void load(const Record& r, int lane) {
#pragma unroll
        for (int i = 0; i < (Q8 ? NB : NB / 2); ++i) w[i] = r.at(lane * 16 + i * 1024);
#pragma unroll
        for (int b = 0; b < NB; ++b) d[b] = r.at((lane >> 4) * (NB * 16) + cache_values(Q8, NB * 32) + b * 16);
    }
    __device__ h8 get(int b, int u) const {                 // 8 tokens of values 16u.. of block b
        if constexpr (Q8) return from_bytes(w[b][2 * u], w[b][2 * u + 1]);
        else {
            const uint32_t x = w[b / 2][(b & 1) * 2], y = w[b / 2][(b & 1) * 2 + 1];
            return join(from_nibbles(x, 4 * u), from_nibbles(x, 8 + 4 * u), from_nibbles(y, 4 * u), from_nibbles(y, 8 + 4 * u));
        }
    }
};

__device__ inline f32x4 mfma(h8 a, h8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

__device__ inline float xor_max(float v) {                  // over the four groups of a column
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ inline float xor_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Four values of a result's row
template <bool F32> __device__ inline void store4(const AttnArgs& a, int64_t row, int head, int D, int d, f32x4 y) {
    const int64_t to = row * a.ldo + (int64_t)head * D + d;
    if constexpr (F32) {
        *reinterpret_cast<f32x4_any*>(static_cast<float*>(a.out) + to) = y;
    } else {
        const u32x2 w = {bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
        *reinterpret_cast<u32x2_any*>(static_cast<uint16_t*>(a.out) + to) = w;
    }
}

// The 16 rows of one product's columns: q's terms and the running sums.
template <int TERMS, int NB> struct Rows {
    h8 q[TERMS][NB];
    f32x4 o[2 * NB];
    float c;                    // from the products of q's terms to the exponent: scale * log2(e) * 2^-e
    float m, off, l;            // the maximum that p is taken from, P_BITS - m (P_BITS before the first), sum of p
    uint64_t bits;              // of the mask
    int i;                      // the row's new token
};

template <int TERMS, int NB>
__device__ inline void load_rows(const AttnArgs& a, const Seq& s, int h, int row, int g, Rows<TERMS, NB>& r) {
    constexpr bool F32 = TERMS == 2;
    r.i = row / a.G;
    r.bits = a.mask ? a.mask[s.first + r.i] : 0;
    r.m = -__builtin_inff();
    r.off = P_BITS;
    r.l = 0.f;
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) r.o[j] = 0.f;
    float v[NB][8];
    float top = 0.f;
    const int64_t at = (int64_t)(s.first + r.i) * a.ldq + (int64_t)(h * a.G + row % a.G) * (NB * 32) + 8 * g;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if constexpr (F32) {
            const u32x4_any* p = reinterpret_cast<const u32x4_any*>(static_cast<const float*>(a.q) + at + 32 * b);
            const u32x4 r0 = p[0], r1 = p[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[b][j] = __builtin_bit_cast(float, (uint32_t)r0[j]);
                v[b][4 + j] = __builtin_bit_cast(float, (uint32_t)r1[j]);
            }
        } else {
            const u32x4 w = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(a.q) + at + 32 * b);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[b][2 * j] = __builtin_bit_cast(float, w[j] << 16);
                v[b][2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[b][j]));
    }
    top = xor_max(top);
    // the row's largest value in [2^13, 2^14)
    const int e = top > 0.f && top < __builtin_inff() ? 14 - __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = __builtin_amdgcn_ldexpf(v[b][j], e);
            const _Float16 hi = (_Float16)y;
            r.q[0][b][j] = hi;
            if constexpr (F32) r.q[1][b][j] = (_Float16)(y - (float)hi);
        }
    // never 0, which times the score of a hidden token would be NaN
    r.c = fmaxf(__builtin_amdgcn_ldexpf(a.scale * 1.44269504088896340736f, -e), 1e-37f);
}

// Waves of a SIMD that the registers are dealt out for.
constexpr int waves_of(int NB, int NQ) { return NB * NQ <= 4 ? 3 : NB * NQ <= 8 ? 2 : 1; }

// What a wave knows of a tile's value scales: their exponent, and the f16 bits from which it must fall.
struct Exponent {
    int k;
    uint32_t limit;
};

// F32: rows of f32 (two terms), or bf16 (one). NQ: groups of 16 rows of a workgroup.
template <bool F32, bool K8, bool V8, int NB, int NQ>
__global__ __launch_bounds__(THREADS, waves_of(NB, NQ)) void cache_attn_kernel(AttnArgs a) {
    constexpr int D = NB * 32, TERMS = F32 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float sh_o[WAVES][16][D + 4];
    __shared__ float sh_m[WAVES][16], sh_l[WAVES][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    // workgroups that share a chunk (one per QG) are 8 apart: on the same die, behind one L2
    const int gx = scalar(((int)blockIdx.x >> 3) / a.QG), qg = ((int)blockIdx.x >> 3) - gx * a.QG;
    const int x = gx * 8 + ((int)blockIdx.x & 7);
    const int unit = scalar(x / a.c.heads), h = x - unit * a.c.heads;
    if (unit >= a.units) return;
    Unit u;
    int splits;
    const bool there = find_unit(a, unit, tid, u, &splits);
    const bool first_of = a.list && h == 0 && qg == 0 && tid == 0;
    if (first_of && unit == 0) a.list[0] = {min(splits, a.splits), 0, 0, 0};
    if (!there) return;
    Seq s = seq_of(a, u.b);
    s = {scalar(s.first), scalar(s.n), scalar(s.len)};
    if (first_of && u.chunks > 1 && u.chunk == 0 && u.split < a.splits)
        a.list[1 + u.split] = {s.first, min(s.n, a.max_q), u.chunks, u.part};
    const int row0 = qg * NQ * 16;
    const int nrows = min(min(s.n, a.max_q) * a.G - row0, NQ * 16);    // this workgroup's
    if (nrows <= 0) return;
    const int ctx = s.len - s.n, len = min(s.len, a.cap);

    // the tiles that any of the rows can see
    int seen = len;
    if (!a.mask) seen = min(seen, ctx + (row0 + nrows - 1) / a.G + 1);
    const int t0 = u.chunk * u.tiles;
    const int t1 = scalar(min(t0 + u.tiles, (max(seen, 0) + CACHE_TILE - 1) / CACHE_TILE));

    Rows<TERMS, NB> r[NQ];                                  // (past the rows: the last one again)
#pragma unroll
    for (int n = 0; n < NQ; ++n) load_rows<TERMS, NB>(a, s, h, row0 + min(n * 16 + col, nrows - 1), g, r[n]);

    Exponent ex = {15, 0};                                  // no scale yet
    // pages by scalar loads: a vector load would be waited for with every load before it
    const auto* table = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)(a.table + (int64_t)u.b * a.ldt);
    const int shift = __builtin_ctz(a.c.tiles);
    const auto record = [&](int t, uint32_t page) {
        return ((uint64_t)page * a.c.heads + h) * a.c.tiles + (t & (a.c.tiles - 1));
    };
    Keys<K8, NB> kw;
    Values<V8, NB> vw;
    const auto load_k = [&](uint64_t rec, bool there) __attribute__((always_inline)) {
        kw.load(Record(a.kc, rec, cache_record(K8, D), there), lane);
    };
    const auto load_v = [&](uint64_t rec, bool there) __attribute__((always_inline)) {
        vw.load(Record(a.vc, rec, cache_record(V8, D), there), lane);
    };
    // A tile's keys are loaded while the products of values of the one before run, its values while the
    // next scores do: the registers are free by then. No such page: its tokens are not seen, and the
    // first page stands in for it.
    int t = t0 + wave;
    bool ok = false;
    uint64_t rec = 0;
    if (t < t1) {
        const uint32_t page = (uint32_t)table[t >> shift];
        ok = page < (uint32_t)a.c.pages;
        rec = record(t, ok ? page : 0);
        load_k(rec, true);
        load_v(rec, true);
    }
#pragma unroll 1
    for (; t < t1; t += WAVES) {
        const int limit = ok ? len : 0;
        const bool more = t + WAVES < t1;
        const uint32_t page = (uint32_t)table[(more ? t + WAVES : t) >> shift];

        // 1. the products of scores
        float sc[NQ][8];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            f32x4 acc[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) acc[n] = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const h8 kv = kw.get(hh, b);
                const h2 d0 = as_h2(kw.d[b][2 * hh]), d1 = as_h2(kw.d[b][2 * hh + 1]);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    f32x4 y = 0.f;
#pragma unroll
                    for (int i = 0; i < TERMS; ++i) y = mfma(kv, r[n].q[i][b], y);
                    acc[n][0] = fmaf(y[0], (float)d0[0], acc[n][0]);
                    acc[n][1] = fmaf(y[1], (float)d0[1], acc[n][1]);
                    acc[n][2] = fmaf(y[2], (float)d1[0], acc[n][2]);
                    acc[n][3] = fmaf(y[3], (float)d1[1], acc[n][3]);
                }
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[n][4 * hh + i] = acc[n][i];
        }

        // (the scores are finished before the loads, whose registers the products' operands leave)
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(sc[n][i]));
        ok = page < (uint32_t)a.c.pages;
        rec = record(t + WAVES, ok ? page : 0);           // (not loaded from where there is none)
        load_k(rec, more);

        // tokens that a row does not see; scales of slots past the sequence are not read as numbers
        if (CACHE_TILE * (t + 1) > min(ctx, limit)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int pos = CACHE_TILE * t + 16 * (i >> 2) + 4 * g + (i & 3), ahead = pos - ctx;
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    bool v = pos < limit;
                    if (ahead >= 0) v = v && (a.mask ? ahead < 64 && (r[n].bits >> ahead & 1) : ahead <= r[n].i);
                    if (!v) sc[n][i] = -__builtin_inff();
                }
                if (pos >= limit) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) vw.d[b][i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                }
            }
        }

        // The exponent k of the value scales. One that is not finite counts as 0, after the sums that it
        // goes into, those of the rows that see its token, are made NaN.
        u16x2 dtop = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) dtop = __builtin_elementwise_max(dtop, as_u16(vw.d[b][i] & 0x7FFF7FFFu));
        uint32_t dmax = max(dtop[0], dtop[1]);
        if (__any(dmax > ex.limit)) {
            if (__any(dmax >= 0x7C00)) {
                dmax = 0;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float bad[NQ] = {};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t d = (vw.d[b][i >> 1] >> (16 * (i & 1))) & 0x7FFF;
                        if (d < 0x7C00) {
                            dmax = max(dmax, d);
                        } else {
                            vw.d[b][i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
                            for (int n = 0; n < NQ; ++n)
                                if (sc[n][i] != -__builtin_inff()) bad[n] = 1.f;
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        if (xor_max(bad[n]) != 0.f) r[n].o[2 * b] = r[n].o[2 * b + 1] = __builtin_nanf("");
                }
            }
            dmax = max(dmax, (uint32_t)__shfl_xor((int)dmax, 16));
            dmax = max(dmax, (uint32_t)__shfl_xor((int)dmax, 32));
            dmax = __builtin_amdgcn_readfirstlane(dmax);
            if (dmax > ex.limit) {
                // the largest scale times 2^k in [1, 2), as far as 2^k is an f16
                const int k = min(15, 1 - __builtin_amdgcn_frexp_expf((float)__builtin_bit_cast(_Float16, (uint16_t)dmax)));
                const float fall = __builtin_amdgcn_ldexpf(1.f, k - ex.k);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i) r[n].o[i] *= fall;
                ex.k = k;
                // the largest f16 below 2^(1 - k)
                ex.limit = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)__builtin_amdgcn_ldexpf(1.f, -k)) | 0x3FF;
            }
        }

        // 2. p, from a maximum that is taken anew where a score is far above it
        uint32_t ph[NQ][4], pl[NQ][4];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float top = sc[n][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, sc[n][i]);
            top *= r[n].c;
            if (__any(top > r[n].m + P_SLACK)) {
                const float m1 = fmaxf(r[n].m, xor_max(top));
                const float base = m1 == -__builtin_inff() ? 0.f : m1;
                const float fall = __builtin_amdgcn_exp2f(r[n].m - base);
                r[n].m = m1;
                r[n].off = P_BITS - base;
                r[n].l *= fall;
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) r[n].o[i] *= fall;
            }
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(fmaf(sc[n][i], r[n].c, r[n].off));
                r[n].l += p[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const h2 hi = {(_Float16)p[2 * i], (_Float16)p[2 * i + 1]};
                ph[n][i] = as_u32(hi);
                if constexpr (F32) {
                    const h2 lo = {(_Float16)(p[2 * i] - (float)hi[0]), (_Float16)(p[2 * i + 1] - (float)hi[1])};
                    pl[n][i] = as_u32(lo);
                }
            }
        }

        const _Float16 two_k = (_Float16)__builtin_amdgcn_ldexpf(1.f, ex.k);

        // 3. the products of values
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            h2 d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = as_h2(vw.d[b][i]) * h2{two_k, two_k};
            h8 pt[NQ][TERMS];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const h2 y = as_h2(ph[n][i]) * d[i];
                    hi[i] = as_u32(y);
                    if constexpr (F32)
                        lo[i] = as_u32(__builtin_elementwise_fma(as_h2(pl[n][i]), d[i],
                                                                 __builtin_elementwise_fma(as_h2(ph[n][i]), d[i], -y)));
                }
                pt[n][0] = __builtin_bit_cast(h8, u32x4{hi[0], hi[1], hi[2], hi[3]});
                if constexpr (F32) pt[n][1] = __builtin_bit_cast(h8, u32x4{lo[0], lo[1], lo[2], lo[3]});
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const h8 vv = vw.get(b, v);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < TERMS; ++i) r[n].o[2 * b + v] = mfma(vv, pt[n][i], r[n].o[2 * b + v]);
            }
        }
        load_v(rec, more);
    }

    // the waves' sums
    const bool split = u.chunks > 1;
    const int64_t part = split ? (((int64_t)(u.part + u.chunk) * a.c.heads + h) * a.QG + qg) * (NQ * 16) : 0;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        if (n * 16 >= nrows) break;
        if (n) __syncthreads();
        const float l = xor_sum(r[n].l);
        if (g == 0) {
            sh_m[wave][col] = r[n].m;
            sh_l[wave][col] = l;
        }
        __syncthreads();
        float top = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = fmaxf(top, sh_m[w][col]);
        // (a wave that saw nothing counts 0, one whose scores are all NaN, NaN)
        const float mine = r[n].m == -__builtin_inff() ? 0.f
                           : __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(r[n].m - top), -ex.k);
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
            *reinterpret_cast<f32x4*>(&sh_o[wave][col][16 * i + 4 * g]) = r[n].o[i] * mine;
        __syncthreads();
        const int left = min(nrows - n * 16, 16);
        for (int e = tid; e < left * (D / 4); e += THREADS) {
            const int rr = e / (D / 4), d = e % (D / 4) * 4;
            float big = -__builtin_inff(), sum = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) big = fmaxf(big, sh_m[w][rr]);
            f32x4 y = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                y += *reinterpret_cast<const f32x4*>(&sh_o[w][rr][d]);
                const float m = sh_m[w][rr];
                sum += sh_l[w][rr] * (m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m - big));
            }
            if (split) {
                const int64_t to = part + n * 16 + rr;
                *reinterpret_cast<f32x4*>(a.part_o + to * D + d) = y;
                if (d == 0) {
                    a.part_m[to] = big;
                    a.part_l[to] = sum;
                }
            } else {
                const int row = row0 + n * 16 + rr;
                store4<F32>(a, s.first + row / a.G, h * a.G + row % a.G, D, d, y * (sum == 0.f ? 0.f : 1.f / sum));
            }
        }
    }
}

// Joins the chunks of the split sequences, a workgroup a row: thread i takes four values of every
// (THREADS / (D/4))th chunk, and the threads of a place are joined in LDS.
template <bool F32, int NB> __global__ __launch_bounds__(THREADS) void cache_join_kernel(AttnArgs a, int rq) {
    constexpr int D = NB * 32, PLACES = D / 4, WAYS = THREADS / PLACES, AT_ONCE = 4;
    __shared__ float sh_f[WAYS * AT_ONCE * 8];
    __shared__ __attribute__((aligned(16))) f32x4 sh_y[WAYS][PLACES];
    __shared__ float sh_w[WAVES], sh_s[WAVES];
    constexpr int MOST = WAYS * AT_ONCE * 8;            // chunks whose factors are kept at once
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int h = (int)blockIdx.y / a.QG, qg = (int)blockIdx.y % a.QG;
    if ((int)blockIdx.z >= a.list[0].x) return;
    const int4 seq = a.list[1 + blockIdx.z];
    const int row = qg * rq + (int)blockIdx.x, chunks = seq.z;
    if (row >= seq.y * a.G) return;
    const int64_t step = (int64_t)a.c.heads * a.QG * rq;
    const int64_t at = ((int64_t)seq.w * a.c.heads + h) * a.QG * rq + row;
    float top = -__builtin_inff();
    for (int c = tid; c < chunks; c += THREADS) top = fmaxf(top, a.part_m[at + c * step]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) sh_w[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, sh_w[w]);
    const int place = tid % PLACES, way = tid / PLACES;
    float sum = 0.f;
    f32x4 y = 0.f;
    for (int c0 = 0; c0 < chunks; c0 += MOST) {
        if (c0) __syncthreads();
        for (int c = tid; c < MOST; c += THREADS) {
            float f = 0.f;
            if (c0 + c < chunks) {
                const float m = a.part_m[at + (c0 + c) * step];
                f = m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m - top);
                sum = fmaf(a.part_l[at + (c0 + c) * step], f, sum);
            }
            sh_f[c] = f;
        }
        __syncthreads();
        const int n = min(chunks - c0, MOST);
        if (way < WAYS) {
            for (int c = way; c < n; c += WAYS * AT_ONCE) {
                f32x4 v[AT_ONCE];
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i) {
                    v[i] = 0.f;
                    if (c + i * WAYS < n)
                        v[i] = *reinterpret_cast<const f32x4*>(a.part_o + (at + (c0 + c + i * WAYS) * step) * D + place * 4);
                }
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i) {
                    const float f = c + i * WAYS < n ? sh_f[c + i * WAYS] : 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = fmaf(v[i][j], f, y[j]);
                }
            }
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) sh_s[wave] = sum;
    if (way < WAYS) sh_y[way][place] = y;
    __syncthreads();
    if (tid >= PLACES) return;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += sh_s[w];
    y = 0.f;
#pragma unroll
    for (int w = 0; w < WAYS; ++w) y += sh_y[w][tid];
    store4<F32>(a, seq.x + row / a.G, h * a.G + row % a.G, D, tid * 4, y * (sum == 0.f ? 0.f : 1.f / sum));
}

// Sizes that the host knows: groups of rows, units at most, split sequences and their parts at most.
struct Plan {
    int64_t NQ, QG, units, splits, parts;
};
Plan plan_of(const CacheShape& c, const AttnShape& a) {
    Plan p;
    const int64_t G = a.Hq / c.heads;
    p.NQ = a.max_q * G <= 16 || c.D > 128 ? 1 : 2;
    p.QG = ceil_div(a.max_q * G, p.NQ * 16);
    const int64_t tiles = std::max<int64_t>(1, a.width * c.tiles);      // of a sequence, at most
    const int64_t aim = std::max<int64_t>(1, TARGET / (c.heads * p.QG));
    // sum over b of ceil(tiles_b / chunk) <= aim + B, and a split sequence has at most twice its share
    const int64_t most = ceil_div(tiles, CHUNK_MIN);
    p.units = std::min(aim + a.B, a.B * most);
    p.splits = most > 1 ? std::min(aim, a.B) : 0;
    p.parts = most > 1 ? std::min(2 * aim, a.B * most) : 0;
    return p;
}

struct Workspace {
    int64_t list, m, l, o, bytes;
};
Workspace workspace_of(const CacheShape& c, const Plan& p) {
    Workspace w = {};
    if (!p.splits) return w;
    const int64_t rows = p.parts * c.heads * p.QG * p.NQ * 16;
    w.list = 0;
    w.m = round_up((p.splits + 1) * 16, REGION_ALIGN);
    w.l = w.m + round_up(rows * 4, REGION_ALIGN);
    w.o = w.l + round_up(rows * 4, REGION_ALIGN);
    w.bytes = w.o + rows * c.D * 4;
    return w;
}

// f(rows' type, K8, V8, blocks) for the call's types
template <typename F> void by_shape(mmq_otype o, mmq_wtype tk, mmq_wtype tv, int D, F f) {
    const auto types = [&](auto nb) {
        const auto k = [&](auto f32) {
            const auto v = [&](auto k8) {
                if (tv == MMQ_Q8_0) f(f32, k8, std::true_type(), nb);
                else f(f32, k8, std::false_type(), nb);
            };
            if (tk == MMQ_Q8_0) v(std::true_type());
            else v(std::false_type());
        };
        if (o == MMQ_OUT_F32) k(std::true_type());
        else k(std::false_type());
    };
    switch (D) {
        case 64: types(std::integral_constant<int, 2>()); break;
        case 128: types(std::integral_constant<int, 4>()); break;
        case 192: types(std::integral_constant<int, 6>()); break;
        default: types(std::integral_constant<int, 8>()); break;
    }
}

}  // namespace

// the first launch's workgroups stay below 2^24, the second's rows of the grid below 2^16
bool cache_attn_grid_ok(const CacheShape& c, const AttnShape& a) {
    const Plan p = plan_of(c, a);
    return p.QG * round_up(p.units * c.heads, 8) < (int64_t(1) << 24) && c.heads * p.QG < 65536;
}

size_t cache_attn_workspace_bytes(const CacheShape& c, const AttnShape& a) {
    return (size_t)workspace_of(c, plan_of(c, a)).bytes;
}

hipError_t launch_cache_attn(mmq_otype o, const void* q, int64_t ldq, mmq_wtype tk, const void* kcache, mmq_wtype tv,
                             const void* vcache, CacheShape c, const int32_t* table, int64_t ldt, const int32_t* lens,
                             const int32_t* starts, AttnShape s, const uint64_t* mask, float scale, void* out,
                             int64_t ldo, void* workspace, hipStream_t stream) {
    const Plan p = plan_of(c, s);
    const Workspace w = workspace_of(c, p);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    AttnArgs a = {};
    a.q = q;
    a.out = out;
    a.kc = static_cast<const uint8_t*>(kcache);
    a.vc = static_cast<const uint8_t*>(vcache);
    a.table = table;
    a.lens = lens;
    a.starts = starts;
    a.mask = mask;
    a.ldq = ldq;
    a.ldo = ldo;
    a.ldt = ldt;
    a.c = c;
    a.scale = scale;
    a.rows = (int)s.rows;
    a.B = (int)s.B;
    a.max_q = (int)s.max_q;
    a.G = s.Hq / c.heads;
    a.QG = (int)p.QG;
    a.cap = (int)std::min<int64_t>(s.width * c.tiles * CACHE_TILE, (int64_t(1) << 31) - CACHE_TILE);
    a.units = (int)p.units;
    a.splits = (int)p.splits;
    if (p.splits) {
        a.list = reinterpret_cast<int4*>(base + w.list);
        a.part_m = reinterpret_cast<float*>(base + w.m);
        a.part_l = reinterpret_cast<float*>(base + w.l);
        a.part_o = reinterpret_cast<float*>(base + w.o);
    }
    const dim3 grid((unsigned)(p.QG * round_up(p.units * c.heads, 8)));
    by_shape(o, tk, tv, c.D, [&](auto f32, auto k8, auto v8, auto nb) {
        constexpr bool F = decltype(f32)::value, K = decltype(k8)::value, V = decltype(v8)::value;
        constexpr int NB = decltype(nb)::value;
        if (p.NQ == 1) hipLaunchKernelGGL((cache_attn_kernel<F, K, V, NB, 1>), grid, dim3(THREADS), 0, stream, a);
        if constexpr (NB <= 4)
            if (p.NQ == 2) hipLaunchKernelGGL((cache_attn_kernel<F, K, V, NB, 2>), grid, dim3(THREADS), 0, stream, a);
        if (p.splits)
            hipLaunchKernelGGL((cache_join_kernel<F, NB>),
                               dim3((unsigned)std::min<int64_t>(p.NQ * 16, s.max_q * a.G), (unsigned)(c.heads * p.QG),
                                    (unsigned)p.splits),
                               dim3(THREADS), 0, stream, a, (int)p.NQ * 16);
    });
    return hipGetLastError();
}

}  // namespace mmq
