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
constexpr int RQ = 16;                      // rows of a workgroup
constexpr int CHUNK_MIN = 4;                // tiles of a chunk at least
constexpr int TARGET = 1024;                // workgroups aimed at
constexpr int P_BITS = 10;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

struct AttnArgs {
    const void* q;
    void* out;
    const uint8_t *kc, *vc;
    const int32_t *table, *lens, *starts;
    const uint64_t* mask;
    float *part_o, *part_m, *part_l;        // parts: [part][RQ][D], [part][RQ] twice
    int32_t* heads_of;                      // split sequences: count, then (sequence, chunks, first part)
    int64_t ldq, ldo, ldt;
    CacheShape c;
    float scale;
    int rows, B, max_q, Hq, G, QG, cap, units, splits;    // cap: tokens a table row can hold
};

__device__ inline h2 as_h2(uint32_t x) { return __builtin_bit_cast(h2, x); }
__device__ inline u16x2 as_u16(uint32_t x) { return __builtin_bit_cast(u16x2, x); }
__device__ inline uint32_t as_u32(h2 x) { return __builtin_bit_cast(uint32_t, x); }

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
    u = found;
    return any != 0;
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

template <bool Q8, int NB> struct Keys {
    u32x4 w[Q8 ? NB : NB / 2];
    __device__ void load(const uint8_t* rec, int lane) {
#pragma unroll
        for (int i = 0; i < (Q8 ? NB : NB / 2); ++i) w[i] = *reinterpret_cast<const u32x4*>(rec + (i * 64 + lane) * 16);
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
    __device__ void load(const uint8_t* rec, int lane) {
#pragma unroll
        for (int i = 0; i < (Q8 ? NB : NB / 2); ++i) w[i] = *reinterpret_cast<const u32x4*>(rec + (i * 64 + lane) * 16);
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

// F32: rows of f32 (two terms), or bf16 (one)
template <bool F32, bool K8, bool V8, int NB> __global__ __launch_bounds__(THREADS) void cache_attn_kernel(AttnArgs a) {
    constexpr int D = NB * 32, TERMS = F32 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float sh_o[WAVES][RQ][D + 4];
    __shared__ float sh_m[WAVES][RQ], sh_l[WAVES][RQ];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    // workgroups that share a chunk (one per QG) are 8 apart: on the same die, behind one L2
    const int qg = ((int)blockIdx.x >> 3) % a.QG;
    const int x = ((int)blockIdx.x >> 3) / a.QG * 8 + ((int)blockIdx.x & 7);
    const int unit = x / a.c.heads, h = x - unit * a.c.heads;
    if (unit >= a.units) return;
    Unit u;
    int splits;
    const bool there = find_unit(a, unit, tid, u, &splits);
    if (unit == 0 && h == 0 && qg == 0 && tid == 0 && a.heads_of) a.heads_of[0] = min(splits, a.splits);
    if (!there) return;
    const Seq s = seq_of(a, u.b);
    if (a.heads_of && u.chunks > 1 && u.chunk == 0 && h == 0 && qg == 0 && tid == 0 && u.split < a.splits) {
        int32_t* to = a.heads_of + 4 + 4 * u.split;
        to[0] = u.b;
        to[1] = u.chunks;
        to[2] = u.part;
    }
    const int nrows = min(min(s.n, a.max_q) * a.G - qg * RQ, RQ);      // this workgroup's
    if (nrows <= 0) return;
    const int row = qg * RQ + col;
    const bool has = col < nrows;
    const int i_row = row / a.G, head = h * a.G + row % a.G;
    const int ctx = s.len - s.n, len = min(s.len, a.cap);

    // q's terms
    h8 qt[TERMS][NB];
    float c_row;
    {
        float v[NB][8];
        float top = 0.f;
        const int64_t at = (int64_t)(s.first + i_row) * a.ldq + (int64_t)head * D + 8 * g;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[b][j] = 0.f;
            if (has) {
                if constexpr (F32) {
                    const u32x4_any* p = reinterpret_cast<const u32x4_any*>(static_cast<const float*>(a.q) + at + 32 * b);
                    const u32x4 r0 = p[0], r1 = p[1];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[b][j] = __builtin_bit_cast(float, (uint32_t)r0[j]);
                        v[b][4 + j] = __builtin_bit_cast(float, (uint32_t)r1[j]);
                    }
                } else {
                    const u32x4 r = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(a.q) + at + 32 * b);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[b][2 * j] = __builtin_bit_cast(float, r[j] << 16);
                        v[b][2 * j + 1] = __builtin_bit_cast(float, r[j] & 0xFFFF0000u);
                    }
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
                qt[0][b][j] = hi;
                if constexpr (F32) qt[1][b][j] = (_Float16)(y - (float)hi);
            }
        c_row = __builtin_amdgcn_ldexpf(a.scale * 1.44269504088896340736f, -e);
    }

    // the tiles that any of the rows can see
    const int last_row = (qg * RQ + nrows - 1) / a.G;
    int seen = len;
    if (!a.mask) seen = min(seen, ctx + last_row + 1);
    const int t0 = u.chunk * u.tiles;
    const int t1 = min(t0 + u.tiles, (max(seen, 0) + CACHE_TILE - 1) / CACHE_TILE);
    const uint64_t bits = a.mask && has ? a.mask[s.first + i_row] : 0;

    f32x4 o[2 * NB];
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) o[i] = 0.f;
    float m = -__builtin_inff(), l = 0.f;
    int k = 100;                                            // the exponent of p d_v; 100: no tile yet
    const int32_t* table = a.table + (int64_t)u.b * a.ldt;
    const uint64_t krec = cache_record(K8, D), vrec = cache_record(V8, D);
#pragma unroll 1
    for (int t = t0 + wave; t < t1; t += WAVES) {
        const uint32_t page = (uint32_t)__builtin_amdgcn_readfirstlane(table[t / a.c.tiles]);
        if (page >= (uint32_t)a.c.pages) continue;          // no such page: its tokens are not seen
        const uint64_t rec = ((uint64_t)page * a.c.heads + h) * a.c.tiles + t % a.c.tiles;
        const uint8_t *kp = a.kc + rec * krec, *vp = a.vc + rec * vrec;
        Keys<K8, NB> kw;
        Values<V8, NB> vw;
        kw.load(kp, lane);
        vw.load(vp, lane);
        u32x4 ks[NB], vs[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            ks[b] = *reinterpret_cast<const u32x4*>(kp + cache_values(K8, D) + (g * NB + b) * 16);
            vs[b] = *reinterpret_cast<const u32x4*>(vp + cache_values(V8, D) + (g * NB + b) * 16);
        }

        float sc[8];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            f32x4 acc = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const h8 kv = kw.get(hh, b);
                f32x4 r = 0.f;
#pragma unroll
                for (int i = 0; i < TERMS; ++i) r = mfma(kv, qt[i][b], r);
                const h2 d0 = as_h2(ks[b][2 * hh]), d1 = as_h2(ks[b][2 * hh + 1]);
                acc[0] = fmaf(r[0], (float)d0[0], acc[0]);
                acc[1] = fmaf(r[1], (float)d0[1], acc[1]);
                acc[2] = fmaf(r[2], (float)d1[0], acc[2]);
                acc[3] = fmaf(r[3], (float)d1[1], acc[3]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[4 * hh + i] = acc[i] * c_row;
        }
        // tokens that this row does not see; scales of slots past the sequence are not read as numbers
        uint32_t see = 0xFF;
        if (CACHE_TILE * (t + 1) > min(ctx, len)) {
            see = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int pos = CACHE_TILE * t + 16 * (i >> 2) + 4 * g + (i & 3), ahead = pos - ctx;
                bool v = pos < len;
                if (ahead >= 0) v = v && (a.mask ? ahead < 64 && (bits >> ahead & 1) : ahead <= i_row);
                see |= (uint32_t)v << i;
                if (pos >= len) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) vs[b][i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                }
            }
        }
        float top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!(see >> i & 1)) sc[i] = -__builtin_inff();
            top = fmaxf(top, sc[i]);
        }
        top = xor_max(top);
        const float m1 = fmaxf(m, top);
        const float base = m1 == -__builtin_inff() ? 0.f : m1;      // nothing seen yet: every p is 0
        const float fall = __builtin_amdgcn_exp2f(m - base);
        m = m1;
        float p[8];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(sc[i] - base + (float)P_BITS);
            sum += p[i];
        }
        l = l * fall + sum;

        // the exponent k, from the scales that are finite (others leave the rest of the tile as it is)
        u16x2 dtop = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) dtop = __builtin_elementwise_max(dtop, as_u16(vs[b][i] & 0x7FFF7FFFu));
        if (__any(max(dtop[0], dtop[1]) >= 0x7C00)) {
            dtop = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint16_t d = as_u16(vs[b][i >> 1] & 0x7FFF7FFFu)[i & 1];
                    if (d < 0x7C00) dtop[0] = max(dtop[0], d);
                }
        }
        float dmax = (float)__builtin_bit_cast(_Float16, max(dtop[0], dtop[1]));
        dmax = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, xor_max(dmax))));
        float fall_k = fall;
        if (dmax > 0.f) {
            const int k1 = min(k, 1 - __builtin_amdgcn_frexp_expf(dmax));
            if (k != 100) fall_k = __builtin_amdgcn_ldexpf(fall, k1 - k);
            k = k1;
        }
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) o[i] *= fall_k;
        const int kk = k == 100 ? 0 : k;
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_ldexpf(p[i], kk);

#pragma unroll
        for (int b = 0; b < NB; ++b) {
            h8 pt[TERMS];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = (float)as_h2(vs[b][i >> 1])[i & 1];
                const float y = see >> i & 1 ? p[i] * d : 0.f;      // also where d is not finite
                const _Float16 hi = (_Float16)y;
                pt[0][i] = hi;
                if constexpr (F32) pt[1][i] = (_Float16)(y - (float)hi);
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const h8 vv = vw.get(b, v);
#pragma unroll
                for (int i = 0; i < TERMS; ++i) o[2 * b + v] = mfma(vv, pt[i], o[2 * b + v]);
            }
        }
    }

    // the waves' sums
    l = xor_sum(l);
    if (g == 0) {
        sh_m[wave][col] = m;
        sh_l[wave][col] = l;
    }
    __syncthreads();
    float top = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, sh_m[w][col]);
    const float mine = m == -__builtin_inff() ? 0.f : __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(m - top), k == 100 ? 0 : -k);
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i)
        *reinterpret_cast<f32x4*>(&sh_o[wave][col][16 * i + 4 * g]) = o[i] * mine;
    __syncthreads();
    const bool split = u.chunks > 1;
    const int64_t part = split ? ((int64_t)(u.part + u.chunk) * a.c.heads + h) * a.QG + qg : 0;
    for (int e = tid; e < nrows * (D / 4); e += THREADS) {
        const int r = e / (D / 4), d = e % (D / 4) * 4;
        float big = -__builtin_inff(), sum = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) big = fmaxf(big, sh_m[w][r]);
        f32x4 y = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            y += *reinterpret_cast<const f32x4*>(&sh_o[w][r][d]);
            if (sh_m[w][r] > -__builtin_inff()) sum += sh_l[w][r] * __builtin_amdgcn_exp2f(sh_m[w][r] - big);
        }
        if (split) {
            *reinterpret_cast<f32x4*>(a.part_o + (part * RQ + r) * D + d) = y;
            if (d == 0) {
                a.part_m[part * RQ + r] = big;
                a.part_l[part * RQ + r] = sum;
            }
        } else {
            const int rr = qg * RQ + r;
            const int64_t to = (int64_t)(s.first + rr / a.G) * a.ldo + (int64_t)(h * a.G + rr % a.G) * D + d;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            if constexpr (F32) {
                float* p = static_cast<float*>(a.out) + to;
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = y[j] * inv;
            } else {
                uint16_t* p = static_cast<uint16_t*>(a.out) + to;
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = bf16_rne(y[j] * inv);
            }
        }
    }
}

// Joins the chunks of the split sequences: a wave a row.
template <bool F32, int NB> __global__ __launch_bounds__(THREADS) void cache_join_kernel(AttnArgs a) {
    constexpr int D = NB * 32;
    const int lane = threadIdx.x & 63;
    const int r = (int)blockIdx.x * WAVES + (int)(threadIdx.x >> 6);
    const int h = (int)blockIdx.y / a.QG, qg = (int)blockIdx.y % a.QG;
    if ((int)blockIdx.z >= a.heads_of[0]) return;
    const int32_t* from = a.heads_of + 4 + 4 * blockIdx.z;
    const int b = from[0], chunks = from[1], first = from[2];
    const Seq s = seq_of(a, b);
    const int row = qg * RQ + r;
    if (row >= min(s.n, a.max_q) * a.G) return;
    const int64_t step = (int64_t)a.c.heads * a.QG * RQ;
    const int64_t at = ((int64_t)first * a.c.heads + h) * a.QG * RQ + (int64_t)qg * RQ + r;
    float top = -__builtin_inff();
    for (int c = 0; c < chunks; ++c) top = fmaxf(top, a.part_m[at + c * step]);
    float sum = 0.f, y[(D + 63) / 64] = {};
    for (int c = 0; c < chunks; ++c) {
        const float m = a.part_m[at + c * step];
        if (m == -__builtin_inff()) continue;
        const float f = __builtin_amdgcn_exp2f(m - top);
        sum = fmaf(a.part_l[at + c * step], f, sum);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) y[i] = fmaf(a.part_o[(at + c * step) * D + i * 64 + lane], f, y[i]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t to = (int64_t)(s.first + row / a.G) * a.ldo + (int64_t)(h * a.G + row % a.G) * D;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        if constexpr (F32) static_cast<float*>(a.out)[to + i * 64 + lane] = y[i] * inv;
        else static_cast<uint16_t*>(a.out)[to + i * 64 + lane] = bf16_rne(y[i] * inv);
    }
}

// Sizes that the host knows: groups of rows, units at most, split sequences and their parts at most.
struct Plan {
    int64_t QG, units, splits, parts;
};
Plan plan_of(const CacheShape& c, const AttnShape& a) {
    Plan p;
    const int64_t G = a.Hq / c.heads;
    p.QG = ceil_div(a.max_q * G, RQ);
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
    const int64_t rows = p.parts * c.heads * p.QG * RQ;
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
    a.Hq = s.Hq;
    a.G = s.Hq / c.heads;
    a.QG = (int)p.QG;
    a.cap = (int)std::min<int64_t>(s.width * c.tiles * CACHE_TILE, (int64_t(1) << 31) - CACHE_TILE);
    a.units = (int)p.units;
    a.splits = (int)p.splits;
    if (p.splits) {
        a.heads_of = reinterpret_cast<int32_t*>(base + w.list);
        a.part_m = reinterpret_cast<float*>(base + w.m);
        a.part_l = reinterpret_cast<float*>(base + w.l);
        a.part_o = reinterpret_cast<float*>(base + w.o);
    }
    const dim3 grid((unsigned)(p.QG * round_up(p.units * c.heads, 8)));
    by_shape(o, tk, tv, c.D, [&](auto f32, auto k8, auto v8, auto nb) {
        constexpr bool F = decltype(f32)::value, K = decltype(k8)::value, V = decltype(v8)::value;
        constexpr int NB = decltype(nb)::value;
        hipLaunchKernelGGL((cache_attn_kernel<F, K, V, NB>), grid, dim3(THREADS), 0, stream, a);
        if (p.splits)
            hipLaunchKernelGGL((cache_join_kernel<F, NB>), dim3(RQ / WAVES, (unsigned)(c.heads * p.QG), (unsigned)p.splits),
                               dim3(THREADS), 0, stream, a);
    });
    return hipGetLastError();
}

}  // namespace mmq
