// cache_attn.hip - attention over the block-quantised cache, for one new token a sequence, chains of
// them and trees of drafted ones.
//
// Rows are (new token, query head) pairs that share a head of the cache; a workgroup has 16 or 32 of them
// and a part of the sequence's tiles of 32 tokens, its waves take the tiles in turn. Per tile:
//   1. scores, transposed: S^T = K q^T on the matrix core. int8 or 4-bit whole numbers are exact in
//      f16; a block of 32 values is one product, whose four sums a lane are scaled by their tokens'
//      scales in f32. q is held as f16 terms of q 2^e (e: the row's exponent, its largest value in
//      [2^13, 2^14)): two for f32 rows, which leave 2^-22 of a value, one for bf16 rows, whose 8 bits
//      it holds exactly down to 2^-30 of the row's largest.
//   2. p = 2^(score - m), m the running maximum, sums of p in f32; 2^8 of headroom keeps small p away
//      from f16's subnormals.
//   3. O^T += V^T P^T. The scale of a token's block of values lies along the sum, so it goes into P:
//      p d_v 2^k, for f32 rows in two f16 terms (the rounding of the first is in the second), for bf16
//      rows in one, two roundings of 2^-11 of a term, where the result's own is 2^-8: errors are 1.004 to
//      1.02 times those of the result's rounding alone. (Two terms leave that alone there too, and take 88
//      us for 73 of 8 trees, 286 for 235 of 2048 tokens behind 2048, 50 for 47 of 64 single tokens in q4_0.)
//      k, the wave's running exponent, keeps the largest d_v 2^k in [4, 8) and is never negative, so that
//      d_v 2^k is exact in f16. Tiles with scales of 8 and more (values from 1016, or 64 in q4_0) come last, in
//      a loop of their own, which makes p d_v 2^k in f32 and holds it in range by m: a token's score counts
//      as higher by as much as its largest scale times 2^k is above 8. So a large value takes bits of a row's
//      result only by its own weight there. (Inside the main loop, a branch around the products took 40 registers.)
// A lane holds the tokens of S^T's rows that it needs as P^T's k: the cache's order of tokens makes
// them the same (cache.h).
// The waves' sums are joined in LDS. Work that several workgroups share leaves its parts in the
// workspace, and a second launch joins them.
//
// What bounds it, and what it reaches (8 heads of 128 values, 4 query heads for each, q8_0 unless said; kernels' times in
// a profiler's trace):
//   - one new token a sequence: memory. 64 sequences of 128 to 8192 tokens, f32, 58.5 us for 277 MB (4.7 TB/s);
//     one of 131072 tokens, bf16, values in q4_0, 43 us for 218 MB (5.0 TB/s); the second launch takes 5 us.
//     With keys and values in q4_0 vector instructions (24 us in bf16, 29 in f32) hide behind the loads (28 us) in
//     part only: the 64 sequences 43.5 us in bf16, 50 in f32 for 146 MB.
//   - many rows: the vector unit, whose time and the matrix core's add up here. A wave's tile costs some 180
//     instructions whatever its rows (8-bit numbers made f16, scales), and for each 16 rows 130 (bf16)
//     or 180 (f32) and 16 or 32 products: 8 trees of 48 to 64 tokens, bf16, 72 us (0.37 PFLOP/s), a chain
//     of 512 behind 3584, f32 with twice the products, 109 us (0.3 PFLOP/s).
#include <algorithm>

#include "cache.h"

namespace mmq {
namespace {

constexpr int WAVES = 4, THREADS = WAVES * 64;
// Tiles of a workgroup's part at least: one a wave, or two where beginning costs more. 3 trees of 5 to 13 tokens
// 17.8 us with 4 and 16.3 with 8, one token of 777 11.4 and 12.2.
constexpr int step_min(int rq) { return rq == 16 ? 4 : 8; }
// What beginning an item costs, in tiles (a tile of two groups of rows takes about twice the time). 64 sequences of 128 to
// 8192 tokens, one group, 83.5, 74, 68.5 and 72 us with 2, 5, 10 and 16; 8 trees, two groups, 81.5, 76, 78 and 79.
constexpr int begin_cost(int rq) { return rq == 16 ? 10 : 5; }
// Tiles of a table's row up to which items are not cut, so that there is no second launch: 32 tokens that see 700
// each (22 tiles) 21.4 us with 16 and 15.5 with 24; one that sees 777 (25) 11.0 with 24 and 12.0 with 32.
constexpr int64_t WHOLE = 24;
// p is held times 2^P_BITS, the maximum may rise by P_SLACK before it is taken anew, and scales times 2^k are below
// 2^D_BITS in the main loop: p d 2^k stays below 2^15. With 10, 2 and 3, 2048 tokens behind 2048 236 us and with 8, 4 and
// 3 233.5; 8 trees 75.7 and 74.8. With 10, 3 and 2 ordinary values in q4_0 are large ones: 131072 tokens 61 us, and 49.5 so.
constexpr float P_BITS = 8.f, P_SLACK = 4.f;
constexpr int D_BITS = 3;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Where a workgroup's part of the launch's range ends inside an item, for the second launch.
struct Cut {
    int64_t start, end, step;               // the item's range; length of a workgroup's part (0: no item is cut here)
    int first, rows, h, qg;                 // first row of the sequence, its rows, the item's head and group of rows
};

struct AttnArgs {
    const void* q;
    void* out;
    const uint8_t *kc, *vc;
    const int32_t *table, *lens, *starts;
    const uint64_t* mask;
    float *part_o, *part_m, *part_l;        // parts: [part][rows][D], [part][rows] twice
    Cut* cuts;                              // of each workgroup's end
    int64_t ldq, ldo, ldt;
    CacheShape c;
    float scale;
    int rows, B, max_q, G, cap;             // cap: tokens a table row can hold
    int even, spare;                        // how work is counted; even: workgroups beyond one an item (0: no cuts)
};

__device__ inline h2 as_h2(uint32_t x) { return __builtin_bit_cast(h2, x); }
__device__ inline u16x2 as_u16(uint32_t x) { return __builtin_bit_cast(u16x2, x); }
__device__ inline uint32_t as_u32(h2 x) { return __builtin_bit_cast(uint32_t, x); }

// A value that is the same in every lane, in a scalar register: what comes from LDS or an integer
// division would be kept, with all that follows from it (loop counts, buffer descriptors), in lanes.
__device__ inline int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline int64_t scalar(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)scalar((int)(v >> 32)) << 32 | (uint32_t)scalar((int)v));
}

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

// The launch's work is one range: for every sequence, head and group of RQ rows (an item) a cost, by its tiles.
// Each workgroup takes an equal part of the range, whatever the sequences' lengths, and finds its place
// from them by itself. An item that is cut leaves parts in the workspace. Two ways to count:
//   even: an item costs 1 for each of its parts, which are equal and at most `share` tiles long. For
//         items few enough that the parts' ends do not matter. (An item of one part is finished by its workgroup. The
//         second launch is made all the same, wherever the table is wide enough for cuts: the host does not know the
//         lengths. It finds nothing to join then.)
//   tiles: an item costs its tiles and begin_cost more, what beginning an item takes; workgroups end anywhere.
struct Found {
    int64_t start;                          // of the sequence
    int b, first, n, len, cost, groups;     // cost of an item; groups of rows
};
template <typename T> __device__ inline T lanes_sum_up(T v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const T u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}
__device__ inline int64_t wave_scan(int64_t v, int lane) {          // inclusive sum over the lanes
    return __any(v >= 1 << 24) ? lanes_sum_up((long long)v, lane) : lanes_sum_up((int)v, lane);
}
__device__ inline int64_t quotient_up(int64_t x, int64_t n) {       // ceil(x / n), x < 2^60, n < 2^31
    int64_t q;                                                      // within 2^8 of it
    if (x < 1 << 24) q = (int)((float)x * __builtin_amdgcn_rcpf((float)n));
    else q = (int64_t)((double)x / (double)n);
    while (q * n >= x + n) --q;
    while (q * n < x) ++q;
    return scalar(q);
}
template <int RQ> struct Work {
    struct Shared {
        int64_t start[THREADS], total[WAVES];           // of a thread's sequences
        Found found;
    };
    const AttnArgs& a;
    Shared& sh;
    int tid, per;                                       // per: sequences of a thread
    int share;
    Seq own;                                            // the thread's first sequence
    __device__ Seq seq(int i) const { return i == 0 ? own : seq_of(a, tid * per + i); }
    __device__ int cost(const Seq& s) const {
        const int tiles = seq_tiles(a, s);
        return !a.even ? (tiles ? tiles + begin_cost(RQ) : 0) : tiles <= share ? min(tiles, 1) : (tiles + share - 1) / share;
    }
    __device__ int groups(const Seq& s) const { return (min(s.n, a.max_q) * a.G + RQ - 1) / RQ; }
    // the sum of f over all items, and that over the sequences before the thread's
    template <typename F> __device__ int64_t sum_up(F f, int64_t& before) {
        before = 0;
        if (a.B == 1) return scalar((int64_t)f(own) * groups(own) * a.c.heads);
        int64_t mine = 0;
        for (int i = 0; i < per && tid * per + i < a.B; ++i) {
            const Seq s = seq(i);
            mine += (int64_t)f(s) * groups(s) * a.c.heads;
        }
        const int64_t sum = wave_scan(mine, tid & 63);
        if ((tid & 63) == 63) sh.total[tid >> 6] = sum;
        __syncthreads();
        before = sum - mine;
        int64_t all = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            if (w < tid >> 6) before += sh.total[w];
            all += sh.total[w];
        }
        return scalar(all);
    }
    // the whole range; every thread calls it once, before find()
    __device__ Work(const AttnArgs& args, Shared& shared, int64_t& all) : a(args), sh(shared), tid(threadIdx.x), own{0, 0, 0} {
        per = (a.B + THREADS - 1) / THREADS;
        if (tid * per < a.B || a.B == 1) own = seq_of(a, a.B == 1 ? 0 : tid * per);
        int64_t before;
        share = 1 << 30;
        if (a.spare) {
            // sum of ceil(tiles / share) <= spare + items = the workgroups
            const int64_t tiles = sum_up([&](const Seq& s) { return seq_tiles(a, s); }, before);
            share = (int)min(max(quotient_up(tiles, a.spare), (int64_t)step_min(RQ)), (int64_t)1 << 30);
            if (a.B > 1) __syncthreads();
        }
        all = sum_up([&](const Seq& s) { return cost(s); }, before);
        sh.start[tid] = before;
    }
    // the sequence at `pos` of the range
    __device__ Found find(int64_t pos) {
        if (a.B == 1) return {0, 0, scalar(own.first), scalar(own.n), scalar(own.len), scalar(cost(own)), scalar(groups(own))};
        if (tid == 0) sh.found.cost = 0;                // there always is one, unless the lengths change meanwhile
        __syncthreads();
        int64_t at = sh.start[tid];
        for (int i = 0; i < per && at <= pos && tid * per + i < a.B; ++i) {
            const Seq s = seq(i);
            const int n = groups(s), c = cost(s);
            const int64_t size = (int64_t)c * n * a.c.heads;
            if (pos < at + size) {                      // one thread's
                sh.found = {at, tid * per + i, s.first, s.n, s.len, c, n};
                break;
            }
            at += size;
        }
        __syncthreads();
        const Found& f = sh.found;
        return {scalar(f.start), scalar(f.b), scalar(f.first), scalar(f.n), scalar(f.len), scalar(f.cost), scalar(f.groups)};
    }
};

// One item's part: tiles [t0, t1) for the rows row0.. of a sequence's head.
struct Segment {
    Found f;
    int h, qg, row0, nrows, ctx, len, t0, t1;
    int part;                               // -1: the whole item
};

// The thread's number, new to the compiler at each segment: what follows from it would else be computed once
// for all of them and held in registers that the main loop has not.
__device__ inline int thread_here() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// Calls one(segment) for each item in the workgroup's part of the range.
template <int RQ, typename F> __device__ inline void each_segment(const AttnArgs& a, F one) {
    __shared__ typename Work<RQ>::Shared shared;
    int64_t all;
    Work<RQ> work(a, shared, all);
    // neighbours in the range on the same die, behind one L2 (the items of one head read the same cache)
    const int per_die = (int)gridDim.x >> 3, w = ((int)blockIdx.x & 7) * per_die + ((int)blockIdx.x >> 3);
    const int64_t step = max(quotient_up(all, gridDim.x), (int64_t)(a.even ? 1 : step_min(RQ)));
    const int64_t begin = w * step, end = min(all, begin + step);
    if (a.cuts && threadIdx.x == 0) a.cuts[w].step = 0;
    int64_t pos = begin;
    while (pos < end) {
        Segment s;
        s.f = work.find(pos);
        if (s.f.cost <= 0 || s.f.groups <= 0) break;
        const int64_t seq_end = s.f.start + (int64_t)s.f.cost * s.f.groups * a.c.heads;
        int item = (int)((float)(pos - s.f.start) / (float)s.f.cost);        // fewer than 2^20: within one of the quotient
        while ((int64_t)item * s.f.cost > pos - s.f.start) --item;
        while ((int64_t)(item + 1) * s.f.cost <= pos - s.f.start) ++item;
        item = scalar(item);
        for (; pos < end && pos < seq_end; ++item) {
            const int64_t start = s.f.start + (int64_t)item * s.f.cost;
            const int from = (int)(pos - start), to = (int)min((int64_t)s.f.cost, end - start);
            pos = start + to;
            s.h = scalar(item / s.f.groups);
            // first and last groups of rows in turn: the first rows of a chain see fewer tokens than the last
            const int i = item - s.h * s.f.groups;
            s.qg = i & 1 ? s.f.groups - 1 - i / 2 : i / 2;
            s.row0 = s.qg * RQ;
            s.nrows = min(min(s.f.n, a.max_q) * a.G - s.row0, RQ);
            s.ctx = s.f.len - s.f.n;
            s.len = min(s.f.len, a.cap);
            const int tiles = (s.len + CACHE_TILE - 1) / CACHE_TILE;
            if (a.even) {
                s.t0 = (int)((int64_t)tiles * from / s.f.cost);
                s.t1 = (int)((int64_t)tiles * to / s.f.cost);
            } else {
                s.t0 = max(from - begin_cost(RQ), 0);
                s.t1 = max(to - begin_cost(RQ), 0);
            }
            // the tiles that any of the rows can see
            const int seen = a.mask ? s.len : min(s.len, s.ctx + (s.row0 + s.nrows - 1) / a.G + 1);
            s.t0 = scalar(s.t0);
            s.t1 = scalar(min(s.t1, (max(seen, 0) + CACHE_TILE - 1) / CACHE_TILE));
            s.part = from == 0 && to == s.f.cost ? -1 : start + from == begin ? 2 * w : 2 * w + 1;
            if (to < s.f.cost && threadIdx.x == 0)
                a.cuts[w] = {start, start + s.f.cost, step, s.f.first, min(s.f.n, a.max_q) * a.G, s.h, s.qg};
            one(s);
        }
    }
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
__device__ inline h2 two_nibbles(uint32_t x, int s) {
    const h2 off = {(_Float16)1032.f, (_Float16)1032.f};
    return as_h2(((x >> s) & 0x000F000Fu) | 0x64006400u) - off;
}
__device__ inline h8 from_nibbles(uint32_t x) {             // keys
    return join(two_nibbles(x, 0), two_nibbles(x, 4), two_nibbles(x, 8), two_nibbles(x, 12));
}
__device__ inline h8 from_nibbles(uint32_t x, uint32_t y, int s) {      // values: s = 0, or 4 for the upper ones
    return join(two_nibbles(x, s), two_nibbles(x, 8 + s), two_nibbles(y, s), two_nibbles(y, 8 + s));
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
            return from_nibbles(x);
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
            return from_nibbles(x, y, 4 * u);
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

// Whether new token i, of mask `bits`, sees the token at `pos`; ctx tokens lie before the new ones.
__device__ inline bool sees(const AttnArgs& a, uint64_t bits, int i, int pos, int ctx, int limit) {
    const int ahead = pos - ctx;
    if (pos >= limit) return false;
    return ahead < 0 || (a.mask ? ahead < 64 && (bits >> ahead & 1) : ahead <= i);
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
__device__ inline void load_rows(const AttnArgs& a, int first, int h, int row, int g, Rows<TERMS, NB>& r) {
    constexpr bool F32 = TERMS == 2;
    r.i = row / a.G;
    r.bits = a.mask ? a.mask[first + r.i] : 0;
    r.m = -__builtin_inff();
    r.off = P_BITS;
    r.l = 0.f;
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) r.o[j] = 0.f;
    float v[NB][8];
    float top = 0.f;
    const int64_t at = (int64_t)(first + r.i) * a.ldq + (int64_t)(h * a.G + row % a.G) * (NB * 32) + 8 * g;
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

// Waves of a SIMD that the registers are dealt out for, and so workgroups of a compute unit.
//   - 8 blocks of values need the 512 registers of one wave: f32, 4 trees of 60 tokens 100 us, with two waves, which
//     spill, 211.
//   - 6 blocks, with one wave or two (with which the f32 forms of q8_0 keys or values and the bf16 form of both spill 20
//     to 104 bytes, none on the main loop's usual path): 512 tokens behind 1488, f32, 121 and 87 us, 8 trees 218 and 167, 64
//     single tokens in q4_0 90 and 68; but in q8_0 95 and 103, and 32 of 8000 149 and 171.
//   - 4 blocks, with three waves, which spill 12 to 480 bytes, or two: 64 single tokens, f32, 88 and 63 us, 8 trees 241 and
//     104. (In q4_0 and bf16 46 and 47.)
//   - 2 blocks, with three waves, of which three forms spill 20 to 36 bytes, or two: 512 tokens behind 1488 47 and 39 us, one
//     single token of 65536 23 and 22; but 64 single tokens in q4_0 and bf16 31.5 and 34.
constexpr int waves_of(int NB) { return NB <= 6 ? 2 : 1; }

// A row's maximum taken anew where a score is far above it, and there alone: its bits do not depend on the other rows
// of the products. top: the lane's largest, times r.c.
template <typename R> __device__ inline void raise_max(float top, R& r) {
    if (__any(top > r.m + P_SLACK)) {
        const float above = xor_max(top), m1 = above > r.m + P_SLACK ? above : r.m;
        const float base = m1 == -__builtin_inff() ? 0.f : m1;
        const float fall = __builtin_amdgcn_exp2f(r.m - base);
        r.m = m1;
        r.off = P_BITS - base;
        r.l *= fall;
#pragma unroll
        for (auto& o : r.o) o *= fall;
    }
}
// A lane's 8 weights, and their sum
template <typename R> __device__ inline void weights(const float (&sc)[8], R& r, float (&p)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(fmaf(sc[i], r.c, r.off));
        r.l += p[i];
    }
}
// A product as the f32 that it is rounded to. Without it, the compiler makes a term's f16 from the product's factors, with
// one rounding, where the term is subtracted, and from their f32, with two, where it is used: where those differ, the
// second term is the first's error no more (one in some thousands, then 2^-11 of the term).
__device__ inline float rounded(float x) {
    asm("" : "+v"(x));
    return x;
}
// Two numbers as f16 terms
template <bool F32> __device__ inline void in_terms(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    const h2 h = {(_Float16)x0, (_Float16)x1};
    hi = as_u32(h);
    if constexpr (F32) {
        const h2 l = {(_Float16)(x0 - (float)h[0]), (_Float16)(x1 - (float)h[1])};
        lo = as_u32(l);
    }
}

// A wave's products go before the other wave's softmax: 512 tokens behind 3488, bf16, 76.6 us and 73 so; 2048 behind 2048
// 242 and 231.5; single tokens alike. (A wave alone on its SIMD has no other: 256 values, 156 us and 174 so.)
template <bool SHARED> __device__ inline void products_first(bool yes) {
    if constexpr (SHARED) {
        if (yes) __builtin_amdgcn_s_setprio(1);
        else __builtin_amdgcn_s_setprio(0);
    }
}

// What a wave knows of its tiles' value scales: their exponent, and the largest f16 bits that it suits.
struct Exponent {
    int k;
    uint32_t limit;
};
constexpr uint32_t WIDE = (15 + D_BITS) << 10;              // 2^D_BITS as f16

// F32: rows of f32 (two terms), or bf16 (one). NQ: groups of 16 rows of a workgroup.
template <bool F32, bool K8, bool V8, int NB, int NQ>
__global__ __launch_bounds__(THREADS, waves_of(NB)) void cache_attn_kernel(AttnArgs a) {
    constexpr int D = NB * 32, TERMS = F32 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float sh_o[WAVES][16][D + 4];
    __shared__ float sh_m[WAVES][16], sh_l[WAVES][16];
    // f32 rows in twos: q's terms would take 64 registers that the main loop has not, and are the same in every wave
    constexpr bool Q_LDS = F32 && NQ == 2;
    constexpr bool SHARED = waves_of(NB) > 1;
    __shared__ __attribute__((aligned(16))) h8 sh_q[Q_LDS ? NQ * TERMS * NB : 1][64];
    each_segment<NQ * 16>(a, [&](const Segment& s) __attribute__((always_inline)) {
        const int tid = thread_here(), lane = tid & 63, wave = scalar(tid >> 6), col = lane & 15, g = lane >> 4;
        const int h = s.h, row0 = s.row0, nrows = s.nrows, ctx = s.ctx, len = s.len, t0 = s.t0, t1 = s.t1;

        Rows<TERMS, NB> r[NQ];                                  // (past the rows: the last one again)
#pragma unroll
        for (int n = 0; n < NQ; ++n) load_rows<TERMS, NB>(a, s.f.first, h, row0 + min(n * 16 + col, nrows - 1), g, r[n]);
        if constexpr (Q_LDS) {
            if (wave == 0) {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < TERMS; ++i)
#pragma unroll
                        for (int b = 0; b < NB; ++b) sh_q[(n * TERMS + i) * NB + b][lane] = r[n].q[i][b];
            }
            __syncthreads();
        }

        Exponent ex = {15, 0};                                  // no scale yet
        // pages by scalar loads: a vector load would be waited for with every load before it
        const auto* table = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)(a.table + (int64_t)s.f.b * a.ldt);
        const int shift = __builtin_ctz(a.c.tiles);
        const auto record = [&](int t, uint32_t page) {
            return ((uint64_t)page * a.c.heads + h) * a.c.tiles + (t & (a.c.tiles - 1));
        };
        Keys<K8, NB> kw;
        Values<V8, NB> vw;
        const auto load_k = [&](uint64_t rec, bool there, int lane) __attribute__((always_inline)) {
            kw.load(Record(a.kc, rec, cache_record(K8, D), there), lane);
        };
        const auto load_v = [&](uint64_t rec, bool there, int lane) __attribute__((always_inline)) {
            vw.load(Record(a.vc, rec, cache_record(V8, D), there), lane);
        };
        const auto scores = [&](int lane, float (&sc)[NQ][8]) __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < 8; ++i) sc[n][i] = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                h8 q[NQ][TERMS];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < TERMS; ++i) q[n][i] = Q_LDS ? sh_q[(n * TERMS + i) * NB + b][lane] : r[n].q[i][b];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const h8 kv = kw.get(hh, b);
                    const h2 d0 = as_h2(kw.d[b][2 * hh]), d1 = as_h2(kw.d[b][2 * hh + 1]);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        f32x4 y = 0.f;
#pragma unroll
                        for (int i = 0; i < TERMS; ++i) y = mfma(kv, q[n][i], y);
                        sc[n][4 * hh] = fmaf(y[0], (float)d0[0], sc[n][4 * hh]);
                        sc[n][4 * hh + 1] = fmaf(y[1], (float)d0[1], sc[n][4 * hh + 1]);
                        sc[n][4 * hh + 2] = fmaf(y[2], (float)d1[0], sc[n][4 * hh + 2]);
                        sc[n][4 * hh + 3] = fmaf(y[3], (float)d1[1], sc[n][4 * hh + 3]);
                    }
                }
            }
        };
        // tokens that a row does not see; scales of slots past the sequence are not read as numbers
        const auto hide = [&](int t, int limit, int g, float (&sc)[NQ][8]) __attribute__((always_inline)) {
            if (__builtin_expect(CACHE_TILE * (t + 1) > min(ctx, limit), 0)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int pos = CACHE_TILE * t + 16 * (i >> 2) + 4 * g + (i & 3);
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        if (!sees(a, r[n].bits, r[n].i, pos, ctx, limit)) sc[n][i] = -__builtin_inff();
                    if (pos >= limit) {
#pragma unroll
                        for (int b = 0; b < NB; ++b) vw.d[b][i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                    }
                }
            }
        };
        const auto product = [&](int b, const h8 (&pt)[NQ][TERMS]) __attribute__((always_inline)) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const h8 vv = vw.get(b, v);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < TERMS; ++i) r[n].o[2 * b + v] = mfma(vv, pt[n][i], r[n].o[2 * b + v]);
            }
        };
        // A tile's keys are loaded while the products of values of the one before run, its values while the
        // next scores do: the registers are free by then. No such page: its tokens are not seen, and the
        // first page stands in for it.
        int t = t0 + wave, left_out = t1;                       // left_out: the first tile with scales from 2^D_BITS on
        bool ok = false;
        uint64_t rec = 0;
        if (t < t1) {
            const uint32_t page = (uint32_t)table[t >> shift];
            ok = page < (uint32_t)a.c.pages;
            rec = record(t, ok ? page : 0);
            load_k(rec, true, lane);
            load_v(rec, true, lane);
        }
#pragma unroll 1
        for (; t < t1; t += WAVES) {
            const int limit = ok ? len : 0;
            const bool more = t + WAVES < t1;
            const uint32_t page = (uint32_t)table[(more ? t + WAVES : t) >> shift];

            // 1. the products of scores
            products_first<SHARED>(true);
            float sc[NQ][8];
            scores(lane, sc);

            // (the scores are finished before the loads, whose registers the products' operands leave)
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(sc[n][i]));
            ok = page < (uint32_t)a.c.pages;
            rec = record(t + WAVES, ok ? page : 0);           // (not loaded from where there is none)
            load_k(rec, more, lane);

            hide(t, limit, g, sc);

            // The exponent k of the value scales. One that is not finite counts as 0, after the sums that it
            // goes into, those of the rows that see its token, are made NaN.
            u16x2 dtop = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dtop = __builtin_elementwise_max(dtop, as_u16(V8 ? vw.d[b][i] : vw.d[b][i] & 0x7FFF7FFFu));
            uint32_t dmax = max(dtop[0], dtop[1]);              // (scales of q8_0 are not negative, or look large)
            if (__builtin_expect(__any(dmax > ex.limit), 0)) {
                if (__builtin_expect(__any(dmax >= 0x7C00), 0)) {
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
                // A tile with such scales is left for later: here none of it is seen. (Selects: a third path to the products,
                // with zeros of its own, cost the main loop up to 27 registers, and bf16 rows in twos a quarter of their time.)
                const bool wide = dmax >= WIDE;
                left_out = wide ? min(left_out, t) : left_out;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) vw.d[b][i] = wide ? 0 : vw.d[b][i];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 8; ++i) sc[n][i] = wide ? -__builtin_inff() : sc[n][i];
                if (!wide && dmax > ex.limit) {
                    // the largest scale times 2^k in [4, 8), as far as 2^k is an f16
                    const int k = min(15, D_BITS - __builtin_amdgcn_frexp_expf((float)__builtin_bit_cast(_Float16, (uint16_t)dmax)));
                    const float fall = __builtin_amdgcn_ldexpf(1.f, k - ex.k);
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int i = 0; i < 2 * NB; ++i) r[n].o[i] *= fall;
                    ex.k = k;
                    // the largest f16 below 2^(D_BITS - k)
                    ex.limit = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)__builtin_amdgcn_ldexpf(1.f, D_BITS - 1 - k)) | 0x3FF;
                }
            }

            products_first<SHARED>(false);

            // 2. p, from a maximum that is taken anew where a score is far above it
            uint32_t ph[NQ][4], pl[NQ][4];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float top = sc[n][0], p[8];
#pragma unroll
                for (int i = 1; i < 8; ++i) top = fmaxf(top, sc[n][i]);
                raise_max(top * r[n].c, r[n]);
                weights(sc[n], r[n], p);
#pragma unroll
                for (int i = 0; i < 4; ++i) in_terms<F32>(p[2 * i], p[2 * i + 1], ph[n][i], pl[n][i]);
            }

            const _Float16 two_k = (_Float16)__builtin_amdgcn_ldexpf(1.f, ex.k);

            // 3. the products of values
            products_first<SHARED>(true);
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
                product(b, pt);
            }
            products_first<SHARED>(false);
            load_v(rec, more, lane);
        }

        // The tiles left out, found by their scales again. Scales that are not finite have made their sums NaN above.
#pragma unroll 1
        for (t = left_out; __builtin_expect(t < t1, 0); t += WAVES) {
            const uint32_t page = (uint32_t)table[t >> shift];
            if (page >= (uint32_t)a.c.pages) continue;
            const int lane = thread_here() & 63;
            load_v(record(t, page), true, lane);
            float sc[NQ][8] = {}, up[8];
            hide(t, len, lane >> 4, sc);                                   // (for the scales)
            uint32_t dmax = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t token = 0;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t d = (vw.d[b][i >> 1] >> (16 * (i & 1))) & 0x7FFF;
                    if (d < 0x7C00) token = max(token, d);
                    else vw.d[b][i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                }
                dmax = max(dmax, token);
                up[i] = (float)max(__builtin_amdgcn_frexp_expf((float)__builtin_bit_cast(_Float16, (uint16_t)token)) + ex.k - D_BITS, 0);
            }
            if (!__any(dmax >= WIDE)) continue;
            load_k(record(t, page), true, lane);
            scores(lane, sc);
            hide(t, len, lane >> 4, sc);
            float p[NQ][8];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float top = fmaf(sc[n][0], r[n].c, up[0]);
#pragma unroll
                for (int i = 1; i < 8; ++i) top = fmaxf(top, fmaf(sc[n][i], r[n].c, up[i]));
                raise_max(top, r[n]);
                weights(sc[n], r[n], p[n]);
            }
            const float two_k = __builtin_amdgcn_ldexpf(1.f, ex.k);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                h8 pt[NQ][TERMS];
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const h2 d = as_h2(vw.d[b][i]);
                        in_terms<F32>(rounded(p[n][2 * i] * ((float)d[0] * two_k)), rounded(p[n][2 * i + 1] * ((float)d[1] * two_k)),
                                      hi[i], lo[i]);
                    }
                    pt[n][0] = __builtin_bit_cast(h8, u32x4{hi[0], hi[1], hi[2], hi[3]});
                    if constexpr (F32) pt[n][1] = __builtin_bit_cast(h8, u32x4{lo[0], lo[1], lo[2], lo[3]});
                }
                product(b, pt);
            }
        }

        // the waves' sums
        const bool split = s.part >= 0;
        const int64_t part = (int64_t)s.part * (NQ * 16);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            if (n * 16 >= nrows) break;
            __syncthreads();
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
                    store4<F32>(a, s.f.first + row / a.G, h * a.G + row % a.G, D, d, y * (sum == 0.f ? 0.f : 1.f / sum));
                }
            }
        }
    });
}

// Joins the parts of cut items. Workgroup (x, w): rows of the item that is cut where workgroup w's range ends,
// if that is its first cut. A row's D/4 threads have four values each, and there are WAYS such groups of
// threads. EACH: each has a row of its own, WAYS x on. Else the workgroup has row x, the groups take its
// parts in turn and are joined in LDS.
constexpr int ways_of(int NB) { return THREADS / (NB * 8); }
template <bool F32, int NB, bool EACH> __global__ __launch_bounds__(THREADS) void cache_join_kernel(AttnArgs a, int rq) {
    constexpr int D = NB * 32, PLACES = D / 4, WAYS = ways_of(NB), STEP = EACH ? 1 : WAYS, AT_ONCE = EACH ? 4 : 8;
    const int place = (int)threadIdx.x % PLACES, way = (int)threadIdx.x / PLACES, w = blockIdx.y;
    const Cut cut = a.cuts[w];
    if (cut.step == 0 || w * cut.step > cut.start) return;
    const int r = EACH ? blockIdx.x * WAYS + way : blockIdx.x, row = cut.qg * rq + r;
    const bool live = way < WAYS && r < rq && row < cut.rows;
    // parts: the first is w's, its first segment or its last; then the first segments of the workgroups up to the item's end
    const int head = w * cut.step == cut.start ? 2 * w : 2 * w + 1;
    const int chunks = (int)min((cut.end - 1) / cut.step + 1, (int64_t)gridDim.y) - w;
    const auto part_at = [&](int c) { return (int64_t)(c == 0 ? head : 2 * (w + c)) * rq + r; };
    float m = -__builtin_inff(), l = 0.f;
    f32x4 y = 0.f;
    for (int c0 = EACH ? 0 : way; live && c0 < chunks; c0 += STEP * AT_ONCE) {
        float pm[AT_ONCE], pl[AT_ONCE];
        f32x4 py[AT_ONCE];
        float top = m;
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int64_t p = part_at(min(c0 + i * STEP, chunks - 1));
            pm[i] = a.part_m[p];
            pl[i] = a.part_l[p];
            py[i] = *reinterpret_cast<const f32x4*>(a.part_o + p * D + place * 4);
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
            if (c0 + i * STEP < chunks) top = fmaxf(top, pm[i]);
        const float base = top == -__builtin_inff() ? 0.f : top;
        const float fall = __builtin_amdgcn_exp2f(m - base);
        m = top;
        l *= fall;
        y *= fall;
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            if (c0 + i * STEP >= chunks) break;
            const float f = __builtin_amdgcn_exp2f(pm[i] - base);
            l = fmaf(pl[i], f, l);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = fmaf(py[i][j], f, y[j]);
        }
    }
    if constexpr (!EACH) {
        __shared__ __attribute__((aligned(16))) f32x4 sh_y[WAYS][PLACES];
        __shared__ float sh_m[WAYS], sh_l[WAYS];
        if (live) sh_y[way][place] = y;
        if (live && place == 0) {
            sh_m[way] = m;
            sh_l[way] = l;
        }
        __syncthreads();
        if (!live || way) return;
        float top = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < WAYS; ++w) top = fmaxf(top, sh_m[w]);
        const float base = top == -__builtin_inff() ? 0.f : top;
        l = 0.f;
        y = 0.f;
#pragma unroll
        for (int w = 0; w < WAYS; ++w) {
            const float f = __builtin_amdgcn_exp2f(sh_m[w] - base);
            l = fmaf(sh_l[w], f, l);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = fmaf(sh_y[w][place][j], f, y[j]);
        }
    }
    if (!live) return;
    store4<F32>(a, cut.first + row / a.G, cut.h * a.G + row % a.G, D, place * 4, y * (l == 0.f ? 0.f : 1.f / l));
}

// What the host knows: the kernel, its rows, and workgroups at most.
struct Plan {
    int64_t NQ, RQ, blocks;
    int64_t spare;
    bool even, cut, each;
};
Plan plan_of(const CacheShape& c, const AttnShape& a) {
    Plan p;
    const int64_t rows = a.max_q * (a.Hq / c.heads);
    // A second group of 16 rows shares the first's work on a tile, which no more than 16 rows do not need. Above 128
    // values it has no registers: 192 values, 4 trees of 60 tokens, bf16, 96 us with two groups and 58 with one;
    // 256 values 79 and 81, 4 chains of 8 tokens 64 and 53 (in f32 the two groups gain a tenth to a fifth there).
    // Four groups leave a SIMD one wave: 8 trees of 48 to 64 tokens 127 us, with two 79.5; 512 tokens 138 and 116.
    p.NQ = rows <= 16 || c.D > 128 ? 1 : 2;
    p.RQ = p.NQ * 16;
    const int64_t most = std::max<int64_t>(1, a.width * c.tiles);      // tiles of a sequence
    const int64_t items = a.B * ceil_div(rows, p.RQ) * c.heads;
    const int64_t card = 256 * waves_of((int)c.D / 32);                 // workgroups that run at once
    p.cut = most > WHOLE;
    // Equal parts of items (even) suit few, up to 64 (32 for heads of 256): 64 of one token, 8000 long, 35 us against 37 cut
    // by tiles, 500 to 8000 long 21 against 25; 32 of 256 values 38 against 41. 128, 8000 long, 63 against 59, and 64 of 256
    // values 66 against 62.5. A call of few short items has one part for each only this way.
    p.even = !p.cut || items <= card / 8;
    p.spare = p.cut && p.even ? card - items : 0;
    // Many items have few parts each: 8 trees of 48 to 64 tokens, both launches, 85.5 us with a row a workgroup and
    // 79.5 with WAYS. Few have many: one token of 131072 54.9, and 72.6 with WAYS.
    p.each = !p.even;
    const int64_t least = step_min((int)p.RQ);
    const int64_t parts = items * (p.cut ? ceil_div(std::min(most + begin_cost((int)p.RQ), card * least), least) : 1);
    p.blocks = std::min(p.cut ? card : 2 * card, round_up(parts, 8));
    return p;
}

struct Workspace {
    int64_t cuts, m, l, o, bytes;
};
Workspace workspace_of(const CacheShape& c, const Plan& p) {
    Workspace w = {};
    if (!p.cut) return w;
    const int64_t rows = 2 * p.blocks * p.RQ;
    w.cuts = 0;
    w.m = round_up(p.blocks * (int64_t)sizeof(Cut), REGION_ALIGN);
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

// an item's number stays an int32
bool cache_attn_grid_ok(const CacheShape& c, const AttnShape& a) {
    return ceil_div(a.max_q * (a.Hq / c.heads), 16) * c.heads < (int64_t(1) << 20);
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
    a.cap = (int)std::min<int64_t>(s.width * c.tiles * CACHE_TILE, (int64_t(1) << 31) - CACHE_TILE);
    a.even = p.even;
    a.spare = (int)p.spare;
    if (p.cut) {
        a.cuts = reinterpret_cast<Cut*>(base + w.cuts);
        a.part_m = reinterpret_cast<float*>(base + w.m);
        a.part_l = reinterpret_cast<float*>(base + w.l);
        a.part_o = reinterpret_cast<float*>(base + w.o);
    }
    const dim3 grid((unsigned)p.blocks);
    by_shape(o, tk, tv, c.D, [&](auto f32, auto k8, auto v8, auto nb) {
        constexpr bool F = decltype(f32)::value, K = decltype(k8)::value, V = decltype(v8)::value;
        constexpr int NB = decltype(nb)::value;
        const dim3 threads(THREADS);
        if constexpr (NB <= 4) {
            if (p.NQ == 2) hipLaunchKernelGGL((cache_attn_kernel<F, K, V, NB, 2>), grid, threads, 0, stream, a);
        }
        if (p.NQ == 1) hipLaunchKernelGGL((cache_attn_kernel<F, K, V, NB, 1>), grid, threads, 0, stream, a);
        const int64_t rows = std::min<int64_t>(p.RQ, s.max_q * a.G);
        if (p.cut && p.each)
            hipLaunchKernelGGL((cache_join_kernel<F, NB, true>), dim3((unsigned)ceil_div(rows, ways_of(NB)), (unsigned)p.blocks),
                               threads, 0, stream, a, (int)p.RQ);
        else if (p.cut)
            hipLaunchKernelGGL((cache_join_kernel<F, NB, false>), dim3((unsigned)rows, (unsigned)p.blocks), threads, 0, stream, a,
                               (int)p.RQ);
    });
    return hipGetLastError();
}

}  // namespace mmq
