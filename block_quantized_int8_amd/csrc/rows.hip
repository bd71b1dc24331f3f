// rows.hip - rows grouped by the adapter or expert they use, and the expert rows' way there and
// back: the plan (a stable counting sort on the device), the gather of token rows into expert
// order, their weighted sum back into tokens and its gradients.
//
// The plan replaces nothing inside mmq_gemm_id (whose route kernel sorts for itself, in any
// order inside an expert); it is for calls that share one grouping: the adapters' products of
// every projection of a step, and rows that leave in expert order. Its order is stable (rising
// pair ids inside a group), so sums over a group's rows have one order and repeat bit for bit.
#include <algorithm>

#include "mmq_internal.h"
#include "rows.h"

namespace mmq {
namespace {

// Sizes of the sort. Up to GROUP_ONE pairs one launch sorts: up to GROUP_WGS workgroups, each of
// which counts all pairs (64 KB of ids at most, from L2) and places a segment. Past that a launch of
// up to GROUP_MAX workgroups counts their segments first. There are two instances: 16 waves for up to
// SMALL_KEYS groups (E + 1, the last being "no group"), whose LDS has room for a counter for each wave
// and key, else 4 waves. Segments of a counted sort, measured with 2048, 4096, 8192 and 16384 pairs
// (us): 32768 pairs of 64 groups 8.4, 9.7, 12.7, 20.0; 800000 of 64 17.5, 16.7, 17.3, 23.3; 240000
// of 4096 428, 232, 145, 124 (each workgroup reads all segments' counts of all keys).
constexpr int64_t GROUP_ONE = 16384;
constexpr int64_t GROUP_WGS = 16;
constexpr int64_t GROUP_MAX = 256;
constexpr int SMALL_KEYS = 1024, MAX_KEYS = 4097;

bool group_counts_first(int64_t P) { return P > GROUP_ONE; }
int64_t group_blocks(int64_t E, int64_t P) {
    const bool small = E + 1 <= SMALL_KEYS;
    return group_counts_first(P) ? std::min<int64_t>(GROUP_MAX, ceil_div(P, small ? 2048 : 16384))
                                 : std::min<int64_t>(GROUP_WGS, ceil_div(P, small ? 1024 : 256));
}

struct GroupArgs {
    const int32_t* ids;
    int P, E, seg;              // seg: pairs per workgroup
    int32_t *offs, *order, *pos, *scratch;
    int4* units;
    int nunits;
};

__device__ inline int key_of(const GroupArgs& a, int e) { return (e >= 0 && e < a.E) ? e : a.E; }

// The ids of up to KEYS_AT_ONCE steps of 64 pairs, loaded together (a step at a time the sort of
// 16384 pairs by one workgroup waited for 32 loads one after another: 21 us against 17.6).
constexpr int KEYS_AT_ONCE = 8;
__device__ inline void load_ids(const GroupArgs& a, int64_t p, int64_t end, int* id) {
#pragma unroll
    for (int i = 0; i < KEYS_AT_ONCE; ++i) {
        const int64_t at = p + 64 * i;
        id[i] = at < end ? a.ids[at] : 0;
    }
}

// Lanes that add to one LDS address wait for each other, so a key has several counters. (16384 pairs
// of 64 groups, a quarter of them without one: 9.1 us with one counter, 7.9 with two, 7.2 with
// four or eight; all of one group: 18.6, 12.0, 9.0, 7.4.)
template <int KEYS> constexpr int COPIES = KEYS <= SMALL_KEYS ? 8 : 1;

// counts of each workgroup's segment: scratch[block][E + 1]
template <int GW, int KEYS>
__global__ __launch_bounds__(GW * 64) void group_count_kernel(GroupArgs a) {
    constexpr int C = COPIES<KEYS>;
    __shared__ int cnt[KEYS][C];
    const int keys = a.E + 1;
    for (int i = threadIdx.x; i < C * keys; i += GW * 64) cnt[0][i] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * a.seg;
    const int p1 = (int)min(p0 + a.seg, (int64_t)a.P);
    for (int64_t p = p0 + threadIdx.x; p < p1; p += GW * 64) atomicAdd(&cnt[key_of(a, a.ids[p])][threadIdx.x % C], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < keys; e += GW * 64) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) n += cnt[e][i];
        a.scratch[(int64_t)blockIdx.x * keys + e] = n;
    }
}

// Inclusive scan of (x, y) over the workgroup's threads.
template <int GW>
__device__ inline int2 block_scan(int2 v, int2* wtot) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int ox = __shfl_up(v.x, d, 64), oy = __shfl_up(v.y, d, 64);
        if (lane >= d) {
            v.x += ox;
            v.y += oy;
        }
    }
    if (lane == 63) wtot[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        v.x += wtot[w].x;
        v.y += wtot[w].y;
    }
    return v;
}

// The stable sort. Every workgroup knows all counts (its own, or the count kernel's where that ran:
// `counted`); wave w of a workgroup places segment w in pair order: 64 pairs
// at a time find the lanes of their own key by one ballot per key bit, so a pair's position is
// the wave's running start of its key plus the lanes before it. Bound by latency: 80 pairs 4.7 us,
// 16384 pairs of 64 groups 7.2 us.
template <int GW, int KEYS>
__global__ __launch_bounds__(GW * 64) void group_kernel(GroupArgs a, int bits, int counted) {
    __shared__ int cur[GW][KEYS];
    constexpr int C = COPIES<KEYS>;
    __shared__ int before[KEYS][C], after[KEYS][C];        // the earlier and later workgroups' pairs
    __shared__ int offs[KEYS + 1], uoff[KEYS + 1];
    __shared__ int2 wtot[GW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int keys = a.E + 1, nblk = (int)gridDim.x, blk = (int)blockIdx.x;
    for (int i = lane; i < keys; i += 64) cur[wave][i] = 0;
    for (int i = tid; i < C * keys; i += GW * 64) before[0][i] = after[0][i] = 0;
    const int64_t b0 = min((int64_t)blk * a.seg, (int64_t)a.P);
    const int64_t b1 = min(b0 + a.seg, (int64_t)a.P);
    const int wseg = (int)(((b1 - b0 + GW - 1) / GW + 63) & ~(int64_t)63);   // pairs per wave
    const int64_t s0 = min(b0 + (int64_t)wave * wseg, b1), s1 = min(s0 + wseg, b1);
    __syncthreads();
    if (!counted && nblk > 1)
        for (int64_t p = (int64_t)wave * 64 * KEYS_AT_ONCE + lane; p - lane < a.P; p += (int64_t)GW * 64 * KEYS_AT_ONCE) {
            int id[KEYS_AT_ONCE];
            load_ids(a, p, a.P, id);
#pragma unroll
            for (int i = 0; i < KEYS_AT_ONCE; ++i) {
                const int64_t at = p + 64 * i;
                if (at < b0) atomicAdd(&before[key_of(a, id[i])][lane % C], 1);
                else if (at >= b1 && at < a.P) atomicAdd(&after[key_of(a, id[i])][lane % C], 1);
            }
        }
    for (int64_t p = s0 + lane; p - lane < s1; p += 64 * KEYS_AT_ONCE) {
        int id[KEYS_AT_ONCE];
        load_ids(a, p, s1, id);
#pragma unroll
        for (int i = 0; i < KEYS_AT_ONCE; ++i)
            if (p + 64 * i < s1) atomicAdd(&cur[wave][key_of(a, id[i])], 1);
    }
    if (counted && KEYS <= SMALL_KEYS) {                     // few keys: a count a thread
        const uint32_t n = (uint32_t)nblk * keys;
#pragma unroll 8
        for (uint32_t x = tid; x < n; x += GW * 64) {
            const int b = (int)(x / (uint32_t)keys), e = (int)x - b * keys, c = a.scratch[x];
            if (b != blk) atomicAdd(b < blk ? &before[e][lane % C] : &after[e][lane % C], c);
        }
    } else if (counted) {                                  // a key a thread
        for (int e = tid; e < keys; e += GW * 64) {
            int x = 0, y = 0;
            for (int b = 0; b < blk; ++b) x += a.scratch[(int64_t)b * keys + e];
            for (int b = blk + 1; b < nblk; ++b) y += a.scratch[(int64_t)b * keys + e];
            before[e][0] = x;
            after[e][0] = y;
        }
    }
    __syncthreads();

    // thread t owns keys [t*KPT, t*KPT + KPT): all pairs of a key, then the waves' starts
    const int KPT = (keys + GW * 64 - 1) / (GW * 64);
    const int e0 = min(tid * KPT, keys), e1 = min(e0 + KPT, keys);
    int2 sum = make_int2(0, 0);
    for (int e = e0; e < e1; ++e) {
        int all = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) all += before[e][i] + after[e][i];
#pragma unroll
        for (int w = 0; w < GW; ++w) all += cur[w][e];
        offs[e] = all;
        sum.x += all;
        sum.y += (all + GROUP_UNIT - 1) / GROUP_UNIT;
    }
    const int2 inc = block_scan<GW>(sum, wtot);
    int px = inc.x - sum.x, py = inc.y - sum.y;
    for (int e = e0; e < e1; ++e) {
        const int all = offs[e];
        int c[GW], run = px;
#pragma unroll
        for (int i = 0; i < C; ++i) run += before[e][i];
#pragma unroll
        for (int w = 0; w < GW; ++w) c[w] = cur[w][e];
#pragma unroll
        for (int w = 0; w < GW; ++w) {
            cur[w][e] = run;
            run += c[w];
        }
        offs[e] = px;
        uoff[e] = py;
        if (blk == 0) a.offs[e] = px;
        px += all;
        py += (all + GROUP_UNIT - 1) / GROUP_UNIT;
    }
    if (tid == GW * 64 - 1) {
        offs[keys] = px;
        uoff[keys] = py;
    }
    __syncthreads();

    for (int u = blk * GW * 64 + tid; u < a.nunits; u += nblk * GW * 64) {
        int4 v = make_int4(0, 0, 0, 0);
        if (u < uoff[keys]) {
            int lo = 0, hi = keys;                           // the last key with uoff <= u
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (uoff[mid] <= u) lo = mid; else hi = mid;
            }
            v.x = lo;
            v.y = offs[lo] + (u - uoff[lo]) * GROUP_UNIT;
            v.z = min(GROUP_UNIT, offs[lo + 1] - v.y);
        }
        a.units[u] = v;
    }

    for (int64_t q = s0 + lane; q - lane < s1; q += 64 * KEYS_AT_ONCE) {
        int id[KEYS_AT_ONCE];
        load_ids(a, q, s1, id);
#pragma unroll
        for (int i = 0; i < KEYS_AT_ONCE; ++i) {
            const int64_t p = q + 64 * i;
            if (p - lane >= s1) break;
            const bool live = p < s1;
            const int key = live ? key_of(a, id[i]) : 0;
            uint64_t same = __ballot(live);
            for (int b = 0; b < bits; ++b) {
                const uint64_t m = __ballot((key >> b) & 1);
                same &= ((key >> b) & 1) ? m : ~m;
            }
            const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
            if (live) {
                const int at = cur[wave][key] + before;
                a.order[at] = (int)p;
                a.pos[p] = key < a.E ? at : -1;
                // the key's first lane moves its start past the wave's pairs, after every lane's read
                if (before == 0) cur[wave][key] = at + __popcll(same);
            }
        }
    }
}

// ------------------------------------------------------------------ token rows
// Rows move in 16-byte pieces, also where a row's size or stride leaves them unaligned (global
// accesses need no alignment; the piece's type says that it has only its values'); a row's last
// piece, if it is shorter, goes value by value.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <typename T> struct Piece {
    static constexpr int V = 16 / (int)sizeof(T);
    u32x4 r;
    __device__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, (uint32_t)r[i]);
        else return __builtin_bit_cast(float, i & 1 ? r[i / 2] & 0xFFFF0000u : r[i / 2] << 16);
    }
    // from V values: f32 as they are, bf16 rounded to nearest even
    __device__ void set(const float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) r[i] = __builtin_bit_cast(uint32_t, v[i]);
            else r[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
        }
    }
    __device__ T bits(int i) const {
        if constexpr (sizeof(T) == 4) return (T)r[i];
        else return (T)(r[i / 2] >> (16 * (i & 1)));
    }
};

// T: uint32_t (f32) or uint16_t (bf16); n: the row's values from p on
template <typename T>
__device__ inline Piece<T> load_piece(const void* row, int64_t at, int n) {
    const T* p = static_cast<const T*>(row) + at;
    Piece<T> q;
    if (n >= Piece<T>::V) {
        q.r = *reinterpret_cast<const u32x4_any*>(p);
        return q;
    }
    q.r = 0;
#pragma unroll
    for (int i = 0; i < Piece<T>::V; ++i)
        if (i < n) {
            if constexpr (sizeof(T) == 4) q.r[i] = p[i];
            else q.r[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
        }
    return q;
}

template <typename T>
__device__ inline void store_piece(void* row, int64_t at, const Piece<T>& q, int n) {
    T* p = static_cast<T*>(row) + at;
    if (n >= Piece<T>::V) {
        *reinterpret_cast<u32x4_any*>(p) = q.r;
        return;
    }
#pragma unroll
    for (int i = 0; i < Piece<T>::V; ++i)
        if (i < n) p[i] = q.bits(i);
}

struct RowArgs {
    const void *x, *z, *dy;
    void *y, *dz;
    const float* w;
    float* dw;
    const int32_t* pos;
    int64_t ldx, ldz, ldy, lddz;
    int T, top_k, N;
    int sorted;                 // z / dz rows: 1 by sorted position, 0 by pair
};

constexpr int ROW_THREADS = 256;

// the pair's sorted position, -1 if it has none (or one outside the rows: a plan of another batch)
__device__ inline int pos_of(const RowArgs& a, int p) {
    const int r = a.pos[p];
    return (uint32_t)r < (uint32_t)(a.T * a.top_k) ? r : -1;
}
// the row of z that holds pair p, -1 if it has none
__device__ inline int pair_row(const RowArgs& a, int p) {
    const int r = pos_of(a, p);
    return r < 0 ? -1 : a.sorted ? r : p;
}

// A token's row is read once and written to each of its pairs' places. Bound by memory: 2048 tokens x 8
// of 4096 bf16 values, a quarter of the pairs without an expert, 118 MB in 23.1 us (5.1 TB/s; a
// large copy reaches 5.2).
template <typename T>
__global__ __launch_bounds__(ROW_THREADS) void gather_kernel(RowArgs a) {
    const int n = ((int)blockIdx.x * ROW_THREADS + (int)threadIdx.x) * Piece<T>::V;
    if (n >= a.N) return;
    for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
        const Piece<T> v = load_piece<T>(a.x, (int64_t)t * a.ldx + n, a.N - n);
        for (int j = 0; j < a.top_k; ++j) {
            const int r = pos_of(a, t * a.top_k + j);
            if (r >= 0) store_piece<T>(a.y, (int64_t)r * a.ldy + n, v, a.N - n);
        }
    }
}

// y[t] = sum over j of w[t][j] z[row(t, j)]: f32 sums in rising j, one rounding at the end. Eight rows'
// loads are in flight before the first is used. 512 tokens x 8 of 2048 f32 values: 38 MB in 8.3 us
// (4.6 TB/s).
template <typename T>
__global__ __launch_bounds__(ROW_THREADS) void combine_kernel(RowArgs a) {
    constexpr int V = Piece<T>::V, J = 8;      // J rows in flight
    const int n = ((int)blockIdx.x * ROW_THREADS + (int)threadIdx.x) * V;
    if (n >= a.N) return;
    for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = 0.f;
        for (int j0 = 0; j0 < a.top_k; j0 += J) {
            Piece<T> z[J];
            float w[J];
            bool has[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int p = t * a.top_k + j0 + j;
                const int r = j0 + j < a.top_k ? pair_row(a, p) : -1;
                has[j] = r >= 0;
                if (has[j]) {
                    w[j] = a.w ? a.w[p] : 1.f;
                    z[j] = load_piece<T>(a.z, (int64_t)r * a.ldz + n, a.N - n);
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (has[j]) {
#pragma unroll
                    for (int i = 0; i < V; ++i) s[i] = fmaf(w[j], z[j].get(i), s[i]);
                }
        }
        Piece<T> o;
        o.set(s);
        store_piece<T>(a.y, (int64_t)t * a.ldy + n, o, a.N - n);
    }
}

// dz[row] = w dy[t] and dw = <dy[t], z[row]> of one pair: W waves each (the dot is summed per
// lane, then over lanes and waves in a fixed order). The four pairs of a workgroup are neighbours, so
// a token's dy comes from L2 for all but the first. 512 tokens x 8 of 2048 f32 values: 71 MB in
// 13.2 us (5.4 TB/s).
template <typename T, int W>
__global__ __launch_bounds__(ROW_THREADS) void combine_grad_kernel(RowArgs a) {
    constexpr int V = Piece<T>::V, PW = ROW_THREADS / 64 / W;   // pairs per workgroup
    __shared__ float red[ROW_THREADS / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int P = a.T * a.top_k;
    for (int p0 = (int)blockIdx.x * PW; p0 < P; p0 += (int)gridDim.x * PW) {
        const int p = p0 + wave / W;
        const int r = p < P ? pair_row(a, p) : -1;
        float dot = 0.f;
        if (r >= 0) {
            const float w = a.w[p];
            const int64_t dy = (int64_t)(p / a.top_k) * a.ldy, z = (int64_t)r * a.ldz, dz = (int64_t)r * a.lddz;
            for (int n = ((wave % W) * 64 + lane) * V; n < a.N; n += W * 64 * V) {
                const Piece<T> g = load_piece<T>(a.dy, dy + n, a.N - n), v = load_piece<T>(a.z, z + n, a.N - n);
                float d[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dot = fmaf(g.get(i), v.get(i), dot);
                    d[i] = w * g.get(i);
                }
                Piece<T> o;
                o.set(d);
                store_piece<T>(a.dz, dz + n, o, a.N - n);
            }
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) dot += __shfl_xor(dot, o);
        if constexpr (W > 1) {
            if (lane == 0) red[wave] = dot;
            __syncthreads();
            dot = 0.f;
            for (int i = 0; i < W; ++i) dot += red[wave / W * W + i];
            __syncthreads();
        }
        if (p < P && wave % W == 0 && lane == 0) a.dw[p] = dot;
    }
}

constexpr int64_t GRID_MAX = int64_t(1) << 20;      // workgroups of a launch; they loop past it
constexpr int GRID_Y = 65535;                        // tokens of a launch's grid; it loops past them

}  // namespace

PlanLayout plan_layout(int64_t E, int64_t P) {
    PlanLayout L;
    L.nunits = P / GROUP_UNIT + std::min<int64_t>(E + 1, P);
    L.offs_off = 0;
    L.order_off = round_up((E + 1) * 4, REGION_ALIGN);
    L.pos_off = L.order_off + round_up(P * 4, REGION_ALIGN);
    L.units_off = L.pos_off + round_up(P * 4, REGION_ALIGN);
    L.scratch_off = L.units_off + round_up(L.nunits * 16, REGION_ALIGN);
    L.bytes = L.scratch_off + (group_counts_first(P) ? round_up(group_blocks(E, P) * (E + 1) * 4, REGION_ALIGN) : 0);
    return L;
}

template <int GW, int KEYS>
static void launch_group(GroupArgs a, int bits, hipStream_t s) {
    const int64_t blocks = group_blocks(a.E, a.P);
    const bool counted = group_counts_first(a.P);
    a.seg = (int)ceil_div(a.P, blocks);
    if (counted) hipLaunchKernelGGL((group_count_kernel<GW, KEYS>), dim3(blocks), dim3(GW * 64), 0, s, a);
    hipLaunchKernelGGL((group_kernel<GW, KEYS>), dim3(blocks), dim3(GW * 64), 0, s, a, bits, counted ? 1 : 0);
}

hipError_t launch_group_rows(const int32_t* ids, int64_t E, int64_t P, void* plan, hipStream_t s) {
    const PlanLayout L = plan_layout(E, P);
    uint8_t* base = static_cast<uint8_t*>(plan);
    GroupArgs a;
    a.ids = ids;
    a.P = (int)P;
    a.E = (int)E;
    a.offs = reinterpret_cast<int32_t*>(base + L.offs_off);
    a.order = reinterpret_cast<int32_t*>(base + L.order_off);
    a.pos = reinterpret_cast<int32_t*>(base + L.pos_off);
    a.units = reinterpret_cast<int4*>(base + L.units_off);
    a.scratch = reinterpret_cast<int32_t*>(base + L.scratch_off);
    a.nunits = (int)L.nunits;
    int bits = 1;
    while ((int64_t(1) << bits) < E + 1) ++bits;
    if (E + 1 <= SMALL_KEYS) launch_group<16, SMALL_KEYS>(a, bits, s);
    else launch_group<4, MAX_KEYS>(a, bits, s);
    return hipGetLastError();
}

namespace {
// workgroups along a row (of T's values) x tokens
template <typename T> dim3 row_grid(const RowArgs& a) {
    return dim3((unsigned)ceil_div(a.N, ROW_THREADS * Piece<T>::V), (unsigned)std::min(a.T, GRID_Y));
}
}  // namespace

hipError_t launch_moe_gather(mmq_otype o, const void* x, int64_t ldx, const void* plan, int64_t E,
                             int64_t T, int64_t top_k, int64_t N, void* rows, int64_t ldr, hipStream_t s) {
    const PlanLayout L = plan_layout(E, T * top_k);
    RowArgs a = {};
    a.x = x;
    a.ldx = ldx;
    a.y = rows;
    a.ldy = ldr;
    a.pos = reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(plan) + L.pos_off);
    a.T = (int)T;
    a.top_k = (int)top_k;
    a.N = (int)N;
    if (o == MMQ_OUT_F32)
        hipLaunchKernelGGL(gather_kernel<uint32_t>, row_grid<uint32_t>(a), dim3(ROW_THREADS), 0, s, a);
    else
        hipLaunchKernelGGL(gather_kernel<uint16_t>, row_grid<uint16_t>(a), dim3(ROW_THREADS), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_combine(mmq_otype o, const void* z, int64_t ldz, bool sorted, const float* w,
                              const void* plan, int64_t E, int64_t T, int64_t top_k, int64_t N, void* y,
                              int64_t ldy, hipStream_t s) {
    const PlanLayout L = plan_layout(E, T * top_k);
    RowArgs a = {};
    a.z = z;
    a.ldz = ldz;
    a.sorted = sorted;
    a.w = w;
    a.y = y;
    a.ldy = ldy;
    a.pos = reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(plan) + L.pos_off);
    a.T = (int)T;
    a.top_k = (int)top_k;
    a.N = (int)N;
    if (o == MMQ_OUT_F32)
        hipLaunchKernelGGL(combine_kernel<uint32_t>, row_grid<uint32_t>(a), dim3(ROW_THREADS), 0, s, a);
    else
        hipLaunchKernelGGL(combine_kernel<uint16_t>, row_grid<uint16_t>(a), dim3(ROW_THREADS), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_combine_grad(mmq_otype o, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                                   bool sorted, const float* w, const void* plan, int64_t E, int64_t T,
                                   int64_t top_k, int64_t N, void* dz, int64_t lddz, float* dw, hipStream_t s) {
    const int64_t P = T * top_k;
    const PlanLayout L = plan_layout(E, P);
    RowArgs a = {};
    a.dy = dy;
    a.ldy = lddy;
    a.z = z;
    a.ldz = ldz;
    a.sorted = sorted;
    a.w = w;
    a.dz = dz;
    a.lddz = lddz;
    a.dw = dw;
    a.pos = reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(plan) + L.pos_off);
    a.T = (int)T;
    a.top_k = (int)top_k;
    a.N = (int)N;
    constexpr int W = ROW_THREADS / 64;
    // A wave per pair, or all four of a workgroup for up to 1024 pairs. Measured, four waves against
    // one, f32: 512 pairs x 2048 4.3 against 5.8 us, 1024 x 2048 6.4 against 6.9, 1024 x 8192 17.6
    // against 29.1, 1536 x 2048 8.3 against 7.5, 4096 x 2048 17.8 against 13.2.
    const bool wide = P <= 1024;
    const dim3 grid((unsigned)std::min<int64_t>(wide ? P : ceil_div(P, W), GRID_MAX));
    if (o == MMQ_OUT_F32) {
        if (wide) hipLaunchKernelGGL((combine_grad_kernel<uint32_t, W>), grid, dim3(ROW_THREADS), 0, s, a);
        else hipLaunchKernelGGL((combine_grad_kernel<uint32_t, 1>), grid, dim3(ROW_THREADS), 0, s, a);
    } else {
        if (wide) hipLaunchKernelGGL((combine_grad_kernel<uint16_t, W>), grid, dim3(ROW_THREADS), 0, s, a);
        else hipLaunchKernelGGL((combine_grad_kernel<uint16_t, 1>), grid, dim3(ROW_THREADS), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace mmq
