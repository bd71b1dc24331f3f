// lora.hip - low-rank adapters of many requests beside a shared projection:
//     v[m] = A_e x^[m],   out[m] = base[m] + s_e B_e v[m],   e the row's adapter (or none)
// on the act buffer that the projection reads and the output that it wrote.
//
// Two launches over the plan's units (up to 64 rows of one adapter):
//   1. lora_down_kernel: v, split over K into S parts so that few rows still fill the chip; a
//      workgroup's four waves take every fourth block of its part and join in LDS. The int8
//      values enter the matrix core as they are (exact in bf16 and f16), each block's product
//      is scaled by its f32 scale; the per-token form accumulates on the matrix core.
//   2. lora_up_kernel: (unit, 256 columns): sums the S parts of v in order, and adds
//      s_e B_e v to the base.
#include <algorithm>

#include "lora.h"

namespace mmq {
namespace {

template <int RT, bool F16, bool Q81>
__global__ __launch_bounds__(LT) void lora_down_kernel(LoraArgs a) {
    __shared__ f32x4 red[4][4 * RT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int u = (int)blockIdx.x / a.S, s = (int)blockIdx.x % a.S;
    const int4 unit = a.units[u];
    if (unit.z == 0 || unit.x >= a.E) return;
    const int r0 = (int)blockIdx.y * LORA_RC;
    const int nt = (unit.z + 15) >> 4;

    const int8_t* xrow[4];
    const uint32_t* srow[4];
    int row[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        // rows past the unit's last repeat it; their columns are not stored
        const int m = a.order[unit.y + min(16 * t + c, unit.z - 1)];
        row[t] = m;
        xrow[t] = a.xq + (int64_t)(m >> 5) * a.KBp * 1024 + ((g >> 1) * 32 + (m & 31)) * 16 + (g & 1) * 8;
        if constexpr (Q81) srow[t] = a.xs2 + (int64_t)(m >> 5) * a.KBp * 32 + (m & 31);
    }
    const uint16_t* arow[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)        // ranks past R repeat the last one; not stored either
        arow[i] = a.A + ((int64_t)unit.x * a.R + min(r0 + 16 * i + c, a.R - 1)) * a.K + 8 * g;

    f32x4 acc[4][RT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[t][i] = 0;

    const int per = (a.KB + a.S - 1) / a.S;
    const int b1 = min((s + 1) * per, a.KB);
    for (int b = s * per + wave; b < b1; b += 4) {
        u32x4 w[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) w[i] = *reinterpret_cast<const u32x4*>(arow[i] + (int64_t)b * 32);
        u32x2 q[4];
        float xs[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (t < nt) {
                q[t] = *reinterpret_cast<const u32x2*>(xrow[t] + (int64_t)b * 1024);
                if constexpr (Q81) xs[t] = (float)__builtin_bit_cast(_Float16, (uint16_t)srow[t][(int64_t)b * 32]);
            }
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (t < nt) {
                const u32x4 x = int8_operand<F16>(q[t]);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const f32x4 from = Q81 ? f32x4(0) : acc[t][i];
                    const f32x4 d = F16 ? mfma_f16(w[i], x, from) : mfma_bf16(w[i], x, from);
                    if constexpr (Q81) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[t][i][j] = fmaf(xs[t], d[j], acc[t][i][j]);
                    } else {
                        acc[t][i] = d;
                    }
                }
            }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
        if (t < nt)
#pragma unroll
            for (int i = 0; i < RT; ++i) red[wave][t * RT + i][lane] = acc[t][i];
    __syncthreads();
    // wave w joins the tiles w, w + 4, ... (RT of them at most)
#pragma unroll
    for (int k = 0; k < RT; ++k) {
        const int tile = wave + 4 * k, t = tile / RT, i = tile % RT;
        if (t >= nt) continue;
        f32x4 d = red[0][tile][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) d += red[w][tile][lane];
        const int at = 16 * t + c, r = r0 + 16 * i + 4 * g;
        if (at >= unit.z || r >= a.R) continue;
        if constexpr (!Q81) d *= a.sa[a.order[unit.y + at]];
        *reinterpret_cast<f32x4*>(a.part + ((int64_t)s * a.M + unit.y + at) * a.R + r) = d;
    }
}

template <bool F16, bool BF16>
__global__ __launch_bounds__(LT) void lora_up_kernel(LoraArgs a, int ntiles) {
    constexpr int LD = LORA_RC + 8;                         // a row's stride in LDS: rows on other banks
    __shared__ __attribute__((aligned(16))) uint16_t vt[3][GROUP_UNIT][LD];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int u = (int)blockIdx.x / ntiles, tile = (int)blockIdx.x % ntiles;
    const int4 unit = a.units[u];
    if (unit.z == 0) return;
    const int nt = (unit.z + 15) >> 4;
    const bool none = unit.x >= a.E;
    const int n0 = tile * UP_COLS + wave * 64;

    int64_t row[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) row[t] = a.order[unit.y + min(16 * t + c, unit.z - 1)];
    f32x4 base[4][4], acc[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[t][i] = 0;
            base[t][i] = 0;
            const int n = n0 + 16 * i + 4 * g;
            if (a.base && t < nt && n < a.N) base[t][i] = load4<BF16>(a.base, row[t] * a.ldb + n, a.N - n);
        }

    for (int r0 = 0; r0 < a.R; r0 += LORA_RC) {
        // the rows' v of these ranks: the parts in order, three bf16 terms each; zeros past the
        // unit's rows and past R
        if (r0) __syncthreads();
        for (int idx = threadIdx.x; idx < nt * 16 * (LORA_RC / 4); idx += LT) {
            const int at = idx / (LORA_RC / 4), r = 4 * (idx % (LORA_RC / 4));
            f32x4 d = 0;
            if (at < unit.z && r0 + r < a.R) {
                if (!none) {
                    const float* p = a.part + ((int64_t)unit.y + at) * a.R + r0 + r;
                    for (int s = 0; s < a.S; ++s) d += *reinterpret_cast<const f32x4*>(p + (int64_t)s * a.M * a.R);
                }
                if (tile == 0) *reinterpret_cast<f32x4*>(a.v + (int64_t)a.order[unit.y + at] * a.R + r0 + r) = d;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                u32x2 w;
                w[0] = pack_hi(d[0], d[1]);
                w[1] = pack_hi(d[2], d[3]);
                *reinterpret_cast<u32x2*>(&vt[k][at][r]) = w;
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] -= cut(d[j]);
            }
        }
        __syncthreads();
        if (none) continue;
#pragma unroll
        for (int kk = 0; kk < LORA_RC; kk += 32) {
            if (r0 + kk >= a.R) break;
            Weights<F16> w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = min(n0 + 16 * i + c, a.N - 1), r = r0 + kk + 8 * g;
                u32x4 raw = 0;
                if (r < a.R) raw = *reinterpret_cast<const u32x4*>(a.B + ((int64_t)unit.x * a.N + n) * a.R + r);
                w[i].set(raw);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t < nt) {
                    u32x4 x[3];
#pragma unroll
                    for (int k = 0; k < 3; ++k) x[k] = *reinterpret_cast<const u32x4*>(&vt[k][16 * t + c][kk + 8 * g]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][i] = mfma_terms(w[i], x, acc[t][i]);
                }
        }
    }

    const float scale = none ? 0.f : a.scale[unit.x];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (t >= nt || 16 * t + c >= unit.z) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 16 * i + 4 * g;
            if (n >= a.N) continue;
            f32x4 o = base[t][i];
            if (!none)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = fmaf(scale, acc[t][i][j], o[j]);
            store4<BF16>(a.out, row[t] * a.ldo + n, o, a.N - n);
        }
    }
}

// parts that K is split into: about 512 workgroups, four blocks (one a wave) at least
int64_t down_parts(int64_t E, int64_t M, int64_t K) {
    const int64_t units = plan_layout(E, M).nunits;
    return std::max<int64_t>(1, std::min<int64_t>(512 / units, ceil_div(K / QK, 4)));
}

template <bool F16, bool Q81>
void launch_down(const LoraArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.nunits * a.S), (unsigned)ceil_div(a.R, LORA_RC));
    if (a.R <= 16) hipLaunchKernelGGL((lora_down_kernel<1, F16, Q81>), grid, dim3(LT), 0, s, a);
    else if (a.R <= 32) hipLaunchKernelGGL((lora_down_kernel<2, F16, Q81>), grid, dim3(LT), 0, s, a);
    else hipLaunchKernelGGL((lora_down_kernel<4, F16, Q81>), grid, dim3(LT), 0, s, a);
}

}  // namespace

size_t lora_workspace_bytes(int64_t E, int64_t M, int64_t K, int64_t R) {
    return (size_t)round_up(down_parts(E, M, K) * M * R * 4, REGION_ALIGN);
}

// both launches' grids stay below 2^32 threads
bool lora_grid_ok(int64_t E, int64_t M, int64_t N, int64_t K) {
    const int64_t units = plan_layout(E, M).nunits;
    return units * std::max(ceil_div(N, UP_COLS), ceil_div(K, UP_COLS)) < (int64_t(1) << 32) / LT;
}

hipError_t launch_lora(mmq_atype t, bool f16, const void* act, const void* A, const void* B, const float* scale,
                       int64_t E, int64_t R, const void* plan, int64_t M, int64_t N, int64_t K, const void* base,
                       int64_t ldb, void* out, int64_t ldo, float* v, void* ws, hipStream_t s) {
    LoraArgs a = lora_args(t, act, A, B, scale, E, R, plan, M, N, K);
    a.part = static_cast<float*>(ws);
    a.S = (int)down_parts(E, M, K);
    a.base = base;
    a.ldb = ldb;
    a.out = out;
    a.ldo = ldo;
    a.v = v;
    const bool q81 = t == MMQ_ACT_Q8_1;
    if (f16) q81 ? launch_down<true, true>(a, s) : launch_down<true, false>(a, s);
    else q81 ? launch_down<false, true>(a, s) : launch_down<false, false>(a, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int ntiles = (int)ceil_div(N, UP_COLS);
    const dim3 grid((unsigned)a.nunits * (unsigned)ntiles);
    if (f16) {
        if (q81) hipLaunchKernelGGL((lora_up_kernel<true, false>), grid, dim3(LT), 0, s, a, ntiles);
        else hipLaunchKernelGGL((lora_up_kernel<true, true>), grid, dim3(LT), 0, s, a, ntiles);
    } else {
        if (q81) hipLaunchKernelGGL((lora_up_kernel<false, false>), grid, dim3(LT), 0, s, a, ntiles);
        else hipLaunchKernelGGL((lora_up_kernel<false, true>), grid, dim3(LT), 0, s, a, ntiles);
    }
    return hipGetLastError();
}

}  // namespace mmq
