// lora_grad.hip - the adapters' gradients, from the 8-bit activations kept as the checkpoint:
//     u[m] = s_e B_e^T dy[m]        dB_e = s_e sum over the rows of e of dy[m] v[m]^T
//     dx[m] = dxb[m] + A_e^T u[m]   dA_e = sum over the rows of e of u[m] x^[m]^T
// The act buffer is read as it is: its int8 values enter the matrix core exactly and each block's
// scale goes to u's side, so no activation is ever restored to f32 in memory.
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

template <bool BF16> __device__ inline float grad_at(const void* p, int64_t at) {
    if constexpr (BF16) return as_f((uint32_t)static_cast<const uint16_t*>(p)[at] << 16);
    else return static_cast<const float*>(p)[at];
}

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

// Eight 16-bit values, `step` apart, as an operand's raw bits.
__device__ inline u32x4 gather8(const uint16_t* p, int64_t step) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (uint32_t)p[2 * i * step] | ((uint32_t)p[(2 * i + 1) * step] << 16);
    return r;
}

// Partial u over the S parts of N: [s][sorted position][R].
template <int RT, bool F16, bool BF16>
__global__ __launch_bounds__(LT) void lora_u_kernel(LoraArgs a) {
    __shared__ f32x4 red[4][4 * RT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int u = (int)blockIdx.x / a.S, s = (int)blockIdx.x % a.S;
    const int4 unit = a.units[u];
    if (unit.z == 0 || unit.x >= a.E) return;
    const int r0 = (int)blockIdx.y * LORA_RC;
    const int nt = (unit.z + 15) >> 4;
    int64_t row[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) row[t] = (int64_t)a.order[unit.y + min(16 * t + c, unit.z - 1)] * a.lddy;
    f32x4 acc[4][RT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[t][i] = 0;
    const int NB = (a.N + 31) / 32, per = (NB + a.S - 1) / a.S;
    const int b1 = min((s + 1) * per, NB);
    for (int b = s * per + wave; b < b1; b += 4) {
        const int n = 32 * b + 8 * g;
        Weights<F16> w[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = min(r0 + 16 * i + c, a.R - 1);
            const uint16_t* p = a.B + ((int64_t)unit.x * a.N) * a.R + r;
            u32x4 raw;
            if (n + 8 <= a.N) raw = gather8(p + (int64_t)n * a.R, a.R);
            else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    raw[j] = (uint32_t)p[(int64_t)min(n + 2 * j, a.N - 1) * a.R] |
                             ((uint32_t)p[(int64_t)min(n + 2 * j + 1, a.N - 1) * a.R] << 16);
            }
            w[i].set(raw);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (t < nt) {
                float x[8];
                const f32x4 lo = n < a.N ? load4<BF16>(a.dy, row[t] + n, a.N - n) : f32x4(0);
                const f32x4 hi = n + 4 < a.N ? load4<BF16>(a.dy, row[t] + n + 4, a.N - n - 4) : f32x4(0);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = lo[j];
                    x[4 + j] = hi[j];
                }
                Grad<BF16> d;
                d.set(x);
#pragma unroll
                for (int i = 0; i < RT; ++i) acc[t][i] = mfma_grad<F16, BF16>(w[i], d, acc[t][i]);
            }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
        if (t < nt)
#pragma unroll
            for (int i = 0; i < RT; ++i) red[wave][t * RT + i][lane] = acc[t][i];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < RT; ++k) {
        const int tile = wave + 4 * k, t = tile / RT, i = tile % RT;
        if (t >= nt) continue;
        f32x4 d = red[0][tile][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) d += red[w][tile][lane];
        const int at = 16 * t + c, r = r0 + 16 * i + 4 * g;
        if (at >= unit.z || r >= a.R) continue;
        *reinterpret_cast<f32x4*>(a.part + ((int64_t)s * a.M + unit.y + at) * a.R + r) = d;
    }
}

// u = s_e times the sum of the parts, in order; a workgroup per unit.
__global__ __launch_bounds__(LT) void lora_u_join_kernel(LoraArgs a) {
    const int4 unit = a.units[blockIdx.x];
    if (unit.z == 0 || unit.x >= a.E) return;
    const float scale = a.scale[unit.x];
    const int64_t at = (int64_t)unit.y * a.R;
    for (int i = 4 * threadIdx.x; i < unit.z * a.R; i += 4 * LT) {
        f32x4 d = 0;
        for (int s = 0; s < a.S; ++s) d += *reinterpret_cast<const f32x4*>(a.part + (int64_t)s * a.M * a.R + at + i);
        *reinterpret_cast<f32x4*>(a.u + at + i) = d * scale;
    }
}

// Joins the four waves' accumulators in LDS: wave w returns the tiles w, w + 4, ... .
template <int NT> __device__ inline void join_waves(f32x4 (*red)[NT][64], f32x4* acc, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < NT; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NT / 4; ++k) {
        f32x4 d = red[0][wave + 4 * k][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) d += red[w][wave + 4 * k][lane];
        acc[k] = d;
    }
}

// dB_e[n][r] over all rows of adapter e: a workgroup has 64 columns n and up to 64 ranks, its
// waves every fourth 32 rows.
template <int RT, bool BF16>
__global__ __launch_bounds__(LT) void lora_dB_kernel(LoraArgs a, int ntiles) {
    __shared__ f32x4 red[4][4 * RT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int e = (int)blockIdx.x / ntiles, n0 = ((int)blockIdx.x % ntiles) * 64;
    const int r0 = (int)blockIdx.y * LORA_RC;
    const int p0 = a.offs[e], p1 = a.offs[e + 1];
    f32x4 acc[4 * RT];
#pragma unroll
    for (int i = 0; i < 4 * RT; ++i) acc[i] = 0;
    for (int p = p0 + 32 * wave; p < p1; p += 128) {
        int64_t row[8];
        bool live[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            live[j] = p + 8 * g + j < p1;
            row[j] = a.order[min(p + 8 * g + j, p1 - 1)];
        }
        u32x4 v[RT][3];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float w = a.v[row[j] * a.R + min(r0 + 16 * i + c, a.R - 1)];
                x[j] = live[j] ? w : 0.f;
            }
            split3(x, v[i]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float x[8];
            const int n = min(n0 + 16 * t + c, a.N - 1);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = grad_at<BF16>(a.dy, row[j] * a.lddy + n);
            Grad<BF16> d;
            d.set(x);
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[t * RT + i] = mfma_3<Grad<BF16>::T>(v[i], d.t, acc[t * RT + i]);
        }
    }
    join_waves<4 * RT>(red, acc, wave, lane);
    const float scale = a.scale[e];
#pragma unroll
    for (int k = 0; k < RT; ++k) {
        const int tile = wave + 4 * k, n = n0 + 16 * (tile / RT) + c, r = r0 + 16 * (tile % RT) + 4 * g;
        if (n < a.N && r < a.R) *reinterpret_cast<f32x4*>(a.dB + ((int64_t)e * a.N + n) * a.R + r) = acc[k] * scale;
    }
}

// dA_e[r][k] over all rows of adapter e: a workgroup has two blocks of K and up to 64 ranks.
template <int RT, bool Q81>
__global__ __launch_bounds__(LT) void lora_dA_kernel(LoraArgs a, int ktiles) {
    __shared__ f32x4 red[4][4 * RT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int e = (int)blockIdx.x / ktiles, b0 = ((int)blockIdx.x % ktiles) * 2;
    const int r0 = (int)blockIdx.y * LORA_RC;
    const int p0 = a.offs[e], p1 = a.offs[e + 1];
    f32x4 acc[4 * RT];
#pragma unroll
    for (int i = 0; i < 4 * RT; ++i) acc[i] = 0;
    for (int p = p0 + 32 * wave; p < p1; p += 128) {
        int m[8];
        float u[RT][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int at = min(p + 8 * g + j, p1 - 1);
            m[j] = a.order[at];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const float w = a.u[(int64_t)at * a.R + min(r0 + 16 * i + c, a.R - 1)];
                u[i][j] = p + 8 * g + j < p1 ? w : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int b = min(b0 + k, a.KB - 1);            // past K: a block's repeat, not stored
            u32x4 x[2];
            float xs[8];
            u32x2 q[2];
            q[0] = q[1] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t cell = (int64_t)(m[j] >> 5) * a.KBp + b;
                const uint8_t* from = reinterpret_cast<const uint8_t*>(a.xq) + cell * 1024 + (m[j] & 31) * 16 + c;
                q[0][j / 4] |= (uint32_t)from[0] << (8 * (j & 3));
                q[1][j / 4] |= (uint32_t)from[512] << (8 * (j & 3));
                if constexpr (Q81) xs[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)a.xs2[cell * 32 + (m[j] & 31)]);
                else xs[j] = a.sa[m[j]];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) x[h] = int8_operand<false>(q[h]);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                float w[8];
                u32x4 t[3];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = u[i][j] * xs[j];
                split3(w, t);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f32x4& s = acc[(2 * k + h) * RT + i];
                    s = mfma_bf16(x[h], t[2], s);
                    s = mfma_bf16(x[h], t[1], s);
                    s = mfma_bf16(x[h], t[0], s);
                }
            }
        }
    }
    join_waves<4 * RT>(red, acc, wave, lane);
#pragma unroll
    for (int k = 0; k < RT; ++k) {
        const int tile = wave + 4 * k, kt = tile / RT, r = r0 + 16 * (tile % RT) + c;
        if (b0 + kt / 2 < a.KB && r < a.R)
            *reinterpret_cast<f32x4*>(a.dA + ((int64_t)e * a.R + r) * a.K + 32 * b0 + 16 * kt + 4 * g) = acc[k];
    }
}

// dx = dxb + A_e^T u over (unit, 256 columns).
template <bool F16>
__global__ __launch_bounds__(LT) void lora_dx_kernel(LoraArgs a, int ktiles) {
    constexpr int LD = LORA_RC + 8;
    __shared__ __attribute__((aligned(16))) uint16_t ut[3][GROUP_UNIT][LD];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int u = (int)blockIdx.x / ktiles, tile = (int)blockIdx.x % ktiles;
    const int4 unit = a.units[u];
    if (unit.z == 0) return;
    const int nt = (unit.z + 15) >> 4;
    const bool none = unit.x >= a.E;
    const int k0 = tile * UP_COLS + wave * 64;
    int64_t row[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) row[t] = a.order[unit.y + min(16 * t + c, unit.z - 1)];
    f32x4 acc[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[t][i] = 0;
            const int k = k0 + 16 * i + 4 * g;
            if (a.dxb && t < nt && k < a.K) acc[t][i] = load4<false>(a.dxb, row[t] * a.lddxb + k, a.K - k);
        }
    if (!none)
        for (int r0 = 0; r0 < a.R; r0 += LORA_RC) {
            if (r0) __syncthreads();
            for (int idx = threadIdx.x; idx < nt * 16 * (LORA_RC / 4); idx += LT) {
                const int at = idx / (LORA_RC / 4), r = 4 * (idx % (LORA_RC / 4));
                f32x4 d = 0;
                if (at < unit.z && r0 + r < a.R)
                    d = *reinterpret_cast<const f32x4*>(a.u + ((int64_t)unit.y + at) * a.R + r0 + r);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    u32x2 w;
                    w[0] = pack_hi(d[0], d[1]);
                    w[1] = pack_hi(d[2], d[3]);
                    *reinterpret_cast<u32x2*>(&ut[k][at][r]) = w;
#pragma unroll
                    for (int j = 0; j < 4; ++j) d[j] -= cut(d[j]);
                }
            }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < LORA_RC; kk += 32) {
                if (r0 + kk >= a.R) break;
                Weights<F16> w[4];
                const int r = r0 + kk + 8 * g;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = min(k0 + 16 * i + c, a.K - 1);
                    u32x4 raw = 0;
                    if (r < a.R) raw = gather8(a.A + ((int64_t)unit.x * a.R + r) * a.K + k, a.K);
                    w[i].set(raw);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t < nt) {
                        u32x4 x[3];
#pragma unroll
                        for (int k = 0; k < 3; ++k) x[k] = *reinterpret_cast<const u32x4*>(&ut[k][16 * t + c][kk + 8 * g]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[t][i] = mfma_terms(w[i], x, acc[t][i]);
                    }
            }
        }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (t >= nt || 16 * t + c >= unit.z) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + 16 * i + 4 * g;
            if (k < a.K) store4<false>(a.dx, row[t] * a.lddx + k, acc[t][i], a.K - k);
        }
    }
}

int64_t u_parts(int64_t E, int64_t M, int64_t N) {
    const int64_t units = plan_layout(E, M).nunits;
    return std::max<int64_t>(1, std::min<int64_t>(512 / units, ceil_div(N, 128)));
}

template <int RT>
void launch_sums(const LoraArgs& a, bool f16, bool q81, hipStream_t s) {
    const unsigned rc = (unsigned)ceil_div(a.R, LORA_RC);
    const dim3 gu((unsigned)(a.nunits * a.S), rc);
    if (f16) {
        if (q81) hipLaunchKernelGGL((lora_u_kernel<RT, true, false>), gu, dim3(LT), 0, s, a);
        else hipLaunchKernelGGL((lora_u_kernel<RT, true, true>), gu, dim3(LT), 0, s, a);
    } else {
        if (q81) hipLaunchKernelGGL((lora_u_kernel<RT, false, false>), gu, dim3(LT), 0, s, a);
        else hipLaunchKernelGGL((lora_u_kernel<RT, false, true>), gu, dim3(LT), 0, s, a);
    }
    hipLaunchKernelGGL(lora_u_join_kernel, dim3((unsigned)a.nunits), dim3(LT), 0, s, a);
    const int nt = (int)ceil_div(a.N, 64), kt = (int)ceil_div(a.KB, 2);
    const dim3 gb((unsigned)(a.E * nt), rc), ga((unsigned)(a.E * kt), rc);
    if (q81) {
        hipLaunchKernelGGL((lora_dB_kernel<RT, false>), gb, dim3(LT), 0, s, a, nt);
        hipLaunchKernelGGL((lora_dA_kernel<RT, true>), ga, dim3(LT), 0, s, a, kt);
    } else {
        hipLaunchKernelGGL((lora_dB_kernel<RT, true>), gb, dim3(LT), 0, s, a, nt);
        hipLaunchKernelGGL((lora_dA_kernel<RT, false>), ga, dim3(LT), 0, s, a, kt);
    }
}

}  // namespace

size_t lora_grad_workspace_bytes(int64_t E, int64_t M, int64_t N, int64_t R) {
    return (size_t)(round_up(u_parts(E, M, N) * M * R * 4, REGION_ALIGN) + round_up(M * R * 4, REGION_ALIGN));
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
    a.S = (int)u_parts(E, M, N);
    a.part = static_cast<float*>(ws);
    a.u = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + round_up((int64_t)a.S * M * R * 4, REGION_ALIGN));
    const bool q81 = t == MMQ_ACT_Q8_1;
    if (R <= 16) launch_sums<1>(a, f16, q81, s);
    else if (R <= 32) launch_sums<2>(a, f16, q81, s);
    else launch_sums<4>(a, f16, q81, s);
    if (dx) {
        const int kt = (int)ceil_div(K, UP_COLS);
        const dim3 grid((unsigned)a.nunits * (unsigned)kt);
        if (f16) hipLaunchKernelGGL(lora_dx_kernel<true>, grid, dim3(LT), 0, s, a, kt);
        else hipLaunchKernelGGL(lora_dx_kernel<false>, grid, dim3(LT), 0, s, a, kt);
    }
    return hipGetLastError();
}

}  // namespace mmq
