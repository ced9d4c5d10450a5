// linattn.cu -- linear attention with a decay per head, token by token, for
// sm_100a.  Per (b, h), with a state S of P values by N keys:
//
//   S_t   = exp(g_t) S_{t-1} + v_t k_t^T,     out_t = scale * S_t q_t
//
// Rows of S (one value p each) are independent of one another, so every kernel
// here gives rows to warps and the N keys of a row to a warp's lanes; S, its
// products and its sums are float32 throughout.
//
//   linattn_generic_kernel  a prompt of any strides, types and sizes (N <= 256):
//                           a warp carries 4 rows of S in registers over the
//                           whole sequence.
//   linattn_step_kernel     one token: S is read and written once, in 16-byte
//                           vectors.
//   linattn_step_generic_kernel  one token, any strides.
//
// The tensor-core form for prompts is linattn_chunk.cu.
#include "../../include/ssm_causal.h"
#include "common.cuh"
#include "problem.h"

namespace ssm {
namespace {

constexpr int kBlock = 128;   // 4 warps
constexpr int kWarpRows = 4;  // rows of S per warp of the generic prompt kernel

// a positive log decay counts as 0 (a NaN stays one)
__device__ __forceinline__ float decay_log(float g) { return g > 0.0f ? 0.0f : g; }

// sum over the warp of each of K values, K a power of two <= 32: the butterfly
// halves the number of values a lane carries at each step while it can, so K
// sums take K + log2(32 / K) - 1 shuffles or so instead of 5 K.  Afterwards
// lane l holds the sum of value l / (32 / K).
template <int K>
__device__ __forceinline__ float reduce_many(float (&v)[K], int lane) {
    int keep = K;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        if (keep > 1) {
            keep >>= 1;
            const bool hi = lane & o;
#pragma unroll
            for (int i = 0; i < K / 2; ++i) {
                if (i < keep) {
                    const float send = hi ? v[i] : v[i + keep];
                    const float mine = hi ? v[i + keep] : v[i];
                    v[i] = mine + __shfl_xor_sync(0xffffffffu, send, o);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return v[0];
}

// Prompt, any layout.  Bound by the latency of a token's chain (decay and FMA,
// then the reduction, whose result nothing waits for): U tokens are loaded
// while the U before them are computed, and their 4 U sums reduced together.
template <typename T, int NE, int U>
__global__ void __launch_bounds__(kBlock) linattn_generic_kernel(const LinAttnProblem p) {
    const int lane = threadIdx.x & 31;
    const int64_t nblk = (p.P + 4 * kWarpRows - 1) / (4 * kWarpRows);
    const int64_t unit = blockIdx.x / nblk;
    const int64_t b = unit / p.H, h = unit - b * p.H;
    const int64_t p0 = ((blockIdx.x - unit * nblk) * 4 + (threadIdx.x >> 5)) * kWarpRows;
    if (p0 >= p.P) return;
    int64_t len = p.L;
    if (p.lens) {
        const int64_t n = p.lens[b * p.len_b];
        len = n < 0 ? 0 : (n < p.L ? n : p.L);
    }
    float s[kWarpRows][NE];
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r)
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int64_t n = lane + 32 * i;
            s[r][i] = p.s_in && p0 + r < p.P && n < p.N
                          ? p.s_in[b * p.si_b + h * p.si_h + (p0 + r) * p.si_p + n * p.si_n] : 0.0f;
        }
    const T* q = static_cast<const T*>(p.q) + b * p.q_b + (h / p.rep) * p.q_h;
    const T* k = static_cast<const T*>(p.k) + b * p.k_b + (h / p.rep) * p.k_h;
    const T* v = static_cast<const T*>(p.v) + b * p.v_b + h * p.v_h;
    const float* g = p.g + b * p.g_b + h * p.g_h;
    T* out = static_cast<T*>(p.out) + b * p.o_b + h * p.o_h;

    float kn[U][NE], qn[U][NE], vn[U][kWarpRows], gn[U];
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u;
            const bool on = t < len;
            gn[u] = on ? decay_log(g[t * p.g_t]) : 0.0f;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int64_t n = lane + 32 * i;
                kn[u][i] = on && n < p.N ? to_f<T>(k[t * p.k_t + n * p.k_n]) : 0.0f;
                qn[u][i] = on && n < p.N ? to_f<T>(q[t * p.q_t + n * p.q_n]) : 0.0f;
            }
#pragma unroll
            for (int r = 0; r < kWarpRows; ++r)
                vn[u][r] = on && p0 + r < p.P ? to_f<T>(v[t * p.v_t + (p0 + r) * p.v_p]) : 0.0f;
        }
    };
    load(0);
    for (int64_t t0 = 0; t0 < len; t0 += U) {
        // The decay is applied as S + (exp(g) - 1) S where it is above a half: the error of a
        // factor close to 1 would add up over the tokens that S remembers, that
        // of its distance from 1 does not.
        float kc[U][NE], qc[U][NE], vc[U][kWarpRows], lam[U];
        bool near1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            near1[u] = gn[u] > -0.6931f;
            lam[u] = near1[u] ? expm1f(gn[u]) : expf(gn[u]);
#pragma unroll
            for (int i = 0; i < NE; ++i) kc[u][i] = kn[u][i], qc[u][i] = qn[u][i];
#pragma unroll
            for (int r = 0; r < kWarpRows; ++r) vc[u][r] = vn[u][r];
        }
        load(t0 + U);
        float sum[U * kWarpRows];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < kWarpRows; ++r) {
                float acc = 0.0f;
                if (t0 + u < len) {  // past the end: the state stays
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        s[r][i] = fmaf(lam[u], s[r][i], fmaf(vc[u][r], kc[u][i], near1[u] ? s[r][i] : 0.0f));
                        acc = fmaf(s[r][i], qc[u][i], acc);
                    }
                }
                sum[u * kWarpRows + r] = acc;
            }
        constexpr int K = U * kWarpRows;  // 8 or 16 sums
        const float o = reduce_many<K>(sum, lane);
        const int idx = lane / (32 / K);
        const int64_t t = t0 + idx / kWarpRows, row = p0 + idx % kWarpRows;
        if (lane % (32 / K) == 0 && t < len && row < p.P)
            out[t * p.o_t + row * p.o_p] = from_f<T>(o * p.scale);
    }
    if (!p.s_out) return;
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r)
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int64_t n = lane + 32 * i;
            if (p0 + r < p.P && n < p.N)
                p.s_out[b * p.so_b + h * p.so_h + (p0 + r) * p.so_p + n * p.so_n] = s[r][i];
        }
}

template <typename T>
cudaError_t generic_t(const LinAttnProblem& p, int grid, cudaStream_t s) {
    if (p.N <= 32) linattn_generic_kernel<T, 1, 4><<<grid, kBlock, 0, s>>>(p);
    else if (p.N <= 64) linattn_generic_kernel<T, 2, 4><<<grid, kBlock, 0, s>>>(p);
    else if (p.N <= 128) linattn_generic_kernel<T, 4, 4><<<grid, kBlock, 0, s>>>(p);
    else linattn_generic_kernel<T, 8, 2><<<grid, kBlock, 0, s>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------- one token --
// Bound by the state's bytes.  A row of N keys is nv = N / VE 16-byte vectors, held by LPR
// = 2^k >= min(nv, 32) lanes with CPL vectors each, so a warp takes 32 / LPR
// rows at once; RU such groups of rows are loaded before the first is used.
__host__ __device__ inline int step_lanes(int nv) {
    int l = 1;
    while (l < nv && l < 32) l <<= 1;
    return l;
}
template <int CPL> struct StepShape { static constexpr int RU = CPL == 1 ? 8 : 4; };

template <typename ST, int CPL>
__global__ void __launch_bounds__(kBlock) linattn_step_kernel(const LinAttnStepProblem p) {
    constexpr int VE = Vec16<ST>::VE, RU = StepShape<CPL>::RU;
    const int lane = threadIdx.x & 31;
    const int nv = (int)(p.N / VE), lpr = step_lanes(nv), rows_at_once = 32 / lpr;
    const int rows_cta = (kBlock / 32) * RU * rows_at_once;
    const int64_t nblk = (p.P + rows_cta - 1) / rows_cta;
    const int64_t unit = blockIdx.x / nblk;
    const int64_t b = unit / p.H, h = unit - b * p.H;
    const int64_t row0 = (blockIdx.x - unit * nblk) * rows_cta +
                         (int64_t)(threadIdx.x >> 5) * RU * rows_at_once + lane / lpr;
    const int64_t slot = p.slot_idx ? p.slot_idx[b * p.ix_b] : b;
    if (slot < 0 || slot >= p.slots) return;
    const int c0 = lane & (lpr - 1);

    const ST* in = static_cast<const ST*>(p.s_in) + slot * p.si_b + h * p.si_h;
    ST* so = static_cast<ST*>(p.s_out) + slot * p.so_b + h * p.so_h;
    uint4 raw[RU][CPL];
#pragma unroll
    for (int r = 0; r < RU; ++r) {
        const int64_t row = row0 + r * rows_at_once;
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            if (row < p.P && c0 + c * lpr < nv)
                raw[r][c] = ld_stream16(in + row * p.si_p + (int64_t)(c0 + c * lpr) * VE);
    }
    float kf[CPL][VE], qf[CPL][VE];
    const int64_t kb = b * p.k_b + (h / p.rep) * p.k_h, qb = b * p.q_b + (h / p.rep) * p.q_h;
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const int64_t n = (int64_t)(c0 + c * lpr) * VE + e;
            const bool on = c0 + c * lpr < nv;
            kf[c][e] = on ? ld_f(p.k, kb + n * p.k_n, p.io_dt) : 0.0f;
            qf[c][e] = on ? ld_f(p.q, qb + n * p.q_n, p.io_dt) : 0.0f;
        }
    const float lam = expf(decay_log(p.g[b * p.g_b + h * p.g_h]));
    float acc[RU];
#pragma unroll
    for (int r = 0; r < RU; ++r) {
        const int64_t row = row0 + r * rows_at_once;
        acc[r] = 0.0f;
        if (row < p.P) {
            const float v = ld_f(p.v, b * p.v_b + h * p.v_h + row * p.v_p, p.io_dt);
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                if (c0 + c * lpr < nv) {
                    float f[VE];
                    Vec16<ST>::unpack(raw[r][c], f);
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        f[e] = fmaf(v, kf[c][e], lam * f[e]);
                        acc[r] = fmaf(f[e], qf[c][e], acc[r]);
                    }
                    st_stream16(so + row * p.so_p + (int64_t)(c0 + c * lpr) * VE, Vec16<ST>::pack(f));
                }
        }
    }
#pragma unroll
    for (int r = 0; r < RU; ++r) {
        for (int o = lpr >> 1; o >= 1; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
        const int64_t row = row0 + r * rows_at_once;
        if (c0 == 0 && row < p.P) st_f(p.out, b * p.o_b + h * p.o_h + row * p.o_p, p.io_dt, acc[r] * p.scale);
    }
}

__global__ void __launch_bounds__(kBlock) linattn_step_generic_kernel(const LinAttnStepProblem p) {
    const int lane = threadIdx.x & 31;
    const int64_t nblk = (p.P + kBlock / 32 - 1) / (kBlock / 32);
    const int64_t unit = blockIdx.x / nblk;
    const int64_t b = unit / p.H, h = unit - b * p.H;
    const int64_t row = (blockIdx.x - unit * nblk) * (kBlock / 32) + (threadIdx.x >> 5);
    const int64_t slot = p.slot_idx ? p.slot_idx[b * p.ix_b] : b;
    if (slot < 0 || slot >= p.slots || row >= p.P) return;  // warp-uniform
    const float lam = expf(decay_log(p.g[b * p.g_b + h * p.g_h]));
    const float v = ld_f(p.v, b * p.v_b + h * p.v_h + row * p.v_p, p.io_dt);
    const int64_t si = slot * p.si_b + h * p.si_h + row * p.si_p;
    const int64_t so = slot * p.so_b + h * p.so_h + row * p.so_p;
    const int64_t kb = b * p.k_b + (h / p.rep) * p.k_h, qb = b * p.q_b + (h / p.rep) * p.q_h;
    float acc = 0.0f;
    for (int64_t n = lane; n < p.N; n += 32) {
        const float f = fmaf(v, ld_f(p.k, kb + n * p.k_n, p.io_dt), lam * ld_f(p.s_in, si + n * p.si_n, p.st_dt));
        acc = fmaf(f, ld_f(p.q, qb + n * p.q_n, p.io_dt), acc);
        st_f(p.s_out, so + n * p.so_n, p.st_dt, f);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) st_f(p.out, b * p.o_b + h * p.o_h + row * p.o_p, p.io_dt, acc * p.scale);
}

template <typename ST>
cudaError_t step_t(const LinAttnStepProblem& p, int grid, cudaStream_t s) {
    if (p.N / Vec16<ST>::VE <= 32) linattn_step_kernel<ST, 1><<<grid, kBlock, 0, s>>>(p);
    else linattn_step_kernel<ST, 2><<<grid, kBlock, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

int linattn_generic_block() { return kBlock; }
int linattn_generic_rows() { return (kBlock / 32) * kWarpRows; }

cudaError_t launch_linattn_generic(const LinAttnProblem& p, int grid, cudaStream_t s) {
    if (p.io_dt == kF16) return generic_t<__half>(p, grid, s);
    if (p.io_dt == kBF16) return generic_t<__nv_bfloat16>(p, grid, s);
    return generic_t<float>(p, grid, s);
}

int linattn_step_block() { return kBlock; }
int linattn_step_rows(int st_dt, int64_t N, bool vec) {
    if (!vec) return kBlock / 32;
    const int nv = (int)(N / (st_dt == kF32 ? 4 : 8));
    const int ru = nv <= 32 ? StepShape<1>::RU : StepShape<2>::RU;
    return (kBlock / 32) * ru * (32 / step_lanes(nv));
}

cudaError_t launch_linattn_step(const LinAttnStepProblem& p, int kernel, int grid, cudaStream_t s) {
    if (kernel == SSM_KERNEL_LINATTN_STEP_GENERIC) {
        linattn_step_generic_kernel<<<grid, kBlock, 0, s>>>(p);
        return cudaGetLastError();
    }
    if (p.st_dt == kF16) return step_t<__half>(p, grid, s);
    if (p.st_dt == kBF16) return step_t<__nv_bfloat16>(p, grid, s);
    return step_t<float>(p, grid, s);
}

}  // namespace ssm
