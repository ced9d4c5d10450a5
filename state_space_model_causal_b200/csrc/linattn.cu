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
//                           a warp carries 4 rows of S (2 where there are few) in
//                           registers over the whole sequence.
//   linattn_step_bulk_kernel one token: S is read and written once, by bulk copies
//                           through shared memory (rows without gaps).
//   linattn_step_kernel     one token, rows of 16-byte vectors with gaps.
//   linattn_step_generic_kernel  one token, any strides.
//
// The tensor-core form for prompts is linattn_chunk.cu.
#include "../../include/ssm_causal.h"
#include "common.cuh"
#include "problem.h"
#include "tma.cuh"

namespace ssm {
namespace {

constexpr int kBlock = 128;   // 4 warps

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

// Prompt, any layout.  A warp holds R rows of S in registers, a lane NE neighbouring
// keys.  The CTA's threads bring the next stage of tokens (1024 numbers of k and of q, so 4 to
// 32 tokens) into registers while its warps work on the last one from shared memory,
// as float32; 4 tokens' sums are reduced together.  Bound by latency with few warps (2 sequences of
// 1024 tokens, 16 heads of 64: 7 warps per SM, 43% of issue slots), so the tokens of a stage are
// unrolled: 108 us, against 123 in a loop over groups of 4 tokens, and 274 when every warp
// loaded its tokens itself.
constexpr int kStageNumbers = 1024;
template <typename T, int NE, int R>
__global__ void __launch_bounds__(kBlock) linattn_generic_kernel(const LinAttnProblem p) {
    constexpr int NP = 32 * NE, U = kStageNumbers / NP, ROWS = 4 * R;   // U: tokens per stage
    constexpr int PER = kStageNumbers / kBlock, VPER = (U * ROWS + kBlock - 1) / kBlock;
    __shared__ __align__(16) float ks[2][kStageNumbers], qs[2][kStageNumbers];
    __shared__ __align__(16) float vs[2][U * ROWS];
    __shared__ float2 gs[2][U];  // the decay's factor, and 1 if that is its distance from 1
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t nblk = (p.P + ROWS - 1) / ROWS;
    const int64_t unit = blockIdx.x / nblk;
    const int64_t b = unit / p.H, h = unit - b * p.H;
    const int64_t c0 = (blockIdx.x - unit * nblk) * ROWS, p0 = c0 + warp * R;  // rows of the CTA, of the warp
    int64_t len = p.L;
    if (p.lens) {
        const int64_t n = p.lens[b * p.len_b];
        len = n < 0 ? 0 : (n < p.L ? n : p.L);
    }
    auto key = [&](int i) { return NE <= 4 ? lane * NE + i : (i >> 2) * 128 + lane * 4 + (i & 3); };
    float s[R][NE];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NE; ++i)
            s[r][i] = p.s_in && p0 + r < p.P && key(i) < p.N
                          ? p.s_in[b * p.si_b + h * p.si_h + (p0 + r) * p.si_p + key(i) * p.si_n] : 0.0f;
    T* const out = static_cast<T*>(p.out) + b * p.o_b + h * p.o_h;

    // this thread's numbers of a stage: of k and q token u0 + j * du, key n0 (NP = 256: both halves in turn)
    constexpr int kSplit = NP > kBlock ? 2 : 1;
    constexpr int du = NP > kBlock ? 1 : kBlock / NP;
    const int u0 = NP > kBlock ? 0 : threadIdx.x / NP, n0 = threadIdx.x % (NP > kBlock ? kBlock : NP);
    const T* const q0 = static_cast<const T*>(p.q) + b * p.q_b + (h / p.rep) * p.q_h + n0 * p.q_n;
    const T* const k0 = static_cast<const T*>(p.k) + b * p.k_b + (h / p.rep) * p.k_h + n0 * p.k_n;
    const T* const v0 = static_cast<const T*>(p.v) + b * p.v_b + h * p.v_h;
    const float* const g0 = p.g + b * p.g_b + h * p.g_h;
    float kn[PER], qn[PER], vn[VPER], gn = 0.0f;
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int64_t t = t0 + u0 + (j / kSplit) * du;
            const int half = (j % kSplit) * kBlock;
            const bool on = t < len && n0 + half < p.N;
            kn[j] = on ? to_f<T>(k0[t * p.k_t + half * p.k_n]) : 0.0f;
            qn[j] = on ? to_f<T>(q0[t * p.q_t + half * p.q_n]) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < VPER; ++j) {
            const int e = threadIdx.x + j * kBlock, u = e / ROWS;
            const int64_t t = t0 + u, row = c0 + e % ROWS;
            vn[j] = u < U && t < len && row < p.P ? to_f<T>(v0[t * p.v_t + row * p.v_p]) : 0.0f;
        }
        if (threadIdx.x < U) gn = t0 + threadIdx.x < len ? decay_log(g0[(t0 + threadIdx.x) * p.g_t]) : 0.0f;
    };
    load(0);
    for (int64_t t0 = 0, buf = 0; t0 < len; t0 += U, buf ^= 1) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int at = (u0 + (j / kSplit) * du) * NP + n0 + (j % kSplit) * kBlock;
            ks[buf][at] = kn[j];
            qs[buf][at] = qn[j];
        }
#pragma unroll
        for (int j = 0; j < VPER; ++j)
            if (threadIdx.x + j * kBlock < U * ROWS) vs[buf][threadIdx.x + j * kBlock] = vn[j];
        // The decay is applied as S + (exp(g) - 1) S where it is above a half: the error of a
        // factor close to 1 would add up over the tokens that S remembers, that
        // of its distance from 1 does not.
        // Tokens past the end have v = 0 and a factor of 1.
        if (threadIdx.x < U)
            gs[buf][threadIdx.x] = t0 + threadIdx.x >= len ? make_float2(1.0f, 0.0f)
                                   : gn > -0.6931f ? make_float2(expm1f(gn), 1.0f) : make_float2(expf(gn), 0.0f);
        __syncthreads();  // (the other buffer is written after the next one)
        if (t0 + U < len) load(t0 + U);
#pragma unroll
        for (int u = 0; u < U; u += 4) {
            float sum[4 * R];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float kf[NE], qf[NE], vf[R];
                const float2 lam = gs[buf][u + x];
                const bool near1 = lam.y != 0.0f;
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    kf[i] = ks[buf][(u + x) * NP + key(i)];
                    qf[i] = qs[buf][(u + x) * NP + key(i)];
                }
#pragma unroll
                for (int r = 0; r < R; ++r) vf[r] = vs[buf][(u + x) * ROWS + warp * R + r];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float acc = 0.0f;
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        s[r][i] = fmaf(lam.x, s[r][i], fmaf(vf[r], kf[i], near1 ? s[r][i] : 0.0f));
                        acc = fmaf(s[r][i], qf[i], acc);
                    }
                    sum[x * R + r] = acc;
                }
            }
            const float o = reduce_many<4 * R>(sum, lane);
            constexpr int share = 32 / (4 * R);  // lanes that hold the same sum
            const int idx = lane / share;
            const int64_t t = t0 + u + idx / R, row = p0 + idx % R;
            if (lane % share == 0 && t < len && row < p.P) out[t * p.o_t + row * p.o_p] = from_f<T>(o * p.scale);
        }
    }
    if (!p.s_out) return;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (p0 + r < p.P && key(i) < p.N)
                p.s_out[b * p.so_b + h * p.so_h + (p0 + r) * p.so_p + key(i) * p.so_n] = s[r][i];
}

template <typename T, int R>
cudaError_t generic_t(const LinAttnProblem& p, int grid, cudaStream_t s) {
    if (p.N <= 32) linattn_generic_kernel<T, 1, R><<<grid, kBlock, 0, s>>>(p);
    else if (p.N <= 64) linattn_generic_kernel<T, 2, R><<<grid, kBlock, 0, s>>>(p);
    else if (p.N <= 128) linattn_generic_kernel<T, 4, R><<<grid, kBlock, 0, s>>>(p);
    else linattn_generic_kernel<T, 8, R><<<grid, kBlock, 0, s>>>(p);
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

// Dense rows: blocks of up to 16 KB of a head's state go through a ring of
// stages in shared memory, brought in and taken out by bulk copies that one thread
// issues; the CTA updates a stage in place.  Loads run kStages - 1 blocks ahead.  What else
// an update reads is small but far away (the slot's index, then k, q, v and the decay),
// so a CTA takes a unit of several blocks of one head, and reads the next unit's small
// operands into registers while it works on this one.
// 245 x 32 heads of 128 x 128 in float32: 185 us, 0.85 of a plain copy's rate (half of the
// bytes are writes); 258 with vectors straight from global memory.
constexpr int kStageBytes = 16384, kStages = 3, kUnitRows = 512;
struct BulkSmem {
    alignas(128) unsigned char stage[kStages][kStageBytes];
    uint64_t full[kStages];
    int64_t slot[kStages];
    float v[2][kUnitRows];
};
constexpr int kBulkCtas = 4;  // per SM
static_assert(kBulkCtas * (sizeof(BulkSmem) + 1024) <= 228 * 1024, "shared memory of an SM");

template <typename ST, int CPL>
__global__ void __launch_bounds__(kBlock, kBulkCtas)
linattn_step_bulk_kernel(const LinAttnStepProblem p, const LinAttnStepBulk sh, DeviceError* err, const BoundedWaits waits) {
    constexpr int VE = Vec16<ST>::VE, VN = kUnitRows / kBlock, RU = StepShape<CPL>::RU;
    extern __shared__ __align__(128) unsigned char raw[];
    BulkSmem& sm = *reinterpret_cast<BulkSmem*>(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nv = (int)(p.N / VE), lpr = step_lanes(nv), rows_at_once = 32 / lpr;
    const int row_bytes = nv * 16, c0 = lane & (lpr - 1);
    struct Unit {
        int64_t b, h, row0;
        int rows, blocks;
    };
    auto unit_at = [&](uint32_t u) {
        Unit t;
        const uint32_t head = u / sh.groups;
        t.row0 = (int64_t)(u - head * sh.groups) * sh.rows * sh.blocks;
        const int64_t left = p.P - t.row0;
        t.rows = (int)(left < (int64_t)sh.rows * sh.blocks ? left : (int64_t)sh.rows * sh.blocks);
        t.blocks = (t.rows + sh.rows - 1) / sh.rows;
        t.b = head / (uint32_t)p.H;
        t.h = head - (uint32_t)t.b * (uint32_t)p.H;
        return t;
    };
    // thread 0: the copies, some blocks ahead of the work
    uint32_t ahead_unit = blockIdx.x, issued = 0;
    int ahead_block = 0;
    Unit ahead;
    int64_t ahead_slot = -1;
    auto fetch = [&] {
        if (ahead_unit >= sh.units) return;
#ifdef SSM_TEST_HOOKS
        if ((int64_t)ahead_unit == waits.drop_item) return;  // never issued
#endif
        if (ahead_block == 0) {
            ahead = unit_at(ahead_unit);
            ahead_slot = p.slot_idx ? p.slot_idx[ahead.b * p.ix_b] : ahead.b;
            if (ahead_slot >= p.slots) ahead_slot = -1;
        }
        const int s = (int)(issued % kStages), r0 = ahead_block * sh.rows;
        const int rows = ahead.rows - r0 < sh.rows ? ahead.rows - r0 : sh.rows;
        const uint32_t bytes = ahead_slot < 0 ? 0u : (uint32_t)(rows * row_bytes);
        sm.slot[s] = ahead_slot;
        mbar_arrive_expect_tx(&sm.full[s], bytes);
        if (bytes)
            tma_load_1d(sm.stage[s], static_cast<const ST*>(p.s_in) + ahead_slot * p.si_b + ahead.h * p.si_h +
                                         (ahead.row0 + r0) * p.si_p, bytes, &sm.full[s]);
        ++issued;
        if (++ahead_block == ahead.blocks) {
            ahead_block = 0;
            ahead_unit += gridDim.x;
        }
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[s], 1);
        mbar_fence_init();
        for (int i = 0; i < kStages - 1; ++i) fetch();
    }
    // a unit's small operands
    float kn[CPL][VE], qn[CPL][VE], vn[VN], gn = 0.0f;
    auto load_small = [&](const Unit& t) {
        const int64_t hk = t.h / (uint32_t)p.rep;
        const int64_t kb = t.b * p.k_b + hk * p.k_h, qb = t.b * p.q_b + hk * p.q_h;
#pragma unroll
        for (int c = 0; c < CPL; ++c)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const int64_t n = (int64_t)(c0 + c * lpr) * VE + e;
                const bool on = c0 + c * lpr < nv;
                kn[c][e] = on ? ld_f(p.k, kb + n * p.k_n, p.io_dt) : 0.0f;
                qn[c][e] = on ? ld_f(p.q, qb + n * p.q_n, p.io_dt) : 0.0f;
            }
#pragma unroll
        for (int j = 0; j < VN; ++j) {
            const int r = threadIdx.x + j * kBlock;
            vn[j] = r < t.rows ? ld_f(p.v, t.b * p.v_b + t.h * p.v_h + (t.row0 + r) * p.v_p, p.io_dt) : 0.0f;
        }
        gn = p.g[t.b * p.g_b + t.h * p.g_h];
    };
    auto put_v = [&](int buf) {
#pragma unroll
        for (int j = 0; j < VN; ++j) sm.v[buf][threadIdx.x + j * kBlock] = vn[j];
    };
    uint32_t u = blockIdx.x, done = 0;
    Unit next = unit_at(u < sh.units ? u : 0);
    if (u < sh.units) {
        load_small(next);
        put_v(0);
    }
    __syncthreads();
    bool ok = true;
    uint32_t unit = u;
    for (int buf = 0; ok && u < sh.units; buf ^= 1) {
        unit = u;
        const Unit t = next;
        float kf[CPL][VE], qf[CPL][VE];
#pragma unroll
        for (int c = 0; c < CPL; ++c)
#pragma unroll
            for (int e = 0; e < VE; ++e) kf[c][e] = kn[c][e], qf[c][e] = qn[c][e];
        const float lam = expf(decay_log(gn));
        u += gridDim.x;
        if (u < sh.units) {
            next = unit_at(u);
            load_small(next);
        }
        for (int blk = 0; blk < t.blocks; ++blk, ++done) {
            const int s = (int)(done % kStages), r0 = blk * sh.rows;
            const int rows = t.rows - r0 < sh.rows ? t.rows - r0 : sh.rows;
            const bool here = mbar_wait_bounded(&sm.full[s], (done / kStages) & 1, waits.budget);
            const int64_t slot = sm.slot[s];
            if (here && slot >= 0) {
                // RU groups of rows at a time: their loads together, their sums together
                for (int g0 = warp * RU; g0 * rows_at_once < rows; g0 += RU * (kBlock / 32)) {
                    float acc[RU];
                    uint4 x[RU][CPL];
#pragma unroll
                    for (int r = 0; r < RU; ++r) {
                        const int row = (g0 + r) * rows_at_once + lane / lpr;
#pragma unroll
                        for (int c = 0; c < CPL; ++c)
                            if (row < rows && c0 + c * lpr < nv)
                                x[r][c] = *(reinterpret_cast<const uint4*>(sm.stage[s] + row * row_bytes) + c0 + c * lpr);
                    }
#pragma unroll
                    for (int r = 0; r < RU; ++r) {
                        const int row = (g0 + r) * rows_at_once + lane / lpr;
                        acc[r] = 0.0f;
                        const float v = row < rows ? sm.v[buf][r0 + row] : 0.0f;
#pragma unroll
                        for (int c = 0; c < CPL; ++c)
                            if (row < rows && c0 + c * lpr < nv) {
                                float f[VE];
                                Vec16<ST>::unpack(x[r][c], f);
#pragma unroll
                                for (int e = 0; e < VE; ++e) {
                                    f[e] = fmaf(v, kf[c][e], lam * f[e]);
                                    acc[r] = fmaf(f[e], qf[c][e], acc[r]);
                                }
                                *(reinterpret_cast<uint4*>(sm.stage[s] + row * row_bytes) + c0 + c * lpr) = Vec16<ST>::pack(f);
                            }
                    }
                    const int64_t o0 = t.b * p.o_b + t.h * p.o_h + (t.row0 + r0) * p.o_p;
                    if (lpr == 32) {
                        const float sum = reduce_many<RU>(acc, lane);
                        const int row = g0 + lane / (32 / RU);
                        if (lane % (32 / RU) == 0 && row < rows) st_f(p.out, o0 + row * p.o_p, p.io_dt, sum * p.scale);
                    } else {
#pragma unroll
                        for (int r = 0; r < RU; ++r) {
                            for (int o = lpr >> 1; o >= 1; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
                            const int row = (g0 + r) * rows_at_once + lane / lpr;
                            if (c0 == 0 && row < rows) st_f(p.out, o0 + row * p.o_p, p.io_dt, acc[r] * p.scale);
                        }
                    }
                }
            }
            if (blk + 1 == t.blocks && u < sh.units) put_v(buf ^ 1);
            fence_proxy_async_smem();
            if (__syncthreads_or(!here)) {
                ok = false;
                break;
            }
            if (threadIdx.x == 0) {
                if (slot >= 0)
                    tma_store_1d(static_cast<ST*>(p.s_out) + slot * p.so_b + t.h * p.so_h + (t.row0 + r0) * p.so_p,
                                 sm.stage[s], (uint32_t)(rows * row_bytes));
                bulk_commit();
                bulk_wait_read<1>();  // the stage of the block before has been read out
                fetch();
            }
        }
    }
    if (threadIdx.x == 0) {
        if (!ok) {  // a copy never came: leave with none in flight
            report_device_error(err, SSM_KERNEL_LINATTN_STEP_BULK, (long long)unit);
            for (; done < issued; ++done) mbar_wait_bounded(&sm.full[done % kStages], (done / kStages) & 1, waits.budget);
        }
        bulk_wait_all();
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
    if constexpr (Vec16<ST>::VE == 4) {  // (rows of 16-bit numbers are 32 vectors at most)
        if (p.N > 128) {
            linattn_step_kernel<ST, 2><<<grid, kBlock, 0, s>>>(p);
            return cudaGetLastError();
        }
    }
    linattn_step_kernel<ST, 1><<<grid, kBlock, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename ST, int CPL>
cudaError_t bulk_t(const LinAttnStepProblem& p, const LinAttnStepBulk& plan, DeviceError* err, const BoundedWaits& waits,
                   cudaStream_t s) {
    auto* fn = linattn_step_bulk_kernel<ST, CPL>;
    int per_sm = 0;
    const cudaError_t e = prepared_launch(
        reinterpret_cast<const void*>(fn), plan.smem, kBlock, &per_sm,
        [&](int bytes) { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); },
        [&](int* n) { *n = kBulkCtas; return cudaSuccess; });
    if (e != cudaSuccess) return e;
    fn<<<plan.grid, kBlock, plan.smem, s>>>(p, plan, err, waits);
    return cudaGetLastError();
}

}  // namespace

int linattn_generic_block() { return kBlock; }
int linattn_generic_rows(int64_t heads, int64_t P, int sms) {
    // rows per CTA: 4 per warp, 2 while that leaves less than 3 CTAs per SM (the kernel waits for a
    // token's chain: more warps hide it, more rows per warp share its loads)
    return heads * ((P + 15) / 16) >= (int64_t)3 * sms ? 16 : 8;
}

cudaError_t launch_linattn_generic(const LinAttnProblem& p, int rows, int grid, cudaStream_t s) {
    if (rows == 8) {
        if (p.io_dt == kF16) return generic_t<__half, 2>(p, grid, s);
        if (p.io_dt == kBF16) return generic_t<__nv_bfloat16, 2>(p, grid, s);
        return generic_t<float, 2>(p, grid, s);
    }
    if (p.io_dt == kF16) return generic_t<__half, 4>(p, grid, s);
    if (p.io_dt == kBF16) return generic_t<__nv_bfloat16, 4>(p, grid, s);
    return generic_t<float, 4>(p, grid, s);
}

int linattn_step_block() { return kBlock; }
int linattn_step_rows(int st_dt, int64_t N, bool vec) {
    if (!vec) return kBlock / 32;
    const int nv = (int)(N / (st_dt == kF32 ? 4 : 8));
    const int ru = nv <= 32 ? StepShape<1>::RU : StepShape<2>::RU;
    return (kBlock / 32) * ru * (32 / step_lanes(nv));
}

int linattn_step_bulk_rows(int st_dt, int64_t N) {
    const int64_t rows = kStageBytes / (N * (st_dt == kF32 ? 4 : 2));
    return (int)(rows < kUnitRows ? rows : kUnitRows);
}

LinAttnStepBulk linattn_step_bulk_plan(int st_dt, int64_t heads, int64_t P, int64_t N, int sms) {
    LinAttnStepBulk plan;
    plan.smem = (int)sizeof(BulkSmem);
    plan.rows = linattn_step_bulk_rows(st_dt, N);
    const int64_t wave = (int64_t)sms * kBulkCtas, per_head = (P + plan.rows - 1) / plan.rows;
    // as many blocks per unit as leave every CTA four units or more
    int64_t blocks = heads * per_head / (4 * wave);
    blocks = blocks < 1 ? 1 : blocks;
    blocks = blocks > per_head ? per_head : blocks;
    if (blocks * plan.rows > kUnitRows) blocks = kUnitRows / plan.rows;
    plan.blocks = (int)blocks;
    plan.groups = (uint32_t)((per_head + blocks - 1) / blocks);
    plan.units = (uint32_t)(heads * plan.groups);
    plan.grid = plan.units < wave ? plan.units : (uint32_t)wave;
    return plan;
}

cudaError_t launch_linattn_step_bulk(const LinAttnStepProblem& p, const LinAttnStepBulk& plan, const BoundedWaits& waits,
                                     int dev, cudaStream_t s) {
    DeviceError* err = device_error_ptr(dev);
    if (!err) return cudaErrorUnknown;
    if (p.st_dt == kF16) return bulk_t<__half, 1>(p, plan, err, waits, s);
    if (p.st_dt == kBF16) return bulk_t<__nv_bfloat16, 1>(p, plan, err, waits, s);
    return p.N <= 128 ? bulk_t<float, 1>(p, plan, err, waits, s) : bulk_t<float, 2>(p, plan, err, waits, s);
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
