// linattn_chunk.cu -- linear attention with a decay per head over a prompt, in
// chunks of 128 tokens on the tensor cores (tcgen05), for sm_100a.
//
// Inside a chunk let G_t be the sum of the log decays up to and including token
// t, S the state before the chunk.  Then
//
//   out_t = scale ( exp(G_t) S q_t  +  sum_{s <= t} (q_t . k_s) exp(G_t - G_s) v_s )
//   S    <- exp(G_C) S + sum_s exp(G_C - G_s) v_s k_s^T
//
// where every exponent is <= 0, so nothing can overflow however strong the
// decay.  That is four products per chunk (Q K^T, P V, Q S, K^T V~) with
// V~_s = exp(G_C - G_s) v_s; only S goes from one chunk to the next, and the
// product that it waits for does not wait for it (S enters its own update
// elementwise), so a chunk's products run while the state of the one before
// is being finished.
//
// A CTA takes one (batch, head, 64 values) and a run of chunks; the keys' size
// is padded to 128 by the loads (zeros).  16 warps:
//   0      loads Q, K, V tiles by TMA, two chunks deep
//   1      issues the products (one thread)
//   2      the chunk's sums G, in double, stored as a float and its remainder:
//          differences of two sums keep float accuracy however large the sums
//   3      allocates tensor memory
//   4-7    scores: tensor memory -> exp(G_t - G_s), mask -> 16 bits -> tensor memory
//   8-11   V~, and the state: float32 in registers (lane = key, 64 values)
//   12-15  output
//
// Precision.  Accumulators and S are float32.  V~ and the S that Q S reads are
// given to the tensor cores as two 16-bit numbers, the second holding what
// rounding the first left over (16 bits of significand for bf16, 22 for f16): the state is
// a float32 result and remembers for long.  The scores are rounded once, as the
// output will be.  For f16, whose range is small, a power of two is taken out of every row of
// scores, of V~ and of S, and put back in float32: it costs three maxima.
//
// Few long sequences: with less than one CTA per SM, each is cut into pieces of
// chunks.  A first launch computes every piece's end state from zero (keys and
// values only), a second starts every piece from the states composed of those.
#include <type_traits>

#include "../../include/ssm_causal.h"
#include "common.cuh"
#include "problem.h"
#include "tcgen05.cuh"

namespace ssm {
namespace {

constexpr int kThreads = 512;
constexpr int C = 128;        // tokens per chunk
constexpr int DV = 64;        // values per CTA
constexpr int kBlockBytes = C * 128;               // a tile: 128 rows of 64 16-bit elements
constexpr int kStageBytes = 5 * kBlockBytes;       // Q (2 tiles), K (2), V (1)
constexpr int kOffVt = 2 * kStageBytes;            // V~ high, low
constexpr int kOffS = kOffVt + 2 * kBlockBytes;    // S high, low
constexpr int kTiles = kOffS + 2 * kBlockBytes;    // 229,376 bytes

struct Small {
    uint64_t full_qk[2], full_v[2], empty_qk[2], empty_v[2];  // loads
    uint64_t g_full[2], g_empty[2];                           // decay sums
    uint64_t sc_full[2], sc_empty[2];                         // scores' accumulators
    uint64_t p_full, vt_full, kv_full, s_full, qs_done, o_full, o_empty, red_full, spare;
    uint32_t tmem;
    int abort;
    float red[2][4];
    int s_lift[2];         // f16: S was divided by 2^s_lift
    int8_t row_lift[2][C]; // f16: a row of scores was divided by 2^row_lift
    alignas(16) float g_hi[2][C], g_lo[2][C];  // read as vectors
};
constexpr int kSmem = kTiles + sizeof(Small);
static_assert(kSmem <= 232448, "shared memory of one CTA");
static_assert(kTiles % 16 == 0, "alignment of the vectors behind the tiles");

// tensor memory columns
constexpr uint32_t kSc = 0, kP = 256, kOa = 320, kOb = 384, kKv = 448, kColumns = 512;

struct ChunkArgs {
    LinAttnProblem p;
    int64_t pt;          // ceil(P / 64)
    int64_t chunks;      // ceil(L / 128)
    int pieces;          // pieces per sequence
    int64_t per_piece;   // chunks per piece
    int states_only;     // first of two launches
    float* rec;          // [unit][S_0, ends of pieces 0 .. pieces - 2][64 values][128 keys]
    double* rec_g;       // [unit][pieces]: log2 of the piece's decay
    DeviceError* err;
    long long wait_budget;
};

// Bounded wait; a wait that runs out ends every role of the CTA.
struct Waiter {
    Small* sm;
    const ChunkArgs* a;
    // by one thread
    __device__ __forceinline__ bool one(uint64_t* bar, uint32_t parity) const {
        if (mbar_try(bar, parity)) return true;
        const long long t0 = clock64();
        for (;;) {
            if (mbar_try(bar, parity)) return true;
            if (*(volatile int*)&sm->abort) return false;
            if (clock64() - t0 > a->wait_budget) {
                *(volatile int*)&sm->abort = 1;
                report_device_error(a->err, SSM_KERNEL_LINATTN_CHUNK, (long long)blockIdx.x);
                return false;
            }
        }
    }
    // by a whole warp, with one answer
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, one(bar, parity));
    }
};

template <typename T> struct Half16;
template <> struct Half16<__half> {
    static constexpr uint32_t kType = 0;
    static constexpr bool kScaled = true;
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float2 back(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
};
template <> struct Half16<__nv_bfloat16> {
    static constexpr uint32_t kType = 1;
    static constexpr bool kScaled = false;
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float2 back(uint32_t u) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
    }
};

// e with top * 2^-e in [2^13, 2^14), where top >= 0 is finite and not 0 (else
// 0); limited so that 2^e and 2^-e are normal numbers.
__device__ __forceinline__ int lift_of(float top) {
    const int e = (int)(__float_as_uint(top) >> 23) - 127 - 13;
    return top > 0.0f && top < INFINITY ? min(max(e, -120), 120) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// two 16-bit numbers per value: f = hi + lo, for 8 values
template <typename T>
__device__ __forceinline__ void split8(const float* f, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = Half16<T>::two(f[2 * i], f[2 * i + 1]);
        const float2 b = Half16<T>::back(h[i]);
        l[i] = Half16<T>::two(f[2 * i] - b.x, f[2 * i + 1] - b.y);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
linattn_chunk_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ ChunkArgs a) {
    using HT = Half16<T>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Small& sm = *reinterpret_cast<Small*>(smem + kTiles);
    const LinAttnProblem& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_pieces = a.states_only ? a.pieces - 1 : a.pieces;
    const int64_t unit = blockIdx.x / n_pieces;
    const int piece = (int)(blockIdx.x - unit * n_pieces);
    const int64_t bh = unit / a.pt, b = bh / p.H, h = bh - b * p.H;
    const int p0 = (int)(unit - bh * a.pt) * DV;
    const bool outputs = !a.states_only;

    int64_t len = p.L;
    if (p.lens) {
        const int64_t n = p.lens[b * p.len_b];
        len = n < 0 ? 0 : (n < p.L ? n : p.L);
    }
    const int64_t seq_chunks = (len + C - 1) / C;
    const int64_t c0 = piece * a.per_piece;
    int64_t c1 = c0 + a.per_piece;
    if (c1 > seq_chunks) c1 = seq_chunks;
    const int n = c1 > c0 ? (int)(c1 - c0) : 0;  // this CTA's chunks

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.full_qk[i], 1);
            mbar_init(&sm.full_v[i], 1);
            mbar_init(&sm.empty_qk[i], 1);
            mbar_init(&sm.empty_v[i], 1);
            mbar_init(&sm.g_full[i], 1);
            mbar_init(&sm.g_empty[i], outputs ? 12 : 4);
            mbar_init(&sm.sc_full[i], 1);
            mbar_init(&sm.sc_empty[i], 4);
        }
        mbar_init(&sm.p_full, 4);
        mbar_init(&sm.vt_full, 4);
        mbar_init(&sm.kv_full, 1);
        mbar_init(&sm.s_full, 4);
        mbar_init(&sm.qs_done, 1);
        mbar_init(&sm.o_full, 1);
        mbar_init(&sm.o_empty, 4);
        mbar_init(&sm.red_full, 4);
        mbar_init(&sm.spare, 1);
        sm.abort = (smem_u32(smem) & 1023u) != 0;  // the swizzle counts from 1024-byte boundaries
        if (sm.abort) report_device_error(a.err, SSM_KERNEL_LINATTN_CHUNK, (long long)blockIdx.x);
        mbar_fence_init();
    }
    if (warp == 3) {
        tmem_alloc(&sm.tmem, kColumns);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    const Waiter wait{&sm, &a};
    const bool start = sm.abort == 0;
    auto q_tile = [&](int s) { return smem + s * kStageBytes; };
    auto k_tile = [&](int s) { return smem + s * kStageBytes + 2 * kBlockBytes; };
    auto v_tile = [&](int s) { return smem + s * kStageBytes + 4 * kBlockBytes; };

    if (warp == 0) {
        // ------------------------------------------------------------- loads --
        if (lane == 0 && start) {
            const int hk = (int)(h / p.rep);
            int issued = 0;
            for (int i = 0; i < n; ++i, ++issued) {
                const int s = i & 1;
                const uint32_t reuse = ((i >> 1) & 1) ^ 1;
                const int t = (int)((c0 + i) * C);
                if (i >= 2 && !wait.one(&sm.empty_qk[s], reuse)) break;
                mbar_arrive_expect_tx(&sm.full_qk[s], (outputs ? 4 : 2) * kBlockBytes);
                tma_load_4d(k_tile(s), &mk, 0, t, hk, (int)b, &sm.full_qk[s]);
                tma_load_4d(k_tile(s) + kBlockBytes, &mk, 64, t, hk, (int)b, &sm.full_qk[s]);
                if (outputs) {
                    tma_load_4d(q_tile(s), &mq, 0, t, hk, (int)b, &sm.full_qk[s]);
                    tma_load_4d(q_tile(s) + kBlockBytes, &mq, 64, t, hk, (int)b, &sm.full_qk[s]);
                }
                if (i >= 2 && !wait.one(&sm.empty_v[s], reuse)) {  // (its Q, K are in flight)
                    mbar_wait_bounded(&sm.full_qk[s], (i >> 1) & 1, a.wait_budget);
                    break;
                }
                mbar_arrive_expect_tx(&sm.full_v[s], kBlockBytes);
                tma_load_4d(v_tile(s), &mv, p0, t, (int)h, (int)b, &sm.full_v[s]);
            }
            if (*(volatile int*)&sm.abort)  // leave with no copy in flight
                for (int i = issued > 2 ? issued - 2 : 0; i < issued; ++i) {
                    mbar_wait_bounded(&sm.full_qk[i & 1], (i >> 1) & 1, a.wait_budget);
                    mbar_wait_bounded(&sm.full_v[i & 1], (i >> 1) & 1, a.wait_budget);
                }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- products --
        if (lane == 0 && start && n > 0) {
            constexpr uint32_t d_qk = mma_desc(HT::kType, false, false, 128, 128);
            constexpr uint32_t d_pv = mma_desc(HT::kType, false, true, 128, DV);
            constexpr uint32_t d_kv = mma_desc(HT::kType, true, true, 128, DV);
            const uint32_t base = smem_u32(smem);
            const uint64_t vt = tile_desc(base + kOffVt, kBlockBytes), st = tile_desc(base + kOffS, kBlockBytes);
            constexpr uint64_t kLow = kBlockBytes >> 4;   // the second number's tile
            auto qd = [&](int s) { return tile_desc(base + s * kStageBytes, kBlockBytes); };
            auto kd = [&](int s) { return tile_desc(base + s * kStageBytes + 2 * kBlockBytes, kBlockBytes); };
            auto vd = [&](int s) { return tile_desc(base + s * kStageBytes + 4 * kBlockBytes, kBlockBytes); };
            // depth step kk of an operand whose row elements are the depth: 32 bytes, 4 to a tile
            auto along = [](int kk) { return (uint64_t)((kk >> 2) * (kBlockBytes >> 4) + (kk & 3) * 2); };
            auto down = [](int kk) { return (uint64_t)kk * (2048 >> 4); };  // whose rows are: 16 rows
            auto qk = [&](int i) {
                const int s = i & 1;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(tm + kSc + s * 128, qd(s) + along(kk), kd(s) + along(kk), d_qk, kk > 0);
                mma_commit(&sm.sc_full[s]);
            };
            bool ok = true;
            if (outputs) {
                ok = wait.one(&sm.full_qk[0], 0);
                if (ok) qk(0);
            }
            for (int i = 0; ok && i < n; ++i) {
                const int s = i & 1;
                const uint32_t ph = (i >> 1) & 1;
                ok = wait.one(&sm.vt_full, i & 1) && wait.one(&sm.full_qk[s], ph);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 16; ++kk)
                    mma_ss(tm + kKv, kd(s) + down(kk & 7), vt + (kk >> 3) * kLow + down(kk & 7), d_kv, kk > 0);
                mma_commit(&sm.kv_full);
                if (!outputs) {
                    mma_commit(&sm.empty_qk[s]);
                    mma_commit(&sm.empty_v[s]);
                    continue;
                }
                ok = wait.one(&sm.s_full, i & 1) && (i == 0 || wait.one(&sm.o_empty, (i - 1) & 1));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 16; ++kk)
                    mma_ss(tm + kOb, qd(s) + along(kk & 7), st + (kk >> 3) * kLow + down(kk & 7), d_pv, kk > 0);
                mma_commit(&sm.qs_done);
                mma_commit(&sm.empty_qk[s]);
                // the next chunk's scores before this one's weighted values, if its tiles are here
                const int j = i + 1, js = j & 1;
                bool early = false;
                if (j < n) {
                    if (j >= 2) ok = wait.one(&sm.sc_empty[js], ((j >> 1) & 1) ^ 1);
                    if (!ok) break;
                    early = mbar_try(&sm.full_qk[js], (j >> 1) & 1);
                    if (early) qk(j);
                }
                ok = wait.one(&sm.p_full, i & 1) && wait.one(&sm.full_v[s], ph);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) mma_ts(tm + kOa, tm + kP + kk * 8, vd(s) + down(kk), d_pv, kk > 0);
                mma_commit(&sm.o_full);
                mma_commit(&sm.empty_v[s]);
                if (j < n && !early) {
                    ok = wait.one(&sm.full_qk[js], (j >> 1) & 1);
                    if (ok) qk(j);
                }
            }
            // every product done before tensor memory is freed
            mma_commit(&sm.spare);
            mbar_wait_bounded(&sm.spare, 0, a.wait_budget);
        }
    } else if (warp == 2) {
        // -------------------------------------------------------- decay sums --
        const float* g = p.g + b * p.g_b + h * p.g_h;
        for (int i = 0; start && i < n; ++i) {
            const int s = i & 1;
            const int64_t t0 = (c0 + i) * C + 4 * lane;
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = t0 + j < len ? g[(t0 + j) * p.g_t] : 0.0f;
                // exp(-256) is 0 in float32: below it only the sums' accuracy would suffer
                v[j] = v[j] > 0.0f ? 0.0f : (v[j] < -256.0f ? -256.0f : v[j]);
            }
            double x[4];
            x[0] = (double)v[0] * 1.4426950408889634;
#pragma unroll
            for (int j = 1; j < 4; ++j) x[j] = x[j - 1] + (double)v[j] * 1.4426950408889634;
            double incl = x[3];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const double before = incl - x[3];
            if (i >= 2) {
                if (!wait(&sm.g_empty[s], ((i >> 1) & 1) ^ 1)) break;
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double G = before + x[j];
                const float hi = (float)G;
                sm.g_hi[s][4 * lane + j] = hi;
                sm.g_lo[s][4 * lane + j] = (float)(G - (double)hi);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.g_full[s]);
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ scores --
        const int w = warp & 3, row = w * 32 + lane;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        for (int i = 0; start && outputs && i < n; ++i) {
            const int s = i & 1;
            const uint32_t ph = (i >> 1) & 1;
            if (!wait(&sm.g_full[s], ph) || !wait(&sm.sc_full[s], ph)) break;
            if (i > 0 && !wait(&sm.o_full, (i - 1) & 1)) break;  // the last weights are used up
            tc_fence_after();
            const float hi = sm.g_hi[s][row], lo = sm.g_lo[s][row];
            float lower = 1.0f;
            if (HT::kScaled) {
                float mx = 0.0f;
                for (int g = 0; g <= w; ++g) {
                    uint32_t r[32];
                    tmem_ld32(tm + lanes + kSc + s * 128 + g * 32, r);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (g < w || j <= lane) mx = fmaxf(mx, fabsf(__uint_as_float(r[j])));
                }
                const int e = lift_of(mx);
                lower = pow2(-e);
                sm.row_lift[s][row] = (int8_t)e;
            }
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                uint32_t out[16];
                if (g <= w) {
                    uint32_t r[32];
                    tmem_ld32(tm + lanes + kSc + s * 128 + g * 32, r);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 h4 = *reinterpret_cast<const float4*>(&sm.g_hi[s][g * 32 + j]);
                        const float4 l4 = *reinterpret_cast<const float4*>(&sm.g_lo[s][g * 32 + j]);
                        const float hs[4] = {h4.x, h4.y, h4.z, h4.w}, ls[4] = {l4.x, l4.y, l4.z, l4.w};
                        float e[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float d = ex2_approx((hi - hs[u]) + (lo - ls[u]));
                            float x = __uint_as_float(r[j + u]);
                            if (HT::kScaled) x *= lower;
                            e[u] = g < w || j + u <= lane ? x * d : 0.0f;
                        }
                        out[j / 2] = HT::two(e[0], e[1]);
                        out[j / 2 + 1] = HT::two(e[2], e[3]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[j] = 0u;
                }
                tmem_st16(tm + lanes + kP + g * 16, out);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.p_full);
                mbar_arrive(&sm.sc_empty[s]);
                mbar_arrive(&sm.g_empty[s]);
            }
        }
    } else if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------ V~ and state --
        const int w = warp & 3, row = w * 32 + lane;  // token of V~, key of the state
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        unsigned char* const vt = smem + kOffVt;
        unsigned char* const st = smem + kOffS;
        float S[DV];
        const bool key = row < p.N;
#pragma unroll
        for (int j = 0; j < DV; ++j)
            S[j] = p.s_in && key && p0 + j < p.P && (a.pieces == 1 || (a.states_only && piece == 0))
                       ? p.s_in[b * p.si_b + h * p.si_h + (p0 + j) * p.si_p + row * p.si_n] : 0.0f;
        float* const rec = a.rec + unit * a.pieces * (DV * C) + row;  // S_0, then each piece's end
        if (a.states_only && piece == 0) {
            // S_0 goes through the workspace: the second launch's last piece may
            // write state_out, in place, before another piece has begun
#pragma unroll
            for (int j = 0; j < DV; ++j) {
                rec[j * C] = S[j];
                S[j] = 0.0f;
            }
        }
        if (outputs && a.pieces > 1) {  // through the pieces before this one
#pragma unroll
            for (int j = 0; j < DV; ++j) S[j] = rec[j * C];
            for (int i = 0; i < piece; ++i) {
                const float f = (float)exp2(a.rec_g[unit * a.pieces + i]);
                const float* end = rec + (i + 1) * (DV * C);
#pragma unroll
                for (int j = 0; j < DV; ++j) S[j] = fmaf(f, S[j], end[j * C]);
            }
        }
        // the largest of the warpgroup's values (two places, used in turn)
        uint32_t reds = 0;
        auto wg_max = [&](float v, float& top) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(v));  // v >= 0: ordered as integers
            float* red = sm.red[reds & 1];
            if (lane == 0) {
                red[w] = __uint_as_float(m);
                mbar_arrive(&sm.red_full);
            }
            if (!wait(&sm.red_full, reds & 1)) return false;
            ++reds;
            top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
            return true;
        };
        auto put_state = [&](int i) {  // for the queries of chunk i
            float lower = 1.0f;
            if (HT::kScaled) {
                float mx = 0.0f;
#pragma unroll
                for (int j = 0; j < DV; ++j) mx = fmaxf(mx, fabsf(S[j]));
                if (!wg_max(mx, mx)) return false;
                const int e = lift_of(mx);
                lower = pow2(-e);
                if (row == 0) sm.s_lift[i & 1] = e;
            }
#pragma unroll
            for (int j = 0; j < DV; j += 8) {
                float f[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) f[u] = HT::kScaled ? S[j + u] * lower : S[j + u];
                uint4 hi, lo;
                split8<T>(f, hi, lo);
                const int at = row * 128 + (((j >> 3) ^ (row & 7)) << 4);
                *reinterpret_cast<uint4*>(st + at) = hi;
                *reinterpret_cast<uint4*>(st + kBlockBytes + at) = lo;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.s_full);
            return true;
        };
        bool ok = start;
        if (outputs && ok && n > 0) ok = put_state(0);
        double total = 0.0;
        for (int i = 0; ok && i < n; ++i) {
            const int s = i & 1;
            const uint32_t ph = (i >> 1) & 1;
            if (!wait(&sm.g_full[s], ph) || !wait(&sm.full_v[s], ph) || !wait(&sm.full_qk[s], ph)) break;
            const int64_t t0 = (c0 + i) * C;
            const bool there = t0 + row < len;
            unsigned char* vrow = v_tile(s) + row * 128;
            const float end_hi = sm.g_hi[s][C - 1], end_lo = sm.g_lo[s][C - 1];
            const float weight = ex2_approx((end_hi - sm.g_hi[s][row]) + (end_lo - sm.g_lo[s][row]));
            if (!there) {  // rows behind the end may hold anything
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    *reinterpret_cast<uint4*>(vrow + 16 * j) = zero;
                    *reinterpret_cast<uint4*>(k_tile(s) + row * 128 + 16 * j) = zero;
                    *reinterpret_cast<uint4*>(k_tile(s) + kBlockBytes + row * 128 + 16 * j) = zero;
                }
            }
            float lift = 1.0f, lower = 1.0f;
            if (HT::kScaled) {
                float mx = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float f[8];
                    Vec16<T>::unpack(*reinterpret_cast<const uint4*>(vrow + 16 * j), f);
#pragma unroll
                    for (int u = 0; u < 8; ++u) mx = fmaxf(mx, fabsf(f[u]));
                }
                if (!wg_max(mx * weight, mx)) break;
                const int e = lift_of(mx);
                lift = pow2(e);
                lower = pow2(-e);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = (j ^ (row & 7)) << 4;
                float f[8];
                Vec16<T>::unpack(*reinterpret_cast<const uint4*>(vrow + at), f);
#pragma unroll
                for (int u = 0; u < 8; ++u) f[u] *= HT::kScaled ? weight * lower : weight;
                uint4 hi, lo;
                split8<T>(f, hi, lo);
                *reinterpret_cast<uint4*>(vt + row * 128 + at) = hi;
                *reinterpret_cast<uint4*>(vt + kBlockBytes + row * 128 + at) = lo;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.vt_full);
                mbar_arrive(&sm.g_empty[s]);
            }
            // the decay over the chunk, as its distance from 1 where it is near 1: the
            // error of a factor near 1 would add up over the chunks S remembers
            const float log2_decay = end_hi + end_lo;
            total += (double)end_hi + (double)end_lo;
            const bool near1 = log2_decay > -1.0f;
            const float f = near1 ? expm1f(log2_decay * kLn2) : ex2_approx(log2_decay);
            if (!wait(&sm.kv_full, i & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t r[32];
                tmem_ld32(tm + lanes + kKv + g * 32, r);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float x = __uint_as_float(r[j]);
                    if (HT::kScaled) x *= lift;
                    float& sj = S[g * 32 + j];
                    sj = fmaf(f, sj, x) + (near1 ? sj : 0.0f);
                }
            }
            tc_fence_before();
            if (outputs && i + 1 < n) {
                if (!wait(&sm.qs_done, i & 1)) break;
                ok = put_state(i + 1);
            }
        }
        if (start && a.states_only) {
#pragma unroll
            for (int j = 0; j < DV; ++j) rec[(piece + 1) * (DV * C) + j * C] = S[j];
            if (row == 0) a.rec_g[unit * a.pieces + piece] = total;
        } else if (start && p.s_out && piece == a.pieces - 1 && key) {
#pragma unroll
            for (int j = 0; j < DV; ++j)
                if (p0 + j < p.P) p.s_out[b * p.so_b + h * p.so_h + (p0 + j) * p.so_p + row * p.so_n] = S[j];
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------ output --
        const int w = warp & 3, row = w * 32 + lane;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        T* const out = static_cast<T*>(p.out) + b * p.o_b + h * p.o_h + p0;
        for (int i = 0; start && outputs && i < n; ++i) {
            const int s = i & 1;
            if (!wait(&sm.g_full[s], (i >> 1) & 1)) break;
            float across = ex2_approx(sm.g_hi[s][row]) * p.scale, inside = p.scale;
            if (!wait(&sm.o_full, i & 1)) break;
            tc_fence_after();
            if (HT::kScaled) {
                across *= pow2(sm.s_lift[i & 1]);
                inside *= pow2(sm.row_lift[s][row]);
            }
            const int64_t t = (c0 + i) * C + row;
            T* const orow = out + t * p.o_t;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t x[32], y[32];
                tmem_ld32(tm + lanes + kOa + g * 32, x);
                tmem_ld32(tm + lanes + kOb + g * 32, y);
                if (g == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.o_empty);
                        mbar_arrive(&sm.g_empty[s]);
                    }
                }
                if (t < len) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        float f[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            f[u] = fmaf(__uint_as_float(y[j + u]), across, __uint_as_float(x[j + u]) * inside);
                        if (p0 + g * 32 + j < p.P) *reinterpret_cast<uint4*>(orow + g * 32 + j) = Vec16<T>::pack(f);
                    }
                }
            }
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_free(tm, kColumns);
}

// ------------------------------------------------------------------- host --
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// (batch, head, token, element) tensor as boxes of 64 elements by 128 tokens
bool make_map(CUtensorMap* m, int io_dt, const void* data, int64_t size, int64_t L, int64_t heads, int64_t batch,
              int64_t s_t, int64_t s_h, int64_t s_b) {
    const EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)size, (cuuint64_t)L, (cuuint64_t)heads, (cuuint64_t)batch};
    // a dimension of size 1 has no stride of its own; any valid one will do
    auto bytes = [](int64_t s, int64_t n) { return (cuuint64_t)(n == 1 ? 16 : s * 2); };
    const cuuint64_t strides[3] = {bytes(s_t, L), bytes(s_h, heads), bytes(s_b, batch)};
    const cuuint32_t box[4] = {64, (cuuint32_t)C, 1, 1}, step[4] = {1, 1, 1, 1};
    return enc(m, io_dt == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(data), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
cudaError_t launch_t(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const ChunkArgs& a, int64_t grid,
                     cudaStream_t s) {
    auto* fn = linattn_chunk_kernel<T>;
    int per_sm = 0;
    const cudaError_t e = prepared_launch(
        reinterpret_cast<const void*>(fn), kSmem, kThreads, &per_sm,
        [&](int smem) { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); },
        [&](int* n) { return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, fn, kThreads, kSmem); });
    if (e != cudaSuccess) return e;
    fn<<<(unsigned)grid, kThreads, kSmem, s>>>(mq, mk, mv, a);
    return cudaGetLastError();
}

}  // namespace

int linattn_chunk_block() { return kThreads; }
int linattn_chunk_smem() { return kSmem; }
int linattn_chunk_tokens() { return C; }
int linattn_chunk_values() { return DV; }
uint64_t linattn_chunk_record_bytes() { return DV * C * 4; }

cudaError_t launch_linattn_chunk(const LinAttnProblem& p, int64_t units, int pieces, int64_t per_piece, float* rec,
                                 double* rec_g, long long wait_budget, int dev, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, p.io_dt, p.q, p.N, p.L, p.Hk, p.Bn, p.q_t, p.q_h, p.q_b) ||
        !make_map(&mk, p.io_dt, p.k, p.N, p.L, p.Hk, p.Bn, p.k_t, p.k_h, p.k_b) ||
        !make_map(&mv, p.io_dt, p.v, p.P, p.L, p.H, p.Bn, p.v_t, p.v_h, p.v_b))
        return cudaErrorInvalidValue;
    ChunkArgs a{};
    a.p = p;
    a.pt = (p.P + DV - 1) / DV;
    a.chunks = (p.L + C - 1) / C;
    a.pieces = pieces;
    a.per_piece = per_piece;
    a.rec = rec;
    a.rec_g = rec_g;
    a.err = device_error_ptr(dev);
    if (!a.err) return cudaErrorUnknown;
    a.wait_budget = wait_budget;
    cudaError_t e = cudaSuccess;
    if (pieces > 1) {
        a.states_only = 1;
        e = p.io_dt == kF16 ? launch_t<__half>(mq, mk, mv, a, units * (pieces - 1), s)
                            : launch_t<__nv_bfloat16>(mq, mk, mv, a, units * (pieces - 1), s);
        if (e != cudaSuccess) return e;
        a.states_only = 0;
    }
    return p.io_dt == kF16 ? launch_t<__half>(mq, mk, mv, a, units * pieces, s)
                           : launch_t<__nv_bfloat16>(mq, mk, mv, a, units * pieces, s);
}

}  // namespace ssm
