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
// is padded to 128 by the loads (zeros).  20 warps:
//   0      loads Q, K, V tiles by TMA, two chunks deep
//   1, 3   issue the products (one thread each): P V and Q K^T, and those with the state
//   2      the chunk's sums G, in double, stored as a float and its remainder:
//          differences of two sums keep float accuracy however large the sums
//   4-7    scores: tensor memory -> exp(G_t - G_s), mask -> 16 bits -> tensor memory.
//          With R the sum at the end of s's 32 tokens, exp(G_t - G_s) =
//          exp(G_t - R) exp(R - G_s), a factor per row and one per column; an exponential
//          per element only where the 32 tokens of the diagonal decay by more than 2^100
//          (f16: or by more than 2^120 times a row's power of two, see below).  These warps
//          take the diagonal block of 32 columns and the one before it
//   8-11   the state: float32 in registers (lane = key, 64 values)
//   12-15  V~
//   16-19  the scores' other blocks, then the output
//
// Precision.  Accumulators and S are float32.  V~ is given to the tensor cores as
// several 16-bit numbers, each holding what rounding those before it left over (three
// for bf16: 24 bits of significand, two for f16: 22, down to 2^-28 of the chunk's largest), because
// the state is a float32 result and remembers for long.  The scores, and the copy of S that Q S reads, are
// rounded once, as the output will be.  For f16, whose range is small, a power of two is taken out of every row of
// scores, of V~ and of S, and put back in float32: it costs three maxima.
//
// Few long sequences: with half a CTA per SM or less, each is cut into pieces of
// chunks.  A first launch computes piece 0, and of the others but the last the end
// states from zero (keys and values only, which takes half as long: piece 0 is half as
// long as the others); a second starts pieces 1, 2, ... from the states composed of those.
#include <climits>
#include <type_traits>

#include "../../include/ssm_causal.h"
#include "common.cuh"
#include "problem.h"
#include "tcgen05.cuh"

namespace ssm {
namespace {

constexpr int kThreads = 640;
constexpr int C = 128;        // tokens per chunk
constexpr int DV = 64;        // values per CTA
constexpr int kBlockBytes = C * 128;               // a tile: 128 rows of 64 16-bit elements
constexpr int kStageBytes = 5 * kBlockBytes;       // Q (2 tiles), K (2), V (1)
constexpr int kOffS = 2 * kStageBytes;             // S
constexpr int kOffVt = kOffS + kBlockBytes;        // V~: Half16<T>::kParts tiles

template <typename T> struct Half16;
template <> struct Half16<__half> {
    static constexpr uint32_t kType = 0;
    static constexpr bool kScaled = true;
    static constexpr int kParts = 2;  // numbers that hold a value of V~
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float2 back(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
};
template <> struct Half16<__nv_bfloat16> {
    static constexpr uint32_t kType = 1;
    static constexpr bool kScaled = false;
    static constexpr int kParts = 3;
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float2 back(uint32_t u) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
    }
};

template <typename T>
struct Small {
    uint64_t full_qk[2], full_v[2], empty_qk[2], empty_v[2];  // loads
    uint64_t g_full[2], g_empty[2];                           // decay sums
    uint64_t sc_full, top_full;                               // scores' accumulator; f16: their largest
    uint64_t p_full, vt_full, kv_full, kv_empty, s_full, qs_done, o_full, o_empty, red_full[2], spare;
    uint64_t v_read[2], out_done, state_done, repaired, repair_sync;
    uint32_t tmem;
    int abort;
    int not_finite;            // the state at the end
    float part[4];             // of a sum, per warp
    int first[4];              // a token, per warp
    uint8_t red[2][2][4];      // f16: exponents of the largest values, per warp
    int s_lift[2], v_lift[2];  // f16: S, V~ were divided by 2^lift
    static constexpr int kRows = Half16<T>::kScaled ? C : 1;
    int8_t row_lift[2][kRows]; // f16: so was a row of scores
    uint8_t row_top[2][kRows]; // f16: exponent of a row's largest score, of either group
    alignas(16) float g_hi[2][C], column[2][C];  // read as vectors
    __half g_lo[2][C];         // remainder of g_hi, below 2^-24 of it
};
template <typename T>
struct Layout {
    static constexpr int kTiles = kOffVt + Half16<T>::kParts * kBlockBytes, kSmem = kTiles + (int)sizeof(Small<T>);
    static_assert(kSmem <= 232448, "shared memory of one CTA");
    static_assert(kTiles % 16 == 0, "alignment of the vectors behind the tiles");
};

// tensor memory columns
constexpr uint32_t kSc = 0, kP = 128, kOa = 192, kOb = 256, kKv = 320, kColumns = 512;
static_assert(kKv + Half16<__nv_bfloat16>::kParts * DV <= kColumns, "tensor memory of one CTA");

struct ChunkArgs {
    LinAttnProblem p;
    int64_t pt;          // ceil(P / 64)
    int pieces;          // pieces per sequence
    int64_t piece0, per_piece;  // chunks of piece 0, and of the others
    int phase;           // 0: one launch, 1: pieces 0 .. pieces - 2, 2: pieces 1 .. pieces - 1
    int out32;           // rows of out are whole, aligned 32-byte sectors
    float* rec;          // [unit][pieces - 1][64 values][128 keys]: end of the piece (from zero, but for 0)
    double* rec_g;       // [unit][pieces - 1]: log2 of the piece's decay
    DeviceError* err;
    BoundedWaits waits;
};

// Bounded wait; a wait that runs out ends every role of the CTA.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, int* abort, DeviceError* err, long long budget) {
    const long long t0 = clock64();
    for (;;) {
        if (mbar_try(bar, parity)) return true;
        if (*(volatile int*)abort) return false;
        if (clock64() - t0 > budget) {
            *(volatile int*)abort = 1;
            report_device_error(err, SSM_KERNEL_LINATTN_CHUNK, (long long)blockIdx.x);
            return false;
        }
    }
}
template <typename T>
struct Waiter {
    Small<T>* sm;
    const ChunkArgs* a;
    // by one thread
    __device__ __forceinline__ bool one(uint64_t* bar, uint32_t parity) const {
        return mbar_try(bar, parity) || wait_long(bar, parity, &sm->abort, a->err, a->waits.budget);
    }
    // by a whole warp, with one answer
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, one(bar, parity));
    }
};

// e with top * 2^-e in [2^13, 2^14), from the exponent field of top >= 0 (0 if top is 0 or not
// finite); limited so that 2^e and 2^-e are normal numbers.
__device__ __forceinline__ int lift_of(uint32_t exponent) {
    return exponent == 0 || exponent == 255 ? 0 : min(max((int)exponent - 127 - 13, -120), 120);
}
__device__ __forceinline__ uint32_t exponent_of(float v) { return __float_as_uint(v) >> 23 & 255u; }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 16-bit numbers that add up to a value, for a pair; f16: the second 2^11 times as large, so that
// it does not fall among the subnormals 2^11 before the first does
constexpr float kSecond = 2048.0f;
template <typename T>
__device__ __forceinline__ void split2(u64 f, uint32_t (&part)[Half16<T>::kParts]) {
#pragma unroll
    for (int i = 0; i < Half16<T>::kParts; ++i) {
        float x, y;
        upk(f, x, y);
        part[i] = Half16<T>::two(x, y);
        const float2 back = Half16<T>::back(part[i]);
        f = fsub2(f, pk(back.x, back.y));
        if (Half16<T>::kScaled) f = fmul2(f, pk(kSecond, kSecond));
    }
}

__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// What a CTA does.
struct Place {
    int64_t unit, b, h;
    int piece, p0;   // p0: first value
    int64_t len;     // tokens of the sequence
    int64_t c0;      // first chunk
    int chunks;
};
__device__ __forceinline__ Place place_of(const ChunkArgs& a, uint32_t block) {
    const LinAttnProblem& p = a.p;
    Place at;
    const int n_pieces = a.phase == 0 ? 1 : a.pieces - 1;
    at.unit = block / n_pieces;
    at.piece = (int)(block - at.unit * n_pieces) + (a.phase == 2 ? 1 : 0);
    const int64_t bh = at.unit / a.pt;
    at.b = bh / p.H;
    at.h = bh - at.b * p.H;
    at.p0 = (int)(at.unit - bh * a.pt) * DV;
    at.len = p.L;
    if (p.lens) {
        const int64_t n = p.lens[at.b * p.len_b];
        at.len = n < 0 ? 0 : (n < p.L ? n : p.L);
    }
    const int64_t seq_chunks = (at.len + C - 1) / C;
    at.c0 = at.piece == 0 ? 0 : a.piece0 + (at.piece - 1) * a.per_piece;
    int64_t c1 = at.piece == 0 ? a.piece0 : at.c0 + a.per_piece;
    if (c1 > seq_chunks) c1 = seq_chunks;
    at.chunks = c1 > at.c0 ? (int)(c1 - at.c0) : 0;
    return at;
}

// Registers per thread: 96 at launch (640 threads), of which the warpgroup that holds the
// state takes 128 and the others keep 88.
constexpr int kRegs = 88, kRegsState = 128;
static_assert(4 * kRegs + kRegsState <= 5 * 96, "no more than the launch has");
template <int R>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Code size: 20 warps run a dozen different loops, each once per chunk.  Unrolled
// throughout, they did not fit the instruction caches, and warps waited for
// instructions more than for anything else (10 of 26 stalled warps per issue; 237 us
// for 4 x 2048 tokens of 32 heads of 128).  So loops over blocks of 32 columns, and the one that
// makes V~, stay loops: 109 us (with V~ unrolled by 4 115, wholly 133).  One sequence of
// 16384 tokens, 32 heads over 8, f16, in pieces: 289 to 294 us.
template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
linattn_chunk_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ ChunkArgs a) {
    using HT = Half16<T>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Small<T>& sm = *reinterpret_cast<Small<T>*>(smem + Layout<T>::kTiles);
    const LinAttnProblem& p = a.p;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const Place at = place_of(a, blockIdx.x);
    const int64_t unit = at.unit, b = at.b, h = at.h, len = at.len, c0 = at.c0;
    const int piece = at.piece, p0 = at.p0, n = at.chunks;
    const bool outputs = a.phase != 1 || piece == 0;


    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.full_qk[i], 1);
            mbar_init(&sm.full_v[i], 1);
            mbar_init(&sm.empty_qk[i], outputs ? 2 : 1);  // both issuers
            mbar_init(&sm.empty_v[i], 5);                 // an issuer, and the warps that make V~
            mbar_init(&sm.g_full[i], 1);
            mbar_init(&sm.g_empty[i], outputs ? 16 : 8);
        }
        mbar_init(&sm.sc_full, 1);
        mbar_init(&sm.top_full, 8);
        mbar_init(&sm.p_full, 8);
        mbar_init(&sm.vt_full, 4);
        mbar_init(&sm.kv_full, 1);
        mbar_init(&sm.kv_empty, 4);
        mbar_init(&sm.s_full, 4);
        mbar_init(&sm.qs_done, 1);
        mbar_init(&sm.o_full, 2);
        mbar_init(&sm.o_empty, 4);
        mbar_init(&sm.red_full[0], 4);
        mbar_init(&sm.red_full[1], 4);
        mbar_init(&sm.v_read[0], 4);
        mbar_init(&sm.v_read[1], 4);
        mbar_init(&sm.out_done, 4);
        mbar_init(&sm.state_done, 4);
        mbar_init(&sm.repaired, 4);
        mbar_init(&sm.repair_sync, 4);
        sm.not_finite = 0;
        mbar_init(&sm.spare, outputs ? 2 : 1);
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
    const uint32_t tm = __shfl_sync(0xffffffffu, sm.tmem, 0);
    const Waiter<T> wait{&sm, &a};
    const bool start = sm.abort == 0;
    auto q_tile = [&](int s) { return smem + s * kStageBytes; };
    auto k_tile = [&](int s) { return smem + s * kStageBytes + 2 * kBlockBytes; };
    auto v_tile = [&](int s) { return smem + s * kStageBytes + 4 * kBlockBytes; };

    // the largest exponent in a warpgroup (group 0: the state's, 1: the values'), at its call i
    auto group_max = [&](float v, int group, int i, uint32_t& top) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, exponent_of(v));
        uint8_t* const red = sm.red[group][i & 1];
        if (lane == 0) {
            red[warp & 3] = (uint8_t)m;
            mbar_arrive(&sm.red_full[group]);
        }
        if (!wait(&sm.red_full[group], i & 1)) return false;
        top = max(max(red[0], red[1]), max(red[2], red[3]));
        return true;
    };

    if (warp < 4) fewer_registers<kRegs>();
    if (warp == 0) {
        // ------------------------------------------------------------- loads --
        if (lane == 0 && start) {
            const int hk = (int)(h / p.rep);
            int issued = 0;
            for (int i = 0; i < n; ++i, ++issued) {
#ifdef SSM_TEST_HOOKS
                if ((int64_t)blockIdx.x == a.waits.drop_item) break;  // never issued
#endif
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
                    mbar_wait_bounded(&sm.full_qk[s], (i >> 1) & 1, a.waits.budget);
                    break;
                }
                mbar_arrive_expect_tx(&sm.full_v[s], kBlockBytes);
                tma_load_4d(v_tile(s), &mv, p0, t, (int)h, (int)b, &sm.full_v[s]);
            }
            if (*(volatile int*)&sm.abort)  // leave with no copy in flight
                for (int i = issued > 2 ? issued - 2 : 0; i < issued; ++i) {
                    mbar_wait_bounded(&sm.full_qk[i & 1], (i >> 1) & 1, a.waits.budget);
                    mbar_wait_bounded(&sm.full_v[i & 1], (i >> 1) & 1, a.waits.budget);
                }
        }
    } else if (warp == 1 || warp == 3) {
        // ---------------------------------------------------------- products --
        // Two warps, so that the products of one can be issued while the other waits
        // for operands: the weights are made while the products with the state run, the
        // state is brought up to date during the others, and a stage is refilled two
        // steps after it was last read.
        constexpr uint32_t d_qk = mma_desc(HT::kType, false, false, 128, 128);
        constexpr uint32_t d_pv = mma_desc(HT::kType, false, true, 128, DV);
        constexpr uint32_t d_kv = mma_desc(HT::kType, true, true, 128, HT::kParts * DV);
        constexpr int kTile = kBlockBytes >> 4, kRows = 2048 >> 4;  // to the next 64 elements, 16 rows
        const uint32_t base = smem_u32(smem);
        auto qd = [&](int s) { return tile_desc(base + s * kStageBytes, kBlockBytes); };
        auto kd = [&](int s) { return tile_desc(base + s * kStageBytes + 2 * kBlockBytes, kBlockBytes); };
        auto vd = [&](int s) { return tile_desc(base + s * kStageBytes + 4 * kBlockBytes, kBlockBytes); };
        if (warp == 1 && start && outputs && n > 0) {
            for (int i = -1; i < n; ++i) {
                const int s = i & 1, j = i + 1, js = j & 1;
                if (i >= 0) {
                    // (V~ made: rows behind the end are 0 by then, in V too.  A barrier per stage:
                    // the next chunk's V~ may be made before this warp looks)
                    if (!wait(&sm.full_v[s], (i >> 1) & 1) || !wait(&sm.v_read[s], (i >> 1) & 1) || !wait(&sm.p_full, i & 1) ||
                        (i > 0 && !wait(&sm.o_empty, (i - 1) & 1)))
                        break;
                    tc_fence_after();
                    product_ts<kRows>(tm + kOa, tm + kP, vd(s), d_pv);
                    mma_commit(&sm.o_full);
                    mma_commit(&sm.empty_v[s]);
                }
                // the scores of the next chunk (the last ones were read when their weights were ready)
                if (j == n || !wait(&sm.full_qk[js], (j >> 1) & 1)) break;
                tc_fence_after();
                product_ss<2, kTile - 6, 2, kTile - 6>(tm + kSc, qd(js), kd(js), d_qk);
                mma_commit(&sm.sc_full);
                mma_commit(&sm.empty_qk[js]);
            }
        } else if (warp == 3 && start) {
            const uint64_t vt = tile_desc(base + kOffVt, kBlockBytes), st = tile_desc(base + kOffS, kBlockBytes);
            for (int i = 0; i < n; ++i) {
                const int s = i & 1;
                // K^T [V~'s parts] (side by side, added up by the state's warps) and Q S
                if (!wait(&sm.vt_full, i & 1) || !wait(&sm.full_qk[s], (i >> 1) & 1) ||
                    (i > 0 && !wait(&sm.kv_empty, (i - 1) & 1)))
                    break;
                tc_fence_after();
                product_ss<kRows, kRows, kRows, kRows>(tm + kKv, kd(s), vt, d_kv);
                mma_commit(&sm.kv_full);
                if (outputs) {
                    if (!wait(&sm.s_full, i & 1) || (i > 0 && !wait(&sm.o_empty, (i - 1) & 1))) break;
                    tc_fence_after();
                    product_ss<2, kTile - 6, kRows, kRows>(tm + kOb, qd(s), st, d_pv);
                    mma_commit(&sm.qs_done);
                    mma_commit(&sm.o_full);
                } else {
                    mma_commit(&sm.empty_v[s]);
                }
                mma_commit(&sm.empty_qk[s]);
            }
        }
        // every product done before tensor memory is freed
        if (start && n > 0 && (warp == 3 || outputs)) {
            mma_commit(&sm.spare);
            mbar_wait_bounded(&sm.spare, 0, a.waits.budget);
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
            // (not incl - x[3]: a NaN would reach the tokens before it)
            const double up = __shfl_up_sync(0xffffffffu, incl, 1), before = lane ? up : 0.0;
            // the sum at the end of this lane's 32 tokens
            const double end = __shfl_sync(0xffffffffu, incl, lane | 7);
            if (i >= 2) {
                if (!wait(&sm.g_empty[s], ((i >> 1) & 1) ^ 1)) break;
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double G = before + x[j];
                const float hi = (float)G;
                sm.g_hi[s][4 * lane + j] = hi;
                sm.g_lo[s][4 * lane + j] = __float2half_rn((float)(G - (double)hi));
                sm.column[s][4 * lane + j] = ex2_approx((float)(end - G));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.g_full[s]);
        }
    } else if ((warp >= 4 && warp < 8) || warp >= 16) {
        // ------------------------------------------------- scores and output --
        fewer_registers<kRegs>();
        const int w = warp & 3, row = w * 32 + lane, group = warp >= 16;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        // blocks of 32 columns: the diagonal and the one before it, or those before them
        const int split = w > 1 ? w - 1 : w, first = group ? 0 : split, last = group ? split : w + 1;
        T* const out = static_cast<T*>(p.out) + b * p.o_b + h * p.o_h + p0;
        auto output = [&](int i, float across) {  // across: scale exp(G_t)
            if (!wait(&sm.o_full, i & 1)) return false;
            tc_fence_after();
            float inside = p.scale, over = across;
            if (HT::kScaled) {
                over *= pow2(sm.s_lift[i & 1]);
                inside *= pow2(sm.row_lift[i & 1][row]);
            }
            const int64_t t = (c0 + i) * C + row;
            T* const orow = out + t * p.o_t;
            const u64 over2 = pk(over, over), inside2 = pk(inside, inside);
#pragma unroll 1
            for (int g = 0; g < DV; g += 16) {
                uint32_t x[16], y[16], o[8];
                tmem_ld16x2(tm + lanes + kOa + g, tm + lanes + kOb + g, x, y);
                if (g == DV - 16) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.o_empty);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    float f0, f1;
                    upk(ffma2(pk(__uint_as_float(y[j]), __uint_as_float(y[j + 1])), over2,
                              fmul2(pk(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), inside2)), f0, f1);
                    o[j / 2] = HT::two(f0, f1);
                }
                if (t < len && p0 + g < p.P) {
                    if (a.out32) {  // a whole 32-byte sector
                        store32(orow + g, o);
                    } else {
                        *reinterpret_cast<uint4*>(orow + g) = make_uint4(o[0], o[1], o[2], o[3]);
                        if (p0 + g + 8 < p.P) *reinterpret_cast<uint4*>(orow + g + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
            return true;
        };
        for (int i = 0; start && outputs && i < n; ++i) {
            const int s = i & 1;
            if (!wait(&sm.g_full[s], (i >> 1) & 1)) break;
            const float hi = sm.g_hi[s][row], lo = __half2float(sm.g_lo[s][row]);
            if (!wait(&sm.sc_full, i & 1)) break;
            tc_fence_after();
            const uint32_t sc = tm + lanes + kSc, pw = tm + lanes + kP;
            float lower = 1.0f;
            // (a product of the two factors on the diagonal is exact enough while the first,
            // which is above 1 there, and the second stay well inside float32)
            const float drop = sm.g_hi[s][w * 32] - sm.g_hi[s][w * 32 + 31];
            bool steep = !(drop <= 100.0f);  // (a NaN among the 32: earlier tokens must not meet R)
            if (HT::kScaled) {
                float mx = 0.0f;
#pragma unroll 1
                for (int g = first; g < last; ++g) {
                    uint32_t r[32];
                    tmem_ld32(sc + g * 32, r);
                    const int end = g < w ? 31 : lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j) mx = fmaxf(mx, j <= end ? fabsf(__uint_as_float(r[j])) : 0.0f);
                }
                sm.row_top[group][row] = (uint8_t)exponent_of(mx);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.top_full);
                if (!wait(&sm.top_full, i & 1)) break;
                const int e = lift_of(max(sm.row_top[0][row], sm.row_top[1][row]));
                lower = pow2(-e);
                sm.row_lift[s][row] = (int8_t)e;  // (both groups write the same)
                // the first factor holds the row's power of two as well, which is large where scores are small
                // (16384 tokens, 32 heads of 128, decays of 2^72 over 32 tokens: 288 us; steep from 2^60 on, 404)
                steep = __any_sync(0xffffffffu, steep || drop - (float)e > 120.0f);
            }
#pragma unroll 1
            for (int g = first; g < last; ++g) {
                uint32_t r[32], out[16];
                const int e = g * 32 + 31;
                const float f = ex2_approx((hi - sm.g_hi[s][e]) + (lo - __half2float(sm.g_lo[s][e]))) * lower;
                tmem_ld32(sc + g * 32, r);
                if (g == w && steep) {
#pragma unroll 1
                    for (int j = 0; j < 32; ++j) {
                        // element j of every lane's row, by rotating the registers
                        const float x = __uint_as_float(r[0]) * lower *
                                        ex2_approx((hi - sm.g_hi[s][w * 32 + j]) + (lo - __half2float(sm.g_lo[s][w * 32 + j])));
#pragma unroll
                        for (int u = 0; u < 31; ++u) r[u] = r[u + 1];
                        r[31] = __float_as_uint(x);
                    }
                } else {
                    const u64 f2 = pk(f, f);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 c4 = *reinterpret_cast<const float4*>(&sm.column[s][g * 32 + j]);
                        float x0, x1, x2, x3;
                        // (the two factors first: a column's, 2^-100 or so, would take a small score out of range)
                        upk(fmul2(fmul2(f2, pk(c4.x, c4.y)), pk(__uint_as_float(r[j]), __uint_as_float(r[j + 1]))), x0, x1);
                        upk(fmul2(fmul2(f2, pk(c4.z, c4.w)), pk(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]))), x2, x3);
                        r[j] = __float_as_uint(x0);
                        r[j + 1] = __float_as_uint(x1);
                        r[j + 2] = __float_as_uint(x2);
                        r[j + 3] = __float_as_uint(x3);
                    }
                }
                if (g == w) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = j <= lane ? r[j] : 0u;
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) out[j / 2] = HT::two(__uint_as_float(r[j]), __uint_as_float(r[j + 1]));
                tmem_st16(pw + g * 16, out);
            }
            if (group) {
#pragma unroll 1
                for (int g = w + 1; g < 4; ++g) {  // behind the diagonal
                    const uint32_t none[16] = {};
                    tmem_st16(pw + g * 16, none);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.p_full);
                mbar_arrive(&sm.g_empty[s]);
            }
            if (group && !output(i, ex2_approx(hi) * p.scale)) break;
        }
        __syncwarp();
        if (group && lane == 0) mbar_arrive(&sm.out_done);
    } else if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------------- state --
        more_registers<kRegsState>();
        const int w = warp & 3, row = w * 32 + lane;  // this thread's key
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        unsigned char* const st = smem + kOffS;
        float S[DV];
        const bool key = row < p.N;
        const int rows = (int)(p.P - p0 < DV ? p.P - p0 : DV);
        {
            // (unconditional loads of something valid, so that all are in flight at once)
            const bool given = p.s_in && key && piece == 0;
            const float* at = given ? p.s_in + b * p.si_b + h * p.si_h + p0 * p.si_p + row * p.si_n : p.g;
            const int64_t step = given ? p.si_p : 0;
#pragma unroll
            for (int j = 0; j < DV; ++j) {
                S[j] = *at;
                if (j + 1 < rows) at += step;
            }
#pragma unroll
            for (int j = 0; j < DV; ++j) S[j] = given && j < rows ? S[j] : 0.0f;
        }
        float* const rec = a.rec + unit * (a.pieces - 1) * (DV * C) + row;
        if (a.phase == 2) {  // through the pieces before this one
            const float* end = rec;
            float f = 0.0f;
#pragma unroll 1
            for (int i = 0;;) {
#pragma unroll
                for (int j = 0; j < DV; ++j) S[j] = fmaf(f, S[j], end[j * C]);
                if (++i == piece) break;
                f = exp2f((float)a.rec_g[unit * (a.pieces - 1) + i]);
                end += DV * C;
            }
        }
        auto put_state = [&](int i) {  // for the queries of chunk i
            float lower = 1.0f;
            if (HT::kScaled) {
                float mx;
                for (;;) {
                    mx = 0.0f;
#pragma unroll
                    for (int j = 0; j < DV; ++j) mx = fmaxf(mx, fabsf(S[j]));
                    if (mx < INFINITY) break;
                    // an infinity becomes a NaN, which a maximum passes over: what is not finite has no
                    // part in the scale.  (290 us at 16384 tokens; a second maximum, of what is finite, 295)
#pragma unroll
                    for (int j = 0; j < DV; j += 2) {
                        const u64 s2 = pk(S[j], S[j + 1]);
                        upk(ffma2(s2, 0, s2), S[j], S[j + 1]);
                    }
                }
                uint32_t top;
                if (!group_max(mx, 0, i, top)) return false;
                const int e = lift_of(top);
                lower = pow2(-e);
                if (row == 0) sm.s_lift[i & 1] = e;
            }
#pragma unroll
            for (int j = 0; j < DV; j += 8) {
                uint32_t x[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float f = S[j + 2 * u], g = S[j + 2 * u + 1];
                    x[u] = HT::kScaled ? HT::two(f * lower, g * lower) : HT::two(f, g);
                }
                *reinterpret_cast<uint4*>(st + row * 128 + (((j >> 3) ^ (row & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.s_full);
            return true;
        };
        double total = 0.0;
        int i = 0;
        for (; start && i < n; ++i) {
            const int s = i & 1;
            if (outputs && !((i == 0 || wait(&sm.qs_done, (i - 1) & 1)) && put_state(i))) break;
            if (!wait(&sm.g_full[s], (i >> 1) & 1)) break;
            // the decay over the chunk, as its distance from 1 where it is near 1: the
            // error of a factor near 1 would add up over the chunks S remembers
            const float end_hi = sm.g_hi[s][C - 1], end_lo = __half2float(sm.g_lo[s][C - 1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.g_empty[s]);
            const float log2_decay = end_hi + end_lo;
            total += (double)end_hi + (double)end_lo;
            const bool near1 = log2_decay > -1.0f;
            const float f = near1 ? expm1f(log2_decay * kLn2) : ex2_approx(log2_decay);
            if (!wait(&sm.kv_full, i & 1)) break;
            tc_fence_after();
            const float lift = HT::kScaled ? pow2(sm.v_lift[i & 1]) : 1.0f;
            const u64 lift2 = pk(lift, lift), f2 = pk(f, f);
#pragma unroll
            for (int g = 0; g < DV; g += 16) {
                uint32_t x[16], y[16], z[16];
                if (HT::kParts == 3)
                    tmem_ld16x3(tm + lanes + kKv + g, tm + lanes + kKv + DV + g, tm + lanes + kKv + 2 * DV + g, x, y, z);
                else
                    tmem_ld16x2(tm + lanes + kKv + g, tm + lanes + kKv + DV + g, x, y);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    u64 add = pk(__uint_as_float(y[j]), __uint_as_float(y[j + 1]));
                    const u64 first = pk(__uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                    if (HT::kScaled) {
                        add = fmul2(ffma2(add, pk(1.0f / kSecond, 1.0f / kSecond), first), lift2);
                    } else {
                        add = fadd2(fadd2(add, pk(__uint_as_float(z[j]), __uint_as_float(z[j + 1]))), first);
                    }
                    const u64 s2 = pk(S[g + j], S[g + j + 1]);
                    u64 to = ffma2(f2, s2, add);
                    if (near1) to = fadd2(to, s2);
                    upk(to, S[g + j], S[g + j + 1]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.kv_empty);
        }
        bool done = start && i == n;  // (no wait ran out)
        if (done && outputs && n > 0) {
            u64 zeros = 0;  // 0 times every number of S: a NaN if one is not finite
#pragma unroll
            for (int j = 0; j < DV; j += 2) zeros = ffma2(pk(S[j], S[j + 1]), 0, zeros);
            float z0, z1;
            upk(zeros, z0, z1);
            if (z0 + z1 != 0.0f) *(volatile int*)&sm.not_finite = 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.state_done);
            done = wait(&sm.state_done, 0);
            // (the repair works longer than a wait may take, and ends this one if it gives up)
            if (done && *(volatile int*)&sm.not_finite)
                done = __all_sync(0xffffffffu, wait_long(&sm.repaired, 0, &sm.abort, a.err, DV * a.waits.budget));
        }
        if (!done) {  // nothing to hand on
        } else if (a.phase == 1) {
#pragma unroll
            for (int j = 0; j < DV; ++j) rec[piece * (DV * C) + j * C] = S[j];
            if (row == 0) a.rec_g[unit * (a.pieces - 1) + piece] = total;
        } else if (p.s_out && piece == a.pieces - 1 && key) {
            float* at = p.s_out + b * p.so_b + h * p.so_h + p0 * p.so_p + row * p.so_n;
#pragma unroll
            for (int j = 0; j < DV; ++j) {
                if (j < rows) *at = S[j];
                at += p.so_p;
            }
        }
    } else if (warp >= 12 && warp < 16) {
        // ---------------------------------------------------------------- V~ --
        fewer_registers<kRegs>();
        const int w = warp & 3, row = w * 32 + lane;  // this thread's token
        unsigned char* const vt = smem + kOffVt;
        auto values = [&](int i) {
            const int s = i & 1;
            const uint32_t ph = (i >> 1) & 1;
            if (!wait(&sm.g_full[s], ph) || !wait(&sm.full_v[s], ph) || !wait(&sm.full_qk[s], ph)) return false;
            unsigned char* const vrow = v_tile(s) + row * 128;
            const float hi = sm.g_hi[s][row], lo = __half2float(sm.g_lo[s][row]);
            const float weight = ex2_approx((sm.g_hi[s][C - 1] - hi) + (__half2float(sm.g_lo[s][C - 1]) - lo));
            if ((c0 + i) * C + row >= len) {  // rows behind the end may hold anything
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                for (int j = 0; j < 8; ++j) {
                    *reinterpret_cast<uint4*>(vrow + 16 * j) = zero;
                    *reinterpret_cast<uint4*>(k_tile(s) + row * 128 + 16 * j) = zero;
                    *reinterpret_cast<uint4*>(k_tile(s) + kBlockBytes + row * 128 + 16 * j) = zero;
                }
            }
            float factor = weight;
            int lift = 0;
            if (HT::kScaled) {
                float mx = 0.0f;
#pragma unroll 2
                for (int j = 0; j < 8; ++j) {
                    float f[8];
                    Vec16<T>::unpack(*reinterpret_cast<const uint4*>(vrow + ((j ^ (row & 7)) << 4)), f);
#pragma unroll
                    for (int u = 0; u < 8; ++u) mx = fmaxf(mx, fabsf(f[u]));
                }
                if (mx == INFINITY) {  // (a NaN does not count as it is)
                    mx = 0.0f;
#pragma unroll 1
                    for (int j = 0; j < DV; ++j) {
                        const float f = fabsf(to_f<T>(reinterpret_cast<const T*>(vrow)[j]));
                        if (f < INFINITY) mx = fmaxf(mx, f);
                    }
                }
                uint32_t top;
                if (!group_max(mx * weight, 1, i, top)) return false;
                lift = lift_of(top);
                factor = weight * pow2(-lift);
            }
            // the products with the last V~ are over
            if (i > 0 && !wait(&sm.kv_full, (i - 1) & 1)) return false;
            if (HT::kScaled && row == 0) sm.v_lift[i & 1] = lift;
            const u64 factor2 = pk(factor, factor);
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                const int at = (j ^ (row & 7)) << 4;
                float f[8];
                Vec16<T>::unpack(*reinterpret_cast<const uint4*>(vrow + at), f);
                uint32_t part[4][HT::kParts];
#pragma unroll
                for (int u = 0; u < 4; ++u) split2<T>(fmul2(factor2, pk(f[2 * u], f[2 * u + 1])), part[u]);
#pragma unroll
                for (int u = 0; u < HT::kParts; ++u)
                    *reinterpret_cast<uint4*>(vt + u * kBlockBytes + row * 128 + at) =
                        make_uint4(part[0][u], part[1][u], part[2][u], part[3][u]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.vt_full);
                mbar_arrive(&sm.v_read[s]);
                mbar_arrive(&sm.empty_v[s]);
                mbar_arrive(&sm.g_empty[s]);
            }
            return true;
        };
        int syncs = 0;
        // the four warps of this group, waiting for one another
        auto sync = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.repair_sync);
            return wait(&sm.repair_sync, syncs++ & 1);
        };
        // A weight of 0 does not keep a NaN or an infinity of V from the tokens before it
        // in a product: its column is NaN from the first token of its chunk on, and so is the
        // state.  When the state ends up like that, the outputs between that token and the
        // first value that is not finite are computed again, token by token (before the new
        // state is written, which may be where the old one is).  Looking at every value of V
        // instead took 4 to 8% of the kernel's time, in whichever warps; this takes 2 to 3.
        auto repair = [&] {
            if (!wait(&sm.out_done, 0)) return false;
            // (found again: kept, these would take registers from the loops above)
            uint32_t block;
            asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(block));
            const Place at = place_of(a, block);
            const int64_t unit = at.unit, b = at.b, h = at.h, end = (at.c0 + at.chunks) * C;
            const int piece = at.piece, p0 = at.p0, t0 = (int)(at.c0 * C), t1 = (int)(end < at.len ? end : at.len);
            const int64_t hk = h / p.rep;
            const int rows = (int)(p.P - p0 < DV ? p.P - p0 : DV);
            const bool key = row < p.N;  // (row: a key here)
            const float* const rec = a.rec + unit * (a.pieces - 1) * (DV * C) + row;
            const T* const k = static_cast<const T*>(p.k) + b * p.k_b + hk * p.k_h + row;
            const T* const q = static_cast<const T*>(p.q) + b * p.q_b + hk * p.q_h + row;
            const float* const g = p.g + b * p.g_b + h * p.g_h;
#pragma unroll 1
            for (int j = 0; j < rows; ++j) {
                const T* const v = static_cast<const T*>(p.v) + b * p.v_b + h * p.v_h + p0 + j;
                int bad = INT_MAX;
                for (int t = t0 + row; t < t1 && bad == INT_MAX; t += C)
                    if (!(fabsf(to_f<T>(v[t * p.v_t])) < INFINITY)) bad = t;
                bad = __reduce_min_sync(0xffffffffu, bad);
                if (lane == 0) sm.first[w] = bad;
                if (!sync()) return false;
                bad = min(min(sm.first[0], sm.first[1]), min(sm.first[2], sm.first[3]));
                if (!sync()) return false;
                const int chunk = bad / C * C;
                if (bad == INT_MAX || bad == chunk) continue;
                float s = 0.0f;
                if (p.s_in && key && piece == 0) s = p.s_in[b * p.si_b + h * p.si_h + (p0 + j) * p.si_p + row * p.si_n];
                if (a.phase == 2)
                    for (int i = 0; i < piece; ++i)
                        s = fmaf(i == 0 ? 0.0f : exp2f((float)a.rec_g[unit * (a.pieces - 1) + i]), s,
                                 rec[(int64_t)(i * DV + j) * C]);
                auto token = [&](int t) {
                    const float decay = g[t * p.g_t];
                    s = fmaf(to_f<T>(v[t * p.v_t]), key ? to_f<T>(k[t * p.k_t]) : 0.0f,
                             expf(decay > 0.0f ? 0.0f : decay) * s);
                };
#pragma unroll 8
                for (int t = t0; t < chunk; ++t) token(t);
#pragma unroll 1
                for (int t = chunk; t < bad; ++t) {
                    token(t);
                    float sum = key ? s * to_f<T>(q[t * p.q_t]) : 0.0f;
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0) sm.part[w] = sum;
                    if (!sync()) return false;
                    if (row == 0)
                        static_cast<T*>(p.out)[b * p.o_b + h * p.o_h + t * p.o_t + p0 + j] =
                            from_f<T>(((sm.part[0] + sm.part[1]) + (sm.part[2] + sm.part[3])) * p.scale);
                    if (!sync()) return false;
                }
            }
            return true;
        };
        int i = 0;
        while (start && i < n && values(i)) ++i;
        if (outputs && n > 0 && i == n && wait(&sm.state_done, 0) && *(volatile int*)&sm.not_finite && repair()) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.repaired);
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
    constexpr int kSmem = Layout<T>::kSmem;
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
int linattn_chunk_smem(int io_dt) { return io_dt == kF16 ? Layout<__half>::kSmem : Layout<__nv_bfloat16>::kSmem; }
int linattn_chunk_tokens() { return C; }
int linattn_chunk_values() { return DV; }
uint64_t linattn_chunk_record_bytes() { return DV * C * 4; }

cudaError_t launch_linattn_chunk(const LinAttnProblem& p, int64_t units, const LinAttnPieces& cut, float* rec, double* rec_g,
                                 const BoundedWaits& waits, int dev, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, p.io_dt, p.q, p.N, p.L, p.Hk, p.Bn, p.q_t, p.q_h, p.q_b) ||
        !make_map(&mk, p.io_dt, p.k, p.N, p.L, p.Hk, p.Bn, p.k_t, p.k_h, p.k_b) ||
        !make_map(&mv, p.io_dt, p.v, p.P, p.L, p.H, p.Bn, p.v_t, p.v_h, p.v_b))
        return cudaErrorInvalidValue;
    ChunkArgs a{};
    a.p = p;
    a.pt = (p.P + DV - 1) / DV;
    a.pieces = cut.pieces;
    a.piece0 = cut.piece0;
    a.per_piece = cut.per_piece;
    a.rec = rec;
    a.rec_g = rec_g;
    a.out32 = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.P % 16 == 0 && p.o_b % 16 == 0 && p.o_h % 16 == 0 &&
              p.o_t % 16 == 0;
    a.err = device_error_ptr(dev);
    if (!a.err) return cudaErrorUnknown;
    a.waits = waits;
    const bool f16 = p.io_dt == kF16;
    const int64_t grid = cut.pieces > 1 ? units * (cut.pieces - 1) : units;
    if (cut.pieces > 1) {
        a.phase = 1;
        const cudaError_t e = f16 ? launch_t<__half>(mq, mk, mv, a, grid, s) : launch_t<__nv_bfloat16>(mq, mk, mv, a, grid, s);
        if (e != cudaSuccess) return e;
        a.phase = 2;
    }
    return f16 ? launch_t<__half>(mq, mk, mv, a, grid, s) : launch_t<__nv_bfloat16>(mq, mk, mv, a, grid, s);
}

}  // namespace ssm
