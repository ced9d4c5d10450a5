// paged.cu -- attention of one new token per sequence over a paged key-value
// cache, split over the length and joined, for sm_100a.
//
//   p[t] = exp(x[t] - m) / l,  x[t] = scale * q . k[t],  m = max x,  l = sum exp(x - m)
//   out  = sum_t p[t] v[t]
//
// One pass over the keys and values with the running maximum and sum of the
// softmax: each key and value row is read once for all query heads of its
// group, so the bound is the cache's bytes (2 D elements per token and
// key-value head), as long as the group's arithmetic stays below it.
//
// Split.  The (sequence, 64 tokens) tiles of all sequences form one list, cut
// into `workers` equal ranges; a CTA takes one range for one (key-value head,
// block of query heads).  Every CTA finds its range from seq_lens itself (a
// prefix sum over the batch), so the lengths never travel to the host, and a
// batch of one long and many short sequences is as balanced as an even one.
// A range that holds a whole sequence writes its output; a part of a sequence
// leaves (maximum, sum, weighted values) in the workspace -- at most two such
// parts per range, its first and its last -- and paged_join_kernel joins them,
// in the order of the ranges, so results do not depend on timing.
//
// 64 sequences of up to 8192 tokens, 32 heads over 8 of 128, bf16: 180 to 190 us, 0.89 to 0.94 of
// a plain copy's rate.  16 sequences of up to 12000, 8 heads of 64, f16, with weights: 54 us, of
// which the first kernel takes 47 (38 without the scores it then leaves), 31 at a copy's rate.
//
// The scores' maximum and sums, the weighted values and all partial results are
// float32.  On the tensor cores the weights p are rounded to the cache's type (their
// sum is of unrounded ones); for groups of up to 8 heads the 8 rows of the matrix
// instruction that would be empty carry the rounding's remainder, itself rounded: a weight
// is off by 2^-16 (bf16) or 2^-22 (f16) of itself at most, in larger groups by 2^-8 or
// 2^-11; f16 weights by 2^-39 of the largest if that is more.
#include <type_traits>

#include "../../include/ssm_causal.h"
#include "common.cuh"
#include "problem.h"

namespace ssm {
namespace {

constexpr int kBlock = 128;
constexpr int kWarps = kBlock / 32;
constexpr int kTile = 64;  // tokens per tile of the work list
constexpr float kNegInf = -INFINITY;

// the larger of two, a NaN if either is one (a score that is a NaN makes its row one)
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Dependent launches: the join and the weights' kernel are launched while the one before
// still runs (its CTAs need not have finished for theirs to start) and wait
// here for its results.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------ work ranges --
struct Range {
    int64_t total;   // tiles of all sequences
    int64_t start, end;  // this worker's tiles
    int64_t b, c;    // the sequence that holds `start`, and its first tile
};

__device__ __forceinline__ int64_t seq_len(const PagedProblem& p, int64_t b) {
    const int64_t n = p.lens[b * p.len_b];
    return n < 0 ? 0 : (n < p.cap ? n : p.cap);
}
__device__ __forceinline__ int64_t seq_tiles(const PagedProblem& p, int64_t b) {
    return (seq_len(p, b) + kTile - 1) / kTile;
}
// Equal ranges: the first `more` workers take one tile more than the others.
struct Cut {
    int64_t each, more;
    __device__ __forceinline__ Cut(int64_t total, int64_t workers) {
        if (total < ((int64_t)1 << 32)) {  // (a 64-bit division takes much longer)
            each = (uint32_t)total / (uint32_t)workers;
        } else {
            each = total / workers;
        }
        more = total - each * workers;
    }
    __device__ __forceinline__ int64_t start(int64_t w) const { return w * each + (w < more ? w : more); }
    // the worker whose range holds tile x
    __device__ __forceinline__ int64_t worker_of(int64_t x) const {
        const int64_t longer = more * (each + 1);
        return x < longer ? x / (each + 1) : more + (x - longer) / each;
    }
};

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* sh) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sh[i];
    __syncthreads();
    return v;
}

// All threads: this worker's range, and the sequence its first tile lies in
// (worker < 0: total only; b = Bn if the range is empty).
__device__ Range find_range(const PagedProblem& p, int64_t worker) {
    __shared__ int64_t sh[kWarps + 2];
    Range r;
    int64_t mine = 0;
    for (int64_t b = threadIdx.x; b < p.Bn; b += kBlock) mine += seq_tiles(p, b);
    r.total = block_sum(mine, sh);
    const Cut cut(r.total, p.workers);
    r.start = cut.start(worker);
    r.end = cut.start(worker + 1);
    r.b = p.Bn;
    r.c = 0;
    if (r.start >= r.end) return r;
    int64_t base = 0;
    for (int64_t b0 = 0; b0 < p.Bn; b0 += kBlock) {
        const int64_t b = b0 + threadIdx.x;
        const int64_t n = b < p.Bn ? seq_tiles(p, b) : 0;
        int64_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if ((threadIdx.x & 31) >= o) incl += up;
        }
        if ((threadIdx.x & 31) == 31) sh[threadIdx.x >> 5] = incl;
        if (threadIdx.x == 0) sh[kWarps] = -1;
        __syncthreads();
        int64_t before = base, all = base;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < (int)(threadIdx.x >> 5)) before += sh[i];
            all += sh[i];
        }
        const int64_t c = before + incl - n;
        if (n > 0 && c <= r.start && r.start < c + n) {  // one thread at most
            sh[kWarps] = b;
            sh[kWarps + 1] = c;
        }
        __syncthreads();
        const int64_t found = sh[kWarps];
        r.c = sh[kWarps + 1];
        __syncthreads();
        if (found >= 0) {
            r.b = found;
            return r;
        }
        base = all;
    }
    return r;  // not reached: every tile lies in a sequence
}

// ------------------------------------------------- joining within a CTA --
// What a warp has of one segment: for query row r the maximum its weights are
// relative to (log2 units), their sum, and D weighted values, put in shared memory by the warp and joined by
// the whole CTA into the output or into the workspace.
template <int HPB, int DP>
struct Join {
    float o[kWarps][HPB][DP + 4];  // + 4: rows start in different banks
    float m[kWarps][HPB], l[kWarps][HPB];
};

template <typename T, int HPB, int DP>
__device__ void write_segment(const PagedProblem& p, Join<HPB, DP>& sm, int64_t b, int64_t hk, int hblk, int heads,
                              bool whole, int64_t part) {
    __syncthreads();
    for (int i = threadIdx.x; i < heads * DP; i += kBlock) {
        const int r = i / DP, d = i - r * DP;
        float m = kNegInf;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = max_nan(m, sm.m[w][r]);
        float acc = 0.0f, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm.m[w][r] == kNegInf ? 0.0f : exp2f(sm.m[w][r] - m);
            if (sm.m[w][r] != kNegInf) {
                acc = fmaf(f, sm.o[w][r][d], acc);
                l = fmaf(f, sm.l[w][r], l);
            }
        }
        const int64_t hq = hk * p.G + (int64_t)hblk * p.hpb + r;
        if (whole) {
            if (d < p.D)
                static_cast<T*>(p.out)[b * p.o_b + hq * p.o_h + d * p.o_d] =
                    from_f<T>(m == kNegInf ? 0.0f : acc / l);
            if (d == 0) {
                const float lse2 = m == kNegInf ? kNegInf : m + log2f(l);
                if (p.lse) p.lse[b * p.lse_b + hq * p.lse_h] = lse2 * kLn2;
                if (p.w) p.ws_lse2[b * p.Hq + hq] = lse2;
            }
        } else {
            if (d < p.D) p.ws_o[(part * p.hpb + r) * p.D + d] = acc;
            if (d == 0) p.ws_ml[part * p.hpb + r] = make_float2(m, l);
        }
    }
    __syncthreads();
}

// the workspace entry of a part: `last` = it is not its worker's first segment
__device__ __forceinline__ int64_t part_of(const PagedProblem& p, int64_t worker, int64_t hk, int hblk, int last) {
    return ((worker * p.Hkv + hk) * p.hblocks + hblk) * 2 + last;
}

// Walks a worker's segments: body(b, first token, end token), then write_segment.
template <typename T, int HPB, int DP, typename Body>
__device__ __forceinline__ void for_segments(const PagedProblem& p, Join<HPB, DP>& sm, Body body) {
    const int64_t worker = blockIdx.x;
    const int64_t hk = blockIdx.y / p.hblocks;
    const int hblk = (int)(blockIdx.y - hk * p.hblocks);
    const int heads = (int)(p.G - (int64_t)hblk * p.hpb < p.hpb ? p.G - (int64_t)hblk * p.hpb : p.hpb);
    let_next_kernel_start();
    const Range r = find_range(p, worker);
    int64_t at = r.start, c = r.c;
    for (int64_t b = r.b; at < r.end; ++b) {
        const int64_t n = seq_tiles(p, b);
        if (n == 0) continue;
        const int64_t to = c + n < r.end ? c + n : r.end;
        const int64_t len = seq_len(p, b);
        const int64_t t0 = (at - c) * kTile, t1 = (to - c) * kTile < len ? (to - c) * kTile : len;
        body(b, hk, hblk, heads, (int)t0, (int)t1);
        write_segment<T>(p, sm, b, hk, hblk, heads, at == c && to == c + n,
                         part_of(p, worker, hk, hblk, at == r.start ? 0 : 1));
        at = to;
        c += n;
    }
}

// ------------------------------------------------------- any type, strides --
// Float32 arithmetic: a warp takes tokens t0 + warp, t0 + warp + 4, ..., U at a
// time, its lanes the D elements of a row; the U * HPB dot products are
// reduced together, then every lane weighs its own elements.
constexpr int kGenHeads = 4, kGenTokens = 4;

template <typename T, int DE>
__global__ void __launch_bounds__(kBlock) paged_generic_kernel(const PagedProblem p) {
    constexpr int HPB = kGenHeads, U = kGenTokens;
    __shared__ Join<HPB, 32 * DE> sm;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* q = static_cast<const T*>(p.q);
    const T* k = static_cast<const T*>(p.k);
    const T* v = static_cast<const T*>(p.v);
    for_segments<T>(p, sm, [&](int64_t b, int64_t hk, int hblk, int heads, int t0, int t1) {
        float qf[HPB][DE], o[HPB][DE], m[HPB], l[HPB];
#pragma unroll
        for (int g = 0; g < HPB; ++g) {
            m[g] = kNegInf;
            l[g] = 0.0f;
            const int64_t hq = hk * p.G + (int64_t)hblk * HPB + g;
#pragma unroll
            for (int i = 0; i < DE; ++i) {
                const int64_t d = lane + 32 * i;
                o[g][i] = 0.0f;
                qf[g][i] = g < heads && d < p.D ? to_f<T>(q[b * p.q_b + hq * p.q_h + d * p.q_d]) : 0.0f;
            }
        }
        for (int t = t0 + warp * U; t < t1; t += kWarps * U) {
            float kf[U][DE], vf[U][DE];
            bool on[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                int64_t pg = -1;
                if (t + u < t1) pg = p.table[b * p.tb_b + (int64_t)((t + u) / p.page) * p.tb_m];
                on[u] = pg >= 0 && pg < p.pages;
                const int row = (t + u) % p.page;
                const int64_t ko = pg * p.k_g + row * p.k_t + hk * p.k_h, vo = pg * p.v_g + row * p.v_t + hk * p.v_h;
#pragma unroll
                for (int i = 0; i < DE; ++i) {
                    const int64_t d = lane + 32 * i;
                    kf[u][i] = on[u] && d < p.D ? to_f<T>(k[ko + d * p.k_d]) : 0.0f;
                    vf[u][i] = on[u] && d < p.D ? to_f<T>(v[vo + d * p.v_d]) : 0.0f;
                }
            }
            float x[U][HPB];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int g = 0; g < HPB; ++g) {
                    float a = 0.0f;
#pragma unroll
                    for (int i = 0; i < DE; ++i) a = fmaf(qf[g][i], kf[u][i], a);
#pragma unroll
                    for (int s = 16; s >= 1; s >>= 1) a += __shfl_xor_sync(0xffffffffu, a, s);
                    x[u][g] = on[u] ? a * p.scale_log2 : kNegInf;
                }
            if (p.w) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int g = 0; g < HPB; ++g)
                        if (lane == u * HPB + g && t + u < t1 && g < heads)
                            p.ws_s[(b * p.Hq + hk * p.G + (int64_t)hblk * HPB + g) * p.ws_cap + t + u] = x[u][g];
            }
#pragma unroll
            for (int g = 0; g < HPB; ++g) {
                float mn = m[g];
#pragma unroll
                for (int u = 0; u < U; ++u) mn = max_nan(mn, x[u][g]);
                if (mn == kNegInf) continue;  // nothing yet
                const float f = m[g] == kNegInf ? 0.0f : exp2f(m[g] - mn);
                float pw[U];
#pragma unroll
                for (int u = 0; u < U; ++u) pw[u] = on[u] ? exp2f(x[u][g] - mn) : 0.0f;
                l[g] *= f;
#pragma unroll
                for (int u = 0; u < U; ++u) l[g] += pw[u];
#pragma unroll
                for (int i = 0; i < DE; ++i) {
                    o[g][i] *= f;
#pragma unroll
                    for (int u = 0; u < U; ++u) o[g][i] = fmaf(pw[u], vf[u][i], o[g][i]);
                }
                m[g] = mn;
            }
        }
#pragma unroll
        for (int g = 0; g < HPB; ++g) {
            if (lane == 0) {
                sm.m[warp][g] = m[g];
                sm.l[warp][g] = l[g];
            }
#pragma unroll
            for (int i = 0; i < DE; ++i) sm.o[warp][g][lane + 32 * i] = o[g][i];
        }
    });
}

// ------------------------------------------------------------ tensor cores --
// 16-bit types.  A warp takes 16 tokens at a time with m16n8k16 products whose
// operands come straight from global memory as 16-byte vectors, nothing staged:
//
//   scores  rows = query heads, columns = tokens, depth = d.  The order of d in
//           a sum is free, so lane (r, c) = (lane / 4, lane % 4) takes
//           q[r][32 i + 8 c ..] and k[token r][32 i + 8 c ..], and its 8 elements are
//           its fragments of two products' depth.
//   values  rows = heads, columns = d, depth = tokens.  The weights come out of the
//           scores' accumulators in the layout the left operand wants; the
//           right operand wants pairs of tokens, so a lane loads 8 elements of
//           4 tokens (2c, 2c+1, 2c+8, 2c+9), d = 64 i + 8 r + j, and pairs them
//           with byte permutes: product j of slab i has columns d = 64 i + 8 n + j.
//
// WIDE: 16 query heads per CTA.  Else 8, and rows 8..15 of the weights hold what
// rounding them to 16 bits left over.  Decode has a few rows against a whole cache:
// tcgen05's tiles of 64 or 128 rows would be all padding, and the bound is HBM.
template <typename T> struct Pack;
template <> struct Pack<__half> {
    // weights are taken relative to 2^-14 of the largest: in [0, 2^14], so that a
    // weight of 2^-38 of the largest still counts (many of them can add up)
    static constexpr float kLift = 14.0f;
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float2 back(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
    __device__ __forceinline__ static void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};
template <> struct Pack<__nv_bfloat16> {
    static constexpr float kLift = 0.0f;
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float2 back(uint32_t u) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
    }
    __device__ __forceinline__ static void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};

__device__ __forceinline__ int64_t shfl64(int64_t v, int src) {
    return __shfl_sync(0xffffffffu, (long long)v, src);
}
__device__ __forceinline__ uint32_t word(const uint4& u, int i) {
    return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
}

// WHOLE: pages of a multiple of 16 tokens, so that a block of 16 lies in one page and has one
// address; else every token's row is looked up by a lane and handed round.
template <typename T, int DP, bool WIDE, bool WHOLE>
__global__ void __launch_bounds__(kBlock, WIDE ? 2 : 3) paged_mma_kernel(const PagedProblem p) {
    constexpr int HPB = WIDE ? 16 : 8, KI = DP / 32, VI = DP / 64;
    constexpr int NB = DP == 64 ? 2 : 1;  // blocks of 16 tokens loaded together
    constexpr int ROWS = WIDE ? 2 : 1;  // query rows per lane
    using M = Pack<T>;
    __shared__ Join<HPB, DP> sm;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for_segments<T>(p, sm, [&](int64_t b, int64_t hk, int hblk, int heads, int t0, int t1) {
        const T* kh = static_cast<const T*>(p.k) + hk * p.k_h;
        const T* vh = static_cast<const T*>(p.v) + hk * p.v_h;
        const int32_t* table = p.table + b * p.tb_b;
        const int64_t hq0 = hk * p.G + (int64_t)hblk * HPB;
        uint4 qf[ROWS][KI];
#pragma unroll
        for (int w = 0; w < ROWS; ++w)
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                const int d = 32 * i + 8 * c;
                qf[w][i] = r + 8 * w < heads && d < p.D
                               ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + b * p.q_b +
                                                                 (hq0 + r + 8 * w) * p.q_h + d)
                               : zero;
            }
        float o[8 * VI][4], m[ROWS], l[ROWS];
#pragma unroll
        for (int j = 0; j < 8 * VI; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
#pragma unroll
        for (int w = 0; w < ROWS; ++w) {
            m[w] = kNegInf;
            l[w] = 0.0f;
        }
        auto page_index = [&](int tok) {
            return p.page_shift >= 0 ? tok >> p.page_shift : (int)((uint32_t)tok / (uint32_t)p.page);
        };
        // the pages of a step, looked up one step ahead: WHOLE: pg[nb] is block nb's;
        // else pg[0] is that of token t + lane
        auto look_up = [&](int t, int32_t (&pg)[NB]) {
#pragma unroll
            for (int nb = 0; nb < (WHOLE ? NB : 1); ++nb) {
                const int tok = WHOLE ? t + 16 * nb : t + (lane & (16 * NB - 1));
                pg[nb] = tok < t1 ? table[(int64_t)page_index(tok) * p.tb_m] : -1;
            }
        };
        int32_t pg[NB];
        look_up(t0 + warp * 16 * NB, pg);
        for (int t2 = t0 + warp * 16 * NB; t2 < t1; t2 += 16 * NB * kWarps) {
            uint4 kf[NB][2][KI], vf[NB][4][VI];
            bool on_all[NB][4];
            int64_t ko = -1, vo = -1;
            if (!WHOLE) {
                const int tok = t2 + (lane & (16 * NB - 1));
                const int64_t row = tok - page_index(tok) * p.page;
                if (pg[0] >= 0 && pg[0] < p.pages) {
                    ko = pg[0] * p.k_g + row * p.k_t;
                    vo = pg[0] * p.v_g + row * p.v_t;
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                int valid = 0;  // WHOLE: tokens of the block that are there
                const T *kb = kh, *vb = vh;
                if (WHOLE) {
                    const int t = t2 + 16 * nb;
                    const int64_t row = t - page_index(t) * p.page;
                    if (pg[nb] >= 0 && pg[nb] < p.pages) {
                        valid = t1 - t;
                        kb = kh + pg[nb] * p.k_g + (row + r) * p.k_t + 8 * c;
                        vb = vh + pg[nb] * p.v_g + (row + 2 * c) * p.v_t + 8 * r;
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t at = WHOLE ? 0 : shfl64(ko, 16 * nb + r + 8 * j);
                    const T* const row = WHOLE ? kb + 8 * j * p.k_t : kh + at + 8 * c;
                    const bool on = WHOLE ? r + 8 * j < valid : at >= 0;
#pragma unroll
                    for (int i = 0; i < KI; ++i) kf[nb][j][i] = on && 32 * i + 8 * c < p.D ? ld_stream16(row + 32 * i) : zero;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int q = (j & 1) + 8 * (j >> 1);  // this lane's token 2 c + q
                    const int64_t at = WHOLE ? 0 : shfl64(vo, 16 * nb + 2 * c + q);
                    const T* const row = WHOLE ? vb + q * p.v_t : vh + at + 8 * r;
                    const bool on = WHOLE ? 2 * c + q < valid : at >= 0;
                    on_all[nb][j] = on;
#pragma unroll
                    for (int i = 0; i < VI; ++i) vf[nb][j][i] = on && 64 * i + 8 * r < p.D ? ld_stream16(row + 64 * i) : zero;
                }
            }
            look_up(t2 + 16 * NB * kWarps, pg);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int t = t2 + 16 * nb;
                const bool (&on)[4] = on_all[nb];
                const uint4 (&kx)[2][KI] = kf[nb];
                const uint4 (&vx)[4][VI] = vf[nb];
                float s[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
#pragma unroll
                    for (int i = 0; i < KI; ++i) {
                        M::mma(s[j], qf[0][i].x, WIDE ? qf[ROWS - 1][i].x : 0u, qf[0][i].y, WIDE ? qf[ROWS - 1][i].y : 0u,
                               kx[j][i].x, kx[j][i].y);
                        M::mma(s[j], qf[0][i].z, WIDE ? qf[ROWS - 1][i].z : 0u, qf[0][i].w, WIDE ? qf[ROWS - 1][i].w : 0u,
                               kx[j][i].z, kx[j][i].w);
                    }
                }
                uint32_t a[4];
                float f[ROWS];
#pragma unroll
                for (int w = 0; w < ROWS; ++w) {
                    float x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = on[j] ? s[j >> 1][2 * w + (j & 1)] * p.scale_log2 : kNegInf;
                    if (p.w && r + 8 * w < heads) {
                        // pairs of tokens (behind the end of the sequence the second is not read)
                        float* ws = p.ws_s + (b * p.Hq + hq0 + r + 8 * w) * p.ws_cap + t + 2 * c;
                        if (t + 2 * c < t1) *reinterpret_cast<float2*>(ws) = make_float2(x[0], x[1]);
                        if (t + 2 * c + 8 < t1) *reinterpret_cast<float2*>(ws + 8) = make_float2(x[2], x[3]);
                    }
                    float mx = max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3]));
                    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float mn = max_nan(m[w], mx);
                    const float base = mn == kNegInf ? 0.0f : mn;  // no token yet: every weight is 0
                    f[w] = ex2_approx(m[w] - base);
                    m[w] = mn;
                    float e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] = ex2_approx(x[j] - base + M::kLift);
                    l[w] = fmaf(l[w], f[w], (e[0] + e[1]) + (e[2] + e[3]));
                    a[w] = M::two(e[0], e[1]);
                    a[2 + w] = M::two(e[2], e[3]);
                    if (!WIDE) {
                        const float2 h0 = M::back(a[0]), h1 = M::back(a[2]);
                        a[1] = M::two(e[0] - h0.x, e[1] - h0.y);
                        a[3] = M::two(e[2] - h1.x, e[3] - h1.y);
                    }
                }
                // the running maximum moves rarely
                if (__any_sync(0xffffffffu, f[0] != 1.0f || f[ROWS - 1] != 1.0f)) {
#pragma unroll
                    for (int j = 0; j < 8 * VI; ++j) {
                        o[j][0] *= f[0];
                        o[j][1] *= f[0];
                        o[j][2] *= f[ROWS - 1];
                        o[j][3] *= f[ROWS - 1];
                    }
                }
#pragma unroll
                for (int i = 0; i < VI; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
                        const uint32_t b0 = __byte_perm(word(vx[0][i], j / 2), word(vx[1][i], j / 2), sel);
                        const uint32_t b1 = __byte_perm(word(vx[2][i], j / 2), word(vx[3][i], j / 2), sel);
                        M::mma(o[8 * i + j], a[0], a[1], a[2], a[3], b0, b1);
                    }
            }
        }
#pragma unroll
        for (int w = 0; w < ROWS; ++w) {
            l[w] += __shfl_xor_sync(0xffffffffu, l[w], 1);
            l[w] += __shfl_xor_sync(0xffffffffu, l[w], 2);
            if (c == 0) {
                sm.m[warp][r + 8 * w] = m[w] - M::kLift;  // what the weights are relative to
                sm.l[warp][r + 8 * w] = l[w];
            }
#pragma unroll
            for (int i = 0; i < VI; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        float4 v4;
                        float* f4 = &v4.x;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float x = o[8 * i + j + u][2 * w + e], rest = o[8 * i + j + u][2 + e];
                            // (an infinity among the values: times a remainder it may be a NaN)
                            f4[u] = WIDE || fabsf(x) == INFINITY ? x : x + rest;
                        }
                        *reinterpret_cast<float4*>(&sm.o[warp][r + 8 * w][64 * i + (2 * c + e) * 8 + j]) = v4;
                    }
        }
    });
}

// ------------------------------------------------------------ joining ranges --
// One CTA per (sequence, query head): the parts of a sequence that was cut, or
// the answer for one without tokens.
__global__ void __launch_bounds__(kBlock) paged_join_kernel(const PagedProblem p) {
    __shared__ int64_t sh[kWarps];
    __shared__ float red[kWarps];
    __shared__ float wgt[kBlock];
    __shared__ int64_t from[kBlock];
    __shared__ float all[kWarps][256];
    const int64_t b = blockIdx.x / (uint32_t)p.Hq, hq = blockIdx.x - b * p.Hq;
    let_next_kernel_start();
    int64_t total = 0, c = 0;
    {
        int64_t mine = 0, before = 0;
        for (int64_t i = threadIdx.x; i < p.Bn; i += kBlock) {
            const int64_t n = seq_tiles(p, i);
            mine += n;
            before += i < b ? n : 0;
        }
        total = block_sum(mine, sh);
        c = block_sum(before, sh);
    }
    const int64_t n = seq_tiles(p, b);
    const int64_t hk = hq / p.G, g = hq - hk * p.G;
    const int hblk = (int)(g / p.hpb), r = (int)(g - (int64_t)hblk * p.hpb);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_previous_kernel();
    if (n == 0) {
        for (int64_t d = threadIdx.x; d < p.D; d += kBlock) st_f(p.out, b * p.o_b + hq * p.o_h + d * p.o_d, p.io_dt, 0.0f);
        if (threadIdx.x == 0) {
            if (p.lse) p.lse[b * p.lse_b + hq * p.lse_h] = kNegInf;
            if (p.w) p.ws_lse2[b * p.Hq + hq] = kNegInf;
        }
        return;
    }
    const Cut cut(total, p.workers);
    const int64_t w0 = cut.worker_of(c), w1 = cut.worker_of(c + n - 1);
    if (w0 == w1) return;  // written whole
    // every range between them holds a part (none is empty: its neighbours are not)
    auto entry = [&](int64_t w) { return part_of(p, w, hk, hblk, cut.start(w) >= c ? 0 : 1) * p.hpb + r; };
    float m = kNegInf;
    for (int64_t w = w0 + threadIdx.x; w <= w1; w += kBlock) m = max_nan(m, p.ws_ml[entry(w)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) m = max_nan(m, red[i]);
    __syncthreads();
    // warp by warp, every fourth part; a lane takes elements lane, lane + 32, ...
    float l = 0.0f, acc[8] = {};
    const int de = (int)(p.D + 31) / 32;
    for (int64_t base = w0; base <= w1; base += kBlock) {
        const int64_t w = base + threadIdx.x;
        if (w <= w1) {
            const int64_t e = entry(w);
            const float2 ml = p.ws_ml[e];
            float f = 0.0f;
            if (ml.x != kNegInf) {
                f = exp2f(ml.x - m);
                l = fmaf(f, ml.y, l);
            }
            wgt[threadIdx.x] = f;
            from[threadIdx.x] = e * p.D;
        }
        __syncthreads();
        const int cnt = (int)(w1 - base + 1 < kBlock ? w1 - base + 1 : kBlock);
        for (int i = warp; i < cnt; i += 4 * kWarps) {
            float fi[4], v[4][8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {  // 4 parts in flight
                const int at = i + u * kWarps;
                fi[u] = at < cnt ? wgt[at] : 0.0f;
                const float* o = p.ws_o + from[at < cnt ? at : i];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[u][e] = e < de && lane + 32 * e < p.D ? o[lane + 32 * e] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = fi[u] != 0.0f ? fmaf(fi[u], v[u][e], acc[e]) : acc[e];  // (a NaN counts)
        }
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) red[warp] = l;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < de) all[warp][lane + 32 * e] = acc[e];
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) l += red[i];
    for (int d = threadIdx.x; d < p.D; d += kBlock) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += all[i][d];
        st_f(p.out, b * p.o_b + hq * p.o_h + d * p.o_d, p.io_dt, m == kNegInf ? 0.0f : sum / l);
    }
    if (threadIdx.x == 0) {
        const float lse2 = m == kNegInf ? kNegInf : m + log2f(l);
        if (p.lse) p.lse[b * p.lse_b + hq * p.lse_h] = lse2 * kLn2;
        if (p.w) p.ws_lse2[b * p.Hq + hq] = lse2;
    }
}

// Accumulated weights: the scores of the first kernel against the joined
// denominators.  A thread takes 4 neighbouring tokens of one key-value head.
constexpr int kWeightTokens = 4 * kBlock;  // tokens per CTA
__global__ void __launch_bounds__(kBlock) paged_weights_kernel(const PagedProblem p) {
    const int64_t blocks = (p.cap + kWeightTokens - 1) / kWeightTokens;
    const int64_t row = blockIdx.x / blocks, b = row / p.Hkv, hk = row - b * p.Hkv;
    const int64_t len = seq_len(p, b);
    const int64_t t = (blockIdx.x - row * blocks) * kWeightTokens + 4 * threadIdx.x;
    const float* const w = p.w + b * p.w_b + hk * p.w_h;
    float* const w_out = p.w_out + b * p.wo_b + hk * p.wo_h;
    float sum[4] = {}, old[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) old[j] = t + j < len ? w[(t + j) * p.w_t] : 0.0f;  // (not the last kernel's)
    wait_for_previous_kernel();
    if (t >= len) return;
#pragma unroll 4
    for (int64_t g = 0; g < p.G; ++g) {
        const int64_t hq = b * p.Hq + hk * p.G + g;
        const float lse2 = p.ws_lse2[hq];
        const float4 x4 = *reinterpret_cast<const float4*>(p.ws_s + hq * p.ws_cap + t);
        const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += lse2 == kNegInf || x[j] == kNegInf ? 0.0f : exp2f(x[j] - lse2);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (t + j < len) w_out[(t + j) * p.wo_t] = old[j] + sum[j];
}

// a launch that may start before the stream's last kernel has finished
cudaError_t launch_after(void (*fn)(const PagedProblem), unsigned grid, const PagedProblem& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kBlock);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

template <typename T, bool WHOLE>
void mma_t(const PagedProblem& p, dim3 grid, cudaStream_t s) {
    if (p.hpb == 16) {
        if (p.D <= 64) paged_mma_kernel<T, 64, true, WHOLE><<<grid, kBlock, 0, s>>>(p);
        else paged_mma_kernel<T, 128, true, WHOLE><<<grid, kBlock, 0, s>>>(p);
    } else {
        if (p.D <= 64) paged_mma_kernel<T, 64, false, WHOLE><<<grid, kBlock, 0, s>>>(p);
        else paged_mma_kernel<T, 128, false, WHOLE><<<grid, kBlock, 0, s>>>(p);
    }
}

template <typename T>
void generic_t(const PagedProblem& p, dim3 grid, cudaStream_t s) {
    if (p.D <= 64) paged_generic_kernel<T, 2><<<grid, kBlock, 0, s>>>(p);
    else if (p.D <= 128) paged_generic_kernel<T, 4><<<grid, kBlock, 0, s>>>(p);
    else paged_generic_kernel<T, 8><<<grid, kBlock, 0, s>>>(p);
}

}  // namespace

int paged_block() { return kBlock; }
int64_t paged_weight_blocks(int64_t cap) { return (cap + kWeightTokens - 1) / kWeightTokens; }
int paged_heads_per_cta(int kernel, int64_t G) {
    return kernel == SSM_KERNEL_PAGED_DECODE ? (G > 8 ? 16 : 8) : kGenHeads;
}
// CTAs resident per SM, as the launch bounds and the registers allow
int paged_ctas_per_sm(int kernel, int64_t G, int64_t D) {
    if (kernel == SSM_KERNEL_PAGED_DECODE) return G > 8 ? 2 : 3;
    return D <= 128 ? 3 : 2;
}

cudaError_t launch_paged(const PagedProblem& p, int kernel, cudaStream_t s) {
    const dim3 grid((unsigned)p.workers, (unsigned)(p.Hkv * p.hblocks));
    if (kernel == SSM_KERNEL_PAGED_DECODE) {
        const bool whole = p.page % 16 == 0;
        if (p.io_dt == kF16) whole ? mma_t<__half, true>(p, grid, s) : mma_t<__half, false>(p, grid, s);
        else whole ? mma_t<__nv_bfloat16, true>(p, grid, s) : mma_t<__nv_bfloat16, false>(p, grid, s);
    } else if (p.io_dt == kF16) generic_t<__half>(p, grid, s);
    else if (p.io_dt == kBF16) generic_t<__nv_bfloat16>(p, grid, s);
    else generic_t<float>(p, grid, s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_after(paged_join_kernel, (unsigned)(p.Bn * p.Hq), p, s);
    if (e != cudaSuccess || !p.w || p.cap == 0) return e;
    return launch_after(paged_weights_kernel, (unsigned)(paged_weight_blocks(p.cap) * p.Bn * p.Hkv), p, s);
}

}  // namespace ssm
