// evict.cu -- eviction from a paged key-value cache by accumulated attention
// weight, for sm_100a.
//
// Of n tokens of a sequence and key-value head, min(keep, n) stay: the last
// `recent`, then those of the largest weight, the lowest position first among
// equals.  Two kernels:
//
//   evict_select_kernel  one CTA per (sequence, head).  Weights are mapped to
//       32-bit keys in their order; four passes over the weights, 8 bits each,
//       find the key of the last token that stays and how many of the tokens
//       with that key do (a radix selection: no sort, no atomics on values, the
//       counts do not depend on the order of arrival); a fifth pass writes the
//       positions in ascending order by prefix sums over the CTA.
//       Bound by the latency of its passes: the loads of a step are issued
//       together, each address clamped instead of branched around (49 to 35 us at 16
//       caches of up to 16000 tokens and 8 heads; 1024 threads instead of 512: 32.6).
//   evict_copy_kernel    copies the kept key and value rows to their new pages,
//       4 D elements read and written per kept token.  Bound by HBM's mix of reads
//       and writes: at 16 caches, 8 heads of 128 in bf16, half of up to 16000
//       tokens kept, both kernels take 139 us, 0.72 of a plain copy's rate.  A
//       thread keeps its place in the rows (142 us against 157 us with a division
//       per piece, with the slower selection).
#include "../../include/ssm_causal.h"
#include "common.cuh"
#include "problem.h"

namespace ssm {
namespace {

constexpr int kSelect = 1024;  // threads of the selection
constexpr int kSelWarps = kSelect / 32;
constexpr int kItems = 4;     // consecutive tokens per thread and step
constexpr int kCached = 48 * 1024;  // keys that fit in shared memory (192 KB)
constexpr int kCopy = 256;

// Order of the weights as an unsigned key: 0 = a token that cannot be kept,
// 1 = a NaN, then the numbers in their order, the largest key for a recent token.
__device__ __forceinline__ uint32_t key_of(float w, bool valid, bool recent) {
    if (!valid) return 0u;
    if (recent) return 0xffffffffu;
    if (w != w) return 1u;
    const uint32_t u = __float_as_uint(w + 0.0f);  // -0 + 0 = +0
    return (u >> 31) ? ~u : u | 0x80000000u;       // -inf -> 0x007fffff, +inf -> 0xff800000
}

// CACHED: the keys are made once and kept in shared memory; else (sequences past
// 48 Ki tokens) every pass makes them again.
template <bool CACHED>
__global__ void __launch_bounds__(kSelect) evict_select_kernel(const EvictProblem p) {
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sh[kSelWarps];
    __shared__ uint32_t pick[2];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
    int64_t n = p.lens[b * p.len_b];
    n = n < 0 ? 0 : (n < p.cap ? n : p.cap);
    const int len = (int)n;
    const int first_recent = len - (int)(p.recent < n ? p.recent : n);
    const float* w = p.w + b * p.w_b + h * p.w_h;
    const int32_t* table = p.table + b * p.tb_b;
    // the keys of U tokens from t on, `step` apart (0 behind the end): loads of clamped
    // addresses, all U in flight (behind a branch each waited for the one before)
    auto make_keys = [&](int t, int step, auto& key) {
        constexpr int U = sizeof(key) / 4;
        int32_t pg[U];
        float wv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = t + u * step < len ? t + u * step : len - 1;
            pg[u] = table[(int64_t)(at / p.page) * p.tb_m];
            wv[u] = w[at * p.w_t];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = t + u * step;
            key[u] = at < len ? key_of(wv[u], pg[u] >= 0 && pg[u] < p.pages, at >= first_recent) : 0u;
        }
    };
    auto make_key = [&](int t) {  // (t < len)
        uint32_t key[1];
        make_keys(t, 0, key);
        return key[0];
    };

    if (CACHED) {
        for (int t = threadIdx.x; t < len; t += 8 * kSelect) {
            uint32_t key[8];
            make_keys(t, kSelect, key);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (t + u * kSelect < len) keys[t + u * kSelect] = key[u];
        }
        __syncthreads();
    }
    auto key_at = [&](int t) { return t < len ? (CACHED ? keys[t] : make_key(t)) : 0u; };

    // passes of 8 bits from the top; `left` tokens are still to be found among
    // the keys that agree with `prefix` in the bits above
    uint32_t prefix = 0, left = 0, valid = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) hist[threadIdx.x] = 0;
        __syncthreads();
        const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        uint32_t mine = 0;
        for (int t0 = 0; t0 < len; t0 += 4 * kSelect) {
            uint32_t key[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) key[u] = key_at(t0 + u * kSelect + threadIdx.x);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                mine += key[u] != 0u;
                const bool on = key[u] != 0u && (key[u] & above) == prefix;
                if (!__any_sync(0xffffffffu, on)) continue;
                const uint32_t digit = on ? (key[u] >> shift) & 255u : 256u;
                if (shift == 24) {
                    // one atomic per distinct digit of the warp: softmax weights share their exponents
                    const uint32_t same = __match_any_sync(0xffffffffu, digit);
                    if (on && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
                } else if (__all_sync(0xffffffffu, digit == __shfl_sync(0xffffffffu, digit, 0))) {
                    if (lane == 0) atomicAdd(&hist[digit], 32u);  // (all equal: weights that never moved)
                } else if (on) {
                    atomicAdd(&hist[digit], 1u);
                }
            }
        }
        if (shift == 24) {  // how many tokens there are, and how many stay
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
            if (lane == 0) sh[warp] = mine;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kSelWarps; ++i) valid += sh[i];
            left = (int64_t)valid < p.keep ? valid : (uint32_t)p.keep;
        }
        __syncthreads();
        // the digit at which the count from the top reaches `left`
        if (warp == 0 && left > 0) {
            uint32_t c[8], sum = 0;  // lane l: digits 255 - 8 l - i
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = hist[255 - 8 * lane - i];
                sum += c[i];
            }
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            uint32_t before = incl - sum;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (before < left && left <= before + c[i]) {
                    pick[0] = 255 - 8 * lane - i;
                    pick[1] = left - before;
                }
                before += c[i];
            }
        }
        __syncthreads();
        if (left > 0) {
            prefix |= pick[0] << shift;
            left = pick[1];
        }
        __syncthreads();
    }
    const uint32_t stay = (int64_t)valid < p.keep ? valid : (uint32_t)p.keep;

    // positions in ascending order: keys above `prefix`, and the first `left` equal to it
    float* nw = p.new_w + b * p.nw_b + h * p.nw_h;
    int32_t* kept = p.kept + b * p.kp_b + h * p.kp_h;
    uint32_t gt_done = 0, eq_done = 0;
    for (int t0 = 0; stay > 0 && t0 < len; t0 += kSelect * kItems) {
        uint32_t gt[kItems], eq[kItems], ngt = 0, neq = 0;
        float wv[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int t = t0 + threadIdx.x * kItems + i;
            const uint32_t key = key_at(t);
            wv[i] = w[(t < len ? t : len - 1) * p.w_t];
            gt[i] = key > prefix;
            eq[i] = key == prefix;
            ngt += gt[i];
            neq += eq[i];
        }
        uint32_t both = ngt | neq << 16;  // at most 4096 of each per step
        uint32_t incl = both;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) sh[warp] = incl;
        __syncthreads();
        uint32_t before = incl - both, all = 0;
#pragma unroll
        for (int i = 0; i < kSelWarps; ++i) {
            if (i < warp) before += sh[i];
            all += sh[i];
        }
        __syncthreads();
        uint32_t g = gt_done + (before & 0xffffu), e = eq_done + (before >> 16);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (gt[i] || (eq[i] && e < left)) {
                const int64_t j = g + (e < left ? e : left);
                kept[j * p.kp_j] = t0 + threadIdx.x * kItems + i;
                nw[j * p.nw_j] = wv[i];
            }
            g += gt[i];
            e += eq[i];
        }
        gt_done += all & 0xffffu;
        eq_done += all >> 16;
    }
    for (int64_t j = stay + threadIdx.x; j < p.keep; j += kSelect) {
        kept[j * p.kp_j] = -1;
        nw[j * p.nw_j] = 0.0f;
    }
    if (h == 0 && threadIdx.x == 0) p.new_lens[b * p.nl_b] = (int32_t)stay;
}

// A CTA takes per_cta kept tokens of one sequence for every head: first the offsets of
// their rows, one thread each (the table look-ups and their arithmetic once per
// row), then the copy, consecutive threads on consecutive pieces of a row.  VEC: pieces
// of 16 bytes (unit element stride, aligned rows), else single elements.
constexpr int kRows = 32, kFewRows = 8;  // the latter while that leaves few CTAs
constexpr int64_t kNoRow = INT64_MIN;

template <typename W, bool VEC>
__global__ void __launch_bounds__(kCopy) evict_copy_kernel(const EvictProblem p, const int per_cta) {
    __shared__ int64_t k_from[kCopy], k_to[kCopy], v_from[kCopy], v_to[kCopy];  // offsets in pieces
    const int64_t blocks = (p.keep + per_cta - 1) / per_cta;
    const int64_t b = blockIdx.x / blocks, j0 = (blockIdx.x - b * blocks) * per_cta;
    const int rows = (int)(p.keep - j0 < per_cta ? p.keep - j0 : per_cta);
    const int entries = rows * (int)p.Hkv;  // (Hkv < 2^26)
    const int pieces = VEC ? (int)(p.D * p.es / 16) : (int)p.D;
    const int shift = VEC ? (p.es == 2 ? 3 : 2) : 0;  // elements per piece: 2^shift, and rows start at whole pieces
    const int width = pieces < kCopy ? (pieces > 0 ? pieces : 1) : kCopy, at_once = kCopy / width;  // threads per row, rows
    const int place = threadIdx.x % width;
    const int first = threadIdx.x / width < at_once ? threadIdx.x / width : 1 << 30;  // (the last few threads may have none)
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the selection
    for (int e0 = 0; e0 < entries; e0 += kCopy) {
        const int e = e0 + threadIdx.x;
        if (e < entries) {
            const int r = e / (int)p.Hkv, h = e - r * (int)p.Hkv;
            const int j = (int)j0 + r;
            const int32_t t = p.kept[b * p.kp_b + h * p.kp_h + j * p.kp_j];
            const int32_t to = p.new_table[b * p.nt_b + (int64_t)(j / p.page) * p.nt_m];
            k_from[threadIdx.x] = kNoRow;
            if (t >= 0 && to >= 0 && to < p.pages) {
                const int64_t from = p.table[b * p.tb_b + (int64_t)(t / p.page) * p.tb_m];
                const int fr = t % p.page, tr = j % p.page;
                k_from[threadIdx.x] = (from * p.k_g + fr * p.k_t + h * p.k_h) >> shift;
                k_to[threadIdx.x] = (to * p.k_g + tr * p.k_t + h * p.k_h) >> shift;
                v_from[threadIdx.x] = (from * p.v_g + fr * p.v_t + h * p.v_h) >> shift;
                v_to[threadIdx.x] = (to * p.v_g + tr * p.v_t + h * p.v_h) >> shift;
            }
        }
        __syncthreads();
        const int here = entries - e0 < kCopy ? entries - e0 : kCopy;
        W* const k = static_cast<W*>(p.k);
        W* const v = static_cast<W*>(p.v);
        const int64_t ks = VEC ? 1 : p.k_d, vs = VEC ? 1 : p.v_d;
        // U rows' pieces of the keys and of the values in flight per thread, whose place
        // in a row stays the same
        constexpr int U = 4;
        for (int d0 = place; d0 < pieces; d0 += width)
            for (int row0 = first; row0 < here; row0 += U * at_once) {
                W kx[U], vx[U];
                const int64_t dk = d0 * ks, dv = d0 * vs;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int row = row0 + u * at_once;
                    if (row < here && k_from[row] != kNoRow) {
                        kx[u] = __ldcs(k + k_from[row] + dk);
                        vx[u] = __ldcs(v + v_from[row] + dv);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int row = row0 + u * at_once;
                    if (row < here && k_from[row] != kNoRow) {
                        __stcs(k + k_to[row] + dk, kx[u]);
                        __stcs(v + v_to[row] + dv, vx[u]);
                    }
                }
            }
        __syncthreads();
    }
}

}  // namespace

int evict_select_block() { return kSelect; }
int64_t evict_copy_ctas(int64_t keep) { return (keep + kFewRows - 1) / kFewRows; }

cudaError_t launch_evict(const EvictProblem& p, bool vec, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (p.cap <= kCached) {
        const int smem = (int)p.cap * 4;
        auto* fn = evict_select_kernel<true>;
        int per_sm = 0;
        e = prepared_launch(
            reinterpret_cast<const void*>(fn), smem > 40960 ? kCached * 4 : 40960, kSelect, &per_sm,
            [&](int bytes) { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); },
            [&](int* n) { *n = 1; return cudaSuccess; });
        if (e != cudaSuccess) return e;
        fn<<<(unsigned)(p.Bn * p.Hkv), kSelect, smem, s>>>(p);
    } else {
        evict_select_kernel<false><<<(unsigned)(p.Bn * p.Hkv), kSelect, 0, s>>>(p);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // the copy may be launched while the selection still runs; it waits for its results
    cudaLaunchConfig_t cfg{};
    const int per_cta = p.Bn * ((p.keep + kRows - 1) / kRows) >= 512 ? kRows : kFewRows;
    cfg.gridDim = dim3((unsigned)(p.Bn * ((p.keep + per_cta - 1) / per_cta)));
    cfg.blockDim = dim3(kCopy);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (vec) return cudaLaunchKernelEx(&cfg, evict_copy_kernel<uint4, true>, p, per_cta);
    return p.es == 2 ? cudaLaunchKernelEx(&cfg, evict_copy_kernel<uint16_t, false>, p, per_cta)
                     : cudaLaunchKernelEx(&cfg, evict_copy_kernel<uint32_t, false>, p, per_cta);
}

}  // namespace ssm
