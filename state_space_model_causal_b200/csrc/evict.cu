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
//   evict_copy_kernel    copies the kept key and value rows to their new pages,
//       bound by HBM: 4 D elements read and written per kept token.
#include "../../include/ssm_causal.h"
#include "common.cuh"
#include "problem.h"

namespace ssm {
namespace {

constexpr int kSelect = 512;  // threads of the selection
constexpr int kSelWarps = kSelect / 32;
constexpr int kItems = 4;     // consecutive tokens per thread and step
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

__global__ void __launch_bounds__(kSelect) evict_select_kernel(const EvictProblem p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sh[kSelWarps];
    __shared__ uint32_t pick[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
    int64_t n = p.lens[b * p.len_b];
    n = n < 0 ? 0 : (n < p.cap ? n : p.cap);
    const int len = (int)n;
    const int first_recent = len - (int)(p.recent < n ? p.recent : n);
    const float* w = p.w + b * p.w_b + h * p.w_h;
    const int32_t* table = p.table + b * p.tb_b;
    auto key_at = [&](int t) {
        if (t >= len) return 0u;
        const int32_t pg = table[(int64_t)(t / p.page) * p.tb_m];
        return key_of(w[t * p.w_t], pg >= 0 && pg < p.pages, t >= first_recent);
    };

    // passes of 8 bits from the top; `left` tokens are still to be found among
    // the keys that agree with `prefix` in the bits above
    uint32_t prefix = 0, left = 0, valid = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) hist[threadIdx.x] = 0;
        __syncthreads();
        const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        uint32_t mine = 0;
        for (int t0 = 0; t0 < len; t0 += kSelect) {
            const uint32_t key = key_at(t0 + threadIdx.x);
            mine += key != 0u;
            const bool on = key != 0u && (key & above) == prefix;
            // one atomic per distinct digit of the warp: softmax weights share their exponents
            const uint32_t digit = on ? (key >> shift) & 255u : 256u;
            const uint32_t same = __match_any_sync(0xffffffffu, digit);
            if (on && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
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
            wv[i] = t < len ? w[t * p.w_t] : 0.0f;
            gt[i] = key > prefix;
            eq[i] = key == prefix;
            ngt += gt[i];
            neq += eq[i];
        }
        uint32_t both = ngt | neq << 16;  // at most 2048 of each per step
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

// VEC: rows of 16-byte vectors (unit element stride, aligned); a thread takes a
// vector of the key row and of the value row.  Else one element.
template <bool VEC>
__global__ void __launch_bounds__(kCopy) evict_copy_kernel(const EvictProblem p) {
    const int64_t per_row = VEC ? p.D * p.es / 16 : p.D;
    const int64_t total = p.Bn * p.keep * p.Hkv * per_row;
    const int64_t unit = VEC ? 16 / p.es : 1;  // elements per item
    for (int64_t i = (int64_t)blockIdx.x * kCopy + threadIdx.x; i < total; i += (int64_t)gridDim.x * kCopy) {
        int64_t r = i / per_row;
        const int64_t d = (i - r * per_row) * unit;
        const int64_t h = r % p.Hkv;
        r /= p.Hkv;
        const int64_t j = r % p.keep, b = r / p.keep;
        const int32_t t = p.kept[b * p.kp_b + h * p.kp_h + j * p.kp_j];
        const int32_t to = p.new_table[b * p.nt_b + j / p.page * p.nt_m];
        if (t < 0 || to < 0 || to >= p.pages) continue;
        const int64_t from = p.table[b * p.tb_b + (int64_t)(t / p.page) * p.tb_m];
        const int64_t fr = t % p.page, tr = j % p.page;
        char* k = static_cast<char*>(p.k);
        char* v = static_cast<char*>(p.v);
        const int64_t ks = (from * p.k_g + fr * p.k_t + h * p.k_h + d * p.k_d) * p.es;
        const int64_t kd = (to * p.k_g + tr * p.k_t + h * p.k_h + d * p.k_d) * p.es;
        const int64_t vs = (from * p.v_g + fr * p.v_t + h * p.v_h + d * p.v_d) * p.es;
        const int64_t vd = (to * p.v_g + tr * p.v_t + h * p.v_h + d * p.v_d) * p.es;
        if (VEC) {
            const uint4 kv = ld_stream16(k + ks), vv = ld_stream16(v + vs);
            st_stream16(k + kd, kv);
            st_stream16(v + vd, vv);
        } else if (p.es == 2) {
            *reinterpret_cast<uint16_t*>(k + kd) = *reinterpret_cast<const uint16_t*>(k + ks);
            *reinterpret_cast<uint16_t*>(v + vd) = *reinterpret_cast<const uint16_t*>(v + vs);
        } else {
            *reinterpret_cast<uint32_t*>(k + kd) = *reinterpret_cast<const uint32_t*>(k + ks);
            *reinterpret_cast<uint32_t*>(v + vd) = *reinterpret_cast<const uint32_t*>(v + vs);
        }
    }
}

}  // namespace

int evict_select_block() { return kSelect; }
int evict_copy_block() { return kCopy; }

cudaError_t launch_evict(const EvictProblem& p, bool vec, int copy_grid, cudaStream_t s) {
    evict_select_kernel<<<(unsigned)(p.Bn * p.Hkv), kSelect, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (vec) evict_copy_kernel<true><<<copy_grid, kCopy, 0, s>>>(p);
    else evict_copy_kernel<false><<<copy_grid, kCopy, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace ssm
