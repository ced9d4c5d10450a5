// api_attn.cpp -- the C ABI of the token mixers of hybrid models: linear
// attention with a decay per head (prompt, one token), attention of one token
// over a paged key-value cache, and eviction from that cache.  As in api.cpp
// every argument is checked before any CUDA call.
#include "../../include/ssm_causal.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "checks.h"
#include "problem.h"

namespace {

using namespace ssm;

constexpr int kMaxN = 256;  // keys per state row, elements per head

uint64_t round256(uint64_t v) { return (v + 255) / 256 * 256; }

BoundedWaits bounded_waits() {
    BoundedWaits w{kWaitBudget, -1};
#ifdef SSM_TEST_HOOKS
    long long v = 0;
    if (env_int("SSM_TEST_WAIT_CYCLES", &v) && v > 0) w.budget = clamp_test_budget(v);
    if (env_int("SSM_TEST_DROP_ITEM", &v) && v >= 0) w.drop_item = v;
#endif
    return w;
}

bool same_view(const ssm_tensor& a, const ssm_tensor& b) {
    if (a.data != b.data || a.dtype != b.dtype || a.ndim != b.ndim) return false;
    for (int i = 0; i < a.ndim; ++i)
        if (a.shape[i] != b.shape[i] || (a.shape[i] > 1 && a.stride[i] != b.stride[i])) return false;
    return true;
}

ssm_status ws_ok(const void* ws, uint64_t have, uint64_t need) {
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0 || have < need) return SSM_ERR_WORKSPACE;
    return SSM_OK;
}

// A caller's workspace as a tensor, for the overlap checks.
ssm_tensor ws_tensor(void* ws, uint64_t bytes) {
    ssm_tensor t{};
    t.data = ws;
    t.dtype = SSM_F32;
    t.ndim = 1;
    t.shape[0] = (int64_t)(bytes / 4);
    t.stride[0] = 1;
    return t;
}

// rows of 16-byte vectors along the last dimension: unit stride there, every
// other stride a multiple of 16 bytes, an aligned pointer
bool rows16(const ssm_tensor& t) {
    const int es = esize(t.dtype), last = t.ndim - 1;
    bool ok = aligned16(t.data) && (t.shape[last] == 1 || t.stride[last] == 1) && (t.shape[last] * es) % 16 == 0;
    for (int i = 0; i < last; ++i) ok = ok && (sd(t, i) * es) % 16 == 0;
    return ok;
}

// -------------------------------------------------- linear attention, prompt --
ssm_status linattn_impl(const ssm_linattn_args* a, cudaStream_t stream, uint64_t* ws_query) {
    if (!a) return SSM_ERR_NULL;
    if (a->struct_size != sizeof(ssm_linattn_args)) return SSM_ERR_VERSION;
    SSM_TRY(info_ok(a->info));
    for (const ssm_tensor* t : {&a->q, &a->k, &a->v, &a->log_decay, &a->out}) SSM_TRY(basic(*t));
    if (a->q.ndim != 4 || a->v.ndim != 4) return SSM_ERR_SHAPE;
    const int64_t B = a->q.shape[0], Hk = a->q.shape[1], L = a->q.shape[2], N = a->q.shape[3];
    const int64_t H = a->v.shape[1], P = a->v.shape[3];
    SSM_TRY(want(a->k, {B, Hk, L, N}));
    SSM_TRY(want(a->v, {B, H, L, P}));
    SSM_TRY(want(a->out, {B, H, L, P}));
    if (N < 1) return SSM_ERR_SHAPE;
    if (N > kMaxN) return SSM_ERR_UNSUPPORTED;
    if (Hk == 0 ? H != 0 : H % Hk != 0) return SSM_ERR_SHAPE;
    const bool per_token = a->log_decay.ndim == 3;
    if (per_token) SSM_TRY(want(a->log_decay, {B, H, L}));
    else SSM_TRY(want(a->log_decay, {H}));
    const int io = a->q.dtype;
    if (!is_float(io) || a->k.dtype != io || a->v.dtype != io || a->out.dtype != io) return SSM_ERR_DTYPE;
    if (a->log_decay.dtype != SSM_F32) return SSM_ERR_DTYPE;
    const bool has_in = present(a->state);
    const ssm_tensor& so = present(a->state_out) ? a->state_out : a->state;
    const bool has_out = present(so);
    if (has_in) {
        SSM_TRY(basic(a->state));
        SSM_TRY(want(a->state, {B, H, P, N}));
        if (a->state.dtype != SSM_F32) return SSM_ERR_DTYPE;
    }
    if (has_out) {
        SSM_TRY(basic(so));
        SSM_TRY(want(so, {B, H, P, N}));
        if (so.dtype != SSM_F32) return SSM_ERR_DTYPE;
        if (!non_overlapping(so)) return SSM_ERR_STRIDE;
    }
    const bool has_lens = present(a->seq_lens);
    if (has_lens) {
        SSM_TRY(basic(a->seq_lens));
        SSM_TRY(want(a->seq_lens, {B}));
        if (a->seq_lens.dtype != SSM_I32) return SSM_ERR_DTYPE;
    }
    if (!non_overlapping(a->out)) return SSM_ERR_STRIDE;
    const ssm_tensor* ins[] = {&a->q, &a->k, &a->v, &a->log_decay, &a->seq_lens};
    for (const ssm_tensor* t : ins) {
        if (!present(*t)) continue;
        if (overlap(a->out, *t)) return SSM_ERR_ALIAS;
        if (has_out && overlap(so, *t)) return SSM_ERR_ALIAS;
    }
    if (has_in && overlap(a->out, a->state)) return SSM_ERR_ALIAS;
    if (has_out && overlap(a->out, so)) return SSM_ERR_ALIAS;
    if (has_in && has_out && !same_view(a->state, so) && overlap(a->state, so)) return SSM_ERR_ALIAS;
    if (ws_query) *ws_query = 0;
    if (B * H * P == 0 || (L == 0 && (!has_out || (has_in && same_view(a->state, so))))) {
        fill_info(a->info, SSM_KERNEL_NONE, 0, 0, 0, 0, 0);
        return SSM_OK;
    }
    const bool dry = (a->flags & SSM_FLAG_DRY_RUN) != 0;

    LinAttnProblem p{};
    p.Bn = B; p.H = H; p.Hk = Hk; p.L = L; p.N = N; p.P = P; p.rep = H / Hk; p.io_dt = io;
    p.q = a->q.data; p.q_b = sd(a->q, 0); p.q_h = sd(a->q, 1); p.q_t = sd(a->q, 2); p.q_n = sd(a->q, 3);
    p.k = a->k.data; p.k_b = sd(a->k, 0); p.k_h = sd(a->k, 1); p.k_t = sd(a->k, 2); p.k_n = sd(a->k, 3);
    p.v = a->v.data; p.v_b = sd(a->v, 0); p.v_h = sd(a->v, 1); p.v_t = sd(a->v, 2); p.v_p = sd(a->v, 3);
    p.g = static_cast<const float*>(a->log_decay.data);
    if (per_token) {
        p.g_b = sd(a->log_decay, 0); p.g_h = sd(a->log_decay, 1); p.g_t = sd(a->log_decay, 2);
    } else {
        p.g_b = 0; p.g_h = sd(a->log_decay, 0); p.g_t = 0;
    }
    if (has_in) {
        p.s_in = static_cast<const float*>(a->state.data);
        p.si_b = sd(a->state, 0); p.si_h = sd(a->state, 1); p.si_p = sd(a->state, 2); p.si_n = sd(a->state, 3);
    }
    if (has_out) {
        p.s_out = static_cast<float*>(so.data);
        p.so_b = sd(so, 0); p.so_h = sd(so, 1); p.so_p = sd(so, 2); p.so_n = sd(so, 3);
    }
    if (has_lens) {
        p.lens = static_cast<const int32_t*>(a->seq_lens.data);
        p.len_b = sd(a->seq_lens, 0);
    }
    p.scale = a->scale;
    p.out = a->out.data;
    p.o_b = sd(a->out, 0); p.o_h = sd(a->out, 1); p.o_t = sd(a->out, 2); p.o_p = sd(a->out, 3);

    // the chunk kernel: TMA boxes of contiguous, aligned rows (no broadcast)
    bool chunk = esize(io) == 2 && N <= 128 && L > 0 && L <= INT32_MAX - 256 && B <= INT32_MAX && H <= INT32_MAX;
    for (const ssm_tensor* t : {&a->q, &a->k, &a->v, &a->out}) {
        chunk = chunk && rows16(*t);
        for (int i = 0; i < 3; ++i)
            chunk = chunk && (t->shape[i] == 1 || (t->stride[i] > 0 && t->stride[i] < ((int64_t)1 << 39)));
    }
    if (chunk) {
        const int64_t units = B * H * ((P + linattn_chunk_values() - 1) / linattn_chunk_values());
        const int64_t chunks = (L + linattn_chunk_tokens() - 1) / linattn_chunk_tokens();
        const int dev = current_device(dry);
        // With half a wave of CTAs or less, each sequence in pieces: `others` after the
        // first, which is half as long; each launch computes `others` pieces at a time.
        // (Two launches of fewer than 6 chunks each would take longer than one of 12.)
        int64_t others = std::min<int64_t>(sm_count(dry, dev) / units, chunks / 2);
        if (others < 2 || chunks < 12 || (!ws_query && !a->workspace)) others = 0;
        LinAttnPieces cut{1, chunks, 0};
        if (others) {
            cut.per_piece = (2 * chunks + 2 * others) / (2 * others + 1);  // about chunks / (others + 1/2), rounded up
            cut.piece0 = std::max<int64_t>(1, chunks - others * cut.per_piece);
            cut.pieces = (int)(1 + (chunks - cut.piece0 + cut.per_piece - 1) / cut.per_piece);
        }
        const int64_t pieces = cut.pieces;
        const uint64_t rec = pieces > 1 ? round256((uint64_t)units * (pieces - 1) * linattn_chunk_record_bytes()) : 0;
        const uint64_t need = pieces > 1 ? rec + round256((uint64_t)units * (pieces - 1) * 8) : 0;
        if (ws_query) {
            *ws_query = need;
            return SSM_OK;
        }
        if (pieces > 1) {
            SSM_TRY(ws_ok(a->workspace, a->workspace_bytes, need));
            const ssm_tensor ws = ws_tensor(a->workspace, need);
            for (const ssm_tensor* t : {&a->q, &a->k, &a->v, &a->log_decay, &a->seq_lens, &a->state, &so, &a->out})
                if (present(*t) && overlap(ws, *t)) return SSM_ERR_ALIAS;
        }
        if (units > INT32_MAX / pieces) return SSM_ERR_UNSUPPORTED;
        fill_info(a->info, SSM_KERNEL_LINATTN_CHUNK, (int)(units * std::max<int64_t>(pieces - 1, 1)), linattn_chunk_block(),
                  linattn_chunk_smem(io), linattn_chunk_values(), units * pieces);
        if (dry) return SSM_OK;
        char* ws = static_cast<char*>(a->workspace);
        return launch_linattn_chunk(p, units, cut, reinterpret_cast<float*>(ws),
                                    reinterpret_cast<double*>(ws + rec), bounded_waits(), dev, stream) == cudaSuccess
                   ? SSM_OK : SSM_ERR_CUDA;
    }
    const int64_t rows = linattn_generic_rows(B * H, P, sm_count(dry)), blocks = (P + rows - 1) / rows;
    if (B * H > INT32_MAX / blocks) return SSM_ERR_UNSUPPORTED;
    const int grid = (int)(B * H * blocks);
    fill_info(a->info, SSM_KERNEL_LINATTN_GENERIC, grid, linattn_generic_block(), 0, rows, B * H * blocks);
    if (dry || ws_query) return SSM_OK;
    return launch_linattn_generic(p, (int)rows, grid, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

// ----------------------------------------------- linear attention, one token --
ssm_status linattn_update_impl(const ssm_linattn_update_args* a, cudaStream_t stream) {
    if (!a) return SSM_ERR_NULL;
    if (a->struct_size != sizeof(ssm_linattn_update_args)) return SSM_ERR_VERSION;
    SSM_TRY(info_ok(a->info));
    for (const ssm_tensor* t : {&a->state, &a->q, &a->k, &a->v, &a->log_decay, &a->out}) SSM_TRY(basic(*t));
    if (a->state.ndim != 4 || a->q.ndim != 3) return SSM_ERR_SHAPE;
    const int64_t S = a->state.shape[0], H = a->state.shape[1], P = a->state.shape[2], N = a->state.shape[3];
    const int64_t B = a->q.shape[0], Hk = a->q.shape[1];
    SSM_TRY(want(a->q, {B, Hk, N}));
    SSM_TRY(want(a->k, {B, Hk, N}));
    SSM_TRY(want(a->v, {B, H, P}));
    SSM_TRY(want(a->out, {B, H, P}));
    if (N < 1) return SSM_ERR_SHAPE;
    if (N > kMaxN) return SSM_ERR_UNSUPPORTED;
    if (Hk == 0 ? H != 0 : H % Hk != 0) return SSM_ERR_SHAPE;
    if (a->log_decay.ndim == 2) SSM_TRY(want(a->log_decay, {B, H}));
    else SSM_TRY(want(a->log_decay, {H}));
    const int io = a->q.dtype, st = a->state.dtype;
    if (!is_float(io) || a->k.dtype != io || a->v.dtype != io || a->out.dtype != io) return SSM_ERR_DTYPE;
    if (!is_float(st) || a->log_decay.dtype != SSM_F32) return SSM_ERR_DTYPE;
    const bool has_ix = present(a->state_batch_indices);
    if (has_ix) {
        SSM_TRY(basic(a->state_batch_indices));
        SSM_TRY(want(a->state_batch_indices, {B}));
        if (a->state_batch_indices.dtype != SSM_I32) return SSM_ERR_DTYPE;
    } else if (S != B) {
        return SSM_ERR_SHAPE;
    }
    const ssm_tensor& so = present(a->state_out) ? a->state_out : a->state;
    SSM_TRY(basic(so));
    SSM_TRY(want(so, {S, H, P, N}));
    if (so.dtype != st) return SSM_ERR_DTYPE;
    if (!non_overlapping(so) || !non_overlapping(a->out)) return SSM_ERR_STRIDE;
    const ssm_tensor* ins[] = {&a->q, &a->k, &a->v, &a->log_decay, &a->state_batch_indices};
    for (const ssm_tensor* t : ins) {
        if (!present(*t)) continue;
        if (overlap(a->out, *t) || overlap(so, *t)) return SSM_ERR_ALIAS;
    }
    if (overlap(a->out, a->state) || overlap(a->out, so)) return SSM_ERR_ALIAS;
    if (!same_view(a->state, so) && overlap(a->state, so)) return SSM_ERR_ALIAS;
    if (B * H * P == 0 || S == 0) {
        fill_info(a->info, SSM_KERNEL_NONE, 0, 0, 0, 0, 0);
        return SSM_OK;
    }
    const bool vec = rows16(a->state) && rows16(so);
    // rows without gaps: bulk copies
    const bool bulk = vec && (P == 1 || (a->state.stride[2] == N && so.stride[2] == N));
    const int64_t rows = bulk ? linattn_step_bulk_rows(st, N) : linattn_step_rows(st, N, vec);
    const int64_t blocks = (P + rows - 1) / rows;
    if (B * H > INT32_MAX / blocks) return SSM_ERR_UNSUPPORTED;
    const int items = (int)(B * H * blocks);
    const int kernel = bulk ? SSM_KERNEL_LINATTN_STEP_BULK : vec ? SSM_KERNEL_LINATTN_STEP : SSM_KERNEL_LINATTN_STEP_GENERIC;
    const bool dry = (a->flags & SSM_FLAG_DRY_RUN) != 0;
    const int dev = current_device(dry), sms = sm_count(dry, dev);
    LinAttnStepBulk plan{};
    if (bulk) {
        plan = linattn_step_bulk_plan(st, B * H, P, N, sms);
        fill_info(a->info, kernel, (int)plan.grid, linattn_step_block(), plan.smem, (int64_t)plan.rows * plan.blocks,
                  plan.units);
    } else {
        fill_info(a->info, kernel, items, linattn_step_block(), 0, rows, items);
    }
    if (dry) return SSM_OK;

    LinAttnStepProblem p{};
    p.Bn = B; p.H = H; p.Hk = Hk; p.N = N; p.P = P; p.slots = S; p.rep = H / Hk; p.io_dt = io; p.st_dt = st;
    p.q = a->q.data; p.q_b = sd(a->q, 0); p.q_h = sd(a->q, 1); p.q_n = sd(a->q, 2);
    p.k = a->k.data; p.k_b = sd(a->k, 0); p.k_h = sd(a->k, 1); p.k_n = sd(a->k, 2);
    p.v = a->v.data; p.v_b = sd(a->v, 0); p.v_h = sd(a->v, 1); p.v_p = sd(a->v, 2);
    p.g = static_cast<const float*>(a->log_decay.data);
    p.g_b = a->log_decay.ndim == 2 ? sd(a->log_decay, 0) : 0;
    p.g_h = sd(a->log_decay, a->log_decay.ndim - 1);
    p.s_in = a->state.data;
    p.si_b = sd(a->state, 0); p.si_h = sd(a->state, 1); p.si_p = sd(a->state, 2); p.si_n = sd(a->state, 3);
    p.s_out = so.data;
    p.so_b = sd(so, 0); p.so_h = sd(so, 1); p.so_p = sd(so, 2); p.so_n = sd(so, 3);
    if (has_ix) {
        p.slot_idx = static_cast<const int32_t*>(a->state_batch_indices.data);
        p.ix_b = sd(a->state_batch_indices, 0);
    }
    p.scale = a->scale;
    p.out = a->out.data; p.o_b = sd(a->out, 0); p.o_h = sd(a->out, 1); p.o_p = sd(a->out, 2);
    const cudaError_t e = bulk ? launch_linattn_step_bulk(p, plan, bounded_waits(), dev, stream)
                               : launch_linattn_step(p, kernel, items, stream);
    return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

// -------------------------------------------------------- paged attention --
constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // per sequence: positions are 32-bit in the kernels

ssm_status paged_impl(const ssm_paged_attention_args* a, cudaStream_t stream, uint64_t* ws_query) {
    if (!a) return SSM_ERR_NULL;
    if (a->struct_size != sizeof(ssm_paged_attention_args)) return SSM_ERR_VERSION;
    SSM_TRY(info_ok(a->info));
    for (const ssm_tensor* t : {&a->q, &a->k_cache, &a->v_cache, &a->block_table, &a->seq_lens, &a->out})
        SSM_TRY(basic(*t));
    if (a->q.ndim != 3 || a->k_cache.ndim != 4 || a->block_table.ndim != 2) return SSM_ERR_SHAPE;
    const int64_t B = a->q.shape[0], Hq = a->q.shape[1], D = a->q.shape[2];
    const int64_t pages = a->k_cache.shape[0], page = a->k_cache.shape[1], Hkv = a->k_cache.shape[2];
    const int64_t M = a->block_table.shape[1];
    SSM_TRY(want(a->k_cache, {pages, page, Hkv, D}));
    SSM_TRY(want(a->v_cache, {pages, page, Hkv, D}));
    SSM_TRY(want(a->block_table, {B, M}));
    SSM_TRY(want(a->seq_lens, {B}));
    SSM_TRY(want(a->out, {B, Hq, D}));
    if (D < 1 || page < 1) return SSM_ERR_SHAPE;
    if (Hkv == 0 ? Hq != 0 : Hq % Hkv != 0) return SSM_ERR_SHAPE;
    if (D > kMaxN || page > kMaxTokens || (M > 0 && page > kMaxTokens / M) || Hkv > 65535) return SSM_ERR_UNSUPPORTED;
    const int64_t cap = M * page;
    const int io = a->q.dtype;
    if (!is_float(io) || a->k_cache.dtype != io || a->v_cache.dtype != io || a->out.dtype != io) return SSM_ERR_DTYPE;
    if (a->block_table.dtype != SSM_I32 || a->seq_lens.dtype != SSM_I32) return SSM_ERR_DTYPE;
    const bool has_w = present(a->weights);
    const ssm_tensor& wo = present(a->weights_out) ? a->weights_out : a->weights;
    if (present(a->weights_out) && !has_w) return SSM_ERR_NULL;
    if (has_w) {
        for (const ssm_tensor* t : {&a->weights, &wo}) {
            SSM_TRY(basic(*t));
            if (t->ndim != 3 || t->shape[0] != B || t->shape[1] != Hkv || t->shape[2] < cap) return SSM_ERR_SHAPE;
            if (t->dtype != SSM_F32) return SSM_ERR_DTYPE;
        }
        if (!non_overlapping(wo)) return SSM_ERR_STRIDE;
        if (!same_view(a->weights, wo) && overlap(a->weights, wo)) return SSM_ERR_ALIAS;
    }
    const bool has_lse = present(a->lse);
    if (has_lse) {
        SSM_TRY(basic(a->lse));
        SSM_TRY(want(a->lse, {B, Hq}));
        if (a->lse.dtype != SSM_F32) return SSM_ERR_DTYPE;
        if (!non_overlapping(a->lse)) return SSM_ERR_STRIDE;
    }
    if (!non_overlapping(a->out)) return SSM_ERR_STRIDE;
    const ssm_tensor* ins[] = {&a->q, &a->k_cache, &a->v_cache, &a->block_table, &a->seq_lens};
    for (const ssm_tensor* t : ins) {
        if (overlap(a->out, *t)) return SSM_ERR_ALIAS;
        if (has_w && overlap(wo, *t)) return SSM_ERR_ALIAS;
        if (has_lse && overlap(a->lse, *t)) return SSM_ERR_ALIAS;
    }
    if (has_w && (overlap(a->out, a->weights) || overlap(a->out, wo))) return SSM_ERR_ALIAS;
    if (has_lse && (overlap(a->lse, a->out) || (has_w && (overlap(a->lse, a->weights) || overlap(a->lse, wo)))))
        return SSM_ERR_ALIAS;
    if (ws_query) *ws_query = 0;
    if (B * Hq == 0) {
        fill_info(a->info, SSM_KERNEL_NONE, 0, 0, 0, 0, 0);
        return SSM_OK;
    }
    const bool dry = (a->flags & SSM_FLAG_DRY_RUN) != 0;
    const bool mma = esize(io) == 2 && D <= 128 && rows16(a->q) && rows16(a->k_cache) && rows16(a->v_cache);
    const int kernel = mma ? SSM_KERNEL_PAGED_DECODE : SSM_KERNEL_PAGED_DECODE_GENERIC;

    PagedProblem p{};
    p.Bn = B; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.page = (int)page; p.pages = pages; p.M = M;
    p.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (page == (int64_t)1 << i) p.page_shift = i;
    p.G = Hq / Hkv; p.cap = cap; p.ws_cap = (cap + 3) / 4 * 4; p.io_dt = io;
    p.hpb = paged_heads_per_cta(kernel, p.G);
    p.hblocks = (int)((p.G + p.hpb - 1) / p.hpb);
    if (Hkv * p.hblocks > 65535 || B > (int64_t)INT32_MAX / Hq ||
        (has_w && B * Hkv > INT32_MAX / std::max<int64_t>(paged_weight_blocks(cap), 1)))
        return SSM_ERR_UNSUPPORTED;
    // ranges: as many CTAs as are resident at once, and no more than there can be tiles
    const int64_t heads = Hkv * p.hblocks, most = B * ((cap + 63) / 64);
    const int64_t slots = (int64_t)sm_count(dry) * paged_ctas_per_sm(kernel, p.G, D);
    p.workers = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(slots / heads, most), 65535));

    const uint64_t parts = (uint64_t)p.workers * heads * 2 * p.hpb;
    const uint64_t at_ml = round256(parts * D * 4), at_lse = at_ml + round256(parts * 8);
    const uint64_t at_s = at_lse + (has_w ? round256((uint64_t)B * Hq * 4) : 0);
    const uint64_t need = at_s + (has_w ? round256((uint64_t)B * Hq * p.ws_cap * 4) : 0);
    if (ws_query) {
        *ws_query = need;
        return SSM_OK;
    }
    fill_info(a->info, kernel, (int)(p.workers * heads), paged_block(), 0, p.hpb, p.workers * heads);
    if (!a->workspace && !dry) return SSM_ERR_WORKSPACE;
    if (a->workspace) {
        SSM_TRY(ws_ok(a->workspace, a->workspace_bytes, need));
        const ssm_tensor ws = ws_tensor(a->workspace, need);
        for (const ssm_tensor* t : {&a->q, &a->k_cache, &a->v_cache, &a->block_table, &a->seq_lens, &a->out, &a->lse,
                                    &a->weights, &wo})
            if (present(*t) && overlap(ws, *t)) return SSM_ERR_ALIAS;
    }
    if (dry) return SSM_OK;

    p.q = a->q.data; p.q_b = sd(a->q, 0); p.q_h = sd(a->q, 1); p.q_d = sd(a->q, 2);
    p.k = a->k_cache.data;
    p.k_g = sd(a->k_cache, 0); p.k_t = sd(a->k_cache, 1); p.k_h = sd(a->k_cache, 2); p.k_d = sd(a->k_cache, 3);
    p.v = a->v_cache.data;
    p.v_g = sd(a->v_cache, 0); p.v_t = sd(a->v_cache, 1); p.v_h = sd(a->v_cache, 2); p.v_d = sd(a->v_cache, 3);
    p.table = static_cast<const int32_t*>(a->block_table.data);
    p.tb_b = sd(a->block_table, 0); p.tb_m = sd(a->block_table, 1);
    p.lens = static_cast<const int32_t*>(a->seq_lens.data);
    p.len_b = sd(a->seq_lens, 0);
    if (has_w) {
        p.w = static_cast<const float*>(a->weights.data);
        p.w_b = sd(a->weights, 0); p.w_h = sd(a->weights, 1); p.w_t = sd(a->weights, 2);
        p.w_out = static_cast<float*>(wo.data);
        p.wo_b = sd(wo, 0); p.wo_h = sd(wo, 1); p.wo_t = sd(wo, 2);
    }
    if (has_lse) {
        p.lse = static_cast<float*>(a->lse.data);
        p.lse_b = sd(a->lse, 0); p.lse_h = sd(a->lse, 1);
    }
    p.scale_log2 = (float)((double)a->scale * 1.4426950408889634);
    p.out = a->out.data; p.o_b = sd(a->out, 0); p.o_h = sd(a->out, 1); p.o_d = sd(a->out, 2);
    char* ws = static_cast<char*>(a->workspace);
    p.ws_o = reinterpret_cast<float*>(ws);
    p.ws_ml = reinterpret_cast<float2*>(ws + at_ml);
    if (has_w) {
        p.ws_lse2 = reinterpret_cast<float*>(ws + at_lse);
        p.ws_s = reinterpret_cast<float*>(ws + at_s);
    }
    return launch_paged(p, kernel, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

// --------------------------------------------------------------- eviction --
ssm_status evict_impl(const ssm_kv_evict_args* a, cudaStream_t stream) {
    if (!a) return SSM_ERR_NULL;
    if (a->struct_size != sizeof(ssm_kv_evict_args)) return SSM_ERR_VERSION;
    SSM_TRY(info_ok(a->info));
    for (const ssm_tensor* t : {&a->k_cache, &a->v_cache, &a->weights, &a->block_table, &a->seq_lens,
                                &a->new_block_table, &a->new_weights, &a->new_seq_lens, &a->kept})
        SSM_TRY(basic(*t));
    if (a->k_cache.ndim != 4 || a->block_table.ndim != 2 || a->new_block_table.ndim != 2) return SSM_ERR_SHAPE;
    const int64_t pages = a->k_cache.shape[0], page = a->k_cache.shape[1], Hkv = a->k_cache.shape[2],
                  D = a->k_cache.shape[3];
    const int64_t B = a->block_table.shape[0], M = a->block_table.shape[1], M2 = a->new_block_table.shape[1];
    SSM_TRY(want(a->v_cache, {pages, page, Hkv, D}));
    SSM_TRY(want(a->new_block_table, {B, M2}));
    SSM_TRY(want(a->seq_lens, {B}));
    SSM_TRY(want(a->new_seq_lens, {B}));
    if (page < 1 || a->keep < 1 || a->recent < 0 || a->recent > a->keep) return SSM_ERR_SHAPE;
    if (page > kMaxTokens || (M > 0 && page > kMaxTokens / M) || (M2 > 0 && page > kMaxTokens / M2) ||
        a->keep > kMaxTokens)
        return SSM_ERR_UNSUPPORTED;
    const int64_t cap = M * page;
    if (M2 * page < a->keep) return SSM_ERR_SHAPE;
    if (a->weights.ndim != 3 || a->weights.shape[0] != B || a->weights.shape[1] != Hkv || a->weights.shape[2] < cap)
        return SSM_ERR_SHAPE;
    SSM_TRY(want(a->new_weights, {B, Hkv, a->keep}));
    SSM_TRY(want(a->kept, {B, Hkv, a->keep}));
    if (!is_float(a->k_cache.dtype) || a->v_cache.dtype != a->k_cache.dtype) return SSM_ERR_DTYPE;
    if (a->weights.dtype != SSM_F32 || a->new_weights.dtype != SSM_F32) return SSM_ERR_DTYPE;
    for (const ssm_tensor* t : {&a->block_table, &a->seq_lens, &a->new_block_table, &a->new_seq_lens, &a->kept})
        if (t->dtype != SSM_I32) return SSM_ERR_DTYPE;
    // (the two caches may be interleaved in one buffer: their extents may overlap)
    const ssm_tensor* outs[] = {&a->k_cache, &a->v_cache, &a->new_weights, &a->new_seq_lens, &a->kept};
    const ssm_tensor* ins[] = {&a->weights, &a->block_table, &a->seq_lens, &a->new_block_table};
    for (int i = 0; i < 5; ++i) {
        if (!non_overlapping(*outs[i])) return SSM_ERR_STRIDE;
        for (const ssm_tensor* t : ins)
            if (overlap(*outs[i], *t)) return SSM_ERR_ALIAS;
        for (int j = i < 2 ? 2 : i + 1; j < 5; ++j)
            if (overlap(*outs[i], *outs[j])) return SSM_ERR_ALIAS;
    }
    if (B == 0 || Hkv == 0) {
        fill_info(a->info, SSM_KERNEL_NONE, 0, 0, 0, 0, 0);
        return SSM_OK;
    }
    if (B > INT32_MAX / Hkv) return SSM_ERR_UNSUPPORTED;
    const bool dry = (a->flags & SSM_FLAG_DRY_RUN) != 0;
    EvictProblem p{};
    p.Bn = B; p.Hkv = Hkv; p.D = D; p.page = (int)page; p.pages = pages; p.M = M; p.M2 = M2; p.cap = cap;
    p.keep = a->keep; p.recent = a->recent; p.es = esize(a->k_cache.dtype);
    const bool vec = D > 0 && rows16(a->k_cache) && rows16(a->v_cache);
    if (B > INT32_MAX / evict_copy_ctas(a->keep) || Hkv > (1 << 25) || D > (1 << 20)) return SSM_ERR_UNSUPPORTED;
    fill_info(a->info, SSM_KERNEL_KV_EVICT, (int)(B * Hkv), evict_select_block(), 0, 1, B * Hkv);
    if (dry) return SSM_OK;

    p.k = a->k_cache.data;
    p.k_g = sd(a->k_cache, 0); p.k_t = sd(a->k_cache, 1); p.k_h = sd(a->k_cache, 2); p.k_d = sd(a->k_cache, 3);
    p.v = a->v_cache.data;
    p.v_g = sd(a->v_cache, 0); p.v_t = sd(a->v_cache, 1); p.v_h = sd(a->v_cache, 2); p.v_d = sd(a->v_cache, 3);
    p.w = static_cast<const float*>(a->weights.data);
    p.w_b = sd(a->weights, 0); p.w_h = sd(a->weights, 1); p.w_t = sd(a->weights, 2);
    p.table = static_cast<const int32_t*>(a->block_table.data);
    p.tb_b = sd(a->block_table, 0); p.tb_m = sd(a->block_table, 1);
    p.lens = static_cast<const int32_t*>(a->seq_lens.data); p.len_b = sd(a->seq_lens, 0);
    p.new_table = static_cast<const int32_t*>(a->new_block_table.data);
    p.nt_b = sd(a->new_block_table, 0); p.nt_m = sd(a->new_block_table, 1);
    p.new_w = static_cast<float*>(a->new_weights.data);
    p.nw_b = sd(a->new_weights, 0); p.nw_h = sd(a->new_weights, 1); p.nw_j = sd(a->new_weights, 2);
    p.new_lens = static_cast<int32_t*>(a->new_seq_lens.data); p.nl_b = sd(a->new_seq_lens, 0);
    p.kept = static_cast<int32_t*>(a->kept.data);
    p.kp_b = sd(a->kept, 0); p.kp_h = sd(a->kept, 1); p.kp_j = sd(a->kept, 2);
    return launch_evict(p, vec, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

}  // namespace

extern "C" {

ssm_status ssm_linear_attention_fwd(const ssm_linattn_args* args, void* stream) {
    return linattn_impl(args, static_cast<cudaStream_t>(stream), nullptr);
}

ssm_status ssm_linear_attention_workspace_size(const ssm_linattn_args* args, uint64_t* bytes) {
    if (!bytes) return SSM_ERR_NULL;
    return linattn_impl(args, nullptr, bytes);
}

ssm_status ssm_linear_attention_update(const ssm_linattn_update_args* args, void* stream) {
    return linattn_update_impl(args, static_cast<cudaStream_t>(stream));
}

ssm_status ssm_paged_attention_decode(const ssm_paged_attention_args* args, void* stream) {
    return paged_impl(args, static_cast<cudaStream_t>(stream), nullptr);
}

ssm_status ssm_paged_attention_workspace_size(const ssm_paged_attention_args* args, uint64_t* bytes) {
    if (!bytes) return SSM_ERR_NULL;
    return paged_impl(args, nullptr, bytes);
}

ssm_status ssm_kv_cache_evict(const ssm_kv_evict_args* args, void* stream) {
    return evict_impl(args, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
