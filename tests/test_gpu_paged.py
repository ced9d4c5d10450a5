"""GPU parity of attention of one token over a paged cache, and of eviction
from that cache, against their float64 definitions.

Tolerances of the attention.  A score is a sum of D products in float32 of
magnitude at most X = scale max_t sum |q||k| (and is scaled to base 2): off by at most
e = (D + 4) 2^-24 X.  A weight is then off by a factor of exp(2 e) at most, and by the
exponential's own error and those of the running sums, at most (n / 16 + 64)
roundings of 2^-22: w = 2 e + (n / 16 + 64) 2^-22.  The values' weighted sum of
magnitude M = sum p |v| is off by (w + c) M, where c = 2^-16 for the tensor
cores' remainder of a weight rounded to 16 bits, or 2^-8 (bf16), 2^-11 (f16)
where a group of more than 8 heads rounds it once.  The output is rounded once: + u |ref|.
"""
import numpy as np
import pytest

from oracle import attention as ref
from state_space_model_causal_b200 import inputs as gen
from tests.parity import N as to_np
from tests.parity import T

pytestmark = pytest.mark.gpu

UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


def cache(pools, page, Hkv, D, io, *tags):
    return [gen.round_to(gen.normal((pools, page, Hkv, D), "paged", x, *tags), io) for x in ("k", "v")]


def table_for(B, M, pool, seed=0):
    return np.random.RandomState(seed).permutation(pool)[: B * M].reshape(B, M).astype(np.int32)


def run(q, k, v, table, lens, scale, io, weights=None, in_place=False, device_kv=None):
    import torch
    from state_space_model_causal_b200 import LaunchInfo, binding, ssm_device_error, ssm_paged_attention_decode
    tk, tv = device_kv if device_kv is not None else (T(k, io), T(v, io))
    info = LaunchInfo()
    B, Hq, _ = q.shape
    lse = torch.full((B, Hq), 5.0, device="cuda")
    w = None if weights is None else T(weights, "f32")
    wo = None if weights is None or in_place else torch.full_like(w, 9.0)
    out = ssm_paged_attention_decode(T(q, io), tk, tv, torch.tensor(table, device="cuda"),
                                     torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=scale, weights=w,
                                     weights_out=wo, lse=lse, info=info)
    torch.cuda.synchronize()
    assert ssm_device_error() == 0
    return to_np(out), to_np(lse), to_np(w if in_place else wo), binding.KERNELS[info.kernel]


def check(q, k, v, table, lens, scale, io, weights=None, in_place=False, device_kv=None, kernel=None):
    out, ps, lse, mag, spread = ref.paged_attention(q, k, v, table, lens, scale)
    got, gl, gw, kern = run(q, k, v, table, lens, scale, io, weights, in_place, device_kv)
    if kernel:
        assert kern == kernel
    B, Hq, D = q.shape
    rep = Hq // k.shape[2]
    n = np.array([p.shape[1] for p in ps])
    e = (D + 4) * 2.0 ** -24 * spread
    w = 2 * e + (n[:, None] / 16 + 64) * 2.0 ** -22
    c = 0.0 if kern != "paged_decode" else (2.0 ** -16 if rep <= 8 else UNIT[io])
    bound = UNIT[io] * np.abs(out) + (w + c)[..., None] * mag + TINY[io]
    worst = np.max(np.abs(got - out) / (bound + 1e-30))
    assert worst <= 1, f"worst {worst:.2f} bounds ({kern})"
    live = lse > -np.inf
    assert (gl[~live] == -np.inf).all()
    assert (np.abs(gl[live] - lse[live]) <= w[live] + 2.0 ** -22 * np.abs(lse[live])).all()
    if weights is not None:
        expect = weights.copy() if in_place else np.full(weights.shape, 9.0)
        tol = np.zeros(weights.shape)
        for b, p in enumerate(ps):
            add = p.reshape(k.shape[2], rep, n[b]).sum(1)
            expect[b, :, : n[b]] = weights[b, :, : n[b]] + add
            worst_w = 2 * w[b].max()  # numerator and denominator
            tol[b, :, : n[b]] = worst_w * add + rep * 2.0 ** -22 * add + 2.0 ** -23 * np.abs(expect[b, :, : n[b]]) + 1e-37
        assert (np.abs(gw - expect) <= tol).all()
    return got


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ([1], 1, 1, 64, 16), ([2, 17, 0, 63], 4, 2, 64, 16), ([64, 65, 127, 128], 8, 1, 128, 16),
    ([1000], 32, 8, 128, 16), ([300, 5, 0, 0, 700], 6, 3, 96, 24), ([129, 1], 16, 1, 64, 7),
    ([333, 500], 24, 1, 128, 32), ([0, 0], 4, 4, 64, 8), ([77, 200], 5, 5, 80, 1), ([90], 3, 1, 256, 16),
    ([90, 40], 4, 2, 40, 16), ([55, 21], 34, 2, 33, 10), ([5000], 2, 2, 64, 64), ([1] * 140, 2, 1, 64, 16)])
def test_attention_matches_definition(io, lens, Hq, Hkv, D, page):
    """One token, none, tile and page borders, pages that end inside a tile,
    groups of 1 to 24 heads, odd sizes, many short sequences, a long one."""
    B, M = len(lens), -(-max(max(lens), 1) // page)
    k, v = cache(B * M + 2, page, Hkv, D, io, tuple(lens), Hq, D)
    q = gen.round_to(gen.normal((B, Hq, D), "paged", "q", tuple(lens), Hq, D), io)
    check(q, k, v, table_for(B, M, B * M + 2), lens, D ** -0.5, io)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("io,lens,Hq,Hkv,D,page", [("f16", [700, 3, 0, 129], 8, 2, 64, 16), ("bf16", [260, 2000], 40, 4, 128, 32),
                                                   ("f32", [70, 500], 6, 3, 72, 24), ("bf16", [513], 12, 1, 96, 16)])
def test_accumulated_weights(io, lens, Hq, Hkv, D, page, in_place):
    B, M = len(lens), -(-max(lens) // page)
    k, v = cache(B * M, page, Hkv, D, io, "w", tuple(lens))
    q = gen.round_to(gen.normal((B, Hq, D), "paged", "wq", tuple(lens)), io)
    w = gen.round_to(gen.uniform((B, Hkv, M * page + 5), 0, 2, "paged", "w", tuple(lens)), "f32")
    check(q, k, v, table_for(B, M, B * M), lens, D ** -0.5, io, weights=w, in_place=in_place)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_pages_that_do_not_exist_and_garbage_behind_the_end(io):
    """Page indices -1 and past the pool hold no tokens (a sequence of such
    pages only is empty); rows behind the end, and whole pages that nobody
    names, may hold NaN.  Lengths beyond the table are limited to it."""
    page, M, B, Hq, Hkv, D = 16, 6, 4, 4, 2, 64
    k, v = cache(B * M + 4, page, Hkv, D, io, "bad")
    q = gen.round_to(gen.normal((B, Hq, D), "paged", "badq"), io)
    table = table_for(B, M, B * M + 4)
    lens = [90, 50, 96, 5000]
    table[0, 1], table[0, 5] = -1, B * M + 4
    table[1, :] = -7
    table[2, 0] = 2 ** 31 - 1
    named = np.zeros(B * M + 4, bool)
    named[table[(table >= 0) & (table < B * M + 4)]] = True
    k[~named], v[~named] = np.nan, np.inf
    last = table[0, 4]  # 90 tokens end in row 10 of page 5 (out of range); cut page 4 of sequence 3 short instead
    lens[3] = 4 * page + 5
    k[table[3, 4], 5:], v[table[3, 4], 5:] = np.nan, np.nan
    k[table[3, 5]], v[table[3, 5]] = np.nan, np.nan
    assert last >= 0
    check(q, k, v, table, lens, 0.3, io, weights=np.ones((B, Hkv, M * page)))
    k, v = cache(B * M + 4, page, Hkv, D, io, "bad2")
    check(q, k, v, table_for(B, M, B * M + 4), [5000, 96, -3, 97], 0.3, io)


@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_extreme_scores(io):
    """One token far above the others, scores of hundreds, and equal scores."""
    page, M, D = 16, 20, 64
    k, v = cache(M, page, 1, D, io, "ext")
    q = gen.round_to(gen.normal((1, 4, D), "paged", "extq", std=30.0), io)
    q[0, 3] = 0.0
    k[7, 3] = q[0, 0] / 4
    check(q, gen.round_to(k, io), v, np.arange(M, dtype=np.int32)[None], [300], 1.0, io)


def test_keys_and_values_interleaved_in_one_pool():
    """K and V as views of one (pages, 2, page, Hkv, D) pool, heads before rows
    in memory, a broadcast table."""
    import torch
    io, page, Hkv, D, M = "bf16", 16, 2, 64, 5
    k, v = cache(M, page, Hkv, D, io, "inter")
    pool = torch.stack([T(k, io), T(v, io)], dim=1).transpose(2, 3).contiguous().transpose(2, 3)
    table = np.broadcast_to(np.arange(M, dtype=np.int32), (3, M))
    q = gen.round_to(gen.normal((3, 4, D), "paged", "inter", "q"), io)
    check(q, k, v, table, [80, 33, 7], 0.125, io, device_kv=(pool[:, 0], pool[:, 1]), kernel="paged_decode")


def test_a_nan_in_the_cache_reaches_its_row_only():
    import torch
    page, M, D = 16, 8, 64
    k, v = cache(2 * M, page, 1, D, "bf16", "nan")
    k[3, 2, 0, 5] = np.nan
    q = gen.round_to(gen.normal((2, 2, D), "paged", "nanq"), "bf16")
    table = np.arange(2 * M, dtype=np.int32).reshape(2, M)
    got, lse, _, _ = run(q, k, v, table, [128, 128], 0.1, "bf16")
    assert np.isnan(got[0]).all() and np.isnan(lse[0]).all()
    assert np.isfinite(got[1]).all() and np.isfinite(lse[1]).all()


def test_the_same_call_twice_gives_the_same_bits():
    page, M, B = 32, 64, 3
    k, v = cache(B * M, page, 2, 128, "bf16", "bits")
    q = gen.round_to(gen.normal((B, 16, 128), "paged", "bitsq"), "bf16")
    args = (q, k, v, table_for(B, M, B * M), [2048, 1500, 9], 0.09, "bf16")
    first, again = run(*args), run(*args)
    np.testing.assert_array_equal(first[0], again[0])
    np.testing.assert_array_equal(first[1], again[1])


# --------------------------------------------------------------- eviction --
def run_evict(k, v, w, table, lens, new_table, keep, recent, io):
    import torch
    from state_space_model_causal_b200 import ssm_kv_cache_evict
    tk, tv = T(k, io), T(v, io)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    n, kept, nw = ssm_kv_cache_evict(tk, tv, T(w, "f32"), i32(table), i32(lens), i32(new_table), keep, recent=recent)
    torch.cuda.synchronize()
    return n.cpu().numpy(), kept.cpu().numpy(), to_np(nw), to_np(tk), to_np(tv)


def check_evict(k, v, w, table, lens, new_table, keep, recent, io):
    n, kept, nw, gk, gv = run_evict(k, v, w, table, lens, new_table, keep, recent, io)
    pages, page = k.shape[:2]
    want = ref.evict(w, table, lens, pages, page, keep, recent)
    ek, ev = k.copy(), v.copy()
    for b in range(len(lens)):
        assert n[b] == len(want[b][0])
        for h in range(k.shape[2]):
            idx = want[b][h]
            np.testing.assert_array_equal(kept[b, h], idx + [-1] * (keep - len(idx)))
            np.testing.assert_array_equal(nw[b, h], np.concatenate([w[b, h, idx], np.zeros(keep - len(idx))]))
            for j, t in enumerate(idx):
                to = new_table[b][j // page]
                if 0 <= to < pages:
                    ek[to, j % page, h] = k[table[b][t // page], t % page, h]
                    ev[to, j % page, h] = v[table[b][t // page], t % page, h]
    np.testing.assert_array_equal(gk, ek)
    np.testing.assert_array_equal(gv, ev)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,Hkv,D,page,keep,recent", [
    ([1], 1, 64, 16, 1, 0), ([40, 0, 17, 5], 2, 64, 16, 16, 4), ([1000, 300], 3, 96, 24, 250, 32),
    ([513, 2048, 2049], 2, 33, 16, 512, 512), ([600], 1, 64, 7, 599, 0), ([64, 64], 4, 128, 32, 200, 10),
    ([5000], 1, 8, 64, 1, 1)])
def test_eviction_matches_definition(io, lens, Hkv, D, page, keep, recent):
    """Equal weights (a quarter of them are 0, some are -0), more room than
    tokens, nothing but recent tokens, steps of the selection and neighbours."""
    B, M, M2 = len(lens), -(-max(lens) // page), -(-keep // page)
    pool = B * (M + M2)
    k, v = cache(pool, page, Hkv, D, io, "ev", tuple(lens))
    tabs = table_for(B, M + M2, pool)
    w = gen.round_to(np.round(gen.uniform((B, Hkv, M * page), -4, 12, "ev", tuple(lens))) / 8, "f32")
    w[w < 0] *= np.arange(1, 1 + (w < 0).sum()) % 2  # 0, -0 and negative numbers
    check_evict(k, v, w, tabs[:, :M], lens, tabs[:, M:], keep, recent, io)


def test_eviction_of_odd_weights_and_bad_pages():
    """Infinities, NaN and subnormal weights; pages that do not exist on either side;
    lengths past the table and negative ones."""
    B, Hkv, page, M, keep = 3, 2, 16, 10, 40
    pool = B * (M + 3)
    k, v = cache(pool, page, Hkv, 64, "bf16", "evbad")
    tabs = table_for(B, M + 3, pool)
    w = gen.round_to(gen.normal((B, Hkv, M * page + 3), "ev", "odd", std=1e-39), "f32")
    w[:, :, ::9], w[:, :, 4::11], w[:, :, 5::13] = np.nan, np.inf, -np.inf
    w[1, 0] = np.nan  # nothing but NaN: the lowest positions
    table, new_table = tabs[:, :M].copy(), tabs[:, M:].copy()
    table[0, 2], table[0, 9] = -1, pool
    new_table[2, 1] = -5
    check_evict(k, v, w, table, [5000, 150, 155], new_table, keep, 10, "bf16")
    check_evict(k, v, w, table, [3 * page, -4, 0], new_table, keep, 0, "bf16")


def test_decode_evict_decode():
    """As a serving loop uses them: attention steps that accumulate weights, an
    eviction, and a step over the smaller cache, against the definitions."""
    import torch
    from state_space_model_causal_b200 import ssm_kv_cache_evict, ssm_paged_attention_decode
    io, B, Hq, Hkv, D, page, M = "bf16", 2, 8, 2, 64, 16, 20
    pool = 2 * B * M
    k, v = cache(pool, page, Hkv, D, io, "loop")
    tabs = table_for(B, 2 * M, pool)
    lens, keep, recent = [300, 120], 100, 16
    tk, tv = T(k, io), T(v, io)
    tt, tn = torch.tensor(tabs[:, :M].copy(), device="cuda"), torch.tensor(tabs[:, M:].copy(), device="cuda")
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w = torch.zeros(B, Hkv, M * page, device="cuda")
    for step in range(3):
        q = gen.round_to(gen.normal((B, Hq, D), "paged", "loop", step), io)
        ssm_paged_attention_decode(T(q, io), tk, tv, tt, tl, weights=w)
    n2, kept, w2 = ssm_kv_cache_evict(tk, tv, w, tt, tl, tn, keep, recent=recent)
    want = ref.evict(to_np(w), tabs[:, :M], lens, pool, page, keep, recent)
    for b in range(B):
        for h in range(Hkv):
            np.testing.assert_array_equal(kept[b, h].cpu().numpy()[: len(want[b][h])], want[b][h])
    q = gen.round_to(gen.normal((B, Hq, D), "paged", "loop", "last"), io)
    out = ssm_paged_attention_decode(T(q, io), tk, tv, tn, n2)
    r, _, _, mag, spread = ref.paged_attention(q, to_np(tk), to_np(tv), tabs[:, M:], [100, 100], D ** -0.5)
    e = (D + 4) * 2.0 ** -24 * spread
    bound = UNIT[io] * np.abs(r) + (2 * e + 80 * 2.0 ** -22 + 2.0 ** -16)[..., None] * mag
    assert (np.abs(to_np(out) - r) <= bound).all()
