"""GPU parity of linear attention with a decay per head (a prompt and one
token) against its float64 definition.

Tolerances.  Let M be the same computation on absolute values (|q|, |k|, |v|,
|S0|): every rounding made on the way to an output is at most its unit times
M.  u = eps / 2 is a type's unit, 2^-24 that of float32.

* float32 arithmetic over L tokens and N keys rounds each contribution to an
  output at most once per token it is carried over for the decay and once for
  the addition, then N times in the sum: (2 L + N + 8) 2^-24 M.  The decay
  itself is exp of a float32 number, 2 units at most per token: + 2 L 2^-24 M.
* the chunk kernel rounds two factors of each product to the I/O type (scores,
  and the state that queries read): 2 u M for the output; its state sums
  products of weighted values split into numbers of the I/O type (two for f16,
  three for bf16), whose remainder is at most u^2 (f16) or u^3 (bf16): + 2^-22 M.
* an output is rounded to its type once: u |ref|.
"""
import numpy as np
import pytest

from oracle import attention as ref
from state_space_model_causal_b200 import inputs as gen
from tests.parity import N as to_np
from tests.parity import T

pytestmark = pytest.mark.gpu

UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}  # half the smallest subnormal


def draw(shape, io, *tags, std=1.0):
    return gen.round_to(gen.normal(shape, "linattn", *tags, std=std), io)


def problem(B, H, Hk, L, N, P, io, decay, seed=0, state=True):
    q = draw((B, Hk, L, N), io, seed, "q", B, H, L, N, P)
    k = draw((B, Hk, L, N), io, seed, "k", B, H, L, N, P, std=N ** -0.5)
    v = draw((B, H, L, P), io, seed, "v", B, H, L, N, P)
    shape = (H,) if decay == "head" else (B, H, L)
    g = gen.round_to(-np.exp(gen.uniform(shape, -6.0, 0.5, "linattn", seed, "g", B, H, L)), "f32")
    s0 = gen.round_to(gen.normal((B, H, P, N), "linattn", seed, "s", B, H, N, P), "f32") if state else None
    return q, k, v, g, s0


def token_major(a, io):
    """(B, H, L, X) values as a transposed view of (B, L, H, X) storage."""
    return T(a.transpose(0, 2, 1, 3), io).transpose(1, 2)


def bounds(q, k, v, g, s0, scale, lens, io, ref_out, chunk):
    """Elementwise bounds of out and state (see the module's docstring)."""
    mo, ms = ref.linear_attention(np.abs(q), np.abs(k), np.abs(v), g, abs(scale),
                                  None if s0 is None else np.abs(s0), lens)
    L, N = q.shape[2], q.shape[3]
    f32 = (4 * L + N + 8) * 2.0 ** -24
    u = UNIT[io]
    out = u * np.abs(ref_out) + (f32 + (2 * u if chunk else 0.0)) * mo + TINY[io]
    return out, (f32 + (2.0 ** -22 if chunk else 0.0)) * ms


def run(q, k, v, g, s0, scale=1.0, lens=None, io="f32", layout="token", workspace="auto", in_place=False):
    import torch
    from state_space_model_causal_b200 import LaunchInfo, binding, ssm_device_error, ssm_linear_attention_fwd
    put = token_major if layout == "token" else T
    tq, tk, tv = (put(a, io) for a in (q, k, v))
    st = T(s0, "f32") if s0 is not None else None
    so = st if in_place else torch.full((v.shape[0], v.shape[1], v.shape[3], q.shape[3]), 7.0, device="cuda")
    out = torch.full_like(tv, 3.0)
    li = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    info = LaunchInfo()
    ssm_linear_attention_fwd(tq, tk, tv, T(g, "f32"), scale=scale, state=st, state_out=so, seq_lens=li,
                             out=out, info=info, workspace=workspace)
    torch.cuda.synchronize()
    assert ssm_device_error() == 0
    return to_np(out), to_np(so), binding.KERNELS[info.kernel]


def check(args, scale, lens, io, got_out, got_state, kernel):
    q, k, v, g, s0 = args
    out, S = ref.linear_attention(q, k, v, g, scale, s0, lens)
    chunk = kernel == "linattn_chunk"
    live = ~np.isnan(out)
    bo, bs = bounds(q, k, v, g, s0, scale, lens, io, np.where(live, out, 0.0), chunk)
    assert np.isfinite(got_out).all() and np.isfinite(got_state).all()
    np.testing.assert_array_equal(got_out[~live], 3.0)  # rows that are not there: left as they were
    bad = np.abs(got_out - out)[live] > bo[live]
    assert not bad.any(), f"{bad.sum()} outputs off, worst {np.nanmax(np.abs(got_out - out) / bo):.2f} bounds"
    bad = np.abs(got_state - S) > bs + 1e-30
    assert not bad.any(), f"{bad.sum()} states off, worst {np.max(np.abs(got_state - S) / (bs + 1e-30)):.2f} bounds"


@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,H,Hk,L,N,P", [
    (1, 1, 1, 1, 64, 64), (2, 3, 3, 7, 32, 16), (1, 2, 1, 127, 64, 64), (1, 2, 2, 128, 128, 64),
    (2, 4, 2, 129, 128, 128), (1, 3, 1, 300, 96, 72), (1, 1, 1, 513, 128, 192), (3, 2, 2, 65, 8, 8),
    (1, 2, 2, 40, 200, 24), (1, 2, 1, 33, 17, 5), (1, 1, 1, 1000, 64, 128)])
def test_prompt_matches_definition(io, decay, B, H, Hk, L, N, P):
    """One token, chunk borders and their neighbours, many chunks, shared keys,
    sizes that are no multiple of a tile or of a vector."""
    args = problem(B, H, Hk, L, N, P, io, decay)
    out, S, kern = run(*args, scale=N ** -0.5, io=io)
    check(args, N ** -0.5, None, io, out, S, kern)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_strides_and_no_state(io):
    """(B, H, L, X) storage instead of token-major, no initial state."""
    args = problem(2, 3, 3, 150, 64, 64, io, "token", state=False)
    out, S, kern = run(*args, io=io, layout="head")
    check(args, 1.0, None, io, out, S, kern)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_padded_batch_with_garbage_behind_the_end(io):
    """Lengths 0, 1, a chunk border, beyond the tensor (limited) and negative
    (none); NaN and infinities behind the ends reach nothing."""
    L = 300
    lens = [0, 1, 128, 129, 300, 1000, -5]
    q, k, v, g, s0 = problem(7, 2, 1, L, 64, 64, io, "token", seed=3)
    for b, n in enumerate(np.clip(lens, 0, L)):
        q[b, :, n:], k[b, :, n:], v[b, :, n:], g[b, :, n:] = np.nan, np.inf, -np.inf, np.nan
    out, S, kern = run(q, k, v, g, s0, lens=lens, io=io)
    clean = [np.where(np.isfinite(a), a, 0.0) for a in (q, k, v, g)]
    check((*clean, s0), 1.0, lens, io, out, S, kern)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_what_is_not_finite_reaches_no_earlier_token(io, in_place):
    """Infinities and NaN among the values and keys of a sequence: the outputs before
    their token, and the other columns and heads, are what they are without them."""
    q, k, v, g, s0 = problem(1, 3, 3, 300, 64, 96, io, "token", seed=9)
    bad_v, bad_k = v.copy(), k.copy()
    bad_v[0, 0, 70, 5], bad_v[0, 0, 200, 66], bad_v[0, 1, 0, 0], bad_v[0, 1, 299, 95] = np.inf, np.nan, -np.inf, np.inf
    bad_k[0, 1, 290, 3] = np.nan
    clean = q, np.where(np.isfinite(bad_k), k, 0.0), np.where(np.isfinite(bad_v), v, 0.0), g, s0
    reach, state_reach = np.zeros(v.shape, bool), np.zeros(s0.shape, bool)
    reach[0, 0, 70:, 5] = reach[0, 0, 200:, 66] = reach[0, 1, :, 0] = reach[0, 1, 299:, 95] = reach[0, 1, 290:] = True
    state_reach[0, 0, [5, 66]] = state_reach[0, 1, [0, 95]] = state_reach[0, 1, :, 3] = True
    out, S, kern = run(q, bad_k, bad_v, g, s0, io=io, in_place=in_place)
    assert not np.isfinite(out[reach]).any() and not np.isfinite(S[state_reach]).any()
    ref_out, ref_S = ref.linear_attention(*clean[:4], 1.0, s0, None)
    check(clean, 1.0, None, io, np.where(reach, ref_out, out), np.where(state_reach, ref_S, S), kern)


@pytest.mark.parametrize("bad", [np.inf, np.nan])
def test_small_values_beside_one_that_is_not_finite(bad):
    """float16 values far below 1, which its two numbers hold by a common power of two:
    what is not finite has no part in that."""
    q, k, v, g, s0 = problem(1, 1, 1, 40, 64, 64, "f16", "token", seed=11, state=False)
    v = gen.round_to(v * 1e-4, "f16")
    bad_v, clean = v.copy(), v.copy()
    bad_v[0, 0, 30, 7], clean[0, 0, 30, 7] = bad, 0.0
    reach, state_reach = np.zeros(v.shape, np.bool_), np.zeros((1, 1, 64, 64), np.bool_)
    reach[0, 0, 30:, 7] = state_reach[0, 0, 7] = True
    out, S, kern = run(q, k, bad_v, g, s0, io="f16")
    assert kern == "linattn_chunk" and not np.isfinite(out[reach]).any() and not np.isfinite(S[state_reach]).any()
    ref_out, ref_S = ref.linear_attention(q, k, clean, g, 1.0, s0, None)
    check((q, k, clean, g, s0), 1.0, None, "f16", np.where(reach, ref_out, out), np.where(state_reach, ref_S, S), kern)


@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_what_is_not_finite_in_pieces_of_a_long_sequence(io):
    """As above where sequences are cut into pieces: in the first, in the others and in
    a padded end."""
    q, k, v, g, s0 = problem(2, 1, 1, 2500, 64, 64, io, "token", seed=10)
    bad = v.copy()
    bad[0, 0, 100, 3], bad[0, 0, 1200, 40], bad[0, 0, 2499, 63] = np.nan, np.inf, -np.inf
    bad[1, 0, 2000, 5], bad[1, 0, 2101:] = np.inf, np.nan
    lens = [2500, 2101]
    reach, state_reach = np.zeros(v.shape, bool), np.zeros(s0.shape, bool)
    reach[0, 0, 100:, 3] = reach[0, 0, 1200:, 40] = reach[0, 0, 2499:, 63] = reach[1, 0, 2000:2101, 5] = True
    state_reach[0, 0, [3, 40, 63]] = state_reach[1, 0, 5] = True
    clean = q, k, np.where(np.isfinite(bad), v, 0.0), g, s0
    out, S, kern = run(q, k, bad, g, s0, io=io, lens=lens)
    assert kern == "linattn_chunk" and not np.isfinite(out[reach]).any() and not np.isfinite(S[state_reach]).any()
    ref_out, ref_S = ref.linear_attention(*clean[:4], 1.0, s0, lens)
    check(clean, 1.0, lens, io, np.where(reach, ref_out, out), np.where(state_reach, ref_S, S), kern)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_decay_extremes(io):
    """No decay at all, a decay that forgets everything (log decay -inf) in the
    middle of a chunk, and one so strong that its sum over a chunk passes
    float32's exponent range."""
    q, k, v, g, s0 = problem(1, 3, 3, 290, 64, 64, io, "token", seed=4)
    g[:, 0] = 0.0
    g[:, 1] = -1e-3
    g[:, 1, [5, 130, 131, 200]] = -np.inf
    g[:, 2] = -300.0
    g[:, 2, ::7] = -1e-4
    out, S, kern = run(q, k, v, g, s0, io=io)
    check((q, k, v, g, s0), 1.0, None, io, out, S, kern)


@pytest.mark.parametrize("io", ["bf16", "f16"])
def test_large_values(io):
    """Scores and states far past float16's largest number; outputs brought
    back into range by the scale."""
    q, k, v, g, s0 = problem(1, 2, 2, 200, 128, 64, io, "head", seed=5)
    q, k, s0 = q * 64, gen.round_to(k * 512, io), s0 * 2.0 ** 20
    scale = 2.0 ** -28
    out, S, kern = run(q, k, v, g, s0, scale=scale, io=io)
    check((q, k, v, g, s0), scale, None, io, out, S, kern)


def test_zero_length_prompt_copies_the_state():
    import torch
    from state_space_model_causal_b200 import ssm_linear_attention_fwd
    q = torch.zeros(2, 3, 0, 64, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros(2, 3, 0, 64, device="cuda", dtype=torch.bfloat16)
    s0 = torch.randn(2, 3, 64, 64, device="cuda")
    so = torch.zeros_like(s0)
    ssm_linear_attention_fwd(q, q, v, torch.zeros(3, device="cuda"), state=s0, state_out=so)
    assert torch.equal(so, s0)
    ssm_linear_attention_fwd(q, q, v, torch.zeros(3, device="cuda"), state_out=so)
    assert torch.equal(so, torch.zeros_like(so))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_then_tokens_equals_one_prompt(io):
    """A prompt of 140 tokens, then 20 single tokens through the same state in
    place, against a definition that sees 160 tokens."""
    import torch
    from state_space_model_causal_b200 import ssm_linear_attention_fwd, ssm_linear_attention_update
    args = problem(2, 4, 2, 160, 64, 64, io, "token", seed=6)
    q, k, v, g, s0 = args
    tq, tk, tv, tg, S = token_major(q, io), token_major(k, io), token_major(v, io), T(g, "f32"), T(s0, "f32")
    first = ssm_linear_attention_fwd(tq[:, :, :140], tk[:, :, :140], tv[:, :, :140], tg[:, :, :140], state=S)
    rest = [ssm_linear_attention_update(S, tq[:, :, t], tk[:, :, t], tv[:, :, t], tg[:, :, t]) for t in range(140, 160)]
    got = torch.cat([first, torch.stack(rest, dim=2)], dim=2)
    out, Sr = ref.linear_attention(q, k, v, g, 1.0, s0)
    bo, bs = bounds(q, k, v, g, s0, 1.0, None, io, out, io != "f32")
    assert (np.abs(to_np(got) - out) <= bo).all()
    assert (np.abs(to_np(S) - Sr) <= bs).all()


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("L,lens", [(3000, None), (1600, [1600, 0, 130, 900]), (2048, [2048, 2047, 128, 1])])
def test_long_sequences_in_pieces_or_whole(io, L, lens):
    """Few long sequences are cut into pieces where a workspace is given (ends
    of sequences before, in and between pieces); with and without it the
    results agree with the definition, the state updated in place too."""
    import torch
    from state_space_model_causal_b200 import ssm_linear_attention_fwd
    B = 1 if lens is None else len(lens)
    args = problem(B, 2, 1, L, 64, 64, io, "token", seed=8)
    for ws in ("auto", None):
        out, S, kern = run(*args, lens=lens, io=io, workspace=ws)
        assert kern == "linattn_chunk"
        check(args, 1.0, lens, io, out, S, kern)
    q, k, v, g, s0 = args
    st = T(s0, "f32")
    li = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    ssm_linear_attention_fwd(token_major(q, io), token_major(k, io), token_major(v, io), T(g, "f32"), state=st, seq_lens=li)
    out, S, _ = run(*args, lens=lens, io=io)
    np.testing.assert_array_equal(to_np(st), S)


# -------------------------------------------------------------- one token --
def step_bounds(state, q, k, v, g, scale, slots, io, st, out, new):
    mo, mn = ref.linear_attention_step(np.abs(state), np.abs(q), np.abs(k), np.abs(v), g, abs(scale), slots)
    f32 = (q.shape[-1] + 8) * 2.0 ** -24
    return (UNIT[io] * np.abs(out) + f32 * mo + TINY[io],
            (UNIT[st] if st != "f32" else 0.0) * np.abs(new) + 8 * 2.0 ** -24 * mn + TINY[st])


@pytest.mark.parametrize("st", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,H,Hk,N,P,slots", [(1, 1, 1, 128, 128, None), (5, 4, 2, 64, 64, 9), (3, 2, 2, 256, 33, 3),
                                              (2, 3, 1, 8, 5, None), (4, 2, 1, 100, 70, 6), (2, 2, 2, 17, 3, 4),
                                              (2, 1, 1, 136, 200, None)])
def test_step_matches_definition(io, st, B, H, Hk, N, P, slots):
    import torch
    from state_space_model_causal_b200 import ssm_linear_attention_update
    n_slots = B if slots is None else slots
    state = gen.round_to(gen.normal((n_slots, H, P, N), "la", "step", B, H, N, P), st)
    q, k, v = (draw(s, io, "step", x, B, H, N, P) for s, x in
               (((B, Hk, N), "q"), ((B, Hk, N), "k"), ((B, H, P), "v")))
    g = gen.round_to(-np.exp(gen.uniform((B, H), -6.0, 0.5, "la", "g", B, H)), "f32")
    idx = None
    if slots is not None:
        idx = np.random.RandomState(1).permutation(n_slots)[:B].astype(np.int32)
        idx[0] = -1 if B % 2 else n_slots  # a padding row
    out, new = ref.linear_attention_step(state, q, k, v, g, 0.5, idx)
    bo, bn = step_bounds(state, q, k, v, g, 0.5, idx, io, st, np.nan_to_num(out), np.nan_to_num(new))
    ti = None if idx is None else torch.tensor(idx, device="cuda")
    for in_place in (True, False):
        S = T(state, st)
        so = None if in_place else torch.full_like(S, 7.0)
        o = torch.full((B, H, P), 3.0, device="cuda", dtype=gen.torch_dtype(io))
        ssm_linear_attention_update(S, T(q, io), T(k, io), T(v, io), T(g, "f32"), scale=0.5, state_batch_indices=ti,
                                    state_out=so, out=o)
        got, after = to_np(o), to_np(S if in_place else so)
        expect = state.copy() if in_place else np.full(state.shape, 7.0)
        bound = np.zeros(state.shape)
        for b in range(B):
            s = b if idx is None else idx[b]
            if 0 <= s < n_slots:
                expect[s], bound[s] = new[b], bn[b]
                assert (np.abs(got[b] - out[b]) <= bo[b]).all()
            else:
                np.testing.assert_array_equal(got[b], 3.0)
        assert (np.abs(after - expect) <= bound).all()
        if not in_place:
            np.testing.assert_array_equal(to_np(S), state)


def test_step_of_a_strided_cache_and_a_decay_that_forgets():
    import torch
    from state_space_model_causal_b200 import LaunchInfo, binding, ssm_linear_attention_update
    big = torch.randn(3, 2, 40, 100, device="cuda")
    before = to_np(big)
    S = big[:, :, 3:35, 1:65]  # rows that start 4 bytes off a vector
    q, k, v = (T(draw(s, "f32", "strided", x), "f32") for s, x in (((3, 2, 64), "q"), ((3, 2, 64), "k"), ((3, 2, 32), "v")))
    g = torch.tensor([0.0, -torch.inf], device="cuda")
    info = LaunchInfo()
    o = ssm_linear_attention_update(S, q, k, v, g, info=info)
    assert binding.KERNELS[info.kernel] == "linattn_step_generic"
    st = before[:, :, 3:35, 1:65]
    out, new = ref.linear_attention_step(st, to_np(q), to_np(k), to_np(v), np.array([0.0, -np.inf]))
    bo, bn = step_bounds(st, to_np(q), to_np(k), to_np(v), np.array([0.0, -np.inf]), 1.0, None, "f32", "f32", out, new)
    assert (np.abs(to_np(o) - out) <= bo).all() and (np.abs(to_np(S) - new) <= bn).all()
    after = to_np(big)
    after[:, :, 3:35, 1:65] = before[:, :, 3:35, 1:65]
    np.testing.assert_array_equal(after, before)  # nothing around the view was written
