"""Linear attention where the numbers are far apart: decays, scores, states and
values whose sizes differ by tens of powers of two, and what is not finite.

Tolerances: those of test_gpu_linattn, and for float16 prompts what a common
power of two leaves of the small numbers beside a large one.  A number held in
float16 under a scale that brings the largest to 2^13 or more is off by at most half a
subnormal step, 2^-25, that is 2^-38 of the largest:

* a score: 2^-38 of the largest |q_t . k_s| of its row, times |v_s|;
* the copy of the state that queries read: 2^-38 of the largest |S| of its
  64 values, times |q|, times the scale.
"""
import numpy as np
import pytest

from oracle import attention as ref
from state_space_model_causal_b200 import inputs as gen
from tests.test_gpu_linattn import bounds, problem, run

pytestmark = pytest.mark.gpu


def common_scale(q, k, v, s0, scale):
    """The float16 terms above, for every output (B, H, L, P)."""
    rep = v.shape[1] // q.shape[1]
    q, k, v = np.repeat(np.abs(q), rep, 1), np.repeat(np.abs(k), rep, 1), np.abs(v)
    row = np.maximum.accumulate(np.einsum("bhtn,bhsn->bhts", q, k), -1)
    top = np.einsum("bhtt->bht", row)  # over s <= t
    S = np.einsum("bhsp,bhsn->bhpn", v, k) + (0.0 if s0 is None else np.abs(s0))
    most = S.max((2, 3))
    return abs(scale) * 2.0 ** -38 * (top[..., None] * v.cumsum(2) + most[:, :, None, None] * q.sum(-1)[..., None])


def check(args, got, scale, io, kernel, skip_out=None, skip_state=None, lens=None):
    """Against the definition; skip: a mask of elements that are not compared here."""
    q, k, v, g, s0 = args
    out, S = ref.linear_attention(q, k, v, g, scale, s0, lens)
    chunk = kernel == "linattn_chunk"
    bo, bs = bounds(q, k, v, g, s0, scale, lens, io, out, chunk)
    if chunk and io == "f16":
        bo = bo + common_scale(q, k, v, s0, scale)
    for what, a, b, bound, skip in (("out", got[0], out, bo, skip_out), ("state", got[1], S, bs, skip_state)):
        on = np.ones(a.shape, bool) if skip is None else ~skip
        assert np.isfinite(a[on]).all(), f"{what}: {(~np.isfinite(a[on])).sum()} not finite"
        err = np.abs(a - b)[on] / (bound[on] + 1e-300)
        assert err.max() <= 1.0, f"{what}: {(err > 1).sum()} of {err.size} off, worst {err.max():.3g} bounds"


# Over 32 tokens these decay by 2^45 to 2^103: on both sides of the border to the form with
# an exponential per element.
DECAYS = [-1.0, -1.35, -1.6, -2.0, -2.2, -2.3, "one"]


def decaying(log_decay, shape):
    g = np.full(shape, log_decay if log_decay != "one" else -0.01)
    if log_decay == "one":  # one token of a block forgets nearly everything, another a good deal
        g[..., 17], g[..., 40] = -65.0, -45.0
    return gen.round_to(g, "f32")


@pytest.mark.parametrize("log_decay", DECAYS)
@pytest.mark.parametrize("small", [0, 7, 10, 14])
def test_float16_scores_below_one_under_strong_decay(log_decay, small):
    """q and k of 2^-small: scores of about 2^(3 - 2 small), put right by the scale."""
    q, k, v, _, s0 = problem(1, 2, 2, 160, 64, 64, "f16", "token", seed=71)
    q, k = gen.round_to(q * 2.0 ** -small, "f16"), gen.round_to(k * 8 * 2.0 ** -small, "f16")
    g, scale = decaying(log_decay, (1, 2, 160)), 2.0 ** (2 * small - 3)
    s0 = s0 * 2.0 ** -small
    out, S, kern = run(q, k, v, g, s0, scale=scale, io="f16")
    assert kern == "linattn_chunk"
    check((q, k, v, g, s0), (out, S), scale, "f16", kern)


@pytest.mark.parametrize("log_decay", DECAYS)
@pytest.mark.parametrize("small", [16, 30])
def test_bfloat16_scores_far_below_one_under_strong_decay(log_decay, small):
    """As above in bfloat16, whose scores can be as small as float32's."""
    q, k, v, _, s0 = problem(1, 2, 2, 160, 64, 64, "bf16", "token", seed=72)
    q, k = q * 2.0 ** -small, k * 8 * 2.0 ** -small
    g, scale = decaying(log_decay, (1, 2, 160)), 2.0 ** (2 * small - 3)
    s0 = s0 * 2.0 ** -small
    out, S, kern = run(q, k, v, g, s0, scale=scale, io="bf16")
    assert kern == "linattn_chunk"
    check((q, k, v, g, s0), (out, S), scale, "bf16", kern)


@pytest.mark.parametrize("size", [20, -20])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("L", [40, 300])
def test_initial_state_with_one_number_that_is_not_finite(L, bad, size):
    """float16: the other value channels keep their common scale, for states above float16's
    largest number and for states among its subnormals."""
    q, k, v, g, s0 = problem(1, 2, 1, L, 64, 64, "f16", "token", seed=73)
    s0, scale = s0 * 2.0 ** size, 2.0 ** -size
    v = gen.round_to(v * 2.0 ** min(size, 0), "f16")
    clean, bad_s0 = s0.copy(), s0.copy()
    bad_s0[0, 0, 5, 3], clean[0, 0, 5, 3] = bad, 0.0
    skip_out, skip_state = np.zeros(v.shape, bool), np.zeros(s0.shape, bool)
    skip_out[0, 0, :, 5] = skip_state[0, 0, 5, 3] = True
    out, S, kern = run(q, k, v, g, bad_s0, scale=scale, io="f16")
    assert kern == "linattn_chunk"
    assert not np.isfinite(out[skip_out]).any() and not np.isfinite(S[skip_state]).any()
    check((q, k, v, g, clean), (out, S), scale, "f16", kern, skip_out, skip_state)


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("L", [5, 200])
def test_value_channels_far_apart_in_size(io, L):
    """Channels of 2^-16 to 2^12 beside one another: the state of each to the accuracy of its
    own size (2^-22, and 2^-49 of the largest value in float16, see the header)."""
    q, k, v, g, _ = problem(1, 2, 2, L, 64, 64, io, "token", seed=74, state=False)
    v = gen.round_to(np.clip(v, -4, 4) * 2.0 ** (4.0 * (np.arange(64) % 8) - 16), io)
    out, S, kern = run(q, k, v, g, None, io=io)
    assert kern == "linattn_chunk"
    _, ref_S = ref.linear_attention(q, k, v, g)
    _, own = bounds(q, k, v, g, None, 1.0, None, io, np.zeros_like(v), True)
    largest = np.abs(v).max((2, 3))[:, :, None, None] * np.abs(k).sum(2)[:, :, None, :]
    err = np.abs(S - ref_S) / (own + 2.0 ** -49 * largest)
    assert err.max() <= 1.0, f"worst {err.max():.3g} bounds, by channel size {err.max((0, 1, 3))[:8].round(2)}"
    want, _ = ref.linear_attention(q, k, v, g)
    bound, _ = bounds(q, k, v, g, None, 1.0, None, io, want, True)
    assert (np.abs(out - want) <= bound + (common_scale(q, k, v, None, 1.0) if io == "f16" else 0.0)).all()


@pytest.mark.parametrize("io,L", [("f32", 300), ("bf16", 300), ("f16", 300), ("bf16", 2500), ("f16", 2500)])
def test_a_decay_that_is_nan_reaches_no_earlier_token(io, L):
    """Outputs before its token are what they are without it; those from it on, and the
    state, are NaN.  The other head sees nothing.  L = 2500: a sequence in pieces."""
    q, k, v, g, s0 = problem(1, 2, 1, L, 64, 64, io, "token", seed=75)
    at = L - 255  # in the middle of 32 tokens
    bad = g.copy()
    bad[0, 1, at] = np.nan
    skip_out, skip_state = np.zeros(v.shape, bool), np.zeros(s0.shape, bool)
    skip_out[0, 1, at:] = skip_state[0, 1] = True
    out, S, kern = run(q, k, v, bad, s0, io=io)
    assert np.isnan(out[skip_out]).all() and np.isnan(S[skip_state]).all()
    check((q, k, v, g, s0), (out, S), 1.0, io, kern, skip_out, skip_state)


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_a_positive_log_decay_counts_as_zero(io, decay):
    """In a prompt, on both kernels."""
    q, k, v, g, s0 = problem(2, 4, 2, 150, 64, 64, io, decay, seed=76)
    up = g.copy()
    up.reshape(-1)[::3] = np.resize([1e-3, 0.7, 90.0, np.inf], up.reshape(-1)[::3].shape)
    out, S, kern = run(q, k, v, up, s0, io=io)
    check((q, k, v, np.minimum(up, 0.0), s0), (out, S), 1.0, io, kern)
