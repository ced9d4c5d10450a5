"""Attention of one token over a paged cache where the values are not finite.
Tolerances of what is: those of test_gpu_paged."""
import numpy as np
import pytest

from oracle import attention as ref
from state_space_model_causal_b200 import inputs as gen
from tests.test_gpu_paged import TINY, UNIT, cache, run, table_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("io,Hq,D", [("bf16", 1, 64), ("bf16", 4, 128), ("bf16", 8, 64), ("bf16", 12, 128),
                                     ("f16", 5, 64), ("f16", 16, 64), ("f32", 4, 64)])
def test_a_value_that_is_not_finite_stays_in_its_column(io, Hq, D, bad):
    """An infinity in the values of tokens that count gives an infinity there, a NaN a NaN, in
    groups of every size; the other columns are what they are without it."""
    lens, page = [200, 900], 16
    M = -(-max(lens) // page)
    k, v = cache(2 * M, page, 1, D, io, "bad", Hq, D)
    q = gen.round_to(0.5 * gen.normal((2, Hq, D), "paged", "badq", Hq, D), io)  # no weight near 0
    table = table_for(2, M, 2 * M)
    dirty, clean = v.copy(), v.copy()
    for b, t, d in ((0, 77, 3), (0, 130, 3), (1, 600, D - 1)):
        at = table[b, t // page], t % page, 0, d
        dirty[at], clean[at] = bad, 0.0
    out, ps, lse, mag, spread = ref.paged_attention(q, k, clean, table, lens, D ** -0.5)
    got, _, _, kern = run(q, k, dirty, table, lens, D ** -0.5, io)
    assert kern == ("paged_decode" if io != "f32" else "paged_decode_generic")
    reach = np.zeros(out.shape, bool)
    reach[0, :, 3] = reach[1, :, D - 1] = True
    np.testing.assert_array_equal(got[reach], bad)
    n = np.array([p.shape[1] for p in ps])
    w = 2 * (D + 4) * 2.0 ** -24 * spread + (n[:, None] / 16 + 64) * 2.0 ** -22
    c = 0.0 if io == "f32" else (2.0 ** -16 if Hq <= 8 else UNIT[io])
    bound = UNIT[io] * np.abs(out) + (w + c)[..., None] * mag + TINY[io]
    assert (np.abs(got - out) <= bound)[~reach].all()
