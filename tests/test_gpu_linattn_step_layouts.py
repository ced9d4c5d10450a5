"""One token of linear attention on every layout of the state cache: rows without
gaps, rows with gaps between them, and rows that start off a vector.

Tolerances: those of test_gpu_linattn."""
import numpy as np
import pytest

from oracle import attention as ref
from state_space_model_causal_b200 import inputs as gen
from tests.parity import N as to_np
from tests.parity import T
from tests.test_gpu_linattn import draw, step_bounds

pytestmark = pytest.mark.gpu

KERNEL = {"dense": "linattn_step_bulk", "gaps": "linattn_step", "shifted": "linattn_step_generic"}


def pool(values, st, layout):
    """The whole buffer (filled with 5), and the view of it that holds the values."""
    import torch
    S, H, P, N = values.shape
    pad, at = {"dense": (0, 0), "gaps": (8, 8), "shifted": (8, 1)}[layout]
    whole = torch.full((S, H, P + 3 if pad else P, N + 2 * pad), 5.0, device="cuda", dtype=gen.torch_dtype(st))
    view = whole[:, :, :P, at:at + N]
    view.copy_(T(values, st))
    return whole, view


@pytest.mark.parametrize("layout", ["dense", "gaps", "shifted"])
@pytest.mark.parametrize("st", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,N,P,slots", [(1, 2, 2, 64, 64, 1), (3, 4, 2, 128, 37, 7), (2, 2, 1, 256, 130, 5),
                                              (4, 3, 3, 8, 300, 4), (2, 3, 1, 200, 1, 3)])
def test_step_layouts(layout, st, io, B, H, Hk, N, P, slots):
    import torch
    from state_space_model_causal_b200 import LaunchInfo, binding, ssm_linear_attention_update
    state = gen.round_to(gen.normal((slots, H, P, N), "layout", B, H, N, P), st)
    q, k, v = (draw(s, io, "layout", x, B, H, N, P) for s, x in (((B, Hk, N), "q"), ((B, Hk, N), "k"), ((B, H, P), "v")))
    g = gen.round_to(-np.exp(gen.uniform((B, H), -6.0, 0.5, "layout", "g", B, H)), "f32")
    idx = np.random.RandomState(B + N).permutation(slots)[:B].astype(np.int32)
    if B > 2:
        idx[1] = -1  # a padding row
    out, new = ref.linear_attention_step(state, q, k, v, g, 0.5, idx)
    bo, bn = step_bounds(state, q, k, v, g, 0.5, idx, io, st, np.nan_to_num(out), np.nan_to_num(new))
    for in_place in (True, False):
        whole, S = pool(state, st, layout)
        whole_out, so = (whole, None) if in_place else pool(np.full(state.shape, 7.0), st, layout)
        before = to_np(whole_out)
        o = torch.full((B, H, P), 3.0, device="cuda", dtype=gen.torch_dtype(io))
        info = LaunchInfo()
        ssm_linear_attention_update(S, T(q, io), T(k, io), T(v, io), T(g, "f32"), scale=0.5,
                                    state_batch_indices=torch.tensor(idx, device="cuda"), state_out=so, out=o, info=info)
        if P > 1:  # (a single row has no gaps)
            assert binding.KERNELS[info.kernel] == KERNEL[layout]
        got, after = to_np(o), to_np(S if in_place else so)
        expect, bound = (state if in_place else np.full(state.shape, 7.0)).copy(), np.zeros(state.shape)
        for b, s in enumerate(idx):
            if 0 <= s < slots:
                expect[s], bound[s] = new[b], bn[b]
                assert (np.abs(got[b] - out[b]) <= bo[b]).all()
            else:
                np.testing.assert_array_equal(got[b], 3.0)
        assert (np.abs(after - expect) <= bound).all()
        # nothing around the view is written, and a state that is only read stays
        (S if in_place else so).copy_(T(np.zeros(state.shape), st))
        view = to_np(S if in_place else so) == 0
        assert view.all()
        around = to_np(whole_out)
        pad, at = {"dense": (0, 0), "gaps": (8, 8), "shifted": (8, 1)}[layout]
        before[:, :, :P, at:at + N] = 0.0
        np.testing.assert_array_equal(around, before)
        if not in_place:
            np.testing.assert_array_equal(to_np(S), state)


@pytest.mark.parametrize("layout", ["dense", "gaps", "shifted"])
@pytest.mark.parametrize("per_head", [True, False])
def test_a_positive_log_decay_counts_as_zero(layout, per_head):
    from state_space_model_causal_b200 import ssm_linear_attention_update
    state = gen.round_to(gen.normal((2, 4, 24, 64), "up", "s"), "f32")
    q, k, v = (draw(s, "f32", "up", x) for s, x in (((2, 2, 64), "q"), ((2, 2, 64), "k"), ((2, 4, 24), "v")))
    g = np.array([0.5, -0.25, np.inf, 88.0])
    g = g if per_head else np.stack([g, -g[::-1]])
    _, S = pool(state, "f32", layout)
    o = ssm_linear_attention_update(S, T(q, "f32"), T(k, "f32"), T(v, "f32"), T(g, "f32"))
    g = np.minimum(g, 0.0)
    out, new = ref.linear_attention_step(state, q, k, v, g)
    bo, bn = step_bounds(state, q, k, v, g, 1.0, None, "f32", "f32", out, new)
    assert (np.abs(to_np(o) - out) <= bo).all() and (np.abs(to_np(S) - new) <= bn).all()
