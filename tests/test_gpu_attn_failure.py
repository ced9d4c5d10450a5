"""Failure detection of the linear attention kernels, without a GPU fault.

Two of them wait for copies into shared memory.  As in the state update, a wait
gives up after a cycle budget, records itself in the library's device error
record, and the kernel returns.  The failure-test build of the library starts no
copies for one work item (a flag that nothing sets) and shortens the budget to
about 10 ms: the call must return without a CUDA error, the record must name
the kernel and the item, everything that other CTAs computed must be complete,
and the next call must match the oracle.  The product library ignores the
switches."""
import numpy as np
import pytest

from oracle import attention as ref
from tests.test_gpu_failure import _env

pytestmark = pytest.mark.gpu
SWITCHES = {"SSM_TEST_DROP_ITEM": "5", "SSM_TEST_WAIT_CYCLES": "20000000"}


def _prompt(L):
    import torch
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(2, 4, L, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    return q, k, v, -torch.rand(4, generator=g).cuda()


def _run_prompt(a, info=None):
    import torch
    from state_space_model_causal_b200 import ssm_linear_attention_fwd
    q, k, v, decay = a
    state = torch.zeros(2, 4, 64, 64, device="cuda")
    out = ssm_linear_attention_fwd(q, k, v, decay, state=state, scale=0.125, info=info)
    torch.cuda.synchronize()  # no CUDA error: the kernel returned
    return out, state


def _step(B):
    import torch
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(B, 8, 128, generator=g).cuda() for _ in range(3))
    return torch.randn(B, 8, 128, 128, generator=g).cuda(), q, k, v, -torch.rand(8, generator=g).cuda()


def _run_step(a, info=None):
    import torch
    from state_space_model_causal_b200 import ssm_linear_attention_update
    state = a[0].clone()
    out = ssm_linear_attention_update(state, *a[1:], scale=0.125, info=info)
    torch.cuda.synchronize()
    return out, state


# L = 160: one launch; 2048: sequences in pieces, two launches, both without their item 5
@pytest.mark.parametrize("run,args,kernel", [(_run_prompt, lambda: _prompt(160), "linattn_chunk"),
                                             (_run_prompt, lambda: _prompt(2048), "linattn_chunk"),
                                             (_run_step, lambda: _step(4), "linattn_step_bulk"),
                                             (_run_step, lambda: _step(512), "linattn_step_bulk")])
def test_a_wait_that_runs_out_is_reported(run, args, kernel):
    from state_space_model_causal_b200 import LaunchInfo, binding, ssm_device_error, ssm_device_error_info
    a = args()
    info = LaunchInfo()
    want, want_state = run(a, info)  # product library, checked against the oracle elsewhere
    assert info.as_dict()["kernel"] == kernel and info.work_items > 5
    with binding.using_library(binding.TESTHOOKS_LIB_PATH):
        assert ssm_device_error() == 0
        with _env(**SWITCHES):
            got, got_state = run(a)
        rep = ssm_device_error_info()
        assert rep == {"code": 1, "kernel": kernel, "first_item": 5}, rep
        assert ssm_device_error() == 0  # read and cleared
        heads = got_state.shape[0] * got_state.shape[1]
        same = [(got_state.flatten(0, 1)[i] == want_state.flatten(0, 1)[i]).all().item() for i in range(heads)]
        if run is _run_prompt:  # item 5 is head 5 of one launch, and one piece of another
            pieces = info.work_items // heads
            lost = 5 if pieces == 1 else 5 // (pieces - 1)
            assert all(x for i, x in enumerate(same) if i != lost)
            if pieces == 1:
                assert not same[lost] and not got_state.flatten(0, 1)[lost].any()  # as it was
        else:
            assert not all(same) and same[0]
        got, got_state = run(a)  # the switches gone: complete again
        assert (got == want).all() and (got_state == want_state).all()
        assert ssm_device_error() == 0


@pytest.mark.parametrize("run,args", [(_run_prompt, lambda: _prompt(160)), (_run_step, lambda: _step(4))])
def test_the_product_library_ignores_the_switches(run, args):
    from state_space_model_causal_b200 import ssm_device_error
    a = args()
    want = run(a)
    with _env(**SWITCHES):
        got = run(a)
    assert ssm_device_error() == 0
    for x, y in zip(want, got):
        assert (x == y).all()


def test_the_runs_compared_with_are_right():
    a = _step(4)
    out, state = _run_step(a)
    n = [x.double().cpu().numpy() for x in a]
    o, s = ref.linear_attention_step(*n, scale=0.125)
    # a few roundings of 2^-24 of |v k|, |S| < 32; 128 products of |S q| < 8 or so in the sum
    np.testing.assert_allclose(state.cpu().numpy(), s, rtol=0, atol=1e-5)
    np.testing.assert_allclose(out.cpu().numpy(), o, rtol=0, atol=1e-4)
