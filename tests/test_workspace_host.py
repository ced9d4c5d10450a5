"""Host-side check of a workspace that a caller gives the binding."""
import pytest

from state_space_model_causal_b200 import binding as bd


def test_a_workspace_that_is_not_contiguous_is_refused():
    """An expanded tensor counts a million elements over one byte of memory."""
    torch = pytest.importorskip("torch")
    whole = torch.empty(1 << 12, dtype=torch.uint8)
    assert bd._given_workspace(whole) == (whole.data_ptr(), 1 << 12)
    assert bd._given_workspace(torch.empty(64))[1] == 256
    for bad in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), whole[::2], torch.empty(8, 8).t()):
        with pytest.raises(ValueError, match="contiguous"):
            bd._given_workspace(bad)


@pytest.mark.gpu
def test_calls_refuse_such_a_workspace():
    import torch
    ws = torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 26)
    q = torch.zeros(1, 2, 4096, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="contiguous"):
        bd.ssm_linear_attention_fwd(q, q, q, torch.zeros(2, device="cuda"), workspace=ws)
    cache = torch.zeros(8, 16, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="contiguous"):
        bd.ssm_paged_attention_decode(q[:, :, 0].contiguous(), cache, cache,
                                      torch.zeros(1, 4, device="cuda", dtype=torch.int32),
                                      torch.ones(1, device="cuda", dtype=torch.int32), workspace=ws)
    x = torch.zeros(1, 64, 32, device="cuda")
    bc = torch.zeros(1, 16, 32, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        bd.ssm_selective_scan_fwd(x, x, -torch.ones(64, 16, device="cuda"), bc, bc, workspace=ws)
