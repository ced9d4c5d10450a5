"""What the binding takes as the size of a workspace that a caller gives it."""
import pytest

from state_space_model_causal_b200 import binding as bd


def test_a_workspace_counts_for_the_memory_it_has():
    """An expanded tensor counts a million elements over one byte."""
    torch = pytest.importorskip("torch")
    whole = torch.empty(1 << 12, dtype=torch.uint8)
    for ws, nbytes in ((whole, 1 << 12), (torch.empty(64), 256), (whole[:0], 0), (whole[::2], 1 << 11),
                       (torch.empty(8, 8).t(), 256), (whole[:1].expand(1 << 20), 1),
                       (torch.empty(1, 64).expand(1000, 64), 256)):
        assert bd._given_workspace(ws) == (ws.data_ptr(), nbytes)


@pytest.mark.gpu
def test_calls_refuse_a_workspace_of_one_byte():
    import torch
    ws = torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 26)
    q = torch.zeros(1, 2, 4096, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(bd.SsmError):
        bd.ssm_linear_attention_fwd(q, q, q, torch.zeros(2, device="cuda"), workspace=ws)
    cache = torch.zeros(8, 16, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(bd.SsmError):
        bd.ssm_paged_attention_decode(q[:, :, 0].contiguous(), cache, cache,
                                      torch.zeros(1, 4, device="cuda", dtype=torch.int32),
                                      torch.ones(1, device="cuda", dtype=torch.int32), workspace=ws)
