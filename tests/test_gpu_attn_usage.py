"""The token mixers of hybrid models as a program uses them: on other streams,
two calls at once, captured into graphs that are replayed together, over pools
whose offsets pass 32 bits, over very many sequences or heads, and the same
call twice (the same bits)."""
import numpy as np
import pytest

from oracle import attention as ref
from state_space_model_causal_b200 import inputs as gen
from tests.parity import N as to_np
from tests.parity import T
from tests.test_gpu_linattn import problem, token_major
from tests.test_gpu_linattn import check as check_prompt
from tests.test_gpu_paged import check as check_paged

pytestmark = pytest.mark.gpu


def prompt_inputs(L=1600, io="bf16", seed=21):
    args = problem(1, 2, 2, L, 64, 64, io, "token", seed=seed)
    q, k, v, g, s0 = args
    return args, (token_major(q, io), token_major(k, io), token_major(v, io), T(g, "f32"), T(s0, "f32"))


def paged_inputs(seed, B=3, M=40, page=16, Hq=8, Hkv=2, D=64):
    import torch
    rs = np.random.RandomState(seed)
    k, v = (gen.round_to(gen.normal((B * M, page, Hkv, D), "usage", x, seed), "bf16") for x in "kv")
    q = gen.round_to(gen.normal((B, Hq, D), "usage", "q", seed), "bf16")
    table = rs.permutation(B * M).reshape(B, M).astype(np.int32)
    lens = rs.randint(1, M * page + 1, B).astype(np.int32)
    want = ref.paged_attention(q, k, v, table, lens, 0.125)[0]
    dev = (T(q, "bf16"), T(k, "bf16"), T(v, "bf16"), torch.tensor(table, device="cuda"), torch.tensor(lens, device="cuda"))
    return dev, want


def near(got, want):
    assert np.abs(to_np(got) - want).max() <= 2.0 ** -7 * np.abs(want).max()


@pytest.mark.parametrize("how", ["argument", "context"])
def test_on_another_stream(how):
    """Inputs are made on a side stream right before the calls, which run there
    without anyone waiting; the default stream is kept busy meanwhile."""
    import torch
    from state_space_model_causal_b200 import (ssm_kv_cache_evict, ssm_linear_attention_fwd,
                                               ssm_linear_attention_update, ssm_paged_attention_decode)
    args, (q, k, v, g, s0) = prompt_inputs()
    (pq, pk, pv, table, lens), want = paged_inputs(1)
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    kw = dict(stream=side) if how == "argument" else {}
    with torch.cuda.stream(side):
        q2, k2, v2, S = q * 1, k * 1, v * 1, s0 * 1
        out, o2, pout = torch.full_like(v2, 3.0), torch.empty_like(v2[:, :, 0]), torch.empty_like(pq)
        so = torch.empty_like(S)
        w = torch.rand(3, 2, 640, device="cuda")
    if how == "argument":
        ssm_linear_attention_fwd(q2, k2, v2, g, state=S, state_out=so, out=out, **kw)
        ssm_linear_attention_update(so, q2[:, :, 0], k2[:, :, 0], v2[:, :, 0], g[:, :, 0], out=o2, **kw)
        ssm_paged_attention_decode(pq, pk, pv, table, lens, scale=0.125, out=pout, **kw)
        n, kept, nw = ssm_kv_cache_evict(pk, pv, w, table, lens, table[:, :2].contiguous(), 32, **kw)
    else:
        with torch.cuda.stream(side):
            ssm_linear_attention_fwd(q2, k2, v2, g, state=S, state_out=so, out=out)
            ssm_linear_attention_update(so, q2[:, :, 0], k2[:, :, 0], v2[:, :, 0], g[:, :, 0], out=o2)
            ssm_paged_attention_decode(pq, pk, pv, table, lens, scale=0.125, out=pout)
            n, kept, nw = ssm_kv_cache_evict(pk, pv, w, table, lens, table[:, :2].contiguous(), 32)
    side.synchronize()
    _, S_ref = ref.linear_attention(*args[:4], 1.0, args[4])
    near(pout, want)
    assert n.tolist() == [min(32, x) for x in lens.tolist()]
    out_ref, S1 = ref.linear_attention_step(S_ref, *(a[:, :, 0] for a in args[:4]))
    assert np.abs(to_np(so) - S1).max() < 1e-3
    assert np.abs(to_np(o2) - out_ref).max() < 0.03 * np.abs(out_ref).max()
    ref_out, _ = ref.linear_attention(*args[:4], 1.0, args[4])
    assert np.abs(to_np(out) - ref_out).max() < 0.03 * np.abs(ref_out).max()


def test_outputs_are_allocated_on_the_stream_that_writes_them():
    """With a stream argument: memory that the current stream freed a moment ago may still
    be read there."""
    import torch
    from state_space_model_causal_b200 import (ssm_kv_cache_evict, ssm_linear_attention_fwd,
                                               ssm_linear_attention_update, ssm_paged_attention_decode)
    _, (q, k, v, g, s0) = prompt_inputs()
    (pq, pk, pv, table, lens), _ = paged_inputs(1)
    w = torch.rand(3, 2, 640, device="cuda")
    new = table.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [ssm_linear_attention_fwd(q, k, v, g, state=s0, stream=side),
            ssm_linear_attention_update(s0, q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous(),
                                        g[:, :, 0].contiguous(), stream=side),
            ssm_paged_attention_decode(pq, pk, pv, table, lens, stream=side),
            *ssm_kv_cache_evict(pk, pv, w, table, lens * 0, new, keep=5, recent=2, stream=side)]
    torch.cuda.synchronize()
    segments = torch.cuda.memory_snapshot()
    for o in outs:
        home = [x for x in segments if x["address"] <= o.data_ptr() < x["address"] + x["total_size"]]
        assert [x["stream"] for x in home] == [side.cuda_stream]


def test_two_calls_at_once():
    """Prompts and decode steps on two streams at the same time."""
    import torch
    from state_space_model_causal_b200 import ssm_linear_attention_fwd, ssm_paged_attention_decode
    sets = [prompt_inputs(seed=s) for s in (31, 32)]
    pages = [paged_inputs(s) for s in (5, 6)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, pouts = [], []
    torch.cuda.synchronize()
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                q, k, v, g, s0 = sets[i][1]
                so = torch.empty_like(s0)
                outs.append((i, ssm_linear_attention_fwd(q, k, v, g, state=s0, state_out=so), so))
                pouts.append((i, ssm_paged_attention_decode(*pages[i][0], scale=0.125)))
    torch.cuda.synchronize()
    for i, o, so in outs:
        full = np.full(sets[i][0][2].shape, np.nan)
        check_prompt(sets[i][0], 1.0, None, "bf16", to_np(o), to_np(so), "linattn_chunk")
        assert full.shape == to_np(o).shape
    for i, o in pouts:
        near(o, pages[i][1])


def test_graphs_replayed_together():
    """Two graphs captured on one stream, each with calls that need a workspace,
    replayed on two streams at the same time and again after their inputs changed: each
    has its own workspace."""
    import torch
    from state_space_model_causal_b200 import ssm_linear_attention_fwd, ssm_paged_attention_decode
    sets = [prompt_inputs(seed=s) for s in (41, 42)]
    pages = [paged_inputs(s) for s in (7, 8)]
    made = []
    cap = torch.cuda.Stream()
    for i in range(2):
        q, k, v, g, s0 = sets[i][1]
        so, out, pout = torch.empty_like(s0), torch.full_like(v, 3.0), torch.empty_like(pages[i][0][0])
        w = torch.zeros(3, 2, 640, device="cuda")
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=cap):
            ssm_linear_attention_fwd(q, k, v, g, state=s0, state_out=so, out=out)
            ssm_paged_attention_decode(*pages[i][0], scale=0.125, out=pout, weights=w)
        made.append((graph, so, out, pout, w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for round_ in range(4):
        for st, (graph, *_rest) in zip(streams, made):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for i, (graph, so, out, pout, w) in enumerate(made):
        check_prompt(sets[i][0], 1.0, None, "bf16", to_np(out), to_np(so), "linattn_chunk")
        near(pout, pages[i][1])
        heads = 8 // 2 * 4  # four replays of weights that sum to 1 per query head
        np.testing.assert_allclose(to_np(w).sum(-1), heads, rtol=1e-4)
    # other inputs at the same addresses
    (pq, pk, pv, table, lens), want = paged_inputs(9)
    for dst, src in zip(pages[0][0], (pq, pk, pv, table, lens)):
        dst.copy_(src)
    made[0][0].replay()
    torch.cuda.synchronize()
    near(made[0][3], want)


def test_the_same_prompt_twice_gives_the_same_bits():
    from tests.test_gpu_linattn import run
    for io in ("bf16", "f16", "f32"):
        args = problem(2, 3, 3, 700, 96, 72, io, "token", seed=51)
        a, b = run(*args, io=io), run(*args, io=io)
        np.testing.assert_array_equal(a[0], b[0])
        np.testing.assert_array_equal(a[1], b[1])


def test_pools_past_32_bits():
    """Cache pools and state pools of more than 2^32 bytes, used at their far end."""
    import torch
    from state_space_model_causal_b200 import (ssm_kv_cache_evict, ssm_linear_attention_update,
                                               ssm_paged_attention_decode)
    pages, page, Hkv, D = 1_300_000, 16, 2, 64  # 2.66e9 elements, 5.3 GB each
    kc, vc = (torch.empty((pages, page, Hkv, D), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    M = 6
    table = (pages - 1 - torch.randperm(4 * M, device="cuda")).to(torch.int32).view(2, 2 * M)
    k, v = (gen.round_to(gen.normal((2 * M, page, Hkv, D), "far", x), "bf16") for x in "kv")
    old = table[:, :M].contiguous()
    kc[old.flatten().long()], vc[old.flatten().long()] = T(k, "bf16"), T(v, "bf16")
    q = gen.round_to(gen.normal((2, 4, D), "far", "q"), "bf16")
    lens = torch.tensor([96, 50], dtype=torch.int32, device="cuda")
    local = np.arange(2 * M, dtype=np.int32).reshape(2, M)
    want = ref.paged_attention(q, k, v, local, [96, 50], 0.125)[0]
    near(ssm_paged_attention_decode(T(q, "bf16"), kc, vc, old, lens, scale=0.125), want)
    w = torch.rand(2, Hkv, M * page, device="cuda")
    n, kept, _ = ssm_kv_cache_evict(kc, vc, w, old, lens, table[:, M:].contiguous(), 40, recent=8)
    rows = ref.evict(to_np(w), local, [96, 50], 2 * M, page, 40, 8)
    for b in range(2):
        for h in range(Hkv):
            assert kept[b, h].tolist() == rows[b][h]
            new = kc[table[b, M:].long()].flatten(0, 1)[:40, h]
            np.testing.assert_array_equal(to_np(new), np.concatenate(k[local[b]])[rows[b][h], h])
    del kc, vc
    S = torch.empty((140_000, 1, 128, 128), device="cuda")  # 9.2 GB
    state = gen.round_to(gen.normal((2, 1, 128, 128), "far", "state"), "f32")
    slots = torch.tensor([139_999, 70_001], dtype=torch.int32, device="cuda")
    S[slots.long()] = T(state, "f32")
    qkv = [gen.round_to(gen.normal((2, 1, 128), "far", x, "s"), "f32") for x in "qkv"]
    g = np.array([-0.1])
    out = ssm_linear_attention_update(S, *(T(x, "f32") for x in qkv), T(g, "f32"), state_batch_indices=slots)
    want, new = ref.linear_attention_step(state, *qkv, gen.round_to(g, "f32"))
    assert np.abs(to_np(out) - want).max() < 1e-3 and np.abs(to_np(S[slots.long()]) - new).max() < 1e-4


def test_prompt_views_past_32_bits():
    """Two sequences of one prompt more than 2^32 bytes apart."""
    import torch
    from state_space_model_causal_b200 import ssm_linear_attention_fwd
    args = problem(2, 2, 2, 200, 64, 64, "bf16", "head", seed=61)
    buf = torch.empty(2_300_000_000 + 400_000, device="cuda", dtype=torch.bfloat16)
    views = []
    for i, a in enumerate(args[:3]):
        view = buf[i * 100_000:].as_strided((2, 2, 200, 64), (2_300_000_000, 64, 128, 1))
        view.copy_(T(a, "bf16"))
        views.append(view)
    so = torch.empty(2, 2, 64, 64, device="cuda")
    out = torch.full((2, 2, 200, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    ssm_linear_attention_fwd(*views, T(args[3], "f32"), state=T(args[4], "f32"), state_out=so, out=out)
    check_prompt(args, 1.0, None, "bf16", to_np(out), to_np(so), "linattn_chunk")


@pytest.mark.parametrize("B,Hq,Hkv", [(3000, 2, 1), (2, 600, 300)])
def test_very_many_sequences_or_heads(B, Hq, Hkv):
    rs = np.random.RandomState(3)
    page, M, D = 8, 3, 32
    lens = rs.randint(0, M * page + 1, B)
    k, v = (gen.round_to(gen.normal((64, page, Hkv, D), "many", x, B), "bf16") for x in "kv")
    q = gen.round_to(gen.normal((B, Hq, D), "many", "q", B), "bf16")
    check_paged(q, k, v, rs.randint(0, 64, (B, M)).astype(np.int32), lens.tolist(), 0.2, "bf16")


def test_a_long_eviction_without_cached_keys():
    """More tokens than keys fit in shared memory, few of them kept; nearly all weights equal."""
    import torch
    from state_space_model_causal_b200 import ssm_kv_cache_evict
    page, M, keep = 256, 300, 700  # 76800 tokens
    lens = torch.tensor([M * page - 3], dtype=torch.int32, device="cuda")
    k = torch.randn(M + 3, page, 1, 16, device="cuda", dtype=torch.float16)
    v = torch.randn_like(k)
    w = torch.zeros(1, 1, M * page, device="cuda")
    w[0, 0, 5000:5300] = 1.0
    w[0, 0, 70000] = 2.0
    table = torch.randperm(M + 3, device="cuda").to(torch.int32)[None]
    n, kept, nw = ssm_kv_cache_evict(k, v, w, table[:, :M].contiguous(), lens, table[:, M:].contiguous(), keep, recent=100)
    end = M * page - 3
    want = list(range(0, keep - 100 - 301)) + list(range(5000, 5300)) + [70000] + list(range(end - 100, end))
    assert n.tolist() == [keep] and kept[0, 0].tolist() == want
    got = k[table[0, M:].long()].flatten(0, 1)[:keep, 0]
    flat = k[table[0, :M].long()].flatten(0, 1)[:, 0]
    assert torch.equal(got, flat[torch.tensor(want, device="cuda")])
