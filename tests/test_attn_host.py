"""Host-side checks of the token mixers of hybrid models (no GPU, nothing is
launched): every invalid argument is refused with its documented status, and
the dry-run mode shows which kernel a valid call would take."""
import ctypes

import pytest

from state_space_model_causal_b200 import binding as bd

F32, F16, BF16, I32 = bd.SSM_F32, bd.SSM_F16, bd.SSM_BF16, bd.SSM_I32
OK, ENULL, ESHAPE, EDTYPE, ESTRIDE, EUNSUP, ECUDA, EINT, EVER, EALIAS, EWS = range(11)


class FakeMem:
    """Distinct, 256-byte-aligned fake device addresses far apart."""

    def __init__(self):
        self.next = 1 << 40

    def __call__(self, dtype, shape, stride=None, offset=0):
        ptr = self.next + offset
        self.next += 1 << 42
        return bd.raw_tensor(ptr, dtype, shape, stride)


@pytest.fixture
def mem():
    return FakeMem()


@pytest.fixture(scope="module")
def lib():
    return bd.library()


def args_of(cls, **fields):
    a = cls()
    a.struct_size = ctypes.sizeof(cls)
    a.flags = bd.SSM_FLAG_DRY_RUN
    info = bd.LaunchInfo()
    info.struct_size = ctypes.sizeof(bd.LaunchInfo)
    a.info = ctypes.pointer(info)
    for k, v in fields.items():
        setattr(a, k, v)
    return a


def call(fn, a):
    st = fn(ctypes.byref(a), None)
    return st, a.info.contents.as_dict() if st == OK else None


# --------------------------------------------------------- linear attention --
def token_major(mem, dt, B, H, L, X):
    """A (B, H, L, X) view of (B, L, H, X) storage."""
    return mem(dt, (B, H, L, X), (L * H * X, X, H * X, 1))


def prompt(mem, B=2, H=4, Hk=2, L=300, N=64, P=64, io=BF16, per_token=False, with_state=True, **over):
    f = dict(q=token_major(mem, io, B, Hk, L, N), k=token_major(mem, io, B, Hk, L, N),
             v=token_major(mem, io, B, H, L, P), out=token_major(mem, io, B, H, L, P),
             log_decay=mem(F32, (B, H, L) if per_token else (H,)), scale=1.0)
    if with_state:
        f.update(state=mem(F32, (B, H, P, N)), state_out=mem(F32, (B, H, P, N)))
    f.update(over)
    return args_of(bd.LinAttnArgs, **f)


def test_prompt_kernels(lib, mem):
    fn = lib.ssm_linear_attention_fwd
    assert call(fn, prompt(mem))[1]["kernel"] == "linattn_chunk"
    assert call(fn, prompt(mem, io=F16, N=128, P=192))[1]["kernel"] == "linattn_chunk"
    assert call(fn, prompt(mem, N=8, P=8, per_token=True, with_state=False))[1]["kernel"] == "linattn_chunk"
    assert call(fn, prompt(mem, io=F32))[1]["kernel"] == "linattn_generic"
    assert call(fn, prompt(mem, N=136))[1]["kernel"] == "linattn_generic"
    assert call(fn, prompt(mem, N=68))[1]["kernel"] == "linattn_generic"  # rows of 136 bytes
    assert call(fn, prompt(mem, P=12))[1]["kernel"] == "linattn_generic"
    shifted = mem(BF16, (2, 2, 300, 64), (300 * 128, 64, 128, 1), offset=2)
    assert call(fn, prompt(mem, q=shifted))[1]["kernel"] == "linattn_generic"
    broadcast = mem(BF16, (2, 2, 300, 64), (0, 64, 128, 1))
    assert call(fn, prompt(mem, k=broadcast))[1]["kernel"] == "linattn_generic"
    apart = mem(BF16, (2, 2, 300, 64), (300 * 256, 128, 256, 2))
    assert call(fn, prompt(mem, k=apart))[1]["kernel"] == "linattn_generic"
    assert call(fn, prompt(mem, L=0, with_state=False))[1]["kernel"] == "none"
    assert call(fn, prompt(mem, B=0))[1]["kernel"] == "none"
    assert call(fn, prompt(mem, L=0))[1]["kernel"] == "linattn_generic"  # copies the state


def test_prompt_workspace(lib, mem):
    """Few long sequences ask for a workspace; one that is too small or misaligned is
    refused, none at all is not."""
    need = ctypes.c_uint64(7)
    size = lib.ssm_linear_attention_workspace_size
    assert size(None, ctypes.byref(need)) == ENULL
    assert size(ctypes.byref(prompt(mem)), None) == ENULL
    assert size(ctypes.byref(prompt(mem, B=8, H=32, Hk=32, L=4096)), ctypes.byref(need)) == OK and need.value == 0
    a = prompt(mem, B=1, L=8192)
    assert size(ctypes.byref(a), ctypes.byref(need)) == OK and need.value > 0
    fn = lib.ssm_linear_attention_fwd
    whole = call(fn, a)[1]["grid"]
    a.workspace, a.workspace_bytes = 1 << 30, need.value
    assert call(fn, a)[1]["grid"] > whole
    a.workspace_bytes = need.value - 1
    assert call(fn, a)[0] == EWS
    a.workspace, a.workspace_bytes = (1 << 30) + 16, need.value + 512
    assert call(fn, a)[0] == EWS
    a.workspace, a.workspace_bytes = a.v.data, need.value
    assert call(fn, a)[0] == EALIAS


@pytest.mark.parametrize("over,status", [
    (dict(struct_size=3), EVER), (dict(q=bd.Tensor()), ENULL), (dict(k=bd.Tensor()), ENULL),
    (dict(out=bd.Tensor()), ENULL), (dict(log_decay=bd.Tensor()), ENULL)])
def test_prompt_missing_arguments(lib, mem, over, status):
    assert call(lib.ssm_linear_attention_fwd, prompt(mem, **over))[0] == status
    assert lib.ssm_linear_attention_fwd(None, None) == ENULL


def test_prompt_refusals(lib, mem):
    fn = lib.ssm_linear_attention_fwd

    def st(**over):
        return call(fn, prompt(mem, **over))[0]

    B, H, Hk, L, N, P = 2, 4, 2, 300, 64, 64
    assert st(k=mem(BF16, (B, Hk, L, N + 1))) == ESHAPE
    assert st(k=mem(BF16, (B, H, L, N))) == ESHAPE
    assert st(v=mem(BF16, (B, H, L - 1, P))) == ESHAPE
    assert st(out=mem(BF16, (B, H, L, P + 1))) == ESHAPE
    assert st(Hk=3) == ESHAPE  # 4 heads over 3
    assert st(log_decay=mem(F32, (H + 1,))) == ESHAPE
    assert st(log_decay=mem(F32, (B, H))) == ESHAPE
    assert st(log_decay=mem(F32, (B, H, L + 1))) == ESHAPE
    assert st(state=mem(F32, (B, H, N, P + 1))) == ESHAPE
    assert st(state_out=mem(F32, (B, H, P))) == ESHAPE
    assert st(seq_lens=mem(I32, (B + 1,))) == ESHAPE
    assert st(N=257) == EUNSUP
    assert st(k=mem(F16, (B, Hk, L, N))) == EDTYPE
    assert st(log_decay=mem(BF16, (H,))) == EDTYPE
    assert st(state=mem(BF16, (B, H, P, N))) == EDTYPE
    assert st(seq_lens=mem(F32, (B,))) == EDTYPE
    assert st(io=I32) == EDTYPE
    assert st(out=mem(BF16, (B, H, L, P), (0, L * P, P, 1))) == ESTRIDE
    assert st(state_out=mem(F32, (B, H, P, N), (H * P * N, P * N, 0, 1))) == ESTRIDE
    assert st(q=mem(BF16, (B, Hk, L, N), (-1, 1, 1, 1))) == ESTRIDE
    a = prompt(mem)
    a.out.data = a.v.data
    assert call(fn, a)[0] == EALIAS
    a = prompt(mem)
    a.state_out.data = a.state.data + 4
    assert call(fn, a)[0] == EALIAS
    a = prompt(mem)
    a.state_out = a.state  # in place, spelled out
    assert call(fn, a)[0] == OK
    a = prompt(mem)
    a.out.data = a.state.data
    assert call(fn, a)[0] == EALIAS


def step(mem, B=3, H=4, Hk=2, N=64, P=32, S=None, io=BF16, st=F32, **over):
    S = B if S is None else S
    f = dict(state=mem(st, (S, H, P, N)), q=mem(io, (B, Hk, N)), k=mem(io, (B, Hk, N)), v=mem(io, (B, H, P)),
             out=mem(io, (B, H, P)), log_decay=mem(F32, (H,)), scale=1.0)
    if S != B:
        f["state_batch_indices"] = mem(I32, (B,))
    f.update(over)
    return args_of(bd.LinAttnUpdateArgs, **f)


def test_step_kernels(lib, mem):
    fn = lib.ssm_linear_attention_update
    assert call(fn, step(mem))[1]["kernel"] == "linattn_step_bulk"
    assert call(fn, step(mem, S=9, st=F16))[1]["kernel"] == "linattn_step_bulk"
    gaps = mem(F32, (3, 4, 32, 64), (4 * 32 * 80, 32 * 80, 80, 1))
    assert call(fn, step(mem, state=gaps))[1]["kernel"] == "linattn_step"
    assert call(fn, step(mem, state_out=gaps))[1]["kernel"] == "linattn_step"
    assert call(fn, step(mem, N=66))[1]["kernel"] == "linattn_step_generic"
    assert call(fn, step(mem, state=mem(F32, (3, 4, 32, 64), offset=4)))[1]["kernel"] == "linattn_step_generic"
    assert call(fn, step(mem, B=0))[1]["kernel"] == "none"


def test_step_refusals(lib, mem):
    fn = lib.ssm_linear_attention_update

    def st(**over):
        return call(fn, step(mem, **over))[0]

    assert fn(None, None) == ENULL
    assert st(struct_size=0) == EVER
    assert st(state=bd.Tensor()) == ENULL
    assert st(state=mem(F32, (4, 4, 32, 64))) == ESHAPE  # slots without indices
    assert st(q=mem(BF16, (3, 2, 65))) == ESHAPE
    assert st(v=mem(BF16, (3, 4, 33))) == ESHAPE
    assert st(Hk=3) == ESHAPE
    assert st(log_decay=mem(F32, (3, 5))) == ESHAPE
    assert st(S=9, state_batch_indices=mem(I32, (4,))) == ESHAPE
    assert st(N=300) == EUNSUP
    assert st(S=9, state_batch_indices=mem(F32, (3,))) == EDTYPE
    assert st(state_out=mem(F16, (3, 4, 32, 64))) == EDTYPE
    assert st(k=mem(F32, (3, 2, 64))) == EDTYPE
    assert st(state=mem(F32, (3, 4, 32, 64), (0, 32 * 64, 64, 1))) == ESTRIDE
    a = step(mem)
    a.out.data = a.v.data
    assert call(fn, a)[0] == EALIAS
    a = step(mem)
    a.state_out = mem(F32, (3, 4, 32, 64))
    a.state_out.data = a.state.data + 64
    assert call(fn, a)[0] == EALIAS


# ---------------------------------------------------------- paged attention --
def paged(mem, B=2, Hq=8, Hkv=2, D=64, pages=40, page=16, M=10, io=BF16, with_weights=False, with_lse=False, **over):
    f = dict(q=mem(io, (B, Hq, D)), out=mem(io, (B, Hq, D)), k_cache=mem(io, (pages, page, Hkv, D)),
             v_cache=mem(io, (pages, page, Hkv, D)), block_table=mem(I32, (B, M)), seq_lens=mem(I32, (B,)), scale=0.1)
    if with_weights:
        f["weights"] = mem(F32, (B, Hkv, M * page))
    if with_lse:
        f["lse"] = mem(F32, (B, Hq))
    f.update(over)
    return args_of(bd.PagedAttentionArgs, **f)


def test_paged_kernels_and_workspace(lib, mem):
    fn, size = lib.ssm_paged_attention_decode, lib.ssm_paged_attention_workspace_size
    assert call(fn, paged(mem))[1]["kernel"] == "paged_decode"
    assert call(fn, paged(mem, D=128, Hq=32, with_weights=True, with_lse=True))[1]["kernel"] == "paged_decode"
    assert call(fn, paged(mem, D=40))[1]["kernel"] == "paged_decode"
    assert call(fn, paged(mem, io=F32))[1]["kernel"] == "paged_decode_generic"
    assert call(fn, paged(mem, D=136))[1]["kernel"] == "paged_decode_generic"
    assert call(fn, paged(mem, D=33))[1]["kernel"] == "paged_decode_generic"
    odd = mem(BF16, (40, 16, 2, 64), (16 * 132, 132, 64, 1))
    assert call(fn, paged(mem, k_cache=odd))[1]["kernel"] == "paged_decode_generic"
    assert call(fn, paged(mem, B=0))[1]["kernel"] == "none"
    need = ctypes.c_uint64(0)
    assert size(ctypes.byref(paged(mem)), None) == ENULL
    a = paged(mem)
    assert size(ctypes.byref(a), ctypes.byref(need)) == OK and need.value > 0
    plain = need.value
    w = paged(mem, with_weights=True)
    assert size(ctypes.byref(w), ctypes.byref(need)) == OK and need.value > plain
    w.workspace, w.workspace_bytes = 1 << 30, plain
    assert call(fn, w)[0] == EWS
    w.workspace, w.workspace_bytes = (1 << 30) + 128, need.value + 512
    assert call(fn, w)[0] == EWS
    w.workspace, w.workspace_bytes = w.weights.data, need.value
    assert call(fn, w)[0] == EALIAS
    a.flags = 0  # a real call without a workspace is refused before anything runs
    assert call(fn, a)[0] == EWS


def test_paged_refusals(lib, mem):
    fn = lib.ssm_paged_attention_decode

    def st(**over):
        return call(fn, paged(mem, **over))[0]

    assert fn(None, None) == ENULL
    assert st(struct_size=1) == EVER
    for name in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "out"):
        assert st(**{name: bd.Tensor()}) == ENULL
    assert st(weights_out=mem(F32, (2, 2, 160))) == ENULL  # without weights
    assert st(Hq=7) == ESHAPE
    assert st(v_cache=mem(BF16, (40, 16, 2, 65))) == ESHAPE
    assert st(v_cache=mem(BF16, (41, 16, 2, 64))) == ESHAPE
    assert st(block_table=mem(I32, (3, 10))) == ESHAPE
    assert st(block_table=mem(I32, (2,))) == ESHAPE
    assert st(seq_lens=mem(I32, (3,))) == ESHAPE
    assert st(out=mem(BF16, (2, 8, 65))) == ESHAPE
    assert st(weights=mem(F32, (2, 2, 159))) == ESHAPE
    assert st(weights=mem(F32, (2, 8, 160))) == ESHAPE
    assert st(lse=mem(F32, (2, 2))) == ESHAPE
    assert st(page=0, pages=4) == ESHAPE
    assert st(D=257) == EUNSUP
    assert st(M=1 << 27) == EUNSUP  # more than 2^30 tokens per sequence
    assert st(k_cache=mem(F16, (40, 16, 2, 64))) == EDTYPE
    assert st(block_table=mem(F32, (2, 10))) == EDTYPE
    assert st(seq_lens=mem(F32, (2,))) == EDTYPE
    assert st(weights=mem(BF16, (2, 2, 160))) == EDTYPE
    assert st(lse=mem(BF16, (2, 8))) == EDTYPE
    assert st(out=mem(BF16, (2, 8, 64), (0, 64, 1))) == ESTRIDE
    assert st(weights=mem(F32, (2, 2, 160), (160, 0, 1))) == ESTRIDE
    a = paged(mem)
    a.out.data = a.q.data
    assert call(fn, a)[0] == EALIAS
    a = paged(mem, with_weights=True)
    a.weights_out = mem(F32, (2, 2, 160))
    a.weights_out.data = a.weights.data + 8
    assert call(fn, a)[0] == EALIAS
    a = paged(mem, with_lse=True)
    a.lse.data = a.out.data
    assert call(fn, a)[0] == EALIAS


# ----------------------------------------------------------------- eviction --
def evict(mem, B=2, Hkv=2, D=64, pages=60, page=16, M=10, keep=70, recent=8, io=BF16, **over):
    M2 = -(-keep // page)
    f = dict(k_cache=mem(io, (pages, page, Hkv, D)), v_cache=mem(io, (pages, page, Hkv, D)),
             weights=mem(F32, (B, Hkv, M * page)), block_table=mem(I32, (B, M)), seq_lens=mem(I32, (B,)),
             new_block_table=mem(I32, (B, M2)), keep=keep, recent=recent, new_weights=mem(F32, (B, Hkv, keep)),
             new_seq_lens=mem(I32, (B,)), kept=mem(I32, (B, Hkv, keep)))
    f.update(over)
    return args_of(bd.KvEvictArgs, **f)


def test_evict_refusals(lib, mem):
    fn = lib.ssm_kv_cache_evict

    def st(**over):
        return call(fn, evict(mem, **over))[0]

    assert fn(None, None) == ENULL
    assert call(fn, evict(mem))[1]["kernel"] == "kv_evict"
    assert call(fn, evict(mem, B=0))[1]["kernel"] == "none"
    assert st(struct_size=1) == EVER
    for name in ("k_cache", "v_cache", "weights", "block_table", "seq_lens", "new_block_table", "new_weights",
                 "new_seq_lens", "kept"):
        assert st(**{name: bd.Tensor()}) == ENULL
    assert st(recent=71) == ESHAPE
    assert st(recent=-1) == ESHAPE
    assert st(keep=0, recent=0) == ESHAPE
    assert st(new_block_table=mem(I32, (2, 4))) == ESHAPE  # room for 64 of 70
    assert st(new_block_table=mem(I32, (1, 5))) == ESHAPE
    assert st(weights=mem(F32, (2, 2, 159))) == ESHAPE
    assert st(kept=mem(I32, (2, 2, 71))) == ESHAPE
    assert st(new_seq_lens=mem(I32, (3,))) == ESHAPE
    assert st(v_cache=mem(BF16, (60, 16, 2, 32))) == ESHAPE
    assert st(v_cache=mem(F32, (60, 16, 2, 64))) == EDTYPE
    assert st(io=I32) == EDTYPE
    assert st(weights=mem(BF16, (2, 2, 160))) == EDTYPE
    assert st(kept=mem(F32, (2, 2, 70))) == EDTYPE
    assert st(k_cache=mem(BF16, (60, 16, 2, 64), (0, 128, 64, 1))) == ESTRIDE
    assert st(kept=mem(I32, (2, 2, 70), (140, 0, 1))) == ESTRIDE
    a = evict(mem)
    a.new_weights.data = a.weights.data
    assert call(fn, a)[0] == EALIAS
    a = evict(mem)
    a.kept.data = a.k_cache.data
    assert call(fn, a)[0] == EALIAS
    a = evict(mem)  # keys and values interleaved in one pool: their extents overlap, they do not
    a.k_cache = bd.raw_tensor(1 << 45, BF16, (60, 16, 2, 64), (2 * 16 * 128, 128, 64, 1))
    a.v_cache = bd.raw_tensor((1 << 45) + 16 * 128 * 2, BF16, (60, 16, 2, 64), (2 * 16 * 128, 128, 64, 1))
    assert call(fn, a)[0] == OK


def test_binding_refuses_cpu_tensors_and_bad_workspaces():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 2, 4, 8)
    with pytest.raises(ValueError):
        bd.ssm_linear_attention_fwd(q, q, q, torch.zeros(2))
    with pytest.raises(ValueError):
        bd.ssm_paged_attention_decode(torch.zeros(1, 2, 8), torch.zeros(4, 4, 2, 8), torch.zeros(4, 4, 2, 8),
                                      torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
