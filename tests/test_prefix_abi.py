"""Refusals of the attention of batches that share prefixes, on the host and before
any launch (no GPU needed)."""
import ctypes

import pytest
import torch

from decode_context_attention_gb300 import binding, build

OK, INVALID, DTYPE, HEADS, MISALIGNED, ALIAS = 0, 1, 2, 3, 4, 5
# plausible, disjoint and never dereferenced addresses
Q, KP, VP, BT, QS, SL, GS, PL, O, LSE, WS = (0x100000000 * (i + 1) for i in range(11))


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def prefix(**c):
    a = dict(dtype=2, N=2, B=3, T=8, H=4, Hkv=2, D=128, q=Q, q_st=512, q_sh=128, kp=KP, kp_sn=65536 * 4, kp_sp=4096,
             kp_st=256, kp_sh=128, vp=VP, vp_sn=65536 * 4, vp_sp=4096, vp_st=256, vp_sh=128, pages=10, page=16, bt=BT,
             bt_sn=12, bt_sb=4, mp=4, qs=QS, sl=SL, L=100, G=2, gs=GS, pl=PL, scale=0.1, causal=1, o=O, o_sn=4096,
             o_st=512, o_sh=128, lse=LSE, l_sn=32, l_st=4, l_sh=1, base=0, ws=WS, wsb=1 << 40, stream=None)
    assert not set(c) - set(a)
    a.update(c)
    return binding.dcp_prefix_attention_paged(*a.values())


@pytest.mark.parametrize("change,status", [
    (dict(dtype=0), DTYPE), (dict(dtype=3), DTYPE), (dict(N=0), INVALID), (dict(B=-1), INVALID), (dict(H=5), HEADS),
    (dict(H=130), INVALID), (dict(D=96), INVALID), (dict(page=24), INVALID), (dict(mp=3), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(base=2), INVALID), (dict(G=-1), INVALID), (dict(G=1 << 30), INVALID),
    (dict(N=4096, G=1 << 18), INVALID), (dict(gs=None), INVALID), (dict(pl=None), INVALID), (dict(gs=GS + 2), MISALIGNED),
    (dict(pl=PL + 1), MISALIGNED), (dict(q=None), INVALID), (dict(o=GS), ALIAS), (dict(lse=PL), ALIAS),
    (dict(ws=GS), ALIAS), (dict(ws=KP), ALIAS), (dict(ws=None), INVALID), (dict(wsb=1000), INVALID),
    (dict(ws=WS + 8), MISALIGNED), (dict(o=Q), ALIAS), (dict(o_sh=64), ALIAS), (dict(q_sh=4), MISALIGNED),
    (dict(kp_sn=-1), INVALID), (dict(L=-1), INVALID),
])
def test_refusals(change, status):
    assert prefix(**change) == status
    assert binding.dcp_last_error_message()


def test_workspace_holds_the_rows_that_are_joined():
    size, extend = binding.dcp_prefix_attention_workspace_size, binding.dcp_extend_attention_workspace_size
    args = (2, 3, 8, 4, 2, 128, 100)
    assert size(*args, 0) == extend(*args)
    assert size(*args, 2) >= extend(*args) + 8 * 2 * 8 * 4 * 129
    need = size(*args, 2)
    assert prefix(wsb=need - 1) == INVALID
    for bad in ((0, 3, 8, 4, 2, 128, 100, 1), (2, 3, 8, 5, 2, 128, 100, 1), (2, 3, 8, 4, 2, 128, 100, -1)):
        assert size(*bad) == 0


def test_empty_problems_succeed_and_launch_nothing():
    assert prefix(B=0) == OK and prefix(T=0) == OK
    assert prefix(T=0, gs=None, pl=None, q=None, ws=None) == OK


def test_torch_layer():
    q, kp = torch.zeros(8, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 10, 16, 2, 128, dtype=torch.bfloat16)
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):     # ordinary host memory
        binding.prefix_attention_paged(q, kp, kp, ints(2, 3, 4), ints(4), ints(3), 100, ints(2), ints(1),
                                       torch.zeros(2, 8, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 8, 4), 0.1)
    for n in (1 << 31, -(1 << 40)):
        with pytest.raises(ValueError):
            binding.prefix_workspace_bytes(2, 3, 8, 4, 2, 128, n, 1)


def test_symbols_are_exported(lib):
    for name in ("dcp_prefix_attention_paged", "dcp_prefix_attention_workspace_size"):
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr)
