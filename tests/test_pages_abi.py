"""Refusals of the page bookkeeping, on the host and before any launch (no GPU
needed): sizes, alignment, strides, overlaps; empty problems succeed; the torch
layer's own checks."""
import ctypes

import pytest
import torch

from decode_context_attention_gb300 import binding, build

OK, INVALID, MISALIGNED, ALIAS = 0, 1, 4, 5
# plausible, disjoint and never dereferenced addresses
CL, NL, GS, PL, BT, FP, FC, FO, MI, QS, SL, POS, SLOT, REQ, KL, LO = (0x100000000 * (i + 1) for i in range(16))


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def reserve(**c):
    a = dict(N=2, B=3, T=8, page=16, pages=10, L=100, lens=CL, new=NL, G=1, gs=GS, pl=PL, bt=BT, bt_sn=12, bt_sb=4,
             mp=4, fp=FP, fp_sn=10, cap=10, fc=FC, fo=FO, mi=MI, qs=QS, sl=SL, pos=POS, slot=SLOT, req=REQ, stream=None)
    assert not set(c) - set(a)
    a.update(c)
    return binding.dcp_page_reserve(*a.values())


def release(**c):
    a = dict(N=2, B=3, page=16, pages=10, L=100, lens=CL, keep=KL, G=1, gs=GS, pl=PL, bt=BT, bt_sn=12, bt_sb=4,
             mp=4, fp=FP, fp_sn=10, cap=10, fc=FC, fo=FO, lo=LO, stream=None)
    assert not set(c) - set(a)
    a.update(c)
    return binding.dcp_page_release(*a.values())


@pytest.mark.parametrize("call", [reserve, release])
@pytest.mark.parametrize("change,status", [
    (dict(N=0), INVALID), (dict(N=5000), INVALID), (dict(B=-1), INVALID), (dict(B=1 << 30), INVALID),
    (dict(N=4096, B=1 << 20), INVALID), (dict(L=-1), INVALID), (dict(L=(1 << 30) + 1, mp=1 << 30), INVALID),
    (dict(page=0), INVALID), (dict(page=24), INVALID), (dict(page=1 << 17), INVALID), (dict(pages=0), INVALID),
    (dict(mp=3), INVALID), (dict(cap=0), INVALID), (dict(G=-1), INVALID),
    (dict(lens=None), INVALID), (dict(gs=None), INVALID), (dict(pl=None), INVALID), (dict(bt=None), INVALID),
    (dict(fp=None), INVALID), (dict(fc=None), INVALID), (dict(fo=None), INVALID),
    (dict(bt_sn=-1), INVALID), (dict(bt_sb=(1 << 52) + 1), INVALID), (dict(fp_sn=-4), INVALID),
    (dict(N=4000, bt_sn=1 << 51), INVALID),
    (dict(lens=CL + 2), MISALIGNED), (dict(bt=BT + 1), MISALIGNED), (dict(fp=FP + 2), MISALIGNED),
    (dict(fo=FO + 2), MISALIGNED), (dict(gs=GS + 2), MISALIGNED),
    (dict(fo=CL), ALIAS), (dict(fo=FC + 4), ALIAS), (dict(fo=BT), ALIAS), (dict(fo=GS), ALIAS), (dict(fp=BT), ALIAS),
])
def test_refusals(call, change, status):
    assert call(**change) == status
    assert binding.dcp_last_error_message()


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(T=(1 << 30) + 1), INVALID), (dict(new=None), INVALID), (dict(mi=None), INVALID),
    (dict(qs=None), INVALID), (dict(sl=None), INVALID), (dict(slot=SLOT + 4), MISALIGNED), (dict(pos=POS + 2), MISALIGNED),
    (dict(bt_sb=3), ALIAS), (dict(bt_sn=0), ALIAS), (dict(sl=CL), ALIAS), (dict(sl=NL), ALIAS), (dict(qs=SL - 4), ALIAS),
    (dict(pos=REQ), ALIAS), (dict(slot=POS), ALIAS), (dict(mi=FO), ALIAS), (dict(bt=FP), ALIAS), (dict(mi=FC), ALIAS),
    (dict(qs=PL), ALIAS),
])
def test_reserve_refusals(change, status):
    assert reserve(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(keep=None), INVALID), (dict(lo=CL), ALIAS), (dict(lo=KL), ALIAS), (dict(lo=FO), ALIAS), (dict(fp_sn=9), ALIAS),
    (dict(lo=LO + 2), MISALIGNED), (dict(fp=KL), ALIAS), (dict(lo=BT + 4), ALIAS),
])
def test_release_refusals(change, status):
    assert release(**change) == status


def test_empty_problems_succeed_and_launch_nothing():
    assert reserve(B=0) == OK and release(B=0) == OK
    assert reserve(B=0, lens=None, bt=None) == OK


def test_torch_layer_checks_devices():
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):     # ordinary host memory
        binding.page_reserve(ints(3), ints(3), 100, 8, 10, 16, ints(2, 3, 4), ints(2, 10), ints(2), ints(2), ints(2),
                             ints(4), ints(3))
    with pytest.raises(ValueError):
        binding.page_release(ints(3), ints(3), 100, 10, 16, ints(2, 3, 4), ints(2, 10), ints(2), ints(2))


def test_symbols_are_exported(lib):
    for name in ("dcp_page_reserve", "dcp_page_release"):
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr)


@pytest.mark.parametrize("call,names", [(reserve, ("lens", "new", "gs", "pl", "fp")), (release, ("lens", "keep", "gs", "pl", "bt"))])
def test_only_the_counts_themselves_may_be_written_in_place(call, names):
    for name in names:
        # another array where both counts are (every call is refused before a launch)
        assert call(**{name: FC, "fo": FC}) == ALIAS, name
