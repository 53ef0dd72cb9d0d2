"""Refusals of the chunk-serving entry points, on the host and before any launch
(no GPU needed): sizes, head counts, alignment, strides, overlaps, workspaces;
empty problems succeed; the torch layer's own checks."""
import ctypes

import pytest
import torch

from decode_context_attention_gb300 import binding, build

OK, INVALID, DTYPE, HEADS, MISALIGNED, ALIAS = 0, 1, 2, 3, 4, 5
F32, F16, BF16 = 0, 1, 2
# plausible, disjoint and never dereferenced addresses
Q, K, V, O, KP, VP, BT, QS, SL, LSE, WS, W, CS, PS, ACC, KL, DT, KEPT, OUT = (0x100000000 * (i + 1) for i in range(19))


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def append(**c):
    a = dict(dtype=BF16, N=2, B=3, T=8, H=4, Hkv=2, D=128, q=Q, q_st=512, q_sh=128, k=K, k_st=256, k_sh=128, v=V,
             v_st=256, v_sh=128, qw=W, kw=W + 256, eps=1e-6, cs=CS, npos=64, rot=128, inter=0, ps=PS, o=O, o_st=512,
             o_sh=128, kp=KP, kp_sn=65536 * 4, kp_sp=4096, kp_st=256, kp_sh=128, vp=VP, vp_sn=65536 * 4, vp_sp=4096,
             vp_st=256, vp_sh=128, pages=10, page=16, bt=BT, bt_sn=12, bt_sb=4, mp=4, qs=QS, sl=SL, L=100, stream=None)
    assert not set(c) - set(a)
    a.update(c)
    return binding.dcp_qk_norm_rope_append(*a.values())


def extend(**c):
    a = dict(dtype=BF16, N=2, B=3, T=8, H=4, Hkv=2, D=128, q=Q, q_st=512, q_sh=128, kp=KP, kp_sn=65536 * 4, kp_sp=4096,
             kp_st=256, kp_sh=128, vp=VP, vp_sn=65536 * 4, vp_sp=4096, vp_st=256, vp_sh=128, pages=10, page=16, bt=BT,
             bt_sn=12, bt_sb=4, mp=4, qs=QS, sl=SL, L=100, scale=0.1, causal=1, o=O, o_sn=4096, o_st=512, o_sh=128,
             lse=LSE, l_sn=32, l_st=4, l_sh=1, base=0, ws=WS, wsb=1 << 40, stream=None)
    assert not set(c) - set(a)
    a.update(c)
    return binding.dcp_extend_attention_paged(*a.values())


def weights(**c):
    a = dict(dtype=BF16, N=2, B=3, T=8, H=4, Hkv=2, D=128, q=Q, q_st=512, q_sh=128, kp=KP, kp_sn=65536 * 4, kp_sp=4096,
             kp_st=256, kp_sh=128, pages=10, page=16, bt=BT, bt_sn=12, bt_sb=4, mp=4, qs=QS, sl=SL, L=100, scale=0.1,
             lse=LSE, l_st=4, l_sh=1, base=0, acc=ACC, a_sn=300, a_sb=100, a_sh=50, stream=None)
    assert not set(c) - set(a)
    a.update(c)
    return binding.dcp_attention_weights_paged(*a.values())


def evict(**c):
    a = dict(dtype=BF16, N=2, B=3, Hkv=2, D=128, kp=KP, kp_sn=65536 * 4, kp_sp=4096, kp_st=256, kp_sh=128, vp=VP,
             vp_sn=65536 * 4, vp_sp=4096, vp_st=256, vp_sh=128, pages=10, page=16, bt=BT, bt_sn=12, bt_sb=4, mp=4, sl=SL,
             L=100, acc=ACC, a_sn=300, a_sb=100, a_sh=50, kl=KL, max_keep=60, recent=8, dt=DT, dt_sn=6, dt_sb=2, dmp=2,
             kept=KEPT, k_sn=180, k_sb=60, k_sh=30, out=OUT, u_sn=180, u_sb=60, u_sh=30, stream=None)
    assert not set(c) - set(a)
    a.update(c)
    return binding.dcp_cache_evict_paged(*a.values())


BATCH = [
    (dict(dtype=F32), DTYPE), (dict(dtype=3), DTYPE), (dict(dtype=9), DTYPE),
    (dict(N=0), INVALID), (dict(N=5000), INVALID), (dict(B=-1), INVALID), (dict(Hkv=0), INVALID),
    (dict(L=-1), INVALID), (dict(L=(1 << 30) + 1, mp=1 << 30), INVALID), (dict(page=0), INVALID),
    (dict(page=24), INVALID), (dict(page=1 << 17), INVALID), (dict(pages=0), INVALID), (dict(mp=3), INVALID),
    (dict(kp=None), INVALID), (dict(bt=None), INVALID), (dict(sl=None), INVALID),
    (dict(kp_sn=-1), INVALID), (dict(kp_sp=(1 << 52) + 1), INVALID), (dict(bt_sn=-4), INVALID),
    (dict(kp_sn=1 << 52, pages=1 << 20, kp_sp=1 << 51), INVALID),
    (dict(kp=KP + 8), MISALIGNED), (dict(kp_st=260), MISALIGNED), (dict(bt=BT + 2), MISALIGNED),
    (dict(sl=SL + 1), MISALIGNED),
]


@pytest.mark.parametrize("call", [append, extend, weights, evict])
@pytest.mark.parametrize("change,status", BATCH)
def test_batch_and_page_arguments(call, change, status):
    assert call(**change) == status
    assert binding.dcp_last_error_message()


HEADS_CASES = [(dict(H=5), HEADS), (dict(H=0), INVALID), (dict(H=130, Hkv=2), INVALID), (dict(D=96), INVALID),
               (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(base=2), INVALID),
               (dict(T=1 << 29), INVALID), (dict(T=-1), INVALID), (dict(q=None), INVALID), (dict(q=Q + 8), MISALIGNED),
               (dict(q_sh=4), MISALIGNED), (dict(qs=None), INVALID), (dict(qs=QS + 2), MISALIGNED),
               (dict(lse=None), INVALID), (dict(lse=LSE + 2), MISALIGNED)]


@pytest.mark.parametrize("call", [extend, weights])
@pytest.mark.parametrize("change,status", HEADS_CASES)
def test_head_arguments(call, change, status):
    assert call(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(H=0), INVALID), (dict(D=24), INVALID), (dict(D=528), INVALID), (dict(rot=24), INVALID),
    (dict(rot=144), INVALID), (dict(npos=0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=-1.0), INVALID),
    (dict(T=1 << 30), INVALID), (dict(cs=None), INVALID), (dict(ps=None), INVALID), (dict(v=None), INVALID),
    (dict(qw=W + 2), MISALIGNED), (dict(cs=CS + 4), MISALIGNED), (dict(ps=PS + 2), MISALIGNED),
    (dict(o=O + 2), MISALIGNED), (dict(k_sh=132), MISALIGNED),
    (dict(o=Q + 256), ALIAS), (dict(o=K), ALIAS), (dict(o=KP), ALIAS), (dict(kp=Q), ALIAS), (dict(vp=V), ALIAS),
    (dict(vp=KP), ALIAS), (dict(vp=KP + 256), ALIAS), (dict(o_sh=64), ALIAS), (dict(kp_st=0), ALIAS),
    (dict(o=CS), ALIAS), (dict(kp=BT), ALIAS),
])
def test_append_refusals(change, status):
    assert append(**change) == status


def test_append_takes_a_fused_projection_in_place():
    # rows [q heads | k heads | v heads] of one buffer, q_out = q: refused only when the rows really meet.  B = 0
    # stops before the launch, so these calls go as far as a device would be needed and no further.
    fused = dict(q=Q, q_st=1024, q_sh=128, k=Q + 4 * 256, k_st=1024, k_sh=128, v=Q + 6 * 256, v_st=1024, v_sh=128, o=Q,
                 o_st=1024, o_sh=128)
    assert append(**{**fused, "k": Q + 3 * 256}) == ALIAS       # the last q head is a k head
    assert append(**{**fused, "o_st": 512, "q_st": 512}) == ALIAS


@pytest.mark.parametrize("change,status", [
    (dict(ws=None), INVALID), (dict(wsb=1000), INVALID), (dict(ws=WS + 8), MISALIGNED), (dict(ws=KP), ALIAS),
    (dict(ws=O), ALIAS), (dict(o=Q), ALIAS), (dict(o=KP), ALIAS), (dict(lse=Q), ALIAS), (dict(lse=O), ALIAS),
    (dict(o_sh=64), ALIAS), (dict(o_st=256), ALIAS), (dict(l_sh=0), ALIAS), (dict(o=O + 2), MISALIGNED),
    (dict(o=None), INVALID), (dict(vp=None), INVALID), (dict(vp_sh=132), MISALIGNED), (dict(o_sn=-1), INVALID),
])
def test_extend_refusals(change, status):
    assert extend(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(acc=None), INVALID), (dict(acc=ACC + 1), MISALIGNED), (dict(acc=LSE), ALIAS), (dict(acc=KP), ALIAS),
    (dict(acc=Q), ALIAS), (dict(a_sh=49), ALIAS), (dict(a_sb=0), ALIAS), (dict(a_sn=-1), INVALID),
])
def test_weights_refusals(change, status):
    assert weights(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(D=4), INVALID), (dict(D=132), INVALID), (dict(D=2048), INVALID), (dict(max_keep=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(dmp=1), INVALID), (dict(kl=None), INVALID), (dict(dt=None), INVALID),
    (dict(kept=None), INVALID), (dict(out=None), INVALID), (dict(acc=None), INVALID), (dict(vp=None), INVALID),
    (dict(kept=KEPT + 2), MISALIGNED), (dict(out=OUT + 2), MISALIGNED), (dict(kl=KL + 2), MISALIGNED),
    (dict(out=ACC), ALIAS), (dict(kept=ACC), ALIAS), (dict(kept=OUT), ALIAS), (dict(kept=KP), ALIAS),
    (dict(k_sh=29), ALIAS), (dict(u_sb=0), ALIAS), (dict(vp=KP), ALIAS), (dict(kp=DT), ALIAS), (dict(k_sn=-1), INVALID),
])
def test_evict_refusals(change, status):
    assert evict(**change) == status


def test_empty_problems_succeed_and_launch_nothing():
    assert append(B=0) == OK and append(T=0) == OK
    assert extend(B=0) == OK and extend(T=0) == OK
    assert weights(B=0) == OK and weights(T=0) == OK and weights(L=0) == OK
    assert evict(B=0) == OK and evict(L=0) == OK and evict(max_keep=0) == OK
    # pointers are not looked at then
    assert extend(T=0, q=None, o=None, ws=None) == OK


def test_workspace_size_refuses_what_the_call_refuses():
    size = binding.dcp_extend_attention_workspace_size
    assert size(2, 3, 8, 4, 2, 128, 100) > 0
    for bad in ((0, 3, 8, 4, 2, 128, 100), (2, -1, 8, 4, 2, 128, 100), (2, 3, 8, 5, 2, 128, 100),
                (2, 3, 8, 4, 2, 96, 100), (2, 3, 8, 260, 2, 128, 100), (2, 3, 8, 4, 2, 128, -1)):
        assert size(*bad) == 0


def test_torch_layer_checks_shapes_and_types():
    def pinned_like(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype)

    q, kp = pinned_like(8, 4, 128), pinned_like(2, 10, 16, 2, 128)
    bt = torch.zeros((2, 3, 4), dtype=torch.int32)
    qs, sl = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    acc = torch.zeros((2, 3, 2, 50))
    lse = torch.zeros((8, 4))
    with pytest.raises(ValueError):     # ordinary host memory
        binding.attention_weights_paged(q, kp, bt, qs, sl, 100, lse, acc, 0.1)


def test_lengths_beyond_32_bits_are_refused():
    for n in (1 << 31, (1 << 32) + 5, -(1 << 40)):
        with pytest.raises(ValueError):
            binding.extend_workspace_bytes(2, 3, 8, 4, 2, 128, n)


def test_symbols_are_exported(lib):
    for name in ("dcp_qk_norm_rope_append", "dcp_extend_attention_workspace_size", "dcp_extend_attention_paged",
                 "dcp_attention_weights_paged", "dcp_cache_evict_paged"):
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr)
