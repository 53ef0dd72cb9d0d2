"""The norm, rotation and append of new tokens against its definition in 64 bits:
odd head counts, partial and interleaved rotation, no norm, fused projections,
padding rows, in place, skipped tokens, bad pages, another stream, a graph."""
import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV, TINY, U, Batch, share

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def inputs(bt, rot, fused=True, positions=None, seed=5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T, H, Hkv, D = bt.T, bt.H, bt.Hkv, bt.D
    if fused:
        qkv = (torch.randn((T, H + 2 * Hkv, D), generator=g, device=DEV) * 3).to(bt.dtype)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:
        q, k, v = ((torch.randn((T, n, D), generator=g, device=DEV) * 3).to(bt.dtype) for n in (H, Hkv, Hkv))
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(bt.dtype) for _ in range(2))
    P = bt.max_len + 9
    cs = None
    if rot:
        ang = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * 100.0 ** (
            -torch.arange(rot // 2, device=DEV, dtype=torch.float64) / max(1, rot // 2))
        cs = torch.cat([ang.cos(), ang.sin()], -1).float()
        if positions is None:
            positions = [l - n + j + 3 for n, l in bt.lens for j in range(n)]
            positions += [0] * (T - len(positions))
        positions = torch.tensor(positions, dtype=torch.int32, device=DEV)
    return q, k, v, qw, kw, cs, positions if rot else None


def turned(x, w, eps, cs, pos, rot, inter):
    """[T, heads, D] in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    if not rot:
        return x
    row = cs.double()[pos.long().clamp(0, cs.shape[0] - 1)][:, None]
    c, s = row[..., : rot // 2], row[..., rot // 2:]
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    return y


def close(got, want, dtype, what):
    # one rounding to the type; the norm, weight and rotation in 32 bits are off by a few units of 2^-24 of the
    # row's largest magnitude (a sum of up to 512 squares: 32 units)
    top = want.abs().amax(-1, keepdim=True)
    tol = U[dtype] * (want.abs() + 64 * 2.0 ** -24 * top) + 64 * 2.0 ** -24 * top + TINY[dtype]
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off"


def run(bt, rot=0, inter=False, norm=True, fused=True, skip=(), bad=(), stream=None, inplace=False, check=True,
        positions=None):
    q, k, v, qw, kw, cs, pos = inputs(bt, rot, fused, positions)
    q0 = q.clone()
    if not norm:
        qw = kw = None
    eps = 1e-5
    out = q if inplace else torch.full((bt.T, bt.H, bt.D), 7.0, dtype=bt.dtype, device=DEV)
    k_was, v_was = bt.k_pages.clone(), bt.v_pages.clone()
    args = (q, k, v, qw, kw, eps, cs, pos, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens,
            bt.max_len, out)
    want_q, want_k = turned(q0, qw, eps, cs, pos, rot, inter), turned(k.clone(), kw, eps, cs, pos, rot, inter)
    binding.qk_norm_rope_append(*args, interleaved=inter, stream=stream)
    torch.cuda.synchronize()
    if not check:
        return args, want_q, want_k
    n = bt.start[-1]
    live = torch.tensor([t not in skip for t in range(n)], device=DEV, dtype=torch.bool)
    close(out[:n][live], want_q[:n][live], bt.dtype, "q")
    left = q0 if inplace else torch.full_like(out, 7.0)
    assert torch.equal(out[n:], left[n:]) and torch.equal(out[:n][~live], left[:n][~live])
    # the pages: what was there, but for the new tokens' slots
    want_kp, want_vp = k_was.double(), v_was.clone()
    at_k = torch.zeros(k_was.shape[:3], dtype=torch.bool, device=DEV)
    for b, (m, l) in enumerate(bt.lens):
        for j in range(m):
            t, g = bt.start[b] + j, l - m + j
            if t in skip or g < 0:
                continue
            r, i = g % bt.N, g // bt.N
            pg = int(bt.block_table[r, b, i // bt.page])
            if not 0 <= pg < bt.num_pages:
                continue
            want_kp[r, pg, i % bt.page] = want_k[t]
            want_vp[r, pg, i % bt.page] = v[t]
            at_k[r, pg, i % bt.page] = True
    assert torch.equal(bt.v_pages.view(torch.int16), want_vp.view(torch.int16)), "V pages"
    assert torch.equal(bt.k_pages[~at_k].view(torch.int16), k_was[~at_k].view(torch.int16)), "K outside the new slots"
    close(bt.k_pages[at_k], want_kp[at_k], bt.dtype, "K")


CASES = [
    # lens, N, H, Hkv, D, page, dtype, rot, interleaved, pad
    ([(1, 1)], 1, 1, 1, 16, 1, torch.bfloat16, 16, False, 0),
    ([(1, 7), (1, 300)], 3, 5, 1, 64, 8, torch.float16, 64, False, 0),
    ([(17, 17), (0, 40), (1, 33), (130, 400)], 4, 8, 2, 128, 16, torch.bfloat16, 128, False, 5),
    ([(17, 19), (0, 0), (64, 100)], 2, 6, 3, 128, 64, torch.float16, 64, True, 1),
    ([(3, 50), (2, 2)], 2, 4, 4, 96, 32, torch.bfloat16, 32, True, 0),
    ([(40, 41)], 8, 12, 1, 256, 16, torch.bfloat16, 256, True, 2),
    ([(9, 20)], 2, 3, 1, 512, 4, torch.float16, 256, False, 0),
    ([(9, 20)], 2, 3, 1, 80, 4, torch.float16, 0, False, 0),
    ([(700, 901), (1, 5)] + [(1, 1 + i) for i in range(70)], 3, 16, 8, 128, 32, torch.bfloat16, 128, False, 3),
]


@pytest.mark.parametrize("lens,N,H,Hkv,D,page,dtype,rot,inter,pad", CASES)
@pytest.mark.parametrize("norm", [True, False])
def test_append_matches_the_definition(lens, N, H, Hkv, D, page, dtype, rot, inter, pad, norm):
    bt = Batch(lens, N, H, Hkv, D, page, dtype, pad, seed=len(lens) + D)
    run(bt, rot, inter, norm)


def test_append_many_rows_per_group():
    # enough tokens that a lane group takes several rows of one
    bt = Batch([(6000, 6100), (2500, 2500)], 2, 8, 2, 128, 64, torch.bfloat16, 1, seed=3)
    run(bt, 128, False)


@pytest.mark.parametrize("D", [64, 128, 16])
def test_append_finds_the_owner_among_many_requests(D):
    run(Batch([(b % 4, 3 + b % 4 + 13 * b % 97) for b in range(1100)], 3, 4, 2, D, 16, torch.bfloat16, 3, seed=D), D, False)


def test_append_in_place_strided_pool_and_stream():
    bt = Batch([(5, 9), (33, 70)], 2, 4, 2, 128, 16, torch.bfloat16, 2, seed=4, strided=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(bt, 64, True, stream=s, inplace=True)
    bt = Batch([(5, 9)], 2, 4, 2, 128, 16, torch.bfloat16, 2, seed=4)
    run(bt, 128, False, fused=False, inplace=True)


def test_append_skips_positions_outside_the_table():
    bt = Batch([(6, 9)], 2, 4, 2, 64, 16, torch.float16, 0, seed=6)
    P = bt.max_len + 9
    run(bt, 64, False, positions=[0, -1, P - 1, P, 2 ** 31 - 1, 3], skip=(1, 3, 4))


def test_append_leaves_out_pages_outside_the_pool_and_negative_indices():
    bt = Batch([(20, 40), (9, 12)], 2, 4, 2, 64, 4, torch.float16, 0, seed=7)
    bt.block_table[0, 0, 3], bt.block_table[1, 0, 4] = bt.num_pages, -1
    run(bt, 64, False)
    # more new tokens than the length says: the first have no place
    bt = Batch([(9, 9)], 2, 4, 2, 64, 4, torch.float16, 0, seed=7)
    bt.lens = [(9, 5)]
    bt.seq_lens.fill_(5)
    run(bt, 64, False, positions=list(range(9)))


def test_append_captured_into_a_graph_follows_its_inputs():
    bt = Batch([(4, 30), (1, 9)], 2, 4, 2, 128, 16, torch.bfloat16, 3, seed=8)
    args, *_ = run(bt, 128, False, check=False)
    q, k, v, qw, kw, eps, cs, pos, kp, vp, table, qs, sl, ml, out = args
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.qk_norm_rope_append(*args)
    q.copy_(torch.randn_like(q))
    sl.copy_(torch.tensor([28, 8], device=DEV))     # other lengths and a shorter batch
    qs.copy_(torch.tensor([0, 2, 3], device=DEV))
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    close(out[:3], turned(q, qw, eps, cs, pos, 128, False)[:3], bt.dtype, "q")
    assert bool((out[3:] == 7.0).all())
    for t, (b, g) in enumerate([(0, 26), (0, 27), (1, 7)]):
        r, i = g % 2, g // 2
        assert torch.equal(vp[r, int(table[r, b, i // 16]), i % 16], v[t])
