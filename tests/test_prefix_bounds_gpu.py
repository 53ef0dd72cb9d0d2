"""Groups' arrays that the documentation does not allow (borders out of order): outputs may be anything, but nothing
beside them is written: padding rows, the gaps between rows, pools, tables, the batch's arrays, and what lies in front of
and behind the workspace and the outputs keep their marks."""
import pytest
import torch

from chunk_ref import DEV
from decode_context_attention_gb300 import binding, build
from test_pages_gpu import State, ints
from test_prefix_attention_gpu import Shared

pytestmark = pytest.mark.gpu
MARK = 0x5A


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def marked(shape, dtype, gap):
    """A tensor within a larger one of marks: (the larger one's bytes, the tensor), its last two dimensions' rows `gap`
    elements apart and with as much in front and behind."""
    wide = (shape[0] + 2, *shape[1:-1], shape[-1] + gap)
    size = torch.empty((), dtype=dtype).element_size()
    n = size
    for x in wide:
        n *= x
    raw = torch.full((n,), MARK, dtype=torch.uint8, device=DEV)
    return raw, raw.view(dtype).view(wide)[1:-1, ..., :shape[-1]]


def untouched(raw, wide_shape, dtype, rows, last):
    """Whether all bytes but those of `rows` (of the dimension after the first) and the first `last` elements are marks."""
    size = torch.empty((), dtype=dtype).element_size()
    x = raw.view(wide_shape[0], wide_shape[1], -1, wide_shape[-1] * size).clone()
    x[1:-1, :rows, :, :last * size] = MARK
    return bool((x == MARK).all())


# (few requests; many and long enough for common parts; chunks that the tensor-core kernel takes)
BATCHES = {
    "few": ([(1, 200), (1, 190), (2, 180)], 96),
    "many": ([(1 + b % 3, 2900 + 3 * b) for b in range(20)], 2880),
    "many, and chunks": ([(1 + 40 * (b % 4 == 3), 6500 + 3 * b) for b in range(20)], 6400),
}
BORDERS = [lambda B: [2, 0, B], lambda B: [0, B, 1], lambda B: [B, B // 2, 0], lambda B: [B // 2, 0, B],
           lambda B: [0, 2 ** 31 - 1, 3], lambda B: [5, -2 ** 31, B], lambda B: [-1, -7, B], lambda B: [B // 2, B, 0]]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("borders", range(len(BORDERS)))
@pytest.mark.parametrize("name", BATCHES)
def test_borders_out_of_order(name, borders, D):
    lens, n = BATCHES[name]
    bt = Shared(lens, [(0, len(lens), n)], D=D, pad=3, strided=True, seed=borders)
    bt.group_start = torch.tensor(BORDERS[borders](bt.B), dtype=torch.int32, device=DEV)
    bt.prefix_lens = torch.tensor([n, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    o_raw, o = marked((bt.N, bt.T, bt.H, D), bt.dtype, 16)
    l_raw, lse = marked((bt.N, bt.T, bt.H), torch.float32, 3)
    need = binding.prefix_workspace_bytes(bt.N, bt.B, bt.T, bt.H, bt.Hkv, D, bt.max_len, 2)
    w_raw = torch.full((need + 1024,), MARK, dtype=torch.uint8, device=DEV)
    kept = [x.clone() for x in (bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens,
                                bt.group_start, bt.prefix_lens)]
    bt.run(workspace=w_raw[512:512 + need], out=(o, lse))
    rows = bt.start[-1]
    assert untouched(o_raw, (bt.N + 2, bt.T, bt.H, D + 16), bt.dtype, rows, D)
    assert untouched(l_raw, (bt.N + 2, bt.T, bt.H + 3), torch.float32, rows, bt.H)
    assert (w_raw[:512] == MARK).all() and (w_raw[512 + need:] == MARK).all()
    for x, y in zip(kept, (bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens, bt.group_start,
                           bt.prefix_lens)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def test_the_marks_are_looked_at():
    raw, x = marked((2, 5, 4, 8), torch.bfloat16, 16)
    shape = (4, 5, 4, 24)
    assert x.shape == (2, 5, 4, 8) and untouched(raw, shape, torch.bfloat16, 3, 8)
    x[:, :3] = 1.0
    assert untouched(raw, shape, torch.bfloat16, 3, 8)
    x[1, 3, 2, 5] = 1.0
    assert not untouched(raw, shape, torch.bfloat16, 3, 8)
    raw, x = marked((2, 5, 4), torch.float32, 3)
    raw.view(torch.float32).view(4, 5, 7)[2, 1, 4] = 0.0
    assert not untouched(raw, (4, 5, 7), torch.float32, 3, 4)


@pytest.mark.parametrize("B", [40, 2600])
@pytest.mark.parametrize("borders", range(len(BORDERS)))
def test_page_bookkeeping_with_borders_out_of_order(borders, B):
    N, page, max_len = 3, 4, 90
    s = State([30 + b % 31 for b in range(B)], N, page, max_len, None, seed=borders, wide=1)
    lens, free, count = ints(s.cached), s.f.clone(), s.c.clone()
    s.g = ints(BORDERS[borders](B)), ints([60, 2 ** 31 - 1])
    T = 2 * B
    x = s.reserve([2] * B, T)
    # what the groups have no say in: lengths, ranges, positions, requests, the stacks
    assert x["query_start"].tolist() == list(range(0, 2 * B + 1, 2)) and x["seq_lens"].tolist() == (lens + 2).tolist()
    assert x["requests"].tolist() == [t // 2 for t in range(T)]
    assert x["positions"].tolist() == [s.cached[t // 2] + t % 2 for t in range(T)]
    assert torch.equal(s.f, free) and torch.equal(s.c, count) and x["missing"].tolist() == [0] * N
    assert (x["slots"] >= -1).all() and (x["slots"] < N * s.num_pages * page).all()
    assert (s.buf[:, B:] == -7).all() and (s.buf[:, :, s.mp:] == -7).all()
    table, out, left = s.buf.clone(), ints([-3] * N), ints([-3] * B)
    beside = s.f.as_strided((N, 2), (s.num_pages + 2, 1), s.num_pages).clone()
    binding.page_release(x["seq_lens"], ints([0] * B), max_len, s.num_pages, page, s.t, s.f, x["free_count"], out,
                         lens_out=left, group_start=s.g[0], prefix_lens=s.g[1])
    assert left.tolist() == [0] * B and torch.equal(table, s.buf)
    assert (out >= x["free_count"]).all() and (out <= s.num_pages).all()
    assert torch.equal(beside, s.f.as_strided((N, 2), (s.num_pages + 2, 1), s.num_pages))
