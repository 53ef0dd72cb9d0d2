"""Random batches of the shared-prefix attention against 64 bits, pools beyond 4 GB,
and slots beyond 32 bits."""
import random

import pytest
import torch

import pages_ref as ref
from chunk_ref import DEV
from decode_context_attention_gb300 import binding, build
from test_prefix_attention_gpu import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def draw(seed):
    r = random.Random(seed)
    D = r.choice((64, 128, 256))
    Hkv = r.choice((1, 2, 3))
    H = Hkv * r.choice((1, 2, 4, 5, 8, 16, 40))
    N = r.choice((1, 2, 3, 5))
    page = r.choice((2, 8, 16, 64, 128))
    lens, groups = [], []
    for _ in range(r.randint(1, 3)):
        for _ in range(r.choice((0, 0, 1, 3))):                # loose ones
            n = r.randint(0, 5)
            lens.append((n, n + r.randint(0, 200)))
        size, prefix, q = r.choice((1, 2, 8, 20)), r.choice((0, 30, 200, 700, 1500, 1100 * N)), r.choice((1, 1, 4, 30))
        lo = len(lens)
        for _ in range(size):
            n = r.choice((0, 1, r.randint(1, q)))
            lens.append((n, n + prefix + r.choice((0, 1, r.randint(0, 300)))))
        groups.append((lo, len(lens), prefix))
    # one array of borders: a gap between groups is a group of nothing in common
    flat, at = [], 0
    for lo, hi, p in groups:
        if at < lo:
            flat.append((at, lo, 0))
        flat.append((lo, hi, p))
        at = hi
    return lens, flat, dict(H=H, Hkv=Hkv, D=D, N=N, page=page, pad=r.choice((0, 0, 2)), strided=r.random() < 0.3,
                            dtype=r.choice((torch.bfloat16, torch.float16)), seed=seed, qscale=r.choice((0.3, 1.0, 4.0)))


@pytest.mark.parametrize("seed", range(36))
def test_random_batches(seed):
    lens, groups, kw = draw(seed)
    bt = Shared(lens, groups, **kw)
    causal, base = seed % 5 != 0, "2" if seed % 3 == 0 else "e"
    o, lse = bt.run(causal=causal, base=base)
    bt.check(o, lse, causal=causal, base=base)


@pytest.mark.parametrize("D", [128, 256])
def test_pools_beyond_four_gigabytes(D):
    """The same batch in the last pages of pools of more than 2^31 elements."""
    small = Shared([(1 + b % 2, 2900 + 3 * b) for b in range(20)], [(0, 20, 2890)], N=2, D=D, H=4, Hkv=1)
    o, lse = small.run()
    n = small.k_pages.shape[1]
    pages = (1 << 31) // (small.page * D) + n + 3
    k, v = (torch.empty((2, pages, small.page, 1, D), dtype=small.dtype, device=DEV) for _ in range(2))
    k[:, -n:], v[:, -n:] = small.k_pages, small.v_pages
    small.k_pages, small.v_pages = k, v
    small.block_table += (small.block_table < n) * (pages - n)
    o1, lse1 = small.run()
    assert torch.equal(o, o1) and torch.equal(lse, lse1)


def test_slots_beyond_32_bits():
    N, B, page, pages, max_len = 3, 4, 64, 1 << 26, 1000
    cached, new = [0, 100, 999, 63], [200, 3, 1, 66]
    free = [[pages - 1 - 7 * i - r for i in range(40)] for r in range(N)]
    table = [[[5] * 6 for _ in range(B)] for _ in range(N)]
    want = ref.reserve(cached, new, max_len, 300, pages, page, table, free, [40] * N)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    t, slots = ints(table), torch.zeros(300, dtype=torch.int64, device=DEV)
    qs, sl, mi, left = ints([0] * (B + 1)), ints([0] * B), ints([0] * N), ints([0] * N)
    binding.page_reserve(ints(cached), ints(new), max_len, 300, pages, page, t, ints(free), ints([40] * N), left, mi, qs,
                         sl, slots=slots)
    n = want["query_start"][-1]
    assert slots[:n].tolist() == want["slots"] and max(want["slots"]) > 1 << 33
    assert t.tolist() == want["block_table"] and left.tolist() == want["free_count"]
