"""A prompt's chunk in front of single tokens without number: the requests that the chunk kernel has nothing to do for
are passed soon enough for its waits, and every row is written."""
import pytest
import torch

from decode_context_attention_gb300 import binding, build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


@pytest.mark.parametrize("B,wide", [(100, [0]), (4000, [0, 31, 32, 33, 64, 3999]), (4200000, [0]), (4200000, [0, 4199999])])
def test_chunks_among_single_tokens(B, wide):
    H, Hkv, D, page, L, n = 1, 1, 64, 8, 12, 300
    g = torch.Generator(device=DEV).manual_seed(B)
    new = torch.ones(B, dtype=torch.int64, device=DEV)
    new[wide] = n
    query_start = torch.cat([new.new_zeros(1), new.cumsum(0)]).int()
    lens = torch.randint(1, L + 1, (B,), generator=g, device=DEV).int()
    lens[wide] = n + 70
    T, max_len = int(query_start[-1]), n + 70
    mp, pages = -(-max_len // page), 997
    table = torch.randint(0, pages, (1, B, 2), generator=g, device=DEV, dtype=torch.int32)
    rows = torch.full((1, B, mp), 2 ** 30, dtype=torch.int32, device=DEV)      # entries behind a request's tokens
    rows[:, :, :2] = table
    rows[:, wide] = torch.randint(0, pages, (1, len(wide), mp), generator=g, device=DEV, dtype=torch.int32)
    k, v = (torch.empty((1, pages, page, Hkv, D), device=DEV).uniform_(-1, 1, generator=g).to(torch.bfloat16)
            for _ in range(2))
    q = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    groups = torch.tensor([0, B], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = torch.full((1, T, H, D), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((1, T, H), 99.0, device=DEV)
    binding.prefix_attention_paged(q, k, v, rows, query_start, lens, max_len, *groups, o, lse, D ** -0.5)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    # single tokens in 64 bits, some hundred thousand at a time
    single = (new == 1).nonzero()[:, 0]
    for some in single.split(200000):
        i = torch.arange(2 * page, device=DEV)
        pg = table[0, some].long().repeat_interleave(page, 1)
        kk, vv = (x[0, pg, i % page, 0].double() for x in (k, v))
        t = query_start[some].long()
        x = torch.einsum("bhd,bld->bhl", q[t].double(), kk) * D ** -0.5
        x = torch.where(i < lens[some, None, None], x, -torch.inf)
        z = torch.logsumexp(x, -1)
        want = torch.einsum("bhl,bld->bhd", (x - z[..., None]).exp(), vv)
        # |v| <= 1 and the weights' sum is 1: P's and the output's rounding, 2^-9 for the 32-bit scores and exponentials
        assert (lse[0, t].double() - z).abs().max() <= 2.0 ** -16
        assert (o[0, t].double() - want).abs().max() <= 2 * 2.0 ** -8 + 2.0 ** -9
        del kk, vv, x, want
    for b in wide:
        i = torch.arange(max_len, device=DEV)
        pg = rows[0, b].long()[i // page]
        kk, vv = (x[0, pg, i % page, 0].double() for x in (k, v))
        t = slice(int(query_start[b]), int(query_start[b + 1]))
        x = torch.einsum("thd,ld->htl", q[t].double(), kk) * D ** -0.5
        x = torch.where(i[None] <= max_len - n + torch.arange(n, device=DEV)[:, None], x, -torch.inf)
        z = torch.logsumexp(x, -1)
        want = torch.einsum("htl,ld->thd", (x - z[..., None]).exp(), vv)
        assert (lse[0, t].double() - z.T).abs().max() <= 2.0 ** -16
        assert (o[0, t].double() - want).abs().max() <= 2 * 2.0 ** -8 + 2.0 ** -9
