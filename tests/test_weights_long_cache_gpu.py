"""Accumulated weights over caches whose (tokens x heads of a group) pass 32 bits: the page table repeats a few
physical pages, so that the cache is long and its memory small."""
import math

import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


@pytest.mark.parametrize("H,D,n", [(48, 64, 1), (48, 128, 1), (48, 64, 3), (64, 64, 1)])
def test_tokens_times_heads_beyond_32_bits(H, D, n):
    page, phys = 65536, 3
    L = 2 ** 31 // H + 5000
    mp = -(-L // page)
    g = torch.Generator(device=DEV).manual_seed(H + D)
    k = torch.randn((1, phys, page, 1, D), generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn((n, H, D), generator=g, device=DEV).to(torch.bfloat16)
    table = (torch.arange(mp, device=DEV) % phys).to(torch.int32).view(1, 1, mp)
    start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    # log-sum-exps of the size of a row's: weights of about 1 / 2^10, and one row that adds nothing
    lse = torch.full((n, H), 10 * math.log(2.0), device=DEV)
    lse[0, 5] = math.inf
    acc = torch.zeros((1, 1, 1, L), device=DEV)
    binding.attention_weights_paged(q, k, table, start, lens, L, lse, acc, D ** -0.5)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    # the definition in 64 bits for one pass over the physical tokens, by new token
    s = torch.einsum("jhd,td->jht", q.double(), k[0].reshape(-1, D).double()) * D ** -0.5
    w = torch.where(lse.isfinite()[..., None], (s - lse.double()[..., None]).exp(), torch.zeros_like(s)).sum(1)
    want = w.sum(0)
    # a weight: the product's error (D / 8 + 4 roundings of the sum of magnitudes), 2^-22 of exponent and 2^-20 of
    # exponential and sums (as the other tests of the weights)
    mag = torch.einsum("jhd,td->jht", q.double().abs(), k[0].reshape(-1, D).double().abs()).amax().item() * D ** -0.5
    rel = 2 * mag * (D / 8 + 4) * 2.0 ** -24 + 2.0 ** -22 * (s.abs().max().item() + 8) + 2.0 ** -20 + n * H * 2.0 ** -24
    got = acc.view(-1)
    for at in range(0, L - n, phys * page):
        part = got[at:min(at + phys * page, L - n)].double()
        off = (part - want[: part.numel()]).abs() - rel * want[: part.numel()]
        assert off.max().item() <= 0, f"tokens from {at}: off by {off.max().item():.3e} beyond the bound"
    for j in range(n):      # the new tokens are seen by themselves and the later ones
        t = L - n + j
        x = w[j:, t % (phys * page)].sum().item()
        assert abs(got[t].item() - x) <= rel * x
