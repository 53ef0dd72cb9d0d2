"""Evictions whose blocks have more keys than shared memory holds (they are read again in every pass): one request in
a cluster of eight blocks, and many heads with a block each."""
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


def pick(a, keep, recent):
    """Kept indices of one head, in order: the latest, then by weight, ties to the lower index, NaN last."""
    n = a.numel()
    older = n - min(recent, n)
    want = max(keep - (n - older), 0)
    x = a[:older].double()
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
    by = x.sort(descending=True, stable=True).indices
    # a stable sort of "is not a number" puts those behind everything else, -inf among it
    by = by[a[:older][by].isnan().int().sort(stable=True).indices]
    late = torch.arange(n - min(keep, n - older), n, device=a.device)
    return torch.cat([by[:want].sort().values, late])


def weights(kind, shape, g):
    if kind == "random":
        return torch.empty(shape, device=DEV).exponential_(1.0, generator=g)
    if kind == "ties":
        return torch.randint(0, 3, shape, generator=g, device=DEV).float()
    x = torch.randn(shape, generator=g, device=DEV)
    x[..., 5::9] = math.nan
    x[..., 7::31] = -math.inf
    return x


@pytest.mark.parametrize("kind", ["random", "ties", "nan"])
@pytest.mark.parametrize("B,Hkv,L,keep,recent", [
    (1, 1, 400_003, 100_001, 77),       # eight blocks of 50,001 keys
    (1, 2, 700_000, 699_990, 0),        # all but ten are kept
    (20, 8, 44_000, 3000, 512),         # 160 heads, a block each
])
def test_slices_beyond_shared_memory(B, Hkv, L, keep, recent, kind):
    D, page = 8, 256
    g = torch.Generator(device=DEV).manual_seed(L)
    mp, kp = -(-L // page), -(-keep // page)
    pages = B * (mp + kp)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table, dst = perm[: B * mp].view(1, B, mp), perm[B * mp:].view(1, B, kp)
    k, v = (torch.randn((1, pages, page, Hkv, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    acc = weights(kind, (1, B, Hkv, L), g)
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    keeps = torch.full((B,), keep, dtype=torch.int32, device=DEV)
    kept = torch.full((1, B, Hkv, keep), -1, dtype=torch.int32, device=DEV)
    out = torch.zeros((1, B, Hkv, keep), device=DEV)
    binding.cache_evict_paged(k, v, table, lens, L, acc, keeps, keep, recent, dst, kept, out)
    torch.cuda.synchronize()
    n = torch.arange(keep, device=DEV)
    for b in range(B):
        for h in range(Hkv):
            ids = pick(acc[0, b, h], keep, recent)
            assert torch.equal(kept[0, b, h].long(), ids)
            assert torch.equal(out[0, b, h].view(torch.int32), acc[0, b, h, ids].view(torch.int32))
            for pool, was in ((k, k0), (v, v0)):
                got = pool[0, dst[0, b].long()[n // page], n % page, h]
                want = was[0, table[0, b].long()[ids // page], ids % page, h]
                assert torch.equal(got, want)
