"""The chunk operators at the longest length they accept, 2^30 tokens, over page tables that repeat a few physical
pages: a new token's slot, its attention (whose log-sum-exp counts every repetition) and the weights it gives."""
import math

import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV, share

pytestmark = pytest.mark.gpu

PAGE, LONG = 65536, 1 << 30


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def table(N, pages):
    n = -(-(-(-LONG // N)) // PAGE)
    return (torch.arange(n, device=DEV) % pages).to(torch.int32).view(1, 1, n).repeat(N, 1, 1)


@pytest.mark.parametrize("N", [1, 3])
@pytest.mark.parametrize("n,L", [(1, LONG), (5, LONG), (2, LONG - 1)])
def test_append_at_the_end(N, n, L):
    H, Hkv, D, pages = 4, 2, 64, 3
    g = torch.Generator(device=DEV).manual_seed(N + n)
    k_pages, v_pages = (torch.zeros((N, pages, PAGE, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, k, v = (torch.randn((n, h, D), generator=g, device=DEV).to(torch.bfloat16) for h in (H, Hkv, Hkv))
    start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    bt = table(N, pages)
    out = torch.zeros_like(q)
    binding.qk_norm_rope_append(q, k, v, None, None, 0.0, None, None, k_pages, v_pages, bt, start, lens, LONG, out)
    torch.cuda.synchronize()
    want_k, want_v = torch.zeros_like(k_pages), torch.zeros_like(v_pages)
    for j in range(n):
        at = L - n + j
        r, i = at % N, at // N
        pg = int(bt[r, 0, i // PAGE])
        want_k[r, pg, i % PAGE], want_v[r, pg, i % PAGE] = k[j], v[j]
    assert torch.equal(out, q) and torch.equal(k_pages, want_k) and torch.equal(v_pages, want_v)


@pytest.mark.parametrize("N,D,causal", [(1, 64, True), (3, 128, True), (2, 64, False)])
def test_attention_and_weights(N, D, causal):
    H, pages, L = 4, 2, LONG
    g = torch.Generator(device=DEV).manual_seed(N + D)
    k, v = (torch.randn((N, pages, PAGE, 1, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, H, D), generator=g, device=DEV).to(torch.bfloat16)
    start = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    bt = table(N, pages)
    o = torch.empty((N, 1, H, D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((N, 1, H), device=DEV)
    binding.extend_attention_paged(q, k, v, bt, start, lens, L, o, lse, D ** -0.5, causal=causal)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    parts = []
    for r in range(N):
        m = share(L, r, N)
        times = torch.full((pages * PAGE,), m // (pages * PAGE), dtype=torch.float64, device=DEV)
        times[: m % (pages * PAGE)] += 1
        x = q[0].double() @ k[r, :, :, 0].reshape(-1, D).double().T * D ** -0.5 + times.log()
        z = torch.logsumexp(x, -1)
        p = (x - z[:, None]).exp()
        want = p @ v[r, :, :, 0].reshape(-1, D).double()
        mass = p @ v[r, :, :, 0].reshape(-1, D).double().abs()
        # the tiles of 128 tokens a CTA joins one after another (152 CTAs, two accumulators), each sum rounded or cut
        # to 2^-23; a thread's row sum takes 32 terms of a tile in each of four accumulators
        tiles = m / 128 / 152 / 2
        tol = (2.0 ** -8 + 2.0 ** -18 + tiles * 2.0 ** -23) * mass + 2.0 ** -8 * want.abs()
        assert bool(((o[r, 0].double() - want).abs() <= tol).all())
        assert bool(((lse[r, 0].double() - z).abs() <= 32 * tiles * 2.0 ** -24 + 2.0 ** -16).all())
        parts.append(z)
    if not causal:
        return
    merged = torch.logsumexp(torch.stack(parts), 0)
    acc = torch.zeros((N, 1, 1, -(-L // N)), device=DEV)
    binding.attention_weights_paged(q, k, bt, start, lens, L, merged.float().view(1, H), acc, D ** -0.5)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    for r in range(N):
        m = share(L, r, N)
        x = q[0].double() @ k[r, :, :, 0].reshape(-1, D).double().T * D ** -0.5
        w = (x - merged.float().double()[:, None]).exp().sum(0)
        # as in the other tests of the weights: scores and log-sum-exps below 32
        rel = 2.0 ** -14
        step = pages * PAGE
        for at in list(range(0, m, 64 * step)) + [m - m % step]:
            got = acc[r, 0, 0, at:min(at + step, m)].double()
            assert bool(((got - w[: got.numel()]).abs() <= rel * w[: got.numel()]).all()), (r, at)
