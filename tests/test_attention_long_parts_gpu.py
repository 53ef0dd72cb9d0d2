"""Chunk attention whose parts take longer than a bounded wait's second: warps that wait for a part, not for a tile,
count only the time in which nothing moves.  The page table repeats two physical pages."""
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


def test_a_part_of_more_than_a_second_is_no_timeout():
    # three new tokens of 64 heads a group over 2^30 tokens of 20 KV heads: 1.1 million tiles a CTA, most of whose
    # last ones are masked
    L, page, Hkv, D, T = 1 << 30, 65536, 20, 64, 3
    H = 64 * Hkv
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn((1, 2, page, Hkv, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((T, H, D), generator=g, device=DEV).to(torch.bfloat16)
    table = (torch.arange(L // page, device=DEV) % 2).to(torch.int32).view(1, 1, -1)
    start = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    o = torch.full((1, T, H, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((1, T, H), float("nan"), device=DEV)
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    binding.extend_attention_paged(q, k, v, table, start, lens, L, o, lse, D ** -0.5)
    t1.record()
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    assert bool(o.isfinite().all()) and bool(lse.isfinite().all())
    assert t0.elapsed_time(t1) > 1000, "too short to reach what is tested"
