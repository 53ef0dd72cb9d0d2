"""Prepared calls of the chunk-serving operators: run again and again on changed inputs they give what the direct call
gives; a workspace that they allocate stays theirs; two graphs of prepared calls follow their own workspaces."""
import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def batch(D=128, seed=3):
    return Batch([(5, 700), (60, 300), (1, 2500)], 2, 8, 2, D, 16, torch.bfloat16, 1, seed=seed)


def churn():
    """What the allocator would hand out of freed memory meanwhile."""
    for n in (1 << 16, 1 << 22, 64 << 20, 256 << 20):
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)


def attention_args(bt, o, lse):
    return (bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens, bt.max_len, o, lse, bt.scale)


@pytest.mark.parametrize("D", [128, 64, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_attention(D, causal):
    bt = batch(D)
    o, o2 = (torch.zeros((2, bt.T, 8, D), dtype=bt.dtype, device=DEV) for _ in range(2))
    lse, lse2 = (torch.zeros((2, bt.T, 8), device=DEV) for _ in range(2))
    call = binding.prepare_extend_attention_paged(*attention_args(bt, o, lse), base="2", causal=causal)
    for step in range(3):
        churn()
        bt.q.copy_(torch.randn(bt.q.shape, generator=bt.g, device=DEV))
        bt.seq_lens[0] = 700 - 31 * step
        call()
        binding.extend_attention_paged(*attention_args(bt, o2, lse2), base="2", causal=causal)
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_weights_append_and_eviction():
    bt = batch()
    acc = torch.zeros((2, bt.B, 2, bt.cap), device=DEV)
    lse = torch.randn((bt.T, 8), generator=bt.g, device=DEV) + 6
    k, v = (torch.randn((bt.T, 2, bt.D), generator=bt.g, device=DEV).to(bt.dtype) for _ in range(2))
    w = torch.ones(bt.D, dtype=bt.dtype, device=DEV)
    out = torch.zeros_like(bt.q)
    rows = 300 // 2
    kp = -(-rows // bt.page)
    grown = [torch.zeros((2, bt.num_pages + bt.B * kp, *t.shape[2:]), dtype=bt.dtype, device=DEV)
             for t in (bt.k_pages, bt.v_pages)]
    for t, was in zip(grown, (bt.k_pages, bt.v_pages)):
        t[:, :bt.num_pages] = was.nan_to_num(0.0)
    dst = (torch.arange(bt.B * kp, dtype=torch.int32, device=DEV) + bt.num_pages).view(1, bt.B, kp).repeat(2, 1, 1)
    keep = torch.full((bt.B,), 300, dtype=torch.int32, device=DEV)
    kept = torch.full((2, bt.B, 2, rows), -1, dtype=torch.int32, device=DEV)
    acc_out = torch.zeros((2, bt.B, 2, rows), device=DEV)
    common = (bt.block_table, bt.query_start, bt.seq_lens, bt.max_len)
    append = (bt.q, k, v, w, w, 1e-6, None, None, *grown, *common, out)
    add = (bt.q, grown[0], *common, lse, acc, bt.scale)
    evict = (*grown, bt.block_table, bt.seq_lens, bt.max_len, acc, keep, 300, 20, dst, kept, acc_out)
    prepared = (binding.prepare_qk_norm_rope_append(*append), binding.prepare_attention_weights_paged(*add),
                binding.prepare_cache_evict_paged(*evict))
    direct = (lambda: binding.qk_norm_rope_append(*append), lambda: binding.attention_weights_paged(*add),
              lambda: binding.cache_evict_paged(*evict))
    state = (*grown, out, acc, kept, acc_out)
    for _ in range(2):
        churn()
        bt.q.copy_(torch.randn(bt.q.shape, generator=bt.g, device=DEV))
        k.copy_(torch.randn(k.shape, generator=bt.g, device=DEV))
        before = [t.clone() for t in state]
        results = []
        for calls in (prepared, direct):
            for t, was in zip(state, before):
                t.copy_(was)
            for call in calls:
                call()
            torch.cuda.synchronize()
            results.append([t.clone() for t in state])
        assert binding.device_status() == 0
        for a, b, was in zip(*results, before):
            assert torch.equal(a, b)
        assert not torch.equal(results[0][3], before[3]) and bool((kept >= 0).any())


def test_two_graphs_of_prepared_calls_replayed_together():
    bts = [batch(seed=4), batch(seed=5)]
    outs, graphs, calls = [], [], []
    for bt in bts:
        o, lse = torch.zeros((2, bt.T, 8, 128), dtype=bt.dtype, device=DEV), torch.zeros((2, bt.T, 8), device=DEV)
        binding.extend_attention_paged(*attention_args(bt, o, lse))
        torch.cuda.synchronize()
        outs.append((o, lse, o.clone(), lse.clone()))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            # prepared on the capturing stream: each call keeps a workspace of its own
            calls.append(binding.prepare_extend_attention_paged(*attention_args(bt, o, lse)))
            calls[-1]()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for o, lse, _, _ in outs:
        o.fill_(7.0)
        lse.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    n = bts[0].start[-1]
    for o, lse, o2, lse2 in outs:
        assert torch.equal(o[:, :n], o2[:, :n]) and torch.equal(lse[:, :n], lse2[:, :n])


def test_a_prepared_call_on_another_stream():
    bt = batch()
    s = torch.cuda.Stream()
    o, lse = torch.zeros((2, bt.T, 8, 128), dtype=bt.dtype, device=DEV), torch.zeros((2, bt.T, 8), device=DEV)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    torch.cuda.synchronize()
    call = binding.prepare_extend_attention_paged(*attention_args(bt, o, lse), stream=s)
    binding.extend_attention_paged(*attention_args(bt, o2, lse2))
    for _ in range(3):
        call()
        churn()
    del call        # the workspace goes back while the stream may still run
    churn()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
