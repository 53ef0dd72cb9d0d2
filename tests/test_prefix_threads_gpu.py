"""Attention behind common prefixes from several host threads at once, whose calls give the last kernel different
amounts of shared memory: no call may take from another's what its launch needs.  (What one thread's opt-in took from
another's launch was met once in some thousand calls: hence their number.)"""
import threading

import pytest
import torch

from decode_context_attention_gb300 import binding, build
from test_prefix_attention_gpu import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_calls_of_few_and_of_many_blocks(D):
    # four warps an item, so 8 and 36 blocks; two warps an item, so 312 and 400 of them: on both sides of two an SM
    batches = [Shared([(1, 40 + b % 9) for b in range(n)], [(0, n, 32)], D=D, H=4, Hkv=2, seed=n)
               for n in (2, 9, 156, 200)]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert 9 * 4 <= 2 * sms < 156 * 4 // 2 and 200 * 4 < 6 * sms
    outs = [bt.outputs() for bt in batches]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(batches))

    def work(bt, out):
        try:
            stream = torch.cuda.Stream()
            call = binding.prepare_prefix_attention_paged(
                bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens, bt.max_len, bt.group_start,
                bt.prefix_lens, *out, bt.scale, stream=stream)
            start.wait()
            for _ in range(1500):
                for _ in range(20):
                    call()
                stream.synchronize()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(batches, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    for bt, out in zip(batches, outs):
        bt.check(*out)
