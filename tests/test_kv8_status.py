"""Calls on the 8-bit cache without a status word: what the device finds wrong is not lost."""
import pytest
import torch

from mla_decode_attention_03_gb300 import ops
from tests._kv8_reference import make_cache, make_pages
from tests.test_kv8_decode import SCALE, inputs

gpu = pytest.mark.gpu


def write(slots, cache, scales):
    x = torch.ones((len(slots), 576), dtype=torch.bfloat16, device="cuda")
    ops.write_cache_fp8(x[:, :512], x[:, 512:].contiguous(), torch.tensor(slots, device="cuda"), cache, scales)


@gpu
def test_errors_without_a_word_are_seen_once():
    ops.check_status()
    cache, scales = ops.empty_cache_fp8(2)
    write([3, 500], cache, scales)
    with pytest.raises(ops.MLAError, match="BLOCK_ID"):
        ops.check_status()
    ops.check_status()
    bt = torch.tensor([[7]], dtype=torch.int32, device="cuda")
    ops.read_cache_fp8(cache, scales, bt, torch.tensor([0, 5], dtype=torch.int32, device="cuda"), 5)
    with pytest.raises(ops.MLAError, match="BLOCK_ID"):
        ops.check_status()
    q, cache, scales, bt, sl = inputs([100], 1, 16, seed=61)
    dec = ops.MLADecoderFP8(1, 1, 16).plan(sl)
    ops.mla_decode_fp8(q, cache, scales, bt + 50, sl, dec.metadata, dec.num_splits, SCALE)
    with pytest.raises(ops.MLAError, match="BLOCK_ID"):
        ops.check_status()
    ops.check_status(dec.status)
    ops.check_status()


@gpu
def test_other_streams_and_a_replayed_graph_report_too():
    ops.check_status()
    cache, scales = ops.empty_cache_fp8(2)
    x = torch.ones((1, 576), dtype=torch.bfloat16, device="cuda")
    k, slot = x[:, 512:].contiguous(), torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        write([-1, 128], cache, scales)
    with pytest.raises(ops.MLAError, match="BLOCK_ID"):
        ops.check_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.write_cache_fp8(x[:, :512], k, slot, cache, scales)
    graph.replay()
    ops.check_status()
    slot.fill_(1000)
    graph.replay()
    with pytest.raises(ops.MLAError, match="BLOCK_ID"):
        ops.check_status()
    slot.fill_(0)
    graph.replay()
    ops.check_status()


@gpu
def test_calls_without_a_word_allocate_nothing():
    cache, scales = make_cache(3, seed=62)
    bt, _ = make_pages([130], seed=62)
    x = torch.ones((2, 576), dtype=torch.bfloat16, device="cuda")
    k, slots = x[:, 512:].contiguous(), torch.tensor([1, 2], device="cuda")
    cu, out = torch.tensor([0, 130], dtype=torch.int32, device="cuda"), torch.empty((130, 576), dtype=torch.bfloat16, device="cuda")

    def calls():
        ops.write_cache_fp8(x[:, :512], k, slots, cache, scales)
        ops.read_cache_fp8(cache, scales, bt, cu, 130, out=out)

    calls()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    calls()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    ops.check_status()
