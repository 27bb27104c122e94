"""A decode over the 8-bit cache reads what the calls before it on its stream have written: the schedule, the lengths, the
page table, the cache and its scales, the queries."""
import pytest
import torch

from mla_decode_attention_03_gb300 import ops
from tests._kv8_reference import ENTRY, make_cache, make_pages

gpu = pytest.mark.gpu
SCALE = ENTRY ** -0.5


@gpu
@pytest.mark.parametrize("h_q,s_q,b", [(16, 1, 3), (48, 1, 3), (128, 1, 3), (128, 2, 3), (128, 1, 120)])
def test_steps_without_a_pause_read_what_came_before(h_q, s_q, b):
    """Steps that each rewrite every input, enqueued without a pause, against the same steps one at a time."""
    longest, steps = 700, 12
    gen = torch.Generator().manual_seed(31)
    lens = [torch.randint(1, longest, (b,), generator=gen, dtype=torch.int32).cuda() for _ in range(steps)]
    bt0, nb = make_pages([longest] * b, seed=30)
    caches = [make_cache(nb, seed=40 + i, device="cuda") for i in range(2)]
    tables = [bt0, bt0.flip(0).contiguous()]
    queries = [torch.randn((b, s_q, h_q, ENTRY), generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    cache, scales, bt, sl, q = (torch.empty_like(t) for t in (caches[0][0].view(torch.uint8), caches[0][1], bt0, lens[0], queries[0]))
    dec = ops.MLADecoderFP8(b, s_q, h_q)
    # inputs that no earlier step left behind
    cache.fill_(0x7F), scales.fill_(1.0), bt.zero_(), sl.fill_(1), q.zero_()
    dec.plan(sl)(q, cache.view(torch.float8_e4m3fn), scales, bt, sl, SCALE)

    def run(pause):
        got = []
        for i in range(steps):
            cache.copy_(caches[i & 1][0].view(torch.uint8))
            scales.copy_(caches[i & 1][1])
            bt.copy_(tables[(i >> 1) & 1])
            q.copy_(queries[(i >> 2) & 1])
            sl.copy_(lens[i])
            if pause:
                torch.cuda.synchronize()
            dec.plan(sl)
            if pause:
                torch.cuda.synchronize()
            got.append(dec(q, cache.view(torch.float8_e4m3fn), scales, bt, sl, SCALE, causal=s_q > 1))
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        ops.check_status(dec.status)
        return got

    for a, c in zip(run(False), run(True)):
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
        assert torch.isfinite(a[0]).all()
