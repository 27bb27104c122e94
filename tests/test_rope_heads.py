"""Rotary positions of tensors without heads beside ones that have some."""
import pytest
import torch

from mla_decode_attention_03_gb300 import ops

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("heads,k_heads", [(0, 1), (0, 3), (2, 0), (0, 0)])
def test_no_heads_on_one_side(heads, k_heads):
    rotary, pos = ops.Rotary(64), torch.arange(5, device="cuda") * 7
    gen = torch.Generator().manual_seed(1)
    x, k = (torch.randn((5, h, 64), generator=gen).cuda() for h in (heads, k_heads))
    out, k_out = torch.full_like(x, 9.0), torch.full_like(k, 9.0)
    got = ops.rope(x, pos, rotary, out=out, k=k, k_out=k_out)
    assert got[0] is out and got[1] is k_out
    if heads:
        assert torch.equal(out, ops.rope(x, pos, rotary))
    if k_heads:
        assert torch.equal(k_out, ops.rope(k, pos, rotary))
