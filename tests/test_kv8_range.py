"""Decode over the 8-bit cache where scales are zero, hidden, or anywhere in the type's range, against the definition in
64 bits.  The bounds are those of _kv8_reference."""
import math

import pytest
import torch

from mla_decode_attention_03_gb300 import ops
from tests._kv8_reference import ENTRY, attention
from tests.test_kv8_decode import SCALE, decode, held, inputs

gpu = pytest.mark.gpu


def at(bt, i, t):
    """(page, 0, slot) of token t of sequence i in the scales."""
    return int(bt[i, t // 64]), 0, t % 64


@gpu
@pytest.mark.parametrize("h_q,s_q", [(16, 2), (10, 3), (40, 2), (96, 3), (128, 2)])
@pytest.mark.parametrize("parts", [None, 1, 40])
def test_hidden_scales_of_any_value(h_q, s_q, parts):
    """Whatever scale the last tokens have, the queries that do not see them keep their results, bit for bit."""
    lens = [300, 63, 1, 2, 129, 190, 65, 128, 700]
    q, cache, scales, bt, sl = inputs(lens, s_q, h_q, seed=50)
    first = decode(q, cache, scales, bt, sl, causal=True, parts=parts)
    held(*first, attention(q, cache, scales, bt, sl, SCALE, True))
    for value in (0.0, -0.0, 2.0 ** -149, 2.0 ** -126, 3e38, math.nan, math.inf):
        hidden = scales.clone()
        for i, L in enumerate(lens):
            hidden[at(bt, i, L - 1)] = value
        out, lse = decode(q, cache, hidden, bt, sl, causal=True, parts=parts)
        assert torch.equal(out[:, :-1], first[0][:, :-1]) and torch.equal(lse[..., :-1], first[1][..., :-1]), value
        if value < 1:  # the last query sees a key of (almost) zero
            held(out, lse, attention(q, cache, hidden, bt, sl, SCALE, True))


@gpu
@pytest.mark.parametrize("h_q", [16, 64, 128])
def test_a_nan_with_a_scale_of_zero_is_seen(h_q):
    q, cache, scales, bt, sl = inputs([300, 64, 129], 2, h_q, seed=51)
    first = decode(q, cache, scales, bt, sl, causal=True)
    for i, L in enumerate((300, 64, 129)):
        scales[at(bt, i, L - 1)] = 0.0
        cache.view(torch.uint8)[int(bt[i, (L - 1) // 64]), (L - 1) % 64, 0, 575] = 0x7F
    out, lse = decode(q, cache, scales, bt, sl, causal=True)
    assert torch.equal(out[:, 0], first[0][:, 0]) and torch.equal(lse[..., 0], first[1][..., 0])
    assert torch.isnan(out[:, 1]).all() and torch.isnan(lse[..., 1]).all()


@gpu
@pytest.mark.parametrize("h_q", [16, 40, 128])
@pytest.mark.parametrize("s_q", [2, 3, 70])
def test_few_tokens_at_the_far_end_of_the_range(h_q, s_q):
    """Lengths where no token, or none of a piece, is seen by every query: one scale decides for those that see it."""
    if s_q == 70 and h_q != 16:
        pytest.skip("one shape of many positions is enough")
    q0, cache, scales0, bt, sl = inputs([1, 2, 65, 129, 200, 3, 64], s_q, h_q, seed=53)
    for power in (-60, 60, 92, 110):
        q = (q0.float() * 2.0 ** -power).to(torch.bfloat16)
        x = (q, cache, scales0 * 2.0 ** power, bt, sl)
        ref = attention(*x, SCALE, True)
        for parts in (None, 1, 4, 60):
            held(*decode(*x, causal=True, parts=parts), ref)


@gpu
@pytest.mark.parametrize("h_q,s_q", [(16, 1), (40, 1), (128, 1), (20, 3), (96, 2)])
@pytest.mark.parametrize("kind", ["scale 0", "written zeros", "scale 2^-70"])
def test_first_tokens_of_next_to_nothing(h_q, s_q, kind):
    """Tokens whose entries are zero or next to it count in the softmax like any others, and those after them too, whatever
    their scales."""
    lens = [256, 300, 700, 1000, 129, 128, 5]
    gone = 190
    q0, cache, scales0, bt, sl = inputs(lens, s_q, h_q, seed=52)
    codes = cache.view(torch.uint8)
    for i, L in enumerate(lens):
        for t in range(min(L, gone)):
            scales0[at(bt, i, t)] = {"scale 0": 0.0, "written zeros": 2.0 ** -126, "scale 2^-70": 2.0 ** -70}[kind]
            if kind == "written zeros":
                codes[int(bt[i, t // 64]), t % 64] = 0
    for power in (0, 4, 20, 46, 60, 100):
        scales = torch.where(scales0 > 2.0 ** -60, scales0 * 2.0 ** power, scales0)
        for level in (1.0, 6.0):  # of the scores
            q = (q0.float() * (level * 2.0 ** -power)).to(torch.bfloat16)
            x = (q, cache, scales, bt, sl)
            ref = attention(*x, SCALE, s_q > 1)
            for parts in (None, 1, 5):
                held(*decode(*x, causal=s_q > 1, parts=parts), ref)


@gpu
@pytest.mark.parametrize("h_q,s_q", [(128, 512), (4, 16384)])
def test_more_rows_than_a_grid_dimension(h_q, s_q):
    """65536 rows a sequence, in two pieces: the merge takes them."""
    x = inputs([200], s_q, h_q, seed=57)
    out, lse = decode(*x, parts=2, causal=False)
    some = [0, 1, s_q // 2, s_q - 1]
    ref = attention(x[0][:, some], *x[1:], SCALE, False)
    held(out[:, some], lse[..., some], ref)


@gpu
@pytest.mark.parametrize("h_q", [16, 64, 128])
def test_infinite_scale_makes_a_row_nan(h_q):
    lens = [64, 700, 129]
    q, cache, scales, bt, sl = inputs(lens, 2, h_q, seed=56)
    for parts in (1, 9):
        first = decode(q, cache, scales, bt, sl, causal=True, parts=parts)
        for t_of in (lambda L: L - 1, lambda L: 0):
            bad = scales.clone()
            for i, L in enumerate(lens):
                bad[at(bt, i, t_of(L))] = math.inf
            out, lse = decode(q, cache, bad, bt, sl, causal=True, parts=parts)
            assert torch.isnan(out[:, 1]).all() and torch.isnan(lse[..., 1]).all()
            if t_of(64):
                assert torch.equal(out[:, 0], first[0][:, 0]) and torch.equal(lse[..., 0], first[1][..., 0])
            else:
                assert torch.isnan(out).all() and torch.isnan(lse).all()


@gpu
@pytest.mark.parametrize("h_q", [16, 40, 128])
@pytest.mark.parametrize("power", [-112, 118])
def test_scores_of_large_and_small_factors(h_q, power):
    """Entries near the ends of bf16's range and queries at the other end: the scores are ordinary."""
    q, cache, scales, bt, sl = inputs([300, 70, 1], 1, h_q, seed=55)
    x = ((q.float() * 2.0 ** -power).to(torch.bfloat16), cache, scales * 2.0 ** power, bt, sl)
    held(*decode(*x), attention(*x, SCALE, False))


@gpu
@pytest.mark.parametrize("h_q", [16, 40, 128])
def test_smallest_entries_keep_their_bits(h_q):
    """Entries of the smallest scale, 2^-126: the outputs are held relative to themselves, down to bf16's smallest step."""
    q, cache, scales, bt, sl = inputs([700, 3, 20000], 1, h_q, seed=54)
    scales.fill_(2.0 ** -126)
    cache.view(torch.uint8)[..., :512] &= 0x7F  # of one sign, so that the outputs are as large as their parts
    x = (q, cache, scales, bt, sl)
    o, l, ob, lb = attention(*x, SCALE, False)
    for parts in (None, 1):
        out, lse = decode(*x, parts=parts)
        held(out, lse, (o, l, ob - 1e-30 + 2.0 ** -133, lb))


@gpu
@pytest.mark.parametrize("h_q,s_q", [(16, 3), (4, 5), (33, 3), (128, 3)])
@pytest.mark.parametrize("kind", ["scale 0", "written zeros", "scale 2^-70"])
def test_last_tokens_after_next_to_nothing(h_q, s_q, kind):
    """Entries next to nothing but for the last ones, which only some queries see: each query has what it sees, and keeps
    it, bit for bit, whatever the last one's scale is."""
    lens = [129, 65, 128, 130, 193, 3, 64, 66]
    q0, cache, scales0, bt, sl = inputs(lens, s_q, h_q, seed=63)
    codes = cache.view(torch.uint8)
    for i, L in enumerate(lens):
        for t in range(max(0, L - s_q + 1)):
            scales0[at(bt, i, t)] = {"scale 0": 0.0, "written zeros": 2.0 ** -126, "scale 2^-70": 2.0 ** -70}[kind]
            if kind == "written zeros":
                codes[int(bt[i, t // 64]), t % 64] = 0
    for power in (0, -40, 30, 70):
        scales = torch.where(scales0 > 2.0 ** -60, scales0 * 2.0 ** power, scales0)
        for level in (1.0, 8.0):
            q = (q0.float() * (level * 2.0 ** -power)).to(torch.bfloat16)
            ref = attention(q, cache, scales, bt, sl, SCALE, True)
            for parts in (None, 1, 2):
                out, lse = decode(q, cache, scales, bt, sl, causal=True, parts=parts)
                held(out, lse, ref)
                for value in (0.0, 1.0, 3e38, math.nan):
                    hidden = scales.clone()
                    for i, L in enumerate(lens):
                        hidden[at(bt, i, L - 1)] = value
                    got = decode(q, cache, hidden, bt, sl, causal=True, parts=parts)
                    assert torch.equal(got[0][:, :-1], out[:, :-1]) and torch.equal(got[1][..., :-1], lse[..., :-1]), value


@gpu
@pytest.mark.parametrize("h_q,s_q", [(16, 3), (33, 5), (128, 2)])
def test_hidden_scales_beside_small_ones(h_q, s_q):
    """Sequences of small entries: a hidden token's scale, as large as it may be, leaves the others' bits alone."""
    lens = [128, 300, 129, 65, 1, 5]
    q, cache, scales, bt, sl = inputs(lens, s_q, h_q, seed=64)
    for power in (-100, -60, -30):
        x = ((q.float() * 2.0 ** -power).to(torch.bfloat16), cache, scales * 2.0 ** power, bt, sl)
        ref = attention(*x, SCALE, True)
        for parts in (None, 1, 20):
            out, lse = decode(*x, causal=True, parts=parts)
            # (the reference's floor of 1e-30 is above these outputs; rows that see nothing have none)
            held(out, lse, (ref[0], ref[1], (ref[2] - 1e-30).clamp(min=0) + 2.0 ** -133, ref[3]))
            for value in (0.0, 1.0, 3e38):
                hidden = x[2].clone()
                for i, L in enumerate(lens):
                    hidden[at(bt, i, L - 1)] = value
                got = decode(x[0], cache, hidden, bt, sl, causal=True, parts=parts)
                assert torch.equal(got[0][:, :-1], out[:, :-1]) and torch.equal(got[1][..., :-1], lse[..., :-1]), value
