"""Measured cases of the 8-bit latent cache and the rotary positions beside it.

Four operators, each with its plain form (elementary torch operations in 32 bits, 64 for rotary angles):

  rope    rotary positions of query rows and of the shared key row, into the buffers the decode and the cache write read
  write   quantises new tokens' entries to e4m3 with one power-of-two scale per token and puts them into the paged cache
  read    gathers entries of ragged sequences back as contiguous bf16 rows
  decode  multi-head latent attention over the 8-bit paged cache, returning out and the log-sum-exp

`own` selects the framework's kernels.  A case is a dict of plain values; lengths, head counts and strides follow from
the case alone, values and page orders from the seed.
"""
import math

import torch

own = False

PAGE, LATENT, ROPE = 64, 512, 64
ENTRY = LATENT + ROPE
E4M3_MAX = 448.0
SOFTMAX_SCALE = ENTRY ** -0.5
GOLDEN = 0.6180339887498949


def listed():
    return [
        # one short conversation, 16 heads: a decode step where latency is all there is
        dict(name="decode_1x16", op="decode", b=1, s_q=1, h=16, lo=256, hi=256, stride=576),
        # a small batch of ragged contexts, 16 heads, padded entries: the cache's bytes count
        dict(name="decode_16x16", op="decode", b=16, s_q=1, h=16, lo=1024, hi=4096, stride=640),
        # a full serving batch, 128 heads: arithmetic and bytes both count
        dict(name="decode_128x128", op="decode", b=128, s_q=1, h=128, lo=4096, hi=4096, stride=576),
        # two drafted positions per sequence, causal, ragged, padded entries
        dict(name="decode_mtp_48x128", op="decode", b=48, s_q=2, h=128, lo=257, hi=7001, stride=640),
        # an odd head count, three positions, lengths from nothing up (some sequences empty)
        dict(name="decode_odd_37x20", op="decode", b=37, s_q=3, h=20, lo=0, hi=3001, stride=576),
        # the new tokens of one decode step
        dict(name="write_128", op="write", tokens=128, blocks=4096, stride=576),
        # a prefill chunk with padding tokens
        dict(name="write_16001", op="write", tokens=16001, blocks=2048, stride=640),
        # one short prefix read back
        dict(name="read_3x100", op="read", b=3, lo=1, hi=211, stride=576),
        # the contexts of a batch read back for a chunk of prefill
        dict(name="read_64x4096", op="read", b=64, lo=1900, hi=6300, stride=640),
        # one token of a 16-head model
        dict(name="rope_1x16", op="rope", tokens=1, h=16, interleaved=True, factor=1.0, far=4096, dtype="bfloat16"),
        # a decode step of 128 sequences, scaled for long contexts
        dict(name="rope_128x128", op="rope", tokens=128, h=128, interleaved=True, factor=40.0, far=163840, dtype="bfloat16"),
        # a prefill chunk, half layout, far positions
        dict(name="rope_8191x32", op="rope", tokens=8191, h=32, interleaved=False, factor=4.0, far=1000000, dtype="float16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "write", "read", "rope"])
    stride = rng.choice([576, 640])
    if op == "decode":
        h = rng.choice([1, 4, 8, 12, 16, 20, 32, 40, 64, 96, 128])
        s_q = rng.choice([1, 1, 1, 2, 3, 4])
        b = _log_int(rng, 1, 128)
        # at most the largest listed case's (token, row) pairs and tokens
        most = min(524288 // b, (524288 * 128) // (b * h * s_q), 16384)
        hi = _log_int(rng, 1, most)
        return dict(op=op, b=b, s_q=s_q, h=h, lo=rng.randint(0, hi), hi=hi, stride=stride)
    if op == "write":
        return dict(op=op, tokens=_log_int(rng, 1, 16001), blocks=rng.randint(300, 2048), stride=stride)
    if op == "read":
        b = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 6300)
        return dict(op=op, b=b, lo=rng.randint(0, hi), hi=hi, stride=stride)
    return dict(op=op, tokens=_log_int(rng, 1, 8191), h=rng.choice([1, 5, 8, 16, 32]), interleaved=rng.random() < 0.5,
                factor=rng.choice([1.0, 2.0, 8.0, 40.0]), far=_log_int(rng, 64, 1000000),
                dtype=rng.choice(["bfloat16", "float16", "float32"]))


def _lengths(case):
    """Sequence lengths, spread over [lo, hi], from the case alone."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int((hi - lo + 1) * ((i * GOLDEN + 0.5) % 1.0)) for i in range(case["b"])]


def _visible(case):
    """(token, query position) pairs that the attention of a decode case has."""
    return sum(max(0, L - case["s_q"] + 1 + j) for L in _lengths(case) for j in range(case["s_q"]))


def work(case):
    if case["op"] == "decode":
        tokens = sum(_lengths(case))
        rows = case["b"] * case["s_q"] * case["h"]
        return {"bytes": tokens * (ENTRY + 4) + rows * (2 * ENTRY + 2 * LATENT + 4),
                "flops": 2.0 * (ENTRY + LATENT) * case["h"] * _visible(case)}
    if case["op"] == "write":
        return {"bytes": case["tokens"] * (2 * ENTRY + 8 + ENTRY + 4), "flops": 2.0 * case["tokens"] * ENTRY}
    if case["op"] == "read":
        return {"bytes": sum(_lengths(case)) * (ENTRY + 4 + 2 * ENTRY), "flops": 1.0 * sum(_lengths(case)) * ENTRY}
    size = 4 if case["dtype"] == "float32" else 2
    rows = case["tokens"] * (case["h"] + 1)
    return {"bytes": rows * ROPE * 2 * size + case["tokens"] * 8, "flops": 3.0 * rows * ROPE}


# ---------------------------------------------------------------- the plain forms
def _split(x):
    """e4m3 codes and the power-of-two scale of each row of x (32 bits): the smallest 2^e with max|x| <= 448 * 2^e."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, -126)).clamp(min=-126)
    scale = ((e + 127) << 23).to(torch.int32).view(torch.float32)  # 2^e
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _plain_decode(s):
    b, s_q, h, _ = s["q"].shape
    pages = s["block_table"].long().clamp(min=0)
    k = s["cache"].view(torch.uint8)[pages][:, :, :, 0].view(torch.float8_e4m3fn).float()
    k = (k * s["scales"][pages][:, :, 0, :, None]).reshape(b, -1, ENTRY)
    q = s["q"].float().reshape(b, s_q * h, ENTRY)
    score = torch.matmul(q, k.transpose(1, 2)) * SOFTMAX_SCALE
    t = torch.arange(k.shape[1], device=k.device)
    j = torch.arange(s_q, device=k.device).repeat_interleave(h)
    end = s["seqlens"].long()[:, None] - (s_q - 1 - j)[None, :]
    hidden = t[None, None, :] >= end[:, :, None]
    score = score.masked_fill_(hidden, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, k[..., :LATENT]) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).reshape(b, s_q, h).transpose(1, 2)
    return {"out": out.reshape(b, s_q, h, LATENT).to(torch.bfloat16), "lse": lse.contiguous()}


def _plain_write(s):
    code, scale = _split(torch.cat([s["kv_c"], s["k_pe"]], -1).float())
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    at = s["slots"][keep]
    s["cache"].view(torch.uint8)[at // PAGE, at % PAGE, 0] = code[keep].view(torch.uint8)
    s["scales"][at // PAGE, 0, at % PAGE] = scale[keep]
    return {"cache": s["cache"], "scales": s["scales"]}


def _plain_read(s):
    row = torch.arange(s["total"], device=s["cu"].device)
    i = torch.searchsorted(s["cu"], row.to(torch.int32), right=True) - 1
    t = row - s["cu"][i]
    page = s["block_table"][i, t // PAGE].long()
    code = s["cache"].view(torch.uint8)[page, t % PAGE, 0].view(torch.float8_e4m3fn)
    return (code.float() * s["scales"][page, 0, t % PAGE, None]).to(torch.bfloat16)


def _plain_turn(x, angle, interleaved, gain):
    c, w = (torch.cos(angle) * gain).float(), (torch.sin(angle) * gain).float()
    x = x.float()
    if interleaved:
        u, v = x[..., 0::2], x[..., 1::2]
        return torch.stack([u * c - v * w, u * w + v * c], -1).flatten(-2)
    u, v = x.chunk(2, -1)
    return torch.cat([u * c - v * w, u * w + v * c], -1)


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["freq"][None, :]
    s["q_out"][..., LATENT:] = _plain_turn(s["q_pe"], angle[:, None], s["interleaved"], s["gain"]).to(s["q_pe"].dtype)
    s["k_out"].copy_(_plain_turn(s["k_pe"], angle, s["interleaved"], s["gain"]).to(s["k_pe"].dtype))
    return {"q": s["q_out"][..., LATENT:], "k": s["k_out"]}


# ---------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _entries(gen, n):
    """n entries as a model makes them: unit latent and rope values, each token at a level of its own."""
    level = torch.exp(0.3 * _randn(gen, n, 1))
    return (_randn(gen, n, ENTRY) * level).to(torch.bfloat16)


def _cache(gen, blocks, stride):
    """A filled cache: e4m3 [blocks, 64, 1, 576] (a view where entries are padded), scales fp32 [blocks, 1, 64]."""
    alloc = torch.zeros((blocks, PAGE, 1, stride), dtype=torch.uint8, device="cuda")
    scales = torch.empty((blocks, 1, PAGE), dtype=torch.float32, device="cuda")
    step = 1024
    for p in range(0, blocks, step):
        n = min(step, blocks - p)
        code, scale = _split(_entries(gen, n * PAGE).float())
        alloc[p:p + n, :, 0, :ENTRY] = code.view(torch.uint8).view(n, PAGE, ENTRY)
        scales[p:p + n, 0] = scale.view(n, PAGE)
    return alloc[..., :ENTRY].view(torch.float8_e4m3fn), scales


def _frequencies(case):
    """Radians per position of the 32 pairs, in 64 bits: low pairs as they are, high ones slowed by `factor`."""
    base, original, fast, slow = 10000.0, 4096, 32.0, 1.0
    i = torch.arange(ROPE // 2, dtype=torch.float64, device="cuda")
    freq = base ** (-2.0 * i / ROPE)
    if case["factor"] == 1.0:
        return freq, 1.0
    edge = [ROPE * math.log(original / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (fast, slow)]
    low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), ROPE - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return freq / case["factor"] * ramp + freq * (1 - ramp), 0.1 * math.log(case["factor"]) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op in ("decode", "read"):
        lengths = _lengths(case)
        pages = [(L + PAGE - 1) // PAGE for L in lengths]
        blocks = max(1, sum(pages))
        s["cache"], s["scales"] = _cache(gen, blocks, case["stride"])
        order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32).tolist()
        table, at = [], 0
        for n in pages:
            table.append(order[at:at + n] + [-1] * (max(max(pages), 1) - n))
            at += n
        s["block_table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
        s["seqlens"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if op == "decode":
        s["q"] = _randn(gen, case["b"], case["s_q"], case["h"], ENTRY).to(torch.bfloat16)
        if own:  # the schedule is made once per step and kept for all layers
            from mla_decode_attention_03_gb300 import ops
            s["decoder"] = ops.MLADecoderFP8(case["b"], case["s_q"], case["h"]).plan(s["seqlens"])
    elif op == "read":
        s["total"] = sum(lengths)
        s["cu"] = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    elif op == "write":
        n = case["tokens"]
        s["cache"], s["scales"] = _cache(gen, case["blocks"], case["stride"])
        new = _entries(gen, n)
        s["kv_c"], s["k_pe"] = new[:, :LATENT], new[:, LATENT:].contiguous()
        slots = torch.randperm(case["blocks"] * PAGE, generator=gen, device="cuda")[:n]
        skip = torch.rand(n, generator=gen, device="cuda") < 0.05  # padding tokens
        s["slots"] = torch.where(skip, torch.full_like(slots, -1), slots)
    elif op == "rope":
        n, h, dtype = case["tokens"], case["h"], getattr(torch, case["dtype"])
        # the query projection's rows hold 128 other values before the 64 that turn
        s["q_pe"] = _randn(gen, n, h, 128 + ROPE).to(dtype)[..., 128:]
        s["k_pe"] = _randn(gen, n, ROPE).to(dtype)
        s["q_out"] = torch.zeros((n, h, ENTRY), dtype=dtype, device="cuda")
        s["k_out"] = torch.zeros((n, ROPE), dtype=dtype, device="cuda")
        s["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device="cuda")
        s["freq"], s["gain"] = _frequencies(case)
        s["interleaved"] = case["interleaved"]
        if own:  # the frequencies belong to the model
            from mla_decode_attention_03_gb300 import ops
            s["rotary"] = ops.Rotary(ROPE, base=10000.0, interleaved=case["interleaved"], factor=case["factor"],
                                     original_length=4096, gain=s["gain"])
    return s


def _own(s):
    from mla_decode_attention_03_gb300 import ops
    if s["op"] == "decode":
        out, lse = s["decoder"](s["q"], s["cache"], s["scales"], s["block_table"], s["seqlens"], SOFTMAX_SCALE,
                                causal=s["q"].shape[1] > 1)
        return {"out": out, "lse": lse}
    if s["op"] == "write":
        ops.write_cache_fp8(s["kv_c"], s["k_pe"], s["slots"], s["cache"], s["scales"])
        return {"cache": s["cache"], "scales": s["scales"]}
    if s["op"] == "read":
        return ops.read_cache_fp8(s["cache"], s["scales"], s["block_table"], s["cu"], s["total"])
    q, k = ops.rope(s["q_pe"], s["positions"], s["rotary"], out=s["q_out"][..., LATENT:], k=s["k_pe"], k_out=s["k_out"])
    return {"q": q, "k": k}


def run(s):
    if own:
        return _own(s)
    return {"decode": _plain_decode, "write": _plain_write, "read": _plain_read, "rope": _plain_rope}[s["op"]](s)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "decode":
        b, s_q, h, _ = s["q"].shape
        out = torch.zeros((b, s_q, h, LATENT), dtype=f64, device="cuda")
        lse = torch.full((b, h, s_q), -math.inf, dtype=f64, device="cuda")
        for i, L in enumerate(_lengths(case)):
            ids = s["block_table"][i, :(L + PAGE - 1) // PAGE].long()
            values = s["cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).to(f64)[:, :, 0]
            k = (values * s["scales"][ids, 0].to(f64)[..., None]).reshape(-1, ENTRY)[:L]
            for j in range(s_q):
                n = L - s_q + 1 + j
                if n > 0:
                    w = torch.einsum("hd,td->ht", s["q"][i, j].to(f64), k[:n]) * SOFTMAX_SCALE
                    lse[i, :, j] = torch.logsumexp(w, 1)
                    out[i, j] = torch.einsum("ht,td->hd", torch.exp(w - lse[i, :, j, None]), k[:n, :LATENT])
        return {"out": out, "lse": lse}
    if case["op"] == "write":
        x = torch.cat([s["kv_c"].to(f64), s["k_pe"].to(f64)], 1)
        top, scale = x.abs().max(1).values, torch.full((len(x),), 2.0 ** -126, dtype=f64, device="cuda")
        for _ in range(254):
            scale = torch.where(top > E4M3_MAX * scale, 2 * scale, scale)
        v = x / scale[:, None]
        step = torch.full_like(v, 2.0 ** -9)
        for e in range(-5, 9):
            step = torch.where(v.abs() >= 2.0 ** e, 2.0 ** (e - 3), step)
        v = torch.round(v / step) * step
        cache, scales = s["cache"].to(f64).reshape(-1, ENTRY), s["scales"].to(f64).reshape(-1)
        kept = torch.nonzero(s["slots"] >= 0).flatten()
        cache[s["slots"][kept]] = v[kept]
        scales[s["slots"][kept]] = scale[kept]
        return {"cache": cache.reshape(s["cache"].shape), "scales": scales.reshape(s["scales"].shape)}
    if case["op"] == "read":
        rows = []
        for i, L in enumerate(_lengths(case)):
            ids = s["block_table"][i, :(L + PAGE - 1) // PAGE].long()
            values = s["cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).to(f64)[:, :, 0]
            rows.append((values * s["scales"][ids, 0].to(f64)[..., None]).reshape(-1, ENTRY)[:L])
        return torch.cat(rows)
    turn = torch.polar(torch.full((case["tokens"], ROPE // 2), s["gain"], dtype=f64, device="cuda"),
                       torch.outer(s["positions"].to(f64), s["freq"]))

    def turned(x, z):
        x = x.to(f64)
        pairs = x.unflatten(-1, (-1, 2)) if case["interleaved"] else x.unflatten(-1, (2, -1)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        return (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2)

    return {"q": turned(s["q_pe"], turn[:, None]), "k": turned(s["k_pe"], turn)}
