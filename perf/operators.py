"""Cases and plain forms of the operators that serve a decoder beside its 4-bit weights: writing and reading a paged
key/value cache held in 4 bits, attention over that cache, and the linear layer in 8-bit integers.

`own = False` computes each operator from its formula with elementary torch operations; `own = True` makes the calls of
this repository's package.

The cache.  A page holds `page` tokens of each kv head.  A token's head vector x of D elements is cut into blocks of B;
per block mn = min(0, min x), mx = max(0, max x), s = f16((mx - mn) / 15), z = clamp(rint(-mn / s), 0, 15) and
q = clamp(rint(x / s) + z, 0, 15) (binary32 divisions; all codes 0 where s = 0), and x^ = s (q - z).  Codes:
uint8 [pages, heads, page, D / 2], as D / 8 words of 8 codes each (low nibble first); word i * (D / B) + j holds elements
8 i .. 8 i + 7 of block j.  Block states: binary16 [pages, heads, page, D / B, 2], the pair (s, z).
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the new tokens of a decode step: one for each of 16 sequences, grouped-query heads of a 70B-class layer
        dict(name="write_step", op="write", dtype="bf16", tokens=16, heads=8, dim=128, block=64, page=64),
        # a prompt's keys and values, the 32 heads of a 7B-class layer, an odd number of tokens
        dict(name="write_prompt", op="write", dtype="f16", tokens=8191, heads=32, dim=128, block=128, page=16),
        # one user's next token after a short dialogue, 7B-class layer
        dict(name="attend_short", op="attend", dtype="f16", batch=1, rows="one", new=1, longest=777, q_heads=32, heads=32,
             dim=128, block=128, page=16, causal=True, window=0),
        # a step of a batch of 16 dialogues of unequal lengths, grouped-query heads
        dict(name="attend_batch", op="attend", dtype="bf16", batch=16, rows="one", new=1, longest=8192, q_heads=64, heads=8,
             dim=128, block=64, page=64, causal=True, window=0),
        # one token over a long document
        dict(name="attend_document", op="attend", dtype="bf16", batch=1, rows="one", new=1, longest=131071, q_heads=64, heads=8,
             dim=128, block=64, page=256, causal=True, window=0),
        # five drafted tokens of each of 24 sequences, looked at together; heads of a 135M-class layer, a sliding window
        dict(name="attend_draft", op="attend", dtype="f16", batch=24, rows="same", new=5, longest=4000, q_heads=9, heads=3,
             dim=64, block=64, page=32, causal=True, window=1500),
        # a chunk of a long prompt behind what the cache already holds
        dict(name="attend_chunk", op="attend", dtype="bf16", batch=1, rows="same", new=2048, longest=8192, q_heads=64, heads=8,
             dim=128, block=64, page=64, causal=True, window=0),
        # several whole prompts of unequal lengths, the small model's heads
        dict(name="attend_prompts", op="attend", dtype="f16", batch=6, rows="whole", new=1500, longest=1500, q_heads=9, heads=3,
             dim=64, block=64, page=16, causal=True, window=0),
        # the linear layer: one token through a square projection
        dict(name="linear_token", op="linear", dtype="f16", m=1, n=4096, k=4096, bias=False),
        # a decode batch through an up projection
        dict(name="linear_batch", op="linear", dtype="bf16", m=24, n=11008, k=4096, bias=False),
        # a short prompt through the small model's up projection, with a bias and an odd number of rows
        dict(name="linear_small", op="linear", dtype="f16", m=331, n=1536, k=576, bias=True),
        # a prompt through a gate projection of a 70B-class layer
        dict(name="linear_prompt", op="linear", dtype="bf16", m=4096, n=28672, k=8192, bias=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "attend", "attend", "attend", "linear", "linear"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "linear":
        m = _log(rng, 1, 4096)
        k = _log(rng, 64, 11008)
        n = _log(rng, 64, 28672)
        return dict(op=op, dtype=dtype, m=m, n=n, k=k, bias=rng.random() < 0.4)
    dim = rng.choice([64, 128])
    block = rng.choice([64, dim])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "write":
        heads = rng.choice([1, 3, 8, 32])
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, 8192), heads=heads, dim=dim, block=block, page=page)
    q_heads, heads = rng.choice([(32, 32), (64, 8), (9, 3), (8, 1), (16, 4), (40, 40), (12, 2)])
    rows = rng.choice(["one", "one", "same", "whole"])
    window = rng.choice([0, 0, 0, _log(rng, 1, 4000)])
    if rows == "one":
        batch, new = _log(rng, 1, 64), 1
        longest = _log(rng, 1, min(65536, 131071 // batch))
    elif rows == "same":
        batch, new = _log(rng, 1, 16), _log(rng, 2, 512)
        longest = _log(rng, max(new, 16), 8192)
        batch = max(1, min(batch, 16384 * 4096 // (new * longest * 4)))
    else:
        batch, longest = _log(rng, 1, 8), _log(rng, 17, 2000)
        new = longest
    return dict(op=op, dtype=dtype, batch=batch, rows=rows, new=new, longest=longest, q_heads=q_heads, heads=heads, dim=dim,
                block=block, page=page, causal=rng.random() < 0.9, window=window)


def lengths(case):
    """(new rows, length with them) of each sequence: the longest first, the others anywhere below it."""
    r = random.Random(case["longest"] * 64 + case["batch"])
    got = []
    for b in range(case["batch"]):
        n = case["longest"] if b == 0 else r.randint(max(1, case["longest"] // 8), case["longest"])
        got.append((n if case["rows"] == "whole" else min(case["new"], n), n))
    return got


def _pairs(case):
    """Attended (row, key) pairs and the keys that any row attends to, over all sequences."""
    pairs = keys = 0
    w = case["window"]
    for n, length in lengths(case):
        p0 = length - n
        if not case["causal"]:
            if w:
                first = [max(0, p - w + 1) for p in range(p0, length)]
                pairs += sum(length - f for f in first)
                keys += length - first[0]
            else:
                pairs += n * length
                keys += length
        else:
            pairs += sum(min(p + 1, w) if w else p + 1 for p in range(p0, length))
            keys += length - (max(0, p0 - w + 1) if w else 0)
    return pairs, keys


def work(case):
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return dict(bytes=2 * m * k + n * k + 4 * n + 2 * n * case["bias"] + 2 * m * n, flops=2 * m * n * k)
    per = case["dim"] + 8 * case["dim"] // case["block"]  # bytes of one token's K and V in one head
    if case["op"] == "write":  # written and read back: 16 bits in, the cache, 16 bits out
        t = case["tokens"] * case["heads"]
        return dict(bytes=t * (8 * case["dim"] + 2 * per) + 16 * case["tokens"], flops=12 * t * case["dim"])
    pairs, keys = _pairs(case)
    rows = sum(n for n, _ in lengths(case))
    return dict(bytes=keys * case["heads"] * per + rows * case["q_heads"] * (4 * case["dim"] + 4) + 4 * keys // case["page"],
                flops=4 * case["dim"] * case["q_heads"] * pairs)


# ------------------------------------------------------------------------------------------------ plain forms

def _div(a, b):
    """The binary32 quotient, 0 where the divisor is."""
    return torch.where(b == 0, torch.zeros_like(a), a / torch.where(b == 0, torch.ones_like(b), b))


def _quantize(x, block):
    """x [..., D] -> codes (int32) [..., D/B, B], s, z (float32) [..., D/B, 1]."""
    v = x.float().unflatten(-1, (-1, block))
    mn, mx = v.amin(-1, keepdim=True).clamp(max=0), v.amax(-1, keepdim=True).clamp(min=0)
    s = ((mx - mn) / torch.full_like(mx, 15)).half().float()
    z = _div(-mn, s).round().clamp(0, 15)
    q = torch.where(s == 0, torch.zeros_like(v), (_div(v, s.expand_as(v)).round() + z).clamp(0, 15))
    return q.to(torch.int32), s, z


def _pack(q):
    """codes [..., D/B, B] -> bytes [..., D/2] in the cache's order of words."""
    w = q.unflatten(-1, (-1, 4, 2)).transpose(-4, -3)  # [..., B/8, D/B, 4 bytes, 2]
    return (w[..., 0] + 16 * w[..., 1]).flatten(-3).to(torch.uint8)


def _unpack(codes, state):
    """bytes [..., D/2] and states [..., D/B, 2] -> values (float32) [..., D]."""
    nb = state.shape[-2]
    w = codes.unflatten(-1, (-1, nb, 4)).transpose(-3, -2)  # [..., D/B, B/8, 4 bytes]
    q = torch.stack([w & 15, w >> 4], -1).flatten(-3).float()
    return ((q - state[..., 1:].float()) * state[..., :1].float()).flatten(-2)


def _write(s):
    got = []
    for x, codes, state in ((s["k"], s["k_codes"], s["k_state"]), (s["v"], s["v_codes"], s["v_state"])):
        q, sc, z = _quantize(x, s["block"])
        page, off = s["slots"] // codes.shape[2], s["slots"] % codes.shape[2]
        codes[page, :, off] = _pack(q)
        state[page, :, off] = torch.cat([sc, z], -1).half()
        got.append(_unpack(codes[page, :, off], state[page, :, off]).to(x.dtype))
    return got


def _attend(s):
    q, lens, starts = s["q"].float(), s["lens"].long(), s["starts"].long()
    batch, heads, dim = lens.numel(), s["k_codes"].shape[1], q.shape[-1]
    page = s["k_codes"].shape[2]
    longest, new = s["longest"], s["new"]
    dev = q.device
    n = starts[1:] - starts[:-1]
    # the keys and values of every sequence, padded to the longest
    j = torch.arange(longest, device=dev)
    there = j[None] < lens[:, None]  # [batch, longest]
    at = s["table"].long()[:, : (longest + page - 1) // page].clamp(min=0).repeat_interleave(page, 1)[:, :longest]
    k = _unpack(s["k_codes"][at, :, j % page], s["k_state"][at, :, j % page]).permute(0, 2, 3, 1)  # [batch, heads, dim, longest]
    x_rows = torch.arange(new, device=dev)
    row = (starts[:-1, None] + x_rows[None]).clamp(max=q.shape[0] - 1)  # [batch, new]
    real = x_rows[None] < n[:, None]
    qp = q[row].unflatten(2, (heads, -1)).permute(0, 2, 3, 1, 4)  # [batch, heads, group, new, dim]
    x = torch.matmul(qp.flatten(2, 3), k).unflatten(2, (-1, new)) * s["scale"]
    del k
    pos = (lens - n)[:, None] + x_rows[None]  # [batch, new]
    seen = there[:, None, :] & real[:, :, None]
    if s["causal"]:
        seen &= j[None, None] <= pos[:, :, None]
    if s["window"]:
        seen &= j[None, None] > pos[:, :, None] - s["window"]
    seen = seen[:, None, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    v = _unpack(s["v_codes"][at, :, j % page], s["v_state"][at, :, j % page]).permute(0, 2, 1, 3)
    v = torch.where(there[:, None, :, None], v, 0.0)
    o = torch.matmul(x.flatten(2, 3), v).unflatten(2, (-1, new)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total))[..., 0]  # [batch, heads, group, new]
    out = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[real]
    return [out.to(s["q"].dtype), lse.permute(0, 3, 1, 2).flatten(2)[real]]


def _linear(s):
    x = s["x"].float()
    top = x.abs().amax(-1, keepdim=True)
    sa = top / torch.full_like(top, 127)
    q = _div(x, sa.expand_as(x)).round()
    # sums of up to K products of 7-bit integers: binary64 holds them exactly
    acc = torch.matmul(q.double(), s["w"].double().t())
    y = acc.float() * (sa * s["ws"][None])
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


# ------------------------------------------------------------------------------------------------ prepare and run

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _kv(shape, g, dtype):
    """Keys or values: Gaussian, some channels of a head larger and some away from zero, as projections give them."""
    d = shape[-1]
    size = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    off = torch.randn(d, generator=g, device="cuda") * (torch.rand(d, generator=g, device="cuda") < 0.1)
    return (torch.randn(*shape, generator=g, device="cuda") * size + off).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    dtype = DT[case["dtype"]]
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        x = torch.randn(m, k, generator=g, device="cuda") * torch.exp(0.7 * torch.randn(k, generator=g, device="cuda"))
        w = torch.randn(n, k, generator=g, device="cuda").mul_(0.02)
        top = w.abs().amax(-1, keepdim=True)
        ws = top / torch.full_like(top, 127)
        bias = torch.randn(n, generator=g, device="cuda").to(dtype) if case["bias"] else None
        # a weight's rows begin at multiples of 16 bytes
        codes = torch.zeros(n, (k + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :k]
        codes.copy_(w.div_(ws).round_())
        return dict(op="linear", x=x.to(dtype), w=codes, ws=ws[:, 0].contiguous(), bias=bias)
    heads, dim, block, page = case["heads"], case["dim"], case["block"], case["page"]
    if case["op"] == "write":
        t = case["tokens"]
        pages = (t + page - 1) // page + 3
        empty = torch.zeros(pages, heads, page, dim // 2, dtype=torch.uint8, device="cuda")
        state = torch.zeros(pages, heads, page, dim // block, 2, dtype=torch.float16, device="cuda")
        return dict(op="write", block=block, k=_kv((t, heads, dim), g, dtype), v=_kv((t, heads, dim), g, dtype),
                    slots=torch.randperm(pages * page, generator=g, device="cuda")[:t].contiguous(),
                    k_codes=empty, v_codes=empty.clone(), k_state=state, v_state=state.clone())
    both = lengths(case)
    need = [(length + page - 1) // page for _, length in both]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(both), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    s = dict(op="attend", block=block, table=table, causal=case["causal"], window=case["window"], scale=1.0 / math.sqrt(dim),
             longest=case["longest"], new=max(n for n, _ in both))
    for name in "kv":
        q, sc, z = _quantize(_kv((pages, heads, page, dim), g, dtype), block)
        s[name + "_codes"], s[name + "_state"] = _pack(q), torch.cat([sc, z], -1).half()
    rows = sum(n for n, _ in both)
    s["q"] = torch.randn(rows, case["q_heads"], dim, generator=g, device="cuda").to(dtype)
    s["lens"] = torch.tensor([n for _, n in both], dtype=torch.int32, device="cuda")
    starts = [0]
    for n, _ in both:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    return s


def _cache(s):
    """The handle of the cache, which a program makes once and keeps."""
    from bit_blockwise_weight_absmax_b200 import q4
    if "cache" not in s:
        s["cache"] = q4.KVCache(s["k_codes"], s["k_state"], s["v_codes"], s["v_state"])
    return s["cache"]


def run(state):
    s = state
    if own:
        from bit_blockwise_weight_absmax_b200 import q4
        if s["op"] == "write":
            q4.kv_append(_cache(s), s["k"], s["v"], s["slots"])
            return q4.kv_dequantize(_cache(s), s["slots"], s["k"].dtype)
        if s["op"] == "attend":
            return q4.kv_attention(s["q"], _cache(s), s["table"], s["lens"], s["starts"], max_q=s["new"], scale=s["scale"],
                                   causal=s["causal"], window=s["window"], return_lse=True)
        return q4.int8_linear(s["x"], s["w"], s["ws"], s["bias"])
    return {"write": _write, "attend": _attend, "linear": _linear}[s["op"]](s)


# ------------------------------------------------------------------------------------------------ in 64 bits

def _values(codes, state, d):
    """The binary64 values of cached vectors, element by element: element e of block j is nibble e % 8 of word
    (e // 8) * blocks + j."""
    nb = state.shape[-2]
    e = torch.arange(d, device=codes.device)
    j, i = e // (d // nb), e % (d // nb)
    byte = ((i // 8) * nb + j) * 4 + (i % 8) // 2
    q = (codes[..., byte].to(torch.int64) >> (4 * (i % 2))) % 16
    return state[..., j, 0].double() * (q.double() - state[..., j, 1].double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x = s["x"].double()
        # the stored scale is a binary32 number, and a code is the rint of a binary32 quotient
        sa = (x.abs().max(1).values / 127.0).float().double()
        q = (x / sa.clamp(min=1e-300)[:, None]).float().round().double()
        y = torch.einsum("mk,nk->mn", q, s["w"].double()) * sa[:, None] * s["ws"].double()[None]
        return y if s["bias"] is None else y + s["bias"].double()
    d = case["dim"]
    if case["op"] == "write":
        got = []
        for x in (s["k"], s["v"]):
            b = x.double().reshape(-1, case["block"])
            lo, hi = torch.clamp(b.min(1).values, max=0), torch.clamp(b.max(1).values, min=0)
            sc = ((hi - lo).float().double() / 15.0).float().half().double()
            safe = torch.where(sc > 0, sc, 1.0)
            z = torch.clamp((-lo / safe).float().round(), 0, 15).double()
            q = torch.clamp((b / safe[:, None]).float().round().double() + z[:, None], 0, 15)
            got.append((sc[:, None] * (q - z[:, None])).reshape(x.shape))
        return got
    page, group = case["page"], case["q_heads"] // case["heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, length) in enumerate(lengths(case)):
        pages = s["table"][b, : (length + page - 1) // page].long()
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None]
        hidden = torch.zeros(n, length, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= j > pos
        if case["window"]:
            hidden |= j <= pos - case["window"]
        for h in range(case["heads"]):
            k = _values(s["k_codes"][pages, h], s["k_state"][pages, h], d).reshape(-1, d)[:length]
            v = _values(s["v_codes"][pages, h], s["v_state"][pages, h], d).reshape(-1, d)[:length]
            for hq in range(h * group, (h + 1) * group):
                x = (s["q"][row:row + n, hq].double() @ k.t() * s["scale"]).masked_fill_(hidden, -math.inf)
                lse[row:row + n, hq] = torch.logsumexp(x, 1)
                out[row:row + n, hq] = torch.exp(x - lse[row:row + n, hq, None]).nan_to_num_(0.0) @ v
        row += n
    return [out, lse]
