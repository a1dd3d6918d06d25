"""The operators of the 8-bit block-scaled KV cache, as cases that can be timed and compared.

Four operators:

norm_rope   tq_qk_norm_rope: per-head RMS norm of queries and keys with the
            position rotation in the same pass
write       tq_cache8_write: new keys and values quantised into their blocks,
            one power-of-two scale for each block of tokens and head
read        tq_cache8_read: tokens of a paged cache back as bf16 or fp32 rows
attend      tq_cache8_attention: attention of the newest queries over the cache

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits; where it is true, it calls the framework.
"""
import math

import torch

own = False

E_MIN = -100                                    # smallest exponent of a block's scale
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One decode step of a batch of 8, heads of the Llama-3.1-8B shape, q and k slices of a fused projection.
        dict(name="norm_rope_step", op="norm_rope", tokens=8, hq=32, hkv=8, d=128, rot=128, dtype="bf16", norm=True,
             base=500000.0),
        # A prompt batch of 16384 tokens of the same shape.
        dict(name="norm_rope_prompt", op="norm_rope", tokens=16384, hq=32, hkv=8, d=128, rot=128, dtype="bf16",
             norm=True, base=500000.0),
        # A protein of 1021 residues, ESM-2-650M heads in fp32: an odd number of tokens, half of each head turned.
        dict(name="norm_rope_odd", op="norm_rope", tokens=1021, hq=20, hkv=20, d=64, rot=32, dtype="f32", norm=True,
             base=10000.0),
        # A decode step's tokens written: 64 sequences of ragged length, one token each.
        dict(name="write_step", op="write", batch=64, new=1, start=2048, hkv=8, d=128, block=64, code="e4m3",
             dtype="bf16"),
        # Eight prompts of ragged length written at once behind a short prefix that ends inside a block.
        dict(name="write_prompt", op="write", batch=8, new=8192, start=40, hkv=8, d=128, block=64, code="e4m3",
             dtype="bf16"),
        # One cached sequence of 1000 tokens read back in fp32 (int8 codes, small pages, d = 64).
        dict(name="read_one", op="read", batch=1, new=1000, start=0, hkv=20, d=64, block=16, code="int8", dtype="f32"),
        # Eight cached prefixes read back to bf16, as for a dense kernel or another host.
        dict(name="read_prompt", op="read", batch=8, new=8192, start=0, hkv=8, d=128, block=64, code="e4m3",
             dtype="bf16"),
        # One token of one short chat: the smallest step, where latency counts.
        dict(name="attend_short", op="attend", batch=1, nq=1, len=777, ragged=False, window=0, hq=32, hkv=8, d=128,
             block=64, code="e4m3", dtype="bf16"),
        # The Llama-3.1-8B decode step of the benchmark: batch 8, context 32768.
        dict(name="attend_step", op="attend", batch=8, nq=1, len=32768, ragged=False, window=0, hq=32, hkv=8, d=128,
             block=64, code="e4m3", dtype="bf16"),
        # The benchmark's long context of 131072 tokens, one sequence, int8 codes.
        dict(name="attend_long", op="attend", batch=1, nq=1, len=131072, ragged=False, window=0, hq=32, hkv=8, d=128,
             block=128, code="int8", dtype="bf16"),
        # Four drafted tokens of 32 ragged sequences, every head its own keys (ESM heads), fp32, a sliding window.
        dict(name="attend_draft", op="attend", batch=32, nq=4, len=8192, ragged=True, window=4096, hq=20, hkv=20, d=64,
             block=16, code="int8", dtype="f32"),
        # A chunk of 1024 prompt tokens of two sequences over the cache they extend.
        dict(name="attend_chunk", op="attend", batch=2, nq=1024, len=8192, ragged=False, window=0, hq=32, hkv=8, d=128,
             block=64, code="e4m3", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv = rng.choice([(32, 8), (20, 20), (16, 2), (8, 1), (28, 4), (12, 12), (24, 8)])
    d = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["norm_rope", "write", "read", "attend", "attend", "attend"])
    if op == "norm_rope":
        most = 16384 * 40 * 128 // ((hq + hkv) * d) // (2 if dtype == "f32" else 1)
        return dict(op=op, tokens=_log(rng, 1, most), hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2]), dtype=dtype,
                    norm=rng.random() < 0.8, base=rng.choice([10000.0, 500000.0]))
    block, code = rng.choice([16, 32, 64, 128]), rng.choice(["e4m3", "int8"])
    if op in ("write", "read"):
        most = 36000 * 8 * 128 // (hkv * d) // (2 if dtype == "f32" else 1)    # about what the listed prompts hold
        batch = _log(rng, 1, 128)
        return dict(op=op, batch=batch, new=rng.choice([1, _log(rng, 1, max(2, most // batch))]),
                    start=_log(rng, 1, 2048) - 1, hkv=hkv, d=d, block=block, code=code, dtype=dtype)
    batch = _log(rng, 1, 64)
    nq = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
    keys = 8 * 32768 * 8 * 128 // (hkv * d)                                     # the keys of attend_step
    if nq > 1:
        keys = min(keys, 2 * 32 * 1024 * 8192 * 128 // 2 // (hq * nq * d))      # half the products of attend_chunk
    batch = max(1, min(batch, keys // 64))
    length = _log(rng, 1, max(64, min(131072, keys // batch)))
    return dict(op=op, batch=batch, nq=nq, len=length, ragged=rng.random() < 0.6,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), hq=hq, hkv=hkv, d=d, block=block, code=code,
                dtype=dtype)


def _lengths(most, batch, ragged):
    """Lengths of a batch, spread over 1 .. most by the golden ratio (the first is the longest)."""
    if not ragged:
        return [most] * batch
    return [most] + [max(1, int(most * math.fmod(0.6180339887498949 * (b + 1), 1.0))) for b in range(1, batch)]


def _plan(case):
    """(tokens before, new tokens) of each sequence."""
    if case["op"] == "attend":
        n = _lengths(case["len"], case["batch"], case["ragged"])
        return [0] * len(n), n
    new = _lengths(case["new"], case["batch"], True)
    start = [s - 1 for s in _lengths(case["start"] + 1, case["batch"], True)][::-1]
    return start, new


def _spans(case):
    """Of each sequence: how many keys the rows of its queries see together, and how many query-key pairs there are."""
    nq, w, keys, pairs = case["nq"], case["window"], 0, 0
    for n in _plan(case)[1]:
        first = min(n, max(1, n - nq + 1))                                      # keys of the first row that sees any
        rows = n - first + 1
        if w and w < n:
            keys += n - max(0, first - w)
            full = rows - max(0, min(rows, w - first))                          # rows that see w keys
            part = rows - full
            pairs += full * w + part * first + part * (part - 1) // 2
        else:
            keys += n
            pairs += rows * (first + n) // 2
    return keys, pairs


def work(case):
    d = case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm_rope":
        rows = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": 2 * rows * d * size + 4 * case["tokens"] + 8 * d, "flops": 7 * rows * d}
    h = case["hkv"]
    if case["op"] in ("write", "read"):
        start, new = _plan(case)
        touched = sum(-(-(s % case["block"] + n) // case["block"]) for s, n in zip(start, new))
        return {"bytes": 2 * sum(new) * h * d * (size + 1) + 8 * touched * h, "flops": 4 * sum(new) * h * d}
    keys, pairs = _spans(case)
    rows = case["batch"] * case["hq"] * case["nq"]
    return {"bytes": 2 * keys * h * d + 8 * h * (keys // case["block"]) + rows * (2 * d * size + 4),
            "flops": 4 * pairs * case["hq"] * d}


# ---------------------------------------------------------------- inputs
def _values(shape, dtype, gen):
    """Normal values with a few channels of several times the others' size, as keys and values have them."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    loud = torch.exp(torch.randn(shape[-1], generator=gen, device="cuda")) * 4.0
    some = torch.rand(shape[-1], generator=gen, device="cuda") < 0.03
    return x.mul_(torch.where(some, loud, 1.0)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, d = DTYPES[case["dtype"]], case["d"]
    s = {"case": case}
    if case["op"] == "norm_rope":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        qkv = _values((t, hq + 2 * hkv, d), dtype, gen)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["qw"], s["kw"] = (1.0 + 0.2 * torch.randn((2, d), generator=gen, device="cuda")).unbind(0)
        if not case["norm"]:
            s["qw"] = s["kw"] = None
        s["pos"] = torch.randint(0, 131072, (t,), generator=gen, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty((t, hq, d), device="cuda", dtype=dtype)
        s["k_out"] = torch.empty((t, hkv, d), device="cuda", dtype=dtype)
        return s
    h, blk, batch = case["hkv"], case["block"], case["batch"]
    start, new = _plan(case)
    per = [-(-(a + n) // blk) for a, n in zip(start, new)]
    total = sum(per) + 3
    # Pages in random order; the slots of the table behind a sequence's last page hold -1.
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((batch, max(per)), -1, dtype=torch.int32)
    at = torch.tensor(per).cumsum(0) - torch.tensor(per)
    col = torch.arange(max(per))[None]
    here = col < torch.tensor(per)[:, None]
    table[here] = (at[:, None] + col)[here].to(torch.int32)
    table = table.cuda()
    s["table"] = torch.where(table >= 0, order[table.clamp(min=0).long()], -1).to(torch.int32)
    s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    n = sum(new)
    s["tokens"] = n
    for name in ("k", "v"):
        # The cache as earlier writes left it.
        codes = torch.empty((total, h, blk, d), dtype=torch.uint8, device="cuda")
        scale = torch.empty((total, h), dtype=torch.float32, device="cuda")
        step = max(1, (1 << 26) // (h * blk * d))
        for a in range(0, total, step):
            x = _values((min(step, total - a), h, blk, d), torch.float32, gen)
            if case["op"] != "attend":
                x.mul_(torch.exp2(torch.randint(-2, 1, (x.shape[0], h, 1, 1), generator=gen, device="cuda").float()))
            e = _exponent(x.abs().amax((2, 3)), case["code"])
            codes[a:a + step] = _codes(x * torch.exp2(-e)[..., None, None], case["code"])
            scale[a:a + step] = torch.exp2(e)
        s[name], s[name + "_scale"] = codes, scale
        if case["op"] == "write":
            s["new_" + name] = _values((n, h, d), dtype, gen)
        if case["op"] == "read":
            s[name + "_out"] = torch.empty((n, h, d), device="cuda", dtype=dtype)
    if case["op"] == "attend":
        q = _values((batch, case["nq"], case["hq"], d), torch.float32, gen)
        s["q"] = q.to(dtype).transpose(1, 2)                                    # [batch, hq, nq, d], token-major
        s["out"] = torch.empty((batch, case["nq"], case["hq"], d), device="cuda", dtype=dtype).transpose(1, 2)
        s["lse"] = torch.empty((batch, case["hq"], case["nq"]), device="cuda")
        s["lens"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        s["ws"] = None
    return s


# ---------------------------------------------------------------- plain forms
def _exponent(amax, code):
    """The smallest e with amax <= 448 * 2^e (e4m3) or 127 * 2^e (int8), at least E_MIN; as a float."""
    m, e = torch.frexp(amax)                                                    # amax = m 2^e, 1/2 <= m < 1
    top, bits = (0.875, 9) if code == "e4m3" else (127.0 / 128.0, 7)
    e = e - bits + (m > top).to(e.dtype)
    return torch.where(amax > 0, e, E_MIN).clamp(min=E_MIN).float()


def _codes(x, code):
    """Bytes of values already divided by their scale: nearest, ties to even."""
    return x.to(torch.float8_e4m3fn).view(torch.uint8) if code == "e4m3" else x.round().to(torch.int8).view(torch.uint8)


def _floats(codes, code):
    return codes.view(torch.float8_e4m3fn).float() if code == "e4m3" else codes.view(torch.int8).float()


def _stored(codes, code):
    """Codes as the numbers that they stand for."""
    return codes.view(torch.float8_e4m3fn if code == "e4m3" else torch.int8)


def _norm_rope(s, name, weight, base, rot):
    x = s[name].float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    angle = s["pos"].double()[:, None, None] * base ** (-2.0 * i / rot)         # far positions: fp64
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b, rest = x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
    s[name + "_out"].copy_(torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1))
    return s[name + "_out"]


def _slots(s, blk):
    """Page and row within it of each token of a ragged batch."""
    t = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], t, right=True) - 1
    pos = s["start"][seq] + t - s["cu"][seq]
    return s["table"][seq, (pos // blk).long()].long(), (pos % blk).long()


def _write(s, name, code, blk):
    codes, scale, x = s[name], s[name + "_scale"], s["new_" + name].float()
    page, row = _slots(s, blk)
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    need = torch.exp2(_exponent(amax, code))
    # Blocks that hold tokens already keep the larger scale; their codes follow it.
    filled = s["start"] % blk
    more = (s["cu"][1:] > s["cu"][:-1]) & (filled > 0)
    first = s["table"].gather(1, (s["start"] // blk).long().clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    first = first.clamp(min=0).long()
    held = torch.zeros(scale.shape[0], dtype=torch.int32, device="cuda").index_add_(0, first, more.int())
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    grown = torch.where(held[:, None] > 0, torch.maximum(scale, need), need)
    ratio = (scale / grown)[first][..., None, None]
    old = codes[first]
    keep = (torch.arange(blk, device="cuda") < filled[:, None]) & more[:, None]
    codes[first] = torch.where(keep[:, None, :, None], _codes(_floats(old, code) * ratio, code), old)
    codes[page, :, row] = _codes(x / grown[page][..., None], code)
    scale.copy_(torch.where(touched[:, None], grown, scale))


def _read(s, name, code, blk):
    page, row = _slots(s, blk)
    s[name + "_out"].copy_(_floats(s[name][page, :, row], code) * s[name + "_scale"][page][..., None])
    return s[name + "_out"]


def _gather(s, name, code):
    """[batch, hkv, tokens, d] in fp32."""
    page = s["table"].clamp(min=0).long()
    x = _floats(s[name][page], code) * s[name + "_scale"][page][..., None, None]
    b, n, h, blk, d = x.shape
    return x.transpose(1, 2).reshape(b, h, n * blk, d)


def _attend(s):
    c = s["case"]
    b, hq, nq, d = s["q"].shape
    h, g = c["hkv"], hq // c["hkv"]
    k = _gather(s, "k", c["code"])
    score = (s["q"].float().reshape(b, h, g * nq, d) @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    del k
    at = torch.arange(score.shape[-1], device="cuda", dtype=torch.int32)
    last = s["lens"][:, None] - nq + torch.arange(nq, device="cuda", dtype=torch.int32)      # a row's own position
    see = at <= last[..., None]
    if c["window"]:
        see &= at > last[..., None] - c["window"]
    score = score.view(b, h, g, nq, -1)
    score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _gather(s, "v", c["code"])
    out = (p.view(b, h, g * nq, -1) @ v).view(b, h, g, nq, d) / total.clamp(min=1e-30)
    s["out"].copy_(out.reshape(b, hq, nq, d))
    s["lse"].copy_((top + total.log()).reshape(b, hq, nq))
    return s["out"], s["lse"]


def _own(s):
    import kv_cache_vector_rope_b200 as tq
    c = s["case"]
    if c["op"] == "norm_rope":
        tq.tq_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                           positions=s["pos"], rope_base=c["base"], rot_dim=c["rot"])
        return s["q_out"], s["k_out"]
    cache = tq.Cache8(s["k"], s["v"], s["k_scale"], s["v_scale"], c["code"])
    if c["op"] == "write":
        tq.tq_cache8_write(cache, s["new_k"], s["new_v"], s["cu"], s["start"], block_table=s["table"])
        return _stored(s["k"], c["code"]), _stored(s["v"], c["code"]), s["k_scale"], s["v_scale"]
    if c["op"] == "read":
        tq.tq_cache8_read(cache, s["k_out"], s["v_out"], s["cu"], s["start"], block_table=s["table"])
        return s["k_out"], s["v_out"]
    if s["ws"] is None:
        s["ws"] = tq.cache8_attention_workspace(cache, *s["q"].shape[:3])
    tq.tq_cache8_attention(cache, s["q"], s["lens"], s["out"], s["ws"], block_table=s["table"], causal=True,
                           window=c["window"], lse_out=s["lse"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "norm_rope":
        return (_norm_rope(state, "q", state["qw"], c["base"], c["rot"]),
                _norm_rope(state, "k", state["kw"], c["base"], c["rot"]))
    if c["op"] == "write":
        _write(state, "k", c["code"], c["block"])
        _write(state, "v", c["code"], c["block"])
        return (_stored(state["k"], c["code"]), _stored(state["v"], c["code"]), state["k_scale"], state["v_scale"])
    if c["op"] == "read":
        return _read(state, "k", c["code"], c["block"]), _read(state, "v", c["code"], c["block"])
    return _attend(state)


# ---------------------------------------------------------------- 64 bits
def _e4m3_table():
    """The value of every e4m3 byte, from the format's definition (0x7f and 0xff are no numbers)."""
    size = [math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10) for e in range(16) for m in range(8)]
    size[127] = math.nan
    return torch.tensor(size + [-x for x in size], dtype=torch.float64, device="cuda")


def _exact_values(codes, code):
    if code == "int8":
        x = codes.double()
        return torch.where(x > 127, x - 256, x)
    return _e4m3_table()[codes.long()]


def _exact_round(x, code):
    """The code's value nearest to x (|x| in its range), ties to the even one."""
    if code == "int8":
        return torch.round(x)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_scale(amax, code):
    top = 448.0 if code == "e4m3" else 127.0
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -300) / top))
    e = torch.where(top * torch.exp2(e - 1) >= amax, e - 1, e)                  # log2 may miss a power by its rounding
    e = torch.where(top * torch.exp2(e) < amax, e + 1, e)
    return torch.exp2(e.clamp(min=E_MIN))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        rot, out = case["rot"], []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            freq = torch.exp(torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) * (-math.log(case["base"]) / rot))
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous())
            z = z * torch.exp(1j * (s["pos"].double()[:, None] * freq))[:, None]
            out.append(torch.cat([z.real, z.imag, x[..., rot:]], -1))
        return tuple(out)
    code, blk, h, d = case["code"], case["block"], case["hkv"], case["d"]
    start, new = _plan(case)
    table = s["table"].cpu().tolist()
    if case["op"] == "read":
        out = []
        for name in ("k", "v"):
            rows = []
            for b, (a, n) in enumerate(zip(start, new)):
                pages = torch.tensor(table[b][a // blk:-(-(a + n) // blk)], device="cuda")
                x = _exact_values(s[name][pages], code) * s[name + "_scale"].double()[pages][..., None, None]
                rows.append(x.permute(0, 2, 1, 3).reshape(-1, h, d)[a % blk:a % blk + n])
            out.append(torch.cat(rows))
        return tuple(out)
    if case["op"] == "write":
        values, scales = [], []
        for name in ("k", "v"):
            val = _exact_values(s[name], code)
            sc = s[name + "_scale"].double()
            at = 0
            for b, (a, n) in enumerate(zip(start, new)):
                x = s["new_" + name][at:at + n].double()
                at += n
                pages = torch.tensor(table[b][a // blk:-(-(a + n) // blk)], device="cuda")
                head, count = a % blk, len(pages)
                full = torch.zeros((count * blk, h, d), dtype=torch.float64, device="cuda")
                full[head:head + n] = x
                full = full.view(count, blk, h, d).transpose(1, 2)
                want = _exact_scale(full.abs().amax((2, 3)), code)
                if head:
                    want[0] = torch.maximum(want[0], sc[pages[0]])
                put = _exact_round(full / want[..., None, None], code)
                if head:
                    kept = val[pages[0], :, :head] * (sc[pages[0]] / want[0])[:, None, None]
                    put[0, :, :head] = _exact_round(kept, code)
                slot = torch.arange(count * blk, device="cuda").view(count, 1, blk, 1)
                val[pages] = torch.where(slot < head + n, put, val[pages])
                sc[pages] = want
            # The numbers that the codes hold, in the types that hold them.
            values.append(val.float().to(torch.float8_e4m3fn) if code == "e4m3" else val.to(torch.int8))
            scales.append(sc)
        return (*values, *scales)
    b, hq, nq, d = s["q"].shape
    g = hq // h
    outs = torch.zeros((b, hq, nq, d), dtype=torch.float64, device="cuda")
    lses = torch.full((b, hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    if b * h > 4000:
        return None
    for i in range(b):
        n = new[i]
        pages = torch.tensor(table[i][:-(-n // blk)], device="cuda")
        first = max(0, nq - n)                                                  # rows before it see nothing
        where = torch.arange(n, device="cuda")
        own_at = n - nq + torch.arange(first, nq, device="cuda")
        see = where[None] <= own_at[:, None]
        if case["window"]:
            see &= where[None] > own_at[:, None] - case["window"]
        for j in range(h):
            k, v = (_exact_values(s[m][pages, j], code) * s[m + "_scale"][pages, j].double()[:, None, None]
                    for m in ("k", "v"))
            k, v = k.reshape(-1, d)[:n], v.reshape(-1, d)[:n]
            for a in range(j * g, j * g + g):
                x = (s["q"][i, a, first:].double() @ k.T) / math.sqrt(d)
                x = x.masked_fill(~see, -math.inf)
                lse = torch.logsumexp(x, -1)
                outs[i, a, first:] = torch.exp(x - lse[:, None]) @ v
                lses[i, a, first:] = lse
    return outs, lses
