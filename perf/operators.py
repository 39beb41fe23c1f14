"""The serving operators beside the INT4 paged cache, as cases that can be measured: rotary
positions applied where new keys enter the cache, decode attention for a batch that shares a long
prefix, decode attention that accumulates every cached token's attention weight, and the eviction
that keeps the heaviest tokens.

With ``own`` false, ``run`` computes an operator in its plain form: elementary torch operations in
32 bits (64 for the angles of the rotary table), rounded once at the end.  With ``own`` true it
makes the calls a user makes of ``bit_paged_kv_block_b200.saw``.

The cache is the library's: pages of 16 tokens, kv uint8 [pages][Hkv][2 (K, V)][16][D / 2] (low
nibble: even index), scales fp16 [pages][Hkv][2][16][2 (scale, zero)]; a cached value stands for
zero + code * scale, rotated by the normalised Hadamard transform of blocks of min(D, 128) unless
the cache is a plain INT4 one.  Codes are defined by fp32 operations in a fixed order, so they are
compared as they are stored.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
LOG2E = 1.4426950408889634


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # the cos / sin table of a model that rotates a quarter of 256-wide heads, 8 k positions
        dict(name="table_8k_r64_banded", op="table", positions=8192, rotary=64, kind="banded",
             base=500000.0, factor=8.0),
        # the table of a long-context model, filled once when it is loaded
        dict(name="table_256k_r128_yarn", op="table", positions=262144, rotary=128, kind="yarn",
             base=10000.0, factor=32.0),
        # one serving step's append: a batch of 64, four of its rows padding
        dict(name="append_step_64", op="append", tokens=64, hq=32, hkv=8, d=128, rotary=128,
             interleaved=False, strided=False, rotate=True, positions=131072, padded=4),
        # slices of a fused QKV output, half of 64-wide heads rotated, neighbours paired
        dict(name="append_4097_d64_fused", op="append", tokens=4097, hq=16, hkv=4, d=64, rotary=32,
             interleaved=True, strided=True, rotate=True, positions=8192, padded=0),
        # the prefill append of 32 sequences x 2048 tokens
        dict(name="append_prefill_65536", op="append", tokens=65536, hq=32, hkv=8, d=128,
             rotary=128, interleaved=False, strided=False, rotate=True, positions=131072, padded=0),
        # a handful of requests behind one short instruction
        dict(name="prefix_4x259", op="prefix", seqs=4, hq=8, hkv=2, d=128, prefix=259, lo=0, hi=41,
             rotate=True),
        # a chat batch behind one long system prompt
        dict(name="prefix_64x8192", op="prefix", seqs=64, hq=32, hkv=8, d=128, prefix=8192, lo=64,
             hi=2048, rotate=True),
        # many questions about one long document
        dict(name="prefix_64x32768_hq64", op="prefix", seqs=64, hq=64, hkv=8, d=128, prefix=32768,
             lo=1, hi=512, rotate=True),
        # a small batch of wide heads, plain INT4 cache
        dict(name="mass_3x333_d256", op="mass", seqs=3, hq=16, hkv=2, d=256, lo=1, hi=333,
             rotate=False),
        # the decode step of a batch of 64 whose cache is bounded by eviction
        dict(name="mass_64x8192", op="mass", seqs=64, hq=32, hkv=8, d=128, lo=512, hi=8192,
             rotate=True),
        # one long sequence brought down to a quarter
        dict(name="evict_1x32768", op="evict", seqs=1, hkv=8, d=128, lo=32768, hi=32768, keep=8192,
             sink=4, recent=1024),
        # a batch brought back to its budget
        dict(name="evict_64x4096", op="evict", seqs=64, hkv=8, d=128, lo=2048, hi=4096, keep=2048,
             sink=4, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# (Hq, Hkv, D): the head layouts of this repository's tests and benchmark, and an odd group
_HEADS = [(32, 8, 128), (64, 8, 128), (8, 2, 128), (16, 4, 64), (16, 2, 256), (12, 4, 128),
          (4, 4, 128), (32, 2, 128), (8, 1, 64), (10, 2, 128), (9, 3, 128)]


def draw(rng):
    op = rng.choice(["table", "append", "append", "prefix", "prefix", "mass", "mass", "evict"])
    hq, hkv, d = rng.choice(_HEADS)
    rotate = rng.random() < 0.75
    if op == "table":
        rotary = 16 * rng.randint(1, 16)
        return dict(op=op, positions=_log(rng, 100, 262144 * 128 // rotary), rotary=rotary,
                    kind=rng.choice(["none", "linear", "ntk", "banded", "yarn"]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    factor=rng.choice([1.0, 2.0, 4.0, 8.0, 32.0]))
    if op == "append":
        most = 65536 * (48 * 128) // ((hq + 2 * hkv) * d)
        tokens = _log(rng, 1, most)
        return dict(op=op, tokens=tokens, hq=hq, hkv=hkv, d=d, rotary=16 * rng.randint(1, d // 16),
                    interleaved=rng.random() < 0.5, strided=rng.random() < 0.5 and hkv != 3,
                    rotate=rotate,
                    positions=rng.choice([2048, 32768, 131072]),
                    padded=rng.randint(0, min(8, tokens - 1)))
    if op == "prefix":
        seqs = _log(rng, 1, 256)
        most = 64 * 64 * 128 * 32768 // (seqs * hq * d)
        own_most = 64 * 8 * 128 * 1024 // (seqs * hkv * d)
        lo = rng.choice([0, 1, 17, 64])
        return dict(op=op, seqs=seqs, hq=hq, hkv=hkv, d=d, prefix=_log(rng, 1, min(32768, most)),
                    lo=lo, hi=lo + _log(rng, 1, max(2, min(4096, own_most))), rotate=rotate)
    if op == "mass":
        seqs = _log(rng, 1, 64)
        most = 64 * 4352 * 8 * 128 // (seqs * hkv * d)
        lo = rng.choice([0, 1, 64, 512])
        return dict(op=op, seqs=seqs, hq=hq, hkv=hkv, d=d, lo=lo,
                    hi=lo + _log(rng, 1, max(2, min(32768, most))), rotate=rotate)
    seqs = _log(rng, 1, 64)
    most = 64 * 4096 * 8 * 128 // (seqs * hkv * d)
    hi = _log(rng, 16, min(65536, most))
    keep = max(1, int(hi * rng.uniform(0.1, 1.1)))
    sink = min(rng.choice([0, 4, 16]), keep)
    return dict(op=op, seqs=seqs, hkv=hkv, d=d, lo=rng.randint(0, hi), hi=hi, keep=keep, sink=sink,
                recent=rng.randint(0, keep - sink))


def _lens(case):
    """Lengths spread evenly over [lo, hi] (the seed only orders them)."""
    lo = case["lo"] if case["seqs"] > 1 else case["hi"]
    return np.linspace(lo, case["hi"], case["seqs"]).round().astype(np.int64)


def _blocks(n):
    return -(-n // PAGE)


def work(case):
    op = case["op"]
    if op == "table":
        n = case["positions"] * case["rotary"]
        return {"bytes": 4.0 * n, "flops": 8.0 * n}
    hkv, d = case["hkv"], case["d"]
    row = d / 2 + 4                                  # codes and (scale, zero) of one cached vector
    if op == "append":
        T, hq, r = case["tokens"] - case["padded"], case["hq"], case["rotary"]
        table = min(T, case["positions"]) * r * 4
        cache = T * hkv * (2 * row + 4)              # K and V rows, and the cleared mass
        return {"bytes": float(T * (2 * hq + 2 * hkv) * d * 2 + table + cache + 16 * T),
                "flops": float(T * (3 * r * (hq + hkv) + hkv * 2 * d * (math.log2(min(d, 128)) + 6)))}
    lens = _lens(case)
    if op == "prefix":
        S, hq, n = case["seqs"], case["hq"], case["prefix"] + int(lens.sum())
        return {"bytes": float(n * hkv * 2 * row + 4 * S * hq * d + 4 * _blocks(n)),
                "flops": float(4 * hq * d * (S * case["prefix"] + int(lens.sum())))}
    if op == "mass":
        S, hq, n = case["seqs"], case["hq"], int(lens.sum())
        return {"bytes": float(n * hkv * (2 * row + 8) + 4 * S * hq * d + 4 * _blocks(n)),
                "flops": float(4 * hq * d * n)}
    kept = int(np.minimum(lens, case["keep"]).sum())
    return {"bytes": float(int(lens.sum()) * hkv * 4 + kept * hkv * (2 * (2 * row) + 4 + 4)),
            "flops": float(int(lens.sum()) * hkv * 4)}


# ---- inputs -----------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000 + seed)


def _values(gen, n, h, d, outliers):
    """bf16 [n][h][d]: N(0, 1), with four channels of each head 10 to 30 times larger (keys)."""
    x = torch.randn(n, h, d, generator=gen, device="cuda")
    if outliers:
        at = torch.rand(h, d, generator=gen, device="cuda").argsort(1)[:, :4]
        x *= torch.ones(h, d, device="cuda").scatter_(
            1, at, 10 + 20 * torch.rand(h, 4, generator=gen, device="cuda"))
    return x.to(torch.bfloat16)


def _filled_cache(gen, pages, h, d, rotate):
    """A cache whose every row was quantized from drawn keys and values."""
    kv = torch.empty(pages, h, 2, PAGE, d // 2, dtype=torch.uint8, device="cuda")
    sc = torch.empty(pages, h, 2, PAGE, 2, dtype=torch.float16, device="cuda")
    step = max(1, (1 << 27) // (h * PAGE * d))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        for half in range(2):
            x = _values(gen, n * PAGE, h, d, half == 0).float()
            codes, pair = _quantize(x, rotate)
            kv[a:a + n, :, half] = codes.view(n, PAGE, h, d // 2).transpose(1, 2)
            sc[a:a + n, :, half] = pair.view(n, PAGE, h, 2).transpose(1, 2)
    return kv, sc


def _tables(gen, lens, extra=0):
    """A shuffled page for every block of every sequence: (int32 [S][max blocks], pages used);
    unused entries hold -1."""
    blocks = [_blocks(int(n)) for n in lens]
    perm = torch.randperm(sum(blocks) + extra, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(blocks))), -1, dtype=torch.int32)
    flat, at = perm.cpu(), 0
    for s, n in enumerate(blocks):
        table[s, :n] = flat[at:at + n]
        at += n
    return table.cuda(), flat[at:].cuda(), sum(blocks) + extra


def prepare(case, seed):
    gen = _gen(seed)
    st = {"case": case}
    op = case["op"]
    if op == "table":
        # positions up to the table's end; the seed moves its first position, as a table that is
        # extended while a conversation grows
        st["first"] = int(torch.randint(0, 4096, (1,), generator=gen, device="cuda"))
        st["table"] = torch.zeros(case["positions"], case["rotary"], device="cuda")
        return st
    hkv, d = case["hkv"], case["d"]
    if op == "append":
        T, hq = case["tokens"], case["hq"]
        q = _values(gen, T, hq, d, False)
        k, v = _values(gen, T, hkv, d, True), _values(gen, T, hkv, d, False)
        if case["strided"]:
            fused = torch.cat([q, k, v], 1)
            q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
        pages = _blocks(T) + 3
        perm = torch.randperm(pages, generator=gen, device="cuda")[:_blocks(T)]
        slots = (perm[:, None] * PAGE + torch.arange(PAGE, device="cuda")).view(-1)[:T].contiguous()
        if case["padded"]:
            slots[T - case["padded"]:] = -1
        angles = torch.rand(case["positions"], case["rotary"] // 2, generator=gen,
                            device="cuda", dtype=torch.float64) * (2 * math.pi)
        st.update(q=q, k=k, v=v, slots=slots,
                  positions=torch.randint(0, case["positions"], (T,), generator=gen, device="cuda"),
                  table=torch.cat([angles.cos(), angles.sin()], 1).float(),
                  q_out=torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda"),
                  kv=torch.zeros(pages, hkv, 2, PAGE, d // 2, dtype=torch.uint8, device="cuda"),
                  sc=torch.zeros(pages, hkv, 2, PAGE, 2, dtype=torch.float16, device="cuda"),
                  mass=torch.rand(pages, hkv, PAGE, generator=gen, device="cuda"))
        return st
    order = torch.randperm(case["seqs"], generator=gen, device="cuda").cpu().numpy()
    lens = _lens(case)[order]
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if op == "evict":
        new = np.minimum(lens, case["keep"])
        st["table"], free, pages = _tables(gen, lens, int(sum(_blocks(int(n)) for n in new)))
        blocks = [_blocks(int(n)) for n in new]
        table, free, at = torch.full((len(new), max(1, max(blocks))), -1, dtype=torch.int32), free.cpu(), 0
        for s, n in enumerate(blocks):
            table[s, :n] = free[at:at + n]
            at += n
        st["new_table"] = table.cuda()
        # moved rows are moved as they are: any bits will do for the codes
        st["kv"] = torch.randint(0, 256, (pages, hkv, 2, PAGE, d // 2), generator=gen, device="cuda",
                                 dtype=torch.uint8)
        st["sc"] = torch.rand(pages, hkv, 2, PAGE, 2, generator=gen, device="cuda").half()
        # accumulated weights: heavy-tailed, in steps of 1 / 1024 so that equal ones occur
        u = torch.rand(pages, hkv, PAGE, generator=gen, device="cuda")
        st["mass"] = (torch.floor(1024 * (0.01 / (u + 1e-3))) / 1024).contiguous()
        st["new_lens"] = torch.zeros(case["seqs"], dtype=torch.int32, device="cuda")
        st["kept"] = torch.zeros(case["seqs"], hkv, case["keep"], dtype=torch.int32, device="cuda")
        return st
    S, hq = case["seqs"], case["hq"]
    extra = _blocks(case["prefix"]) if op == "prefix" else 2
    st["table"], spare, pages = _tables(gen, lens, extra)
    st["kv"], st["sc"] = _filled_cache(gen, pages, hkv, d, case["rotate"])
    st["q"] = _values(gen, S, hq, d, False)
    st["out"] = torch.zeros(S, hq, d, dtype=torch.bfloat16, device="cuda")
    if op == "prefix":
        st["prefix_table"] = spare
    else:
        st["mass"] = torch.rand(pages, hkv, PAGE, generator=gen, device="cuda")
    if own:
        # the workspace, which a program keeps for the shapes it serves
        from bit_paged_kv_block_b200 import saw
        if op == "prefix":
            st["ws"] = saw.allocate_prefix_workspace(hkv, hq, S, case["prefix"], head_dim=d)
        else:
            st["ws"] = saw.allocate_mass_workspace(hkv, hq, S, st["table"].shape[1], head_dim=d)
    return st


# ---- plain forms ------------------------------------------------------------------------------

def _frequencies(kind, rotary, base, factor, original=8192, low=1.0, high=4.0, fast=32.0, slow=1.0):
    """Angle per position of each pair and the amplitude, in 64 bits."""
    i = torch.arange(rotary // 2, dtype=torch.float64)
    if kind == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    inv = base ** (-2 * i / rotary)
    amplitude = 1.0
    if kind == "linear":
        inv = inv / factor
    elif kind == "banded":
        turns = original * inv / (2 * math.pi)       # turns over the original context
        t = ((turns - low) / (high - low)).clamp(0, 1)
        inv = inv * ((1 - t) / factor + t)
    elif kind == "yarn":
        at = lambda b: rotary * math.log(original / (2 * math.pi * b)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(at(fast))), min(rotary - 1, math.ceil(at(slow)))
        t = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        inv = inv * (t / factor + (1 - t))
        amplitude = 0.1 * math.log(factor) + 1.0
    return inv, amplitude


def _butterfly(x):
    """The normalised Hadamard transform of each block of min(D, 128), stages h = 1, 2, ..., every
    step one fp32 operation."""
    d = x.shape[-1]
    block = min(d, 128)
    lead = x.shape[:-1]
    h = 1
    while h < block:
        a, b = x.view(-1, d // (2 * h), 2, h).unbind(2)
        x = torch.stack([a + b, a - b], 2)
        h *= 2
    return (x * (0.125 if block == 64 else 0.0883883461356163)).view(*lead, d)


def _quantize(x, rotate):
    """Packed codes uint8 [..., D / 2] and fp16 (scale, zero) [..., 2] of fp32 vectors."""
    y = _butterfly(x) if rotate else x
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    scale = (hi - lo) / torch.full((), 15.0, device=y.device)
    codes = torch.where(scale > 0, torch.round((y - lo) / scale), 0).clamp(0, 15).to(torch.uint8)
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return packed, torch.cat([scale, lo + 0.0], -1).half()


def _rope(x, cos, sin, rotary, interleaved):
    """Rotate pairs of the first `rotary` elements of each head (fp32 in, bf16 out)."""
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
        y[..., 0:rotary:2], y[..., 1:rotary:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rotary // 2], x[..., rotary // 2:rotary]
        y[..., :rotary // 2], y[..., rotary // 2:rotary] = a * cos - b * sin, b * cos + a * sin
    return y.to(torch.bfloat16)


def _dequant(kv, sc, pages):
    """fp32 K, V of the pages (any shape [...]): each [..., Hkv, 16, D]."""
    c, p = kv[pages], sc[pages].float()
    x = torch.stack([c & 15, c >> 4], -1).flatten(-2).float()
    x = x * p[..., 0:1] + p[..., 1:2]
    return x.unbind(-3)


def _rotated(x, rotate):
    return _butterfly(x) if rotate else x


def _plain_table(st):
    case = st["case"]
    inv, amp = _frequencies(case["kind"], case["rotary"], case["base"], case["factor"])
    pos = torch.arange(st["first"], st["first"] + case["positions"], dtype=torch.float64, device="cuda")
    angle = pos[:, None] * inv.cuda()
    st["table"].copy_(torch.cat([angle.cos() * amp, angle.sin() * amp], 1))
    return {"table": st["table"]}


def _plain_append(st):
    case = st["case"]
    at = (st["slots"] >= 0).nonzero()[:, 0]          # the tokens that are not padding
    half = case["rotary"] // 2
    cs = st["table"][st["positions"][at]]
    cos, sin = cs[:, :half], cs[:, half:]
    rope = lambda x: _rope(x[at].float(), cos, sin, case["rotary"], case["interleaved"])
    st["q_out"][at] = rope(st["q"])
    page, off = st["slots"][at] // PAGE, st["slots"][at] % PAGE
    k, v = rope(st["k"]).float(), st["v"][at].float()
    st["kv"][page, :, 0, off], st["sc"][page, :, 0, off] = _quantize(k, case["rotate"])
    st["kv"][page, :, 1, off], st["sc"][page, :, 1, off] = _quantize(v, case["rotate"])
    st["mass"][page, :, off] = 0.0
    return {"q": st["q_out"], "pages": st["kv"], "scales": st["sc"], "mass": st["mass"]}


def _own_logits(st, q):
    """Logits [S, Hkv, G, L] and values [S, Hkv, L, D] of each sequence's own tokens; -inf past
    its length."""
    S, hkv, g, d = q.shape
    blocks = st["table"].shape[1]
    k, v = (x.transpose(1, 2).reshape(S, hkv, blocks * PAGE, d)
            for x in _dequant(st["kv"], st["sc"], st["table"].clamp(min=0).long()))
    logits = q @ k.transpose(2, 3)
    live = torch.arange(blocks * PAGE, device="cuda") < st["lens"][:, None]
    return torch.where(live[:, None, None], logits, -math.inf), v


def _plain_prefix(st):
    case = st["case"]
    S, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
    q = (_rotated(st["q"].float(), case["rotate"]) / math.sqrt(d)).view(S, hkv, hq // hkv, d)
    own_logits, own_v = _own_logits(st, q)
    k, v = (x.transpose(0, 1).reshape(hkv, -1, d)[:, :case["prefix"]]
            for x in _dequant(st["kv"], st["sc"], st["prefix_table"].long()))
    logits = q.transpose(0, 1).reshape(hkv, -1, d) @ k.transpose(1, 2)       # [Hkv, S G, P]
    top = torch.maximum(logits.amax(-1).view(hkv, S, -1).transpose(0, 1), own_logits.amax(-1))
    w = torch.exp(logits - top.transpose(0, 1).reshape(hkv, -1, 1))
    own_w = torch.exp(own_logits - top[..., None])
    total = w.sum(-1).view(hkv, S, -1).transpose(0, 1) + own_w.sum(-1)
    o = (w @ v).view(hkv, S, -1, d).transpose(0, 1) + own_w @ own_v
    o = (o / total[..., None]).reshape(S, hq, d)
    st["out"].copy_(_rotated(o, case["rotate"]))
    return {"out": st["out"]}


def _plain_mass(st):
    case = st["case"]
    S, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
    q = (_rotated(st["q"].float(), case["rotate"]) / math.sqrt(d)).view(S, hkv, hq // hkv, d)
    logits, v = _own_logits(st, q)
    top = logits.amax(-1, keepdim=True)
    w = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0)
    st["out"].copy_(_rotated((w @ v).reshape(S, hq, d), case["rotate"]))
    added = w.sum(2).view(S, hkv, -1, PAGE).transpose(1, 2).reshape(-1, hkv, PAGE)
    st["mass"].index_add_(0, st["table"].clamp(min=0).view(-1).long(), added)
    return {"out": st["out"], "mass": st["mass"]}


def _plain_evict(st):
    case = st["case"]
    S, hkv, keep = case["seqs"], case["hkv"], case["keep"]
    lens = st["lens"].long()
    n = torch.minimum(lens, torch.full_like(lens, keep))
    L = st["table"].shape[1] * PAGE
    at = torch.arange(L, device="cuda")
    score = st["mass"][st["table"].clamp(min=0).long()].transpose(1, 2).reshape(S, hkv, L)
    fixed = (at < case["sink"]) | (at >= lens[:, None] - case["recent"])
    score = torch.where(fixed[:, None], math.inf, score)
    score = torch.where((at < lens[:, None])[:, None], score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices   # ties: lowest first
    j = torch.arange(keep, device="cuda")
    pick = torch.nn.functional.pad(best, (0, max(0, keep - L)), value=L)[..., :keep]
    pick = torch.where((j < n[:, None])[:, None], pick, L).sort(-1).values   # cache order
    live = (j < n[:, None])[:, None].expand(S, hkv, keep)
    st["kept"].copy_(torch.where(live, pick, -1))
    s, h, k = live.nonzero().unbind(1)
    src = pick[s, h, k]
    page, off = st["table"][s, src // PAGE].long(), src % PAGE
    to, to_off = st["new_table"][s, k // PAGE].long(), k % PAGE
    st["kv"][to, h, :, to_off] = st["kv"][page, h, :, off]
    st["sc"][to, h, :, to_off] = st["sc"][page, h, :, off]
    st["mass"][to, h, to_off] = st["mass"][page, h, off]
    st["new_lens"].copy_(n)
    return {"pages": st["kv"], "scales": st["sc"], "mass": st["mass"], "lens": st["new_lens"],
            "kept": st["kept"]}


# ---- the library's calls ----------------------------------------------------------------------

def _run_own(st):
    from bit_paged_kv_block_b200 import saw
    case = st["case"]
    op = case["op"]
    if op == "table":
        scaling = saw.rope_scaling(case["kind"], base=case["base"], factor=case["factor"],
                                   original_positions=8192, low=1.0, high=4.0, fast=32.0, slow=1.0)
        saw.saw_rope_table(st["table"], scaling, first_position=st["first"])
        return {"table": st["table"]}
    if op == "append":
        saw.saw_rope_rotate_quantize_paged(
            st["q"], st["k"], st["v"], st["positions"], st["slots"],
            (st["table"], case["interleaved"]), st["q_out"], st["kv"], st["sc"], mass=st["mass"],
            rotate=case["rotate"])
        return {"q": st["q_out"], "pages": st["kv"], "scales": st["sc"], "mass": st["mass"]}
    if op == "prefix":
        saw.saw_paged_decode_attn_prefix(
            st["q"], st["kv"], st["sc"], st["prefix_table"], case["prefix"], st["table"],
            st["lens"], st["out"], st["ws"], rotate=case["rotate"])
        return {"out": st["out"]}
    if op == "mass":
        saw.saw_paged_decode_attn_mass(
            st["q"], st["kv"], st["sc"], st["mass"], st["table"], st["lens"], st["out"], st["ws"],
            rotate=case["rotate"])
        return {"out": st["out"], "mass": st["mass"]}
    saw.saw_evict_paged(
        st["kv"], st["sc"], st["mass"], st["table"], st["lens"], st["new_table"], st["new_lens"],
        st["kept"], sink=case["sink"], recent=case["recent"])
    return {"pages": st["kv"], "scales": st["sc"], "mass": st["mass"], "lens": st["new_lens"],
            "kept": st["kept"]}


def run(state):
    if own:
        return _run_own(state)
    return {"table": _plain_table, "append": _plain_append, "prefix": _plain_prefix,
            "mass": _plain_mass, "evict": _plain_evict}[state["case"]["op"]](state)


# ---- the definitions in 64 bits ---------------------------------------------------------------

def _hadamard64(d):
    """The normalised block-diagonal Hadamard matrix: entry (i, j) of a block has the sign
    (-1)^popcount(i & j)."""
    b = min(d, 128)
    i = np.arange(b)
    sign = 1.0 - 2.0 * (np.array([bin(x).count("1") for x in range(b)])[i[:, None] & i[None]] % 2)
    return torch.tensor(np.kron(np.eye(d // b), sign) / math.sqrt(b), device="cuda")


def _vectors64(st, pages, n, h):
    """K and V of one head's first n tokens in the given pages, rotated back: fp64 [n][D] each."""
    c = st["kv"][pages, h].long()                    # [blocks][2][16][D / 2]
    p = st["sc"][pages, h].double()
    d = 2 * c.shape[-1]
    x = torch.empty(*c.shape[:-1], d, dtype=torch.float64, device="cuda")
    x[..., 0::2], x[..., 1::2] = (c % 16).double(), (c // 16).double()
    x = x * p[..., :1] + p[..., 1:]
    if st["case"]["rotate"]:
        x = x @ _hadamard64(d)
    k, v = x[:, 0].reshape(-1, d)[:n], x[:, 1].reshape(-1, d)[:n]
    return k, v


def _attend64(st, shared):
    """fp64 attention one sequence and head at a time: outputs [S][Hq][D] and the weights."""
    case = st["case"]
    S, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    lens = st["lens"].tolist()
    out = torch.zeros(S, hq, d, dtype=torch.float64, device="cuda")
    mass = None if shared else st["mass"].double()
    for h in range(hkv):
        if shared:
            pk, pv = _vectors64(st, st["prefix_table"].long(), case["prefix"], h)
        for s in range(S):
            pages = st["table"][s, :_blocks(lens[s])].long()
            k, v = _vectors64(st, pages, lens[s], h)
            if shared:
                k, v = torch.cat([pk, k]), torch.cat([pv, v])
            if not len(k):
                continue
            w = torch.softmax(st["q"][s, h * g:(h + 1) * g].double() @ k.T / math.sqrt(d), 1)
            out[s, h * g:(h + 1) * g] = w @ v
            if not shared:
                full = torch.zeros(len(pages) * PAGE, dtype=torch.float64, device="cuda")
                full[:lens[s]] = w.sum(0)
                mass[pages, h] += full.view(-1, PAGE)
    return out, mass


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "table":
        inv, amp = _frequencies(case["kind"], case["rotary"], case["base"], case["factor"])
        pos = np.arange(st["first"], st["first"] + case["positions"], dtype=np.float64)
        z = amp * np.exp(1j * (pos[:, None] * inv.numpy()[None]))
        return {"table": np.concatenate([z.real, z.imag], 1)}
    if op == "prefix":
        return {"out": _attend64(st, True)[0]}
    if op == "mass":
        out, mass = _attend64(st, False)
        return {"out": out, "mass": mass}
    if op == "append":
        r, d = case["rotary"], case["d"]
        live = [t for t, s in enumerate(st["slots"].tolist()) if s >= 0]
        at = torch.tensor(live, device="cuda")
        turn = torch.complex(*st["table"][st["positions"][at]].double().split(r // 2, 1))[:, None]

        def turned(x):
            y = x[at].double()
            pair = y[..., :r].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
            if not case["interleaved"]:
                pair = pair.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            y[..., :r] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
            return y

        q = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        q[at] = turned(st["q"])
        scales, mass = st["sc"].double(), st["mass"].double()
        slot = st["slots"][at]
        # keys are held in bf16 between the rotary step and the quantizer, by definition
        for half, x in enumerate((turned(st["k"]).to(torch.bfloat16).double(), st["v"][at].double())):
            y = x @ _hadamard64(d) if case["rotate"] else x
            lo, hi = y.amin(-1), y.amax(-1)
            scales[slot // PAGE, :, half, slot % PAGE] = torch.stack([(hi - lo) / 15, lo], -1)
        mass[slot // PAGE, :, slot % PAGE] = 0
        # the codes are defined by 32-bit operations
        return {"q": q, "pages": None, "scales": scales, "mass": mass}
    lens, keep = st["lens"].tolist(), case["keep"]
    scales, mass = st["sc"].cpu().numpy().astype(np.float64), st["mass"].cpu().numpy().astype(np.float64)
    table, new = st["table"].cpu().numpy(), st["new_table"].cpu().numpy()
    for s, n in enumerate(lens):
        t = np.arange(n)
        held = (t < case["sink"]) | (t >= n - case["recent"])
        for h in range(case["hkv"]):
            m = mass[table[s, t // PAGE], h, t % PAGE]
            order = np.lexsort((t, -m, ~held))       # held ones, then by weight, then by place
            k = np.sort(order[:keep])
            j = np.arange(len(k))
            scales[new[s, j // PAGE], h, :, j % PAGE] = scales[table[s, k // PAGE], h, :, k % PAGE]
            mass[new[s, j // PAGE], h, j % PAGE] = m[k]
    return {"pages": None, "scales": scales, "mass": mass, "lens": None, "kept": None}
