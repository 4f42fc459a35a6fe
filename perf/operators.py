"""What is measured of the attention operators: rotary positions, the paged
key/value cache (written and read back) and attention, over that cache and
over whole prompts.

``listed()`` holds the cases, ``draw()`` makes more of the same ranges,
``prepare()`` the inputs of a case, ``run()`` one pass (elementary torch
operations in fp32, or the library's calls where ``own`` is set), ``work()``
what a pass cannot do without and ``exact()`` the definition in 64 bits.

Sizes: 32 query and 8 key/value heads of 128 are the 4096-wide q / o and
1024-wide k / v matrices of the 8B-shaped body; the others are generic.
"""
import math

import numpy as np
import torch

own = False

HALF, INTERLEAVED = 0, 1
BF16, INT8 = 0, 1


# ---------------------------------------------------------------------------
# Cases.

def listed():
    return [
        # one new token of one sequence: the rotation of q between the q product (fp32 output) and attention
        {"name": "rope, one token", "op": "rope", "n": 1, "heads": 32, "dim": 128, "rot": 128, "layout": HALF,
         "scaling": "none", "factor": 1.0, "first": 4097, "in": "f32", "out": "bf16", "pad": 0},
        # q and k of a long prompt in one fused buffer, a quarter of the head left alone, context extended by parts
        {"name": "rope, long prompt", "op": "rope", "n": 16001, "heads": 40, "dim": 128, "rot": 96,
         "layout": INTERLEAVED, "scaling": "parts", "factor": 8.0, "first": 100000, "in": "bf16", "out": "bf16",
         "pad": 1024},
        # 37 sequences decoding: q and k rotated, k and v of one token each into a bf16 cache
        {"name": "cache write, decode step", "op": "write", "n": 37, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "layout": HALF, "scaling": "none", "factor": 1.0, "first": 900, "in": "f32", "page": 16,
         "fmt": BF16, "spare": 200, "back": False},
        # a prompt's k and v quantised as they are written, and read back (a prefix taken up again)
        {"name": "cache write and read, prompt", "op": "write", "n": 8191, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "layout": HALF, "scaling": "linear", "factor": 4.0, "first": 0, "in": "f32", "page": 64,
         "fmt": INT8, "spare": 16, "back": True},
        # a long prefix read back from the int8 cache, pages in any order
        {"name": "cache read, long prefix", "op": "read", "n": 100003, "kv_heads": 8, "dim": 128, "page": 64,
         "fmt": INT8, "out": "bf16"},
        # one sequence, one new token, a short context: latency counts
        {"name": "decode, one sequence", "op": "paged", "seqs": 1, "max_new": 1, "max_len": 517, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "fmt": BF16},
        # a serving batch of uneven lengths over the int8 cache
        {"name": "decode, batch of 64, int8", "op": "paged", "seqs": 64, "max_new": 1, "max_len": 8192, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "fmt": INT8},
        # one long document: the context is what can be split
        {"name": "decode, long context", "op": "paged", "seqs": 1, "max_new": 1, "max_len": 131001, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 32, "fmt": BF16},
        # a mixed step: chunks of uneven size next to sequences with a token or two
        {"name": "chunks, mixed batch", "op": "paged", "seqs": 13, "max_new": 301, "max_len": 4100, "q_heads": 16,
         "kv_heads": 4, "dim": 64, "page": 16, "fmt": BF16},
        # a long prompt taken in pieces: one piece near its end, over the int8 cache
        {"name": "chunk, long prompt, int8", "op": "paged", "seqs": 1, "max_new": 2048, "max_len": 32768,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "fmt": INT8},
        # several short prompts packed one after another, wide heads, 5 query heads to each key head
        {"name": "prompts, packed", "op": "prompt", "seqs": 9, "max_len": 777, "q_heads": 10, "kv_heads": 2,
         "dim": 256, "causal": True},
        # a whole long prompt
        {"name": "prompt, long", "op": "prompt", "seqs": 1, "max_len": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "causal": True},
    ]


def _log(rng, a, b):
    """A whole number in [a, b], spread over its logarithm."""
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "paged", "paged", "prompt"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    rotary = {"rot": rng.choice([dim, dim, dim // 2, dim - 32]), "layout": rng.choice([HALF, INTERLEAVED])}
    rotary["scaling"] = rng.choice(["none", "linear", "ntk", "parts"])
    rotary["factor"] = 1.0 if rotary["scaling"] == "none" else rng.choice([2.0, 4.0, 8.0])
    if op == "rope":
        heads = rng.randint(1, 40)
        return {"op": op, "n": _log(rng, 1, max(1, 16001 * 40 * 128 // (heads * dim * 2))), "heads": heads, "dim": dim,
                **rotary, "first": _log(rng, 1, 1000000), "in": rng.choice(["f32", "bf16"]),
                "out": rng.choice(["f32", "bf16"]), "pad": rng.choice([0, 64, 1024])}
    if op == "write":
        return {"op": op, "n": _log(rng, 1, 8000), "q_heads": kv_heads * min(group, 4), "kv_heads": kv_heads,
                "dim": min(dim, 128), "rot": min(rotary["rot"], min(dim, 128)), "layout": rotary["layout"],
                "scaling": rotary["scaling"], "factor": rotary["factor"], "first": _log(rng, 1, 100000),
                "in": rng.choice(["f32", "bf16"]), "page": rng.choice([16, 32, 64, 128]),
                "fmt": rng.choice([BF16, INT8]), "spare": rng.randint(1, 50), "back": True}
    if op == "read":
        return {"op": op, "n": _log(rng, 1, 100003 * 1024 // (kv_heads * dim) // 2), "kv_heads": kv_heads, "dim": dim,
                "page": rng.choice([16, 32, 64, 128]), "fmt": rng.choice([BF16, INT8]),
                "out": rng.choice(["f32", "bf16"])}
    if op == "paged":
        kind = rng.choice(["decode", "few", "chunk"])
        seqs = _log(rng, 1, 64) if kind != "chunk" else rng.randint(1, 8)
        new = {"decode": 1, "few": rng.randint(2, 16), "chunk": _log(rng, 17, 1024)}[kind]
        most = {"decode": 131001, "few": 32768, "chunk": 16384}[kind]
        most = min(most, 524288 * 1024 // (seqs * kv_heads * dim), 2 ** 38 // (seqs * new * kv_heads * group * dim))
        return {"op": op, "seqs": seqs, "max_new": new, "max_len": _log(rng, new, max(new + 1, most)),
                "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128]),
                "fmt": rng.choice([BF16, INT8])}
    seqs, q_heads = rng.randint(1, 12), kv_heads * min(group, 32 // kv_heads)
    most = min(8192, math.isqrt(2 ** 37 // (seqs * q_heads * dim)))
    return {"op": op, "seqs": seqs, "max_len": _log(rng, 16, most), "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "causal": rng.random() < 0.8}


# ---------------------------------------------------------------------------
# Inputs.

def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _random(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return lambda *shape: torch.randn(shape, generator=g, device="cuda")


def _spread(count, most, least):
    """Whole numbers between least and most, the first of them the largest."""
    parts = [(1 - (0.6180339887 * i) % 1.0) ** 1.5 for i in range(count)]
    return [max(least, int(round(least + (most - least) * x))) for x in parts]


def _lengths(case):
    """New tokens and context (the new tokens among it) of each sequence."""
    new = _spread(case["seqs"], case["max_new"], 1)
    return new, [max(n, x) for n, x in zip(new, _spread(case["seqs"], case["max_len"], 1 + case["max_len"] // 16))]


def _frequencies(case):
    """Radians per position of each pair, and the factor on the rotated values."""
    rot, base, s = case["rot"], 1e6, case["factor"]
    if case["scaling"] == "ntk":
        base *= s ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        f = [w / s for w in f]
    if case["scaling"] != "parts":
        return f, 1.0
    keep = [min(1.0, max(0.0, (32768 * w / (2 * math.pi) - 1) / 31)) for w in f]
    return [w * (g + (1 - g) / s) for w, g in zip(f, keep)], 0.1 * math.log(s) + 1


def _rotary(case, seed):
    f, magnitude = _frequencies(case)
    turns = torch.tensor([int(round(w / (2 * math.pi) * 2.0 ** 64)) for w in f], dtype=torch.int64, device="cuda")
    pos = torch.arange(case["n"], dtype=torch.int32, device="cuda") + case["first"] + seed % 5
    return {"turns": turns, "pos": pos, "magnitude": magnitude}


def _rows(rand, n, width, pad, dtype):
    """[n][width] inside rows that are pad wider, some columns much larger than others as keys have them."""
    t = torch.empty((n, width + pad), dtype=dtype, device="cuda")[:, :width]
    gain = torch.exp(0.5 * rand(width))
    t.copy_(rand(n, width) * gain)
    return t


def _cache_parts(case, pages):
    """Byte offsets of the cache's planes: keys, values, and for int8 their scales; and its size."""
    values = pages * case["page"] * case["kv_heads"] * case["dim"] * (2 if case["fmt"] == BF16 else 1)
    sizes = [values, values] + ([values // case["dim"] * 4] * 2 if case["fmt"] == INT8 else [])
    at, off = [], 0
    for b in sizes:
        at.append(off)
        off += -(-b // 256) * 256
    return at, sizes, off


def _cache(case, pages, rand):
    """A cache of random rows: the bytes, and its planes as tensors [pages][kv heads][page][dim] (scales without dim)."""
    at, sizes, total = _cache_parts(case, pages)
    data = torch.zeros(total, dtype=torch.uint8, device="cuda")
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    part = lambda i, t, s: data[at[i]:at[i] + sizes[i]].view(t).view(s)  # noqa: E731
    planes = [part(i, torch.bfloat16 if case["fmt"] == BF16 else torch.int8, shape) for i in (0, 1)]
    planes += [part(i, torch.float32, shape[:3]) for i in (2, 3)] if case["fmt"] == INT8 else [None, None]
    if rand is not None:
        gain = torch.exp(0.5 * rand(2, case["kv_heads"], 1, case["dim"]))
        gain[1] = 1.0
        for i in (0, 1):
            x = rand(*shape)
            x *= gain[i]
            if case["fmt"] == BF16:
                planes[i].copy_(x)
            else:
                top = x.abs().amax(-1)
                planes[2 + i].copy_(top * (1.0 / 127.0))
                planes[i].copy_((x * (127.0 / top)[..., None]).round())
    return data, planes


def prepare(case, seed):
    rand, op = _random(seed), case["op"]
    s = {"case": case, "ws": None}
    if op == "rope":
        s.update(_rotary(case, seed))
        width = case["heads"] * case["dim"]
        s["x"] = _rows(rand, case["n"], width, case["pad"], _type(case["in"]))
        s["out"] = torch.zeros((case["n"], width), dtype=_type(case["out"]), device="cuda")
        return s
    if op in ("write", "read"):
        width = case["kv_heads"] * case["dim"]
        s["pages"] = pages = -(-case["n"] // case["page"]) + case.get("spare", 3)
        s["cache"], s["planes"] = _cache(case, pages, rand)
        if op == "write" and not case["back"]:   # a token for each of n sequences: a place in a page of its own
            s["pages"] = pages = case["n"] + case["spare"]
            s["cache"], s["planes"] = _cache(case, pages, rand)
            at = torch.randint(0, case["page"], (case["n"],), generator=torch.Generator().manual_seed(seed))
            order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:case["n"]]
            s["slots"] = (order * case["page"] + at).to(torch.int32).cuda()
        else:
            order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
            i = torch.arange(case["n"])
            s["slots"] = (order[i // case["page"]] * case["page"] + i % case["page"]).to(torch.int32).cuda()
        back = _type(case["out"]) if op == "read" else torch.bfloat16
        s["k_back"], s["v_back"] = (torch.zeros((case["n"], width), dtype=back, device="cuda") for _ in range(2))
        if op == "write":
            s.update(_rotary(case, seed))
            s["k"], s["v"] = (_rows(rand, case["n"], width, 0, _type(case["in"])) for _ in range(2))
            s["q"] = _rows(rand, case["n"], case["q_heads"] * case["dim"], 0, _type(case["in"]))
            s["q_out"] = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
        return s
    s["scale"] = case["dim"] ** -0.5
    if op == "paged":
        new, lens = _lengths(case)
        counts = [-(-x // case["page"]) for x in lens]
        s["pages"] = pages = sum(counts) + 3
        s["cache"], s["planes"] = _cache(case, pages, rand)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        tables, used = np.zeros((case["seqs"], max(counts)), np.int32), 0
        for i, c in enumerate(counts):
            tables[i, :c] = order[used:used + c]
            used += c
        s["tables"] = torch.from_numpy(tables).cuda()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        width = case["q_heads"] * case["dim"]
        total = sum(new)
        s["q"] = rand(total, width).to(torch.bfloat16)
    else:
        new = _spread(case["seqs"], case["max_len"], 1)
        total, wide = sum(new), (case["q_heads"] + 2 * case["kv_heads"]) * case["dim"]
        a = case["q_heads"] * case["dim"]
        b = a + case["kv_heads"] * case["dim"]
        width, fused = a, rand(total, wide).to(torch.bfloat16)   # q, k and v side by side in each token's row
        s["q"], s["k"], s["v"] = fused[:, :a], fused[:, a:b], fused[:, b:]
    s["starts"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    s["out"] = torch.zeros((total, width), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass.

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_rope(s):
    import ternary_hybrid_bit_amd as wal
    c = s["case"]
    return wal.wal_rope(s["x"], s["out"], s["pos"], s["turns"], c["dim"], layout=c["layout"],
                        magnitude=s["magnitude"])


def _own_desc(wal, s):
    c = s["case"]
    return wal.make_kv_desc(s["pages"], c["page"], c["kv_heads"], c["dim"], c["fmt"])


def _own_write(s):
    import ternary_hybrid_bit_amd as wal
    c, desc = s["case"], _own_desc(wal, s)
    wal.wal_kv_write(desc, s["cache"], s["slots"], s["k"], s["v"], pos=s["pos"], turns=s["turns"], layout=c["layout"],
                     magnitude=s["magnitude"], Q=s["q"], Q_out=s["q_out"])
    if c["back"]:
        return (s["q_out"],) + tuple(wal.wal_kv_read(desc, s["cache"], s["slots"], s["k_back"], s["v_back"]))
    return s["q_out"], s["planes"][0], s["planes"][1]


def _own_read(s):
    import ternary_hybrid_bit_amd as wal
    return wal.wal_kv_read(_own_desc(wal, s), s["cache"], s["slots"], s["k_back"], s["v_back"])


def _own_paged(s):
    import ternary_hybrid_bit_amd as wal
    c, desc = s["case"], _own_desc(wal, s)
    if s["ws"] is None:   # kept by the program, as every workspace is
        n = wal.wal_attn_paged_workspace_size(desc, c["q_heads"], c["seqs"], s["q"].shape[0], c["max_new"],
                                              c["max_len"])
        s["ws"] = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    return wal.wal_attn_paged(desc, s["cache"], s["tables"], s["lens"], s["starts"], s["q"], s["out"], s["ws"],
                              scale=s["scale"], max_new=c["max_new"], max_len=c["max_len"])


def _own_prompt(s):
    import ternary_hybrid_bit_amd as wal
    c = s["case"]
    return wal.wal_attn_prompt(s["q"], s["k"], s["v"], s["starts"], s["out"], c["dim"], c["max_len"],
                               scale=s["scale"], causal=c["causal"])


_own = {"rope": _own_rope, "write": _own_write, "read": _own_read, "paged": _own_paged, "prompt": _own_prompt}


def _turn(x, s):
    """x [n][heads][dim] in fp32, rotated."""
    c = s["case"]
    a = (s["pos"].long()[:, None] * s["turns"]).float() * (2 * math.pi * 2.0 ** -64)   # the product mod 2^64: turns
    cos, sin = (torch.cos(a) * s["magnitude"])[:, None], (torch.sin(a) * s["magnitude"])[:, None]
    r = c["rot"]
    if c["layout"] == HALF:
        u, v = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([u * cos - v * sin, v * cos + u * sin, x[..., r:]], -1)
    u, v = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2), x[..., r:]], -1)


def _plain_rope(s):
    x = s["x"].float().unflatten(-1, (-1, s["case"]["dim"]))
    return _turn(x, s).flatten(-2).to(s["out"].dtype)


def _places(s):
    p = s["case"]["page"]
    slots = s["slots"].long()
    return slots // p, slots % p


def _plain_write(s):
    c = s["case"]
    split = lambda t: t.float().unflatten(-1, (-1, c["dim"]))  # noqa: E731
    page, at = _places(s)
    for x, plane, scales in ((_turn(split(s["k"]), s), s["planes"][0], s["planes"][2]),
                             (split(s["v"]), s["planes"][1], s["planes"][3])):
        if c["fmt"] == INT8:
            top = x.abs().amax(-1)
            scales[page, :, at] = top * (1.0 / 127.0)
            x = (x * torch.where(top > 0, 127.0 / top, 0.0)[..., None]).round()
        plane[page, :, at] = x.to(plane.dtype)
    q = _turn(split(s["q"]), s).flatten(-2).to(torch.bfloat16)
    return (q,) + tuple(_plain_read(s)) if c["back"] else (q, s["planes"][0], s["planes"][1])


def _plain_read(s):
    page, at = _places(s)
    got = []
    for plane, scales, back in zip(s["planes"][:2], s["planes"][2:], (s["k_back"], s["v_back"])):
        x = plane[page, :, at].float()
        if scales is not None:
            x = x * scales[page, :, at][..., None]
        got.append(x.flatten(-2).to(back.dtype))
    return tuple(got)


def _attend(q, k, v, seen, scale):
    """q [seqs][kv heads][group][new][dim] over k, v [seqs][kv heads][keys][dim]; seen [seqs][new][keys]."""
    shape = q.shape
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2).contiguous()).view(*shape[:-1], k.shape[-2])
    x = (x * scale).masked_fill(~seen[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-3e38))
    x = x / x.sum(-1, keepdim=True).clamp_min(1e-38)
    return torch.matmul(x.flatten(2, 3), v).view(shape)


def _padded(t, starts, most, heads, dim):
    """Rows of each sequence side by side, [seqs][heads][most][dim] in fp32, and the rows' places in t."""
    at = starts[:-1, None].long() + torch.arange(most, device=t.device)
    at = at.clamp_max(t.shape[0] - 1)
    return t[at].float().unflatten(-1, (heads, dim)).transpose(1, 2), at


def _plain_paged(s):
    c = s["case"]
    h, g, d = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["dim"]
    kv = []
    for plane, scales in zip(s["planes"][:2], s["planes"][2:]):
        x = plane[s["tables"].long()].float()
        if scales is not None:
            x = x * scales[s["tables"].long()][..., None]
        kv.append(x.transpose(1, 2).flatten(2, 3))   # [seqs][kv heads][keys][dim]
    q, _ = _padded(s["q"], s["starts"], c["max_new"], c["q_heads"], d)
    lens, new = s["lens"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(c["max_new"], device="cuda")
    last = (lens - new)[:, None] + i                 # the last key that row i of a sequence sees
    seen = torch.arange(kv[0].shape[2], device="cuda") <= last[..., None]
    o = _attend(q.unflatten(1, (h, g)), kv[0], kv[1], seen, s["scale"])
    o = o.flatten(1, 2).transpose(1, 2).flatten(2).to(torch.bfloat16)
    return o[i < new[:, None]]


def _plain_prompt(s):
    c = s["case"]
    h, g, d, n = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["dim"], c["max_len"]
    q, _ = _padded(s["q"], s["starts"], n, h * g, d)
    k, _ = _padded(s["k"], s["starts"], n, h, d)
    v, _ = _padded(s["v"], s["starts"], n, h, d)
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(n, device="cuda")
    seen = (i < new[:, None])[:, None].expand(-1, n, -1)
    if c["causal"]:
        seen = seen & (i <= i[:, None])
    o = _attend(q.unflatten(1, (h, g)), k, v, seen, s["scale"])
    return o.flatten(1, 2).transpose(1, 2).flatten(2).to(torch.bfloat16)[i < new[:, None]]


_plain = {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "paged": _plain_paged,
          "prompt": _plain_prompt}


# ---------------------------------------------------------------------------
# What a pass cannot do without.

def work(case):
    op, b = case["op"], {"f32": 4, "bf16": 2}
    d = case["dim"]
    if op == "rope":
        n = case["n"] * case["heads"] * d
        return {"bytes": n * (b[case["in"]] + b[case["out"]]) + 4 * case["n"] + 4 * case["rot"],
                "flops": 3 * n * case["rot"] // d}
    if op in ("write", "read"):
        row = case["kv_heads"] * (2 * d if case["fmt"] == BF16 else d + 4)   # bytes of a token's keys in the cache
        n, kv = case["n"], case["kv_heads"] * d
        if op == "read":
            return {"bytes": n * (2 * row + 2 * kv * b[case["out"]] + 4), "flops": 2 * n * kv}
        q = case["q_heads"] * d
        back = 2 * row + 4 * kv if case["back"] else 0
        return {"bytes": n * ((q + 2 * kv) * b[case["in"]] + 2 * q + 2 * row + back + 8) + 4 * case["rot"],
                "flops": n * (3 * (q + kv) + 4 * kv)}
    if op == "paged":
        new, lens = _lengths(case)
        row = case["kv_heads"] * (4 * d if case["fmt"] == BF16 else 2 * d + 8)
        pairs = sum(n * (x - n) + n * (n + 1) // 2 for n, x in zip(new, lens))
        return {"bytes": sum(lens) * row + sum(new) * case["q_heads"] * d * 4, "flops": 4 * pairs * case["q_heads"] * d}
    new = _spread(case["seqs"], case["max_len"], 1)
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in new)
    return {"bytes": sum(new) * d * (4 * case["q_heads"] + 4 * case["kv_heads"]),
            "flops": 4 * pairs * case["q_heads"] * d}


# ---------------------------------------------------------------------------
# The definition, in 64 bits.

def _exact_turn(x, case, pos):
    """Each pair as a complex number times magnitude * exp(i * position * frequency)."""
    f, magnitude = _frequencies(case)
    r = case["rot"]
    f = torch.tensor(f, dtype=torch.float64, device=x.device)
    w = magnitude * torch.exp(1j * pos.double()[:, None] * f)[:, None]
    first, second = (slice(0, r // 2), slice(r // 2, r)) if case["layout"] == HALF else (slice(0, r, 2), slice(1, r, 2))
    z = torch.complex(x[..., first], x[..., second]) * w
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rows(x, case):
    """Rows as a cache of this format holds them."""
    if case["fmt"] == BF16:
        return x
    unit = x.abs().amax(-1, keepdim=True) / 127
    return torch.where(unit > 0, torch.round(x / torch.where(unit > 0, unit, torch.ones_like(unit))) * unit, 0.0)


def _exact_cache(s, plane):
    x = s["planes"][plane].double()
    return x * s["planes"][2 + plane].double()[..., None] if s["case"]["fmt"] == INT8 else x


def _exact_softmax(q, k, v, scale, last):
    """Rows q [new][heads][dim]; row i sees keys 0 .. last[i]."""
    group = q.shape[1] // k.shape[1]
    out = torch.zeros_like(q)
    for h in range(q.shape[1]):
        z = (q[:, h] @ k[:, h // group].T) * scale
        z[torch.arange(k.shape[0], device=z.device)[None] > last[:, None]] = -math.inf
        w = torch.softmax(z, -1)
        w[last < 0] = 0
        out[:, h] = w @ v[:, h // group]
    return out.flatten(1)


def exact(case, seed):
    s, op, d = prepare(case, seed), case["op"], case["dim"]
    heads = lambda t: t.double().unflatten(-1, (-1, d))  # noqa: E731
    if op == "rope":
        return _exact_turn(heads(s["x"]), case, s["pos"]).flatten(1)
    if op in ("write", "read"):
        slot, page = s["slots"].long(), case["page"]
        if op == "read":
            return tuple(_exact_cache(s, i)[slot // page, :, slot % page].flatten(1) for i in (0, 1))
        q = _exact_turn(heads(s["q"]), case, s["pos"]).flatten(1)
        rows = [_exact_rows(_exact_turn(heads(s["k"]), case, s["pos"]), case), _exact_rows(heads(s["v"]), case)]
        if case["back"]:
            return q, rows[0].flatten(1), rows[1].flatten(1)
        planes = [_exact_cache(s, i) for i in (0, 1)]
        for x, plane in zip(rows, planes):
            plane[slot // page, :, slot % page] = x
        return q, planes[0], planes[1]
    starts = s["starts"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["seqs"]):
        a, b = starts[i], starts[i + 1]
        row = torch.arange(b - a, device="cuda")
        if op == "paged":
            n = int(s["lens"][i])
            pages = s["tables"][i, :-(-n // case["page"])].long()
            k, v = (_exact_cache(s, j)[pages].transpose(1, 2).flatten(0, 1)[:n] for j in (0, 1))
            last = n - (b - a) + row
        else:
            k, v = heads(s["k"][a:b]), heads(s["v"][a:b])
            last = row if case["causal"] else torch.full_like(row, b - a - 1)
        out[a:b] = _exact_softmax(heads(s["q"][a:b]), k, v, s["scale"], last)
    return out
