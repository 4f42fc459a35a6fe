"""What is measured of the operators around the products of blocks with head
norms and of delta-rule blocks: norms of single heads with the rotation or a
gate in the same pass (also on the way into the paged cache), the causal
convolution with kept state, and the gated delta rule.

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
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases.

def listed():
    return [
        # a delta-rule block's output for one new token: normed by heads and gated, before the o product
        {"name": "gated norm, one token", "op": "norm", "n": 1, "heads": 48, "dim": 128, "then": "gate", "in": "bf16",
         "gate": "f32", "out": "bf16", "weight": "bf16", "pad": 0},
        # the same of a long prompt
        {"name": "gated norm, long prompt", "op": "norm", "n": 8192, "heads": 48, "dim": 128, "then": "gate",
         "in": "bf16", "gate": "f32", "out": "bf16", "weight": "bf16", "pad": 0},
        # q of a long prompt that needs no cache (scoring): normed, a quarter of each head rotated, wide heads
        {"name": "norm and rotation, long prompt", "op": "norm", "n": 8001, "heads": 20, "dim": 256, "then": "rotate",
         "rot": 64, "layout": HALF, "first": 100000, "in": "f32", "out": "bf16", "weight": "f32", "pad": 0},
        # 37 sequences decoding: q and k normed and rotated, k and v of one token each into a bf16 cache
        {"name": "normed cache write, decode", "op": "write", "n": 37, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "layout": HALF, "first": 900, "in": "f32", "weight": "bf16", "page": 16, "fmt": BF16, "spare": 200},
        # a prompt's keys normed, rotated and quantised as they are written, then read back (a prefix taken up again)
        {"name": "normed cache write, prompt", "op": "write", "n": 8191, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "layout": HALF, "first": 0, "in": "f32", "weight": "bf16", "page": 64, "fmt": INT8, "spare": 16},
        # q | k | v of one new token of a delta-rule block (16 key and 48 value heads of 128)
        {"name": "convolution, one token", "op": "conv", "seqs": 1, "max_new": 1, "channels": 10240, "taps": 4,
         "in": "f32", "out": "bf16", "weight": "bf16", "bias": False, "silu": True},
        # several prompts packed one after another
        {"name": "convolution, packed prompts", "op": "conv", "seqs": 7, "max_new": 4099, "channels": 8192, "taps": 4,
         "in": "f32", "out": "bf16", "weight": "bf16", "bias": True, "silu": True},
        # one new token of one sequence: latency counts
        {"name": "delta rule, one token", "op": "delta", "seqs": 1, "max_new": 1, "key_heads": 16, "value_heads": 48,
         "key_dim": 128, "value_dim": 128, "gates": "raw"},
        # a serving batch: the states are what is moved
        {"name": "delta rule, batch of 64", "op": "delta", "seqs": 64, "max_new": 1, "key_heads": 16,
         "value_heads": 48, "key_dim": 128, "value_dim": 128, "gates": "raw"},
        # a few tokens of each sequence at once (guesses that are checked together)
        {"name": "delta rule, few tokens", "op": "delta", "seqs": 13, "max_new": 5, "key_heads": 16, "value_heads": 32,
         "key_dim": 128, "value_dim": 128, "gates": "raw"},
        # uneven prompts packed, narrow heads, gates from the caller
        {"name": "delta rule, packed prompts", "op": "delta", "seqs": 9, "max_new": 1111, "key_heads": 4,
         "value_heads": 8, "key_dim": 64, "value_dim": 96, "gates": "given"},
        # a whole long prompt
        {"name": "delta rule, long prompt", "op": "delta", "seqs": 1, "max_new": 8192, "key_heads": 16,
         "value_heads": 48, "key_dim": 128, "value_dim": 128, "gates": "raw"},
    ]


def _log(rng, a, b):
    """A whole number in [a, b], spread over its logarithm."""
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 1)))))))


def draw(rng):
    op, types = rng.choice(["norm", "write", "conv", "delta", "delta"]), ["f32", "bf16"]
    if op == "norm":
        dim, heads = rng.choice([64, 80, 128, 128, 192, 256]), rng.randint(1, 48)
        case = {"op": op, "n": _log(rng, 1, max(1, 8192 * 48 * 128 // (heads * dim * 2))), "heads": heads, "dim": dim,
                "then": rng.choice(["gate", "rotate", "nothing"]), "in": rng.choice(types), "out": rng.choice(types),
                "weight": rng.choice(types), "pad": rng.choice([0, 64, 1024])}
        if case["then"] == "gate":
            case["gate"] = rng.choice(types)
        if case["then"] == "rotate":
            case.update(rot=rng.choice([dim, dim - 16, 32, 64]), layout=rng.choice([HALF, INTERLEAVED]),
                        first=_log(rng, 1, 1000000))
        return case
    if op == "write":
        dim, kv_heads = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 5, 8])
        return {"op": op, "n": _log(rng, 1, 8000 * 128 // max(dim, 128)), "q_heads": kv_heads * rng.randint(1, 4),
                "kv_heads": kv_heads, "dim": dim, "rot": rng.choice([dim, dim // 2, dim // 4]),
                "layout": rng.choice([HALF, INTERLEAVED]), "first": _log(rng, 1, 100000), "in": rng.choice(types),
                "weight": rng.choice(types), "page": rng.choice([16, 32, 64, 128]), "fmt": rng.choice([BF16, INT8]),
                "spare": rng.randint(1, 50)}
    if op == "conv":
        seqs, channels = _log(rng, 1, 64), 8 * _log(rng, 1, 1500)
        most = max(1, min(8192, 7 * 4099 * 8192 // (3 * seqs * channels)))
        return {"op": op, "seqs": seqs, "max_new": rng.choice([1, _log(rng, 1, most), _log(rng, 1, most)]),
                "channels": channels, "taps": rng.randint(2, 4), "in": rng.choice(types), "out": rng.choice(types),
                "weight": rng.choice(types), "bias": rng.random() < 0.5, "silu": rng.random() < 0.8}
    key_heads, key_dim = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128, 128])
    value_heads, value_dim = key_heads * rng.randint(1, 4), rng.choice([32, 64, 96, 128, 128, 256])
    kind = rng.choice(["one", "few", "chunk", "chunk"])
    state = value_heads * key_dim * value_dim
    seqs = _log(rng, 1, min(64, 64 * 48 * 128 * 128 // state)) if kind != "chunk" else rng.randint(1, 12)
    most = max(65, min(8192, 8192 * 48 * 128 * 128 // (2 * seqs * state)))
    return {"op": op, "seqs": seqs, "max_new": {"one": 1, "few": rng.randint(2, 16), "chunk": _log(rng, 17, most)}[kind],
            "key_heads": key_heads, "value_heads": value_heads, "key_dim": key_dim, "value_dim": value_dim,
            "gates": rng.choice(["raw", "given"])}


# ---------------------------------------------------------------------------
# Inputs.

def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _random(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return lambda *shape: torch.randn(shape, generator=g, device="cuda")


def _new_tokens(case):
    """New tokens of each sequence, the first of them the most."""
    parts = [(1 - (0.6180339887 * i) % 1.0) ** 1.5 for i in range(case["seqs"])]
    return [max(1, int(round(1 + (case["max_new"] - 1) * x))) for x in parts]


def _frequencies(case):
    """Radians per position of each pair."""
    return [1e6 ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]


def _rotary(case, seed):
    turns = [int(round(w / (2 * math.pi) * 2.0 ** 64)) for w in _frequencies(case)]
    pos = torch.arange(case["n"], dtype=torch.int32, device="cuda") + case["first"] + seed % 5
    return {"turns": torch.tensor(turns, dtype=torch.int64, device="cuda"), "pos": pos}


def _rows(rand, n, width, dtype, pad=0):
    """[n][width] inside rows that are pad wider, some columns much larger than others."""
    t = torch.empty((n, width + pad), dtype=dtype, device="cuda")[:, :width]
    t.copy_(rand(n, width) * torch.exp(0.5 * rand(width)))
    return t


def _slots(case, seed):
    """A place of its own for each sequence's state, in any order."""
    order = torch.randperm(case["seqs"] + 2, generator=torch.Generator().manual_seed(seed))
    return order[:case["seqs"]].to(torch.int32).cuda()


def _cache(case, pages):
    """An empty cache: its bytes, and its planes as tensors [pages][kv heads][page][dim] (scales without dim)."""
    values = pages * case["page"] * case["kv_heads"] * case["dim"] * (2 if case["fmt"] == BF16 else 1)
    sizes = [values, values] + ([values // case["dim"] * 4] * 2 if case["fmt"] == INT8 else [])
    at = np.cumsum([0] + [-(-b // 256) * 256 for b in sizes]).tolist()
    data = torch.zeros(at[-1], dtype=torch.uint8, device="cuda")
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    part = lambda i, t, s: data[at[i]:at[i] + sizes[i]].view(t).view(s)  # noqa: E731
    planes = [part(i, torch.bfloat16 if case["fmt"] == BF16 else torch.int8, shape) for i in (0, 1)]
    return data, planes + ([part(i, torch.float32, shape[:3]) for i in (2, 3)] if case["fmt"] == INT8 else [None, None])


def _starts(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    rand, op = _random(seed), case["op"]
    s = {"case": case, "ws": None}
    if op == "norm":
        width = case["heads"] * case["dim"]
        s["x"] = _rows(rand, case["n"], width, _type(case["in"]), case["pad"])
        s["weight"] = (1 + 0.3 * rand(case["dim"])).to(_type(case["weight"]))
        s["out"] = torch.zeros((case["n"], width), dtype=_type(case["out"]), device="cuda")
        if case["then"] == "gate":
            s["gate"] = _rows(rand, case["n"], width, _type(case["gate"]))
        if case["then"] == "rotate":
            s.update(_rotary(case, seed))
        return s
    if op == "write":
        s["pages"] = pages = -(-case["n"] // case["page"]) + case["spare"]
        s["cache"], s["planes"] = _cache(case, pages)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
        i = torch.arange(case["n"])
        s["slots"] = (order[i // case["page"]] * case["page"] + i % case["page"]).to(torch.int32).cuda()
        s.update(_rotary(case, seed))
        kv, q = case["kv_heads"] * case["dim"], case["q_heads"] * case["dim"]
        s["q"], s["k"], s["v"] = (_rows(rand, case["n"], w, _type(case["in"])) for w in (q, kv, kv))
        s["q_norm"], s["k_norm"] = ((1 + 0.3 * rand(case["dim"])).to(_type(case["weight"])) for _ in range(2))
        s["q_out"] = torch.zeros((case["n"], q), dtype=torch.bfloat16, device="cuda")
        s["k_back"], s["v_back"] = (torch.zeros((case["n"], kv), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return s
    new = _new_tokens(case)
    n = sum(new)
    s["starts"], s["slots"] = _starts(new), _slots(case, seed)
    if op == "conv":
        c, t = case["channels"], _type(case["in"])
        s["x"] = _rows(rand, n, c, t)
        s["state"] = rand(case["seqs"] + 2, case["taps"] - 1, c).to(t)
        s["weight"] = (0.5 * rand(c, case["taps"])).to(_type(case["weight"]))
        s["bias"] = (0.2 * rand(c)).to(_type(case["weight"])) if case["bias"] else None
        s["out"] = torch.zeros((n, c), dtype=_type(case["out"]), device="cuda")
        return s
    # q, k and v side by side as the convolution leaves them: through silu, columns of different size
    kw, vw = case["key_heads"] * case["key_dim"], case["value_heads"] * case["value_dim"]
    x = rand(n, 2 * kw + vw) * torch.exp(0.3 * rand(2 * kw + vw))
    fused = (x * torch.sigmoid(x)).to(torch.bfloat16)
    s["q"], s["k"], s["v"] = fused[:, :kw], fused[:, kw:2 * kw], fused[:, 2 * kw:]
    h = case["value_heads"]
    gates = rand(n, 2 * h)
    s["decay"] = s["shift"] = None
    if case["gates"] == "raw":
        # a step of 0.001 to 0.1 at a = 0, decays of 1 to 16 per unit of it
        step = torch.exp(rand(h).sigmoid() * math.log(100.0) + math.log(0.001))
        s["shift"] = torch.log(torch.expm1(step))
        s["decay"] = 1 + 15 * rand(h).sigmoid()
    else:
        gates[:, :h] = -0.1 * torch.exp(gates[:, :h])
        gates[:, h:].sigmoid_()
    s["a"], s["b"] = gates[:, :h], gates[:, h:]
    s["state"] = 0.2 * rand(case["seqs"] + 2, h, case["key_dim"], case["value_dim"])
    s["out"] = torch.zeros((n, vw), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass.

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_norm(s):
    import ternary_hybrid_bit_amd as wal
    c = s["case"]
    return wal.wal_head_norm(s["x"], s["out"], s["weight"], c["dim"], eps=EPS, pos=s.get("pos"), turns=s.get("turns"),
                             layout=c.get("layout", HALF), gate=s.get("gate"))


def _own_write(s):
    import ternary_hybrid_bit_amd as wal
    c = s["case"]
    desc = wal.make_kv_desc(s["pages"], c["page"], c["kv_heads"], c["dim"], c["fmt"])
    wal.wal_kv_write(desc, s["cache"], s["slots"], s["k"], s["v"], pos=s["pos"], turns=s["turns"], layout=c["layout"],
                     Q=s["q"], Q_out=s["q_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
    if c["fmt"] == INT8:
        return (s["q_out"],) + tuple(wal.wal_kv_read(desc, s["cache"], s["slots"], s["k_back"], s["v_back"]))
    return s["q_out"], s["planes"][0], s["planes"][1]


def _own_conv(s):
    import ternary_hybrid_bit_amd as wal
    wal.wal_conv(s["x"], s["weight"], s["starts"], s["out"], state=s["state"], slots=s["slots"], bias=s["bias"],
                 silu=s["case"]["silu"])
    return s["out"], s["state"]


def _own_delta(s):
    import ternary_hybrid_bit_amd as wal
    c = s["case"]
    desc = wal.make_delta_desc(c["key_heads"], c["value_heads"], c["key_dim"], c["value_dim"], norm_eps=EPS)
    if s["ws"] is None:   # kept by the program, as every workspace is
        n = wal.wal_delta_workspace_size(desc, c["seqs"], s["q"].shape[0], c["max_new"])
        s["ws"] = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    wal.wal_delta(desc, s["q"], s["k"], s["v"], s["a"], s["b"], s["starts"], s["out"], state=s["state"],
                  slots=s["slots"], ws=s["ws"], decay=s["decay"], shift=s["shift"], max_new=c["max_new"])
    return s["out"], s["state"]


_own = {"norm": _own_norm, "write": _own_write, "conv": _own_conv, "delta": _own_delta}


def _turn(x, s):
    """x [n][heads][dim] in fp32, rotated."""
    a = (s["pos"].long()[:, None] * s["turns"]).float() * (2 * math.pi * 2.0 ** -64)   # the product mod 2^64: turns
    cos, sin, r = torch.cos(a)[:, None], torch.sin(a)[:, None], s["case"]["rot"]
    if s["case"]["layout"] == HALF:
        u, v = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([u * cos - v * sin, v * cos + u * sin, x[..., r:]], -1)
    u, v = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2), x[..., r:]], -1)


def _normed(x, weight):
    """x [n][heads * dim] -> fp32 [n][heads][dim]."""
    x = x.float().unflatten(-1, (-1, weight.shape[0]))
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _plain_norm(s):
    y = _normed(s["x"], s["weight"])
    if s["case"]["then"] == "rotate":
        y = _turn(y, s)
    y = y.flatten(-2)
    if s["case"]["then"] == "gate":
        g = s["gate"].float()
        y = y * (g * torch.sigmoid(g))
    return y.to(s["out"].dtype)


def _plain_write(s):
    c, p, slots = s["case"], s["case"]["page"], s["slots"].long()
    for x, plane, scales in ((_turn(_normed(s["k"], s["k_norm"]), s), s["planes"][0], s["planes"][2]),
                             (s["v"].float().unflatten(-1, (-1, c["dim"])), s["planes"][1], s["planes"][3])):
        if c["fmt"] == INT8:
            top = x.abs().amax(-1)
            scales[slots // p, :, slots % p] = top * (1.0 / 127.0)
            x = (x * torch.where(top > 0, 127.0 / top, 0.0)[..., None]).round()
        plane[slots // p, :, slots % p] = x.to(plane.dtype)
    q = _turn(_normed(s["q"], s["q_norm"]), s).flatten(-2).to(torch.bfloat16)
    if c["fmt"] == BF16:
        return q, s["planes"][0], s["planes"][1]
    at = (slots // p, slice(None), slots % p)
    return (q,) + tuple((s["planes"][i][at].float() * s["planes"][2 + i][at][..., None]).flatten(1).to(torch.bfloat16)
                        for i in (0, 1))


def _padded(s):
    """Rows of each sequence side by side, [seqs][most]: their places among the call's rows, and whether there are such."""
    starts = s["starts"].long()
    i = torch.arange(s["case"]["max_new"], device="cuda")
    there = i < (starts[1:] - starts[:-1])[:, None]
    return torch.where(there, starts[:-1, None] + i, 0), there


def _plain_conv(s):
    c, slots, (at, there) = s["case"], s["slots"].long(), _padded(s)
    n = c["max_new"]
    x = torch.cat([s["state"][slots], s["x"][at]], 1)            # a sequence's state and its rows
    w = s["weight"].float()
    y = sum(x[:, j:j + n].float() * w[:, j] for j in range(c["taps"]))
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["silu"]:
        y = y * torch.sigmoid(y)
    out = y[there].to(s["out"].dtype)
    last = there.sum(1)[:, None] + torch.arange(c["taps"] - 1, device="cuda")
    s["state"][slots] = x[torch.arange(c["seqs"], device="cuda")[:, None], last]
    return out, s["state"]


def _gates(s):
    """Logarithms of the decays, in 64 bits since they are added up, and the steps, both [n][value heads]."""
    if s["decay"] is None:
        return s["a"].double(), s["b"].float()
    x = s["a"] + s["shift"]
    return (-s["decay"] * (x.clamp_min(0) + torch.log1p(torch.exp(-x.abs())))).double(), torch.sigmoid(s["b"])


def _chunks(x, size):
    """[seqs][rows][heads][...] -> [chunks][seqs][heads][size][...], zeros behind the last row."""
    x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, -x.shape[1] % size))
    return x.unflatten(1, (-1, size)).transpose(0, 1).transpose(2, 3).contiguous()


def _plain_delta(s):
    c, slots, (at, there) = s["case"], s["slots"].long(), _padded(s)
    h, group, size = c["value_heads"], c["value_heads"] // c["key_heads"], min(64, c["max_new"])
    g, b = (torch.where(there[..., None], x[at], 0) for x in _gates(s))

    def heads(t, dim):
        return t[at].float().unflatten(-1, (-1, dim)) * there[..., None, None]

    q, k = (heads(s[t], c["key_dim"]) for t in ("q", "k"))
    q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS) for x in (q, k))
    q = q * c["key_dim"] ** -0.5
    q, k, v = (_chunks(x, size) for x in (q.repeat_interleave(group, 2), k.repeat_interleave(group, 2),
                                          heads(s["v"], c["value_dim"])))
    g, b = (_chunks(x[..., None], size) for x in (g, b))          # [chunks][seqs][heads][size][1]
    far = g.cumsum(-2)
    end = far[..., -1:, :]
    i = torch.arange(size, device="cuda")
    apart = torch.exp((far - far.transpose(-1, -2)).masked_fill(i[:, None] < i, -math.inf)).float()
    kt = k.transpose(-1, -2).contiguous()
    a = torch.matmul(k, kt) * apart * b * (i[:, None] > i)
    p = torch.matmul(q, kt) * apart
    t = torch.eye(size, device="cuda").expand_as(a).contiguous()   # (1 + a)^-1, a row after the other
    for r in range(1, size):
        t[..., r, :] -= torch.matmul(a[..., r:r + 1, :r], t[..., :r, :])[..., 0, :]
    far, end, left = torch.exp(far).float(), torch.exp(end).float(), torch.exp(end - far).float()
    kt = (k * left).transpose(-1, -2).contiguous()
    state, out = s["state"][slots], []
    for j in range(q.shape[0]):
        u = torch.matmul(t[j], b[j] * (v[j] - far[j] * torch.matmul(k[j], state)))
        out.append(far[j] * torch.matmul(q[j], state) + torch.matmul(p[j], u))
        state = end[j] * state + torch.matmul(kt[j], u)
    s["state"][slots] = state
    out = torch.stack(out, 1).transpose(2, 3).flatten(1, 2)[:, :c["max_new"]]   # [seqs][rows][heads][dim]
    return out[there].flatten(1).to(torch.bfloat16), s["state"]


_plain = {"norm": _plain_norm, "write": _plain_write, "conv": _plain_conv, "delta": _plain_delta}


# ---------------------------------------------------------------------------
# What a pass cannot do without.

def work(case):
    op, b = case["op"], {"f32": 4, "bf16": 2}
    if op == "norm":
        n = case["n"] * case["heads"] * case["dim"]
        gate = b[case["gate"]] if case["then"] == "gate" else 0
        return {"bytes": n * (b[case["in"]] + b[case["out"]] + gate) + case["dim"] * b[case["weight"]],
                "flops": 4 * n + (6 * n if gate else 0)}
    if op == "write":
        n, d = case["n"], case["dim"]
        q, kv = case["q_heads"] * d, case["kv_heads"] * d
        row = case["kv_heads"] * (2 * d if case["fmt"] == BF16 else d + 4)   # bytes of a token's keys in the cache
        back = 2 * row + 4 * kv if case["fmt"] == INT8 else 0
        return {"bytes": n * ((q + 2 * kv) * b[case["in"]] + 2 * q + 2 * row + back + 8),
                "flops": n * (7 * (q + kv) + 4 * kv)}
    n = sum(_new_tokens(case))
    if op == "conv":
        c, t = case["channels"], case["taps"]
        return {"bytes": n * c * (b[case["in"]] + b[case["out"]]) + 2 * case["seqs"] * (t - 1) * c * b[case["in"]]
                + c * t * b[case["weight"]], "flops": n * c * (2 * t + 4)}
    h, state = case["value_heads"], case["value_heads"] * case["key_dim"] * case["value_dim"]
    row = 2 * (2 * case["key_heads"] * case["key_dim"] + 2 * h * case["value_dim"]) + 8 * h
    return {"bytes": n * row + 8 * case["seqs"] * state, "flops": 7 * n * state}


# ---------------------------------------------------------------------------
# The definition, in 64 bits.

def _exact_normed(x, weight):
    x = x.double().unflatten(-1, (-1, weight.numel()))
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) / weight.numel() + EPS) * weight.double()


def _exact_turn(x, s):
    """Each pair as a complex number times exp(i * position * frequency)."""
    r = s["case"]["rot"]
    f = torch.tensor(_frequencies(s["case"]), dtype=torch.float64, device=x.device)
    w = torch.exp(1j * s["pos"].double()[:, None] * f)[:, None]
    first, second = (slice(0, r // 2), slice(r // 2, r)) if s["case"]["layout"] == HALF else (slice(0, r, 2), slice(1, r, 2))
    z = torch.complex(x[..., first], x[..., second]) * w
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_int8_rows(x):
    unit = x.abs().amax(-1, keepdim=True) / 127
    return torch.round(x / unit) * unit


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        y = _exact_normed(s["x"], s["weight"])
        if case["then"] == "rotate":
            y = _exact_turn(y, s)
        y = y.flatten(1)
        return y * torch.nn.functional.silu(s["gate"].double()) if case["then"] == "gate" else y
    if op == "write":
        k = _exact_turn(_exact_normed(s["k"], s["k_norm"]), s)
        v = s["v"].double().unflatten(-1, (-1, case["dim"]))
        q = _exact_turn(_exact_normed(s["q"], s["q_norm"]), s).flatten(1)
        if case["fmt"] == INT8:
            return q, _exact_int8_rows(k).flatten(1), _exact_int8_rows(v).flatten(1)
        slot, planes = s["slots"].long(), [torch.zeros(p.shape, dtype=torch.float64, device="cuda") for p in s["planes"][:2]]
        for x, plane in zip((k, v), planes):
            plane[slot // case["page"], :, slot % case["page"]] = x
        return (q, *planes)
    starts, slots = s["starts"].tolist(), s["slots"].tolist()
    state = s["state"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    if op == "conv":
        w, t = s["weight"].double(), case["taps"]
        for i, slot in enumerate(slots):
            rows = torch.cat([state[slot], s["x"][starts[i]:starts[i + 1]].double()])
            y = torch.einsum("ncj,cj->nc", rows.unfold(0, t, 1), w)
            if s["bias"] is not None:
                y = y + s["bias"].double()
            out[starts[i]:starts[i + 1]] = torch.nn.functional.silu(y) if case["silu"] else y
            state[slot] = rows[rows.shape[0] - (t - 1):]
        return out, state
    # one token of every sequence after the other
    h, group = case["value_heads"], case["value_heads"] // case["key_heads"]

    def unit(x):
        x = x.double().unflatten(-1, (-1, case["key_dim"]))
        return (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)).repeat_interleave(group, 1)

    q, k, v = unit(s["q"]), unit(s["k"]), s["v"].double().unflatten(-1, (h, -1))
    if s["decay"] is None:
        alpha, beta = torch.exp(s["a"].double()), s["b"].double()
    else:
        alpha = torch.exp(-s["decay"].double() * torch.logaddexp(s["a"].double() + s["shift"].double(),
                                                                 torch.zeros((), dtype=torch.float64, device="cuda")))
        beta = torch.special.expit(s["b"].double())
    got = out.unflatten(1, (h, -1))
    counts = torch.tensor(_new_tokens(case))
    for i in range(case["max_new"]):
        live = (counts > i).nonzero()[:, 0].cuda() if int(counts.min()) <= i else slice(None)
        row, at = s["starts"][:-1].long()[live] + i, s["slots"].long()[live]
        m = state[at] * alpha[row][..., None, None]
        miss = v[row] - (m * k[row][..., None]).sum(-2)
        m = m + k[row][..., None] * (beta[row][..., None] * miss)[..., None, :]
        got[row] = (m * q[row][..., None]).sum(-2) * case["key_dim"] ** -0.5
        state[at] = m
    return out, state
