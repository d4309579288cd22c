"""Workloads of the operators around the paged KV cache of a serving step: the linear map with low-rank
adapters of many requests beside the shared weights, the norms of q and k with the rotation by one or
several position axes and the append to the cache, and the block tables and slot maps that say where
the step's tokens go.

``listed()`` names the workloads, ``draw(rng)`` makes one more of the same ranges, ``prepare`` builds
the inputs on the GPU, ``run`` makes one pass.  With ``own`` false a pass is the operators' plain form
in elementary torch operations (32-bit arithmetic, angles in 64, one rounding at the end); with
``own`` true it calls the library.  ``exact`` is the operators' definition in 64 bits.

Shapes come from this repository's configurations (the tiny, 1B and 8B decoder shapes, batches of 8,
prompts of 4096 tokens) and go beyond them where an operator's range does.
"""
import math
import random

import numpy as np
import torch

own = False

FLOP_CAP = 2.5e11          # a drawn linear map costs no more than the largest listed one
ADAPTER_CAP = 1 << 29      # bytes of all adapters of a drawn case


def listed():
    return [
        # one token through the attention output projection of the 1B shape, with its request's adapter, added to the residual
        dict(name="adapted_token", op="adapted", rows=1, k=2048, n=2048, rank=16, adapters=8, act="", bias=False, residual="f32",
             out="f32", pad=0, runs=0, mix=1),
        # a decode batch of 8 requests with 8 different adapters of 64 loaded ones, gate/up with SwiGLU (1B)
        dict(name="adapted_batch8_swiglu", op="adapted", rows=8, k=2048, n=8192, rank=16, adapters=64, act="swiglu", bias=False,
             residual="", out="bf16", pad=0, runs=0, mix=2),
        # odd sizes: tokens of any adapter or of none, a rank that is no power of two, strided rows, bias and GELU
        dict(name="adapted_odd_gelu", op="adapted", rows=333, k=688, n=1001, rank=24, adapters=5, act="gelu", bias=True, residual="bf16",
             out="bf16", pad=24, runs=3, mix=3),
        # 64 requests, each with its own adapter of rank 64, through the q/k/v projection of the 8B shape: adapters outweigh weights
        dict(name="adapted_batch64_qkv", op="adapted", rows=64, k=4096, n=6144, rank=64, adapters=64, act="", bias=False, residual="",
             out="f32", pad=0, runs=0, mix=4),
        # prompts of 4096 tokens in all, a few requests with an adapter each, gate/up with SwiGLU (1B): products are the floor
        dict(name="adapted_prompt_swiglu", op="adapted", rows=4096, k=2048, n=8192, rank=16, adapters=8, act="swiglu", bias=False,
             residual="", out="bf16", pad=0, runs=600, mix=5),
        # one token far along (1B heads), contiguous cache
        dict(name="rope_token", op="rope", tokens=1, nq=32, nkv=8, d=64, rot=64, pairs="halves", sections=0, norm=False, dtype="bf16",
             block=0, far=100000, padded=0, mix=1),
        # odd widths: a part of each head rotated in neighbouring pairs, norms, fp32 rows, a padded batch
        dict(name="rope_odd_padded", op="rope", tokens=333, nq=12, nkv=4, d=80, rot=48, pairs="neighbours", sections=0, norm=True,
             dtype="f32", block=16, far=5000, padded=60, mix=2),
        # a 4096-token prompt (8B heads) with norms of q and k into a paged cache, from the projection's 32-bit sums
        dict(name="rope_prompt_norm", op="rope", tokens=4096, nq=32, nkv=8, d=128, rot=128, pairs="halves", sections=0, norm=True,
             dtype="f32", block=128, far=8192, padded=0, mix=3),
        # 16384 tokens of video and text (8B heads): three axes of position, norms, bf16 rows, paged
        dict(name="rope_video_axes", op="rope", tokens=16384, nq=32, nkv=8, d=128, rot=128, pairs="halves", sections=3, norm=True,
             dtype="bf16", block=256, far=0, padded=0, mix=4),
        # a decode step of 8 requests, one token each, blocks of 128 positions
        dict(name="pages_step", op="pages", batch=8, block=128, most=4096, tokens=1, ends=0, prefix=0, mix=1),
        # 200 requests: some end and give their blocks back, some begin, chunks of up to 512 tokens behind a shared prefix
        dict(name="pages_ragged", op="pages", batch=200, block=16, most=8192, tokens=512, ends=30, prefix=1000, mix=2),
        # 256 prompts of up to 8192 tokens at once: a million slots
        dict(name="pages_prompts", op="pages", batch=256, block=128, most=16384, tokens=8192, ends=0, prefix=0, mix=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["adapted", "adapted", "rope", "rope", "pages"])
    mix = rng.randrange(1 << 20)
    if kind == "adapted":
        while True:
            c = dict(op="adapted", rows=_log(rng, 1, 4096), k=8 * _log(rng, 8, 1024), n=_log(rng, 16, 8192),
                     rank=rng.choice([8, 16, 16, 24, 32, 64, 128]), adapters=_log(rng, 1, 128),
                     act=rng.choice(["", "", "silu", "gelu", "swiglu"]), bias=rng.random() < 0.5,
                     residual=rng.choice(["", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]), pad=rng.choice([0, 0, 8, 40]), runs=0, mix=mix)
            if c["rows"] > 256 or rng.random() < 0.4:   # prompts: neighbouring tokens share a request's adapter
                c["runs"] = max(1, c["rows"] // rng.choice([1, 3, 8, 20]))
            size = 2 * c["adapters"] * c["rank"] * (c["k"] + (2 if c["act"] == "swiglu" else 1) * c["n"])
            if work(c)["flops"] <= FLOP_CAP and size <= ADAPTER_CAP and size * c["rows"] <= FLOP_CAP:   # (the plain form takes all)
                return c
    if kind == "rope":
        nkv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([32, 64, 64, 80, 96, 128, 128, 256])
        most = min(16384, 16384 * 48 * 128 // (nkv * (group + 2) * d))
        return dict(op="rope", tokens=_log(rng, 1, most), nq=nkv * group, nkv=nkv, d=d,
                    rot=d if rng.random() < 0.7 else 16 * rng.randint(1, d // 16), pairs=rng.choice(["halves", "halves", "neighbours"]),
                    sections=rng.choice([0, 0, 2, 3]), norm=rng.random() < 0.6, dtype=rng.choice(["bf16", "f32"]),
                    block=rng.choice([0, 16, 48, 128]), far=rng.choice([0, 0, 7000, 1000000]), padded=rng.choice([0, 0, 30]), mix=mix)
    batch = _log(rng, 1, 1024)
    tokens = min(_log(rng, 1, 8192), (1 << 20) // batch)
    return dict(op="pages", batch=batch, block=rng.choice([8, 16, 48, 128, 256]), most=_log(rng, 2 * tokens, 32768), tokens=tokens,
                ends=rng.choice([0, 0, 10, 40]), prefix=rng.choice([0, 0, 100, 512]), mix=mix)


def _index(case):
    """The adapter of every token (-1: none): each its own, or runs of neighbouring tokens."""
    r = random.Random(case["mix"])
    rows, n = case["rows"], case["adapters"]
    if not case["runs"]:
        order = list(range(n))
        r.shuffle(order)
        return [order[i % n] for i in range(rows)] if rows <= n else [r.randrange(-1, n) for _ in range(rows)]
    out = []
    while len(out) < rows:
        out += [r.randrange(-1, n)] * r.randint(1, 2 * case["runs"])
    return out[:rows]


def _lengths(case):
    """Cached positions of each request before and after the step, the shared prefix's among them (a
    request that has ended: 0 after the step, one that is not there at all: 0 and 0)."""
    r = random.Random(case["mix"])
    old, new = [], []
    for _ in range(case["batch"]):
        n = r.randint(1, case["tokens"])
        a = case["prefix"] + (r.randint(0, case["most"] - n) if r.random() < 0.8 else 0)
        if r.randrange(100) < case["ends"]:
            a, n = (a, -a) if r.random() < 0.7 else (0, 0)
        old.append(a)
        new.append(a + n)
    return old, new


def work(case):
    if case["op"] == "adapted":
        m, k, n, r = case["rows"], case["k"], case["n"], case["rank"]
        f = 2 if case["act"] == "swiglu" else 1
        size = {"": 0, "bf16": 2, "f32": 4}
        index = _index(case)
        used, with_one = len(set(index) - {-1}), sum(i >= 0 for i in index)
        return {"bytes": 2 * m * k + 2 * f * n * k + (2 * f * n if case["bias"] else 0) + m * n * (size[case["residual"]] + size[case["out"]]) +
                2 * used * r * (k + f * n) + 4 * m, "flops": 2 * f * m * n * k + 2 * with_one * r * (k + f * n)}
    if case["op"] == "rope":
        t, nq, nkv, d = case["tokens"], case["nq"], case["nkv"], case["d"]
        kept = t - case["padded"] * t // 100
        return {"bytes": t * (nq + 2 * nkv) * d * (2 if case["dtype"] == "bf16" else 4) + 2 * t * nq * d + 4 * kept * nkv * d +
                4 * t * (1 + max(case["sections"], 1)), "flops": t * (nq + nkv) * (3 * case["rot"] + (5 * d if case["norm"] else 0))}
    old, new = _lengths(case)
    b, p = case["block"], case["prefix"] // case["block"]
    tokens = sum(max(y - x, 0) for x, y in zip(old, new))
    moved = sum(abs(max(-(-y // b), p) - max(-(-x // b), p)) for x, y in zip(old, new))
    return {"bytes": 12 * tokens + 8 * moved + 16 * case["batch"], "flops": 8 * tokens}


def _normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


class Cache:
    """K and V as the decoder keeps them: [batch, layers, heads, positions, d], or the pool of a paged cache."""

    def __init__(self, k, v):
        self.k, self.v = k, v


_KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}


def _prepare_adapted(case, seed, s):
    m, k, n, pad, r, count = (case[x] for x in ("rows", "k", "n", "pad", "rank", "adapters"))
    f = 2 if case["act"] == "swiglu" else 1
    s["x"] = _normal((m, k + pad), seed * 16 + 1).to(torch.bfloat16)[:, :k]
    s["w"] = _normal((f * n, k), seed * 16 + 2, 1.0 / math.sqrt(k)).to(torch.bfloat16)   # pre-activations of about 1
    s["b"] = _normal((f * n,), seed * 16 + 3, 0.5).to(torch.bfloat16) if case["bias"] else None
    s["r"] = _normal((m, n + pad), seed * 16 + 4).to(_KINDS[case["residual"]])[:, :n] if case["residual"] else None
    s["down"] = _normal((count, r, k), seed * 16 + 5, 1.0 / math.sqrt(k)).to(torch.bfloat16)
    s["up"] = _normal((count, f * n, r), seed * 16 + 6, 1.0 / math.sqrt(r)).to(torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(seed * 16 + 7)
    s["scale"] = torch.rand(count, generator=g, device="cuda") * 0.75 + 0.25             # alpha / rank
    s["index"] = torch.tensor(_index(case), dtype=torch.int32, device="cuda")
    s["dtype"] = _KINDS[case["out"]]


def _sections(case):
    """Pairs of each axis: the first a quarter, the others equal shares, any rest to the last."""
    pairs, n = case["rot"] // 2, case["sections"]
    if not n:
        return [pairs]
    first = pairs // 4 if n == 3 else pairs // 2
    rest = pairs - first
    return [first, rest] if n == 2 else [first, rest // 2, rest - rest // 2]


def _prepare_rope(case, seed, s):
    t, nq, nkv, d, block = (case[x] for x in ("tokens", "nq", "nkv", "d", "block"))
    s["qkv"] = _normal((t, (nq + 2 * nkv) * d), seed * 16 + 1, 1.5).to(_KINDS[case["dtype"]])
    r = random.Random(case["mix"])
    # sequences of uneven lengths, each behind what its cache holds already
    lens = []
    while sum(lens) < t:
        lens.append(min(r.randint(1, max(1, t // 2)), t - sum(lens)))
    before = [r.randint(0, 300) for _ in lens]
    top = max(a + b for a, b in zip(lens, before))
    if block:
        per = -(-top // block)
        order = torch.randperm(len(lens) * per, generator=torch.Generator().manual_seed(seed)).tolist()
        shape = (1, nkv, len(lens) * per * block, d)
    else:
        per, order, shape = 1, range(len(lens)), (len(lens), 1, nkv, top, d)
    slots, at = [], []
    for b, (n, a) in enumerate(zip(lens, before)):
        p = np.arange(a, a + n)
        size = block or top
        slots.append(np.asarray(order)[b * per + p // size] * size + p % size)
        at.append(p + case["far"])
    slots, at = np.concatenate(slots), np.concatenate(at)
    if case["padded"]:   # the last rows of a padded batch have no place in the cache
        kept = t - case["padded"] * t // 100
        slots[kept:], at[kept:] = -1, 0
    if case["sections"]:   # frames of 28 x 46 patches behind one another, the first axis time
        axes = np.stack([at, at % 1288 // 46, at % 46] if case["sections"] == 3 else [at // 46, at % 46])
        axes = np.where(np.arange(t) % 2000 < 100, at, axes)      # and text, whose axes are alike
    else:
        axes = at
    s["positions"] = torch.tensor(axes, dtype=torch.int32, device="cuda")
    s["slots"] = torch.tensor(slots, dtype=torch.int32, device="cuda")
    s["kv"] = Cache(_normal(shape, seed * 16 + 2).to(torch.bfloat16), _normal(shape, seed * 16 + 3).to(torch.bfloat16))
    s["gains"] = [(1 + _normal((d,), seed * 16 + i, 0.1)).to(torch.bfloat16) for i in (4, 5)] if case["norm"] else [None, None]
    s["eps"], s["theta"] = 1e-5, 500000.0
    s["freqs"] = s["theta"] ** (-2.0 * torch.arange(case["rot"] // 2, dtype=torch.float64) / case["rot"])   # radians a position
    s["rates"], s["parts"] = s["freqs"].cuda(), _sections(case)
    s["axis"] = torch.repeat_interleave(torch.arange(len(s["parts"])), torch.tensor(s["parts"])).cuda()


def _prepare_pages(case, seed, s):
    block, p = case["block"], case["prefix"] // case["block"]
    old, new = _lengths(case)
    per = max(-(-max(old + new) // block), p, 1)
    held = [max(-(-a // block), p) for a in old]
    wanted = [max(-(-a // block), p) for a in new]
    grown = sum(max(w - h, 0) for h, w in zip(held, wanted))
    total = p + sum(h - p for h in held) + grown + random.Random(case["mix"]).randint(1, 200)
    ids = np.random.default_rng(seed).permutation(total)
    table = np.full((case["batch"], per), -1)
    table[:, :p], taken = ids[:p], p                 # the shared prefix's whole blocks are in every row
    for b, h in enumerate(held):
        table[b, p:h] = ids[taken:taken + h - p]
        taken += h - p
    free = total - taken
    head = int(np.random.default_rng(seed + 1).integers(total))
    ring = np.full(total, -1)
    ring[(head + np.arange(free)) % total] = ids[taken:]
    i32 = dict(dtype=torch.int32, device="cuda")
    s["lens"], s["new"] = torch.tensor(old, **i32), torch.tensor(new, **i32)
    s["table"], s["ring"] = torch.tensor(table, **i32), torch.tensor(ring, **i32)
    s["ends"], s["next"] = torch.tensor([head, free, 0], **i32), torch.zeros(3, **i32)
    s["most_tokens"] = sum(max(b - a, 0) for a, b in zip(old, new)) + 5   # (rows of a padded batch behind the tokens)


def prepare(case, seed):
    s = dict(case)
    {"adapted": _prepare_adapted, "rope": _prepare_rope, "pages": _prepare_pages}[case["op"]](case, seed, s)
    return s


_ACTS = {"": lambda y: y, "silu": lambda y: y / (1 + torch.exp(-y)), "gelu": lambda y: 0.5 * y * (1 + torch.erf(y / math.sqrt(2.0)))}


def _adapted(s):
    x, count = s["x"].float(), s["adapters"]
    y = x @ s["w"].float().T
    if s["b"] is not None:
        y = y + s["b"].float()
    # every adapter's low-rank rows for every token, of which a token keeps its own adapter's
    t = (x @ s["down"].float().reshape(-1, s["k"]).T).reshape(len(x), count, -1)
    mine = s["index"][:, None] == torch.arange(count, device=x.device)
    t = torch.where(mine[:, :, None], t * s["scale"][:, None], 0.0).reshape(len(x), -1)
    y = y + t @ s["up"].float().transpose(1, 2).reshape(-1, y.shape[1])
    if s["act"] == "swiglu":
        gate, up = y[:, :s["n"]], y[:, s["n"]:]
        y = gate / (1 + torch.exp(-gate)) * up
    else:
        y = _ACTS[s["act"]](y)
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(s["dtype"])


def _append(s, cache, rows):
    kept = s["slots"] >= 0
    slots, rows = s["slots"][kept].long(), rows[kept]
    if s["block"]:
        cache[0, :, slots] = rows.transpose(0, 1)
    else:
        cache[slots // cache.shape[3], 0, :, slots % cache.shape[3]] = rows


def _rope(s):
    t, nq, nkv, d, rot = (s[x] for x in ("tokens", "nq", "nkv", "d", "rot"))
    x = s["qkv"].float().reshape(t, nq + 2 * nkv, d)
    qk = x[:, :nq + nkv]
    if s["norm"]:
        gain = torch.cat([g.float().expand(n, d) for g, n in zip(s["gains"], (nq, nkv))])
        qk = qk / torch.sqrt((qk * qk).mean(-1, keepdim=True) + s["eps"]) * gain
    at = s["positions"] if s["sections"] else s["positions"][None]
    angle = at.double().T[:, s["axis"]] * s["rates"]                           # [tokens, pairs]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if s["pairs"] == "halves":
        a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    qk = torch.cat([turned, qk[..., rot:]], -1).to(torch.bfloat16)
    _append(s, s["kv"].k, qk[:, nq:])
    _append(s, s["kv"].v, x[:, nq + nkv:].to(torch.bfloat16))
    return [qk[:, :nq], s["kv"].k, s["kv"].v]


def _pages(s):
    b, p, dev = s["block"], s["prefix"] // s["block"], s["lens"].device
    old, new, table, ring = s["lens"].long(), s["new"].long(), s["table"], s["ring"]
    n, head, free = len(ring), s["ends"][0].long(), s["ends"][1].long()
    held, wanted = ((x + b - 1).div(b, rounding_mode="floor").clamp(min=p) for x in (old, new))
    column = torch.arange(table.shape[1], device=dev)
    # blocks given back go behind the free ones, in order of request and place; blocks are taken from the front
    back, take = ((column >= lo[:, None]) & (column < hi[:, None]) for lo, hi in ((wanted, held), (held, wanted)))
    back_at, take_at = ((m.reshape(-1).cumsum(0) - 1).reshape(m.shape) for m in (back, take))
    returned, taken = back.sum(), take.sum()
    dump = torch.cat([ring, ring.new_zeros(1)])      # (a last place for what is not given back)
    dump[torch.where(back, (head + free + back_at) % n, n).reshape(-1)] = table.reshape(-1)
    ring.copy_(dump[:n])
    table.copy_(torch.where(take, ring[(head + take_at) % n], table))
    s["next"].copy_(torch.stack([(head + taken) % n, free + returned - taken, torch.zeros_like(head)]))
    first = torch.cat([old.new_zeros(1), (new - old).clamp(min=0).cumsum(0)])
    i = torch.arange(s["most_tokens"], device=dev)
    seq = torch.searchsorted(first, i, right=True) - 1
    real = i < first[-1]
    seq = torch.where(real, seq, 0)
    at = old[seq] + i - first[seq]
    slot = table[seq, torch.where(real, at, 0).div(b, rounding_mode="floor")].long() * b + at % b
    out = [torch.where(real, x, fill).to(torch.int32) for x, fill in ((slot, -1), (at, 0), (seq, -1))]
    return [table, ring, s["next"], *out, first.to(torch.int32)]


def run(state):
    s = state
    if own:
        import persistent_megakernel_decode_sm_gb300 as mk
        if s["op"] == "adapted":
            return mk.adapted_linear(s["x"], s["w"], (s["down"], s["up"], s["scale"]), s["index"], bias=s["b"],
                                     activation=s["act"] or None, residual=s["r"], out_dtype=s["dtype"])
        if s["op"] == "rope":
            q = mk.rope_append(s["qkv"], s["kv"], s["positions"], s["slots"], s["freqs"], sections=s["parts"] if s["sections"] else None,
                               neighbours=s["pairs"] == "neighbours", q_gain=s["gains"][0], k_gain=s["gains"][1], eps=s["eps"])
            return [q, s["kv"].k, s["kv"].v]
        out = mk.assign_pages(s["ring"], s["ends"], s["table"], s["lens"], s["new"], s["block"], s["most_tokens"],
                              shared_prefix=s["prefix"], ends_out=s["next"])
        return [s["table"], s["ring"], s["next"], *out]
    return {"adapted": _adapted, "rope": _rope, "pages": _pages}[s["op"]](s)


def exact(case, seed):
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    if case["op"] == "adapted":
        x, index = s["x"].double(), s["index"].tolist()
        y = x @ s["w"].double().T
        for a in sorted(set(index) - {-1}):
            rows = torch.tensor([i for i, v in enumerate(index) if v == a], device="cuda")
            y[rows] += s["scale"][a].double() * (x[rows] @ s["down"][a].double().T @ s["up"][a].double().T)
        if s["b"] is not None:
            y += s["b"].double()
        if case["act"] == "swiglu":
            y = y[:, :case["n"]] * torch.sigmoid(y[:, :case["n"]]) * y[:, case["n"]:]
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        return y if s["r"] is None else y + s["r"].double()
    t, nq, nkv, d, rot = (case[x] for x in ("tokens", "nq", "nkv", "d", "rot"))
    x = s["qkv"].double().reshape(t, nq + 2 * nkv, d)
    place = s["positions"].reshape(-1, t).double()
    heads, pair = [], 0
    turn = torch.empty(t, rot // 2, dtype=torch.complex128, device="cuda")
    for axis, n in enumerate(_sections(case)):
        for _ in range(n):
            turn[:, pair] = torch.exp(1j * place[axis] * s["theta"] ** (-2.0 * pair / rot))
            pair += 1
    low, high = (slice(0, rot // 2), slice(rot // 2, rot)) if case["pairs"] == "halves" else (slice(0, rot, 2), slice(1, rot, 2))
    for h in range(nq + nkv):
        y = x[:, h].clone()
        if case["norm"]:
            y *= (y.square().mean(1, keepdim=True) + s["eps"]).rsqrt() * s["gains"][h >= nq].double()
        z = torch.complex(y[:, low], y[:, high]) * turn
        y[:, low], y[:, high] = z.real, z.imag
        heads.append(y)
    kept = (s["slots"] >= 0).nonzero().reshape(-1)
    slots = s["slots"][kept].long()
    out = [torch.stack(heads[:nq], 1)]
    for c, rows in ((s["kv"].k, heads[nq:]), (s["kv"].v, list(x[:, nq + nkv:].unbind(1)))):
        c = c.double()
        for g in range(nkv):
            if case["block"]:
                c[0, g].index_copy_(0, slots, rows[g][kept])
            else:
                size = c.shape[3]
                c[slots // size, 0, g, slots % size] = rows[g][kept]
        out.append(c)
    return out
