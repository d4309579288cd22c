"""Workloads of the prompt-side operators: the linear map with a fused epilogue, attention of query
tokens over the decode KV cache (causal, sliding window with sinks), and the same attention for a
batch whose sequences share a long prefix.

``listed()`` names the workloads, ``draw(rng)`` makes one more of the same ranges, ``prepare`` builds
the inputs on the GPU, ``run`` makes one pass.  With ``own`` false a pass is the operators' plain form
in elementary torch operations (32-bit arithmetic, one rounding at the end); with ``own`` true it
calls the library.  ``exact`` is the operators' definition in 64 bits.

Shapes come from this repository's configurations (the tiny, 1B and 8B decoder shapes, KV lengths
512 to 8192, batches of 8) and go beyond them where an operator's range does.
"""
import math
import random

import numpy as np
import torch

own = False

SCORE_CAP = 1 << 31          # scores of one attention pass in the plain form, at most (elements)
FLOP_CAP = 5.0e11          # a drawn pass costs no more than the largest listed one


def listed():
    return [
        # one token through the attention output projection of the 1B shape, added to the residual
        dict(name="linear_token", op="linear", rows=1, k=2048, n=2048, act="", bias=False, residual="f32", out="f32", pad=0),
        # a batch of 8 tokens through gate/up with SwiGLU (1B): the weights' bytes are the floor
        dict(name="linear_batch8_swiglu", op="linear", rows=8, k=2048, n=8192, act="swiglu", bias=False, residual="", out="bf16", pad=0),
        # odd sizes, rows that are views of a wider buffer, bias and GELU (the tiny shape's row length)
        dict(name="linear_odd_gelu", op="linear", rows=333, k=688, n=1001, act="gelu", bias=True, residual="bf16", out="bf16", pad=24),
        # a 512-token prompt through the down projection (1B), residual stream in 32 bits
        dict(name="linear_prompt_down", op="linear", rows=512, k=8192, n=2048, act="", bias=False, residual="f32", out="f32", pad=0),
        # a 4096-token prompt chunk through gate/up with SwiGLU (1B): the tensor cores are the floor
        dict(name="linear_prompt_swiglu", op="linear", rows=4096, k=2048, n=8192, act="swiglu", bias=False, residual="", out="bf16", pad=0),
        # one token over a cache of 8192 positions (1B)
        dict(name="attend_token_8192", op="attend", batch=1, nq=32, nkv=8, d=64, q_min=1, q_max=1, kv_min=8192, kv_max=8192,
             window=0, sinks=0, prefix=0, block=0, lens=0),
        # eight single tokens far along, each seeing 4 sinks and a window of 4096 (8B heads)
        dict(name="attend_tokens_window", op="attend", batch=8, nq=32, nkv=8, d=128, q_min=1, q_max=1, kv_min=9001, kv_max=16384,
             window=4096, sinks=4, prefix=0, block=0, lens=1),
        # a whole 4096-token prompt, causal (1B)
        dict(name="attend_prompt_4096", op="attend", batch=1, nq=32, nkv=8, d=64, q_min=4096, q_max=4096, kv_min=4096, kv_max=4096,
             window=0, sinks=0, prefix=0, block=0, lens=0),
        # a 2048-token chunk of a long prompt with window and sinks (8B heads), paged cache
        dict(name="attend_chunk_window", op="attend", batch=1, nq=32, nkv=8, d=128, q_min=2048, q_max=2048, kv_min=16000, kv_max=16000,
             window=4096, sinks=4, prefix=0, block=512, lens=0),
        # a ragged batch of short and long chunks, 3 heads per KV head, paged in blocks of 48 positions
        dict(name="attend_ragged_paged", op="attend", batch=5, nq=12, nkv=4, d=64, q_min=1, q_max=777, kv_min=1, kv_max=2111,
             window=300, sinks=7, prefix=0, block=48, lens=2),
        # 8 single tokens behind one 8192-position prefix (1B), each with a short tail of its own
        dict(name="prefix_tokens_8", op="attend", batch=8, nq=32, nkv=8, d=64, q_min=1, q_max=1, kv_min=8200, kv_max=8448,
             window=0, sinks=0, prefix=8192, block=0, lens=3),
        # 32 short questions of up to 24 tokens behind one 16384-position prefix (8B heads), paged
        dict(name="prefix_questions_32", op="attend", batch=32, nq=32, nkv=8, d=128, q_min=3, q_max=24, kv_min=16411, kv_max=16600,
             window=0, sinks=0, prefix=16384, block=256, lens=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.45:
        while True:
            act = rng.choice(["", "", "silu", "gelu", "swiglu"])
            c = dict(op="linear", rows=_log(rng, 1, 4096), k=8 * _log(rng, 8, 2048), n=_log(rng, 16, 16384), act=act,
                     bias=rng.random() < 0.5, residual=rng.choice(["", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                     pad=rng.choice([0, 0, 8, 40]))
            if work(c)["flops"] <= FLOP_CAP / 2:
                return c
    prefixed = rng.random() < 0.4
    while True:
        nkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
        c = dict(op="attend", batch=_log(rng, 2 if prefixed else 1, 48), nq=nkv * group, nkv=nkv, d=rng.choice([32, 64, 128]),
                 q_min=1, q_max=_log(rng, 1, 4096), kv_min=1, kv_max=_log(rng, 16, 32768), window=0, sinks=0, prefix=0,
                 block=rng.choice([0, 0, 16, 128, 256]), lens=rng.randrange(1 << 20))
        if rng.random() < 0.5:
            c["q_max"] = 1
        if prefixed:
            c["q_max"] = min(c["q_max"], 64)
            c["prefix"] = _log(rng, 64, 16384)
            c["kv_min"] = c["prefix"] + c["q_max"]
            c["kv_max"] = c["kv_min"] + _log(rng, 1, 512)
        else:
            c["q_max"] = min(c["q_max"], c["kv_max"])
            if rng.random() < 0.5:
                c["window"], c["sinks"] = _log(rng, 1, 8192), rng.choice([0, 1, 4, 64, 200])
        if c["batch"] * c["nq"] * c["q_max"] * c["kv_max"] <= SCORE_CAP // 2 and c["batch"] * nkv * c["kv_max"] * c["d"] <= 1 << 29:
            return c


def lengths(case):
    """Query tokens and cached positions (the query tokens' own included) of each sequence."""
    r = random.Random(case["lens"])
    kv = [r.randint(case["kv_min"], case["kv_max"]) for _ in range(case["batch"])]
    ql = [min(r.randint(case["q_min"], case["q_max"]), k) for k in kv]
    return ql, kv


def work(case):
    if case["op"] == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        f = 2 if case["act"] == "swiglu" else 1
        size = {"": 0, "bf16": 2, "f32": 4}
        return {"bytes": 2 * m * k + 2 * f * n * k + (2 * f * n if case["bias"] else 0) + m * n * (size[case["residual"]] + size[case["out"]]),
                "flops": 2 * f * m * n * k}
    d, nq, nkv, w, s, p = (case[x] for x in ("d", "nq", "nkv", "window", "sinks", "prefix"))
    pairs, rows = 0, p
    for n, length in zip(*lengths(case)):
        t = np.arange(length - n, length)
        pairs += int((t + 1 if w == 0 else np.minimum(t + 1, w) + np.clip(t + 1 - w, 0, s)).sum())
        low = max(0, length - n - w + 1) if w else 0
        rows += length - p if p else length - low + min(s, low)
    return {"bytes": sum(lengths(case)[0]) * nq * d * 4 + rows * nkv * d * 4, "flops": 4 * d * nq * pairs}


def _normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


class Cache:
    """K and V as the decoder keeps them: [batch, layers, heads, positions, d], or the pool of a paged cache."""

    def __init__(self, k, v):
        self.k, self.v = k, v


def prepare(case, seed):
    s = dict(case)
    if case["op"] == "linear":
        m, k, n, pad = case["rows"], case["k"], case["n"], case["pad"]
        f = 2 if case["act"] == "swiglu" else 1
        s["x"] = _normal((m, k + pad), seed * 8 + 1).to(torch.bfloat16)[:, :k]
        s["w"] = _normal((f * n, k), seed * 8 + 2, 1.0 / math.sqrt(k)).to(torch.bfloat16)   # pre-activations of about 1
        s["b"] = _normal((f * n,), seed * 8 + 3, 0.5).to(torch.bfloat16) if case["bias"] else None
        kind = {"bf16": torch.bfloat16, "f32": torch.float32}
        s["r"] = _normal((m, n + pad), seed * 8 + 4).to(kind[case["residual"]])[:, :n] if case["residual"] else None
        s["dtype"] = kind[case["out"]]
        return s
    ql, kvl = lengths(case)
    batch, nkv, d, block, prefix = (case[x] for x in ("batch", "nkv", "d", "block", "prefix"))
    top = max(kvl)
    s["ql"], s["kvl"] = ql, kvl
    s["q"] = _normal((sum(ql), case["nq"], d), seed * 8 + 1, 1.5).to(torch.bfloat16)
    if block:   # a pool of blocks in shuffled order; a shared prefix's whole blocks appear in every table
        per, common = -(-top // block), prefix // block
        total = common + batch * (per - common)
        order = torch.randperm(total, generator=torch.Generator().manual_seed(seed), dtype=torch.int64)
        table = torch.empty((batch, per), dtype=torch.int64)
        table[:, :common] = order[:common]
        table[:, common:] = order[common:].reshape(batch, per - common)
        s["table"] = table.to(device="cuda", dtype=torch.int32)
        s["blocks"] = total
        shape = (1, nkv, total * block, d)
    else:
        shape = (batch, 1, nkv, top, d)
    s["kv"] = Cache(_normal(shape, seed * 8 + 2).to(torch.bfloat16), _normal(shape, seed * 8 + 3).to(torch.bfloat16))
    if block and prefix % block:   # the block that the prefix ends in: every sequence has its own copy of the prefix's part
        at, cut = (table[:, prefix // block] * block).tolist(), prefix % block
        for t in (s["kv"].k, s["kv"].v):
            for a in at[1:]:
                t[:, :, a:a + cut] = t[:, :, at[0]:at[0] + cut]
    # where each query token stands: its row in a padded batch, and the position it has
    first = torch.tensor([0] + ql).cumsum(0)[:-1]
    most = max(ql)
    step = torch.arange(most)
    n = torch.tensor(ql)[:, None]
    s["pick"] = (first[:, None] + torch.minimum(step, n - 1)).cuda()              # [batch, most]: rows of q
    s["keep"] = (step < n).reshape(-1).nonzero().reshape(-1).cuda()               # rows of the padded output
    s["at"] = (torch.tensor(kvl)[:, None] - n + step).cuda()                      # positions
    return s


_ACTS = {"": lambda y: y, "silu": lambda y: y / (1 + torch.exp(-y)), "gelu": lambda y: 0.5 * y * (1 + torch.erf(y / math.sqrt(2.0)))}


def _linear(s, t):
    y = s["x"].to(t) @ s["w"].to(t).T
    if s["b"] is not None:
        y = y + s["b"].to(t)
    if s["act"] == "swiglu":
        gate, up = y[:, :s["n"]], y[:, s["n"]:]
        y = gate / (1 + torch.exp(-gate)) * up
    else:
        y = _ACTS[s["act"]](y)
    return y if s["r"] is None else y + s["r"].to(t)


def _rows(s, cache, top):
    """[batch, heads, top, d]: each sequence's cached rows in order of position."""
    if s["block"]:
        at = torch.arange(top, device=cache.device)
        slot = s["table"][:, at // s["block"]].long() * s["block"] + at % s["block"]
        return cache[0][:, slot].transpose(0, 1)
    rows = cache[:, 0, :, :top]
    p = s["prefix"]   # a contiguous cache holds a shared prefix once, in sequence 0's rows
    return torch.cat([rows[:1, :, :p].expand(rows.shape[0], -1, -1, -1), rows[:, :, p:]], 2) if p else rows


def _seen(s, at, top):
    """[..., top]: whether the query at each position sees each cached position."""
    key = torch.arange(top, device=at.device)
    at = at[..., None]
    seen = key <= at
    if s["window"]:
        seen = seen & ((key > at - s["window"]) | (key < s["sinks"]))
    return seen


def _attend(s):
    top, d, nkv = max(s["kvl"]), s["d"], s["nkv"]
    k, v = (_rows(s, c, top).float() for c in (s["kv"].k, s["kv"].v))
    q = s["q"].float()[s["pick"]]                                               # [batch, most, heads, d]
    b, n = s["pick"].shape
    q = q.reshape(b, n, nkv, -1, d).permute(0, 2, 3, 1, 4).reshape(b, nkv, -1, d)
    score = (q @ k.transpose(2, 3) * (1 / math.sqrt(d))).reshape(b, nkv, -1, n, top)
    score = score.masked_fill(~_seen(s, s["at"], top)[:, None, None], -math.inf)
    high = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(high > -math.inf, high, 0.0))
    o = p.reshape(b, nkv, -1, top) @ v
    total = p.sum(-1).reshape(b, nkv, -1, 1)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.reshape(b, nkv, -1, n, d).permute(0, 3, 1, 2, 4).reshape(b * n, s["nq"], d)
    return o[s["keep"]]


def run(state):
    s = state
    if own:
        import persistent_megakernel_decode_sm_gb300 as mk
        if s["op"] == "linear":
            return mk.linear(s["x"], s["w"], bias=s["b"], activation=s["act"] or None, residual=s["r"], out_dtype=s["dtype"])
        pages = (s["table"], s["block"], s["blocks"]) if s["block"] else None
        return mk.attend(s["q"], s["kv"], s["ql"], s["kvl"], window=s["window"], sinks=s["sinks"], shared_prefix=s["prefix"],
                         pages=pages)
    if s["op"] == "linear":
        return _linear(s, torch.float32).to(s["dtype"])
    return _attend(s).to(torch.bfloat16)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "linear":
        out = []
        for a in range(0, case["rows"], 1024):   # in 64 bits, a piece of the rows at a time
            piece = dict(s, x=s["x"][a:a + 1024], r=None if s["r"] is None else s["r"][a:a + 1024])
            y = piece["x"].double() @ s["w"].double().T
            if s["b"] is not None:
                y += s["b"].double()
            if case["act"] == "swiglu":
                g = y[:, :case["n"]]
                y = g * torch.sigmoid(g) * y[:, case["n"]:]
            elif case["act"] == "silu":
                y = y * torch.sigmoid(y)
            elif case["act"] == "gelu":
                y = y * torch.special.ndtr(y)
            if s["r"] is not None:
                y = y + piece["r"].double()
            out.append(y)
        return torch.cat(out)
    group, d, block, prefix = case["nq"] // case["nkv"], case["d"], case["block"], case["prefix"]
    out, row = [], 0
    for b, (n, length) in enumerate(zip(s["ql"], s["kvl"])):
        pos = torch.arange(length, device="cuda")
        if block:
            slot = s["table"][b, pos // block].long() * block + pos % block
            k, v = s["kv"].k[0][:, slot], s["kv"].v[0][:, slot]
        else:
            own_rows = [torch.cat([c[0, 0, :, :prefix], c[b, 0, :, prefix:length]], 1) for c in (s["kv"].k, s["kv"].v)]
            k, v = own_rows
        t = torch.arange(length - n, length, device="cuda")[:, None]
        hidden = pos > t
        if case["window"]:
            hidden |= (pos <= t - case["window"]) & (pos >= case["sinks"])
        heads = []
        for h in range(case["nq"]):
            score = s["q"][row:row + n, h].double() @ k[h // group].double().T / math.sqrt(d)
            score[hidden] = -math.inf
            heads.append(torch.softmax(score, -1) @ v[h // group].double())
        out.append(torch.stack(heads, 1))
        row += n
    return torch.cat(out)
