"""The definition of the cache attention in 64 bits, for the GPU tests, and the error a kernel may make.

A kernel takes scores in fp32 (d products of bf16 values, error at most d 2^-23 of their absolute
sum), rounds its softmax weights to bf16 (half a step, 2^-8 relative) and its output to bf16 (2^-8
relative); exponentials, running sums and a merge of parts add less than 2^-16 together.  At head
dims other than 64 the rows are divided by the sum of the rounded weights: with weights p_i (1 + e_i),
|e_i| <= 2^-8, and e their mean under p, the output is off by sum p_i |e_i - e| |v_i| / (1 + e), where
|e_i - e| <= 2 2^-8 (two keys, one of them with a small v, come near it): twice the bound of exact sums."""
import math

import torch


def visible(t, pos, window, sinks):
    see = pos <= t
    if window:
        see &= (pos > t - window) | (pos < sinks)
    return see


def attend_reference(q, kv, q_lens, kv_lens, layer=0, window=0, sinks=0, shared_prefix=0, scale=None, pages=None):
    """(out, bound): both [tokens, heads, d] in fp64; bound is the largest error the formats allow."""
    tokens, nq, d = q.shape
    nkv = kv.k.shape[-3]
    group = nq // nkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.zeros((tokens, nq, d), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    row = 0
    weights = 2.0 ** -8 if d == 64 else 2.0 ** -7 + 2.0 ** -15   # (the last term: 1 / (1 + e))
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        if n == 0:
            continue
        pos = torch.arange(length, device=q.device)
        src = torch.where(pos < shared_prefix, 0, b)
        if pages is None:
            k, v = (c[src, layer, :, pos].transpose(0, 1) for c in (kv.k, kv.v))
            ok = torch.ones(length, dtype=torch.bool, device=q.device)
        else:
            table, block, blocks = pages
            e = table[src, pos // block].long()
            ok = (e >= 0) & (e < blocks)
            slot = torch.where(ok, e, 0) * block + pos % block
            k, v = (c[layer][:, slot] for c in (kv.k, kv.v))
        t = torch.arange(length - n, length, device=q.device)[:, None]
        see = visible(t, pos, window, sinks) & ok
        used = see.any(0)                                   # positions no token sees may hold anything
        for h in range(nq):
            kk = torch.where(used[:, None], k[h // group].double(), 0.0)
            vv = torch.where(used[:, None], v[h // group].double(), 0.0)
            qq = q[row:row + n, h].double()
            s = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
            any_ = see.any(1, keepdim=True)
            p = torch.where(any_, torch.softmax(torch.where(any_, s, 0.0), -1), 0.0)
            o = p @ vv
            ds = (qq.abs() @ kk.abs().T * scale * d * 2.0 ** -23).masked_fill(~see, 0.0).amax(1, keepdim=True) if length else 0.0
            out[row:row + n, h] = o
            bound[row:row + n, h] = 2.0 ** -8 * o.abs() + (weights + 2 * ds + 2.0 ** -16) * (p @ vv.abs()) + 1e-37
        row += n
    return out, bound
