"""The operators of a serving step run together, as they are used: pages assigned on the device, the projection with every
request's adapter, norms and rotation with the append through those slots, attention over the block table that they made, and the
output projection added to the residual stream; and the decoder on a table made so.

The step is compared with the same chain in 64 bits that rounds where the operators round (q, k, v and attention's output to
bf16).  Each of those roundings is off by at most 2^-8 of a value, attention's weights by 2^-9 of theirs; the residual stream itself is
fp32, so a step's output is off by at most 5 2^-8 of the projected part's norm."""
import gc
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from workload import KVCache, get_workload, make_weights, token_ids, empty_kv  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def nothing_left_behind():
    """Tracebacks of refused calls hold tensors in cycles: they go before the next module's tests look at the memory."""
    yield
    gc.collect()


def randn(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Layer:
    def __init__(self, nq, nkv, d, hidden, adapters, rank, axes=None):
        self.nq, self.nkv, self.d, self.axes = nq, nkv, d, axes
        width = (nq + 2 * nkv) * d
        self.wqkv, self.wo = randn((width, hidden), 1, hidden ** -0.5), randn((hidden, nq * d), 2, (nq * d) ** -0.5)
        self.qkv_adapters = (randn((adapters, rank, hidden), 3, hidden ** -0.5), randn((adapters, width, rank), 4, rank ** -0.5),
                             randn((adapters,), 5, 0.3, F32))
        self.o_adapters = (randn((adapters, rank, nq * d), 6, (nq * d) ** -0.5), randn((adapters, hidden, rank), 7, rank ** -0.5))
        self.gains = [(1 + randn((d,), 8 + i, 0.1, F32)).to(BF) for i in range(2)]
        self.freqs = 500000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)

    def step(self, x, kv, pages, slots, positions, adapter, q_lens, kv_lens, status=None):
        """x fp32 [tokens, hidden], the residual stream: one attention block of a decoder layer."""
        xb = x.to(BF)
        qkv = mk.adapted_linear(xb, self.wqkv, self.qkv_adapters, adapter, out_dtype=F32, status=status)
        at = positions if self.axes is None else positions.expand(len(self.axes), -1).contiguous()
        q = mk.rope_append(qkv, kv, at, slots, self.freqs, sections=self.axes, q_gain=self.gains[0], k_gain=self.gains[1], status=status)
        o = mk.attend(q, kv, q_lens, kv_lens, pages=pages, status=status)
        return mk.adapted_linear(o.reshape(len(x), -1), self.wo, self.o_adapters, adapter, residual=x, out_dtype=F32, status=status)

    def reference(self, x, history, positions, sequences, adapter):
        """The same in 64 bits: history[b] is the list of (k, v) rows of sequence b, grown by this call's tokens."""
        def adapted(a, w, ad):
            y = a @ w.double().T
            for r, i in enumerate(adapter.tolist()):
                if i >= 0:
                    f = 1.0 if len(ad) == 2 else ad[2][i].double()
                    y[r] += f * (ad[1][i].double() @ (ad[0][i].double() @ a[r]))
            return y
        nq, nkv, d = self.nq, self.nkv, self.d
        h = adapted(x.to(BF).double(), self.wqkv, self.qkv_adapters).reshape(len(x), nq + 2 * nkv, d)
        for lo, hi, g in ((0, nq, 0), (nq, nq + nkv, 1)):
            h[:, lo:hi] *= (h[:, lo:hi].square().mean(-1, keepdim=True) + 1e-5).rsqrt() * self.gains[g].double()
        angle = positions.double()[:, None] * self.freqs.cuda()
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = h[:, :nq + nkv, :d // 2].clone(), h[:, :nq + nkv, d // 2:].clone()
        h[:, :nq + nkv, :d // 2], h[:, :nq + nkv, d // 2:] = a * c - b * s, a * s + b * c
        h = h.to(BF).double()
        out = torch.zeros(len(x), nq, d, dtype=torch.float64, device="cuda")
        for r, b in enumerate(sequences.tolist()):
            history[b].append((h[r, nq:nq + nkv], h[r, nq + nkv:]))
            k, v = (torch.stack([row[i] for row in history[b]], 1).repeat_interleave(nq // nkv, 0) for i in range(2))
            out[r] = torch.einsum("hp,hpd->hd", torch.softmax(torch.einsum("hd,hpd->hp", h[r, :nq], k) / math.sqrt(d), -1), v)
        return adapted(out.to(BF).double().reshape(len(x), -1), self.wo, self.o_adapters) + x.double()


@pytest.mark.parametrize("nq,nkv,d,hidden,rank,axes", [(4, 2, 64, 256, 8, None), (8, 2, 128, 512, 24, [16, 24, 24])])
def test_steps_of_a_changing_batch(nq, nkv, d, hidden, rank, axes):
    batch, block, columns, n_blocks, adapters = 6, 16, 12, 60, 4
    layer = Layer(nq, nkv, d, hidden, adapters, rank, axes)
    kv = KVCache(*(torch.full((1, nkv, n_blocks * block, d), 9.0, dtype=BF, device="cuda") for _ in range(2)))
    order = list(range(n_blocks))
    random.Random(1).shuffle(order)
    ring, ends, table = i32(order), i32([0, n_blocks, 0]), torch.full((batch, columns), -1, dtype=torch.int32, device="cuda")
    lens, status = [0] * batch, torch.zeros(1, dtype=torch.int32, device="cuda")
    history = [[] for _ in range(batch)]
    # prompts, single tokens, a request that ends and another that takes its place, mixed chunks
    for number, new in enumerate(([33, 5, 100, 0, 1, 16], [34, 6, 101, 20, 2, 17], [35, 0, 102, 21, 40, 0], [36, 9, 103, 60, 41, 30])):
        q_lens = [max(b - a, 0) for a, b in zip(lens, new)]
        tokens = sum(q_lens)
        slots, positions, sequences, first = mk.assign_pages(ring, ends, table, i32(lens), i32(new), block, tokens, status=status)
        for b, n in enumerate(new):
            if n == 0:
                history[b] = []
        x = randn((tokens, hidden), 50 + number, dtype=F32)
        adapter = i32([-1, 0, 1, 2, 3, 1])[sequences.long()]
        got = layer.step(x, kv, (table, block, n_blocks), slots, positions, adapter, q_lens, [n if n else 0 for n in new], status)
        want = layer.reference(x, history, positions, sequences, adapter)
        off = (got.double() - want).norm() / (want - x.double()).norm()
        assert status.item() == 0 and off <= 5 * 2.0 ** -8, off.item()
        assert first.tolist() == [sum(q_lens[:i]) for i in range(batch + 1)]
        lens = list(new)


def test_a_captured_step_of_a_padded_batch():
    # a graph for up to 8 tokens, replayed with other lengths: attention is not part of it (its lengths are the host's)
    nq, nkv, d, hidden, batch, block, n_blocks = 4, 2, 64, 256, 4, 8, 40
    layer = Layer(nq, nkv, d, hidden, 3, 16)
    kv = KVCache(*(torch.zeros((1, nkv, n_blocks * block, d), dtype=BF, device="cuda") for _ in range(2)))
    ring, ends, table = i32(list(range(n_blocks))), i32([0, n_blocks, 0]), torch.full((batch, 8), -1, dtype=torch.int32, device="cuda")
    lens, new, names = i32([0] * batch), i32([0] * batch), i32([0, 1, 2, -1])
    x = torch.zeros((8, hidden), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        slots, positions, sequences, _ = mk.assign_pages(ring, ends, table, lens, new, block, 8, status=status)
        adapter = torch.where(sequences >= 0, names[sequences.clamp(min=0).long()], -1)
        qkv = mk.adapted_linear(x.to(BF), layer.wqkv, layer.qkv_adapters, adapter, out_dtype=F32)
        q = mk.rope_append(qkv, kv, positions, slots, layer.freqs, q_gain=layer.gains[0], k_gain=layer.gains[1])
        lens.copy_(new)
    history, old = [[] for _ in range(batch)], [0] * batch
    for number, wanted in enumerate(([3, 1, 0, 2], [4, 2, 1, 3], [5, 0, 5, 4], [6, 8, 0, 4])):
        for b, n in enumerate(wanted):
            if n == 0:
                history[b] = []
        new.copy_(i32(wanted))
        x.copy_(randn(x.shape, number, dtype=F32))
        before = kv.k.clone()
        g.replay()
        torch.cuda.synchronize()
        real = sum(max(b - a, 0) for a, b in zip(old, wanted))
        if real > 8:                                                        # the last step's 1 + 8 tokens: more than the graph has rows for
            assert number == 3 and status.item() == mk.MK_ERR_CAPACITY and (slots == -1).all() and torch.equal(kv.k, before)
            break
        assert (sequences[real:] == -1).all() and (slots[real:] == -1).all() and status.item() == 0
        changed = (kv.k != before).any(-1).any(1)[0].nonzero().reshape(-1).tolist()
        assert changed == sorted(slots[:real].tolist())                     # padded rows store nothing
        layer.reference(x[:real], history, positions[:real], sequences[:real], adapter[:real])
        for r in range(real):
            want = history[sequences[r].item()][positions[r].item()][0]
            got = kv.k[0, :, slots[r].item()].double()
            assert (got - want).norm() <= 2 * 2.0 ** -8 * want.norm()
        old = wanted


def test_the_decoder_on_a_table_made_on_the_device():
    wl = get_workload("tiny")
    cfg = wl.cfg
    sms = mk.device_sm_count()
    block = mk.Schedule(cfg, sms).attn_chunk
    columns, n_blocks = -(-cfg.max_seq // block), 7
    weights = make_weights(cfg, seed=0, device="cuda")
    plain = empty_kv(cfg, device="cuda")
    pool = KVCache(*(torch.zeros((cfg.n_layers, cfg.n_kv_heads, n_blocks * block, cfg.head_dim), dtype=BF, device="cuda") for _ in range(2)))
    table = torch.full((cfg.batch, columns), -1, dtype=torch.int32, device="cuda")
    mk.assign_pages(i32([5, 2, 6, 0, 1, 4, 3]), i32([2, 7, 0]), table, i32([0] * cfg.batch), i32([cfg.max_seq] * cfg.batch), block,
                    cfg.batch * cfg.max_seq)
    assert table[0].tolist() == [6, 0, 1, 4, 3, 5, 2][:columns]
    a = mk.Decoder(mk.Schedule(cfg, sms), weights, plain)
    b = mk.Decoder(mk.Schedule(cfg, sms), weights, pool, pages=(table, block, n_blocks))
    prompt = token_ids(cfg, wl.prompt_len, seed=0, tag="prompt")
    for dec in (a, b):
        dec.prefill([prompt[:-1]])
    tokens, pos = [prompt[-1]], [wl.prompt_len - 1]
    for _ in range(4):
        ta, tb = a.step(tokens, pos), b.step(tokens, pos)
        assert ta == tb and torch.equal(a.logits, b.logits)
        tokens, pos = ta, [pos[0] + 1]
    a.close()
    b.close()


class Python:
    """In the place of the C call module: leaves every call to Python."""
    linear = attend = adapted_linear = rope_append = assign_pages = staticmethod(lambda *a: None)


def test_c_and_python_calls_agree_and_keep_nothing(monkeypatch):
    import sys
    x, w, index = randn((5, 64), 1), randn((96, 64), 2), i32([0, 2, -1, 1, 0])
    down, up, scale = randn((3, 8, 64), 3), randn((3, 96, 8), 4), randn((3,), 5, dtype=F32)
    kv = KVCache(*(randn((2, 1, 2, 16, 16), 6 + i) for i in range(2)))
    pool = KVCache(*(randn((1, 2, 32, 16), 8 + i) for i in range(2)))
    qkv, at, slots, f = randn((5, 96), 10), i32([3, 1, 4, 1, 5]), i32([0, 9, 17, -1, 31]), torch.linspace(1, 0.1, 8, dtype=torch.float64)
    gain, status, ws = randn((16,), 11), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    ring, ends, spare, table, lens, new = i32(list(range(20))), i32([4, 12, 0]), i32([0, 0, 0]), i32([[0, 1, -1], [2, -1, -1]]), i32([12, 3]), i32([17, 4])
    out4 = tuple(i32([7] * n) for n in (9, 9, 9, 3))
    ad = (down, up, scale)
    calls = [lambda: mk.adapted_linear(x, w, ad, index), lambda: mk.adapted_linear(x, w, (down, up), index, activation="silu", out_dtype=F32, workspace=ws),
             lambda: mk.adapted_linear(x, w, [down, up, None], index, activation="swiglu", residual=x[:, :48], status=status), lambda: mk.adapted_linear(x[:0], w, ad, index[:0]),
             lambda: mk.rope_append(qkv, kv, at, slots, f), lambda: mk.rope_append(qkv.float(), pool, at, slots, f[:0], q_gain=gain, k_gain=gain, neighbours=True, status=status),
             lambda: mk.rope_append(qkv, pool, torch.stack([at, at]), slots, f, sections=[3, 5], eps=1e-3), lambda: mk.rope_append(qkv, pool, torch.stack([at, at]), slots, f, sections=(8, 0), k_gain=gain),
             lambda: mk.assign_pages(ring, ends, table, lens, new, 8, 9, ends_out=spare), lambda: mk.assign_pages(ring, ends, table, lens, new, 8, 9, ends_out=spare, out=out4, status=status),
             lambda: mk.assign_pages(ring, ends, table, lens, new, 8, 9, ends_out=spare, shared_prefix=8, out=list(out4))]
    bad = [lambda: mk.adapted_linear(x, w, ad, index[:4]), lambda: mk.adapted_linear(x, w, (down[:, :7], up, scale), index), lambda: mk.adapted_linear(x, w, (down, up.mT, scale), index),
           lambda: mk.adapted_linear(x, w, (down, up, scale[:2]), index), lambda: mk.adapted_linear(x, w, ad, index, workspace=ws[:64]), lambda: mk.adapted_linear(x, w, ad, index, workspace=ws.cpu()),
           lambda: mk.adapted_linear(x, w, ad, index, activation="relu"), lambda: mk.adapted_linear(x, w, ad, index.long()),
           lambda: mk.rope_append(qkv, kv, at[:4], slots, f), lambda: mk.rope_append(qkv, kv, at, slots, f.float()), lambda: mk.rope_append(qkv, kv, at, slots, f[:7]),
           lambda: mk.rope_append(qkv, pool, torch.stack([at, at]), slots, f, sections=[3, 4]), lambda: mk.rope_append(qkv, pool, at, slots, f, sections=[8]), lambda: mk.rope_append(qkv, kv, at, slots, f, layer=1),
           lambda: mk.rope_append(qkv, kv, at, slots, f, eps=-1.0), lambda: mk.rope_append(qkv[:, :64], kv, at, slots, f), lambda: mk.rope_append(qkv, kv, at, slots, f, q_gain=gain[:8]),
           lambda: mk.assign_pages(ring, ends, table, lens, new, 0, 9), lambda: mk.assign_pages(ring, ends, table[:1], lens, new, 8, 9), lambda: mk.assign_pages(ring, ends[:2], table, lens, new, 8, 9),
           lambda: mk.assign_pages(ring, ends, table, lens, new, 8, 9, out=out4[:3]), lambda: mk.assign_pages(ring, ends, table, lens, new, 8, 8, out=out4)]

    def run(call):
        try:
            y = call()
            return [t.clone() for t in (y if isinstance(y, tuple) else (y, kv.k, kv.v, pool.k, pool.v))]
        except (ValueError, mk.MkError) as e:
            return str(e)

    first = [run(c) for c in calls]
    taken = [run(c) for c in calls]
    refused = [run(c) for c in bad]
    assert all(isinstance(t, list) for t in first) and all(isinstance(r, str) for r in refused)
    with monkeypatch.context() as m:
        m.setattr(mk, "_fast", Python)
        for c, t in zip(calls, taken):
            assert all(torch.equal(a, b) for a, b in zip(run(c), t))
        assert [run(c) for c in bad] == refused
    held = (x, w, index, down, up, scale, kv.k, qkv, at, slots, f, gain, status, ws, ring, ends, spare, table, lens, new, *out4)
    del first, taken
    gc.collect()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in held]
    for _ in range(60):
        for c in calls + bad:
            run(c)
    gc.collect()
    assert (torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in held]) == before
