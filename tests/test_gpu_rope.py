"""mk_rope_append against the formula in 64 bits: norms, rotated widths, pairs, axes, positions far along, caches of
both layouts, padded batches.

Tolerance per element: x and gains enter in fp32; cosines and sines are off by at most 2^-20.9 (the special-function unit's bound
on [-pi, pi]) and the rounding of the angle, 2^-22; the arithmetic of the norm and of the rotation is about 12 roundings of 2^-24.
So values are off by at most 2^-19 of the pair's sum before the output's own rounding (half a step of bf16, 2^-8 of the value)."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from workload import KVCache  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def nothing_left_behind():
    """Tracebacks of refused calls hold tensors in cycles: they go before the next module's tests look at the memory."""
    yield
    gc.collect()


def randn(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def freqs_of(rotary, theta=10000.0):
    return theta ** (-2.0 * torch.arange(rotary // 2, dtype=torch.float64) / max(rotary, 1))


def reference(qkv, nq, nkv, d, positions, freqs, sections, neighbours, gains, eps):
    """([tokens, nq + 2 nkv, d] in fp64, bound without the output's rounding)."""
    t, rotary = qkv.shape[0], 2 * len(freqs)
    x = qkv.double().reshape(t, nq + 2 * nkv, d).clone()
    for lo, hi, gain in ((0, nq, gains[0]), (nq, nq + nkv, gains[1])):
        if gain is not None:
            x[:, lo:hi] *= (x[:, lo:hi].square().mean(-1, keepdim=True) + eps).rsqrt() * gain.double()
    bound = x.abs() * 2.0 ** -19
    axis = torch.repeat_interleave(torch.arange(len(sections or [1])), torch.tensor(sections or [rotary // 2]))
    at = positions.reshape(-1, t).double()[axis.cuda()]                          # [pairs, tokens]
    angle = (at * freqs.cuda()[:, None]).T[:, None]
    c, s = angle.cos(), angle.sin()
    i = torch.arange(rotary // 2)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + rotary // 2)
    xa, xb = x[:, :nq + nkv, a], x[:, :nq + nkv, b]
    size = (xa.abs() + xb.abs()) * 2.0 ** -19
    x[:, :nq + nkv, a], x[:, :nq + nkv, b] = xa * c - xb * s, xa * s + xb * c
    bound[:, :nq + nkv, a], bound[:, :nq + nkv, b] = size, size
    return x, bound


def check(t, nq, nkv, d, rotary, *, dtype=BF, sections=None, neighbours=False, norm=True, paged=0, sequences=2, layers=1, layer=0, far=0,
          freqs=None, seed=1, slots=None, positions=None, pad=0, eps=1e-5):
    width = (nq + 2 * nkv) * d
    qkv = randn((t, width + pad), seed, 1.5, dtype)[:, :width]
    gains = [(1 + randn((d,), seed + i, 0.1, F32)).to(BF) if norm is True or norm == which else None
             for i, which in ((4, "q"), (5, "k"))]
    freqs = freqs_of(rotary) if freqs is None else freqs
    g = torch.Generator().manual_seed(seed)
    if paged:
        shape = (layers, nkv, (t // paged + 2) * paged, d)
        total = shape[2]
    else:
        shape = (sequences, layers, nkv, t + 3, d)
        total = sequences * (t + 3)
    if slots is None:
        slots = torch.randperm(total, generator=g)[:t].to(torch.int32).cuda()
    if positions is None:
        positions = (torch.randint(0, 5000, (len(sections), t) if sections else (t,), generator=g) + far).to(torch.int32).cuda()
    kv = KVCache(randn(shape, seed + 8), randn(shape, seed + 9))
    before = [c.clone() for c in (kv.k, kv.v)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = mk.rope_append(qkv, kv, positions, slots, freqs, layer=layer, sections=sections, neighbours=neighbours, q_gain=gains[0],
                       k_gain=gains[1], eps=eps, status=status)
    want, bound = reference(qkv, nq, nkv, d, positions, freqs, sections, neighbours, gains, eps)
    bound = bound + 2.0 ** -8 * want.abs() + 1e-37
    assert q.shape == (t, nq, d) and q.dtype == BF
    off = ((q.double() - want[:, :nq]).abs() / bound[:, :nq]).max().item()
    assert off <= 1, off
    kept = slots >= 0
    where = slots[kept].long()
    for c, old, lo in ((kv.k, before[0], nq), (kv.v, before[1], nq + nkv)):
        rows = c[layer] if paged else c[:, layer]
        got = rows[:, where].transpose(0, 1) if paged else rows[where // (t + 3), :, where % (t + 3)]
        off = ((got.double() - want[kept, lo:lo + nkv]).abs() / bound[kept, lo:lo + nkv]).max().item() if len(where) else 0
        assert off <= 1, off
        if paged:
            old[layer][:, where] = rows[:, where]
        else:
            old[where // (t + 3), layer, :, where % (t + 3)] = got
        assert torch.equal(c, old)                      # nothing else is written
    assert status.item() == 0
    return q


@pytest.mark.parametrize("t", [1, 2, 7, 64, 1000])
@pytest.mark.parametrize("nq,nkv,d", [(4, 2, 64), (32, 8, 64), (32, 8, 128), (3, 1, 32), (5, 5, 80), (12, 4, 96), (2, 1, 256), (7, 1, 16), (6, 3, 48)])
def test_sizes(t, nq, nkv, d):
    check(t, nq, nkv, d, d)
    check(t, nq, nkv, d, d, dtype=F32, norm=False, paged=16)


@pytest.mark.parametrize("d,rotary", [(64, 0), (64, 16), (64, 48), (128, 64), (128, 112), (256, 32), (80, 48)])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("norm", [False, True, "q", "k"])
def test_rotated_part_pairs_and_gains(d, rotary, neighbours, norm):
    for dtype in (BF, F32):
        check(9, 6, 2, d, rotary, dtype=dtype, neighbours=neighbours, norm=norm, paged=8)


@pytest.mark.parametrize("sections", [[32], [16, 16], [8, 12, 12], [16, 24, 24], [0, 32], [1, 2, 3, 58], [64, 0, 0]])
def test_axes(sections):
    d = 2 * sum(sections)
    check(50, 6, 2, d, d, sections=sections, paged=16, dtype=F32)
    check(50, 6, 2, 128, d, sections=sections, neighbours=True)


@pytest.mark.parametrize("far", [100000, 2 ** 24 + 1, 2 ** 31 - 6000])
def test_positions_far_along(far):
    # the 64-bit reference's own angles are off by 2^-53 of themselves (5e-7 radians at 2^31)
    check(40, 4, 2, 64, 64, far=far, freqs=freqs_of(64, 500000.0) if far < 2 ** 25 else freqs_of(64, 500000.0) * 2.0 ** -8, norm=False)


def test_negative_positions_and_any_frequency():
    positions = torch.tensor([-1, -7000, 0, 5], dtype=torch.int32, device="cuda")
    check(4, 4, 2, 32, 32, positions=positions, norm=False)
    check(4, 4, 2, 32, 32, positions=positions, norm=False, freqs=torch.linspace(-20.0, 20.0, 16, dtype=torch.float64))
    a = check(4, 4, 2, 32, 32, positions=positions, norm=False, freqs=torch.zeros(16, dtype=torch.float64))
    assert torch.equal(a, check(4, 4, 2, 32, 0, positions=positions, norm=False))


def test_layers_sequences_and_strided_rows():
    for dtype, pad in ((BF, 8), (F32, 4)):
        check(21, 4, 2, 64, 64, layers=3, layer=2, sequences=3, dtype=dtype, pad=pad)
        check(21, 4, 2, 64, 64, layers=3, layer=1, paged=8, dtype=dtype, pad=pad)


def test_tokens_without_a_place_and_places_behind_the_cache():
    t, nq, nkv, d = 40, 4, 2, 64
    slots = torch.arange(t, dtype=torch.int32, device="cuda")
    slots[25:] = -1
    slots[3] = -2 ** 31
    check(t, nq, nkv, d, d, slots=slots, paged=8)
    check(t, nq, nkv, d, d, slots=slots.clamp(min=-1))
    check(t, nq, nkv, d, d, slots=torch.full_like(slots, -1), paged=8)
    kv = KVCache(*(torch.zeros(2, 1, nkv, 8, d, dtype=BF, device="cuda") for _ in range(2)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qkv = randn((3, 8 * d), 1)
    args = (torch.arange(3, dtype=torch.int32, device="cuda"), torch.tensor([15, 16, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), freqs_of(d))
    q = mk.rope_append(qkv, kv, *args, status=status)
    assert status.item() == mk.MK_ERR_BOUNDS and torch.equal(kv.k[1, 0, :, 7] != 0, torch.ones(nkv, d, dtype=torch.bool, device="cuda"))
    kv.k[1, 0, :, 7] = 0
    assert not kv.k.any() and torch.isfinite(q).all()


def test_no_tokens_and_rows_that_are_not_finite():
    kv = KVCache(*(torch.zeros(1, 1, 2, 8, 32, dtype=BF, device="cuda") for _ in range(2)))
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert mk.rope_append(randn((0, 256), 1), kv, none, none, freqs_of(32)).shape == (0, 4, 32)
    qkv = randn((3, 256), 1)
    qkv[1, 5] = float("nan")                            # one head of one token
    i = torch.arange(3, dtype=torch.int32, device="cuda")
    gain = torch.ones(32, dtype=BF, device="cuda")
    q = mk.rope_append(qkv, kv, i, i, freqs_of(32), q_gain=gain, k_gain=gain)
    assert q[1, 0].isnan().all() and torch.isfinite(q[[0, 2]]).all() and torch.isfinite(q[1, 1:]).all() and torch.isfinite(kv.k).all()
    zero = mk.rope_append(torch.zeros_like(qkv), kv, i, i, freqs_of(32), q_gain=gain, k_gain=gain)
    assert not zero.any()


def test_q_in_place_and_beside_other_columns():
    t, nq, nkv, d = 30, 6, 2, 64
    qkv, i = randn((t, 10 * d), 1), torch.arange(t, dtype=torch.int32, device="cuda")
    kv = KVCache(*(torch.zeros(1, 1, nkv, t, d, dtype=BF, device="cuda") for _ in range(2)))
    gain = randn((d,), 2)
    want = mk.rope_append(qkv, kv, i, i, freqs_of(d), q_gain=gain)
    k = kv.k.clone()
    wide = torch.full((t, 8 * d), 7.0, dtype=BF, device="cuda")
    mk.rope_append(qkv, kv, i, i, freqs_of(d), q_gain=gain, out=wide[:, d:7 * d].unflatten(1, (nq, d)))
    assert torch.equal(wide[:, d:7 * d].reshape(t, nq, d), want) and (wide[:, :d] == 7).all() and (wide[:, 7 * d:] == 7).all()
    rest = qkv[:, nq * d:].clone()
    got = mk.rope_append(qkv, kv, i, i, freqs_of(d), q_gain=gain, out=qkv[:, :nq * d].unflatten(1, (nq, d)))
    assert got.data_ptr() == qkv.data_ptr() and torch.equal(got, want) and torch.equal(kv.k, k) and torch.equal(qkv[:, nq * d:], rest)


def test_cache_offsets_past_2_to_the_31():
    # a pool of 2.2e9 elements a side: the last slot of the last head
    nkv, d = 2, 128
    positions = (1 << 31) // (nkv * d) + 40000
    kv = KVCache(*(torch.zeros(1, nkv, positions, d, dtype=BF, device="cuda") for _ in range(2)))
    qkv, i = randn((2, 4 * nkv * d), 1), torch.zeros(2, dtype=torch.int32, device="cuda")
    slots = torch.tensor([positions - 1, 0], dtype=torch.int32, device="cuda")
    mk.rope_append(qkv, kv, i, slots, freqs_of(d))
    rows = qkv.reshape(2, 4 * nkv, d)
    for c, lo in ((kv.k, 2 * nkv), (kv.v, 3 * nkv)):
        assert torch.equal(c[0, :, -1], rows[0, lo:lo + nkv]) and torch.equal(c[0, :, 0], rows[1, lo:lo + nkv]) and not c[0, :, 1:-1].any()


def test_streams_and_graphs():
    t, nq, nkv, d = 8, 32, 8, 64
    qkv, at = randn((t, (nq + 2 * nkv) * d), 1), torch.arange(t, dtype=torch.int32, device="cuda")
    slots = at + 5
    kv = KVCache(*(torch.zeros(1, nkv, 64, d, dtype=BF, device="cuda") for _ in range(2)))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        q = mk.rope_append(qkv, kv, at, slots, freqs_of(d))
    for seed in (2, 3):
        qkv.copy_(randn(qkv.shape, seed))
        at.add_(100)
        slots.add_(t)
        g.replay()
        other = KVCache(torch.zeros_like(kv.k), torch.zeros_like(kv.v))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = mk.rope_append(qkv, other, at, slots, freqs_of(d))
        torch.cuda.synchronize()
        assert torch.equal(q, want) and torch.equal(kv.k[:, :, slots.long()], other.k[:, :, slots.long()])


@pytest.mark.parametrize("nq,nkv,d", [(4094, 1, 16), (4094, 1, 256), (2, 2047, 32)])
def test_the_most_heads(nq, nkv, d):
    check(3, nq, nkv, d, d)
    check(3, nq, nkv, d, 16, dtype=F32, paged=4)


def test_two_tokens_of_one_slot_leave_either_ones_values():
    t, nq, nkv, d = 200, 4, 2, 64
    qkv, at = randn((t, 8 * d), 1), torch.arange(t, dtype=torch.int32, device="cuda")
    kv, each = (KVCache(*(torch.zeros(1, nkv, t, d, dtype=BF, device="cuda") for _ in range(2))) for _ in range(2))
    want = mk.rope_append(qkv, each, at, at, freqs_of(d))
    got = mk.rope_append(qkv, kv, at, torch.full_like(at, 7), freqs_of(d))
    assert torch.equal(got, want)
    for c, e in ((kv.k, each.k), (kv.v, each.v)):
        assert (c[:, :, 7:8] == e).any(2).all()          # (of every element some token's)
        c[:, :, 7] = 0
        assert not c.any()


def test_calls_on_two_streams_at_once():
    t, nq, nkv, d = 3000, 8, 2, 128
    qkv, at = randn((t, 12 * d), 1), torch.arange(t, dtype=torch.int32, device="cuda")
    gain = randn((d,), 2)
    caches = [KVCache(*(torch.zeros(1, nkv, t, d, dtype=BF, device="cuda") for _ in range(2))) for _ in range(3)]
    want = mk.rope_append(qkv, caches[2], at, at, freqs_of(d), q_gain=gain, k_gain=gain)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        for s, c in zip(streams, caches):
            with torch.cuda.stream(s):
                outs.append(mk.rope_append(qkv, c, at, at, freqs_of(d), q_gain=gain, k_gain=gain))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    for c in caches[:2]:
        assert torch.equal(c.k, caches[2].k) and torch.equal(c.v, caches[2].v)


def test_refusals():
    nkv, d, t = 2, 32, 4
    kv = KVCache(*(torch.zeros(1, 1, nkv, 8, d, dtype=BF, device="cuda") for _ in range(2)))
    qkv, i = randn((t, 8 * d), 1), torch.arange(t, dtype=torch.int32, device="cuda")
    f = freqs_of(d)
    for call in (lambda: mk.rope_append(qkv[:, :7 * d + 8], kv, i, i, f), lambda: mk.rope_append(qkv[:, :4 * d], kv, i, i, f),
                 lambda: mk.rope_append(qkv.half(), kv, i, i, f), lambda: mk.rope_append(qkv, kv, i[:3], i, f), lambda: mk.rope_append(qkv, kv, i, i[:3], f),
                 lambda: mk.rope_append(qkv, kv, i.long(), i, f), lambda: mk.rope_append(qkv, kv, i, i, f.float()), lambda: mk.rope_append(qkv, kv, i, i, f.cuda()),
                 lambda: mk.rope_append(qkv, kv, i, i, f, layer=1), lambda: mk.rope_append(qkv, kv, i, i, f, sections=[8, 8]),
                 lambda: mk.rope_append(qkv, kv, i, i, f, q_gain=torch.ones(16, dtype=BF, device="cuda")),
                 lambda: mk.rope_append(qkv, kv, i, i, f, out=torch.empty(t, 4, d, device="cuda")), lambda: mk.rope_append(qkv.cpu(), kv, i, i, f)):
        with pytest.raises(ValueError):
            call()
    two = torch.stack([i, i])
    for call in (lambda: mk.rope_append(qkv, kv, two, i, f, sections=[8, 9]), lambda: mk.rope_append(qkv, kv, two, i, f, sections=[-8, 24]),
                 lambda: mk.rope_append(qkv, kv, i, i, freqs_of(24)), lambda: mk.rope_append(qkv, kv, i, i, freqs_of(64)),
                 lambda: mk.rope_append(qkv, kv, i, i, f, eps=-1.0), lambda: mk.rope_append(qkv, kv, i, i, f, eps=float("inf")),
                 lambda: mk.rope_append(qkv, kv, i, i, f * float("nan")),
                 lambda: mk.rope_append(qkv, KVCache(kv.k, kv.k), i, i, f), lambda: mk.rope_append(qkv[:, 1:1 + 6 * d], kv, i, i, f),
                 lambda: mk.rope_append(qkv, kv, i, i, f, out=qkv[:, d:5 * d].unflatten(1, (4, d)))):
        with pytest.raises(mk.MkError) as e:
            call()
        assert e.value.status == mk.MK_ERR_ARG
