"""mk_attend over caches whose dimensions of one have odd strides, and with an output right behind the cache:
the same bits as over an ordinary cache."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from workload import KVCache  # noqa: E402


class _Python:
    """In the place of the C call module: leaves every call to Python."""

    @staticmethod
    def attend(*args):
        return None


def randn(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def restride(t, strides):
    """t's values behind other strides (None: t's own) for its dimensions of one."""
    return t.as_strided(t.shape, [s if new is None else new for s, new in zip(t.stride(), strides)], t.storage_offset())


@pytest.mark.parametrize("python", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_dimensions_of_one(d, python, monkeypatch):
    if python:
        monkeypatch.setattr(mk, "_fast", _Python)
    q = randn((9, 4, d), 5)
    # one head of a cache that keeps its heads outermost: the stride of heads is the largest
    heads = [randn((3, 2, 1, 900, d), 10 + i) for i in range(2)]
    plain = KVCache(*(h[1][:, :, None].contiguous() for h in heads))
    outer = KVCache(*(h.permute(1, 2, 0, 3, 4)[:, :, 1:2] for h in heads))
    want = mk.attend(q, plain, [4, 5], [900, 77])
    assert torch.equal(mk.attend(q, outer, [4, 5], [900, 77]), want)
    # one sequence, one layer, one head
    one = KVCache(*(t[:1] for t in (plain.k, plain.v)))
    want = mk.attend(q, one, [9], [900])
    for strides in ((1, 1, 1, None, None), (0, 0, 0, None, None), (1 << 40, 1 << 40, 1 << 40, None, None)):
        assert torch.equal(mk.attend(q, KVCache(*(restride(t, strides) for t in (one.k, one.v))), [9], [900]), want)
    # a pool of one layer and one head
    pool = KVCache(*(t[0] for t in (one.k, one.v)))
    pages = (torch.arange(7, device="cuda", dtype=torch.int32).reshape(1, 7), 128, 7)
    want = mk.attend(q, one, [9], [896])
    for strides in ((None, None, None, None), (1, 1, None, None), (1 << 40, 1 << 40, None, None)):
        assert torch.equal(mk.attend(q, KVCache(*(restride(t, strides) for t in (pool.k, pool.v))), [9], [896], pages=pages), want)


def test_an_output_right_behind_the_last_position():
    n, d, wide = 130, 64, 200
    q = randn((7, 4, d), 5)
    k = randn((2, 1, 2, wide, d), 1)
    v = randn((2, 1, 2, wide, d), 2)
    want = mk.attend(q, KVCache(k[:, :, :, wide - n:].contiguous(), v[:, :, :, wide - n:].contiguous()), [3, 4], [n, 60])
    buf = torch.zeros(k.numel() + q.numel(), device="cuda", dtype=torch.bfloat16)
    buf[:k.numel()] = k.reshape(-1)
    kv = KVCache(buf[:k.numel()].view(k.shape)[:, :, :, wide - n:], v[:, :, :, wide - n:])       # ends where k's storage does
    out = buf[k.numel():].view(q.shape)
    assert torch.equal(mk.attend(q, kv, [3, 4], [n, 60], out=out), want) and torch.equal(buf[:k.numel()], k.reshape(-1))
