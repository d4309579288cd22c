"""mk_attend with scores that are not finite: the softmax of a row with a NaN score, with one of +infinity, or
with -infinity alone is NaN; a score of -infinity among others has no weight; zeros are for rows without a
visible position.  Rows beside such a row stay as they are, bit for bit: a row's arithmetic does not depend on
its neighbours' values."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from workload import KVCache  # noqa: E402

BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")
# one share of the keys and several, whole blocks of queries and parts, behind a shared prefix, with a window
CALLS = [dict(n=1, length=1), dict(n=1, length=100), dict(n=1, length=5000), dict(n=70, length=300), dict(n=3, length=700, shared_prefix=600),
         dict(n=40, length=900, window=130, sinks=5)]


def randn(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("call", CALLS)
def test_scores_that_are_not_finite(d, call):
    call = dict(call)
    n, length = call.pop("n"), call.pop("length")
    lens = [n, n], [length, length]
    kv = KVCache(randn((2, 1, 1, length, d), 1), randn((2, 1, 1, length, d), 2))
    q = randn((2 * n, 4, d), 3)
    # keys' and queries' first elements are positive: an infinity there gives scores of its sign
    kv.k[..., 0], q[..., 0] = kv.k[..., 0].abs() + 0.01, q[..., 0].abs() + 0.01
    clean = mk.attend(q, kv, *lens, **call)
    assert torch.isfinite(clean).all()
    row = n + n // 2
    rest = torch.ones((2 * n, 4), dtype=torch.bool)
    rest[row, 1] = False
    for where, value in ((slice(None), NAN), (d - 1, NAN), (0, INF), (0, -INF)):
        bad = q.clone()
        bad[row, 1, where] = value
        got = mk.attend(bad, kv, *lens, **call)
        assert got[row, 1].isnan().all(), (where, value)
        assert same(got[rest], clean[rest])
    # a key: seen by the tokens of its sequence from its position on, of both where it lies in the shared prefix
    window, sinks, prefix = (call.get(k, 0) for k in ("window", "sinks", "shared_prefix"))
    for b, p in ((1, length - 1), (1, length - n), (0, 0), (0, max(0, length - n - 20))):
        t = torch.arange(length - n, length).repeat(2)
        see = (t >= p) & ((t < p + window) | (p < sinks) if window else True)
        if p >= prefix:
            see &= torch.arange(2).repeat_interleave(n) == b
        bad = KVCache(kv.k.clone(), kv.v)
        for value in (NAN, INF):
            bad.k[b, 0, 0, p, 0] = value
            got = mk.attend(q, bad, *lens, **call)
            assert got[see].isnan().all() and same(got[~see], clean[~see]), (b, p, value)
        if length > 1:   # no weight, as with a finite score that is as good as -infinity (another visible key outweighs it)
            bad.k[b, 0, 0, p, 0] = -1e30
            want = mk.attend(q, bad, *lens, **call)
            bad.k[b, 0, 0, p, 0] = -INF
            assert torch.isfinite(want).all() and same(mk.attend(q, bad, *lens, **call), want), (b, p)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_rows_without_a_key_stay_zeros(d):
    # more tokens than positions, and a table that leads nowhere, beside a NaN query and one with keys of -infinity alone
    n, block = 9, 16
    kv = KVCache(randn((1, 1, 64 * block, d), 1), randn((1, 1, 64 * block, d), 2))
    kv.k[..., 0] = kv.k[..., 0].abs() + 0.01
    table = torch.arange(64, dtype=torch.int32, device="cuda").reshape(4, 16)
    table[1] = -1
    q = randn((4 * n, 2, d), 3)
    q[0, 0, 0] = NAN          # sees nothing: its scores do not count
    q[n - 1, 1, 0] = NAN      # sees 4 positions
    q[3 * n, :, 0] = -INF
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mk.attend(q, kv, [n] * 4, [4, 200, 200, 0], pages=(table, block, 64), status=status)
    assert (got[:n - 4] == 0).all() and torch.isfinite(got[n - 4:n - 1]).all() and (got[n - 4:n - 1] != 0).any()
    assert got[n - 1, 1].isnan().all() and torch.isfinite(got[n - 1, 0]).all()
    assert (got[n:2 * n] == 0).all() and torch.isfinite(got[2 * n:3 * n]).all() and (got[3 * n:] == 0).all()
    assert status.item() == mk.MK_ERR_BOUNDS
    seen = mk.attend(q[3 * n:], kv, [n], [200], pages=(table[3:].contiguous(), block, 64))
    assert seen[0].isnan().all() and torch.isfinite(seen[1:]).all()
