"""mk_attend against its definition in 64 bits: head layouts, lengths from none to many tiles, windows
and sinks, ragged batches, paged caches, shared prefixes, what masked places hold, strides, streams
and graphs.  The tolerance is derived in attend_reference."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from attend_reference import attend_reference  # noqa: E402
from workload import KVCache  # noqa: E402

BF = torch.bfloat16


def randn(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def cache(batch, nkv, d, max_seq, layers=1, seed=0):
    shape = (batch, layers, nkv, max_seq, d)
    return KVCache(randn(shape, seed + 1), randn(shape, seed + 2))


def pool(batch, nkv, d, max_seq, block, layers=1, seed=0, spare=3):
    """A paged cache: (kv, pages) with blocks in shuffled order."""
    per = -(-max_seq // block)
    n = batch * per + spare
    table = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:batch * per].reshape(batch, per)
    shape = (layers, nkv, n * block, d)
    return KVCache(randn(shape, seed + 1), randn(shape, seed + 2)), (table.to(device="cuda", dtype=torch.int32), block, n)


def check(q, kv, q_lens, kv_lens, out=None, **kw):
    want, bound = attend_reference(q, kv, q_lens, kv_lens, **kw)
    got = mk.attend(q, kv, q_lens, kv_lens, out=out, **kw)
    rows = sum(q_lens)
    off = (got[:rows].double() - want[:rows]).abs() / bound[:rows]
    assert torch.isfinite(got[:rows]).all()
    assert off.numel() == 0 or off.max().item() <= 1, off.max().item()
    return got


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("nkv,group", [(1, 1), (2, 2), (1, 3), (2, 4), (1, 5), (1, 6), (1, 7), (2, 8)])
def test_head_layouts(d, nkv, group):
    kv = cache(2, nkv, d, 300)
    check(randn((1 + 70, nkv * group, d), 5, 1.5), kv, [1, 70], [300, 211])


@pytest.mark.parametrize("q_len,kv_len", [(1, 1), (1, 2), (2, 2), (1, 127), (1, 128), (1, 129), (1, 1000), (16, 16), (17, 128),
                                          (31, 131), (32, 256), (33, 257), (64, 640), (129, 129), (130, 513), (400, 400)])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_lengths(q_len, kv_len, d):
    check(randn((q_len, 4, d), 5, 1.5), cache(1, 1, d, kv_len), [q_len], [kv_len])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (5, 3), (64, 4), (127, 0), (128, 128), (130, 64), (300, 150),
                                          (1000, 4), (40, 1000), (2000, 0)])
@pytest.mark.parametrize("q_len,kv_len", [(1, 700), (40, 700), (300, 700), (700, 700)])
def test_windows(window, sinks, q_len, kv_len):
    check(randn((q_len, 8, 64), 5, 1.5), cache(1, 2, 64, 704), [q_len], [kv_len], window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(1, 1), (5, 3), (63, 0), (64, 64), (65, 10), (130, 64), (300, 150), (1000, 4), (40, 1000)])
@pytest.mark.parametrize("q_len,kv_len", [(1, 700), (40, 700), (333, 333)])
@pytest.mark.parametrize("d", [32, 128])
def test_windows_at_other_widths(d, window, sinks, q_len, kv_len):
    check(randn((q_len, 4, d), 5, 1.5), cache(1, 1, d, 704), [q_len], [kv_len], window=window, sinks=sinks)


@pytest.mark.parametrize("q_len,kv_len", [(1, 63), (1, 64), (1, 65), (63, 63), (64, 64), (65, 65), (128, 192), (200, 321), (17, 64 * 31 + 1)])
@pytest.mark.parametrize("group", [1, 4, 7])
def test_lengths_about_a_tile_of_64(group, q_len, kv_len):
    check(randn((q_len, group, 128), 5, 1.5), cache(1, 1, 128, kv_len), [q_len], [kv_len])


def test_masked_places_and_rising_maxima_at_width_128():
    kv = cache(2, 2, 128, 384)
    q_lens, kv_lens = [60, 200], [200, 333]
    q = randn((260, 4, 128), 5)
    for window, sinks in ((0, 0), (90, 5)):
        want = mk.attend(q, kv, q_lens, kv_lens, window=window, sinks=sinks)
        bad = KVCache(kv.k.clone(), kv.v.clone())
        for c, fill in ((bad.k, float("nan")), (bad.v, float("inf"))):
            for b, n in enumerate(kv_lens):
                c[b, :, :, n:] = fill
                if window:
                    c[b, :, :, sinks:n - q_lens[b] - window + 1] = fill
        assert torch.equal(mk.attend(q, bad, q_lens, kv_lens, window=window, sinks=sinks), want)
    # a maximum that rises and falls from one tile of 64 keys to the next, and alternates between them
    kv, one = cache(1, 1, 128, 900), torch.ones((64, 4, 128), device="cuda", dtype=BF)
    at = torch.arange(900, device="cuda")
    for ramp in (at // 64 * 4.0, at // 64 * -4.0, at // 64 % 2 * 12.0, at // 64 % 3 * -9.0, (at == 700) * 30.0):
        kv.k[0, 0, 0] = (ramp[:, None] * torch.ones(128, device="cuda")).to(BF)
        for q in (one, -one):
            check(q, kv, [64], [900])
            check(q, kv, [64], [900], window=500, sinks=70)


@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_ragged_batch(window, sinks):
    q_lens, kv_lens = [1, 0, 37, 200, 1, 3, 0, 129], [1, 17, 300, 200, 513, 3, 0, 400]
    q = randn((sum(q_lens) + 9, 6, 64), 5, 1.5)
    kv = cache(8, 2, 64, 520)
    out = torch.full_like(q, 3.0)
    check(q, kv, q_lens, kv_lens, out=out, window=window, sinks=sinks)
    assert (out[sum(q_lens):] == 3).all()          # rows behind the last sequence are left as they were


def test_tokens_without_a_visible_position_get_zeros():
    q_lens, kv_lens = [5, 300, 2], [2, 170, 0]
    q, kv = randn((307, 4, 64), 5), cache(3, 1, 64, 300)
    got = check(q, kv, q_lens, kv_lens)
    assert (got[:3] == 0).all() and (got[5:5 + 130] == 0).all() and (got[305:] == 0).all() and (got[3:5] != 0).any()


@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [200, 333]), ([60, 200], [200, 333])])
def test_what_masked_places_hold(window, sinks, q_lens, kv_lens):
    # positions that no token of the call sees hold NaN and infinities: they change nothing
    kv = cache(2, 2, 64, 384)
    q = randn((sum(q_lens), 8, 64), 5)
    clean = mk.attend(q, kv, q_lens, kv_lens, window=window, sinks=sinks)
    for b in range(2):
        for t, bad in ((kv.k, float("nan")), (kv.v, float("nan"))):
            t[b, :, :, kv_lens[b]:] = bad
        low = kv_lens[b] - q_lens[b] - window + 1
        if window and low > sinks:
            kv.k[b, :, :, sinks:low] = float("inf")
            kv.v[b, :, :, sinks:low] = float("nan")
    assert torch.equal(mk.attend(q, kv, q_lens, kv_lens, window=window, sinks=sinks), clean)


@pytest.mark.parametrize("block", [8, 16, 48, 64, 128, 200, 256, 512])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_paged(block, d):
    kv, pages = pool(3, 2, d, 777, block)
    q_lens, kv_lens = [1, 90, 3], [777, 400, 129]
    check(randn((94, 8, d), 5, 1.5), kv, q_lens, kv_lens, pages=pages)
    check(randn((94, 8, d), 6, 1.5), kv, q_lens, kv_lens, pages=pages, window=150, sinks=9)


def test_a_bad_table_entry_is_not_followed():
    kv, pages = pool(2, 1, 64, 512, 64)
    q_lens, kv_lens = [2, 40], [512, 500]
    q = randn((42, 4, 64), 5)
    for bad in (-1, pages[2], 1 << 30):
        pages[0][0, 1] = bad
        pages[0][1, 7] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        want, bound = attend_reference(q, kv, q_lens, kv_lens, pages=pages)
        got = mk.attend(q, kv, q_lens, kv_lens, pages=pages, status=status)
        assert ((got.double() - want).abs() <= bound).all()
        assert status.item() == mk.MK_ERR_BOUNDS


def test_unused_table_entries_may_hold_anything():
    kv, pages = pool(2, 1, 64, 512, 64)
    pages[0][0, 4:] = -7
    pages[0][1, 1:5] = 1 << 29          # between the sinks and the window of every token
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = randn((11, 4, 64), 5)
    got = mk.attend(q, kv, [1, 10], [256, 500], pages=pages, window=100, sinks=3, status=status)
    want, bound = attend_reference(q, kv, [1, 10], [256, 500], pages=pages, window=100, sinks=3)
    assert ((got.double() - want).abs() <= bound).all() and status.item() == 0


@pytest.mark.parametrize("block", [0, 64, 128])
@pytest.mark.parametrize("prefix", [1, 100, 128, 1000])
@pytest.mark.parametrize("q_lens,tails", [([1, 1, 1], [1, 2, 140]), ([1, 0, 33, 7], [1, 0, 200, 7]), ([60] * 9, [60] * 9)])
def test_shared_prefix(block, prefix, q_lens, tails):
    kv_lens = [prefix + t for t in tails]
    batch, top = len(q_lens), max(kv_lens)
    if block:
        kv, pages = pool(batch, 2, 64, top, block)
    else:
        kv, pages = cache(batch, 2, 64, top), None
        for b in range(1, batch):          # the prefix is read through sequence 0 alone
            kv.k[b, :, :, :prefix] = float("nan")
            kv.v[b, :, :, :prefix] = float("nan")
    check(randn((sum(q_lens), 8, 64), 5, 1.5), kv, q_lens, kv_lens, shared_prefix=prefix, pages=pages)


@pytest.mark.parametrize("d,group", [(32, 1), (64, 3), (128, 8)])
def test_shared_prefix_heads(d, group):
    q_lens = [1, 4, 2, 50, 1]
    kv_lens = [400 + n + 3 * b for b, n in enumerate(q_lens)]
    check(randn((sum(q_lens), 2 * group, d), 5, 1.5), cache(5, 2, d, 500), q_lens, kv_lens, shared_prefix=400)


def test_strides_layers_and_scale():
    kv = cache(3, 2, 64, 400, layers=3)
    wide = KVCache(*(torch.full((3, 3, 2, 500, 64), float("nan"), device="cuda", dtype=BF)[:, :, :, :400] for _ in range(2)))
    wide.k.copy_(kv.k)
    wide.v.copy_(kv.v)
    buf = randn((60, 1000), 5, 1.5)
    q = buf[:, 8:8 + 512].unflatten(1, (8, 64))
    obuf = torch.full((60, 800), 2.0, device="cuda", dtype=BF)
    out = obuf[:, 16:16 + 512].unflatten(1, (8, 64))
    for c in (kv, wide):
        for layer in (0, 2):
            got = check(q, c, [10, 50], [400, 123], out=out, layer=layer, scale=0.3)
            assert (obuf[:, :16] == 2).all() and (obuf[:, 528:] == 2).all()
    assert torch.equal(got, check(q.contiguous(), kv, [10, 50], [400, 123], layer=2, scale=0.3))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("q_len", [1, 64])
def test_sharp_and_flat_softmax(d, q_len):
    # scores far apart (one weight near 1), all alike, far above and below zero, and a maximum that rises along
    # the row by much more than the formats hold, within a tile and from tile to tile
    kv = cache(1, 1, d, 600)
    check(randn((q_len, 4, d), 5, 12.0), kv, [q_len], [600])
    one = torch.ones((q_len, 4, d), device="cuda", dtype=BF)
    for ramp in (torch.arange(600, device="cuda") / 20.0, torch.arange(600, device="cuda") // 128 * 8.0,
                 torch.arange(600, device="cuda") // 128 * -8.0, torch.full((600,), 30.0, device="cuda")):
        kv.k[0, 0, 0] = (ramp[:, None] * torch.ones(d, device="cuda")).to(BF)
        for q in (one, -one, 0 * one):
            check(q, kv, [q_len], [600])
            check(q, kv, [q_len], [600], window=300, sinks=2)


def test_one_weight_that_outweighs_the_rest_is_exact():
    # rows that see one key, or one that matters, return its value as it is
    for d in (32, 64, 128):
        kv = cache(1, 1, d, 300)
        got = mk.attend(randn((7, 4, d), 5), kv, [7], [300], window=1)
        assert torch.equal(got, kv.v[0, 0, 0, 293:300, None].expand(7, 4, d))


def test_far_positions():
    # offsets past 2^31 elements: only the window's tail of a long cache is read
    d, top = 64, (1 << 25) + 700
    kv = KVCache(torch.zeros((1, 1, 1, top, d), device="cuda", dtype=BF), torch.zeros((1, 1, 1, top, d), device="cuda", dtype=BF))
    kv.k[0, 0, 0, -1000:] = randn((1000, d), 1)
    kv.v[0, 0, 0, -1000:] = randn((1000, d), 2)
    kv.v[0, 0, 0, :4] = 1.0
    q = randn((30, 4, d), 5)
    got = mk.attend(q, kv, [30], [top], window=300, sinks=4)
    near = KVCache(kv.k[:, :, :, -1000:].contiguous(), kv.v[:, :, :, -1000:].contiguous())
    near.k[0, 0, 0, :4], near.v[0, 0, 0, :4] = 0.0, 1.0
    want, bound = attend_reference(q, near, [30], [1000], window=300, sinks=4)
    assert ((got.double() - want).abs() <= bound).all()


def test_repeatable_on_streams_and_with_a_given_workspace():
    kv = cache(4, 2, 64, 3000)
    q = randn((4, 8, 64), 5)
    args = (q, kv, [1] * 4, [3000, 1, 2000, 700])
    a = mk.attend(*args)
    for _ in range(3):
        assert torch.equal(mk.attend(*args), a)
    ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")      # whatever it holds
    assert torch.equal(mk.attend(*args, workspace=ws), a)
    s = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for x in s:
        x.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(x):
            got.append(mk.attend(*args))
    torch.cuda.synchronize()
    assert torch.equal(got[0], a) and torch.equal(got[1], a)


def test_captured_and_replayed():
    kv, pages = pool(2, 2, 64, 2000, 128)
    q = randn((5, 8, 64), 5)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    mk.attend(q, kv, [1, 4], [2000, 1500], pages=pages)
    torch.cuda.synchronize()
    for lens in ([2000, 1500], [900, 2000]):          # two graphs, one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mk.attend(q, kv, [1, 4], lens, pages=pages, workspace=ws))
        graphs.append(g)
    kv.v.copy_(randn(tuple(kv.v.shape), 77))
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for lens, o in zip(([2000, 1500], [900, 2000]), outs):
        assert torch.equal(o, mk.attend(q, kv, [1, 4], lens, pages=pages))


def test_captured_without_a_workspace_of_its_own():
    # the workspace of each captured call is the graph's: eager calls in between take other memory
    kv = cache(2, 2, 64, 3000)
    q = randn((2, 8, 64), 5)
    want = [mk.attend(q, kv, [1, 1], lens) for lens in ([3000, 2500], [1200, 3000])]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [mk.attend(q, kv, [1, 1], lens) for lens in ([3000, 2500], [1200, 3000])]
    for _ in range(3):
        other = mk.attend(randn((2, 8, 64), 6), kv, [1, 1], [3000, 3000])
        g.replay()
        other = mk.attend(randn((2, 8, 64), 7), kv, [1, 1], [2000, 3000])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.isfinite(other).all()


def test_workspace_is_checked():
    kv, q = cache(1, 1, 64, 4000), randn((1, 4, 64), 5)
    for ws, status in ((torch.empty(256, dtype=torch.uint8, device="cuda"), mk.MK_ERR_CAPACITY),
                       (torch.empty(1 << 22, dtype=torch.uint8, device="cuda")[16:], mk.MK_ERR_ARG)):
        with pytest.raises(mk.MkError) as e:
            mk.attend(q, kv, [1], [4000], workspace=ws)
        assert e.value.status == status
    with pytest.raises(ValueError):
        mk.attend(q, kv, [1], [4000], workspace=torch.empty(1 << 22, dtype=torch.uint8))


def test_more_queries_than_positions_need_little_workspace():
    # most of the tokens see nothing: the shares must not multiply their parts (one part here is 41 MB a 20000 tokens)
    kv, q = cache(1, 1, 128, 5000), randn((20000, 4, 128), 5)
    parts = 20000 * 4 * (128 * 4 + 8)
    ws = torch.empty(4 * parts, dtype=torch.uint8, device="cuda")
    got = mk.attend(q, kv, [20000], [5000], workspace=ws)
    assert (got[:15000] == 0).all()
    check(q, kv, [20000], [5000])


def test_a_single_kv_head_taken_out_of_a_cache():
    kv = cache(2, 4, 64, 200)
    one = KVCache(kv.k[:, :, 1:2], kv.v[:, :, 1:2])
    odd = KVCache(*(x.as_strided(x.shape, (x.stride(0), x.stride(1), 0, 64, 1), x.storage_offset()) for x in (one.k, one.v)))
    q = randn((9, 4, 64), 5)
    a = check(q, one, [4, 5], [200, 90])
    assert torch.equal(mk.attend(q, odd, [4, 5], [200, 90]), a)


def test_many_short_sequences_and_many_tokens():
    q_lens = [1 + b % 3 for b in range(256)]
    kv_lens = [n + 7 * b % 90 for b, n in enumerate(q_lens)]
    check(randn((sum(q_lens), 4, 32), 5), cache(256, 2, 32, 100), q_lens, kv_lens)
    check(randn((sum(q_lens), 4, 32), 5), cache(256, 2, 32, 200), q_lens, [90 + k for k in kv_lens], shared_prefix=90)
    check(randn((20000, 1, 32), 5), cache(1, 1, 32, 20000), [20000], [20000], window=40, sinks=1)


class _Python:
    """In the place of the C call module: leaves every call to Python."""

    @staticmethod
    def linear(*args):
        return None

    attend = linear


def test_c_and_python_calls_agree_and_keep_nothing(monkeypatch):
    import sys
    kv, q = cache(3, 2, 64, 500), randn((9, 4, 64), 5)
    pool = KVCache(kv.k[:, 0].permute(1, 0, 2, 3).reshape(1, 2, 1500, 64).contiguous(),
                   kv.v[:, 0].permute(1, 0, 2, 3).reshape(1, 2, 1500, 64).contiguous())
    table = torch.arange(15, device="cuda", dtype=torch.int32).reshape(3, 5)
    out, status = torch.empty_like(q), torch.zeros(1, device="cuda", dtype=torch.int32)
    ws = torch.empty(1 << 22, device="cuda", dtype=torch.uint8)
    calls = [(kv, [1, 3, 5], [500, 200, 60], {}), (kv, (1, 3, 5), (500, 200, 60), dict(window=40, sinks=3, scale=0.3, status=status)),
             (kv, [2, 0, 1], [500, 0, 300], dict(out=out, workspace=ws)), (kv, [1, 1, 1], [400, 300, 450], dict(shared_prefix=128)),
             (pool, [1, 3, 5], [480, 200, 60], dict(pages=(table, 96, 15)))]
    bad = [(kv, [1, 3, 5], [500, 200], {}), (kv, [1, 3, 5], [500, 200, 501], {}), (kv, [9, 9, 9], [500, 200, 60], {}),
           (kv, [1, 3, 5], [500, 200, 60], dict(layer=1)), (kv, [1, 3, 5], [500, 200, 60], dict(scale=-1.0)),
           (kv, [1, 3, 5], [500, 200, 60], dict(scale=1e-60)), (kv, [1, 3, 5], [500, 200, 60], dict(workspace=ws.cpu())),
           (kv, [1, 3, 5], [500, 200, 60], dict(out=q)), (kv, [1, 3, 5], [500, 200, 60], dict(status=status.float())),
           (pool, [1, 3, 5], [480, 200, 60], dict(pages=(table, 96, 16))), (kv, [], [], {})]

    def run(c):
        try:
            return mk.attend(q, c[0], c[1], c[2], **c[3]).clone()
        except (ValueError, mk.MkError) as e:
            return str(e)

    taken = [run(c) for c in calls]
    refused = [run(c) for c in bad]
    assert all(isinstance(t, torch.Tensor) for t in taken) and all(isinstance(r, str) for r in refused)
    with monkeypatch.context() as m:
        m.setattr(mk, "_fast", _Python)
        for c, t in zip(calls, taken):
            n = sum(c[1])
            assert torch.equal(run(c)[:n], t[:n])
        assert [run(c) for c in bad] == refused
    del taken
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in (q, out, ws, table, status, kv.k, torch.bfloat16)]
    for _ in range(100):
        for c in calls + bad:
            run(c)
    assert (torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in (q, out, ws, table, status, kv.k, torch.bfloat16)]) == held


def test_lengths_may_be_any_sequence_of_ints():
    import numpy as np
    kv, q = cache(2, 1, 64, 300), randn((5, 4, 64), 5)
    want = mk.attend(q, kv, [2, 3], [300, 40])
    assert torch.equal(mk.attend(q, kv, np.array([2, 3]), np.array([300, 40])), want)
    assert torch.equal(mk.attend(q, kv, range(2, 4), (300, 40)), want)


def test_refuses_tensors_it_cannot_take():
    kv, (pk, pages) = cache(2, 2, 64, 100), pool(2, 2, 64, 100, 16)
    q = randn((3, 8, 64), 5)
    for bad in (lambda: mk.attend(q.cpu(), kv, [1, 2], [9, 9]), lambda: mk.attend(q.float(), kv, [1, 2], [9, 9]),
                lambda: mk.attend(q, kv, [1, 2], [9]), lambda: mk.attend(q, kv, [2, 2], [9, 9]),
                lambda: mk.attend(q, kv, [1, 1, 1], [9, 9, 9]), lambda: mk.attend(q, kv, [1, 2], [9, 9], layer=1),
                lambda: mk.attend(q, pk, [1, 2], [9, 9]), lambda: mk.attend(q, kv, [1, 2], [9, 9], pages=pages),
                lambda: mk.attend(q, kv, [1, 2], [9, 9], scale=0.0), lambda: mk.attend(q[:, ::2], kv, [1, 2], [9, 9]),
                lambda: mk.attend(q, pk, [1, 2], [9, 9], pages=(pages[0], 16, pages[2] + 1)),
                lambda: mk.attend(q, pk, [1, 2], [9, 9], pages=(pages[0][:1], 16, pages[2])),
                lambda: mk.attend(q, kv, [1, 2], [9, 9], out=torch.empty_like(q[:2])),
                lambda: mk.attend(q, KVCache(kv.k, kv.v[:, :, :, :50]), [1, 2], [9, 9])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mk.attend(q, kv, [1, 2], [9, 101]), lambda: mk.attend(q, kv, [1, 2], [9, 9], out=q),
                lambda: mk.attend(q, kv, [1, 2], [9, 9], shared_prefix=9),
                lambda: mk.attend(randn((3, 18, 64), 5), kv, [1, 2], [9, 9])):
        with pytest.raises(mk.MkError) as e:
            bad()
        assert e.value.status == mk.MK_ERR_ARG
