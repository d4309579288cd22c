"""mk_linear_adapted against the formula in 64 bits: tokens of every mixture of adapters, ranks, sizes, types and
activations, streams, graphs, workspaces.

Tolerance per output.  The linear map's part as for mk_linear: a tensor-core step adds 16 products to the running sum with an
error of at most 2^-22 of the absolute sum, so a contraction of k has at most (k / 16 + 2) 2^-22 of it.  A low-rank value
t = scale x . down has (k / 16 + 20) 2^-22 of its own absolute sum (up to 16 partial sums joined in fp32, the scale); it enters
the second product in two bf16 parts, each off by at most 2^-9 of what is left (2^-18 together), or three (2^-27, below fp32's
own 2^-24); the second product adds 3 steps per 16 columns of the rank to the contraction.  Activations and output as
for mk_linear."""
import gc
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def nothing_left_behind():
    """Tracebacks of refused calls hold tensors in cycles: they go before the next module's tests look at the memory."""
    yield
    gc.collect()


def randn(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def adapters(count, rank, k, n, seed=50, scaled=True):
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    return (randn((count, rank, k), seed, k ** -0.5), randn((count, n, rank), seed + 1, rank ** -0.5),
            torch.rand(count, generator=g, device="cuda") + 0.25 if scaled else None)


def index_of(rows, count, how, seed=7):
    r = torch.Generator().manual_seed(seed)
    if how == "own":
        i = torch.arange(rows) % count
    elif how == "any":
        i = torch.randint(-1, count, (rows,), generator=r)
    elif how == "runs":
        i = (torch.arange(rows) * 3 // max(rows, 1)) % (count + 1) - 1
    else:
        i = torch.full((rows,), -1)
    return i.to(torch.int32).cuda()


def reference(x, w, ad, index, bias, act, residual, out_dtype):
    """(value, bound) in fp64."""
    down, up, scale = ad
    k, r = x.shape[1], down.shape[1]
    x64 = x.double()
    y, s = x64 @ w.double().T, x64.abs() @ w.double().abs().T
    if bias is not None:
        y, s = y + bias.double(), s + bias.double().abs()
    e = torch.zeros_like(y)
    for a in range(down.shape[0]):
        rows = (index == a).nonzero().reshape(-1)
        if not len(rows):
            continue
        f = 1.0 if scale is None else scale[a].double()
        t, ta = f * (x64[rows] @ down[a].double().T), f * (x64[rows].abs() @ down[a].double().abs().T)
        u = up[a].double().T
        y[rows] += t @ u
        s[rows] += t.abs() @ u.abs()
        e[rows] += (k / 16 + 20) * 2.0 ** -22 * (ta @ u.abs()) + (2.0 ** -18 if out_dtype == BF else 2.0 ** -24) * (t.abs() @ u.abs())
    e = e + (k / 16 + 2 + 3 * math.ceil(r / 16)) * 2.0 ** -22 * s
    if act == "swiglu":
        n = w.shape[0] // 2
        g, u, eg, eu = y[:, :n], y[:, n:], e[:, :n], e[:, n:]
        sg = g * torch.sigmoid(g)
        y, e = sg * u, 1.13 * eg * u.abs() + sg.abs() * eu + 1.13 * eg * eu
    elif act == "silu":
        y, e = y * torch.sigmoid(y), 1.13 * e
    elif act == "gelu":
        y, e = y * torch.special.ndtr(y), 1.13 * e
    e = e + 2.0 ** -20 * y.abs()
    if residual is not None:
        y = y + residual.double()
    return y, e + torch.finfo(out_dtype).eps / 2 * (y.abs() + e) * (1 if out_dtype == BF else 2) + 1e-37


def check(x, w, ad, index, bias=None, act=None, residual=None, out=None, out_dtype=BF, **more):
    want, bound = reference(x, w, ad, index, bias, act, residual, out_dtype)
    got = mk.adapted_linear(x, w, ad, index, bias=bias, activation=act, residual=residual, out=out, out_dtype=out_dtype, **more)
    assert got.dtype == out_dtype and (out is None or got is out)
    off = (got.double() - want).abs() / bound
    assert torch.isfinite(got).all() and off.max().item() <= 1, off.max().item()
    return got


@pytest.mark.parametrize("rows", [1, 2, 8, 16, 17, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("how", ["own", "any", "runs", "none"])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_mixtures(rows, how, out_dtype):
    n, k, count = 257, 136, 5
    check(randn((rows, k), 1), randn((n, k), 2, k ** -0.5), adapters(count, 16, k, n), index_of(rows, count, how), out_dtype=out_dtype)


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 128, 256])
@pytest.mark.parametrize("rows", [3, 70, 600])
def test_ranks(rank, rows):
    n, k, count = 130, 264, 3
    for dtype in (BF, F32):
        check(randn((rows, k), 1), randn((n, k), 2, k ** -0.5), adapters(count, rank, k, n), index_of(rows, count, "any"), out_dtype=dtype)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("residual", [None, BF, F32])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_epilogues(act, residual, out_dtype):
    f = 2 if act == "swiglu" else 1
    for rows, n, k, bias in ((3, 77, 136, True), (200, 264, 256, False), (520, 100, 72, True)):
        check(randn((rows, k), 1), randn((f * n, k), 2, k ** -0.5), adapters(4, 16, k, f * n, scaled=bias), index_of(rows, 4, "any"),
              randn((f * n,), 3) if bias else None, act, None if residual is None else randn((rows, n), 4, dtype=residual), out_dtype=out_dtype)


@pytest.mark.parametrize("rows,n,k,act,count,rank,how", [
    (1, 2048, 2048, None, 3, 16, "own"), (8, 8192, 2048, "swiglu", 40, 16, "own"), (64, 2048, 4096, None, 64, 64, "own"),
    (256, 1000, 1032, "silu", 256, 16, "own"), (2100, 520, 1032, "swiglu", 7, 32, "runs"), (1500, 700, 512, None, 90, 8, "any"),
    (4096, 2048, 2048, "swiglu", 4, 16, "runs")])
def test_large(rows, n, k, act, count, rank, how):
    f = 2 if act == "swiglu" else 1
    for dtype in (BF, F32):
        check(randn((rows, k), 1), randn((f * n, k), 2, k ** -0.5), adapters(count, rank, k, f * n), index_of(rows, count, how), act=act,
              residual=randn((rows, n), 3, dtype=F32), out_dtype=dtype)


def test_one_input_feature_block_and_one_output():
    check(randn((5, 8), 1), randn((1, 8), 2), adapters(2, 8, 8, 1), index_of(5, 2, "any"), out_dtype=F32)


def test_no_adapter_is_the_linear_map():
    for rows in (1, 9, 150):
        x, w = randn((rows, 264), 1), randn((130, 264), 2, 0.1)
        got = mk.adapted_linear(x, w, adapters(3, 16, 264, 130), index_of(rows, 3, "none"), out_dtype=F32)
        want, bound = reference(x, w, adapters(3, 16, 264, 130), index_of(rows, 3, "none"), None, None, None, F32)
        assert ((got.double() - want).abs() <= bound).all()


def test_no_rows():
    assert mk.adapted_linear(randn((0, 64), 1), randn((32, 64), 2), adapters(2, 8, 64, 32), index_of(0, 2, "none")).shape == (0, 32)


def test_adapters_that_no_token_names_are_not_read_and_bad_entries_count_as_none():
    rows, n, k, count = 70, 200, 136, 6
    x, w, ad = randn((rows, k), 1), randn((n, k), 2, k ** -0.5), adapters(count, 16, k, n)
    index = index_of(rows, 3, "any")                       # names 0, 1, 2
    poisoned = tuple(t.clone() for t in ad)
    for t in poisoned:
        t[3:] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(check(x, w, ad, index, status=status), mk.adapted_linear(x, w, poisoned, index, status=status))
    assert status.item() == 0
    bad = index.clone()
    bad[5], bad[40], index[5], index[40] = count, 2 ** 31 - 1, -1, -1
    assert torch.equal(mk.adapted_linear(x, w, ad, bad, status=status), mk.adapted_linear(x, w, ad, index))
    assert status.item() == mk.MK_ERR_BOUNDS
    index[7] = -2 ** 31
    mk.adapted_linear(x, w, ad, index)


@pytest.mark.parametrize("rows,n,k,rank", [(5, 257, 136, 16), (12, 300, 2048, 8), (40, 130, 1032, 24), (70, 257, 136, 64), (130, 600, 2048, 16),
                                           (300, 257, 264, 32), (700, 1000, 520, 16), (2100, 2048, 264, 40), (9000, 4096, 72, 8)])
@pytest.mark.parametrize("act", [None, "silu", "swiglu"])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_infinities_and_nan_of_an_adapter_stay_with_its_tokens(rows, n, k, rank, act, out_dtype):
    f, count = 2 if act == "swiglu" else 1, 4
    x, w, ad, index = randn((rows, k), 1), randn((f * n, k), 2, k ** -0.5), adapters(count, rank, k, f * n), index_of(rows, count, "any")
    index[:5] = torch.tensor([1, 0, 2, -1, 3], dtype=torch.int32)
    bias, residual = randn((f * n,), 3), randn((rows, n), 4, dtype=out_dtype)
    want, bound = reference(x, w, ad, index, bias, act, residual, out_dtype)
    down, up, scale = (t.clone() for t in ad)
    up[1, ::3, rank - 1] = float("nan")
    up[2, 1::4, 0] = float("inf")
    up[2, 5, 1] = -float("inf")
    down[3, 2, 5] = float("nan")
    for out in (None, residual.clone()):   # (the second time in place)
        got = mk.adapted_linear(x, w, (down, up, scale), index, bias, act, residual if out is None else out, out, out_dtype)
        sound = (index <= 0).nonzero().reshape(-1)
        off = (got[sound].double() - want[sound]).abs() / bound[sound]
        assert torch.isfinite(got[sound]).all() and off.max().item() <= 1, off.max().item()
        if act is None:   # theirs are what the formula gives, and finite elsewhere
            x64 = x.double()
            for a in (1, 2, 3):
                mine = (index == a).nonzero().reshape(-1)
                t = x64[mine] @ down[a].double().T
                e = (t[:, None, :] * up[a].double()[None]).sum(2) if a < 3 else torch.full((len(mine), n), float("nan"), device="cuda").double()
                assert torch.equal(got[mine].isnan(), e.isnan()) and torch.equal(got[mine].isposinf(), e.isposinf())
                assert torch.equal(got[mine].isneginf(), e.isneginf())


def test_tokens_that_are_not_finite_leave_the_others_alone():
    rows, n, k = 60, 200, 264
    x, w, ad, index = randn((rows, k), 1), randn((n, k), 2, k ** -0.5), adapters(3, 16, k, n), index_of(rows, 3, "any")
    want = check(x, w, ad, index)
    bad = x.clone()
    bad[7, 3], bad[20], bad[21, 0] = float("nan"), float("inf"), -float("inf")
    got = mk.adapted_linear(bad, w, ad, index)
    rest = [i for i in range(rows) if i not in (7, 20, 21)]
    assert torch.equal(got[rest], want[rest]) and not torch.isfinite(got[[7, 20]]).any()


def test_large_and_tiny_low_rank_values():
    # a low-rank value near fp32's largest leaves no rest that is not finite; a tiny one keeps its parts
    x, w, index = randn((20, 64), 1), randn((40, 64), 2, 0.1), index_of(20, 2, "own")
    down, up, _ = adapters(2, 8, 64, 40)
    for big, small in ((2.0 ** 60, 2.0 ** -60), (2.0 ** -60, 2.0 ** 60)):
        check(x, w, (down * big, up * small, None), index, out_dtype=F32)


def test_strided_rows_and_residual_in_place():
    rows, n, k = 140, 99, 136
    x, w, ad, index = randn((rows, 200), 1)[:, 8:144], randn((n, k), 2, 0.1), adapters(4, 24, k, n), index_of(rows, 4, "any")
    wide = torch.full((rows, 300), 7.0, device="cuda")
    check(x, w, ad, index, residual=randn((rows, 131), 3)[:, 1:100], out=wide[:, 3:102], out_dtype=F32)
    assert (wide[:, :3] == 7).all() and (wide[:, 102:] == 7).all()
    r = randn((rows, n), 5, dtype=F32)
    want = mk.adapted_linear(x, w, ad, index, residual=r, out_dtype=F32)
    assert torch.equal(mk.adapted_linear(x, w, ad, index, residual=r, out=r), want)


def test_pieces_of_rows_where_the_terms_are_many():
    # 128 adapters of rank 256: a piece of the rows' terms fills the workspace's bound, the call is made in several
    rows, n, k, count = 5000, 64, 64, 128
    ad = adapters(count, 256, k, n)
    check(randn((rows, k), 1), randn((n, k), 2, 0.1), ad, index_of(rows, count, "any"), residual=randn((rows, n), 3), out_dtype=F32)


def test_streams_workspaces_and_repeats():
    import ctypes
    rows, n, k = 40, 300, 520
    x, w, ad, index = randn((rows, k), 1), randn((n, k), 2, 0.05), adapters(9, 16, k, n), index_of(rows, 9, "any")
    want = check(x, w, ad, index)
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s in side:
            with torch.cuda.stream(s):
                outs.append(mk.adapted_linear(x, w, ad, index))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    _, _, args = mk._linear_args(x, w, None, None, None, None, None, None)
    pack = mk._ADAPTERS.pack(9, 16, ad[0].data_ptr(), ad[1].data_ptr(), ad[2].data_ptr(), index.data_ptr())
    need = mk.lib.mk_linear_adapted_workspace(args, pack)
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    assert torch.equal(mk.adapted_linear(x, w, ad, index, workspace=ws[:need]), want) and (ws[need:] == 0x5A).all()
    with pytest.raises(mk.MkError) as e:
        mk.adapted_linear(x, w, ad, index, workspace=ws[:need - 1])
    assert e.value.status == mk.MK_ERR_CAPACITY
    with pytest.raises(mk.MkError):
        mk.adapted_linear(x, w, ad, index, workspace=ws[8:])


def test_captured_and_replayed_with_other_adapters():
    rows, n, k = 24, 640, 512
    x, w, ad, index = randn((rows, k), 1), randn((n, k), 2, 0.05), adapters(9, 16, k, n), index_of(rows, 9, "any")
    x2 = randn((rows, n), 5)
    w2, ad2 = randn((k, n), 6, 0.05), adapters(9, 32, n, k, seed=60)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y = mk.adapted_linear(x, w, ad, index, activation="silu")
        z = mk.adapted_linear(y, w2, ad2, index, residual=x, out_dtype=F32)
    for seed in (7, 8, 9):
        index.copy_(index_of(rows, 9, "any", seed))
        x.copy_(randn((rows, k), seed))
        g.replay()
        torch.cuda.synchronize()
        y1 = check(x, w, ad, index, act="silu")
        assert torch.equal(y, y1)
        assert torch.equal(z, check(y1, w2, ad2, index, residual=x, out_dtype=F32))


def test_a_call_behind_kernels_that_make_its_inputs():
    # x comes from the kernel right in front, the output is overwritten by the next call: no call starts too early
    rows, k = 16, 2048
    x0, w, ad, index = randn((rows, k), 1), randn((k, k), 2, k ** -0.5), adapters(8, 16, k, k), index_of(rows, 8, "own")
    want = [x0]
    for _ in range(4):
        want.append(mk.adapted_linear(want[-1], w, ad, index))
        torch.cuda.synchronize()
    for _ in range(20):
        a, b = torch.empty_like(x0), torch.empty_like(x0)
        x = x0
        for i in range(4):
            x = mk.adapted_linear(x, w, ad, index, out=(a, b)[i % 2])
        assert torch.equal(x, want[4])


def test_adapters_past_2_to_the_32_elements():
    # 65536 adapters of 16 x 4160: 4.4e9 elements of up; those that no token names hold whatever was there
    count, rank, n, k, rows = 65536, 16, 4160, 24, 40
    down, up = (torch.empty(shape, dtype=BF, device="cuda") for shape in ((count, rank, k), (count, n, rank)))
    names = [0, 65535, 64600, 32768]
    few = adapters(4, rank, k, n, scaled=False)
    down[names], up[names] = few[0], few[1]
    x, w, index = randn((rows, k), 1), randn((n, k), 2, k ** -0.5), index_of(rows, 4, "any")
    far = torch.tensor(names + [-1], dtype=torch.int32, device="cuda")[index.long()]
    assert torch.equal(mk.adapted_linear(x, w, (down, up), far), check(x, w, few, index))
    one = torch.full((rows,), 65535, dtype=torch.int32, device="cuda")
    assert torch.equal(mk.adapted_linear(x, w, (down, up), one, out_dtype=F32), check(x, w, few, torch.ones_like(one), out_dtype=F32))


def test_two_captured_graphs_of_one_workspace():
    rows, n, k = 30, 264, 512
    x, w, index = randn((rows, k), 1), randn((n, k), 2, 0.05), index_of(rows, 9, "any")
    sets = [adapters(9, 16, k, n, seed=s) for s in (50, 70)]
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    want = [check(x, w, ad, index) for ad in sets]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in sets], []
    torch.cuda.synchronize()
    for g, ad in zip(graphs, sets):
        with torch.cuda.graph(g):
            outs.append(mk.adapted_linear(x, w, ad, index, workspace=ws))
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])


def test_refusals():
    x, w, ad, index = randn((5, 64), 1), randn((32, 64), 2), adapters(3, 8, 64, 32), index_of(5, 3, "own")
    down, up, scale = ad
    for call in (lambda: mk.adapted_linear(x, w, (down[:, :, :56], up, scale), index), lambda: mk.adapted_linear(x, w, (down, up[:, :31], scale), index),
                 lambda: mk.adapted_linear(x, w, (down, up, scale[:2]), index), lambda: mk.adapted_linear(x, w, (down, up, scale.bfloat16()), index),
                 lambda: mk.adapted_linear(x, w, ad, index[:4]), lambda: mk.adapted_linear(x, w, ad, index.long()),
                 lambda: mk.adapted_linear(x, w, ad, index.cpu()), lambda: mk.adapted_linear(x, w, (down.float(), up, scale), index),
                 lambda: mk.adapted_linear(x, w, (down.transpose(1, 2), up, scale), index), lambda: mk.adapted_linear(x, w[:, :56], ad, index),
                 lambda: mk.adapted_linear(x, w, (down[:2], up, scale), index)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mk.MkError):
        mk.adapted_linear(x, w, (down[:, :4].contiguous(), up[:, :, :4].contiguous(), scale), index)
    with pytest.raises(mk.MkError):
        mk.adapted_linear(x, w, ad, index, out=up.reshape(-1)[:160].reshape(5, 32))
