"""mk_linear_adapted where outputs are NaN in their own right (a token, a weight, a bias or the token's own adapter is not finite): they are
NaN, nothing else changes, and the call takes no longer for them than for others.  Only another adapter's infinity or NaN beside a token in its tile,
or the token's own infinities, have its outputs worked out again."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from test_gpu_adapted import BF, F32, adapters, index_of, randn, reference  # noqa: E402

NAN, INF = float("nan"), float("inf")
SHAPES = [(1, 300, 264, 16), (5, 257, 136, 16), (12, 300, 2048, 8), (70, 257, 136, 64), (130, 600, 2048, 24), (300, 257, 264, 32), (2100, 1030, 264, 40)]


@pytest.fixture(scope="module", autouse=True)
def nothing_left_behind():
    yield
    gc.collect()


@pytest.mark.parametrize("rows,n,k,rank", SHAPES)
@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("foreign", [False, True])
def test_what_is_nan_in_its_own_right(rows, n, k, rank, act, out_dtype, foreign):
    """Every kind of NaN at once, without and with another adapter (the last) that is not finite for some features."""
    f, count = 2 if act == "swiglu" else 1, 4
    x, w, index = randn((rows, k), 1), randn((f * n, k), 2, k ** -0.5), index_of(rows, count, "any")
    ad, bias, residual = adapters(count, rank, k, f * n), randn((f * n,), 3), randn((rows, n), 4, dtype=out_dtype)
    want, bound = reference(x, w, ad, index, bias, act, residual, out_dtype)
    down, up, scale = (t.clone() for t in ad)
    nan = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
    lost = torch.arange(rows, device="cuda") % 7 == 3
    x[lost, k - 1] = NAN
    nan |= lost[:, None]
    w[2], bias[f * n - 1], residual[rows // 2, 4] = NAN, NAN, NAN
    nan[:, 2] = True
    nan[:, n - 1] = True
    nan[rows // 2, 4] = True
    up[1, 9], down[2, rank // 2, 1] = NAN, NAN
    nan[index == 1, 9] = True
    nan[index == 2] = True
    if foreign:
        up[3, 1::5] = NAN
        nan[:, torch.arange(1, f * n, 5, device="cuda") % n] |= (index == 3)[:, None]
    for out in (None, residual.clone()):   # (the second time in place)
        got = mk.adapted_linear(x, w, (down, up, scale), index, bias, act, residual if out is None else out, out, out_dtype)
        assert torch.equal(got.isnan(), nan)
        assert not bool((((got.double() - want).abs() > bound) & ~nan).any())


@pytest.mark.parametrize("rows,n,k,rank", SHAPES)
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_own_infinities_are_the_formula_s(rows, n, k, rank, out_dtype):
    """Infinite `up` rows times low-rank values whose parts have either sign, alone in their tile and beside others."""
    x, w = randn((rows, k), 1), randn((n, k), 2, k ** -0.5)
    for count in (1, 3):
        down, up, scale = adapters(count, rank, k, n)
        index = index_of(rows, count, "own")
        want, bound = reference(x, w, (down, up, scale), index, None, None, None, out_dtype)
        up[0, ::3, 0], up[0, 1::3, rank - 1] = INF, -INF
        t = x.double() @ down[0].double().T
        mine = index == 0
        got = mk.adapted_linear(x, w, (down, up, scale), index, out_dtype=out_dtype)
        for column, sign, features in ((0, 1, slice(0, None, 3)), (rank - 1, -1, slice(1, None, 3))):
            assert torch.equal(got[mine, features], (sign * t[mine, column].sign() * INF)[:, None].expand_as(got[mine, features]).to(out_dtype))
            want[mine, features] = 0
            got[mine, features] = 0
        assert not bool(((got.double() - want).abs() > bound).any())


def test_parts_that_overflow_are_taken_in_one_piece():
    # t u is beyond fp32's range in t's two parts of different signs, and so is the sum: an infinity, not NaN
    rows, n, k, rank = 20, 40, 64, 8
    x, w, index = randn((rows, k), 1), randn((n, k), 2, 0.1), index_of(rows, 1, "own")
    x[:, 0] = 1
    down, up = torch.zeros(1, rank, k, dtype=BF, device="cuda"), torch.zeros(1, n, rank, dtype=BF, device="cuda")
    down[0, 0, 0], down[0, 1, 0], up[0, :, 0] = 2.0 ** 100, 0, 2.0 ** 60
    down[0, 0, 1], x[:, 1] = -2.0 ** 91, 1   # (t = 2^100 - 2^91: its parts are 2^100 and -2^91)
    for dtype in (BF, F32):
        assert bool((mk.adapted_linear(x, w, (down, up, None), index, out_dtype=dtype) == INF).all())


@pytest.mark.parametrize("what", ["tokens", "all tokens", "own up", "own down"])
def test_takes_no_longer(what):
    """4096 tokens, of which 512 or all are NaN, or one adapter that is, alone in its tiles: taking each of these outputs again took 30
    times as long as the call."""
    rows, n, k, rank, count = 4096, 2048, 1024, 16, 4
    x, w, ad = randn((rows, k), 1), randn((2 * n, k), 2, k ** -0.5), adapters(count, rank, k, 2 * n)
    index = (torch.arange(rows) // 1024).to(torch.int32).cuda()   # (a tile of 256 names one)

    def us():
        call = lambda: mk.adapted_linear(x, w, ad, index, activation="swiglu")   # noqa: E731
        call()
        best = 1e9
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                call()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) * 250)
        return best

    clean = us()
    if what == "tokens":
        x[:512] = NAN
    elif what == "all tokens":
        x[:] = NAN
    elif what == "own up":
        ad[1][2] = NAN
    else:
        ad[0][2] = NAN
    assert us() < 4 * clean + 100
