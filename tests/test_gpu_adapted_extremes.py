"""mk_linear_adapted with low-rank values at the end of fp32's range and beyond it.  Tolerances are test_gpu_adapted.py's: they are
relative to the absolute sums, which these values do not change."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from test_gpu_adapted import BF, F32, adapters, check, index_of, randn, reference  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def nothing_left_behind():
    yield
    gc.collect()


@pytest.mark.parametrize("rows", [2, 20, 300])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_low_rank_values_that_bf16_would_round_to_infinity(rows, out_dtype):
    # (2 - 2^-9) 2^127 is finite in fp32 and above bf16's largest value, (2 - 2^-7) 2^127, by more than half a step
    n, k, rank = 70, 64, 8
    x, w = randn((rows, k), 1), randn((n, k), 2, 0.1)
    x[:, :2] = 1
    down, up = torch.zeros(2, rank, k, dtype=BF, device="cuda"), randn((2, n, rank), 3, 2.0 ** -120)
    down[:, :, 0], down[:, :, 1] = (2 - 2.0 ** -7) * 2.0 ** 127, 0.75 * 2.0 ** 120
    down[1] *= -1
    check(x, w, (down, up, None), index_of(rows, 2, "own"), out_dtype=out_dtype)
    check(x, w, (down / 2, up, torch.full((2,), 2.0, device="cuda")), index_of(rows, 2, "any"), out_dtype=out_dtype)


@pytest.mark.parametrize("rows,n,k,rank", [(1, 2048, 2048, 8), (5, 257, 136, 16), (12, 300, 2048, 8), (40, 130, 1032, 24), (70, 257, 136, 64),
                                           (300, 257, 264, 40), (2100, 2048, 264, 8)])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("where", ["down", "scale", "scale_negative", "x"])
def test_infinite_low_rank_rows(rows, n, k, rank, out_dtype, where):
    # products of one sign, so that the formula's sums are infinities, not NaN; the rank's padding must not make them NaN
    count = 4
    x, w = randn((rows, k), 1).abs() + 0.5, randn((n, k), 2, k ** -0.5)
    down, up, scale = adapters(count, rank, k, n)
    down, up = (down.abs() + 0.001).to(BF), (up.abs() + 0.01).to(BF)
    index = index_of(rows, count, "any")
    index[:1] = 1
    mine = (index == 1).nonzero().reshape(-1)
    rest = (index != 1).nonzero().reshape(-1)
    want, bound = reference(x, w, (down, up, scale), index, None, None, None, out_dtype)
    if where == "down":
        down[1, rank - 1, 5] = float("inf")
    elif where == "x":
        w = w.abs()
        want, bound = reference(x, w, (down, up, scale), index, None, None, None, out_dtype)
        x[mine, 7] = float("inf")
    else:
        scale[1] = float("inf") if where == "scale" else -float("inf")
    got = mk.adapted_linear(x, w, (down, up, scale), index, out_dtype=out_dtype)
    assert bool((got[mine] == (-float("inf") if where == "scale_negative" else float("inf"))).all())
    if len(rest):
        off = (got[rest].double() - want[rest]).abs() / bound[rest]
        assert torch.isfinite(got[rest]).all() and off.max().item() <= 1, off.max().item()
    # and with a zero among the adapter's values the formula's inf times 0: NaN for its tokens alone
    up[1, n // 2] = 0
    if where != "down":
        got = mk.adapted_linear(x, w, (down, up, scale), index, out_dtype=out_dtype)
        assert got[mine, n // 2].isnan().all() and torch.isfinite(got[rest]).all()
        got[:, n // 2] = 0
        assert not got.isnan().any()
