"""mk_linear_adapted's tiles of tokens where tokens name many adapters: a wide tile multiplies each of its tokens by every adapter that any
of them names, so the tile's width has to go by how many that may be.  The workspace, [rows][parts][columns of the tile's adapters], shows it."""
import ctypes
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from test_gpu_adapted import BF, F32, adapters, check, index_of, randn  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def nothing_left_behind():
    yield
    gc.collect()


def adapters_of_a_tile(rows, n, k, rank, count, dtype):
    a, ad = mk.mk_linear_args(rows=rows, n=n, k=k, out_dtype=dtype), mk.mk_adapters(n_adapters=count, rank=rank)
    need = mk.lib.mk_linear_adapted_workspace(ctypes.addressof(a), ctypes.addressof(ad))
    return need / (rows * (3 if dtype else 2) * 2 * rank)   # (a little above: the list of adapters, alignment)


@pytest.mark.parametrize("rows,n,k,rank,most", [(128, 4096, 4096, 64, 64), (256, 4096, 4096, 64, 64), (512, 4096, 4096, 16, 128), (512, 4096, 4096, 64, 128),
                                                (2048, 2048, 2048, 64, 128)])
@pytest.mark.parametrize("dtype", [mk.BF16, mk.F32])
def test_tiles_are_narrower_where_adapters_may_be_many(rows, n, k, rank, most, dtype):
    assert adapters_of_a_tile(rows, n, k, rank, 256, dtype) < 1.1 * most


def test_tiles_stay_wide_where_they_are_few():
    for rows, count in ((4096, 8), (4096, 64)):   # (pairs of CTAs: 256 tokens, or all the adapters there are)
        assert adapters_of_a_tile(rows, 8192, 2048, 16, count, mk.BF16) > 0.99 * count


@pytest.mark.parametrize("rows", [63, 64, 65, 96, 128, 257, 511, 513, 1100])
@pytest.mark.parametrize("rank", [16, 64])
def test_every_token_its_own(rows, rank):
    n, k = 330, 520
    for dtype in (BF, F32):
        check(randn((rows, k), 1), randn((n, k), 2, k ** -0.5), adapters(256, rank, k, n), index_of(rows, 256, "own"), out_dtype=dtype)
