"""mk_linear_adapted_workspace before any buffer exists: the size of a call is that of its sizes, activation and types."""
import ctypes
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def nothing_left_behind():
    """A later module's tests look at the memory."""
    yield
    gc.collect()


def size(linear, adapters):
    return mk.lib.mk_linear_adapted_workspace(ctypes.addressof(linear), ctypes.addressof(adapters))


@pytest.mark.parametrize("rows,n,k,rank,count", [(1, 64, 64, 8, 1), (8, 512, 256, 16, 40), (64, 1001, 688, 64, 64), (300, 2048, 264, 256, 7), (5000, 64, 64, 256, 128)])
@pytest.mark.parametrize("act", [0, 3])
@pytest.mark.parametrize("dtype", [mk.BF16, mk.F32])
def test_sized_before_its_buffers(rows, n, k, rank, count, act, dtype):
    f = 2 if act == 3 else 1
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w, down, up = torch.zeros(rows, k, **bf), torch.zeros(f * n, k, **bf), torch.zeros(count, rank, k, **bf), torch.ones(count, f * n, rank, **bf)
    index, out = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.ones(rows, n, dtype=torch.float32 if dtype else torch.bfloat16, device="cuda")
    sizes = dict(rows=rows, n=n, k=k, activation=act, out_dtype=dtype)
    a = mk.mk_linear_args(**sizes, x=x.data_ptr(), x_stride=k, w=w.data_ptr(), out=out.data_ptr(), out_stride=n)
    ad = mk.mk_adapters(n_adapters=count, rank=rank, down=down.data_ptr(), up=up.data_ptr(), index=index.data_ptr())
    need = size(a, ad)
    assert need > 0 and size(mk.mk_linear_args(**sizes), mk.mk_adapters(n_adapters=count, rank=rank)) == need
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    call = lambda bytes_: mk.lib.mk_linear_adapted(ctypes.addressof(a), ctypes.addressof(ad), ws.data_ptr(), bytes_, stream)   # noqa: E731
    assert call(need - 1) == mk.MK_ERR_CAPACITY and call(need) == mk.MK_OK
    assert not out.any()


def test_sizes_that_are_not_valid_have_none():
    good = dict(rows=4, n=64, k=64)
    ad = mk.mk_adapters(n_adapters=3, rank=8)
    assert size(mk.mk_linear_args(**good), ad) > 0
    for over in (dict(rows=0), dict(rows=-1), dict(n=0), dict(k=60), dict(activation=4), dict(out_dtype=7)):
        assert size(mk.mk_linear_args(**{**good, **over}), ad) == 0
    for bad in (dict(n_adapters=0, rank=8), dict(n_adapters=65537, rank=8), dict(n_adapters=3, rank=12), dict(n_adapters=3, rank=264)):
        assert size(mk.mk_linear_args(**good), mk.mk_adapters(**bad)) == 0
