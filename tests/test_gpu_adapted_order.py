"""mk_linear_adapted behind kernels that have only just written its operands: what it reads beside the kernel in front of its
products is what was written last, call after call on the same addresses."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def nothing_left_behind():
    yield
    gc.collect()


def randn(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("rows,n,k,act", [(1, 2048, 2048, None), (9, 640, 512, "swiglu"), (64, 1030, 2048, None), (150, 514, 264, "gelu"),
                                          (1024, 2048, 256, None), (1024, 1024, 256, "swiglu")])
@pytest.mark.parametrize("captured", [False, True])
def test_operands_written_right_in_front(rows, n, k, act, captured):
    f, count, sets = 2 if act == "swiglu" else 1, 5, 3
    w = randn((f * n, k), 2, k ** -0.5)
    ad = randn((count, 16, k), 3, k ** -0.5), randn((count, f * n, 16), 4, 0.25), None
    given = []
    for s in range(sets):   # x, bias, residual, index
        r = torch.Generator().manual_seed(s)
        given.append((randn((rows, k), 10 + s), randn((f * n,), 20 + s), randn((rows, n), 30 + s, dtype=F32),
                      torch.randint(-1, count, (rows,), generator=r).to(torch.int32).cuda()))
    want = []
    for x, bias, residual, index in given:
        want.append(mk.adapted_linear(x, w, ad, index, bias, act, residual))
        torch.cuda.synchronize()
    at = [t.clone() for t in given[0]]
    outs = [torch.empty_like(want[0]) for _ in range(4 * sets)]

    def steps():
        for i, out in enumerate(outs):
            for t, v in zip(at, given[i % sets]):
                t.copy_(v)
            mk.adapted_linear(at[0], w, ad, at[3], at[1], act, at[2], out=out)

    if captured:
        steps()   # (kernels' attributes are set outside of the capture too)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            steps()
        run = g.replay
    else:
        run = steps
    for _ in range(5):
        for out in outs:
            out.zero_()
        run()
        for i, out in enumerate(outs):
            assert torch.equal(out, want[i % sets])


@pytest.mark.parametrize("rows,n,k,rank,count", [(64, 514, 2048, 64, 64), (300, 257, 688, 24, 5), (1024, 512, 264, 16, 40)])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_rows_in_another_order(rows, n, k, rank, count, out_dtype):
    """Each order is within its bound, and the same again; bits may differ between them."""
    from test_gpu_adapted import adapters, check, index_of
    x, w, ad, index = randn((rows, k), 1), randn((n, k), 2, k ** -0.5), adapters(count, rank, k, n), index_of(rows, count, "any")
    for seed in range(3):
        order = torch.randperm(rows, generator=torch.Generator().manual_seed(seed)).cuda()
        got = check(x[order], w, ad, index[order], out_dtype=out_dtype)
        assert torch.equal(got, mk.adapted_linear(x[order], w, ad, index[order], out_dtype=out_dtype))
