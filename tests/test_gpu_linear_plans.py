"""mk_linear in every way it cuts a call: each tile width and the CTA pairs, the contraction in one piece and shared
out, a CTA's several tiles, both output types, with and without SwiGLU.  The shapes are found by asking mk_linear_plan,
whose choice depends on how many clusters the GPU at hand keeps resident.

Error in norm of an fp32 output: sums are taken 512 terms at a time in the tensor core, 32 steps of 16, and each step
cuts the running sum off, by 2^-24 of it in the mean (uniform up to 2^-23).  The sum's size grows like the root of the step, so a
piece is off by at most (2/3 32 + 1) 2^-24 = 1.4e-6 of its size, and the sum of pieces, which are independent, by the
same of its own.  (In one piece 16392 terms are off by some 3e-6.)"""
import ctypes
import functools
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from test_gpu_linear import BF, F32, check, randn  # noqa: E402

A = 1 << 20   # an aligned address: plans read no operand
ROWS = (1, 5, 16, 17, 33, 40, 64, 65, 100, 129, 200, 257, 300, 511, 600, 900, 1025, 1300, 2049, 3000, 4097)
OUTS = (1, 129, 300, 520, 1030, 2056, 3000, 4100, 8200, 20000)
INS = (64, 136, 520, 1032, 2056, 4104, 8200, 16392)


def plan(rows, n, k, act, dtype):
    a = mk.mk_linear_args(rows, n, k, mk.ACTIVATIONS[act], A, k, 1 << 40, None, None, 0, 0, mk.F32 if dtype == F32 else mk.BF16, 1 << 42, n, None)
    p = (ctypes.c_int32 * 6)()
    assert mk.lib.mk_linear_plan(ctypes.byref(a), p) == mk.MK_OK, mk.lib.mk_last_error()
    return tuple(p)


@functools.lru_cache(None)
def shapes(act, dtype):
    """{(unit, tokens, split, whether a CTA makes several tiles): the least work found for it}"""
    torch.zeros(1, device="cuda")
    found = {}
    for rows, n, k in itertools.product(ROWS, OUTS, INS):
        if rows * n * k <= 1.5e11:
            unit, _, tokens, split, tiles, clusters = plan(rows, n, k, act, dtype)
            key, work = (unit, tokens, split, tiles > clusters), rows * n * k
            if key not in found or work < found[key][0]:
                found[key] = (work, (rows, n, k))
    return {key: shape for key, (_, shape) in found.items()}


@pytest.mark.parametrize("unit,tokens,split", [(1, t, s) for t in (16, 32, 64, 128) for s in (0, 1, 2, 3, 4, 5, 6, 8)] +
                         [(2, 256, s) for s in (0, 1, 2, 3, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_every_plan(act, dtype, unit, tokens, split):
    key = (unit, tokens, max(split, 1), split == 0)       # (0: uncut tiles, several a CTA)
    shape = shapes(act, dtype).get(key)
    if shape is None and (unit, split) in ((1, 3), (1, 5), (1, 6), (2, 3), (2, 4)):
        pytest.skip("not chosen on this GPU")
    rows, n, k = shape
    f = 2 if act else 1
    x, w, b = randn((rows, k), 1), randn((f * n, k), 2, k ** -0.5), randn((f * n,), 3)
    r = randn((rows, n), 4, dtype=dtype)
    got = check(x, w, b, act, r, out_dtype=dtype)
    assert torch.equal(mk.linear(x, w, bias=b, activation=act, residual=r, out=r), got)       # in place


@pytest.mark.parametrize("act,bias", [("silu", True), ("gelu", True), (None, False)])
@pytest.mark.parametrize("split", [0, 2])
def test_pairs_with_other_epilogues(act, bias, split):
    rows, n, k = shapes(None, BF)[2, 256, max(split, 1), split == 0]
    check(randn((rows, k), 1), randn((n, k), 2, k ** -0.5), randn((n,), 3) if bias else None, act, randn((rows, n), 4, dtype=F32))


@pytest.mark.parametrize("rows,n,k", [(3, 1030, 16392), (300, 2056, 16392), (1025, 2056, 16392), (4097, 4100, 2056), (4097, 2056, 8200)])
def test_fp32_error_in_norm(rows, n, k):
    x, w = randn((rows, k), 1), randn((n, k), 2)
    got = mk.linear(x, w, out_dtype=F32)
    want = x.double() @ w.double().T
    off = ((got.double() - want).norm() / want.norm()).item()
    assert off <= 1.4e-6, off


def test_plan_refusals():
    p = (ctypes.c_int32 * 6)()
    good = mk.mk_linear_args(4, 24, 64, 0, A, 64, 2 * A, None, None, 0, 0, 0, 3 * A, 24, None)
    assert mk.lib.mk_linear_plan(ctypes.byref(good), p) == mk.MK_OK and list(p)[:3] == [1, 128, 16]
    for over in (dict(rows=0), dict(rows=-1), dict(k=60), dict(out=A), dict(x=None)):
        a = mk.mk_linear_args.from_buffer_copy(good)
        for name, value in over.items():
            setattr(a, name, value)
        assert mk.lib.mk_linear_plan(ctypes.byref(a), p) == mk.MK_ERR_ARG
    assert mk.lib.mk_linear_plan(ctypes.byref(good), None) == mk.MK_ERR_ARG
    assert mk.lib.mk_linear_plan(None, p) == mk.MK_ERR_ARG
