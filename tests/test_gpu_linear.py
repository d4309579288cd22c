"""mk_linear against the formula in 64 bits: sizes from one row to many tiles, odd sizes, strides,
types, activations, residuals in place, streams and graphs.

Tolerance per output: sums are fp32 over products that are exact in fp32.  A tensor-core step adds 16
products to the running sum with an error of at most 2^-22 of the absolute sum S = sum |x w| + |b|,
so a row of k has at most (k / 16 + 2) 2^-22 S; the activations' slopes are at most 1.13 (the up
factor of SwiGLU enters as it is), expf, erff and the divisions add 2^-20 of the value; the output's rounding
is half a step of its type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def randn(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def reference(x, w, bias, act, residual, out_dtype):
    """(value, bound) in fp64."""
    y = x.double() @ w.double().T
    s = x.double().abs() @ w.double().abs().T
    if bias is not None:
        y, s = y + bias.double(), s + bias.double().abs()
    e = (x.shape[1] / 16 + 2) * 2.0 ** -22 * s
    if act == "swiglu":
        n = w.shape[0] // 2
        g, u, eg, eu = y[:, :n], y[:, n:], e[:, :n], e[:, n:]
        sg = g * torch.sigmoid(g)
        y, e = sg * u, 1.13 * eg * u.abs() + sg.abs() * eu + 1.13 * eg * eu
    elif act == "silu":
        y, e = y * torch.sigmoid(y), 1.13 * e
    elif act == "gelu":
        y, e = 0.5 * y * (1 + torch.erf(y / math.sqrt(2))), 1.13 * e
    e = e + 2.0 ** -20 * y.abs()
    if residual is not None:
        y = y + residual.double()
    return y, e + torch.finfo(out_dtype).eps / 2 * (y.abs() + e) * (1 if out_dtype == BF else 2) + 1e-37


def check(x, w, bias=None, act=None, residual=None, out=None, out_dtype=BF):
    want, bound = reference(x, w, bias, act, residual, out_dtype)
    got = mk.linear(x, w, bias=bias, activation=act, residual=residual, out=out, out_dtype=out_dtype)
    assert got.dtype == out_dtype and (out is None or got is out)
    off = (got.double() - want).abs() / bound
    assert torch.isfinite(got).all() and off.max().item() <= 1, off.max().item()
    return got


@pytest.mark.parametrize("rows", [1, 2, 8, 9, 16, 17, 33, 64, 65, 128, 129, 257, 300])
@pytest.mark.parametrize("n,k", [(1, 8), (130, 72), (257, 688)])
def test_sizes(rows, n, k):
    check(randn((rows, k), 1), randn((n, k), 2, k ** -0.5), out_dtype=F32)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [None, BF, F32])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_epilogues(act, bias, residual, out_dtype):
    for rows, n, k in ((3, 77, 136), (200, 264, 256)):
        f = 2 if act == "swiglu" else 1
        check(randn((rows, k), 1), randn((f * n, k), 2, k ** -0.5), randn((f * n,), 3) if bias else None, act,
              None if residual is None else randn((rows, n), 4, dtype=residual), out_dtype=out_dtype)


@pytest.mark.parametrize("rows,n,k,act", [(1, 2048, 2048, None), (8, 8192, 2048, "swiglu"), (40, 2048, 8192, None),
                                          (1000, 1000, 4096, "silu"), (5, 40000, 512, None), (2100, 520, 1032, "swiglu")])
def test_large(rows, n, k, act):
    f = 2 if act == "swiglu" else 1
    check(randn((rows, k), 1), randn((f * n, k), 2, k ** -0.5), act=act, residual=randn((rows, n), 3, dtype=F32), out_dtype=F32)


def test_strided_rows_and_a_broadcast_residual():
    for rows in (1, 5, 140):
        x = randn((rows, 200), 1)[:, 8:144]
        w = randn((99, 136), 2, 0.1)
        wide = torch.full((rows, 300), 7.0, device="cuda")
        check(x, w, residual=randn((rows, 131), 3)[:, 1:100], out=wide[:, 3:102], out_dtype=F32)
        assert (wide[:, :3] == 7).all() and (wide[:, 102:] == 7).all()       # nothing beside the output is written
        check(x, w, residual=randn((1, 99), 4).expand(rows, 99))


@pytest.mark.parametrize("rows", [1, 7, 64, 200])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_residual_in_place(rows, dtype):
    x, w, r = randn((rows, 264), 1), randn((130, 264), 2, 0.1), randn((rows, 130), 3, dtype=dtype)
    want = mk.linear(x, w, residual=r, out_dtype=dtype)
    assert torch.equal(mk.linear(x, w, residual=r, out=r), want)


def test_outputs_past_2_to_the_31():
    # 2.2e9 outputs: offsets need 64 bits; a few rows and columns of every corner are checked
    rows, n, k = 40000, 55000, 16
    x, w = randn((rows, k), 1), randn((n, k), 2, k ** -0.5)
    got = mk.linear(x, w)
    for r in (slice(0, 3), slice(39040, 39060), slice(rows - 3, rows)):
        want, bound = reference(x[r], w, None, None, None, BF)
        assert ((got[r].double() - want).abs() <= bound).all()


def test_captured_before_any_other_call():
    # a process whose first calls are captured: kernels are loaded and set up during the capture
    import os
    import subprocess
    import sys
    code = """
import torch, persistent_megakernel_decode_sm_gb300 as mk
from workload import KVCache
x, w = torch.randn(300, 64, device="cuda").bfloat16(), torch.randn(96, 64, device="cuda").bfloat16()
kv = KVCache(*(torch.randn(1, 1, 1, 900, 64, device="cuda").bfloat16() for _ in range(2)))
q = torch.randn(1, 4, 64, device="cuda").bfloat16()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y, o = mk.linear(x, w), mk.attend(q, kv, [1], [900])
g.replay()
torch.cuda.synchronize()
assert torch.equal(y, mk.linear(x, w)) and torch.equal(o, mk.attend(q, kv, [1], [900]))
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_c_and_python_calls_agree_and_keep_nothing(monkeypatch):
    import sys
    x, w, b = randn((5, 64), 1), randn((32, 64), 2), randn((32,), 3)
    r, out = randn((5, 32), 4), torch.empty((5, 32), device="cuda", dtype=torch.float32)
    calls = [(x, w, {}), (x, w, dict(bias=b, activation="gelu")), (x, w, dict(residual=r, out_dtype=torch.float32)),
             (x, w, dict(residual=r.float(), out=out)), (x, w, dict(bias=b, activation="swiglu", residual=r[:, :16])),
             (x[:0], w, {}), (x[1:2], w, dict(activation="silu", residual=r[:1].expand(1, 32)))]
    bad = [(x, w[:, :56], {}), (x.float(), w, {}), (x, w, dict(bias=b[:31])), (x, w, dict(activation="relu")), (x, w, dict(out=out[:4])),
           (x, w, dict(out=out, out_dtype=torch.bfloat16)), (x, w, dict(out_dtype=torch.float16)), (x, w[:31], dict(activation="swiglu")),
           (x, w, dict(residual=r[:4])), (x[0], w, {}), (x[:, 1:57], w[:, :56].contiguous(), {}), (x.T, w, {})]

    class Python:
        linear = staticmethod(lambda *a: None)

    def run(c):
        try:
            return mk.linear(c[0], c[1], **c[2]).clone()
        except (ValueError, mk.MkError) as e:
            return str(e)

    taken, refused = [run(c) for c in calls], [run(c) for c in bad]
    assert all(isinstance(t, torch.Tensor) for t in taken) and all(isinstance(t, str) for t in refused)
    with monkeypatch.context() as m:
        m.setattr(mk, "_fast", Python)
        assert all(torch.equal(run(c), t) and run(c).dtype == t.dtype for c, t in zip(calls, taken))
        assert [run(c) for c in bad] == refused
    del taken
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in (x, w, b, r, out, torch.bfloat16, torch.float32)]
    for _ in range(100):
        for c in calls + bad:
            run(c)
    assert (torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in (x, w, b, r, out, torch.bfloat16, torch.float32)]) == held


def test_no_rows():
    assert mk.linear(randn((0, 64), 1), randn((10, 64), 2)).shape == (0, 10)


def test_infinities_and_nan_stay_in_their_rows():
    x, w = randn((150, 72), 1), randn((140, 72), 2)
    clean = mk.linear(x, w, out_dtype=F32)
    x[3] = float("nan")
    x[140, 5] = float("inf")
    w[139] = float("nan")
    got = mk.linear(x, w, out_dtype=F32)
    keep = torch.ones(150, dtype=torch.bool)
    keep[[3, 140]] = False
    assert torch.equal(got[keep][:, :139], clean[keep][:, :139])
    assert got[3].isnan().all() and got[:, 139].isnan().all() and not got[140, :139].isfinite().any()


def test_extreme_activations():
    # pre-activations from -200 to 200: exp overflows, the outputs do not
    x = torch.zeros((3, 8), device="cuda", dtype=BF)
    x[:, 0] = torch.tensor([-200.0, 0.0, 200.0])
    w = torch.zeros((2, 8), device="cuda", dtype=BF)
    w[:, 0] = 1
    for act in ("silu", "gelu"):
        y = mk.linear(x, w, activation=act, out_dtype=F32)
        assert y[0].abs().max() < 1e-30 and (y[1] == 0).all() and (y[2] == 200).all()
    y = mk.linear(x, w, activation="swiglu", out_dtype=F32)
    assert y[0].abs().max() < 1e-30 and y[1] == 0 and y[2] == 40000


def test_repeatable_and_on_another_stream():
    x, w = randn((70, 2056), 1), randn((1030, 2056), 2)
    a = mk.linear(x, w, out_dtype=F32)
    for _ in range(3):
        assert torch.equal(mk.linear(x, w, out_dtype=F32), a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = mk.linear(x, w, out_dtype=F32)
    s.synchronize()
    assert torch.equal(a, b)


def test_captured_and_replayed():
    x, w, r = randn((20, 520), 1), randn((2 * 260, 520), 2, 0.05), randn((20, 260), 3)
    mk.linear(x, w, activation="swiglu", residual=r)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = mk.linear(x, w, activation="swiglu", residual=r)
    x.copy_(randn((20, 520), 9))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, mk.linear(x, w, activation="swiglu", residual=r))


def test_refuses_tensors_it_cannot_take():
    x, w = randn((4, 64), 1), randn((10, 64), 2)
    for bad in (lambda: mk.linear(x.cpu(), w), lambda: mk.linear(x.float(), w), lambda: mk.linear(x.T, w),
                lambda: mk.linear(x, w[:, :32]), lambda: mk.linear(x, w, activation="tanh"),
                lambda: mk.linear(x, w, bias=randn((9,), 3)), lambda: mk.linear(x, w, residual=randn((4, 9), 3)),
                lambda: mk.linear(x, w, out=randn((4, 9), 3)), lambda: mk.linear(x[0], w),
                lambda: mk.linear(x, randn((9, 64), 2), activation="swiglu"), lambda: mk.linear(x, w, out_dtype=torch.float16),
                lambda: mk.linear(x, w, out=randn((4, 10), 3), out_dtype=F32), lambda: mk.linear(x, w.T.contiguous().T)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(mk.MkError) as e:
        mk.linear(randn((4, 68), 1)[:, :64], w)      # rows 136 bytes apart
    assert e.value.status == mk.MK_ERR_ARG
    with pytest.raises(mk.MkError):
        mk.linear(randn((4, 60), 1), randn((10, 60), 2))
    with pytest.raises(mk.MkError):
        mk.linear(x, randn((64, 64), 2), out=x)
