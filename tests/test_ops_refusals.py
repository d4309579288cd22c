"""The prompt operators' C entry points refuse bad arguments before anything is launched (no GPU
needed: every call below fails its host checks, or has nothing to do)."""
import ctypes

import pytest

mk = pytest.importorskip("persistent_megakernel_decode_sm_gb300")

A = 1 << 20          # an aligned address that is never dereferenced


def linear_args(**over):
    f = dict(rows=4, n=24, k=64, activation=0, x=A, x_stride=64, w=2 * A, bias=None, residual=None, residual_stride=0,
             residual_dtype=mk.BF16, out_dtype=mk.BF16, out=3 * A, out_stride=24, status=None)
    f.update(over)
    return mk.mk_linear_args(*[f[n] for n, _ in mk.mk_linear_args._fields_])


@pytest.mark.parametrize("over", [
    dict(rows=-1), dict(rows=(1 << 30) + 1), dict(n=(1 << 30) + 1, out_stride=1 << 31), dict(n=0), dict(k=0), dict(k=60), dict(activation=4), dict(activation=-1), dict(out_dtype=2),
    dict(residual=4 * A, residual_stride=24, residual_dtype=5), dict(x=None), dict(w=None), dict(out=None),
    dict(x=A + 2), dict(w=2 * A + 8), dict(out=3 * A + 1), dict(out_dtype=mk.F32, out=3 * A + 2), dict(bias=A + 1),
    dict(residual=4 * A + 2, residual_stride=24, residual_dtype=mk.F32), dict(status=A + 2),
    dict(x_stride=56), dict(x_stride=68), dict(out_stride=23), dict(residual=4 * A, residual_stride=23),
    dict(residual=4 * A, residual_stride=-24),
    dict(out=A), dict(out=A + 64 * 2 - 16), dict(out=2 * A + 8), dict(bias=3 * A),          # out overlaps an input
    dict(residual=3 * A + 2, residual_stride=24),                                            # and a shifted residual
    dict(residual=3 * A, residual_stride=24, residual_dtype=mk.F32),                         # and one of another type
    dict(residual=3 * A, residual_stride=0),                                                 # and one broadcast row
])
def test_linear_refuses(over):
    assert mk.lib.mk_linear(ctypes.byref(linear_args(**over)), None) == mk.MK_ERR_ARG
    assert mk.lib.mk_last_error()


def test_linear_refuses_null_and_takes_no_rows():
    assert mk.lib.mk_linear(None, None) == mk.MK_ERR_ARG
    assert mk.lib.mk_linear(ctypes.byref(linear_args(rows=0, x=None, w=None, out=None)), None) == mk.MK_OK


def attend_args(q_lens=(1, 2), kv_lens=(5, 9), kv=None, pages=None, **over):
    n = len(q_lens)
    kv = kv or mk.mk_kv(5 * A, 6 * A, 2 * 64 * 32, 2 * 64 * 32, 64 * 32)
    f = dict(n_q_heads=4, n_kv_heads=2, head_dim=32, batch=n, q_lens=(ctypes.c_int32 * max(n, 1))(*q_lens),
             kv_lens=(ctypes.c_int32 * max(n, 1))(*kv_lens), q=A, q_stride=128, out=2 * A, out_stride=128, kv=ctypes.pointer(kv),
             pages=None if pages is None else ctypes.pointer(pages), layer=0, max_seq=64, window=0, sinks=0,
             shared_prefix=0, scale=0.0, status=None)
    f.update(over)
    return mk.mk_attend_args(*[f[n] for n, _ in mk.mk_attend_args._fields_])


@pytest.mark.parametrize("over", [
    dict(n_q_heads=5), dict(n_kv_heads=0), dict(n_q_heads=0), dict(n_q_heads=18), dict(head_dim=48), dict(head_dim=256),
    dict(batch=0), dict(batch=257), dict(q_lens=(-1, 2)), dict(kv_lens=(5, -9)), dict(kv_lens=(5, 65)), dict(max_seq=0),
    dict(layer=-1), dict(window=-1), dict(sinks=-1), dict(shared_prefix=-1), dict(shared_prefix=5), dict(scale=-1.0),
    dict(shared_prefix=3, window=8), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(out=None),
    dict(q=A + 8), dict(out=2 * A + 4), dict(q_stride=120), dict(q_stride=132), dict(out_stride=64), dict(status=A + 1),
    dict(out=A), dict(out=A + 64),                                                           # out overlaps q
    dict(out=5 * A + 64), dict(out=6 * A), dict(layer=1, out=5 * A + 2 * 4096),                # and the cache
    dict(layer=1, kv=mk.mk_kv(5 * A, 6 * A, 4096, 2048, 2048)),                              # layers overlap
    dict(kv=mk.mk_kv(None, A, 4096, 4096, 2048)), dict(kv=mk.mk_kv(5 * A + 8, 6 * A, 4096, 4096, 2048)),
    dict(kv=mk.mk_kv(5 * A, 6 * A, 4096, 4096, 2040)),                                       # heads do not cover max_seq
    dict(kv=mk.mk_kv(5 * A, 6 * A, 4088, 4096, 2048)),                                       # sequences overlap
    dict(kv=mk.mk_kv(5 * A, 6 * A, 4100, 4096, 2048)),
    dict(pages=mk.mk_kv_pages(None, 16, 4, 9)), dict(pages=mk.mk_kv_pages(7 * A, 12, 9, 4)),
    dict(pages=mk.mk_kv_pages(7 * A, 16, 3, 4)),                                             # the table does not cover max_seq
    dict(pages=mk.mk_kv_pages(7 * A, 16, 4, 0)), dict(pages=mk.mk_kv_pages(7 * A, 16, 4, 5)),  # pool larger than a head
])
def test_attend_refuses(over):
    a = attend_args(**over)
    assert mk.lib.mk_attend(ctypes.byref(a), None, 0, None) == mk.MK_ERR_ARG
    assert mk.lib.mk_last_error()


def test_attend_refuses_null_and_takes_no_tokens():
    assert mk.lib.mk_attend(None, None, 0, None) == mk.MK_ERR_ARG
    assert mk.lib.mk_attend_workspace(None) == 0
    assert mk.lib.mk_attend_workspace(ctypes.byref(attend_args(head_dim=48))) == 0
    a = attend_args(q_lens=(0, 0), q=None, out=None)
    assert mk.lib.mk_attend_workspace(ctypes.byref(a)) == 0
    assert mk.lib.mk_attend(ctypes.byref(a), None, 0, None) == mk.MK_OK


def test_operands_off_the_gpu_are_named():
    torch = pytest.importorskip("torch")
    x = torch.ones(2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        mk.linear(x, x)
    kv = type("KV", (), dict(k=torch.ones(1, 1, 1, 8, 32, dtype=torch.bfloat16), v=torch.ones(1, 1, 1, 8, 32, dtype=torch.bfloat16)))
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        mk.attend(torch.ones(1, 1, 32, dtype=torch.bfloat16), kv, [1], [8])
    with pytest.raises(AttributeError):
        mk.linear(None, x)


def test_call_module_hands_over_what_it_does_not_take():
    # nothing is kept or raised by a call that it leaves to Python
    import sys
    torch = pytest.importorskip("torch")
    fast = mk._fast or mk._setup()
    x = torch.ones(2, 16, dtype=torch.bfloat16)
    linear = ((), (x,), (x, x, None, None, None, None, None, None), (1, 2, 3, 4, 5, 6, 7, 8), (x, x, x, "tanh", x, x, 5, x))
    attend = ((), (x,) * 14, (x, x, x, [1], [2], 0, 0, 0, 0, None, None, None, None, None), (None,) * 14)

    def counts():
        return sys.getrefcount(x), sys.getrefcount(torch.bfloat16)

    before = counts()
    results = {id(f(*args)) for _ in range(50) for f, calls in ((fast.linear, linear), (fast.attend, attend)) for args in calls}
    after = counts()
    assert results == {id(None)} and after == before
    with pytest.raises(TypeError):
        fast.setup(1)
