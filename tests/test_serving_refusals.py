"""The C entry points around the paged cache refuse bad arguments before anything is launched (no GPU needed: every call below
fails its host checks, or has nothing to do)."""
import ctypes
import math

import pytest

mk = pytest.importorskip("persistent_megakernel_decode_sm_gb300")

A = 1 << 20          # an aligned address that is never dereferenced


def fields(struct, f, over):
    assert set(over) <= set(f)
    f.update(over)
    return struct(*[f[n] for n, _ in struct._fields_])


def linear_args(**over):
    return fields(mk.mk_linear_args, dict(rows=4, n=24, k=64, activation=0, x=A, x_stride=64, w=2 * A, bias=None, residual=None, residual_stride=0,
                                          residual_dtype=mk.BF16, out_dtype=mk.BF16, out=3 * A, out_stride=24, status=None), over)


def adapters(**over):
    return fields(mk.mk_adapters, dict(n_adapters=3, rank=8, down=4 * A, up=5 * A, scale=6 * A, index=7 * A), over)


@pytest.mark.parametrize("linear,over", [
    (dict(rows=-1), {}), (dict(k=60), {}), (dict(activation=9), {}), (dict(x=None), {}), (dict(out=A), {}), (dict(x_stride=56), {}),
    ({}, dict(n_adapters=0)), ({}, dict(n_adapters=65537)), ({}, dict(rank=0)), ({}, dict(rank=12)), ({}, dict(rank=264)), ({}, dict(rank=-8)),
    ({}, dict(down=None)), ({}, dict(up=None)), ({}, dict(index=None)), ({}, dict(down=4 * A + 8)), ({}, dict(up=5 * A + 2)),
    ({}, dict(scale=6 * A + 2)), ({}, dict(index=7 * A + 1)),
    ({}, dict(down=3 * A)), ({}, dict(up=3 * A + 32)), ({}, dict(scale=3 * A + 4)), ({}, dict(index=3 * A)),   # out overlaps an input
    (dict(out=5 * A + 3 * 24 * 8 * 2 - 16), {}), (dict(out=4 * A + 3 * 8 * 64 * 2 - 32), {}),
])
def test_linear_adapted_refuses(linear, over):
    a, ad = linear_args(**linear), adapters(**over)
    assert mk.lib.mk_linear_adapted(ctypes.byref(a), ctypes.byref(ad), 8 * A, 1 << 30, None) == mk.MK_ERR_ARG
    assert mk.lib.mk_last_error()


def test_linear_adapted_refuses_null_and_takes_no_rows():
    a, none = linear_args(), linear_args(rows=0, x=None, w=None, out=None)
    ad, empty = adapters(), adapters(down=None, up=None, index=None, scale=None)
    for args in ((None, ctypes.byref(ad)), (ctypes.byref(a), None), (None, None)):
        assert mk.lib.mk_linear_adapted(*args, 8 * A, 1 << 30, None) == mk.MK_ERR_ARG
        assert mk.lib.mk_linear_adapted_workspace(*args) == 0
    assert mk.lib.mk_linear_adapted(ctypes.byref(none), ctypes.byref(empty), None, 0, None) == mk.MK_OK
    assert mk.lib.mk_linear_adapted_workspace(ctypes.byref(none), ctypes.byref(empty)) == 0
    assert mk.lib.mk_linear_adapted_workspace(ctypes.byref(a), ctypes.byref(adapters(rank=9))) == 0


KEEP = []


def rope_args(kv=None, freqs=None, sections=None, **over):
    kv = kv or mk.mk_kv(5 * A, 6 * A, 2 * 64 * 32, 2 * 64 * 32, 64 * 32)
    freqs = (ctypes.c_double * 128)(*(freqs or [1.0] * 128))
    sections = None if sections is None else (ctypes.c_int32 * max(len(sections), 1))(*sections)
    KEEP.append((kv, freqs, sections))
    return fields(mk.mk_rope_args, dict(
        tokens=4, n_q_heads=4, n_kv_heads=2, head_dim=32, qkv=A, qkv_stride=256, qkv_dtype=mk.BF16, rotary=32, q_gain=None, k_gain=None, eps=1e-5,
        neighbours=0, n_axes=1, sections=sections, freqs=freqs, positions=2 * A, position_stride=0, slots=3 * A, kv=ctypes.pointer(kv), layer=0, max_seq=64,
        sequences=2, q=4 * A, q_stride=128, status=None), over)


@pytest.mark.parametrize("over", [
    dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(head_dim=0), dict(head_dim=24), dict(head_dim=272), dict(n_q_heads=0), dict(n_kv_heads=0),
    dict(n_q_heads=4096), dict(n_kv_heads=2 ** 31 - 1), dict(rotary=-16), dict(rotary=24), dict(rotary=48), dict(neighbours=2), dict(qkv_dtype=2), dict(eps=-1.0),
    dict(eps=math.inf), dict(eps=math.nan), dict(n_axes=0), dict(n_axes=5), dict(n_axes=2), dict(n_axes=2, sections=[8, 9], position_stride=4),
    dict(n_axes=2, sections=[-4, 20], position_stride=4), dict(n_axes=1, sections=[15]), dict(n_axes=2, sections=[8, 8], position_stride=3),
    dict(freqs=[math.nan] + [1.0] * 127), dict(freqs=[1.0] * 15 + [math.inf] + [1.0] * 112), dict(max_seq=0), dict(sequences=0), dict(max_seq=1 << 30, sequences=2),
    dict(layer=-1), dict(qkv=None), dict(q=None), dict(slots=None), dict(positions=None), dict(qkv=A + 8), dict(q=4 * A + 2), dict(q_gain=A + 4),
    dict(k_gain=A + 8), dict(positions=2 * A + 2), dict(slots=3 * A + 1), dict(status=A + 2), dict(qkv_stride=248), dict(qkv_stride=252), dict(q_stride=120),
    dict(q_stride=132), dict(qkv_dtype=mk.F32, qkv_stride=258), dict(kv=mk.mk_kv(None, A, 4096, 4096, 2048)), dict(kv=mk.mk_kv(5 * A + 8, 6 * A, 4096, 4096, 2048)),
    dict(kv=mk.mk_kv(5 * A, 6 * A, 4096, 4096, 2040)), dict(kv=mk.mk_kv(5 * A, 6 * A, 4088, 4096, 2048)), dict(kv=mk.mk_kv(5 * A, 6 * A, 4100, 4096, 2048)),
    dict(kv=mk.mk_kv(5 * A, 5 * A, 4096, 4096, 2048)), dict(layer=1, kv=mk.mk_kv(5 * A, 6 * A, 4096, 2048, 2048)),
    dict(q=A, q_stride=264), dict(q=A + 256), dict(q=5 * A), dict(q=6 * A + 4096), dict(qkv=5 * A + 8192), dict(slots=4 * A), dict(positions=5 * A + 64),
    dict(q=A, qkv_dtype=mk.F32), dict(layer=2, q=5 * A + 2 * 2 * 4096 + 64),                                            # overlaps
])
def test_rope_append_refuses(over):
    assert mk.lib.mk_rope_append(ctypes.byref(rope_args(**over)), None) == mk.MK_ERR_ARG
    assert mk.lib.mk_last_error()


def test_rope_append_refuses_null_and_takes_no_tokens():
    assert mk.lib.mk_rope_append(None, None) == mk.MK_ERR_ARG
    assert mk.lib.mk_rope_append(ctypes.byref(rope_args(kv=None, tokens=0, qkv=None, q=None, slots=None, positions=None)), None) == mk.MK_OK
    a = rope_args()
    a.kv = None
    assert mk.lib.mk_rope_append(ctypes.byref(a), None) == mk.MK_ERR_ARG
    a = rope_args()
    a.freqs = None
    assert mk.lib.mk_rope_append(ctypes.byref(a), None) == mk.MK_ERR_ARG


def pages_args(**over):
    return fields(mk.mk_pages_args, dict(batch=4, block_size=8, max_blocks=5, n_blocks=30, shared_prefix=0, max_tokens=16, ring=A, ends=2 * A, ends_out=2 * A,
                                         table=3 * A, lens=4 * A, new_lens=5 * A, slots=6 * A, positions=7 * A, sequences=8 * A, first=9 * A, status=10 * A), over)


@pytest.mark.parametrize("over", [
    dict(batch=0), dict(batch=1025), dict(block_size=0), dict(block_size=-8), dict(max_blocks=0), dict(n_blocks=0), dict(n_blocks=1 << 28), dict(max_blocks=1 << 28),
    dict(shared_prefix=-1), dict(shared_prefix=48), dict(max_tokens=-1), dict(ring=None), dict(ends=None), dict(ends_out=None), dict(table=None), dict(lens=None),
    dict(new_lens=None), dict(slots=None), dict(ring=A + 2), dict(ends=2 * A + 1), dict(table=3 * A + 2), dict(first=9 * A + 2), dict(status=10 * A + 1),
    dict(ring=3 * A), dict(ends_out=2 * A + 4), dict(table=4 * A - 8), dict(lens=6 * A + 32), dict(slots=5 * A), dict(positions=6 * A), dict(sequences=7 * A + 60),
    dict(first=8 * A + 60), dict(status=9 * A + 16), dict(ends_out=A + 4), dict(ends=A, ends_out=A),                       # overlaps
])
def test_assign_pages_refuses(over):
    assert mk.lib.mk_assign_pages(ctypes.byref(pages_args(**over)), None) == mk.MK_ERR_ARG
    assert mk.lib.mk_last_error()


def test_assign_pages_refuses_null():
    assert mk.lib.mk_assign_pages(None, None) == mk.MK_ERR_ARG


def test_operands_off_the_gpu_are_named():
    torch = pytest.importorskip("torch")
    x, i = torch.ones(2, 16, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        mk.adapted_linear(x, x, (torch.ones(1, 8, 16, dtype=torch.bfloat16), torch.ones(1, 2, 8, dtype=torch.bfloat16)), i)
    kv = type("KV", (), dict(k=torch.ones(1, 1, 1, 8, 16, dtype=torch.bfloat16), v=torch.ones(1, 1, 1, 8, 16, dtype=torch.bfloat16)))
    with pytest.raises(ValueError, match="qkv must be a CUDA tensor"):
        mk.rope_append(torch.ones(2, 48, dtype=torch.bfloat16), kv, i, i, torch.ones(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="ring must be a CUDA tensor"):
        mk.assign_pages(i, torch.zeros(3, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32), i, i, 8, 4)


def test_call_module_hands_over_what_it_does_not_take():
    torch = pytest.importorskip("torch")
    fast = mk._fast or mk._setup()
    x = torch.ones(2, 16, dtype=torch.bfloat16)
    for f, n in ((fast.adapted_linear, 13), (fast.rope_append, 14), (fast.assign_pages, 11)):
        for args in ((), (x,), (None,) * n, (x,) * n, (1,) * n):
            assert f(*args) is None
