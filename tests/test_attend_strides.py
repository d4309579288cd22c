"""mk_attend's checks of the cache's strides and extent: a dimension of one has no stride to speak of, and what lies
behind the last position is not the cache.  No GPU needed, and nothing is launched on one: the calls below ask for
parts to join (a shared prefix) and bring a workspace of no bytes."""
import ctypes

import pytest

mk = pytest.importorskip("persistent_megakernel_decode_sm_gb300")

A = 1 << 20          # an aligned address that is never dereferenced


def call(kv, pages=None, **over):
    q_lens, kv_lens = over.pop("q_lens", (1, 2)), over.pop("kv_lens", (5, 9))
    n = len(q_lens)
    f = dict(n_q_heads=4, n_kv_heads=2, head_dim=32, batch=n, q_lens=(ctypes.c_int32 * n)(*q_lens), kv_lens=(ctypes.c_int32 * n)(*kv_lens),
             q=A, q_stride=128, out=2 * A, out_stride=128, kv=ctypes.pointer(kv), pages=None if pages is None else ctypes.pointer(pages), layer=0,
             max_seq=64, window=0, sinks=0, shared_prefix=3, scale=0.0, status=None)
    f.update(over)
    a = mk.mk_attend_args(*[f[n] for n, _ in mk.mk_attend_args._fields_])
    return mk.lib.mk_attend(ctypes.byref(a), 9 * A, 0, None)


TAKEN = (mk.MK_ERR_CAPACITY, mk.MK_ERR_CUDA)   # past the checks of arguments (the second: no GPU to ask for its size)
ROWS = 64 * 32                                 # elements of a head
POOL = mk.mk_kv_pages(7 * A, 16, 4, 4)


@pytest.mark.parametrize("kv,pages,over", [
    (mk.mk_kv(5 * A, 6 * A, ROWS, 0, 1), None, dict(n_kv_heads=1)),                              # one head
    (mk.mk_kv(5 * A, 6 * A, ROWS, 0, 100 * ROWS), None, dict(n_kv_heads=1)),
    (mk.mk_kv(5 * A, 6 * A, 1, 0, ROWS), None, dict(q_lens=(1,), kv_lens=(5,))),                 # one sequence
    (mk.mk_kv(5 * A, 6 * A, 2 * ROWS, 1, ROWS), None, {}),                                       # the first layer
    (mk.mk_kv(5 * A, 6 * A, 1, 1, ROWS), POOL, {}),                                              # a pool has no sequences
    (mk.mk_kv(5 * A, 6 * A, 1, 1, 1), POOL, dict(n_kv_heads=1)),
    (mk.mk_kv(5 * A, 6 * A, 4 * ROWS, 0, 2 * ROWS), None, dict(out=5 * A + 2 * 7 * ROWS)),       # behind the last position
    (mk.mk_kv(5 * A, 6 * A, 0, 0, 2 * ROWS), POOL, dict(out=5 * A + 2 * 3 * ROWS)),
    (mk.mk_kv(5 * A, 6 * A, 8 * ROWS, 4 * ROWS, 2 * ROWS), None, dict(layer=1, out=5 * A + 2 * 15 * ROWS)),
])
def test_taken(kv, pages, over):
    assert call(kv, pages, **over) in TAKEN, mk.lib.mk_last_error()


@pytest.mark.parametrize("kv,pages,over", [
    (mk.mk_kv(5 * A, 6 * A, ROWS, 0, 1), None, {}),
    (mk.mk_kv(5 * A, 6 * A, ROWS - 8, 0, 1), None, dict(n_kv_heads=1)),
    (mk.mk_kv(5 * A, 6 * A, 1, 0, ROWS), None, {}),
    (mk.mk_kv(5 * A, 6 * A, 2 * ROWS, 1, ROWS), None, dict(layer=1)),
    (mk.mk_kv(5 * A, 6 * A, 1, 0, ROWS - 8), POOL, {}),
    (mk.mk_kv(5 * A, 6 * A, 1, 4, ROWS), POOL, dict(layer=1)),
    (mk.mk_kv(5 * A, 6 * A, 1, -8, ROWS), POOL, dict(layer=1)),
    (mk.mk_kv(5 * A, 6 * A, 4 * ROWS, 0, 2 * ROWS), None, dict(out=5 * A + 2 * 7 * ROWS - 16)),
    (mk.mk_kv(5 * A, 6 * A, 0, 0, 2 * ROWS), POOL, dict(out=6 * A + 2 * 3 * ROWS - 16)),
    (mk.mk_kv(5 * A, 6 * A, 8 * ROWS, 4 * ROWS, 2 * ROWS), None, dict(layer=1, out=6 * A + 2 * 15 * ROWS - 16)),
])
def test_refused(kv, pages, over):
    assert call(kv, pages, **over) == mk.MK_ERR_ARG
