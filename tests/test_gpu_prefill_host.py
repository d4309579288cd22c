"""mk_prefill at its C entry: when it has read its host arrays, and where its device errors surface."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from workload import KVCache, empty_kv, make_weights, small_config, token_ids  # noqa: E402

I32P = ctypes.POINTER(ctypes.c_int32)


def prefill(dec, tokens, n, pos, prefix=0):
    """mk_prefill without the wait for its errors; tokens: the address of its int32 host tokens, or a list."""
    B = dec.cfg.batch
    c_n, c_p = (ctypes.c_int32 * B)(*n), (ctypes.c_int32 * B)(*pos)
    if not isinstance(tokens, int):
        tokens = (ctypes.c_int32 * len(tokens))(*tokens)
    need = mk.lib.mk_prefill_workspace(dec.handle, c_n, c_p, prefix)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = mk.lib.mk_prefill(dec.handle, ctypes.cast(tokens, I32P), c_n, c_p, prefix, ws.data_ptr(), need)
    return st, ws


def paged(cfg, sched):
    C = sched.attn_chunk
    per = -(-cfg.max_seq // C)
    n = cfg.batch * per + 1
    table = torch.arange(cfg.batch * per, dtype=torch.int32, device="cuda").reshape(cfg.batch, per)
    shape = (cfg.n_layers, cfg.n_kv_heads, n * C, cfg.head_dim)
    kv = KVCache(*(torch.zeros(shape, device="cuda", dtype=torch.bfloat16) for _ in range(2)))
    return kv, (table, C, n)


@pytest.mark.parametrize("lens", [[1, 70], [900, 2300]])
def test_tokens_are_read_before_the_call_returns(lens):
    # a page-locked array behind work that keeps the stream busy, refilled as soon as the call has returned
    cfg = small_config(batch=2, max_seq=2304)
    w = make_weights(cfg, device="cuda", std=0.05)
    S = mk.device_sm_count()
    toks = token_ids(cfg, sum(lens), tag="prompt")
    a, b = empty_kv(cfg, device="cuda"), empty_kv(cfg, device="cuda")
    da, db = (mk.Decoder(mk.Schedule(cfg, S), w, kv) for kv in (a, b))
    db.prefill([toks[:lens[0]], toks[lens[0]:]])
    pinned = torch.tensor(toks, dtype=torch.int32).pin_memory()
    torch.cuda._sleep(200_000_000)          # about 0.1 s
    st, ws = prefill(da, pinned.data_ptr(), lens, [0, 0])
    pinned.copy_(torch.tensor([(t + 1) % cfg.vocab for t in toks], dtype=torch.int32))
    assert st == mk.MK_OK
    da.status()
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    da.close()
    db.close()


@pytest.mark.parametrize("then", ["step_static", "status", "step"])
@pytest.mark.parametrize("before", [False, True])
def test_a_device_error_surfaces_at_the_next_synchronous_call(then, before):
    # a table entry outside the pool while the prompt runs, put right before the next call: that call reports it
    cfg = small_config(max_seq=128)
    w = make_weights(cfg, device="cuda")
    sched = mk.Schedule(cfg, mk.device_sm_count(), attn_chunk=32)
    kv, pages = paged(cfg, sched)
    dec = mk.Decoder(sched, w, kv, pages=pages)
    if before:
        dec.step_static([1], [0])
    good = int(pages[0][0, 1])
    pages[0][0, 1] = pages[2] + 5
    st, ws = prefill(dec, token_ids(cfg, 80), [80], [0])
    assert st == mk.MK_OK
    torch.cuda.synchronize()
    pages[0][0, 1] = good
    torch.cuda.synchronize()
    calls = {"step_static": lambda: dec.step_static([1], [80]), "status": dec.status, "step": lambda: dec.step([1], [80])}
    with pytest.raises(mk.MkError) as e:
        calls[then]()
    assert e.value.status == mk.MK_ERR_BOUNDS
    with pytest.raises(mk.MkError) as e:
        dec.step([1], [80])
    assert e.value.status == mk.MK_ERR_POISONED
    dec.close()


def test_a_good_prompt_between_steps_on_the_static_scratch():
    cfg = small_config(max_seq=128)
    w = make_weights(cfg, device="cuda", std=0.05)
    kvs = [empty_kv(cfg, device="cuda") for _ in range(2)]
    decs = [mk.Decoder(mk.Schedule(cfg, mk.device_sm_count()), w, kv) for kv in kvs]
    toks = token_ids(cfg, 40, tag="prompt")
    decs[0].step_static(toks[:1], [0])
    decs[1].step(toks[:1], [0])
    for d in decs:
        st, ws = prefill(d, toks[1:39], [38], [1])
        assert st == mk.MK_OK
        torch.cuda.synchronize()
    out = [decs[0].step_static(toks[39:], [39]), decs[1].step(toks[39:], [39])]
    assert out[0] == out[1] and torch.equal(decs[0].logits, decs[1].logits)
    for d in decs:
        d.status()
        d.close()

