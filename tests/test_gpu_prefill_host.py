"""mk_prefill at its C entry: when it has read its host arrays."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from workload import empty_kv, make_weights, small_config, token_ids  # noqa: E402

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

