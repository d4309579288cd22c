"""mk_prefill: the prompt path's operators run together, as a user runs them -- prompts into the cache (in one
piece, in several, ragged batches, paged, behind a shared prefix), then decode steps that read it.

Tolerances.  The prompt path rounds its activations to bf16 where the decode step keeps fp32: per layer the
normed inputs (twice), q, the softmax weights, the attention output, the SwiGLU output, and K or V itself, each off by at
most half a step, 2^-8 relative in norm.  Cache rows of layer l therefore agree with the decode step's in norm to
(2 + 7 l) 2^-8 (the residual stream only dilutes what a layer adds).  Logits are held to the parity tests' 1e-2 of
the largest."""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from gpu_helpers import REL_TOL  # noqa: E402
from oracle import HostWeights, Oracle, kv_to_host  # noqa: E402
from workload import KVCache, empty_kv, get_workload, make_weights, small_config, token_ids  # noqa: E402


def prompts(cfg, lens, seed=0):
    return [token_ids(cfg, n, seed=seed, tag=f"prompt{b}") for b, n in enumerate(lens)]


def step_by_step(dec, toks, pos):
    """Feeds the prompts through decode steps, one position at a time (shorter ones repeat their last
    token at its own position, which rewrites the same row)."""
    for i in range(max(len(t) for t in toks)):
        k = [min(i, len(t) - 1) for t in toks]
        out = dec.step([t[j] for t, j in zip(toks, k)], [p + j for p, j in zip(pos, k)])
    return out


def check_rows(got, want, lens, pos):
    for name in ("k", "v"):
        a, b = getattr(got, name).double(), getattr(want, name).double()
        for s, (n, p) in enumerate(zip(lens, pos)):
            for layer in range(a.shape[1]):
                x, y = a[s, layer, :, p:p + n], b[s, layer, :, p:p + n]
                rel = (x - y).norm() / y.norm()
                assert rel.item() <= (2 + 7 * layer) * 2.0 ** -8, (name, s, layer, rel.item())


def check_logits(a, b):
    assert ((a - b).abs().amax(1) <= REL_TOL * b.abs().amax(1)).all(), ((a - b).abs().amax(1) / b.abs().amax(1)).tolist()


@pytest.mark.parametrize("name,n", [("tiny", 16), ("llama1b_reduced", 200)])
def test_prompt_then_step_matches_the_oracle(name, n):
    cfg = get_workload(name).cfg
    w = make_weights(cfg, device="cuda")
    kv = empty_kv(cfg, device="cuda")
    prompt = token_ids(cfg, n, tag="prompt")
    dec = mk.Decoder(mk.Schedule(cfg, mk.device_sm_count()), w, kv)
    dec.prefill([prompt[:-1]])
    nxt = dec.step([prompt[-1]], [n - 1])
    orc, hw = Oracle("f32"), HostWeights(w)
    kh, vh = kv_to_host(empty_kv(cfg))
    for i, t in enumerate(prompt):
        logits, want = orc.decode_step(cfg, hw, kh, vh, [t], [i])
    check_logits(dec.logits.cpu().double(), torch.from_numpy(np.asarray(logits)).double())
    top = np.sort(logits[0])[-2:]
    if top[1] - top[0] > 0.05:
        assert nxt == want
    dec.close()


@pytest.mark.parametrize("head_dim,nq,nkv", [(64, 4, 2), (32, 8, 1), (128, 3, 3)])
@pytest.mark.parametrize("gain", [0.0, 0.2])
def test_prompt_matches_decode_steps(head_dim, nq, nkv, gain):
    cfg = small_config(n_layers=3, head_dim=head_dim, n_q_heads=nq, n_kv_heads=nkv, max_seq=200)
    w = make_weights(cfg, device="cuda", std=0.05, gain_std=gain)
    a, b = empty_kv(cfg, device="cuda"), empty_kv(cfg, device="cuda")
    toks = prompts(cfg, [150])
    da, db = (mk.Decoder(mk.Schedule(cfg, mk.device_sm_count()), w, kv) for kv in (a, b))
    step_by_step(db, toks, [0])
    da.prefill([toks[0][:-1]])
    da.step(toks[0][-1:], [149])
    check_rows(a, b, [150], [0])
    check_logits(da.logits, db.logits)
    assert (a.k[:, :, :, 150:] == 0).all() and (a.v[:, :, :, 150:] == 0).all()
    da.close()
    db.close()


@pytest.mark.parametrize("lens,pos", [([1, 40, 130], [0, 0, 0]), ([7, 1, 33], [100, 60, 0])])
def test_ragged_batch_in_pieces(lens, pos):
    cfg = small_config(batch=3, max_seq=256)
    w = make_weights(cfg, device="cuda", std=0.05)
    start = KVCache(*(torch.randn(empty_kv(cfg).k.shape, device="cuda").to(torch.bfloat16) for _ in range(2)))
    toks = prompts(cfg, lens)
    kvs = [start.clone() for _ in range(4)]
    S = mk.device_sm_count()
    decs = [mk.Decoder(mk.Schedule(cfg, S), w, kv) for kv in kvs]
    step_by_step(decs[0], toks, pos)
    for dec, chunk in zip(decs[1:], (4096, 32, 1)):
        dec.prefill(toks, pos, chunk=chunk)
    for kv in kvs[1:]:
        check_rows(kv, kvs[0], lens, pos)
        for b, (n, p) in enumerate(zip(lens, pos)):          # nothing else of the cache is touched
            keep = torch.ones(cfg.max_seq, dtype=torch.bool)
            keep[p:p + n] = False
            assert torch.equal(kv.k[b][:, :, keep], start.k[b][:, :, keep])
            assert torch.equal(kv.v[b][:, :, keep], start.v[b][:, :, keep])
    for d in decs:
        d.close()


def paged(cfg, sched, tables=None, seed=0):
    C = sched.attn_chunk
    per = -(-cfg.max_seq // C)
    n = cfg.batch * per + 2
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:cfg.batch * per].reshape(cfg.batch, per)
    if tables:
        tables(order)
    shape = (cfg.n_layers, cfg.n_kv_heads, n * C, cfg.head_dim)
    kv = KVCache(torch.zeros(shape, device="cuda", dtype=torch.bfloat16), torch.zeros(shape, device="cuda", dtype=torch.bfloat16))
    return kv, (order.to(device="cuda", dtype=torch.int32), C, n)


@pytest.mark.parametrize("chunk", [16, 128])
def test_paged_cache(chunk):
    cfg = small_config(batch=2, max_seq=300)
    w = make_weights(cfg, device="cuda", std=0.05)
    S = mk.device_sm_count()
    sched = mk.Schedule(cfg, S, attn_chunk=chunk)
    kv, pages = paged(cfg, sched)
    flat = empty_kv(cfg, device="cuda")
    toks = prompts(cfg, [270, 19])
    a = mk.Decoder(sched, w, kv, pages=pages)
    b = mk.Decoder(mk.Schedule(cfg, S, attn_chunk=chunk), w, flat)
    for d in (a, b):
        d.prefill([t[:-1] for t in toks])
        d.step([t[-1] for t in toks], [len(t) - 1 for t in toks])
    # the same kernels over the same values, in other places: identical
    assert torch.equal(a.logits, b.logits)
    for b_, n in enumerate((270, 19)):
        pos = torch.arange(n, device="cuda")
        slot = pages[0][b_, pos // chunk].long() * chunk + pos % chunk
        assert torch.equal(kv.k[:, :, slot], flat.k[b_, :, :, :n]) and torch.equal(kv.v[:, :, slot], flat.v[b_, :, :, :n])
    a.close()
    b.close()


def test_shared_prefix_then_questions_then_decode():
    # a system prompt once, blocks shared by every sequence's table; each sequence's own question; decoding
    cfg = small_config(batch=4, max_seq=400)
    w = make_weights(cfg, device="cuda", std=0.05)
    S = mk.device_sm_count()
    sched = mk.Schedule(cfg, S, attn_chunk=64)
    prefix, asks = prompts(cfg, [128], seed=5)[0], prompts(cfg, [9, 40, 1, 70], seed=6)

    def share(order):
        order[:, :2] = order[0, :2]

    kv, pages = paged(cfg, sched, share)
    dec = mk.Decoder(sched, w, kv, pages=pages)
    dec.prefill([prefix, [], [], []])
    dec.prefill([a[:-1] for a in asks], [128] * 4, shared_prefix=128)
    first = dec.step([a[-1] for a in asks], [127 + len(a) for a in asks])
    logits = dec.logits.clone()
    more = dec.steps(first, [128 + len(a) for a in asks], 3)
    flat = empty_kv(cfg, device="cuda")
    ref = mk.Decoder(mk.Schedule(cfg, S, attn_chunk=64), w, flat)
    ref.prefill([prefix + a[:-1] for a in asks])
    ref.step([a[-1] for a in asks], [127 + len(a) for a in asks])
    check_logits(logits, ref.logits)
    assert len(more) == 3
    dec.close()
    ref.close()


def test_shared_prefix_in_a_contiguous_cache():
    cfg = small_config(batch=2, max_seq=300)
    w = make_weights(cfg, device="cuda", std=0.05)
    S = mk.device_sm_count()
    prefix, asks = prompts(cfg, [100], seed=5)[0], prompts(cfg, [9, 60], seed=6)
    a, b = empty_kv(cfg, device="cuda"), empty_kv(cfg, device="cuda")
    da, db = (mk.Decoder(mk.Schedule(cfg, S), w, kv) for kv in (a, b))
    da.prefill([prefix, []])
    da.prefill(asks, [100, 100], shared_prefix=100)          # read through sequence 0's rows
    db.prefill([prefix + q for q in asks])
    check_rows(a, b, [9, 60], [100, 100])
    da.close()
    db.close()


def test_runs_are_identical_and_the_streams_own():
    cfg = small_config(max_seq=300)
    w = make_weights(cfg, device="cuda", std=0.05)
    toks = prompts(cfg, [250])
    kvs = []
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        kv = empty_kv(cfg, device="cuda")
        torch.cuda.synchronize()
        dec = mk.Decoder(mk.Schedule(cfg, mk.device_sm_count()), w, kv, stream=stream)
        dec.prefill(toks, workspace=torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda") if stream is None else None)
        kvs.append(kv)
        dec.close()
    for kv in kvs[1:]:
        assert torch.equal(kv.k, kvs[0].k) and torch.equal(kv.v, kvs[0].v)


def test_refusals_leave_the_context_usable():
    cfg = small_config(batch=2, max_seq=64)
    w = make_weights(cfg, device="cuda")
    dec = mk.Decoder(mk.Schedule(cfg, mk.device_sm_count()), w, empty_kv(cfg, device="cuda"))
    good = prompts(cfg, [5, 6])
    for bad in (lambda: dec.prefill([good[0]]), lambda: dec.prefill(good, [0]), lambda: dec.prefill(good, chunk=0)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dec.prefill([good[0], [cfg.vocab]]), lambda: dec.prefill([good[0], [-1]]),
                lambda: dec.prefill(good, [0, 60]), lambda: dec.prefill(good, [-1, 0]),
                lambda: dec.prefill(good, [3, 2], shared_prefix=3), lambda: dec.prefill(good, shared_prefix=-1)):
        with pytest.raises(mk.MkError) as e:
            bad()
        assert e.value.status == mk.MK_ERR_ARG
    with pytest.raises(mk.MkError) as e:
        dec.prefill(good, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))
    assert e.value.status == mk.MK_ERR_CAPACITY
    dec.prefill([[], []])
    dec.prefill(good)
    run = dec.persistent_start([1, 2], [5, 6], 4)
    with pytest.raises(mk.MkError) as e:
        dec.prefill(good)
    assert e.value.status == mk.MK_ERR_ARG
    dec.persistent_wait()
    assert run.numel() == 8
    dec.close()


def test_blocks_that_are_not_multiples_of_8_are_refused():
    cfg = small_config(max_seq=60)
    w = make_weights(cfg, device="cuda")
    sched = mk.Schedule(cfg, mk.device_sm_count(), attn_chunk=20)
    kv, pages = paged(cfg, sched)
    dec = mk.Decoder(sched, w, kv, pages=pages)
    with pytest.raises(mk.MkError) as e:
        dec.prefill([[1, 2, 3]])
    assert e.value.status == mk.MK_ERR_ARG
    dec.close()


def test_a_bad_table_entry_is_reported_and_not_followed():
    cfg = small_config(max_seq=128)
    w = make_weights(cfg, device="cuda")
    sched = mk.Schedule(cfg, mk.device_sm_count(), attn_chunk=32)
    kv, pages = paged(cfg, sched)
    dec = mk.Decoder(sched, w, kv, pages=pages)
    pages[0][0, 1] = pages[2] + 5
    with pytest.raises(mk.MkError) as e:
        dec.prefill([token_ids(cfg, 80)])
    assert e.value.status == mk.MK_ERR_BOUNDS
    with pytest.raises(mk.MkError) as e:
        dec.prefill([[1]])
    assert e.value.status == mk.MK_ERR_POISONED
    dec.close()


def test_workspace_size_and_null_arguments():
    assert mk.lib.mk_prefill_workspace(None, None, None, 0) == 0
    n = (ctypes.c_int32 * 8)(1)
    assert mk.lib.mk_prefill(None, n, n, n, 0, None, 0) == mk.MK_ERR_ARG
