"""Whole models' prompts against decode steps, which keep activations in fp32: the 1B shape's 16 layers, the 8B shape's 32.

Tolerance.  A cache row of layer l has 2 + 7 l roundings to bf16 behind it that the decode step does not make (per
layer the normed inputs (two), q, the softmax weights, the attention and SwiGLU outputs, K or V).  They are independent of one
another, so they add in squares: in norm sqrt(2 + 7 l) times that of one, whose rms is at most 2^-8 / sqrt 3.  Each is counted
at 2^-8 instead, which leaves a factor of sqrt 3 for what magnifies it (SwiGLU's two factors share one rounded
input); the residual stream dilutes what a layer adds.  Logits: one row behind the last layer, 2 + 7 n_layers roundings."""
import dataclasses
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from workload import empty_kv, get_workload, make_weights, token_ids  # noqa: E402


def relative(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


@pytest.mark.parametrize("name,n", [("llama1b_ctx512", 1500), ("llama8b_ctx2048", 400)])
def test_prompt_of_a_whole_model(name, n):
    cfg = dataclasses.replace(get_workload(name).cfg, max_seq=1536)
    w = make_weights(cfg, device="cuda")
    toks = token_ids(cfg, n, tag="prompt")
    kvs, decs = [], []
    for _ in range(2):
        kvs.append(empty_kv(cfg, device="cuda"))
        decs.append(mk.Decoder(mk.Schedule(cfg, mk.device_sm_count()), w, kvs[-1]))
    decs[0].prefill([toks[:-1]])
    decs[0].step(toks[-1:], [n - 1])
    for i, t in enumerate(toks):
        decs[1].step([t], [i])
    for layer in range(cfg.n_layers):
        for c in ("k", "v"):
            off = relative(getattr(kvs[0], c)[0, layer, :, :n], getattr(kvs[1], c)[0, layer, :, :n])
            assert off <= math.sqrt(2 + 7 * layer) * 2.0 ** -8, (layer, c, off)
    off = relative(decs[0].logits, decs[1].logits)
    assert off <= math.sqrt(2 + 7 * cfg.n_layers) * 2.0 ** -8, off
    for d in decs:
        d.close()
