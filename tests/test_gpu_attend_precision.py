"""How far mk_attend is from its definition in 64 bits, in norm and where one weight outweighs the rest.

In norm.  A rounding to bf16 is off by at most half a step, 2^-8 relative, and uniform within it: its rms is at most
2^-8 / sqrt 3 relative.  An output is rounded once; and its weights are: with errors e_i of the weights independent of the
values, sum p_i e_i v_i has the norm of o = sum p_i v_i times that of e (values of mean zero: |o|^2 = sum p_i^2 |v_i|^2), at
most.  Together sqrt 2 times 2^-8 / sqrt 3; the rest (scores, exponentials, sums in fp32) is below 2^-16.  The least rows
below, 64 tokens by 4 heads, make the mean of the squares certain to a few per cent, which lie between the bound and the mean
over a binade (0.74 of it)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402
from attend_reference import attend_reference  # noqa: E402
from workload import KVCache  # noqa: E402

BF = torch.bfloat16
NORM = math.sqrt(2 / 3) * 2.0 ** -8 + 2.0 ** -16


def randn(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,kw", [
    ([64], [64], {}), ([64], [2000], {}), ([300, 90], [1000, 90], {}), ([64, 64], [1500, 900], dict(window=300, sinks=4)),
    ([20] * 8, [1020] * 8, dict(shared_prefix=1000)), ([1] * 64, [3000] * 64, {})])
@pytest.mark.parametrize("std", [0.3, 1.5, 5.0])
def test_error_in_norm(d, q_lens, kv_lens, kw, std):
    kv = KVCache(*(randn((len(q_lens), 1, 1, max(kv_lens), d), s) for s in (1, 2)))
    q = randn((sum(q_lens), 4, d), 3, std)
    want, _ = attend_reference(q, kv, q_lens, kv_lens, **kw)
    got = mk.attend(q, kv, q_lens, kv_lens, **kw).double()
    off = ((got - want).norm() / want.norm()).item()
    assert off <= NORM, off / NORM


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("at", [5, 130, 299, 599])          # in the first tile that a row sees, and in later ones
@pytest.mark.parametrize("power", [0.3, 6.1, 6.6, 7.3, 7.9, 8.4, 30.7])
def test_one_key_that_outweighs_the_rest(d, at, power):
    # key 0 has score 0, key `at` one whose weight is 2^power against it, the others 2^-40
    k = torch.zeros((1, 1, 1, 600, d), device="cuda")
    k[..., 0] = -40 * math.log(2)
    k[..., 0, 0], k[..., at, 0] = 0, power * math.log(2)
    kv = KVCache(k.to(BF), randn((1, 1, 1, 600, d), 2))
    q = torch.zeros((40, 2, d), device="cuda", dtype=BF)
    q[..., 0] = 1
    q[3, 0, 0] = 0.75          # (rows of their own weights)
    kw = dict(scale=1.0)
    want, bound = attend_reference(q, kv, [40], [600], **kw)
    got = mk.attend(q, kv, [40], [600], **kw)
    off = ((got.double() - want).abs() / bound).max().item()
    assert off <= 1, off
