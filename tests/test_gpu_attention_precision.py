"""Attention on the GPU where numbers are far apart in size: rows of NaN, keys
that dominate, small weights and small gradients (MI355X only)."""
import math

import pytest
import torch

from tests import layer_cases as lc
from tests.test_gpu_attention import Call

pytestmark = pytest.mark.gpu

NAN = float("nan")
H16 = 2.0 ** -11        # half a step of fp16


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


POISONED = {
    "prompt": dict(S=260, d=64, Hq=4, Hkv=2, window=45, sinks=2),
    "prompt_fp16": dict(S=260, d=128, Hq=4, Hkv=2, dtype="fp16"),
    "prompt_fp32": dict(S=150, d=40, Hq=2, Hkv=1, window=45, dtype="fp32"),
    "last_tokens": dict(B=2, S=70, d=64, Hq=4, Hkv=2, queries=3),
    "last_tokens_joined": dict(B=2, S=3000, d=128, Hq=4, Hkv=1, queries=2),
    "last_tokens_joined_fp32": dict(B=2, S=1300, d=64, Hq=4, Hkv=1, queries=2, dtype="fp32"),
}


@pytest.mark.parametrize("name", POISONED)
def test_lse_of_rows_without_a_score(name):
    """NaN where every score in sight is NaN (the query holds one, or the only key
    in sight does), -infinity for rows that see nothing and for no others."""
    c = lc.Attention(**POISONED[name])
    q, k, v, do = c.inputs(2)
    lengths = [c.S] * c.B
    lengths[-1] = c.S - 1 if c.queries < c.S else c.S - 30
    bad = c.queries // 2
    q[0, 1, bad, 3] = NAN
    starts = [0] * c.B if c.queries == c.S else [c.S - c.queries] * c.B     # the last row of the last sequence is beyond it
    call = Call(c, q, k, v, do, starts, lengths)
    call.forward()
    torch.cuda.synchronize()
    lse, o = call.lse.t.view(c.shards, c.hq, c.queries).cpu(), c.shaped(call.o.t.cpu(), c.hq, c.queries)
    want = torch.zeros_like(lse)
    want[0, 1, bad] = NAN
    for n, s in enumerate(c.sequence):
        want[n, :, ~c.sees(starts[s], lengths[s]).any(1)] = -math.inf
    assert bool((torch.isnan(lse) == torch.isnan(want)).all())
    assert bool((torch.isneginf(lse) == torch.isneginf(want)).all())
    assert bool(torch.isnan(o[0, 1, bad]).all()) and bool((o[torch.isneginf(want)] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_lse_of_a_key_of_nan(dtype):
    c = lc.Attention(S=100, d=64, window=1, dtype=dtype)
    q, k, v, do = c.inputs(2)
    k[0, 0, 41] = NAN
    call = Call(c, q, k, v, do)
    call.forward()
    torch.cuda.synchronize()
    got = torch.isnan(call.lse.t.cpu())
    assert bool(got[41]) and int(got.sum()) == 1
