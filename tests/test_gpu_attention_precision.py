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


def dominant(c, size):
    """A first key 17.5 above all others, which are equal; its value is 0, theirs
    are 1.  Exact o of position p and dv of the keys but the first for do = size."""
    q, k, v, do = (torch.zeros_like(x) for x in c.inputs(0))
    q[..., 0] = 1.0
    k[:, :, 0, 0] = 17.5
    v[:, :, 1:] = 1.0
    do[:] = size
    p = (c.S - c.queries + torch.arange(c.queries)).double()
    w = math.exp(-17.5)
    o = p * w / (1 + p * w)
    # row p gives each of the keys 1 to p the weight w / (1 + p w)
    each = torch.zeros(c.S, dtype=torch.float64)
    each[c.S - c.queries:] = w / (1 + p * w)
    return (q, k, v, do), o, size * each.flip(0).cumsum(0).flip(0) * (c.hq // c.hkv)


DOMINANT = {
    "prompt": dict(S=4096, d=64, Hq=4, Hkv=4, dtype="fp16"),
    "prompt_heads": dict(S=4096, d=128, Hq=8, Hkv=4, dtype="fp16"),
    "few_tokens": dict(S=9000, d=64, Hq=8, Hkv=1, queries=2, dtype="fp16"),
    "block_of_keys_shared": dict(S=700, d=40, Hq=2, Hkv=1, dtype="fp16"),
}


@pytest.mark.parametrize("name", DOMINANT)
def test_small_weights_in_fp16(name):
    """Many weights of 2^-25 of the largest.  They are rounded to fp16 after a
    shift by 2^7, so each is off by half a step of its size or by 2^-25 / 2^7 of the
    largest weight."""
    c = lc.Attention(**DOMINANT[name])
    (q, k, v, do), want, _ = dominant(c, 1.0)
    call = Call(c, q, k, v, do, scale=1.0)
    call.forward()
    torch.cuda.synchronize()
    o = c.shaped(call.o.t.cpu().double(), c.hq, c.queries)
    # the weights' rounding, the result's, and fp32: 2 (n + 8) 2^-24 of it
    allowed = (c.S * 2.0 ** -32 + want * (2 * H16 + 2 * (c.S + 8) * lc.U) + 2.0 ** -25)[None, None, :, None]
    assert bool(((o - want[None, None, :, None]).abs() <= allowed).all())


@pytest.mark.parametrize("S,queries", [(600, 600), (600, 3), (4000, 4000)])
@pytest.mark.parametrize("first", [False, True])
def test_scores_of_fifty_million_in_fp16(S, queries, first):
    """Every key's score is 10^4 and more from its neighbours': a row's value is that
    of its largest."""
    c = lc.Attention(S=S, d=64, queries=queries, dtype="fp16")
    q, k, v, do = c.inputs(1)
    q[:], k[:] = 0.0, 0.0
    step = 64 if S < 1000 else 16
    j = torch.arange(S).double()
    q[..., 0], k[..., 0] = 60000.0, (step * (-1 - j if first else 1 + j)).half().double()
    call = Call(c, q, k, v, do, scale=2.0 ** -6)
    call.forward()
    torch.cuda.synchronize()
    top = torch.zeros(queries, dtype=torch.long) if first else torch.arange(S - queries, S)
    if S > 1000:        # past 2^11 * 16 two neighbours have the same key
        top = top[:2000]
    o = c.shaped(call.o.t.cpu().double(), 1, queries)[0, 0, :len(top)]
    # one weight of 1: its rounding, the result's, and the sum's
    assert bool(((o - v[0, 0, top]).abs() <= 2.5 * H16 * v[0, 0, top].abs()).all())
    lse, want = call.lse.t.cpu().double()[:len(top)], 60000.0 / 64 * k[0, 0, top, 0]
    assert bool(((lse - want).abs() <= 8 * lc.U * want.abs()).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("large", [2.0 ** 10, 2.0 ** 16, 2.0 ** 20, 2.0 ** 22, 2.0 ** 23, 2.0 ** 24, 2.0 ** 25])
def test_weights_of_large_scores_stay_in_range(large, d):
    """Scores that rise by 0 to 40 a row above a large one, which fp32 holds in steps
    of up to 4: a mean of ones is 1."""
    c = lc.Attention(B=4, S=1000, d=d, Hq=4, Hkv=4, dtype="fp16")
    q, k, v, do = c.inputs(1)
    noise = torch.rand(k.shape[:-1], dtype=torch.float64, generator=torch.Generator().manual_seed(int(large))) * 40
    for sign in (1.0, -1.0):
        q[:], k[:], v[:] = 0.0, 0.0, 1.0
        q[..., 0], q[..., 1] = 1024.0, 1.0
        k[..., 0] = sign * 2.0
        k[..., 1] = (noise / (large / 2048.0)).half().double()
        q, k = q.half().double(), k.half().double()
        call = Call(c, q, k, v, do, scale=large / 2048.0)
        call.forward()
        torch.cuda.synchronize()
        # weights and the result are rounded once each
        assert bool(((call.o.t.double() - 1.0).abs() <= 3 * H16).all()), sign


@pytest.mark.parametrize("name", DOMINANT)
def test_small_weights_in_the_gradient_of_values(name):
    c = lc.Attention(**DOMINANT[name])
    (q, k, v, do), _, want = dominant(c, 1024.0)
    call = Call(c, q, k, v, do, scale=1.0)
    call.forward()
    call.backward()
    torch.cuda.synchronize()
    dv = c.shaped(call.dv.t.cpu().double(), c.hkv, c.S)[:, :, 1:]
    want = want[1:, None]
    # rounding of the weights and of the result; lse and the exponent in fp32: 17.5
    # and its logarithm to the base of 2 have a half step of 2^-20 at most, four times
    n = c.queries * c.hq // c.hkv
    assert bool(((dv - want).abs() <= want * (2 * H16 + 4 * 2.0 ** -20 + 2 * (n + 4) * lc.U) + 2.0 ** -25).all())


@pytest.mark.parametrize("keys", [3000, 50000])
def test_equal_weights_in_the_gradient_of_values(keys):
    """1/50000 is below fp16's normal numbers: a step there is 1/335 of it."""
    c = lc.Attention(S=keys, d=64, queries=1, dtype="fp16")
    q, k, v, do = (torch.zeros_like(x) for x in c.inputs(0))
    do[:] = 100.0
    call = Call(c, q, k, v, do, scale=1.0)
    call.forward()
    call.backward()
    torch.cuda.synchronize()
    dv = call.dv.t.cpu().double()
    assert bool(((dv - 100.0 / keys).abs() <= 100.0 / keys * (2 * H16 + 4 * 2.0 ** -20) + 2.0 ** -25).all())


def two_norm(got, want, extra=0.0):
    """Relative error in 2-norm, and half a smallest subnormal of fp16 an element of it."""
    return float((got - want).norm() / want.norm()), 2.0 ** -25 * want.numel() ** 0.5 / float(want.norm())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [3e2, 1.0, 1e-2, 1e-3, 1e-4, 1e-6])
def test_small_gradients_in_fp16(size, d):
    """dS of thousands of keys is far below dout.  Its rounding to fp16 and those of
    the weights, of o in delta and of the result are off by half a step each, in
    the mean square by 1 / sqrt(3) of that: two half steps in 2-norm, and the
    result's smallest subnormal."""
    c = lc.Attention(S=6000, d=d, Hq=2, Hkv=1, queries=64, dtype="fp16")
    q, k, v, do = c.inputs(6)
    for shift in (64.0, 1.0 / 64.0):        # the scores stay, dq and dk in turn are in range
        call = Call(c, q / shift, k * shift, v, (do * size).half().double())
        call.forward()
        call.backward()
        torch.cuda.synchronize()
        want = c.exact(call_values(call.q, c, c.hq, c.queries), call_values(call.k, c, c.hkv, c.S), v, call_values(call.do, c, c.hq, c.queries),
                       [c.S - c.queries], [c.S], call.scale)
        for name, got in (("dq", call.dq), ("dk", call.dk), ("dv", call.dv)):
            exact = want[name][0]
            off, least = two_norm(c.shaped(got.t.cpu().double(), exact.shape[1], exact.shape[2]), exact)
            assert off <= 2 * H16 + least, (name, shift, off, least)


def call_values(x, c, heads, tokens):
    return c.shaped(x.cpu().double(), heads, tokens)


GROWING = {
    "prompt": dict(S=600, d=64, Hq=2, Hkv=1, dtype="fp16"),
    "prompt_128": dict(S=500, d=128, Hq=2, Hkv=1, window=90, sinks=3, dtype="fp16"),
    "by_heads": dict(S=300, d=64, Hq=8, Hkv=1, dtype="fp16"),
    "ragged": dict(S=333, d=33, Hq=2, Hkv=2, window=100, dtype="fp16", order="token"),
}


@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("name", GROWING)
def test_gradients_of_growing_size(name, down):
    """dout from 2^-20 to 2^12 along the queries, and keys whose scores rise: a
    column's largest dS moves all along."""
    c = lc.Attention(**GROWING[name])
    q, k, v, do = c.inputs(3)
    ramp = torch.linspace(-20, 12, c.S, dtype=torch.float64)
    do = (do * torch.exp2(ramp.flip(0) if down else ramp)[:, None]).to(c.dtype).double()
    k = (k * torch.linspace(0.0, 2.0, c.S, dtype=torch.float64)[:, None]).to(c.dtype).double()
    call = Call(c, q, k, v, do)
    call.forward()
    call.backward()
    call.check(c.exact(q, k, v, do, [0], [c.S], call.scale))


def test_gradients_beyond_fp16_on_the_way():
    """dS of 10^5 and more, whose sums times the scale are in range."""
    c = lc.Attention(S=200, d=64, Hq=2, Hkv=1, window=8, dtype="fp16")
    q, k, v, do = c.inputs(6)
    do, v = (do * 8000).half().double(), v * 16
    call = Call(c, q, k, v, do, scale=2.0 ** -7)
    call.forward()
    call.backward()
    want = c.exact(q, k, v, do, [0], [c.S], call.scale)
    torch.cuda.synchronize()
    for name, got, heads in (("dq", call.dq, c.hq), ("dk", call.dk, c.hkv)):
        got = c.shaped(got.t.cpu().double(), heads, c.S)
        off, least = two_norm(got, want[name][0])
        assert bool(torch.isfinite(got).all()) and off <= 2 * H16 + least, (name, off)


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** 6])
@pytest.mark.parametrize("of", [dict(S=3000, d=64, Hq=2, queries=32), dict(S=200, d=128, Hq=4, Hkv=2, window=20), dict(S=700, d=40, Hq=1)])
def test_gradients_by_size_of_the_values(size, of):
    """Values far from 1, of which one key's are larger still."""
    c = lc.Attention(dtype="fp16", **{"Hkv": 1, **of})
    q, k, v, do = c.inputs(8)
    v = v * size
    v[:, :, c.S // 2] *= 64.0
    v, do = v.half().double(), (do / 1024).half().double()
    q, k = q / 8, k * 8
    call = Call(c, q, k, v, do)
    call.forward()
    call.backward()
    torch.cuda.synchronize()
    want = c.exact(q, k, v, do, [c.S - c.queries], [c.S], call.scale)
    for name, got, heads in (("dq", call.dq, c.hq), ("dk", call.dk, c.hkv)):
        exact, err = want[name]
        got = c.shaped(got.t.cpu().double(), heads, exact.shape[2])
        off, least = two_norm(got, exact)
        # a half step each of the weights, of o in delta, of dS and of the result
        assert off <= 4 * H16 + least, (name, off, least)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["v", "do", "k"])
def test_infinities_beside_large_gradients(what, d):
    """A column whose largest dS is infinite next to one whose dS has to come down."""
    c = lc.Attention(S=260, d=d, Hq=4, Hkv=2, window=45, sinks=2, dtype="fp16")
    q, k, v, do = c.inputs(5)
    v, do = v * 16, (do * 8000).half().double()
    x = {"v": v, "do": do, "k": k}[what]
    x[0, 0, 100, 0] = math.inf
    x[0, 1, 200] = NAN
    call = Call(c, q, k, v, do, scale=2.0 ** -8)
    call.forward()
    call.backward()
    torch.cuda.synchronize()
    want = c.exact(q, k, v, do, [0], [c.S], call.scale)
    for name, got, heads in (("dq", call.dq, c.hq), ("dk", call.dk, c.hkv), ("dv", call.dv, c.hkv)):
        exact, err = want[name]
        got = c.shaped(got.t.cpu().double(), heads, c.S)
        fine = torch.isfinite(exact) & torch.isfinite(err) & (exact.abs() + err < 65000)
        assert bool(torch.isfinite(got[fine]).all()), name
        assert not bool(torch.isfinite(got[~torch.isfinite(exact)]).any()), name
        assert bool(((got - exact).abs()[fine] <= (err + H16 * (exact.abs() + err) + 2.0 ** -25)[fine]).all()), name


def test_equal_weights_in_fp32_gradients():
    """3000 keys of nearly equal scores, 128 channels.  lse is 8: its half step,
    2^-21, and that of the exponent to the base of 2, three times in its way, are
    each off by 1 / sqrt(3) in the mean square, 5e-7 together.  Sums of 32 rows add a
    fifth of that.  dk is a sum of dS, whose dP are off by less: 2 sqrt(128) 2^-24
    / sqrt(3) of their size, 8e-7."""
    c = lc.Attention(S=3000, d=128, queries=32, dtype="fp32")
    q, k, v, do = c.inputs(4, 0.05)
    call = Call(c, q, k, v, do)
    call.forward()
    call.backward()
    torch.cuda.synchronize()
    want = c.exact(q, k, v, do, [c.S - c.queries], [c.S], call.scale)
    off = {}
    for name, got, heads in (("dv", call.dv, c.hkv), ("dk", call.dk, c.hkv), ("dq", call.dq, c.hq)):
        exact = want[name][0]
        off[name] = float((c.shaped(got.t.cpu().double(), heads, exact.shape[2]) - exact).norm() / exact.norm())
    assert off["dv"] <= 1e-6 and off["dk"] <= 1.3e-6, off


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 128), ("fp32", 40), ("bf16", 33)])
@pytest.mark.parametrize("what", ["v", "k", "q", "do"])
def test_infinities_and_nan_of_rows_without_weight(what, dtype, d):
    """Scores of hundreds: most weights are below fp32's numbers.  What such a row
    or key holds reaches the rows that see it all the same, in tiles that are seen as
    a whole and in others, and no other rows."""
    c = lc.Attention(S=330, d=d, Hq=4, Hkv=2, window=140, sinks=2, dtype=dtype)
    q, k, v, do = c.inputs(5, 60.0)
    x = {"q": q, "k": k, "v": v, "do": do}[what]
    x[0, 0, 70, 0] = math.inf
    x[0, 1, 150, 1] = NAN
    x[0, 1, 1, d // 2] = -math.inf
    call = Call(c, q, k, v, do)
    call.forward()
    call.backward()
    torch.cuda.synchronize()
    want = c.exact(q, k, v, do, [0], [c.S], call.scale)
    for name, got, heads in (("o", call.o, c.hq), ("dq", call.dq, c.hq), ("dk", call.dk, c.hkv), ("dv", call.dv, c.hkv)):
        exact = want[name][0]
        got = c.shaped(got.t.cpu().double(), heads, c.S)
        assert bool((torch.isfinite(got) == torch.isfinite(exact)).all()), name


ONE_KEY = {
    "window_1": dict(S=70, d=64, Hq=2, Hkv=1, window=1),
    "window_1_128": dict(S=300, d=128, window=1),
    "one_token": dict(S=1, d=64),
    "one_token_odd": dict(B=3, S=1, d=33, Hq=3, Hkv=1),
    "first_key_only": dict(S=200, d=64, window=1, sinks=1),
    "sharp": dict(S=500, d=64, Hq=2, Hkv=1, sharp=300.0),
    "sharp_128": dict(S=500, d=128, Hq=2, Hkv=1, window=70, sharp=300.0),
}


@pytest.mark.parametrize("size", [1.0, 1e-3, 3e3])
@pytest.mark.parametrize("name", ONE_KEY)
def test_rows_of_one_weight_in_fp16(name, size):
    """Rows whose weight is all on one key: dS is 0 but for the rounding of dP and
    delta, which is another one in the two kernels."""
    of = dict(ONE_KEY[name])
    sharp = of.pop("sharp", 1.0)
    if sharp > 1.0:
        size = min(size, 1.0)       # dk is beyond fp16 else
    c = lc.Attention(dtype="fp16", **of)
    q, k, v, do = c.inputs(3, sharp)
    do = (do * size).half().double()
    call = Call(c, q, k, v, do)
    call.forward()
    call.backward()
    call.check(c.exact(q, k, v, do, [0] * c.B, [c.S] * c.B, call.scale))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("of", [dict(S=64), dict(S=2048, queries=2), dict(S=1500, Hq=4, Hkv=4)])
def test_lse_of_equal_scores(dtype, of):
    """log(n) to its last bits: the logarithm to the base of 2 is off by a step of its
    size, the product with log(2) and that constant by half a step each."""
    c = lc.Attention(d=64, dtype=dtype, **of)
    q, k, v, do = c.inputs(0)
    call = Call(c, torch.zeros_like(q), k, v, do)
    call.forward()
    torch.cuda.synchronize()
    want = torch.log((c.S - c.queries + 1 + torch.arange(c.queries)).double())
    got = call.lse.t.view(c.hq, c.queries).cpu().double()
    assert bool(((got - want).abs() <= 4 * lc.U * want).all()), float(((got - want).abs() / want.clamp(1e-9)).max())


@pytest.mark.parametrize("of,sharp,values,size", [(dict(d=64), 12.0, 64.0, 16.0), (dict(d=64), 12.0, 128.0, 8.0), (dict(d=96), 8.0, 64.0, 16.0),
                                                  (dict(d=128, Hq=2), 8.0, 128.0, 16.0)])
def test_small_ds_beside_large_ones(of, sharp, values, size):
    """dS of thousands, which need no power of two: small ones beside them are off by
    no more than fp16's rounding of them as they are."""
    c = lc.Attention(B=2, S=257, window=17, dtype="fp16", **of)
    q, k, v, do = c.inputs(182, sharp)
    v, do = v * values, do * size
    call = Call(c, q, k, v, do)
    call.forward()
    call.backward()
    call.check(c.exact(q, k, v, do, [0, 0], [c.S] * 2, call.scale))


@pytest.mark.parametrize("of,lengths", [(dict(S=700, d=64, Hq=4, window=100, sinks=130), None), (dict(S=300, d=128, Hq=8, window=60), None),
                                        (dict(B=5, S=100, d=64, Hq=6, window=30, sinks=2), [100, 1, 0, 57, 99]),
                                        (dict(S=500, d=40, Hq=3, queries=70), None), (dict(S=129, d=33, order="token"), [77])])
def test_same_bits_whatever_the_workspace_holds(of, lengths):
    c = lc.Attention(dtype="fp16", **{"Hkv": 1, **of})
    q, k, v, do = c.inputs(9)
    runs = []
    for fill in (0, 255, 0x7e, 0xfe, 1):
        call = Call(c, q, k, v, do, None, lengths)
        call.ws.fill_(fill)
        call.gws.fill_(fill)
        call.forward()
        call.backward()
        torch.cuda.synchronize()
        runs.append([g.t.clone() for g in call.outputs()])
    assert all(torch.equal(x, y) for run in runs[1:] for x, y in zip(runs[0], run))
