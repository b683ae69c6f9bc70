"""Attention on head shards on the GPU, forward and gradients, against plain
forms in 64 bits (MI355X only)."""
import math

import pytest
import torch

from tests import index_cases as ic
from tests import layer_cases as lc

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sequence_re_layout_amd import binding as b
else:  # collected on a machine without a GPU: every test here is skipped
    b = None

NAN = float("nan")
INF = float("inf")


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Call:
    """A plan, its inputs on the device and guarded outputs full of NaN."""

    def __init__(self, c, q, k, v, do, starts=None, lengths=None, scale=None, shift=0):
        self.c, self.scale = c, c.d ** -0.5 if scale is None else scale
        code = {torch.bfloat16: b.BASP_BF16, torch.float16: b.BASP_FP16, torch.float32: b.BASP_FP32}[c.dtype]
        order = b.BASP_LAYOUT_HEAD_MAJOR if c.order == "head" else b.BASP_LAYOUT_TOKEN_MAJOR
        layout = b.basp_plan_create_groups(c.N, c.B, c.S, c.Hq, c.Hkv, c.d, code, c.G, order)
        self.plan = b.basp_attention_plan_create(layout, c.queries, c.window, c.sinks)
        i = self.plan.info
        assert (i["shards"], i["Hl_q"], i["Hl_kv"]) == (c.shards, c.hq, c.hkv)
        put = lambda x: ic.shifted(c.buffer(x.to(c.dtype)), shift).cuda() if not shift else ic.shifted(c.buffer(x.to(c.dtype)).cuda(), shift)
        self.q, self.k, self.v, self.do = put(q), put(k), put(v), put(do)
        each = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
        self.starts, self.lengths = each(starts), each(lengths)
        out = lambda n, dt=c.dtype: ic.Guarded(n, dt, NAN, shift)
        self.o, self.lse = out(i["q_elems"]), ic.Guarded(i["lse_elems"], torch.float32, NAN)
        self.dq, self.dk, self.dv = out(i["q_elems"]), out(i["kv_elems"]), out(i["kv_elems"])
        self.ws = torch.full((max(1, i["workspace_bytes"]),), 255, dtype=torch.uint8, device="cuda")
        self.gws = torch.full((max(1, i["grad_workspace_bytes"]),), 255, dtype=torch.uint8, device="cuda")

    def forward(self, lse=True):
        b.basp_attention(self.plan, self.q, self.k, self.v, self.starts, self.lengths, self.scale, self.o.t,
                         self.lse.t if lse else None, self.ws)

    def backward(self):
        b.basp_attention_grad(self.plan, self.q, self.k, self.v, self.o.t, self.lse.t, self.do, self.starts, self.lengths, self.scale,
                              self.dq.t, self.dk.t, self.dv.t, self.gws)

    def outputs(self, grads=True):
        return [self.o, self.lse] + ([self.dq, self.dk, self.dv] if grads else [])

    def check(self, exact, grads=True, near=False):
        """near: the errors' squares, too.  A rounding is off by h / sqrt(3) in the
        mean square, and the weights, dS and the result take one each: h together,
        and as much again for what has a hundredth of that in fp32."""
        torch.cuda.synchronize()
        c = self.c
        names = ("o", "lse", "dq", "dk", "dv") if grads else ("o", "lse")
        for name, g in zip(names, self.outputs(grads)):
            g.check(name)
            want, err = exact[name]
            got = g.t.cpu()
            got = got.view(want.shape) if name == "lse" else c.shaped(got, want.shape[1], want.shape[2])
            lc.check(got.contiguous(), want, err, name)
            if near and name != "lse":
                off = float((got.double() - want).norm() / want.norm())
                assert off <= max(2 * lc.half_step(c.dtype)[0], 4e-6), (name, off)


CASES = {
    "one_token": dict(S=1, d=64),
    "two_tokens_window_1": dict(S=2, window=1, d=16, dtype="fp32"),
    "window_1": dict(S=70, window=1, d=32),
    "window_1_sinks": dict(S=150, window=1, sinks=2, d=64, Hq=2),
    "one_channel": dict(S=37, d=1, dtype="fp16"),
    "odd_channels": dict(S=65, d=33, Hq=3, Hkv=1, window=20, sinks=5),
    "odd_channels_fp32": dict(S=65, d=7, Hq=3, Hkv=1, window=20, sinks=5, dtype="fp32"),
    "three_heads_a_key": dict(S=200, d=72, Hq=6, Hkv=2, window=50, sinks=3, dtype="fp16"),
    "whole": dict(S=257, d=64, Hq=2),
    "whole_128": dict(S=130, d=128, Hq=4, Hkv=2),
    "whole_fp32_128": dict(S=130, d=128, Hq=2, Hkv=1, dtype="fp32"),
    "tile_edges": dict(S=192, d=64, window=64, sinks=64),
    "sinks_in_the_window": dict(S=300, d=64, window=150, sinks=200),
    "many_sinks": dict(S=600, d=40, window=33, sinks=300, dtype="fp32"),
    "sinks_of_two_blocks": dict(S=700, d=64, Hq=4, Hkv=1, window=100, sinks=130),
    "token_order": dict(N=4, B=2, G=2, S=128, Hq=8, Hkv=4, d=48, window=40, sinks=1, order="token"),
    "token_order_fp32": dict(N=2, B=3, G=1, S=90, Hq=4, Hkv=2, d=24, window=31, sinks=2, order="token", dtype="fp32"),
    "groups": dict(N=4, B=4, G=2, S=66, Hq=4, Hkv=4, d=64, window=30),
    "long_chunks": dict(S=2100, d=64, window=300, sinks=4),
    "long_whole": dict(S=1500, d=128, dtype="fp16"),
    "heads_apart": dict(S=300, d=64, Hq=8, Hkv=1, window=60, sinks=2, dtype="fp32"),
    "heads_and_sinks_apart": dict(S=520, d=128, Hq=6, Hkv=1, window=200, sinks=130),
    "heads_apart_whole": dict(S=700, d=40, Hq=12, Hkv=2, dtype="fp16"),
    "few_rows_many_heads": dict(N=2, S=8, d=80, Hq=32, Hkv=4, dtype="fp32"),
    "three_channels": dict(S=75, d=3, Hq=2, window=40),
    "channels_past_a_chunk": dict(S=75, d=11, Hq=2, Hkv=1, dtype="fp16"),
    "sharp": dict(S=300, d=64, Hq=2, sharp=30.0),
    "sharp_fp16": dict(S=300, d=128, Hq=2, sharp=30.0, dtype="fp16"),
}


@pytest.mark.parametrize("name", CASES)
def test_forward_and_gradients(name):
    of = dict(CASES[name])
    sharp = of.pop("sharp", 1.0)
    c = lc.Attention(**of)
    q, k, v, do = c.inputs(len(name), sharp)
    call = Call(c, q, k, v, do)
    call.forward()
    call.backward()
    call.check(c.exact(q, k, v, do, [0] * c.B, [c.S] * c.B, call.scale), near=sharp == 1.0 and min(c.S, c.window) >= 16)


PADDED = {
    "lengths": dict(of=dict(B=5, S=100, d=64, Hq=4, Hkv=2, window=30, sinks=2), starts=None, lengths=[100, 1, 0, 57, 99]),
    "lengths_outside": dict(of=dict(B=3, S=70, d=32, dtype="fp32"), starts=None, lengths=[-5, 71, 2 ** 31 - 1]),
    "starts_anywhere": dict(of=dict(B=6, S=80, d=64, queries=20, window=25, sinks=3, Hq=2),
                            starts=[0, 60, 70, -10, -25, 100], lengths=[80, 80, 75, 80, 30, 80]),
    "starts_far": dict(of=dict(B=4, S=50, d=64, queries=7, Hq=2), starts=[2 ** 31 - 1, -2 ** 31, 49, 43], lengths=[50] * 4),
    "all_rows_empty": dict(of=dict(B=2, S=64, d=64, Hq=2), starts=None, lengths=[0, 0]),
    "training_padded": dict(of=dict(N=2, B=4, G=2, S=300, d=128, Hq=4, Hkv=2, window=90, sinks=4), starts=None,
                            lengths=[300, 10, 129, 250]),
    "chunk_of_a_prompt": dict(of=dict(B=2, S=500, d=64, Hq=2, Hkv=1, queries=150, window=200, sinks=4), starts=[100, 350],
                              lengths=[250, 500]),
}


@pytest.mark.parametrize("name", PADDED)
def test_padding_is_not_read(name):
    """Lengths and starts of every sequence; NaN in all keys and values after a
    sequence's end, and in rows that see nothing."""
    p = PADDED[name]
    c = lc.Attention(**p["of"])
    q, k, v, do = c.inputs(7)
    lengths = [max(0, min(n, c.S)) for n in p["lengths"]]
    starts = p["starts"] or [0] * c.B
    for n, s in enumerate(c.sequence):
        k[n, :, lengths[s]:] = NAN
        v[n, :, lengths[s]:] = INF
        dead = ~c.sees(starts[s], lengths[s]).any(1)
        q[n, :, dead] = NAN
        do[n, :, dead] = NAN
    call = Call(c, q, k, v, do, p["starts"], p["lengths"])
    call.forward()
    call.backward()
    call.check(c.exact(q, k, v, do, starts, lengths, call.scale))


STEPS = {
    "one_of_many": dict(N=2, B=4, S=600, d=64, Hq=8, Hkv=2, queries=1, window=200, sinks=4),
    "whole_cache": dict(B=2, S=3000, d=128, Hq=4, Hkv=1, queries=1, dtype="fp16"),
    "whole_cache_fp32": dict(B=2, S=1300, d=128, Hq=4, Hkv=1, queries=1, dtype="fp32"),
    "few": dict(B=3, S=700, d=40, Hq=6, Hkv=2, queries=5, window=300, sinks=70, order="token"),
    "more_than_a_block": dict(B=1, S=1500, d=64, Hq=8, Hkv=1, queries=9),
    "prompt_on_a_long_cache": dict(B=1, S=4000, d=64, Hq=2, Hkv=1, queries=70),
    "odd_rows": dict(B=2, S=900, d=20, Hq=3, Hkv=1, queries=2, dtype="bf16"),
    "two_blocks_fp32": dict(B=2, S=305, d=96, Hq=16, Hkv=2, queries=5, dtype="fp32"),
    "tiny_cache": dict(B=2, S=3, d=64, Hq=2, Hkv=1, queries=2),
}


@pytest.mark.parametrize("name", STEPS)
def test_last_tokens_of_a_cache(name):
    """starts NULL: the last queries of every sequence."""
    c = lc.Attention(**STEPS[name])
    q, k, v, do = c.inputs(3)
    lengths = [max(1, c.S - 97 * i) for i in range(c.B)]
    call = Call(c, q, k, v, do, None, lengths)
    call.forward()
    want = c.exact(q, k, v, do, [n - c.queries for n in lengths], lengths, call.scale)
    call.check(want, grads=False)
    first = call.o.t.clone()
    call.o.t.fill_(NAN)
    call.forward(lse=False)
    torch.cuda.synchronize()
    assert torch.equal(call.o.t, first)
    call.forward()
    call.backward()
    call.check(want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shift", [1, 4])
def test_any_element_address(dtype, shift):
    """Buffers that start off a 16-byte boundary, in whole and in ragged rows."""
    for d in (64, 50, 128):
        c = lc.Attention(S=150, d=d, Hq=2, Hkv=1, window=70, sinks=3, dtype=dtype)
        q, k, v, do = c.inputs(d)
        call = Call(c, q, k, v, do, shift=shift)
        call.forward()
        call.backward()
        call.check(c.exact(q, k, v, do, [0], [c.S], call.scale))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 128), ("fp32", 64), ("bf16", 33)])
@pytest.mark.parametrize("what", ["v", "k", "q", "do"])
def test_infinities_and_nan_stay_where_they_are_seen(dtype, d, what):
    """A token's infinities and NaN reach the rows (or keys) that see it and no
    others: rows before it, rows whose window has passed it, other heads."""
    c = lc.Attention(S=260, d=d, Hq=4, Hkv=2, window=45, sinks=2, dtype=dtype)
    q, k, v, do = c.inputs(5)
    x = {"q": q, "k": k, "v": v, "do": do}[what]
    x[0, 0, 100, 0] = INF if what in ("v", "do") else NAN
    x[0, 0, 130, d // 2] = -INF if what in ("v", "do") else NAN
    x[0, 1, 200] = NAN
    call = Call(c, q, k, v, do)
    call.forward()
    call.backward()
    torch.cuda.synchronize()
    want = c.exact(q, k, v, do, [0], [c.S], call.scale)
    for name, g in zip(("o", "lse", "dq", "dk", "dv"), call.outputs()):
        value, err = want[name]
        got = g.t.cpu()
        got = (got.view(value.shape) if name == "lse" else c.shaped(got, value.shape[1], value.shape[2])).double()
        fine = torch.isfinite(value) & torch.isfinite(err)
        assert bool(torch.isfinite(got[fine]).all()), name
        assert not bool(torch.isfinite(got[~torch.isfinite(value)]).any()), name
        over = (got - value).abs() > err + lc.half_step(c.dtype if name != "lse" else torch.float32)[0] * (value.abs() + err) + lc.half_step(c.dtype)[1]
        assert not bool((over & fine).any()), name


@pytest.mark.parametrize("name", ["sinks_of_two_blocks", "heads_apart", "heads_and_sinks_apart", "long_chunks", "token_order_fp32", "whole_128"])
def test_same_bits_every_time(name):
    c = lc.Attention(**CASES[name])
    q, k, v, do = c.inputs(9)
    runs = []
    for fill in (0, 255):
        call = Call(c, q, k, v, do)
        call.ws.fill_(fill)
        call.gws.fill_(fill)
        call.forward()
        call.backward()
        torch.cuda.synchronize()
        runs.append([g.t.clone() for g in call.outputs()])
    assert all(torch.equal(x, y) for x, y in zip(*runs))


def test_scales():
    """Scores of any size: the running maximum moves up all along, and weights
    below the type's range."""
    for scale, dtype in ((3.0, "fp16"), (1e-6, "bf16"), (20.0, "fp32"), (2.0 ** -60, "bf16"), (2.0 ** -100, "fp32")):
        c = lc.Attention(S=333, d=64, Hq=2, Hkv=1, dtype=dtype)
        q, k, v, do = c.inputs(1)
        k *= torch.linspace(0.0, 2.0, c.S, dtype=torch.float64)[:, None].expand(c.S, c.d)
        k = k.to(c.dtype).double()
        call = Call(c, q, k, v, do, scale=scale)
        call.forward()
        call.backward()
        call.check(c.exact(q, k, v, do, [0], [c.S], call.scale))


def test_gradient_against_differences():
    """The gradient of a sum of o * do by central differences of the exact o."""
    c = lc.Attention(S=40, d=8, Hq=2, Hkv=1, window=9, sinks=2, dtype="fp32")
    q, k, v, do = c.inputs(4)
    call = Call(c, q, k, v, do)
    call.forward()
    call.backward()
    torch.cuda.synchronize()
    loss = lambda q, k, v: float((c.exact(q, k, v, do, [0], [c.S], call.scale)["o"][0] * do).sum())
    g = torch.Generator()
    g.manual_seed(8)
    for which, got, heads in ((0, call.dq, c.hq), (1, call.dk, c.hkv), (2, call.dv, c.hkv)):
        x = [q, k, v]
        way = torch.randn(x[which].shape, generator=g, dtype=torch.float64)
        step = 1e-4
        up, down = list(x), list(x)
        up[which], down[which] = x[which] + step * way, x[which] - step * way
        want = (loss(*up) - loss(*down)) / (2 * step)
        have = float((c.shaped(got.t.cpu().double(), heads, c.S) * way).sum())
        # differences are off by the third derivative, step^2 of the terms' size; the gradient by 1e-6 of its terms
        terms = float((c.shaped(got.t.cpu().double(), heads, c.S) * way).abs().sum())
        assert abs(have - want) <= 1e-5 * terms, which


def test_beyond_four_gib():
    """The last token of a cache of 2^25 tokens: keys and values 8 GiB each, the
    window at the far end, the sinks at the near one."""
    S, d, window, sinks = 1 << 25, 128, 300, 3
    layout = b.basp_plan_create_groups(1, 1, S, 2, 1, d, b.BASP_FP16, 1, b.BASP_LAYOUT_HEAD_MAJOR)
    plan = b.basp_attention_plan_create(layout, 1, window, sinks)
    k, v = (torch.empty(S * d, dtype=torch.float16, device="cuda") for _ in range(2))
    for x in (k, v):
        x.view(torch.int16).fill_(0x7e00)            # NaN wherever nothing is to be read
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    seen = list(range(sinks)) + list(range(S - window, S))
    for x in (k, v):
        for part in (slice(0, sinks), slice(S - window, S)):
            x.view(S, d)[part] = torch.randn(x.view(S, d)[part].shape, generator=g, device="cuda").half()
    q = torch.randn(2 * d, generator=g, device="cuda").half()
    o, lse = torch.empty_like(q), torch.empty(2, device="cuda")
    ws = torch.empty(max(1, plan.info["workspace_bytes"]), dtype=torch.uint8, device="cuda")
    b.basp_attention(plan, q, k, v, None, None, d ** -0.5, o, lse, ws)
    pick = torch.tensor(seen, device="cuda")
    ks, vs = k.view(S, d)[pick].double(), v.view(S, d)[pick].double()
    p = torch.softmax(q.view(2, d).double() @ ks.T * d ** -0.5, 1)
    want = p @ vs
    # weights and result are rounded once each: 2^-11 of the terms and of the result, twice for the rest
    assert bool(((o.view(2, d).double() - want).abs() <= 2.0 ** -10 * (p @ vs.abs())).all())
    assert bool(torch.allclose(lse.double(), torch.logsumexp(q.view(2, d).double() @ ks.T * d ** -0.5, 1), rtol=0, atol=1e-4))


def test_empty_cache():
    layout = b.basp_plan_create_groups(2, 1, 0, 2, 2, 64, b.BASP_BF16, 1)
    plan = b.basp_attention_plan_create(layout, 0, 1)
    b.basp_attention(plan, None, None, None, None, None, 1.0, None, None, None)
    b.basp_attention_grad(plan, *[None] * 8, 1.0, *[None] * 4)
    torch.cuda.synchronize()
