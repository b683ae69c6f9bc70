"""The index-driven re-layouts as a program uses them (MI355X only): through
autograd, together with the attention boundary, on side streams, in captured
graphs, timed, and refused."""
import numpy as np
import pytest
import torch

from tests import index_cases as ic

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sequence_re_layout_amd import autograd as ag
    from sequence_re_layout_amd import binding as b
else:  # collected on a machine without a GPU: every test here is skipped
    ag = b = None

NAN = float("nan")


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Model:
    """Embedding -> attention boundary and back -> experts (one matrix each)
    -> weighted sum.  Linear in each of table, expert matrices and weights, so
    the same graph on absolute values bounds every rounding error."""

    N, B, S, H, d, V, E, K = 4, 2, 48, 4, 12, 61, 6, 3

    def __init__(self, seed):
        self.D, self.T = self.H * self.d, self.B * self.S
        rng = np.random.default_rng(seed)
        self.ids = rng.integers(0, self.V, self.T)
        self.chosen = ic.choices(rng, self.T, self.K, self.E, 0.1)
        self.scale = 1.5
        self.table = rng.standard_normal((self.V, self.D)).astype(np.float32)
        self.mats = rng.standard_normal((self.E, self.D, self.D)).astype(np.float32)
        self.w = rng.random((self.T, self.K)).astype(np.float32)
        self.g = rng.standard_normal((self.T, self.D)).astype(np.float32)

    def library(self, align):
        """Output and gradients through the library, expert products by torch
        in fp32 over whole padded segments."""
        layout = b.basp_plan_create(self.N, self.B, self.S, self.H, self.H, self.d, b.BASP_FP32, b.BASP_MODE_ULYSSES)
        embed = b.basp_embed_plan_create(layout, self.T, self.V, self.D, dtype=b.BASP_FP32, grad_dtype=b.BASP_FP32)
        experts = b.basp_expert_plan_create(self.T, self.K, self.E, self.D, align=align, dtype=b.BASP_FP32)
        table, mats, w = (torch.from_numpy(v).cuda().requires_grad_() for v in (self.table, self.mats, self.w))
        h = ag.embed_to_seq(embed, torch.from_numpy(self.ids).cuda(), table, self.scale)
        flat = h.reshape(-1)
        qkv = ag.seq_to_head_qkv(layout, flat, flat, flat)
        h = ag.head_to_seq_o(layout, qkv[:layout.info["q_elems"]]).view(self.T, self.D)
        rows, index = ag.route_to_expert(experts, h, torch.from_numpy(self.chosen).cuda())
        ends = index.offsets.tolist()
        parts = [rows[ends[e]:ends[e + 1]] @ mats[e] for e in range(self.E)]
        out = torch.cat(parts + [rows[ends[-1]:]])
        y = ag.expert_to_seq(experts, out, w, index)
        return (y, *torch.autograd.grad(y, (table, mats, w), torch.from_numpy(self.g).cuda()))

    def exact(self, absolute):
        t = lambda v: torch.from_numpy(v).double().abs() if absolute else torch.from_numpy(v).double()
        table, mats, w = (t(v).requires_grad_() for v in (self.table, self.mats, self.w))
        place = torch.from_numpy(ic.seq_place(self.N, self.B, self.S, 1))
        back = torch.empty_like(place)
        back[place] = torch.arange(self.T)
        h = table[torch.from_numpy(self.ids)[back]] * self.scale
        y = torch.zeros(self.T, self.D, dtype=torch.float64)
        for k in range(self.K):
            e = torch.from_numpy(self.chosen[:, k])
            kept = (e >= 0) & (e < self.E)
            prod = torch.einsum("td,tde->te", h, mats[e.clamp(0, self.E - 1)])
            y = y + torch.where(kept, w[:, k], 0.0)[:, None] * prod
        grads = torch.autograd.grad(y, (table, mats, w), t(self.g))
        return [v.detach().numpy() for v in (y, *grads)]


@pytest.mark.parametrize("align", [1, 16])
def test_model_with_gradients(align):
    """Output and all gradients; a value passes at most one rounding per
    addend of each sum on its way."""
    m = Model(3)
    got, want, terms = m.library(align), m.exact(False), m.exact(True)
    n = 4 * m.D + 4 * m.K + 3 * m.T
    for v, x, a, what in zip(got, want, terms, ("y", "dtable", "dmats", "dw")):
        ic.check(v.detach(), x, a, n, what)


def test_gradients_against_differences():
    """Every call is linear in each input, so a central difference of any step
    is exact: <g, f(x + v) - f(x - v)> / 2 = <gradient, v>, up to the fp32
    roundings of f at both points and of the gradient."""
    T, K, E, D, V = 70, 3, 5, 40, 33
    rng = np.random.default_rng(5)
    normal = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()
    plan = b.basp_expert_plan_create(T, K, E, D, align=4, dtype=b.BASP_FP32)
    ids = torch.from_numpy(ic.choices(rng, T, K, E, 0.2)).cuda()
    index = ag.sort_by_expert(plan, ids)
    R = plan.info["max_rows"]
    rows, w = normal(R, D), normal(T, K)
    ep = b.basp_embed_plan_create(None, T, V, D, dtype=b.BASP_FP32, grad_dtype=b.BASP_FP32)
    tokens = torch.from_numpy(rng.integers(-1, V, T)).cuda()
    steps = {
        "seq_to_expert": (lambda x: ag.seq_to_expert(plan, x, index), normal(T, D), K),
        "route_to_expert": (lambda x: ag.route_to_expert(plan, x, ids)[0], normal(T, D), K),
        "expert_to_seq, rows": (lambda x: ag.expert_to_seq(plan, x, w, index), rows, K),
        "expert_to_seq, weights": (lambda x: ag.expert_to_seq(plan, rows, x, index), w, D),
        "embed_to_seq": (lambda x: ag.embed_to_seq(ep, tokens, x, 0.5), normal(V, D), T),
    }
    for what, (f, x, n) in steps.items():
        x = x.requires_grad_()
        y = f(x)
        g, v = normal(*y.shape), normal(*x.shape)
        (grad,) = torch.autograd.grad(y, (x,), g)
        with torch.no_grad():
            plus, minus = f(x + v).double(), f(x - v).double()
        diff = float((g.double() * (plus - minus)).sum() / 2)
        dot = float((grad.double() * v.double()).sum())
        # roundings: x +- v (one each), n + 1 in f and n + 1 in the gradient,
        # all relative to the sum of the absolute products
        with torch.no_grad():
            big = {"expert_to_seq, rows": lambda z: ag.expert_to_seq(plan, z, w.abs(), index),
                   "expert_to_seq, weights": lambda z: ag.expert_to_seq(plan, rows.abs(), z, index)}.get(what, f)
            terms = float((g.abs().double() * big(x.abs() + v.abs()).double()).sum())
        assert abs(diff - dot) <= 2 * (2 * n + 4) * 2.0 ** -24 * terms, what
        if what == "embed_to_seq":
            untouched = torch.ones(V, dtype=torch.bool, device="cuda")
            untouched[tokens[tokens >= 0]] = False
            assert bool((grad[untouched] == 0).all())


class Step:
    """One training step's calls on fixed buffers, for capture and replay."""

    def __init__(self, T=300, K=3, E=20, D=136, V=5000, S=150):
        self.T, self.K, self.E, self.D, self.V = T, K, E, D, V
        new = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")
        layout = b.basp_plan_create(2, T // S, S, 2, 2, 8, b.BASP_BF16, b.BASP_MODE_ULYSSES)
        self.embed = b.basp_embed_plan_create(layout, T, V, D)
        self.plan = b.basp_expert_plan_create(T, K, E, D, align=8)
        R = self.plan.info["max_rows"]
        self.tokens, self.table = new(T, dt=torch.int64), new(V, D)
        self.ids, self.w, self.g = new(T, K, dt=torch.int64), new(T, K, dt=torch.float32), new(T, D)
        self.index = [new(n, dt=torch.int32) for n in (T * K, R, E + 1, E)]
        self.h, self.y, self.dx, self.rows, self.drows = new(T, D), new(T, D), new(T, D), new(R, D), new(R, D)
        self.dw, self.dtable = new(T, K, dt=torch.float32), new(V, D)
        self.ws = [new(max(1, p.info["workspace_bytes"]), dt=torch.uint8) for p in (self.plan, self.embed)]

    def fill(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.tokens.copy_(torch.randint(0, self.V, (self.T,), generator=g, device="cuda"))
        self.ids.copy_(torch.randint(-1, self.E + 1, (self.T, self.K), generator=g, device="cuda"))
        for t in (self.table, self.w, self.g):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    def outputs(self):
        return [*self.index, self.h, self.rows, self.y, self.drows, self.dw, self.dx, self.dtable]

    def spoil(self):
        for t in self.outputs():
            t.fill_(-9)
        for t in self.ws:
            t.fill_(170)

    def run(self):
        pos, order = self.index[0], self.index[1]
        b.basp_embed_to_seq(self.embed, self.tokens, self.table, 2.0, self.h)
        b.basp_route_to_expert(self.plan, self.h, self.ids, *self.index, self.rows, self.ws[0])
        b.basp_expert_to_seq(self.plan, self.rows, pos, self.w, self.y)
        b.basp_expert_to_seq_grad(self.plan, self.g, self.rows, pos, order, self.w, self.drows, self.dw)
        b.basp_seq_to_expert_grad(self.plan, self.drows, pos, self.dx)
        b.basp_embed_to_seq_grad(self.embed, self.tokens, self.dx, 2.0, False, self.dtable, self.ws[1])

    def want(self, seed):
        self.fill(seed)
        self.spoil()
        self.run()
        torch.cuda.synchronize()
        return [t.clone() for t in self.outputs()]


SIZES = [dict(), dict(T=1200, K=2, S=600), dict(T=9000, K=1, E=64, D=64, V=70000, S=4500)]


@pytest.mark.parametrize("size", SIZES, ids=["small", "more slots", "many tokens"])
def test_graph_replays(size):
    """A captured step, replayed on new inputs with eager work in between,
    gives the eager step's bits."""
    s, eager = Step(**size), Step(**size)
    s.fill(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (11, 12, 13):
        want = eager.want(seed)
        s.fill(seed)
        s.spoil()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, w) in enumerate(zip(s.outputs(), want)):
            assert torch.equal(a, w), (seed, i)


def test_streams_at_the_same_time():
    """Two steps on two side streams, each with workspaces of its own and on
    plans that both use; and a stream given by its handle."""
    one, two = Step(T=9000, K=2, E=64, D=64, V=70000, S=4500), Step(T=9000, K=2, E=64, D=64, V=70000, S=4500)
    want = [one.want(21), two.want(22)]
    two.plan, two.embed = one.plan, one.embed
    for s in (one, two):
        s.spoil()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, stream in zip((one, two), streams):
            with torch.cuda.stream(stream):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip((one, two), want):
        assert all(torch.equal(a, x) for a, x in zip(s.outputs(), w))
    two.y.fill_(-9)
    torch.cuda.synchronize()
    b.basp_expert_to_seq(two.plan, two.rows, two.index[0], two.w, two.y, stream=streams[1].cuda_stream)
    streams[1].synchronize()
    assert torch.equal(two.y, want[1][6])


def test_backward_in_a_graph():
    """Forward and backward through the autograd wrappers inside one capture,
    on leaves of its own."""
    T, K, E, D = 200, 2, 8, 64
    plan = b.basp_expert_plan_create(T, K, E, D, dtype=b.BASP_FP32)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    ids = torch.randint(0, E, (T, K), generator=gen, device="cuda")
    x = torch.randn(T, D, generator=gen, device="cuda").requires_grad_()
    w = torch.rand(T, K, generator=gen, device="cuda").requires_grad_()
    g = torch.randn(T, D, generator=gen, device="cuda")

    def step():
        rows, index = ag.route_to_expert(plan, x, ids)
        y = ag.expert_to_seq(plan, rows * 2, w, index)
        return (y.detach(), *torch.autograd.grad(y, (x, w), g))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (3, 4, 5):
        gen.manual_seed(seed)
        with torch.no_grad():
            x.copy_(torch.randn(T, D, generator=gen, device="cuda"))
            g.copy_(torch.randn(T, D, generator=gen, device="cuda"))
            ids.copy_(torch.randint(0, E, (T, K), generator=gen, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        # the exact values: x twice over with all weights, and the gradients
        xe, we, ge = x.detach().double(), w.detach().double(), g.double()
        want = (2 * xe * we.sum(1, keepdim=True), 2 * ge * we.sum(1, keepdim=True),
                (2 * xe * ge).sum(1, keepdim=True).expand(T, K))
        terms = (2 * xe.abs() * we.sum(1, keepdim=True), 2 * ge.abs() * we.sum(1, keepdim=True),
                 (2 * xe * ge).abs().sum(1, keepdim=True).expand(T, K))
        for v, e, a in zip(kept, want, terms):
            ic.check(v, e.cpu().numpy(), a.cpu().numpy(), D + 4, "replay %d" % seed)


def test_timed_calls():
    """basp_time_next_call covers every launch of a call, and one call only."""
    s = Step(T=9000, K=2, E=64, D=64, V=70000, S=4500)
    want = s.want(31)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in ev:
        e.record()
    torch.cuda.synchronize()
    pos, order = s.index[0], s.index[1]
    for call in (lambda: b.basp_route_to_expert(s.plan, s.h, s.ids, *s.index, s.rows, s.ws[0]),
                 lambda: b.basp_expert_sort(s.plan, s.ids, *s.index, s.ws[0]),
                 lambda: b.basp_seq_to_expert(s.plan, s.h, pos, order, s.rows),
                 lambda: b.basp_expert_to_seq(s.plan, s.rows, pos, s.w, s.y),
                 lambda: b.basp_expert_to_seq_grad(s.plan, s.g, s.rows, pos, order, s.w, s.drows, s.dw),
                 lambda: b.basp_embed_to_seq_grad(s.embed, s.tokens, s.dx, 2.0, False, s.dtable, s.ws[1])):
        b.basp_time_next_call(*ev)
        call()
        torch.cuda.synchronize()
        ms = ev[0].elapsed_time(ev[1])
        assert 0 < ms < 50
        call()                                  # not timed: the events keep their times
        torch.cuda.synchronize()
        assert ev[0].elapsed_time(ev[1]) == ms
    assert all(torch.equal(a, x) for a, x in zip(s.outputs(), want))


def test_binding_refuses():
    """What the binding checks before the library is called."""
    s = Step()
    s.fill(1)
    pos, order = s.index[0], s.index[1]
    with pytest.raises(TypeError, match="pos"):
        b.basp_expert_to_seq(s.plan, s.rows, pos.long(), s.w, s.y)
    with pytest.raises(TypeError, match="weights"):
        b.basp_expert_to_seq(s.plan, s.rows, pos, s.w.bfloat16(), s.y)
    with pytest.raises(TypeError, match="ids"):
        b.basp_route_to_expert(s.plan, s.h, s.ids.int(), *s.index, s.rows, s.ws[0])
    with pytest.raises(ValueError, match="rows must be contiguous"):
        b.basp_expert_to_seq(s.plan, s.rows.t(), pos, s.w, s.y)
    with pytest.raises(ValueError, match="out holds"):
        b.basp_expert_to_seq(s.plan, s.rows, pos, s.w, s.y[1:])
    with pytest.raises(ValueError, match="device tensor"):
        b.basp_expert_to_seq(s.plan, s.rows, pos, s.w.cpu(), s.y)
    with pytest.raises(ValueError, match="ws holds"):
        b.basp_embed_to_seq_grad(s.embed, s.tokens, s.dx, 1.0, False, s.dtable, s.ws[1][:-1])
    with pytest.raises(ValueError, match="contiguous device tensor"):
        b.basp_embed_to_seq_grad(s.embed, s.tokens, s.dx, 1.0, False, s.dtable, s.ws[1].cpu())
    with pytest.raises(b.BaspError) as e:
        b.basp_embed_to_seq_grad(s.embed, s.tokens, s.dx, 1.0, False, s.dtable, None)
    assert e.value.status == b.BASP_ERR_INVALID
    with pytest.raises(b.BaspError) as e:
        b.basp_seq_to_expert(s.plan, s.rows.view(-1)[:s.h.numel()].view_as(s.h), pos, order, s.rows)
    assert e.value.status == b.BASP_ERR_ALIAS


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_all_values(dtype):
    """Every 16-bit pattern: moved bit for bit, and through a factor of one
    unchanged (subnormals and signed zeros too), NaN staying NaN."""
    dt = ic.FLOATS[dtype]
    code = {"bf16": b.BASP_BF16, "fp16": b.BASP_FP16}[dtype]
    bits = torch.arange(-32768, 32768, device="cuda").to(torch.int16)
    x = bits.view(dt).view(256, 256)
    plan = b.basp_expert_plan_create(256, 1, 4, 256, dtype=code)
    ids = (torch.arange(256, device="cuda") * 7 % 4).view(256, 1)
    rows, index = ag.route_to_expert(plan, x, ids)
    assert torch.equal(rows.view(torch.int16), x.view(torch.int16)[index.order.long()])
    y = ag.expert_to_seq(plan, rows, torch.ones(256, 1, device="cuda"), index)
    ep = b.basp_embed_plan_create(None, 256, 256, 256, dtype=code, grad_dtype=code)
    tokens = torch.arange(256, device="cuda")
    z = ag.embed_to_seq(ep, tokens, x, 1.0)
    g = torch.empty_like(x)
    ws = torch.empty(ep.info["workspace_bytes"], dtype=torch.uint8, device="cuda")
    b.basp_embed_to_seq_grad(ep, tokens, x, 1.0, False, g, ws)
    nan = torch.isnan(x)
    for what, got, zeros in (("expert_to_seq", y, False), ("embed_to_seq", z, True), ("gradient", g, False)):
        assert bool(torch.isnan(got[nan]).all()), what
        if zeros:
            assert torch.equal(got.view(torch.int16)[~nan], x.view(torch.int16)[~nan]), what
        else:               # a sum that starts at +0: the sign of a zero may be lost
            assert torch.equal(got[~nan], x[~nan]), what


def test_one_input_needs_its_gradient():
    """Gradients of rows or of weights alone, and of expanded inputs."""
    T, K, E, D = 64, 2, 4, 32
    plan = b.basp_expert_plan_create(T, K, E, D, dtype=b.BASP_FP32)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    ids = torch.randint(0, E, (T, K), generator=gen, device="cuda")
    index = ag.sort_by_expert(plan, ids)
    rows = torch.randn(plan.info["max_rows"], D, generator=gen, device="cuda")
    w = torch.rand(T, K, generator=gen, device="cuda")
    both = [t.clone().requires_grad_() for t in (rows, w)]
    want = torch.autograd.grad(ag.expert_to_seq(plan, *both, index).sum(), both)   # an expanded gradient
    for i in range(2):
        one = [t.clone().requires_grad_(i == j) for j, t in enumerate((rows, w))]
        (got,) = torch.autograd.grad(ag.expert_to_seq(plan, *one, index).sum(), (one[i],))
        assert torch.equal(got, want[i])
    # one weight for every token: its gradient is the sum over the tokens
    s = torch.full((1, K), 0.5, device="cuda").requires_grad_()
    (got,) = torch.autograd.grad(ag.expert_to_seq(plan, rows, s.expand(T, K).contiguous(), index).sum(), (s,))
    terms = want[1].double().sum(0, keepdim=True)
    assert torch.allclose(got.double(), terms, rtol=0, atol=2 * (T + D) * 2.0 ** -24 * float(rows.abs().sum()))


def test_plan_of_another_thread_and_stream():
    """One plan used by several threads at once, each on its own stream."""
    import threading
    steps = [Step() for _ in range(4)]
    want = [s.want(40 + i) for i, s in enumerate(steps)]
    for s in steps:
        s.plan, s.embed = steps[0].plan, steps[0].embed
        s.spoil()
    torch.cuda.synchronize()
    failed = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    s.run()
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001  (reported by the main thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, x) for a, x in zip(s.outputs(), w))
