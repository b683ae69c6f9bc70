"""Attention, norm and balance loss together with the re-layouts, as a layer uses
them: a model with gradients, captured graphs, streams, refusals (MI355X only)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sequence_re_layout_amd import autograd as ag
    from sequence_re_layout_amd import binding as b
else:  # collected on a machine without a GPU: every test here is skipped
    ag = b = None


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


N, B, G, S, HQ, HKV, D_HEAD, V, E, K = 4, 2, 2, 48, 8, 4, 16, 90, 6, 2
D = HQ * D_HEAD
WINDOW, SINKS, EPS, COEF = 13, 2, 1e-5, 0.05


def parameters(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    return dict(table=n(V, D), w1=1 + 0.1 * n(D), b1=0.1 * n(D), wq=n(D, HQ * D_HEAD) * D ** -0.5, wk=n(D, HKV * D_HEAD) * D ** -0.5,
                wv=n(D, HKV * D_HEAD) * D ** -0.5, wo=n(D, D) * D ** -0.5, w2=1 + 0.1 * n(D), b2=0.1 * n(D),
                router=n(D, E) * D ** -0.5, experts=n(E, D, D) * D ** -0.5)


def library(p, tokens, lengths, plans, target):
    """One layer through the library: the loss."""
    boundary, embed, norm, attend, experts = plans
    h = ag.embed_to_seq(embed, tokens, p["table"], 2.0)
    x = ag.layer_norm(norm, h, p["w1"], p["b1"], EPS)
    qkv = ag.seq_to_head_qkv(boundary, *((x @ p[n]).view(-1) for n in ("wq", "wk", "wv")))
    o = ag.head_to_seq_o(boundary, ag.attention_qkv(attend, qkv, lengths=lengths))
    h = h + o.view(B * S, D) @ p["wo"]
    x = ag.layer_norm(norm, h, p["w2"], p["b2"], EPS)
    logits = x @ p["router"]
    live = (torch.arange(S, device="cuda")[None] < lengths[:, None]).reshape(-1)
    scores, ids = torch.topk(logits, K, dim=1)
    balance, counts = ag.balance_loss(experts, logits, ids, live, COEF)
    rows, index = ag.route_to_expert(experts, x, ids)
    ends = index.offsets.tolist()
    out = torch.cat([rows[ends[e]:ends[e + 1]] @ p["experts"][e] for e in range(E)] + [rows[ends[E]:]])
    y = h + ag.expert_to_seq(experts, out, torch.softmax(scores, 1), index)
    return ((y - target) * live[:, None]).square().sum() / 100 + balance.sum(), ids


def plain(p, tokens, lengths, target, ids):
    """The same in 64 bits on the CPU, from the definitions, with the router's choices given."""
    h = p["table"][tokens] * 2.0

    def norm(x, w, c):
        m = x.mean(1, keepdim=True)
        return (x - m) / ((x - m).square().mean(1, keepdim=True) + EPS).sqrt() * w + c

    x = norm(h, p["w1"], p["b1"])
    q, k, v = ((x @ p[n]).view(B, S, -1, D_HEAD).transpose(1, 2) for n in ("wq", "wk", "wv"))
    k, v = (t.repeat_interleave(HQ // HKV, 1) for t in (k, v))
    i, j = torch.arange(S)[:, None], torch.arange(S)[None]
    sees = ((j <= i) & ((i - j < WINDOW) | (j < SINKS)))[None, None] & (i < lengths[:, None, None, None])
    s = (q @ k.transpose(2, 3) * D_HEAD ** -0.5).masked_fill(~sees, -1e300)
    w = torch.softmax(s, 3) * sees
    h = h + (w @ v).transpose(1, 2).reshape(B * S, D) @ p["wo"]
    x = norm(h, p["w2"], p["b2"])
    logits = x @ p["router"]
    live = (j < lengths[:, None]).reshape(-1)
    prob = torch.softmax(logits, 1)
    L = live.sum()
    counts = torch.bincount(ids[live].reshape(-1), minlength=E).double()
    balance = COEF * E * (counts / (K * L) * prob[live].mean(0)).sum()
    weight = torch.softmax(logits.gather(1, ids), 1)
    y = h + sum(weight[:, c:c + 1] * torch.einsum("td,tde->te", x, p["experts"][ids[:, c]]) for c in range(K))
    return ((y - target) * live[:, None]).square().sum() / 100 + balance


def make_plans():
    boundary = b.basp_plan_create_groups(N, B, S, HQ, HKV, D_HEAD, b.BASP_FP32, G)
    embed = b.basp_embed_plan_create(boundary, B * S, V, D, dtype=b.BASP_FP32, grad_dtype=b.BASP_FP32)
    return (boundary, embed, b.basp_norm_plan_create(B * S, D, b.BASP_FP32, b.BASP_FP32),
            b.basp_attention_plan_create(boundary, S, WINDOW, SINKS),
            b.basp_expert_plan_create(B * S, K, E, D, align=4, dtype=b.BASP_FP32, weight_dtype=b.BASP_FP32))


def test_layer_with_gradients():
    """G = B groups: the sequence-sharded order is that of the tokens."""
    g = torch.Generator()
    g.manual_seed(5)
    tokens = torch.randint(0, V, (B * S,), generator=g)
    lengths = torch.tensor([S, 31])
    target = torch.randn(B * S, D, generator=g)
    p = parameters(1)
    dev = {n: t.cuda().requires_grad_() for n, t in p.items()}
    loss, ids = library(dev, tokens.cuda(), lengths.int().cuda(), make_plans(), target.cuda())
    grads = torch.autograd.grad(loss, list(dev.values()))
    exact = {n: t.double().requires_grad_() for n, t in p.items()}
    want = plain(exact, tokens, lengths, target.double(), ids.cpu())
    wants = torch.autograd.grad(want, list(exact.values()))
    # a chain of about ten products and sums of up to 128 terms in fp32, each off
    # by at most 2 * 130 * 2^-24 = 1.6e-5 of its terms and by a tenth of that in the
    # mean square: 2e-5 in 2-norm, five times that is allowed
    assert abs(loss.item() - want.item()) <= 1e-4 * want.item()
    for (n, got), w in zip(zip(dev, grads), wants):
        off = float((got.cpu().double() - w).norm() / w.norm())
        assert off <= 1e-4, (n, off)


def attention_step(dtype=None, seed=0, queries=None):
    """A call of every kernel of the attention, norm and balance loss on buffers of its own."""
    dt = torch.bfloat16
    g = torch.Generator(device="cuda")

    class Step:
        pass
    s = Step()
    layout = b.basp_plan_create_groups(2, 2, 320, 8, 4, 64, b.BASP_BF16, 1)
    s.plan = b.basp_attention_plan_create(layout, 320, 100, 4)
    s.last = b.basp_attention_plan_create(layout, 1, 320, 0)
    s.norm = b.basp_norm_plan_create(640, 512, b.BASP_BF16, b.BASP_FP32)
    s.route = b.basp_expert_plan_create(640, 2, 16, 1, weight_dtype=b.BASP_BF16)
    i, j = s.plan.info, s.last.info
    empty = lambda n, d=dt: torch.empty(n, dtype=d, device="cuda")
    s.q, s.k, s.v, s.do = empty(i["q_elems"]), empty(i["kv_elems"]), empty(i["kv_elems"]), empty(i["q_elems"])
    s.one = empty(j["q_elems"])
    s.lengths = empty(2, torch.int32)
    s.x, s.dy, s.w = empty((640, 512)), empty((640, 512)), empty(512, torch.float32)
    s.logits, s.ids = empty((640, 16)), empty((640, 2), torch.int64)
    f = torch.float32
    s.outputs = dict(o=empty(i["q_elems"]), lse=empty(i["lse_elems"], f), dq=empty(i["q_elems"]), dk=empty(i["kv_elems"]),
                     dv=empty(i["kv_elems"]), last=empty(j["q_elems"]), y=empty((640, 512)), mean=empty(640, f), rstd=empty(640, f),
                     dx=empty((640, 512)), dw=empty(512, f), db=empty(512, f), loss=empty(1, f), counts=empty(16, torch.int32),
                     slope=empty(16, f), dlogits=empty((640, 16)))
    s.ws = [empty(max(1, n), torch.uint8) for n in (i["workspace_bytes"], i["grad_workspace_bytes"], j["workspace_bytes"],
                                                    s.norm.info["workspace_bytes"], s.route.balance_bytes)]

    def fill(seed):
        g.manual_seed(seed)
        for t in (s.q, s.k, s.v, s.do, s.one, s.x, s.dy, s.w, s.logits):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        s.lengths.copy_(torch.randint(200, 321, (2,), generator=g, device="cuda"))
        s.ids.copy_(torch.randint(0, 16, (640, 2), generator=g, device="cuda"))

    def run(stream=None):
        o = s.outputs
        b.basp_attention(s.plan, s.q, s.k, s.v, None, s.lengths, 0.125, o["o"], o["lse"], s.ws[0], stream)
        b.basp_attention_grad(s.plan, s.q, s.k, s.v, o["o"], o["lse"], s.do, None, s.lengths, 0.125, o["dq"], o["dk"], o["dv"],
                              s.ws[1], stream)
        b.basp_attention(s.last, s.one, s.k, s.v, None, s.lengths, 0.125, o["last"], None, s.ws[2], stream)
        b.basp_layer_norm(s.norm, s.x, s.w, None, 1e-5, o["y"], o["mean"], o["rstd"], stream)
        b.basp_layer_norm_grad(s.norm, s.dy, s.x, s.w, o["mean"], o["rstd"], o["dx"], o["dw"], o["db"], s.ws[3], stream)
        b.basp_balance_loss(s.route, s.logits, s.ids, None, 0.1, o["loss"], o["counts"], o["slope"], s.ws[4], stream)
        b.basp_balance_loss_grad(s.route, s.logits, None, o["slope"], o["loss"], o["dlogits"], stream)

    def spoil():
        for t in s.outputs.values():
            t.fill_(-9)

    s.fill, s.run, s.spoil = fill, run, spoil
    return s


def results(s, seed):
    s.fill(seed)
    s.spoil()
    s.run()
    torch.cuda.synchronize()
    return {n: t.clone() for n, t in s.outputs.items()}


def test_graph_replays():
    s, eager = attention_step(), attention_step()
    s.fill(1)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (11, 12, 13):
        want = results(eager, seed)
        s.fill(seed)
        s.spoil()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in s.outputs.items():
            assert torch.equal(t, want[n]), (seed, n)


def test_streams_at_the_same_time():
    """Plans are shared, workspaces are not; and a stream given by its handle."""
    one, two = attention_step(), attention_step()
    want = [results(one, 21), results(two, 22)]
    for n in ("plan", "last", "norm", "route"):
        setattr(two, n, getattr(one, n))
    one.spoil()
    two.spoil()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        one.run(streams[0].cuda_stream)
        with torch.cuda.stream(streams[1]):
            two.run()
    torch.cuda.synchronize()
    for s, w in zip((one, two), want):
        for n, t in s.outputs.items():
            assert torch.equal(t, w[n]), n


def test_backward_in_a_graph():
    """Forward and backward of the autograd wrappers inside one capture, on leaves of its own."""
    plans = make_plans()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    i = plans[3].info
    qkv = torch.randn(i["q_elems"] + 2 * i["kv_elems"], generator=gen, device="cuda").requires_grad_()
    x = torch.randn(B * S, D, generator=gen, device="cuda").requires_grad_()
    w, c = (torch.randn(D, generator=gen, device="cuda").requires_grad_() for _ in range(2))
    logits = torch.randn(B * S, E, generator=gen, device="cuda").requires_grad_()
    ids = torch.randint(0, E, (B * S, K), generator=gen, device="cuda")
    do, dy = torch.randn(i["q_elems"], generator=gen, device="cuda"), torch.randn(B * S, D, generator=gen, device="cuda")

    def step(qkv, x, w, c, logits):
        o = ag.attention_qkv(plans[3], qkv)
        y = ag.layer_norm(plans[2], x, w, c, EPS)
        loss, _ = ag.balance_loss(plans[4], logits, ids)
        return (o.detach(), y.detach(), loss.detach(), *torch.autograd.grad((o, y, loss), (qkv, x, w, c, logits), (do, dy, torch.ones_like(loss))))

    leaves = [qkv, x, w, c, logits]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            step(*leaves)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*leaves)
    for seed in (3, 4, 5):
        gen.manual_seed(seed)
        with torch.no_grad():
            for t in leaves + [do, dy]:
                t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
            ids.copy_(torch.randint(0, E, (B * S, K), generator=gen, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        eager = step(*[t.detach().clone().requires_grad_() for t in leaves])
        torch.cuda.synchronize()
        for n, (a, e) in enumerate(zip(kept, eager)):
            assert torch.equal(a, e), (seed, n)


def test_gradients_are_not_differentiated_again():
    plans = make_plans()
    i = plans[3].info
    qkv = torch.randn(i["q_elems"] + 2 * i["kv_elems"], device="cuda").requires_grad_()
    x, w = torch.randn(B * S, D, device="cuda").requires_grad_(), torch.randn(D, device="cuda").requires_grad_()
    logits = torch.randn(B * S, E, device="cuda").requires_grad_()
    ids = torch.randint(0, E, (B * S, K), device="cuda")
    for out, leaf in ((ag.attention_qkv(plans[3], qkv), qkv), (ag.layer_norm(plans[2], x, w), x), (ag.layer_norm(plans[2], x, w), w),
                      (ag.balance_loss(plans[4], logits, ids)[0], logits)):
        (grad,) = torch.autograd.grad(out.square().sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="not themselves differentiable"):
            torch.autograd.grad(grad.square().sum(), leaf)


def test_separate_q_k_v_agree_with_the_fused_buffer():
    plans = make_plans()
    i = plans[3].info
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    qkv = torch.randn(i["q_elems"] + 2 * i["kv_elems"], generator=g, device="cuda").requires_grad_()
    parts = [t.detach().clone().requires_grad_() for t in qkv.split([i["q_elems"], i["kv_elems"], i["kv_elems"]])]
    lengths = torch.tensor([S, 20], dtype=torch.int32, device="cuda")
    do = torch.randn(i["q_elems"], generator=g, device="cuda")
    one, two = ag.attention_qkv(plans[3], qkv, lengths=lengths), ag.attention(plans[3], *parts, lengths=lengths)
    assert torch.equal(one, two)
    a, = torch.autograd.grad(one, qkv, do)
    assert torch.equal(a, torch.cat(torch.autograd.grad(two, parts, do)))


def test_binding_refuses():
    s = attention_step()
    o = s.outputs
    call = lambda **k: b.basp_attention(*[dict(plan=s.plan, q=s.q, k=s.k, v=s.v, starts=None, lengths=s.lengths, scale=0.1, o=o["o"],
                                               lse=o["lse"], ws=s.ws[0], **{})[n] if n not in k else k[n]
                                          for n in ("plan", "q", "k", "v", "starts", "lengths", "scale", "o", "lse", "ws")])
    call()
    for bad, error in ((dict(q=s.q.float()), TypeError), (dict(k=s.q), ValueError), (dict(v=s.v.cpu()), ValueError),
                       (dict(q=s.q.view(-1, 2).t()), ValueError), (dict(lengths=s.lengths.long()), TypeError),
                       (dict(lengths=s.lengths[:1]), ValueError), (dict(starts=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
                       (dict(lse=o["lse"].half()), TypeError), (dict(q=None), b.BaspError), (dict(o=s.q), b.BaspError),
                       (dict(scale=float("nan")), b.BaspError)):
        with pytest.raises(error):
            call(**bad)
    with pytest.raises(ValueError):
        b.basp_attention(s.last, s.one, s.k, s.v, None, None, 0.1, o["last"], None, s.ws[2][:-1])
    with pytest.raises(ValueError):
        b.basp_attention_grad(s.plan, s.q, s.k, s.v, o["o"], o["lse"], s.do, None, None, 0.1, o["dq"], o["dk"], o["dv"], s.ws[1][:-1])
    with pytest.raises(ValueError):
        b.basp_layer_norm(s.norm, s.x[:-1], s.w, None, 1e-5, o["y"], None, None)
    with pytest.raises(TypeError):
        b.basp_layer_norm(s.norm, s.x, s.w.half(), None, 1e-5, o["y"], None, None)
    with pytest.raises(TypeError):
        b.basp_balance_loss(s.route, s.logits, s.ids, torch.ones(640, device="cuda"), 0.1, o["loss"], o["counts"], o["slope"], s.ws[4])
    with pytest.raises(ValueError):
        b.basp_balance_loss(s.route, s.logits, s.ids, None, 0.1, o["loss"], o["counts"], o["slope"], s.ws[4][:-1])
    with pytest.raises(ValueError):
        b.basp_balance_loss_grad(s.route, s.logits, torch.ones(639, dtype=torch.bool, device="cuda"), o["slope"], o["loss"], o["dlogits"])


def test_timed_calls():
    s = attention_step()
    s.fill(1)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in events:
        e.record()
    o = s.outputs
    for call in (lambda: b.basp_attention(s.plan, s.q, s.k, s.v, None, None, 0.1, o["o"], o["lse"], s.ws[0]),
                 lambda: b.basp_attention_grad(s.plan, s.q, s.k, s.v, o["o"], o["lse"], s.do, None, None, 0.1, o["dq"], o["dk"], o["dv"], s.ws[1]),
                 lambda: b.basp_attention(s.last, s.one, s.k, s.v, None, None, 0.1, o["last"], None, s.ws[2]),
                 lambda: b.basp_layer_norm(s.norm, s.x, s.w, None, 1e-5, o["y"], o["mean"], o["rstd"]),
                 lambda: b.basp_layer_norm_grad(s.norm, s.dy, s.x, s.w, o["mean"], o["rstd"], o["dx"], o["dw"], o["db"], s.ws[3]),
                 lambda: b.basp_balance_loss(s.route, s.logits, s.ids, None, 0.1, o["loss"], o["counts"], o["slope"], s.ws[4]),
                 lambda: b.basp_balance_loss_grad(s.route, s.logits, None, o["slope"], o["loss"], o["dlogits"])):
        call()
        torch.cuda.synchronize()
        b.basp_time_next_call(*events)
        call()
        torch.cuda.synchronize()
        assert 0.0 < events[0].elapsed_time(events[1]) < 100.0
