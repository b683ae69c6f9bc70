"""The autograd wrappers' gradients are not themselves differentiable: a loss
with a gradient in it is refused, and not differentiated as if that gradient
were a constant (MI355X only)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sequence_re_layout_amd import autograd as ag
    from sequence_re_layout_amd import binding as b
else:  # collected on a machine without a GPU: every test here is skipped
    ag = b = None

T, K, E, D, V = 48, 3, 5, 24, 31


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def experts():
    """The calls on experts as functions of the tensors that need gradients."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    plan = b.basp_expert_plan_create(T, K, E, D, align=4, dtype=b.BASP_FP32)
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda")
    index = ag.sort_by_expert(plan, ids)
    table = b.basp_embed_plan_create(None, T, V, D, dtype=b.BASP_FP32, grad_dtype=b.BASP_FP32)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").requires_grad_()
    x, w, rows, emb = normal(T, D), normal(T, K), normal(plan.info["max_rows"], D), normal(V, D)
    return {
        "sums, of rows": (lambda: ag.expert_to_seq(plan, rows, w, index), rows, (rows, w)),
        "sums, of weights": (lambda: ag.expert_to_seq(plan, rows, w, index), w, (rows, w)),
        "routed and back": (lambda: ag.expert_to_seq(plan, ag.route_to_expert(plan, x, ids)[0], w, index), x, (x, w)),
        "squared rows": (lambda: ag.seq_to_expert(plan, x, index) ** 2, x, (x,)),
        "squared embedding": (lambda: ag.embed_to_seq(table, tokens, emb, 2.0) ** 2, emb, (emb,)),
    }


@pytest.mark.parametrize("what", ["sums, of rows", "sums, of weights", "routed and back", "squared rows",
                                  "squared embedding"])
def test_a_gradient_in_the_loss_of_the_experts(what):
    f, of, leaves = experts()[what]
    want = torch.autograd.grad(f().sum(), of)[0]
    y = f()
    (grad,) = torch.autograd.grad(y.sum(), of, create_graph=True)
    assert torch.equal(grad, want)
    with pytest.raises(RuntimeError, match="differentia"):
        torch.autograd.grad(y.sum() + (grad * grad).sum(), leaves)
    # the loss without it is as it was
    assert torch.equal(torch.autograd.grad(f().sum(), of, create_graph=True)[0], want)


@pytest.mark.parametrize("what", ["qkv, of q", "qkv, of k", "qkv, of v", "output"])
def test_a_gradient_in_the_loss_of_the_boundary(what):
    plan = b.basp_plan_create(2, 2, 8, 4, 2, 16, b.BASP_FP32, b.BASP_MODE_ULYSSES)
    i = plan.info
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    q, k, v, o = (torch.randn(n, generator=g, device="cuda").requires_grad_()
                  for n in (i["q_elems"], i["kv_elems"], i["kv_elems"], i["q_elems"]))
    of = {"qkv, of q": q, "qkv, of k": k, "qkv, of v": v, "output": o}[what]
    f = (lambda: ag.head_to_seq_o(plan, o) ** 3) if what == "output" else (lambda: ag.seq_to_head_qkv(plan, q, k, v) ** 3)
    leaves = (o,) if what == "output" else (q, k, v)
    want = torch.autograd.grad(f().sum(), of)[0]
    assert torch.allclose(want, 3 * of.detach() ** 2, rtol=8 * 2.0 ** -24, atol=0)   # two roundings a side
    y = f()
    (grad,) = torch.autograd.grad(y.sum(), of, create_graph=True)
    assert torch.equal(grad, want)
    with pytest.raises(RuntimeError, match="differentia"):
        torch.autograd.grad(y.sum() + (grad * grad).sum(), leaves)
