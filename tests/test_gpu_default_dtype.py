"""The autograd wrappers under another default type of torch (MI355X only)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sequence_re_layout_amd import autograd as ag
    from sequence_re_layout_amd import binding as b
else:  # collected on a machine without a GPU: every test here is skipped
    ag = b = None

F32 = torch.float32


@pytest.fixture(params=[torch.float16, torch.bfloat16, torch.float64])
def default(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield
    torch.set_default_dtype(before)


def leaf(*shape):
    return torch.randn(*shape, dtype=F32, device="cuda").requires_grad_()


def layout():
    return b.basp_plan_create_groups(2, 1, 64, 4, 2, 16, b.BASP_FP32, 1)


def test_balance_loss(default):
    plan = b.basp_expert_plan_create(50, 2, 8, 1, weight_dtype=b.BASP_FP32)
    logits, ids = leaf(50, 8), torch.randint(0, 8, (50, 2), device="cuda")
    loss, counts = ag.balance_loss(plan, logits, ids, coef=0.5)
    loss.sum().backward()
    assert loss.dtype is F32 and counts.dtype is torch.int32 and logits.grad.dtype is F32
    f = torch.bincount(ids.reshape(-1), minlength=8).double() * 8 / 100
    want = 0.5 * (f * torch.softmax(logits.detach().double(), 1).mean(0)).sum()
    # sums of 50 and of 8 products in fp32, at most 2 * 60 steps of 2^-24
    assert abs(loss.item() - want.item()) <= 120 * 2.0 ** -24 * want.item()


def test_attention_and_norm(default):
    boundary = layout()
    plan = b.basp_attention_plan_create(boundary, 64, 20, 2)
    qkv = leaf(boundary.info["qkv_elems"])
    ag.attention_qkv(plan, qkv).square().sum().backward()
    norm = b.basp_norm_plan_create(64, 32, b.BASP_FP32, b.BASP_FP32)
    x, w, c = leaf(64, 32), leaf(32), leaf(32)
    ag.layer_norm(norm, x, w, c).square().sum().backward()
    for t in (qkv, x, w, c):
        assert t.grad.dtype is F32 and bool(torch.isfinite(t.grad).all())


def test_re_layouts(default):
    boundary = layout()
    i = boundary.info
    q, k, v = leaf(i["q_elems"]), leaf(i["kv_elems"]), leaf(i["kv_elems"])
    ag.seq_to_head_qkv(boundary, q, k, v).square().sum().backward()
    experts = b.basp_expert_plan_create(64, 2, 4, 32, dtype=b.BASP_FP32, weight_dtype=b.BASP_FP32)
    x, weights, ids = leaf(64, 32), leaf(64, 2), torch.randint(0, 4, (64, 2), device="cuda")
    rows, index = ag.route_to_expert(experts, x, ids)
    ag.expert_to_seq(experts, rows, weights, index).square().sum().backward()
    embed = b.basp_embed_plan_create(boundary, 64, 100, 32, dtype=b.BASP_FP32, grad_dtype=b.BASP_FP32)
    table = leaf(100, 32)
    ag.embed_to_seq(embed, torch.randint(0, 100, (64,), device="cuda"), table).square().sum().backward()
    for t in (q, k, v, x, weights, table):
        assert t.grad.dtype is F32 and bool(torch.isfinite(t.grad).all())
