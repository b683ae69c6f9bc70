"""Layer norm and the balance loss on the GPU against plain forms in 64 bits
(MI355X only)."""
import numpy as np
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


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def code(name):
    return {"bf16": b.BASP_BF16, "fp16": b.BASP_FP16, "fp32": b.BASP_FP32}[name]


def values(g, shape, dtype, size=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g) * size + mean).to(lc.FLOATS[dtype]).double()


NORMS = [  # T, D, dtype, weights, bias, mean of the rows, shift of the buffers
    (1, 1, "fp32", "fp32", True, 0.0, 0),
    (1, 2, "bf16", "bf16", True, 0.0, 0),
    (3, 3, "fp16", "fp32", False, 1.0, 1),
    (17, 7, "bf16", "fp32", True, 0.0, 1),
    (70, 8, "bf16", "bf16", True, 0.0, 0),
    (33, 31, "fp32", "bf16", True, 3.0, 1),
    (5, 100, "fp16", "fp16", True, 0.0, 0),
    (129, 130, "bf16", "fp32", True, 0.5, 1),
    (300, 500, "fp32", "fp32", True, 0.0, 0),
    (64, 512, "bf16", "fp32", False, 0.0, 0),
    (77, 777, "fp32", "fp32", True, 10.0, 1),
    (1030, 1000, "bf16", "fp32", True, 0.0, 3),
    (2049, 1024, "fp16", "fp32", True, 0.0, 0),
    (50, 1025, "fp32", "fp32", False, 0.0, 0),
    (9, 2048, "bf16", "bf16", True, 0.0, 0),
    (600, 2050, "bf16", "fp32", True, 0.0, 1),
    (4, 4095, "fp32", "fp32", True, 0.0, 0),
    (11, 4100, "bf16", "fp32", True, 0.0, 0),
    (5, 8200, "fp16", "fp32", True, 0.0, 0),
    (3, 8193, "fp32", "fp32", True, 0.0, 1),
    (3, 16400, "bf16", "fp32", True, 0.0, 0),
    (2, 40001, "fp32", "bf16", True, 1.0, 0),
    (5000, 16, "bf16", "fp32", True, 0.0, 0),
    (1100, 4200, "bf16", "fp32", True, 0.0, 0),
    (530, 5001, "fp32", "fp32", True, 0.0, 1),
    (520, 9000, "fp16", "fp16", False, 0.0, 0),
    (300, 12000, "fp32", "bf16", True, 1.0, 0),
]


@pytest.mark.parametrize("T,D,dtype,wdtype,has_bias,mean,shift", NORMS)
def test_norm(T, D, dtype, wdtype, has_bias, mean, shift):
    g = torch.Generator()
    g.manual_seed(T + D)
    x = values(g, (T, D), dtype, 2.0, mean)
    w, bias = values(g, (D,), wdtype, 0.3, 1.0), values(g, (D,), wdtype)
    dy = values(g, (T, D), dtype)
    eps, dt, wt = 1e-5, lc.FLOATS[dtype], lc.FLOATS[wdtype]
    plan = b.basp_norm_plan_create(T, D, code(dtype), code(wdtype))
    put = lambda t, d: ic.shifted(t.to(d).cuda(), shift)
    xd, dyd, wd, bd = put(x, dt), put(dy, dt), put(w, wt), put(bias, wt) if has_bias else None
    out = lambda n, d, s=shift: ic.Guarded(n, d, NAN, s)
    y, mu, rs = out(T * D, dt), out(T, torch.float32, 0), out(T, torch.float32, 0)
    b.basp_layer_norm(plan, xd, wd, bd, eps, y.t, mu.t, rs.t)
    bias_e = bias if has_bias else None
    want = lc.norm_exact(x, w, bias_e, eps)
    errs = lc.norm_errors(x, w, bias_e, eps)
    torch.cuda.synchronize()
    for got, e, err, name in zip((y, mu, rs), want, errs, ("y", "mean", "rstd")):
        got.check(name)
        lc.check(got.t, e, err, name)
    only = out(T * D, dt)
    b.basp_layer_norm(plan, xd, wd, bd, eps, only.t, None, None)
    assert torch.equal(only.t, y.t)

    dx, dw, db = out(T * D, dt), out(D, wt), out(D, wt)
    ws = torch.full((max(1, plan.info["workspace_bytes"]),), 255, dtype=torch.uint8, device="cuda")
    b.basp_layer_norm_grad(plan, dyd, xd, wd, mu.t, rs.t, dx.t, dw.t, db.t if has_bias else None, ws)
    torch.cuda.synchronize()
    grads = lc.norm_grad_exact(dy, x, w, mu.t.cpu().double(), rs.t.cpu().double())
    for got, (e, err), name in zip((dx, dw, db), grads, ("dx", "dweight", "dbias")):
        got.check(name)
        if name != "dbias" or has_bias:
            lc.check(got.t, e, err, name)
    again = [t.t.clone() for t in (dx, dw)]
    ws.fill_(0)
    b.basp_layer_norm_grad(plan, dyd, xd, wd, mu.t, rs.t, dx.t, dw.t, None, ws)
    assert torch.equal(dx.t, again[0]) and torch.equal(dw.t, again[1])


def test_norm_of_no_rows():
    plan = b.basp_norm_plan_create(0, 100, b.BASP_BF16, b.BASP_FP32)
    w = torch.ones(100, device="cuda")
    b.basp_layer_norm(plan, None, w, None, 1e-5, None, None, None)
    dw, db = torch.full_like(w, 7), torch.full_like(w, 7)
    b.basp_layer_norm_grad(plan, None, None, w, None, None, None, dw, db, None)
    assert float(dw.abs().max()) == 0 and float(db.abs().max()) == 0


def test_norm_of_bad_rows_stays_in_them():
    """NaN and infinities of one row reach no other row's results."""
    T, D = 40, 300
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(T, D, generator=g, device="cuda")
    w = torch.ones(D, device="cuda")
    plan = b.basp_norm_plan_create(T, D, b.BASP_FP32, b.BASP_FP32)
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    b.basp_layer_norm(plan, x, w, None, 1e-5, y0, None, None)
    x[7, 3], x[9] = NAN, float("inf")
    b.basp_layer_norm(plan, x, w, None, 1e-5, y1, None, None)
    rest = [t for t in range(T) if t not in (7, 9)]
    assert torch.equal(y0[rest], y1[rest]) and bool(torch.isnan(y1[7]).all()) and bool(torch.isnan(y1[9]).all())


def test_norm_of_equal_numbers():
    """No variance: 1 / sqrt(eps), and with eps 0 whatever the division gives, of that row only."""
    x = torch.full((2, 64), 3.0, device="cuda")
    x[1] += torch.arange(64, device="cuda")
    w = torch.ones(64, device="cuda")
    plan = b.basp_norm_plan_create(2, 64, b.BASP_FP32, b.BASP_FP32)
    y, rstd = torch.empty_like(x), torch.empty(2, device="cuda")
    b.basp_layer_norm(plan, x, w, None, 1e-4, y, None, rstd)
    assert float(y[0].abs().max()) == 0 and abs(float(rstd[0]) - 100) < 1e-3
    b.basp_layer_norm(plan, x, w, None, 0.0, y, None, rstd)
    assert not bool(torch.isfinite(rstd[0])) and bool(torch.isfinite(y[1]).all())


def test_norm_gradient_against_differences():
    T, D, eps = 5, 60, 1e-5
    g = torch.Generator()
    g.manual_seed(2)
    x, w, bias, dy = (values(g, s, "fp32") for s in ((T, D), (D,), (D,), (T, D)))
    plan = b.basp_norm_plan_create(T, D, b.BASP_FP32, b.BASP_FP32)
    dev = [t.float().cuda() for t in (x, w, bias, dy)]
    y, mean, rstd = torch.empty_like(dev[0]), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    b.basp_layer_norm(plan, *dev[:3], eps, y, mean, rstd)
    dx, dw, db = (torch.empty_like(t) for t in dev[:3])
    ws = torch.empty(plan.info["workspace_bytes"], dtype=torch.uint8, device="cuda")
    b.basp_layer_norm_grad(plan, dev[3], dev[0], dev[1], mean, rstd, dx, dw, db, ws)
    for i, got in enumerate((dx, dw, db)):
        way = torch.randn(got.shape, generator=g, dtype=torch.float64)
        args = [[t for t in (x, w, bias)] for _ in range(2)]
        args[0][i], args[1][i] = args[0][i] + 1e-5 * way, args[1][i] - 1e-5 * way
        up, down = ((lc.norm_exact(*a, eps)[0] * dy).sum() for a in args)
        terms = (got.cpu().double() * way).abs().sum()
        # differences are off by step^2, the gradient by some 100 * 2^-24 of its terms
        assert abs((got.cpu().double() * way).sum() - (up - down) / 2e-5) <= 2e-5 * terms


BALANCES = [  # T, K, E, dtype, id_bytes, share masked, share of ids outside
    (1, 1, 1, "fp32", 8, 0.0, 0.0),
    (1, 2, 4, "bf16", 4, 0.0, 0.0),
    (5, 1, 3, "fp16", 8, 0.5, 0.0),
    (50, 2, 2, "bf16", 8, 0.0, 0.3),
    (64, 4, 7, "fp32", 4, 0.2, 0.1),
    (100, 8, 8, "fp16", 8, 0.0, 0.0),
    (257, 3, 33, "bf16", 4, 0.3, 0.2),
    (300, 2, 64, "fp32", 8, 0.0, 0.0),
    (1000, 6, 129, "fp32", 8, 0.1, 0.1),
    (700, 2, 257, "fp16", 4, 0.0, 0.0),
    (513, 3, 320, "bf16", 8, 0.2, 0.0),
    (260, 2, 1000, "bf16", 8, 0.0, 0.1),
    (300, 5, 1023, "fp32", 4, 0.1, 0.0),
    (90, 1, 1024, "fp32", 8, 0.0, 0.0),
    (20000, 2, 16, "fp32", 8, 0.1, 0.0),
    (9000, 4, 513, "fp16", 4, 0.1, 0.1),
    (400, 2, 408, "bf16", 8, 0.1, 0.0),
    (400, 3, 700, "fp32", 8, 0.0, 0.1),
    (3000, 2, 128, "fp32", 4, 0.1, 0.0),
    (70, 2, 96, "fp32", 8, 0.1, 0.0),
    (2, 2, 1000, "fp16", 8, 0.0, 0.0),
]


@pytest.mark.parametrize("T,K,E,dtype,id_bytes,masked,gone", BALANCES)
def test_balance(T, K, E, dtype, id_bytes, masked, gone):
    rng = np.random.default_rng(T + E)
    g = torch.Generator()
    g.manual_seed(T + E)
    logits = values(g, (T, E), dtype, 2.0)
    ids = ic.choices(rng, T, K, E, gone, id_bytes)
    live = rng.random(T) >= masked
    coef, dt = 0.37, lc.FLOATS[dtype]
    if masked:                                         # what a masked token's scores are does not count
        logits[~torch.from_numpy(live)] = NAN
    for shift, mask in ((0, torch.from_numpy(live)), (1, torch.from_numpy(live.astype(np.uint8) * 200))):
        plan = b.basp_expert_plan_create(T, K, E, 1, id_bytes=id_bytes, weight_dtype=code(dtype))
        x = ic.shifted(logits.to(dt).cuda(), shift)
        idd = torch.from_numpy(ids).to(torch.int64 if id_bytes == 8 else torch.int32).cuda()
        mask_d = mask.cuda() if masked else None
        f32 = torch.float32
        loss, slope, counts = ic.Guarded(1, f32, NAN), ic.Guarded(E, f32, NAN), ic.Guarded(E, torch.int32, -7)
        dlogits = ic.Guarded(T * E, dt, NAN, shift)
        ws = torch.full((plan.balance_bytes,), 255, dtype=torch.uint8, device="cuda")
        b.basp_balance_loss(plan, x, idd, mask_d, coef, loss.t, counts.t, slope.t, ws)
        dloss = torch.tensor([1.7], device="cuda")
        b.basp_balance_loss_grad(plan, x, mask_d, slope.t, dloss, dlogits.t)
        torch.cuda.synchronize()
        for t, name in ((loss, "loss"), (slope, "slope"), (counts, "counts"), (dlogits, "dlogits")):
            t.check(name)
        want, n, s, p = lc.balance_exact(logits, ids, live, coef, E)
        assert np.array_equal(counts.t.cpu().numpy(), n)
        U = lc.U
        lc.check(slope.t, s, 8 * U * s, "slope")
        # a probability is off by the rounding of its exponent, about |x - max| u, a step of the power of two, and its row's sum
        wide = torch.where(torch.isfinite(logits), logits, torch.zeros_like(logits))
        r = 2 * (wide.amax(1) - wide.amin(1) + E + 8)[:, None] * U
        lc.check(loss.t, want.reshape(1), ((s * (p * r).sum(0)).sum() + 2 * (T + E + 4) * U * want).reshape(1), "loss")
        dot = (p * s).sum(1, keepdim=True)
        grad = 1.7 * p * (s - dot)
        err = 1.7 * p * (r * ((s - dot).abs() + 2 * dot) + 2 * (E + 8) * U * (s + dot))
        assert lc.check(dlogits.t, grad, err, "dlogits") is None


def test_balance_with_nothing_alive():
    plan = b.basp_expert_plan_create(10, 2, 6, 1, weight_dtype=b.BASP_FP32)
    x = torch.full((10, 6), NAN, device="cuda")
    ids = torch.zeros(10, 2, dtype=torch.int64, device="cuda")
    mask = torch.zeros(10, dtype=torch.bool, device="cuda")
    out = [torch.full((n,), 5.0, device="cuda") for n in (1, 6)] + [torch.full((6,), 5, dtype=torch.int32, device="cuda")]
    ws = torch.empty(plan.balance_bytes, dtype=torch.uint8, device="cuda")
    b.basp_balance_loss(plan, x, ids, mask, 1.0, out[0], out[2], out[1], ws)
    d = torch.full_like(x, 5.0)
    b.basp_balance_loss_grad(plan, x, mask, out[1], torch.ones(1, device="cuda"), d)
    assert all(float(t.float().abs().max()) == 0 for t in out + [d])
    empty = b.basp_expert_plan_create(0, 2, 6, 1)
    for t in out:
        t.fill_(5)
    b.basp_balance_loss(empty, None, None, None, 1.0, out[0], out[2], out[1],
                        torch.empty(empty.balance_bytes, dtype=torch.uint8, device="cuda"))
    b.basp_balance_loss_grad(empty, None, None, out[1], torch.ones(1, device="cuda"), None)
    assert all(float(t.float().abs().max()) == 0 for t in out)


def test_balance_of_banned_experts():
    """Scores of -infinity and of the type's lowest value: no probability, no gradient, nothing else disturbed."""
    T, E = 30, 12
    for dt, low in ((torch.float32, -float("inf")), (torch.bfloat16, torch.finfo(torch.bfloat16).min),
                    (torch.float16, torch.finfo(torch.float16).min)):
        plan = b.basp_expert_plan_create(T, 1, E, 1, weight_dtype={torch.float32: b.BASP_FP32, torch.bfloat16: b.BASP_BF16,
                                                                   torch.float16: b.BASP_FP16}[dt])
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        x = torch.randn(T, E, generator=g, device="cuda").to(dt)
        x[:, 4:7] = low
        ids = x.float().argmax(1, keepdim=True)
        loss, slope = torch.empty(1, device="cuda"), torch.empty(E, device="cuda")
        counts = torch.empty(E, dtype=torch.int32, device="cuda")
        ws = torch.empty(plan.balance_bytes, dtype=torch.uint8, device="cuda")
        b.basp_balance_loss(plan, x, ids, None, 1.0, loss, counts, slope, ws)
        d = torch.empty_like(x)
        b.basp_balance_loss_grad(plan, x, None, slope, torch.ones(1, device="cuda"), d)
        p = torch.softmax(x.double(), 1)
        assert float(d[:, 4:7].float().abs().max()) == 0 and bool(torch.isfinite(d.float()).all())
        assert abs(float(loss) - float((slope.double() * p.sum(0)).sum())) <= 1e-5 * float(loss)


def test_balance_counts_are_those_of_the_sort():
    T, K, E = 5000, 3, 40
    ids = torch.from_numpy(ic.choices(np.random.default_rng(1), T, K, E, 0.2)).cuda()
    plan = b.basp_expert_plan_create(T, K, E, 1, weight_dtype=b.BASP_FP32)
    pos, order = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (T * K, plan.info["max_rows"]))
    offsets, counts, mine = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, E, E))
    ws = torch.empty(max(plan.balance_bytes, plan.info["workspace_bytes"]), dtype=torch.uint8, device="cuda")
    b.basp_expert_sort(plan, ids, pos, order, offsets, counts, ws)
    b.basp_balance_loss(plan, torch.zeros(T, E, device="cuda"), ids, None, 1.0, torch.empty(1, device="cuda"), mine,
                        torch.empty(E, device="cuda"), ws)
    assert torch.equal(counts, mine)


def test_balance_same_bits_every_time():
    """Work-groups that finish in any order, on a workspace that holds anything."""
    T, K, E = 9000, 4, 700
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn(T, E, generator=g, device="cuda")
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda")
    plan = b.basp_expert_plan_create(T, K, E, 1, weight_dtype=b.BASP_FP32)
    first = None
    for fill in range(0, 256, 15):
        ws = torch.full((plan.balance_bytes,), fill, dtype=torch.uint8, device="cuda")
        loss, slope = torch.empty(1, device="cuda"), torch.empty(E, device="cuda")
        counts = torch.empty(E, dtype=torch.int32, device="cuda")
        b.basp_balance_loss(plan, x, ids, None, 1.0, loss, counts, slope, ws)
        out = [t.clone() for t in (loss, slope, counts)]
        first = first or out
        assert all(torch.equal(a, c) for a, c in zip(first, out))
