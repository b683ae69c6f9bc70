"""Tokens sorted by expert and back on the GPU, against plain forms in 64 bits
(MI355X only)."""
import numpy as np
import pytest
import torch

from tests import index_cases as ic

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


class Routing:
    """A plan, a routing of its tokens and the exact index."""

    def __init__(self, T, K, E, D, align=1, dtype="bf16", wdtype="fp32", id_bytes=8, drop=0.0, seed=0, ids=None):
        self.T, self.K, self.E, self.D, self.dt, self.wdt = T, K, E, D, ic.FLOATS[dtype], ic.FLOATS[wdtype]
        self.rng = np.random.default_rng(seed)
        self.ids = ic.choices(self.rng, T, K, E, drop, id_bytes) if ids is None else np.asarray(ids).reshape(T, K)
        self.plan = b.basp_expert_plan_create(T, K, E, D, align, id_bytes, code(dtype), code(wdtype))
        self.rows = self.plan.info["max_rows"]
        assert self.rows == ic.max_rows(T, K, E, align)
        self.pos, self.order, self.offsets, self.counts = ic.index(self.ids, E, align)
        self.ids_d = torch.from_numpy(self.ids).to(torch.int64 if id_bytes == 8 else torch.int32).cuda()
        self.ws = torch.full((max(1, self.plan.info["workspace_bytes"]),), 255, dtype=torch.uint8, device="cuda")
        self.index_d = [torch.from_numpy(v).to(torch.int32).cuda() for v in (self.pos, self.order)]

    def normal(self, *shape, dtype=None):
        return torch.from_numpy(self.rng.standard_normal(shape).astype(np.float32)).to(dtype or self.dt).cuda()

    def out_index(self):
        return [ic.Guarded(n, torch.int32, -7) for n in (self.pos.size, self.rows, self.E + 1, self.E)]

    def check_index(self, got):
        torch.cuda.synchronize()
        for g, want, what in zip(got, (self.pos, self.order, self.offsets, self.counts),
                                 ("pos", "order", "offsets", "counts")):
            assert np.array_equal(g.t.cpu().numpy(), want), what
            g.check(what)

    def slots(self, per_row):
        """Rows of the slots [T*K][...] in 64 bits, zeros for dropped ones."""
        v = np.where((self.pos >= 0)[:, None], per_row[np.maximum(self.pos, 0)] if per_row.size else 0.0, 0.0)
        return v.reshape(self.T, self.K, self.D)


SIZES = [  # T, K, E, D, align, dtype, weights, id_bytes, drop
    (1, 1, 1, 1, 1, "bf16", "fp32", 8, 0.0),
    (1, 2, 4, 7, 1, "fp16", "fp16", 4, 0.0),
    (3, 3, 5, 9, 2, "fp32", "fp32", 8, 0.5),
    (16, 4, 64, 2048, 1, "bf16", "fp32", 8, 0.0),
    (16, 8, 128, 256, 16, "bf16", "bf16", 8, 0.0),
    (33, 2, 7, 3, 4, "bf16", "fp32", 4, 0.3),
    (65, 5, 1024, 65, 1, "fp16", "fp32", 8, 0.2),
    (129, 9, 33, 513, 8, "bf16", "fp32", 8, 0.1),
    (200, 17, 20, 31, 1, "fp32", "bf16", 4, 0.1),
    (255, 1, 3, 100, 128, "fp16", "fp16", 8, 0.9),
    (511, 4, 64, 1000, 1, "fp16", "fp32", 4, 0.0),
    (700, 3, 1000, 24, 3, "fp32", "fp32", 8, 0.1),
    (1023, 5, 40, 777, 4, "fp32", "fp32", 4, 0.2),
    (512, 4, 512, 40, 5, "bf16", "fp32", 8, 0.1),
    (683, 3, 77, 40, 128, "bf16", "fp32", 4, 0.0),
    (2049, 2, 8, 520, 1, "bf16", "fp32", 8, 0.0),
    (4099, 3, 20, 1001, 16, "bf16", "fp32", 8, 0.1),
    (5000, 8, 256, 8, 1, "bf16", "fp32", 4, 0.0),
    (600, 2, 16, 9001, 1, "bf16", "fp32", 8, 0.05),
]
IDS = ["x".join(map(str, s)) for s in SIZES]


@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_sort(size):
    r = Routing(*size)
    got = r.out_index()
    b.basp_expert_sort(r.plan, r.ids_d, *[g.t for g in got], r.ws)
    r.check_index(got)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_seq_to_expert(size, shift):
    """The move alone and the sort with the move, bit for bit."""
    r = Routing(*size)
    x = r.normal(r.T, r.D)
    want = torch.zeros(r.rows, r.D, dtype=r.dt)
    has = r.order >= 0
    want[torch.from_numpy(has)] = x.cpu()[torch.from_numpy(r.order[has] // r.K)]
    xs = ic.shifted(x, shift)
    out = ic.Guarded(r.rows * r.D, r.dt, NAN, shift)
    b.basp_seq_to_expert(r.plan, xs, r.index_d[0], r.index_d[1], out.t)
    torch.cuda.synchronize()
    assert torch.equal(out.t.cpu().view(r.rows, r.D), want)
    out.check("rows")
    out = ic.Guarded(r.rows * r.D, r.dt, NAN, shift)
    got = r.out_index()
    b.basp_route_to_expert(r.plan, xs, r.ids_d, *[g.t for g in got], out.t, r.ws)
    r.check_index(got)
    assert torch.equal(out.t.cpu().view(r.rows, r.D), want)
    out.check("rows of the combined call")


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_sums(size, shift):
    """expert -> seq, and the gradient of seq -> expert; rows without a slot
    hold NaN and the weights of dropped slots infinities."""
    r = Routing(*size)
    rows = r.normal(r.rows, r.D)
    rows[torch.from_numpy(r.order < 0).cuda()] = NAN
    w = r.normal(r.T * r.K, dtype=r.wdt)
    w[torch.from_numpy(r.pos < 0).cuda()] = float("inf")
    terms = r.slots(rows.double().cpu().numpy())
    weights = np.where(r.pos < 0, 0.0, w.double().cpu().numpy()).reshape(r.T, r.K, 1)
    rs, ws = ic.shifted(rows, shift), ic.shifted(w, shift)
    out = ic.Guarded(r.T * r.D, r.dt, NAN, shift)
    b.basp_expert_to_seq(r.plan, rs, r.index_d[0], ws, out.t)
    torch.cuda.synchronize()
    ic.check(out.t, (terms * weights).sum(1), np.abs(terms * weights).sum(1), r.K, "expert -> seq")
    out.check("out")
    dx = ic.Guarded(r.T * r.D, r.dt, NAN, shift)
    b.basp_seq_to_expert_grad(r.plan, rs, r.index_d[0], dx.t)
    torch.cuda.synchronize()
    ic.check(dx.t, terms.sum(1), np.abs(terms).sum(1), r.K, "gradient of seq -> expert")
    dx.check("dx")


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_expert_to_seq_grad(size, shift):
    r = Routing(*size)
    rows, dout = r.normal(r.rows, r.D), r.normal(r.T, r.D)
    rows[torch.from_numpy(r.order < 0).cuda()] = NAN
    w = r.normal(r.T * r.K, dtype=r.wdt)
    w[torch.from_numpy(r.pos < 0).cuda()] = NAN
    g = dout.double().cpu().numpy()
    prod = r.slots(rows.double().cpu().numpy()) * g[:, None, :]
    has = r.order >= 0
    want = np.zeros((r.rows, r.D))
    want[has] = w.double().cpu().numpy()[r.order[has], None] * g[r.order[has] // r.K]
    drows = ic.Guarded(r.rows * r.D, r.dt, NAN, shift)
    dw = ic.Guarded(r.T * r.K, r.wdt, NAN, shift)
    b.basp_expert_to_seq_grad(r.plan, ic.shifted(dout, shift), ic.shifted(rows, shift), r.index_d[0], r.index_d[1],
                              ic.shifted(w, shift), drows.t, dw.t)
    torch.cuda.synchronize()
    ic.check(drows.t, want, np.abs(want), 1, "drows")
    ic.check(dw.t, prod.sum(2).reshape(-1), np.abs(prod).sum(2).reshape(-1), r.D, "dweights")
    drows.check("drows")
    dw.check("dweights")


@pytest.mark.parametrize("ids", [[[-1, 9]] * 5, [[2, 2]] * 5, [[0, 0], [7, 7], [0, 7], [8, 0], [-5, 7]]],
                         ids=["all dropped", "one expert twice", "ends"])
@pytest.mark.parametrize("align", [1, 4])
def test_odd_routings(ids, align):
    r = Routing(5, 2, 8, 40, align, "fp32", ids=np.array(ids))
    x, rows, w = r.normal(5, 40), r.normal(r.rows, 40), r.normal(10, dtype=torch.float32)
    got, out = r.out_index(), ic.Guarded(r.rows * 40, r.dt, NAN)
    b.basp_route_to_expert(r.plan, x, r.ids_d, *[g.t for g in got], out.t, r.ws)
    r.check_index(got)
    want = np.where((r.order >= 0)[:, None], x.double().cpu().numpy()[np.maximum(r.order, 0) // 2], 0.0)
    assert np.array_equal(out.t.double().cpu().numpy().reshape(want.shape), want)
    y = ic.Guarded(200, r.dt, NAN)
    b.basp_expert_to_seq(r.plan, rows, got[0].t, w, y.t)
    t = r.slots(rows.double().cpu().numpy()) * w.double().cpu().numpy().reshape(5, 2, 1)
    ic.check(y.t, t.sum(1), np.abs(t).sum(1), 2, "expert -> seq")


def test_no_tokens():
    r = Routing(0, 2, 8, 16, 4)
    got, out = r.out_index(), ic.Guarded(0, r.dt, NAN)
    b.basp_route_to_expert(r.plan, out.t, r.ids_d, *[g.t for g in got], out.t, None)
    r.check_index(got)
    b.basp_expert_to_seq(r.plan, out.t, got[0].t, out.t.float(), out.t)
    b.basp_expert_to_seq_grad(r.plan, out.t, out.t, got[0].t, got[1].t, out.t.float(), out.t, out.t.float())
    b.basp_seq_to_expert_grad(r.plan, out.t, got[0].t, out.t)
    torch.cuda.synchronize()
    out.check("rows")


def test_damaged_index_stays_inside():
    """Entries of pos and order outside their range count as -1."""
    r = Routing(40, 2, 4, 72, 8, "bf16")
    pos, order = r.index_d[0].clone(), r.index_d[1].clone()
    pos[3], pos[5], order[1] = r.rows, 2**31 - 1, 80
    order[r.pos[3]] = order[r.pos[5]] = -1
    x, rows, w = r.normal(40, 72), r.normal(r.rows, 72), r.normal(80, dtype=torch.float32)
    out, y = ic.Guarded(r.rows * 72, r.dt, NAN), ic.Guarded(40 * 72, r.dt, NAN)
    drows, dw = ic.Guarded(r.rows * 72, r.dt, NAN), ic.Guarded(80, torch.float32, NAN)
    b.basp_seq_to_expert(r.plan, x, pos, order, out.t)
    b.basp_expert_to_seq(r.plan, rows, pos, w, y.t)
    b.basp_expert_to_seq_grad(r.plan, x, rows, pos, order, w, drows.t, dw.t)
    torch.cuda.synchronize()
    for g, what in ((out, "rows"), (y, "out"), (drows, "drows"), (dw, "dweights")):
        g.check(what)
    assert dw.t[3] == 0 and dw.t[5] == 0
    assert bool((out.t.view(r.rows, 72)[torch.from_numpy(r.pos[[3, 5]]).cuda()] == 0).all())


@pytest.mark.parametrize("T", [70001, 140001, 290001])
def test_many_groups_of_the_sort(T):
    """More slots than 256 work-groups of 1024 (and of 4096): the groups grow."""
    r = Routing(T, 4, 300, 1, 1, "bf16", id_bytes=4, drop=0.01)
    got = r.out_index()
    b.basp_expert_sort(r.plan, r.ids_d, *[g.t for g in got], r.ws)
    r.check_index(got)


def test_rows_past_four_gib():
    """Row offsets above 2^32 bytes: the last rows of a 5 GiB buffer."""
    T, D = 82000, 16384
    plan = b.basp_expert_plan_create(T, 2, 4, D)
    ids = (torch.arange(2 * T, device="cuda") // 5 % 4).view(T, 2)
    index = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (2 * T, 2 * T, 5, 4)]
    ws = torch.empty(plan.info["workspace_bytes"], dtype=torch.uint8, device="cuda")
    x = (torch.arange(T, device="cuda") % 251).to(torch.bfloat16)[:, None].expand(T, D).contiguous()
    rows = torch.full((2 * T, D), NAN, dtype=torch.bfloat16, device="cuda")
    b.basp_route_to_expert(plan, x, ids, *index, rows, ws)
    token = index[1].long() // 2
    assert rows.numel() * 2 > 2**32
    assert torch.equal(rows[:, 0], x[token, 0]) and torch.equal(rows[:, -1], x[token, -1])
    assert torch.equal(rows[-3:], x[token[-3:]])
    y = torch.full((T, D), NAN, dtype=torch.bfloat16, device="cuda")
    w = torch.full((T, 2), 0.5, device="cuda")
    b.basp_expert_to_seq(plan, rows, index[0], w, y)
    assert torch.equal(y, x)
    y.fill_(NAN)
    b.basp_seq_to_expert_grad(plan, rows, index[0], y)
    assert torch.equal(y, x + x)
    drows, dw = torch.full_like(rows, NAN), torch.full_like(w, NAN)
    one = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    one[:, 5] = 2.0
    b.basp_expert_to_seq_grad(plan, one, rows, index[0], index[1], w, drows, dw)
    assert torch.equal(dw, (2 * x[:, :1].float()).expand(T, 2))
    assert bool((drows[:, 5] == 1).all()) and int(torch.count_nonzero(drows)) == 2 * T
