"""Embedding lookup and its gradient on the GPU, against plain forms in 64 bits
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


class Lookup:
    """A plan, ids, and where each token's row lies."""

    def __init__(self, layout, V, D, dtype="bf16", grad="bf16", id_bytes=8, padding=-1, outside=0.0, seed=0, ids=None):
        N, B, S, G = layout if isinstance(layout, tuple) else (1, 1, layout, 1)
        self.T, self.V, self.D, self.padding = B * S, V, D, padding
        self.dt, self.gdt = ic.FLOATS[dtype], ic.FLOATS[grad]
        self.rng = np.random.default_rng(seed)
        if ids is None:
            ids = np.minimum((np.exp(self.rng.random(self.T) * np.log(V + 1)) - 1).astype(np.int64), V - 1)
            gone = self.rng.random(self.T) < outside
            out = [-1, V, -2**31, 2**31 - 1] + ([2**32, 2**40 + 1] if id_bytes == 8 else [])
            ids[gone] = self.rng.choice(np.array(out, dtype=np.int64), size=int(gone.sum()))
        self.ids = np.asarray(ids, dtype=np.int64)
        of = None if not isinstance(layout, tuple) else b.basp_plan_create_groups(N, B, S, N, N, 8, b.BASP_BF16, G)
        self.place = ic.seq_place(N, B, S, G)
        self.plan = b.basp_embed_plan_create(of, self.T, V, D, padding, id_bytes, code(dtype), code(grad))
        self.ids_d = torch.from_numpy(self.ids).to(torch.int64 if id_bytes == 8 else torch.int32).cuda()
        self.ws = torch.full((max(1, self.plan.info["workspace_bytes"]),), 255, dtype=torch.uint8, device="cuda")

    def normal(self, *shape, dtype=None):
        return torch.from_numpy(self.rng.standard_normal(shape).astype(np.float32)).to(dtype or self.dt).cuda()

    def grad(self, dy, scale):
        """Exact gradient, its absolute terms and the tokens of each row."""
        g, a, n = np.zeros((self.V, self.D)), np.zeros((self.V, self.D)), np.zeros(self.V, dtype=np.int64)
        used = (self.ids >= 0) & (self.ids < self.V) & (self.ids != self.padding)
        dy = dy.double().cpu().numpy()[self.place[used]] * scale
        np.add.at(g, self.ids[used], dy)
        np.add.at(a, self.ids[used], np.abs(dy))
        np.add.at(n, self.ids[used], 1)
        return g, a, n


SIZES = [  # layout (N, B, S, groups) or tokens, V, D, dtype, grad, id_bytes, padding, outside
    (1, 1, 1, "bf16", "bf16", 8, -1, 0.0),
    (2, 5, 3, "fp16", "fp32", 4, 0, 0.0),
    (31, 7, 9, "fp32", "bf16", 8, -1, 0.3),
    (33, 1000, 2048, "bf16", "fp32", 8, 2, 0.1),
    ((4, 2, 8, 1), 50, 64, "bf16", "bf16", 8, -1, 0.0),
    ((6, 4, 33, 2), 300, 65, "fp16", "fp16", 4, -1, 0.1),
    ((8, 2, 512, 1), 2000, 520, "bf16", "bf16", 8, 1, 0.0),
    ((8, 8, 96, 2), 1023, 31, "fp32", "fp32", 8, -1, 0.0),
    ((3, 6, 100, 3), 1024, 1001, "bf16", "fp32", 4, -1, 0.05),
    (4095, 8191, 501, "fp32", "fp32", 4, -1, 0.0),
    (2500, 3, 260, "bf16", "fp16", 8, -1, 0.0),
    (5001, 2000, 8, "bf16", "bf16", 8, -1, 0.0),
    (3000, 1500000, 16, "bf16", "bf16", 8, -1, 0.0),
    (700, 40, 9001, "fp16", "fp32", 8, -1, 0.0),
    (8192, 300, 40, "bf16", "fp32", 8, -1, 0.01),
    (8193, 300, 40, "bf16", "fp32", 8, -1, 0.01),
    (11264, 381299, 9, "bf16", "bf16", 8, -1, 0.01),
    (11265, 40, 33, "bf16", "fp32", 8, -1, 0.01),
    (7168, 1 << 22, 3, "bf16", "bf16", 8, -1, 0.01),
    ((2, 2, 10000, 1), 70001, 24, "fp16", "bf16", 4, 5, 0.02),
    (9000, 1500000, 9, "bf16", "bf16", 8, -1, 0.0),
    (20001, 511, 520, "bf16", "fp32", 4, -1, 0.0),
    (30000, 1023, 16, "fp16", "fp32", 8, 700, 0.3),
    (30000, 1024, 16, "bf16", "fp32", 4, -1, 0.3),
    (12000, 1 << 20, 12, "bf16", "bf16", 8, -1, 0.05),
    (530001, 1000, 2, "fp32", "fp32", 4, -1, 0.1),
    (1100001, 3000, 2, "bf16", "fp32", 8, -1, 0.01),
]
IDS = ["x".join(map(str, s)).replace(" ", "") for s in SIZES]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_lookup(size, shift):
    r = Lookup(*size)
    table = r.normal(r.V, r.D)
    scale = 3.3
    inside = (r.ids >= 0) & (r.ids < r.V)
    want = np.zeros((r.T, r.D))
    want[r.place[inside]] = table.double().cpu().numpy()[r.ids[inside]] * np.float64(np.float32(scale))
    out = ic.Guarded(r.T * r.D, r.dt, NAN, shift)
    b.basp_embed_to_seq(r.plan, r.ids_d, ic.shifted(table, shift), scale, out.t)
    torch.cuda.synchronize()
    ic.check(out.t, want, np.abs(want), 1, "rows")
    out.check("rows")


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_gradient(size, shift):
    """Overwriting and accumulating; the rows of ignored tokens hold NaN."""
    r = Lookup(*size)
    dy, scale = r.normal(r.T, r.D), 0.75
    ignored = (r.ids < 0) | (r.ids >= r.V) | (r.ids == r.padding)
    dy[torch.from_numpy(r.place[ignored]).cuda()] = NAN
    g, terms, n = r.grad(dy, scale)
    dys = ic.shifted(dy, shift)
    out = ic.Guarded(r.V * r.D, r.gdt, NAN, shift)
    b.basp_embed_to_seq_grad(r.plan, r.ids_d, dys, scale, False, out.t, r.ws)
    torch.cuda.synchronize()
    ic.check(out.t, g, terms, n[:, None], "gradient")
    out.check("gradient")
    first = out.t.clone()
    out.t.fill_(NAN)
    r.ws.fill_(17)
    b.basp_embed_to_seq_grad(r.plan, r.ids_d, dys, scale, False, out.t, r.ws)
    assert torch.equal(first, out.t), "not the same bits again"
    # into a gradient that is there
    base = r.normal(r.V, r.D, dtype=r.gdt)
    acc = ic.Guarded(r.V * r.D, r.gdt, NAN, shift)
    acc.t.copy_(base.view(-1))
    b.basp_embed_to_seq_grad(r.plan, r.ids_d, dys, scale, True, acc.t, r.ws)
    torch.cuda.synchronize()
    old = base.double().cpu().numpy()
    ic.check(acc.t, old + g, terms + np.abs(old), n[:, None] + 1, "accumulated gradient")
    acc.check("accumulated gradient")
    untouched = torch.from_numpy(n == 0).cuda()
    assert torch.equal(acc.t.view(r.V, r.D)[untouched], base[untouched])


@pytest.mark.parametrize("ids", ["same", "two", "all outside", "distinct", "runs of 32", "runs of 33"])
@pytest.mark.parametrize("T", [32, 33, 1000, 5000, 10000, 20000])
def test_long_and_short_runs(ids, T):
    """One id for all tokens, ids that fill whole chunks, and none repeated."""
    t = np.arange(T)
    V = 20000
    of = {"same": t * 0 + 17, "two": (t * 7 % 13 > 5) * 5999, "all outside": t * 0 + V, "distinct": t[::-1].copy(),
          "runs of 32": t // 32, "runs of 33": t // 33}[ids]
    r = Lookup(T, V, 72, "bf16", "fp32", ids=of)
    dy = r.normal(r.T, r.D)
    g, terms, n = r.grad(dy, 1.0)
    out = ic.Guarded(V * 72, r.gdt, NAN)
    b.basp_embed_to_seq_grad(r.plan, r.ids_d, dy, 1.0, False, out.t, r.ws)
    torch.cuda.synchronize()
    ic.check(out.t, g, terms, n[:, None], "gradient")
    out.check("gradient")


def test_no_tokens():
    r = Lookup(0, 70, 24)
    none = torch.empty(0, dtype=r.dt, device="cuda")
    out = ic.Guarded(70 * 24, r.gdt, NAN)
    b.basp_embed_to_seq(r.plan, r.ids_d, None, 1.0, none)
    b.basp_embed_to_seq_grad(r.plan, r.ids_d, none, 1.0, True, out.t, None)
    torch.cuda.synchronize()
    assert bool(torch.isnan(out.t).all())
    b.basp_embed_to_seq_grad(r.plan, r.ids_d, none, 1.0, False, out.t, None)
    torch.cuda.synchronize()
    assert bool((out.t == 0).all())
    out.check("gradient")


def test_table_past_four_gib():
    """Row offsets above 2^32 bytes in the table and its gradient."""
    V, D = 140000, 16384
    assert V * D * 2 > 2**32
    plan = b.basp_embed_plan_create(None, 6, V, D)
    ids = torch.tensor([V - 1, 0, V - 2, 131072, V - 1, 131071], device="cuda")
    table = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    table[ids] = torch.tensor([1.0, 2.0, 3.0, 4.0, 1.0, 6.0], device="cuda").bfloat16()[:, None]
    out = torch.full((6, D), NAN, dtype=torch.bfloat16, device="cuda")
    b.basp_embed_to_seq(plan, ids, table, 2.0, out)
    want = torch.tensor([2.0, 4.0, 6.0, 8.0, 2.0, 12.0], device="cuda").bfloat16()[:, None]
    assert torch.equal(out, want.expand(6, D))
    table.fill_(NAN)
    ws = torch.empty(plan.info["workspace_bytes"], dtype=torch.uint8, device="cuda")
    b.basp_embed_to_seq_grad(plan, ids, out, 1.0, False, table, ws)
    assert torch.equal(table[ids], torch.tensor([4.0, 4.0, 6.0, 8.0, 4.0, 12.0], device="cuda").bfloat16()[:, None]
                       .expand(6, D))
    table[ids] = 0
    assert not bool(table.any())


def test_activations_past_four_gib():
    """Row offsets above 2^32 bytes in the activations, looked up and summed."""
    T, D, V = 140000, 16384, 9
    plan = b.basp_embed_plan_create(None, T, V, D)
    ids = torch.arange(T, device="cuda") % V
    table = torch.arange(1, V + 1, device="cuda").bfloat16()[:, None].expand(V, D).contiguous()
    out = torch.full((T, D), NAN, dtype=torch.bfloat16, device="cuda")
    assert out.numel() * 2 > 2**32
    b.basp_embed_to_seq(plan, ids, table, 1.0, out)
    assert torch.equal(out, table[ids])
    out.fill_(0)
    out[T - V:] = table      # only the last token of each id has a gradient
    ws = torch.empty(plan.info["workspace_bytes"], dtype=torch.uint8, device="cuda")
    got = torch.full((V, D), NAN, dtype=torch.bfloat16, device="cuda")
    b.basp_embed_to_seq_grad(plan, ids, out, 1.0, False, got, ws)
    want = torch.empty_like(table)
    want[ids[T - V:]] = table
    assert torch.equal(got, want)
