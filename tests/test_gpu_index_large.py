"""The index-driven re-layouts at the sizes where they take other paths: sums
whose output streams past the caches, and tables whose rows of zeros are shared
out over several launches (MI355X only).  Exact forms in 64 bits on the device;
the bounds are those of tests/index_cases.py."""
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
MIB = 1 << 20
STREAMED = 32 * MIB     # bytes of output from which sums may take another store


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def code(name):
    return {"bf16": b.BASP_BF16, "fp16": b.BASP_FP16, "fp32": b.BASP_FP32}[name]


def check(got, exact, terms, n, what):
    """ic.check on the device: n is a number or a column of them."""
    fi = torch.finfo(got.dtype)
    got = got.view(exact.shape).double()
    assert bool(torch.isfinite(got).all()), "%s: not finite, or not written" % what
    err = 2 * (n + 1) * 2.0 ** -24 * terms
    over = (got - exact).abs() > err + fi.eps / 2 * (exact.abs() + err) + fi.smallest_normal * fi.eps / 2
    assert not bool(over.any()), "%s: %d of %d over the bound" % (what, int(over.sum()), over.numel())


# dtype, D: rows of whole waves of 16-byte vectors; the odd ones end inside a
# vector, so that their last vector starts anywhere
WIDTHS = [("bf16", 2048), ("fp16", 2048), ("fp32", 1024), ("bf16", 509), ("fp16", 505), ("fp32", 253), ("bf16", 1018)]


@pytest.mark.parametrize("above", [False, True], ids=["below", "above"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("K", [1, 2, 5])
@pytest.mark.parametrize("dtype,D", WIDTHS)
def test_sums_on_both_sides_of_streaming(dtype, D, K, shift, above):
    dt = ic.FLOATS[dtype]
    row = D * dt.itemsize
    T = -(-STREAMED // row) - (0 if above else 1)
    assert (T * row >= STREAMED) == above and -(-row // 16) % 64 == 0
    rng = np.random.default_rng(T + K)
    ids = ic.choices(rng, T, K, 16, 0.1)
    pos, order, _, _ = ic.index(ids, 16, 4)
    plan = b.basp_expert_plan_create(T, K, 16, D, 4, dtype=code(dtype))
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    rows = torch.randn(order.size, D, generator=g, device="cuda").to(dt)
    rows[torch.from_numpy(order < 0).cuda()] = NAN
    w = torch.randn(T, K, generator=g, device="cuda")
    pos_d = torch.from_numpy(pos).int().cuda()
    at = torch.from_numpy(pos).cuda().view(T, K)
    for weighted in (True, False):
        exact, terms = (torch.zeros(T, D, dtype=torch.float64, device="cuda") for _ in range(2))
        for k in range(K):
            t = torch.nonzero(at[:, k] >= 0)[:, 0]
            v = rows[at[t, k]].double()
            if weighted:
                v *= w[t, k, None].double()
            exact[t] += v
            terms[t] += v.abs()
        out = ic.Guarded(T * D, dt, NAN, shift)
        if weighted:
            b.basp_expert_to_seq(plan, ic.shifted(rows, shift), pos_d, ic.shifted(w, shift), out.t)
        else:
            b.basp_seq_to_expert_grad(plan, ic.shifted(rows, shift), pos_d, out.t)
        torch.cuda.synchronize()
        what = "expert -> seq" if weighted else "gradient of seq -> expert"
        check(out.t, exact, terms, K, what)
        out.check(what)


TABLES = [  # V, D, dtype, grad, tokens
    (131072, 2048, "bf16", "bf16", 12001),      # one piece of zeros a row, two digits
    (50021, 5001, "bf16", "bf16", 12500),       # three pieces a row
    ((1 << 22) + 3, 64, "bf16", "bf16", 12001),     # 32 rows a piece, three digits
    (131071, 1000, "fp16", "fp32", 20000),
    (3000017, 45, "fp32", "fp32", 13001),       # 22 rows a piece, an odd width
]


@pytest.mark.parametrize("named", ["around", "at"])
@pytest.mark.parametrize("V,D,dtype,grad,T", TABLES)
def test_zeros_shared_out_over_launches(V, D, dtype, grad, T, named):
    """More zeros than the sort's launches take: every row is written once,
    also where one launch's share ends and the next one's begins (multiples of
    32 MiB), whether the rows there have tokens or their neighbours do."""
    dt, gdt = ic.FLOATS[dtype], ic.FLOATS[grad]
    row = D * gdt.itemsize
    assert V * row > 448 * MIB
    rng = np.random.default_rng(V)
    ids = rng.integers(0, V, T)
    ends = np.arange(32 * MIB, V * row, 32 * MIB) // row
    near = np.concatenate([ends + d for d in range(-2, 3)])
    ids = ids[~np.isin(ids, near)]
    take = np.concatenate([ends - 2, ends + 1, [0]] if named == "around" else [ends - 1, ends, [V - 1]])
    ids = np.concatenate([ids, take, take])[-T:]
    ids = np.concatenate([ids, np.full(T - ids.size, take[0])])
    rng.shuffle(ids)
    plan = b.basp_embed_plan_create(None, T, V, D, dtype=code(dtype), grad_dtype=code(grad))
    ids_d = torch.from_numpy(ids).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    dy = torch.randn(T, D, generator=g, device="cuda").to(dt)
    ws = torch.full((plan.info["workspace_bytes"],), 255, dtype=torch.uint8, device="cuda")
    out = ic.Guarded(V * D, gdt, NAN)
    b.basp_embed_to_seq_grad(plan, ids_d, dy, 0.75, False, out.t, ws)
    torch.cuda.synchronize()
    out.check("gradient")
    rows, which = torch.unique(ids_d, return_inverse=True)
    got = out.t.view(V, D)
    exact, terms = (torch.zeros(rows.numel(), D, dtype=torch.float64, device="cuda") for _ in range(2))
    exact.index_add_(0, which, dy.double() * 0.75)
    terms.index_add_(0, which, dy.double().abs() * 0.75)
    n = torch.bincount(which)[:, None]
    check(got[rows], exact, terms, n, "gradient")
    has = torch.zeros(V, dtype=torch.bool, device="cuda")
    has[rows] = True
    zero = torch.cat([(part == 0).all(1) for part in got.split(1 << 16)])
    assert bool((zero | has).all()), "rows without a token: %d are not zeros" % int((~(zero | has)).sum())


@pytest.mark.parametrize("major", ["head", "token"])
@pytest.mark.parametrize("N,B,S,G", [(4, 2, 24, 1), (8, 4, 16, 2), (6, 6, 9, 2), (4, 4, 12, 4), (3, 1, 30, 1)])
def test_embedded_batch_through_the_boundary(N, B, S, G, major):
    """Embedded rows re-laid by the boundary's call are the head-sharded
    buffer of the batch, and the head-sharded gradient reaches the table: the
    embedding's order is the boundary's.  Whole numbers, so both are exact."""
    H, d, V = 2 * N, 4, 37
    P, Bl, Hl, D = N // G, B // G, 2 * N // (N // G), 2 * N * 4
    major_code = {"head": b.BASP_LAYOUT_HEAD_MAJOR, "token": b.BASP_LAYOUT_TOKEN_MAJOR}[major]
    layout = b.basp_plan_create_groups(N, B, S, H, H, d, b.BASP_FP32, G, major_code)
    embed = b.basp_embed_plan_create(layout, B * S, V, D, dtype=b.BASP_FP32, grad_dtype=b.BASP_FP32)
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    ids = torch.randint(0, V, (B, S), generator=g, device="cuda")
    table = torch.randint(-1000, 1000, (V, D), generator=g, device="cuda").float()

    def head_sharded(batch):
        """[B][S][H][d] by rank: group n // P has sequences, member n % P heads."""
        parts = []
        for n in range(N):
            of = batch[n // P * Bl:(n // P + 1) * Bl, :, n % P * Hl:(n % P + 1) * Hl]
            parts.append((of.transpose(1, 2) if major == "head" else of).reshape(-1))
        return torch.cat(parts)

    rows = torch.full((B * S * D,), NAN, device="cuda")
    b.basp_embed_to_seq(embed, ids, table, 2.0, rows)
    got = torch.full_like(rows, NAN)
    b.basp_seq_to_head_o(layout, rows, got)
    assert torch.equal(got, head_sharded(2.0 * table[ids].view(B, S, H, d)))

    dy = torch.randint(-1000, 1000, (B, S, H, d), generator=g, device="cuda").float()
    b.basp_head_to_seq(layout, head_sharded(dy), rows)
    dtable = torch.full((V, D), NAN, device="cuda")
    ws = torch.empty(embed.info["workspace_bytes"], dtype=torch.uint8, device="cuda")
    b.basp_embed_to_seq_grad(embed, ids, rows, 2.0, False, dtable, ws)
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids.view(-1), 2.0 * dy.view(-1, D).double())
    assert torch.equal(dtable.double(), want)
