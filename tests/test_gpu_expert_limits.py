"""The sort by expert at the largest sizes a plan accepts, on the GPU (MI355X
only)."""
import pytest
import torch

from tests import index_cases as ic

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sequence_re_layout_amd import binding as b
else:  # collected on a machine without a GPU: every test here is skipped
    b = None


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def is_range(t, first):
    """t is first, first + 1, ... (looked at in parts: t is several GiB)."""
    part = 1 << 28
    return all(torch.equal(t[i:i + part], torch.arange(first + i, first + min(i + part, t.numel()), dtype=torch.int32,
                                                       device=t.device))
               for i in range(0, t.numel(), part))


@pytest.mark.parametrize("T,align", [(2147482999, 1000), (2147483646, 1)])
def test_one_expert_with_nearly_2_to_31_slots(T, align):
    """Counts whose rounding up to a multiple of align passes 2^31."""
    plan = b.basp_expert_plan_create(T, 1, 1, 1, align, id_bytes=4)
    rows = plan.info["max_rows"]
    assert rows == ic.max_rows(T, 1, 1, align) and T <= rows < 2**31
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos, order, offsets, counts = (ic.Guarded(n, torch.int32, -7) for n in (T, rows, 2, 1))
    ws = torch.empty(plan.info["workspace_bytes"], dtype=torch.uint8, device="cuda")
    b.basp_expert_sort(plan, ids, pos.t, order.t, offsets.t, counts.t, ws)
    torch.cuda.synchronize()
    assert counts.t.tolist() == [T] and offsets.t.tolist() == [0, rows]
    assert is_range(pos.t, 0) and is_range(order.t[:T], 0) and bool((order.t[T:] == -1).all())
    for g, what in ((pos, "pos"), (offsets, "offsets"), (counts, "counts")):
        g.check(what)
    assert bool((order.whole[:order.at] == -7).all()) and bool((order.whole[order.at + rows:] == -7).all())
