"""Attention, layer norm and balance loss on the host (no GPU): plans and their
refusals, sizes, and the pre-launch checks of every pointer and number.  No call
here reaches a kernel launch."""
import ctypes

import pytest

from sequence_re_layout_amd import binding as b
from tests.test_index_abi import refusals, status_of

BF, F16, F32, I32 = 0, 1, 2, 3
OK, INVALID, INDIVISIBLE, UNSUPPORTED = b.BASP_OK, b.BASP_ERR_INVALID, b.BASP_ERR_INDIVISIBLE, b.BASP_ERR_UNSUPPORTED


def layout(N=4, B=2, S=64, Hq=8, Hkv=4, d=16, dtype=BF, G=2, order=0):
    return b.basp_plan_create_groups(N, B, S, Hq, Hkv, d, dtype, G, order)


@pytest.mark.parametrize("of,args,status", [
    (dict(), (64, 64, 0), OK),
    (dict(), (1, 1, 0), OK),
    (dict(), (64, 1 << 62, 1 << 62), OK),
    (dict(S=0), (0, 1, 0), OK),
    (dict(dtype=F32, d=128), (64, 8, 70), OK),
    (dict(d=1), (64, 8, 4), OK),
    (dict(), (0, 8, 0), INVALID),                       # no queries of a cache that holds tokens
    (dict(), (65, 8, 0), INVALID),
    (dict(), (-1, 8, 0), INVALID),
    (dict(S=0), (1, 8, 0), INVALID),
    (dict(), (64, 0, 0), INVALID),
    (dict(), (64, -5, 0), INVALID),
    (dict(), (64, 8, -1), INVALID),
    (dict(Hq=12, Hkv=8), (64, 8, 0), INDIVISIBLE),
    (dict(dtype=I32), (64, 8, 0), UNSUPPORTED),
    (dict(d=129), (64, 8, 0), UNSUPPORTED),
    (dict(N=1, B=1, G=1, Hq=1, Hkv=1, d=1, S=(1 << 29) - 1), (1, 1 << 40, 3), OK),
    (dict(N=1, B=1, G=1, Hq=1, Hkv=1, d=1, S=1 << 29), (1, 8, 0), UNSUPPORTED),
    (dict(N=1, B=1, G=1, Hq=16, Hkv=1, d=1, S=1 << 27), ((1 << 26) - 1, 8, 0), OK),
    (dict(N=1, B=1, G=1, Hq=16, Hkv=1, d=1, S=1 << 27), (1 << 26, 8, 0), UNSUPPORTED),    # 2^30 columns
    (dict(N=1, B=1, G=1, Hq=1 << 17, Hkv=1, d=128, S=1), (1, 1, 0), UNSUPPORTED),         # a token of over 2^24 bytes
])
def test_attention_plan_status(of, args, status):
    plan = layout(**of)
    lib = b.library()
    assert status_of(lib.basp_attention_plan_create, lib.basp_attention_plan_destroy, plan.handle, *args) == status


def test_attention_plan_needs_a_layout():
    lib = b.library()
    assert status_of(lib.basp_attention_plan_create, lib.basp_attention_plan_destroy, None, 1, 1, 0) == INVALID
    with pytest.raises(TypeError):
        b.basp_attention_plan_create(b.basp_norm_plan_create(4, 4), 1, 1)
    with pytest.raises(TypeError):
        b.basp_attention_plan_create(None, 1, 1)
    gone = layout()
    b.basp_plan_destroy(gone)
    with pytest.raises(b.BaspError) as e:
        b.basp_attention_plan_create(gone, 1, 1)
    assert e.value.status == INVALID
    with pytest.raises(ValueError):
        b.basp_attention_plan_create(layout(), 1, 1 << 63)
    with pytest.raises(b.BaspError) as e:
        b.basp_attention_plan_create(layout(), 1, 0)
    assert e.value.status == INVALID


@pytest.mark.parametrize("order", [0, 1])
def test_attention_plan_sizes(order):
    l = layout(N=8, B=4, S=96, Hq=16, Hkv=8, d=24, G=2, order=order)
    i = b.basp_attention_plan_create(l, 10, 20, 3).info
    of = l.info
    # a shard for each rank and sequence of its group; heads of a rank
    assert i["shards"] == 8 * 2 and (i["Hl_q"], i["Hl_kv"]) == (of["Hl_q"], of["Hl_kv"]) == (4, 2)
    assert (i["S"], i["queries"], i["window"], i["sinks"], i["B"], i["d"], i["layout"]) == (96, 10, 20, 3, 4, 24, order)
    assert i["kv_elems"] == of["kv_elems"] and i["q_elems"] * 96 == of["q_elems"] * 10
    assert i["lse_elems"] * 24 == i["q_elems"]
    # with all queries the parts of the fused buffer
    assert b.basp_attention_plan_create(l, 96, 20, 3).info["q_elems"] == of["q_elems"]


def test_attention_workspaces_stay_small():
    """Unfinished sums are those of at most about two work-groups a compute unit, whatever the sinks are."""
    for sinks in (0, 4, 200, 5000, 30000):
        l = layout(N=8, B=2, S=32768, Hq=24, Hkv=8, d=128, G=2)
        i = b.basp_attention_plan_create(l, 32768, 1024, sinks).info
        assert i["workspace_bytes"] == 0
        assert i["grad_workspace_bytes"] <= i["lse_elems"] * 8 + 256 + 1500 * 2 * 128 * 128 * 4, sinks
    i = b.basp_attention_plan_create(layout(N=1, B=1, G=1, S=1 << 20, Hq=8, Hkv=1, d=128), 1, 1 << 20).info
    assert 0 < i["workspace_bytes"] <= 512 * 32 * 130 * 4


@pytest.mark.parametrize("args,status", [
    ((16, 64, BF, F32), OK),
    ((0, 1, F16, F16), OK),
    (((1 << 31) - 2, 1, BF, BF), OK),
    ((16, (1 << 28) - 1, F32, BF), OK),
    ((-1, 64, BF, F32), INVALID),
    ((16, 0, BF, F32), INVALID),
    ((16, 64, I32, F32), INVALID),
    ((16, 64, BF, I32), INVALID),
    ((16, 64, 7, F32), INVALID),
    (((1 << 31) - 1, 64, BF, F32), UNSUPPORTED),
    ((16, 1 << 28, BF, F32), UNSUPPORTED),
])
def test_norm_plan_status(args, status):
    lib = b.library()
    assert status_of(lib.basp_norm_plan_create, lib.basp_norm_plan_destroy, *args) == status


def test_norm_plan_arguments():
    i = b.basp_norm_plan_create(100, 48, b.BASP_FP16, b.BASP_BF16).info
    assert (i["T"], i["D"], i["dtype"], i["weight_dtype"]) == (100, 48, F16, BF) and i["workspace_bytes"] > 0
    with pytest.raises(ValueError):
        b.basp_norm_plan_create(1 << 63, 4)
    with pytest.raises(ValueError):
        b.basp_norm_plan_create(4, 4, dtype=1 << 31)


def test_balance_workspace():
    for T, E in ((0, 4), (1, 1024), (100000, 64)):
        plan = b.basp_expert_plan_create(T, 2, E, 1)
        assert b.basp_balance_workspace_bytes(plan) >= (2 * E + 1) * 4
    assert b.library().basp_balance_workspace_bytes(None) == 0 and b.basp_last_error() == INVALID


def test_null_plans():
    lib = b.library()
    assert lib.basp_attention_plan_query(None, None) == INVALID and lib.basp_norm_plan_query(None, None) == INVALID
    assert lib.basp_attention(None, *[None] * 5, 1.0, *[None] * 4) == INVALID
    assert lib.basp_attention_grad(None, *[None] * 8, 1.0, *[None] * 5) == INVALID
    assert lib.basp_layer_norm(None, *[None] * 3, 1e-5, *[None] * 4) == INVALID
    assert lib.basp_layer_norm_grad(None, *[None] * 10) == INVALID
    assert lib.basp_balance_loss(None, *[None] * 3, 1.0, *[None] * 5) == INVALID
    assert lib.basp_balance_loss_grad(None, *[None] * 6) == INVALID
    lib.basp_attention_plan_destroy(None)
    lib.basp_norm_plan_destroy(None)
    assert b.basp_last_error() == OK


def optional_refusals(call, buffers, optional):
    """refusals() with NULL allowed at some places, tried with and without them;
    a NULL there is not refused for itself, so it is left out of that check."""
    every = [x for x in buffers]
    refusals(lambda *a: call(*a) if all(a[i] is not None for i in optional) else INVALID, every)


@pytest.mark.parametrize("dtype,es", [(BF, 2), (F32, 4)])
def test_attention_refuses_pointers(dtype, es):
    lib = b.library()
    l = layout(S=4096, d=64, dtype=dtype, N=1, B=2, G=1, Hq=2, Hkv=1)
    for queries in (1, 4096):
        plan = b.basp_attention_plan_create(l, queries, 512 if queries > 1 else 4096, 4)
        i = plan.info
        nq, nkv, rows = i["q_elems"] * es, i["kv_elems"] * es, i["lse_elems"] * 4
        h = plan.handle
        if i["workspace_bytes"]:
            ws = [(i["workspace_bytes"], 16, True)]
        else:
            ws = []
        fwd = [(nq, es, False), (nkv, es, False), (nkv, es, False), (8, 4, False), (8, 4, False), (nq, es, True), (rows, 4, True)] + ws
        optional_refusals(lambda *a: lib.basp_attention(h, *a[:5], 0.1, *a[5:7], a[7] if ws else None, None), fwd, (3, 4, 6))
        bwd = [(nq, es, False), (nkv, es, False), (nkv, es, False), (nq, es, False), (rows, 4, False), (nq, es, False), (8, 4, False),
               (8, 4, False), (nq, es, True), (nkv, es, True), (nkv, es, True), (i["grad_workspace_bytes"], 16, True)]
        optional_refusals(lambda *a: lib.basp_attention_grad(h, *a[:8], 0.1, *a[8:], None), bwd, (6, 7))


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 101, 1e-45, 3e38])
def test_attention_refuses_scales(scale):
    lib = b.library()
    h = b.basp_attention_plan_create(layout(), 64, 8)
    assert lib.basp_attention(h.handle, *[1 << 40] * 5, scale, *[1 << 41] * 4) == INVALID
    assert lib.basp_attention_grad(h.handle, *[1 << 40] * 8, scale, *[1 << 41] * 5) == INVALID


def test_norm_refuses_pointers_and_numbers():
    lib = b.library()
    plan = b.basp_norm_plan_create(100, 48, b.BASP_BF16, b.BASP_FP32)
    h, n, cols, stats = plan.handle, 100 * 48 * 2, 48 * 4, 400
    optional_refusals(lambda *a: lib.basp_layer_norm(h, *a[:3], 1e-5, *a[3:], None),
                      [(n, 2, False), (cols, 4, False), (cols, 4, False), (n, 2, True), (stats, 4, True), (stats, 4, True)], (2, 4, 5))
    optional_refusals(lambda *a: lib.basp_layer_norm_grad(h, *a, None),
                      [(n, 2, False), (n, 2, False), (cols, 4, False), (stats, 4, False), (stats, 4, False), (n, 2, True),
                       (cols, 4, True), (cols, 4, True), (plan.info["workspace_bytes"], 16, True)], (7,))
    for eps in (-1e-6, float("nan"), float("inf")):
        assert lib.basp_layer_norm(h, *[1 << 40] * 3, eps, *[1 << 41] * 4) == INVALID


def test_balance_refuses_pointers_and_numbers():
    lib = b.library()
    plan = b.basp_expert_plan_create(300, 2, 16, 1, id_bytes=4, weight_dtype=b.BASP_FP16)
    h, n, E = plan.handle, 300 * 16 * 2, 64
    optional_refusals(lambda *a: lib.basp_balance_loss(h, *a[:3], 0.1, *a[3:], None),
                      [(n, 2, False), (2400, 4, False), (300, 1, False), (4, 4, True), (E, 4, True), (E, 4, True),
                       (plan.balance_bytes, 16, True)], (2,))
    optional_refusals(lambda *a: lib.basp_balance_loss_grad(h, *a, None),
                      [(n, 2, False), (300, 1, False), (E, 4, False), (4, 4, False), (n, 2, True)], (1,))
    for coef in (float("nan"), float("inf")):
        assert lib.basp_balance_loss(h, *[1 << 40] * 3, coef, *[1 << 41] * 5) == INVALID


def test_structs_match_the_header():
    """Sizes that a C program sees: the fields in their order, without gaps but those of alignment."""
    assert ctypes.sizeof(b.basp_attention_info) == 3 * 8 + 8 * 4 + 5 * 8
    assert ctypes.sizeof(b.basp_norm_info) == 2 * 8 + 2 * 4 + 8
