"""The index-driven re-layouts on the host (no GPU): plan creation and its
refusals, sizes, the pre-launch pointer checks, the place of a token in the
sequence-sharded layout, and the cover of the launches that write zeros.  No
call here reaches a kernel launch."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from sequence_re_layout_amd import binding as b
from tests import index_cases as ic

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sequence_re_layout_amd", "csrc")
BASE = 1 << 40   # fake addresses: never dereferenced


def status_of(create, destroy, *args):
    h = create(*args)
    st = b.basp_last_error()
    if h:
        destroy(h)
    return st


BF, F16, F32, I32 = 0, 1, 2, 3


@pytest.mark.parametrize("args,status", [
    ((16, 2, 8, 64, 1, 8, BF, F32), b.BASP_OK),
    ((0, 2, 8, 64, 1, 8, BF, F32), b.BASP_OK),                       # no tokens
    ((16, 2, 1, 1, 1, 4, F32, BF), b.BASP_OK),                       # more choices than experts
    ((-1, 2, 8, 64, 1, 8, BF, F32), b.BASP_ERR_INVALID),
    ((16, 0, 8, 64, 1, 8, BF, F32), b.BASP_ERR_INVALID),
    ((16, 2, 0, 64, 1, 8, BF, F32), b.BASP_ERR_INVALID),
    ((16, 2, 8, 0, 1, 8, BF, F32), b.BASP_ERR_INVALID),
    ((16, 2, 8, 64, 0, 8, BF, F32), b.BASP_ERR_INVALID),
    ((16, 2, 8, 64, 1, 2, BF, F32), b.BASP_ERR_INVALID),             # id_bytes
    ((16, 2, 8, 64, 1, 8, I32, F32), b.BASP_ERR_INVALID),            # rows of whole numbers
    ((16, 2, 8, 64, 1, 8, BF, I32), b.BASP_ERR_INVALID),
    ((16, 2, 8, 64, 1, 8, 9, F32), b.BASP_ERR_INVALID),
    ((16, 2, 1024, 64, 65536, 8, BF, F32), b.BASP_OK),
    ((16, 2, 1025, 64, 1, 8, BF, F32), b.BASP_ERR_UNSUPPORTED),
    ((16, 2, 8, 64, 65537, 8, BF, F32), b.BASP_ERR_UNSUPPORTED),
    ((16, 2, 8, (1 << 29) - 1, 1, 8, BF, F32), b.BASP_OK),
    ((16, 2, 8, 1 << 29, 1, 8, BF, F32), b.BASP_ERR_UNSUPPORTED),    # a row of 2^30 bytes
    ((16, 2, 8, 1 << 28, 1, 8, F32, F32), b.BASP_ERR_UNSUPPORTED),
    ((16, 2, 8, 1 << 62, 1, 8, BF, F32), b.BASP_ERR_UNSUPPORTED),
    (((1 << 30) - 1, 2, 8, 64, 1, 8, BF, F32), b.BASP_OK),           # 2^31 - 2 slots
    ((1 << 30, 2, 8, 64, 1, 8, BF, F32), b.BASP_ERR_UNSUPPORTED),
    ((1 << 62, 1 << 30, 8, 64, 1, 8, BF, F32), b.BASP_ERR_UNSUPPORTED),
    (((1 << 30) - 1, 2, 8, 64, 2, 8, BF, F32), b.BASP_ERR_UNSUPPORTED),   # rows with padding
])
def test_expert_plan_status(args, status):
    lib = b.library()
    assert status_of(lib.basp_expert_plan_create, lib.basp_expert_plan_destroy, *args) == status


@pytest.mark.parametrize("T,K,E,align", [(0, 2, 8, 4), (1, 1, 1, 1), (16, 4, 64, 1), (16, 4, 64, 128), (7, 3, 5, 3),
                                         (4099, 3, 20, 16), (140001, 4, 300, 1)])
def test_expert_plan_sizes(T, K, E, align):
    i = b.basp_expert_plan_create(T, K, E, 24, align).info
    assert (i["T"], i["K"], i["E"], i["D"], i["align"]) == (T, K, E, 24, align)
    assert i["slots"] == T * K and i["max_rows"] == ic.max_rows(T, K, E, align)
    # enough for the worst ids: one slot in each expert first, then anywhere
    M = T * K
    ones = min(E, M)
    assert i["max_rows"] >= ones * align if align <= M // max(1, ones) or ones == M else True
    worst = (ones - 1) * align + -(-(M - ones + 1) // align) * align if M else 0
    assert i["max_rows"] >= worst and i["max_rows"] % align == 0


@pytest.mark.parametrize("args,status", [
    ((10, 8, 64, -1, 8, BF, BF), b.BASP_OK),
    ((0, 8, 64, 7, 4, F32, BF), b.BASP_OK),
    ((-1, 8, 64, -1, 8, BF, BF), b.BASP_ERR_INVALID),
    ((10, 0, 64, -1, 8, BF, BF), b.BASP_ERR_INVALID),
    ((10, 8, 0, -1, 8, BF, BF), b.BASP_ERR_INVALID),
    ((10, 8, 64, 8, 8, BF, BF), b.BASP_ERR_INVALID),       # padding row outside the table
    ((10, 8, 64, -2, 8, BF, BF), b.BASP_ERR_INVALID),
    ((10, 8, 64, -1, 1, BF, BF), b.BASP_ERR_INVALID),
    ((10, 8, 64, -1, 8, I32, BF), b.BASP_ERR_INVALID),
    ((10, 8, 64, -1, 8, BF, I32), b.BASP_ERR_INVALID),
    ((10, 1 << 30, 64, -1, 8, BF, BF), b.BASP_OK),
    ((10, (1 << 30) + 1, 64, -1, 8, BF, BF), b.BASP_ERR_UNSUPPORTED),
    ((10, 8, (1 << 28) - 1, -1, 8, BF, BF), b.BASP_OK),
    ((10, 8, 1 << 28, -1, 8, BF, BF), b.BASP_ERR_UNSUPPORTED),
    (((1 << 31) - 2, 8, 1, -1, 8, BF, BF), b.BASP_OK),
    (((1 << 31) - 1, 8, 1, -1, 8, BF, BF), b.BASP_ERR_UNSUPPORTED),
    (((1 << 31) - 2, 8, 8192, -1, 8, BF, BF), b.BASP_ERR_UNSUPPORTED),   # 32 TiB of activations
])
def test_embed_plan_status(args, status):
    lib = b.library()
    assert status_of(lib.basp_embed_plan_create, lib.basp_embed_plan_destroy, None, *args) == status


def test_embed_plan_follows_a_layout():
    layout = b.basp_plan_create(8, 2, 64, 8, 8, 16)
    i = b.basp_embed_plan_create(layout, 128, 100, 24, padding=3, id_bytes=4, grad_dtype=b.BASP_FP32).info
    assert (i["T"], i["V"], i["D"], i["padding"], i["id_bytes"]) == (128, 100, 24, 3, 4)
    assert i["grad_dtype"] == b.BASP_FP32 and i["workspace_bytes"] > 0
    with pytest.raises(b.BaspError) as e:
        b.basp_embed_plan_create(layout, 127, 100, 24)
    assert e.value.status == b.BASP_ERR_INVALID


def test_null_plans():
    lib = b.library()
    inv = b.BASP_ERR_INVALID
    assert lib.basp_expert_plan_query(None, None) == inv and lib.basp_embed_plan_query(None, None) == inv
    assert lib.basp_expert_sort(None, *[None] * 7) == inv
    assert lib.basp_seq_to_expert(None, *[None] * 5) == inv
    assert lib.basp_route_to_expert(None, *[None] * 9) == inv
    assert lib.basp_seq_to_expert_grad(None, *[None] * 4) == inv
    assert lib.basp_expert_to_seq(None, *[None] * 5) == inv
    assert lib.basp_expert_to_seq_grad(None, *[None] * 8) == inv
    assert lib.basp_embed_to_seq(None, None, None, 1.0, None, None) == inv
    assert lib.basp_embed_to_seq_grad(None, None, None, 1.0, 0, None, None, None) == inv
    assert b.basp_last_error() == inv
    lib.basp_expert_plan_destroy(None)
    lib.basp_embed_plan_destroy(None)
    assert b.basp_last_error() == b.BASP_OK


def refusals(call, buffers):
    """call(*addresses) for buffers of (bytes, alignment, output): every NULL,
    every misalignment, every overlap of an output is refused."""
    at, addr = BASE, []
    for n, _, _ in buffers:
        addr.append(at)
        at += (n + 4096) // 256 * 256
    for i, (n, align, out) in enumerate(buffers):
        def with_(v):
            a = list(addr)
            a[i] = v
            return call(*a)
        if n:
            assert with_(None) == b.BASP_ERR_INVALID, i
        if align > 1:
            assert with_(addr[i] + align // 2) == b.BASP_ERR_ALIGN, i
        for j, (m, _, other_out) in enumerate(buffers):
            if i != j and n and m and (out or other_out):
                assert with_(addr[j]) == b.BASP_ERR_ALIAS, (i, j)
                last = (m - 1) // align * align          # over the other's last byte
                assert with_(addr[j] + last) == b.BASP_ERR_ALIAS, (i, j)


def test_pointer_checks_of_the_expert_calls():
    lib = b.library()
    p = b.basp_expert_plan_create(700, 3, 40, 72, 8, id_bytes=8, dtype=b.BASP_BF16, weight_dtype=b.BASP_FP32)
    i = p.info
    assert i["workspace_bytes"] > 0
    ids, pos, order = (i["slots"] * 8, 8), (i["slots"] * 4, 4), (i["max_rows"] * 4, 4)
    offsets, counts, ws = (41 * 4, 4), (40 * 4, 4), (i["workspace_bytes"], 16)
    x, rows, w = (700 * 72 * 2, 2), (i["max_rows"] * 72 * 2, 2), (i["slots"] * 4, 4)
    I, O = (False,), (True,)
    h = p.handle
    refusals(lambda *a: lib.basp_expert_sort(h, *a, None),
             [ids + I, pos + O, order + O, offsets + O, counts + O, ws + O])
    refusals(lambda *a: lib.basp_seq_to_expert(h, *a, None), [x + I, pos + I, order + I, rows + O])
    refusals(lambda *a: lib.basp_route_to_expert(h, *a, None),
             [x + I, ids + I, pos + O, order + O, offsets + O, counts + O, rows + O, ws + O])
    refusals(lambda *a: lib.basp_seq_to_expert_grad(h, *a, None), [rows + I, pos + I, x + O])
    refusals(lambda *a: lib.basp_expert_to_seq(h, *a, None), [rows + I, pos + I, w + I, x + O])
    refusals(lambda *a: lib.basp_expert_to_seq_grad(h, *a, None),
             [x + I, rows + I, pos + I, order + I, w + I, rows + O, w + O])


def test_pointer_checks_of_the_embedding_calls():
    lib = b.library()
    p = b.basp_embed_plan_create(None, 500, 100, 24, id_bytes=4, dtype=b.BASP_FP16, grad_dtype=b.BASP_FP32)
    ids, rows, table, grad = (500 * 4, 4), (500 * 24 * 2, 2), (100 * 24 * 2, 2), (100 * 24 * 4, 4)
    ws = (p.info["workspace_bytes"], 16)
    I, O = (False,), (True,)
    refusals(lambda i, t, o: lib.basp_embed_to_seq(p.handle, i, t, 1.0, o, None), [ids + I, table + I, rows + O])
    refusals(lambda i, d, g, w: lib.basp_embed_to_seq_grad(p.handle, i, d, 1.0, 0, g, w, None),
             [ids + I, rows + I, grad + O, ws + O])


def test_calls_on_no_tokens_need_no_device():
    lib = b.library()
    p = b.basp_expert_plan_create(0, 2, 8, 64, 4)
    assert lib.basp_seq_to_expert(p.handle, *[None] * 5) == b.BASP_OK
    assert lib.basp_seq_to_expert_grad(p.handle, *[None] * 4) == b.BASP_OK
    assert lib.basp_expert_to_seq(p.handle, *[None] * 5) == b.BASP_OK
    assert lib.basp_expert_to_seq_grad(p.handle, *[None] * 8) == b.BASP_OK
    e = b.basp_embed_plan_create(None, 0, 8, 64)
    assert lib.basp_embed_to_seq(e.handle, None, None, 1.0, None, None) == b.BASP_OK
    # the table itself is still an output, unless it is accumulated into
    assert lib.basp_embed_to_seq_grad(e.handle, None, None, 1.0, 0, None, None, None) == b.BASP_ERR_INVALID
    assert lib.basp_embed_to_seq_grad(e.handle, None, None, 1.0, 1, BASE, None, None) == b.BASP_OK


@pytest.fixture(scope="module")
def emu(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("emu") / "libindex_emu.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Werror", "-DBASP_HD=",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC]
                   + [os.path.join(CSRC, f) for f in ("plan.cpp", "launch.cpp", "index_plan.cpp")]
                   + [os.path.join(ROOT, "tests", "emu", "index_emu.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    lib.basp_plan_create_groups.argtypes = [i32, i32, i64, i32, i32, i32, i32, i32, i32]
    lib.basp_plan_create_groups.restype = vp
    lib.basp_plan_destroy.argtypes = [vp]
    lib.basp_embed_plan_create.argtypes = [vp, i64, i64, i64, i64, i32, i32, i32]
    lib.basp_embed_plan_create.restype = vp
    lib.basp_embed_plan_destroy.argtypes = [vp]
    lib.emu_seq_rows.argtypes = [vp, vp]
    lib.emu_zero_cover.argtypes = [i64, i64, i64, i32, vp]
    lib.emu_zero_cover.restype = i64
    return lib


@pytest.mark.parametrize("N,B,S,G", [(1, 1, 7, 1), (4, 2, 8, 1), (8, 2, 16, 2), (6, 4, 33, 2), (8, 8, 96, 2), (3, 6, 5, 3),
                                     (4, 8, 12, 4), (2, 2, 0, 1), (12, 6, 36, 2)])
def test_place_of_a_token(emu, N, B, S, G):
    layout = emu.basp_plan_create_groups(N, B, S, N, N, 8, 0, G, 0)
    p = emu.basp_embed_plan_create(layout, B * S, 100, 8, -1, 8, 0, 0)
    assert layout and p
    got = np.full(B * S, -1, dtype=np.int64)
    emu.emu_seq_rows(p, got.ctypes.data)
    assert np.array_equal(got, ic.seq_place(N, B, S, G))
    emu.basp_embed_plan_destroy(p)
    emu.basp_plan_destroy(layout)


@pytest.mark.parametrize("waves", [4, 8])
@pytest.mark.parametrize("row", [2, 6, 48, 100, 2046, 2048, 2050, 4096, 4098, 20000])
@pytest.mark.parametrize("begin,end", [(0, 0), (0, 1), (3, 300), (0, 1025), (64, 5000)])
def test_zeros_cover_every_row_once(emu, begin, end, row, waves):
    seen = np.zeros(max(1, (end - begin) * row), dtype=np.uint8)
    assert emu.emu_zero_cover(begin, end, row, waves, seen.ctypes.data) == 0
    if end > begin:
        assert (seen == 1).all()
