"""The limits of attention plans that include/basp.h states, met and passed by
one (no GPU)."""
import pytest

from sequence_re_layout_amd import binding as b


def status(order, Hq, d, S=1, queries=1, dtype=b.BASP_BF16):
    layout = b.basp_plan_create_groups(1, 1, S, Hq, 1, d, dtype, 1, order)
    try:
        b.basp_attention_plan_create(layout, queries, 1)
    except b.BaspError as e:
        return e.status
    return b.BASP_OK


@pytest.mark.parametrize("order", [b.BASP_LAYOUT_HEAD_MAJOR, b.BASP_LAYOUT_TOKEN_MAJOR])
def test_bytes_of_a_token(order):
    assert status(order, 1 << 16, 128) == b.BASP_OK
    assert status(order, (1 << 16) + 1, 128) == b.BASP_ERR_UNSUPPORTED
    assert status(order, 1 << 15, 128, dtype=b.BASP_FP32) == b.BASP_OK
    assert status(order, (1 << 15) + 1, 128, dtype=b.BASP_FP32) == b.BASP_ERR_UNSUPPORTED
    assert status(order, (1 << 23) - 1, 1) == b.BASP_OK


def test_columns():
    assert status(0, 8, 1, S=1 << 27, queries=(1 << 27) - 1) == b.BASP_OK
    assert status(0, 8, 1, S=1 << 27, queries=1 << 27) == b.BASP_ERR_UNSUPPORTED
