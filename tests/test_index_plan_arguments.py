"""Arguments of the index-driven plans that ctypes alone would let through as
something else (no GPU)."""
import pytest

from sequence_re_layout_amd import binding as b


def test_a_destroyed_layout_is_refused():
    """Not taken for None, which would leave the rows in the order of the ids."""
    layout = b.basp_plan_create(8, 2, 64, 8, 8, 16, mode=b.BASP_MODE_ULYSSES)
    b.basp_plan_destroy(layout)
    with pytest.raises(b.BaspError) as e:
        b.basp_embed_plan_create(layout, 128, 100, 24)
    assert e.value.status == b.BASP_ERR_INVALID


def test_a_layout_is_a_plan_of_the_boundary():
    """The handle of another kind of plan would be read as a basp_plan."""
    for other in (b.basp_embed_plan_create(None, 128, 100, 24), b.basp_expert_plan_create(128, 2, 8, 24)):
        with pytest.raises(TypeError, match="layout"):
            b.basp_embed_plan_create(other, 128, 100, 24)
    assert b.basp_embed_plan_create(None, 128, 100, 24).info["T"] == 128
