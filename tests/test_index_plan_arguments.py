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


WIDE = 1 << 32          # a multiple of it is cut off by a 32-bit argument
EXPERTS = dict(T=16, K=2, E=8, D=24, align=4, id_bytes=8, dtype=b.BASP_BF16, weight_dtype=b.BASP_FP32)
EMBED = dict(T=16, V=100, D=24, padding=3, id_bytes=8, dtype=b.BASP_BF16, grad_dtype=b.BASP_FP32)


@pytest.mark.parametrize("name", ["K", "E", "align", "id_bytes", "dtype", "weight_dtype"])
@pytest.mark.parametrize("by", [WIDE, -WIDE])
def test_expert_plans_take_no_part_of_a_number(name, by):
    assert b.basp_expert_plan_create(**EXPERTS).info[name] == EXPERTS[name]
    with pytest.raises(ValueError, match=name):
        b.basp_expert_plan_create(**{**EXPERTS, name: EXPERTS[name] + by})


@pytest.mark.parametrize("name", ["id_bytes", "dtype", "grad_dtype"])
@pytest.mark.parametrize("by", [WIDE, -WIDE])
def test_embed_plans_take_no_part_of_a_number(name, by):
    assert b.basp_embed_plan_create(None, **EMBED).info[name] == EMBED[name]
    with pytest.raises(ValueError, match=name):
        b.basp_embed_plan_create(None, **{**EMBED, name: EMBED[name] + by})


@pytest.mark.parametrize("by", [1 << 64, -(1 << 64)])
def test_sizes_beyond_64_bits(by):
    for name in ("T", "D"):
        with pytest.raises(ValueError, match=name):
            b.basp_expert_plan_create(**{**EXPERTS, name: EXPERTS[name] + by})
    for name in ("T", "V", "D", "padding"):
        with pytest.raises(ValueError, match=name):
            b.basp_embed_plan_create(None, **{**EMBED, name: EMBED[name] + by})
