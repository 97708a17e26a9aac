"""The sizes that the GPU tests of the grouped products run at reach every form of every type."""
import pytest

from tests import op_forms

TYPES = ["bf16", "fp16", "fp32"]


def reached(dtype):
    out = {"forward": set(), "dx": set(), "dw": set()}
    for counts, n, k in op_forms.SHAPES:
        for direction, form in op_forms.forms(dtype, op_forms.rows_of(counts), len(counts), n, k).items():
            out[direction].add(form)
    return out


@pytest.mark.parametrize("dtype", TYPES)
def test_every_form_is_reached(dtype):
    forward = ["16x32 thin", "16x128"] + (["32x128 fp32", "32x256 fp32"] if dtype == "fp32" else
                                          ["32x128 span 16", "32x128 span 8", "64x128", "64x256", "128x128", "128x256"])
    got = reached(dtype)
    assert got["forward"] == {(f, whole) for f in forward for whole in (True, False)}
    assert got["dx"] == {(f,) for f in op_forms.DX}
    assert got["dw"] == ({("128x128 fp32",)} if dtype == "fp32" else {("128x128",), ("256x256",)})


def test_spans_repeat():
    """Every forward form runs over more than two of its spans, with whole spans and without."""
    for dtype in TYPES:
        most = {}
        for counts, n, k in op_forms.SHAPES:
            form, whole = op_forms.forms(dtype, op_forms.rows_of(counts), len(counts), n, k)["forward"]
            spans = k / (32 * (8 if form == "16x128" and dtype == "fp32" else op_forms.SPAN[form]))
            most[form, whole] = max(spans, most.get((form, whole), 0))
        assert all(v > 2 for v in most.values()), most


def test_large_gradient_tiles_end_at_every_step():
    """The 128 x 256 form of dx takes 32 of the contraction a step, four steps a turn: every remainder; and the
    256 x 256 form of dW too, over the groups' rows."""
    left, groups = set(), set()
    for counts, n, k in op_forms.SHAPES:
        f = op_forms.forms("bf16", op_forms.rows_of(counts), len(counts), n, k)
        if f["dx"] == ("128x256",):
            left.add(-(-n // 32) % 4)
        if f["dw"] == ("256x256",):
            groups |= {(-(-c // 32) % 4, c > 128) for c in counts}
    assert left == {0, 1, 2, 3}
    assert {r for r, turned in groups if turned} == {0, 1, 2, 3}
