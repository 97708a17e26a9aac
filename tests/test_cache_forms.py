"""The plans that the GPU tests of the cache run at reach every kernel, in each state that a sequence can be in."""
import pytest

from tests import cache_forms as forms
from tests import cache_reference as ref


def test_the_border_is_the_librarys():
    assert forms.rules().few() == forms.FEW
    assert [forms.FORMS[forms.rules().form(r, s)] for r, s in ((16, 1), (17, 1), (128, 9), (129, 1), (129, 2))] == \
        ["tokens of 16 rows", "tokens of 32 rows", "tokens of 32 rows", "rows", "both"]


@pytest.mark.parametrize("group", [1, 2])
def test_both_kernels_meet_every_state(group):
    """Missing pages, none, lengths past the table, rows before the first token, of causal tiles that are many."""
    plan = forms.awkward()
    assert forms.form(plan, group) == "both"
    for seqs in (forms.by_rows(plan, group), forms.by_tokens(plan, group)):
        holes = [s for s in seqs if any(plan.page_at(s, p) < 0 for p in range(0, max(0, plan.lengths[s]), plan.page))]
        assert any(plan.page_at(s, 0) >= 0 for s in holes) and any(plan.page_at(s, 0) < 0 for s in holes)
        assert any(plan.lengths[s] > plan.max_pages * plan.page for s in seqs) and any(plan.lengths[s] < 0 for s in seqs)
        assert any(0 < plan.lengths[s] < plan.new[s] for s in seqs)
    assert plan.offsets[0] > 0 and plan.offsets[-1] < plan.tokens
    assert any(plan.new[s] * group > 2 * forms.FEW and plan.lengths[s] < plan.new[s] for s in forms.by_rows(plan, group))


def test_a_sequence_by_itself():
    for spec in forms.ALONE.values():
        assert forms.form(forms.alone(spec), 1) == "rows" and forms.by_rows(forms.alone(spec), 1) == [0]


def test_many_heads_take_both_kernels():
    plan = ref.Plan(forms.MANY_HEADS, 32)
    assert forms.form(plan, 1) == "both" and forms.by_rows(plan, 1) == [0] and forms.by_tokens(plan, 1) == [1]


def test_append_and_read_take_several_turns():
    """From so many tokens on a workgroup goes over its heads: several turns, the last one whole and in part, of every
    width; and below, none. 96 values are appended unit by unit, without turns."""
    at = [sum(n for n, _ in spec) for spec in forms.TOKENS]
    assert at[:2] == [1023, 1024]
    rest = {d: set() for d in (64, 96, 128, 192, 256)}
    for heads, kv in forms.HEADS:
        for d in rest:
            rows, lanes = heads + 2 * kv, 128
            assert forms.rules().append(1023, rows, d) == forms.rules().read(1023, kv, d) == 1
            assert forms.rules().append(1024, rows, d) > 1 and forms.rules().read(1024, kv, d) > 1
            rest[d] |= {("append", rows % (lanes // (d // 16)) == 0), ("read", 2 * kv * (d // 8) % lanes == 0)}
    every = {(call, whole) for call in ("append", "read") for whole in (True, False)}
    assert all(r == every or d in (96, 192) and r == every - {("append", True)} for d, r in rest.items())
    pairs = {(d, r, i): bool(forms.rules().pairs(d, r, i)) for d in rest for r in (0, d // 2, d) for i in (0, 1)}
    assert set(pairs.values()) == {True, False} and pairs[128, 64, 0] and not pairs[64, 32, 0] and not pairs[96, 0, 0]
