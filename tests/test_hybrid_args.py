"""hybrid_step hands every entry to its optimizer, whatever holds the list, and refuses before anything is enqueued (no GPU is needed)."""
import pytest

from test_layer_args import ops, torch  # noqa: F401 (fixtures)


@pytest.fixture
def seen(ops, monkeypatch):
    calls = []
    for name in ("muon_step_grouped", "adamw_step", "adamw8_step"):
        monkeypatch.setattr(ops, name, lambda *a, _n=name, **k: calls.append((_n, a, k)))
    return calls


@pytest.mark.parametrize("held", [list, tuple, iter, lambda v: (e for e in v), lambda v: map(tuple, v)], ids=["list", "tuple", "iter", "generator", "map"])
def test_entries_of_both_kinds_from_anything_that_can_be_iterated(torch, ops, seen, held):
    p = [torch.zeros(4) for _ in range(3)]
    s = [ops.adamw8_state(t) for t in p]
    entries = [(p[0], p[0], s[0]), (p[1], p[1], p[1], p[1]), (p[2], p[2], s[2])]
    ops.hybrid_step([], held(entries), muon={}, adamw=dict(lr=1e-3, step=2, bias_correction=True), seed=5)
    assert [c[0] for c in seen] == ["adamw_step", "adamw8_step"]
    assert [len(c[1][0]) for c in seen] == [1, 2]
    assert seen[1][1][0][0] is p[0] and seen[1][1][0][1] is p[2] and seen[1][2]["seed"] == 5


def test_a_step_on_the_device_with_an_iterator(torch, ops, seen):
    p, step = torch.zeros(4), torch.tensor(1)
    with pytest.raises(ValueError, match="on the host"):
        ops.hybrid_step([], iter([(p, p, p, p)]), muon={}, adamw=dict(lr=1e-3, step=step, bias_correction=True))
    ops.hybrid_step([], iter([(p, p, ops.adamw8_state(p))]), muon={}, adamw=dict(lr=1e-3, step=step, bias_correction=True))
    assert [c[0] for c in seen] == ["adamw8_step"]


def test_refusals_come_before_the_first_update(torch, ops, seen):
    p = torch.zeros(4)
    s = ops.adamw8_state(p)
    with pytest.raises(TypeError, match="step"):
        ops.hybrid_step([(p, p, p)], [(p, p, p, p), (p, p, s)], muon={}, adamw=dict(lr=1e-3))
    for entry in ((p, p), (p, p, *s[:3]), ()):
        with pytest.raises(ValueError, match="entry 1"):
            ops.hybrid_step([(p, p, p)], [(p, p, p, p), entry], muon={}, adamw=dict(lr=1e-3, step=1))
    assert not seen
    ops.hybrid_step([], [], muon={}, adamw={})
    ops.hybrid_step([], None, muon={}, adamw={})
    assert not seen


def test_entries_that_are_iterators_and_no_adamw(torch, ops, seen):
    p = torch.zeros(4)
    s = ops.adamw8_state(p)
    ops.hybrid_step([], (iter(e) for e in [(p, p, s), (p, p, p, p)]), muon={}, adamw=dict(lr=1e-3, step=2))
    assert [(c[0], len(c[1][0])) for c in seen] == [("adamw_step", 1), ("adamw8_step", 1)]
    ops.hybrid_step([(p, p, p)], [], muon={}, adamw=None)                    # nothing for AdamW to do
    assert seen[-1][0] == "muon_step_grouped"
