"""The D = 128 backward kernel's barrier protocol over packed sequences with a window, where tiles end their sequence
and the rows behind it are zeroed: K and V land on a barrier of their own, the loader zeroes them after the unit's
first Q and dO are on their way and then arrives on the barrier that the other roles wait for; the key-row warps zero
Q and dO themselves, once S^T and dP^T are formed and before they publish P^T. The model of
test_bwd_barrier_protocol.py with such producers and key-row warps."""
import random

import pytest

import test_bwd_barrier_protocol as model

STAGES = model.STAGES


def _with_cuts(cut, early=False):
    """_roles whose producer and key-row warps take a tile that ends its sequence where ``cut()`` says so. ``early``:
    dV is let go before dP^T is formed from the dO that is being zeroed (wrong)."""
    plain = model._roles

    def producer(ops):
        pairs, held = 0, False
        for op in ops:
            name = op[1] if op[0] == "async" else ""
            if name == "KVFull" and cut():
                yield ("async", "Cut")
                held = True
                continue
            yield op
            if name.startswith("DOFull") and held:
                yield ("wait", "Cut", pairs)
                pairs += 1
                held = False
                yield ("arrive", "KVFull")

    def key_rows(ops):
        J, wait_dp = 0, None
        for op in ops:
            if op[0] == "arrive" and op[1].startswith("PTFull") and cut():
                st, b = J % STAGES, J & 1
                yield ("wait", f"QFull{st}", J // STAGES)
                yield ("wait", f"DOFull{st}", J // STAGES)
                if early:
                    yield op
                yield ("wait", f"DPFull{b}", J >> 1)
                yield ("zeroed", J)
                if not early:
                    yield op
            else:
                yield op
            if op[0] == "arrive" and op[1].startswith("PFull"):
                J += 1

    def roles(units, **kw):
        load, s_issuer, products, rows, *others = plain(units, **kw)
        return [producer(load), s_issuer, products, key_rows(rows), *others]

    return roles


@pytest.mark.parametrize("share", [0.1, 0.5, 1.0])
@pytest.mark.parametrize("case", range(6))
def test_cut_tiles_have_no_deadlock_aliasing_or_overwrite(monkeypatch, case, share):
    rnd = random.Random(case)
    monkeypatch.setattr(model, "_roles", _with_cuts(lambda: rnd.random() < share))
    for seed in range(80):
        units = [rnd.choice([0, 1, 1, 2, 3, 5, 9, 17]) for _ in range(rnd.randrange(1, 10))]
        assert model.simulate(units, seed) == "ok", (units, seed)


def _dv_before_zeroed(ops_by_role):
    """Runs the roles' orders one step at a time; whether a PTFull arrival can precede its sub-step's zeroing."""
    J = 0
    for op in ops_by_role:
        if op[0] == "arrive" and op[1].startswith("PTFull"):
            return True
        if op == ("zeroed", J):
            return False
    return False


def test_p_is_published_after_the_zeroing():
    rows = _with_cuts(lambda: True)([3])[3]
    assert not _dv_before_zeroed(rows)
    assert _dv_before_zeroed(_with_cuts(lambda: True, early=True)([3])[3])
