"""The chunked form's operand splits on the CPU: its numpy model is within the
room of tests/chunk_cases.py with all parts, and every lost part or product shows."""
import numpy as np
import pytest

from ssm_decode_b200 import synth
from tests import chunk_cases as cases
from tests import many_token_util as U

FAM = {"mamba2": synth.MAMBA2, "gdn": synth.GDN}


def far(family, dk, dv, lead, **lost):
    """The cases whose room the model leaves."""
    out = []
    for name in cases.names(family):
        d, S, out_room, S_room = cases.make(name, family, dk, dv, lead)
        o, S1 = cases.model(family, d, S, **lost)
        ref, ref_S = U.reference(family, S[None], d, [len(o)], [0])
        if (np.abs(o - ref) > out_room).any() or (np.abs(S1 - ref_S[0]) > S_room).any():
            out.append(name)
    return out


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
@pytest.mark.parametrize("lead", [0, 64])
@pytest.mark.parametrize("family", list(FAM))
def test_all_parts_are_within_the_room(family, lead, dk, dv):
    assert far(FAM[family], dk, dv, lead) == []


@pytest.mark.parametrize("family", list(FAM))
def test_every_lost_part_shows(family):
    fam = FAM[family]
    assert "read" in far(fam, 64, 64, 0, cut_S=2)
    assert far(fam, 64, 64, 0, cut_U=2)
    for lost in [(0, 1), (0, 2)] if family == "mamba2" else cases.PAIRS[1:]:
        left = [p for p in cases.PAIRS if p != lost and not (family == "mamba2" and p[1] > lost[1])]
        assert far(fam, 64, 64, 0, pairs=left), lost


def test_dropped_products_are_below_2_to_the_minus_21():
    """x y against its six products, on random values and on those whose second and third parts are largest."""
    r = np.random.default_rng(1)
    x, y = (r.uniform(1, 2, 200_000).astype(np.float32) for _ in "xy")
    worst = np.float32(1 + 2.0 ** -7 - 2.0 ** -23)                    # ones behind the first part's last place
    x[:2], y[:2] = worst, worst
    px, py = cases.parts(x), cases.parts(y)
    assert np.array_equal(sum(px), x.astype(np.float64))
    exact = x.astype(np.float64) * y
    left = np.abs(sum(px[i] * py[j] for i, j in cases.PAIRS) - exact) / exact
    assert left.max() < 2.0 ** -21 and left[0] > 2.0 ** -22


@pytest.mark.parametrize("family", list(FAM))
def test_model_is_the_recurrence(family):
    """The model on random tokens, against the recurrence: the tests' formulas are the kernel's."""
    fam = FAM[family]
    d = U.draw(fam, 150, 2, 1, 64, 64, 2)
    S = np.random.default_rng(2).standard_normal((2, 64, 64)).astype(np.float32)
    o, S1 = cases.model(fam, d, S)
    ref, ref_S = U.reference(fam, S[None], d, [150], [0])
    assert np.abs(o - ref).max() < 1e-6 * np.abs(ref).max() and np.abs(S1 - ref_S[0]).max() < 1e-6 * np.abs(ref_S).max()
