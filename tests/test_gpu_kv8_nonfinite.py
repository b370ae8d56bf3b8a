"""Infinities and NaN that a node sees, in every form of the attention over an
8-bit prefix."""
import numpy as np
import pytest

from helpers_kv8 import INF_BF16, NAN_BF16, Kv8Run, aim, assert_attention, kv8_case
from tree_verification_jsv_b200 import jsv, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_jsv_b200 import build
    build.build()
    jsv.load()


# name -> (nodes, prefix, Hq, Hkv, D)
FORMS = {
    "one split": (6, 150, 4, 2, 64),
    "splits": (2, 9001, 8, 2, 128),
    "16 rows": (8, 9001, 32, 8, 64),
    "tiles": (130, 3500, 8, 1, 64),
    "tiles, shared out": (12, 40007, 8, 2, 128),
}


def run(case, fmt):
    r = Kv8Run(case, fmt)
    r.run()
    got = r.result()
    assert int(r.status.item()) == 0
    return got


@pytest.mark.parametrize("what", ["v_scale nan", "v_scale inf", "v code"])
@pytest.mark.parametrize("away", [1, 8, 60])
@pytest.mark.parametrize("form", list(FORMS))
def test_v_whose_weight_underflows(form, away, what):
    """A node sees it all the same: its weight is small, not zero.  Near the
    key that the queries point at, in the next tile, and in another split."""
    n, P, Hq, Hkv, D = FORMS[form]
    case = kv8_case([np.arange(-1, n - 1)], [P], "e4m3", Hq, Hkv, D, seed=70, spread=0.0)
    at = 4 if P < 200 else 16
    away = min(away, 4) if P < 200 else away
    aim(case, "e4m3", 0, at, 5, 600.0)
    pg = case["page_table8"][0, at + away]
    if what == "v code":
        case["v8"][pg, Hkv - 1, 9] = 0x7F
    else:
        case["v_scale"][pg, Hkv - 1] = np.nan if what == "v_scale nan" else np.inf
    got = run(case, "e4m3")
    G = Hq // Hkv
    assert not np.isfinite(got[:, (Hkv - 1) * G:]).any()
    assert np.isfinite(got[:, :(Hkv - 1) * G]).all()
