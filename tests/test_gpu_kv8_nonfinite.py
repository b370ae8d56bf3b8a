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


@pytest.mark.parametrize("scale", [np.inf, np.nan])
@pytest.mark.parametrize("form", list(FORMS))
def test_k_scale(form, scale):
    """Codes of zero and an infinite scale make NaN of a key."""
    n, P, Hq, Hkv, D = FORMS[form]
    case = kv8_case([np.arange(-1, n - 1)], [P], "int8", Hq, Hkv, D, seed=71)
    # keys opposite to the queries: the finished sum, scaled, would be minus infinity
    aim(case, "int8", 0, 1, 5, 5.0)
    at = case["page_table8"][0, P // 16 - 2]
    case["k8"][at] = -case["k8"][case["page_table8"][0, 1], :, 5:6]
    case["k_scale"][at, Hkv - 1] = scale
    got = run(case, "int8")
    G = Hq // Hkv
    assert not np.isfinite(got[:, (Hkv - 1) * G:]).any()
    assert np.isfinite(got[:, :(Hkv - 1) * G]).all()


@pytest.mark.parametrize("sign", [0, 0x8000])
@pytest.mark.parametrize("form", list(FORMS))
def test_infinite_key_of_a_node(form, sign):
    """Its score is plus or minus infinity.  Plus: no weight is defined, the
    output is NaN.  Minus: the weight is zero, and the nodes below it are as
    without it."""
    n, P, Hq, Hkv, D = FORMS[form]
    chain = np.arange(-1, n - 1)
    case = kv8_case([chain], [P], "e4m3", Hq, Hkv, D, seed=72)
    at = 0 if n == 2 else 1                            # the node with the infinite key
    rng = np.random.default_rng(5)
    plus = rng.random((n, Hq)) < 0.4
    q9 = np.where(plus, 0.25, -0.25) * (-1 if sign else 1)
    case["q"][:, :, 9] = synth.f32_to_bf16_bits(q9.astype(np.float32))
    without = dict(case)
    parent = chain.copy()
    parent[at + 1:at + 2] = at - 1                     # below it, the tree without that node
    slot = P + at
    case["k_cache"] = case["k_cache"].copy()
    case["k_cache"][case["page_table"][0, slot // 16], slot % 16, :, 9] = INF_BF16 | sign
    got = run(case, "e4m3")
    below = np.arange(n) > at
    assert np.isnan(got[at:][plus[at:]]).all()
    assert np.isfinite(got[:at]).all() and np.isfinite(got[~plus]).all()
    if at > 0:
        without["parent"] = parent.astype(np.int32)
        rows = (below[:, None] & ~plus)[:, :, None] & np.ones(got.shape, bool)
        assert_attention(np.where(rows, got, 0), without, "e4m3", rows=rows)


@pytest.mark.parametrize("n,P,Hq,Hkv,D", [(2, 40, 4, 2, 64), (9, 700, 32, 8, 128), (130, 3500, 8, 1, 64)])
def test_no_finite_score(n, P, Hq, Hkv, D):
    """All scores minus infinity: there are no weights, the output is NaN (a
    node of another request is as ever)."""
    case = kv8_case([np.array([-1]), np.arange(-1, n - 1)], [0, P], "e4m3", Hq, Hkv, D, seed=73)
    case["q"][0, :, 3] = synth.f32_to_bf16_bits(np.full(Hq, -0.5, np.float32))
    case["k_cache"][case["page_table"][0, 0], 0, :, 3] = INF_BF16
    got = run(case, "e4m3")
    assert np.isnan(got[0]).all()
    with np.errstate(all="ignore"):
        assert_attention(got, case, "e4m3", rows=np.arange(len(got)) > 0)


@pytest.mark.parametrize("form", list(FORMS))
def test_nan_key_of_a_node(form):
    n, P, Hq, Hkv, D = FORMS[form]
    case = kv8_case([np.arange(-1, n - 1)], [P], "e4m3", Hq, Hkv, D, seed=74)
    slot = P + n - 1
    case["k_cache"][case["page_table"][0, slot // 16], slot % 16, Hkv - 1, 9] = NAN_BF16
    got = run(case, "e4m3")
    assert np.isnan(got[n - 1, (Hkv - 1) * (Hq // Hkv):]).all() and np.isfinite(got[:n - 1]).all()
