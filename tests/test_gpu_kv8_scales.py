"""V scales far apart: a row whose weight lies on a page of small values gets
those values, as exactly as if no other page had larger ones."""
import functools

import numpy as np
import pytest

from helpers_kv8 import Kv8Run, aim, assert_attention_tight, kv8_case
from oracle import kv8
from tree_verification_jsv_b200 import jsv, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_jsv_b200 import build
    build.build()
    jsv.load()


def tree(seed, n):
    return synth.tiny_tree(np.random.default_rng(seed), n, 9, 4)


# name -> (tree, prefix, Hq, Hkv, D, tcgen05 form)
FORMS = {
    "one split": (tree(1, 5), 150, 4, 2, 64, False),
    "splits": (tree(2, 2), 9001, 8, 2, 128, False),
    "16 rows": (tree(3, 8), 9001, 32, 8, 64, False),
    "tiles": (tree(4, 130), 3500, 8, 1, 128, True),
    "tiles, shared out": (tree(5, 12), 40007, 8, 2, 64, True),
}


@functools.lru_cache(maxsize=None)
def made(form, fmt, seed):
    t, P, Hq, Hkv, D, _ = FORMS[form]
    return kv8_case([t], [P], fmt, Hq, Hkv, D, seed=seed, spread=0.0)


def case_of(form, fmt, seed):
    return {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in made(form, fmt, seed).items()}


def check(case, fmt, tiles, what):
    r = Kv8Run(case, fmt)
    r.run()
    got = r.result()
    assert int(r.status.item()) == 0
    assert_attention_tight(got, case, fmt, tiles, what)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("factor", [1e-4, 1e-6, 1e-8, 1e-12])
@pytest.mark.parametrize("pages", [1, 8])
@pytest.mark.parametrize("form", list(FORMS))
def test_weight_on_a_page_of_small_values(form, pages, factor, fmt):
    """One page, or the eight pages of a 128-slot tile, with V scales far below
    the others', and every query on a key there."""
    t, P, Hq, Hkv, D, tiles = FORMS[form]
    case = case_of(form, fmt, 60)
    at = 3 if P < 200 else P // 16 // 2 // 8 * 8 + 3
    small = [at] if pages == 1 else np.arange(at // 8 * 8, at // 8 * 8 + 8)
    case["v_scale"][case["page_table8"][0, small]] *= np.float32(factor)
    aim(case, fmt, 0, at, 5, 200.0)
    check(case, fmt, tiles, f"{form} {factor}")


@pytest.mark.parametrize("form", list(FORMS))
def test_scales_up_and_down_along_the_prefix(form):
    """Flat queries over pages whose V scales rise and fall by 2^40, zeros
    among them; then sharp ones on the smallest."""
    t, P, Hq, Hkv, D, tiles = FORMS[form]
    case = case_of(form, "int8", 60)
    n = P // 16
    swing = 2.0 ** (20 * np.cos(np.arange(n) * (2 * np.pi / min(n, 64))))
    case["v_scale"][case["page_table8"][0, :n]] *= swing[:, None].astype(np.float32)
    case["v_scale"][case["page_table8"][0, 6:n:13]] = 0.0
    check(case, "int8", tiles, form)
    low = int(np.argmin(swing))
    low -= low % 13 == 6
    aim(case, "int8", 0, low, 2, 200.0)
    check(case, "int8", tiles, form + ", sharp")


@pytest.mark.parametrize("scale,code", [(1e38, 1), (1e-36, 100), (2e-37, 127)])
@pytest.mark.parametrize("form", list(FORMS))
def test_scales_at_the_ends_of_their_range(form, scale, code):
    """V scales whose values a bf16 result still holds."""
    t, P, Hq, Hkv, D, tiles = FORMS[form]
    case = case_of(form, "int8", 60)
    case["v8"] = np.where(np.random.default_rng(1).random(case["v8"].shape) < 0.5, code, 256 - code).astype(np.uint8)
    case["v_scale"][:] = scale
    case["v_cache"][:] = 0
    aim(case, "int8", 0, 3, 5, 200.0)
    r = Kv8Run(case, "int8")
    r.run()
    got = r.result()
    want = kv8.decode(case["v8"][case["page_table8"][0, 3], :, 5], "int8") * np.float64(np.float32(scale))
    want = np.repeat(want, Hq // Hkv, axis=0)
    # the output's rounding and as much again for the weight and the value
    assert np.all(np.abs(got - want) <= 2.0 ** -7 * np.abs(want))
