"""Further refusals of the 8-bit cache's entry points (no GPU)."""
import ctypes

import pytest

from test_kv8_abi import INVALID, UNSUPPORTED, attention, batch, cache, lib  # noqa: F401
from tree_verification_jsv_b200 import jsv


@pytest.mark.parametrize("scale", [2.4e38, 2.9e38, 3.4e38])
def test_scale_whose_base_two_form_overflows(lib, scale):  # noqa: F811
    assert attention(lib, batch(), cache(), scale=scale) == INVALID


def test_plan(lib):  # noqa: F811
    """Its refusals are the attention's; the form follows rows and length."""
    b = batch(max_nodes=8, total_nodes=8, Hq=32, Hkv=8, max_prefix=32, max_pages_per_req=4000)
    assert jsv.jsv_tree_attention_kv8_plan(b, cache()).rows == 8
    long8 = dict(num_pages=2048, max_pages_per_req=2048)
    b = batch(max_nodes=8, total_nodes=8, Hq=32, Hkv=8, max_prefix=32763, max_pages_per_req=4000)
    pl = jsv.jsv_tree_attention_kv8_plan(b, cache(**long8))
    assert pl.rows == 16 and pl.splits >= 1 and pl.splits * pl.split_units >= 32763 // 16
    b = batch(max_nodes=256, total_nodes=256, Hq=32, Hkv=8, max_prefix=16384, max_pages_per_req=4000)
    assert jsv.jsv_tree_attention_kv8_plan(b, cache(**long8)).rows == 256
    for bad in (batch(D=96), batch(B=40000, total_nodes=40000)):
        assert lib.jsv_tree_attention_kv8_plan(ctypes.byref(bad), ctypes.byref(cache()), ctypes.byref(pl)) == UNSUPPORTED
    assert lib.jsv_tree_attention_kv8_plan(ctypes.byref(b), ctypes.byref(cache()), None) == INVALID
    assert lib.jsv_tree_attention_kv8_plan(ctypes.byref(b), None, ctypes.byref(pl)) == INVALID
