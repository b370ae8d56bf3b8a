"""The largest numbers of rows that the 8-bit cache's and the page pool's calls
take."""
import numpy as np
import pytest
import torch

from helpers_kv8 import dev_i32
from oracle import kv8, pages
from test_gpu_kv8 import QuantRun
from test_gpu_pages import Pool
from tree_verification_jsv_b200 import jsv

pytestmark = pytest.mark.gpu

ROWS = jsv.PAGES_MAX_ROWS


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_jsv_b200 import build
    build.build()
    jsv.load()


def test_quantize_of_the_most_requests_with_several_heads():
    to = [0] * ROWS
    to[0], to[17], to[ROWS - 1] = 33, 16, 50
    r = QuantRun([0] * ROWS, to, "e4m3", 8, 64, seed=80)
    r.check(r.run())
    assert int(r.status.item()) == 0
