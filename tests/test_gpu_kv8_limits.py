"""The largest numbers of rows that the 8-bit cache's and the page pool's calls
take."""
import numpy as np
import pytest
import torch

from oracle import pages
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


@pytest.mark.parametrize("num", [900, 9000])
def test_the_most_rows_of_a_page_table(num):
    """Alloc, fork, trim and compact with 8,192 rows, with and without enough
    pages for them."""
    rng = np.random.default_rng(num)
    p = Pool(num, ROWS, 3)
    p.ws = torch.full((jsv.jsv_pages_workspace_size(num, ROWS),), 255, dtype=torch.uint8, device="cuda")
    half = ROWS // 2
    length = np.concatenate([rng.integers(0, 20, half), np.zeros(half, int)])
    errors = p.alloc(None, length)
    assert errors == ({pages.NO_PAGES} if num < half else set())
    mapped = np.flatnonzero((p.table >= 0).any(1))
    src = rng.choice(mapped, half)
    p.fork(src, half + rng.permutation(half), np.minimum(length[src], 16))
    p.trim(None, rng.integers(0, 33, ROWS))
    p.compact()
    p.compact(in_place=True)


def test_the_most_forks_in_one_call():
    p = Pool(50, ROWS, 2)
    p.ws = torch.full((jsv.jsv_pages_workspace_size(50, ROWS),), 255, dtype=torch.uint8, device="cuda")
    p.alloc(None, [32] + [0] * (ROWS - 1))
    assert p.fork([0] * ROWS, [(i + 1) % ROWS for i in range(ROWS)], [32] * ROWS) == {pages.DEVICE_INPUT}
    assert (p.table[1:] == p.table[0]).all()
