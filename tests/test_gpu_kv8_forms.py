"""The forms that the attention over an 8-bit prefix chooses from, each by the
library's own account of its choice: every page of a long prefix is seen to
count, and the streaming form with 16 rows a warp at its edges."""
import numpy as np
import pytest
import torch

from helpers_kv8 import INF_BF16, NAN_BF16, Kv8Run, aim, assert_attention, assert_attention_tight, kv8_case
from oracle import kv8
from tree_verification_jsv_b200 import jsv, synth

pytestmark = pytest.mark.gpu

ROOT1 = np.array([-1])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_jsv_b200 import build
    build.build()
    jsv.load()


def tree(seed, n, depth=9, width=4):
    return synth.tiny_tree(np.random.default_rng(seed), n, depth, width)


def with_spare(case, pages):
    """The same pool with pages of nobody behind it, NaN all through."""
    for name in ("k", "v"):
        c, s = case[name + "8"], case[name + "_scale"]
        case[name + "8"] = np.concatenate([c, np.full((pages,) + c.shape[1:], 0x7F, np.uint8)])
        case[name + "_scale"] = np.concatenate([s, np.full((pages,) + s.shape[1:], np.nan, np.float32)])
    return case


def plan(r):
    return jsv.jsv_tree_attention_kv8_plan(r.batch, r.cache8)


# name -> (tree, prefix, Hq, Hkv, D, host bound on the prefix, rows taken together)
LONG = {
    "8 rows, splits": (ROOT1, 9001, 8, 2, 128, None, 8),
    "8 rows, one split": (tree(1, 2), 9605, 8, 2, 64, 1_000_000, 8),
    "16 rows, splits": (tree(2, 8), 9001, 32, 8, 64, None, 16),
    "16 rows, one split": (tree(3, 8), 9605, 32, 8, 128, 1_000_000, 16),
    "tiles": (tree(4, 130), 3500, 8, 1, 128, None, 256),
    "tiles, shared out": (tree(5, 10), 46003, 8, 2, 64, None, 256),
    "tiles, one split": (tree(6, 12), 40007, 8, 2, 64, 4_000_000, 256),
}


def long_case(name, fmt):
    t, P, Hq, Hkv, D, bound, rows = LONG[name]
    case = kv8_case([t], [P], fmt, Hq, Hkv, D, seed=90, spread=0.0)
    over = {} if bound is None else dict(max_prefix=bound)
    return case, over, rows


def check_plan(r, name):
    pl, pages = plan(r), int(r.case["prefix_len"][0]) // 16
    assert pl.rows == LONG[name][6]
    if "one split" in name:
        # one split's pages by its four warps: past the third group of 32
        assert pl.split_units >= pages + 40 if pl.rows < 256 else pl.split_units >= pages // 8 + 4
        assert pl.rows == 256 or pages > 4 * 3 * 32
    elif "splits" in name or "shared" in name:
        assert 2 * pl.split_units < (pages if pl.rows < 256 else pages // 8)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("name", list(LONG))
def test_every_page_counts(name, fmt):
    """Flat queries, and V zero but for D pages at a time, each with a
    dimension of its own: that dimension is the page's alone, so that a page
    lost, taken twice or scaled by another's scale shows in full.  The weights
    are equal; a value is off by its roundings to fp16 (2^-10) and its
    weight's (2^-11), the output by 2^-8."""
    case, over, _ = long_case(name, fmt)
    D, P, Hkv, Hq = case["D"], int(case["prefix_len"][0]), case["Hkv"], case["Hq"]
    full, offs, G = P // 16, case["node_offsets"], Hq // Hkv
    pg = case["page_table8"][0, :full]
    rng = np.random.default_rng(7)
    case["q"][:] = 0
    case["v_cache"][:] = 0
    case["v_scale"] = (0.01 * rng.uniform(0.5, 1.5, case["v_scale"].shape)).astype(np.float32)
    depth = np.zeros(offs[1], int)
    for i, p in enumerate(case["parent"]):
        depth[i] = 1 + (depth[p] if p >= 0 else 0)
    code = kv8.encode(np.array([96.0]), fmt)[0]
    case["v8"][:] = 0
    r = Kv8Run(case, fmt, **over)
    check_plan(r, name)
    for w0 in range(0, full, D):
        here = np.arange(w0, min(w0 + D, full))
        case["v8"][:] = 0
        case["v8"][pg[here], :, :, here % D] = code
        r.dev["v8"].copy_(torch.from_numpy(case["v8"]))
        r.run()
        got = r.result()
        want = np.zeros((Hkv, D))
        want[:, here % D] = 16 * 96.0 * case["v_scale"][pg[here]].astype(np.float64).T
        want = np.repeat(want, G, axis=0)[None] / (P + depth)[:, None, None]
        assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -9) * want), w0
    assert int(r.status.item()) == 0


@pytest.mark.parametrize("name", list(LONG))
def test_keys_and_values_of_one_page_belong_together(name):
    """Sharp queries on keys over the whole prefix, ends of groups and splits
    among them: the output is that key's value."""
    case, over, _ = long_case(name, "int8")
    full = int(case["prefix_len"][0]) // 16
    r = Kv8Run(case, "int8", **over)
    check_plan(r, name)
    for i, lp in enumerate(sorted({x for x in (0, 1, 124, 127, 128, 131, 255, 256, 259, 384, 512, full // 2, full - 2, full - 1)
                                   if x < full})):
        aim(case, "int8", 0, lp, (5 * i) % 16, 200.0)
        r.dev["q"].view(torch.int16).copy_(torch.from_numpy(case["q"].view(np.int16)))
        r.run()
        got = r.result()
        at = case["page_table8"][0, lp]
        v = kv8.decode(case["v8"][at, :, (5 * i) % 16], "int8") * case["v_scale"][at].astype(np.float64)[:, None]
        want = np.repeat(v, case["Hq"] // case["Hkv"], axis=0)[None]
        # 2^-8 of the output, 2^-9 of weight and value; other keys' weights are below e^-60
        assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -9) * np.abs(want) + 1e-20), lp


def wide_run(trees, prefixes, fmt, Hq, Hkv, D, units, seed, spread=0.5):
    """A batch under host bounds that give it ``units`` of (page, KV head, 8
    rows), in a pool with room for them."""
    rows8 = -(-max(len(t) for t in trees) * (Hq // Hkv) // 8)
    pages = -(-units // (len(trees) * Hkv * rows8))
    case = kv8_case(trees, prefixes, fmt, Hq, Hkv, D, seed=seed, spread=spread)
    assert 16 * pages >= max(prefixes)
    return with_spare(case, len(trees) * pages), dict(max_prefix=16 * pages)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nodes,Hq,Hkv,units", [(9, 2, 2, 17000), (3, 8, 2, 17000), (16, 1, 1, 17000), (17, 2, 2, 17000),
                                                (32, 2, 2, 30000), (8, 8, 2, 30000), (5, 14, 2, 20000), (33, 2, 2, 20000),
                                                (50, 1, 1, 20000)])
def test_16_rows(nodes, Hq, Hkv, units, D, fmt):
    """9 to 32 rows of a KV head, and more below the tcgen05 form's border;
    long, short and no prefixes, one with scales far apart."""
    trees = [tree(10, nodes), ROOT1, tree(11, max(nodes - 1, 1)), tree(12, max(nodes // 2, 1))]
    case, over = wide_run(trees, [7003, 0, 15, 800], fmt, Hq, Hkv, D, units, 91, spread=2.0)
    case["k_scale"] = np.minimum(case["k_scale"], 0.02).astype(np.float32)
    r = Kv8Run(case, fmt, **over)
    assert plan(r).rows == 16
    r.run()
    got = r.result()
    assert int(r.status.item()) == 0
    assert_attention_tight(got, case, fmt, False)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nodes,G", [(20, 1), (8, 4)])
def test_16_rows_what_a_node_does_not_see_does_not_reach_it(nodes, G, D):
    parent = np.array([-1] + [0] * (nodes - 1))
    P = 4005
    case, over = wide_run([parent, ROOT1], [P, 21], "e4m3", G, 1, D, 20000, 92)
    used = np.zeros(case["k_cache"].shape[:2], dtype=bool)
    for b, m in ((0, nodes), (1, 1)):
        for s in range(int(case["prefix_len"][b]) // 16 * 16, int(case["prefix_len"][b]) + m):
            used[case["page_table"][b, s // 16], s % 16] = True
    case["k_cache"][~used] = NAN_BF16
    case["v_cache"][~used] = INF_BF16
    s = P + nodes - 1
    case["v_cache"][case["page_table"][0, s // 16], s % 16, 0, 5] = INF_BF16
    case["k_cache"][case["page_table"][0, (s - 1) // 16], (s - 1) % 16, 0, 9] = NAN_BF16
    r = Kv8Run(case, "e4m3", **over)
    assert plan(r).rows == 16
    r.run()
    got = r.result()
    assert int(r.status.item()) == 0
    assert np.all(np.isnan(got[nodes - 2:nodes]))
    clean = np.ones(len(got), dtype=bool)
    clean[nodes - 2:nodes] = False
    with np.errstate(all="ignore"):
        assert_attention(got, case, "e4m3", rows=clean)


def test_16_rows_repeat_bit_for_bit():
    case, over = wide_run([tree(13, 20), tree(14, 7)], [6000, 900], "int8", 2, 2, 128, 20000, 93)
    r = Kv8Run(case, "int8", **over)
    assert plan(r).rows == 16
    r.run()
    first, side = r.result(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.run()
    for turn in range(4):
        r.out[:r.T] = 0
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay() if turn % 2 else r.run()
        assert np.array_equal(r.result(), first)
