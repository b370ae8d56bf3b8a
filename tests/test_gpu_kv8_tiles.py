"""Tree attention over an 8-bit prefix at sizes that take the tcgen05 form:
above 32 query rows of a KV head and above 28,000 units of (page, KV head, 8
rows).  The cases in test_gpu_kv8.py stay below."""
import numpy as np
import pytest
import torch

from helpers import bf16
from helpers_kv8 import INF_BF16, NAN_BF16, Kv8Run, assert_attention, kv8_case
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


def units(trees, prefixes, Hq, Hkv):
    """The entry point's own measure of a call, for pools of 3 spare pages."""
    B, most, nodes = len(trees), max(prefixes), max(len(t) for t in trees)
    load = min(1.0, (sum(p // 16 for p in prefixes) + 3 + B) / (B * (most // 16 + 1)))
    rows = nodes * Hq // Hkv
    return rows, load * B * Hkv * ((most + nodes + 15) / 16) * ((rows + 7) // 8)


# name -> (trees, prefixes, Hq, Hkv, D)
CASES = {
    # 1040 rows: four CTAs' 256 and one of 16, whose groups share out the tiles
    "rows_1040": ([tree(1, 130)], [3500], 8, 1, 128),
    "rows_1024_aligned": ([tree(2, 128)], [3584], 8, 1, 64),
    # 40 rows: every CTA's groups share out the tiles
    "rows_40": ([tree(3, 10)], [46003], 8, 2, 64),
    "rows_128_ragged": ([tree(4, 32), tree(5, 9), ROOT1], [16011, 7000, 15], 8, 2, 128),
    # no prefix, less than a page, less than a tile, a page more than a tile,
    # many tiles; trees of one node and of several tiles
    "ragged": ([tree(6, 200), ROOT1, tree(7, 70), tree(8, 5), np.arange(-1, 60), tree(9, 64)],
               [0, 9, 127, 144, 5000, 1600], 8, 2, 128),
    "chain_512": ([np.arange(-1, 511)], [2000], 4, 2, 64),
    "tree_512_g1": ([synth.budget_tree(np.random.default_rng(13), 512, 16, 8)], [1777], 4, 4, 64),
    "g3": ([tree(10, 100), tree(11, 77)], [5000, 4321], 6, 2, 128),
    "g16": ([tree(12, 40), tree(13, 3)], [3001, 4096], 16, 1, 128),
    # one request many times as long as the others: its splits, their one
    "one_long": ([tree(14, 60)] + [tree(20 + i, 20) for i in range(4)], [20000, 16, 200, 0, 33], 8, 2, 64),
}


def run(case, fmt, **kw):
    r = Kv8Run(case, fmt, **kw)
    r.run()
    got = r.result()
    assert int(r.status.item()) == 0
    return got


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("name", list(CASES))
def test_attention(name, fmt):
    trees, pre, Hq, Hkv, D = CASES[name]
    rows, n = units(trees, pre, Hq, Hkv)
    assert rows > 32 and n > 28000
    case = kv8_case(trees, pre, fmt, Hq, Hkv, D, seed=50)
    assert_attention(run(case, fmt), case, fmt, name)


@pytest.mark.parametrize("dual", [False, True])
@pytest.mark.parametrize("q_scale", [0.0, 8.0, 1e-30, 1e20])
def test_flat_sharp_and_extreme_queries(q_scale, dual):
    trees, pre = ([tree(30, 12)], [40007]) if dual else ([tree(30, 130)], [3500])
    case = kv8_case(trees, pre, "int8", 8, 2 if dual else 1, 64, seed=51, q_scale=min(q_scale, 8.0))
    if q_scale > 8:
        case["q"] = bf16(synth.bf16_bits_to_f32(case["q"]) * np.float32(q_scale / 8))
        case["scale"] = float(np.float32(case["scale"] * 8 / q_scale))
    assert_attention(run(case, "int8"), case, "int8")


@pytest.mark.parametrize("dual", [False, True])
@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_scales_far_apart_zero_and_growing(spread, dual):
    trees, pre = ([tree(31, 12)], [40007]) if dual else ([tree(31, 130)], [3500])
    case = kv8_case(trees, pre, "e4m3", 8, 2 if dual else 1, 128, seed=52, spread=spread)
    for name in ("k", "v"):
        case[name + "_scale"][::5] = 0.0
    case["k_scale"] = np.minimum(case["k_scale"], 0.02).astype(np.float32)
    # the reference scale has to follow: page after page twice as large, in places
    order = case["page_table8"][0, 20:30]
    case["v_scale"][order] = (2.0 ** np.arange(-6, 4))[:, None].astype(np.float32) * 1e-2
    assert_attention(run(case, "e4m3"), case, "e4m3")


@pytest.mark.parametrize("n,P", [(400, 1957), (20, 40005)])
def test_what_a_node_does_not_see_does_not_reach_it(n, P):
    parent = np.array([-1] + [0] * (n - 1))
    case = kv8_case([parent, ROOT1], [P, 21], "e4m3", 8 if n < 30 else 4, 2 if n < 30 else 1, 128, seed=53)
    assert units([parent, ROOT1], [P, 21], case["Hq"], case["Hkv"])[1] > 28000
    used = np.zeros(case["k_cache"].shape[:2], dtype=bool)
    for b, m in ((0, n), (1, 1)):
        for s in range(int(case["prefix_len"][b]) // 16 * 16, int(case["prefix_len"][b]) + m):
            used[case["page_table"][b, s // 16], s % 16] = True
    case["k_cache"][~used] = NAN_BF16
    case["v_cache"][~used] = INF_BF16
    s = P + n - 1
    case["v_cache"][case["page_table"][0, s // 16], s % 16, 0, 5] = INF_BF16
    case["k_cache"][case["page_table"][0, (s - 1) // 16], (s - 1) % 16, 0, 9] = NAN_BF16
    got = run(case, "e4m3")
    G = case["Hq"] // case["Hkv"]
    assert np.all(np.isnan(got[n - 2:n, :G]))          # KV head 0's query heads
    clean = np.ones(got.shape, dtype=bool)
    clean[n - 2:n, :G] = False
    got[~clean] = 0
    with np.errstate(all="ignore"):
        assert_attention(got, case, "e4m3", rows=clean)


def test_non_finite_codes_and_scales_are_seen():
    case = kv8_case([tree(32, 130)], [3500], "e4m3", 8, 1, 64, seed=54)
    case["k8"][case["page_table8"][0, 100], 0, 3, 7] = 0x7F
    assert np.isnan(run(case, "e4m3")).all()
    case = kv8_case([tree(32, 130)], [3500], "e4m3", 8, 1, 64, seed=54)
    case["v_scale"][case["page_table8"][0, 0], 0] = np.inf
    assert not np.isfinite(run(case, "e4m3")).any()


@pytest.mark.parametrize("where", ["page_table8", "page_table"])
def test_bad_pages_are_reported_and_other_requests_served(where):
    case = kv8_case([tree(33, 100), tree(34, 80)], [3000, 2500], "int8", 8, 2, 64, seed=55)
    good = {k: v.copy() for k, v in case.items() if isinstance(v, np.ndarray)}
    case[where][0, 20 if where == "page_table8" else 3000 // 16 + 2] = 1 << 20
    r = Kv8Run(case, "int8")
    r.run()
    got = r.result()
    assert int(r.status.item()) == jsv.JSV_ERR_DEVICE_INPUT
    assert_attention(got, {**case, **good}, "int8", rows=np.arange(len(got)) >= 100)


def test_repeats_bit_for_bit_on_other_streams_and_in_graphs():
    cases = [kv8_case([tree(40 + i, 90), tree(42, 16)], [5000 + 17 * i, 900], "e4m3", 8, 2, 128, seed=56 + i) for i in range(2)]
    runs = [Kv8Run(c, "e4m3") for c in cases]
    for r in runs:
        r.run()
    first = [r.result() for r in runs]
    side, graphs = [torch.cuda.Stream() for _ in runs], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.run()
        graphs.append(g)
    for turn in range(2):
        for r in runs:
            r.out[:r.T] = 0
        torch.cuda.synchronize()
        for r, s, g in zip(runs, side, graphs):
            with torch.cuda.stream(s):
                g.replay() if turn else r.run(stream=s)
        for r, f in zip(runs, first):
            assert np.array_equal(r.result(), f)


@pytest.mark.parametrize("seed", range(6))
def test_random_geometry(seed):
    rng = np.random.default_rng(2000 + seed)
    Hkv, G = int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 5, 8]))
    while True:
        B = int(rng.integers(1, 6))
        sizes = [int(rng.integers(1, 200)) for _ in range(B)]
        pre = [int(rng.integers(0, 5000)) for _ in range(B)]
        trees = [tree(int(rng.integers(1 << 30)), n) for n in sizes]
        rows, n = units(trees, pre, Hkv * G, Hkv)
        if rows > 32 and n > 28000:
            break
    D, fmt = int(rng.choice([64, 128])), str(rng.choice(["e4m3", "int8"]))
    case = kv8_case(trees, pre, fmt, Hkv * G, Hkv, D, seed=seed, q_scale=float(rng.choice([1.0, 3.0])))
    assert_attention(run(case, fmt), case, fmt, f"seed {seed}")
