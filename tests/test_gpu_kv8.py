"""The 8-bit cache on the GPU, through the C ABI: tree attention over a prefix
held in 8 bits, and the write of that cache, against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from helpers import bf16
from helpers_kv8 import INF_BF16, NAN_BF16, Kv8Run, assert_attention, bits, dev_bf16, dev_i32, kv8_case
from oracle import kv8
from tree_verification_jsv_b200 import jsv, synth

pytestmark = pytest.mark.gpu

ROOT1 = np.array([-1])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_jsv_b200 import build
    build.build()
    jsv.load()


def tree(seed, n, depth=6, width=3):
    return synth.tiny_tree(np.random.default_rng(seed), n, depth, width)


# name -> (trees, prefixes, Hq, Hkv, D)
CASES = {
    "one_token_no_prefix": ([ROOT1], [0], 4, 2, 128),
    "one_token_15": ([ROOT1], [15], 4, 2, 128),
    "one_token_16": ([ROOT1], [16], 4, 2, 64),
    "one_token_17": ([ROOT1], [17], 4, 1, 128),
    "decode_batch": ([ROOT1] * 7, [0, 1, 31, 32, 333, 64, 1000], 8, 2, 128),
    "decode_long": ([ROOT1], [9001], 8, 2, 128),
    "decode_g16": ([ROOT1] * 2, [700, 80], 16, 1, 64),
    "tree_within_a_page": ([tree(1, 5)], [40], 4, 4, 64),
    "tree_over_pages": ([tree(2, 40)], [29], 8, 2, 128),
    "chain_no_prefix": ([np.arange(-1, 40)], [0], 4, 2, 128),
    "ragged": ([tree(3, 23), ROOT1, tree(4, 70, 9, 4), np.array([-1, 0])], [300, 16, 0, 47], 8, 2, 128),
    "g5": ([tree(5, 60, 8, 4)], [700], 10, 2, 128),
    "g3_d64": ([tree(6, 50), tree(7, 9)], [130, 33], 6, 2, 64),
    "g1": ([tree(8, 150, 9, 3)], [300], 2, 2, 128),
    "rows_33": ([tree(9, 33)], [160], 2, 2, 64),
    "rows_129": ([tree(10, 129)], [512], 1, 1, 128),
    "rows_256": ([tree(11, 64)], [2048 + 5], 4, 1, 128),
    "rows_257": ([tree(12, 257, 12, 4)], [130], 1, 1, 64),
    "tree_512": ([synth.budget_tree(np.random.default_rng(13), 512, 16, 8)], [100], 2, 1, 64),
    "many_requests": ([tree(100 + i, 1 + i % 5, 3, 2) for i in range(40)], [(37 * i) % 211 for i in range(40)], 4, 2, 64),
    "short_and_long": ([tree(200 + i, 30) for i in range(5)], [20, 3000, 16, 0, 200], 8, 2, 128),
}


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("name", list(CASES))
def test_attention(name, fmt):
    trees, pre, Hq, Hkv, D = CASES[name]
    case = kv8_case(trees, pre, fmt, Hq, Hkv, D, seed=11)
    r = Kv8Run(case, fmt)
    r.run()
    got = r.result()
    assert int(r.status.item()) == 0
    assert_attention(got, case, fmt, name)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("q_scale", [0.0, 8.0, 1e-30, 1e20])
def test_attention_flat_sharp_and_extreme_queries(fmt, q_scale):
    case = kv8_case([tree(20, 17), ROOT1], [200, 333], fmt, 8, 2, 128, seed=12, q_scale=min(q_scale, 8.0))
    if q_scale > 8:      # a large query against a small scale: the product is ordinary
        case["q"] = bf16(synth.bf16_bits_to_f32(case["q"]) * np.float32(q_scale / 8))
        case["scale"] = float(np.float32(case["scale"] * 8 / q_scale))
    r = Kv8Run(case, fmt)
    r.run()
    assert_attention(r.result(), case, fmt)


@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_attention_scales_far_apart_and_zero(spread):
    """Scales over several orders of magnitude, some pages zero altogether."""
    case = kv8_case([tree(21, 9), ROOT1], [500, 260], "e4m3", 4, 2, 64, seed=13, spread=spread)
    for name in ("k", "v"):
        case[name + "_scale"][::5] = 0.0
    # keys of a page with a large scale would leave nothing for the others
    case["k_scale"] = np.minimum(case["k_scale"], 0.02).astype(np.float32)
    r = Kv8Run(case, "e4m3")
    r.run()
    assert_attention(r.result(), case, "e4m3")


@pytest.mark.parametrize("rows", [4, 80, 400])
def test_what_a_node_does_not_see_does_not_reach_it(rows):
    """NaN and infinities in the unused slots of the last page, in pages of
    nobody and in one branch of the tree: rows outside that branch are as
    exact as ever, rows in it are not finite."""
    n = rows // 4
    parent = np.array([-1] + [0] * (n - 1)) if n > 1 else ROOT1
    P = 37
    case = kv8_case([parent, ROOT1], [P, 21], "e4m3", 4, 1, 128, seed=14)
    used = np.zeros(case["k_cache"].shape[:2], dtype=bool)
    for b, m in ((0, n), (1, 1)):
        for s in range(int(case["prefix_len"][b]) // 16 * 16, int(case["prefix_len"][b]) + m):
            used[case["page_table"][b, s // 16], s % 16] = True
    for c, bad in (("k_cache", NAN_BF16), ("v_cache", INF_BF16)):
        case[c][~used] = bad
    case["k8"][case["page_table8"].max() + 1:] = 0x7F
    if n > 2:
        s = P + n - 1                                  # the last leaf's own slot
        case["v_cache"][case["page_table"][0, s // 16], s % 16, 0, 5] = INF_BF16
        case["k_cache"][case["page_table"][0, (s - 1) // 16], (s - 1) % 16, 0, 9] = NAN_BF16
    r = Kv8Run(case, "e4m3")
    r.run()
    got = r.result()
    assert int(r.status.item()) == 0
    clean = np.ones(len(got), dtype=bool)
    if n > 2:
        clean[n - 2:n] = False
        assert np.all(np.isnan(got[n - 2:n]))
    with np.errstate(all="ignore"):
        assert_attention(got, case, "e4m3", rows=clean)


def test_non_finite_scale_is_seen():
    case = kv8_case([tree(22, 6), ROOT1], [100, 40], "int8", 4, 2, 64, seed=15)
    case["v_scale"][case["page_table8"][0, 2], 1] = np.nan
    r = Kv8Run(case, "int8")
    r.run()
    got = r.result()
    assert np.all(~np.isfinite(got[:6, 2:])) and np.all(np.isfinite(got[:6, :2])) and np.all(np.isfinite(got[6:]))


@pytest.mark.parametrize("where", ["page_table8", "page_table"])
def test_bad_pages_are_reported_and_other_requests_served(where):
    case = kv8_case([tree(23, 6), tree(24, 4)], [100, 70], "e4m3", 4, 2, 64, seed=16)
    good = {k: v.copy() for k, v in case.items() if isinstance(v, np.ndarray)}
    case[where][0, 2 if where == "page_table8" else 6] = 1 << 20
    r = Kv8Run(case, "e4m3")
    r.run()
    got = r.result()
    assert int(r.status.item()) == jsv.JSV_ERR_DEVICE_INPUT
    assert_attention(got, {**case, **good}, "e4m3", rows=np.arange(len(got)) >= 6)


@pytest.mark.parametrize("fault", ["offsets", "prefix", "parent", "table8"])
def test_malformed_requests_are_reported(fault):
    case = kv8_case([tree(25, 6), tree(26, 4)], [100, 70], "e4m3", 4, 2, 64, seed=17)
    over = {}
    if fault == "offsets":
        case["node_offsets"] = np.array([0, 6, 9], dtype=np.int32)
        over = dict(total_nodes=10)
    elif fault == "prefix":
        over = dict(max_prefix=90)
    elif fault == "parent":
        case["parent"] = case["parent"].copy()
        case["parent"][3] = 4
    else:
        case["page_table8"] = np.ascontiguousarray(case["page_table8"][:, :5])     # 100 tokens need 6
    r = Kv8Run(case, "e4m3", **over)
    r.run()
    torch.cuda.synchronize()
    assert int(r.status.item()) == jsv.JSV_ERR_DEVICE_INPUT


def test_attention_repeats_bit_for_bit_on_other_streams_and_in_graphs():
    cases = [kv8_case([tree(30 + i, 20), ROOT1], [900 + 17 * i, 45], "e4m3", 8, 2, 128, seed=30 + i) for i in range(2)]
    runs = [Kv8Run(c, "e4m3") for c in cases]
    for r in runs:
        r.run()
    first = [r.result() for r in runs]
    side = [torch.cuda.Stream() for _ in runs]
    for r in runs:
        r.out.zero_()
        r.out[r.T:] = 7.0
    torch.cuda.synchronize()
    for _ in range(3):
        for r, s in zip(runs, side):
            r.run(stream=s)
    for r, f in zip(runs, first):
        assert np.array_equal(r.result(), f)
    graphs = []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.run()
        graphs.append(g)
    for r in runs:
        r.out[:r.T] = 0
    torch.cuda.synchronize()
    for s, g in zip(side, graphs):
        with torch.cuda.stream(s):
            g.replay()
    for r, f in zip(runs, first):
        assert np.array_equal(r.result(), f)


@pytest.mark.parametrize("seed", range(6))
def test_attention_random_geometry(seed):
    rng = np.random.default_rng(1000 + seed)
    B = int(rng.integers(1, 9))
    trees = [tree(int(rng.integers(1 << 30)), int(rng.integers(1, 60)), 8, 4) for _ in range(B)]
    pre = [int(rng.integers(0, 900)) for _ in range(B)]
    Hkv, G = int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 4, 7, 16]))
    D, fmt = int(rng.choice([64, 128])), str(rng.choice(["e4m3", "int8"]))
    case = kv8_case(trees, pre, fmt, Hkv * G, Hkv, D, seed=seed, q_scale=float(rng.choice([1.0, 3.0])))
    r = Kv8Run(case, fmt)
    r.run()
    got = r.result()
    assert int(r.status.item()) == 0
    assert_attention(got, case, fmt, f"seed {seed}")


# ---------------------------------------------------------------------------
# The write of the cache
# ---------------------------------------------------------------------------

class QuantRun:
    def __init__(self, frm, to, fmt, Hkv, D, seed=0, width=None):
        rng = np.random.default_rng([seed, 9])
        self.frm, self.to, self.fmt, B = frm, to, fmt, len(to)
        lo, hi = [f // 16 for f in frm], [t // 16 for t in to]
        n16, n8 = sum(-(-t // 16) for t in to) + 1, sum(hi) + 2
        width = width or max(-(-t // 16) for t in to) + 1
        self.table, self.table8 = np.full((B, width), -1, np.int32), np.full((B, max(max(hi), 1)), -1, np.int32)
        p16, p8, a, c = rng.permutation(n16), rng.permutation(n8), 0, 0
        for b in range(B):
            k = -(-to[b] // 16)
            self.table[b, lo[b]:k] = p16[a:a + k - lo[b]]
            self.table8[b, :hi[b]] = p8[c:c + hi[b]]
            a, c = a + k - lo[b], c + hi[b]
        self.kv = [bf16(rng.standard_normal((n16, 16, Hkv, D)) * np.exp(rng.standard_normal((n16, 1, Hkv, 1))))
                   for _ in range(2)]
        self.codes = [rng.integers(0, 256, (n8, Hkv, 16, D)).astype(np.uint8) for _ in range(2)]
        self.scales = [rng.standard_normal((n8, Hkv)).astype(np.float32) for _ in range(2)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, null_from=False):
        B, Hkv, D = len(self.to), self.kv[0].shape[2], self.kv[0].shape[3]
        one = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        t, t8, f, to = dev_i32(self.table), dev_i32(self.table8), dev_i32(self.frm), dev_i32(self.to)
        kv = [dev_bf16(x) for x in self.kv]
        codes, scales = [torch.from_numpy(x).cuda() for x in self.codes], [torch.from_numpy(x).cuda() for x in self.scales]
        batch = jsv.make_batch(B=B, Hq=Hkv, Hkv=Hkv, D=D, max_pages_per_req=t.shape[1], num_pages=kv[0].shape[0],
                               total_nodes=B, max_nodes=1, max_prefix=1, page_table=t, prefix_len=f, node_offsets=one,
                               parent=one, dev_status=self.status)
        cache = jsv.make_kv8(format=self.fmt, num_pages=codes[0].shape[0], max_pages_per_req=t8.shape[1], k=codes[0],
                             v=codes[1], k_scale=scales[0], v_scale=scales[1], page_table=t8)
        jsv.jsv_kv8_quantize(batch, cache, *kv, None if null_from else f, to)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in codes], [x.cpu().numpy() for x in scales]

    def check(self, got, skip=()):
        codes, scales = [x.copy() for x in self.codes], [x.copy() for x in self.scales]
        keep = [b for b in range(len(self.to)) if b not in skip]
        for x, c, s in zip(self.kv, codes, scales):
            kv8.quantize(x, self.table[keep], self.table8[keep], [self.frm[b] for b in keep], [self.to[b] for b in keep],
                         c, s, self.fmt)
        for g, w in zip(got[0] + got[1], codes + scales):
            assert np.array_equal(g, w, equal_nan=g.dtype.kind == "f")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (2, 128), (5, 64), (8, 128)])
def test_quantize_is_exact(fmt, Hkv, D):
    """Codes and scales bit for bit, pages outside the ranges untouched."""
    r = QuantRun([0, 5, 16, 31, 100, 64], [15, 40, 16, 64, 333, 80], fmt, Hkv, D, seed=Hkv)
    r.check(r.run())
    assert int(r.status.item()) == 0


def test_quantize_ties_zeros_and_extremes():
    r = QuantRun([0], [16 * 8], "e4m3", 1, 64, seed=3)
    vals = np.array([448.0, 17, 19, 21, 1.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, -0.0, -17.0, 232, 248], np.float32)
    rng = np.random.default_rng(4)
    for page, factor in zip(r.table[0, :7], [1, 2.0 ** -60, 2.0 ** 110, 3.0, 2.0 ** -118, 0.0, 5.0]):
        x = rng.choice(vals, (16, 1, 64)) * np.float32(factor)
        x[0, 0, 0] = 448 * factor
        for k in range(2):
            r.kv[k][page] = bf16(x)
    r.check(r.run(null_from=True))
    r.fmt = "int8"
    r.check(r.run())
    assert int(r.status.item()) == 0


@pytest.mark.parametrize("bad", [NAN_BF16, INF_BF16, INF_BF16 | 0x8000])
def test_quantize_reports_non_finite_blocks(bad):
    r = QuantRun([0, 0], [48, 40], "int8", 2, 64, seed=5)
    r.kv[1][r.table[0, 1], 7, 1, 33] = bad
    r.check(r.run())
    assert int(r.status.item()) == jsv.JSV_ERR_DEVICE_INPUT


@pytest.mark.parametrize("frm,to,table8", [([50, 0], [40, 32], None), ([-1, 0], [40, 32], None),
                                           ([0, 0], [400, 32], None), ([0, 0], [40, 32], 999)])
def test_quantize_skips_what_is_malformed(frm, to, table8):
    r = QuantRun([0, 0], [40, 32], "e4m3", 2, 64, seed=6)
    r.frm, r.to = frm, to
    if table8:
        r.table8[0, :] = table8
    r.check(r.run(), skip=(0,))
    assert int(r.status.item()) == jsv.JSV_ERR_DEVICE_INPUT


def test_quantize_no_pages_and_many_requests():
    r = QuantRun([0] * 300, [(7 * i) % 50 for i in range(300)], "e4m3", 1, 64, seed=7)
    r.check(r.run())
    r = QuantRun([3, 17], [14, 31], "e4m3", 2, 64, seed=8)
    r.check(r.run())
    assert int(r.status.item()) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_quantized_prefix_gives_the_bf16_attention_within_the_codes_error(fmt):
    """Write the cache with the library's own call, then attend: the result
    differs from attention over the bf16 originals by what the codes round."""
    rng = np.random.default_rng(40)
    case = kv8_case([tree(41, 12)], [250], fmt, 8, 2, 64, seed=41)
    full = 250 // 16
    n16 = case["k_cache"].shape[0] + full
    for c in ("k_cache", "v_cache"):
        case[c] = bf16(rng.standard_normal((n16, 16, 2, 64)))
    case["page_table"][0, :full] = n16 - 1 - np.arange(full)
    r = Kv8Run(case, fmt, num_pages=n16)
    jsv.jsv_kv8_quantize(r.batch, r.cache8, r.dev["k_cache"], r.dev["v_cache"], None, r.dev["prefix_len"])
    r.run()
    got = r.result()
    for name in ("k", "v"):
        case[name + "8"], case[name + "_scale"] = r.dev[name + "8"].cpu().numpy(), r.dev[name + "_scale"].cpu().numpy()
    assert_attention(got, case, fmt)
    from helpers import run_oracle_attention
    exact = run_oracle_attention(case)
    step = 2.0 ** -4 if fmt == "e4m3" else 4.5 / 127 / 2      # of a value; of a block's largest (about 4.5)
    # scores move by at most step * |q| |k| scale per product; loose, for the wiring only
    assert np.abs(got - exact).max() <= 8 * step * np.abs(exact).max() + 8 * step
    assert int(r.status.item()) == 0
