"""Steps over an 8-bit prefix whose trees change size, and the step's pinned
inputs."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from helpers_kv8 import assert_attention, bits
from oracle import kv8, pages
from test_gpu_kv8_step import put_tree, workload
from tree_verification_jsv_b200 import jsv, synth

pytestmark = pytest.mark.gpu

TREES = [synth.tiny_tree(np.random.default_rng(19), 40, 12, 3), np.arange(-1, 12), np.array([-1])]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_jsv_b200 import build
    build.build()
    jsv.load()


@pytest.mark.parametrize("on_device", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_trees_of_other_sizes(graph, on_device):
    from tree_verification_jsv_b200.step import VerifyStepKv8
    rng = np.random.default_rng(4)
    wl, tokens, arg = workload([90, 0, 47], TREES, 5, 8)
    st = VerifyStepKv8(wl, tokens, "e4m3")
    width, B = wl.page_table.shape[1], wl.B
    m = dict(wl=wl, table=wl.page_table.copy(), prefix_len=wl.prefix_len.astype(np.int64), k_cache=wl.k_cache.copy(),
             v_cache=wl.v_cache.copy(), ref=np.bincount(wl.page_table[wl.page_table >= 0], minlength=wl.num_pages).astype(np.int32),
             table8=np.full((B, width), -1, np.int32), ref8=np.zeros(B * width, np.int32),
             codes=[np.zeros((B * width, wl.Hkv, 16, wl.D), np.uint8) for _ in range(2)],
             scales=[np.zeros((B * width, wl.Hkv), np.float32) for _ in range(2)])

    def write_full(frm, to):
        assert not pages.alloc(m["ref8"], m["table8"], None, to, True)
        for x, c, s in zip((m["k_cache"], m["v_cache"]), m["codes"], m["scales"]):
            kv8.quantize(x, m["table"], m["table8"], frm, to, c, s, "e4m3")

    write_full([0] * B, m["prefix_len"])
    assert not pages.trim(m["ref"], m["table"], m["prefix_len"], m["prefix_len"] + np.diff(wl.node_offsets))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if graph:
        before = [x.clone() for x in (st.k_cache, st.v_cache)]
        st.capture_host()
        for x, y in zip((st.k_cache, st.v_cache), before):
            x.copy_(y)
    for step in range(5):
        put_tree(st, m, rng)
        now = m["wl"]
        st.host_inputs()["parent"].copy_(torch.from_numpy(np.ascontiguousarray(now.parent, dtype=np.int32)))
        torch.cuda.synchronize()
        if graph:
            with torch.cuda.stream(side):
                out = st.replay_host()
        else:
            out = st.run_host(side)
        torch.cuda.synchronize()
        assert int(st.status.item()) == 0, f"step {step}"
        case = dict(Hq=wl.Hq, Hkv=wl.Hkv, D=wl.D, scale=wl.scale, q=wl.q, prefix_len=m["prefix_len"], parent=now.parent,
                    node_offsets=now.node_offsets, page_table=m["table"], page_table8=m["table8"], k_cache=m["k_cache"],
                    v_cache=m["v_cache"], k8=m["codes"][0], v8=m["codes"][1], k_scale=m["scales"][0], v_scale=m["scales"][1])
        assert_attention(synth.bf16_bits_to_f32(bits(st.out)).astype(np.float64), case, "e4m3", f"step {step}")
        ref = oracle.accept_batch(now.node_offsets, now.parent, tokens, arg)
        new_len = oracle.kv_compact(m["k_cache"], m["v_cache"], m["table"], m["prefix_len"], [r[0] for r in ref])
        assert np.array_equal(out["new_len"].numpy(), new_len)
        # the next step's trees: each request gets another's
        order = np.roll(np.arange(B), step + 1)
        trees = [TREES[i] for i in order]
        offs = np.concatenate([[0], np.cumsum([len(t) for t in trees])]).astype(np.int32)
        m["wl"] = dataclasses.replace(wl, node_offsets=offs, parent=np.concatenate(trees).astype(np.int32))
        st.advance(side, torch.from_numpy(offs).cuda() if on_device else offs)
        torch.cuda.synchronize()
        write_full(m["prefix_len"], new_len)
        assert not pages.trim(m["ref"], m["table"], new_len, new_len)
        m["prefix_len"] = new_len.astype(np.int64)
        assert not pages.alloc(m["ref"], m["table"], new_len, new_len + np.diff(offs), False)
        for got, want in ((st.page_table, m["table"]), (st.page_table8, m["table8"]), (st.refcount, m["ref"]),
                          (st.refcount8, m["ref8"]), (st.prefix_len, m["prefix_len"]), (st.node_offsets, offs)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert int(st.status.item()) == 0


def test_refused_sizes_and_what_the_host_may_write():
    from tree_verification_jsv_b200.step import VerifyStepKv8
    wl, tokens, _ = workload([90, 0, 47], TREES, 5, 8)
    st = VerifyStepKv8(wl, tokens, "int8")
    assert set(st.host_inputs()) == {"parent", "tokens", "q", "hidden"}
    assert st.h2d_bytes() >= sum(v.numel() * v.element_size() for v in st.host_inputs().values())
    st.run()
    torch.cuda.synchronize()
    before = [x.clone() for x in (st.page_table, st.page_table8, st.refcount, st.prefix_len, st.node_offsets)]
    T = wl.T
    for offs in ([0, 1, T], [0, 1, 2, T - 1], [0, 0, 1, T], [1, 2, 3, T], [0, T - 2, T - 1, T], [0, 5, 4, T],
                 torch.zeros(3, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            st.advance(node_offsets=offs)
    for x, y in zip((st.page_table, st.page_table8, st.refcount, st.prefix_len, st.node_offsets), before):
        assert torch.equal(x, y)


def test_bound_on_the_prefix():
    """By a bound of its own the step gives the same results, and flags a
    prefix that has grown past it."""
    from tree_verification_jsv_b200.step import VerifyStepKv8
    wl, tokens, _ = workload([90, 0, 47], TREES, 5, 300)
    steps = [VerifyStepKv8(wl, tokens, "int8", max_prefix=m) for m in (None, 90)]
    for st in steps:
        st.run()
    torch.cuda.synchronize()
    a, b = steps
    assert a.batch.max_prefix == wl.page_table.shape[1] * 16 - 1 and b.batch.max_prefix == 90
    assert (a.out.float() - b.out.float()).abs().max() <= 2.0 ** -7 * a.out.float().abs().max()
    for name in ("path", "accept_len", "bonus", "new_len"):
        assert torch.equal(getattr(a, name), getattr(b, name))
    for st in steps:
        st.advance()
        st.run()
    torch.cuda.synchronize()
    assert int(a.new_len.max().item()) > 91
    assert int(a.status.item()) == 0 and int(b.status.item()) == jsv.JSV_ERR_DEVICE_INPUT


@pytest.mark.parametrize("bound", [0, 89, 1 << 30])
def test_refused_bounds(bound):
    from tree_verification_jsv_b200.step import VerifyStepKv8
    wl, tokens, _ = workload([90, 0, 47], TREES, 5, 8)
    with pytest.raises(ValueError):
        VerifyStepKv8(wl, tokens, max_prefix=bound)
