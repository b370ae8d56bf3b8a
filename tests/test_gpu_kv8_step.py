"""The verify step over an 8-bit prefix, its calls together as they are used:
several steps in a row, the page tables turning over on the device between
them, every buffer against a host model made of the oracles."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from helpers import golden_workload, small_case
from helpers_kv8 import assert_attention, bits
from oracle import kv8, pages
from tree_verification_jsv_b200 import jsv, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_jsv_b200 import build
    build.build()
    jsv.load()


def workload(prefixes, trees, seed, spare):
    """A ragged workload with room for the prefixes to grow, and tokens that
    follow the argmax down a chain of each tree."""
    rng = np.random.default_rng(seed)
    case = small_case(trees, prefixes, Hq=8, Hkv=2, D=64, seed=seed)
    extra = spare * len(prefixes)
    table = np.concatenate([case["page_table"], np.full((len(prefixes), spare), -1, np.int32)], 1)
    grow = lambda x: np.concatenate([x, synth.f32_to_bf16_bits(rng.standard_normal((extra,) + x.shape[1:]).astype(np.float32))])
    T, d, V = int(case["node_offsets"][-1]), 64, 300
    wl = synth.Workload(name="small", seed=seed, B=len(prefixes), Hq=8, Hkv=2, D=64, d=d, V=V,
                        prefix_len=case["prefix_len"], node_offsets=case["node_offsets"], parent=case["parent"],
                        match_p=np.zeros(len(prefixes)), page_table=table, num_pages=case["num_pages"] + extra,
                        q=case["q"], k_cache=grow(case["k_cache"]), v_cache=grow(case["v_cache"]),
                        hidden=synth.f32_to_bf16_bits(rng.standard_normal((T, d)).astype(np.float32)),
                        w=synth.f32_to_bf16_bits(rng.standard_normal((V, d)).astype(np.float32)))
    arg, t1, t2 = oracle.lmhead_top2(wl.hidden, wl.w)
    ok, _ = oracle.certify_margin(wl.hidden, wl.w, arg, t1, t2)
    assert ok.all()
    wl.tok_flag = rng.random(T) < 0.8
    wl.tok_uniform = rng.integers(0, V, T).astype(np.int32)
    return wl, synth.plant_tokens(wl, arg), arg


def put_tree(st, model, rng):
    """The next tree's K/V and queries, on the device and in the model."""
    wl = model["wl"]
    for name in ("k_cache", "v_cache"):
        new = synth.f32_to_bf16_bits(rng.standard_normal((wl.T, wl.Hkv, wl.D)).astype(np.float32))
        for b in range(wl.B):
            for j in range(int(wl.node_offsets[b + 1] - wl.node_offsets[b])):
                s = int(model["prefix_len"][b]) + j
                model[name][model["table"][b, s // 16], s % 16] = new[wl.node_offsets[b] + j]
        getattr(st, name).view(torch.int16).copy_(torch.from_numpy(model[name].view(np.int16)))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_in_a_row(fmt, graph):
    from tree_verification_jsv_b200.step import VerifyStepKv8
    rng = np.random.default_rng(3)
    trees = [synth.tiny_tree(np.random.default_rng(9), 40, 12, 3), np.arange(-1, 12), np.array([-1])]
    wl, tokens, arg = workload([90, 0, 47], trees, 5, 8)
    st = VerifyStepKv8(wl, tokens, fmt)
    width, B = wl.page_table.shape[1], wl.B
    nodes = np.diff(wl.node_offsets)
    # the model: what the constructor does, then step after step
    m = dict(wl=wl, table=wl.page_table.copy(), prefix_len=wl.prefix_len.astype(np.int64), k_cache=wl.k_cache.copy(),
             v_cache=wl.v_cache.copy(), ref=np.bincount(wl.page_table[wl.page_table >= 0], minlength=wl.num_pages).astype(np.int32),
             table8=np.full((B, width), -1, np.int32), ref8=np.zeros(B * width, np.int32),
             codes=[np.zeros((B * width, wl.Hkv, 16, wl.D), np.uint8) for _ in range(2)],
             scales=[np.zeros((B * width, wl.Hkv), np.float32) for _ in range(2)])

    def write_full(frm, to):
        assert not pages.alloc(m["ref8"], m["table8"], None, to, True)
        for x, c, s in zip((m["k_cache"], m["v_cache"]), m["codes"], m["scales"]):
            kv8.quantize(x, m["table"], m["table8"], frm, to, c, s, fmt)

    write_full([0] * B, m["prefix_len"])
    assert not pages.trim(m["ref"], m["table"], m["prefix_len"], m["prefix_len"] + nodes)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if graph:
        before = [x.clone() for x in (st.k_cache, st.v_cache)]
        st.capture()
        for x, y in zip((st.k_cache, st.v_cache), before):      # capture ran the step once
            x.copy_(y)
    crossed = 0
    for step in range(7):
        put_tree(st, m, rng)
        torch.cuda.synchronize()
        if graph:
            with torch.cuda.stream(side):
                st.replay()
        elif step % 2:
            with torch.cuda.stream(side):
                st.run(side)
        else:
            out = st.run_host()
        torch.cuda.synchronize()
        assert int(st.status.item()) == 0
        # attention, on the caches as they were; the tables as the model has them
        case = dict(Hq=wl.Hq, Hkv=wl.Hkv, D=wl.D, scale=wl.scale, q=wl.q, prefix_len=m["prefix_len"], parent=wl.parent,
                    node_offsets=wl.node_offsets, page_table=m["table"], page_table8=m["table8"], k_cache=m["k_cache"],
                    v_cache=m["v_cache"], k8=m["codes"][0], v8=m["codes"][1], k_scale=m["scales"][0], v_scale=m["scales"][1])
        assert_attention(synth.bf16_bits_to_f32(bits(st.out)).astype(np.float64), case, fmt, f"step {step}")
        assert np.array_equal(st.argmax.cpu().numpy(), arg)
        ref = oracle.accept_batch(wl.node_offsets, wl.parent, tokens, arg)
        new_len = oracle.kv_compact(m["k_cache"], m["v_cache"], m["table"], m["prefix_len"], [r[0] for r in ref])
        assert np.array_equal(st.new_len.cpu().numpy(), new_len)
        if not graph and not step % 2:
            assert np.array_equal(out["new_len"].numpy(), new_len)
        with torch.cuda.stream(side):
            st.advance(side)
        torch.cuda.synchronize()
        write_full(m["prefix_len"], new_len)
        assert not pages.trim(m["ref"], m["table"], new_len, new_len)
        crossed += int((new_len // 16 > m["prefix_len"] // 16).sum())
        m["prefix_len"] = new_len.astype(np.int64)
        assert not pages.alloc(m["ref"], m["table"], new_len, new_len + nodes, False)
        for got, want in ((st.page_table, m["table"]), (st.page_table8, m["table8"]), (st.refcount, m["ref"]),
                          (st.refcount8, m["ref8"]), (st.k8, m["codes"][0]), (st.v8, m["codes"][1]),
                          (st.k_scale, m["scales"][0]), (st.v_scale, m["scales"][1]), (st.prefix_len, m["prefix_len"])):
            assert np.array_equal(got.cpu().numpy(), want)
        assert np.array_equal(bits(st.k_cache), m["k_cache"]) and np.array_equal(bits(st.v_cache), m["v_cache"])
        assert int(st.status.item()) == 0
    assert crossed >= 3                 # pages moved to the 8-bit cache on the way


def test_step_over_the_8_bit_prefix_accepts_what_the_bf16_step_accepts():
    """The named workload: the walk goes by the LM head, which the attention's
    rounding does not touch, and the outputs stay near the bf16 ones."""
    from tree_verification_jsv_b200.step import VerifyStep, VerifyStepKv8
    wl, tokens, _ = golden_workload("tiny")
    a, b = VerifyStep(wl, tokens), VerifyStepKv8(dataclasses.replace(wl), tokens, "int8")
    for st in (a, b):
        st.run()
    torch.cuda.synchronize()
    assert int(a.status.item()) == int(b.status.item()) == 0
    for name in ("path", "accept_len", "bonus", "new_len"):
        assert torch.equal(getattr(a, name), getattr(b, name))
    # int8 codes: off by at most 2^-8 of a block's largest value, about 4.5 standard deviations
    x, y = a.out.float(), b.out.float()
    assert (x - y).abs().max() <= 8 * 4.5 / 254 * wl.D ** -0.5
