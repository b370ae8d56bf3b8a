"""The oracles of the 8-bit cache and of the page pool against closed forms,
other libraries' conversions and their own invariants."""
import numpy as np
import pytest
import torch

from helpers import run_oracle_attention, small_case
from oracle import bf16_to_f64, kv8, pages
from tree_verification_jsv_b200 import synth


def test_e4m3_codes_are_torch_s():
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    got = kv8.decode(c, "e4m3")
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)]) and np.array_equal(np.isnan(got), np.isnan(want))
    y = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 10.0 ** np.random.default_rng(1).uniform(-4, 2, 4000),
                        (want[:126] + want[1:127]) / 2, want[:127], -want[:127]])
    y = np.clip(y, -448, 448).astype(np.float32)
    assert np.array_equal(kv8.encode(y, "e4m3"), torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_int8_codes_round_half_to_even():
    assert kv8.decode(kv8.encode(np.array([0.5, 1.5, -0.5, -2.5, 127.0, -127.0]), "int8"), "int8").tolist() == \
        [0, 2, 0, -2, 127, -127]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_block_comes_back_within_half_a_step(fmt):
    x = bf16_to_f64(synth.f32_to_bf16_bits(np.random.default_rng(2).standard_normal((16, 64)).astype(np.float32)))
    c, s = kv8.quantize_block(x, fmt)
    back = kv8.decode(c, fmt) * float(s)
    amax = np.abs(x).max()
    half = 2.0 ** -4 * np.abs(x) + amax / 448 * 2.0 ** -10 if fmt == "e4m3" else amax / 127 / 2
    assert np.all(np.abs(back - x) <= half * (1 + 1e-6))


def test_kv8_attention_agrees_with_the_bf16_oracle_on_representable_values():
    """A cache whose bf16 values are code times scale gives the same output."""
    rng = np.random.default_rng(5)
    case = small_case([np.array([-1, 0, 0, 1]), np.array([-1])], [37, 48], Hq=4, Hkv=2, D=64, seed=3)
    n = case["num_pages"]
    for name in ("k", "v"):
        code = rng.integers(-100, 101, (n, 2, 16, 64))
        scale = 2.0 ** rng.integers(-9, -5, (n, 2))
        case[name + "8"], case[name + "_scale"] = code.astype(np.int8).view(np.uint8), scale.astype(np.float32)
        full = (code * scale[:, :, None, None]).transpose(0, 2, 1, 3)
        case[name + "_cache"] = synth.f32_to_bf16_bits(full.astype(np.float32))
    case["page_table8"] = case["page_table"]
    out, mag, _, _ = kv8.tree_attention(case, "int8")
    assert np.allclose(out, run_oracle_attention(case), rtol=1e-12, atol=1e-12)
    assert np.all(mag >= np.abs(out) - 1e-12)


def test_page_pool_keeps_its_counts():
    """Random turns: each count is the number of entries that hold the page,
    a partial page is held once, and compaction keeps the rows' contents."""
    rng = np.random.default_rng(7)
    ref, table = np.zeros(60, np.int32), np.full((6, 12), -1, np.int32)
    length = np.zeros(6, int)

    def check():
        assert np.array_equal(np.bincount(table[table >= 0], minlength=60), ref)

    for turn in range(60):
        for b in range(6):
            if rng.random() < 0.3:
                length[b] = 0
        assert not pages.trim(ref, table, None, length)
        check()
        empty = [b for b in range(6) if length[b] == 0]
        held = [b for b in range(6) if length[b]]
        if held and len(empty) > 1:
            src = rng.choice(held, 1)
            errors, copies = pages.fork(ref, table, src, np.array(empty[:1]), length[src], False)
            if not errors:
                length[empty[0]] = length[src[0]]
                assert (copies[0, 0] >= 0) == (length[src[0]] % 16 != 0)
            check()
        want = np.minimum(length + rng.integers(0, 60, 6), 192)
        errors = pages.alloc(ref, table, length, want, False)
        check()
        if not errors:
            length = want
        errors, t2, r2, moves = pages.compact(ref, table)
        assert not errors and np.array_equal(np.flatnonzero(r2 > 0), np.arange((ref > 0).sum()))
        content = np.arange(60)
        for a, d in moves:
            content[d] = content[a]
        assert np.array_equal(content[t2[table >= 0]], table[table >= 0]) and np.array_equal(t2 >= 0, table >= 0)


def test_alloc_serves_rows_in_order_while_pages_last():
    ref, table = np.zeros(5, np.int32), np.full((4, 8), -1, np.int32)
    assert pages.alloc(ref, table, None, [40, 0, 60, 10], False) == {pages.NO_PAGES}
    assert table[0, :3].tolist() == [0, 1, 2] and (table[1:3] == -1).all() and (table[3] == -1).all()
