"""Cases of the 8-bit cache and device state around them (test-side only)."""
import math

import numpy as np
import torch

from helpers import bf16, small_case
from oracle import kv8
from tree_verification_jsv_b200 import jsv, synth

NAN_BF16 = 0x7FC0
INF_BF16 = 0x7F80


def dev_i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def dev_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits, dtype=np.uint16).view(np.int16)).view(torch.bfloat16).cuda()


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def kv8_case(parents, prefixes, fmt, Hq=4, Hkv=2, D=64, seed=0, q_scale=1.0, spread=0.5):
    """A small case whose full prefix pages are random codes with scales
    spread over e^(+-2 spread), in pages of their own order; the bf16 table's
    entries of those pages hold an index no pool has."""
    case = small_case(parents, prefixes, Hq=Hq, Hkv=Hkv, D=D, seed=seed, q_scale=q_scale * math.sqrt(D))
    rng = np.random.default_rng([seed, 77])
    full = [p // 16 for p in prefixes]
    n8 = sum(full) + 3
    perm, at = rng.permutation(n8), 0
    t8 = np.full((len(prefixes), max(max(full), 1) + 1), -1, dtype=np.int32)
    for b, k in enumerate(full):
        t8[b, :k] = perm[at:at + k]
        case["page_table"][b, :k] = 1 << 30
        at += k
    case["page_table8"] = t8
    for name in ("k", "v"):
        x = rng.standard_normal((n8, Hkv, 16, D))
        s = np.exp(spread * rng.standard_normal((n8, Hkv))).astype(np.float32)
        top = np.abs(x).max(axis=(2, 3), keepdims=True)
        case[name + "8"] = kv8.encode(x * kv8.QMAX[fmt] / top, fmt)
        case[name + "_scale"] = (s * top[:, :, 0, 0] / kv8.QMAX[fmt]).astype(np.float32)
    return case


class Kv8Run:
    """A case's device buffers and descriptors; ``run()`` issues the call."""

    def __init__(self, case, fmt, **over):
        self.case, offs = case, case["node_offsets"]
        self.T, nodes = int(offs[-1]), np.diff(offs)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dev = {k: dev_i32(case[k]) for k in ("page_table", "prefix_len", "node_offsets", "parent", "page_table8")}
        self.dev.update({k: dev_bf16(case[k]) for k in ("q", "k_cache", "v_cache")})
        self.dev.update({k: torch.from_numpy(np.ascontiguousarray(case[k])).cuda() for k in ("k8", "v8", "k_scale", "v_scale")})
        kw = dict(B=len(nodes), Hq=case["Hq"], Hkv=case["Hkv"], D=case["D"], max_pages_per_req=case["page_table"].shape[1],
                  num_pages=case["k_cache"].shape[0], total_nodes=self.T, max_nodes=int(nodes.max()),
                  max_prefix=int(max(case["prefix_len"])), dev_status=self.status,
                  **{k: self.dev[k] for k in ("page_table", "prefix_len", "node_offsets", "parent")})
        kw.update(over)
        self.batch = jsv.make_batch(**kw)
        self.cache8 = jsv.make_kv8(format=fmt, num_pages=case["k8"].shape[0], max_pages_per_req=case["page_table8"].shape[1],
                                   k=self.dev["k8"], v=self.dev["v8"], k_scale=self.dev["k_scale"],
                                   v_scale=self.dev["v_scale"], page_table=self.dev["page_table8"])
        # rows behind the last node, which the call must leave as they were
        self.out = torch.full((self.T + 2, case["Hq"], case["D"]), 7.0, dtype=torch.bfloat16, device="cuda")
        nws = jsv.jsv_tree_attention_kv8_workspace_size(self.batch, self.cache8)
        self.ws = torch.full((max(nws, 256),), 255, dtype=torch.uint8, device="cuda")      # NaN patterns

    def run(self, stream=None):
        d = self.dev
        jsv.jsv_tree_attention_kv8(self.batch, self.cache8, d["q"], d["k_cache"], d["v_cache"], self.case["scale"],
                                   self.out, self.ws, stream=stream)

    def result(self):
        torch.cuda.synchronize()
        got = synth.bf16_bits_to_f32(bits(self.out)).astype(np.float64)
        assert np.all(got[self.T:] == 7.0)
        return got[:self.T]


def assert_attention(got, case, fmt, what="", rows=None):
    """Against the fp64 oracle.  Per element, with A = sum p |v| / sum p and X
    the row's largest scale * sum_d |q_d k_d|:
      2^-8 |o|             the output's rounding to bf16
      2^-8 A               weights of the bf16 pages rounded to bf16 (those of
                           the 8-bit pages to fp16, 2^-11, twice as much again
                           left for the sums)
      2 * D * 2^-23 X A    a score is a sum of D exact products in fp32 (each
                           step off by at most one unit of the magnitudes'
                           sum); a score off by e changes weights by a factor
                           exp(+-e), in the numerator and in the sum
      2^-9 A               exponentials, sums and merge in fp32, the code
                           values scaled in fp16, far below this
      2^-31 W              W = (largest V scale) * sum |V code|.  A weight of an
                           8-bit page is held in fp16 as 2^6 e vs / vref with
                           vref at most the largest V scale; below 2^-14 fp16
                           has a step of 2^-24, so e vs is off by up to
                           2^-25 2^-6 vref.  The sum of the weights is at
                           least 1 (the running maximum is at most the largest
                           score), so the output is off by up to 2^-31 W: what
                           is left where a row's large weights meet zeros"""
    want, A, X, W = kv8.tree_attention(case, fmt)
    tol = 2.0 ** -8 * np.abs(want) + A * (2.0 ** -8 + 2.0 ** -9 + 2 * case["D"] * 2.0 ** -23 * X[:, :, None]) + \
        2.0 ** -31 * W + 1e-30
    err = np.abs(got - want)
    bad = ~(err <= tol)
    if rows is not None:
        bad = bad[rows]
    assert not bad.any(), f"{what}: {bad.sum()} elements off, worst {np.nanmax(err / tol):.2f} of the bound"


def aim(case, fmt, b, page, slot, strength):
    """Every query of request b points at one key of its KV head's 8-bit
    prefix; with keys of about unit normal values the key's score is
    ``strength`` and the others' within about 0.6 of that."""
    s0, s1 = case["node_offsets"][b], case["node_offsets"][b + 1]
    q, G = synth.bf16_bits_to_f32(case["q"]).copy(), case["Hq"] // case["Hkv"]
    for g in range(case["Hkv"]):
        pg = case["page_table8"][b, page]
        k = kv8.decode(case["k8"][pg, g, slot], fmt) * case["k_scale"][pg, g]
        q[s0:s1, g * G:(g + 1) * G] = strength / case["scale"] * k / (k @ k)
    case["q"] = bf16(q)


def assert_attention_tight(got, case, fmt, tiles, what=""):
    """As ``assert_attention``, but what is held in few bits counts by each
    key's own weight and value (``kv8.held_terms``) and not by the request's
    largest scale: a page of small values that has a row's weight to itself
    has to come out as exactly as any other.  The tcgen05 form rounds a V value
    twice to fp16, 2^-10 of itself, which the 2^-9 A leaves room for beside
    its weights' 2^-11."""
    want, A, X, _ = kv8.tree_attention(case, fmt)
    tol = 2.0 ** -8 * np.abs(want) + A * (2.0 ** -8 + 2.0 ** -9 + 2 * case["D"] * 2.0 ** -23 * X[:, :, None]) + \
        kv8.held_terms(case, fmt, tiles) + 1e-30
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} elements off, worst {np.nanmax(err / tol):.2f} of the bound"
