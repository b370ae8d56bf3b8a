"""Cases of the 8-bit key/value cache and of the page pool, with their plain forms.

Four operators, each measured as a user's program calls it:

  attn     tree attention over a prefix whose full 16-token pages are held in
           8 bits (e4m3 or int8 codes, one scale for each page and KV head);
           the last, partial page and the tree's own slots are bf16
  quant    the write of that cache: full pages of the bf16 cache to codes and
           scales
  fork     one turn of a serving loop's page bookkeeping: drop the pages past
           each row's kept length, fork rows (full pages shared, the partial
           one copied), map the next tree's pages, copy the page contents
  compact  plan moving the used pages to the front of the pool, and the copy

A case's sizes for each request come from its own numbers (``shape``), its
values from the seed.
"""
import math
import random

import torch

own = False

PAGE = 16
QMAX = {"e4m3": 448.0, "int8": 127.0}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the smallest verify step of the framework's configurations: latency
        dict(name="attn tiny tree", op="attn", fmt="e4m3", B=1, Hq=2, Hkv=1, D=64, nodes_lo=16, nodes_hi=16,
             prefix_lo=128, prefix_hi=128, shape=1),
        # plain decoding of a ragged batch, one token a request: bound by the cache's bytes
        dict(name="attn decode batch", op="attn", fmt="int8", B=16, Hq=32, Hkv=8, D=128, nodes_lo=1, nodes_hi=1,
             prefix_lo=512, prefix_hi=8192, shape=2),
        # one long request, a small tree: the split along the cache
        dict(name="attn 8 nodes, 32768", op="attn", fmt="e4m3", B=1, Hq=32, Hkv=8, D=128, nodes_lo=8, nodes_hi=8,
             prefix_lo=32763, prefix_hi=32763, shape=3),
        # a 256-node tree over one 16384-token request
        dict(name="attn tree 256", op="attn", fmt="int8", B=1, Hq=32, Hkv=8, D=128, nodes_lo=256, nodes_hi=256,
             prefix_lo=16384, prefix_hi=16384, shape=4),
        # the ragged batch of 16 requests, 32 to 128 nodes each
        dict(name="attn ragged 16", op="attn", fmt="e4m3", B=16, Hq=32, Hkv=8, D=128, nodes_lo=32, nodes_hi=128,
             prefix_lo=512, prefix_hi=8192, shape=5),
        # the largest: four 512-node trees over 32768-token prefixes
        dict(name="attn 4 x 512 nodes", op="attn", fmt="e4m3", B=4, Hq=32, Hkv=4, D=128, nodes_lo=512, nodes_hi=512,
             prefix_lo=32768, prefix_hi=32768, shape=6),
        # after a verify step: each request has accepted a few tokens, some completed a page
        dict(name="quant after a step", op="quant", fmt="e4m3", B=16, Hkv=8, D=128, from_lo=512, from_hi=8192,
             new_lo=1, new_hi=17, shape=7),
        # after a prefill: every full page of four prompts
        dict(name="quant prefill", op="quant", fmt="int8", B=4, Hkv=8, D=128, from_lo=0, from_hi=0,
             new_lo=9001, new_hi=16384, shape=8),
        # one prompt forked into four samples
        dict(name="fork 1 into 4", op="fork", parents=1, children=4, len_lo=2040, len_hi=2040, nodes=64, layers=2,
             Hkv=8, D=128, shape=9),
        # a batch forked: 16 prompts, four samples each, four layers' caches
        dict(name="fork 16 into 64", op="fork", parents=16, children=4, len_lo=512, len_hi=8192, nodes=128, layers=4,
             Hkv=8, D=128, shape=10),
        # a small pool with holes
        dict(name="compact small", op="compact", rows=8, len_lo=100, len_hi=1000, free=0.4, layers=1, Hkv=2, D=64,
             shape=11),
        # a large pool, a third of it free
        dict(name="compact large", op="compact", rows=32, len_lo=512, len_hi=8192, free=0.35, layers=2, Hkv=8, D=128,
             shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    shape = rng.randrange(1 << 30)
    op = rng.choice(["attn", "attn", "attn", "quant", "fork", "compact"])
    if op == "attn":
        Hq, Hkv = rng.choice([(2, 1), (4, 2), (4, 4), (10, 2), (16, 2), (16, 1), (32, 8), (32, 4)])
        D = rng.choice([64, 128, 128])
        while True:
            B, hi, pre = _log(rng, 1, 48), _log(rng, 1, 512), _log(rng, 1, 40000)
            if B * hi * pre * Hq <= 4 * 512 * 32768 * 32 and B * hi * Hq * pre <= 2.2e9:
                break
        return dict(op="attn", fmt=rng.choice(["e4m3", "int8"]), B=B, Hq=Hq, Hkv=Hkv, D=D,
                    nodes_lo=rng.randint(1, hi), nodes_hi=hi, prefix_lo=rng.randint(0, pre), prefix_hi=pre, shape=shape)
    if op == "quant":
        while True:
            new = _log(rng, 1, 16384)
            B = _log(rng, 1, 32) if new < 2048 else _log(rng, 1, 4)
            frm = 0 if rng.random() < 0.3 else _log(rng, 1, 8192)
            case = dict(op="quant", fmt=rng.choice(["e4m3", "int8"]), B=B, Hkv=rng.choice([1, 2, 4, 8]),
                        D=rng.choice([64, 128]), from_lo=rng.randint(0, frm), from_hi=frm, new_lo=rng.randint(1, new),
                        new_hi=new, shape=shape)
            if any(b // PAGE > a // PAGE for a, b in zip(*_sizes(case))):  # some page is completed
                return case
    if op == "fork":
        ln = _log(rng, 1, 8192)
        return dict(op="fork", parents=_log(rng, 1, 16), children=_log(rng, 1, 8), len_lo=rng.randint(1, ln), len_hi=ln,
                    nodes=_log(rng, 1, 512), layers=rng.choice([1, 2, 4]), Hkv=rng.choice([1, 2, 4, 8]),
                    D=rng.choice([64, 128]), shape=shape)
    ln = _log(rng, 16, 8192)
    return dict(op="compact", rows=_log(rng, 1, 32), len_lo=rng.randint(1, ln), len_hi=ln,
                free=round(rng.uniform(0.05, 0.7), 3), layers=rng.choice([1, 2]), Hkv=rng.choice([1, 2, 4, 8]),
                D=rng.choice([64, 128]), shape=shape)


def _sizes(case):
    """Per-request host sizes, from the case alone."""
    r = random.Random(case["shape"])
    if case["op"] == "attn":
        n = [r.randint(case["nodes_lo"], case["nodes_hi"]) for _ in range(case["B"])]
        p = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["B"])]
        return n, p
    if case["op"] == "quant":
        a = [r.randint(case["from_lo"], case["from_hi"]) for _ in range(case["B"])]
        return a, [x + r.randint(case["new_lo"], case["new_hi"]) for x in a]
    if case["op"] == "fork":
        return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["parents"])]
    return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["rows"])]


def _up(x):
    return -(-x // PAGE)


def work(case):
    if case["op"] == "attn":
        n, p = _sizes(case)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        pages = sum(x // PAGE for x in p)
        tail = sum(x % PAGE + m for x, m in zip(p, n))
        by = 2 * pages * Hkv * (PAGE * D + 4) + tail * Hkv * D * 4 + sum(n) * (Hq * D * 4 + 4) + pages * 4
        return {"bytes": by, "flops": 4 * Hq * D * sum(m * (x + 1) for x, m in zip(p, n))}
    if case["op"] == "quant":
        pages = sum(b // PAGE - a // PAGE for a, b in zip(*_sizes(case)))
        el = pages * case["Hkv"] * PAGE * case["D"]
        return {"bytes": 2 * (3 * el + 4 * pages * case["Hkv"]) + 8 * pages + 8 * case["B"], "flops": 6 * el}
    page = PAGE * case["Hkv"] * case["D"] * 2
    if case["op"] == "fork":
        ln = _sizes(case)
        rows = case["parents"] * (1 + case["children"])
        shared = sum(_up(x) for x in ln) * case["children"]
        new = rows * _up(case["nodes"])
        copies = sum(1 for x in ln if x % PAGE) * case["children"]
        return {"bytes": 16 * shared + 8 * new + 2 * copies * page * 2 * case["layers"], "flops": 0}
    pages, used, num = _compact_pages(case)
    return {"bytes": 8 * num + 8 * pages + 2 * 2 * case["layers"] * page * (used * (num - used) // num), "flops": 0}


def _compact_pages(case):
    """(table entries, used pages, pool pages) of a compaction case: every odd
    row shares the first half of the row before it."""
    need = [_up(x) for x in _sizes(case)]
    own_pages = sum(k - (min(need[i - 1], k) // 2 if i % 2 else 0) for i, k in enumerate(need))
    return sum(need), own_pages, int(own_pages / (1 - case["free"])) + 2


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(need, num_pages, gen, first=None):
    """Rows of a page table with need[b] entries from first[b] on, drawn from
    a random order of the pool's pages; -1 elsewhere."""
    first = first or [0] * len(need)
    width = max(max(f + k for f, k in zip(first, need)), 1)
    perm = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    t = torch.full((len(need), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        t[b, first[b]:first[b] + k] = perm[at:at + k]
        at += k
    return t


def _kv(pages, Hkv, D, gen):
    """Key or value rows [pages][16][Hkv][D] in bf16: normal values with a
    channel's own offset and a page's own size, a few large."""
    x = torch.randn(pages, PAGE, Hkv, D, generator=gen, device="cuda")
    x += 0.5 * torch.randn(1, 1, Hkv, D, generator=gen, device="cuda")
    x *= torch.exp(0.4 * torch.randn(pages, 1, Hkv, 1, generator=gen, device="cuda"))
    return x.to(torch.bfloat16)


def _codes(x, fmt):
    """Codes [pages][Hkv][16][D] and scales [pages][Hkv] of bf16 rows."""
    y = x.float().transpose(1, 2)
    amax = y.abs().amax(dim=(2, 3))
    a = amax[:, :, None, None].clamp_min(1e-30)
    y = y * QMAX[fmt] / a
    c = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" \
        else y.round().to(torch.int8).view(torch.uint8)
    return c.contiguous(), amax / QMAX[fmt]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    host = random.Random(seed)
    return {"attn": _prepare_attn, "quant": _prepare_quant, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, gen, host)


def _prepare_attn(case, gen, host):
    n, p = _sizes(case)
    Hq, Hkv, D, B = case["Hq"], case["Hkv"], case["D"], case["B"]
    T = sum(n)
    offs = [0]
    for m in n:
        offs.append(offs[-1] + m)
    parent = [x for m in n for x in [-1] + [host.randint(max(0, i - 12), i - 1) for i in range(1, m)]]
    full = [x // PAGE for x in p]
    pages8, tail = sum(full) + 2, [_up(x + m) - x // PAGE for x, m in zip(p, n)]
    pages16 = sum(tail) + 2
    s = dict(case=case, T=T, max_nodes=max(n), max_prefix=max(p),
             offs=_i32(offs), parent=_i32(parent), prefix=_i32(p),
             table8=_tables(full, pages8, gen), table=_tables(tail, pages16, gen, full),
             pages8=pages8, pages16=pages16,
             q=torch.randn(T, Hq, D, generator=gen, device="cuda").to(torch.bfloat16),
             k=_kv(pages16, Hkv, D, gen), v=_kv(pages16, Hkv, D, gen), scale=1 / math.sqrt(D),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    for name in ("k", "v"):
        code, sc = zip(*[_codes(_kv(min(2048, pages8 - at), Hkv, D, gen), case["fmt"]) for at in range(0, pages8, 2048)])
        s[name + "8"], s[name + "_scale"] = torch.cat(code), torch.cat(sc)
    return s


def _prepare_quant(case, gen, host):
    a, b = _sizes(case)
    Hkv, D = case["Hkv"], case["D"]
    first, need = [x // PAGE for x in a], [_up(y) - x // PAGE for x, y in zip(a, b)]
    pages16, pages8 = sum(need) + 1, sum(y // PAGE for y in b) + 1
    s = dict(case=case, frm=_i32(a), to=_i32(b), most=max(y // PAGE - x // PAGE for x, y in zip(a, b)),
             most_len=max(b), table=_tables(need, pages16, gen, first), pages16=pages16,
             table8=_tables([y // PAGE for y in b], pages8, gen), pages8=pages8,
             k=_kv(pages16, Hkv, D, gen), v=_kv(pages16, Hkv, D, gen),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    # one page more than the pool holds: the plain form writes there what it does not keep
    for name in ("k", "v"):
        s[name + "8"] = torch.zeros(pages8 + 1, Hkv, PAGE, D, dtype=torch.uint8, device="cuda")
        s[name + "_scale"] = torch.zeros(pages8 + 1, Hkv, device="cuda")
    return s


def _buffers(count, pages, case, gen):
    # one page more than the pool holds, as above
    return [torch.randint(-30000, 30000, (pages + 1, PAGE * case["Hkv"] * case["D"]), generator=gen, device="cuda",
                          dtype=torch.int16) for _ in range(count)]


def _prepare_fork(case, gen, host):
    ln, c = _sizes(case), case["children"]
    P = len(ln)
    B = P * (1 + c)
    need = [_up(x) for x in ln]
    width = max(need) + _up(case["nodes"]) + 1
    num = sum(need) + B * (2 + _up(case["nodes"]))
    num += num // 4 + 1
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[:P, :max(need)] = _tables(need, num, gen)
    # the children of the turn before: each holds the first half of its prompt
    for i, x in enumerate(ln):
        table[P + i * c:P + (i + 1) * c, :x // 2 // PAGE] = table[i, :x // 2 // PAGE]
    ref = torch.zeros(num, dtype=torch.int32, device="cuda")
    held = table[table >= 0].long()
    ref.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    every = ln + [x for x in ln for _ in range(c)]
    return dict(case=case, B=B, n=P * c, width=width, num=num, table=table, ref=ref,
                keep=_i32(ln + [0] * (P * c)), src=_i32([i for i in range(P) for _ in range(c)]),
                dst=_i32(list(range(P, B))), flen=_i32([x for x in ln for _ in range(c)]),
                begin=_i32(every), end=_i32([x + case["nodes"] for x in every]),
                buffers=_buffers(2 * case["layers"], num, case, gen),
                copy_src=torch.full((P * c,), -1, dtype=torch.int32, device="cuda"),
                copy_dst=torch.full((P * c,), -1, dtype=torch.int32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_compact(case, gen, host):
    need = [_up(x) for x in _sizes(case)]
    _, _, num = _compact_pages(case)
    perm = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(need):
        half = min(need[i - 1], k) // 2 if i % 2 else 0
        if half:
            table[i, :half] = table[i - 1, :half]
        table[i, half:k] = perm[at:at + k - half]
        at += k - half
    ref = torch.zeros(num, dtype=torch.int32, device="cuda")
    held = table[table >= 0].long()
    ref.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    most = max(num // 2, 1)
    return dict(case=case, B=len(need), width=table.shape[1], num=num, most=most, table=table, ref=ref,
                buffers=_buffers(2 * case["layers"], num, case, gen),
                new_table=torch.empty_like(table), new_ref=torch.empty_like(ref),
                copy_src=torch.empty(most, dtype=torch.int32, device="cuda"),
                copy_dst=torch.empty(most, dtype=torch.int32, device="cuda"),
                count=torch.zeros(1, dtype=torch.int32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"attn": _own_attn, "quant": _own_quant, "fork": _own_fork, "compact": _own_compact}[op](s)
    return {"attn": _plain_attn, "quant": _plain_quant, "fork": _plain_fork, "compact": _plain_compact}[op](s)


def _values(code, fmt):
    return code.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8)


def _plain_attn(s):
    c = s["case"]
    Hq, Hkv, D, B, G = c["Hq"], c["Hkv"], c["D"], c["B"], c["Hq"] // c["Hkv"]
    N, dev = s["max_nodes"], s["q"].device
    P, offs = s["prefix"].long(), s["offs"].long()
    n, P0 = offs[1:] - offs[:-1], P // PAGE * PAGE
    # keys and values: the 8-bit pages, then the bf16 slots from the last page boundary on
    t8 = s["table8"].long().clamp_min(0)

    def prefix(name):
        x = _values(s[name + "8"], c["fmt"])[t8].float() * s[name + "_scale"][t8][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)

    slot = P0[:, None] + torch.arange(PAGE - 1 + N, device=dev)
    at = torch.minimum(slot, (P + n)[:, None] - 1)
    page = s["table"].long().gather(1, at // PAGE)

    def tail(name):
        return s[name][page, at % PAGE].float().transpose(1, 2)

    K = torch.cat([prefix("k"), tail("k")], 2)
    V = torch.cat([prefix("v"), tail("v")], 2)
    # ancestors: reach doubles with each product
    i = torch.arange(N, device=dev)
    node = torch.minimum(offs[:-1, None] + i, offs[1:, None] - 1)
    par = torch.where(i < n[:, None], s["parent"].long()[node], -1)
    sees = ((par[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(max(N - 1, 1).bit_length()):
        sees = ((sees @ sees) > 0).float()
    j = slot - P[:, None]
    seen = sees.gather(2, j.clamp(0, N - 1)[:, None, :].expand(B, N, -1)) > 0
    seen = torch.where(j[:, None] < 0, True, seen & (j < n[:, None])[:, None])
    full = (torch.arange(t8.shape[1] * PAGE, device=dev) < P0[:, None])[:, None].expand(B, N, -1)
    mask = torch.cat([full, seen], 2)[:, None, None]
    Q = s["q"][node].float().reshape(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4)
    S = (Q.reshape(B, Hkv, G * N, D) @ K.transpose(2, 3)).reshape(B, Hkv, G, N, -1).mul_(s["scale"])
    S.masked_fill_(~mask, -math.inf)
    S = S.sub_(S.amax(-1, keepdim=True)).exp_()
    O = (S.reshape(B, Hkv, G * N, -1) @ V).reshape(B, Hkv, G, N, D) / S.sum(-1, keepdim=True)
    b = torch.repeat_interleave(torch.arange(B, device=dev), n, output_size=s["T"])
    O = O.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)
    return O[b, torch.arange(s["T"], device=dev) - offs[b]].to(torch.bfloat16)


def _plain_quant(s):
    c = s["case"]
    f, t = s["frm"].long() // PAGE, s["to"].long() // PAGE
    lp = f[:, None] + torch.arange(max(s["most"], 1), device=f.device)
    ok = lp < t[:, None]
    src = s["table"].long().gather(1, lp.clamp_max(s["table"].shape[1] - 1)).clamp_min(0)
    dst = torch.where(ok, s["table8"].long().gather(1, lp.clamp_max(s["table8"].shape[1] - 1)), s["pages8"])
    for name in ("k", "v"):
        x = s[name][src].float().transpose(2, 3)
        amax = x.abs().amax(dim=(3, 4))
        # x * qmax is exact, so the quotient is rounded once before the code
        y = x * QMAX[c["fmt"]] / torch.where(amax > 0, amax, 1.0)[..., None, None]
        code = y.to(torch.float8_e4m3fn).view(torch.uint8) if c["fmt"] == "e4m3" else y.round().to(torch.int8).view(torch.uint8)
        s[name + "8"][dst] = code
        s[name + "_scale"][dst] = amax / QMAX[c["fmt"]]
    return _quant_out(s)


def _quant_out(s):
    k = s["pages8"]
    return {"k": _values(s["k8"][:k], s["case"]["fmt"]), "v": _values(s["v8"][:k], s["case"]["fmt"]),
            "k_scale": s["k_scale"][:k], "v_scale": s["v_scale"][:k]}


def _free_first(ref):
    """Pages in order of use: the free ones first, by index."""
    return torch.argsort((ref > 0).to(torch.int32), stable=True)


def _add(ref, page, on, by):
    ref.index_add_(0, torch.where(on, page, 0).reshape(-1).long(), on.reshape(-1).to(torch.int32) * by)


def _copy(buffers, src, dst):
    for x in buffers:  # a place past the pool takes what is not copied
        x[torch.where(src < 0, x.shape[0] - 1, dst).long()] = x[torch.where(src < 0, x.shape[0] - 1, src).long()]


def _plain_fork(s):
    table, ref = s["table"], s["ref"]
    col = torch.arange(s["width"], device=table.device)
    # drop what lies past the kept length
    drop = (table >= 0) & (col * PAGE >= s["keep"][:, None])
    _add(ref, table, drop, -1)
    table.masked_fill_(drop, -1)
    # fork: full pages shared, a partial one copied to the lowest free page
    order = _free_first(ref)
    src, dst, ln = s["src"].long(), s["dst"].long(), s["flen"].long()
    rows = table[src]
    full = (col < (ln // PAGE)[:, None]) & (rows >= 0)
    _add(ref, rows, full, 1)
    part = ln % PAGE > 0
    page = order[(torch.cumsum(part, 0) - 1).clamp_min(0)].to(torch.int32)
    _add(ref, page, part, 1)
    at = (col == (ln // PAGE)[:, None]) & part[:, None]
    table[dst] = torch.where(at, page[:, None], torch.where(full, rows, -1))
    s["copy_src"].copy_(torch.where(part, rows.gather(1, (ln // PAGE)[:, None])[:, 0], -1))
    s["copy_dst"].copy_(torch.where(part, page, -1))
    # the next tree's pages
    order = _free_first(ref)
    need = (col >= (s["begin"] // PAGE)[:, None]) & (col < ((s["end"] + PAGE - 1) // PAGE)[:, None]) & (table < 0)
    page = order[(torch.cumsum(need.reshape(-1), 0) - 1).clamp_min(0)].to(torch.int32).reshape(need.shape)
    table.copy_(torch.where(need, page, table))
    _add(ref, page, need, 1)
    _copy(s["buffers"], s["copy_src"], s["copy_dst"])
    return _fork_out(s)


def _fork_out(s):
    return {"table": s["table"], "refcount": s["ref"], "copy_src": s["copy_src"], "copy_dst": s["copy_dst"],
            "pages": [x[:s["num"]] for x in s["buffers"]]}


def _plain_compact(s):
    ref, i = s["ref"], torch.arange(s["num"], device=s["ref"].device)
    used = ref > 0
    count = used.sum()
    move, hole = used & (i >= count), ~used & (i < count)
    src = torch.argsort((~move).to(torch.int32), stable=True)
    dst = torch.argsort((~hole).to(torch.int32), stable=True)
    m = move.sum()
    to = torch.where(move, dst[(torch.cumsum(move, 0) - 1).clamp_min(0)], i)
    s["new_table"].copy_(torch.where(s["table"] >= 0, to[s["table"].long().clamp_min(0)], -1))
    s["new_ref"].zero_()
    s["new_ref"].index_add_(0, torch.where(used, to, 0), torch.where(used, ref, 0))
    k = i[:s["most"]]
    s["copy_src"].copy_(torch.where(k < m, src[:s["most"]], -1))
    s["copy_dst"].copy_(torch.where(k < m, dst[:s["most"]], -1))
    s["count"].copy_(m[None])
    _copy(s["buffers"], s["copy_src"], s["copy_dst"])
    return _compact_out(s)


def _compact_out(s):
    return {"table": s["new_table"], "refcount": s["new_ref"], "copy_src": s["copy_src"], "copy_dst": s["copy_dst"],
            "count": s["count"], "pages": [x[:s["num"]] for x in s["buffers"]]}


# --------------------------------------------------------------------------
# The framework's calls.  A state keeps its batch descriptor, output buffer
# and workspace from its first pass on, as a serving loop does.
# --------------------------------------------------------------------------

def _jsv():
    from tree_verification_jsv_b200 import jsv
    return jsv


def _workspace(nbytes):
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")


def _own_attn(s):
    jsv = _jsv()
    if "plan" not in s:
        c = s["case"]
        batch = jsv.make_batch(B=c["B"], Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], max_pages_per_req=s["table"].shape[1],
                               num_pages=s["pages16"], total_nodes=s["T"], max_nodes=s["max_nodes"],
                               max_prefix=s["max_prefix"], page_table=s["table"], prefix_len=s["prefix"],
                               node_offsets=s["offs"], parent=s["parent"], dev_status=s["status"])
        cache = jsv.make_kv8(format=c["fmt"], num_pages=s["pages8"], max_pages_per_req=s["table8"].shape[1],
                             k=s["k8"], v=s["v8"], k_scale=s["k_scale"], v_scale=s["v_scale"], page_table=s["table8"])
        s["plan"] = (batch, cache, torch.empty_like(s["q"]),
                     _workspace(jsv.jsv_tree_attention_kv8_workspace_size(batch, cache)))
    batch, cache, out, ws = s["plan"]
    jsv.jsv_tree_attention_kv8(batch, cache, s["q"], s["k"], s["v"], s["scale"], out, ws)
    return out


def _own_quant(s):
    jsv = _jsv()
    if "plan" not in s:
        c = s["case"]
        one = torch.zeros(c["B"] + 1, dtype=torch.int32, device="cuda")
        batch = jsv.make_batch(B=c["B"], Hq=c["Hkv"], Hkv=c["Hkv"], D=c["D"], max_pages_per_req=s["table"].shape[1],
                               num_pages=s["pages16"], total_nodes=c["B"], max_nodes=1, max_prefix=s["most_len"],
                               page_table=s["table"], prefix_len=s["frm"], node_offsets=one, parent=one,
                               dev_status=s["status"])
        cache = jsv.make_kv8(format=c["fmt"], num_pages=s["pages8"], max_pages_per_req=s["table8"].shape[1],
                             k=s["k8"], v=s["v8"], k_scale=s["k_scale"], v_scale=s["v_scale"], page_table=s["table8"])
        s["plan"] = batch, cache, one
    batch, cache, _ = s["plan"]
    jsv.jsv_kv8_quantize(batch, cache, s["k"], s["v"], s["frm"], s["to"])
    return _quant_out(s)


def _pool_plan(s):
    jsv = _jsv()
    if "plan" not in s:
        pool = jsv.make_page_pool(num_pages=s["num"], refcount=s["ref"], dev_status=s["status"])
        s["plan"] = (pool, _workspace(jsv.jsv_pages_workspace_size(s["num"], s["B"])),
                     jsv.make_page_buffers(s["buffers"], [x[0].numel() * x.element_size() for x in s["buffers"]]))
    return jsv, *s["plan"]


def _own_fork(s):
    jsv, pool, ws, buffers = _pool_plan(s)
    jsv.jsv_pages_trim(pool, s["table"], s["B"], s["width"], None, s["keep"])
    jsv.jsv_pages_fork(pool, s["table"], s["B"], s["width"], s["n"], s["src"], s["dst"], s["flen"], False,
                       s["copy_src"], s["copy_dst"], ws)
    jsv.jsv_pages_alloc(pool, s["table"], s["B"], s["width"], s["begin"], s["end"], False, ws)
    jsv.jsv_pages_copy(pool, buffers, s["copy_src"], s["copy_dst"], s["n"], None)
    return _fork_out(s)


def _own_compact(s):
    jsv, pool, ws, buffers = _pool_plan(s)
    jsv.jsv_pages_compact(pool, s["table"], s["B"], s["width"], s["new_table"], s["new_ref"], s["copy_src"],
                          s["copy_dst"], s["most"], s["count"], ws)
    jsv.jsv_pages_copy(pool, buffers, s["copy_src"], s["copy_dst"], s["most"], s["count"])
    return _compact_out(s)


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "attn":
        return _exact_attn(prepare(case, seed))
    if case["op"] == "quant":
        return _exact_quant(prepare(case, seed))
    return None  # whole numbers only


def _decode(code, fmt):
    """Codes to their values in 64 bits, from the bits."""
    c = code.to(torch.int64)
    if fmt == "int8":
        return (c - 256 * (c >= 128)).double()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    return torch.where(c >= 128, -mag, mag)


def _exact_attn(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    n, p = _sizes(c)
    out = torch.empty(s["T"], Hq, D, dtype=torch.float64, device="cuda")
    parent, base = s["parent"].tolist(), 0
    for b, (m, P) in enumerate(zip(n, p)):
        full = P // PAGE
        L = P % PAGE + m
        mask = torch.zeros(m, L, dtype=torch.bool)
        mask[:, :P % PAGE] = True
        for i in range(m):
            if i:
                mask[i] |= mask[parent[base + i]]
            mask[i, P % PAGE + i] = True
        mask = mask.cuda()
        pg8 = s["table8"][b, :full].long()
        pos = torch.arange(full * PAGE, P + m, device="cuda")
        pg = s["table"][b].long()[pos // PAGE]
        for g in range(Hkv):
            kv = []
            for name in ("k", "v"):
                x = _decode(s[name + "8"][pg8, g], c["fmt"]) * s[name + "_scale"][pg8, g].double()[:, None, None]
                kv.append(torch.cat([x.reshape(-1, D), s[name][pg, pos % PAGE, g].double()]))
            for h in range(g * G, (g + 1) * G):
                w = (s["q"][base:base + m, h].double() @ kv[0].T) * s["scale"]
                w[:, full * PAGE:] = torch.where(mask, w[:, full * PAGE:], -math.inf)
                out[base:base + m, h] = torch.softmax(w, 1) @ kv[1]
        base += m
    return out


def _exact_quant(s):
    c = s["case"]
    a, b = _sizes(c)
    got = {}
    for name in ("k", "v"):
        code = torch.zeros(s["pages8"], c["Hkv"], PAGE, c["D"], dtype=torch.float64, device="cuda")
        scale = torch.zeros(s["pages8"], c["Hkv"], dtype=torch.float64, device="cuda")
        for r, (x, y) in enumerate(zip(a, b)):
            if y // PAGE == x // PAGE:
                continue
            w = s[name][s["table"][r, x // PAGE:y // PAGE].long()].double().permute(0, 2, 1, 3)
            top = w.abs().flatten(2).amax(2)
            z = w * QMAX[c["fmt"]] / torch.where(top == 0, 1.0, top)[:, :, None, None]
            if c["fmt"] == "e4m3":
                # three bits after the leading one; steps of 2^-9 below 2^-6
                step = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6))) - 3)
                z = torch.round(z / step) * step
            at = s["table8"][r, x // PAGE:y // PAGE].long()
            code[at], scale[at] = z, top / QMAX[c["fmt"]]
        got[name], got[name + "_scale"] = (code if c["fmt"] == "e4m3" else None), scale
    return got
