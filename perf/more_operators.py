"""Drafted trees over the paged cache and eviction from it, in plain torch and through this library.

Five operators over a key/value cache kept in pages ([pages, kv heads, slots, d], a sequence's pages listed in a
row of a page table):
  mask    the parents of drafted tokens (nodes) as the bits of the nodes that each one sees, and their rotary positions
  tree    attention of a sequence's nodes over its context and over the nodes that a mask shows to each
  weigh   what every cached token got of the queries' attention, added to what it had
  select  the tokens of every sequence and head that stay: the first, the last and the heaviest
  keep    the keys and values of the tokens that stay to the front of their sequence, or into other pages

`own` chooses the library's calls; otherwise every operator is spelled out in elementary torch operations
in 32 bits.  `exact` computes the same from the definitions in 64 bits, one sequence at a time.
"""
import math
import random

import torch

own = False

# (query heads, kv heads, head size)
HEADS = [(12, 12, 64), (14, 2, 64), (16, 16, 128), (32, 8, 128), (64, 8, 128)]


def listed():
    return [
        # one sequence's small tree: what a call costs at least
        dict(name="mask_one", op="mask", B=1, new_lo=8, new_hi=8, len_lo=500, len_hi=500, spread=4, lens=1),
        # a serving batch's trees, some of them deep
        dict(name="mask_batch", op="mask", B=256, new_lo=20, new_hi=256, len_lo=10, len_hi=8000, spread=12, lens=2),
        # a small tree on one short sequence
        dict(name="tree_one", op="tree", B=1, new_lo=12, new_hi=12, len_lo=1000, len_hi=1000, spread=4, Hq=12, Hkv=12, d=64,
             page=16, dtype="f16", slots_first=False, lens=3),
        # a ragged serving batch with trees of its own sizes
        dict(name="tree_batch", op="tree", B=16, new_lo=8, new_hi=64, len_lo=100, len_hi=8192, spread=16, Hq=32, Hkv=8, d=128,
             page=64, dtype="bf16", slots_first=False, lens=4),
        # large trees on long contexts
        dict(name="tree_long", op="tree", B=2, new_lo=50, new_hi=64, len_lo=60001, len_hi=131007, spread=20, Hq=64, Hkv=8,
             d=128, page=128, dtype="bf16", slots_first=True, lens=5),
        # after the next token of one sequence
        dict(name="weigh_one", op="weigh", B=1, new_lo=1, new_hi=1, len_lo=1000, len_hi=1000, Hq=12, Hkv=12, d=64, page=16,
             dtype="f16", causal=True, slots_first=False, old=True, decay=1.0, lens=6),
        # after the next tokens of a ragged serving batch, older steps counting for less
        dict(name="weigh_batch", op="weigh", B=32, new_lo=1, new_hi=1, len_lo=200, len_hi=8192, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16", causal=True, slots_first=False, old=True, decay=0.98, lens=7),
        # chunks of prompts, their weights counted from nothing
        dict(name="weigh_prompts", op="weigh", B=4, new_lo=700, new_hi=2048, len_lo=2000, len_hi=9000, Hq=32, Hkv=8, d=128,
             page=64, dtype="bf16", causal=True, slots_first=False, old=False, decay=1.0, lens=8),
        # short sequences of a small model
        dict(name="select_short", op="select", B=2, heads=2, len_lo=600, len_hi=1000, budget=256, sink=4, recent=32, lens=9),
        # few heads, very long sequences
        dict(name="select_long", op="select", B=4, heads=8, len_lo=90001, len_hi=131071, budget=16384, sink=16, recent=1024,
             lens=10),
        # the accepted tokens of drafted trees, moved up behind the context
        dict(name="keep_paths", op="keep", B=64, Hkv=8, d=128, page=64, dtype="bf16", slots_first=False, path=True, len_lo=100,
             len_hi=2000, new_lo=20, new_hi=64, budget=6, lens=11),
        # what stays of long sequences, into pages of its own (the old ones may be shared with others)
        dict(name="keep_evicted", op="keep", B=8, Hkv=8, d=128, page=64, dtype="bf16", slots_first=False, path=False,
             len_lo=16384, len_hi=32768, budget=8192, lens=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 0.6)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["mask", "tree", "tree", "weigh", "weigh", "select", "keep"])
    Hq, Hkv, d = rng.choice(HEADS)
    c = dict(op=op, lens=rng.randrange(1 << 30))
    if op in ("tree", "weigh", "keep"):
        c.update(Hkv=Hkv, d=d, page=rng.choice([16, 32, 64, 128, 256]), dtype=rng.choice(["f16", "bf16"]),
                 slots_first=rng.random() < 0.4)
    if op == "mask":
        c.update(B=_spread(rng, 1, 256), new_hi=_spread(rng, 1, 256), len_hi=_spread(rng, 1, 8000), spread=_spread(rng, 1, 40))
    elif op == "tree":
        c.update(B=_spread(rng, 1, 32), new_hi=_spread(rng, 1, 128), len_hi=_spread(rng, 1, 120000), spread=_spread(rng, 1, 40),
                 Hq=Hq)
    elif op == "weigh":
        chunk = rng.random() < 0.4
        c.update(B=_spread(rng, 1, 4 if chunk else 64), new_hi=_spread(rng, 2, 3000) if chunk else 1,
                 len_hi=_spread(rng, 1, 8000 if chunk else 120000), Hq=Hq, causal=rng.random() < 0.85, old=rng.random() < 0.7,
                 decay=rng.choice([1.0, 0.98]))
    elif op == "select":
        c.update(B=_spread(rng, 1, 64), heads=rng.choice([1, 2, 8, 12]), len_hi=_spread(rng, 100, 131072),
                 sink=rng.randint(0, 16), recent=_spread(rng, 1, 64))
        c["budget"] = _spread(rng, 80, 20000)
    else:
        path = rng.random() < 0.4
        c.update(B=_spread(rng, 1, 64), path=path, len_hi=_spread(rng, 64, 4000 if path else 32768))
        if path:
            c["new_hi"] = rng.randint(20, 128)
        c["budget"] = rng.randint(1, 10) if path else _spread(rng, 32, 8192)
    # no dearer than the largest listed one of its kind
    top = [work(x) for x in listed() if x["op"] == op]
    while True:
        c["len_lo"] = max(1, c["len_hi"] // rng.randint(1, 12))
        if op == "keep" and c["path"]:
            c["new_lo"] = 20
        elif op in ("mask", "tree", "weigh"):
            c["new_lo"] = max(1, c["new_hi"] // rng.randint(1, 6))
        w = work(c)
        if w["bytes"] <= max(t["bytes"] for t in top) and w["flops"] <= max(t["flops"] for t in top):
            return c
        big = max(("B", "len_hi", "new_hi"), key=lambda n: c.get(n, 0) * (1000 if n == "B" and c["len_hi"] < 100 else 1))
        c[big] = max(21 if op == "keep" and big == "new_hi" else 1, c[big] * 2 // 3)


def _lengths(case):
    """(new tokens, tokens in the cache with them) of every sequence."""
    rng = random.Random(case["lens"])
    had = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["B"])]
    if "new_hi" not in case:
        return [0] * case["B"], had
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return new, [a + b for a, b in zip(new, had)]


def _words(case):
    return -(-max(_lengths(case)[0]) // 32)


def _kept(case):
    """How many tokens of every sequence stay, and are moved."""
    new, lens = _lengths(case)
    if case["path"]:
        rng = random.Random(case["lens"] + 1)
        return [rng.randint(1, case["budget"]) for _ in new]
    return [min(n, case["budget"]) for n in lens]


def work(case):
    op = case["op"]
    new, lens = _lengths(case)
    T, B = sum(new), case["B"]
    if op == "mask":
        return {"bytes": 4 * T * (2 + _words(case)) + 8 * B, "flops": 0}
    if op == "select":
        W = max(lens)
        return {"bytes": 4 * case["heads"] * (sum(lens) + B * (W + case["budget"])) + 8 * B, "flops": 0}
    Hkv, d = case["Hkv"], case["d"]
    tables = 4 * (sum(-(-n // case["page"]) for n in lens) + 2 * B)
    if op == "keep":
        heads = 1 if case["path"] else Hkv
        return {"bytes": sum(_kept(case)) * (2 * 2 * Hkv * d * 2 + 4 * heads) + tables, "flops": 0}
    Hq = case["Hq"]
    if op == "tree":
        pairs = sum(a * (n - a) + a * (a + 1) // 2 for a, n in zip(new, lens))
        return {"bytes": T * (2 * Hq * d * 2 + 4 * _words(case)) + sum(lens) * 2 * Hkv * d * 2 + tables,
                "flops": 4 * pairs * Hq * d}
    pairs = sum(a * (n - a) + a * (a + 1) // 2 if case["causal"] else a * n for a, n in zip(new, lens))
    return {"bytes": T * Hq * (d * 2 + 4) + sum(lens) * Hkv * (d * 2 + (8 if case["old"] else 4)) + tables,
            "flops": 2 * pairs * Hq * d}


def _parents(case, seed):
    """Every sequence's nodes, parents first: the parent of each, -1 where it follows the context."""
    rng = random.Random(seed)
    return [[rng.randint(max(-1, i - case["spread"]), i - 1) for i in range(n)] for n in _lengths(case)[0]]


def _signed(x):
    return x - (1 << 32) if x >= 1 << 31 else x


def _mask_rows(parents, words):
    """The nodes that each node sees, itself and its ancestors, as bits."""
    rows = []
    for tree in parents:
        seen = []
        for i, p in enumerate(tree):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        rows += [[_signed(m >> 32 * w & 0xffffffff) for w in range(words)] for m in seen]
    return rows


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, (new, lens) = case["op"], _lengths(case)
    B, T = case["B"], sum(new)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case, "max_new": max(new), "seq_lens": ints(lens), "cu_seqlens": ints([0] + torch.tensor(new).cumsum(0).tolist())}
    if op == "mask":
        s["parents"] = ints(sum(_parents(case, seed), []))
        return s
    if op == "select":
        # weights as attention leaves them: a few heavy tokens, many light ones, some that nothing has looked at yet
        w = (randn(B, case["heads"], max(lens)) * 2).exp()
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.05] = 0.0
        live = torch.arange(max(lens), device="cuda") < s["seq_lens"][:, None, None]
        s["weights"] = torch.where(live, w, 0.0)
        return s
    Hkv, d, S, dt = case["Hkv"], case["d"], case["page"], {"f16": torch.float16, "bf16": torch.bfloat16}[case["dtype"]]
    # pages in any order, a few that belong to nobody; entries behind a sequence's last page are not valid
    need = [-(-n // S) for n in lens]
    need_out = [-(-n // S) for n in _kept(case)] if op == "keep" and not case["path"] else []
    count = sum(need) + sum(need_out) + 3
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)

    def table(need, start):
        n = torch.tensor(need, device="cuda")
        col = torch.arange(max(need + [1]) + 1, device="cuda")
        at = start + (n.cumsum(0) - n)[:, None] + col
        return torch.where(col < n[:, None], order[at.clamp(max=count - 1)], -1).to(torch.int32)

    s["page_table"] = table(need, 0)
    # keys carry a channel's own offset, as projections with rotary halves do; values do not
    shape = (count, S, Hkv, d) if case["slots_first"] else (count, Hkv, S, d)
    offset = randn(Hkv, d) if case["slots_first"] else randn(Hkv, 1, d)
    pages = [(randn(*shape) + offset).to(dt), randn(*shape).to(dt)]
    s["k_pages"], s["v_pages"] = (p.transpose(1, 2) if case["slots_first"] else p for p in pages)
    if op == "keep":
        kept = _kept(case)
        s["counts"] = ints(kept)
        if case["path"]:
            # an accepted path's nodes lie behind the places that they go to, so that a pass can be made again
            rng = random.Random(seed)
            paths = [sorted(rng.sample(range(c, a), c) if a >= 2 * c else range(c)) for c, a in zip(kept, new)]
            s["keep"] = ints([[n - a + i for i in p] + [-1] * (case["budget"] - len(p)) for p, n, a in zip(paths, lens, new)])[:, None]
            s["first"] = s["seq_lens"] - ints(new)
        else:
            s["out_table"] = table(need_out, sum(need))
            at = torch.arange(max(lens), device="cuda")
            r = torch.rand(B, Hkv, max(lens), generator=g, device="cuda")
            r = torch.where((at < 4) | (at >= s["seq_lens"][:, None, None] - 16), 2.0, r)  # the first and the last stay
            r = torch.where(at < s["seq_lens"][:, None, None], r, -1.0)
            top = r.argsort(-1, descending=True)[..., :case["budget"]]
            rank = torch.arange(top.shape[-1], device="cuda")
            top = torch.where(rank < s["counts"][:, None, None], top, 1 << 30).sort(-1).values
            s["keep"] = torch.where(top < 1 << 30, top, -1).to(torch.int32)
        return s
    Hq = case["Hq"]
    s["q"] = (randn(T, Hq, d) * 1.5).to(dt)
    if op == "tree":
        s["mask"] = ints(_mask_rows(_parents(case, seed), _words(case)))
        return s
    # the log-sum-exp that the attention of the same queries has returned
    s["lse"] = torch.empty(T, Hq, device="cuda")
    at = 0
    for b, (a, n) in enumerate(zip(new, lens)):
        own_pages = s["page_table"][b, :need[b]].long()
        for h in range(Hkv):
            G = Hq // Hkv
            keys = s["k_pages"][own_pages, h].reshape(-1, d)[:n].float()
            x = s["q"][at:at + a, h * G:(h + 1) * G].float() @ keys.T / math.sqrt(d)
            if case["causal"]:
                x.masked_fill_(torch.ones(a, n, dtype=torch.bool, device="cuda").triu(n - a + 1)[:, None], -math.inf)
            s["lse"][at:at + a, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
        at += a
    W = max(lens)
    live = torch.arange(W, device="cuda") < s["seq_lens"][:, None, None]
    s["weights"] = torch.where(live, torch.rand(B, Hkv, W, generator=g, device="cuda").pow(4) * 3, 0.0) if case["old"] else None
    s["out"] = torch.zeros(B, Hkv, W, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _token_rows(s, T):
    """The sequence of every packed token, and its place among the sequence's new ones."""
    cu = s["cu_seqlens"].long()
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, t - cu[b]


def _plain_mask(s):
    words, N, parents = -(-s["max_new"] // 32), s["max_new"], s["parents"].long()
    b, i = _token_rows(s, parents.numel())
    sees = torch.zeros(s["seq_lens"].numel(), N, N, device="cuda")
    has = parents >= 0
    sees[b[has], i[has], parents[has]] = 1.0
    sees += torch.eye(N, device="cuda")
    for _ in range(max(1, (N - 1).bit_length())):  # itself and its parent, then four levels, then ...
        sees = ((sees @ sees) > 0).float()
    rows = sees[b, i]
    count = s["cu_seqlens"].long().diff()
    positions = s["seq_lens"].long()[b] - count[b] + rows.sum(-1).long() - 1
    bits = torch.zeros(rows.shape[0], words * 32, dtype=torch.long, device="cuda")
    bits[:, :N] = rows.long()
    mask = (bits.view(-1, words, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32), positions.to(torch.int32)


def _gathered(pages, table):
    """[B, n] page ids -> [B, kv heads, n * slots, d] in 32 bits."""
    return pages[table.clamp(min=0).long()].float().transpose(-4, -3).flatten(-3, -2)


def _padded(s, x, fill):
    """[T, Hq, ...] rows -> [B, kv heads, most new tokens, group, ...]."""
    case = s["case"]
    b, i = _token_rows(s, x.shape[0])
    y = torch.full((case["B"], s["max_new"]) + x.shape[1:], fill, device="cuda")
    y[b, i] = x.float()
    return y.unflatten(2, (case["Hkv"], case["Hq"] // case["Hkv"])).transpose(1, 2)


def _plain_tree(s):
    case, d = s["case"], s["case"]["d"]
    T, N = s["q"].shape[0], s["max_new"]
    k, v = _gathered(s["k_pages"], s["page_table"]), _gathered(s["v_pages"], s["page_table"])
    q = _padded(s, s["q"], 0.0).flatten(2, 3)  # [B, kv heads, N * group, d]
    scores = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).unflatten(2, (N, -1))
    b, i = _token_rows(s, T)
    L = k.shape[2]
    past = s["seq_lens"].long() - s["cu_seqlens"].long().diff()
    at = torch.arange(L, device="cuda")
    node = (at - past[:, None]).clamp(min=0, max=32 * s["mask"].shape[1] - 1)  # [B, L]
    seen = torch.zeros(case["B"], N, L, dtype=torch.bool, device="cuda")
    words = s["mask"].long().gather(1, (node // 32)[b])
    seen[b, i] = ((words >> (node % 32)[b] & 1) > 0) & (at >= past[b, None]) & (at < s["seq_lens"][b, None])
    seen |= (at < past[:, None])[:, None]
    scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (scores - m).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, (p.flatten(2, 3) @ v).unflatten(2, (N, -1)) / total, 0.0)
    return o.transpose(1, 2).flatten(2, 3)[b, i].to(s["q"].dtype)


def _plain_weigh(s):
    case, d, N, W = s["case"], s["case"]["d"], s["max_new"], s["out"].shape[2]
    k = _gathered(s["k_pages"], s["page_table"])[:, :, :W]
    if k.shape[2] < W:
        W = k.shape[2]
    q, lse = _padded(s, s["q"], 0.0).flatten(2, 3), _padded(s, s["lse"], math.inf).flatten(2, 3)  # rows that are not there weigh nothing
    p = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).sub_(lse[..., None]).exp_().unflatten(2, (N, -1))
    at, i, n = torch.arange(W, device="cuda"), torch.arange(N, device="cuda"), s["seq_lens"].long()[:, None]
    seen = (at < n)[:, None].expand(-1, N, -1)
    if case["causal"]:
        seen = seen & (at <= n[..., None] - s["cu_seqlens"].long().diff()[:, None, None] + i[:, None])
    p.mul_(seen[:, None, :, None])
    w = p.sum((2, 3))
    if s["weights"] is not None:
        w += case["decay"] * s["weights"]
    live = at < n[..., None]
    s["out"].copy_(torch.where(live, w, s["out"]))
    return s["out"]


def _plain_select(s):
    case, W, n = s["case"], s["weights"].shape[2], s["seq_lens"][:, None, None]
    at = torch.arange(W, device="cuda")
    always = (at < case["sink"]) | (at >= n - case["recent"])
    x = torch.where(at < n, torch.where(always, math.inf, s["weights"]), -1.0)
    order = x.sort(dim=-1, descending=True, stable=True).indices[..., :case["budget"]]
    order = torch.nn.functional.pad(order, (0, case["budget"] - order.shape[-1]))
    counts = s["seq_lens"].clamp(max=case["budget"])
    rank = torch.arange(case["budget"], device="cuda")
    live = rank < counts[:, None, None]
    keep = torch.where(live, order, 1 << 30).sort(-1).values
    kept = torch.zeros_like(s["weights"])
    m = min(W, case["budget"])
    kept[..., :m] = torch.where(live[..., :m], s["weights"].gather(-1, keep[..., :m].clamp(max=W - 1)), 0.0)
    return torch.where(live, keep, -1).to(torch.int32), counts, kept


def _plain_keep(s):
    S, N = s["case"]["page"], s["keep"].shape[2]
    live = torch.arange(N, device="cuda") < s["counts"][:, None, None]
    b, h, i = live.expand_as(s["keep"]).nonzero(as_tuple=True)
    src, dst = s["keep"][b, h, i].long(), i + (s["first"].long()[b] if "first" in s else 0)
    from_page = s["page_table"][b, src // S].long()
    to_page = s.get("out_table", s["page_table"])[b, dst // S].long()
    for pages in (s["k_pages"], s["v_pages"]):
        if s["keep"].shape[1] == 1:
            pages[to_page, :, dst % S] = pages[from_page, :, src % S]
        else:
            pages[to_page, h, dst % S] = pages[from_page, h, src % S]
    return s["k_pages"], s["v_pages"]


def run(s):
    op, case = s["case"]["op"], s["case"]
    if not own:
        return {"mask": _plain_mask, "tree": _plain_tree, "weigh": _plain_weigh, "select": _plain_select, "keep": _plain_keep}[op](s)
    from attention_forward_prefill_gb300 import binding
    if op == "mask":
        return binding.tree_mask(s["parents"], s["cu_seqlens"], s["max_new"], s["seq_lens"])
    if op == "tree":
        return binding.prefill_tree(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["cu_seqlens"],
                                    s["max_new"], s["mask"])
    if op == "weigh":
        return binding.cache_weigh(s["q"], s["lse"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["cu_seqlens"],
                                   s["max_new"], causal=case["causal"], weights=s["weights"], decay=case["decay"], out=s["out"])
    if op == "select":
        return binding.cache_select(s["weights"], s["seq_lens"], case["budget"], sink=case["sink"], recent=case["recent"])
    return binding.cache_keep(s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["keep"], s["counts"],
                              first=s.get("first"), out_table=s.get("out_table"))


# ---------------------------------------------------------------- definitions
def exact(case, seed):
    s, (new, lens) = prepare(case, seed), _lengths(case)
    op, B = case["op"], case["B"]
    if op == "mask":
        cu, parents, n = s["cu_seqlens"].tolist(), s["parents"].tolist(), s["seq_lens"].tolist()
        trees = [parents[cu[b]:cu[b + 1]] for b in range(B)]
        rows = torch.tensor(_mask_rows(trees, -(-s["max_new"] // 32)), dtype=torch.int32)
        positions = []
        for b, t in enumerate(trees):
            depth = []
            for p in t:
                depth.append(depth[p] + 1 if p >= 0 else 0)
            positions += [n[b] - len(t) + x for x in depth]
        return rows, torch.tensor(positions, dtype=torch.int32)
    if op == "select":
        weights = s["weights"].double().cpu()
        keep = torch.full((B, case["heads"], case["budget"]), -1, dtype=torch.int32)
        kept, counts = torch.zeros(weights.shape, dtype=torch.float64), []
        for b, n in enumerate(lens):
            c = min(n, case["budget"])
            counts.append(c)
            middle = list(range(case["sink"], n - case["recent"])) if c < n else []
            for h in range(case["heads"]):
                w = weights[b, h].tolist()
                if c < n:
                    mine = sorted(middle, key=lambda i: (-w[i], i))[:c - case["sink"] - case["recent"]]
                    mine = sorted(mine + list(range(case["sink"])) + list(range(n - case["recent"], n)))
                else:
                    mine = list(range(n))
                keep[b, h, :c] = torch.tensor(mine, dtype=torch.int32)
                kept[b, h, :c] = weights[b, h, mine]
        return keep, torch.tensor(counts, dtype=torch.int32), kept
    S, table = case["page"], s["page_table"].cpu().tolist()
    if op == "keep":
        k, v = s["k_pages"].double().clone(), s["v_pages"].double().clone()
        first = s["first"].tolist() if "first" in s else [0] * B
        to = s["out_table"].cpu().tolist() if "out_table" in s else table
        pages = lambda t, i: torch.tensor(t, device="cuda")[i // S]  # noqa: E731
        for b, c in enumerate(s["counts"].tolist()):
            dst = torch.arange(first[b], first[b] + c, device="cuda")
            for h in range(case["Hkv"]):
                src = s["keep"][b, h if s["keep"].shape[1] > 1 else 0, :c].long()
                k[pages(to[b], dst), h, dst % S] = s["k_pages"][pages(table[b], src), h, src % S].double()
                v[pages(to[b], dst), h, dst % S] = s["v_pages"][pages(table[b], src), h, src % S].double()
        return k, v
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    G, t0 = Hq // Hkv, 0
    if op == "tree":
        out, trees = torch.empty(sum(new), Hq, d, dtype=torch.float64, device="cuda"), _parents(case, seed)
    else:
        out = s["out"].double()
    for b, (a, n) in enumerate(zip(new, lens)):
        own_pages = torch.tensor(table[b][:-(-n // S)], dtype=torch.long, device="cuda")
        if op == "tree":
            hidden = torch.ones(a, n, dtype=torch.bool)
            hidden[:, :n - a] = False
            for i in range(a):
                j = i
                while j >= 0:
                    hidden[i, n - a + j] = False
                    j = trees[b][j]
            hidden = hidden.cuda()[:, None]
        else:
            hidden = torch.ones(a, n, dtype=torch.bool, device="cuda").triu(n - a + 1)[:, None]
        for h in range(Hkv):
            k = s["k_pages"][own_pages, h].reshape(-1, d)[:n].double()
            q = s["q"][t0:t0 + a, h * G:(h + 1) * G].double()
            x = torch.einsum("tgd,jd->tgj", q, k) / math.sqrt(d)
            if op == "tree":
                v = s["v_pages"][own_pages, h].reshape(-1, d)[:n].double()
                out[t0:t0 + a, h * G:(h + 1) * G] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v
                continue
            p = torch.exp(x - s["lse"][t0:t0 + a, h * G:(h + 1) * G].double()[..., None])
            if case["causal"]:
                p = p.masked_fill(hidden, 0.0)
            out[b, h, :n] = p.sum((0, 1))
            if case["old"]:
                out[b, h, :n] += case["decay"] * s["weights"][b, h, :n].double()
        t0 += a
    return out
