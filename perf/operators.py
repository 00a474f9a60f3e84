"""The paged-cache operators at the sizes they are used at, in plain torch and through this library.

Three operators over one key/value cache kept in pages ([pages, kv heads, slots, d], a sequence's pages
listed in a row of a page table):
  append  the keys and values of new tokens into their slots, with the rotary position rotation of q and k
  paged   attention over the pages: one query token per sequence, or a chunk of them
  shared  one query token per sequence over a prefix that the whole batch shares and the sequence's own pages

`own` chooses the library's calls; otherwise every operator is spelled out in elementary torch operations
in 32 bits.  `exact` computes the same from the definitions in 64 bits, one sequence at a time.
"""
import math
import random

import torch

own = False

# (query heads, kv heads, head size)
HEADS = [(12, 12, 64), (14, 2, 64), (16, 16, 128), (32, 8, 128), (64, 8, 128)]
ROPE_BASE = 10000.0


def listed():
    return [
        # one more token of one sequence, 12 heads of 64: what a call costs at least
        dict(name="append_one", op="append", B=1, new_lo=1, new_hi=1, len_lo=1000, len_hi=1000, Hq=12, Hkv=12, d=64,
             page=16, dtype="f16", rot=64, inter=False, slots_first=False, fused=False, lens=1),
        # a serving batch's step: one token each at ragged lengths, a quarter of the head left unrotated
        dict(name="append_batch", op="append", B=256, new_lo=1, new_hi=1, len_lo=1, len_hi=512, Hq=32, Hkv=8, d=128,
             page=64, dtype="bf16", rot=96, inter=False, slots_first=False, fused=False, lens=2),
        # ragged prompts out of one fused projection, into pages that keep the heads of a token together
        dict(name="append_prompts", op="append", B=12, new_lo=100, new_hi=5000, len_lo=100, len_hi=6000, Hq=32, Hkv=8,
             d=128, page=16, dtype="bf16", rot=128, inter=True, slots_first=True, fused=True, lens=3),
        # the next token of one sequence
        dict(name="decode_one", op="paged", B=1, new_lo=1, new_hi=1, len_lo=1000, len_hi=1000, Hq=12, Hkv=12, d=64,
             page=16, dtype="f16", causal=True, slots_first=False, lens=4),
        # the next tokens of a ragged serving batch
        dict(name="decode_ragged", op="paged", B=32, new_lo=1, new_hi=1, len_lo=200, len_hi=8192, Hq=32, Hkv=8, d=128,
             page=64, dtype="bf16", causal=True, slots_first=False, lens=5),
        # few sequences, very long ones
        dict(name="decode_long", op="paged", B=4, new_lo=1, new_hi=1, len_lo=90001, len_hi=131071, Hq=64, Hkv=8, d=128,
             page=128, dtype="bf16", causal=True, slots_first=True, lens=6),
        # a few drafted tokens per sequence, checked in one pass
        dict(name="check_drafts", op="paged", B=16, new_lo=3, new_hi=6, len_lo=50, len_hi=4096, Hq=14, Hkv=2, d=64,
             page=16, dtype="f16", causal=True, slots_first=False, lens=7),
        # the next chunk of prompts that are in the cache in part
        dict(name="prompt_chunks", op="paged", B=4, new_lo=700, new_hi=2048, len_lo=3000, len_hi=10000, Hq=32, Hkv=8,
             d=128, page=64, dtype="bf16", causal=True, slots_first=False, lens=8),
        # whole prompts, small heads
        dict(name="prompt_whole", op="paged", B=3, new_lo=3500, new_hi=5000, len_lo=0, len_hi=0, Hq=12, Hkv=12, d=64,
             page=256, dtype="f16", causal=True, slots_first=False, lens=9),
        # a handful of continuations of one short prefix
        dict(name="shared_few", op="shared", B=4, prefix=777, len_lo=0, len_hi=64, Hq=12, Hkv=12, d=64, page=16,
             dtype="f16", slots_first=False, lens=10),
        # a batch under one long instruction
        dict(name="shared_long", op="shared", B=64, prefix=32801, len_lo=1, len_hi=512, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16", slots_first=False, lens=11),
        # many samples of one prompt
        dict(name="shared_many", op="shared", B=256, prefix=16500, len_lo=16, len_hi=1024, Hq=64, Hkv=8, d=128, page=32,
             dtype="bf16", slots_first=True, lens=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 0.6)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "shared"])
    Hq, Hkv, d = rng.choice(HEADS)
    c = dict(op=op, Hq=Hq, Hkv=Hkv, d=d, page=rng.choice([16, 32, 64, 128, 256]), dtype=rng.choice(["f16", "bf16"]),
             slots_first=rng.random() < 0.4, lens=rng.randrange(1 << 30))
    if op == "append":
        c["B"] = _spread(rng, 1, 256)
        c["new_hi"] = 1 if rng.random() < 0.5 else _spread(rng, 2, 5000)
        c["len_hi"] = _spread(rng, 1, 6000)
        c.update(rot=16 * rng.randint(0, d // 16), inter=rng.random() < 0.4, fused=rng.random() < 0.5)
    elif op == "paged":
        kind = rng.choice(["token", "token", "drafts", "chunk"])
        c["B"] = _spread(rng, 1, 64 if kind == "token" else 16 if kind == "drafts" else 4)
        c["new_hi"] = {"token": 1, "drafts": rng.randint(2, 9), "chunk": _spread(rng, 64, 4000)}[kind]
        c["len_hi"] = _spread(rng, 16, 120000 if kind == "token" else 8000)
        c["causal"] = rng.random() < 0.85
    else:
        c["B"] = _spread(rng, 2, 256)
        c["prefix"] = _spread(rng, 16, 32768)
        c["len_hi"] = _spread(rng, 1, 1024)
    # no dearer than the largest listed one of its kind
    top = [work(x) for x in listed() if x["op"] == op]
    while True:
        c["len_lo"] = c["len_hi"] // rng.randint(1, 12)
        if op != "shared":
            c["new_lo"] = max(1, c["new_hi"] // rng.randint(1, 6))
        w = work(c)
        if w["bytes"] <= max(t["bytes"] for t in top) and w["flops"] <= max(t["flops"] for t in top):
            return c
        big = max(("B", "len_hi", "new_hi", "prefix"), key=lambda n: c.get(n, 0))
        c[big] = max(1, c[big] * 2 // 3)


def _lengths(case):
    """(new tokens, tokens in the cache with them) of every sequence; a case of shared has one new token each."""
    rng = random.Random(case["lens"])
    had = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["B"])]
    if case["op"] == "shared":
        return [1] * case["B"], had
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return new, [a + b for a, b in zip(new, had)]


def work(case):
    new, lens = _lengths(case)
    Hq, Hkv, d, T = case["Hq"], case["Hkv"], case["d"], sum(new)
    kv_row = 2 * Hkv * d * 2
    tables = 4 * (sum(-(-n // case["page"]) for n in lens) + 2 * case["B"])
    if case["op"] == "append":
        # q, k and v in; q, and the cache's slots, out; a row of the angle table for each distinct position
        rows = len({p for a, n in zip(new, lens) for p in range(n - a, n)})
        return {"bytes": 2 * T * (Hq * d * 2 + kv_row) + rows * case["rot"] * 4 + tables, "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    qo = 2 * T * Hq * d * 2
    if case["op"] == "paged":
        if case["causal"]:
            pairs = sum(a * (n - a) + a * (a + 1) // 2 for a, n in zip(new, lens))
        else:
            pairs = sum(a * n for a, n in zip(new, lens))
        return {"bytes": qo + sum(lens) * kv_row + tables, "flops": 4 * pairs * Hq * d}
    keys = sum(lens) + case["prefix"]
    pairs = sum(lens) + case["prefix"] * case["B"]
    return {"bytes": qo + keys * kv_row + tables + 4 * -(-case["prefix"] // case["page"]), "flops": 4 * pairs * Hq * d}


def _angles(count, rot):
    """cos and sin of position x base^(-2 i / rot): [count, rot], the cosines first; in 64 bits."""
    freq = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    a = torch.arange(count, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[case["dtype"]]
    new, lens = _lengths(case)
    B, Hq, Hkv, d, S, T = case["B"], case["Hq"], case["Hkv"], case["d"], case["page"], sum(new)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case, "max_new": max(new)}

    # pages in any order, a few that belong to nobody; entries behind a sequence's last page are not valid
    need = [-(-n // S) for n in lens]
    shared = -(-case["prefix"] // S) if case["op"] == "shared" else 0
    count = sum(need) + shared + 3
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    width = max(need + [1]) + 1
    col = torch.arange(width, device="cuda")
    first = torch.tensor(need, device="cuda").cumsum(0) - torch.tensor(need, device="cuda")
    live = col < torch.tensor(need, device="cuda")[:, None]
    s["page_table"] = torch.where(live, order[(first[:, None] + col).clamp(max=count - 1)], -1).to(torch.int32)
    if shared:
        s["prefix_table"] = order[sum(need):sum(need) + shared].clone()
        s["prefix_len"] = ints([case["prefix"]])
    # keys carry a channel's own offset, as projections with rotary halves do; values do not
    shape = (count, S, Hkv, d) if case["slots_first"] else (count, Hkv, S, d)
    offset = randn(Hkv, d) if case["slots_first"] else randn(Hkv, 1, d)
    pages = [(randn(*shape) + offset).to(dt), randn(*shape).to(dt)]
    s["k_pages"], s["v_pages"] = (p.transpose(1, 2) if case["slots_first"] else p for p in pages)
    s["seq_lens"] = ints(lens)
    s["cu_seqlens"] = ints([0] + torch.tensor(new).cumsum(0).tolist())
    if case["op"] == "append":
        if case["fused"]:
            qkv = randn(T, Hq + 2 * Hkv, d).to(dt)
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = randn(T, Hq, d).to(dt), randn(T, Hkv, d).to(dt), randn(T, Hkv, d).to(dt)
        s["rope"] = _angles(max(lens), case["rot"]).float()
    else:
        s["q"] = (randn(T, Hq, d) * 1.5).to(dt)
    return s


# ---------------------------------------------------------------- plain forms
def _rotated(x, cs, case):
    rot = case["rot"]
    x = x.float()
    c, n = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if case["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * n, a * n + b * c], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _token_rows(s):
    """The sequence and the position of every packed token."""
    cu = s["cu_seqlens"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, s["seq_lens"].long()[b] - cu[b + 1] + t


def _plain_append(s):
    case, S, dt = s["case"], s["case"]["page"], s["q"].dtype
    b, pos = _token_rows(s)
    cs = s["rope"][pos]
    page, slot = s["page_table"][b, pos // S].long(), pos % S
    s["k_pages"][page, :, slot] = _rotated(s["k"], cs, case).to(dt)
    s["v_pages"][page, :, slot] = s["v"]
    return _rotated(s["q"], cs, case).to(dt), s["k_pages"], s["v_pages"]


def _gathered(pages, table):
    """[..., n] page ids -> [..., kv heads, n * slots, d] in 32 bits."""
    x = pages[table.clamp(min=0).long()].float()
    return x.transpose(-4, -3).flatten(-3, -2)


def _normed(scores, v):
    m = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (scores - m).exp()
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p @ v / total, 0.0)


def _plain_paged(s):
    case = s["case"]
    Hq, Hkv, d, B, N = case["Hq"], case["Hkv"], case["d"], case["B"], s["max_new"]
    k, v = _gathered(s["k_pages"], s["page_table"]), _gathered(s["v_pages"], s["page_table"])
    b, pos = _token_rows(s)
    row = torch.arange(b.numel(), device="cuda") - s["cu_seqlens"].long()[b]
    q = torch.zeros(B, N, Hq, d, device="cuda")
    q[b, row] = s["q"].float()
    q = q.view(B, N, Hkv, Hq // Hkv, d).transpose(1, 2).flatten(2, 3)  # [B, kv heads, N * group, d]
    lens = s["seq_lens"].long()
    last = lens[:, None].expand(B, N) - 1
    if case["causal"]:
        new = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long()
        last = (lens - new)[:, None] + torch.arange(N, device="cuda")
    seen = torch.arange(k.shape[2], device="cuda") <= torch.minimum(last, lens[:, None] - 1)[..., None]
    scores = (q @ k.transpose(-1, -2)) * d ** -0.5
    scores.masked_fill_(~seen.repeat_interleave(Hq // Hkv, 1)[:, None], -math.inf)
    o = _normed(scores, v).view(B, Hkv, N, Hq // Hkv, d).transpose(1, 2).reshape(B, N, Hq, d)
    return o[b, row].to(s["q"].dtype)


def _plain_shared(s):
    case = s["case"]
    Hq, Hkv, d, B, P = case["Hq"], case["Hkv"], case["d"], case["B"], case["prefix"]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    k0, v0 = _gathered(s["k_pages"], s["prefix_table"]), _gathered(s["v_pages"], s["prefix_table"])
    k1, v1 = _gathered(s["k_pages"], s["page_table"]), _gathered(s["v_pages"], s["page_table"])
    rows = q.transpose(0, 1).reshape(Hkv, -1, d)
    a = ((rows @ k0[:, :P].transpose(-1, -2)) * d ** -0.5).view(Hkv, B, Hq // Hkv, P)
    c = (q @ k1.transpose(-1, -2)) * d ** -0.5
    c.masked_fill_((torch.arange(k1.shape[2], device="cuda") >= s["seq_lens"][:, None])[:, None, None], -math.inf)
    m = torch.maximum(a.amax(-1).transpose(0, 1), c.amax(-1))[..., None]
    ea, ec = (a - m.transpose(0, 1)).exp(), (c - m).exp()
    total = ea.sum(-1).transpose(0, 1) + ec.sum(-1)
    o = (ea.flatten(1, 2) @ v0[:, :P]).view(Hkv, B, Hq // Hkv, d).transpose(0, 1) + ec @ v1
    return (o / total[..., None]).reshape(B, Hq, d).to(s["q"].dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        from attention_forward_prefill_gb300 import binding
        if op == "append":
            out = binding.cache_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"],
                                       cu_seqlens=s["cu_seqlens"], rope=s["rope"], interleaved=s["case"]["inter"])
            return out, s["k_pages"], s["v_pages"]
        if op == "shared":
            return binding.decode_shared(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix_len"],
                                         s["page_table"], s["seq_lens"])
        if s["max_new"] == 1:
            return binding.decode_paged(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"])
        return binding.prefill_paged(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["cu_seqlens"],
                                     s["max_new"], causal=s["case"]["causal"])
    return {"append": _plain_append, "paged": _plain_paged, "shared": _plain_shared}[op](s)


# ---------------------------------------------------------------- definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    new, lens = _lengths(case)
    Hq, Hkv, d, S, G = case["Hq"], case["Hkv"], case["d"], case["page"], case["Hq"] // case["Hkv"]
    table = s["page_table"].cpu().tolist()
    if case["op"] == "append":
        q, kp, vp = s["q"].double(), s["k_pages"].double(), s["v_pages"].double()
        rot, t0 = case["rot"], 0
        # (x1, x2) -> (x1 + i x2) e^{i angle}
        freq = torch.tensor([ROPE_BASE ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device="cuda")

        def turn(x, pos):
            if rot == 0:
                return x
            y = x.clone()
            one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(x[..., one].contiguous(), x[..., two].contiguous())
            angle = pos.double()[:, None] * freq
            z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
            y[..., one], y[..., two] = z.real, z.imag
            return y

        out = torch.empty_like(q)
        for b, (a, n) in enumerate(zip(new, lens)):
            pos = torch.arange(n - a, n, device="cuda")
            page = torch.tensor([table[b][p // S] for p in range(n - a, n)], device="cuda")
            rows = slice(t0, t0 + a)
            out[rows] = turn(q[rows], pos)
            kp[page, :, pos % S] = turn(s["k"][rows].double(), pos)
            vp[page, :, pos % S] = s["v"][rows].double()
            t0 += a
        return out, kp, vp
    out, t0 = torch.empty(sum(new), Hq, d, dtype=torch.float64, device="cuda"), 0
    front = s["prefix_table"].cpu().tolist() if case["op"] == "shared" else []
    for b, (a, n) in enumerate(zip(new, lens)):
        def keys(pages):
            own_pages = torch.tensor(table[b][:-(-n // S)], dtype=torch.long, device="cuda")
            mine = pages[own_pages].transpose(1, 2).reshape(-1, Hkv, d)[:n]
            if not front:
                return mine
            return torch.cat([pages[torch.tensor(front, device="cuda")].transpose(1, 2).reshape(-1, Hkv, d)[:case["prefix"]], mine])
        k, v = keys(s["k_pages"]), keys(s["v_pages"])
        for h in range(Hkv):
            q = s["q"][t0:t0 + a, h * G:(h + 1) * G].double()
            x = torch.einsum("tgd,jd->tgj", q, k[:, h].double()) / math.sqrt(d)
            if case.get("causal"):
                x = x.masked_fill(torch.ones(a, n, dtype=torch.bool, device="cuda").triu(n - a + 1)[:, None], -math.inf)
            out[t0:t0 + a, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", torch.softmax(x, -1), v[:, h].double())
        t0 += a
    return out
