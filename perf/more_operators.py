"""Operators of speculative decoding over the paged cache, as measured: page lists and slots of a step, positions
and ancestors of drafted trees, storing tokens by slot and position, attention of the drafted trees over the
cache, and keeping the accepted branch.

Each case names an operator (`op`) and its sizes.  `run` computes it in plain torch operations, or, with `own`
set, by the library's entry points."""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
BASE = 10000.0


def ops():
    from context_causal_attention_gb300 import ops as F
    return F


# ------------------------------------------------------------------ cases
def pages_case(name, B, new, old, back, ended, page, base, pad=0):
    """B sequences with up to `new` new tokens behind up to `old` cached ones, of which up to `back` drafted ones were
    rejected; every `ended`-th sequence (0: none) has ended and gives all its pages back."""
    return {"name": name, "op": "pages", "B": B, "new": new, "old": old, "back": back, "ended": ended, "page": page,
            "base": base, "pad": pad}


def branches_case(name, B, new, ragged, base, pad=0):
    return {"name": name, "op": "branches", "B": B, "new": new, "old": 500, "ragged": ragged, "prompts": 0, "prompt": 0,
            "base": base, "pad": pad}


def store_case(name, B, new, ragged, N, Nkv, D, page, dt, order, rot, norm, base, pad=0):
    return {"name": name, "op": "store", "B": B, "new": new, "old": 300, "ragged": ragged, "prompts": 0, "prompt": 0,
            "N": N, "Nkv": Nkv, "D": D, "page": page, "dt": dt, "order": order, "rot": rot, "norm": norm, "base": base,
            "pad": pad}


def attn_case(name, B, new, old, ragged, prefix, N, Nkv, D, page, pad=0, prompts=0, prompt=0):
    """Trees of up to `new` drafted tokens for each of B sequences, and `prompts` more sequences with an ordinary
    prompt of up to `prompt` tokens."""
    return {"name": name, "op": "attn", "B": B, "new": new, "old": old, "ragged": ragged, "prompts": prompts,
            "prompt": prompt, "prefix": prefix, "N": N, "Nkv": Nkv, "D": D, "page": page, "pad": pad}


def keep_case(name, B, new, most, layers, Nkv, D, page):
    """Up to `most` accepted tokens of trees of `new`, in the caches of K and V of `layers` layers."""
    return {"name": name, "op": "keep", "B": B, "new": new, "old": 60, "ragged": False, "prompts": 0, "prompt": 0,
            "most": most, "layers": layers, "Nkv": Nkv, "D": D, "page": page}


def listed():
    return [
        # a decode step of 64 sequences: a page now and then, only latency
        pages_case("pages_decode_b64", 64, 1, 4000, 0, 0, 16, 8192),
        # a large batch: prompts come in, some sequences end, drafted tokens were rejected
        pages_case("pages_mixed_b1000", 1000, 60, 3000, 20, 9, 32, 0, 40),
        # trees of up to 61 drafted tokens for 64 sequences, another tree in every step
        branches_case("branches_b64", 64, 61, True, 8192),
        # many wide trees, the largest masks
        branches_case("branches_b300_wide", 300, 500, True, 0, 7),
        # 16 drafted tokens for each of 64 sequences, q, k normed and rotated by their depth, k and v into the pages
        store_case("store_trees_b64", 64, 16, False, 32, 8, 128, 16, "bf16", "half", 128, True, 8192),
        # fp32 rows, keys and values alone, half of the head rotated, odd sizes and padding
        store_case("store_odd_fp32", 97, 131, True, 0, 5, 64, 64, "fp32", "interleaved", 32, False, 1001, 3),
        # one user, a tree of 27 tokens: latency
        attn_case("tree_attn_user", 1, 27, 4096, False, 0, 32, 8, 128, 16),
        # a step of 64 sequences of ragged lengths, 16 drafted tokens each
        attn_case("tree_attn_b64", 64, 16, 4096, True, 0, 32, 8, 128, 16),
        # 7 sequences behind a shared document, one KV head for each query head, odd lengths
        attn_case("tree_attn_prefix_b7", 7, 13, 1500, True, 100003, 16, 16, 64, 64, 2),
        # wide trees of 24 users beside the prompts of 6 others, behind a shared document
        attn_case("tree_attn_mixed", 24, 60, 1000, True, 16384, 32, 8, 128, 128, 0, 6, 1024),
        # one user of a small model: latency
        keep_case("keep_user", 1, 27, 6, 16, 2, 64, 16),
        # 64 sequences, 32 layers
        keep_case("keep_b64", 64, 16, 6, 32, 8, 128, 16),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def heads(rng):
    kv = rng.choice([1, 2, 3, 4, 8])
    return kv * rng.choice([1, 1, 2, 3, 4, 5, 7, 8]), kv


def draw(rng):
    op = rng.choice(["pages", "branches", "store", "keep", "attn", "attn", "attn"])
    N, Nkv = heads(rng)
    D = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "pages":
        B = spread(rng, 1, 2000)
        c = pages_case("", B, spread(rng, 1, max(1, 60000 // B)), spread(rng, 1, 6000) - 1, rng.choice([0, 1, 7, 60]),
                       rng.choice([0, 0, 3, 20]), page, rng.randrange(0, 200000), rng.choice([0, 0, 5, 300]))
    elif op == "branches":
        B = spread(rng, 1, 400)
        c = branches_case("", B, spread(rng, 1, min(512, max(1, 100000 // B))), rng.random() < 0.7,
                          rng.randrange(0, 200000), rng.choice([0, 0, 3]))
    elif op == "store":
        B = spread(rng, 1, 128)
        c = store_case("", B, spread(rng, 1, max(1, 16384 // B)), rng.random() < 0.7, rng.choice([0, N]), Nkv, D, page,
                       rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["half", "interleaved"]),
                       rng.choice([D, D, D // 2, D // 4]), rng.random() < 0.5, rng.randrange(0, 200000),
                       rng.choice([0, 0, 3]))
    elif op == "keep":
        B = spread(rng, 1, 64)
        new = spread(rng, 2, 64)
        c = keep_case("", B, new, rng.randrange(1, min(9, new // 2 + 1) + 1), rng.randrange(1, 33), Nkv, D, page)
    else:
        B = spread(rng, 1, 64)
        new = rng.choice([1, rng.randrange(2, 9), rng.randrange(9, 33), spread(rng, 1, max(1, min(200, 3500 // B)))])
        prompts = rng.choice([0, 0, 0, rng.randrange(1, 4)])
        prompt = rng.randrange(-(-new // 32) * 32 + 1, 700) if prompts else 0
        rows = B * new + prompts * prompt
        most = max(64, min(120000, 1_500_000_000 // (rows * N)))
        c = attn_case("", B, new, spread(rng, 1, max(64, min(6000, 300000 // B))) - 1, rng.random() < 0.8,
                      rng.choice([0, 0, spread(rng, 1, most)]), N, Nkv, D, page, rng.choice([0, 0, 3]), prompts, prompt)
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes that follow from a case
def words(case):
    """32-bit words of a row's mask: the widest tree's."""
    return -(-case["new"] // 32)


def lengths(case):
    """(new tokens, all own tokens) of each sequence; ragged ones spread from one token up to the case's size."""
    r = random.Random("%d %d %d" % (case["B"], case["new"], case["old"]))
    new, length = [], []
    for b in range(case["B"] + case["prompts"]):
        tree = b < case["B"]
        least, size = (1, case["new"]) if tree else (32 * words(case) + 1, case["prompt"])
        n = size if not case["ragged"] or b == 0 else r.randint(least, size)
        o = case["old"] if not case["ragged"] or b == 0 else r.randint(0, case["old"])
        new.append(n)
        length.append(o + n)
    return new, length


def accepted(case):
    """(kept tokens, how many of them stay where they are) of each sequence; -1 where all new tokens stay."""
    r = random.Random("%d %d %d" % (case["B"], case["new"], case["most"]))
    out = []
    for b in range(case["B"]):
        n = r.randint(1, case["most"]) if b else case["most"]
        n = min(n, case["new"] // 2 + 1)
        out.append((-1, 0) if b % 16 == 15 else (n, r.randint(max(1, 2 * n - case["new"]), n) if b else 1))
    return out


def step(case):
    """(tokens that had pages, tokens that stay, new tokens) of each sequence of a `pages` case."""
    r = random.Random("%d %d %d" % (case["B"], case["new"], case["old"]))
    had, stay, new = [], [], []
    for b in range(case["B"]):
        h = r.randint(0, case["old"])
        ended = bool(case["ended"]) and b % case["ended"] == case["ended"] - 1
        had.append(h)
        stay.append(0 if ended else max(0, h - r.randint(0, case["back"])))
        new.append(0 if ended else r.randint(1, case["new"]))
    return had, stay, new


def work(case):
    if case["op"] == "pages":
        had, stay, new = step(case)
        ps = case["page"]
        moved = sum(abs(-(-(s + n) // ps) - -(-h // ps)) for h, s, n in zip(had, stay, new))
        R = sum(new) + case["pad"]
        return {"bytes": 5.0 * 4 * case["B"] + 2.0 * 4 * moved + 8.0 * R, "flops": 0.0}
    new, length = lengths(case)
    R, B = sum(new), len(new)
    if case["op"] == "branches":
        return {"bytes": 8.0 * B + R * (8.0 + 4 * words(case)), "flops": 0.0}
    Nkv, D = case["Nkv"], case["D"]
    if case["op"] == "keep":
        moved = sum(n - s for n, s in accepted(case) if n > 0)
        return {"bytes": moved * 2.0 * case["layers"] * 2 * Nkv * D * 2 + 4.0 * B * (4 + case["most"]), "flops": 0.0}
    N = case["N"]
    if case["op"] == "store":
        es = 2 if case["dt"] == "bf16" else 4
        return {"bytes": R * (2.0 * Nkv + N) * D * (es + 2) + 8.0 * R, "flops": 3.0 * R * (N + Nkv) * case["rot"]}
    # every row sees its whole context; of its own step's tokens at least itself, at most those before it
    pairs = R * case["prefix"] + sum(n * (m - n) + n for n, m in zip(new, length))
    pairs += sum(n * (n - 1) // 2 for n in new[case["B"]:])
    return {"bytes": 2.0 * (case["prefix"] + sum(length)) * Nkv * D * 2 + R * (N * (D * 4.0 + 4) + 4 * words(case)),
            "flops": 4.0 * N * D * pairs}


# ------------------------------------------------------------------ inputs
def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def int32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def starts(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def pages_of(seed, counts, extra):
    """Distinct page numbers in random order: a list for each of `counts`, the `extra` spare ones, and how many."""
    total = sum(counts) + extra
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    out, at = [], 0
    for c in counts:
        out.append(order[at:at + c])
        at += c
    return out, order[at:], total


def table_of(lists, width):
    t = torch.zeros((len(lists), width), dtype=torch.int32)
    for b, x in enumerate(lists):
        t[b, :len(x)] = x
    return t.cuda()


def parents_of(g, st, rows):
    """A tree over each sequence's new tokens: each hangs on one of the eight before it, now and then on the cached
    tokens themselves (-1), as the first always does."""
    b, j = owners(st)
    u, v = (torch.rand(len(j), generator=g, device="cuda") for _ in range(2))
    p = j - 1 - (u * j.clamp(max=8)).long().clamp(max=7)
    p = torch.where((v < 0.03) | (j == 0), -1, p)
    out = torch.full((rows,), -5, dtype=torch.int32, device="cuda")
    out[:len(j)] = p.to(torch.int32)
    return out


def prepare_pages(case, seed, st):
    had, stay, new = step(case)
    ps = case["page"]
    counts = [-(-h // ps) for h in had]
    need = [-(-(s + n) // ps) for s, n in zip(stay, new)]
    lists, spare, total = pages_of(seed, counts, sum(max(0, n - c) for n, c in zip(need, counts)) + 5)
    st["rows"] = sum(new) + case["pad"]
    st["table"] = table_of(lists, max(1, max(need), max(counts)))
    st["had"], st["stay"], st["new_tokens"] = int32(had), int32(stay), int32(new)
    st["free"] = torch.full((total,), -1, dtype=torch.int32)
    st["free"][:len(spare)] = spare
    st["free"] = st["free"].cuda()
    st["n_free"] = int32([len(spare), 0])
    st["kv_len"], st["cu"] = torch.zeros_like(st["had"]), int32([0] * (case["B"] + 1))
    st["slots"], st["pos"] = (int32([0] * st["rows"]) for _ in range(2))
    st["n_free_out"] = torch.zeros_like(st["n_free"])
    return st


def prepare(case, seed):
    g = generator(seed)
    st = {"case": case}
    if case["op"] == "pages":
        return prepare_pages(case, seed, st)
    new, length = lengths(case)
    B, R = len(new), sum(new) + case.get("pad", 0)
    st["new"], st["length"] = new, length
    st["cu"], st["kv_len"] = int32(starts(new)), int32(length)
    if case["op"] != "keep":
        st["parent"] = parents_of(g, st, R)
    if case["op"] == "branches":
        st["mask"] = torch.zeros(R, words(case), dtype=torch.int32, device="cuda")
        st["pos"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        return st
    Nkv, D, ps, prefix = case["Nkv"], case["D"], case["page"], case.get("prefix", 0)
    counts = [-(-m // ps) for m in length]
    lists, _, total = pages_of(seed, counts + [-(-prefix // ps)], 3)
    st["table"] = table_of(lists[:-1], max(1, max(counts)))
    if case["op"] == "keep":
        st["caches"] = torch.randn(2 * case["layers"], total, ps, Nkv, D, generator=g, device="cuda", dtype=torch.bfloat16)
        r = random.Random(seed)
        kept = torch.full((B, case["most"]), -9, dtype=torch.int32)
        for b, (n, s) in enumerate(accepted(case)):
            # a level-ordered tree's branch: the places that it moves to are not the ones that it moves from, so
            # a pass can be repeated on its own result
            if n > 0:
                kept[b, :n] = torch.tensor(list(range(s)) + sorted(r.sample(range(n, case["new"]), n - s)))
        st["kept"], st["n_kept"] = kept.cuda(), int32([n for n, _ in accepted(case)])
        st["moving"] = sum(max(0, n) for n, _ in accepted(case))
        st["kv_keep"] = torch.zeros_like(st["kv_len"])
        if own:
            st["handle"] = ops().CpCaches(list(st["caches"]))
        return st
    N = case["N"]
    st["k_cache"], st["v_cache"] = (torch.randn(total, ps, Nkv, D, generator=g, device="cuda", dtype=torch.bfloat16)
                                    for _ in range(2))
    if case["op"] == "store":
        dt = DT[case["dt"]]
        # one row of the fused projection holds the q, k and v heads of a token
        qkv = torch.randn(R, N + 2 * Nkv, D, generator=g, device="cuda").to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :N] if N else None, qkv[:, N:N + Nkv], qkv[:, N + Nkv:]
        st["wk"] = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda") if case["norm"] else None
        st["wq"] = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda") if case["norm"] and N else None
        st["q_out"] = torch.zeros(R, N, D, dtype=torch.bfloat16, device="cuda") if N else None
        b, i = own_index(st)
        rows = len(i)
        st["slots"] = torch.full((R,), -1, dtype=torch.int32, device="cuda")
        st["slots"][:rows] = (st["table"].long()[b, i // ps] * ps + i % ps).to(torch.int32)
        st["pos"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        st["pos"][:rows] = tree_of(st)[1].to(torch.int32) + case["base"]
        if own:
            F = ops()
            st["rope"] = F.cp_rope_freqs(case["rot"], base=BASE, device="cuda",
                                         order=F.CP_ROPE_HALF if case["order"] == "half" else F.CP_ROPE_INTERLEAVED)
        return st
    st["prefix_pages"] = torch.cat([lists[-1], torch.zeros(1 if not len(lists[-1]) else 0, dtype=torch.int32)]).cuda()
    # a prompt's rows have no mask: whatever stands there is not read
    st["mask"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (R, words(case)), generator=g, device="cuda", dtype=torch.int32)
    drafted = starts(new)[case["B"]]
    st["mask"][:drafted] = packed(tree_of(st)[0], words(case))[:drafted]
    st["q"] = torch.randn(R, N, D, generator=g, device="cuda", dtype=torch.bfloat16)
    st["o"] = torch.zeros(R, N, D, dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.zeros(N, R, device="cuda")
    if own:
        n = ops().cp_tree_attn_workspace_size(R, B, max(new), words(case), prefix, N, Nkv, D, ps, st["table"].shape[1])
        st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def owners(st):
    """Sequence and place among its new tokens of each new token, in the order of the rows."""
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    rows = sum(st["new"])
    b = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=rows)
    return b, torch.arange(rows, device="cuda") - st["cu"].long()[b]


def own_index(st):
    """Sequence and own index of each new token."""
    b, j = owners(st)
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    return b, (st["kv_len"].long() - n)[b] + j


def tree_of(st):
    """([rows, widest tree] truth values: token i is row's ancestor or itself; own position by depth [rows]).  Rows of
    prompts (more tokens than the mask's words hold) get their index, and no ancestors that matter."""
    case = st["case"]
    b, j = owners(st)
    wide = 32 * words(case)
    # a prompt's tokens behind the mask's width share one more place
    jt, up = j.clamp(max=wide), st["parent"][:len(b)].long()
    edge = torch.zeros(len(st["new"]), wide + 1, wide + 1, device="cuda")
    edge[b, jt, jt] = 1.0
    # an edge to the parent; a token without one has its own place marked twice
    edge[b, jt, torch.where((up < 0) | (j >= wide), jt, up)] = 1.0
    # paths of up to 1, 2, 4, ... edges
    for _ in range(max(1, wide - 1).bit_length()):
        edge = (torch.bmm(edge, edge) > 0).float()
    seen = edge[b, jt, :wide] > 0
    n = (st["cu"][1:] - st["cu"][:-1]).long()[b]
    depth = torch.where(n > wide, j, seen.sum(-1) - 1)
    return seen, (st["kv_len"].long()[b] - n) + depth


def packed(seen, w):
    """Truth values [rows, 32 w] as 32-bit words."""
    bits = seen.view(-1, w, 32).long() << torch.arange(32, device="cuda")
    return bits.sum(-1).to(torch.int32)


def plain_branches(st):
    seen, pos = tree_of(st)
    rows = len(pos)
    st["mask"][:rows] = packed(seen, words(st["case"]))
    st["pos"][:rows] = (pos + st["case"]["base"]).to(torch.int32)
    return [st["mask"], st["pos"]]


def plain_pages(st):
    case = st["case"]
    ps, R, dev = case["page"], st["rows"], "cuda"
    had, stay, new = st["had"].long(), st["stay"].long(), st["new_tokens"].long()
    length = stay + new
    owned, need = (had + ps - 1) // ps, (length + ps - 1) // ps
    take, give = (need - owned).clamp(min=0), (owned - need).clamp(min=0)
    width = torch.arange(st["table"].shape[1], device=dev)
    # pages given back go on the stack in the order of the sequences
    back = (width >= need[:, None]) & (width < owned[:, None])
    top = st["n_free"][0].long() + (give.cumsum(0) - give)[:, None] + width - need[:, None]
    last = len(st["free"])
    stack = torch.cat([st["free"], st["free"][:1]])
    stack[torch.where(back, top, last)] = st["table"]
    st["free"].copy_(stack[:last])
    # pages taken come off its top, in the same order
    top = st["n_free"][0].long() + give.sum()
    fresh = (width >= owned[:, None]) & (width < need[:, None])
    at = top - 1 - ((take.cumsum(0) - take)[:, None] + width - owned[:, None])
    st["table"].copy_(torch.where(fresh, st["free"][torch.where(fresh, at, 0)], st["table"]))
    st["n_free_out"][0] = top - take.sum()
    st["n_free_out"][1] = 0
    st["kv_len"].copy_(length)
    ends = new.cumsum(0)
    st["cu"][1:] = ends
    row = torch.arange(R, device=dev)
    b = torch.searchsorted(ends, row, right=True).clamp(max=len(had) - 1)
    i = stay[b] + row - (ends - new)[b]
    real = row < ends[-1]
    i = torch.where(real, i, 0)
    st["slots"].copy_(torch.where(real, st["table"].long()[b, i // ps] * ps + i % ps, -1))
    st["pos"].copy_(torch.where(real, i + case["base"], 0))
    return [st["kv_len"], st["cu"], st["slots"], st["pos"], st["table"], st["free"], st["n_free_out"]]


def angles(pos, rot):
    """cos and sin of every (position, pair) in 32 bits, from angles in 64."""
    theta = BASE ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    a = pos.double()[..., None] * theta
    return torch.cos(a).float(), torch.sin(a).float()


def turned_rows(x, w, cs, order, rot):
    """Rows x [R, heads, D] through the norm (where it has weights) and the rotation, in fp32."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    c, s = cs[0][:, None, :], cs[1][:, None, :]
    y = x.clone()
    if order == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    return y


def plain_store(st):
    case = st["case"]
    rows = sum(st["new"])
    at, cs = st["slots"][:rows].long(), angles(st["pos"][:rows], case["rot"])
    keys = turned_rows(st["k"][:rows], st["wk"], cs, case["order"], case["rot"])
    st["k_cache"].view(-1, case["Nkv"], case["D"])[at] = keys.to(torch.bfloat16)
    st["v_cache"].view(-1, case["Nkv"], case["D"])[at] = st["v"][:rows].to(torch.bfloat16)
    if st["q"] is None:
        return [st["k_cache"], st["v_cache"]]
    st["q_out"][:rows] = turned_rows(st["q"][:rows], st["wq"], cs, case["order"], case["rot"]).to(torch.bfloat16)
    return [st["k_cache"], st["v_cache"], st["q_out"]]


def plain_keep(st):
    ps = st["case"]["page"]
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    first, kept = st["kv_len"].long() - n, st["n_kept"].long()
    moved = kept.clamp(min=0)
    b = torch.repeat_interleave(torch.arange(len(n), device="cuda"), moved, output_size=st["moving"])
    j = torch.arange(st["moving"], device="cuda") - (moved.cumsum(0) - moved)[b]
    table = st["table"].long()
    source, target = first[b] + st["kept"].long()[b, j], first[b] + j
    source, target = (table[b, i // ps] * ps + i % ps for i in (source, target))
    rows = st["caches"].flatten(1, 2)
    rows[:, target] = rows[:, source]
    st["kv_keep"].copy_(torch.where(kept < 0, st["kv_len"].long(), first + kept))
    return [st["caches"], st["kv_keep"]]


def partial(q, k, v, hidden=None):
    """q [B, n, Nkv, G, D] against k, v [B, L, Nkv, D]: row maxima, sums and values of exp(scores - maximum), each
    [B, n, Nkv, G(, D)]; `hidden` [B, n, L] marks the keys that a row does not see."""
    s = torch.einsum("bnhgd,blhd->bnhgl", q, k) / math.sqrt(q.shape[-1])
    if hidden is not None:
        s = s.masked_fill(hidden[:, :, None, None], -math.inf)
    m = s.amax(-1)
    p = torch.exp(s - m[..., None])
    return m, p.sum(-1), torch.einsum("bnhgl,blhd->bnhgd", p, v)


def plain_attn(st):
    case = st["case"]
    N, Nkv, D, ps, P = case["N"], case["Nkv"], case["D"], case["page"], case["prefix"]
    b, j = owners(st)
    rows, most, longest = len(j), max(st["new"]), max(st["length"])
    B = len(st["new"])
    q = st["q"][:rows].float().view(rows, Nkv, N // Nkv, D)
    # each sequence's own keys, in a batch padded to the longest
    padded = torch.zeros(B, most, *q.shape[1:], device="cuda")
    padded[b, j] = q
    pages = st["table"][:, :-(-longest // ps)].long()
    k, v = (c[pages].flatten(1, 2)[:, :longest].float() for c in (st["k_cache"], st["v_cache"]))
    # which of its own step's tokens a row sees: its mask's bits, or in a prompt those up to itself
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    w = words(case)
    i = torch.arange(longest, device="cuda") - (st["kv_len"].long() - n)[:, None]  # of each key among the new tokens
    bits = torch.zeros(B, most, w + 1, dtype=torch.int32, device="cuda")
    bits[b, j, :w] = st["mask"][:rows]
    word = torch.where((i >= 0) & (i < 32 * w), i >> 5, w)
    bit = bits.gather(2, word[:, None].expand(B, most, longest)) >> (i & 31)[:, None] & 1
    late = i[:, None] > torch.arange(most, device="cuda")[:, None]
    hidden = torch.where((n > 32 * w)[:, None, None], late, (i >= 0)[:, None] & (bit == 0))
    hidden = hidden | (i >= n[:, None])[:, None]
    del bit, late
    m, total, acc = (t[b, j] for t in partial(padded, k, v, hidden))
    if P:
        pages = st["prefix_pages"][:-(-P // ps)].long()
        k, v = (c[pages].flatten(0, 1)[None, :P].float() for c in (st["k_cache"], st["v_cache"]))
        m2, total2, acc2 = (t[0] for t in partial(q[None], k, v))
        top = torch.maximum(m, m2)
        f, f2 = torch.exp(m - top), torch.exp(m2 - top)
        m, total, acc = top, total * f + total2 * f2, acc * f[..., None] + acc2 * f2[..., None]
    st["o"][:rows] = (acc / total[..., None]).flatten(1, 2).to(st["o"].dtype)
    st["lse"][:, :rows] = (m + torch.log(total)).flatten(1, 2).T
    return [st["o"], st["lse"]]


PLAIN = {"pages": plain_pages, "branches": plain_branches, "store": plain_store, "keep": plain_keep, "attn": plain_attn}


def run(state):
    return run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the library's entry points
def run_own(st):
    F, case = ops(), st["case"]
    if case["op"] == "pages":
        F.cp_cache_plan(st["had"], st["stay"], st["new_tokens"], st["table"], st["free"], st["n_free"], case["page"],
                        st["rows"], pos_base=case["base"], kv_len=st["kv_len"], cu_new=st["cu"], slots=st["slots"],
                        pos=st["pos"], n_free_out=st["n_free_out"])
        return [st["kv_len"], st["cu"], st["slots"], st["pos"], st["table"], st["free"], st["n_free_out"]]
    if case["op"] == "branches":
        return list(F.cp_tree_plan(st["parent"], st["cu"], st["kv_len"], words(case), pos_base=case["base"],
                                   mask=st["mask"], pos=st["pos"]))
    if case["op"] == "store":
        F.cp_cache_append_at(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"], st["pos"], rope=st["rope"],
                             q=st["q"], q_out=st["q_out"], wq=st["wq"], wk=st["wk"], eps=EPS)
        return [st["k_cache"], st["v_cache"]] + ([] if st["q"] is None else [st["q_out"]])
    if case["op"] == "keep":
        F.cp_cache_keep(st["handle"], st["table"], st["cu"], st["kv_len"], st["kept"], st["n_kept"], kv_keep=st["kv_keep"])
        return [st["caches"], st["kv_keep"]]
    return list(F.cp_tree_attn_fwd(st["q"], st["k_cache"], st["v_cache"], st["mask"], st["prefix_pages"],
                                   case["prefix"], st["table"], st["cu"], st["kv_len"], max(st["new"]), o=st["o"],
                                   lse=st["lse"], workspace=st["ws"]))


# ------------------------------------------------------------------ 64 bits
def exact_store(st):
    case = st["case"]
    rot, ps = case["rot"], case["page"]
    freq = torch.tensor([math.exp(-2.0 * i / rot * math.log(BASE)) for i in range(rot // 2)], dtype=torch.float64).cuda()
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    qo = st["q_out"].double() if st["q"] is not None else None
    n = sum(st["new"])
    phase = torch.outer(st["pos"][:n].double(), freq)
    z = torch.polar(torch.ones_like(phase), phase)[:, None]
    page, place = st["slots"][:n].long() // ps, st["slots"][:n].long() % ps

    def normed_and_turned(x, w):
        y = x[:n].double()
        if w is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["D"] + EPS) * w.double()
        r = y[..., :rot]
        half = case["order"] == "half"
        pairs = r.unflatten(-1, (2, rot // 2)).movedim(-2, -1) if half else r.unflatten(-1, (rot // 2, 2))
        t = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        return torch.cat([(t.movedim(-1, -2) if half else t).flatten(-2), y[..., rot:]], -1)

    kc[page, place] = normed_and_turned(st["k"], st["wk"])
    vc[page, place] = st["v"][:n].double()
    if qo is None:
        return [kc, vc]
    qo[:n] = normed_and_turned(st["q"], st["wq"])
    return [kc, vc, qo]


def exact_keep(st):
    caches, ps = st["caches"].double(), st["case"]["page"]
    table, kept = st["table"].tolist(), st["kept"].tolist()
    for b, (n, m, count) in enumerate(zip(st["new"], st["length"], st["n_kept"].tolist())):
        def place(i):
            return table[b][(m - n + i) // ps], (m - n + i) % ps
        rows = [caches[:, place(i)[0], place(i)[1]].clone() for i in kept[b][:max(0, count)]]
        for i, x in enumerate(rows):
            caches[:, place(i)[0], place(i)[1]] = x
    return [caches, None]


def exact_attn(st):
    case = st["case"]
    N, Nkv, ps, P = case["N"], case["Nkv"], case["page"], case["prefix"]
    o, lse = st["o"].double(), st["lse"].double()
    kc, vc = (c.flatten(0, 1) for c in (st["k_cache"], st["v_cache"]))
    parent = st["parent"].tolist()

    def at(pages, count):
        i = torch.arange(count, device="cuda")
        return pages.long()[i // ps] * ps + i % ps

    shared = at(st["prefix_pages"], P)
    row = 0
    for b, (n, m) in enumerate(zip(st["new"], st["length"])):
        where = torch.cat([shared, at(st["table"][b], m)])
        seen = torch.ones(n, P + m, dtype=torch.bool)
        seen[:, P + m - n:] = torch.tril(torch.ones(n, n, dtype=torch.bool))
        if b < case["B"]:
            # from each token up to the last without a parent
            branch = torch.zeros(n, n, dtype=torch.bool)
            for j in range(n):
                up = parent[row + j]
                if up >= 0:
                    branch[j] = branch[up]
                branch[j, j] = True
            seen[:, P + m - n:] = branch
        seen = seen.cuda()
        for h in range(N):
            k, v = kc[where, h // (N // Nkv)].double(), vc[where, h // (N // Nkv)].double()
            s = st["q"][row:row + n, h].double() @ k.T / math.sqrt(case["D"])
            s = torch.where(seen, s, -math.inf)
            e = torch.logsumexp(s, -1)
            lse[h, row:row + n] = e
            o[row:row + n, h] = torch.exp(s - e[:, None]) @ v
        row += n
    return [o, lse]


def exact(case, seed):
    if case["op"] in ("pages", "branches"):
        return None  # whole numbers
    if case["op"] == "attn" and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    return {"store": exact_store, "keep": exact_keep, "attn": exact_attn}[case["op"]](st)
