"""Operators around the attention, as measured: rotary positions, per-head norm
with rotation, appending to a paged cache, and attention over a shared prefix.

Each case names an operator (`op`) and its sizes.  `run` computes it in plain
torch operations, or, with `own` set, by the library's entry points."""
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
def rope_case(name, dirn, C, B, s, N, Nkv, D, dt, order, rot, scaling="none", pos0=0, fused=False):
    return {"name": name, "op": "rope", "dir": dirn, "C": C, "B": B, "s": s, "N": N, "Nkv": Nkv, "D": D, "dt": dt,
            "order": order, "rot": rot, "scaling": scaling, "pos0": pos0, "fused": fused}


def norm_case(name, dirn, C, B, s, N, Nkv, D, dt, order, rot, scaling="none", pos0=0, fused=False):
    return dict(rope_case(name, dirn, C, B, s, N, Nkv, D, dt, order, rot, scaling, pos0, fused), op="norm")


def append_case(name, B, new, old, ragged, N, Nkv, D, page, dt, order, rot, norm, base, pad=0):
    return {"name": name, "op": "append", "B": B, "new": new, "old": old, "ragged": ragged, "N": N, "Nkv": Nkv, "D": D,
            "page": page, "dt": dt, "order": order, "rot": rot, "norm": norm, "base": base, "pad": pad}


def attn_case(name, B, new, old, ragged, prefix, N, Nkv, D, page, out, pad=0):
    return {"name": name, "op": "attn", "B": B, "new": new, "old": old, "ragged": ragged, "prefix": prefix, "N": N,
            "Nkv": Nkv, "D": D, "page": page, "out": out, "pad": pad}


def listed():
    return [
        # q and k of the four zigzag shards of a 32768-token sequence, before the ring
        rope_case("rope_fwd_ring_s32k", "fwd", 4, 1, 8192, 32, 32, 128, "bf16", "half", 128),
        # gradients on their way back, fp32 shards of two 4096-token sequences, half of the head rotated
        rope_case("rope_bwd_ring_s4k", "bwd", 4, 2, 1024, 16, 16, 64, "fp32", "interleaved", 32, "by_parts"),
        # one token of one user: only latency
        norm_case("norm_fwd_token", "fwd", 1, 1, 1, 32, 8, 128, "bf16", "half", 128, "none", 70000),
        # a long prompt, q and k read out of the fused projection's rows
        norm_case("norm_fwd_s32k", "fwd", 4, 1, 8192, 32, 8, 128, "bf16", "half", 128, "none", 0, True),
        # its gradient in training
        norm_case("norm_bwd_s32k", "bwd", 4, 1, 8192, 32, 8, 128, "bf16", "half", 128),
        # odd batch and length, full precision, a quarter of the head rotated at far positions
        norm_case("norm_bwd_odd_fp32", "bwd", 1, 3, 777, 12, 4, 64, "fp32", "interleaved", 16, "linear", 1000003),
        # a decode step of 64 sequences: q, k normed and rotated, k and v put into the pages
        append_case("append_decode_b64", 64, 1, 4000, True, 32, 8, 128, 16, "bf16", "half", 128, True, 8192),
        # ragged prompts of eight sequences behind a shared prefix, some rows of padding at the end
        append_case("append_prompts", 8, 4096, 0, True, 0, 8, 128, 64, "bf16", "half", 128, False, 1001, 13),
        # one user, one token: only latency
        attn_case("attn_token", 1, 1, 300, False, 4096, 32, 8, 128, 16, "bf16"),
        # a decode step of 64 sequences behind a shared prefix
        attn_case("attn_decode_b64", 64, 1, 2048, True, 32768, 32, 8, 128, 16, "bf16"),
        # five drafted tokens for each of 7 sequences, one KV head for each query head, odd lengths
        attn_case("attn_draft_b7", 7, 5, 1500, True, 100003, 16, 16, 64, 64, "bf16", 2),
        # ragged questions of eight users behind a shared document
        attn_case("attn_prompts", 8, 1024, 100, True, 16384, 32, 8, 128, 128, "bf16"),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def heads(rng):
    kv = rng.choice([1, 2, 3, 4, 8])
    return kv * rng.choice([1, 1, 2, 3, 4, 5, 7, 8]), kv


def draw(rng):
    op = rng.choice(["rope", "norm", "append", "attn", "attn"])
    N, Nkv = heads(rng)
    D = rng.choice([64, 128])
    order = rng.choice(["half", "interleaved"])
    rot = rng.choice([D, D, D // 2, D // 4])
    dt = rng.choice(["bf16", "bf16", "fp32"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("rope", "norm"):
        C = rng.choice([1, 1, 2, 4])
        B = rng.choice([1, 1, 2, 3])
        s = spread(rng, 1, 8192 // B)
        c = rope_case("", rng.choice(["fwd", "bwd"]), C, B, s, N, Nkv, D, dt, order, rot,
                      rng.choice(["none", "linear", "base", "by_parts"]), rng.randrange(0, 1 << 20),
                      rng.random() < 0.4)
        c["op"] = op
        if c["dir"] == "bwd":
            c["fused"] = False
    elif op == "append":
        B = spread(rng, 1, 128)
        c = append_case("", B, spread(rng, 1, max(1, 16384 // B)), rng.randrange(0, 3000), rng.random() < 0.7,
                        rng.choice([0, N]), Nkv, D, page, dt, order, rot, rng.random() < 0.5, rng.randrange(0, 200000),
                        rng.choice([0, 0, 3]))
    else:
        B = spread(rng, 1, 96)
        new = rng.choice([1, 1, rng.randrange(1, 9), spread(rng, 1, max(1, 3500 // B))])
        most = max(64, min(120000, 1_500_000_000 // (B * new * N)))
        c = attn_case("", B, new, spread(rng, 1, 4000) - 1, rng.random() < 0.8,
                      rng.choice([0, spread(rng, 1, most), spread(rng, 1, most)]), N, Nkv, D, page,
                      "bf16", rng.choice([0, 0, 3]))
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes that follow from a case
def lengths(case):
    """(new tokens, all own tokens) of each sequence; ragged ones spread from one token up to the case's size."""
    r = random.Random("%d %d %d" % (case["B"], case["new"], case["old"]))
    new, length = [], []
    for b in range(case["B"]):
        n = case["new"] if not case["ragged"] or b == 0 else r.randint(1, case["new"])
        o = case["old"] if not case["ragged"] or b == 0 else r.randint(0, case["old"])
        new.append(n)
        length.append(o + n)
    return new, length


def work(case):
    es = 2 if case.get("dt", "bf16") == "bf16" else 4
    N, Nkv, D = case["N"], case["Nkv"], case["D"]
    if case["op"] in ("rope", "norm"):
        t = case["C"] * case["B"] * case["s"]
        passes = 3 if case["op"] == "norm" and case["dir"] == "bwd" else 2
        b = t * (N + Nkv) * D * es * passes + 4 * case["C"] * case["s"]
        f = t * (N + Nkv) * (3.0 * case["rot"] + (4.0 * D if case["op"] == "norm" else 0) * (passes - 1))
        return {"bytes": float(b), "flops": f}
    new, length = lengths(case)
    R = sum(new)
    if case["op"] == "append":
        return {"bytes": float(R * (2 * Nkv + N) * D * (es + 2)), "flops": 3.0 * R * (N + Nkv) * case["rot"]}
    pairs = R * case["prefix"] + sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(new, length))
    out = 2 if case["out"] == "bf16" else 4
    return {"bytes": float(2 * (case["prefix"] + sum(length)) * Nkv * D * 2 + R * N * (D * (2 + out) + 4)),
            "flops": 4.0 * N * D * pairs}


# ------------------------------------------------------------------ inputs
SCALING = {"none": (1.0, 0), "linear": (4.0, 0), "base": (8.0, 0), "by_parts": (16.0, 4096)}


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def shard_positions(C, s, pos0):
    """Global positions of C zigzag shards of s tokens (contiguous ones where s is odd)."""
    if s % 2:
        p = torch.arange(C * s).view(C, s)
    else:
        t = s // 2
        p = torch.stack([torch.cat([torch.arange(r * t, r * t + t), torch.arange((2 * C - 1 - r) * t, (2 * C - r) * t)])
                         for r in range(C)])
    return (p + pos0).to(torch.int32).cuda()


def pages_of(seed, counts, extra):
    """Distinct page numbers in random order: a list for each of `counts`, out of all pages and `extra` spare ones."""
    total = sum(counts) + extra
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    out, at = [], 0
    for c in counts:
        out.append(order[at:at + c])
        at += c
    return out, total


def table_of(lists):
    t = torch.zeros((len(lists), max(1, max(len(x) for x in lists))), dtype=torch.int32)
    for b, x in enumerate(lists):
        t[b, :len(x)] = x
    return t.cuda()


def own_rope(case, rot, order, scaling):
    F = ops()
    kind = {"none": F.CP_ROPE_PLAIN, "linear": F.CP_ROPE_LINEAR, "base": F.CP_ROPE_BASE, "by_parts": F.CP_ROPE_BY_PARTS}
    factor, length = SCALING[scaling]
    return F.cp_rope_freqs(rot, base=BASE, scaling=kind[scaling], factor=factor, original_len=length,
                           order=F.CP_ROPE_HALF if order == "half" else F.CP_ROPE_INTERLEAVED, device="cuda")


def weights(g, D):
    return [1.0 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]


def prepare(case, seed):
    g = generator(seed)
    st = {"case": case}
    N, Nkv, D = case["N"], case["Nkv"], case["D"]
    if case["op"] in ("rope", "norm"):
        dt = DT[case["dt"]]
        lead = (case["C"], case["B"], case["s"])
        if case["fused"]:
            # one row of the fused projection holds the q, k and v heads of a token
            qkv = torch.randn(*lead, N + 2 * Nkv, D, generator=g, device="cuda").to(dt)
            st["q"], st["k"] = qkv[..., :N, :], qkv[..., N:N + Nkv, :]
        else:
            st["q"] = torch.randn(*lead, N, D, generator=g, device="cuda").to(dt)
            st["k"] = torch.randn(*lead, Nkv, D, generator=g, device="cuda").to(dt)
        st["pos"] = shard_positions(case["C"], case["s"], case["pos0"])
        st["wq"], st["wk"] = weights(g, D) if case["op"] == "norm" else (None, None)
        if case["dir"] == "bwd" and case["op"] == "norm":
            st["gq"] = torch.randn(*lead, N, D, generator=g, device="cuda").to(dt)
            st["gk"] = torch.randn(*lead, Nkv, D, generator=g, device="cuda").to(dt)
        if own:
            st["rope"] = own_rope(case, case["rot"], case["order"], case["scaling"])
            st["oq"] = torch.empty(*lead, N, D, dtype=dt, device="cuda")
            st["ok"] = torch.empty(*lead, Nkv, D, dtype=dt, device="cuda")
            if case["dir"] == "bwd" and case["op"] == "norm":
                st["dwq"], st["dwk"] = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
                n = ops().cp_qk_norm_rope_bwd_workspace_size(case["C"], case["B"], case["s"], N, Nkv, D)
                st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        return st
    new, length = lengths(case)
    ps, R = case["page"], sum(new) + case["pad"]
    st["new"], st["length"] = new, length
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
    st["kv_len"] = torch.tensor(length, dtype=torch.int32).cuda()
    prefix = case.get("prefix", 0)
    lists, total = pages_of(seed, [-(-m // ps) for m in length] + [-(-prefix // ps)], 3)
    st["table"] = table_of(lists[:-1])
    st["prefix_pages"] = torch.cat([lists[-1], torch.zeros(1 if not len(lists[-1]) else 0, dtype=torch.int32)]).cuda()
    st["k_cache"] = torch.randn(total, ps, Nkv, D, generator=g, device="cuda").to(torch.bfloat16)
    st["v_cache"] = torch.randn(total, ps, Nkv, D, generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] == "append":
        dt = DT[case["dt"]]
        qkv = torch.randn(R, N + 2 * Nkv, D, generator=g, device="cuda").to(dt)
        st["q"] = qkv[:, :N] if N else None
        st["k"], st["v"] = qkv[:, N:N + Nkv], qkv[:, N + Nkv:]
        st["wq"], st["wk"] = weights(g, D) if case["norm"] else (None, None)
        if not N:
            st["wq"] = None
        st["q_out"] = torch.zeros(R, N, D, dtype=torch.bfloat16, device="cuda") if N else None
        if own:
            st["rope"] = own_rope(case, case["rot"], case["order"], "none")
        return st
    st["q"] = torch.randn(R, N, D, generator=g, device="cuda").to(torch.bfloat16)
    st["o"] = torch.zeros(R, N, D, dtype=DT[case["out"]], device="cuda")
    st["lse"] = torch.zeros(N, R, device="cuda")
    if own:
        n = ops().cp_prefix_attn_workspace_size(R, case["B"], max(new), prefix, N, Nkv, D, ps, st["table"].shape[1])
        st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def frequencies(rot, scaling):
    """Radians per position of each pair, and the factor on the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    s, length = SCALING[scaling]
    theta = BASE ** (-2.0 * i / rot)
    if scaling == "linear":
        return theta / s, 1.0
    if scaling == "base":
        return (BASE * s ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    if scaling == "by_parts":
        turns = length * theta / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return theta * keep + theta / s * (1 - keep), 0.1 * math.log(s) + 1.0
    return theta, 1.0


def angles(pos, rot, scaling):
    """cos and sin of every (position, pair), with the factor, in 32 bits from angles in 64."""
    theta, amp = frequencies(rot, scaling)
    a = pos.double()[..., None] * theta
    return (torch.cos(a) * amp).float(), (torch.sin(a) * amp).float()


def rotate(x, cs, order, rot, back=False):
    """x [..., heads, D] in fp32 turned by cs = (cos, sin) [..., rot/2]; `back` by the negative angles."""
    c, s = cs[0][..., None, :], cs[1][..., None, :]
    if back:
        s = -s
    y = x.clone()
    if order == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    return y


def normed(x):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def plain_turned(st, cs, x, w):
    """One of q and k through the norm (where it has weights) and the rotation."""
    case, y = st["case"], x.float()
    if w is not None:
        y = normed(y)[0] * w
    return rotate(y, cs, case["order"], case["rot"])


def plain_norm_bwd(st, cs, x, w, g):
    """Gradients of one of q and k and of its weights from the gradient g of the rotated rows."""
    case = st["case"]
    g = rotate(g.float(), cs, case["order"], case["rot"], True)
    xh, r = normed(x.float())
    u = g * w
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xh).flatten(0, -2).double().sum(0).float()


def plain_rows(st):
    """rope and norm, forward and backward."""
    case, q, k = st["case"], st["q"], st["k"]
    cs = tuple(t[:, None] for t in angles(st["pos"], case["rot"], case["scaling"]))
    if case["dir"] == "fwd":
        return [plain_turned(st, cs, q, st["wq"]).to(q.dtype), plain_turned(st, cs, k, st["wk"]).to(k.dtype)]
    if case["op"] == "rope":
        return [rotate(q.float(), cs, case["order"], case["rot"], True).to(q.dtype),
                rotate(k.float(), cs, case["order"], case["rot"], True).to(k.dtype)]
    dq, dwq = plain_norm_bwd(st, cs, q, st["wq"], st["gq"])
    dk, dwk = plain_norm_bwd(st, cs, k, st["wk"], st["gk"])
    return [dq, dk, dwq, dwk]


def owners(st):
    """Sequence and own index of each new token, in the order of the rows."""
    n = st["cu"][1:] - st["cu"][:-1]
    rows = sum(st["new"])
    b = torch.repeat_interleave(torch.arange(len(st["new"]), device="cuda"), n.long(), output_size=rows)
    first = (st["kv_len"] - n - st["cu"][:-1]).long()
    return b, torch.arange(rows, device="cuda") + first[b]


def plain_append(st):
    case = st["case"]
    b, i = owners(st)
    rows, ps = len(i), case["page"]
    cs = angles(i + case["base"], case["rot"], "none")
    at = st["table"].long()[b, i // ps] * ps + i % ps
    st["k_cache"].view(-1, case["Nkv"], case["D"])[at] = plain_turned(st, cs, st["k"][:rows], st["wk"]).to(torch.bfloat16)
    st["v_cache"].view(-1, case["Nkv"], case["D"])[at] = st["v"][:rows].to(torch.bfloat16)
    if st["q"] is None:
        return [st["k_cache"], st["v_cache"]]
    st["q_out"][:rows] = plain_turned(st, cs, st["q"][:rows], st["wq"]).to(torch.bfloat16)
    return [st["k_cache"], st["v_cache"], st["q_out"]]


def partial(q, k, v, late=None):
    """q [B, n, Nkv, G, D] against k, v [B, L, Nkv, D]: row maxima, sums and values of exp(scores - maximum), each
    [B, n, Nkv, G(, D)]; `late` [B, n, L] marks the keys that a row does not see."""
    s = torch.einsum("bnhgd,blhd->bnhgl", q, k) / math.sqrt(q.shape[-1])
    if late is not None:
        s = s.masked_fill(late[:, :, None, None], -math.inf)
    m = s.amax(-1)
    p = torch.exp(s - m[..., None])
    return m, p.sum(-1), torch.einsum("bnhgl,blhd->bnhgd", p, v)


def plain_attn(st):
    case = st["case"]
    N, Nkv, D, ps, P = case["N"], case["Nkv"], case["D"], case["page"], case["prefix"]
    b, i = owners(st)
    rows, most, longest = len(i), max(st["new"]), max(st["length"])
    q = st["q"][:rows].float().view(rows, Nkv, N // Nkv, D)
    # each sequence's own keys, in a batch padded to the longest
    row = torch.arange(rows, device="cuda") - st["cu"].long()[b]
    padded = torch.zeros(case["B"], most, *q.shape[1:], device="cuda")
    padded[b, row] = q
    last = torch.zeros(case["B"], most, dtype=torch.long, device="cuda")
    last[b, row] = i
    pages = st["table"][:, :-(-longest // ps)].long()
    k, v = (c[pages].flatten(1, 2)[:, :longest].float() for c in (st["k_cache"], st["v_cache"]))
    late = torch.arange(longest, device="cuda") > last[..., None]
    m, total, acc = (t[b, row] for t in partial(padded, k, v, late))
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


def run(state):
    case = state["case"]
    if own:
        return run_own(state)
    return {"rope": plain_rows, "norm": plain_rows, "append": plain_append, "attn": plain_attn}[case["op"]](state)


# ------------------------------------------------------------------ the library's entry points
def run_own(st):
    F, case = ops(), st["case"]
    if case["op"] == "rope":
        f = F.cp_rope_fwd if case["dir"] == "fwd" else F.cp_rope_bwd
        return list(f(st["q"], st["k"], st["pos"], st["rope"], st["oq"], st["ok"]))
    if case["op"] == "norm" and case["dir"] == "fwd":
        return list(F.cp_qk_norm_rope_fwd(st["q"], st["k"], st["wq"], st["wk"], st["pos"], st["rope"], eps=EPS,
                                          q_out=st["oq"], k_out=st["ok"]))
    if case["op"] == "norm":
        return list(F.cp_qk_norm_rope_bwd(st["gq"], st["gk"], st["q"], st["k"], st["wq"], st["wk"], st["pos"],
                                          st["rope"], eps=EPS, dq=st["oq"], dk=st["ok"], dwq=st["dwq"], dwk=st["dwk"],
                                          workspace=st["ws"]))
    if case["op"] == "append":
        F.cp_cache_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["cu"], st["kv_len"],
                          rope=st["rope"], q=st["q"], q_out=st["q_out"], wq=st["wq"], wk=st["wk"], eps=EPS,
                          pos_base=case["base"])
        return [st["k_cache"], st["v_cache"]] + ([] if st["q"] is None else [st["q_out"]])
    return list(F.cp_prefix_attn_fwd(st["q"], st["k_cache"], st["v_cache"], st["prefix_pages"], case["prefix"],
                                     st["table"], st["cu"], st["kv_len"], max(st["new"]), o=st["o"], lse=st["lse"],
                                     workspace=st["ws"]))


# ------------------------------------------------------------------ 64 bits
def unit(pos, rot, scaling):
    """amplitude * e^(i angle) of every (position, pair), as complex numbers of 64-bit parts."""
    f, length = SCALING[scaling]
    out, amp = [], 1.0
    for i in range(rot // 2):
        base = BASE * f ** (rot / (rot - 2)) if scaling == "base" else BASE
        w = math.exp(-2.0 * i / rot * math.log(base))
        if scaling == "linear":
            w /= f
        if scaling == "by_parts":
            amp = 1.0 + math.log(f) / 10
            r = length * w / math.tau
            w *= 1.0 if r >= 32 else 1.0 / f if r <= 1 else 1.0 / f + (1.0 - 1.0 / f) * (r - 1) / 31
        out.append(w)
    a = torch.outer(pos.flatten().double(), torch.tensor(out, dtype=torch.float64, device="cuda"))
    return torch.polar(torch.full_like(a, amp), a).view(*pos.shape, rot // 2)


def turned(x, z, order, rot):
    """x [..., heads, D] in 64 bits with its rotated pairs as complex numbers times z [..., rot/2]."""
    r = x[..., :rot]
    pairs = r.unflatten(-1, (2, rot // 2)).movedim(-2, -1) if order == "half" else r.unflatten(-1, (rot // 2, 2))
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z[..., None, :])
    y = y.movedim(-1, -2) if order == "half" else y
    return torch.cat([y.flatten(-2), x[..., rot:]], -1)


def exact_rows(st):
    case = st["case"]
    z = unit(st["pos"], case["rot"], case["scaling"])[:, None]
    out, dws = [], []
    for x, w, g in ((st["q"], st["wq"], st.get("gq")), (st["k"], st["wk"], st.get("gk"))):
        parts, dw = [], 0
        for c in range(case["C"]):
            y = x[c:c + 1].double()
            zc = z[c:c + 1]
            if case["op"] == "rope":
                parts.append(turned(y, zc if case["dir"] == "fwd" else zc.conj(), case["order"], case["rot"]))
                continue
            n = torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["D"] + EPS)
            if case["dir"] == "fwd":
                parts.append(turned(y / n * w.double(), zc, case["order"], case["rot"]))
                continue
            t = turned(g[c:c + 1].double(), zc.conj(), case["order"], case["rot"])
            dw = dw + (t * (y / n)).sum((0, 1, 2, 3))
            t = t * w.double()
            parts.append(t / n - y * ((t * y).sum(-1, keepdim=True) / (case["D"] * n ** 3)))
        out.append(torch.cat(parts))
        if torch.is_tensor(dw):
            dws.append(dw)
    return out + dws


def exact_append(st):
    case = st["case"]
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    qo = st["q_out"].double() if st["q"] is not None else None
    row = 0
    for b, (n, m) in enumerate(zip(st["new"], st["length"])):
        i = torch.arange(m - n, m, device="cuda")
        z = unit(i + case["base"], case["rot"], "none")
        page = st["table"][b].long()[torch.div(i, case["page"], rounding_mode="floor")]
        for x, w, dst in ((st["k"], st["wk"], "k"), (st["v"], None, "v"), (st["q"], st["wq"], "q")):
            if x is None:
                continue
            y = x[row:row + n].double()
            if w is not None:
                y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["D"] + EPS) * w.double()
            if dst != "v":
                y = turned(y, z, case["order"], case["rot"])
            if dst == "q":
                qo[row:row + n] = y
            else:
                (kc if dst == "k" else vc)[page, i % case["page"]] = y
        row += n
    return [kc, vc] + ([] if qo is None else [qo])


def exact_attn(st):
    case = st["case"]
    N, Nkv, ps, P = case["N"], case["Nkv"], case["page"], case["prefix"]
    o, lse = st["o"].double(), st["lse"].double()
    kc, vc = (c.flatten(0, 1) for c in (st["k_cache"], st["v_cache"]))

    def at(pages, count):
        i = torch.arange(count, device="cuda")
        return pages.long()[i // ps] * ps + i % ps

    shared = at(st["prefix_pages"], P)
    row = 0
    for b, (n, m) in enumerate(zip(st["new"], st["length"])):
        where = torch.cat([shared, at(st["table"][b], m)])
        seen = torch.arange(P + m, device="cuda") <= torch.arange(P + m - n, P + m, device="cuda")[:, None]
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
    w = work(case)
    if case["op"] == "attn" and w["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    return {"rope": exact_rows, "norm": exact_rows, "append": exact_append, "attn": exact_attn}[case["op"]](st)
