"""Pages and slots of a step, storing by slots and positions, the kept branch of a drafted tree, and the trees'
ancestors, against the plain forms of tree_ref.py and rows_ref.py.  Whole numbers and moved rows are equal; normed and
rotated rows have the tolerance of test_gpu_rope.py (bf16 outputs)."""
import numpy as np
import pytest
import torch

import rows_ref as R
import tree_ref as T
from context_causal_attention_gb300 import ops as F
from test_gpu_rope import f64, rand, rope_of, within

pytestmark = pytest.mark.gpu


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Step:
    """A step's lists on the host: lengths, table, stack of free pages."""

    def __init__(self, seed, had, keep, new, page, width, spare, base=0, pad=0):
        g = np.random.default_rng(seed)
        counts = [-(-h // page) for h in had]
        self.n_pages = sum(counts) + spare
        order = g.permutation(self.n_pages).tolist()
        self.table = [[-9] * width for _ in had]
        at = 0
        for b, c in enumerate(counts):
            self.table[b][:c] = order[at:at + c]
            at += c
        self.stack, self.n_free = order[at:] + [-3] * at, spare
        self.had, self.keep, self.new, self.page, self.base = had, keep, new, page, base
        self.R = max(1, sum(new) + pad)

    def call(self, dev, in_place=None, stream=None):
        """The call's results and the table and stack behind it, as lists."""
        self.lists = [i32(x, dev) for x in (self.had, self.keep, self.new, self.table, self.stack)]
        had, keep, new, table, stack = self.lists
        n_free = i32([self.n_free, 77], dev)
        kw = {}
        if in_place:
            kw = dict(kv_len={"had": had, "keep": keep}[in_place], n_free_out=n_free)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        kv_len, cu, slots, pos, n_out = F.cp_cache_plan(had, keep, new, table, stack, n_free, self.page, self.R,
                                                        pos_base=self.base, stream=stream, **kw)
        if stream is not None:
            stream.synchronize()
        if in_place:
            assert kv_len is kw["kv_len"] and n_out is n_free
        return dict(kv_len=kv_len.tolist(), cu=cu.tolist(), slots=slots.tolist(), pos=pos.tolist(), n_free=n_out.tolist(),
                    table=table.tolist(), stack=stack.tolist())

    def want(self):
        table, stack = [list(r) for r in self.table], list(self.stack)
        r = T.plan(self.had, self.keep, self.new, table, stack, self.n_free, self.page, self.R, self.base)
        return dict(r, table=table, stack=stack)


def same(got, want):
    for k in want:
        if k == "stack":  # behind the top it is unspecified
            n = want["n_free"][0]
            assert got[k][:n] == want[k][:n], k
        else:
            assert got[k] == want[k], k


def random_step(seed, B, most_new, most_old, back, page, base=0, pad=0, spare=None, ended=0):
    g = np.random.default_rng(seed + 1000)
    had = [int(g.integers(0, most_old + 1)) for _ in range(B)]
    keep = [max(0, h - int(g.integers(0, back + 1))) for h in had]
    new = [int(g.integers(0, most_new + 1)) for _ in range(B)]
    for b in range(B):
        if ended and b % ended == 0:
            keep[b] = new[b] = 0
    need = [-(-(k + n) // page) for k, n in zip(keep, new)]
    if spare is None:
        spare = sum(max(0, n + h // -page) for n, h in zip(need, had)) + 3
    return Step(seed, had, keep, new, page, max(1, max(need), max(-(-h // page) for h in had)) + 1, spare, base, pad)


STEPS = {
    "one_token": lambda: Step(1, [0], [0], [1], 16, 1, 1),
    "nothing": lambda: Step(2, [5, 0], [5, 0], [0, 0], 16, 2, 0, pad=4),
    "page_edges": lambda: Step(3, [15, 16, 17, 32, 0], [15, 16, 17, 32, 0], [1, 1, 1, 1, 16], 16, 4, 9, 100, 1),
    "all_back": lambda: Step(4, [100, 33, 1], [0, 0, 0], [0, 0, 0], 16, 9, 0),
    "back_and_forth": lambda: Step(5, [100, 33, 1, 64], [3, 33, 1, 64], [1, 90, 1, 0], 16, 9, 0, -5),
    "decode": lambda: random_step(6, 64, 1, 4000, 0, 16, 8192),
    "rejected": lambda: random_step(7, 100, 9, 300, 40, 32, 7, 3, ended=5),
    "large_pages": lambda: random_step(8, 33, 700, 900, 500, 256, pad=100, ended=4),
    "prompts": lambda: random_step(9, 5, 9000, 10, 3, 16, 1 << 20, 17),
    "each_of_1025": lambda: random_step(10, 1025, 3, 90, 5, 16, ended=9),
    "most_sequences": lambda: random_step(11, 4096, 30, 200, 30, 64, 0, 1000, ended=11),
    "only_one_long": lambda: random_step(12, 1, 70000, 3, 0, 16),
}


@pytest.mark.parametrize("name", sorted(STEPS))
@pytest.mark.parametrize("in_place", [None, "had", "keep"])
def test_plan(cuda_dev, name, in_place):
    s = STEPS[name]()
    same(s.call(cuda_dev, in_place), s.want())


@pytest.mark.parametrize("short", [1, 5, 1000])
def test_plan_without_enough_pages(cuda_dev, short):
    """All or nothing: lists, table and stack stay, and how many pages are lacking is told."""
    s = random_step(20, 90, 70, 200, 10, 16, 3, 5, ended=7)
    free = T.plan(s.had, s.keep, s.new, [list(r) for r in s.table], list(s.stack), s.n_free, 16, s.R)["n_free"][0]
    needed = s.n_free - free  # pages that the step takes from the stack over what it gives
    s.n_free = max(0, needed - short)
    if needed - short < 0:
        s.n_free, s.new[0] = 0, 100000 % (16 * len(s.table[0]) - s.keep[0])
        s.R = sum(s.new) + 5  # (rows for all of them: too few would be reported instead)
    want = s.want()
    assert want["n_free"][1] > 0
    got = s.call(cuda_dev)
    same(got, want)
    assert got["stack"] == s.stack and got["n_free"][1] > 0 and set(got["slots"]) == {-1}
    assert F.cp_device_status() == 0


@pytest.mark.parametrize("what", ["negative_new", "negative_keep", "keep_over_had", "long", "rows", "n_free", "stack_over",
                                  "page"])
def test_plan_reports_lists_out_of_range(cuda_dev, what):
    s = Step(21, [20, 40, 5], [18, 40, 0], [3, 20, 0], 16, 4, 6, 0, 2)
    if what == "negative_new":
        s.new[1] = -1
    elif what == "negative_keep":
        s.keep[0] = -4
    elif what == "keep_over_had":
        s.keep[0] = 21
    elif what == "long":
        s.new[1] = 25
    elif what == "rows":
        s.R = 22
    elif what == "n_free":
        s.n_free = -1
    elif what == "stack_over":
        s.n_free = s.n_pages
    elif what == "page":
        s.stack[s.n_free - 1] = s.n_pages
        s.had[2] = s.keep[2] = 5
    got = s.call(cuda_dev)
    assert F.cp_device_status() == 11
    assert F.cp_device_status() == 0
    if what == "page":
        # the bad page's rows have no slot, the others theirs: sequence 1's tokens from own index 48 on
        bad = [r for r, x in enumerate(got["slots"]) if x < 0]
        assert got["n_free"] == [5, 0] and bad == list(range(11, 25)), (got["n_free"], bad)
        return
    assert got["n_free"] == [s.n_free, -1] and got["cu"] == [0] * 4 and got["kv_len"] == s.had
    assert set(got["slots"]) == {-1} and got["table"] == s.table and got["stack"] == s.stack


@pytest.mark.parametrize("bad", [-1, 999, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("taken", [False, True])
def test_plan_reports_bad_pages_that_are_given_back(cuda_dev, bad, taken):
    """A page number out of range in the table of a sequence that gives it back: the step that puts it on the stack
    says so, whether or not the same step hands it on."""
    s = Step(22, [40, 33, 5], [10, 33, 5], [0, 40 if taken else 1, 0], 16, 6, 0, 0, 2)
    s.table[0][2] = bad  # pages 1 and 2 of sequence 0 go back
    got = s.call(cuda_dev)
    assert F.cp_device_status() == 11
    assert F.cp_device_status() == 0
    assert got["kv_len"] == [10, 73 if taken else 34, 5]
    if not taken:
        assert got["slots"][0] == s.table[1][2] * 16 + 1 and got["n_free"] == [2, 0]
    else:
        # the page was pushed last and popped first: own indexes 48 to 63 of sequence 1 have no slot
        assert got["n_free"] == [0, 0] and [r for r, x in enumerate(got["slots"][:40]) if x < 0] == list(range(15, 31))


@pytest.mark.parametrize("base,first", [(2 ** 31 - 60, 0), (2 ** 31 - 59, 1), (2 ** 31 - 1, 1)])
def test_plan_reports_positions_past_32_bits(cuda_dev, base, first):
    """The last new position is base + 59: beyond 32 bits nothing is handed out.  (A longer sequence without new tokens
    has no new position.)"""
    s = Step(23, [20, 40, 64], [18, 40, 64], [3, 20, 0], 16, 4, 6, base, 2)
    got = s.call(cuda_dev)
    assert F.cp_device_status() == (11 if first else 0)
    if not first:
        same(got, s.want())
        assert max(got["pos"]) == 2 ** 31 - 1
        return
    assert F.cp_device_status() == 0
    assert got["n_free"] == [s.n_free, -1] and got["cu"] == [0] * 4 and got["kv_len"] == s.had
    assert set(got["slots"]) == {-1} and got["table"] == s.table and got["stack"] == s.stack


def test_plan_over_many_steps_in_a_graph(cuda_dev):
    """One captured call, replayed with new lengths: its own results are the next step's lists; every page is
    handed out once."""
    g = np.random.default_rng(30)
    B, page, width, n_pages, rows = 40, 16, 30, 700, 2000
    s = Step(30, [0] * B, [0] * B, [0] * B, page, width, n_pages, 50)
    table, stack = i32(s.table, cuda_dev), i32(s.stack, cuda_dev)
    had, keep, new = (i32([0] * B, cuda_dev) for _ in range(3))
    n_free, cu = i32([n_pages, 0], cuda_dev), i32([0] * (B + 1), cuda_dev)
    slots, pos = i32([0] * rows, cuda_dev), i32([0] * rows, cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.cp_cache_plan(had, keep, new, table, stack, n_free, page, rows, 50, kv_len=had, cu_new=cu, slots=slots, pos=pos,
                        n_free_out=n_free)
    h, t, st, nf = [0] * B, [list(r) for r in s.table], list(s.stack), n_pages
    refused = 0
    for step in range(60):
        k = [int(g.integers(0, x + 1)) if g.random() < 0.2 else x for x in h]
        n = [int(g.integers(0, min(50, width * page - x) + 1)) for x in k]
        keep.copy_(torch.tensor(k, dtype=torch.int32))
        new.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        r = T.plan(h, k, n, t, st, nf, page, rows, 50)
        h, nf = r["kv_len"], r["n_free"][0]
        refused += r["n_free"][1] > 0
        assert had.tolist() == h and n_free.tolist() == r["n_free"] and cu.tolist() == r["cu"], step
        assert slots.tolist() == r["slots"] and pos.tolist() == r["pos"]
        got = table.tolist()
        for b in range(B):
            c = -(-h[b] // page)
            assert got[b][:c] == t[b][:c]
        assert stack.tolist()[:nf] == st[:nf]
    assert 0 < refused < 60


def test_plan_on_another_stream_and_outputs_in_bounds(cuda_dev):
    s = random_step(40, 70, 90, 300, 30, 32, 11, 6, ended=4)
    want = s.want()
    same(s.call(cuda_dev, stream=torch.cuda.Stream()), want)
    sizes = (70, 71, s.R, s.R, 2)
    bufs = [torch.full((n + 8,), 55, dtype=torch.int32, device=cuda_dev) for n in sizes]
    had, keep, new = (i32(x, cuda_dev) for x in (s.had, s.keep, s.new))
    width = len(s.table[0])
    table = torch.full((70 * width + 8,), 55, dtype=torch.int32, device=cuda_dev)
    table[4:-4] = i32(s.table, cuda_dev).flatten()
    stack = torch.full((s.n_pages + 8,), 55, dtype=torch.int32, device=cuda_dev)
    stack[4:-4] = i32(s.stack, cuda_dev)
    outs = dict(zip(("kv_len", "cu_new", "slots", "pos", "n_free_out"), (x[4:-4] for x in bufs)))
    F.cp_cache_plan(had, keep, new, table[4:-4].view(70, width), stack[4:-4], i32([s.n_free], cuda_dev), 32, s.R, 11, **outs)
    for x in bufs + [table, stack]:
        assert (x[:4] == 55).all() and (x[-4:] == 55).all()
    assert outs["slots"].tolist() == want["slots"] and outs["cu_new"].tolist() == want["cu"]
    assert [had.tolist(), keep.tolist(), new.tolist()] == [s.had, s.keep, s.new]


# ------------------------------------------------------------------ ancestors
@pytest.mark.parametrize("words", [1, 2, 5, 16])
@pytest.mark.parametrize("kind", ["chain", "star", "heap", "roots", "random"])
def test_tree_plan(cuda_dev, words, kind):
    """Trees of every size up to the mask's, empty sequences, a prompt, padding."""
    g = np.random.default_rng(words)
    new = [1, 0, 32 * words, 2, 32 * words - 1, 31, 0, 32 * words + 1, min(33, 32 * words), 3 * 32 * words]
    before = [int(g.integers(0, 90)) for _ in new]
    rows, pad, base = sum(new), 5, 1000
    parent = []
    for n in new:
        parent += T.random_parents(g, n, kind) if n <= 32 * words else [12345] * n
    cu = np.concatenate([[0], np.cumsum(new)])
    mask = torch.full((rows + pad, words), 7, dtype=torch.int32, device=cuda_dev)
    pos = torch.full((rows + pad,), 7, dtype=torch.int32, device=cuda_dev)
    F.cp_tree_plan(i32(parent + [99] * pad, cuda_dev), i32(cu.tolist(), cuda_dev),
                   i32([a + b for a, b in zip(before, new)], cuda_dev), words, base, mask, pos)
    assert F.cp_device_status() == 0
    mask, pos = mask.cpu().numpy(), pos.cpu().numpy()
    for b, n in enumerate(new):
        at = slice(cu[b], cu[b] + n)
        if n > 32 * words:
            assert (mask[at] == 7).all() and (pos[at] == base + before[b] + np.arange(n)).all()
            continue
        seen, depth = T.branches(parent[cu[b]:cu[b] + n])
        assert np.array_equal(mask[at], T.packed(seen, words)), (b, n)
        assert np.array_equal(pos[at], base + before[b] + depth)
    assert (mask[rows:] == 7).all() and (pos[rows:] == 7).all()


def test_tree_plan_of_the_most_sequences(cuda_dev):
    g = np.random.default_rng(3)
    new = [int(g.integers(0, 9)) for _ in range(4096)]
    parent = sum((T.random_parents(g, n, "random") for n in new), [])
    cu = np.concatenate([[0], np.cumsum(new)])
    mask, pos = F.cp_tree_plan(i32(parent, cuda_dev), i32(cu.tolist(), cuda_dev), i32([n + 3 for n in new], cuda_dev), 1)
    want = [T.branches(parent[cu[b]:cu[b + 1]]) for b in range(4096)]
    assert np.array_equal(mask.cpu().numpy(), np.concatenate([T.packed(s, 1) for s, _ in want]))
    assert np.array_equal(pos.cpu().numpy(), 3 + np.concatenate([d for _, d in want]))


@pytest.mark.parametrize("what", ["late", "self", "low", "counts", "past"])
def test_tree_plan_reports_lists_out_of_range(cuda_dev, what):
    parent, cu = [-1, 0, 1, -1, 0, 0], [0, 3, 6]
    if what in ("late", "self", "low"):
        parent[1] = {"late": 2, "self": 1, "low": -2}[what]
    elif what == "counts":
        cu[1] = -1
    else:
        cu[2] = 7
    mask = torch.full((6, 1), 9, dtype=torch.int32, device=cuda_dev)
    pos = torch.full((6,), 9, dtype=torch.int32, device=cuda_dev)
    F.cp_tree_plan(i32(parent, cuda_dev), i32(cu, cuda_dev), i32([13, 23], cuda_dev), 1, mask=mask, pos=pos)
    assert F.cp_device_status() == 11
    assert F.cp_device_status() == 0
    mask, pos = mask.flatten().tolist(), pos.tolist()
    if what in ("late", "self", "low"):  # counts as a token without a parent
        assert mask == [1, 2, 6, 1, 3, 5] and pos == [10, 10, 11, 20, 21, 21]
    elif what == "past":
        assert mask == [1, 3, 7, 9, 9, 9] and pos == [10, 11, 12, 9, 9, 9]
    else:
        assert mask == [9] * 6 and pos == [9] * 6


@pytest.mark.parametrize("what,length", [("short", 2), ("none", 0), ("negative", -7), ("lowest", -2 ** 31)])
@pytest.mark.parametrize("n", [3, 40])
def test_tree_plan_reports_lengths_below_the_new_tokens(cuda_dev, what, length, n):
    """A tree (or a prompt) of more new tokens than its sequence has: its rows stay, as cp_cache_keep keeps nothing of it."""
    parent, cu = [-1, 0, 1] + [-1, 0, 0] * 14, [0, 3, 3 + n, 6 + n]
    rows = 6 + n
    mask = torch.full((rows, 1), 9, dtype=torch.int32, device=cuda_dev)
    pos = torch.full((rows,), 9, dtype=torch.int32, device=cuda_dev)
    parent[3 + n:] = [-1, 0, 1]
    F.cp_tree_plan(i32(parent, cuda_dev), i32(cu, cuda_dev), i32([13, length, 3], cuda_dev), 1, 100, mask=mask, pos=pos)
    assert F.cp_device_status() == 11
    assert F.cp_device_status() == 0
    mask, pos = mask.flatten().tolist(), pos.tolist()
    assert mask == [1, 3, 7] + [9] * n + [1, 3, 7] and pos == [110, 111, 112] + [9] * n + [100, 101, 102]


@pytest.mark.parametrize("n", [6, 40])
@pytest.mark.parametrize("base,bad", [(2 ** 31 - 90, 0), (2 ** 31 - 89, 1)])
def test_tree_plan_reports_positions_past_32_bits(cuda_dev, n, base, bad):
    """A sequence of 90 tokens: its last position is base + 89, beyond 32 bits its rows stay."""
    parent = [j - 1 for j in range(n)]
    mask = torch.full((n, 1), 9, dtype=torch.int32, device=cuda_dev)
    pos = torch.full((n,), 9, dtype=torch.int32, device=cuda_dev)
    F.cp_tree_plan(i32(parent, cuda_dev), i32([0, n], cuda_dev), i32([90], cuda_dev), 1, base, mask=mask, pos=pos)
    assert F.cp_device_status() == (11 if bad else 0)
    assert F.cp_device_status() == 0
    assert pos.tolist() == ([9] * n if bad else list(range(2 ** 31 - n, 2 ** 31)))


# ------------------------------------------------------------------ storing by slots
@pytest.mark.parametrize("name,rows,N,Nkv,D,page", [("one", 1, 4, 1, 64, 16), ("odd", 37, 15, 3, 128, 64),
                                                    ("no_q", 200, 0, 2, 128, 256), ("units", 5000, 2, 1, 64, 16),
                                                    ("many", 170000, 1, 1, 64, 32)])
@pytest.mark.parametrize("dt,order,norm", [("bf16", "half", True), ("fp32", "interleaved", False), ("fp32", "half", True),
                                           ("bf16", "interleaved", False)])
def test_append_at(cuda_dev, name, rows, N, Nkv, D, page, dt, order, norm):
    """Rows at random slots and positions, some without a slot: every slot and query that got a row, and all
    others as they were."""
    g = torch.Generator().manual_seed(rows)
    pages = rows // page + 3
    slots = torch.randperm(pages * page, generator=g)[:rows].to(torch.int32)
    slots[3::7] = -1
    pos = torch.randint(-9, 1 << 20, (rows,), generator=g, dtype=torch.int32)
    rope, th, amp = rope_of(D // 2, order, "by_parts")
    x = rand(g, (rows, N + 2 * Nkv, D), dt, 2.0)
    wq, wk = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)]
    d = x.to(cuda_dev)
    kc, vc = (torch.full((pages, page, Nkv, D), 9.0, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
    qo = torch.full((rows, N, D), 7.0, dtype=torch.bfloat16, device=cuda_dev) if N else None
    w = dict(wq=wq.to(cuda_dev) if N else None, wk=wk.to(cuda_dev)) if norm else {}
    got = F.cp_cache_append_at(d[:, N:N + Nkv], d[:, N + Nkv:], kc, vc, slots.to(cuda_dev), pos.to(cuda_dev), rope=rope,
                               q=d[:, :N] if N else None, q_out=qo, eps=1e-5, **w)
    assert got is qo and F.cp_device_status() == 0
    to = slots >= 0
    at = slots[to].long().numpy()
    rest = np.ones(pages * page, bool)
    rest[at] = False
    keys, values = (c.view(-1, Nkv, D).cpu() for c in (kc, vc))
    assert (keys[rest] == 9).all() and (values[rest] == 9).all()
    assert torch.equal(values[at], x[to][:, N + Nkv:].to(torch.bfloat16))

    def check(got, cut, w, what):
        y = f64(x[to][:, cut])
        y = R.norm(y, f64(w), 1e-5) if norm else y
        within(got, R.turn(y, pos[to].numpy(), th, amp, order), "bf16", 24 * R.U32 * amp * R.pair_size(y, th, order), what)

    check(keys[at], slice(N, N + Nkv), wk, "keys")
    if N:
        check(qo.cpu()[to], slice(0, N), wq, "queries")
        assert (qo.cpu()[~to] == 7).all()


def test_append_at_agrees_with_append(cuda_dev):
    """The plan's slots and positions: the bits of cp_cache_append by the plan's other lists."""
    g = torch.Generator().manual_seed(5)
    s = random_step(50, 30, 40, 200, 20, 32, 4000, 9, ended=6)
    want = s.want()
    r = s.call(cuda_dev)
    table, n = s.lists[3], sum(s.new)
    q, k, v = (rand(g, (s.R, h, 64), "bf16").to(cuda_dev) for h in (4, 2, 2))
    rope, _, _ = rope_of(64, "half")
    a, b = ([torch.zeros(s.n_pages, 32, 2, 64, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2)] for _ in range(2))
    qa = F.cp_cache_append(k, v, *a, table, i32(r["cu"], cuda_dev), i32(r["kv_len"], cuda_dev), rope=rope, q=q, pos_base=4000)
    qb = F.cp_cache_append_at(k, v, *b, i32(r["slots"], cuda_dev), i32(r["pos"], cuda_dev), rope=rope, q=q)
    assert torch.equal(qa[:n], qb[:n]) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert int((a[1].view(-1, 128) != 0).any(1).sum()) == n and r["slots"] == want["slots"]


@pytest.mark.parametrize("bad", [-2, 5 * 16, 2 ** 31 - 1, -2 ** 31])
def test_append_at_reports_slots_out_of_range(cuda_dev, bad):
    g = torch.Generator().manual_seed(6)
    k, v = (rand(g, (3, 2, 64), "bf16").to(cuda_dev) for _ in range(2))
    kc, vc = (torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
    F.cp_cache_append_at(k, v, kc, vc, i32([79, bad, 0], cuda_dev), i32([0, 0, 0], cuda_dev))
    assert F.cp_device_status() == 11
    assert F.cp_device_status() == 0
    flat = kc.view(-1, 2, 64)
    assert torch.equal(flat[79], k[0]) and torch.equal(flat[0], k[2]) and not flat[1:79].any()


def test_append_at_past_32_bits_of_offset(cuda_dev):
    pages, page, Nkv, D = 20500, 256, 8, 128
    kc = torch.zeros(pages, page, Nkv, D, dtype=torch.bfloat16, device=cuda_dev)
    vc = torch.zeros_like(kc)
    k, v = (torch.ones(2, Nkv, D, dtype=torch.bfloat16, device=cuda_dev) * x for x in (3, 5))
    F.cp_cache_append_at(k, v, kc, vc, i32([pages * page - 1, 17000 * page], cuda_dev), i32([0, 0], cuda_dev))
    torch.cuda.synchronize()
    assert (kc[-1, -1] == 3).all() and (vc[-1, -1] == 5).all() and (kc[17000, 0] == 3).all() and (vc[17000, 0] == 5).all()
    for c in (kc, vc):
        assert int((c.view(torch.int16).view(-1, Nkv * D)[:, 0] != 0).sum()) == 2
    # and moved on from there
    kc[17000, 0] = 4
    table = i32([[pages - 1, 17000]], cuda_dev)
    F.cp_cache_keep([kc, vc], table, i32([0, 2], cuda_dev), i32([257], cuda_dev), i32([[1]], cuda_dev), i32([1], cuda_dev))
    torch.cuda.synchronize()
    assert (kc[-1, -1] == 4).all() and (kc[17000, 0] == 4).all() and (vc[-1, -1] == 5).all()
    for c in (kc, vc):
        assert int((c.view(torch.int16).view(-1, Nkv * D)[:, 0] != 0).sum()) == 2


# ------------------------------------------------------------------ the kept branch
class Branch:
    """Sequences with new tokens and a kept path each, over pages in random order."""

    def __init__(self, seed, new, before, page, most, layers, Nkv, D, dev):
        g = np.random.default_rng(seed)
        length = [a + b for a, b in zip(new, before)]
        counts = [-(-m // page) for m in length]
        order = g.permutation(sum(counts) + 2).tolist()
        self.new, self.length, self.page, self.dev = new, length, page, dev
        self.table = [[-5] * max(counts + [1]) for _ in new]
        at = 0
        for b, c in enumerate(counts):
            self.table[b][:c] = order[at:at + c]
            at += c
        self.kept = [[-8] * most for _ in new]
        self.n_kept = []
        for b, n in enumerate(new):
            k = int(g.integers(0, min(n, most) + 1)) if b % 5 else min(n, most)
            if b % 7 == 6:
                k = -1
            if k > 0:
                self.kept[b][:k] = sorted(g.choice(n, k, replace=False).tolist())
            self.n_kept.append(k)
        t = torch.Generator().manual_seed(seed)
        self.caches = [torch.randn(sum(counts) + 2, page, Nkv, D, generator=t).to(torch.bfloat16).to(dev)
                       for _ in range(2 * layers)]
        self.before = [c.clone() for c in self.caches]

    def call(self, **kw):
        cu = np.concatenate([[0], np.cumsum(self.new)]).tolist()
        self.lists = [i32(x, self.dev) for x in (self.table, cu, self.length, self.kept, self.n_kept)]
        return F.cp_cache_keep(self.caches, *self.lists, **kw)

    def slot(self, b, i):
        return self.table[b][i // self.page] * self.page + i % self.page

    def check(self, got, kept=None):
        """`kept`: the paths that count (those of the lists else)."""
        source, target, stay = [], [], []
        for b, (n, m, k) in enumerate(zip(self.new, self.length, self.n_kept)):
            path = self.kept[b][:max(0, k)] if kept is None else kept[b]
            source += [self.slot(b, m - n + i) for i in path]
            target += [self.slot(b, m - n + j) for j in range(len(path))]
            stay.append(m if k < 0 else m - n + len(path))
        assert got.tolist() == stay
        for c, old in zip(self.caches, self.before):
            want = old.clone().flatten(0, 1)
            want[target] = old.flatten(0, 1)[source]
            assert torch.equal(c.flatten(0, 1), want)


@pytest.mark.parametrize("name,new,page,most,layers,Nkv,D", [
    ("one", [5], 16, 5, 1, 1, 64), ("pages", [60, 3, 0, 33, 17, 1, 9, 40], 16, 30, 3, 2, 64),
    ("layers", [27] * 20, 64, 6, 32, 8, 128), ("most_caches", [9, 30], 32, 9, 128, 1, 64),
    ("many", [7, 0, 3, 16] * 600, 16, 8, 1, 3, 128), ("long_paths", [512, 700, 512, 300, 5, 512], 128, 512, 2, 1, 128)])
def test_keep(cuda_dev, name, new, page, most, layers, Nkv, D):
    """Paths of every length, also over their own sources, against a copy made before; all other slots as they were."""
    g = np.random.default_rng(len(name))
    b = Branch(len(name), new, [int(g.integers(0, 50)) for _ in new], page, most, layers, Nkv, D, cuda_dev)
    got = b.call(R=sum(new)) if len(name) % 2 else b.call()
    assert F.cp_device_status() == 0
    b.check(got)


def test_keep_shifts_a_whole_tree(cuda_dev):
    """Every path entry is the next one's target: a shift by one through 300 tokens over pages of 16."""
    b = Branch(60, [301, 301], [7, 16], 16, 300, 2, 2, 64, cuda_dev)
    b.kept, b.n_kept = [list(range(1, 301))] * 2, [300, 300]
    b.check(b.call())


@pytest.mark.parametrize("what", ["falls", "equal", "late", "low", "count", "over_most", "page", "counts", "short"])
def test_keep_reports_lists_out_of_range(cuda_dev, what):
    b = Branch(61, [9, 9, 9], [20, 30, 7], 16, 5, 2, 2, 64, cuda_dev)
    b.kept, b.n_kept = [[0, 2, 4, 6, 8], [1, 3, 5, 7, -8], [0, 1, 2, 3, 8]], [5, 4, 5]
    want = [list(x) for x in b.kept]
    want[1] = [1, 3, 5, 7]
    if what in ("falls", "equal", "late", "low"):
        b.kept[1][2] = {"falls": 0, "equal": 3, "late": 9, "low": -3}[what]
        want[1] = [1, 3]
    elif what == "count":
        b.n_kept[1], want[1] = 10, []
    elif what == "over_most":
        b.n_kept[1], want[1] = 6, []
    elif what == "page":
        b.table[1][2] = 999  # own indexes 32 and on: new token 2 and on.  The first entry comes from index 31
        want[1] = [1]
    elif what == "short":
        b.length[1] = 8
    if what == "counts":
        cu = [0, 9, 8, 27]
        lists = [i32(x, cuda_dev) for x in (b.table, cu, b.length, b.kept, b.n_kept)]
        got = F.cp_cache_keep(b.caches, *lists, R=27).tolist()
        assert F.cp_device_status() == 11 and got[0] == 25 and got[1] == 39
        return
    got = b.call()
    assert F.cp_device_status() == 11
    assert F.cp_device_status() == 0
    if what == "short":
        want[1] = []
        assert got.tolist()[1] == 8
        got[1] = -1
        b.new[1], b.length[1] = 9, 8
    b.check(got, want)


def test_keep_in_a_graph_and_on_another_stream(cuda_dev):
    b = Branch(62, [12] * 9, [40] * 9, 16, 5, 3, 2, 64, cuda_dev)
    handle = F.CpCaches(b.caches)
    cu = np.concatenate([[0], np.cumsum(b.new)]).tolist()
    lists = [i32(x, cuda_dev) for x in (b.table, cu, b.length, b.kept, b.n_kept)]
    out = i32([0] * 9, cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.cp_cache_keep(handle, *lists, kv_keep=out)
    graph.replay()
    b.check(out)
    for c, o in zip(b.caches, b.before):
        c.copy_(o)
    b.kept, b.n_kept = [[1, 4, 5, 7, 11]] * 9, [0, 1, 2, 3, 4, 5, 5, -1, 5]
    lists[3].copy_(i32(b.kept, cuda_dev))
    lists[4].copy_(i32(b.n_kept, cuda_dev))
    graph.replay()
    b.check(out)
    for c, o in zip(b.caches, b.before):
        c.copy_(o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = F.cp_cache_keep(handle, *lists, stream=s)
    s.synchronize()
    b.check(got)


def test_keep_follows_pages_that_move_between_calls(cuda_dev):
    """Plans and keeps in turns in one graph: every plan hands other pages to the sequences, and the keep that starts
    under it reads that plan's table, lengths and counts."""
    B, page, width, n_pages, steps, most, Nkv, D = 9, 16, 8, 60, 12, 6, 2, 64
    g = np.random.default_rng(63)
    s = Step(63, [0] * B, [0] * B, [0] * B, page, width, n_pages, 0)
    new = [[int(g.integers(1, 60)) for _ in range(B)] for _ in range(steps)]
    n_kept = [[min(n, int(g.integers(0, most + 1))) for n in row] for row in new]
    kept = [[sorted(g.choice(n, k, replace=False).tolist()) + [-1] * (most - k) for n, k in zip(a, b)]
            for a, b in zip(new, n_kept)]
    for row in n_kept:  # and a step that ends in an empty sequence for some
        row[3] = 0
    t = torch.Generator().manual_seed(63)
    caches = [torch.randn(n_pages, page, Nkv, D, generator=t).to(torch.bfloat16).to(cuda_dev) for _ in range(4)]
    before = [c.clone() for c in caches]
    first = [c.flatten(0, 1).clone() for c in caches]
    table, stack = i32(s.table, cuda_dev), i32(s.stack, cuda_dev)
    had, keep, n_free = i32([0] * B, cuda_dev), i32([0] * B, cuda_dev), i32([n_pages, 0], cuda_dev)
    lists = [[i32(x[i], cuda_dev) for x in (new, kept, n_kept)] for i in range(steps)]
    cu, R = i32([0] * (B + 1), cuda_dev), 60 * B
    rows = [i32([0] * R, cuda_dev) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for n, k, c in lists:
            F.cp_cache_plan(had, keep, n, table, stack, n_free, page, R, 0, kv_len=had, cu_new=cu, slots=rows[0],
                            pos=rows[1], n_free_out=n_free)
            F.cp_cache_keep(caches, table, cu, had, k, c, kv_keep=keep)
    graph.replay()
    h, m, nf, tb, st = [0] * B, [0] * B, n_pages, [list(r) for r in s.table], list(s.stack)
    moved = 0
    for i in range(steps):
        old = [list(r) for r in tb]
        r = T.plan(h, m, new[i], tb, st, nf, page, R, 0)
        assert r["n_free"][1] == 0
        h, nf = r["kv_len"], r["n_free"][0]
        moved += tb != old
        at = lambda b, j: tb[b][j // page] * page + j % page  # noqa: E731
        pairs = [(at(b, h[b] - new[i][b] + x), at(b, h[b] - new[i][b] + j))
                 for b in range(B) for j, x in enumerate(kept[i][b][:n_kept[i][b]])]
        source, target = [x for x, _ in pairs], [y for _, y in pairs]
        for c in first:
            c[target] = c[source]
        m = [h[b] - new[i][b] + n_kept[i][b] for b in range(B)]
    assert moved > steps // 2 and keep.tolist() == m and n_free.tolist() == [nf, 0]
    for c, w, o in zip(caches, first, before):
        assert torch.equal(c.flatten(0, 1), w) and not torch.equal(c, o)
