"""Plain forms of the page plan, the drafted trees' ancestors and the kept branch, for the tests."""
import numpy as np


def plan(had, keep, new, table, stack, n_free, page, R, base=0):
    """cp_cache_plan on lists -> dict of its results; `table` (list of rows) and `stack` are changed in place."""
    B = len(had)
    pages = lambda n: -(-n // page)  # noqa: E731
    length = [k + n for k, n in zip(keep, new)]
    give = [max(0, pages(h) - pages(m)) for h, m in zip(had, length)]
    take = [max(0, pages(m) - pages(h)) for h, m in zip(had, length)]
    lacking = sum(take) - n_free - sum(give)
    if lacking > 0:
        return dict(kv_len=list(had), cu=[0] * (B + 1), slots=[-1] * R, pos=[0] * R, n_free=[n_free, lacking])
    top = n_free
    for b in range(B):
        for i in range(pages(length[b]), pages(length[b]) + give[b]):
            stack[top] = table[b][i]
            top += 1
    for b in range(B):
        for i in range(pages(had[b]), pages(had[b]) + take[b]):
            top -= 1
            table[b][i] = stack[top]
    cu, slots, pos = [0], [], []
    for b in range(B):
        for i in range(keep[b], length[b]):
            slots.append(table[b][i // page] * page + i % page)
            pos.append(base + i)
        cu.append(len(slots))
    pad = R - len(slots)
    return dict(kv_len=length, cu=cu, slots=slots + [-1] * pad, pos=pos + [0] * pad, n_free=[top, 0])


def branches(parent):
    """(truth values [n, n]: token i is j's ancestor or j itself, depth [n]) of one sequence's parents."""
    n = len(parent)
    seen, depth = np.zeros((n, n), bool), np.zeros(n, np.int64)
    for j, p in enumerate(parent):
        if p >= 0:
            seen[j], depth[j] = seen[p], depth[p] + 1
        seen[j, j] = True
    return seen, depth


def packed(seen, words):
    """Truth values [n, m] as int32 words [n, words]."""
    bits = np.zeros((len(seen), 32 * words), np.uint64)
    bits[:, :seen.shape[1]] = seen
    w = (bits.reshape(-1, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def random_parents(g, n, kind):
    """Parents of n tokens: a chain, a star, a binary heap, a random tree, or several trees."""
    if kind == "chain":
        return [j - 1 for j in range(n)]
    if kind == "star":
        return ([-1] + [0] * (n - 1))[:n]
    if kind == "heap":
        return [(j - 1) // 2 if j else -1 for j in range(n)]
    if kind == "roots":
        return [-1] * n
    return [int(g.integers(-1, j)) if j else -1 for j in range(n)]
