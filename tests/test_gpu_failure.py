"""Failure detection on the GPU without a GPU fault: a kernel whose bounded
wait runs out (its producer held on a flag that nothing sets) must give up,
record CP_ERR_DEVICE_TIMEOUT in the device status word that the host reads,
and leave the context usable for the next call."""
import numpy as np
import pytest
import torch

import oracle as O
from context_causal_attention_gb300 import ops as F

pytestmark = pytest.mark.gpu

CP_ERR_DEVICE_TIMEOUT = 9


def test_bounded_wait_gives_up_and_reports(cuda_dev):
    assert F.cp_device_status() == 0
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, 128, 1, 64, generator=g).to(torch.bfloat16).to(cuda_dev) for _ in range(3))
    pos = torch.arange(128, dtype=torch.int32, device=cuda_dev)
    o = torch.full((1, 128, 1, 64), 7.0, dtype=torch.float32, device=cuda_dev)
    lse = torch.full((1, 1, 128), 7.0, dtype=torch.float32, device=cuda_dev)
    F.cp_selftest_stalled_producer(q, k, v, pos, o, lse, 20_000_000)  # 20 ms limit
    torch.cuda.synchronize()
    assert F.cp_device_status() == CP_ERR_DEVICE_TIMEOUT      # read and cleared
    assert F.cp_device_status() == 0
    assert torch.all(o == 7.0) and torch.all(lse == 7.0)    # nothing was written
    # the context is intact: the same problem runs normally afterwards
    o2, l2 = F.cp_attn_partial(q, k, v, pos, pos)
    torch.cuda.synchronize()
    f = lambda t: t.float().cpu().numpy().astype(np.float64)
    o_ref, l_ref = O.attn_direct(f(q), f(k), f(v), np.arange(128), np.arange(128))
    assert np.max(np.abs(f(o2) - o_ref)) <= 2e-2
    assert np.max(np.abs(f(l2) - l_ref)) <= 1e-3
    assert F.cp_device_status() == 0


def test_timeout_status_survives_until_read(cuda_dev):
    """Two timed-out launches, then one read: the word is sticky, not a count."""
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(1, 128, 1, 64, generator=g).to(torch.bfloat16).to(cuda_dev) for _ in range(3))
    pos = torch.arange(128, dtype=torch.int32, device=cuda_dev)
    o = torch.empty((1, 128, 1, 64), dtype=torch.float32, device=cuda_dev)
    lse = torch.empty((1, 1, 128), dtype=torch.float32, device=cuda_dev)
    F.cp_selftest_stalled_producer(q, k, v, pos, o, lse, 5_000_000)
    F.cp_selftest_stalled_producer(q, k, v, pos, o, lse, 5_000_000)
    assert F.cp_device_status(clear=False) == CP_ERR_DEVICE_TIMEOUT
    assert F.cp_device_status() == CP_ERR_DEVICE_TIMEOUT
    assert F.cp_device_status() == 0


@pytest.mark.parametrize("kernel", [0, 1, 2], ids=["bf16_forward", "tf32_forward", "backward"])
def test_every_kernel_gives_up_a_stalled_wait(cuda_dev, kernel):
    """Each attention kernel's bounded waits: its producer held on a flag that
    nothing sets gives up after 10 ms, the status word reads
    CP_ERR_DEVICE_TIMEOUT (sticky until read), and the next call on the same
    context computes correctly (the backward's two launches both give up)."""
    assert F.cp_device_status() == 0
    F.cp_selftest_stalled_kernel(kernel, 10_000_000)
    torch.cuda.synchronize()
    assert F.cp_device_status() == CP_ERR_DEVICE_TIMEOUT
    assert F.cp_device_status() == 0
    g = torch.Generator().manual_seed(8)
    q, k, v, do = (torch.randn(1, 256, 2, 64, generator=g) for _ in range(4))
    pos = torch.arange(256, dtype=torch.int32, device=cuda_dev)
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    gp = np.arange(256)
    if kernel == 1:
        o, l = F.cp_attn_partial_f32(q.to(cuda_dev), k.to(cuda_dev), v.to(cuda_dev), pos, pos)
        o_ref, l_ref = O.attn_direct(f(q), f(k), f(v), gp, gp)
        assert np.max(np.abs(f(o) - o_ref)) <= 4e-3 and np.max(np.abs(f(l) - l_ref)) <= 2e-3
    else:
        qb, kb, vb, dob = (t.to(torch.bfloat16) for t in (q, k, v, do))
        o, l = F.cp_attn_partial(qb.to(cuda_dev), kb.to(cuda_dev), vb.to(cuda_dev), pos, pos)
        o_ref, l_ref = O.attn_direct(f(qb), f(kb), f(vb), gp, gp)
        assert np.max(np.abs(f(o) - o_ref)) <= 2e-2 and np.max(np.abs(f(l) - l_ref)) <= 1e-3
        if kernel == 2:
            dq, dk, dv = F.cp_attn_bwd_partial(qb.to(cuda_dev), kb.to(cuda_dev), vb.to(cuda_dev), o, dob.to(cuda_dev),
                                               l, pos, pos)
            ref = O.attn_bwd(f(qb), f(kb), f(vb), o_ref, f(dob), l_ref, gp, gp)
            for got, r in zip((dq, dk, dv), ref):
                assert np.max(np.abs(f(got) - r)) <= 1e-2 * np.max(np.abs(r))
    assert F.cp_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", ["narrow", "wide_tma", "wide_small_pages", "both_tma", "both_small_pages"])
def test_prefix_attention_gives_up_a_stalled_wait(cuda_dev, form, D):
    """Every kernel of the shared-prefix attention, its loads held on a word that nothing sets: it
    gives up after 10 ms, the status word says so, nothing outside the workspace is written,
    and the same call computes correctly afterwards, in the workspace that was left."""
    from test_gpu_prefix import Call
    new, length, prefix, page = {
        "narrow": ([1], [300], 1000, 16), "wide_tma": ([40, 9], [300, 900], 500, 64),
        "wide_small_pages": ([40, 9], [300, 900], 500, 16), "both_tma": ([1] * 20, [90 + 9 * i for i in range(20)], 1000, 64),
        "both_small_pages": ([1] * 20, [90 + 9 * i for i in range(20)], 1000, 32)}[form]
    c = Call(21, new, length, prefix, 8, 2, D, page)
    o, lse = c.run(cuda_dev)
    c.check(o, lse)
    assert F.cp_device_status() == 0
    q, k, v, pages, table, cu, kv_len = c.dev
    need = F.cp_prefix_attn_workspace_size(c.R, len(new), max(new), prefix, 8, 2, D, page, table.shape[1])
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=cuda_dev)
    lists = (q, k, v, pages, prefix, table, cu, kv_len, max(new))
    F.cp_selftest_stalled_prefix_attn(10_000_000, *lists, workspace=ws[256:256 + need])
    assert F.cp_device_status() == CP_ERR_DEVICE_TIMEOUT
    assert F.cp_device_status() == 0
    o2, lse2 = F.cp_prefix_attn_fwd(*lists, workspace=ws[256:256 + need])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()
    assert F.cp_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", ["items", "items_of_many_tiles", "items_ordered", "clusters", "clusters_of_many_tiles",
                                  "clusters_few_tiles", "line_narrow", "line_wide"])
def test_tree_attention_gives_up_a_stalled_wait(cuda_dev, form, D):
    """The tree attention's own kernels (a block an item, a cluster an item: their blocks still meet when all of them
    have given up) and the line's: as above."""
    from test_gpu_tree import TreeCall
    new, length, prefix, hint, wide = {
        "items": ([20, 9], [300, 90], 100, 20, 0),
        "items_of_many_tiles": ([60, 200, 3], [300, 200, 90], 0, 1, 0),
        "items_ordered": ([3 + i % 9 for i in range(100)], [700 + 9 * i for i in range(100)], 0, 11, 0),
        "clusters": ([20, 9], [300, 1900], 100, 20, 0),
        "clusters_of_many_tiles": ([60, 200, 3], [300, 2000, 90], 0, 1, 0),
        "clusters_few_tiles": ([5, 40], [90, 40], 0, 40, 700),
        "line_narrow": ([1, 2], [300, 200], 0, 2, 140000),
        "line_wide": ([40, 9], [300, 900], 500, 40, 140000)}[form]
    c = TreeCall(23, new, length, prefix, 16, 4, D, 16, 2)
    c.table = torch.cat([c.table, torch.full((len(new), wide // 16), -3, dtype=torch.int32)], 1)
    o, lse = c.run(cuda_dev, hint=hint)
    c.check(o, lse)
    assert F.cp_device_status() == 0
    q, k, v, mask, pages, table, cu, kv_len = c.dev
    need = F.cp_tree_attn_workspace_size(c.R, len(new), hint, 2, prefix, 16, 4, D, 16, table.shape[1])
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=cuda_dev)
    lists = (q, k, v, mask, pages, prefix, table, cu, kv_len, hint)
    F.cp_selftest_stalled_tree_attn(10_000_000, *lists, workspace=ws[256:256 + need])
    assert F.cp_device_status() == CP_ERR_DEVICE_TIMEOUT
    assert F.cp_device_status() == 0
    o2, lse2 = F.cp_tree_attn_fwd(*lists, workspace=ws[256:256 + need])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()
    assert F.cp_device_status() == 0


@pytest.mark.parametrize("order", ["wait_first", "list_first"])
def test_a_bad_list_does_not_hide_a_wait_that_ran_out(cuda_dev, order):
    """A stalled call and calls with a page number out of range (the append's and the
    attention's), in either order: the status word is the wait's; without it, the list's."""
    from test_gpu_prefix import Call
    c = Call(22, [1, 1], [40, 70], 100, 4, 2, 64, 16)
    c.run(cuda_dev)
    q, k, v, pages, table, cu, kv_len = c.dev
    bad = table.clone()
    bad[:, :3] = c.b.total

    def lists():
        F.cp_cache_append(k[0, :2], v[0, :2], k.clone(), v.clone(), bad, cu, kv_len)
        F.cp_prefix_attn_fwd(q, k, v, pages, 100, bad, cu, kv_len, 1)

    def stall():
        F.cp_selftest_stalled_prefix_attn(5_000_000, q, k, v, pages, 100, table, cu, kv_len, 1)

    for call in (stall, lists) if order == "wait_first" else (lists, stall):
        call()
    assert F.cp_device_status(clear=False) == CP_ERR_DEVICE_TIMEOUT
    assert F.cp_device_status() == CP_ERR_DEVICE_TIMEOUT
    assert F.cp_device_status() == 0
    lists()
    assert F.cp_device_status() == 11
    assert F.cp_device_status() == 0
