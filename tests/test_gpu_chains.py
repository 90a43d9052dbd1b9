"""Attention launched right behind this library's kernels that write its inputs: the list of a
selection, appended cells, the tables, offsets and limits of a page map.  Every call of a run with
nothing between is bitwise what it is with a synchronisation after each call."""
import numpy as np
import pytest

import qsa_workloads as wl
from kv4_cases import Attend

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def qsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_selection_int8_gb300 import build
    build.build()
    import sparse_selection_int8_gb300 as q
    return q


def run_twice(step, n, repeats=20):
    """step(i, wait): a chain over input set i of n, wait() after each call but the last, an attention, whose output it returns."""
    want = []
    for i in range(n):
        want.append(step(i, torch.cuda.synchronize))
        torch.cuda.synchronize()
    assert all(torch.isfinite(w).all() and w.any() for w in want) and not torch.equal(want[0], want[1])
    got = [(i, step(i, lambda: None)) for _ in range(repeats) for i in range(n)]
    torch.cuda.synchronize()
    for i, o in got:
        assert torch.equal(o, want[i])


@pytest.mark.parametrize("cells", ["int8", "kv4"])
@pytest.mark.parametrize("n_seq,G", [(1, 1), (3, 2)])
def test_attention_behind_the_selection(qsa, cells, n_seq, G):
    draw = dict(n_seq=n_seq, n_queries=2, idx_heads=4, idx_dim=64, block_cells=16, max_blocks=256, top_k=20)
    sets = [qsa.DeviceSelection(wl.make_selection(seed=9800 + i, **draw)) for i in range(2)]
    sets[1].sel, sets[1].sel_offsets = sets[0].sel, sets[0].sel_offsets  # the same list, rewritten
    most = sets[0].max_selected
    n = 256 * 16
    p = wl.make_problem(n_seq=n_seq, n_kv_heads=G, n_queries=2, pool_cells=n, n_selected=[600] * n_seq, chunk_cells=128, seed=9810)
    d = qsa.DeviceProblem(p, max_selected=most)
    c = Attend(seed=9811, n_seq=n_seq, G=G, T=2, lens=(600,), context=n)
    shape = qsa.make_shape(n_kv_heads=G, q_per_kv=12, n_queries=2, pool_cells=c.pool_cells, page_table_len=c.table_len,
                           chunk_cells=1, softmax_scale=1 / 16)
    q, pool, scale, table = (torch.from_numpy(x).cuda() for x in (c.q, c.kv_pool, c.kv_scale, c.page_table))
    ws = torch.empty(qsa.qsa_kv4_attn_workspace_bytes(shape, n_seq, most), dtype=torch.uint8, device="cuda")

    def step(i, wait):
        s = sets[i]
        s.run()
        wait()
        out = torch.empty((n_seq, 2, G * 12, 256), device="cuda")
        if cells == "int8":
            qsa.qsa_decode_attn_batch(d.shape, n_seq, d.q, d.k_pool, d.v_pool, d.k_scale, d.v_scale, d.page_table, s.sel,
                                      s.sel_offsets, most, out, d.workspace, d.ws_bytes, d.status)
        else:
            qsa.qsa_kv4_attn_batch(shape, n_seq, n_seq, q, pool, scale, table, s.sel, s.sel_offsets, most, None, qsa.QSA_F32,
                                   out, ws, ws.numel(), d.status)
        return out
    run_twice(step, 2)
    assert int(d.status.item()) == 0


@pytest.mark.parametrize("n_seq,G", [(1, 1), (4, 2)])
def test_attention_behind_the_int8_append(qsa, n_seq, G):
    n = 512
    p = wl.make_problem(n_seq=n_seq, n_kv_heads=G, n_queries=2, pool_cells=n, n_selected=[n] * n_seq, chunk_cells=128, seed=9820)
    d = qsa.DeviceProblem(p)
    rng = np.random.default_rng(9821)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(n_seq, 1)
    table = pos.clone()
    rows = [[torch.from_numpy(rng.standard_normal((n_seq, n, G, 256)).astype(np.float32)).cuda() for _ in "kv"] for _ in range(2)]

    def step(i, wait):
        qsa.qsa_kv_append(d.shape, n_seq, n, qsa.QSA_F32, *rows[i], pos, table, d.k_pool, d.v_pool, d.k_scale, d.v_scale, d.status)
        wait()
        out = torch.empty((n_seq, 2, G * 12, 256), device="cuda")
        qsa.qsa_decode_attn_batch(d.shape, n_seq, d.q, d.k_pool, d.v_pool, d.k_scale, d.v_scale, table, d.sel, d.sel_offsets,
                                  n, out, d.workspace, d.ws_bytes, d.status)
        return out
    run_twice(step, 2)
    assert int(d.status.item()) == 0


@pytest.mark.parametrize("n_seq,G", [(1, 1), (4, 2)])
def test_int8_attention_behind_ordinary_kernels(qsa, n_seq, G):
    """Each input in turn written by a framework's kernel, another ordinary kernel between it and the call."""
    sets = [qsa.DeviceProblem(wl.make_problem(n_seq=n_seq, n_kv_heads=G, n_queries=2, pool_cells=2048, n_selected=[900] * n_seq,
                                              chunk_cells=128, seed=9840 + i)) for i in range(2)]
    d = qsa.DeviceProblem(sets[0].p)
    names = ["sel", "sel_offsets", "page_table", "q", "k_scale", "v_scale", "k_pool", "v_pool"]
    other = torch.zeros(1, device="cuda")
    for last in range(len(names)):
        def step(i, wait):
            for n in names[last + 1:] + names[:last + 1]:
                torch.add(getattr(sets[i], n), 0, out=getattr(d, n))
            other.add_(1)
            wait()
            out = torch.empty((n_seq, 2, G * 12, 256), device="cuda")
            qsa.qsa_decode_attn_batch(d.shape, n_seq, d.q, d.k_pool, d.v_pool, d.k_scale, d.v_scale, d.page_table, d.sel,
                                      d.sel_offsets, 900, out, d.workspace, d.ws_bytes, d.status)
            return out
        run_twice(step, 2, 5)


@pytest.mark.parametrize("T", [4, 700])  # the maps by one launch, by two
def test_limited_attention_behind_the_page_map(qsa, T):
    """INT8 pools whose tables, offsets and limits are the page map's: a window of T tokens that comes and goes."""
    B, P, L = 8, 16, 64
    n = L * P
    p = wl.make_problem(n_seq=B, n_kv_heads=1, n_queries=T, q_per_kv=2, pool_cells=n, n_selected=[n] * B, chunk_cells=128, seed=9830)
    d = qsa.DeviceProblem(p)
    shape = qsa.make_shape(n_kv_heads=1, q_per_kv=2, n_queries=T, pool_cells=n, page_table_len=L, chunk_cells=128,
                           softmax_scale=1 / 16, page_cells=P)
    ws = torch.empty(qsa.qsa_workspace_bytes(shape, B, n), dtype=torch.uint8, device="cuda")
    sel = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B)
    every = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((B, L), -1, **i32)
    free = torch.arange(L - 1, -1, -1, **i32).repeat(B, 1)
    count = torch.full((B,), L, **i32)
    out_len, offsets = torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
    positions, slots, limit = (torch.zeros((B, T), **i32) for _ in range(3))
    first = [0, T // 4]  # each set's first position
    length = {x: torch.full((B,), x, **i32) for f in first for x in (f, f + T)}
    held = [0]

    def step(i, wait):
        # emptied, grown to the window's start, then by the window
        for x in (0, first[i], first[i] + T):
            qsa.qsa_page_map(B, B, T, P, L, L, length[held[0]], length[x], table, free, count, out_len, offsets, positions,
                             slots, limit, d.status)
            held[0] = x
            wait()
        out = torch.empty((B, T, 2, 256), device="cuda")
        qsa.qsa_decode_attn_batch_limited(shape, B, d.q, d.k_pool, d.v_pool, d.k_scale, d.v_scale, table, sel, every, n, limit, out, ws,
                                          ws.numel(), d.status)
        return out
    # (the list names every position of the table: the pages that a sequence does not hold are masked)
    run_twice(step, 2)
    assert int(d.status.item()) == 0
