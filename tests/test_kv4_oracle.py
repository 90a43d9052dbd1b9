"""The oracles of the 4-bit cells and the page bookkeeping, on the CPU: hand-worked
values and properties; and the refusals of their entry points (no kernel runs)."""
import ctypes

import numpy as np
import pytest

import sparse_selection_int8_gb300 as qsa
from kv4_cases import Attend, bf16_round
from oracle import kv4, page_map as pm
from sparse_selection_int8_gb300 import build as qsa_build


# ------------------------------------------------------------------ quantiser

def test_quantise_by_hand():
    # 0, 1, ..., 15 repeated: scale 1, zero 0, the codes are the values
    x = np.tile(np.arange(16, dtype=np.float32), 16)
    u, s, z = kv4.quantise(x)
    assert s == 1 and z == 0 and np.array_equal(u, x.astype(np.uint8))
    # shifted and scaled by powers of two: the same codes
    u2, s2, z2 = kv4.quantise(x * np.float32(0.25) - np.float32(2))
    assert s2 == 0.25 and z2 == -2 and np.array_equal(u2, u)
    # halves go to the even code
    x = np.zeros(256, np.float32)
    x[:4] = [15, 0.5, 1.5, 2.5]
    u, s, z = kv4.quantise(x)
    assert s == 1 and u[:4].tolist() == [15, 0, 2, 2]
    # a constant row: scale 0, zero codes, the value itself
    u, s, z = kv4.quantise(np.full(256, -3.25, np.float32))
    assert s == 0 and z == -3.25 and not u.any()


def test_quantise_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, 256)) * np.exp(rng.uniform(-20, 20, (50, 1)))).astype(np.float32)
    u, s, z = kv4.quantise(x)
    y = u * s[:, None].astype(np.float64) + z[:, None]
    # half a step, and the scale's own roundings (15 codes of 1/15's, the difference's and the product's, 2^-24 each)
    assert (np.abs(y - x) <= s[:, None] * (0.5 + 15 * 4 * 2.0 ** -24)).all()
    assert (u.min(1) == 0).all() and (u.max(1) == 15).all()


def test_pack_places_dimensions():
    u = np.zeros(256, np.uint8)
    u[2], u[3], u[255] = 5, 9, 12
    b = kv4.pack(u)
    assert b[1] == 5 | 9 << 4 and b[127] == 12 << 4 and np.array_equal(kv4.unpack(b), u)


# ------------------------------------------------------------------ attention

def test_attend_single_cell_is_its_value():
    c = Attend(seed=5, G=2, T=2, lens=(1,), context=9)
    out, _, status = c.reference()
    slot = c.page_table[0, c.sel[0]]
    for g in range(2):
        _, v = kv4.values(c.kv_pool[0, g, slot], c.kv_scale[0, g, slot])
        assert np.allclose(out[0, :, 12 * g:12 * g + 12], v, rtol=1e-14)
    assert status == 0


def test_attend_equal_scores_give_the_mean():
    c = Attend(seed=6, lens=(40,))
    c.q[:] = 0
    out, _, _ = c.reference()
    _, v = kv4.values(c.kv_pool[0, 0, c.page_table[0, c.sel]], c.kv_scale[0, 0, c.page_table[0, c.sel]])
    assert np.allclose(out[0, 0], v.mean(0), rtol=1e-12)


def test_attend_matches_brute_force():
    c = Attend(seed=7, n_seq=2, G=2, H=3, T=3, lens=(5, 0), P=4, dense=True, causal=True, shared=True)
    out, aux, _ = c.reference()
    for t in range(3):
        for h in range(6):
            s, v = [], []
            for pos in range(min(5, int(c.q_limit[0, t]))):
                slot = c.page_table[0, pos // 4] * 4 + pos % 4
                u = [(int(c.kv_pool[0, h // 3, slot, i // 2 + 128 * kv]) >> (4 * (i % 2))) & 15 for kv in (0, 1) for i in range(256)]
                f = c.kv_scale[0, h // 3, slot].astype(float)
                s.append(sum(float(c.q[0, t, h, i]) * (u[i] * f[0] + f[1]) for i in range(256)) / 16)
                v.append([u[256 + i] * f[2] + f[3] for i in range(256)])
            w = np.exp(np.array(s) - max(s))
            assert np.allclose(out[0, t, h], w @ np.array(v) / w.sum(), rtol=1e-10)
    assert not out[1].any() and not aux["n"][1].any()


def test_masked_and_bad_cells_are_left_out():
    c = Attend(seed=8, lens=(30,), context=40)
    full = Attend(seed=8, lens=(30,), context=40)
    keep = np.ones(30, bool)
    keep[[3, 17]] = False
    c.page_table[0, c.sel[3]] = -1
    c.page_table[0, c.sel[17]] = c.pool_cells
    full.sel, full.offsets = full.sel[keep], np.array([0, 28], np.int32)
    out, _, status = c.reference()
    assert np.allclose(out, full.reference()[0], rtol=1e-13) and status == kv4.STATUS_BAD_SLOT


def test_bf16_round():
    assert bf16_round(np.float32([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -2.5])).tolist() == [1.0, 1 + 2.0 ** -6, -2.5]


# ---------------------------------------------------------------------- pages

def draw_pages(seed, n_seq, max_new, P, L, shared, spare, grow=None, holes=0.0):
    """Lengths, tables and free lists of sequences that hold the pages of their lengths."""
    rng = np.random.default_rng(seed)
    cap = L * P
    cur = rng.integers(0, cap + 1, n_seq)
    step = rng.integers(-cap, max_new + 1, n_seq) if grow is None else rng.integers(0, max_new + 1, n_seq) * grow
    new = np.clip(cur + step, 0, cap)
    held = -(-cur // P)
    if shared:
        pool = int(held.sum()) + spare
        order = rng.permutation(pool)
        ends = np.concatenate([[0], np.cumsum(held)])
        free = [order[ends[-1]:]]
        own = [order[ends[b]:ends[b + 1]] for b in range(n_seq)]
    else:
        pool = L + spare
        order = [rng.permutation(pool) for _ in range(n_seq)]
        own = [order[b][:held[b]] for b in range(n_seq)]
        free = [order[b][held[b]:] for b in range(n_seq)]
    pool = max(pool, 1)
    table = np.full((n_seq, L), -1, np.int32)
    for b in range(n_seq):
        table[b, :held[b]] = np.where(rng.random(held[b]) < holes, -1, own[b])
    pages = np.full((len(free), pool), -7, np.int32)
    for i, f in enumerate(free):
        pages[i, :len(f)] = f
    return dict(cur_len=cur.astype(np.int32), new_len=new.astype(np.int32), page_table=table, free_pages=pages,
                free_count=np.array([len(f) for f in free], np.int32), max_new=max_new, page_cells=P, pool_pages=pool)


def test_pages_by_hand():
    table = np.array([[4, 7, -1], [2, -1, -1]], np.int32)
    free = np.array([[9, 1, 3, 0, 0, 0, 0, 0, 0, 0]], np.int32)
    count = np.array([3], np.int32)
    # sequence 0 gives back page 7, sequence 1 grows from 3 to 9 cells (2 more pages of 4)
    out = pm.page_map([8, 3], [4, 9], table, free, count, 6, 4, 10)
    assert out[0].tolist() == [4, 9] and out[1].tolist() == [0, 4, 13]
    assert table.tolist() == [[4, -1, -1], [2, 7, 3]] and count.tolist() == [2] and free[0, :2].tolist() == [9, 1]
    assert out[2][1].tolist() == [3, 4, 5, 6, 7, 8] and out[3][1].tolist() == [11, 28, 29, 30, 31, 12]
    assert out[4][0].tolist() == [0] * 6 and out[4][1].tolist() == [4, 5, 6, 7, 8, 9] and out[5] == 0


def test_pages_shrink_and_grow_back_is_identity():
    c = draw_pages(11, 9, 50, 4, 20, True, 13, grow=1)
    before = {k: c[k].copy() for k in ("page_table", "free_pages", "free_count")}
    kw = dict(max_new=80, page_cells=4, pool_pages=c["pool_pages"])
    pm.page_map(c["cur_len"], c["cur_len"] // 2, c["page_table"], c["free_pages"], c["free_count"], **kw)
    out = pm.page_map(c["cur_len"] // 2, c["cur_len"], c["page_table"], c["free_pages"], c["free_count"], **kw)
    assert out[5] == 0 and np.array_equal(c["page_table"], before["page_table"])
    n = int(before["free_count"][0])
    assert c["free_count"][0] == n and np.array_equal(c["free_pages"][0, :n], before["free_pages"][0, :n])


def test_pages_exhausted_serves_a_prefix():
    table = np.full((4, 4), -1, np.int32)
    free, count = np.arange(8, dtype=np.int32)[None].copy(), np.array([5], np.int32)
    out = pm.page_map([0, 0, 0, 0], [2, 4, 1, 0], table, free, count, 4, 1, 8)
    assert out[0].tolist() == [2, 0, 0, 0] and out[5] == pm.STATUS_NO_PAGES and count[0] == 3


# ------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def lib():
    qsa_build.build()
    return qsa.load_library()


MB = 1 << 20
AT = 1 << 32  # aligned addresses that are never read: every call fails its checks


def shape(**kw):
    f = dict(n_kv_heads=2, q_per_kv=12, n_queries=2, pool_cells=4096, page_table_len=256, chunk_cells=128,
             softmax_scale=1 / 16, page_cells=16)
    f.update(kw)
    return qsa.make_shape(**f)


def rows_call(lib, name, s=None, **over):
    a = dict(n_seq=3, n_pools=1, n_new=4, dtype=qsa.QSA_F32, k=AT, v=AT + MB, positions=AT + 2 * MB, table=AT + 3 * MB,
             pool=AT + 4 * MB, scale=AT + 5 * MB, status=None)
    a.update(over)
    s = ctypes.byref(s or shape())
    if name == "append":
        return lib.qsa_kv4_append(s, a["n_seq"], a["n_pools"], a["n_new"], a["dtype"], a["k"], a["v"], a["positions"],
                                  a["table"], a["pool"], a["scale"], a["status"], None)
    return lib.qsa_kv4_read(s, a["n_seq"], a["n_pools"], a["n_new"], a["dtype"], a["positions"], a["table"], a["pool"],
                            a["scale"], a["k"], a["v"], a["status"], None)


INVALID, UNSUPPORTED = qsa.QSA_ERR_INVALID_ARG, qsa.QSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["append", "read"])
@pytest.mark.parametrize("over,code", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(positions=None), INVALID), (dict(table=None), INVALID),
    (dict(pool=None), INVALID), (dict(scale=None), INVALID), (dict(k=AT + 8), INVALID), (dict(pool=AT + 4 * MB + 16), INVALID),
    (dict(scale=AT + 4), INVALID), (dict(positions=AT + 2), INVALID), (dict(status=AT + 1), INVALID),
    (dict(n_new=-1), INVALID), (dict(n_seq=-1, n_pools=-1), INVALID), (dict(n_pools=2), INVALID), (dict(n_pools=0), INVALID),
    (dict(dtype=5), INVALID), (dict(k=AT + 4 * MB), INVALID), (dict(v=AT + 5 * MB), INVALID),
    (dict(n_seq=1 << 16, n_new=1 << 15), UNSUPPORTED), (dict(n_seq=2 ** 31 - 1, n_new=2 ** 31 - 1), UNSUPPORTED),
])
def test_rows_refused(lib, name, over, code):
    assert rows_call(lib, name, **over) == code


@pytest.mark.parametrize("name", ["append", "read"])
@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 128, UNSUPPORTED), ("n_kv_heads", 0, INVALID), ("n_kv_heads", 65536, UNSUPPORTED),
    ("pool_cells", 0, INVALID), ("pool_cells", 4097, INVALID), ("page_table_len", 0, INVALID), ("page_cells", -1, INVALID),
    ("page_table_len", 1 << 28, INVALID),
])
def test_rows_shape_refused(lib, name, field, value, code):
    s = shape()
    setattr(s, field, value)
    assert rows_call(lib, name, s) == code


@pytest.mark.parametrize("name", ["append", "read"])
def test_rows_nothing_to_do(lib, name):
    assert rows_call(lib, name, n_new=0) == qsa.QSA_OK
    assert rows_call(lib, name, n_seq=0, n_pools=0, k=None, v=None, positions=None) == qsa.QSA_OK


def attn_call(lib, s=None, **over):
    a = dict(n_seq=3, n_pools=3, q=AT, pool=AT + MB, scale=AT + 2 * MB, table=AT + 3 * MB, sel=AT + 4 * MB,
             offsets=AT + 5 * MB, most=100, limit=AT + 6 * MB, dtype=qsa.QSA_F32, out=AT + 7 * MB, ws=AT + 8 * MB,
             size=1 << 40, status=None)
    a.update(over)
    return lib.qsa_kv4_attn_batch(ctypes.byref(s or shape()), a["n_seq"], a["n_pools"], a["q"], a["pool"], a["scale"],
                                  a["table"], a["sel"], a["offsets"], a["most"], a["limit"], a["dtype"], a["out"],
                                  a["ws"], a["size"], a["status"], None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), INVALID), (dict(pool=None), INVALID), (dict(scale=None), INVALID), (dict(table=None), INVALID),
    (dict(offsets=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(q=AT + 4), INVALID),
    (dict(pool=AT + MB + 16), INVALID), (dict(scale=AT + 8), INVALID), (dict(ws=AT + 64), INVALID), (dict(out=AT + 8), INVALID),
    (dict(sel=AT + 2), INVALID), (dict(limit=AT + 1), INVALID), (dict(offsets=AT + 3), INVALID), (dict(status=AT + 2), INVALID),
    (dict(out=AT), INVALID), (dict(out=AT + MB), INVALID), (dict(out=AT + 2 * MB), INVALID), (dict(ws=AT), INVALID),
    (dict(dtype=9), INVALID), (dict(most=-1), INVALID), (dict(n_seq=0, n_pools=1), INVALID), (dict(n_pools=2), INVALID),
    (dict(n_seq=65536, n_pools=1), UNSUPPORTED), (dict(size=16), qsa.QSA_ERR_WORKSPACE),
])
def test_attn_refused(lib, over, code):
    assert attn_call(lib, **over) == code


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 128, UNSUPPORTED), ("q_per_kv", 0, INVALID), ("q_per_kv", 65, UNSUPPORTED), ("n_queries", 0, INVALID),
    ("n_queries", 65537, UNSUPPORTED), ("q_dtype", 3, INVALID), ("softmax_scale", float("inf"), INVALID),
    ("softmax_scale", float("nan"), INVALID), ("pool_cells", 4097, INVALID), ("n_kv_heads", 0, INVALID),
])
def test_attn_shape_refused(lib, field, value, code):
    s = shape()
    setattr(s, field, value)
    assert attn_call(lib, s) == code
    if field != "pool_cells":
        assert lib.qsa_kv4_attn_workspace_bytes(ctypes.byref(s), 3, 100, ctypes.byref(ctypes.c_size_t(0))) == code


@pytest.mark.parametrize("value,ok", [(2.0 ** 100, False), (-2.0 ** 127, False), (3e38, False), (2.0 ** 99, True), (0.0, True)])
def test_attn_softmax_scale_refused(lib, value, ok):
    """Scales that the kernels' scaling by powers of two would overflow."""
    bytes_ = ctypes.c_size_t(0)
    s = shape(softmax_scale=value)
    assert lib.qsa_kv4_attn_workspace_bytes(ctypes.byref(s), 3, 100, ctypes.byref(bytes_)) == (qsa.QSA_OK if ok else INVALID)
    if not ok:
        assert attn_call(lib, s) == INVALID


def test_attn_pools_of_2_to_32_rows_refused(lib):
    """Refused by the host's checks, before the device is asked anything."""
    assert attn_call(lib, shape(n_kv_heads=65535, pool_cells=1 << 16, page_table_len=4096), n_seq=2, n_pools=2) == UNSUPPORTED
    assert attn_call(lib, shape(n_kv_heads=1, pool_cells=1 << 30, page_table_len=1 << 20), n_seq=4, n_pools=4) == UNSUPPORTED


def test_attn_workspace_bytes(lib):
    size = qsa.qsa_kv4_attn_workspace_bytes(shape(), 3, 100)
    assert size > 0 and size % 256 == 0
    assert attn_call(lib, size=size - 1) == qsa.QSA_ERR_WORKSPACE
    assert lib.qsa_kv4_attn_workspace_bytes(ctypes.byref(shape()), 3, 100, None) == INVALID
    assert lib.qsa_kv4_attn_workspace_bytes(None, 3, 100, ctypes.byref(ctypes.c_size_t(0))) == INVALID


def page_call(lib, **over):
    names = ("cur", "new", "table", "free", "count", "len", "offsets", "positions", "slots", "limit")
    a = dict(n_seq=3, n_pools=1, max_new=4, P=16, L=64, pool=200, status=None,
             **{n: AT + i * MB for i, n in enumerate(names)})
    a.update(over)
    return lib.qsa_page_map(a["n_seq"], a["n_pools"], a["max_new"], a["P"], a["L"], a["pool"], *[a[n] for n in names],
                            a["status"], None)


@pytest.mark.parametrize("over,code", [
    (dict(cur=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(count=None), INVALID), (dict(len=None), INVALID), (dict(offsets=None), INVALID), (dict(positions=None), INVALID),
    (dict(slots=None), INVALID), (dict(limit=None), INVALID), (dict(table=AT + 2), INVALID), (dict(status=AT + 1), INVALID),
    (dict(n_seq=0), INVALID), (dict(max_new=-1), INVALID), (dict(P=0), INVALID), (dict(L=0), INVALID), (dict(pool=0), INVALID),
    (dict(n_pools=2), INVALID), (dict(len=AT), INVALID), (dict(slots=AT + 7 * MB), INVALID), (dict(offsets=AT + MB), INVALID),
    (dict(n_seq=65536), UNSUPPORTED), (dict(L=1 << 28), UNSUPPORTED), (dict(n_seq=60000, max_new=60000), UNSUPPORTED),
    (dict(pool=1 << 28), UNSUPPORTED), (dict(n_seq=3, L=1 << 26), UNSUPPORTED),
])
def test_page_map_refused(lib, over, code):
    assert page_call(lib, **over) == code


def test_binding_refuses_what_is_no_device_array():
    """Host tensors, strided ones and numbers past 32 bits raise before anything is launched."""
    torch = pytest.importorskip("torch")
    import sparse_selection_int8_gb300 as qsa
    shape = qsa.make_shape(n_kv_heads=1, q_per_kv=1, n_queries=1, pool_cells=4, page_table_len=4, chunk_cells=1,
                           softmax_scale=1.0)
    host = torch.zeros(1, 1, 1, 256)
    a = 1 << 32
    with pytest.raises(ValueError, match="device tensor"):
        qsa.qsa_kv4_append(shape, 1, 1, 1, qsa.QSA_F32, host, a, a, a, a, a, None, 0)
    with pytest.raises(ValueError, match="device tensor"):
        qsa.qsa_kv4_read(shape, 1, 1, 1, qsa.QSA_F32, a, a, a, a, a, host, None, 0)
    with pytest.raises(ValueError, match="device tensor"):
        qsa.qsa_kv4_attn_batch(shape, 1, 1, a, a, a, a, None, host, 4, None, qsa.QSA_F32, a, a, 1 << 30, None, 0)
    with pytest.raises(ValueError, match="device tensor"):
        qsa.qsa_page_map(1, 1, 1, 1, 4, 4, *[a + (i << 20) for i in range(9)], host, None, 0)
    with pytest.raises(OverflowError):
        qsa.qsa_page_map(1, 1, 1, 1, 4, 1 << 31, *[a + (i << 20) for i in range(10)], None, 0)
    with pytest.raises(TypeError):
        qsa.qsa_kv4_append(shape, 1.5, 1, 1, qsa.QSA_F32, a, a, a, a, a, a, None, 0)
    with pytest.raises(TypeError):
        qsa.qsa_kv4_append(None, 1, 1, 1, qsa.QSA_F32, a, a, a, a, a, a, None, 0)
    with pytest.raises(TypeError):
        qsa.qsa_kv4_append(b"short", 1, 1, 1, qsa.QSA_F32, a, a, a, a, a, a, None, 0)
    with pytest.raises(qsa.QsaError):  # an address that is not aligned
        qsa.qsa_kv4_append(shape, 1, 1, 1, qsa.QSA_F32, a + 4, a, a, a, a, a, None, 0)
