"""The 4-bit cells on the GPU against their oracle: append and read bit for bit, attention
within bounds derived from its arithmetic, and the three of them with the page maps in a run."""
import numpy as np
import pytest

from kv4_cases import Attend, assert_attend, bf16_round
from oracle import kv4, page_map as pm
from test_kv4_oracle import draw_pages

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


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(dtype) if dtype is not None else t


# ------------------------------------------------------------ append and read

class Rows:
    def __init__(self, seed, n_seq, G, n_new, P, shared, dtype, spoil=True):
        rng = np.random.default_rng(seed)
        self.n_seq, self.G, self.n_new, self.P, self.dtype = n_seq, G, n_new, P, dtype
        self.L = -(-(n_new + 50) // P)
        pages = self.L + 1
        self.n_pools = 1 if shared else n_seq
        self.cells = pages * P * (n_seq if shared else 1)
        order = rng.permutation(pages * n_seq)
        self.table = (order[:n_seq * self.L].reshape(n_seq, -1) if shared
                      else np.stack([rng.permutation(pages)[:self.L] for _ in range(n_seq)])).astype(np.int32)
        self.pos = np.stack([rng.permutation(self.L * P)[:n_new] for _ in range(n_seq)]).astype(np.int32)
        self.pos[rng.random(self.pos.shape) < 0.1] = -1
        if spoil and n_new > 4:
            self.pos[0, 0], self.pos[-1, 1] = self.L * P, -5
            self.table[-1, self.pos[-1, 2] // P if self.pos[-1, 2] >= 0 else 0] = -1
            self.table[0, self.pos[0, 3] // P if self.pos[0, 3] >= 0 else 0] = self.cells // P
        shape = (n_seq, n_new, G, 256)
        self.k, self.v = (rng.standard_normal(shape) * np.exp(rng.uniform(-30, 30, shape[:3] + (1,)))
                          + rng.standard_normal(shape[:3] + (1,)) for _ in "kv")
        self.k, self.v = self.k.astype(np.float32), self.v.astype(np.float32)
        if dtype == "bf16":
            self.k, self.v = bf16_round(self.k), bf16_round(self.v)
        self.pool = rng.integers(0, 256, (self.n_pools, G, self.cells, 256), dtype=np.uint8)
        self.scale = rng.standard_normal((self.n_pools, G, self.cells, 4)).astype(np.float32)

    def shape(self, qsa):
        return qsa.make_shape(n_kv_heads=self.G, q_per_kv=1, n_queries=1, pool_cells=self.cells,
                              page_table_len=self.L, chunk_cells=1, softmax_scale=1.0, page_cells=self.P)


def check_append(qsa, a):
    t = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    code = qsa.QSA_BF16 if a.dtype == "bf16" else qsa.QSA_F32
    pool, scale, status = dev(a.pool), dev(a.scale), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (a.shape(qsa), a.n_seq, a.n_pools, a.n_new)
    qsa.qsa_kv4_append(*args, code, dev(a.k, t), dev(a.v, t), dev(a.pos), dev(a.table), pool, scale, status)
    want_pool, want_scale = a.pool.copy(), a.scale.copy()
    want_status = kv4.append(a.k, a.v, a.pos, a.table, a.P, want_pool, want_scale)
    got = pool.cpu().numpy()
    assert np.array_equal(got, want_pool), f"{np.argwhere(got != want_pool)[:4].tolist()}"
    assert np.array_equal(scale.cpu().numpy().view(np.uint32), want_scale.view(np.uint32))
    assert int(status.item()) == want_status
    # and back
    for out, half in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -24 + 2.0 ** -8)):
        k, v = (torch.full(a.k.shape, 7.0, dtype=out, device="cuda") for _ in "kv")
        status.zero_()
        qsa.qsa_kv4_read(*args, qsa.QSA_F32 if out == torch.float32 else qsa.QSA_BF16, dev(a.pos), dev(a.table), pool,
                         scale, k, v, status)
        k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
        bad = 0
        for b in range(a.n_seq):
            for i in range(a.n_new):
                slot, why = kv4.resolve(a.table[b], int(a.pos[b, i]), a.P, a.cells)
                bad |= why & ~kv4.STATUS_NOT_RESIDENT
                if slot < 0:
                    assert not k[b, i].any() and not v[b, i].any()
                    continue
                at = 0 if a.n_pools == 1 else b
                ek, ev = kv4.values(want_pool[at, :, slot], want_scale[at, :, slot])
                # one rounding to fp32 (and one to bf16); below 2^-120 in units of the smallest normals
                assert (np.abs(k[b, i] - ek) <= half * np.abs(ek) + 2.0 ** -120).all()
                assert (np.abs(v[b, i] - ev) <= half * np.abs(ev) + 2.0 ** -120).all()
        assert int(status.item()) == bad


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n_seq,G,n_new,P,shared", [(1, 1, 1, 1, False), (3, 2, 37, 1, True), (5, 3, 200, 16, True),
                                                    (2, 1, 1000, 24, False), (16, 2, 4, 64, False), (1, 5, 7, 2, True),
                                                    (2, 5, 3001, 16, True)])
def test_append_and_read(qsa, dtype, n_seq, G, n_new, P, shared):
    check_append(qsa, Rows(100 + n_new, n_seq, G, n_new, P, shared, dtype))


def test_append_borders(qsa):
    """Quotients on and beside the borders between codes, constant rows, tiny and huge ranges."""
    a = Rows(9, 1, 1, 64, 1, False, "f32", spoil=False)
    rng = np.random.default_rng(10)
    for i in range(64):
        s = np.float32(np.exp(rng.uniform(-60, 60)))
        row = (rng.integers(0, 15, 256).astype(np.float32) + np.float32(0.5)) * s
        near = rng.integers(-1, 2, 256)
        row = np.where(near > 0, np.nextafter(row, np.float32(np.inf)), np.where(near < 0, np.nextafter(row, np.float32(0)), row))
        row[:2] = 0, 15 * s
        a.k[0, i, 0] = row if i % 2 else row - np.float32(7) * s
        a.v[0, i, 0] = bf16_round(row)
    a.k[0, 0, 0] = 3.5
    a.k[0, 1, 0] = np.float32(1e-44) * np.arange(256)
    a.k[0, 2, 0] = np.float32(2.0 ** 125) * np.linspace(-1, 1, 256)
    a.k[0, 3, 0] = 0
    a.k[0, 4, 0] = np.float32(1) + np.float32(2.0 ** -23) * (np.arange(256) % 5)
    check_append(qsa, a)


# -------------------------------------------------------------------- attention

class Call:
    """A drawn attention call on the device."""

    def __init__(self, qsa, c, out_dtype):
        self.qsa, self.c = qsa, c
        bf = c.q_dtype == "bf16"
        self.shape = qsa.make_shape(n_kv_heads=c.G, q_per_kv=c.H, n_queries=c.T, pool_cells=c.pool_cells,
                                    page_table_len=c.table_len, chunk_cells=1, softmax_scale=c.softmax_scale,
                                    q_dtype=qsa.QSA_BF16 if bf else qsa.QSA_F32, page_cells=c.P)
        self.q = dev(c.q, torch.bfloat16 if bf else torch.float32)
        self.pool, self.scale, self.table = dev(c.kv_pool), dev(c.kv_scale), dev(c.page_table)
        self.sel = None if c.sel is None else dev(c.sel if len(c.sel) else np.zeros(1, np.int32))
        self.offsets = dev(c.offsets)
        self.limit = None if c.q_limit is None else dev(c.q_limit)
        self.code = qsa.QSA_BF16 if out_dtype == "bf16" else qsa.QSA_F32
        self.out = torch.full(c.q.shape, 3.0, dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32, device="cuda")
        self.ws = torch.full((qsa.qsa_kv4_attn_workspace_bytes(self.shape, c.n_seq, c.max_selected),), 255,
                             dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def __call__(self, stream=None):
        c = self.c
        self.qsa.qsa_kv4_attn_batch(self.shape, c.n_seq, c.n_pools, self.q, self.pool, self.scale, self.table, self.sel,
                                    self.offsets, c.max_selected, self.limit, self.code, self.out, self.ws, self.ws.numel(),
                                    self.status, stream)
        return self.out

    def check(self, what=""):
        self()
        torch.cuda.synchronize()
        rel, status = assert_attend(self.out.float().cpu().numpy(), self.c, self.code == self.qsa.QSA_BF16, what)
        assert int(self.status.item()) == status, what
        return rel


DTYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")]


@pytest.mark.parametrize("n", [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 255, 256, 257, 600])
@pytest.mark.parametrize("q,o", DTYPES[:2])
def test_attend_list_lengths(qsa, n, q, o):
    Call(qsa, Attend(seed=n, lens=(n,), q_dtype=q), o).check()


@pytest.mark.parametrize("H,T", [(1, 1), (7, 1), (8, 1), (9, 1), (12, 1), (16, 1), (17, 1), (12, 2), (5, 5), (12, 3), (12, 4),
                                 (10, 5), (64, 1), (13, 5), (12, 8), (12, 17)])
@pytest.mark.parametrize("q,o", DTYPES)
def test_attend_row_counts(qsa, H, T, q, o):
    """Rows per KV head on both sides of every block and tile size, with limits that leave some rows few cells."""
    c = Attend(seed=H * 100 + T, n_seq=2, G=2, H=H, T=T, lens=(301, 77), P=8, dense=True, causal=True, q_dtype=q)
    Call(qsa, c, o).check()


@pytest.mark.parametrize("H", [1, 4, 7, 8, 12, 13, 16, 20, 24, 25, 32, 33, 48])
@pytest.mark.parametrize("q,o", DTYPES)
def test_attend_row_counts_of_many_tiles(qsa, H, q, o):
    """The same with more tiles than multiprocessors, where blocks hold up to 32 rows."""
    c = Attend(seed=H, n_seq=20, G=2, H=H, lens=(700, 12, 640, 129), P=4, q_dtype=q, holes=0.02)
    Call(qsa, c, o).check()


@pytest.mark.parametrize("kw", [
    dict(n_seq=5, G=3, lens=(0, 700, 1, 0, 257), P=1),
    dict(n_seq=4, G=2, T=4, lens=(2051, 600, 33, 1500), P=16, holes=0.05, causal=True),
    dict(n_seq=3, G=1, T=2, lens=(900,), P=24, shared=True, order="shuffled"),
    dict(n_seq=2, G=2, lens=(500, 40), P=3, shared=True, order="repeats", holes=0.2),
    dict(n_seq=40, G=1, lens=(65, 3, 0, 129), P=64, dense=True, shared=True),
    dict(n_seq=3, G=4, H=8, lens=(4000, 10, 999), P=64, dense=True, causal=True, shared=True, holes=0.1),
    dict(n_seq=1, G=1, T=1, lens=(40000,), P=1),
    dict(n_seq=70, G=2, H=4, lens=(5,), P=2, dense=True),
], ids=str)
@pytest.mark.parametrize("q,o", DTYPES[:2])
def test_attend_batches(qsa, kw, q, o):
    Call(qsa, Attend(seed=77, q_dtype=q, **kw), o).check()


@pytest.mark.parametrize("gain", [1e-3, 8.0, 60.0])
@pytest.mark.parametrize("q,o", DTYPES[:2])
def test_attend_peaked_and_flat(qsa, gain, q, o):
    """Scores from flat to a single dominant cell; the running maximum moves often in an ascending list."""
    c = Attend(seed=4, lens=(3000,), T=2, q_dtype=q, q_gain=gain, order="shuffled")
    Call(qsa, c, o).check()


@pytest.mark.parametrize("q,o", DTYPES[:2])
def test_attend_scores_that_rise(qsa, q, o):
    """Every cell scores above the one before it (the maximum moves at every cell), then every one below."""
    for way in (1, -1):
        c = Attend(seed=12, lens=(1200,), q_dtype=q)
        c.kv_pool[..., :128] = 0
        slots = c.page_table[0, c.sel]
        c.q[0, 0, :, :] = 1.0
        c.kv_scale[0, 0, slots, 1] = (np.arange(1200)[::way] * 0.01).astype(np.float32)
        Call(qsa, c, o).check()


@pytest.mark.parametrize("q,o", DTYPES[:2])
def test_attend_scale_ranges(qsa, q, o):
    """V scales over many binary orders, zeros among them."""
    c = Attend(seed=13, lens=(700,), T=2, q_dtype=q)
    rng = np.random.default_rng(14)
    s = np.exp2(rng.uniform(-40, 20, c.kv_scale.shape[:3])).astype(np.float32)
    s[rng.random(s.shape) < 0.1] = 0
    c.kv_scale[..., 2], c.kv_scale[..., 3] = s, -7 * s
    Call(qsa, c, o).check()


def test_attend_garbage_in_unseen_cells(qsa):
    """NaN and infinities in cells that are masked, beyond a limit or not listed do not reach the output."""
    for bad in (np.nan, np.inf, -np.inf):
        c = Attend(seed=15, n_seq=2, G=2, T=3, lens=(500, 90), P=4, dense=True, causal=True, holes=0.1)
        c.q_limit = c.q_limit - 150
        clean = c.reference()[0]
        used = np.zeros((2, c.pool_cells), bool)
        for b in range(2):
            for pos in range(max(0, int(c.q_limit[b].max()))):
                e = c.page_table[b, pos // 4]
                if e >= 0:
                    used[b, e * 4 + pos % 4] = True
        for b in range(2):
            c.kv_scale[b, :, ~used[b]] = bad
        assert not c.q_limit[1].max() > 0  # the second sequence's rows see nothing
        call = Call(qsa, c, "f32")
        got = call().cpu().numpy()
        assert np.isfinite(got).all()
        assert np.linalg.norm(got - clean) <= 2e-5 * np.linalg.norm(clean)
        assert not got[1].any()


def test_attend_limits_in_any_order(qsa):
    """A cell that one row sees and its neighbour does not may hold anything for the latter."""
    c = Attend(seed=16, lens=(400,), T=4, P=1, dense=True, causal=True)
    c.q_limit[0] = [400, 0, 1, 33]
    Call(qsa, c, "f32").check()
    clean = c.reference()[0]
    c.kv_scale[0, :, c.page_table[0, 33:]] = np.nan
    got = Call(qsa, c, "f32")().cpu().numpy()
    assert np.isnan(got[0, 0]).all()  # the row that sees them
    assert not got[0, 1].any()
    assert np.linalg.norm(got[0, 2:] - clean[0, 2:]) <= 2e-5 * np.linalg.norm(clean[0, 2:])


@pytest.mark.parametrize("big", [2.0 ** 14, 2.0 ** 20, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("kw,q,o", [(dict(lens=(300,), T=4), "f32", "f32"), (dict(lens=(300,), T=4), "bf16", "bf16"),
                                    (dict(lens=(3000,), T=4, G=2), "f32", "f32"), (dict(lens=(3000,), T=4, H=3), "bf16", "bf16"),
                                    (dict(n_seq=40, lens=(500, 90), T=4, G=2, H=4), "bf16", "f32"),
                                    (dict(lens=(4097,), T=100), "bf16", "bf16")], ids=str)
def test_attend_unseen_scales_of_any_size(qsa, big, kw, q, o):
    """Finite V scales that a row does not see do not reach it, in pairs of one part and of several, also
    where the row has seen no cell yet; padding rows (limit 0) are zeros."""
    c = Attend(seed=80, P=4, dense=True, causal=True, q_dtype=q, **kw)
    n = int(c.offsets[1])
    c.kv_scale[..., 2:] *= np.float32(big ** -0.5)
    c.q_limit[:, :] = np.linspace(0, n // 3, c.T).astype(int)
    c.q_limit[:, -1] = n
    for b in range(c.n_seq):
        pos = np.arange(n // 3, c.context)
        e = c.page_table[b, pos // 4]
        c.kv_scale[b, :, e * 4 + pos % 4, 2:] *= np.float32(big ** 0.75)
        c.kv_scale[b, :, e * 4 + pos % 4, 2:] *= np.float32(big ** 0.75)
    Call(qsa, c, o).check()


@pytest.mark.parametrize("kw,t", [(dict(lens=(300, 77), n_seq=2, holes=0.1, T=2), "f32"), (dict(lens=(3001,), G=2, holes=0.1), "bf16"),
                                  (dict(lens=(700,), T=3, dense=True, causal=True), "f32"),
                                  (dict(lens=(4100,), T=100, holes=0.05), "bf16"),
                                  (dict(lens=(4097,), T=100, dense=True, causal=True), "bf16")], ids=str)
@pytest.mark.parametrize("scale", [0.0, -0.0, -1.0 / 16, 2.0 ** -30, -(2.0 ** -60), 2.0 ** -120])
def test_attend_softmax_scales(qsa, scale, kw, t):
    """No scale (the mean of the values), negative and tiny ones, with masked pages and lists that end inside a tile."""
    c = Attend(seed=81, P=4, q_dtype=t, **kw)
    c.softmax_scale = scale
    Call(qsa, c, t).check()
    c.q[0, 0, 0] = 0  # a row of zeros
    Call(qsa, c, t).check("zeros")
    if abs(scale) < 1e-3:
        c.kv_scale[..., :2] *= np.float32(2.0 ** 122)  # scores stay small beside the scale
        c.q *= np.float32(2.0 ** -112)
        Call(qsa, c, t).check("K scales")


def test_attend_nonfinite_queries_stay_in_their_row(qsa):
    c = Attend(seed=17, lens=(300,), T=2)
    clean = c.reference()[0]
    c.q[0, 0, 3, 7], c.q[0, 1, 5, 0] = np.nan, np.inf
    got = Call(qsa, c, "f32")().cpu().numpy()
    rows = np.ones((2, 12), bool)
    rows[0, 3] = rows[1, 5] = False
    assert not np.isfinite(got[0][~rows]).any()
    assert np.linalg.norm(got[0][rows] - clean[0][rows]) <= 2e-5 * np.linalg.norm(clean[0][rows])


def test_attend_bad_inputs_are_masked_and_reported(qsa):
    c = Attend(seed=18, n_seq=2, lens=(300, 200), P=4)
    c.sel[5], c.sel[310], c.sel[17] = -1, c.table_len * 4, -2 ** 31
    c.page_table[0, c.sel[40] // 4] = c.pool_pages
    c.page_table[1, c.sel[320] // 4] = -9
    Call(qsa, c, "f32").check()
    # offsets that decrease, and a list above the bound
    c = Attend(seed=19, n_seq=3, lens=(300, 200, 50))
    c.offsets[2] = 250
    c.max_selected = 150
    call = Call(qsa, c, "f32")
    call.check()


def test_attend_repeats_bitwise_and_on_a_stream(qsa):
    c = Attend(seed=20, n_seq=3, G=2, T=2, lens=(900, 5000, 30), P=16, holes=0.05)
    call = Call(qsa, c, "f32")
    first = call().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side):
        call.ws.fill_(170)
        call.out.fill_(9)
        torch.cuda.synchronize()
        call(stream)
        torch.cuda.synchronize()
        assert torch.equal(call.out, first)


@pytest.mark.parametrize("kw", [dict(n_seq=300, G=2, H=4, lens=(100, 1, 129, 40, 0, 128)), dict(n_seq=30, G=16, H=12, T=2, lens=(60, 200)),
                                dict(n_seq=700, G=1, H=1, lens=(3, 90), dense=True, P=8, shared=True)], ids=str)
@pytest.mark.parametrize("q,o", DTYPES)
def test_attend_whole_pairs_in_a_row(qsa, kw, q, o):
    """Several short (sequence, KV head) pairs to a multiprocessor, each written to its own place, time after time."""
    call = Call(qsa, Attend(seed=71, q_dtype=q, **kw), o)
    call.check()
    first = call.out.clone()
    for _ in range(40):
        call.out.fill_(9)
        call()
        assert torch.equal(call.out, first)


def test_attend_captured(qsa):
    """One graph serves other lengths within the bound: lists, limits and tables are read at replay."""
    a = Attend(seed=21, n_seq=4, G=2, lens=(700, 20, 300, 1), P=8, dense=True, causal=True)
    call = Call(qsa, a, "bf16")
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(torch.cuda.current_stream())
    for lens in ((1, 700, 0, 64), (0, 0, 0, 0), (700, 700, 700, 700)):
        b = Attend(seed=22, n_seq=4, G=2, lens=lens, P=8, dense=True, causal=True, context=700)
        a.offsets, a.q_limit, a.q = b.offsets, b.q_limit, b.q
        for x, y in ((call.offsets, a.offsets), (call.limit, a.q_limit), (call.q, a.q)):
            x.copy_(dev(y))
        g.replay()
        torch.cuda.synchronize()
        assert_attend(call.out.float().cpu().numpy(), a, True, str(lens))


def test_attend_two_calls_on_two_streams(qsa):
    """Two calls at once, each with its own workspace."""
    calls = [Call(qsa, Attend(seed=30 + i, n_seq=4, G=2, T=2, lens=(3000, 700), P=4), "f32") for i in range(2)]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for c, s in zip(calls, streams):
            c(s)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c.out, w)


# bf16 windows of so many rows and cells that the kernel with 128 rows a block takes them
WIDE = dict(q_dtype="bf16", H=12, T=100, lens=(4100,))


@pytest.mark.parametrize("kw", [
    dict(H=12, T=100, lens=(4100,)),
    dict(H=12, T=100, lens=(4097,), P=16, dense=True, causal=True),
    dict(H=12, T=11, n_seq=6, G=2, lens=(4000, 3900, 128), P=16, holes=0.05),
    dict(H=64, T=4, n_seq=5, G=2, lens=(1900, 77, 0, 640, 1800), P=24, dense=True, causal=True, shared=True),
    dict(H=7, T=70, n_seq=40, G=1, lens=(190, 3, 0, 129), P=64, order="repeats", shared=True),
    dict(H=16, T=64, n_seq=2, G=2, lens=(3000, 2500), P=1, order="shuffled", causal=True, q_gain=20.0),
    dict(H=1, T=1500, n_seq=1, G=3, lens=(2000,), P=3, dense=True, causal=True),
    dict(H=12, T=260, lens=(1600,), q_gain=60.0, order="shuffled"),
    dict(H=12, T=260, lens=(1600,), q_gain=1e-3),
], ids=str)
def test_attend_wide_windows(qsa, kw):
    Call(qsa, Attend(seed=50, q_dtype="bf16", **kw), "bf16").check()


def test_attend_wide_window_rows_of_their_own(qsa):
    """Limits in any order; what unseen cells hold, and rows that are not finite, stay where they are."""
    c = Attend(seed=51, dense=True, causal=True, **{**WIDE, "lens": (4097,)})
    rng = np.random.default_rng(52)
    c.q_limit[0] = rng.integers(0, 4098, c.T)
    c.q_limit[0, :4] = 4097, 0, 1, 3000
    Call(qsa, c, "bf16").check()
    clean = c.reference()[0]
    c.q_limit[0] = np.minimum(c.q_limit[0], 4000)
    c.q_limit[0, 0] = 4097
    c.kv_scale[0, :, c.page_table[0, 4000:]] = (np.nan, np.inf, np.inf, np.nan)
    c.q[0, 7, 3, 5], c.q[0, 8, 11, 0] = np.nan, np.inf
    got = Call(qsa, c, "bf16")().float().cpu().numpy()
    assert not np.isfinite(got[0, 0]).any()  # the row that sees them
    assert not np.isfinite(got[0, 7, 3]).any() and not np.isfinite(got[0, 8, 11]).any()
    assert not got[0, 1].any()
    rows = np.ones((c.T, 12), bool)
    rows[0] = rows[7, 3] = rows[8, 11] = False
    rows &= (c.q_limit[0] < 4000)[:, None]
    assert rows.sum() > 1000
    assert np.linalg.norm(got[0][rows] - clean[0][rows]) <= 2.0 ** -8 * np.linalg.norm(clean[0][rows])


def test_attend_wide_window_scores_that_rise(qsa):
    """Every tile outgrows the last one's reference, then none does; V scales from 2^-20 to 2^20."""
    c = Attend(seed=53, **{**WIDE, "T": 60, "lens": (8300,)})
    at = c.page_table[0, c.sel]
    n = len(at)
    c.kv_scale[0, :, at, 0] *= np.linspace(1, 60, n, dtype=np.float32)[:, None]
    c.kv_scale[0, :, at, 1] = -7.5 * c.kv_scale[0, :, at, 0]
    Call(qsa, c, "bf16").check("rise")
    c.sel = c.sel[::-1].copy()
    Call(qsa, c, "bf16").check("fall")
    c.kv_scale[0, :, at, 2:] *= np.exp2(np.random.default_rng(54).integers(-20, 21, n)).astype(np.float32)[:, None, None]
    Call(qsa, c, "bf16").check("V scales")


def test_attend_wide_window_repeats_bitwise(qsa):
    """On another stream, from a dirty workspace, in a graph that serves fewer cells."""
    c = Attend(seed=55, n_seq=2, P=8, dense=True, causal=True, **{**WIDE, "lens": (4100, 3000)})
    call = Call(qsa, c, "bf16")
    first = call().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side):
        call.ws.fill_(170)
        call.out.fill_(9)
        torch.cuda.synchronize()
        call(stream)
        torch.cuda.synchronize()
        assert torch.equal(call.out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(torch.cuda.current_stream())
    for lens in ((900, 4100), (0, 129), (0, 0)):
        d = Attend(seed=56, n_seq=2, P=8, dense=True, causal=True, context=4100, **{**WIDE, "lens": lens})
        c.offsets, c.q_limit, c.q = d.offsets, d.q_limit, d.q
        for x, y in ((call.offsets, c.offsets), (call.limit, c.q_limit), (call.q, c.q)):
            x.copy_(dev(y))
        g.replay()
        torch.cuda.synchronize()
        assert_attend(call.out.float().cpu().numpy(), c, True, str(lens))


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kw", [dict(H=12, T=100, lens=(4100,)), dict(lens=(300,)), dict(lens=(2000,), T=4), dict(n_seq=9, G=2, T=3, lens=(1500, 80))], ids=str)
def test_attend_output_is_the_next_query(qsa, t, kw):
    """Calls in a row, each reading what the one before wrote: eagerly one at a time, then with nothing between."""
    c = Attend(seed=35, q_dtype=t, q_gain=20.0, **kw)
    call = Call(qsa, c, t)
    n = 12
    x = [call.q.clone()] + [torch.empty_like(call.q) for _ in range(n)]

    def steps(wait):
        for i in range(n):
            call.q, call.out = x[i], x[i + 1]
            call()
            if wait:
                torch.cuda.synchronize()
    steps(True)
    want = [y.clone() for y in x]
    assert torch.isfinite(want[-1]).all() and not torch.equal(want[-1], want[-2])

    def check():
        torch.cuda.synchronize()
        for y, w in zip(x, want):
            assert torch.equal(y, w)
    for _ in range(5):
        for y in x[1:]:
            y.fill_(1)
        steps(False)
        check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        steps(False)
    for _ in range(5):
        for y in x[1:]:
            y.fill_(1)
        g.replay()
        check()


@pytest.mark.parametrize("what", ["table", "sel", "offsets", "limit"])
@pytest.mark.parametrize("kw,t", [(dict(H=12, lens=(300,)), "f32"), (dict(H=12, T=100, lens=(4100,)), "bf16")], ids=str)
def test_attend_output_is_another_input_of_the_next(qsa, what, kw, t):
    """A call whose rows see nothing writes zeros over the table, list, offsets or limits that the next call,
    launched right behind it, reads."""
    first = Attend(seed=72, H=20, lens=(12800,), P=64, dense=True, causal=True)
    first.q_limit[:] = 0
    c = Attend(seed=73, q_dtype=t, causal=True, context=5000, **kw)
    name = dict(table="page_table", sel="sel", offsets="offsets", limit="q_limit")[what]
    old = getattr(c, name)
    a, b = Call(qsa, first, "f32"), Call(qsa, c, t)
    assert old.size <= a.out.numel()
    a.out = torch.empty(a.out.numel(), dtype=torch.int32, device="cuda")
    buf = a.out[:old.size].view(old.shape)
    setattr(b, what, buf)
    setattr(c, name, np.zeros_like(old))
    data = dev(old)
    b.out.fill_(3)
    for _ in range(10):
        buf.copy_(data)
        a()
        b.check(what)


@pytest.mark.parametrize("kw,t", [(dict(lens=(600,)), "f32"), (dict(n_seq=16, G=2, T=4, lens=(2000, 100, 700)), "bf16"),
                                  (dict(H=12, T=100, lens=(4100,)), "bf16")], ids=str)
def test_attend_behind_ordinary_kernels(qsa, kw, t):
    """Each input in turn written by a framework's kernel right before the call."""
    calls = [Call(qsa, Attend(seed=74 + i, q_dtype=t, P=4, causal=True, context=4500, **kw), t) for i in range(2)]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    names = ["sel", "offsets", "table", "limit", "q", "scale", "pool"]
    got = Call(qsa, calls[0].c, t)
    for last in range(len(names)):
        for i in range(12):
            for n in names[last + 1:] + names[:last + 1]:
                torch.add(getattr(calls[i & 1], n), 0, out=getattr(got, n))
            got()
            assert torch.equal(got.out, want[i & 1]), names[last]


def test_attend_behind_the_append_at_once(qsa):
    """Cells appended right before they are attended to, over and over into the same slots."""
    c = Attend(seed=76, lens=(256,), P=1, dense=True)
    call = Call(qsa, c, "f32")
    rng = np.random.default_rng(77)
    pos = dev(np.arange(256, dtype=np.int32)[None])
    rows = [[dev(rng.standard_normal((1, 256, 1, 256)).astype(np.float32)) for _ in "kv"] for _ in range(2)]

    def step(i):
        qsa.qsa_kv4_append(call.shape, 1, 1, 256, qsa.QSA_F32, *rows[i], pos, call.table, call.pool, call.scale)
    want = []
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        want.append(call().clone())
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    outs = [torch.empty_like(call.out) for _ in range(60)]
    for i, o in enumerate(outs):
        step(i & 1)
        call.out = o
        call()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i & 1])


def test_attend_fewer_cells_than_the_workspace_was_sized_for(qsa):
    """A workspace of the largest bound serves every smaller one."""
    big = Attend(seed=36, n_seq=3, T=4, lens=(4000,))
    ws = Call(qsa, big, "f32").ws
    for n in (0, 1, 130, 700, 1800, 3999):
        call = Call(qsa, Attend(seed=37, n_seq=3, T=4, lens=(n, n // 2, n)), "f32")
        call.ws = ws
        call.check(str(n))


@pytest.mark.parametrize("kw,t", [(dict(lens=(600,)), "f32"), (dict(n_seq=6, G=2, T=4, lens=(2000, 100)), "f32"),
                                  (dict(n_seq=20, G=2, H=8, lens=(2000,)), "bf16"),
                                  (dict(H=12, T=100, lens=(4100,)), "bf16")], ids=str)
def test_attend_times_out_and_recovers(qsa, kw, t):
    """A correct call whose waits are bounded by 16 clock cycles ends, says so, and the next one is right."""
    call = Call(qsa, Attend(seed=38, q_dtype=t, **kw), t)
    call.check()
    qsa.qsa_set_wait_limit(16)
    try:
        call()
    finally:
        qsa.qsa_set_wait_limit(0)
    torch.cuda.synchronize()
    assert int(call.status.item()) == qsa.QSA_STATUS_TIMEOUT
    call.status.zero_()
    call.out.fill_(3)
    call.check()


TIMED = [(dict(lens=(600,)), "f32"), (dict(n_seq=6, G=2, T=4, lens=(2000, 100)), "f32"),
         (dict(n_seq=20, G=2, H=8, lens=(2000,)), "bf16"), (dict(n_seq=9, G=2, T=3, lens=(1500, 80)), "bf16"),
         (dict(H=12, T=100, lens=(4100,)), "bf16")]


@pytest.mark.parametrize("kw,t", TIMED, ids=str)
def test_attend_times_out_behind_other_kernels(qsa, kw, t):
    """A call whose waits all run out reads rows of the pool alone, whatever other kernels left in shared memory:
    a wide window's operands, small blocks' codes, scores of fp32 windows."""
    before = [Call(qsa, Attend(seed=70 + i, q_dtype=u, **k), u) for i, (k, u) in enumerate(TIMED)]
    call = Call(qsa, Attend(seed=39, q_dtype=t, **kw), t)
    want = call().clone()
    pool, scale = call.pool.clone(), call.scale.clone()
    for other in before:
        qsa.qsa_set_wait_limit(0)
        other()
        qsa.qsa_set_wait_limit(16)
        try:
            call()
        finally:
            qsa.qsa_set_wait_limit(0)
        torch.cuda.synchronize()
        assert int(call.status.item()) == qsa.QSA_STATUS_TIMEOUT
        call.status.zero_()
    assert torch.equal(call.pool, pool) and torch.equal(call.scale, scale)
    call.out.fill_(3)
    assert torch.equal(call(), want)


@pytest.mark.parametrize("H", [1, 2, 12, 24, 32])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_attend_long_sums(qsa, H, t):
    """8,192 cells a row and multiprocessor.  The tensor cores round their sums towards zero: a step of 16
    cells loses up to 2^-23 of the sum so far, half of that on average, and sums of 1,024 cells (64 steps)
    are added up to nearest; a sum that grows from zero loses half of 64 * 2^-24, 1.9e-6, and what the scores
    and exponentials lose (2^-21 each, of random sign) is below 1e-6 in quadrature.  bf16 outputs: their
    rounding, 2^-8 at most."""
    G, n = 76, 16384
    g = torch.Generator(device="cuda").manual_seed(60 + H)
    pool = torch.randint(0, 256, (1, G, n, 256), generator=g, dtype=torch.uint8, device="cuda")
    r = torch.rand(1, G, n, 4, generator=g, device="cuda")
    scale = torch.empty_like(r)
    scale[..., 0::2] = 0.15 + 0.15 * r[..., 0::2]
    scale[..., 1::2] = -7.5 * scale[..., 0::2] + 0.6 * (r[..., 1::2] - 0.5)
    dt, code = (torch.float32, qsa.QSA_F32) if t == "f32" else (torch.bfloat16, qsa.QSA_BF16)
    q = torch.randn(1, 1, G * H, 256, generator=g, device="cuda").to(dt)
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda")[None]
    shape = qsa.make_shape(n_kv_heads=G, q_per_kv=H, n_queries=1, pool_cells=n, page_table_len=n // 64, chunk_cells=1,
                           softmax_scale=1 / 16, q_dtype=code, page_cells=64)
    ws = torch.empty(qsa.qsa_kv4_attn_workspace_bytes(shape, 1, n), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    qsa.qsa_kv4_attn_batch(shape, 1, 1, q, pool, scale, table, None, dev(np.array([0, n], np.int32)), n, None, code, out, ws, ws.numel())
    err = norm = 0.0
    for h in range(G):
        u = torch.stack([pool[0, h] & 15, pool[0, h] >> 4], -1).flatten(-2).double()
        f = scale[0, h].double()
        k, v = u[:, :256] * f[:, 0:1] + f[:, 1:2], u[:, 256:] * f[:, 2:3] + f[:, 3:4]
        ref = torch.softmax(q[0, 0, h * H:(h + 1) * H].double() @ k.T / 16, -1) @ v
        err += float((out[0, 0, h * H:(h + 1) * H].double() - ref).square().sum())
        norm += float(ref.square().sum())
    assert (err / norm) ** 0.5 <= (3e-6 if t == "f32" else 2.0 ** -8)


@pytest.mark.parametrize("kw,t", [(dict(n_seq=3, G=2, lens=(600, 0, 77)), "f32"), (dict(n_seq=2, H=12, T=8, lens=(900, 5)), "bf16"),
                                  (dict(n_seq=40, lens=(300, 2), T=2), "f32")], ids=str)
def test_attend_short_lists_under_the_largest_bound(qsa, kw, t):
    """max_selected at its limit (and so the work list in 64 bits): short lists as ever."""
    c = Attend(seed=82, q_dtype=t, **kw)
    c.max_selected = 2 ** 31 - 1 - 1024
    Call(qsa, c, t).check()


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_attend_as_many_sequences_as_there_can_be(qsa, t):
    """65,535 contexts of no or one cell: zeros, or that cell's values."""
    B = 65535
    dt, code = (torch.float32, qsa.QSA_F32) if t == "f32" else (torch.bfloat16, qsa.QSA_BF16)
    g = torch.Generator(device="cuda").manual_seed(83)
    pool = torch.randint(0, 256, (1, 1, B, 256), generator=g, dtype=torch.uint8, device="cuda")
    scale = torch.rand(1, 1, B, 4, generator=g, device="cuda") + 0.1
    q = torch.randn(B, 1, 3, 256, generator=g, device="cuda").to(dt)
    table = torch.randperm(B, generator=g, device="cuda").int()[:, None].contiguous()
    one = torch.rand(B, generator=g, device="cuda") < 0.7
    offsets = torch.cat([torch.zeros(1, device="cuda"), one.cumsum(0)]).int()
    shape = qsa.make_shape(n_kv_heads=1, q_per_kv=3, n_queries=1, pool_cells=B, page_table_len=1, chunk_cells=1, softmax_scale=1 / 16,
                           q_dtype=code)
    ws = torch.empty(qsa.qsa_kv4_attn_workspace_bytes(shape, B, 1), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 3.0)
    qsa.qsa_kv4_attn_batch(shape, B, 1, q, pool, scale, table, None, offsets, 1, None, code, out, ws, ws.numel())
    f = scale[0, 0, table[:, 0].long()].double()
    v = pool[0, 0, table[:, 0].long(), 128:]
    want = torch.stack([v & 15, v >> 4], -1).flatten(-2).double() * f[:, 2:3] + f[:, 3:4]
    assert not out[~one].any()
    # one weight of 1: P' (2^-22, or 2^-11 of a code's part) and the output's rounding
    err = (out[one].double() - want[one][:, None, None]).abs()
    part = (7.5 * f[one][:, 2:3])[:, None, None]
    eps = 2.0 ** -20 * (want[one][:, None, None].abs() + part) if t == "f32" else 2.0 ** -11 * part + 2.0 ** -8 * (want[one][:, None, None] + part * 2.0 ** -11)
    assert bool((err <= eps + 2.0 ** -20 * part).all())


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_attend_widest_window(qsa, t):
    """65,536 queries of 64 heads: 2^22 rows, their offsets past 2^31 bytes, over five cells with limits of their own."""
    H, T, n = 64, 65536, 5
    dt, code = (torch.float32, qsa.QSA_F32) if t == "f32" else (torch.bfloat16, qsa.QSA_BF16)
    g = torch.Generator(device="cuda").manual_seed(84)
    pool = torch.randint(0, 256, (1, 1, n, 256), generator=g, dtype=torch.uint8, device="cuda")
    r = torch.rand(1, 1, n, 4, generator=g, device="cuda")
    scale = torch.empty_like(r)
    scale[..., 0::2] = 0.05 + 0.3 * r[..., 0::2]
    scale[..., 1::2] = -7.5 * scale[..., 0::2] + r[..., 1::2] - 0.5
    q = torch.randn(1, T, H, 256, generator=g, device="cuda").to(dt)
    limit = torch.randint(0, n + 1, (1, T), generator=g, device="cuda").int()
    table = torch.arange(n, device="cuda").int()[None].contiguous()
    shape = qsa.make_shape(n_kv_heads=1, q_per_kv=H, n_queries=T, pool_cells=n, page_table_len=n, chunk_cells=1, softmax_scale=1 / 16,
                           q_dtype=code)
    ws = torch.empty(qsa.qsa_kv4_attn_workspace_bytes(shape, 1, n), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 3.0)
    qsa.qsa_kv4_attn_batch(shape, 1, 1, q, pool, scale, table, None, dev(np.array([0, n], np.int32)), n, limit, code, out, ws, ws.numel())
    u = torch.stack([pool[0, 0] & 15, pool[0, 0] >> 4], -1).flatten(-2).double()
    f = scale[0, 0].double()
    k, v = u[:, :256] * f[:, 0:1] + f[:, 1:2], u[:, 256:] * f[:, 2:3] + f[:, 3:4]
    for t0 in range(0, T, 4096):
        x = q[0, t0:t0 + 4096].double() @ k.T / 16
        seen = torch.arange(n, device="cuda") < limit[0, t0:t0 + 4096, None, None]
        w = torch.where(seen, (x - x.masked_fill(~seen, -1e300).amax(-1, keepdim=True)).exp(), torch.zeros_like(x))
        ref = torch.nan_to_num(w / w.sum(-1, keepdim=True)) @ v
        got = out[0, t0:t0 + 4096].double()
        assert not got[limit[0, t0:t0 + 4096] == 0].any()
        err = (got - ref).norm(dim=-1) / ref.norm(dim=-1).clamp_min(1e-30)  # by row: no row in another's place
        assert float(err.max()) <= (2e-5 if t == "f32" else 2.0 ** -8), t0


def test_attend_cells_past_32_bit_offsets(qsa):
    """Slots whose rows lie past 2^32 bytes of the pool."""
    cells = 18_000_000
    pool = torch.empty((1, 1, cells, 256), dtype=torch.uint8, device="cuda")
    scale = torch.empty((1, 1, cells, 4), device="cuda")
    c = Attend(seed=23, lens=(500,), T=2)
    rng = np.random.default_rng(24)
    far = np.sort(rng.permutation(cells - 16_900_000)[:c.table_len] + 16_900_000).astype(np.int32)
    near = c.page_table[0].copy()
    pool[0, 0, dev(far).long()] = dev(c.kv_pool[0, 0, near])
    scale[0, 0, dev(far).long()] = dev(c.kv_scale[0, 0, near])
    want = Call(qsa, c, "f32")
    ref = want().clone()
    want.pool, want.scale, want.table = pool, scale, dev(far[None])
    want.shape.pool_cells = cells
    assert torch.equal(want(), ref)
    rows = Rows(25, 1, 1, 40, 1, False, "f32", spoil=False)
    rows.table = far[None, :rows.L].copy()
    shape = rows.shape(qsa)
    shape.pool_cells = cells
    qsa.qsa_kv4_append(shape, 1, 1, 40, qsa.QSA_F32, dev(rows.k), dev(rows.v), dev(rows.pos), dev(rows.table), pool, scale)
    for i, pos in enumerate(rows.pos[0]):
        if pos >= 0:
            u, s, z = kv4.quantise(rows.v[0, i, 0])
            assert np.array_equal(pool[0, 0, int(far[pos]), 128:].cpu().numpy(), kv4.pack(u))
            assert scale[0, 0, int(far[pos])].cpu().numpy()[2:].tolist() == [s, z]


# ------------------------------------------------------------------------ pages

PAGE_OUT = ("out_len", "len_offsets", "positions", "slots", "q_limit")


def gpu_page_map(qsa, c, cur, new, state):
    B, L = c["page_table"].shape
    if "out_len" not in state:
        state["out_len"] = torch.full((B,), 77, dtype=torch.int32, device="cuda")
        state["len_offsets"] = torch.full((B + 1,), 77, dtype=torch.int32, device="cuda")
        for n in PAGE_OUT[2:]:
            state[n] = torch.full((B, c["max_new"]), 77, dtype=torch.int32, device="cuda")
        state["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    qsa.qsa_page_map(B, c["free_pages"].shape[0], c["max_new"], c["page_cells"], L, c["pool_pages"], cur, new,
                     state["page_table"], state["free_pages"], state["free_count"],
                     *[state[n] if state[n].numel() else None for n in PAGE_OUT], state["status"])


def check_pages(qsa, c):
    state = {n: dev(c[n]) for n in ("page_table", "free_pages", "free_count")}
    gpu_page_map(qsa, c, dev(c["cur_len"]), dev(c["new_len"]), state)
    want = pm.page_map(c["cur_len"], c["new_len"], c["page_table"], c["free_pages"], c["free_count"], c["max_new"],
                       c["page_cells"], c["pool_pages"])
    for n, w in zip(PAGE_OUT, want):
        got = state[n].cpu().numpy()
        assert np.array_equal(got, w), f"{n}: {np.argwhere(got != w)[:4].tolist()}"
    assert np.array_equal(state["page_table"].cpu().numpy(), c["page_table"])
    count = state["free_count"].cpu().numpy()
    assert np.array_equal(count, c["free_count"])
    for i, k in enumerate(count):
        assert np.array_equal(state["free_pages"][i, :k].cpu().numpy(), c["free_pages"][i, :k])
    assert int(state["status"].item()) == want[5]
    return want


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("n_seq,max_new,P,L,spare,grow,holes", [
    (1, 1, 1, 40, 9, 1, 0), (16, 4, 16, 50, 30, 1, 0), (7, 0, 4, 9, 3, None, 0), (33, 50, 3, 31, 200, None, 0),
    (300, 300, 16, 40, 500, None, 0.1), (1025, 5, 2, 8, 4000, None, 0.2), (2500, 3, 1, 6, 20000, None, 0),
    (64, 2000, 64, 64, 4000, 1, 0), (200, 40, 8, 20, 25, 1, 0), (5, 900, 1, 3000, 2, None, 0.3), (3, 10, 7, 1, 5, None, 0),
])
def test_page_map(qsa, shared, n_seq, max_new, P, L, spare, grow, holes):
    check_pages(qsa, draw_pages(n_seq + max_new, n_seq, max_new, P, L, shared, spare, grow, holes))


@pytest.mark.parametrize("shared", [True, False])
def test_page_map_bad_inputs(qsa, shared):
    c = draw_pages(3, 40, 30, 4, 20, shared, 60)
    c["cur_len"][[1, 5, 9]] = -3, 81, 40
    c["new_len"][[2, 9, 11]] = 500, 75, -1
    c["page_table"][7, :3] = c["pool_pages"], -5, 2 ** 30
    c["cur_len"][7], c["new_len"][7] = 12, 0
    want = check_pages(qsa, c)
    assert want[5] & pm.STATUS_BAD_EXTENT and want[5] & pm.STATUS_BAD_SLOT
    # a stack too full for what is freed, and counts outside it
    c = draw_pages(4, 6, 5, 2, 10, shared, 0)
    c["new_len"][:] = 0
    c["free_count"][:] = c["pool_pages"] - 1
    c["free_pages"][:] = 0
    check_pages(qsa, c)
    for count in (-4, 10 ** 6):
        c = draw_pages(5, 6, 5, 2, 10, shared, 4, 1)
        c["free_pages"][:] = 1
        c["free_count"][:] = count
        check_pages(qsa, c)


@pytest.mark.parametrize("shared", [True, False])
def test_page_map_roll_back_and_grow(qsa, shared):
    """A window rolled back and grown again gives the same tables, stack and maps; captured too."""
    c = draw_pages(6, 50, 400, 16, 60, shared, 3000, 1)
    old, new = dev(c["cur_len"]), dev(np.minimum(c["new_len"], 60 * 16))
    state = {n: dev(c[n]) for n in ("page_table", "free_pages", "free_count")}
    gpu_page_map(qsa, c, old, new, state)
    first = {n: t.clone() for n, t in state.items()}

    def turn():
        gpu_page_map(qsa, c, new, old, state)
        gpu_page_map(qsa, c, old, new, state)
    turn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        turn()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for n, t in state.items():
        if n == "free_pages":
            for i, k in enumerate(state["free_count"].tolist()):
                assert torch.equal(t[i, :k], first[n][i, :k])
        else:
            assert torch.equal(t, first[n]), n
    assert not state["status"].any()


@pytest.mark.parametrize("max_new", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 - 2 ** 20 + 3])
def test_page_map_widest_maps(qsa, max_new):
    """Maps near the largest width: the stride behind the last token passes 2^31."""
    P, L, cur, new = 64, 1 << 22, 5, 200_000_007
    table = torch.full((1, L), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    pages = L
    free = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    count = dev(np.array([pages - 1], np.int32))
    out_len, offsets, status = (torch.full((k,), v, dtype=torch.int32, device="cuda") for k, v in ((1, 7), (2, 7), (1, 0)))
    guard = 4096
    maps = [torch.full((max_new + guard,), 77, dtype=torch.int32, device="cuda") for _ in range(3)]
    qsa.qsa_page_map(1, 1, max_new, P, L, pages, dev(np.array([cur], np.int32)), dev(np.array([new], np.int32)), table, free,
                     count, out_len, offsets, *maps, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and int(out_len.item()) == new
    n = new - cur
    want = torch.arange(cur, new, dtype=torch.int32, device="cuda")
    assert torch.equal(maps[0][:n], want) and torch.equal(maps[2][:n], want + 1)
    assert torch.equal(maps[1][:n], want)  # pages taken in order: 1, 2, ...
    for m, fill in zip(maps, (-1, -1, 0)):
        for part in m[n:max_new].split(1 << 28):
            assert bool((part == fill).all())
        assert bool((m[max_new:] == 77).all())


@pytest.mark.parametrize("max_new", [8, 300])
def test_page_map_then_attention_at_once(qsa, max_new):
    """The attention launched right behind the page map reads the tables and offsets that it has written."""
    B, P, L = 16, 16, 40
    c = draw_pages(8, B, max_new, P, L, True, 3000, 1)
    old = np.maximum(c["cur_len"], 200)
    c["cur_len"][:] = 0
    c["page_table"][:] = -1
    pages = c["pool_pages"]
    a = Attend(seed=9, n_seq=B, lens=(64,), P=P, dense=True)
    pool, scale = (torch.from_numpy(x).cuda() for x in (
        np.random.default_rng(1).integers(0, 256, (1, 1, pages * P, 256), dtype=np.uint8),
        np.random.default_rng(2).uniform(0.1, 0.2, (1, 1, pages * P, 4)).astype(np.float32)))
    shape = qsa.make_shape(n_kv_heads=1, q_per_kv=12, n_queries=1, pool_cells=pages * P, page_table_len=L, chunk_cells=1,
                           softmax_scale=1 / 16, page_cells=P)
    q, ws = dev(a.q), torch.empty(qsa.qsa_kv4_attn_workspace_bytes(shape, B, L * P), dtype=torch.uint8, device="cuda")
    zero = dev(np.zeros(B, np.int32))
    lens = [dev(np.minimum(old * 0 + n, max_new).astype(np.int32)) for n in (3, 8, 1, 5)]

    def run(state, wait):
        out, cur = [], zero
        for new in lens + [zero]:
            gpu_page_map(qsa, c, cur, new, state)
            if wait:
                torch.cuda.synchronize()
            o = torch.empty((B, 1, 12, 256), device="cuda")
            qsa.qsa_kv4_attn_batch(shape, B, 1, q, pool, scale, state["page_table"], None, state["len_offsets"], L * P, None,
                                   qsa.QSA_F32, o, ws, ws.numel(), state["status"])
            if wait:
                torch.cuda.synchronize()
            out.append(o)
            cur = new
        torch.cuda.synchronize()
        return out
    fresh = lambda: dict(page_table=dev(c["page_table"]), free_pages=dev(np.arange(pages, dtype=np.int32)[None]),  # noqa: E731
                         free_count=dev(np.array([pages], np.int32)))
    want = run(fresh(), True)
    assert want[0].any() and not want[-1].any()
    for _ in range(10):
        for x, w in zip(run(fresh(), False), want):
            assert torch.equal(x, w)


# --------------------------------------------------------------- a run of them

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_serving_steps(qsa, dtype):
    """Steps of a server over one shared pool: lengths to pages and maps, the new rows appended through
    them, the window's causal attention over the whole contexts; a draft rolled back, a request finished."""
    rng = np.random.default_rng(40)
    B, G, H, P, L, window = 5, 2, 4, 16, 24, 37
    pool_pages = B * L - 20
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    code = qsa.QSA_F32 if dtype == "f32" else qsa.QSA_BF16
    state = dict(page_table=torch.full((B, L), -1, dtype=torch.int32, device="cuda"),
                 free_pages=dev(rng.permutation(pool_pages).astype(np.int32)[None]),
                 free_count=dev(np.array([pool_pages], np.int32)))
    c = dict(page_table=np.empty((B, L)), free_pages=np.empty((1, pool_pages)), max_new=window, page_cells=P, pool_pages=pool_pages)
    shape = qsa.make_shape(n_kv_heads=G, q_per_kv=H, n_queries=window, pool_cells=pool_pages * P, page_table_len=L,
                           chunk_cells=1, softmax_scale=1 / 16, q_dtype=code, page_cells=P)
    pool = torch.zeros((1, G, pool_pages * P, 256), dtype=torch.uint8, device="cuda")
    scale = torch.full((1, G, pool_pages * P, 4), float("nan"), device="cuda")
    ws = torch.empty(qsa.qsa_kv4_attn_workspace_bytes(shape, B, L * P), dtype=torch.uint8, device="cuda")
    past = [[np.zeros((0, G, 256)) for _ in "kv"] for _ in range(B)]  # what the cells stand for
    cur = np.zeros(B, np.int32)
    for step, add in enumerate(([37, 20, 1, 0, 33], [4, 4, 4, 37, 4], [-3, -2, 1, -4, 4], [4, -22, 4, 4, 3], [37] * B)):
        new = cur + np.array(add, np.int32)
        gpu_page_map(qsa, c, dev(cur), dev(new), state)
        k, v = (torch.from_numpy(rng.standard_normal((B, window, G, 256)).astype(np.float32)).cuda().to(t) for _ in "kv")
        q = torch.from_numpy(rng.standard_normal((B, window, G * H, 256)).astype(np.float32)).cuda().to(t)
        qsa.qsa_kv4_append(shape, B, 1, window, code, k, v, state["positions"], state["page_table"], pool, scale, state["status"])
        out = torch.empty_like(q)
        qsa.qsa_kv4_attn_batch(shape, B, 1, q, pool, scale, state["page_table"], None, state["len_offsets"], L * P,
                               state["q_limit"], code, out, ws, ws.numel(), state["status"])
        torch.cuda.synchronize()
        assert int(state["status"].item()) == 0 and state["out_len"].tolist() == new.tolist()
        got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
        ref = np.zeros_like(got)
        for b in range(B):
            rows = []
            for old, x in zip(past[b], (k, v)):
                u, s, z = kv4.quantise(x[b, :max(0, add[b])].float().cpu().numpy())
                y = u * s[..., None].astype(np.float64) + z[..., None]
                rows.append(np.concatenate([old[:min(cur[b], new[b])], y]))
            past[b] = rows
            assert len(rows[0]) == new[b]
            for i in range(max(0, add[b])):
                for h in range(G * H):
                    s = rows[0][:cur[b] + i + 1, h // H] @ qd[b, i, h] / 16
                    w = np.exp(s - s.max())
                    ref[b, i, h] = w @ rows[1][:cur[b] + i + 1, h // H] / w.sum()
        assert np.linalg.norm(got - ref) <= (2e-5 if dtype == "f32" else 2.0 ** -8) * np.linalg.norm(ref), step
        assert not got[ref == 0].any()
        cur = new
