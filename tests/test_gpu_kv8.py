"""8-bit cache on the GPU against the float64 oracle: write, append, decode, selection, sparse decode, fork, compaction.

Tolerances: what a write stores is compared bit for bit.  A float32 output may differ from the float64 one by the bound
that oracle.kv8.attend_bound derives; a BF16 output by that plus half a BF16 step (2^-8 of the value) of rounding.
"""
import numpy as np
import pytest

from oracle import kv8 as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {0: torch.float32, 1: torch.bfloat16}


@pytest.fixture(scope="module")
def osc():
    from int2_rotated_paged_oscar_gb300 import build
    build.build()
    import int2_rotated_paged_oscar_gb300 as m
    m.load()
    return m


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


class Rig:
    """One context with a bound 8-bit cache on the GPU and the oracle's image of one of its layers."""

    def __init__(self, osc, fmt=O.INT8, P=16, d=64, heads=2, G=2, layers=2, layer=1, slots=5, per_req=12, pages=48, int2=False,
                 oracle=True):
        self.osc, self.P, self.d, self.heads, self.G, self.layer, self.fmt = osc, P, d, heads, G, layer, fmt
        self.cfg = osc.make_config(num_layers=layers, n_q_heads=heads * G, n_kv_heads=heads, head_dim=d, page_size=P, sink=4,
                                   recent=16, max_requests=slots, max_pages_per_req=per_req, num_pages=pages)
        self.block = osc.oscar_kv8_block_bytes(self.cfg)
        self.pool = torch.full((layers, pages, heads, self.block), 0xA5, dtype=torch.uint8, device="cuda")
        self.tail = torch.full((layers, slots, heads, 2, P, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.int2 = None
        if int2:
            self.int2 = torch.randint(0, 256, (osc.oscar_int2_pool_bytes(self.cfg),), dtype=torch.uint8, device="cuda")
            self.slab = torch.zeros(osc.oscar_window_slab_bytes(self.cfg), dtype=torch.uint8, device="cuda")
            self.ctx = osc.oscar_create(self.cfg, self.int2, self.slab)
        else:
            self.ctx = osc.oscar_create(self.cfg)
        osc.oscar_kv8_bind(self.ctx, fmt, self.pool, self.tail)
        if oracle:
            self.ref = O.Cache(P, d, heads, fmt, self.pool[layer].cpu().numpy().copy(),
                               self.tail[layer].double().cpu().numpy().copy())

    def __enter__(self):
        return self

    def __exit__(self, *a):
        torch.cuda.synchronize()
        self.osc.oscar_destroy(self.ctx)

    def status(self):
        return self.osc.oscar_check_status(self.ctx)

    def rows(self, x, dtype, gap=0):
        t = torch.from_numpy(np.asarray(x, np.float32)).to(DT[dtype]).cuda()
        if gap:
            wide = torch.full((t.shape[0], t.shape[1] * t.shape[2] + gap), 7.0, dtype=t.dtype, device="cuda")
            wide[:, :t[0].numel()] = t.reshape(t.shape[0], -1)
            return wide[:, :t[0].numel()].unflatten(1, t.shape[1:])
        return t

    def write(self, K, V, dtype, lens, starts, bt, slots, gap=0, ref=True):
        """K, V: one array of [tokens][heads][d] per request."""
        cu = np.concatenate([[0], np.cumsum(lens)])
        k, v = (self.rows(np.concatenate(x), dtype, gap) for x in (K, V))
        bt_d = dev(bt)
        self.osc.oscar_kv8_write(self.ctx, self.layer, k, v, dtype, dev(cu), dev(starts), len(lens), int(cu[-1]), bt_d,
                                 bt_d.shape[1], dev(slots))
        if ref:
            for b in range(len(lens)):
                self.ref.write(bt[b], slots[b], starts[b], bf16(K[b]), bf16(V[b]))

    def append(self, K, V, dtype, lens, bt, slots, gap=0):
        bt_d = dev(bt)
        self.osc.oscar_kv8_append(self.ctx, self.layer, self.rows(K, dtype, gap), self.rows(V, dtype, gap), dtype, dev(lens),
                                  len(lens), bt_d, bt_d.shape[1], dev(slots))
        for b in range(len(lens)):
            self.ref.write(bt[b], slots[b], lens[b], bf16(K[b:b + 1]), bf16(V[b:b + 1]), append=True)

    def same(self):
        """The layer's pool and tail equal the oracle's, bit for bit, and the other layers are as they were."""
        got = self.pool.cpu().numpy()
        assert np.array_equal(got[self.layer], self.ref.pool)
        assert np.array_equal(self.tail[self.layer].double().cpu().numpy(), self.ref.tail, equal_nan=True)
        for i in range(got.shape[0]):
            if i != self.layer:
                assert np.all(got[i] == 0xA5) and torch.isnan(self.tail[i]).all()

    def decode(self, q, qd, od, bt, lens, slots, max_seq=None, pages=None, stream=None, gap=0, ws=None):
        B, o = len(lens), self.osc
        max_seq = max(lens) if max_seq is None else max_seq
        qt = self.rows(q, qd, gap)
        out = torch.full((B + 1, self.heads * self.G, self.d), 123.0, dtype=DT[od], device="cuda")
        bt_d = bt if torch.is_tensor(bt) else dev(bt)
        n, sl = dev(lens), dev(slots)
        if pages is None:
            size = o.oscar_kv8_decode_workspace_size(self.cfg, B, max_seq)
            ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
            o.oscar_kv8_decode_attn(self.ctx, self.layer, qt, qd, out, od, bt_d, bt_d.shape[1], n, sl, B, max_seq, ws, size, stream)
        else:
            idx = pages if torch.is_tensor(pages) else dev(pages)
            size = o.oscar_kv8_sparse_workspace_size(self.cfg, B, idx.shape[2])
            ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
            o.oscar_kv8_sparse_decode_attn(self.ctx, self.layer, qt, qd, out, od, idx, idx.shape[2], bt_d, bt_d.shape[1], n, sl, B,
                                           ws, size, stream)
        assert torch.all(out[B] == 123.0)         # rows behind the last request stay as they are
        return out[:B]

    def select(self, q, qd, bt, lens, first, last, k, max_seq=None, gap=0):
        B, o = len(lens), self.osc
        max_seq = max(lens) if max_seq is None else max_seq
        idx = torch.full((B + 1, self.heads, k), -7, dtype=torch.int32, device="cuda")
        size = o.oscar_kv8_select_workspace_size(self.cfg, B, max_seq)
        ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device="cuda")
        bt_d = dev(bt)
        o.oscar_kv8_select_pages(self.ctx, self.layer, self.rows(q, qd, gap), qd, bt_d, bt_d.shape[1], dev(lens), B, max_seq, first,
                                 last, k, idx, ws, size)
        assert torch.all(idx[B] == -7)
        return idx[:B]

    def check(self, out, q, qd, od, bt, lens, slots, pages=None):
        q = bf16(q) if qd == 1 else np.asarray(q, np.float32).astype(np.float64)
        got = out.double().cpu().numpy()
        for b in range(len(lens)):
            want, bound = self.ref.attend(q[b], bt[b], slots[b], lens[b], None if pages is None else pages[b])
            if od == 1:
                bound = bound + np.abs(want) * 2.0 ** -8
            off = np.abs(got[b] - want)
            assert np.all(off <= bound), (b, lens[b], float((off / bound).max()))


def acts(rng, shape, outliers=True):
    x = rng.normal(size=shape) * np.exp(0.5 * rng.normal(size=shape[-2:]))
    if outliers:
        x[..., rng.integers(shape[-1])] *= 20
    return x


def tables(rng, B, per_req, pages, used):
    ids = rng.permutation(pages)
    bt, at = np.full((B, per_req), -1, np.int32), 0
    for b in range(B):
        bt[b, :used[b]] = ids[at:at + used[b]]
        at += used[b]
    return bt


def filled(osc, rng, lens, scale=1.0, **kw):
    """A rig whose cache holds requests of the given lengths, written by the library and by the oracle."""
    rig = Rig(osc, **kw)
    slots = rng.permutation(rig.cfg.max_requests)[:len(lens)]
    bt = tables(rng, len(lens), rig.cfg.max_pages_per_req, rig.cfg.num_pages, [n // rig.P for n in lens])
    K, V = ([acts(rng, (n, rig.heads, rig.d)) * scale for n in lens] for _ in range(2))
    rig.write(K, V, 1, lens, [0] * len(lens), bt, slots)
    return rig, bt, slots


# ------------------------------------------------------------------------------------------------ refusals first
def test_refusals(osc):
    with Rig(osc) as r:
        o, c = osc, r.ctx
        K = r.rows(np.ones((4, 2, 64)), 1)
        q = r.rows(np.ones((4, 4, 64)), 1)
        i4, bt = dev([0, 1, 2, 3, 4]), dev(np.zeros((4, 12)))
        out = torch.zeros(4, 4, 64, device="cuda")
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        idx = dev(np.zeros((4, 2, 3)))

        def refused(f, *a):
            with pytest.raises(o.OscarError) as e:
                f(*a)
            assert e.value.status in (o.ERR_INVALID, o.ERR_UNSUPPORTED)

        good = dict(write=(c, 0, K, K, 1, i4, i4, 4, 4, bt, 12, i4), append=(c, 0, K, K, 1, i4, 4, bt, 12, i4),
                    decode=(c, 0, q, 1, out, 0, bt, 12, i4, i4, 4, 64, ws, 1 << 20),
                    select=(c, 0, q, 1, bt, 12, i4, 4, 64, 1, 1, 3, idx, ws, 1 << 20),
                    sparse=(c, 0, q, 1, out, 0, idx, 3, bt, 12, i4, i4, 4, ws, 1 << 20))
        fn = dict(write=o.oscar_kv8_write, append=o.oscar_kv8_append, decode=o.oscar_kv8_decode_attn, select=o.oscar_kv8_select_pages,
                  sparse=o.oscar_kv8_sparse_decode_attn)
        k32 = K.float()
        odd = torch.zeros(4 * 128 + 8, dtype=torch.bfloat16, device="cuda")[1:4 * 128 + 1].view(4, 2, 64)     # not 16-byte aligned
        skew = torch.zeros(4, 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[:, :128].unflatten(1, (2, 64))  # nor is the stride
        turned = torch.zeros(4, 64, 2, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        bad = {
            "write": [(1, 2), (1, -1), (2, None), (3, None), (2, odd), (2, skew), (2, turned), (2, k32), (2, K[:3]), (2, K[:, :1]),
                      (2, K.cpu()), (4, 2), (5, None), (6, None), (5, i4.long()), (7, -1), (7, 65536), (8, -1), (9, None),
                      (9, bt.cpu()), (10, 0), (11, None), (5, i4[:4])],
            "append": [(1, 2), (2, None), (3, odd), (4, 7), (5, None), (6, -1), (6, 65536), (7, None), (8, 0), (9, None), (2, K[:3])],
            "decode": [(1, 2), (2, None), (2, q[:3]), (2, q.float()), (3, 5), (4, None), (4, out.to(torch.bfloat16)), (4, out[:3]),
                       (5, 3), (6, None), (7, 0), (8, None), (9, None), (10, -1), (10, 65536), (11, -1), (11, 12 * 16 + 1),
                       (12, None), (12, ws[1:]), (13, 64), (13, 1 << 21)],
            "select": [(1, 2), (2, None), (3, 9), (4, None), (5, 0), (6, None), (7, -1), (8, -1), (8, 193), (9, -1), (10, -1),
                       (9, 3), (11, 0), (11, 1), (11, 1 << 25), (12, None), (12, idx[:3]), (13, None), (14, 8)],
            "sparse": [(1, 2), (2, None), (3, 9), (4, None), (5, 4), (6, None), (6, idx[:, :, :2].contiguous()), (7, 0), (8, None),
                       (9, 0), (10, None), (11, None), (12, -1), (13, None), (14, 64)],
        }
        for name, cases in bad.items():
            for at, value in cases:
                a = list(good[name])
                a[at] = value
                refused(fn[name], *a)
        before = o.oscar_launch_count(c)
        for name, at in (("write", 7), ("write", 8), ("append", 6), ("decode", 10), ("select", 7), ("sparse", 12)):   # nothing to do
            a = list(good[name])
            a[at] = 0
            fn[name](*a)
        assert o.oscar_launch_count(c) == before and r.status() == 0
        refused(o.oscar_kv8_bind, c, 0, r.pool, r.tail)                     # once per context
        refused(o.oscar_kv8_fork, c, [0], 16, 0, [1], 12)                   # page 0 is not allocated
        r.same()


# ------------------------------------------------------------------------------------------------ write
GEO = [(16, 64), (32, 64), (64, 64), (16, 128), (32, 128), (64, 128)]


@pytest.mark.parametrize("P,d", GEO)
@pytest.mark.parametrize("fmt", [O.INT8, O.E4M3])
@pytest.mark.parametrize("dtype", [0, 1])
def test_write(osc, P, d, fmt, dtype):
    rng = np.random.default_rng([P, d, fmt, dtype])
    with Rig(osc, fmt, P, d, heads=3 if d == 64 else 2, pages=80) as r:
        lens0, slots = [0, P + 3, 2 * P, 5, 3 * P - 1], rng.permutation(5)
        lens1 = [2 * P + 1, 1, 0, P - 5, 4 * P + 2]
        bt = tables(rng, 5, 12, 80, [12] * 5)
        for starts, lens, gap in (([0] * 5, lens0, 0), (lens0, lens1, 8)):
            K, V = ([acts(rng, (n, r.heads, d)) for n in lens] for _ in range(2))
            r.write(K, V, dtype, lens, starts, bt, slots, gap)
            r.same()
        assert r.status() == 0


def test_write_many_requests_and_a_long_one(osc):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 40, 70)]
    lens[33] = 64 * 11 + 5
    with Rig(osc, O.E4M3, 16, 64, heads=1, slots=70, per_req=45, pages=400) as r:
        bt, slots = tables(rng, 70, 45, 400, [n // 16 for n in lens]), rng.permutation(70)
        K, V = ([acts(rng, (n, 1, 64)) for n in lens] for _ in range(2))
        r.write(K, V, 1, lens, [0] * 70, bt, slots)
        r.same()
        assert r.status() == 0


@pytest.mark.parametrize("fmt", [O.INT8, O.E4M3])
@pytest.mark.parametrize("P,d,dtype", [(16, 64, 0), (32, 128, 1)])
def test_appends_leave_what_a_write_leaves(osc, fmt, P, d, dtype):
    rng = np.random.default_rng([P, fmt])
    with Rig(osc, fmt, P, d) as r, Rig(osc, fmt, P, d) as whole:
        B, n0, steps = 3, [0, P - 2, 2 * P + 1], 2 * P + 3
        slots, bt = [3, 0, 2], tables(rng, B, 12, 48, [6] * B)
        K, V = (acts(rng, (B, max(n0) + steps, 2, d)) for _ in range(2))
        r.write([K[b, :n0[b]] for b in range(B)], [V[b, :n0[b]] for b in range(B)], dtype, n0, [0] * B, bt, slots)
        for i in range(steps):
            n = [x + i for x in n0]
            r.append(np.stack([K[b, n[b]] for b in range(B)]), np.stack([V[b, n[b]] for b in range(B)]), dtype, n, bt, slots,
                     gap=16 * (i % 2))
        r.same()
        end = [x + steps for x in n0]
        whole.write([K[b, :end[b]] for b in range(B)], [V[b, :end[b]] for b in range(B)], dtype, end, [0] * B, bt, slots)
        assert torch.equal(r.pool, whole.pool)
        for b in range(B):
            at = (whole.layer, slots[b], slice(None), slice(None), slice(end[b] % P))
            assert torch.equal(r.tail[at], whole.tail[at])


@pytest.mark.parametrize("fmt", [O.INT8, O.E4M3])
def test_every_quotient(osc, fmt):
    """All pairs of BF16 mantissas of a value and of its block's maximum, the value up to 2^15 smaller: every tie between two
    codes and every quotient next to one."""
    P, d = 64, 128
    x = np.outer(2.0 ** -np.arange(16), np.arange(128, 256)).reshape(-1)            # 2048 values
    rows = np.zeros((128, P * d))
    for i, m in enumerate(range(128, 256)):
        own = x[x <= m]
        rows[i, :2 * len(own)] = np.concatenate([own, -own])
        rows[i, -1] = m
    K = np.concatenate([rows, rows[::-1] * 2.0 ** 90]).reshape(-1, 1, d)
    with Rig(osc, fmt, P, d, heads=1, per_req=256, pages=256, slots=1) as r:
        bt = np.arange(256, dtype=np.int32)[None]
        r.write([K], [K[::-1] * 2.0 ** -180], 0, [256 * P], [0], bt, [0])
        r.same()
        assert r.status() == 0


def test_write_shuffled_rows_of_a_thousand_requests(osc):
    """More requests than one probe of the search covers twice over, many of them empty, rows with a gap before the first."""
    rng = np.random.default_rng(6)
    B, P = 1100, 16
    lens = [int(x) for x in rng.integers(0, 30, B) * (rng.random(B) < 0.7)]
    starts = [0] * B
    with Rig(osc, O.INT8, P, 64, heads=1, slots=B, per_req=2, pages=sum(n // P for n in lens) + 1) as r:
        bt, slots = tables(rng, B, 2, r.cfg.num_pages, [n // P for n in lens]), rng.permutation(B)
        cu = 5 + np.concatenate([[0], np.cumsum(lens)])
        K, V = (acts(rng, (int(cu[-1]) + 3, 1, 64)) for _ in range(2))
        osc.oscar_kv8_write(r.ctx, r.layer, r.rows(K, 1), r.rows(V, 1), 1, dev(cu), dev(starts), B, len(K), dev(bt), 2, dev(slots))
        for b in range(B):
            r.ref.write(bt[b], slots[b], 0, bf16(K[cu[b]:cu[b + 1]]), bf16(V[cu[b]:cu[b + 1]]))
        r.same()
        assert r.status() == 0


def test_padded_batch(osc):
    """Padding in a batch: appends of length -1 and writes of no rows are skipped whatever their slot says."""
    rng = np.random.default_rng(7)
    P, d = 16, 64
    with Rig(osc, O.E4M3, P, d) as r:
        bt = tables(rng, 4, 12, 48, [2, 0, 2, 0])
        lens, slots = [20, 0, 31, 0], [1, -1, 3, 99]
        K, V = ([acts(rng, (n, 2, d)) for n in lens] for _ in range(2))
        r.write(K, V, 1, lens, [0, -5, 0, 1 << 30], bt, slots, ref=False)
        k, v = acts(rng, (4, 2, d)), acts(rng, (4, 2, d))
        osc.oscar_kv8_append(r.ctx, r.layer, r.rows(k, 1), r.rows(v, 1), 1, dev([20, -1, 31, -1]), 4, dev(bt), 12, dev(slots))
        for b in (0, 2):
            r.ref.write(bt[b], slots[b], 0, bf16(K[b]), bf16(V[b]))
            r.ref.write(bt[b], slots[b], lens[b], bf16(k[b:b + 1]), bf16(v[b:b + 1]), append=True)
        assert r.status() == 0
        r.same()
        q = acts(rng, (4, 4, d), False)
        out = r.decode(q, 1, 0, bt, [21, 0, 32, 0], slots)
        assert torch.all(out[[1, 3]] == 0) and r.status() == 0
        for b in (0, 2):
            r.check(out[b:b + 1], q[b:b + 1], 1, 0, bt[b:b + 1], [[21, 0, 32, 0][b]], [slots[b]])


@pytest.mark.parametrize("fmt", [O.INT8, O.E4M3])
def test_special_values(osc, fmt):
    """Zero and tiny blocks, negative zeros, the largest numbers, infinities and NaNs (with their status)."""
    rng = np.random.default_rng(9)
    P, d = 16, 64
    with Rig(osc, fmt, P, d, heads=1) as r:
        bt, slots = tables(rng, 2, 12, 48, [8, 1]), [1, 2]
        x = rng.normal(size=(7 * P, 1, d))
        x[:P] = 0
        x[P:2 * P] *= 2.0 ** -120
        x[2 * P:3 * P] = -0.0
        x[2 * P, 0, 0] = 1
        x[3 * P:4 * P] = 3.3e38 * np.sign(x[3 * P:4 * P])
        x[4 * P:5 * P] *= 2.0 ** -98
        r.write([x, x[:3]], [x[::-1], x[:3]], 1, [7 * P, 3], [0, 0], bt, slots)
        assert r.status() == 0
        r.same()
        y = rng.normal(size=(P, 1, d))
        y[3, 0, 5], y[4, 0, 6], y[5, 0, 7] = np.inf, -np.inf, np.nan
        with np.errstate(all="ignore"):
            r.write([y], [np.abs(y)], 1, [P], [7 * P], bt[:1], slots[:1])
        assert r.status() == osc.DEV_BAD_VALUE
        r.same()
        assert r.status() == 0


def test_bad_pages_lengths_and_slots(osc):
    """Each sets its status bit, stores nothing out of place, and leaves the other requests right."""
    rng = np.random.default_rng(11)
    P, d = 16, 64
    for what in ("unmapped", "far page", "short table", "negative start", "too long", "cu", "slot"):
        with Rig(osc, O.INT8, P, d) as r:
            bt = tables(rng, 3, 12, 48, [4, 4, 4])
            lens, starts, slots = [2 * P + 1] * 3, [0, 0, 0], [0, 1, 2]
            cu = np.concatenate([[0], np.cumsum(lens)])
            K, V = (acts(rng, (cu[-1], 2, d)) for _ in range(2))
            t, n_cols, bit = bt.copy(), 12, osc.DEV_BAD_LEN
            if what == "unmapped":
                t[1, 1], bit = -1, osc.DEV_BAD_PAGE
            elif what == "far page":
                t[1, 1], bit = 48, osc.DEV_BAD_PAGE
            elif what == "short table":
                t, n_cols, bit = np.ascontiguousarray(t[:, :1]), 1, osc.DEV_BAD_PAGE
            elif what == "negative start":
                starts[1] = -1
            elif what == "too long":
                starts[1] = 12 * P
            elif what == "cu":
                cu = np.array([0, lens[0], lens[0] - 1, lens[0] * 2])
            else:
                slots[1], bit = 5, osc.DEV_BAD_SLOT
            osc.oscar_kv8_write(r.ctx, r.layer, r.rows(K, 0), r.rows(V, 0), 0, dev(cu), dev(starts), 3, len(K), dev(t), n_cols,
                                dev(slots))
            assert r.status() == bit, what
            for b in range(3):
                a = cu[b]
                k, v = bf16(K[a:a + lens[b]]), bf16(V[a:a + lens[b]])
                if b != 1 and what not in ("short table", "cu"):
                    r.ref.write(bt[b], slots[b], 0, k, v)
            got, want = r.pool[r.layer].cpu().numpy(), r.ref.pool
            for b in (0, 2) if what not in ("short table", "cu") else ():
                assert np.array_equal(got[bt[b, :2]], want[bt[b, :2]])
            untouched = [p for p in range(48) if p not in bt]
            assert np.all(got[untouched] == 0xA5) and torch.all(r.pool[1 - r.layer] == 0xA5)


# ------------------------------------------------------------------------------------------------ decode
@pytest.mark.parametrize("P,d", GEO)
@pytest.mark.parametrize("G,fmt,qd,od", [(1, 0, 1, 0), (2, 1, 0, 0), (4, 0, 1, 1), (4, 1, 0, 0), (8, 1, 1, 1), (8, 0, 0, 0), (8, 1, 0, 0)])
def test_decode(osc, P, d, G, fmt, qd, od):
    rng = np.random.default_rng([P, d, G, fmt])
    lens = [0, 1, P - 1, P, P + 1, 3 * P + 7, 11 * P + 15]
    rig, bt, slots = filled(osc, rng, lens, fmt=fmt, P=P, d=d, G=G, slots=8, heads=2 if G > 1 else 3)
    with rig as r:
        q = acts(rng, (len(lens), r.heads * G, d), False)
        out = r.decode(q, qd, od, bt, lens, slots, gap=8 if G == 4 else 0)
        assert r.status() == 0
        r.check(out, q, qd, od, bt, lens, slots)
        assert torch.all(out[0] == 0)
        longer = r.decode(q, qd, od, bt, lens, slots, max_seq=12 * P)          # another split, the same result within the bound
        r.check(longer, q, qd, od, bt, lens, slots)


@pytest.mark.parametrize("B,n,G,fmt,P,d", [(1, 9001, 4, 0, 64, 128), (3, 5000, 8, 1, 64, 128), (2, 3001, 2, 1, 16, 64),
                                           (40, 700, 8, 0, 32, 128)])
def test_decode_long(osc, B, n, G, fmt, P, d):
    rng = np.random.default_rng([B, n])
    lens = [int(x) for x in rng.integers(n // 2, n + 1, B)]
    rig, bt, slots = filled(osc, rng, lens, fmt=fmt, P=P, d=d, G=G, heads=1, slots=B + 1, per_req=n // P + 1,
                            pages=sum(x // P for x in lens) + 2)
    with rig as r:
        q = acts(rng, (B, G, d), False)
        for qd, od in ((1, 0), (0, 0)):
            r.check(r.decode(q, qd, od, bt, lens, slots), q, qd, od, bt, lens, slots)
        assert r.status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("loud", [1e-30, 1e-4, 1.0, 300.0, 1e12])
def test_decode_magnitudes(osc, fmt, loud):
    """Peaked and flat weights, values far from 1, and pages whose scales lie 2^40 apart."""
    rng = np.random.default_rng(13)
    P, d, n = 16, 64, 16 * 7 + 3
    with Rig(osc, fmt, P, d, G=4) as r:
        bt = tables(rng, 1, 12, 48, [7])
        K, V = (acts(rng, (n, 2, d)) for _ in range(2))
        K *= loud
        V *= 10.0 ** rng.integers(-6, 7, (8, 1, 1)).repeat(P, 0)[:n]
        r.write([K], [V], 0, [n], [0], bt, [2])
        q = acts(rng, (1, 8, d), False) * min(1 / loud, 1e25)
        r.check(r.decode(q, 0, 0, bt, [n], [2]), q, 0, 0, bt, [n], [2])


@pytest.mark.parametrize("G,qd", [(1, 0), (2, 0), (4, 0), (8, 0), (4, 1), (8, 1)])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("P,d", [(16, 64), (64, 64), (64, 128)])
def test_decode_large_scores(osc, P, d, fmt, G, qd):
    """Scores of 2e4 to 1e5, nearly the same for every token, from query components whose digits beyond f16's count for tens
    in the exponent, in either direction."""
    rng = np.random.default_rng([P, d, fmt, G])
    lens, loud = [3 * P, 3 * P + 5, P // 2], [513.25, 513.75, 700.3, -513.25, -700.3, 1201.7, 2100.1, -1999.9]
    with Rig(osc, fmt, P, d, heads=2, G=G) as r:
        bt, slots = tables(rng, 3, 12, 48, [3, 3, 0]), [1, 4, 0]
        K, V = ([rng.normal(size=(n, 2, d)) for n in lens] for _ in range(2))
        for k in K:
            k[:, :, 0] = 500 * (1 if d == 64 else 1.5)
        r.write(K, V, 0, lens, [0] * 3, bt, slots)
        for i in range(0, 8, G):
            q = rng.normal(size=(3, 2 * G, d))
            q[:, :, 0] = (loud * 2)[i:i + 2 * G]
            out = r.decode(q, qd, 0, bt, lens, slots)
            assert torch.isfinite(out).all()
            r.check(out, q, qd, 0, bt, lens, slots)
        assert r.status() == 0


@pytest.mark.parametrize("G,qd", [(2, 0), (4, 1), (8, 0), (8, 1)])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("size", [1e8, 1e11, 1e15, 1e25, 1e33])
def test_decode_where_one_key_leads_by_far(osc, fmt, G, qd, size):
    """Finite scores up to 1e33 of which one is twice the next: the output is that token's value row, in a page or in the
    tail.  The others' weights are exp(-size / 2) = 0 whatever a score's rounding, so what is left is the roundings of one
    weight, its scales and its division: 8 of 2^-24."""
    rng = np.random.default_rng([fmt, G])
    P, d = 16, 64
    for n, top in ((5 * P + 3, 2 * P + 7), (5 * P + 3, 5 * P + 1), (3, 2), (90 * P, 77 * P)):
        with Rig(osc, fmt, P, d, heads=2, G=G, per_req=90, pages=90) as r:
            bt = tables(rng, 1, 90, 90, [n // P])
            K, V = (rng.normal(size=(n, 2, d)) for _ in range(2))
            K[:, :, 5] = 0.5 * size ** 0.5
            K[top, :, 5] = size ** 0.5
            r.write([K], [V], 0, [n], [0], bt, [0])
            q = rng.normal(size=(1, 2 * G, d))
            q[:, :, 5] = 8 * size ** 0.5
            out = r.decode(q, qd, 0, bt, [n], [0])[0].double().cpu().numpy()
            for h in range(2):
                v = r.ref.rows(bt[0], 0, n, h)[1][top]
                assert np.all(np.abs(out[h * G:(h + 1) * G] - v) <= 8 * 2.0 ** -24 * np.abs(v)), (n, top)
            assert r.status() == 0


@pytest.mark.parametrize("G,qd", [(1, 1), (2, 0), (4, 1), (4, 0), (8, 0), (8, 1)])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("P,d", [(16, 64), (64, 64), (32, 128), (64, 128)])
def test_decode_where_the_loudest_query_channel_meets_no_key(osc, P, d, fmt, G, qd):
    """A query component 10^3 to 10^30 times the others over a channel of zero keys: the others decide the weights."""
    rng = np.random.default_rng([P, d, fmt, G])
    lens = [9 * P, 9 * P + 3]
    with Rig(osc, fmt, P, d, heads=2, G=G) as r:
        bt, slots = tables(rng, 2, 12, 48, [9, 9]), [1, 4]
        K, V = ([rng.normal(size=(n, 2, d)) for n in lens] for _ in range(2))
        for k in K:
            k[:, :, 3] = 0
            k[4 * P:5 * P, 0, 3] = 1e-30                 # (a code of 0 as well, but for this page of one head)
            k[4 * P:5 * P, 0] *= 1e-30
        r.write(K, V, 0, lens, [0, 0], bt, slots)
        for loud in (1e3, 1e6, 1e9, 1e12, 1e20, 1e30):
            q = 3 * rng.normal(size=(2, 2 * G, d))
            q[:, ::2, 3] = loud
            q[:, 1::2, 3] = -loud
            r.check(r.decode(q, qd, 0, bt, lens, slots), q, qd, 0, bt, lens, slots)
            pages = np.tile(np.array([1, 3, 4, 8, -1], np.int32), (2, 2, 1))
            r.check(r.decode(q, qd, 0, bt, lens, slots, pages=pages), q, qd, 0, bt, lens, slots, pages)
            small = q * (1e-25 if loud > 1e6 else 1e-3)     # and where the query as a whole is quiet
            r.check(r.decode(small, 0, 0, bt, lens, slots), small, 0, 0, bt, lens, slots)
        assert r.status() == 0


@pytest.mark.parametrize("P,d", [(16, 64), (32, 128), (64, 64)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_write_from_slices_of_one_projection(osc, P, d, dtype):
    """K and V as 16-byte aligned slices of one wider tensor, from an odd row on; then a chunk that completes the page."""
    rng = np.random.default_rng([P, d, dtype])
    heads, unit = 2, 4 if dtype == 0 else 8                       # elements of 16 bytes
    with Rig(osc, P=P, d=d, heads=heads, fmt=O.E4M3) as r:
        bt, lens = tables(rng, 2, 12, 48, [4, 2]), [2 * P + 5, P + 1]
        at = [0, 0]
        for step in (lens, [P, 1]):
            x = torch.from_numpy(rng.normal(size=(sum(step) + 3, 3 * unit + 2 * heads * d)).astype(np.float32)).to(DT[dtype]).cuda()
            k = x[3:, unit:unit + heads * d].unflatten(1, (heads, d))
            v = x[3:, 2 * unit + heads * d:2 * unit + 2 * heads * d].unflatten(1, (heads, d))
            bt_d = dev(bt)
            osc.oscar_kv8_write(r.ctx, r.layer, k, v, dtype, dev([0, step[0], sum(step)]), dev(at), 2, sum(step), bt_d, 12, dev([3, 1]))
            for b, (lo, hi) in enumerate(((0, step[0]), (step[0], sum(step)))):
                r.ref.write(bt[b], [3, 1][b], at[b], bf16(k[lo:hi].float().cpu().numpy()), bf16(v[lo:hi].float().cpu().numpy()))
            at = [a + s for a, s in zip(at, step)]
        r.same()
        assert r.status() == 0


def test_decode_reports_bad_arguments_on_the_device(osc):
    rng = np.random.default_rng(17)
    lens = [50, 60, 70]
    rig, bt, slots = filled(osc, rng, lens)
    with rig as r:
        q = acts(rng, (3, 4, 64), False)
        good = r.decode(q, 1, 0, bt, lens, slots)
        for what, bit in (("page", osc.DEV_BAD_PAGE), ("long", osc.DEV_BAD_LEN), ("negative", osc.DEV_BAD_LEN), ("slot", osc.DEV_BAD_SLOT)):
            t, n, s = bt.copy(), list(lens), list(slots)
            if what == "page":
                t[1, 2] = 48
            elif what == "slot":
                s[1] = -1
            else:
                n[1] = 71 if what == "long" else -1
            out = r.decode(q, 1, 0, t, n, s, max_seq=70)
            assert r.status() == bit
            assert torch.equal(out[[0, 2]], good[[0, 2]]) and torch.isfinite(out).all()
            if bit == osc.DEV_BAD_LEN:
                assert torch.all(out[1] == 0)
            if what == "page":       # left out
                want, bound = r.ref.attend(bf16(q[1]), bt[1], slots[1], lens[1], [[0, 1]] * 2)
                assert np.all(np.abs(out[1].double().cpu().numpy() - want) <= bound)


@pytest.mark.parametrize("G,fmt,qd", [(2, 0, 0), (2, 1, 1), (8, 0, 1), (8, 1, 0)])
@pytest.mark.parametrize("n", [1, 16 * 3, 16 * 3 + 5, 16 * 80 + 7])
def test_decode_carries_nan(osc, G, fmt, qd, n):
    """A NaN or an infinity in a query head, or a NaN in a tail row, makes NaN of what depends on it and of nothing else."""
    rng = np.random.default_rng([G, fmt, n])
    P, d, heads = 16, 64, 2
    rig, bt, slots = filled(osc, rng, [n], fmt=fmt, P=P, d=d, G=G, heads=heads, per_req=81, pages=81)
    with rig as r:
        lists = np.full((1, heads, 81), -1, np.int32)
        lists[:, :, :n // P] = np.arange(n // P)
        q = acts(rng, (1, heads * G, d), False)
        for pages in (None, lists) if n >= P else (None,):
            good = r.decode(q, qd, 0, bt, [n], slots, pages=pages)
            assert torch.isfinite(good).all()
            for bad in (np.nan, np.inf, -np.inf):
                x = q.copy()
                x[0, G, 7] = bad                      # the second kv head's first query head
                out = r.decode(x, qd, 0, bt, [n], slots, pages=pages)
                keep = torch.arange(heads * G, device="cuda") != G
                assert torch.isnan(out[0, G]).all() and torch.equal(out[0, keep], good[0, keep])
            if n % P == 0:
                continue
            rows = r.tail[r.layer, slots[0], 1]       # [2][P][d] of the second kv head
            for kv in range(2):
                was = rows[kv, n % P - 1, 9].clone()
                rows[kv, n % P - 1, 9] = float("nan")
                out = r.decode(q, qd, 0, bt, [n], slots, pages=pages)
                rows[kv, n % P - 1, 9] = was
                reach = torch.zeros_like(out, dtype=torch.bool)
                reach[0, G:] = True
                if kv:
                    reach[:] = False
                    reach[0, G:, 9] = True
                assert torch.isnan(out[reach]).all() and torch.equal(out[~reach], good[~reach])
        assert r.status() == 0


# ------------------------------------------------------------------------------------------------ selection, sparse decode
@pytest.mark.parametrize("P,d", GEO)
@pytest.mark.parametrize("G,fmt,qd", [(1, 0, 1), (4, 1, 0), (8, 0, 0), (8, 1, 1)])
def test_select_and_sparse_decode(osc, P, d, G, fmt, qd):
    rng = np.random.default_rng([P, d, G, fmt])
    lens = [0, P - 1, 3 * P, 9 * P + 5, 25 * P + 1, 40 * P]
    rig, bt, slots = filled(osc, rng, lens, fmt=fmt, P=P, d=d, G=G, slots=7, per_req=41, pages=90)
    with rig as r:
        q = acts(rng, (len(lens), 2 * G, d), False)
        qx = bf16(q) if qd else q.astype(np.float32).astype(np.float64)
        for first, last, k in ((0, 0, 1), (1, 2, 7), (2, 0, 9), (0, 5, 39), (0, 0, 40), (3, 3, 100)):
            idx = r.select(q, qd, bt, lens, first, last, k, gap=8 if k == 7 else 0)
            got = idx.cpu().numpy()
            for b in range(len(lens)):
                assert np.array_equal(got[b], r.ref.select(qx[b], bt[b], lens[b], first, last, k)), (b, k)
            out = r.decode(q, qd, 0, bt, lens, slots, pages=idx)
            r.check(out, q, qd, 0, bt, lens, slots, pages=got)
        dense = r.decode(q, qd, 0, bt, lens, slots)
        r.check(out, q, qd, 0, bt, lens, slots)            # k = 100: every page
        assert torch.allclose(out, dense, rtol=1e-4, atol=1e-4) and r.status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_select_ties_and_near_ties(osc, fmt):
    """Equal pages go by the lower index; pages that differ in the last bit of a bound keep their float64 order."""
    rng = np.random.default_rng(23)
    P, d, pages = 16, 128, 300
    with Rig(osc, fmt, P, d, heads=2, G=2, per_req=pages, pages=pages) as r:
        bt = rng.permutation(pages)[None].astype(np.int32)
        K = np.tile(acts(rng, (P, 2, d)), (pages, 1, 1))               # every page the same
        r.write([K], [K], 1, [P * pages], [0], bt, [0])
        q = acts(rng, (1, 4, d), False)
        want = np.concatenate([np.arange(2 + 40), np.arange(pages - 3, pages)])
        assert np.array_equal(r.select(q, 1, bt, [P * pages], 2, 3, 45).cpu().numpy()[0], np.stack([want] * 2))
        # scales one float32 step apart: scores 2^-23 apart, far below what float32 sums tell apart
        sc = r.pool[r.layer][torch.from_numpy(bt[0].astype(np.int64)).cuda()][:, :, 2 * P * d:2 * P * d + 4].contiguous().view(torch.int32)
        step = torch.from_numpy(rng.integers(-3, 4, (pages, 2, 1)).astype(np.int32)).cuda()
        r.pool[r.layer, torch.from_numpy(bt[0].astype(np.int64)).cuda(), :, 2 * P * d:2 * P * d + 4] = (sc + step).view(torch.uint8)
        r.ref.pool[:] = r.pool[r.layer].cpu().numpy()
        for k in (1, 45, 150, 299):
            got = r.select(q, 1, bt, [P * pages], 0, 1, k).cpu().numpy()[0]
            assert np.array_equal(got, r.ref.select(bf16(q)[0], bt[0], P * pages, 0, 1, k))
        # a query of zeros: every bound is 0
        assert np.array_equal(r.select(q * 0, 1, bt, [P * pages], 0, 0, 9).cpu().numpy()[0], np.stack([np.arange(9)] * 2))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("P,d", [(16, 64), (32, 128)])
def test_select_where_the_loudest_query_channel_meets_no_key(osc, fmt, P, d):
    """A query component 10^12 times the others over a channel of zero keys: the order is that of the others."""
    rng = np.random.default_rng([d, fmt])
    lens = [40 * P + 3]
    with Rig(osc, fmt, P, d, heads=2, G=2, per_req=41, pages=41) as r:
        bt = tables(rng, 1, 41, 41, [40])
        K = rng.normal(size=(lens[0], 2, d))
        K[:, :, 3] = 0
        r.write([K], [K], 1, lens, [0], bt, [0])
        q = rng.normal(size=(1, 4, d))
        q[:, :, 3] = 1e12
        for k in (1, 7, 39):
            got = r.select(q, 0, bt, lens, 0, 0, k).cpu().numpy()[0]
            assert np.array_equal(got, r.ref.select(q[0].astype(np.float32).astype(np.float64), bt[0], lens[0], 0, 0, k))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("keys,query", [(-75, -50), (-75, -60), (-90, -40), (-90, -20), (-60, -66), (-60, -90), (-97, 100), (90, 20), (110, 100)])
def test_select_where_scores_leave_the_normal_numbers(osc, fmt, keys, query):
    """Keys near 2^keys and queries near 2^query: bounds whose size float32 holds with few digits, or not at all."""
    rng = np.random.default_rng([fmt, 200 + keys, 200 + query])
    lens = [60 * 16 + 3]
    with Rig(osc, fmt, 16, 64, heads=2, G=2, per_req=61, pages=61) as r:
        bt = tables(rng, 1, 61, 61, [60])
        K = rng.normal(size=(lens[0], 2, 64)) * 2.0 ** keys
        r.write([K], [K], 0, lens, [0], bt, [0])
        q = (rng.normal(size=(1, 4, 64)) * 2.0 ** query).astype(np.float32).astype(np.float64)
        for k in (1, 7, 30, 59):
            got = r.select(q, 0, bt, lens, 0, 0, k).cpu().numpy()[0]
            assert np.array_equal(got, r.ref.select(q[0], bt[0], lens[0], 0, 0, k)), k
        assert r.status() == 0


@pytest.mark.parametrize("pages", [2100, 9000])
@pytest.mark.parametrize("fmt", [0, 1])
def test_select_among_thousands_of_equal_and_nearly_equal_pages(osc, fmt, pages):
    """More pages than are ranked one by one: equal ones by the lower index, nearly equal ones in their float64 order."""
    rng = np.random.default_rng([fmt, pages])
    P, d = 16, 64
    with Rig(osc, fmt, P, d, heads=1, G=2, per_req=pages, pages=pages, layers=1, layer=0, oracle=False) as r:
        bt, n = rng.permutation(pages)[None].astype(np.int32), [pages * P]
        K = np.tile(acts(rng, (P, 1, d)), (pages, 1, 1))
        r.write([K], [K], 1, n, [0], bt, [0], ref=False)
        r.ref = O.Cache(P, d, 1, fmt, r.pool[0].cpu().numpy().copy(), np.zeros((5, 1, 2, P, d)))
        q = acts(rng, (1, 2, d), False)
        some = (1, 45, pages // 2, pages - 1)
        for k in some:                                                  # every page the same
            want = np.concatenate([np.arange(k - 1), [pages - 1]])
            assert np.array_equal(r.select(q, 1, bt, n, 0, 1, k).cpu().numpy()[0, 0], want)
            assert np.array_equal(r.select(q * 0, 1, bt, n, 0, 0, k).cpu().numpy()[0, 0], np.arange(k))
        at = torch.from_numpy(bt[0].astype(np.int64)).cuda()
        field = (0, at, slice(None), slice(2 * P * d, 2 * P * d + 4))
        step = torch.from_numpy(rng.integers(-3, 4, (pages, 1, 1)).astype(np.int32)).cuda()
        r.pool[field] = (r.pool[field].contiguous().view(torch.int32) + step).view(torch.uint8)
        r.ref.pool[:] = r.pool[0].cpu().numpy()
        for k in some:
            got = r.select(q, 1, bt, n, 0, 1, k).cpu().numpy()[0]
            assert np.array_equal(got, r.ref.select(bf16(q)[0], bt[0], n[0], 0, 1, k))
        assert r.status() == 0


@pytest.mark.parametrize("bad", [np.inf, -np.inf, 3.4e38])
def test_select_lists_stay_valid(osc, bad):
    """Whatever a query holds, a list is full, ascending and of complete pages, the kept ones among them."""
    rng = np.random.default_rng(59)
    lens = [40 * 16 + 3]
    rig, bt, slots = filled(osc, rng, lens, fmt=1, G=4, per_req=41, pages=41)
    with rig as r:
        q = acts(rng, (1, 8, 64), False)
        q[0, 2, 7] = bad
        idx = r.select(q, 0, bt, lens, 2, 1, 9).cpu().numpy()[0]
        assert np.all(np.diff(idx, axis=1) > 0) and idx.min() == 0 and idx.max() == 39
        assert np.array_equal(idx[:, [0, 1, 8]], [[0, 1, 39]] * 2)
        good = r.ref.select(q[0].astype(np.float32).astype(np.float64), bt[0], lens[0], 2, 1, 9) if np.isfinite(bad) else idx
        assert np.array_equal(idx, good) and r.status() == 0


def test_select_long(osc):
    rng = np.random.default_rng(29)
    P, d, pages = 16, 64, 4500
    with Rig(osc, O.INT8, P, d, heads=1, G=4, per_req=pages, pages=pages, layers=1, layer=0) as r:
        bt = rng.permutation(pages)[None].astype(np.int32)
        K = rng.normal(size=(P * pages, 1, d)) * np.exp(0.3 * rng.normal(size=(pages, 1, 1))).repeat(P, 0)
        r.write([K], [K], 1, [P * pages], [0], bt, [0])
        q = rng.normal(size=(1, 4, d))
        for k in (3, 64, 1025, 4499):
            got = r.select(q, 1, bt, [P * pages], 1, 1, k).cpu().numpy()[0]
            assert np.array_equal(got, r.ref.select(bf16(q)[0], bt[0], P * pages, 1, 1, k))
        assert r.status() == 0


def test_select_and_sparse_report_bad_arguments(osc):
    rng = np.random.default_rng(31)
    lens = [160, 170]
    rig, bt, slots = filled(osc, rng, lens)
    with rig as r:
        q = acts(rng, (2, 4, 64), False)
        t = bt.copy()
        t[0, 3] = -1
        idx = r.select(q, 1, t, lens, 0, 0, 5)
        assert r.status() == osc.DEV_BAD_PAGE and 3 not in idx[0].cpu().numpy()
        idx = r.select(q, 1, bt, [160, 171], 0, 0, 5, max_seq=170)
        assert r.status() == osc.DEV_BAD_LEN and torch.all(idx[1] == -1)
        qn = q.copy()
        qn[0, 0, 0] = np.nan
        idx = r.select(qn, 1, bt, lens, 0, 0, 5).cpu().numpy()
        assert np.all(np.diff(idx, axis=2) > 0) and idx.min() >= 0 and idx.max() < 10 and r.status() == 0
        good = np.array([[[0, 4, 9], [1, 2, -1]]] * 2, np.int32)
        want = r.decode(q, 1, 0, bt, lens, slots, pages=good)
        r.check(want, q, 1, 0, bt, lens, slots, pages=good)
        for row in ([4, 4, 9], [4, 0, 9], [0, 4, 10], [0, -1, 9], [0, 4, 1 << 30]):
            pages = good.copy()
            pages[0, 0] = row
            out = r.decode(q, 1, 0, bt, lens, slots, pages=pages)
            assert r.status() == osc.DEV_BAD_PAGE
            assert torch.equal(out[1], want[1]) and torch.equal(out[0, 2:], want[0, 2:]) and torch.isfinite(out).all()


# ------------------------------------------------------------------------------------------------ fork, compaction
@pytest.mark.parametrize("n", [0, 5, 16, 16 * 3 + 15])
@pytest.mark.parametrize("ways", [1, 3, 4])
def test_fork(osc, n, ways):
    with Rig(osc, O.INT8, layers=3, layer=0) as r:
        before = torch.randn(r.tail.shape, device="cuda").to(torch.bfloat16)
        r.tail.copy_(before)
        src = osc.oscar_alloc_pages(r.ctx, 3)
        dst = [4, 0, 3, 1][:ways]
        t = osc.oscar_kv8_fork(r.ctx, src, n, 2, dst, 12)
        assert np.all(t[:, :n // 16] == src[:n // 16]) and np.all(t[:, n // 16:] == -1)
        want = before.clone()
        want[:, dst, :, :, :n % 16] = before[:, 2, :, :, :n % 16][:, None]
        assert torch.equal(r.tail, want)
        assert [osc.oscar_page_refcount(r.ctx, p) for p in src] == [1 + ways * (i < n // 16) for i in range(3)]


@pytest.mark.parametrize("pages,live,int2", [(48, 20, True), (48, 47, False), (2300, 1100, True)])
def test_compaction(osc, pages, live, int2):
    rng = np.random.default_rng([pages, live])
    with Rig(osc, O.E4M3, layers=3, pages=pages, int2=int2, per_req=pages) as r:
        r.pool.copy_(torch.randint(0, 256, r.pool.shape, dtype=torch.uint8, device="cuda"))
        old, old2 = r.pool.clone(), r.int2.clone() if int2 else None
        osc.oscar_alloc_pages(r.ctx, pages)
        gone = rng.permutation(pages)[:pages - live]
        osc.oscar_unref_pages(r.ctx, gone)
        keep = np.setdiff1d(np.arange(pages), gone)
        bt = np.full((5, pages), -1, np.int32)
        for row in bt:
            row[:live // 2] = rng.permutation(keep)[:live // 2]
        t = dev(bt)
        table, n = osc.oscar_compact_pages(r.ctx, t, 5, pages, pages)
        assert n == live and sorted(table[keep].tolist()) == list(range(live))
        assert np.array_equal(t.cpu().numpy(), np.where(bt >= 0, table[bt], -1))
        at, to = torch.from_numpy(keep).cuda(), torch.from_numpy(table[keep].astype(np.int64)).cuda()
        assert torch.equal(r.pool[:, to], old[:, at]) and torch.equal(r.pool[:, live:], old[:, live:])
        if int2:
            a, b = (x.view(3, pages, -1) for x in (r.int2, old2))
            assert torch.equal(a[:, to], b[:, at]) and torch.equal(a[:, live:], b[:, live:])


# ------------------------------------------------------------------------------------------------ as they are used together
@pytest.mark.parametrize("fmt", [0, 1])
def test_serving_run(osc, fmt):
    """Two prompts; one forks in two; all decode for some steps, sparsely every other one; one request ends, the pages are
    compacted, and the others go on from where they were."""
    rng = np.random.default_rng(37 + fmt)
    P, d, per_req = 16, 64, 20
    with Rig(osc, fmt, P, d, heads=2, G=4, per_req=per_req, pages=60) as r:
        o = osc
        bt = np.full((3, per_req), -1, np.int32)
        lens, slots = [133, 133, 90], [0, 3, 4]
        for b in (2, 0):
            bt[b, :lens[b] // P] = o.oscar_alloc_pages(r.ctx, lens[b] // P)
        K, V = ([acts(rng, (lens[b], 2, d)) for b in (0, 2)] for _ in range(2))
        r.write(K, V, 1, [133, 90], [0, 0], bt[[0, 2]], [0, 4])
        bt[1] = o.oscar_kv8_fork(r.ctx, bt[0], 133, 0, [3], per_req)[0]
        r.ref.tail[3, :, :, :133 % P] = r.ref.tail[0, :, :, :133 % P]
        r.same()
        rows = [0, 1, 2]

        def steps(count):
            for i in range(count):
                for b in rows:
                    if (lens[b] + 1) % P == 0:
                        bt[b, lens[b] // P] = o.oscar_alloc_pages(r.ctx, 1)[0]
                n, s, t = [lens[b] for b in rows], [slots[b] for b in rows], bt[rows]
                r.append(acts(rng, (len(rows), 2, d)), acts(rng, (len(rows), 2, d)), 1, n, t, s)
                n = [x + 1 for x in n]
                for b in rows:
                    lens[b] += 1
                q = acts(rng, (len(rows), 8, d), False)
                idx = r.select(q, 1, t, n, 1, 1, 4) if i % 2 else None
                r.check(r.decode(q, 1, 0, t, n, s, pages=idx), q, 1, 0, t, n, s, None if idx is None else idx.cpu().numpy())

        steps(30)
        o.oscar_unref_pages(r.ctx, bt[2, :lens[2] // P])
        rows = [0, 1]
        q = acts(rng, (2, 8, d), False)
        n, s = [lens[b] for b in rows], [slots[b] for b in rows]
        before = r.decode(q, 1, 0, bt[rows], n, s)
        t = dev(bt[rows])
        table, live = o.oscar_compact_pages(r.ctx, t, 2, per_req, 60)
        assert live == len(set(bt[rows][bt[rows] >= 0].tolist()))
        bt[rows] = np.where(bt[rows] >= 0, table[bt[rows]], -1)
        assert np.array_equal(t.cpu().numpy(), bt[rows])
        assert torch.equal(r.decode(q, 1, 0, t, n, s), before)
        r.ref.pool = r.pool[r.layer].cpu().numpy().copy()
        steps(20)
        assert r.status() == 0


def test_graphs_streams_and_shared_workspace(osc):
    """An append, a selection and both decodes captured once and replayed on new inputs; two graphs that share a workspace,
    replayed in turn; decodes on two streams at once, each with its own workspace."""
    rng = np.random.default_rng(41)
    P, d, lens = 16, 128, [200, 333]
    rig, bt, slots = filled(osc, rng, lens, fmt=1, P=P, d=d, G=8, per_req=24)
    with rig as r:
        o, B, max_seq = osc, 2, 24 * P
        bt[:, 20:] = [[40, 41, 42, 43], [44, 45, 46, 47]]
        bt[0, 12:16] = [36, 37, 38, 39]
        qt, kt = (torch.zeros(B, h, d, dtype=torch.bfloat16, device="cuda") for h in (16, 2))
        out = [torch.zeros(B, 16, d, device="cuda") for _ in range(2)]
        idx = torch.zeros(B, 2, 6, dtype=torch.int32, device="cuda")
        n0, n1, sl, t = dev(lens), dev([x + 1 for x in lens]), dev(slots), dev(bt)
        size = max(o.oscar_kv8_decode_workspace_size(r.cfg, B, max_seq), o.oscar_kv8_sparse_workspace_size(r.cfg, B, 6))
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        sws = torch.zeros(o.oscar_kv8_select_workspace_size(r.cfg, B, max_seq), dtype=torch.uint8, device="cuda")

        def dense():
            o.oscar_kv8_append(r.ctx, r.layer, kt, kt, 1, n0, B, t, 24, sl)
            o.oscar_kv8_decode_attn(r.ctx, r.layer, qt, 1, out[0], 0, t, 24, n1, sl, B, max_seq, ws, size)

        def sparse():
            o.oscar_kv8_select_pages(r.ctx, r.layer, qt, 1, t, 24, n1, B, max_seq, 1, 1, 6, idx, sws, sws.numel())
            o.oscar_kv8_sparse_decode_attn(r.ctx, r.layer, qt, 1, out[1], 0, idx, 6, t, 24, n1, sl, B, ws, size)

        dense()
        sparse()
        torch.cuda.synchronize()
        graphs = []
        for f in (dense, sparse):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                f()
            graphs.append(g)
        for i in range(2):
            K, q = acts(rng, (B, 2, d)), acts(rng, (B, 16, d), False)
            kt.copy_(r.rows(K, 1))
            qt.copy_(r.rows(q, 1))
            n0.copy_(dev([x + i for x in lens]))
            n1.copy_(dev([x + i + 1 for x in lens]))
            for g in graphs:
                g.replay()
            for b in range(B):
                r.ref.write(bt[b], slots[b], lens[b] + i, bf16(K[b:b + 1]), bf16(K[b:b + 1]), append=True)
            n = [x + i + 1 for x in lens]
            r.check(out[0], q, 1, 0, bt, n, slots)
            r.check(out[1], q, 1, 0, bt, n, slots, idx.cpu().numpy())
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        qs = [acts(rng, (B, 16, d), False) for _ in range(2)]
        got = []
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append([r.decode(q, 1, 0, bt, n, slots) for _ in range(3)])
        torch.cuda.synchronize()
        for q, outs in zip(qs, got):
            for x in outs:
                r.check(x, q, 1, 0, bt, n, slots)
        assert r.status() == 0


def test_outputs_repeat_bit_for_bit(osc):
    """The same call gives the same bits, wherever its request lies in a batch: nothing is summed in the order of arrival."""
    rng = np.random.default_rng(61)
    lens = [16 * 150 + 3] * 3
    rig, bt, slots = filled(osc, rng, lens, fmt=1, G=8, per_req=151, pages=460)
    with rig as r:
        q = np.tile(acts(rng, (1, 16, 64), False), (3, 1, 1))
        pages = r.select(q, 0, bt, lens, 1, 1, 40)
        for idx in (None, pages):
            first = r.decode(q, 0, 0, bt, lens, slots, pages=idx)
            for _ in range(5):
                assert torch.equal(r.decode(q, 0, 0, bt, lens, slots, pages=idx), first)
            turned = r.decode(q, 0, 0, bt[[2, 0, 1]], lens, slots[[2, 0, 1]], pages=None if idx is None else idx[[2, 0, 1]].contiguous())
            assert torch.equal(turned, first[[2, 0, 1]])
        for _ in range(5):
            assert torch.equal(r.select(q, 0, bt, lens, 1, 1, 40), pages)
        assert r.status() == 0


def test_page_moves_are_refused_during_capture(osc):
    """The allocator changes at the call, so neither can be part of a graph; the capture goes on."""
    with Rig(osc, O.INT8, layers=2, layer=0) as r:
        src = osc.oscar_alloc_pages(r.ctx, 5)
        osc.oscar_unref_pages(r.ctx, src[:2])
        t, x = dev([src[2:]]), torch.zeros(4, device="cuda")
        x.add_(1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x.add_(1)
            for n in (16, 20):
                with pytest.raises(osc.OscarError, match="captured"):
                    osc.oscar_kv8_fork(r.ctx, src[2:], n, 0, [1], 12)
            with pytest.raises(osc.OscarError, match="captured"):
                osc.oscar_compact_pages(r.ctx, t, 1, 3, 48)
        graph.replay()
        assert torch.all(x == 2) and t.tolist() == [src[2:]]
        assert [osc.oscar_page_refcount(r.ctx, p) for p in src] == [0, 0, 1, 1, 1]
        osc.oscar_kv8_fork(r.ctx, src[2:], 20, 0, [1], 12)
        assert osc.oscar_compact_pages(r.ctx, t, 1, 3, 48)[1] == 3 and sorted(t[0].tolist()) == [0, 1, 2] and r.status() == 0


def test_offsets_past_32_bits(osc):
    """A pool of 4.7 GB: pages at its end are written, read, selected and moved."""
    rng = np.random.default_rng(43)
    P, d, pages = 64, 128, 35100
    n = 64 * 9 + 20
    with Rig(osc, O.E4M3, P, d, heads=8, G=1, pages=pages, layers=1, layer=0, oracle=False) as r:
        small = O.Cache(P, d, 8, O.E4M3, np.zeros((9, 8, r.block), np.uint8), np.zeros((5, 8, 2, P, d)))
        ids = np.arange(pages - 9, pages)
        bt = np.full((1, 12), -1, np.int32)
        bt[0, :9] = rng.permutation(ids)
        K, V = (acts(rng, (n, 8, d)) for _ in range(2))
        r.write([K], [V], 1, [n], [0], bt, [4], ref=False)
        ref_bt = bt[0, :9] - ids[0]
        small.write(ref_bt, 4, 0, bf16(K), bf16(V))
        used = np.r_[0:2 * P * d + 8, 2 * P * d + 16:2 * P * d + 16 + 2 * d]
        assert np.array_equal(r.pool[0, ids[0]:].cpu().numpy()[..., used], small.pool[..., used])
        q = acts(rng, (1, 8, d), False)
        r.ref = small
        r.check(r.decode(q, 1, 0, bt, [n], [4]), q, 1, 0, [ref_bt], [n], [4])
        idx = r.select(q, 1, bt, [n], 0, 1, 4).cpu().numpy()
        assert np.array_equal(idx[0], small.select(bf16(q)[0], ref_bt, n, 0, 1, 4))
        osc.oscar_alloc_pages(r.ctx, pages)
        osc.oscar_unref_pages(r.ctx, np.arange(pages - 9))
        t = dev(bt)
        _, live = osc.oscar_compact_pages(r.ctx, t, 1, 12, pages)
        assert live == 9 and t.max() < 9
        r.check(r.decode(q, 1, 0, t, [n], [4]), q, 1, 0, [ref_bt], [n], [4])
        assert r.status() == 0


def test_kernel_times_by_name(osc):
    rng = np.random.default_rng(47)
    lens = [100]
    rig, bt, slots = filled(osc, rng, lens, per_req=200)
    with rig as r:
        osc.oscar_set_timing(r.ctx, True)
        q = acts(rng, (1, 4, 64), False)
        r.select(q, 1, bt, lens, 0, 0, 2)
        r.check(r.decode(q, 1, 0, bt, lens, slots, max_seq=3200), q, 1, 0, bt, lens, slots)    # split: decode and merge
        r.check(r.decode(q, 1, 0, bt, lens, slots), q, 1, 0, bt, lens, slots)                  # short: decode alone
        for name, calls in (("kv8_select", 1), ("kv8_decode", 2), ("kv8_combine", 1)):
            ms, count = osc.oscar_kernel_time(r.ctx, name)
            assert ms > 0 and count == calls, name


def test_launch_count(osc):
    """Every kernel counts: two of a selection that has to choose, one of one that takes every page."""
    rng = np.random.default_rng(53)
    lens = [100]
    rig, bt, slots = filled(osc, rng, lens, per_req=200)
    with rig as r:
        q = acts(rng, (1, 4, 64), False)
        for call, kernels in ((lambda: r.select(q, 1, bt, lens, 0, 0, 2), 2), (lambda: r.select(q, 1, bt, lens, 0, 0, 9), 1),
                              (lambda: r.decode(q, 1, 0, bt, lens, slots), 1),
                              (lambda: r.decode(q, 1, 0, bt, lens, slots, max_seq=3200), 2)):
            before = osc.oscar_launch_count(r.ctx)
            call()
            assert osc.oscar_launch_count(r.ctx) - before == kernels
