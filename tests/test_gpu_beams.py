"""Several continuations of one prompt in the 8-bit cache, on the GPU against the float64 oracle: decode of requests that share
a prefix, the choice of the next beams, the reordering of their states, and a run of them together.

Tolerances of the shared decode: the bound of a float32 evaluation (oracle.kv8.attend_bound); the shared part's weights enter
their products as f16 numbers, of weight times V scale, the largest being 2^2 or more: two of them (22 bits) where the output is float32,
one (11 bits, 2^-12 of the weight) where it is BF16, and no finer than f16's last place, 2^-25 / 2^2 of the largest weight times
its page's largest value; a BF16 output is rounded once more (2^-8 of the value).  Selections: keys within 10^-6 of the oracle's and a float32 rounding (2^-24); tokens and parents are
equal unless the keys of two beams' candidates are closer than 2 10^-6.  Reordered states are equal.
"""
import numpy as np
import pytest

from oracle import beams as OB
from oracle import kv8 as O
from tests.test_gpu_kv8 import DT, Rig, acts, bf16, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def osc():
    from int2_rotated_paged_oscar_gb300 import build
    build.build()
    import int2_rotated_paged_oscar_gb300 as m
    m.load()
    return m


# ------------------------------------------------------------------------------------------------ shared prefixes
def family(osc, rng, sizes, shared, own, scale=1.0, **kw):
    """A rig whose requests lie in groups: group i has sizes[i] requests with shared[i] common pages, then own[...] tokens each
    (None: an empty request).  Written by the library and by the oracle."""
    P, total = kw.get("P", 16), sum(sizes)
    lens, group = [], np.repeat(np.arange(len(sizes)), sizes)
    for b, x in enumerate(own):
        lens.append(0 if x is None else int(shared[group[b]]) * P + x)
    per_req = max([n // P + 1 for n in lens] + [max(shared) + 1]) + 2
    pages = sum(shared) + sum(max(n // P - shared[g], 0) for n, g in zip(lens, group)) + 5
    rig = Rig(osc, per_req=per_req, pages=pages, slots=total + 2, **kw)
    ids, at = rng.permutation(pages), 0
    bt = np.full((total, per_req), -1, np.int32)
    slots = rng.permutation(total + 2)[:total]
    heads, d = rig.heads, rig.d
    pre = {}
    for g, s in enumerate(shared):
        pre[g] = (ids[at:at + s], [acts(rng, (s * P, heads, d)) * scale for _ in range(2)])
        at += s
    K, V = [], []
    for b in range(total):
        if lens[b] == 0:
            K.append(np.zeros((0, heads, d)))
            V.append(np.zeros((0, heads, d)))
            continue
        pg, (k, v) = pre[group[b]]
        mine = lens[b] // P - len(pg)
        bt[b, :len(pg)] = pg
        bt[b, len(pg):len(pg) + mine] = ids[at:at + mine]
        at += mine
        new = [acts(rng, (lens[b] - len(k), heads, d)) * scale for _ in range(2)]
        K.append(np.concatenate([k, new[0]]))
        V.append(np.concatenate([v, new[1]]))
    # (every request of a group writes the same codes into the shared pages: one call each)
    for b in range(total):
        if lens[b]:
            rig.write([K[b]], [V[b]], 1, [lens[b]], [0], bt[b:b + 1], slots[b:b + 1])
    rig.K, rig.V = K, V
    return rig, bt, slots, lens


def shared_decode(r, q, qd, od, sizes, shared, bt, lens, slots, max_shared=None, max_own=None, starts=None, gap=0, stream=None, ws=None):
    o, B = r.osc, len(lens)
    group = np.repeat(np.arange(len(sizes)), sizes)
    max_shared = max(shared) if max_shared is None else max_shared
    if max_own is None:
        max_own = max([max(n - shared[g] * r.P, 0) for n, g in zip(lens, group)])
    starts = np.concatenate([[0], np.cumsum(sizes)]) if starts is None else starts
    qt = q if torch.is_tensor(q) else r.rows(q, qd, gap)
    out = torch.full((B + 1, r.heads * r.G, r.d), 123.0, dtype=DT[od], device="cuda")
    size = o.oscar_kv8_shared_workspace_size(r.cfg, B, len(shared), max_shared, max_own)
    ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
    bt_d = dev(bt)
    o.oscar_kv8_shared_decode_attn(r.ctx, r.layer, qt, qd, out, od, dev(starts), dev(shared), len(shared), max_shared, bt_d,
                                   bt_d.shape[1], dev(lens), dev(slots), B, max_own, ws, size, stream)
    assert torch.all(out[B] == 123.0)          # rows behind the last request stay as they are
    return out[:B]


def within(r, out, q, qd, od, bt, lens, slots):
    q = bf16(q) if qd == 1 else np.asarray(q, np.float32).astype(np.float64)
    got = out.double().cpu().numpy()
    for b in range(len(lens)):
        if lens[b] == 0:
            assert not got[b].any()
            continue
        for h in range(r.heads):
            k, v = r.ref.rows(bt[b], slots[b], lens[b], h)
            for i in range(h * r.G, (h + 1) * r.G):
                want, bound = O.attend_bound(q[b, i], k, v, r.P)
                s = k @ q[b, i] / np.sqrt(r.d)
                e = np.exp(s - s.max())
                p = e / e.sum()
                page = np.concatenate([np.full(min(r.P, len(p) - t), np.abs(v[t:t + r.P]).max()) for t in range(0, len(p), r.P)])
                bound = bound + 2.0 ** (-22 if od == 0 else -12) * (p @ np.abs(v)) + 2.0 ** -27 * len(p) * (p * page).max()
                if od == 1:
                    bound = bound + (np.abs(want) + bound) * 2.0 ** -8
                off = np.abs(got[b, i] - want)
                assert np.all(off <= bound), (b, i, lens[b], float((off / bound).max()))


def test_shared_refusals(osc):
    with Rig(osc) as r:
        o, c = osc, r.ctx
        q, i4, bt = r.rows(np.ones((4, 4, 64)), 1), dev([0, 1, 2, 3, 4]), dev(np.zeros((4, 12)))
        out = torch.zeros(4, 4, 64, device="cuda")
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        good = (c, 0, q, 1, out, 0, i4, i4, 4, 2, bt, 12, i4, i4, 4, 64, ws, 1 << 20)
        before = o.oscar_launch_count(c)
        for at, value in [(1, 2), (1, -1), (2, None), (2, q[:3]), (2, q.float()), (3, 5), (4, None), (4, out[:3]), (5, 7), (6, None),
                          (6, i4[:4]), (6, i4.long()), (7, None), (7, i4[:3]), (8, 0), (8, -1), (8, 65536), (9, -1), (9, 13), (10, None),
                          (11, 0), (12, None), (13, None), (14, -1), (14, 65536), (15, -1), (15, 193), (16, None), (16, ws[1:]), (17, 64)]:
            a = list(good)
            a[at] = value
            with pytest.raises(o.OscarError) as e:
                o.oscar_kv8_shared_decode_attn(*a)
            assert e.value.status in (o.ERR_INVALID, o.ERR_UNSUPPORTED), (at, value)
        a = list(good)
        a[14] = 0
        o.oscar_kv8_shared_decode_attn(*a)      # nothing to do
        assert o.oscar_launch_count(c) == before


GEO = [(16, 64), (32, 64), (64, 64), (16, 128), (32, 128), (64, 128)]


@pytest.mark.parametrize("P,d", GEO)
@pytest.mark.parametrize("G,fmt,qd,od", [(1, 0, 1, 0), (2, 1, 0, 0), (4, 0, 1, 1), (4, 1, 0, 1), (8, 1, 1, 1), (8, 0, 0, 0), (8, 1, 1, 0)])
def test_shared_decode(osc, P, d, G, fmt, qd, od):
    """Groups of several sizes: pages that end inside a tile, requests with nothing of their own, empty ones, an empty group, a group
    that shares nothing."""
    rng = np.random.default_rng([P, d, G, fmt, qd, od])
    sizes, shared = [3, 1, 0, 2, 2], [7, 200 // P, 2, 0, 1]
    own = [0, 2 * P + 3, None, 1, 3 * P, 5, P - 1, 40]
    rig, bt, slots, lens = family(osc, rng, sizes, shared, own, P=P, d=d, G=G, fmt=fmt)
    with rig as r:
        q = acts(rng, (len(lens), r.heads * G, d), False)
        out = shared_decode(r, q, qd, od, sizes, shared, bt, lens, slots, gap=(0 if d == 64 else 64))
        assert r.status() == 0
        within(r, out, q, qd, od, bt, lens, slots)
        assert torch.equal(out, shared_decode(r, q, qd, od, sizes, shared, bt, lens, slots))


@pytest.mark.parametrize("sizes,shared,G,fmt,P,d,qd,od", [
    ([40], [60], 8, 1, 64, 128, 1, 0), ([33, 2], [300, 17], 4, 0, 16, 64, 1, 1), ([5, 5, 5], [40, 90, 3], 8, 0, 32, 128, 0, 0),
    ([130], [9], 1, 1, 64, 64, 0, 1), ([2], [700], 2, 0, 16, 128, 1, 0)])
def test_shared_decode_equals_decode(osc, sizes, shared, G, fmt, P, d, qd, od):
    """Rows of more than one tile and prefixes of many splits, against the attention that reads every request's pages."""
    rng = np.random.default_rng([len(sizes), sizes[0], G])
    own = [int(x) for x in rng.integers(0, 5 * P, sum(sizes))]
    rig, bt, slots, lens = family(osc, rng, sizes, shared, own, P=P, d=d, G=G, fmt=fmt)
    with rig as r:
        q = acts(rng, (len(lens), r.heads * G, d), False)
        out = shared_decode(r, q, qd, od, sizes, shared, bt, lens, slots)
        assert r.status() == 0
        want = r.decode(q, qd, 0, bt, lens, slots).double()
        some = sorted({0, sizes[0] - 1, len(lens) - 1})
        within(r, out[some], q[some], qd, od, bt[some], [lens[b] for b in some], [slots[b] for b in some])
        # both evaluations are within their bounds; those of the rows above carry over to the rest, which have the same keys
        scale = want.abs().amax(dim=2, keepdim=True)
        assert ((out.double() - want).abs() <= scale * (2.0 ** -7 if od == 1 else 2.0 ** -15)).all()


@pytest.mark.parametrize("fmt,qd,od", [(0, 1, 1), (1, 1, 0)])
def test_shared_decode_of_many_groups_on_the_same_pages(osc, fmt, qd, od):
    """More groups than a warp has lanes, most of them empty; splits of as many pages as a CTA takes; a page of several groups."""
    rng = np.random.default_rng(9)
    rig, bt, slots, lens = family(osc, rng, [3], [4096], [0, 37, 5], G=2, d=64, fmt=fmt)
    with rig as r:
        q = acts(rng, (3, r.heads * 2, 64), False)
        sizes = [0] * 40 + [1] + [0] * 59 + [2] + [0] * 59
        shared = [7] * 40 + [4096] + [0] * 59 + [4090] + [4096] * 59
        out = shared_decode(r, q, qd, od, sizes, shared, bt, lens, slots)
        assert r.status() == 0
        within(r, out, q, qd, od, bt, lens, slots)


@pytest.mark.parametrize("fmt,qd,od", [(0, 1, 0), (1, 0, 0), (1, 1, 1)])
def test_shared_requests_do_not_depend_on_their_company(osc, fmt, qd, od):
    """A request's output has the same bits wherever it lies in its group."""
    rng = np.random.default_rng(5)
    rig, bt, slots, lens = family(osc, rng, [37], [11], [int(x) for x in rng.integers(0, 50, 37)], G=8, d=128, fmt=fmt)
    with rig as r:
        q = acts(rng, (37, 16, 128), False)
        out = shared_decode(r, q, qd, od, [37], [11], bt, lens, slots)
        turn = rng.permutation(37)
        again = shared_decode(r, q[turn], qd, od, [37], [11], bt[turn], [lens[b] for b in turn], slots[turn])
        assert torch.equal(again, out[torch.from_numpy(turn).cuda()])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("qd", [0, 1])
@pytest.mark.parametrize("loud", [1e-30, 1e-4, 300.0, 1e12])
def test_shared_magnitudes(osc, fmt, qd, loud):
    """Pages far louder or quieter than the next: a row that looks at a quiet page keeps its digits."""
    rng = np.random.default_rng(6)
    rig, bt, slots, lens = family(osc, rng, [2, 1], [9, 9], [7, 33, 1], P=16, d=64, G=2, fmt=fmt)
    with rig as r:
        for g, b in ((0, 0), (1, 2)):
            k, v = r.K[b][:144].copy(), r.V[b][:144].copy()
            v[16 * 3:16 * 5] *= loud
            k[16 * 3:16 * 5] *= min(loud, 4.0)
            r.write([k], [v], 1, [144], [0], bt[b:b + 1], slots[b:b + 1])
            for other in (0, 1) if g == 0 else (2,):
                rest = lens[other] - 144
                r.write([r.K[other][144:]], [r.V[other][144:]], 1, [rest], [144], bt[other:other + 1], slots[other:other + 1])
        q = acts(rng, (3, 4, 64), False)
        out = shared_decode(r, q, qd, 0, [2, 1], [9, 9], bt, lens, slots)
        within(r, out, q, qd, 0, bt, lens, slots)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("qd,od", [(0, 0), (1, 0), (1, 1), (0, 1)])
@pytest.mark.parametrize("loud", [1e6, 1e12, 1e25])
def test_shared_loud_pages_that_no_one_looks_at(osc, fmt, qd, od, loud):
    """Values of any size with weights that vanish leave the digits of the others; a page of zero values counts in the sum alone."""
    rng = np.random.default_rng(61)
    P, d = 16, 128
    rig, bt, slots, lens = family(osc, rng, [3], [24], [0, 5, 20], P=P, d=d, G=2, fmt=fmt)
    with rig as r:
        u = np.zeros((1, 2, d))
        u[..., ::2] = 3.0
        k, v = r.K[0][:384] * 0.3 + u, r.V[0][:384].copy()
        far = np.zeros(384, bool)
        far[32:64] = far[200:240] = True                    # whole pages and, at 200, the middle of them
        k[far] -= 2 * u[0]
        v[far] *= loud
        v[96:112] = 0
        r.write([k], [v], 1, [384], [0], bt[:1], slots[:1])
        for b in (1, 2):
            r.write([r.K[b][384:] * 0.3 + u], [r.V[b][384:]], 1, [lens[b] - 384], [384], bt[b:b + 1], slots[b:b + 1])
        q = acts(rng, (3, 4, d), False) * 0.3
        q[..., ::2] += 5.0                                  # scores of the loud tokens: some 150 below the others
        out = shared_decode(r, q, qd, od, [3], [24], bt, lens, slots)
        assert r.status() == 0
        within(r, out, q, qd, od, bt, lens, slots)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("qd", [0, 1])
@pytest.mark.parametrize("size", [1e3, 1e8, 1e15, 1e30])
def test_shared_where_one_key_leads_by_far(osc, fmt, qd, size):
    """Scores of any size: finite outputs, and the value of the leading key where one leads by more than a float32 score's error."""
    rng = np.random.default_rng(7)
    P, d = 16, 64
    rig, bt, slots, lens = family(osc, rng, [3], [6], [0, 5, 20], P=P, d=d, G=2, fmt=fmt)
    with rig as r:
        k, v = r.K[0][:96] * 0.01, r.V[0][:96]
        k[41] = np.sign(rng.normal(size=k[41].shape)) * 3.0
        r.write([k], [v], 1, [96], [0], bt[:1], slots[:1])
        for b in (1, 2):
            r.write([r.K[b][96:] * 0.01], [r.V[b][96:]], 1, [lens[b] - 96], [96], bt[b:b + 1], slots[b:b + 1])
        q = np.repeat(k[41][None], 3, 0).repeat(2, 1) * size
        out = shared_decode(r, q, qd, 0, [3], [6], bt, lens, slots).double().cpu().numpy()
        assert np.isfinite(out).all()
        for b in range(3):
            for h in range(2):
                want = r.ref.rows(bt[b], slots[b], lens[b], h)[1][41]
                assert np.allclose(out[b, 2 * h:2 * h + 2], want, rtol=0, atol=np.abs(want).max() * 2.0 ** -20)


DTYPES = [(0, 0), (1, 0), (1, 1), (0, 1)]                  # of queries and outputs


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("below,loud,size", [(0.3, 1e6, 1.0), (0.3, 1e10, 1.0), (0.3, 1e13, 1.0), (0.6, 1e20, 1.0), (0.6, 1e23, 1.0),
                                             (2.0, 1e36, 1e-3), (0.9, 1e32, 1e-3), (0.9, 1e34, 1e-3), (0.9, 1e36, 1e-3)])
@pytest.mark.parametrize("zeros", [False, True])
def test_shared_loud_values_of_small_weights(osc, fmt, below, loud, size, zeros):
    """Weights of e^-26 (below = 0.3) to e^-170 on values up to 10^39 times the others': they count for what they are, in a tile with a
    page of zeros too, and a weight of 0 on the largest values is 0."""
    rng = np.random.default_rng(62)
    P, d = 16, 128
    rig, bt, slots, lens = family(osc, rng, [3], [24], [0, 5, 20], P=P, d=d, G=2, fmt=fmt)
    with rig as r:
        u = np.zeros((1, 2, d))
        u[..., ::2] = 3.0
        k, v = r.K[0][:384] * 0.3 + u, r.V[0][:384] * size
        far = np.zeros(384, bool)
        far[32:64] = far[208:240] = True
        k[far] -= below * u[0]
        v[far] *= loud
        if zeros:
            v[96:112] = v[160:176] = 0
        r.write([k], [v], 1, [384], [0], bt[:1], slots[:1])
        for b in (1, 2):
            r.write([r.K[b][384:] * 0.3 + u], [r.V[b][384:] * size], 1, [lens[b] - 384], [384], bt[b:b + 1], slots[b:b + 1])
        q = acts(rng, (3, 4, d), False) * 0.3
        q[..., ::2] += 5.0
        for qd, od in DTYPES:
            within(r, r.decode(q, qd, od, bt, lens, slots), q, qd, od, bt, lens, slots)
            out = shared_decode(r, q, qd, od, [3], [24], bt, lens, slots)
            assert r.status() == 0
            within(r, out, q, qd, od, bt, lens, slots)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("size", [1e-34, 1e-36, 1e-37, 1e-38, 1e36])
def test_shared_values_near_the_ends_of_float32(osc, fmt, size):
    rng = np.random.default_rng(63)
    rig, bt, slots, lens = family(osc, rng, [3], [24], [0, 5, 20], P=16, d=128, G=2, fmt=fmt)
    with rig as r:
        r.write([r.K[0][:384]], [r.V[0][:384] * size], 1, [384], [0], bt[:1], slots[:1])
        for b in (1, 2):
            r.write([r.K[b][384:]], [r.V[b][384:] * size], 1, [lens[b] - 384], [384], bt[b:b + 1], slots[b:b + 1])
        q = acts(rng, (3, 4, 128), False)
        for qd, od in DTYPES:
            within(r, r.decode(q, qd, od, bt, lens, slots), q, qd, od, bt, lens, slots)
            out = shared_decode(r, q, qd, od, [3], [24], bt, lens, slots)
            assert r.status() == 0
            within(r, out, q, qd, od, bt, lens, slots)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rise", [0.05, 0.09, 0.12])
def test_shared_large_values_while_the_reference_lags(osc, fmt, rise):
    """Scores that rise by 4 to 10 after a split's first tiles, on values of 10^35: no sum leaves float32."""
    rng = np.random.default_rng(64)
    P, d, empty = 16, 128, 63                                # (so many groups that a split has all of the prefix)
    sizes, shared = [3] + [0] * empty, [24] + [0] * empty
    rig, bt, slots, lens = family(osc, rng, sizes, shared, [0, 5, 20], P=P, d=d, G=2, fmt=fmt)
    with rig as r:
        u = np.zeros((1, 2, d))
        u[..., ::2] = 3.0
        k, v = r.K[0][:384] * 0.1 + u, r.V[0][:384] * 1e35
        k[128:] += rise * u
        r.write([k], [v], 1, [384], [0], bt[:1], slots[:1])
        for b in (1, 2):
            r.write([r.K[b][384:] * 0.1 + u], [r.V[b][384:] * 1e35], 1, [lens[b] - 384], [384], bt[b:b + 1], slots[b:b + 1])
        q = acts(rng, (3, 4, d), False) * 0.1
        q[..., ::2] += 5.0
        for qd, od in DTYPES:
            within(r, r.decode(q, qd, od, bt, lens, slots), q, qd, od, bt, lens, slots)
            out = shared_decode(r, q, qd, od, sizes, shared, bt, lens, slots)
            assert r.status() == 0
            within(r, out, q, qd, od, bt, lens, slots)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("below", [0.2, 0.5, 0.8, 1.0])
@pytest.mark.parametrize("loud", [1.0, 1e14, 1e30])
def test_shared_leading_pages_of_zeros(osc, monkeypatch, fmt, below, loud):
    """Zero values under scores 17 to 85 above the rest, in the first tiles of a split: the rest keeps its digits, as far as
    float32 has weights.  (Below 2^-126 it has none: that much of every value may be missing.)"""
    bound = O.attend_bound

    def flushed(q, k, v, P):
        want, off = bound(q, k, v, P)
        return want, off + 2.0 ** -126 * np.abs(v).sum(0)

    monkeypatch.setattr(O, "attend_bound", flushed)
    rng = np.random.default_rng(65)
    P, d, empty = 16, 128, 63                                # (so many groups that a split has all of the prefix)
    sizes, shared = [3] + [0] * empty, [32] + [0] * empty
    rig, bt, slots, lens = family(osc, rng, sizes, shared, [0, 5, 20], P=P, d=d, G=2, fmt=fmt)
    with rig as r:
        u = np.zeros((1, 2, d))
        u[..., ::2] = 3.0
        k, v = r.K[0][:512] * 0.1, r.V[0][:512] * loud
        k[:256] += below * u
        v[:256] = 0
        v[400:416] /= loud
        r.write([k], [v], 1, [512], [0], bt[:1], slots[:1])
        for b in (1, 2):
            r.write([r.K[b][512:] * 0.1], [r.V[b][512:]], 1, [lens[b] - 512], [512], bt[b:b + 1], slots[b:b + 1])
        q = acts(rng, (3, 4, d), False) * 0.1
        q[..., ::2] += 5.0
        for qd, od in DTYPES:
            out = shared_decode(r, q, qd, od, sizes, shared, bt, lens, slots)
            assert r.status() == 0
            within(r, out, q, qd, od, bt, lens, slots)


# (token, its key as a share of the leading key, how loud its page's values are) of keys along the queries; the other keys' scores are of ordinary size
FAR = {"between": [(700, 1.0, 1.0)], "at_a_sum": [(512, 1.0, 1.0)], "last": [(1595, 1.0, 1.0)], "first": [(3, 1.0, 1.0)],
       "rises": [(100, 0.5, 1.0), (1000, 1.0, 1.0)], "halves": [(100, 1.0, 1.0), (1000, 0.5, 1.0)],
       "ties": [(300, 1.0, 1.0), (1100, 1.0, 1.0)], "ties_in_a_tile": [(515, 1.0, 1.0), (618, 1.0, 1.0)],
       "louder": [(300, 1.0, 1.0), (1100, 1.0, 50.0)], "quieter": [(300, 1.0, 50.0), (1100, 1.0, 1.0)],
       "unseen_in_a_tile": [(700, 1.0, 1.0), (655, 0.0, 1e12)], "unseen_before": [(700, 1.0, 1.0), (40, 0.0, 1e12)],
       "unseen_after": [(700, 1.0, 1.0), (1400, 0.0, 1e12)], "loud_then_quiet": [(100, 0.5, 1e12), (1000, 1.0, 1.0)],
       "quiet_then_loud": [(100, 0.5, 1e-12), (1000, 1.0, 1.0)]}


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e8, 1e15, 1e30])
@pytest.mark.parametrize("case", list(FAR))
def test_shared_far_scores_in_any_tile(osc, fmt, size, case):
    """A CTA's tiles in turn, scores of ordinary size among very large ones: the output is the value of the leading key, or the mean of
    those that lead alike, whatever the values of the pages without weight.  Off by 2^-20 of the largest.  A BF16 output's weights are
    f16 numbers, off by half a step, 2^-11 of themselves, and their scores' exponents, unless formed from differences (scores of 2^22 in
    log2 on), float32 numbers of the size of the score, off by 2^-24 of it: so the mean of the values v_j is off by
    (2^-11 + ln 2 2^-24 |s|) mean |v_j|, and it is rounded once more, by 2^-8 of what it then is."""
    rng = np.random.default_rng(71)
    P, d, N, empty = 16, 64, 1600, 63                        # (so many groups that a split has all of the prefix)
    sizes, shared = [3] + [0] * empty, [N // P] + [0] * empty
    rig, bt, slots, lens = family(osc, rng, sizes, shared, [0, 5, 20], P=P, d=d, G=2, fmt=fmt)
    with rig as r:
        k, v = r.K[0][:N] * (0.3 / size), r.V[0][:N].copy()
        w = np.sign(rng.normal(size=k[0].shape)) * 3.0
        for t, u, loud in FAR[case]:
            k[t // P * P:t // P * P + P] = 0
            k[t] = u * w
            v[t // P * P:t // P * P + P] *= loud
        r.write([k], [v], 1, [N], [0], bt[:1], slots[:1])
        for b in (1, 2):
            r.write([r.K[b][N:] * (0.3 / size)], [r.V[b][N:]], 1, [lens[b] - N], [N], bt[b:b + 1], slots[b:b + 1])
        q = np.repeat(w[None], 3, 0).repeat(2, 1) * size
        lead = [t for t, u, _ in FAR[case] if u == 1.0]
        for qd, od in DTYPES:
            for out in (r.decode(q, qd, od, bt, lens, slots), shared_decode(r, q, qd, od, sizes, shared, bt, lens, slots)):
                got = out.double().cpu().numpy()
                for b in range(3):
                    for h in range(2):
                        v = r.ref.rows(bt[b], slots[b], lens[b], h)[1][lead]
                        want = v.mean(0)
                        bound = np.abs(want).max() * 2.0 ** -20
                        if od == 1:
                            top = 9 * d * size / np.sqrt(d) * np.log2(np.e)
                            bound = bound + (2.0 ** -11 + np.log(2) * 2.0 ** -24 * top * (top < 2.0 ** 22)) * np.abs(v).mean(0)
                            bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
                        assert np.all(np.abs(got[b, 2 * h:2 * h + 2] - want) <= bound), (b, h)
            assert r.status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("size", [1e3, 1e8, 1e30])
@pytest.mark.parametrize("until", [16, 400, 512, 1584])
@pytest.mark.parametrize("loud", [1.0, 1e12])
def test_shared_far_below_first(osc, fmt, size, until, loud):
    """Tokens whose scores are far below those of the rest come first: nothing of them is left, loud or not."""
    rng = np.random.default_rng(72)
    P, d, N, empty = 16, 64, 1600, 63
    sizes, shared = [3] + [0] * empty, [N // P] + [0] * empty
    rig, bt, slots, lens = family(osc, rng, sizes, shared, [0, 5, 20], P=P, d=d, G=2, fmt=fmt)
    with rig as r:
        k, v = r.K[0][:N] * (0.3 / size), r.V[0][:N].copy()
        w = np.sign(rng.normal(size=k[0].shape)) * 3.0
        k[:until] = -w * (0.5 + 0.5 * rng.random((until, 1, 1)))
        v[:until] *= loud
        r.write([k], [v], 1, [N], [0], bt[:1], slots[:1])
        for b in (1, 2):
            r.write([r.K[b][N:] * (0.3 / size)], [r.V[b][N:]], 1, [lens[b] - N], [N], bt[b:b + 1], slots[b:b + 1])
        q = np.repeat(w[None], 3, 0).repeat(2, 1) * size * (1 + 0.1 * acts(rng, (3, 4, d), False))
        rows = r.ref.rows
        r.ref.rows = lambda *a: [x[until:] for x in rows(*a)]        # (what the other tokens give)
        for qd, od in DTYPES:
            out = shared_decode(r, q, qd, od, sizes, shared, bt, lens, slots)
            assert r.status() == 0
            within(r, out, q, qd, od, bt, lens, slots)


@pytest.mark.parametrize("qd", [0, 1])
def test_shared_decode_carries_nan_in_its_own_row(osc, qd):
    rng = np.random.default_rng(8)
    rig, bt, slots, lens = family(osc, rng, [4], [5], [3, 0, 17, 40], P=16, d=128, G=2, fmt=1)
    with rig as r:
        q = acts(rng, (4, 4, 128), False)
        clean = shared_decode(r, q, qd, 0, [4], [5], bt, lens, slots)
        q2 = q.copy()
        q2[1, 2, 7] = np.nan
        q2[2, 0, 0] = np.inf
        out = shared_decode(r, q2, qd, 0, [4], [5], bt, lens, slots)
        hurt = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
        hurt[1, 2] = hurt[2, 0] = True
        assert torch.isnan(out[1, 2]).all() and torch.isnan(out[2, 0]).any()
        assert torch.equal(out[~hurt], clean[~hurt])


def test_shared_decode_reports_bad_arguments_on_the_device(osc):
    rng = np.random.default_rng(9)
    sizes, shared, own = [3, 2], [6, 4], [3, 0, 17, 40, 5]
    rig, bt, slots, lens = family(osc, rng, sizes, shared, own, P=16, d=64, G=4, fmt=0)
    with rig as r:
        q = acts(rng, (5, 8, 64), False)
        good = shared_decode(r, q, 1, 0, sizes, shared, bt, lens, slots)
        assert r.status() == 0

        def same(out, rows):
            assert torch.equal(out[rows], good[rows])

        short = list(lens)
        short[1] = 6 * 16 - 1                                   # shorter than its group's pages
        out = shared_decode(r, q, 1, 0, sizes, shared, bt, short, slots, max_own=40)
        assert r.status() == osc.DEV_BAD_LEN and not out[1].any()
        same(out, [0, 2, 3, 4])
        out = shared_decode(r, q, 1, 0, sizes, shared, bt, lens, slots, max_own=39)      # one has more of its own
        assert r.status() == osc.DEV_BAD_LEN and not out[3].any()
        same(out, [0, 1, 2, 4])
        neg = list(lens)
        neg[4] = -5
        out = shared_decode(r, q, 1, 0, sizes, shared, bt, neg, slots)
        assert r.status() == osc.DEV_BAD_LEN and not out[4].any()
        same(out, [0, 1, 2, 3])
        out = shared_decode(r, q, 1, 0, sizes, shared, bt, lens, slots, max_shared=5)     # the first group shares more
        assert r.status() == osc.DEV_BAD_LEN and not out[:3].any()
        same(out, [3, 4])
        out = shared_decode(r, q, 1, 0, sizes, shared, bt, lens, slots, starts=[0, 3, 4])  # nobody's request
        assert r.status() == osc.DEV_BAD_LEN and not out[4].any()
        same(out, [0, 1, 2, 3])
        for starts in ([3, 0, 5], [0, 9, 5], [-4, 3, 1 << 30], [5, 5, 5]):                 # no groups at all: flagged, nothing out of range
            shared_decode(r, q, 1, 0, sizes, shared, bt, lens, slots, starts=starts)
            assert r.status() == osc.DEV_BAD_LEN
        out = shared_decode(r, q, 1, 0, sizes, [6, -1], bt, lens, slots)
        assert r.status() == osc.DEV_BAD_LEN and not out[3:].any()
        same(out, [0, 1, 2])
        # an empty first request: the prefix is found through the next one's row
        empty, hole = list(lens), bt.copy()
        empty[0], hole[0] = 0, -1
        out = shared_decode(r, q, 1, 0, sizes, shared, hole, empty, slots)
        assert r.status() == 0 and not out[0].any()
        same(out, [1, 2, 3, 4])
        # a page that is not mapped is left out of every request of its group
        for bad in (-1, r.cfg.num_pages):
            hole = bt.copy()
            hole[:3, 2] = bad
            out = shared_decode(r, q, 1, 0, sizes, shared, hole, lens, slots)
            assert r.status() == osc.DEV_BAD_PAGE
            same(out, [3, 4])
            keep = [0, 1, 3, 4, 5]
            for b in range(3):
                rest = list(range(6, lens[b] // 16))
                want, bound = r.ref.attend(bf16(q)[b], bt[b], slots[b], lens[b], [keep + rest] * 2)
                assert np.all(np.abs(out[b].double().cpu().numpy() - want) <= 2 * bound + 2.0 ** -20 * np.abs(want).max())
        wrong = list(slots)
        wrong[2] = 99
        out = shared_decode(r, q, 1, 0, sizes, shared, bt, lens, wrong)
        assert r.status() == osc.DEV_BAD_SLOT
        same(out, [0, 1, 3, 4])


@pytest.mark.parametrize("word", [0x7fffffff, 0x7fffffe0, 0x40000000, 1 << 20, -0x80000000, -2])
def test_shared_page_counts_of_any_size_are_reported(osc, word):
    """A count of shared pages beyond the bound, to the largest word: the group's requests get zeros, the others what they had."""
    rng = np.random.default_rng(13)
    sizes, shared, own = [3, 2], [6, 4], [3, 0, 17, 40, 5]
    rig, bt, slots, lens = family(osc, rng, sizes, shared, own, P=16, d=64, G=4, fmt=0)
    with rig as r:
        q = acts(rng, (5, 8, 64), False)
        kw = dict(max_shared=6, max_own=40)
        good = shared_decode(r, q, 1, 0, sizes, shared, bt, lens, slots, **kw)
        for at, rows, rest in ((0, [0, 1, 2], [3, 4]), (1, [3, 4], [0, 1, 2])):
            bad = list(shared)
            bad[at] = word
            out = shared_decode(r, q, 1, 0, sizes, bad, bt, lens, slots, **kw)
            assert r.status() == osc.DEV_BAD_LEN and not out[rows].any()
            assert torch.equal(out[rest], good[rest])


def test_shared_workspace_serves_a_shrinking_batch(osc):
    """One workspace of the largest batch's size, as requests finish and groups end: the same bits as with one of the call's own."""
    rng = np.random.default_rng(14)
    sizes, shared = [24, 5, 3], [300, 300, 40]
    own = [int(x) for x in rng.integers(0, 90, 32)]
    rig, bt, slots, lens = family(osc, rng, sizes, shared, own, P=16, d=64, G=8, fmt=0)
    with rig as r:
        o, q = osc, r.rows(acts(rng, (32, 16, 64), False), 1)
        bounds = dict(max_shared=300, max_own=96)
        size = o.oscar_kv8_shared_workspace_size(r.cfg, 32, 3, 300, 96)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        for left in ([24, 5, 3], [24, 5], [24], [17], [16], [9], [4], [1]):
            B, n = sum(left), len(left)
            want = shared_decode(r, q[:B], 1, 0, left, shared[:n], bt[:B], lens[:B], slots[:B], **bounds)
            got = torch.full_like(want, 5.0)
            t = dev(bt[:B])
            o.oscar_kv8_shared_decode_attn(r.ctx, r.layer, q[:B], 1, got, 0, dev(np.concatenate([[0], np.cumsum(left)])), dev(shared[:n]),
                                           n, 300, t, t.shape[1], dev(lens[:B]), dev(slots[:B]), B, 96, ws, size)
            assert r.status() == 0 and torch.equal(got, want)


def test_shared_graphs_and_streams(osc):
    """Captured once and replayed on new inputs; two graphs with one workspace replayed in turn; two streams at once."""
    rng = np.random.default_rng(10)
    sizes, shared, own = [5, 3], [20, 33], [int(x) for x in rng.integers(0, 60, 8)]
    rig, bt, slots, lens = family(osc, rng, sizes, shared, own, P=16, d=128, G=8, fmt=1)
    with rig as r:
        o, cfg, B = osc, r.cfg, 8
        q = [acts(rng, (B, 16, 128), False) for _ in range(4)]
        want = [shared_decode(r, x, 1, 0, sizes, shared, bt, lens, slots) for x in q]
        size = o.oscar_kv8_shared_workspace_size(cfg, B, 2, 33, 64)
        qt = [torch.zeros(B, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        out = [torch.zeros(B, 16, 128, device="cuda") for _ in range(2)]
        ws = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
        st, sh, t, n, sl = dev(np.concatenate([[0], np.cumsum(sizes)])), dev(shared), dev(bt), dev(lens), dev(slots)
        call = lambda i, w, s=None: o.oscar_kv8_shared_decode_attn(   # noqa: E731
            r.ctx, r.layer, qt[i], 1, out[i], 0, st, sh, 2, 33, t, t.shape[1], n, sl, B, 64, ws[w], size, s)
        call(0, 0)
        torch.cuda.synchronize()
        graphs = []
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(i, 0)
            graphs.append(g)
        close = lambda a, b: ((a - b).abs() <= 2.0 ** -18 * b.abs().amax(dim=2, keepdim=True)).all()   # noqa: E731  (splits by max_own)
        for k in range(4):
            qt[k % 2].copy_(r.rows(q[k], 1))
            graphs[k % 2].replay()
            torch.cuda.synchronize()
            assert close(out[k % 2], want[k])
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(20):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    call(i, i)
        torch.cuda.synchronize()
        assert close(out[0], want[2]) and close(out[1], want[3]) and r.status() == 0


# ------------------------------------------------------------------------------------------------ the next beams
class Chooser:
    def __init__(self, osc):
        self.osc = osc
        cfg = osc.make_config(num_layers=1, n_q_heads=1, n_kv_heads=1, head_dim=64, page_size=16, sink=0, recent=1, max_requests=1,
                              max_pages_per_req=1, num_pages=1)
        self.pool = torch.zeros(osc.oscar_kv8_pool_bytes(cfg), dtype=torch.uint8, device="cuda")
        self.tail = torch.zeros(osc.oscar_kv8_tail_bytes(cfg), dtype=torch.uint8, device="cuda")
        self.ctx = osc.oscar_create(cfg)
        osc.oscar_kv8_bind(self.ctx, 0, self.pool, self.tail)

    def __call__(self, x, scores, n_out, finished=None, pad=0, stream=None):
        """x [batch][beams][vocab] (a CUDA tensor), scores [batch][beams]."""
        o, (B, K, V) = self.osc, x.shape
        dt = o.DTYPE_BF16 if x.dtype == torch.bfloat16 else o.DTYPE_F32
        size = o.oscar_beam_select_workspace_size(B, K, V, n_out)
        ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device="cuda")
        key = torch.full((B + 1, n_out), 5.0, device="cuda")
        tok, par = (torch.full((B + 1, n_out), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        s = torch.as_tensor(np.asarray(scores, np.float32)).cuda()
        f = None if finished is None else torch.as_tensor(np.asarray(finished, np.uint8)).cuda()
        o.oscar_beam_select(self.ctx, x, dt, s, f, pad, B, K, V, n_out, key, tok, par, ws, size, stream)
        assert (key[B] == 5).all() and (tok[B] == -9).all() and (par[B] == -9).all()
        return key[:B].cpu().numpy(), tok[:B].cpu().numpy(), par[:B].cpu().numpy()

    def check(self, x, scores, n_out, finished=None, pad=0):
        got = self(x, scores, n_out, finished, pad)
        xs = x.double().cpu().numpy()
        for b in range(x.shape[0]):
            want = OB.select(xs[b], np.asarray(scores, np.float32)[b], n_out, None if finished is None else finished[b], pad)
            some = want[1] >= 0
            assert np.array_equal(got[2][b] >= 0, some) and np.array_equal(got[1][b] >= 0, some)
            assert np.all(got[0][b][~some] == -np.inf)
            off = np.abs(got[0][b][some] - want[0][some])
            assert np.all(off <= 1e-6 + np.abs(want[0][some]) * 2.0 ** -24), (b, off.max())
            diff = (got[1][b] != want[1]) | (got[2][b] != want[2])
            if diff.any():     # only candidates of different beams that are closer than the normalisers are known
                key = want[0][diff]
                near = np.abs(want[0][:, None] - key) + 10.0 * (want[2][:, None] == want[2][diff]) <= 2e-6
                assert np.all(near.any(0)), (b, want, got[1][b], got[2][b])

    def status(self):
        return self.osc.oscar_check_status(self.ctx)


@pytest.fixture(scope="module")
def choose(osc):
    c = Chooser(osc)
    yield c
    torch.cuda.synchronize()
    osc.oscar_destroy(c.ctx)


def logits(rng, B, K, V, dtype):
    x = rng.normal(size=(B, K, V)) * 2 - 2 * np.log1p(np.arange(V) / 50.0) + rng.normal(size=(B, 1, V)) * 2
    return torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()


BOTH = [torch.float32, torch.bfloat16]


def test_choice_refusals(osc, choose):
    o, x, f = osc, torch.zeros(2, 3, 50, device="cuda"), torch.zeros(2, 3, device="cuda")
    fin = torch.zeros(2, 3, dtype=torch.uint8, device="cuda")
    out, tok, par = torch.zeros(2, 4, device="cuda"), dev(np.zeros((2, 4))), dev(np.zeros((2, 4)))
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    good = (choose.ctx, x, 0, f, fin, 0, 2, 3, 50, 4, out, tok, par, ws, 4096)
    before = o.oscar_launch_count(choose.ctx)
    for at, value in [(1, None), (1, x.cpu()), (1, x[:1]), (1, x.to(torch.bfloat16)), (1, x[:, :, ::2]), (2, 3), (3, None), (3, f[:1]),
                      (3, f.double()), (4, fin.int()), (4, fin[:1]), (5, -1), (5, 50), (6, -1), (6, 65536), (7, 0), (7, 65), (8, 0),
                      (8, (1 << 24) + 1), (9, 0), (9, 65), (10, None), (10, out[:1]), (10, x.view(-1)[:8]), (10, f.view(-1)[:6]), (11, None),
                      (11, tok.float()), (12, None), (12, par[:1]), (13, None), (13, ws[8:]), (14, 8), (14, -1)]:
        a = list(good)
        a[at] = value
        with pytest.raises(o.OscarError) as e:
            o.oscar_beam_select(*a)
        assert e.value.status in (o.ERR_INVALID, o.ERR_UNSUPPORTED), (at, value)
    with pytest.raises(o.OscarError):    # outputs over inputs
        o.oscar_beam_select(*good[:3], out.view(-1)[:6], *good[4:])
    a = list(good)
    a[6] = 0
    o.oscar_beam_select(*a)
    assert o.oscar_launch_count(choose.ctx) == before
    assert choose.status() == 0


def test_choice_outputs_and_workspace_over_one_another_are_refused(osc, choose):
    o, B, K, V, N = osc, 2, 3, 2000, 4
    size = o.oscar_beam_select_workspace_size(B, K, V, N)
    room = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    at = lambda i, n, t: room[i:i + n].view(t)  # noqa: E731
    f, i4 = torch.float32, torch.int32
    good = [choose.ctx, at(0, 4 * B * K * V, f).view(B, K, V), 0, at(48128, 4 * B * K, f), None, 0, B, K, V, N, at(48640, 32, f), at(48672, 32, i4),
            at(48704, 32, i4), at(48896, size, torch.uint8), size]
    before = o.oscar_launch_count(choose.ctx)
    for where, value in [(11, at(48704, 32, i4)), (11, at(48660, 32, i4)), (12, at(48640, 32, i4)), (10, at(48700, 32, f)), (12, at(48900, 32, i4)),
                         (10, at(48896 + size - 4, 32, f)), (13, at(48640, size, torch.uint8)), (13, at(47872, size, torch.uint8)),
                         (13, at(48128, size, torch.uint8)), (4, at(48640, B * K, torch.uint8)), (4, at(48896, B * K, torch.uint8))]:
        a = list(good)
        a[where] = value
        with pytest.raises(o.OscarError, match="overlap") as e:
            o.oscar_beam_select(*a)
        assert e.value.status == o.ERR_INVALID
    assert o.oscar_launch_count(choose.ctx) == before
    o.oscar_beam_select(*good)                               # next to one another is fine
    assert o.oscar_launch_count(choose.ctx) == before + 2 and choose.status() == 0


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("B,K,V,n_out", [(1, 1, 1, 1), (1, 1, 1, 4), (2, 2, 7, 4), (1, 2, 997, 2), (3, 5, 1024, 10), (2, 4, 1025, 8), (2, 3, 4097, 64),
                                         (1, 64, 333, 64), (2, 8, 32768, 16), (1, 5, 50021, 10), (1, 1, 131072, 1), (1, 4, 300001, 8)])
def test_choice(choose, dtype, B, K, V, n_out):
    rng = np.random.default_rng([B, K, V, n_out])
    choose.check(logits(rng, B, K, V, dtype), -20 * rng.random((B, K)), n_out)
    assert choose.status() == 0


@pytest.mark.parametrize("dtype", BOTH)
def test_choice_of_a_first_step(choose, dtype):
    rng = np.random.default_rng(1)
    s = np.full((3, 4), -np.inf)
    s[:, 0] = 0
    choose.check(logits(rng, 3, 1, 5000, dtype).expand(3, 4, 5000).contiguous(), s, 8)
    assert (choose(logits(rng, 3, 4, 5000, dtype), np.full((3, 4), -np.inf), 8)[1] == -1).all()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("V,n_out", [(3, 9), (2000, 12), (50021, 64)])
def test_equal_candidates_come_in_order(choose, dtype, V, n_out):
    """All logits equal, rows and scores equal: the lowest (beam, token) first; and whole numbers, where ties are everywhere."""
    key, tok, par = choose(torch.zeros(2, 3, V, dtype=dtype, device="cuda"), np.zeros((2, 3)), n_out)
    want = np.arange(n_out)
    assert np.array_equal(tok, np.tile(want % V, (2, 1))) and np.array_equal(par, np.tile(want // V, (2, 1)))
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.integers(-3, 4, (2, 1, V)).astype(np.float32)).to(dtype).cuda().expand(2, 3, V).contiguous()
    choose.check(x, np.full((2, 3), -1.5), n_out)
    choose.check(x, np.array([[-3.0, -2.0, -1.0]] * 2), n_out)
    low = torch.finfo(dtype).min
    key, tok, par = choose(torch.full((1, 2, V), low, dtype=dtype, device="cuda"), np.zeros((1, 2)), 2)
    assert tok.tolist() == [[0, 1]] and np.allclose(key, -np.log(V), atol=1e-5)       # masks of the lowest value leave an even choice


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("kept", [0.0, 0.0005, 0.3])
def test_masked_tokens_are_never_taken(choose, dtype, kept):
    rng = np.random.default_rng(3)
    x = logits(rng, 2, 4, 6001, dtype)
    x[torch.from_numpy(rng.random(x.shape) >= kept).cuda()] = -torch.inf
    x[0, 2] = -torch.inf                               # a row without tokens
    x[1, 1, :] = -torch.inf
    x[1, 1, 6000] = 3.0                                # and one with a single token: probability 1
    choose.check(x, -rng.random((2, 4)), 16)
    assert choose.status() == 0


@pytest.mark.parametrize("dtype", BOTH)
def test_finished_beams_keep_their_score(choose, dtype):
    rng = np.random.default_rng(4)
    x, s = logits(rng, 3, 4, 2500, dtype), -20 * rng.random((3, 4))
    fin = np.array([[0, 1, 0, 1], [1, 1, 1, 1], [0, 0, 0, 0]])
    s[1, 2] = -np.inf
    x[0, 1] = torch.nan                                # not read
    for pad in (0, 1234, 2499):
        choose.check(x, s, 6, fin, pad)
    assert choose.status() == 0
    same = np.zeros((1, 3))                            # equal scores: in the order of the beams
    assert choose(x[:1, :3], same, 3, np.ones((1, 3)), 7)[2].tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_bad_beams_are_left_out_and_reported(choose, osc, dtype, bad):
    rng = np.random.default_rng(5)
    for at in (0, 1023, 2000, 2999):
        x = logits(rng, 2, 3, 3000, dtype)
        x[1, 2, at] = bad
        choose.check(x, -rng.random((2, 3)), 6)
        assert choose.status() == osc.DEV_BAD_VALUE
    s = -rng.random((2, 3))
    s[0, 1] = bad
    choose.check(logits(rng, 2, 3, 3000, dtype), s, 6)
    assert choose.status() == osc.DEV_BAD_VALUE


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("gap,skip", [(0, 0), (8, 0), (1, 0), (13, 3), (5, 1)])
@pytest.mark.parametrize("V", [9, 4100, 20011])
def test_choice_from_rows_of_any_alignment(choose, dtype, gap, skip, V):
    """The same rows at other addresses give the same bits, at the start and the end of an allocation too."""
    rng = np.random.default_rng(6)
    x, s = logits(rng, 2, 3, V, dtype), -rng.random((2, 3))
    want = choose(x, s, 7)
    flat = torch.full((6 * (V + gap) + skip,), torch.inf, dtype=dtype, device="cuda")[:skip + 5 * (V + gap) + V]
    at = flat.as_strided((2, 3, V), (3 * (V + gap), V + gap, 1), skip)
    at.copy_(x)
    got = choose(at, s, 7)
    assert all(np.array_equal(a, b) for a, b in zip(want, got)) and choose.status() == 0


def test_wide_range_of_logits(choose):
    rng = np.random.default_rng(7)
    for scale in (1e-30, 1e-3, 1e3, 1e30):
        choose.check(torch.from_numpy((rng.normal(size=(2, 3, 3000)) * scale).astype(np.float32)).cuda(), -rng.random((2, 3)), 8)
    x = rng.normal(size=(1, 2, 3000)).astype(np.float32)
    choose.check(torch.from_numpy(x + np.array([[[1000.0], [-1e5]]], np.float32)).cuda(), np.zeros((1, 2)), 8)


def test_scores_and_logits_near_the_largest_float32(choose):
    """score - top is below float32's range where every key is inside it."""
    x = np.zeros((1, 2, 40), np.float32)
    x[0, 0] = 1.9e38
    x[0, 0, 5] = 2e38
    choose.check(torch.from_numpy(x).cuda(), [[-2e38, -3e38]], 4)
    choose.check(torch.from_numpy(x[:, ::-1].copy()).cuda(), [[-3e38, -2e38]], 4)
    wide = np.zeros((1, 3, 5000), np.float32)
    wide[0, 1], wide[0, 1, 4000:] = 1.9e38, 2e38
    choose.check(torch.from_numpy(wide).cuda(), [[-3e38, -2e38, -3.2e38]], 64)


def test_rising_rows_and_one_beam_that_leads(choose):
    x = torch.linspace(-5, 5, 60000, device="cuda").expand(1, 3, 60000).contiguous()
    choose.check(x, [[0.0, -0.5, -1.0]], 32)                    # all of a beam's candidates in its last chunk
    choose.check(x.flip(2).contiguous(), [[0.0, -0.5, -1.0]], 32)
    choose.check(x, [[0.0, -50.0, -100.0]], 64)


def test_choice_graphs_and_streams(osc, choose):
    rng = np.random.default_rng(8)
    o, B, K, V, N = osc, 2, 3, 9001, 6
    x = [logits(rng, B, K, V, torch.bfloat16) for _ in range(3)]
    s = torch.from_numpy(-rng.random((B, K)).astype(np.float32)).cuda()
    want = [choose(y, s.cpu().numpy(), N) for y in x]
    size = o.oscar_beam_select_workspace_size(B, K, V, N)
    buf = [torch.zeros_like(x[0]) for _ in range(2)]
    ws = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [(torch.zeros(B, N, device="cuda"), dev(np.zeros((B, N))), dev(np.zeros((B, N)))) for _ in range(2)]
    call = lambda i, w: o.oscar_beam_select(choose.ctx, buf[i], 1, s, None, 0, B, K, V, N, *out[i], ws[w], size)   # noqa: E731
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, 0)
        graphs.append(g)
    for k in range(3):
        buf[k % 2].copy_(x[k])
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(out[k % 2], want[k]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                call(i, i)
    torch.cuda.synchronize()
    for i, k in ((0, 2), (1, 1)):
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(out[i], want[k]))


# ------------------------------------------------------------------------------------------------ reordering
def reorder(r, parents, bt, lens, slots, batch, beams):
    o, rows = r.osc, batch * beams
    new = [torch.full((rows + 1, bt.shape[1]), 77, dtype=torch.int32, device="cuda")] + \
        [torch.full((rows + 1,), 77, dtype=torch.int32, device="cuda") for _ in range(2)]
    o.oscar_kv8_reorder(r.ctx, dev(parents), batch, beams, dev(bt), bt.shape[1], dev(lens), dev(slots), *new)
    assert all((x[rows] == 77).all() for x in new)
    return [x[:rows].cpu().numpy() for x in new]


def reorder_oracle(parents, bt, lens, slots, tail, P, batch, beams):
    got = [np.empty_like(x) for x in (bt, lens, slots)]
    for b in range(batch):
        at = slice(b * beams, (b + 1) * beams)
        for to, x in zip(got, OB.reorder(np.asarray(parents).reshape(batch, beams)[b], bt[at], lens[at], slots[at], tail, P)):
            to[at] = x
    return got


def test_reorder_refusals(osc):
    with Rig(osc) as r:
        o = osc
        i = [dev(np.zeros(24)) for _ in range(8)]
        good = (r.ctx, i[0], 2, 2, i[1], 6, i[2], i[3], i[4], i[5], i[6])
        before = o.oscar_launch_count(r.ctx)
        for at, value in [(1, None), (1, i[0][:3]), (1, i[0].long()), (2, -1), (2, 40000), (3, 0), (3, 65), (4, None), (4, i[1][:23]), (5, 0), (6, None),
                          (7, None), (8, None), (8, i[1]), (9, None), (9, i[2]), (9, i[0]), (10, None), (10, i[3]), (10, i[1][20:])]:
            a = list(good)
            a[at] = value
            with pytest.raises(o.OscarError) as e:
                o.oscar_kv8_reorder(*a)
            assert e.value.status in (o.ERR_INVALID, o.ERR_UNSUPPORTED), at
        a = list(good)
        a[2] = 0
        o.oscar_kv8_reorder(*a)
        assert o.oscar_launch_count(r.ctx) == before


def test_reorder_outputs_over_one_another_are_refused(osc):
    with Rig(osc) as r:
        o = osc
        i, room = [dev(np.zeros(24)) for _ in range(8)], dev(np.zeros(64))
        good = (r.ctx, i[0], 2, 2, i[1], 6, i[2], i[3], room[:24], room[24:28], room[28:32])
        before = o.oscar_launch_count(r.ctx)
        for at, value in [(9, room[:4]), (9, room[23:27]), (10, room[12:16]), (10, room[24:28]), (10, room[27:31]), (10, room[21:25]), (8, room[8:32])]:
            a = list(good)
            a[at] = value
            with pytest.raises(o.OscarError, match="overlap") as e:
                o.oscar_kv8_reorder(*a)
            assert e.value.status == o.ERR_INVALID
        assert o.oscar_launch_count(r.ctx) == before
        o.oscar_kv8_reorder(*good)                           # next to one another is fine
        assert o.oscar_launch_count(r.ctx) == before + 1 and r.status() == 0


@pytest.mark.parametrize("P,d", GEO)
@pytest.mark.parametrize("batch,beams,layers", [(1, 1, 1), (1, 3, 2), (3, 4, 5), (2, 64, 1)])
def test_reorder(osc, P, d, batch, beams, layers):
    rng = np.random.default_rng([P, d, batch, beams])
    rows = batch * beams
    with Rig(osc, P=P, d=d, layers=layers, layer=0, slots=rows + 3, oracle=False) as r:
        for kind in range(4):
            r.tail.copy_(torch.randn(r.tail.shape, device="cuda"))
            lens = rng.integers(0, 12 * P + 1, rows).astype(np.int32)
            slots, bt = rng.permutation(rows + 3)[:rows].astype(np.int32), rng.integers(-1, 99, (rows, 13)).astype(np.int32)
            parents = [rng.integers(-1, beams, (batch, beams)), np.stack([rng.permutation(beams) for _ in range(batch)]),
                       np.full((batch, beams), beams - 1), np.full((batch, beams), -1)][kind]
            tail = r.tail.float().cpu().numpy()
            got = reorder(r, parents, bt, lens, slots, batch, beams)
            want = reorder_oracle(parents, bt, lens, slots, tail, P, batch, beams)
            assert all(np.array_equal(a, b) for a, b in zip(got, want))
            assert np.array_equal(r.tail.float().cpu().numpy(), tail)          # every other row as it was
            assert r.status() == 0


def test_reorder_reports_bad_arguments_on_the_device(osc):
    rng = np.random.default_rng(1)
    P = 16
    with Rig(osc, P=P, slots=6, oracle=False) as r:
        r.tail.copy_(torch.randn(r.tail.shape, device="cuda"))
        bt, lens, slots = rng.integers(0, 9, (4, 5)).astype(np.int32), np.array([5, 20, 33, 7], np.int32), np.array([5, 0, 3, 2], np.int32)
        tail = r.tail.float().cpu().numpy()
        got = reorder(r, [4, 1, -2, 1], bt, lens, slots, 1, 4)
        assert r.status() == osc.DEV_BAD_SLOT
        want = reorder_oracle([-1, 1, -1, 1], bt, lens, slots, tail, P, 1, 4)
        assert all(np.array_equal(a, b) for a, b in zip(got, want)) and np.array_equal(r.tail.float().cpu().numpy(), tail)
        for bad in (6, -1, 1 << 30):
            s = slots.copy()
            s[0] = bad                                       # the slot that the second child of beam 1 would take
            got = reorder(r, [1, 1, 2, 3], bt, lens, s, 1, 4)
            assert r.status() == osc.DEV_BAD_SLOT and got[2].tolist() == [0, bad, 3, 2]
            assert np.array_equal(r.tail.float().cpu().numpy(), tail)
        for bad in (-3, 12 * P + 1):
            n = lens.copy()
            n[1] = bad
            reorder(r, [1, 1, 2, 3], bt, n, slots, 1, 4)
            assert r.status() == osc.DEV_BAD_LEN
            assert np.array_equal(r.tail.float().cpu().numpy(), tail)


def test_reorder_reports_states_that_do_not_move(osc):
    """A length or slot out of range is reported where no row is copied too: with a parent's only child, and with the slot of an empty beam."""
    rng = np.random.default_rng(2)
    P = 16
    with Rig(osc, P=P, slots=6, oracle=False) as r:
        r.tail.copy_(torch.randn(r.tail.shape, device="cuda"))
        bt, lens, slots = rng.integers(0, 9, (4, 5)).astype(np.int32), np.array([5, 20, 33, 32], np.int32), np.array([5, 0, 3, 2], np.int32)
        tail = r.tail.float().cpu().numpy()
        for parents in ([0, 1, 2, 3], [3, 2, 1, 0], [2, -1, 3, 1]):
            got = reorder(r, parents, bt, lens, slots, 1, 4)
            assert r.status() == 0
            for bad in (6, -1, 1 << 30):
                s = slots.copy()
                s[0 if -1 in parents else 2] = bad           # (beam 0's slot goes to the empty beam)
                got = reorder(r, parents, bt, lens, s, 1, 4)
                assert r.status() == osc.DEV_BAD_SLOT
                want = reorder_oracle(parents, bt, lens, s, tail.copy(), P, 1, 4)
                assert all(np.array_equal(a, b) for a, b in zip(got, want))
            for bad in (-3, 12 * P + 1):
                n = lens.copy()
                n[2] = bad
                got = reorder(r, parents, bt, n, slots, 1, 4)
                assert r.status() == osc.DEV_BAD_LEN
                want = reorder_oracle(parents, bt, n, slots, tail.copy(), P, 1, 4)
                assert all(np.array_equal(a, b) for a, b in zip(got, want))
            assert np.array_equal(r.tail.float().cpu().numpy(), tail)
        n, s = lens.copy(), slots.copy()                     # tails of no rows: nothing would be copied, the states are bad all the same
        n[3], s[0] = 32, 6
        reorder(r, [3, 3, 1, 2], bt, n, s, 1, 4)
        assert r.status() == osc.DEV_BAD_SLOT
        n[3], s[0] = -16, 5
        reorder(r, [3, 3, 1, 2], bt, n, s, 1, 4)
        assert r.status() == osc.DEV_BAD_LEN
        n[0], n[3] = -1, 32                                  # a childless beam's length is nobody's
        reorder(r, [3, 3, 1, 2], bt, n, s, 1, 4)
        assert r.status() == 0 and np.array_equal(r.tail.float().cpu().numpy(), tail)


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt,G", [(0, 4), (1, 8)])
def test_beam_search_run(osc, fmt, G):
    """Two prompts forked into four beams, searched for many steps across page borders: append, shared decode, choice, reordering.  Every beam's
    attention equals that of a request with the same history in a cache of its own; the allocator ends where it began."""
    rng = np.random.default_rng(11)
    P, d, heads, layers, K, prompt = 16, 64, 2, 2, 4, [85, 40]
    B, steps, V = 2, 40, 300
    rows = B * K
    with Rig(osc, fmt=fmt, P=P, d=d, heads=heads, G=G, layers=layers, layer=1, slots=rows, per_req=12, pages=90, oracle=False) as r:
        o, per = osc, 12
        free0 = o.oscar_free_page_count(r.ctx)
        hist = []                                            # every beam's tokens: (K, V) rows [tokens][heads][d]
        bt = np.full((rows, per), -1, np.int32)
        slots = rng.permutation(rows).astype(np.int32)
        for b, n in enumerate(prompt):
            kv = [bf16(acts(rng, (n, heads, d))) for _ in range(2)]
            pages = o.oscar_alloc_pages(r.ctx, n // P)
            bt[b * K, :n // P] = pages
            for layer in range(layers):
                k, v = (r.rows(x, 1) for x in kv)
                o.oscar_kv8_write(r.ctx, layer, k, v, 1, dev([0, n]), dev([0]), 1, n, dev(bt[b * K:b * K + 1]), per, dev(slots[b * K:b * K + 1]))
            table = o.oscar_kv8_fork(r.ctx, list(pages), n, int(slots[b * K]), slots[b * K + 1:(b + 1) * K], per)
            bt[b * K + 1:(b + 1) * K] = table
            hist += [[kv[0].copy(), kv[1].copy()] for _ in range(K)]
        shared, starts = [n // P for n in prompt], [0, K, 2 * K]
        lens = np.repeat(prompt, K).astype(np.int32)
        scores = np.full((B, K), -np.inf, np.float32)
        scores[:, 0] = 0
        c = Chooser(osc)
        emb = bf16(acts(rng, (V, 2, heads, d)))              # what a token appends
        proj = rng.normal(size=(heads * G * d, V)) / np.sqrt(d)
        q0 = acts(rng, (rows, heads * G, d), False)
        tokens = np.zeros((B, K), int)
        dbt, dn, dsl = dev(bt), dev(lens), dev(slots)
        nbt, nn, nsl = torch.empty_like(dbt), torch.empty_like(dn), torch.empty_like(dsl)
        most_own = steps + P
        size = o.oscar_kv8_shared_workspace_size(r.cfg, rows, B, max(shared), most_own)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        out = torch.zeros(rows, heads * G, d, device="cuda")
        copies = 0
        for step in range(steps):
            new = emb[tokens.reshape(-1)] + (0.01 * step)
            new = bf16(new)
            # a page for every beam whose page this token completes
            if ((lens + 1) % P == 0).any():
                for j in np.flatnonzero((lens + 1) % P == 0):
                    bt[j, lens[j] // P] = o.oscar_alloc_pages(r.ctx, 1)[0]
                dbt.copy_(dev(bt))
            for layer in range(layers):
                o.oscar_kv8_append(r.ctx, layer, r.rows(new[:, 0], 1), r.rows(new[:, 1], 1), 1, dn, rows, dbt, per, dsl)
            dn += 1
            lens = lens + 1
            for j in range(rows):
                hist[j] = [np.concatenate([hist[j][i], new[j:j + 1, i]]) for i in range(2)]
            q = np.cos(step) * q0 + np.sin(step) * np.roll(q0, 3, axis=2)
            o.oscar_kv8_shared_decode_attn(r.ctx, 1, r.rows(q, 1), 1, out, 0, dev(starts), dev(shared), B, max(shared), dbt, per, dn, dsl,
                                           rows, most_own, ws, size)
            got = out.double().cpu().numpy()
            if step % 6 == 0 or step == steps - 1:
                for j in range(rows):
                    ref = O.Cache(P, d, heads, fmt, np.zeros((per, heads, r.block), np.uint8), np.zeros((1, heads, 2, P, d)))
                    ref.write(list(range(per)), 0, 0, *hist[j])
                    want, bound = ref.attend(bf16(q)[j], list(range(per)), 0, int(lens[j]))
                    assert np.all(np.abs(got[j] - want) <= 2 * bound + 2.0 ** -20 * np.abs(want).max()), (step, j)
            x = torch.from_numpy((got.reshape(rows, -1) @ proj + 3 * np.cos(np.arange(V) * (step + 1) + tokens.reshape(-1, 1))).astype(np.float32))
            x = x.to(torch.bfloat16).cuda().view(B, K, V)
            c.check(x, scores, K)
            key, tok, par = c(x, scores, K)
            o.oscar_kv8_reorder(r.ctx, dev(par), B, K, dbt, per, dn, dsl, nbt, nn, nsl)
            (dbt, nbt), (dn, nn), (dsl, nsl) = (nbt, dbt), (nn, dn), (nsl, dsl)
            # the host's books: tables, lengths, references
            old = bt.copy()
            flat = (np.arange(B)[:, None] * K + par).reshape(-1)
            kids = np.bincount(flat, minlength=rows)
            for j in range(rows):
                mine = [int(p) for p in old[j] if p >= 0]
                for _ in range(kids[j] - 1):
                    o.oscar_ref_pages(r.ctx, mine)
                copies += max(kids[j] - 1, 0)
            for j in np.flatnonzero(kids == 0):
                o.oscar_unref_pages(r.ctx, [int(p) for p in old[j] if p >= 0])
            bt, lens, hist = old[flat], lens[flat], [[x.copy() for x in hist[j]] for j in flat]
            assert np.array_equal(dbt.cpu().numpy(), bt) and np.array_equal(dn.cpu().numpy(), lens)
            assert sorted(dsl.cpu().numpy().tolist()) == list(range(rows))
            scores, tokens = key, tok
        assert r.status() == 0 and copies > rows
        for j in range(rows):
            o.oscar_unref_pages(r.ctx, [int(p) for p in bt[j] if p >= 0])
        assert o.oscar_free_page_count(r.ctx) == free0
        torch.cuda.synchronize()
        o.oscar_destroy(c.ctx)


def test_kernel_times_and_launches_by_name(osc, choose):
    rng = np.random.default_rng(12)
    rig, bt, slots, lens = family(osc, rng, [3], [4], [0, 5, 20], P=16, d=64, G=2, fmt=0)
    with rig as r:
        q = acts(rng, (3, 4, 64), False)
        want = shared_decode(r, q, 1, 0, [3], [4], bt, lens, slots)
        before = osc.oscar_launch_count(r.ctx)
        osc.oscar_set_timing(r.ctx, True)
        osc.oscar_reset_timing(r.ctx)
        got = shared_decode(r, q, 1, 0, [3], [4], bt, lens, slots)
        reorder(r, [2, 0, 2], bt, np.asarray(lens, np.int32), slots.astype(np.int32), 1, 3)
        assert torch.equal(got, want)
        for name in ("kv8_decode", "kv8_prefix", "kv8_combine", "kv8_reorder"):
            ms, n = osc.oscar_kernel_time(r.ctx, name)
            assert n == 1 and 0 < ms < 100, name
        osc.oscar_set_timing(r.ctx, False)
        assert osc.oscar_launch_count(r.ctx) == before + 4
    before = osc.oscar_launch_count(choose.ctx)
    osc.oscar_set_timing(choose.ctx, True)
    choose(logits(rng, 1, 2, 500, torch.float32), np.zeros((1, 2)), 2)
    assert [osc.oscar_kernel_time(choose.ctx, n)[1] for n in ("beam_units", "beam_pick")] == [1, 1]
    osc.oscar_set_timing(choose.ctx, False)
    osc.oscar_reset_timing(choose.ctx)
    assert osc.oscar_launch_count(choose.ctx) == before + 2
