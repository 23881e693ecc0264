"""8-bit cache on the CPU: oracle pins, sizes, refusals, and the host part of forks and compaction (no kernel runs)."""
import numpy as np
import pytest

from oracle import kv8 as O


@pytest.fixture(scope="module")
def osc():
    from int2_rotated_paged_oscar_gb300 import build
    build.build()
    import int2_rotated_paged_oscar_gb300 as m
    m.load()
    return m


def _cfg(osc, **kw):
    base = dict(num_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16, sink=0, recent=1, max_requests=6,
                max_pages_per_req=12, num_pages=40)
    base.update(kw)
    return osc.make_config(**base)


# ------------------------------------------------------------------------------------------------ oracle pins
def test_code_values():
    v = O.code_values(O.E4M3)
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7E] == 448.0 and v[0xFE] == -448.0
    assert np.all(np.diff(v[:127]) > 0) and np.isnan(v[127])
    assert O.code_values(O.INT8)[[1, 128, 255]].tolist() == [-127, 0, 127]


@pytest.mark.parametrize("fmt", [O.INT8, O.E4M3])
def test_encode_takes_the_nearest_code(fmt):
    rng = np.random.default_rng(0)
    x = rng.normal(size=(16, 64)) * np.exp(rng.normal(size=64))
    x = (x.astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)
    code, scale = O.encode(x, fmt)
    v = O.code_values(fmt)
    v = v[np.isfinite(v) & (np.abs(v) <= O.TOP[fmt])]
    y = x * O.TOP[fmt] / np.abs(x).max()
    best = np.abs(y[..., None] - v).min(-1)
    assert np.allclose(np.abs(y - O.code_values(fmt)[code]), best, rtol=0, atol=1e-12)
    assert np.abs(O.code_values(fmt)[code]).max() == O.TOP[fmt] and scale == np.float32(np.abs(x).max()) / np.float32(O.TOP[fmt])


def test_encode_ties_go_to_the_even_code():
    x = np.zeros((1, 64))
    x[0, :5] = [448, 17, 19, -17, 2.0 ** -10]          # E4M3 has 16, 18, 20 here, and 0 and 2^-9 around 2^-10
    code, scale = O.encode(x, O.E4M3)
    assert scale == 1 and O.code_values(O.E4M3)[code][0, :5].tolist() == [448, 16, 20, -16, 0]
    x[0, :4] = [127, 0.5, 1.5, -2.5]
    x[0, 4] = 0
    assert (O.encode(x, O.INT8)[0][0, :4].astype(int) - 128).tolist() == [127, 0, 2, -2]


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_places_are_a_bijection_within_lines(P, d):
    for is_v in (False, True):
        at = O.place(P, d, is_v)
        assert sorted(at.reshape(-1)) == list(range(P * d))
        assert np.array_equal(at // 128, (np.arange(P)[:, None] * d + np.arange(d)) // 128)


def test_bound_is_an_upper_bound_of_the_scores():
    rng = np.random.default_rng(1)
    P, d, heads, G = 16, 64, 2, 4
    c = O.Cache(P, d, heads, O.E4M3, np.zeros((5, heads, O.block_bytes(P, d)), np.uint8), np.zeros((1, heads, 2, P, d)))
    c.write([3, 1, 4, 0], 0, 0, rng.normal(size=(64, heads, d)), rng.normal(size=(64, heads, d)))
    q = rng.normal(size=(heads * G, d))
    for h in range(heads):
        u = c.bounds(q[h * G:(h + 1) * G], [3, 1, 4, 0], 64, h)
        k, _ = c.rows([3, 1, 4, 0], 0, 64, h)
        s = (q[h * G:(h + 1) * G] @ k.T).reshape(G, 4, P).max(2).sum(0)
        assert np.all(u >= s - 1e-9)


def test_arrival_order_does_not_matter_to_the_oracle():
    rng = np.random.default_rng(2)
    P, d, heads, n = 16, 64, 1, 53
    K, V = rng.normal(size=(2, n, heads, d))
    make = lambda: O.Cache(P, d, heads, O.INT8, np.zeros((4, heads, O.block_bytes(P, d)), np.uint8), np.zeros((1, heads, 2, P, d)))  # noqa: E731
    a, b = make(), make()
    a.write([2, 0, 3], 0, 0, K, V)
    b.write([2, 0, 3], 0, 0, K[:20], V[:20])
    for t in range(20, n):
        b.write([2, 0, 3], 0, t, K[t:t + 1], V[t:t + 1], append=True)
    assert np.array_equal(a.pool, b.pool) and np.array_equal(a.tail[..., :n % P, :], b.tail[..., :n % P, :])


# ------------------------------------------------------------------------------------------------ sizes, refusals
def test_sizes(osc):
    c = _cfg(osc)
    assert osc.oscar_kv8_block_bytes(c) == O.block_bytes(16, 64) == 2304
    assert osc.oscar_kv8_pool_bytes(c) == 2 * 40 * 2 * 2304
    assert osc.oscar_kv8_tail_bytes(c) == 2 * 6 * 2 * 2 * 16 * 64 * 2
    big = _cfg(osc, head_dim=128, page_size=64, n_q_heads=64, n_kv_heads=8)
    assert osc.oscar_kv8_block_bytes(big) == O.block_bytes(64, 128) == 16768
    assert [osc.oscar_kv8_pages_needed(c, n) for n in (0, 15, 16, 17, 160)] == [0, 0, 1, 1, 10]
    assert osc.oscar_kv8_pages_needed(c, -1) == -1
    bad = _cfg(osc, head_dim=96)
    assert osc.oscar_kv8_pool_bytes(bad) == osc.oscar_kv8_tail_bytes(bad) == osc.oscar_kv8_block_bytes(bad) == 0


def test_workspace_sizes(osc):
    c = _cfg(osc)
    for f in (osc.oscar_kv8_decode_workspace_size, osc.oscar_kv8_select_workspace_size):
        with pytest.raises(osc.OscarError):
            f(c, -1, 10)
        with pytest.raises(osc.OscarError):
            f(c, 1, -1)
        with pytest.raises(osc.OscarError):
            f(_cfg(osc, page_size=8), 1, 10)
    with pytest.raises(osc.OscarError):
        osc.oscar_kv8_sparse_workspace_size(c, 1, 0)
    with pytest.raises(osc.OscarError) as e:
        osc.oscar_kv8_sparse_workspace_size(c, 1, (1 << 24) + 1)
    assert e.value.status == osc.ERR_UNSUPPORTED
    assert osc.oscar_kv8_decode_workspace_size(c, 3, 100) >= 3 * 8 * 68 * 4
    assert osc.oscar_kv8_decode_workspace_size(c, 0, 100) >= 0


def test_calls_without_a_bound_cache_are_refused(osc):
    ctx = osc.oscar_create(_cfg(osc))
    try:
        lib = osc.load()
        calls = [
            lib.oscar_kv8_write(ctx, 0, 256, 0, 256, 0, 1, 256, 256, 1, 1, 256, 1, 256, None),
            lib.oscar_kv8_append(ctx, 0, 256, 0, 256, 0, 1, 256, 1, 256, 1, 256, None),
            lib.oscar_kv8_decode_attn(ctx, 0, 256, 0, 1, 256, 1, 256, 1, 256, 256, 1, 16, 256, 1 << 20, None),
            lib.oscar_kv8_select_pages(ctx, 0, 256, 0, 1, 256, 1, 256, 1, 16, 0, 0, 1, 256, 256, 1 << 20, None),
            lib.oscar_kv8_sparse_decode_attn(ctx, 0, 256, 0, 1, 256, 1, 256, 1, 256, 1, 256, 256, 1, 256, 1 << 20, None)]
        assert calls == [osc.ERR_INVALID] * 5
        assert "oscar_kv8_bind" in lib.oscar_last_error().decode()
        assert lib.oscar_check_status(ctx, None, None) == osc.ERR_INVALID
    finally:
        osc.oscar_destroy(ctx)
    assert osc.load().oscar_kv8_append(None, 0, 256, 0, 256, 0, 1, 256, 1, 256, 1, 256, None) == osc.ERR_INVALID


@pytest.mark.parametrize("fmt,pool,tail", [(2, 256, 256), (-1, 256, 256), (0, None, 256), (0, 256, None), (0, 264, 256),
                                           (1, 256, 8)])
def test_bind_refusals(osc, fmt, pool, tail):
    ctx = osc.oscar_create(_cfg(osc))
    try:
        with pytest.raises(osc.OscarError) as e:
            osc.oscar_kv8_bind(ctx, fmt, pool, tail)
        assert e.value.status == osc.ERR_INVALID
    finally:
        osc.oscar_destroy(ctx)
    with pytest.raises(osc.OscarError):
        osc.oscar_kv8_bind(ctx, 0, 256, 256)      # destroyed


def test_tensors_on_the_host_are_refused(osc):
    torch = pytest.importorskip("torch")
    c = _cfg(osc)
    ctx = osc.oscar_create(c)
    try:
        t = torch.zeros(osc.oscar_kv8_pool_bytes(c), dtype=torch.uint8)
        with pytest.raises(osc.OscarError):
            osc.oscar_kv8_bind(ctx, osc.KV8_INT8, t, t)
        rows, ints = torch.zeros(1, 2, 64), torch.zeros(4, dtype=torch.int32)
        with pytest.raises(osc.OscarError):
            osc.oscar_kv8_append(ctx, 0, rows, rows, osc.DTYPE_F32, ints, 1, ints, 1, ints, stream=256)
    finally:
        osc.oscar_destroy(ctx)


class Elsewhere:
    """What the binding asks of a tensor, on the given CUDA device."""

    def __init__(self, t, device):
        self.t, self.device, self.is_cuda = t, f"cuda:{device}", True
        self.get_device = lambda: device

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_tensors_on_another_device_are_refused(osc):
    torch = pytest.importorskip("torch")
    ctx = osc.oscar_create(_cfg(osc))
    try:
        osc._configs[ctx].device = 0              # as after a bind on device 0; the library has no cache, so it refuses all
        rows, ints, byte = torch.zeros(1, 2, 64), torch.zeros(12, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
        q = torch.zeros(1, 8, 64)
        calls = (
            (osc.oscar_kv8_write, [rows, rows, osc.DTYPE_F32, ints, ints, 1, 1, ints, 12, ints]),
            (osc.oscar_kv8_append, [rows, rows, osc.DTYPE_F32, ints, 1, ints, 12, ints]),
            (osc.oscar_kv8_decode_attn, [q, osc.DTYPE_F32, q, osc.DTYPE_F32, ints, 12, ints, ints, 1, 100, byte, 64]),
            (osc.oscar_kv8_select_pages, [q, osc.DTYPE_F32, ints, 12, ints, 1, 100, 0, 0, 2, ints, byte, 64]),
            (osc.oscar_kv8_sparse_decode_attn, [q, osc.DTYPE_F32, q, osc.DTYPE_F32, ints, 2, ints, 12, ints, ints, 1, byte, 64]))
        for call, args in calls:
            on = [Elsewhere(x, 0) if torch.is_tensor(x) else x for x in args]
            with pytest.raises(osc.OscarError, match="no 8-bit cache"):
                call(ctx, 0, *on, stream=256)
            for i, x in enumerate(args):
                if torch.is_tensor(x):
                    with pytest.raises(osc.OscarError, match="device 0"):
                        call(ctx, 0, *on[:i], Elsewhere(x, 1), *on[i + 1:], stream=256)
        with pytest.raises(osc.OscarError, match="device 0"):
            osc.oscar_compact_pages(ctx, Elsewhere(ints, 1), 1, 12, osc._configs[ctx].num_pages, stream=0)
    finally:
        osc.oscar_destroy(ctx)


@pytest.mark.parametrize("layout", ["broadcast", "overlapping"])
def test_rows_that_share_memory_are_refused(osc, layout):
    """One row for every token (the step after a fork, say) has a token stride of 0, which means adjacent rows to the library:
    it would read past the tensor's end.  A single token has no such stride."""
    torch = pytest.importorskip("torch")
    ctx = osc.oscar_create(_cfg(osc))
    try:
        osc._configs[ctx].device = 0
        on = lambda x: Elsewhere(x, 0)  # noqa: E731

        def rows(n, heads):
            one = torch.zeros(1, heads, 64)
            return on(one.expand(n, heads, 64) if layout == "broadcast" else
                      torch.zeros(4 * n + heads * 64).as_strided((n, heads, 64), (4, 64, 1)))

        i, t, byte = on(torch.zeros(12, dtype=torch.int32)), on(torch.zeros(72, dtype=torch.int32)), on(torch.zeros(64, dtype=torch.uint8))
        f32 = osc.DTYPE_F32

        def calls(B):
            kv, q, good = rows(B, 2), rows(B, 8), on(torch.zeros(B, 8, 64))
            good_kv = on(torch.zeros(B, 2, 64))
            return ((osc.oscar_kv8_write, (kv, good_kv, f32, i, i, 1, B, t, 12, i)), (osc.oscar_kv8_write, (good_kv, kv, f32, i, i, 1, B, t, 12, i)),
                    (osc.oscar_kv8_append, (kv, good_kv, f32, i, B, t, 12, i)), (osc.oscar_kv8_append, (good_kv, kv, f32, i, B, t, 12, i)),
                    (osc.oscar_kv8_decode_attn, (q, f32, good, f32, t, 12, i, i, B, 100, byte, 64)),
                    (osc.oscar_kv8_select_pages, (q, f32, t, 12, i, B, 100, 0, 0, 1, t, byte, 64)),
                    (osc.oscar_kv8_sparse_decode_attn, (q, f32, good, f32, t, 1, t, 12, i, i, B, byte, 64)))

        for call, args in calls(5):
            with pytest.raises(osc.OscarError, match="elements apart"):
                call(ctx, 0, *args, stream=256)
        for call, args in calls(1):
            with pytest.raises(osc.OscarError, match="no 8-bit cache"):
                call(ctx, 0, *args, stream=256)
        assert osc._rows(rows(5, 2), "K", 0, f32, 1, 2, 64)[1] == 0         # one of several rows is read
    finally:
        osc.oscar_destroy(ctx)


def test_negative_workspace_sizes_are_refused(osc):
    """As a size_t a negative number of bytes is a very large one, and no buffer would be too small for the library."""
    torch = pytest.importorskip("torch")
    ctx = osc.oscar_create(_cfg(osc))
    try:
        osc._configs[ctx].device = 0
        q, i, byte = (Elsewhere(x, 0) for x in (torch.zeros(1, 8, 64), torch.zeros(12, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)))
        f32 = osc.DTYPE_F32
        for ws in (byte, 256):
            for call, args in ((osc.oscar_kv8_decode_attn, (q, f32, q, f32, i, 12, i, i, 1, 100, ws)),
                               (osc.oscar_kv8_select_pages, (q, f32, i, 12, i, 1, 100, 0, 0, 2, i, ws)),
                               (osc.oscar_kv8_sparse_decode_attn, (q, f32, q, f32, i, 2, i, 12, i, i, 1, ws))):
                with pytest.raises(osc.OscarError, match="no 8-bit cache"):
                    call(ctx, 0, *args, 64, stream=256)
                for bad in (-1, -64, -(1 << 40)):
                    with pytest.raises(osc.OscarError, match="workspace cannot have"):
                        call(ctx, 0, *args, bad, stream=256)
    finally:
        osc.oscar_destroy(ctx)


def test_long_lists_of_pages_take_what_short_ones_take(osc):
    np = pytest.importorskip("numpy")
    torch = pytest.importorskip("torch")
    want = list(range(20))
    for seq in (want, tuple(want), np.arange(20), np.arange(20, dtype=np.int16), torch.arange(20), [np.int64(i) for i in want],
                list(torch.arange(20)), range(20), [float(i) for i in want]):
        assert list(osc._i32_array(seq)) == want


# ------------------------------------------------------------------------------------------------ host part of page moves
def test_fork_shares_complete_pages(osc):
    ctx = osc.oscar_create(_cfg(osc))
    try:
        src = osc.oscar_alloc_pages(ctx, 4)
        t = osc.oscar_kv8_fork(ctx, src, 16 * 3 + 5, 0, [2, 4], 12, stream=0)
        assert t.shape == (2, 12) and np.array_equal(t[0], t[1])
        assert t[0, :3].tolist() == src[:3] and np.all(t[0, 3:] == -1)
        assert [osc.oscar_page_refcount(ctx, p) for p in src] == [3, 3, 3, 1]
        assert osc.oscar_kv8_fork(ctx, src, 5, 0, [1], 12, stream=0).tolist() == [[-1] * 12]
        assert osc.oscar_kv8_fork(ctx, [], 0, 0, [1], 12, stream=0).tolist() == [[-1] * 12]
        assert osc.oscar_kv8_fork(ctx, src, 16, 0, [], 12, stream=0).shape == (0, 12)
        for bad in (dict(n=-1), dict(n=16 * 12 + 1), dict(src_slot=6), dict(src_slot=-1), dict(dst_slots=[6]), dict(dst_slots=[-1]),
                    dict(dst_slots=[2, 2]), dict(dst_slots=[0]), dict(src_bt=src[:2]), dict(src_bt=[src[0], 99, src[2]]),
                    dict(src_bt=[src[0], 39, src[2]]), dict(max_pages=11)):
            kw = dict(src_bt=src, n=48, src_slot=0, dst_slots=[1], max_pages=12, stream=0) | bad
            with pytest.raises(osc.OscarError):
                osc.oscar_kv8_fork(ctx, **kw)
        assert [osc.oscar_page_refcount(ctx, p) for p in src] == [3, 3, 3, 1]
    finally:
        osc.oscar_destroy(ctx)


def test_compaction_plan(osc):
    ctx = osc.oscar_create(_cfg(osc))
    try:
        ids = osc.oscar_alloc_pages(ctx, 40)
        rng = np.random.default_rng(3)
        gone = sorted(rng.permutation(40)[:23].tolist())
        keep = [i for i in ids if i not in gone]
        osc.oscar_ref_pages(ctx, [keep[-1], keep[-1]])
        osc.oscar_unref_pages(ctx, gone)
        table, live = osc.oscar_compact_pages(ctx, None, 0, 1, 40, stream=0)
        assert live == 17 and sorted(table[keep].tolist()) == list(range(17)) and np.all(table[gone] == -1)
        assert all(table[i] == i for i in keep if i < 17)
        assert osc.oscar_page_refcount(ctx, int(table[keep[-1]])) == 3
        assert sum(osc.oscar_page_refcount(ctx, i) for i in range(40)) == 19
        assert osc.oscar_free_page_count(ctx) == 23 and osc.oscar_alloc_pages(ctx, 2) == [17, 18]
        again, live = osc.oscar_compact_pages(ctx, None, 0, 1, 40, stream=0)
        assert live == 19 and again.tolist() == list(range(19)) + [-1] * 21     # nothing moves
        osc.oscar_unref_pages(ctx, [i for i in range(19) for _ in range(osc.oscar_page_refcount(ctx, i))])
        empty, live = osc.oscar_compact_pages(ctx, None, 0, 1, 40, stream=0)
        assert live == 0 and np.all(empty == -1)
        with pytest.raises(osc.OscarError):
            osc.oscar_compact_pages(ctx, None, 0, 1, 39, stream=0)
        with pytest.raises(osc.OscarError):
            osc.oscar_compact_pages(ctx, None, 2, 4, 40, stream=0)
        with pytest.raises(osc.OscarError):
            osc.oscar_compact_pages(ctx, 256, 2, 4, 40, stream=0)               # a table, but no device buffers
    finally:
        osc.oscar_destroy(ctx)


def test_failed_launches_leave_pages_and_tables_as_they_were(tmp_path):
    """Compactions of more pages than one launch takes, each launch of one failing in turn, and a fork whose copy fails."""
    import os
    import shutil
    import subprocess
    from int2_rotated_paged_oscar_gb300 import build
    here = os.path.dirname(os.path.abspath(__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc())))
    program = tmp_path / "page_moves"
    r = subprocess.run([shutil.which("g++"), "-std=c++17", "-O1", "-I", os.path.join(cuda, "include"), "-o", str(program),
                        os.path.join(here, "page_moves_host.cpp"), os.path.join(build.CSRC, "kv8_abi.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
