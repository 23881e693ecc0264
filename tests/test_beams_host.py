"""Beam search and shared prefixes on the CPU: oracle pins, sizes and refusals (no kernel runs)."""
import ctypes

import numpy as np
import pytest

from oracle import beams as OB
from tests.test_kv8_host import Elsewhere, _cfg


@pytest.fixture(scope="module")
def osc():
    from int2_rotated_paged_oscar_gb300 import build
    build.build()
    import int2_rotated_paged_oscar_gb300 as m
    m.load()
    return m


# ------------------------------------------------------------------------------------------------ oracle pins
def test_candidates_are_log_probabilities():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.125, 0.125, 0.75]]))
    key, tok, par = OB.select(x, [0.0, -1.0], 4)
    assert tok.tolist() == [0, 2, 1, 2] and par.tolist() == [0, 1, 0, 0]
    assert np.allclose(np.exp(key), [0.5, 0.75 / np.e, 0.25, 0.25])


def test_masked_finished_and_bad_beams():
    x = np.zeros((4, 3))
    x[0, 1:] = -np.inf
    x[1] = -np.inf
    x[3, 0] = np.nan
    key, tok, par = OB.select(x, [-5.0, 0.0, -2.0, 0.0], 4, finished=[0, 0, 1, 0], pad=2)
    assert tok.tolist() == [2, 0, -1, -1] and par.tolist() == [2, 0, -1, -1] and key[:2].tolist() == [-2.0, -5.0]


@pytest.mark.parametrize("parents,want", [
    ([0, 1, 2], [(0, 0), (1, 0), (2, 0)]), ([2, 0, 1], [(2, 0), (0, 0), (1, 0)]), ([1, 1, 1], [(1, 0), (0, 1), (2, 1)]),
    ([2, 2, 0, 0], [(2, 0), (1, 1), (0, 0), (3, 1)]), ([-1, 3, -1, 3], [(0, 0), (3, 0), (1, 0), (2, 1)]), ([-1, -1], [(0, 0), (1, 0)])])
def test_places(parents, want):
    assert [(k, int(c)) for k, c in OB.places(parents)] == want
    assert sorted(k for k, _ in OB.places(parents)) == list(range(len(parents)))


# ------------------------------------------------------------------------------------------------ sizes, refusals
def test_workspace_sizes(osc):
    c = _cfg(osc)
    shared = osc.oscar_kv8_shared_workspace_size
    assert shared(c, 3, 1, 4, 30) >= 3 * 8 * 2 * 68 * 4 and shared(c, 0, 0, 0, 0) >= 0
    for bad in ((-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1), (1, 1, 1, -1), (1, 1, 13, 1), (1, 1, 1, 12 * 16 + 1)):
        with pytest.raises(osc.OscarError) as e:
            shared(c, *bad)
        assert e.value.status == osc.ERR_INVALID
    with pytest.raises(osc.OscarError) as e:
        shared(c, 1, 65536, 1, 1)
    assert e.value.status == osc.ERR_UNSUPPORTED
    beam = osc.oscar_beam_select_workspace_size
    assert beam(2, 3, 1000, 3) >= 2 * 3 * 8 and beam(0, 1, 1, 1) == 0
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0)):
        with pytest.raises(osc.OscarError) as e:
            beam(*bad)
        assert e.value.status == osc.ERR_INVALID
    for big in ((65536, 1, 1, 1), (1, 65, 1, 1), (1, 1, (1 << 24) + 1, 1), (1, 1, 1, 65)):
        with pytest.raises(osc.OscarError) as e:
            beam(*big)
        assert e.value.status == osc.ERR_UNSUPPORTED
    lib = osc.load()
    assert lib.oscar_beam_select_workspace_size(1, 1, 1, 1, None) == osc.ERR_INVALID
    assert lib.oscar_kv8_shared_workspace_size(ctypes.byref(c), 1, 1, 1, 1, None) == osc.ERR_INVALID


@pytest.mark.parametrize("heads,G,d,P", [(8, 8, 128, 64), (2, 4, 64, 16), (8, 4, 128, 64), (1, 8, 128, 16), (8, 1, 64, 32)])
@pytest.mark.parametrize("shared,own", [(0, 0), (1, 5), (128, 300), (512, 1024), (4096, 9000)])
def test_a_workspace_serves_fewer_requests_and_groups(osc, heads, G, d, P, shared, own):
    """A smaller batch is split into more parts; the size covers every smaller batch and every smaller number of groups."""
    cfg = osc.make_config(num_layers=1, n_q_heads=heads * G, n_kv_heads=heads, head_dim=d, page_size=P, sink=0, recent=1, max_requests=4,
                          max_pages_per_req=4096, num_pages=4)
    size = lambda b, n: osc.oscar_kv8_shared_workspace_size(cfg, b, n, shared, own)  # noqa: E731
    batches, groups = [*range(1, 70), 127, 128, 129, 160, 255, 256, 257, 300], [1, 2, 3, 4, 7, 12, 13, 16, 19, 20, 33, 64]
    table = np.array([[size(b, n) for n in groups] for b in batches], dtype=np.int64)
    assert (np.diff(table, axis=0) >= 0).all() and (np.diff(table, axis=1) >= 0).all()
    # a place of (m, l, O) for every query head at least, in the prefix and in a request's own part
    assert (table >= np.array(batches)[:, None] * heads * G * 2 * (d + 4) * 4).all()
    assert size(1, 1) <= size(2, 0) <= size(2, 1)             # (no group counts as one)


@pytest.mark.parametrize("beams", [1, 2, 7, 64])
@pytest.mark.parametrize("vocab", [1, 1024, 1025, 50021, 131072, 1 << 24])
def test_the_workspace_holds_two_numbers_for_every_1024_logits(osc, beams, vocab):
    for n_out in (1, 16, 64):
        assert osc.oscar_beam_select_workspace_size(3, beams, vocab, n_out) == 3 * beams * -(-vocab // 1024) * 8


def test_calls_without_a_bound_cache_are_refused(osc):
    lib = osc.load()
    ctx = osc.oscar_create(_cfg(osc))
    try:
        assert lib.oscar_kv8_shared_decode_attn(ctx, 0, 256, 0, 1, 256, 1, 256, 256, 1, 1, 256, 1, 256, 256, 1, 16, 256, 1 << 20,
                                                None) == osc.ERR_INVALID
        assert lib.oscar_kv8_reorder(ctx, 256, 1, 2, 256, 1, 256, 256, 512, 768, 1024, None) == osc.ERR_INVALID
        assert "oscar_kv8_bind" in lib.oscar_last_error().decode()
        assert lib.oscar_beam_select(ctx, 256, 0, 1, 256, None, 0, 1, 1, 8, 1, 1024, 2048, 4096, 256, 1 << 20, None) == osc.ERR_INVALID
        assert "device buffers" in lib.oscar_last_error().decode()
    finally:
        osc.oscar_destroy(ctx)
    assert lib.oscar_kv8_reorder(None, 256, 1, 2, 256, 1, 256, 256, 512, 768, 1024, None) == osc.ERR_INVALID
    assert lib.oscar_beam_select(None, 256, 0, 1, 256, None, 0, 1, 1, 8, 1, 1024, 2048, 4096, 256, 64, None) == osc.ERR_INVALID


def test_tensors_on_another_device_are_refused(osc):
    torch = pytest.importorskip("torch")
    ctx = osc.oscar_create(_cfg(osc))
    try:
        osc._configs[ctx].device = 0
        ints, byte, f = torch.zeros(12, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8), torch.zeros(4)
        q, x = torch.zeros(1, 8, 64), torch.zeros(1, 2, 30)
        F32 = osc.DTYPE_F32
        calls = ((osc.oscar_kv8_shared_decode_attn, [0, q, F32, q, F32, ints, ints, 1, 2, ints, 12, ints, ints, 1, 100, byte, 64], "no 8-bit"),
                 (osc.oscar_kv8_reorder, [ints, 1, 2, ints, 6, ints, ints, ints, ints, ints], "no 8-bit"),
                 (osc.oscar_beam_select, [x, F32, f, byte, 0, 1, 2, 30, 2, f, ints, ints, byte, 64], "device buffers"))
        for call, args, why in calls:
            on = [Elsewhere(a, 0) if torch.is_tensor(a) else a for a in args]
            with pytest.raises(osc.OscarError, match=why):
                call(ctx, *on, stream=256)
            for i, a in enumerate(args):
                if torch.is_tensor(a):
                    with pytest.raises(osc.OscarError, match="device 0"):
                        call(ctx, *on[:i], Elsewhere(a, 1), *on[i + 1:], stream=256)
    finally:
        osc.oscar_destroy(ctx)


def test_logits_of_other_shapes_and_strides_are_refused(osc):
    torch = pytest.importorskip("torch")
    on = lambda t: Elsewhere(t, 0)  # noqa: E731
    F32, BF16 = osc.DTYPE_F32, osc.DTYPE_BF16
    wide = torch.zeros(3, 2, 40)
    assert osc._logits(on(wide), 0, F32, 3, 2, 40)[1] == 40
    assert osc._logits(on(wide[:, :, :33]), 0, F32, 3, 2, 33)[1] == 40
    assert osc._logits(on(wide[:, :1]), 0, F32, 3, 1, 40)[1] == 80         # a beam each: rows 80 apart
    assert osc._logits(on(wide.reshape(6, 40)), 0, F32, 3, 2, 40)[1] == 40
    assert osc._logits(on(wide.reshape(6, 40)), 0, F32, 2, 2, 40)[1] == 40  # some of the rows
    assert osc._logits(on(wide[:1, :1]), 0, F32, 1, 1, 40)[1] == 0
    for batch, beams in ((1, 6), (6, 1), (2, 3), (1, 1)):                    # rows of other beams
        with pytest.raises(osc.OscarError):
            osc._logits(on(wide), 0, F32, batch, beams, 40)
    for bad in (wide[:, :, ::2], wide.transpose(1, 2), wide[:, :1].expand(3, 2, 40), wide[:2], torch.zeros(3, 3, 40)[:, :2],
                wide.to(torch.bfloat16), wide.reshape(-1), torch.zeros(60).as_strided((3, 2, 40), (8, 4, 1))):
        with pytest.raises(osc.OscarError):
            osc._logits(on(bad), 0, F32, 3, 2, bad.shape[-1] if bad.shape[-1] == 20 else 40)
    with pytest.raises(osc.OscarError):
        osc._logits(on(wide), 0, BF16, 3, 2, 40)
