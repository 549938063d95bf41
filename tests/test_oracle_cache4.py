"""Pins of the oracle's rotary positions and 4-bit cache, and the library's parts of them that need no GPU:
frequencies, page sizes and refusals."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import cache4, rotary

FAKE, WS, BIG = 0x1000, 0x10000, 1 << 40


@pytest.fixture(scope="module")
def lib():
    from serving_draft_verify_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    from serving_draft_verify_gb300 import _binding
    return _binding.load()


# ------------------------------------------------------------------ rotary ---
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    r = np.random.default_rng(0)
    x, freq, pos = r.normal(size=(5, 2, 16)), np.array([1.0, 0.3, 0.01, 2.0]), np.array([0, 1, 7, 100, 12345])
    y = rotary.rotate(x, pos, freq, interleaved, magnitude=1.25)
    pair = (lambda a: a[..., 0:8:2] + 1j * a[..., 1:8:2]) if interleaved else (lambda a: a[..., :4] + 1j * a[..., 4:8])
    want = 1.25 * pair(x) * np.exp(1j * pos[:, None] * freq)[:, None]
    np.testing.assert_allclose(pair(y), want, atol=1e-11)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    np.testing.assert_array_equal(y[0, :, 8:], x[0, :, 8:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_transposed_rotation_is_the_gradient(interleaved):
    """Inner products with a rotated row, as a function of the row, by central differences."""
    r = np.random.default_rng(1)
    x, dy = r.normal(size=(3, 1, 12)), r.normal(size=(3, 1, 12))
    freq, pos = np.array([0.7, 0.1, 0.02, 1.3]), np.array([3, 50, 999])
    got = rotary.rotate(dy, pos, freq, interleaved, transposed=True, magnitude=0.8)
    for n in range(3):
        for d in range(12):
            e = np.zeros_like(x)
            e[n, 0, d] = 1e-4
            f = lambda z: (rotary.rotate(z, pos, freq, interleaved, magnitude=0.8) * dy).sum()  # noqa: E731
            assert abs((f(x + e) - f(x - e)) / 2e-4 - got[n, 0, d]) < 1e-8
    back = rotary.rotate(rotary.rotate(x, pos, freq, interleaved), pos, freq, interleaved, transposed=True)
    np.testing.assert_allclose(back, x, atol=1e-12)


def test_scores_depend_on_distances():
    r = np.random.default_rng(2)
    q, k, freq = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8)), np.array([1.0, 0.5, 0.1, 0.003])
    s = [float((rotary.rotate(q, [n + 17], freq) * rotary.rotate(k, [n], freq)).sum()) for n in (0, 5, 1000)]
    np.testing.assert_allclose(s, s[0], atol=1e-11)
    assert np.isnan(rotary.rotate(q, [-1], freq)).all()


def test_frequencies_closed_forms():
    f, m = rotary.frequencies(8, 1e4)
    np.testing.assert_allclose(f, [1, 0.1, 0.01, 0.001])
    assert m == 1
    np.testing.assert_allclose(rotary.frequencies(8, 1e4, "linear", 4)[0], f / 4)
    base = rotary.frequencies(8, 1e4, "base", 16)[0]
    np.testing.assert_allclose(base[[0, 3]], [1, f[3] / 16])        # the last pair slows by the whole factor
    bands, _ = rotary.frequencies(8, 1e4, "bands", 8, original=8192, low=1, high=4)
    np.testing.assert_allclose(bands[:3], f[:3])                    # 1304, 130 and 13 turns
    keep = (8192 * 0.001 / (2 * np.pi) - 1) / 3
    np.testing.assert_allclose(bands[3], f[3] * (keep + (1 - keep) / 8))
    ramp, m = rotary.frequencies(128, 1e4, "ramp", 4, original=4096)
    f = rotary.frequencies(128, 1e4)[0]
    # turns over 4096 positions: pair 20 more than 32, pair 46 fewer than 1
    np.testing.assert_allclose(ramp[:21], f[:21])
    np.testing.assert_allclose(ramp[46:], f[46:] / 4)
    assert (np.diff(ramp) < 0).all() and abs(m - (0.1 * np.log(4) + 1)) < 1e-15


@pytest.mark.parametrize("rot,base,scaling,kw", [
    (128, 1e6, "plain", {}), (64, 1e4, "linear", dict(factor=8)), (96, 5e5, "base", dict(factor=3.5)),
    (128, 1e6, "ramp", dict(factor=4, original=32768, low=1, high=32)), (32, 1e4, "ramp", dict(factor=40, original=4096)),
    (16, 1e4, "ramp", dict(factor=2, original=10.0)), (128, 5e5, "bands", dict(factor=8, original=8192, low=1, high=4)),
    (2, 1e4, "plain", {}), (256, 1e6, "bands", dict(factor=2.5, original=1000, low=0.5, high=0.75))])
def test_frequencies(lib, rot, base, scaling, kw):
    import serving_draft_verify_gb300 as dsv
    freq, m = dsv.dspark_rotary_frequencies(rot, base, scaling, device="cpu", **kw)
    want, wm = rotary.frequencies(rot, base, scaling, **kw)
    # rounded once to float32; the doubles before it within 2^-45
    np.testing.assert_allclose(freq.double().numpy(), want, rtol=2.0 ** -24 + 2.0 ** -45)
    assert abs(m - wm) <= 2.0 ** -24 * wm


def test_frequencies_refusals(lib):
    f, buf = lib.dspark_rotary_frequencies, (ctypes.c_float * 128)()
    ok = dict(rot=64, base=1e4, scaling=3, factor=4.0, original=4096.0, low=1.0, high=32.0, freq=ctypes.addressof(buf), m=None)
    assert f(*ok.values()) == 0
    nan, inf = float("nan"), float("inf")
    for bad in (dict(rot=0), dict(rot=63), dict(rot=258), dict(base=1.0), dict(base=nan), dict(base=inf), dict(scaling=-1),
                dict(scaling=5), dict(factor=0.5), dict(factor=nan), dict(factor=inf), dict(original=0.0), dict(original=nan),
                dict(original=inf), dict(low=0.0), dict(low=32.0), dict(high=inf), dict(high=nan), dict(freq=None),
                dict(scaling=2, rot=2)):
        assert f(*{**ok, **bad}.values()) == 1, bad


# ------------------------------------------------------------ 4-bit format ---
def test_codes_nearest_and_even():
    levels = np.concatenate([cache4.LEVELS, -cache4.LEVELS])
    np.testing.assert_array_equal(cache4.to_code(levels), np.arange(16))
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    np.testing.assert_array_equal(cache4.to_code(mid), [0, 2, 2, 4, 4, 6, 6])
    np.testing.assert_array_equal(cache4.to_code(np.nextafter(mid, 9)), np.arange(1, 8))
    np.testing.assert_array_equal(cache4.to_code(np.nextafter(mid, 0)), np.arange(7))
    np.testing.assert_array_equal(cache4.to_code(np.array([7.0, 1e30, np.inf, -np.inf])), [7, 7, 7, 15])


def test_scale_bytes():
    t = torch.arange(128, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(cache4.e4m3_value(np.arange(128)), t)
    for b in range(128):
        assert cache4.e4m3_byte(t[b]) == b


@pytest.mark.parametrize("g", [1.0, 0.0021, 300.0])
def test_quantised_values_are_near(g):
    """With s* = max |x| / (6 g): s is off by e = max(2^-4 s*, 2^-10 (below the normal range), s* - 448) at most.  An
    element is off by one unit s g of its code at most (half a step below 6, where steps are 2), and
    by what it exceeds 6 s g, 6 g e at most; s <= s* + e."""
    r = np.random.default_rng(3)
    x = r.normal(size=(40, 2, 64)).astype(np.float32) * 3
    gs = np.array([g, g / 3], np.float32)
    codes, s = cache4.quantise(x, gs)
    got = cache4.values(codes, s, gs)
    best = np.repeat(np.abs(x.reshape(40, 2, 4, 16)).max(-1), 16, -1) / (6.0 * gs[:, None])
    e = np.maximum(np.maximum(best / 16, 2.0 ** -10), best - 448)
    assert (np.abs(got - x) <= gs[:, None] * (np.minimum(best + e, 448) + 6 * e) * (1 + 1e-6)).all()
    if g == 1.0:
        assert np.abs(got - x).mean() < 0.12 * np.abs(x).mean()


def test_blocks_of_zeros_infinities_and_nan():
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, 16] = 1e-30
    x[0, 0, 33], x[0, 0, 40] = np.inf, -2.0
    x[0, 0, 50] = np.nan
    g = np.ones(1, np.float32)
    v = cache4.values(*cache4.quantise(x, g), g)[0, 0]
    assert (v[:33] == 0).all() and v[33] == 6 * 448 and (v[34:48] == 0).all() and np.isnan(v[48:]).all()


@pytest.mark.parametrize("page,D", [(1, 32), (5, 96), (16, 128), (24, 64), (7, 160), (64, 256)])
def test_layout(lib, page, D):
    import serving_draft_verify_gb300 as dsv
    code, scale, whole = cache4.layout(page, D)
    assert lib.dspark_kv_page_bytes(page, D, 3) == whole == dsv.kv4_page_bytes(page, D)
    r = np.random.default_rng(4)
    cache = np.full((3, 2, whole), 0xA5, np.uint8)
    codes, s = r.integers(0, 16, (3 * page, 2, D)).astype(np.uint8), r.integers(0, 127, (3 * page, 2, D // 16)).astype(np.uint8)
    for slot in range(3 * page):
        for h in range(2):
            cache4.put(cache, page, D, slot, h, codes[slot, h], s[slot, h])
    c, t = cache4.get(cache, page, D)
    np.testing.assert_array_equal(c.transpose(0, 2, 1, 3).reshape(3 * page, 2, D), codes)
    np.testing.assert_array_equal(t.transpose(0, 2, 1, 3).reshape(3 * page, 2, D // 16), s)
    assert dsv.kv4_cache(3, 2, page, D, device="cpu").shape == cache.shape


def test_page_bytes(lib):
    f = lib.dspark_kv_page_bytes
    assert [f(16, 128, t) for t in range(4)] == [8192, 4096, 2048, 16 * 72]
    assert f(0, 128, 3) == f(16, 48, 3) == f(16, 288, 1) == f(16, 12, 0) == f(16, 128, 4) == f(16, 128, -1) == 0
    assert f(1 << 30, 128, 3) == 0 and f(1 << 30, 128, 0) == 1 << 39


# --------------------------------------------------------------- refusals ---
def _call(fn, defaults, **changes):
    assert set(changes) <= set(defaults), changes
    return fn(*{**defaults, **changes}.values())


def test_rotate(lib):
    d = dict(rows=4, heads=8, D=128, rot=128, inter=0, back=0, dt=1, x=0x100000, xs=1024, position=FAKE, freq=FAKE,
             magnitude=1.0, out=0x200000, os=1024, ws=WS, ws_bytes=BIG, stream=None)
    f = lib.dspark_rotate
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(heads=0), dict(heads=4097), dict(D=0), dict(D=24), dict(D=272),
                dict(rot=0), dict(rot=8), dict(rot=144), dict(rot=120), dict(inter=2), dict(back=-1), dict(dt=2), dict(dt=3),
                dict(x=None), dict(x=0x100008), dict(xs=1023), dict(xs=1028), dict(position=None), dict(freq=None),
                dict(magnitude=float("nan")), dict(magnitude=float("inf")), dict(out=None), dict(out=0x200008), dict(os=8),
                dict(ws=None), dict(ws=WS + 16),
                dict(out=0x100000, os=2048),                 # the same rows at another stride
                dict(out=0x100000 + 16), dict(out=0x100000 + 3 * 2048),
                dict(xs=2048, os=2048, out=0x100000 + 1024)):       # half of a head's neighbour
        assert _call(f, d, **bad) == 1, bad
    assert _call(f, d, ws_bytes=16) == 3
    # rows of one buffer that lie beside each other pass the check (and meet the workspace's)
    assert _call(f, d, xs=4096, os=4096, out=0x100000 + 2048, ws_bytes=16) == 3
    assert _call(f, d, out=0x100000, ws_bytes=16) == 3


def test_rotate_write_kv(lib):
    d = dict(rows=4, Hq=32, Hkv=8, D=128, rot=64, inter=0, page=16, nb=64, dt=1, cdt=3, q=0x100000, qs=6144, k=0x102000,
             ks=6144, v=0x102800, vs=6144, position=FAKE, freq=FAKE, magnitude=1.0, slot=FAKE, kscale=FAKE, vscale=FAKE,
             out=0x200000, os=4096, kc=FAKE, vc=FAKE, ws=WS, ws_bytes=BIG, stream=None)
    f = lib.dspark_rotate_write_kv
    for bad in (dict(rows=-1), dict(Hq=-1), dict(Hkv=0), dict(Hkv=1025), dict(D=112), dict(D=288), dict(rot=48), dict(rot=0),
                dict(rot=160), dict(inter=3), dict(page=0), dict(nb=0), dict(dt=2), dict(cdt=0), dict(cdt=4), dict(q=None),
                dict(k=None), dict(v=None), dict(ks=8), dict(vs=1020), dict(qs=4095), dict(position=None), dict(freq=None),
                dict(magnitude=float("inf")), dict(slot=None), dict(kscale=None), dict(vscale=None), dict(cdt=2, vscale=None),
                dict(out=None), dict(os=100), dict(kc=None), dict(vc=FAKE + 8), dict(ws=None), dict(ws=WS + 128),
                dict(out=0x102000, os=6144), dict(out=0x102800 - 4096, os=6144), dict(out=0x100010, os=6144)):
        assert _call(f, d, **bad) == 1, bad
    assert _call(f, d, page=1 << 25) == 2
    assert _call(f, d, ws_bytes=255) == 3
    assert _call(f, d, Hq=0, q=None, out=None, ws_bytes=255) == 3
    assert _call(f, d, out=0x100000, os=6144, ws_bytes=255) == 3
    assert _call(f, d, cdt=2, rot=48, ws_bytes=255) == 3


def test_read_kv(lib):
    d = dict(rows=4, Hkv=8, D=128, page=16, nb=64, dt=1, cdt=3, slot=FAKE, kc=FAKE, vc=FAKE, kscale=FAKE, vscale=FAKE,
             k=0x100000, ks=1024, v=0x200000, vs=1024, ws=WS, ws_bytes=BIG, stream=None)
    f = lib.dspark_read_kv
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(Hkv=0), dict(Hkv=1025), dict(D=0), dict(D=48), dict(D=264), dict(page=0),
                dict(nb=0), dict(dt=2), dict(cdt=4), dict(cdt=-1), dict(cdt=2, D=24), dict(kscale=None), dict(cdt=2, vscale=None),
                dict(slot=None), dict(kc=None), dict(vc=None), dict(kc=FAKE + 8), dict(k=None), dict(v=None), dict(k=0x100008),
                dict(ks=1000), dict(vs=1028), dict(ws=None), dict(ws=WS + 16)):
        assert _call(f, d, **bad) == 1, bad
    assert _call(f, d, page=1 << 25) == 2
    assert _call(f, d, ws_bytes=16) == 3


def test_four_bits_in_write_and_attention(lib):
    d = dict(rows=4, Hkv=8, D=128, page=16, num_blocks=64, dt=1, cache_dt=3, k=FAKE, k_stride=1024, v=FAKE,
             v_stride=1024, slot=FAKE, ks=FAKE, vs=FAKE, kc=FAKE, vc=FAKE, ws=WS, ws_bytes=BIG, stream=None)
    for bad in (dict(D=48), dict(ks=None), dict(vs=None), dict(dt=3)):
        assert _call(lib.dspark_write_kv, d, **bad) == 1, bad
    assert _call(lib.dspark_write_kv, d, page=1 << 25) == 2
    a = dict(B=2, rows=4, max_rows=4, Hq=32, Hkv=8, D=128, page=16, max_blocks=8, num_blocks=64, dt=1, cache_dt=3,
             q=FAKE, q_stride=4096, off=FAKE, len=FAKE, table=FAKE, ld=8, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE,
             scale=0.1, window=0, out=FAKE, lse=None, ws=WS, ws_bytes=BIG, stream=None)
    for bad in (dict(D=48), dict(D=16), dict(ks=None), dict(vs=None), dict(dt=3), dict(cache_dt=4)):
        assert _call(lib.dspark_paged_attention, a, **bad) == 1, bad
    assert _call(lib.dspark_paged_attention, a, page=1 << 25, max_blocks=4) == 2


def test_binding_refuses(lib):
    import serving_draft_verify_gb300 as dsv
    x, i, f = torch.zeros((3, 2, 64)), torch.zeros(3, dtype=torch.int32), torch.zeros(32)
    s, c, g = torch.zeros(3, dtype=torch.int64), torch.zeros((4, 2, 576), dtype=torch.uint8), torch.ones(2)
    for call in (lambda: dsv.dspark_rotate(x, i, f), lambda: dsv.dspark_rotate_write_kv(x, x, x, i, f, s, c, c, g, g),
                 lambda: dsv.dspark_read_kv(s, c, c, g, g, D=64), lambda: dsv.dspark_write_kv(x, x, s, c, c, g, g)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(ValueError):
        dsv.kv4_cache(4, 2, 16, 48, device="cpu")
    with pytest.raises(KeyError):
        dsv.dspark_rotary_frequencies(64, scaling="other", device="cpu")
