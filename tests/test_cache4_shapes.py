"""Rows whose heads are not a 4-bit cache's are refused before anything is launched, although the cache's shape gives
only its pages' bytes: by the calls' checks with stand-ins on the CPU, and by the calls themselves."""
import os

import pytest
import torch

PAGES = [(16, 128, 64), (16, 128, 32), (16, 128, 224), (16, 128, 256), (18, 96, 64), (18, 96, 128), (32, 64, 128)]


@pytest.fixture(scope="module")
def dsv():
    from serving_draft_verify_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    import serving_draft_verify_gb300 as m
    m.load()
    return m


class _OnGpu:
    """A tensor of the CPU that says it is on the first GPU."""

    def __init__(self, t):
        self.t, self.is_cuda = t, True
        self.__dict__.update(t.__dict__)

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


def _calls(dsv, D, kc, vc, on, **kw):
    """The four calls with two rows of two heads of D."""
    x = on(torch.zeros((2, 2, D), dtype=torch.bfloat16))
    i = lambda *v: on(torch.tensor(v, dtype=torch.int32))  # noqa: E731
    slot, g, freq = on(torch.zeros(2, dtype=torch.int64)), on(torch.ones(2)), on(torch.ones(D // 2))
    return (lambda: dsv.dspark_write_kv(x, x, slot, kc, vc, g, g, **kw),
            lambda: dsv.dspark_rotate_write_kv(None, x, x, i(0, 1), freq, slot, kc, vc, g, g, **kw),
            lambda: dsv.dspark_read_kv(slot, kc, vc, g, g, D=D, **kw),
            lambda: dsv.dspark_read_kv(slot, kc, vc, g, g, out=dict(k=x, v=x), **kw),
            lambda: dsv.dspark_paged_attention(x, i(0, 2), i(0), on(torch.zeros((1, 2), dtype=torch.int32)), kc, vc, 2, k_scale=g,
                                               v_scale=g, **kw))


@pytest.fixture
def one_gpu(dsv, monkeypatch):
    monkeypatch.setattr(dsv._binding, "_several", False)


@pytest.mark.parametrize("page,D,other", PAGES)
def test_rows_of_other_heads_are_refused(dsv, one_gpu, page, D, other):
    """The same bytes are whole pages of the other heads, so nothing but the cache itself, or `page`, can tell."""
    made = [dsv.kv4_cache(3, 2, page, D, device="cpu") for _ in range(2)]
    assert any(dsv.kv4_page_bytes(n, other) == made[0].shape[2] for n in range(1, 200))
    kc, vc = (_OnGpu(t) for t in made)
    for call in _calls(dsv, other, kc, vc, _OnGpu):
        with pytest.raises(ValueError, match=f"holds heads of {D}, the rows have heads of {other}"):
            call()
    # one of the two is enough to tell, and without either `page` is
    plain = [_OnGpu(t.clone()) for t in made]
    for pair in ((kc, plain[1]), (plain[0], vc)):
        for call in _calls(dsv, other, *pair, _OnGpu):
            with pytest.raises(ValueError, match=f"holds heads of {D}"):
                call()
    for call in _calls(dsv, other, *plain, _OnGpu, page=page):
        with pytest.raises(ValueError, match=f"no 4-bit cache of heads of {other} has pages of {made[0].shape[2]} bytes for {page} rows"):
            call()


def test_other_pages_are_refused(dsv, one_gpu):
    kc, vc = (_OnGpu(dsv.kv4_cache(3, 2, 16, 128, device="cpu")) for _ in range(2))
    for call in _calls(dsv, 128, kc, vc, _OnGpu, page=32):
        with pytest.raises(ValueError, match="k_cache has pages of 16 rows, not 32"):
            call()
    wide = _OnGpu(torch.zeros((3, 2, 16, 128), dtype=torch.float8_e4m3fn))
    for call in _calls(dsv, 128, wide, wide, _OnGpu, page=32):
        with pytest.raises(ValueError, match="pages of 16 rows, not 32"):
            call()
    odd = _OnGpu(torch.zeros((3, 2, 1153), dtype=torch.uint8))
    for call in _calls(dsv, 128, odd, odd, _OnGpu):
        with pytest.raises(ValueError, match="no 4-bit cache of heads of 128 has pages of 1153 bytes"):
            call()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float8_e4m3fn])
def test_heads_asked_of_other_caches_are_refused(dsv, one_gpu, dtype):
    """Reading with a D that is not the cache's: a cache whose shape says its heads holds it against them."""
    cache = _OnGpu(torch.zeros((3, 2, 16, 128)).to(dtype))
    g = _OnGpu(torch.ones(2)) if dtype is torch.float8_e4m3fn else None
    slot = _OnGpu(torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="heads of 64 asked of caches of heads of 128"):
        dsv.dspark_read_kv(slot, cache, cache, g, g, D=64)


@pytest.mark.gpu
def test_calls_on_the_gpu(dsv):
    """A cache for heads of 128 on pages of 16 rows refuses heads of 64 and 256 and is left as it was; its own heads are
    taken with and without `page`, and so is a copy of it."""
    kc, vc = dsv.kv4_cache(3, 2, 16, 128), dsv.kv4_cache(3, 2, 16, 128)
    kc.fill_(0x21), vc.fill_(0x21)
    on = lambda t: t.cuda()  # noqa: E731
    for D in (64, 256):
        for call in _calls(dsv, D, kc, vc, on):
            with pytest.raises(ValueError, match="holds heads of 128"):
                call()
    assert (kc == 0x21).all() and (vc == 0x21).all()
    slot, g = torch.arange(48, device="cuda"), torch.ones(2, device="cuda")
    want = dsv.dspark_read_kv(slot, kc, vc, g, g)
    assert want["k"].shape == (48, 2, 128)
    for pair, kw in (((kc, vc), dict(page=16)), ((kc.clone(), vc.clone()), dict(page=16, D=128)), ((kc.clone(), vc[:]), dict(D=128))):
        got = dsv.dspark_read_kv(slot, *pair, g, g, **kw)
        assert torch.equal(got["k"], want["k"]) and torch.equal(got["v"], want["v"])
    for call in _calls(dsv, 128, kc, vc, on, page=16):
        call()
    torch.cuda.synchronize()
