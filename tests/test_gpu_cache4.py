"""The cache in 4 bits on the GPU: written, read back, attended over.

Codes and scales are defined by single float32 operations and have to be equal bit for bit; reading back is one
product and one rounding.  Attention's error bound is the one in test_gpu_target.py's text: stored values
are exact in f16, so 4 bits add nothing to it.  What they bring is values that are zero, often those of the
keys that weigh most, so that small weights decide an element.  For bf16 rows a weight e <= 1 (of the largest so far)
enters as f16(2^14 e): below e = 2^-28 that is no normal number and is off by 2^-25, 2^-39 of the largest, not by
2^-12 of itself.  The sum of the weights is 1 at least, so with n keys and values up to v
  2^-39 n v = 2^-11 (2^-28 n v)
comes on top: W becomes W + 2^-28 n v in that bound.
"""
import numpy as np
import pytest
import torch

from oracle import cache4, target
from tests.test_gpu_target import U, _check_attend, _code, _gpu, _ws, dsv  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = dict(bf16=torch.bfloat16, f32=torch.float32)


def _rows(seed, n, heads, D, dtype, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, D), generator=g) * torch.exp(spread * torch.randn((n, heads, 1), generator=g))
    return x.to(TYPES[dtype])


def _scales(seed, heads, size=0.002):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(heads, generator=g) + 0.5) * size


def _slots(seed, n, page, blocks, skip=True):
    g = torch.Generator().manual_seed(seed)
    slot = torch.randperm(blocks * page, generator=g)[:n]
    if skip and n > 2:
        slot[1::5] = -1
    return slot


def _expect(cache, page, slot, x, g):
    """`cache` (numpy bytes) with rows x (float32 values) stored."""
    D = x.shape[-1]
    codes, s = cache4.quantise(x.float().numpy(), g.numpy())
    for i, at in enumerate(slot.tolist()):
        if at >= 0:
            for h in range(x.shape[1]):
                cache4.put(cache, page, D, at, h, codes[i, h], s[i, h])
    return cache


# ------------------------------------------------------------------- write ---
WRITES = [(1, 1, 32, 1), (3, 2, 64, 5), (40, 3, 128, 16), (7, 2, 96, 24), (300, 1, 160, 64), (33, 4, 256, 3),
          (600, 2, 128, 16), (5, 40, 32, 7)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [0.002, 1.0, 700.0])
@pytest.mark.parametrize("n,Hkv,D,page", WRITES)
def test_write(dsv, n, Hkv, D, page, size, dtype):  # noqa: F811
    blocks = -(-n // page) + 2
    kc = torch.full((blocks, Hkv, dsv.kv4_page_bytes(page, D)), 0xA5, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    qkv = _rows(n, n, 2 + 2 * Hkv, D, dtype)
    k, v = qkv[:, 2:2 + Hkv], qkv[:, 2 + Hkv:]
    ks, vs = _scales(1, Hkv, size), _scales(2, Hkv, size)
    slot = _slots(n, n, page, blocks)
    G = qkv.cuda()
    ws = _ws()
    dsv.dspark_write_kv(G[:, 2:2 + Hkv], G[:, 2 + Hkv:], slot.cuda(), kc, vc, ks.cuda(), vs.cuda(), workspace=ws)
    assert _code(ws)[0] == 0
    old = np.full(kc.shape, 0xA5, np.uint8)
    np.testing.assert_array_equal(kc.cpu().numpy(), _expect(old.copy(), page, slot, k, ks))
    np.testing.assert_array_equal(vc.cpu().numpy(), _expect(old.copy(), page, slot, v, vs))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_odd_values(dsv, dtype):  # noqa: F811
    """Zeros of both signs, infinities, NaN, the type's smallest and largest, ties, scales that round to nothing."""
    big, small = torch.finfo(TYPES[dtype]).max, torch.finfo(TYPES[dtype]).tiny
    rows = torch.zeros((12, 1, 64))
    rows[0, 0, 3] = -0.0
    rows[1, 0, :20] = torch.linspace(-6, 6, 20)
    rows[2, 0, 5], rows[2, 0, 6] = float("inf"), -1.0
    rows[3, 0, 17], rows[3, 0, 18] = float("nan"), float("inf")
    rows[4, 0, :] = big
    rows[5, 0, :] = -small
    rows[6, 0, :16] = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -6, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25])
    rows[7, 0, :16] = rows[6, 0, :16] * 2.0 ** -9
    rows[8, 0, :16] = rows[6, 0, :16] * 2.0 ** -10
    rows[9, 0, :16] = rows[6, 0, :16] * 449
    rows[10, 0, 47] = -float("inf")
    rows[11, 0, 48:] = small
    x = rows.to(TYPES[dtype])
    for g in (1.0, 2.0 ** -64, 2.0 ** 64, 0.37):
        gs = torch.tensor([g])
        kc = torch.zeros((1, 1, dsv.kv4_page_bytes(12, 64)), dtype=torch.uint8, device="cuda")
        vc = torch.zeros_like(kc)
        slot = torch.arange(12)
        dsv.dspark_write_kv(x.cuda(), (-x).cuda(), slot.cuda(), kc, vc, gs.cuda(), gs.cuda())
        zero = np.zeros(kc.shape, np.uint8)
        np.testing.assert_array_equal(kc.cpu().numpy(), _expect(zero.copy(), 12, slot, x, gs))
        np.testing.assert_array_equal(vc.cpu().numpy(), _expect(zero.copy(), 12, slot, -x, gs))


def test_write_status(dsv):  # noqa: F811
    for n in (4, 500):
        kc = dsv.kv4_cache(3, 2, 8, 64)
        vc = dsv.kv4_cache(3, 2, 8, 64)
        slot = torch.full((n,), -1)
        slot[:4] = torch.tensor([0, 24, 1 << 40, 23])
        x, one = torch.ones((n, 2, 64), device="cuda"), torch.ones(2, device="cuda")
        ws = _ws()
        dsv.dspark_write_kv(x, x, slot.cuda(), kc, vc, one, one, workspace=ws)
        assert _code(ws) == [6, 1]
        got = dsv.dspark_read_kv(torch.arange(24, device="cuda"), kc, vc, one, one, D=64, dtype=torch.float32)
        assert (got["k"][[0, 23]] == got["v"][[0, 23]]).all() and got["k"].count_nonzero().item() == 2 * 2 * 64
    dsv.dspark_write_kv(x[:0], x[:0], slot[:0].cuda(), kc, vc, one, one)


# ---------------------------------------------------------- rotate and store ---
@pytest.mark.parametrize("cache", ["same", "e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,D,rot,page", [(1, 4, 1, 64, 64, 16), (37, 6, 2, 128, 64, 5), (9, 0, 3, 96, 32, 16),
                                                 (301, 32, 8, 128, 128, 16), (18, 3, 1, 256, 256, 24), (5, 1, 40, 32, 32, 1)])
def test_rotate_write(dsv, n, Hq, Hkv, D, rot, page, inter, dtype, cache):  # noqa: F811
    """The rotated keys in float32 are those of dspark_rotate on float32 copies; stored, they have to be what
    the cache's definition makes of them, bit for bit."""
    blocks = -(-n // page) + 2
    kind = torch.uint8 if cache == "e2m1" else torch.float8_e4m3fn if cache == "e4m3" else TYPES[dtype]
    shape = (blocks, Hkv, dsv.kv4_page_bytes(page, D)) if cache == "e2m1" else (blocks, Hkv, page, D)
    kc, vc = (torch.zeros(shape, dtype=kind, device="cuda") for _ in range(2))
    size = 0.002 if cache == "e2m1" else 0.02
    ks, vs = (None, None) if cache == "same" else (_scales(1, Hkv, size), _scales(2, Hkv, size))
    g = torch.Generator().manual_seed(n)
    position = torch.randint(0, 50000, (n,), generator=g, dtype=torch.int32)
    slot = _slots(n, n, page, blocks)
    if n > 4:
        position[3] = -1
    freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    qkv = _rows(n, n, Hq + 2 * Hkv, D, dtype, 0.3).cuda()
    q, k, v = qkv[:, :Hq] if Hq else None, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    P = position.cuda()
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    ws = _ws()
    out = torch.full((n, Hq, D), 7.0, dtype=TYPES[dtype], device="cuda") if Hq else None
    got = dsv.dspark_rotate_write_kv(q, k, v, P, freq, slot.cuda(), kc, vc, dev(ks), dev(vs), inter, 1.1, out=out, workspace=ws)
    assert _code(ws)[0] == 0
    live = P >= 0
    if Hq:
        want = dsv.dspark_rotate(q, P, freq, inter, False, 1.1)
        assert torch.equal(got[live], want[live]) and (got[~live] == 7).all()
    else:
        assert got is None
    turned = dsv.dspark_rotate(k.float().contiguous(), P, freq, inter, False, 1.1).cpu()
    slot = torch.where(position >= 0, slot, -1)
    turned[position < 0] = 0
    v = v.cpu()
    if cache == "e2m1":
        zero = np.zeros(kc.shape, np.uint8)
        np.testing.assert_array_equal(kc.cpu().numpy(), _expect(zero.copy(), page, slot, turned, ks))
        np.testing.assert_array_equal(vc.cpu().numpy(), _expect(zero.copy(), page, slot, v, vs))
        return
    zero = np.zeros((blocks, Hkv, page, D))
    f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
    stored = turned.to(TYPES[dtype]) if cache == "same" else turned
    wk, wv = target.write_kv(f(stored), f(v), slot.numpy(), zero, zero, f(ks), f(vs))
    np.testing.assert_array_equal(kc.double().cpu().numpy(), wk)
    np.testing.assert_array_equal(vc.double().cpu().numpy(), wv)


def test_rotate_write_in_place_status_and_graph(dsv):  # noqa: F811
    n, Hq, Hkv, D = 600, 4, 2, 64
    qkv = _rows(3, n, Hq + 2 * Hkv, D, "bf16").cuda()
    P = torch.arange(n, dtype=torch.int32, device="cuda")
    freq, _ = dsv.dspark_rotary_frequencies(64)
    one = torch.ones(Hkv, device="cuda") * 0.01
    kc, vc = dsv.kv4_cache(40, Hkv, 16, D), dsv.kv4_cache(40, Hkv, 16, D)
    slot = torch.arange(n, device="cuda")
    want = dsv.dspark_rotate_write_kv(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], P, freq, slot, kc, vc, one, one)
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    same = qkv.clone()
    ws = _ws()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsv.dspark_rotate_write_kv(same[:, :Hq], same[:, Hq:Hq + Hkv], same[:, Hq + Hkv:], P, freq, slot, k2, v2, one, one,
                                   out=same[:, :Hq], workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(same[:, :Hq], want) and torch.equal(same[:, Hq:], qkv[:, Hq:])
    assert torch.equal(k2, kc) and torch.equal(v2, vc)
    slot[5], slot[599] = 640, 1 << 33
    ws = _ws()
    k2.zero_(), v2.zero_()
    got = dsv.dspark_rotate_write_kv(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], P, freq, slot, k2, v2, one, one, workspace=ws)
    assert _code(ws) == [6, 1] and torch.equal(got, want)
    a = dsv.dspark_read_kv(torch.arange(600, device="cuda"), kc, vc, one, one, D=D)
    b = dsv.dspark_read_kv(torch.arange(600, device="cuda"), k2, v2, one, one, D=D)
    keep = [i for i in range(600) if i not in (5, 599)]
    assert torch.equal(a["k"][keep], b["k"][keep]) and (b["v"][[5, 599]] == 0).all()


# -------------------------------------------------------------------- read ---
@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hkv,D,page", [(1, 1, 32, 1), (30, 2, 128, 16), (300, 3, 96, 5), (700, 1, 256, 24), (3, 40, 64, 8)])
def test_read(dsv, n, Hkv, D, page, dtype, cache):  # noqa: F811
    blocks = 20
    r = np.random.default_rng(n)
    g = torch.Generator().manual_seed(n)
    gs = [None, None] if cache in TYPES else [_scales(1, Hkv), _scales(2, Hkv)]
    caches, values = [], []
    for i in range(2):
        if cache == "e2m1":
            raw = r.integers(0, 256, (blocks, Hkv, dsv.kv4_page_bytes(page, D))).astype(np.uint8)
            caches.append(torch.from_numpy(raw).cuda())
            c, s = cache4.get(raw, page, D)
            values.append(cache4.values(c.transpose(0, 2, 1, 3), s.transpose(0, 2, 1, 3), gs[i].numpy()))
        else:
            x = torch.randn((blocks, Hkv, page, D), generator=g) * 50
            x = x.clamp(-448, 448).to(torch.float8_e4m3fn) if cache == "e4m3" else x.to(TYPES[cache])
            caches.append(x.cuda())
            y = x.float() if gs[i] is None else x.float() * gs[i][:, None, None]
            values.append(y.double().numpy().transpose(0, 2, 1, 3))
    slot = torch.randint(0, blocks * page, (n,), generator=g)              # some twice
    slot[n // 2:n // 2 + 2] = -1
    out = {x: torch.full((n, Hkv + 1, D), 7.0, dtype=TYPES[dtype], device="cuda") for x in "kv"}
    part = {x: out[x][:, :Hkv] for x in "kv"}
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    ws = _ws()
    dsv.dspark_read_kv(slot.cuda(), *caches, dev(gs[0]), dev(gs[1]), out=part, workspace=ws)
    assert _code(ws)[0] == 0
    gone = slot < 0
    for x, y in zip("kv", values):
        # the product in float32 (as defined), then one rounding
        rows = y.reshape(blocks * page, Hkv, D)[slot.numpy()]
        want = torch.from_numpy(rows).float().to(TYPES[dtype])
        got = part[x].cpu()
        assert (got[gone] == 7).all() and (out[x][:, Hkv] == 7).all()
        same = (got == want) | (torch.isnan(got) & torch.isnan(want))
        assert same[~gone].all()


def test_read_status(dsv):  # noqa: F811
    for n in (5, 400):
        kc = dsv.kv4_cache(2, 1, 4, 32)
        one = torch.ones(1, device="cuda")
        slot = torch.zeros(n, dtype=torch.int64)
        slot[1], slot[2] = 8, 1 << 50
        out = {x: torch.full((n, 1, 32), 7.0, device="cuda") for x in "kv"}
        ws = _ws()
        dsv.dspark_read_kv(slot.cuda(), kc, kc, one, one, out=out, workspace=ws)
        assert _code(ws) == [6, 1] and (out["k"][1:3] == 7).all() and (out["v"][3:] == 0).all() and (out["v"][0] == 0).all()
    assert dsv.dspark_read_kv(slot[:0].cuda(), kc, kc, one, one, D=32)["k"].shape == (0, 1, 32)


# ------------------------------------------------------------------ attend ---
def _attend_case(seed, lens, Hq, Hkv, D, page, dtype, window, size=0.002):
    """Caches of quantised normal values; places that no row may see read as NaN, the tables' unused entries are bad."""
    r = np.random.default_rng(seed)
    pages = [-(-(n + m) // page) for n, m in lens]
    total = sum(pages)
    ids = r.permutation(total + 3)
    table = np.full((len(lens), max(max(pages), 1) + 2), -5, np.int32)
    seen = np.zeros((total + 3, page), bool)
    at = 0
    for b, (n, m) in enumerate(lens):
        mine = ids[at:at + pages[b]]
        table[b, :pages[b]] = mine
        if pages[b]:
            seen[mine] = (np.arange(pages[b] * page) < n + m).reshape(-1, page)
        at += pages[b]
    code, scale, whole = cache4.layout(page, D)
    got, vals, gs = [], [], []
    for i in range(2):
        g = ((r.random(Hkv) + 0.5) * size).astype(np.float32)
        c, s = cache4.quantise(r.normal(size=(total + 3, page, Hkv, D)).astype(np.float32), g)
        vals.append(cache4.values(c, s, g).transpose(0, 2, 1, 3))
        c, s = c.transpose(0, 2, 1, 3), s.transpose(0, 2, 1, 3).copy()
        s[np.broadcast_to(~seen[:, None, :, None], s.shape)] = 0x7F
        raw = np.full((total + 3, Hkv, whole), 0xFF, np.uint8)
        raw[..., :page * code] = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(total + 3, Hkv, -1)
        padded = np.full((total + 3, Hkv, page, scale), 0x7F, np.uint8)
        padded[..., :D // 16] = s
        raw[..., page * code:page * (code + scale)] = padded.reshape(total + 3, Hkv, -1)
        got.append(torch.from_numpy(raw).cuda())
        gs.append(g)
    offset = np.concatenate([[0], np.cumsum([m for _, m in lens])]).astype(np.int32)
    q = torch.from_numpy(r.normal(size=(int(offset[-1]), Hq + 2, D)) * 2).to(TYPES[dtype]).cuda()[:, 1:1 + Hq]
    c = dict(q=q, row_offset=_gpu(offset), length=torch.tensor([n for n, _ in lens], dtype=torch.int32).cuda(),
             block_table=_gpu(table), k_cache=got[0], v_cache=got[1], k_scale=_gpu(gs[0]), v_scale=_gpu(gs[1]), window=window,
             max_rows=max(max(m for _, m in lens), 1))
    return c, vals


def _oracle(c, vals, scale=None):
    i = lambda x: x.cpu().numpy().astype(np.int64)  # noqa: E731
    D = c["q"].shape[2]
    return target.paged_attention(c["q"].double().cpu().numpy(), i(c["row_offset"]), i(c["length"]), i(c["block_table"]),
                                  vals[0], vals[1], D ** -0.5 if scale is None else scale, c["window"])


def _check(out, ref, vals, dtype, D):
    weight = ref["weight"]
    if dtype == "bf16":
        weight = weight + 2.0 ** -28 * ref["keys"][:, None, None] * np.nanmax(np.abs(vals[1]))
    _check_attend(out, dict(ref, weight=weight), dtype, D)


def _run_attend(dsv, c, **kw):  # noqa: F811
    ws = torch.full((dsv.load().dspark_paged_attention_workspace_size(c["q"].shape[2]),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    args = {k: c[k] for k in ("q", "row_offset", "length", "block_table", "k_cache", "v_cache", "max_rows", "window",
                              "k_scale", "v_scale")}
    out = dsv.dspark_paged_attention(**args, workspace=ws, **kw)
    return out, _code(ws)


SHAPES = [  # lens, Hq, Hkv, D, page, window
    ("one key", [(0, 1)], 4, 2, 64, 16, 0),
    ("one row", [(300, 1)], 32, 8, 128, 16, 0),
    ("ragged", [(0, 3), (17, 1), (64, 8), (5, 0), (129, 5), (31, 1)], 8, 2, 128, 16, 0),
    ("no group", [(40, 2), (3, 1)], 3, 3, 96, 24, 0),
    ("wide group", [(200, 3), (7, 2)], 12, 1, 128, 16, 0),
    ("group of seven", [(90, 4), (1, 4)], 28, 4, 64, 32, 0),
    ("odd page", [(61, 2), (7, 7)], 4, 2, 96, 5, 0),
    ("page of one", [(20, 2)], 4, 4, 32, 1, 0),
    ("big page", [(20, 2), (300, 3)], 8, 4, 64, 256, 0),
    ("window", [(500, 4), (3, 2), (130, 6)], 8, 2, 128, 16, 100),
    ("window of one", [(50, 3)], 4, 2, 64, 16, 1),
    ("verify 8", [(100, 8), (33, 8), (0, 8), (250, 3)], 32, 8, 128, 16, 0),
    ("verify 17", [(100, 17), (33, 17), (0, 17), (250, 9)], 32, 8, 128, 16, 0),
    ("verify 17 window", [(400, 17), (2, 16)], 16, 2, 128, 32, 65),
    ("verify 17 odd page", [(400, 17), (2, 16)], 16, 2, 64, 3, 65),
    ("prompt", [(30, 150), (0, 77)], 8, 2, 128, 16, 0),
    ("wide heads", [(70, 5), (600, 1)], 4, 1, 256, 16, 0),
    ("wide heads, many rows", [(70, 33), (6, 1)], 4, 1, 256, 16, 0),
    ("small heads", [(70, 5), (600, 1)], 8, 4, 32, 16, 0),
    ("odd heads", [(70, 20), (9, 3)], 10, 2, 160, 16, 0),
    ("odd heads, odd page", [(70, 20), (9, 3)], 10, 2, 224, 6, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name,lens,Hq,Hkv,D,page,window", SHAPES, ids=[s[0] for s in SHAPES])
def test_attention(dsv, name, lens, Hq, Hkv, D, page, window, dtype):  # noqa: F811
    c, vals = _attend_case(len(name), lens, Hq, Hkv, D, page, dtype, window)
    out, code = _run_attend(dsv, c)
    assert code[0] == 0
    _check(out, _oracle(c, vals), vals, dtype, D)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,Hq", [(1, 8), (8, 8), (17, 32), (40, 16)])
def test_attention_split_over_many_blocks(dsv, dtype, rows, Hq):  # noqa: F811
    c, vals = _attend_case(7, [(9000, rows), (1, 1), (700, rows), (0, 1)], Hq, Hq // 4, 128, 16, dtype, 0)
    out, code = _run_attend(dsv, c)
    assert code[0] == 0
    _check(out, _oracle(c, vals), vals, dtype, 128)
    again, _ = _run_attend(dsv, c)
    assert torch.equal(out["out"], again["out"]) and torch.equal(out["lse"], again["lse"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-0.25, 0.0, 1.5])
@pytest.mark.parametrize("size", [0.002, 30.0])
def test_attention_scales(dsv, dtype, scale, size):  # noqa: F811
    c, vals = _attend_case(17, [(70, 4), (3, 1), (0, 17)], 16, 4, 64, 16, dtype, 40, size)
    out, code = _run_attend(dsv, c, scale=scale)
    assert code[0] == 0
    _check(out, _oracle(c, vals, scale), vals, dtype, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,Hq,D", [(4, 4, 64), (3, 32, 128), (8, 16, 128), (17, 32, 128), (4, 8, 256)])
def test_hidden_blocks_may_be_nan(dsv, dtype, rows, Hq, D):  # noqa: F811
    """A block that is not a number at a step's last row does not reach the rows before, and reaches its own
    columns of that row alone."""
    lens = [(37, rows), (64, rows)]
    c, _ = _attend_case(12, lens, Hq, 4, D, 16, dtype, 0)
    want, _ = _run_attend(dsv, c)
    code, scale, _ = cache4.layout(16, D)
    for b, (n, m) in enumerate(lens):
        last = n + m - 1
        blk = int(c["block_table"][b, last // 16])
        c["v_cache"][blk, :, 16 * code + last % 16 * scale + 1] = 0x7F + 128 * b       # elements 16 .. 31
    got, status = _run_attend(dsv, c)
    assert status[0] == 0
    keep = [i for i in range(2 * rows) if i % rows != rows - 1]
    assert torch.equal(got["out"][keep], want["out"][keep]) and torch.equal(got["lse"], want["lse"])
    odd = got["out"][rows - 1::rows]
    assert torch.isnan(odd[..., 16:32]).all()
    rest = [i for i in range(D) if not 16 <= i < 32]
    assert torch.equal(odd[..., rest], want["out"][rows - 1::rows][..., rest])
    # a key that is not a number: its row's scores are none
    last = 37 + rows - 1
    c["k_cache"][int(c["block_table"][0, last // 16]), :, 16 * code + last % 16 * scale] = 0x7F
    got, _ = _run_attend(dsv, c)
    assert torch.equal(got["out"][keep], want["out"][keep]) and torch.isnan(got["lse"][rows - 1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page,window", [
    ([(500, 1), (37, 1)], 8, 2, 128, 16, 100), ([(500, 4), (70, 3)], 8, 2, 64, 16, 33), ([(300, 3)], 4, 2, 96, 5, 41),
    ([(90, 2)], 4, 4, 32, 1, 7), ([(700, 17), (140, 17)], 32, 8, 128, 16, 130), ([(600, 2)], 4, 1, 256, 24, 200)])
def test_pages_before_the_window_may_be_gone(dsv, lens, Hq, Hkv, D, page, window, dtype):  # noqa: F811
    c, vals = _attend_case(33, lens, Hq, Hkv, D, page, dtype, window)
    want, code = _run_attend(dsv, c)
    assert code[0] == 0
    _check(want, _oracle(c, vals), vals, dtype, D)
    for b, (n, _r) in enumerate(lens):
        c["block_table"][b, :max(0, n - window + 1) // page] = -1
    got, code = _run_attend(dsv, c)
    assert code[0] == 0 and torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_attention_status_and_untouched_rows(dsv):  # noqa: F811
    c, _ = _attend_case(15, [(20, 2), (30, 3), (9, 2)], 8, 2, 64, 16, "bf16", 0)
    want, _ = _run_attend(dsv, c)
    fill = lambda: dict(out=torch.full((9, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                        lse=torch.full((9, 8), 7.0, device="cuda"))
    c["q"] = torch.cat([c["q"], c["q"][:2]])
    out, code = _run_attend(dsv, c, out=fill())
    assert code[0] == 0 and (out["out"][7:] == 7).all() and (out["lse"][7:] == 7).all()
    assert torch.equal(out["out"][:7], want["out"])
    bad = dict(c, length=torch.tensor([20, 10 ** 6, 9], dtype=torch.int32, device="cuda"))
    out, code = _run_attend(dsv, bad, out=fill())
    assert code == [6, 1] and (out["out"][2:5] == 7).all() and torch.equal(out["out"][:2], want["out"][:2])
    table = c["block_table"].clone()
    table[0, 0] = 10 ** 6
    table[2, 0] = -1
    out, code = _run_attend(dsv, dict(c, block_table=table), out=fill())
    assert code == [6, 2] and torch.equal(out["out"][2:5], want["out"][2:5])
    empty, _ = _attend_case(34, [(20, 0), (3, 0)], 4, 2, 64, 16, "bf16", 0)
    out, code = _run_attend(dsv, dict(empty, max_rows=0))
    assert code[0] == 0 and out["out"].shape == (0, 4, 64)


def test_far_places_of_a_large_cache(dsv):  # noqa: F811
    """Byte offsets past 2^32: the pages of one request lie at the end of a 5 GB cache."""
    blocks, Hkv, page, D = 290000, 8, 32, 128
    kc, vc = dsv.kv4_cache(blocks, Hkv, page, D), dsv.kv4_cache(blocks, Hkv, page, D)
    assert kc.numel() > 1 << 32
    gs = torch.full((Hkv,), 0.002, device="cuda")
    ids = [blocks - 1, 66000, blocks - 7]
    x = _rows(1, 80, 4 * Hkv, D, "bf16", 0.0).cuda()
    slot = torch.tensor([ids[i // page] * page + i % page for i in range(80)], device="cuda")
    ks, vs = dsv.kv4_cache(3, Hkv, page, D), dsv.kv4_cache(3, Hkv, page, D)
    near = torch.arange(80, device="cuda")
    args = dict(row_offset=torch.tensor([0, 3], dtype=torch.int32, device="cuda"), max_rows=3,
                length=torch.tensor([77], dtype=torch.int32, device="cuda"), k_scale=gs, v_scale=gs)
    for k, v, s in ((kc, vc, slot), (ks, vs, near)):
        dsv.dspark_write_kv(x[:, :Hkv], x[:, Hkv:2 * Hkv], s, k, v, gs, gs)
    a = dsv.dspark_read_kv(slot, kc, vc, gs, gs, D=D)
    b = dsv.dspark_read_kv(near, ks, vs, gs, gs, D=D)
    assert torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"]) and a["k"].count_nonzero() > 0
    for q in (x[77:, :2 * Hkv], x[77:, :2 * Hkv].float()):
        far = dsv.dspark_paged_attention(q, block_table=torch.tensor([ids], dtype=torch.int32, device="cuda"), k_cache=kc,
                                         v_cache=vc, **args)
        close = dsv.dspark_paged_attention(q, block_table=torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"),
                                           k_cache=ks, v_cache=vs, **args)
        assert torch.equal(far["out"], close["out"]) and torch.equal(far["lse"], close["lse"])


def test_streams_graphs_and_one_workspace(dsv):  # noqa: F811
    """A captured run of rotation, storing and attention, replayed with other inputs, beside eager calls."""
    Hq, Hkv, D, page, n = 8, 2, 128, 16, 24
    freq, _ = dsv.dspark_rotary_frequencies(D, 1e6)
    gs = torch.full((Hkv,), 0.002, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4).contiguous()
    offset, length = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 20, 24], [0, 30]))
    position = torch.cat([torch.arange(20), torch.arange(30, 34)]).int().cuda()
    slot = torch.cat([torch.arange(20), 64 + torch.arange(30, 34)]).cuda()

    def step(qkv, kc, vc, out, ws, stream=None):
        q = dsv.dspark_rotate_write_kv(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], position, freq, slot, kc, vc, gs, gs,
                                       out=out["q"], workspace=ws, stream=stream)
        dsv.dspark_paged_attention(q, offset, length, table, kc, vc, 20, k_scale=gs, v_scale=gs,
                                   out=dict(out=out["out"], lse=out["lse"]), workspace=ws, stream=stream)
        return out

    new = lambda: dict(q=torch.zeros((n, Hq, D), dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                       out=torch.zeros((n, Hq, D), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((n, Hq), device="cuda"))
    inputs = [_rows(s, n, Hq + 2 * Hkv, D, "bf16", 0.0).cuda() for s in (1, 2)]
    size = dsv.load().dspark_paged_attention_workspace_size(D)
    want = [step(x, dsv.kv4_cache(8, Hkv, page, D), dsv.kv4_cache(8, Hkv, page, D), new(), _ws(size)) for x in inputs]
    qkv, kc, vc, out, ws = inputs[1].clone(), dsv.kv4_cache(8, Hkv, page, D), dsv.kv4_cache(8, Hkv, page, D), new(), _ws(size)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(qkv, kc, vc, out, ws)
    side = torch.cuda.Stream()
    for i in (0, 1, 0):
        qkv.copy_(inputs[i])
        kc.zero_(), vc.zero_()
        side.wait_stream(torch.cuda.current_stream())
        other = step(inputs[1 - i], dsv.kv4_cache(8, Hkv, page, D), dsv.kv4_cache(8, Hkv, page, D), new(), _ws(size), stream=side)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("q", "out", "lse"):
            assert torch.equal(out[k], want[i][k]) and torch.equal(other[k], want[1 - i][k])


@pytest.mark.parametrize("four_bits", [False, True])
def test_rounds_with_rotary_positions(dsv, four_bits):  # noqa: F811
    """Whole decoding rounds whose target rotates, stores and attends: greedy speculative decoding emits what
    decoding token by token does, with keys and values as the cache holds them."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import paged_round
    m = paged_round.Model(D=32, seed=5)
    prompts = [[1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11], [8, 9], [10, 300, 7]]
    s = paged_round.Rounds(m, prompts, gamma=4, page=8, blocks=64, rotary=True, four_bits=four_bits)
    s.prefill()
    for i in range(8):
        s.round(seed=i)
    torch.cuda.synchronize()
    g = np.full(m.Hkv, 0.002, np.float32)

    def stored(x):
        return torch.from_numpy(cache4.values(*cache4.quantise(x.float().cpu().numpy(), g), g)).to(x.device)

    steps = int((s.history_len - s.prompt_len).max())
    want = paged_round.token_by_token(m, prompts, steps, freq=s.freq, stored=stored if four_bits else None)
    for b in range(3):
        p, n = int(s.prompt_len[b]), int(s.history_len[b])
        assert n - p >= 8 and s.history[b, p:n].tolist() == want[b][:n - p]
