"""The target model's side of a round on the GPU against the float64 oracle.

Error bound of attention, fixed before the first run.  With u = 2^-24: a score is a
float32 sum of D products of scaled queries, off by at most (D + 8) u A with A the
largest sum_d |scale q_d k_d| of the row, so a weight is off by the factor 1 +- (2 (D +
8) u A + 2^-20) (2^-20: ex2, the running maximum's factors).  The sum over n keys adds
n u.  Weights enter the second product in at least 11 bits (2^-12 relative) where the
rows are bf16, exactly where they are float32.  With W = sum_j p_j |v_j| that gives
  |out - exact| <= W (2 (D + 8) u A + 2^-20 + 2 n u + [bf16: 2^-11]) + |exact| eps / 2
  |lse - exact| <= (D + 8) u A + 2^-20 + 2 n u + |exact| 2^-22.
An 8-bit cache adds nothing: the oracle reads the same stored values.
"""
import numpy as np
import pytest
import torch

from oracle import target

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dsv():
    import serving_draft_verify_gb300 as m
    m.load()
    return m


def _gpu(x, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def _ws(n=1 << 16):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")     # not zero on entry


def _code(ws):
    torch.cuda.synchronize()
    return ws[:8].cpu().view(torch.int32).tolist()


# -------------------------------------------------------------------- plan ---
def _plan_case(seed, B, page, width, extra, most, finish=0.2):
    r = np.random.default_rng(seed)
    cap_rows = width * page
    length = r.integers(0, max(1, cap_rows // 2), B)
    last = r.integers(0, 18, B)
    advance = np.array([r.integers(0, n + 1) for n in last])
    rows = np.array([r.integers(0, min(most, cap_rows - int(n + a)) + 1) for n, a in zip(length, advance)])
    held = np.minimum(-(-(length + last) // page), width)
    advance = np.minimum(advance, held * page - length)
    done = r.random(B) < finish
    length[done], advance[done], rows[done] = 0, 0, 0
    total = int(held.sum())
    need = -(-(length + advance + rows) // page)
    extra = extra + int(np.maximum(0, need - held).sum())
    ids = r.permutation(total + extra)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    cap = total + extra
    ring = np.full(cap, -7)
    head = int(r.integers(0, cap))
    ring[(head + np.arange(extra)) % cap] = ids[total:]
    i = lambda x: np.asarray(x, np.int32)  # noqa: E731
    return dict(length=i(length), advance=i(advance), rows=i(rows), held=i(held), free_state=i([head, extra]),
                free_ring=i(ring), block_table=i(table), page=page, max_rows=int(rows.sum()) + 3)


def _run_plan(dsv, c, in_place=False, stream=None):
    g = {k: _gpu(v) for k, v in c.items() if isinstance(v, np.ndarray)}
    ws = _ws()
    out = None
    if in_place:
        n = c["max_rows"]
        new = lambda k, t=torch.int32: torch.full((k,), 99, dtype=t, device="cuda")  # noqa: E731
        out = dict(length=g["length"], held=g["held"], free_state=g["free_state"],
                   row_offset=new(len(c["rows"]) + 1), row_request=new(n), position=new(n),
                   slot=new(n, torch.int64))
    o = dsv.dspark_plan_rows(g["length"], g["rows"], g["held"], g["free_state"], g["free_ring"], g["block_table"],
                             c["page"], c["max_rows"], advance=g["advance"], out=out, workspace=ws, stream=stream)
    code, detail = _code(ws)
    got = {k: v.cpu().numpy() for k, v in o.items()}
    got.update(block_table=g["block_table"].cpu().numpy(), free_ring=g["free_ring"].cpu().numpy())
    return got, code, detail


def _same_plan(got, want):
    for k, v in want.items():
        if k != "detail":
            np.testing.assert_array_equal(got[k], v, err_msg=k)


PLANS = [(1, 1, 5, 0, 1), (1, 16, 4, 3, 40), (7, 3, 30, 5, 17), (64, 16, 40, 9, 17), (511, 8, 20, 0, 9),
         (512, 16, 12, 1, 3), (513, 24, 10, 77, 60), (1500, 64, 6, 4, 200), (3, 16, 400, 2, 3000)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,width,extra,most", PLANS)
def test_plan_rows(dsv, B, page, width, extra, most, in_place):
    c = _plan_case(B + page, B, page, width, extra, most)
    got, code, _ = _run_plan(dsv, c, in_place)
    assert code == 0
    _same_plan(got, target.plan_rows(**c))


def test_plan_rows_without_rows_or_advance(dsv):
    c = _plan_case(3, 40, 16, 20, 5, 17)
    c["rows"][:] = 0
    c["max_rows"] = 0
    got, code, _ = _run_plan(dsv, c)
    assert code == 0
    _same_plan(got, target.plan_rows(**c))
    c = _plan_case(4, 40, 16, 20, 5, 17)
    c["advance"][:] = 0
    g = {k: _gpu(v) for k, v in c.items() if isinstance(v, np.ndarray)}
    o = dsv.dspark_plan_rows(g["length"], g["rows"], g["held"], g["free_state"], g["free_ring"], g["block_table"], 16,
                             c["max_rows"])
    want = target.plan_rows(**c)
    assert all((o[k].cpu().numpy() == want[k]).all() for k in o)


@pytest.mark.parametrize("B", [9, 700])
@pytest.mark.parametrize("detail", [1, 2, 3, 4])
def test_plan_rows_refuses_whole_steps(dsv, B, detail):
    c = _plan_case(5, B, 8, 20, 4, 17, finish=0.0)
    c["rows"][B // 2] = 1
    c["max_rows"] = int(c["rows"].sum())
    if detail == 1:
        c["length"][B - 1] = -1
    elif detail == 2:
        c["rows"][0] = 8 * 20 + 1
        c["max_rows"] += 200
    elif detail == 3:
        c["free_state"][1] = 0
    else:
        c["max_rows"] -= 1
    want = target.plan_rows(**c)
    assert want["detail"] == detail
    for in_place in (False, True):
        got, code, why = _run_plan(dsv, c, in_place)
        assert (code, why) == (6, detail)
        _same_plan(got, want)


# ------------------------------------------------------------------- write ---
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
@pytest.mark.parametrize("n,Hkv,D,page,fused", [(0, 2, 64, 16, False), (1, 1, 16, 1, False), (5, 3, 48, 7, True),
                                                (33, 8, 128, 16, True), (300, 4, 256, 24, True), (257, 2, 80, 64, False)])
def test_write_kv(dsv, dtype, cache, n, Hkv, D, page, fused):
    types = dict(bf16=torch.bfloat16, f32=torch.float32, e4m3=torch.float8_e4m3fn)
    g = torch.Generator().manual_seed(n + D)
    blocks = -(-n // page) + 3
    t = types[dtype]
    if fused:
        qkv = torch.randn((n, 3 * Hkv, D), generator=g).to(t).cuda()
        k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
    else:
        k, v = torch.randn((n, Hkv, D), generator=g).to(t).cuda(), torch.randn((n, Hkv, D), generator=g).to(t).cuda()
    if n > 4:
        k[1, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30], dtype=t)
        v[2, 0, :3] = torch.tensor([0.0, -0.0, 1e-30], dtype=t)
    kc = torch.randn((blocks, Hkv, page, D), generator=g).to(types[cache]).cuda()
    vc = torch.randn((blocks, Hkv, page, D), generator=g).to(types[cache]).cuda()
    ks = vs = None
    if cache == "e4m3":
        ks, vs = (torch.rand(Hkv, generator=g).cuda() + 0.01) * 0.02, torch.rand(Hkv, generator=g).cuda() + 0.01
    slot = torch.randperm(blocks * page, generator=g)[:n].cuda()
    slot[::5] = -1
    f = lambda x: x.detach().double().cpu().numpy()  # noqa: E731
    want = target.write_kv(f(k), f(v), slot.tolist(), f(kc), f(vc), None if ks is None else f(ks), None if vs is None else f(vs))
    ws = _ws()
    dsv.dspark_write_kv(k, v, slot, kc, vc, k_scale=ks, v_scale=vs, workspace=ws)
    assert _code(ws)[0] == 0
    np.testing.assert_array_equal(f(kc), want[0])
    np.testing.assert_array_equal(f(vc), want[1])


def test_write_kv_skips_slots_past_the_cache(dsv):
    k = torch.ones((4, 2, 64), device="cuda")
    kc, vc = torch.zeros((3, 2, 8, 64), device="cuda"), torch.zeros((3, 2, 8, 64), device="cuda")
    ws = _ws()
    dsv.dspark_write_kv(k, k, torch.tensor([0, 24, 1 << 40, 23], device="cuda"), kc, vc, workspace=ws)
    assert _code(ws) == [6, 1]
    assert kc.sum().item() == vc.sum().item() == 2 * 2 * 64 and kc[2, 0, 7, 0].item() == 1


# ------------------------------------------------------------------ attend ---
def _attend_case(seed, lens, Hq, Hkv, D, page, dtype, cache, window, poison=True):
    """lens: (keys before the step, rows) of each request.  Unused places of the cache hold
    values that would show if they were read into a result."""
    types = dict(bf16=torch.bfloat16, f32=torch.float32, e4m3=torch.float8_e4m3fn)
    g = torch.Generator().manual_seed(seed)
    pages = [-(-(n + r) // page) for n, r in lens]
    total = sum(pages)
    ids = torch.randperm(total + 3, generator=g)
    table = torch.full((len(lens), max(max(pages), 1) + 2), -5, dtype=torch.int32)
    shape = (total + 3, Hkv, page, D)
    kc, vc = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
    ks = vs = None
    if cache == "e4m3":
        kc, vc = kc * 60, vc * 60
        ks, vs = (torch.rand(Hkv, generator=g) + 0.5) / 60, (torch.rand(Hkv, generator=g) + 0.5) / 60
    at = 0
    seen = torch.zeros((total + 3, page), dtype=torch.bool)
    for b, (n, r) in enumerate(lens):
        table[b, :pages[b]] = ids[at:at + pages[b]].to(torch.int32)
        if pages[b]:
            flat = torch.arange(pages[b] * page) < n + r
            seen[ids[at:at + pages[b]]] = flat.view(-1, page)
        at += pages[b]
    if poison:
        kc[~seen[:, None].expand(-1, Hkv, -1)] = float("nan")
        vc[~seen[:, None].expand(-1, Hkv, -1)] = float("nan")
    offset = np.concatenate([[0], np.cumsum([r for _, r in lens])])
    t = types[dtype]
    q = (torch.randn((int(offset[-1]), Hq + 2, D), generator=g) * 2).to(t).cuda()[:, 1:1 + Hq]
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    return dict(q=q, row_offset=_gpu(offset.astype(np.int32)),
                length=torch.tensor([n for n, _ in lens], dtype=torch.int32).cuda(), block_table=table.cuda(),
                k_cache=kc.to(types[cache]).cuda(), v_cache=vc.to(types[cache]).cuda(), k_scale=dev(ks),
                v_scale=dev(vs), window=window, max_rows=max(max(r for _, r in lens), 1))


def _oracle(c, scale=None):
    f = lambda x: None if x is None else x.detach().double().cpu().numpy()  # noqa: E731
    i = lambda x: x.cpu().numpy().astype(np.int64)  # noqa: E731
    D = c["q"].shape[2]
    return target.paged_attention(f(c["q"]), i(c["row_offset"]), i(c["length"]), i(c["block_table"]), f(c["k_cache"]),
                                  f(c["v_cache"]), D ** -0.5 if scale is None else scale, c["window"], f(c["k_scale"]),
                                  f(c["v_scale"]))


def _check_attend(out, ref, dtype, D):
    bf16 = dtype == "bf16"
    n = ref["keys"][:, None]
    ds = (D + 8) * U * ref["size"] + 2.0 ** -21 + n * U
    tol = ref["weight"] * (2 * ds + (2.0 ** -11 if bf16 else 0.0))[..., None] + \
        np.abs(ref["out"]) * (torch.finfo(torch.bfloat16 if bf16 else torch.float32).eps / 2) + 1e-30
    err = np.abs(out["out"].double().cpu().numpy() - ref["out"])
    assert np.isfinite(err).all() and (err <= tol).all(), float((err / tol).max())
    lerr = np.abs(out["lse"].double().cpu().numpy() - ref["lse"])
    ltol = 2 * ds + np.abs(ref["lse"]) * 2.0 ** -22
    assert (lerr <= ltol).all(), float((lerr / ltol).max())


def _run_attend(dsv, c, **kw):
    ws = torch.full((dsv.load().dspark_paged_attention_workspace_size(c["q"].shape[2]),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    args = {k: c[k] for k in ("q", "row_offset", "length", "block_table", "k_cache", "v_cache", "max_rows", "window",
                              "k_scale", "v_scale")}
    out = dsv.dspark_paged_attention(**args, workspace=ws, **kw)
    return out, _code(ws)


KINDS = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")]
SHAPES = [  # lens, Hq, Hkv, D, page, window
    ("one key", [(0, 1)], 4, 2, 64, 16, 0),
    ("one row", [(300, 1)], 32, 8, 128, 16, 0),
    ("ragged", [(0, 3), (17, 1), (64, 8), (5, 0), (129, 5), (31, 1)], 8, 2, 128, 16, 0),
    ("no group", [(40, 2), (3, 1)], 3, 3, 96, 24, 0),
    ("wide group", [(200, 3), (7, 2)], 12, 1, 128, 16, 0),
    ("group of seven", [(90, 4), (1, 4)], 28, 4, 64, 32, 0),
    ("odd page", [(61, 2), (7, 7)], 4, 2, 48, 5, 0),
    ("page of one", [(20, 2)], 4, 4, 32, 1, 0),
    ("big page", [(20, 2), (300, 3)], 8, 4, 64, 256, 0),
    ("window", [(500, 4), (3, 2), (130, 6)], 8, 2, 128, 16, 100),
    ("window of one", [(50, 3)], 4, 2, 64, 16, 1),
    ("verify 17", [(100, 17), (33, 17), (0, 17), (250, 9)], 32, 8, 128, 16, 0),
    ("verify 17 window", [(400, 17), (2, 16)], 16, 2, 128, 32, 65),
    ("prompt", [(30, 150), (0, 77)], 8, 2, 128, 16, 0),
    ("wide heads", [(70, 5), (600, 1)], 4, 1, 256, 16, 0),
    ("wide heads, many rows", [(70, 33), (6, 1)], 4, 1, 256, 16, 0),
    ("small heads", [(70, 5), (600, 1)], 8, 4, 16, 16, 0),
    ("odd heads", [(70, 20), (9, 3)], 10, 2, 80, 16, 0),
]


@pytest.mark.parametrize("dtype,cache", KINDS, ids=["-".join(k) for k in KINDS])
@pytest.mark.parametrize("name,lens,Hq,Hkv,D,page,window", SHAPES, ids=[s[0] for s in SHAPES])
def test_attention(dsv, name, lens, Hq, Hkv, D, page, window, dtype, cache):
    c = _attend_case(len(name), lens, Hq, Hkv, D, page, dtype, cache, window)
    out, code = _run_attend(dsv, c)
    assert code[0] == 0
    _check_attend(out, _oracle(c), dtype, D)


@pytest.mark.parametrize("dtype,cache", KINDS, ids=["-".join(k) for k in KINDS])
@pytest.mark.parametrize("rows,Hq", [(1, 8), (8, 8), (17, 32)])
def test_attention_split_over_many_blocks(dsv, dtype, cache, rows, Hq):
    """One long request next to short ones: its keys go to many blocks and are joined."""
    c = _attend_case(7, [(9000, rows), (1, 1), (700, rows), (0, 1)], Hq, Hq // 4, 128, 16, dtype, cache, 0)
    out, code = _run_attend(dsv, c)
    assert code[0] == 0
    ref = _oracle(c)
    _check_attend(out, ref, dtype, 128)
    again, _ = _run_attend(dsv, c)
    assert torch.equal(out["out"], again["out"]) and torch.equal(out["lse"], again["lse"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,Hq,D", [(4, 4, 64), (4, 16, 128), (17, 32, 128)])
def test_hidden_keys_may_hold_anything(dsv, dtype, rows, Hq, D):
    """NaN and infinities at the step's later rows do not reach the earlier ones."""
    c = _attend_case(11, [(37, rows), (64, rows)], Hq, 4, D, 16, dtype, dtype, 0)
    want, _ = _run_attend(dsv, c)
    for b, (n, last) in enumerate([(37, 37 + rows - 1), (64, 64 + rows - 1)]):
        blk = c["block_table"][b, last // 16]
        c["k_cache"][blk, :, last % 16] = float("nan")
        c["v_cache"][blk, :, last % 16] = float("inf") if b else float("nan")
    got, _ = _run_attend(dsv, c)
    keep = [i for i in range(2 * rows) if i % rows != rows - 1]
    assert torch.equal(got["out"][keep], want["out"][keep]) and torch.equal(got["lse"][keep], want["lse"][keep])
    assert torch.isnan(got["out"][rows - 1]).all() and torch.isnan(got["lse"][rows - 1]).all()


@pytest.mark.parametrize("rows,Hq,D", [(4, 8, 64), (3, 32, 128), (17, 32, 128)])
def test_hidden_keys_of_an_8_bit_cache(dsv, rows, Hq, D):
    c = _attend_case(12, [(37, rows), (64, rows)], Hq, 4, D, 16, "bf16", "e4m3", 0)
    want, _ = _run_attend(dsv, c)
    nan = torch.tensor(0x7F, dtype=torch.uint8, device="cuda")
    for b, last in enumerate([37 + rows - 1, 64 + rows - 1]):
        blk = c["block_table"][b, last // 16]
        c["k_cache"].view(torch.uint8)[blk, :, last % 16] = nan
        c["v_cache"].view(torch.uint8)[blk, :, last % 16] = nan
    got, _ = _run_attend(dsv, c)
    keep = [i for i in range(2 * rows) if i % rows != rows - 1]
    assert torch.equal(got["out"][keep], want["out"][keep]) and torch.equal(got["lse"][keep], want["lse"][keep])
    assert torch.isnan(got["out"][rows - 1]).all()


@pytest.mark.parametrize("dtype,cache", KINDS, ids=["-".join(k) for k in KINDS])
@pytest.mark.parametrize("scale", [-0.25, 0.0, 1.5])
def test_attention_scales(dsv, dtype, cache, scale):
    c = _attend_case(17, [(70, 4), (3, 1), (0, 17)], 16, 4, 64, 16, dtype, cache, 40)
    out, code = _run_attend(dsv, c, scale=scale)
    assert code[0] == 0
    _check_attend(out, _oracle(c, scale), dtype, 64)


@pytest.mark.parametrize("page", [3, 12, 16])
def test_attention_of_many_rows_on_any_page(dsv, page):
    c = _attend_case(18, [(150, 30), (0, 20), (301, 7)], 8, 2, 128, page, "bf16", "bf16", 0)
    out, code = _run_attend(dsv, c)
    assert code[0] == 0
    _check_attend(out, _oracle(c), "bf16", 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_scores(dsv, dtype):
    """Scores of the type's range, and keys that score -inf."""
    c = _attend_case(13, [(40, 2)], 4, 2, 64, 16, dtype, dtype, 0)
    c["q"][0] *= 1e4
    c["q"][1, :, :] = 1.0
    blk = int(c["block_table"][0, 1])
    c["k_cache"][blk, :, 3] = -float("inf")
    c["q"][0] = c["q"][0].abs()
    out, _ = _run_attend(dsv, c)
    with np.errstate(all="ignore"):
        ref = _oracle(c)
    assert torch.isfinite(out["out"]).all()
    size = np.where(np.isfinite(ref["size"]), ref["size"], 1e5 * 64)
    _check_attend(out, dict(ref, size=size), dtype, 64)
    # every key at -inf: nothing to attend to
    c = _attend_case(14, [(20, 1)], 4, 2, 64, 16, dtype, dtype, 0)
    c["q"][:] = 1.0
    c["k_cache"][:] = -float("inf")
    out, _ = _run_attend(dsv, c)
    assert (out["out"] == 0).all() and torch.isneginf(out["lse"]).all()


def test_attention_status_and_untouched_rows(dsv):
    c = _attend_case(15, [(20, 2), (30, 3), (9, 2)], 8, 2, 64, 16, "bf16", "bf16", 0)
    want, _ = _run_attend(dsv, c)
    fill = lambda: dict(out=torch.full((9, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                        lse=torch.full((9, 8), 7.0, device="cuda"))
    c["q"] = torch.cat([c["q"], c["q"][:2]])
    out, code = _run_attend(dsv, c, out=fill())
    assert code[0] == 0 and (out["out"][7:] == 7).all() and (out["lse"][7:] == 7).all()
    assert torch.equal(out["out"][:7], want["out"])
    # a request longer than its table, one with more rows than max_rows: only they are left out
    bad = dict(c, length=torch.tensor([20, 10 ** 6, 9], dtype=torch.int32, device="cuda"))
    out, code = _run_attend(dsv, bad, out=fill())
    assert code == [6, 1] and (out["out"][2:5] == 7).all()
    assert torch.equal(out["out"][:2], want["out"][:2]) and torch.equal(out["out"][5:7], want["out"][5:])
    out, code = _run_attend(dsv, dict(c, max_rows=2), out=fill())
    assert code == [6, 1] and (out["out"][2:5] == 7).all() and torch.equal(out["out"][:2], want["out"][:2])
    # offsets that go backwards or past q
    for off in ([0, 5, 2, 7], [0, 2, 5, 100], [-4, 2, 5, 7]):
        out, code = _run_attend(dsv, dict(c, row_offset=torch.tensor(off, dtype=torch.int32, device="cuda")), out=fill())
        assert code == [6, 1]
    # a page outside the cache is told, and page 0 read in its place
    table = c["block_table"].clone()
    table[0, 0] = 10 ** 6
    table[2, 0] = -1
    out, code = _run_attend(dsv, dict(c, block_table=table), out=fill())
    assert code == [6, 2] and torch.equal(out["out"][2:5], want["out"][2:5])
    # without lse
    out = dsv.dspark_paged_attention(c["q"], c["row_offset"], c["length"], c["block_table"], c["k_cache"], c["v_cache"],
                                     3, out=dict(out=torch.empty((9, 8, 64), dtype=torch.bfloat16, device="cuda")))
    assert torch.equal(out["out"][:7], want["out"])


def test_far_places_of_a_large_cache(dsv):
    """Element offsets past 2^31: the pages of one request lie at the end of an 8 GB cache."""
    blocks, Hkv, page, D = 130000, 8, 32, 128                       # 4.26e9 elements of 8 bits
    kc = torch.zeros((blocks, Hkv, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc = torch.zeros_like(kc.view(torch.uint8)).view(torch.float8_e4m3fn)
    one = torch.ones(Hkv, device="cuda")
    ids = [blocks - 1, 66000, blocks - 7]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    k = torch.randn((80, Hkv, D), generator=g).to(torch.bfloat16).cuda()
    v = torch.randn((80, Hkv, D), generator=g).to(torch.bfloat16).cuda()
    slot = torch.tensor([ids[i // page] * page + i % page for i in range(80)], device="cuda")
    dsv.dspark_write_kv(k, v, slot, kc, vc, k_scale=one, v_scale=one)
    for rows in (1, 17):
        q = torch.randn((rows, 32, D), generator=g).to(torch.bfloat16).cuda()
        off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        n = torch.tensor([80 - rows], dtype=torch.int32, device="cuda")
        out = dsv.dspark_paged_attention(q, off, n, table, kc, vc, rows, k_scale=one, v_scale=one)
        small = [x[torch.tensor(ids, device="cuda")].contiguous() for x in (kc.view(torch.uint8), vc.view(torch.uint8))]
        near = dsv.dspark_paged_attention(q, off, n, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"),
                                          small[0].view(torch.float8_e4m3fn), small[1].view(torch.float8_e4m3fn), rows,
                                          k_scale=one, v_scale=one)
        assert torch.equal(out["out"], near["out"]) and out["out"].abs().max() > 0


# ------------------------------------------------------------------ adjust ---
def _adjust_case(seed, B, R, V, dtype, L, bias, masks, ell=True, draft=True):
    r = np.random.default_rng(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    logits = torch.from_numpy(r.normal(size=(B, R, V)) * 3).to(t)
    pick = np.unique(np.concatenate([[0, V - 1], r.integers(0, V, 40)]))       # few tokens: many repeats
    c = dict(logits=logits, history=None, prompt_len=None, history_len=None, draft=None, ell=None, repetition=None,
             frequency=None, presence=None, bias_token=None, bias_value=None, mask_row=None, mask=None)
    i = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32))  # noqa: E731
    if L:
        n = r.integers(0, L + 1, B)
        n[0] = L
        c.update(history=i(r.choice(pick, (B, L))), history_len=i(n), prompt_len=i([r.integers(0, x + 1) for x in n]))
    if draft and R > 1:
        c["draft"] = i(r.choice(pick, (B, R - 1)))
    if ell:
        c["ell"] = i(r.integers(0, R, B))
    for k in ("repetition", "frequency", "presence"):
        c[k] = torch.from_numpy(r.uniform(0.5, 1.7, B).astype(np.float32))
    if bias:
        c["bias_token"] = i(r.choice(np.concatenate([pick, [-1]]), (B, bias)))
        c["bias_value"] = torch.from_numpy(r.normal(size=(B, bias)).astype(np.float32) * 4)
    if masks:
        words = r.integers(-2 ** 31, 2 ** 31, (masks, -(-V // 32)))
        words[0] = 0                                                            # allows nothing
        c["mask"], c["mask_row"] = i(words), i(r.integers(-1, masks, (B, R)))
    return c


def _check_adjust(got, c, fill):
    """Every step of the definition rounds once in float32, relative to the largest value on the way."""
    f = lambda x: None if x is None else x.double().numpy() if x.is_floating_point() else x.numpy()  # noqa: E731
    n = {k: f(v) for k, v in c.items()}
    with np.errstate(all="ignore"):
        want = target.adjust_logits(out=np.full(n["logits"].shape, fill), **n)
    got = got.double().cpu().numpy()
    inf = ~np.isfinite(want)
    np.testing.assert_array_equal(got[inf], want[inf])
    eps = torch.finfo(c["logits"].dtype).eps / 2
    big = np.abs(n["logits"]).max() * 2 + 1.7 * (3000 + 1) + (np.abs(n["bias_value"]).sum(-1).max() if c["bias_value"] is not None else 0)
    touched = want != n["logits"]
    tol = np.abs(want) * eps + touched * big * 40 * U
    assert (np.abs(got[~inf] - want[~inf]) <= tol[~inf]).all()


ADJUST = [(1, 1, 8, 5, 0, 0), (1, 1, 1000, 0, 3, 2), (3, 4, 5000, 300, 0, 0), (2, 8, 40000, 2500, 20, 5),
          (5, 33, 1032, 60, 2047, 3), (40, 2, 33000, 17, 1, 1), (300, 1, 4104, 9, 4, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,R,V,L,bias,masks", ADJUST)
def test_adjust_logits(dsv, B, R, V, L, bias, masks, dtype):
    c = _adjust_case(B + V, B, R, V, dtype, L, bias, masks)
    g = {k: v.cuda() if v is not None else None for k, v in c.items()}
    ws = _ws()
    out = torch.full_like(g["logits"], 5.0)
    dsv.dspark_adjust_logits(**g, out=out, workspace=ws)
    assert _code(ws)[0] == 0
    _check_adjust(out, c, 5.0)
    inplace = g["logits"].clone()
    dsv.dspark_adjust_logits(**{**g, "logits": inplace}, out=inplace)
    wanted = torch.arange(R, device="cuda")[None] <= g["ell"][:, None]
    assert torch.equal(inplace[wanted], out[wanted]) and torch.equal(inplace[~wanted], g["logits"][~wanted])


def test_adjust_with_nothing_on_copies_bits(dsv):
    x = torch.randn((2, 3, 4096), device="cuda").to(torch.bfloat16)
    x[0, 0, :3] = torch.tensor([float("nan"), float("inf"), -0.0], dtype=torch.bfloat16)
    out = dsv.dspark_adjust_logits(x)
    assert torch.equal(out.view(torch.int16), x.view(torch.int16))
    # a mask covers whatever stands there
    mask = torch.full((1, 128), -1, dtype=torch.int32, device="cuda")
    mask[0, 0] = ~0b101
    out = dsv.dspark_adjust_logits(x, mask=mask, mask_row=torch.zeros((2, 3), dtype=torch.int32, device="cuda"))
    assert torch.isneginf(out[:, :, 0]).all() and torch.isneginf(out[:, :, 2]).all()
    assert torch.equal(out[:, :, 3:], x[:, :, 3:]) and torch.equal(out[:, :, 1], x[:, :, 1])


def test_adjust_status(dsv):
    def run(**kw):
        c = _adjust_case(3, 2, 3, 2000, "f32", 50, 4, 2)
        c["ell"] = torch.tensor([2, 2], dtype=torch.int32)
        c["history_len"] = torch.tensor([50, 50], dtype=torch.int32)
        c["prompt_len"] = torch.tensor([10, 10], dtype=torch.int32)
        for k, (at, x) in kw.items():
            c[k][at] = x
        g = {k: v.cuda() if v is not None else None for k, v in c.items()}
        ws = _ws()
        out = torch.full_like(g["logits"], 5.0)
        dsv.dspark_adjust_logits(**g, out=out, workspace=ws)
        return out, _code(ws), c
    for at in (-1, 3):
        out, code, _ = run(ell=(1, at))
        assert code == [6, 1] and (out[1] == 5).all()
    assert run(history_len=(0, 51))[1] == [6, 2] and run(prompt_len=(0, 51))[1] == [6, 2]
    assert run(prompt_len=(0, -1))[1] == [6, 2]
    for at in (2000, -1, 2 ** 31 - 1):
        assert run(history=((1, 7), at))[1] == [6, 3] and run(draft=((1, 0), at))[1] == [6, 3]
    assert run(bias_token=((0, 1), -2))[1] == [6, 4] and run(bias_token=((0, 1), 2000))[1] == [6, 4]
    out, code, c = run(mask_row=((0, 1), 2))
    assert code == [6, 5]
    c["mask_row"][0, 1] = -1
    _check_adjust(out, c, 5.0)


# ------------------------------------------------------- streams and graphs ---
def test_on_another_stream_and_in_a_graph(dsv):
    c = _attend_case(21, [(300, 4), (20, 2)], 8, 2, 128, 16, "bf16", "bf16", 0)
    want, _ = _run_attend(dsv, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = {k: c[k] for k in ("q", "row_offset", "length", "block_table", "k_cache", "v_cache", "max_rows")}
    got = dsv.dspark_paged_attention(**args, stream=s)
    s.synchronize()
    assert torch.equal(got["out"], want["out"])
    # one captured call, replayed with other lengths
    ws = torch.empty(dsv.load().dspark_paged_attention_workspace_size(128), dtype=torch.uint8, device="cuda")
    out = dict(out=torch.zeros_like(want["out"]), lse=torch.zeros_like(want["lse"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsv.dspark_paged_attention(**args, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["out"], want["out"])
    c["length"].copy_(torch.tensor([100, 7], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    _check_attend(out, _oracle(c), "bf16", 128)
