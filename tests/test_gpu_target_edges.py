"""Edges of the target model's side of a round: values that are not finite at visible keys, windows
whose early pages are gone, refusals by every reason, empty steps, other streams, graphs and one
workspace for many calls.  The bounds of attention are those of test_gpu_target.py's text.
"""
import numpy as np
import pytest
import torch

from oracle import target
from tests.test_gpu_target import (KINDS, U, _adjust_case, _attend_case, _check_attend, _code, _gpu, _oracle, _plan_case,
                                   _run_attend, _run_plan, _same_plan, _ws, dsv)  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attend ---
# lens, Hq, Hkv, D: 17 rows of groups of four and more go to 128-row tiles, the others to 16-row ones
VISIBLE = [([(900, 1), (130, 1)], 8, 4, 64), ([(900, 4), (130, 4)], 8, 4, 128), ([(900, 2)], 4, 4, 256),
           ([(900, 17), (130, 17)], 32, 8, 128), ([(900, 17)], 16, 2, 64), ([(9000, 1)], 8, 2, 128),
           ([(9000, 17)], 32, 8, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hkv,D", VISIBLE)
def test_infinite_values_at_visible_keys(dsv, lens, Hq, Hkv, D, dtype):  # noqa: F811
    """A weight is positive, so a value of +-inf makes its column +-inf wherever its key stands, both
    signs make it NaN, and the other columns stay as they are."""
    c = _attend_case(31, lens, Hq, Hkv, D, 16, dtype, dtype, 0)
    inf = float("inf")
    for b, (n, r) in enumerate(lens):
        places = [0, 5, n // 3, n // 2 + 1, n - 70, n - 1, n, n + r - 1]
        for i, p in enumerate(places):
            blk = int(c["block_table"][b, p // 16])
            c["v_cache"][blk, :, p % 16, 3 * i] = -inf if i & 1 else inf
        for p, x in ((n // 4, inf), (n // 4 + 1, -inf)):
            c["v_cache"][int(c["block_table"][b, p // 16]), :, p % 16, 31] = x
    out, code = _run_attend(dsv, c)
    assert code[0] == 0
    with np.errstate(invalid="ignore"):
        ref = _oracle(c)
    odd = ~np.isfinite(ref["out"])
    assert np.isposinf(ref["out"]).any() and np.isneginf(ref["out"]).any() and np.isnan(ref["out"]).any()
    got = out["out"].double().cpu().numpy()
    np.testing.assert_array_equal(got[odd], ref["out"][odd])
    rest = dict(ref, out=np.where(odd, 0.0, ref["out"]), weight=np.where(odd, 0.0, ref["weight"]))
    _check_attend(dict(out, out=torch.from_numpy(np.where(odd, 0.0, got))), rest, dtype, D)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_hidden_values_in_later_units(dsv, value):  # noqa: F811
    """Pieces of several units of 128 keys, the last row's value (in the last of them) not finite."""
    rows, B = 17, 20
    lens = [(900 + 13 * b, rows) for b in range(B)]
    c = _attend_case(32, lens, 32, 8, 128, 16, "bf16", "bf16", 0)
    want, _ = _run_attend(dsv, c)
    for b, (n, _r) in enumerate(lens):
        last = n + rows - 1
        c["v_cache"][int(c["block_table"][b, last // 16]), :, last % 16] = value
    got, _ = _run_attend(dsv, c)
    keep = [i for i in range(B * rows) if i % rows != rows - 1]
    assert torch.equal(got["out"][keep], want["out"][keep]) and torch.equal(got["lse"], want["lse"])
    last = got["out"][rows - 1::rows].float()
    assert torch.isnan(last).all() if value != value else torch.isposinf(last).all()


WINDOWS = [  # lens, Hq, Hkv, D, page, window
    ([(500, 1), (37, 1)], 8, 2, 128, 16, 100), ([(500, 4), (70, 3)], 8, 2, 64, 16, 33), ([(300, 3)], 4, 2, 48, 5, 41),
    ([(90, 2)], 4, 4, 32, 1, 7), ([(1000, 3)], 8, 4, 64, 256, 300), ([(700, 17), (140, 17)], 32, 8, 128, 16, 130),
    ([(700, 17)], 16, 2, 64, 8, 65), ([(1100, 17)], 32, 8, 128, 32, 500), ([(600, 2)], 4, 1, 256, 24, 200),
    ([(5000, 4)], 8, 2, 128, 16, 1500)]


@pytest.mark.parametrize("dtype,cache", KINDS, ids=["-".join(k) for k in KINDS])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page,window", WINDOWS)
def test_pages_before_the_window_may_be_gone(dsv, lens, Hq, Hkv, D, page, window, dtype, cache):  # noqa: F811
    if cache == "e4m3" and D % 16:
        pytest.skip("8-bit heads are multiples of 16")
    c = _attend_case(33, lens, Hq, Hkv, D, page, dtype, cache, window)
    want, code = _run_attend(dsv, c)
    assert code[0] == 0
    _check_attend(want, _oracle(c), dtype, D)
    gone = 0
    for b, (n, _r) in enumerate(lens):
        first = max(0, n - window + 1)                       # the first key that any row of the step sees
        c["block_table"][b, :first // page] = -1
        gone += first // page
    assert gone > 0
    got, code = _run_attend(dsv, c)
    assert code[0] == 0
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_attention_of_an_empty_step(dsv):  # noqa: F811
    c = _attend_case(34, [(20, 0), (3, 0)], 4, 2, 64, 16, "bf16", "bf16", 0)
    out, code = _run_attend(dsv, dict(c, max_rows=0))
    assert code[0] == 0 and out["out"].shape == (0, 4, 64)


@pytest.mark.parametrize("dtype,cache", KINDS, ids=["-".join(k) for k in KINDS])
@pytest.mark.parametrize("rows,Hq", [(1, 8), (6, 8), (17, 32)])
def test_lse_bound(dsv, dtype, cache, rows, Hq):  # noqa: F811
    """|lse - exact| <= (D + 8) u A + 2^-20 + 2 n u + |exact| 2^-22: half of what the scores' term is
    allowed elsewhere."""
    D = 128
    c = _attend_case(35, [(700, rows), (40, rows)], Hq, Hq // 4, D, 16, dtype, cache, 0)
    out, _ = _run_attend(dsv, c)
    ref = _oracle(c)
    err = np.abs(out["lse"].double().cpu().numpy() - ref["lse"])
    tol = (D + 8) * U * ref["size"] + 2.0 ** -20 + 2 * ref["keys"][:, None] * U + np.abs(ref["lse"]) * 2.0 ** -22
    assert (err <= tol).all(), float((err / tol).max())


def _dense(c):
    """The oracle of one request by dense float64 products on the GPU (for thousands of rows)."""
    q, page, D = c["q"].double(), c["k_cache"].shape[2], c["q"].shape[2]
    n, Hq = q.shape[:2]
    total = int(c["length"][0]) + n
    ids = c["block_table"][0, :-(-total // page)].long()
    Hkv = c["k_cache"].shape[1]
    out, weight = torch.empty_like(q), torch.empty_like(q)
    lse, size = (torch.empty((n, Hq), dtype=torch.float64, device="cuda") for _ in range(2))
    hide = torch.arange(total, device="cuda")[None] > (total - n + torch.arange(n, device="cuda"))[:, None]
    for h in range(Hq):
        g = h // (Hq // Hkv)
        k, v = (x[ids, g].double().reshape(-1, D)[:total] * (1.0 if s is None else s[g].double())
                for x, s in ((c["k_cache"], c["k_scale"]), (c["v_cache"], c["v_scale"])))
        s = (q[:, h] @ k.T * D ** -0.5).masked_fill(hide, -float("inf"))
        lse[:, h] = torch.logsumexp(s, 1)
        p = torch.exp(s - lse[:, h, None])
        out[:, h], weight[:, h] = p @ v, p @ v.abs()
        size[:, h] = (q[:, h].abs() @ k.abs().T * D ** -0.5).masked_fill(hide, 0).amax(1)
    np_ = lambda x: x.cpu().numpy()  # noqa: E731
    return dict(out=np_(out), lse=np_(lse), weight=np_(weight), size=np_(size), keys=total - n + 1 + np.arange(n))


@pytest.mark.parametrize("dtype,cache", KINDS, ids=["-".join(k) for k in KINDS])
@pytest.mark.parametrize("before,rows,Hq,Hkv,D", [(0, 2500, 8, 2, 64), (777, 1300, 4, 1, 128), (100, 600, 4, 2, 256)])
def test_prompts_of_thousands_of_rows(dsv, dtype, cache, before, rows, Hq, Hkv, D):  # noqa: F811
    c = _attend_case(36, [(before, rows)], Hq, Hkv, D, 16, dtype, cache, 0, poison=False)
    out, code = _run_attend(dsv, c)
    assert code[0] == 0
    _check_attend(out, _dense(c), dtype, D)


# -------------------------------------------------------------------- plan ---
@pytest.mark.parametrize("B,first,second", [(1500, 3, 1027), (1500, 1027, 3), (9, 1, 2), (2100, 2049, 1025)])
def test_plan_tells_the_first_reason(dsv, B, first, second):  # noqa: F811
    """An inconsistent request (detail 1) and a full table (2) in one step: 1, whichever comes first."""
    c = _plan_case(41, B, 8, 20, 4, 17, finish=0.0)
    c["length"][first] = -1
    c["rows"][second] = 8 * 20 + 1
    c["max_rows"] = int(c["rows"].sum()) + 1
    want = target.plan_rows(**c)
    assert want["detail"] == 1
    got, code, why = _run_plan(dsv, c)
    assert (code, why) == (6, 1)
    _same_plan(got, want)


@pytest.mark.parametrize("B", [9, 1500])
def test_plan_refuses_a_negative_advance(dsv, B):  # noqa: F811
    c = _plan_case(42, B, 8, 20, 4, 17, finish=0.0)
    c["length"][B - 1], c["advance"][B - 1] = 5, -1
    got, code, why = _run_plan(dsv, c)
    assert (code, why) == (6, 1)
    want = target.plan_rows(**c)
    assert want["detail"] == 1
    _same_plan(got, want)


@pytest.mark.parametrize("B", [9, 1500])
@pytest.mark.parametrize("where", ["table", "ring"])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_plan_tells_pages_outside_the_cache(dsv, B, where, bad):  # noqa: F811
    c = _plan_case(43, B, 8, 20, 4, 17, finish=0.0)
    clean = target.plan_rows(**c)
    base = c["length"] + c["advance"]
    need = -(-(base + c["rows"]) // 8)
    if where == "table":
        b = next(b for b in range(B) if base[b] % 8 and c["rows"][b] and base[b] // 8 < c["held"][b])
        page = base[b] // 8
        c["block_table"][b, page] = bad
    else:
        b = next(b for b in range(B) if need[b] > c["held"][b])
        page = c["held"][b]
        head = c["free_state"][0] + int(np.maximum(0, need - c["held"])[:b].sum())
        c["free_ring"][head % len(c["free_ring"])] = bad
    hit = (clean["row_request"] == b) & (clean["position"] // 8 == page)
    assert hit.any()
    want = target.plan_rows(**c)
    want["slot"][hit] = -1
    got, code, why = _run_plan(dsv, c)
    assert (code, why) == (6, 5)
    _same_plan(got, want)


# ------------------------------------------------------------------- write ---
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.0625, 2.0 ** -140, 3.0e38])
def test_write_ties_and_far_scales(dsv, dtype, scale):  # noqa: F811
    """Scales of a power of two make a sixteenth of bf16 rows exact ties; scales whose reciprocal is not
    a normal number take the quotient proper."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(51)
    k = (torch.randn((90, 2, 64), generator=g) * 50 * min(scale, 1e30)).to(t).cuda()
    kc, vc = (torch.zeros((8, 2, 16, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    s = torch.full((2,), scale, device="cuda")
    slot = torch.randperm(128, generator=g)[:90].cuda()
    dsv.dspark_write_kv(k, k, slot, kc, vc, k_scale=s, v_scale=s)
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    zero = np.zeros((8, 2, 16, 64))
    want = target.write_kv(f(k), f(k), slot.tolist(), zero, zero, f(s), f(s))[0]
    np.testing.assert_array_equal(f(kc), want)
    np.testing.assert_array_equal(f(vc), want)


# ------------------------------------------------------------------ adjust ---
def _adjust_bound(c, fill):
    """The oracle and each element's bound: every float32 operation of the definition rounds its own
    result by 2^-24, and the output's type rounds once."""
    n = {k: None if v is None else v.double().numpy() if v.is_floating_point() else v.numpy() for k, v in c.items()}
    with np.errstate(all="ignore"):
        want = target.adjust_logits(out=np.full(n["logits"].shape, fill), **n)
    B, R, V = n["logits"].shape
    tol = np.zeros((B, R, V))
    for b in range(B):
        p, h = (int(n[k][b]) if n[k] is not None else 0 for k in ("prompt_len", "history_len"))
        count, seen = np.zeros(V), np.zeros(V, bool)
        if h:
            seen[n["history"][b, :h]] = True
            np.add.at(count, n["history"][b, p:h], 1)
        bias, size, many = np.zeros(V), np.zeros(V), np.zeros(V)
        if n["bias_token"] is not None:
            live = n["bias_token"][b] >= 0
            np.add.at(bias, n["bias_token"][b][live], n["bias_value"][b][live])
            np.add.at(size, n["bias_token"][b][live], np.abs(n["bias_value"][b][live]))
            np.add.at(many, n["bias_token"][b][live], 1)
        for k in range(R):
            if k:
                count[n["draft"][b, k - 1]] += 1
                seen[n["draft"][b, k - 1]] = True
            x = n["logits"][b, k]
            y = np.where(seen, np.where(x > 0, x / n["repetition"][b], x * n["repetition"][b]), x)
            e = np.where(seen, np.abs(y), 0)
            y = y - n["frequency"][b] * count
            e += np.where(count > 0, n["frequency"][b] * count + np.abs(y), 0)
            y = np.where(count > 0, y - n["presence"][b], y)
            e += np.where(count > 0, np.abs(y), 0)
            y = y + bias
            e += np.where(many > 0, np.maximum(many - 1, 0) * size + np.abs(y), 0)
            tol[b, k] = 1.01 * U * e
    return want, tol + np.abs(np.where(np.isfinite(want), want, 0)) * torch.finfo(c["logits"].dtype).eps / 2 * (tol > 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,R,V,L,bias,masks", [(1, 1, 1000, 5, 3, 0), (3, 4, 5000, 300, 0, 2), (2, 8, 40000, 2500, 20, 5),
                                                (40, 2, 33000, 17, 1, 1)])
def test_adjust_within_its_own_roundings(dsv, B, R, V, L, bias, masks, dtype):  # noqa: F811
    c = _adjust_case(61 + B, B, R, V, dtype, L, bias, masks, ell=False)
    want, tol = _adjust_bound(c, 0.0)
    got = dsv.dspark_adjust_logits(**{k: v if v is None else v.cuda() for k, v in c.items()}).double().cpu().numpy()
    inf = ~np.isfinite(want)
    np.testing.assert_array_equal(got[inf], want[inf])
    err = np.abs(np.where(inf, 0, got - np.where(inf, 0, want)))
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-30)).max())


def test_adjust_with_a_history_of_no_columns(dsv):  # noqa: F811
    """Requests without a token yet: the history has no columns, and its lengths are zero."""
    c = _adjust_case(62, 3, 2, 512, "f32", 0, 2, 0)
    g = {k: v if v is None else v.cuda() for k, v in c.items()}
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = _ws()
    want = dsv.dspark_adjust_logits(**g, out=torch.zeros_like(g["logits"]))
    g.update(history=torch.zeros((3, 0), dtype=torch.int32, device="cuda"), history_len=none, prompt_len=none)
    got = dsv.dspark_adjust_logits(**g, out=torch.zeros_like(g["logits"]), workspace=ws)
    assert _code(ws)[0] == 0 and torch.equal(got, want)
    g["history_len"] = none + 1
    dsv.dspark_adjust_logits(**g, out=torch.zeros_like(g["logits"]), workspace=ws)
    assert _code(ws) == [6, 2]


# ---------------------------------------------- streams, graphs, workspaces ---
def _sleep(ms=50):
    torch.cuda._sleep(int(ms * 2e6))


@pytest.mark.parametrize("call", ["plan", "attend", "adjust"])
def test_memory_made_for_another_stream(dsv, call):  # noqa: F811
    """Memory that the current stream has still to read is not what a call on another stream writes."""
    side = torch.cuda.Stream()
    if call == "plan":
        c = _plan_case(71, 2000, 16, 40, 9, 17)
        g = {k: _gpu(v) for k, v in c.items() if isinstance(v, np.ndarray)}
        run = lambda s: dsv.dspark_plan_rows(g["length"], g["rows"], g["held"], g["free_state"], g["free_ring"],  # noqa: E731
                                             g["block_table"], 16, c["max_rows"], advance=g["advance"], stream=s)["slot"]
        size, dtype = (c["max_rows"],), torch.int64
    elif call == "attend":
        c = _attend_case(72, [(300, 64), (20, 2)], 8, 2, 128, 16, "bf16", "bf16", 0)
        args = {k: c[k] for k in ("q", "row_offset", "length", "block_table", "k_cache", "v_cache", "max_rows")}
        run = lambda s: dsv.dspark_paged_attention(**args, stream=s)["out"]  # noqa: E731
        size, dtype = c["q"].shape, torch.bfloat16
    else:
        x = torch.randn((4, 3, 40000), device="cuda")
        run = lambda s: dsv.dspark_adjust_logits(x, stream=s)  # noqa: E731
        size, dtype = x.shape, torch.float32
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.full(size, 77, dtype=dtype, device="cuda")
    later = torch.zeros_like(old)
    _sleep()
    later.copy_(old)
    del old                                              # its memory is free for the current stream's next use
    out = run(side)
    torch.cuda.synchronize()
    assert (later == 77).all() and not (out == 77).all()


def _write_case(seed, n=40):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn((n, 8, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    slot = torch.randperm(6 * 16, generator=g)[:n].cuda()
    want = torch.zeros((2, 6, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    for x, to in ((k, want[0]), (v, want[1])):
        to[slot // 16, :, slot % 16] = x
    return k, v, slot, want


@pytest.mark.parametrize("n", [3, 40, 90])
def test_write_in_a_graph_and_on_another_stream(dsv, n):  # noqa: F811
    k, v, slot, want = _write_case(81, n)
    kc, vc = torch.zeros_like(want[0]), torch.zeros_like(want[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dsv.dspark_write_kv(k, v, slot, kc, vc, stream=s)
    s.synchronize()
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    ws, graph = _ws(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsv.dspark_write_kv(k, v, slot, kc, vc, workspace=ws)
    for seed in (82, 83):
        k2, v2, slot2, want = _write_case(seed, n)
        k.copy_(k2), v.copy_(v2), slot.copy_(slot2), kc.zero_(), vc.zero_()
        graph.replay()
        assert _code(ws)[0] == 0 and torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    slot[0] = 96                                         # past the cache: told by the replay, gone in the next
    graph.replay()
    assert _code(ws) == [6, 1]
    slot[0] = -1
    graph.replay()
    assert _code(ws)[0] == 0


@pytest.mark.parametrize("B", [5, 700, 1500])
def test_plan_in_a_graph_and_on_another_stream(dsv, B):  # noqa: F811
    c = _plan_case(84, B, 16, 40, 9, 17)
    names = [k for k, v in c.items() if isinstance(v, np.ndarray)]
    g = {k: _gpu(c[k]) for k in names}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dsv.dspark_plan_rows(g["length"], g["rows"], g["held"], g["free_state"], g["free_ring"], g["block_table"], 16,
                               c["max_rows"], advance=g["advance"], stream=s)
    s.synchronize()
    _same_plan({**{k: v.cpu().numpy() for k, v in got.items()}, "block_table": g["block_table"].cpu().numpy(),
                "free_ring": g["free_ring"].cpu().numpy()}, target.plan_rows(**c))
    ws, graph, room = _ws(), torch.cuda.CUDAGraph(), 17 * B
    new = lambda n, t=torch.int32: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
    out = dict(length=new(B), held=new(B), free_state=new(2), row_offset=new(B + 1), row_request=new(room),
               position=new(room), slot=new(room, torch.int64))
    with torch.cuda.graph(graph):
        dsv.dspark_plan_rows(g["length"], g["rows"], g["held"], g["free_state"], g["free_ring"], g["block_table"], 16,
                             room, advance=g["advance"], out=out, workspace=ws)
    for spoil in (False, True, False):
        again = {k: c[k].copy() for k in names}
        again["rows"] = np.minimum(again["rows"], 3 if spoil else 17)
        if spoil:
            again["length"][B - 1] = -1
        for k in names:
            g[k].copy_(torch.from_numpy(again[k]))
        graph.replay()
        want = target.plan_rows(**again, page=16, max_rows=room)
        assert _code(ws) == ([6, 1] if spoil else [0, 0]) and want["detail"] == int(spoil)
        _same_plan({**{k: v.cpu().numpy() for k, v in out.items()}, "block_table": g["block_table"].cpu().numpy(),
                    "free_ring": g["free_ring"].cpu().numpy()}, want)


@pytest.mark.parametrize("B", [1, 6])
def test_adjust_in_a_graph_and_on_another_stream(dsv, B):  # noqa: F811
    c = _adjust_case(85, B, 4, 20000, "bf16", 200, 5, 3)
    g = {k: v if v is None else v.cuda() for k, v in c.items()}
    want = dsv.dspark_adjust_logits(**g, out=torch.zeros_like(g["logits"]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    s.wait_stream(torch.cuda.current_stream())
    dsv.dspark_adjust_logits(**g, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    ws, graph = _ws(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsv.dspark_adjust_logits(**g, out=out, workspace=ws)
    for seed, bad in ((86, False), (87, True), (88, False)):
        c2 = _adjust_case(seed, B, 4, 20000, "bf16", 200, 5, 3)
        for k, v in c2.items():
            if v is not None:
                g[k].copy_(v)
        if bad:
            g["draft"][0, 0] = 20000
            g["ell"][0] = 3
        out.zero_()
        want = dsv.dspark_adjust_logits(**g, out=torch.zeros_like(out))
        graph.replay()
        assert _code(ws) == ([6, 3] if bad else [0, 0]) and torch.equal(out, want)


def test_one_workspace_for_calls_back_to_back(dsv):  # noqa: F811
    """The four calls queued one behind the other on one workspace, each with and without an error:
    none of them sees what the one before left there."""
    ws = torch.full((dsv.load().dspark_paged_attention_workspace_size(128),), 0xC3, dtype=torch.uint8, device="cuda")
    k, v, slot, stored = _write_case(91, 90)
    a = _attend_case(92, [(300, 17), (20, 2), (3000, 9)], 32, 8, 128, 16, "bf16", "bf16", 0)
    small = dict(_attend_case(93, [(300, 3), (2000, 1)], 8, 2, 128, 16, "bf16", "bf16", 0))
    d = _adjust_case(94, 6, 4, 20000, "f32", 200, 5, 3)
    d = {n: x if x is None else x.cuda() for n, x in d.items()}
    p = _plan_case(95, 1500, 16, 40, 9, 17)
    keys = ("q", "row_offset", "length", "block_table", "k_cache", "v_cache", "max_rows")

    def attend(c, ws):
        return dsv.dspark_paged_attention(**{n: c[n] for n in keys}, workspace=ws)

    alone = [attend(a, None), attend(small, None), dsv.dspark_adjust_logits(**d, out=torch.zeros_like(d["logits"]))]
    plan = target.plan_rows(**p)
    bad_slot = slot.clone()
    bad_slot[7] = 10 ** 9
    g = [{n: _gpu(x) for n, x in p.items() if isinstance(x, np.ndarray)} for _ in range(3)]
    kc, vc = torch.zeros_like(stored[0]), torch.zeros_like(stored[0])
    outs = []
    torch.cuda.synchronize()
    for i in range(3):
        dsv.dspark_write_kv(k, v, bad_slot, kc, vc, workspace=ws)
        pl = dsv.dspark_plan_rows(g[i]["length"], g[i]["rows"], g[i]["held"], g[i]["free_state"], g[i]["free_ring"],
                                  g[i]["block_table"], 16, p["max_rows"], advance=g[i]["advance"], workspace=ws)
        outs.append((pl, attend(a, ws), attend(small, ws), attend(a, ws),
                     dsv.dspark_adjust_logits(**d, out=torch.zeros_like(d["logits"]), workspace=ws)))
        dsv.dspark_write_kv(k, v, bad_slot, kc, vc, workspace=ws)
        dsv.dspark_write_kv(k, v, slot, kc, vc, workspace=ws)
    assert _code(ws)[0] == 0
    assert torch.equal(kc, stored[0]) and torch.equal(vc, stored[1])
    for i, (pl, x, y, z, w) in enumerate(outs):
        _same_plan({**{n: t.cpu().numpy() for n, t in pl.items()}, "block_table": g[i]["block_table"].cpu().numpy(),
                    "free_ring": g[i]["free_ring"].cpu().numpy()}, plan)
        assert torch.equal(x["out"], alone[0]["out"]) and torch.equal(z["out"], alone[0]["out"])
        assert torch.equal(y["out"], alone[1]["out"]) and torch.equal(x["lse"], alone[0]["lse"])
        assert torch.equal(w, alone[2])
