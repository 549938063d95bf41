"""The oracle of the target model's side against closed forms, other formulations and
planted mistakes."""
import numpy as np
import pytest
import torch

from oracle import target


def _plan_case(seed, B=9, page=4, width=12, extra=40):
    r = np.random.default_rng(seed)
    length = r.integers(0, 20, B).astype(np.int32)
    last = r.integers(0, 6, B)
    advance = np.array([r.integers(0, n + 1) for n in last], np.int32)
    held = (-(-(length + last) // page)).astype(np.int32)
    rows = r.integers(0, 9, B).astype(np.int32)
    finished = r.random(B) < 0.2
    length[finished], advance[finished], rows[finished] = 0, 0, 0
    total = int(held.sum())
    ids = r.permutation(total + extra).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    cap = total + extra
    ring = np.full(cap, -7, np.int32)
    head = int(r.integers(0, cap))
    for i in range(extra):
        ring[(head + i) % cap] = ids[total + i]
    return dict(length=length, advance=advance, rows=rows, held=held,
                free_state=np.array([head, extra], np.int32), free_ring=ring, block_table=table, page=page,
                max_rows=int(rows.sum()) + 3)


@pytest.mark.parametrize("seed", range(6))
def test_plan_keeps_every_page_exactly_once(seed):
    c = _plan_case(seed)
    o = target.plan_rows(**c)
    assert o["detail"] == 0
    cap = len(c["free_ring"])
    held = [o["block_table"][b, :o["held"][b]] for b in range(len(c["rows"]))]
    head, count = o["free_state"]
    free = [o["free_ring"][(head + i) % cap] for i in range(count)]
    assert sorted(np.concatenate(held + [free])) == list(range(cap))
    n = int(c["rows"].sum())
    assert len(set(o["slot"][:n])) == n and (o["slot"][n:] == -1).all()
    # positions of a request are consecutive and lie in its own pages
    for i in range(n):
        b, pos = o["row_request"][i], o["position"][i]
        assert pos == o["length"][b] + i - o["row_offset"][b]
        assert o["block_table"][b, pos // c["page"]] == o["slot"][i] // c["page"]


def test_plan_refuses_whole_steps():
    c = _plan_case(1)
    for change, detail in ((dict(free_state=np.array([c["free_state"][0], 0], np.int32)), 3),
                           (dict(max_rows=int(c["rows"].sum()) - 1), 4),
                           (dict(rows=np.where(np.arange(9) == 2, 500, c["rows"]).astype(np.int32)), 2),
                           (dict(held=np.where(np.arange(9) == 2, -1, c["held"]).astype(np.int32)), 1)):
        o = target.plan_rows(**{**c, **change})
        assert o["detail"] == detail
        assert (o["block_table"] == c["block_table"]).all() and (o["slot"] == -1).all()


def test_e4m3_rounding_matches_torch_on_every_midpoint():
    g = target.e4m3_values()
    assert len(g) == 127 and g[-1] == 448 and g[1] == 2.0 ** -9
    mid = (g[1:] + g[:-1]) / 2
    x = np.concatenate([g, mid, np.nextafter(mid, 0), np.nextafter(mid, 500), [0.0, 1e-9, 460, 1e9]]).astype(np.float32)
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert (target.to_e4m3(x) == want).all()
    assert np.isnan(target.to_e4m3([np.nan])).all()


def _attend_case(seed, window=0, Hq=6, Hkv=2, D=8, page=3):
    r = np.random.default_rng(seed)
    length, rows = np.array([5, 0, 11, 2]), np.array([3, 1, 0, 4])
    offset = np.concatenate([[0], np.cumsum(rows)])
    pages = -(-(length + rows) // page)
    ids = r.permutation(pages.sum() + 4)
    table = np.zeros((4, pages.max()), np.int64)
    at = 0
    for b in range(4):
        table[b, :pages[b]] = ids[at:at + pages[b]]
        at += pages[b]
    shape = (len(ids), Hkv, page, D)
    return dict(q=r.normal(size=(offset[-1], Hq, D)), row_offset=offset, length=length, block_table=table,
                k_cache=r.normal(size=shape), v_cache=r.normal(size=shape), scale=0.7, window=window)


@pytest.mark.parametrize("window", [0, 1, 4])
def test_attention_against_a_dense_masked_softmax(window):
    c = _attend_case(3, window)
    o = target.paged_attention(**c)
    page = c["k_cache"].shape[2]
    for b in range(4):
        lo, hi = c["row_offset"][b], c["row_offset"][b + 1]
        if hi == lo:
            continue
        L = c["length"][b] + hi - lo
        flat = [x[c["block_table"][b]].transpose(0, 2, 1, 3).reshape(-1, 2, 8)[:L] for x in (c["k_cache"], c["v_cache"])]
        K, V = (torch.from_numpy(np.repeat(x, 3, axis=1)) for x in flat)
        s = torch.einsum("rhd,khd->rhk", torch.from_numpy(c["q"][lo:hi]), K) * 0.7
        pos, key = torch.arange(c["length"][b], L)[:, None, None], torch.arange(L)
        hide = key > pos
        if window:
            hide = hide | (key <= pos - window)
        s = s.masked_fill(hide, float("-inf"))
        np.testing.assert_allclose(o["out"][lo:hi], torch.einsum("rhk,khd->rhd", s.softmax(-1), V), atol=1e-12)
        np.testing.assert_allclose(o["lse"][lo:hi], torch.logsumexp(s, -1), atol=1e-12)
    assert page == 3


def test_attention_of_parts_joins_to_the_whole():
    c = _attend_case(5)
    whole = target.paged_attention(**c)
    i = int(c["row_offset"][1]) - 1                      # last row of request 0: eight keys
    at = np.arange(8)
    ids = c["block_table"][0, at // 3]
    K, V = c["k_cache"][ids, 0, at % 3], c["v_cache"][ids, 0, at % 3]
    parts = []
    for part in (slice(0, 3), slice(3, 8)):
        s = 0.7 * K[part] @ c["q"][i, 0]
        parts.append((s.max(), np.exp(s - s.max()).sum(), np.exp(s - s.max()) @ V[part]))
    m = max(p[0] for p in parts)
    z = sum(p[1] * np.exp(p[0] - m) for p in parts)
    np.testing.assert_allclose(whole["out"][i, 0], sum(p[2] * np.exp(p[0] - m) for p in parts) / z, atol=1e-12)


def test_masked_keys_have_no_part():
    c = _attend_case(7)
    want = target.paged_attention(**c)["out"]
    pos, page = 5, c["k_cache"].shape[2]                 # request 0's first new key: hidden from nobody but earlier rows
    k, v = c["k_cache"].copy(), c["v_cache"].copy()
    last = 7
    k[c["block_table"][0, last // page], :, last % page] = np.nan
    v[c["block_table"][0, last // page], :, last % page] = np.inf
    got = target.paged_attention(**{**c, "k_cache": k, "v_cache": v})["out"]
    assert (got[:2] == want[:2]).all() and not np.isfinite(got[2]).all()
    assert pos == c["length"][0]


def test_adjust_closed_forms():
    V = 64
    x = np.zeros((1, 3, V))
    x[0, :, 1], x[0, :, 2], x[0, :, 3] = 2.0, -2.0, 1.0
    kw = dict(history=np.array([[1, 2, 2, 3, 3, 9]]), prompt_len=np.array([3]), history_len=np.array([5]),
              draft=np.array([[1, 1]]), repetition=np.array([2.0]), frequency=np.array([0.25]),
              presence=np.array([0.5]))
    y = target.adjust_logits(x, np.zeros_like(x), **kw)
    assert y[0, 0, 1] == 1.0 and y[0, 0, 2] == -4.0            # prompt tokens: repetition only
    assert y[0, 0, 3] == 0.5 - 2 * 0.25 - 0.5                  # twice in the output
    assert y[0, 1, 1] == 1.0 - 0.25 - 0.5 and y[0, 2, 1] == 1.0 - 2 * 0.25 - 0.5
    assert (y[0, :, 9] == 0).all()                             # past history_len
    kw.update(bias_token=np.array([[5, -1, 5]]), bias_value=np.array([[1.0, 9.0, 2.0]]),
              mask_row=np.array([[-1, 0, 1]]), mask=np.array([[0, 0], [-1, 1]]), ell=np.array([1]))
    y = target.adjust_logits(x, np.full_like(x, 7.0), **kw)
    assert y[0, 0, 5] == 3.0 and np.isneginf(y[0, 1]).all() and (y[0, 2] == 7.0).all()
    kw.update(ell=np.array([2]))
    y = target.adjust_logits(x, x, **kw)
    assert np.isfinite(y[0, 2, :33]).all() and np.isneginf(y[0, 2, 33:]).all()


def test_planted_mistakes_are_seen():
    """A window off by one, a forgotten scale and counts that include the prompt change the result."""
    c = _attend_case(2, window=4)
    want = target.paged_attention(**c)["out"]
    assert np.abs(target.paged_attention(**{**c, "window": 5})["out"] - want).max() > 1e-3
    ones = np.full(2, 1.25)
    assert np.abs(target.paged_attention(**c, k_scale=ones, v_scale=np.ones(2))["out"] - want).max() > 1e-3
    x = np.ones((1, 1, 8))
    kw = dict(history=np.array([[1, 2]]), history_len=np.array([2]), frequency=np.array([0.5]))
    a = target.adjust_logits(x, x, prompt_len=np.array([1]), **kw)
    b = target.adjust_logits(x, x, prompt_len=np.array([0]), **kw)
    assert (a != b).any()
