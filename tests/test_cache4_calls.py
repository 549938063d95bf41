"""Rotary positions and 4-bit caches as programs may use them: another device, side streams,
two captured graphs with one workspace, the most heads."""
import os

import numpy as np
import pytest
import torch

from oracle import cache4, rotary
from tests.test_gpu_cache4 import _attend_case, _check, _expect, _oracle, _rows, _run_attend, _scales
from tests.test_gpu_rotate import _case, _tolerance
from tests.test_gpu_target import _code, _ws


@pytest.fixture(scope="module")
def dsv():
    from serving_draft_verify_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    import serving_draft_verify_gb300 as m
    m.load()
    return m


class _Elsewhere:
    """A stand-in for a tensor on the second GPU; anything but its device is out of bounds."""

    shape = (4, 2, 64)
    device = torch.device("cuda", 1)
    dtype = torch.float32

    def get_device(self):
        return 1


def test_tensors_of_another_device_are_refused(dsv, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(dsv._binding, "_several", None)
    x = _Elsewhere()
    for call in (lambda: dsv.dspark_rotate(x, x, x), lambda: dsv.dspark_rotate_write_kv(x, x, x, x, x, x, x, x, x, x),
                 lambda: dsv.dspark_read_kv(x, x, x, x, x, D=64)):
        with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
            call()


@pytest.mark.gpu
def test_made_outputs_on_a_side_stream(dsv):
    """Outputs and workspaces that the calls make themselves, on a stream that is not the current one."""
    n, Hq, Hkv, D, page = 90, 4, 2, 128, 16
    x, position, freq = (t.cuda() for t in _case(3, n, Hq + 2 * Hkv, D, D, "bf16", 5000, 0))
    position = position.abs()
    slot = torch.randperm(8 * page, generator=torch.Generator().manual_seed(1))[:n].cuda()
    g = torch.full((Hkv,), 0.002, device="cuda")
    kc, vc, kd, vd = (dsv.kv4_cache(8, Hkv, page, D) for _ in range(4))
    args = (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], position, freq, slot)
    want = dsv.dspark_rotate_write_kv(*args, kc, vc, g, g)
    back = dsv.dspark_read_kv(slot, kc, vc, g, g, D=D, dtype=torch.float32)
    turned = dsv.dspark_rotate(x, position, freq, transposed=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q = dsv.dspark_rotate_write_kv(*args, kd, vd, g, g, stream=side)
    b = dsv.dspark_read_kv(slot, kd, vd, g, g, D=D, dtype=torch.float32, stream=side)
    r = dsv.dspark_rotate(x, position, freq, transposed=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(q, want) and torch.equal(kc, kd) and torch.equal(vc, vd) and torch.equal(r, turned)
    assert torch.equal(b["k"], back["k"]) and torch.equal(b["v"], back["v"]) and b["k"].count_nonzero() > 0


@pytest.mark.gpu
def test_two_graphs_share_a_workspace(dsv):
    """Captured with one workspace and replayed in turn, one of them with a bad slot and a bad page: each replay
    answers for itself, and a clean one leaves no status behind."""
    Hq, Hkv, D, page, blocks = 8, 2, 64, 16, 6
    freq, _ = dsv.dspark_rotary_frequencies(D)
    g = torch.full((Hkv,), 0.002, device="cuda")
    ws = _ws(dsv.load().dspark_paged_attention_workspace_size(D))
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").view(1, blocks)

    def record(seed, n, length, bad):
        """(graphs of storing and of attending, what they write, what that has to be, what they read)."""
        x = _rows(seed, n, Hq + 2 * Hkv, D, "bf16", 0.0).cuda()
        kc, vc = dsv.kv4_cache(blocks, Hkv, page, D), dsv.kv4_cache(blocks, Hkv, page, D)
        slot = torch.arange(length, length + n, device="cuda")
        if bad:
            slot[1] = blocks * page
        at = torch.arange(length, length + n, dtype=torch.int32, device="cuda")
        off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        ln = torch.tensor([length], dtype=torch.int32, device="cuda")
        q, out, lse = torch.zeros_like(x[:, :Hq].contiguous()), torch.zeros((n, Hq, D), dtype=torch.bfloat16, device="cuda"), \
            torch.zeros((n, Hq), device="cuda")
        store = lambda: dsv.dspark_rotate_write_kv(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], at, freq, slot, kc, vc,  # noqa: E731
                                                   g, g, out=q, workspace=ws)
        attend = lambda: dsv.dspark_paged_attention(q, off, ln, table, kc, vc, n, k_scale=g, v_scale=g,  # noqa: E731
                                                    out=dict(out=out, lse=lse), workspace=ws)
        store(), attend()
        torch.cuda.synchronize()
        want = [t.clone() for t in (q, out, lse, kc)]
        graphs = []
        for call in (store, attend):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                call()
        return graphs, (q, out, lse, kc), want, (x, vc, slot, at, off, ln)

    a, b = record(1, 7, 30, False), record(2, 80, 0, True)
    for one in (a, b, b, a, b, a):
        for t in one[1]:
            t.zero_()
        one[0][0].replay()
        assert _code(ws) == ([6, 1] if one is b else [0, 0])
        one[0][1].replay()
        assert _code(ws)[0] == 0
        for t, w in zip(one[1], one[2]):
            assert torch.equal(t, w)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_most_heads(dsv, dtype):
    """4096 heads rotated, 1024 heads stored and read, at a width of 256 and 32."""
    x, position, freq = _case(11, 3, 4096, 256, 256, dtype, 100000, 0)
    got = dsv.dspark_rotate(x.cuda(), position.cuda(), freq.cuda()).double().cpu().numpy()
    live = position.numpy() >= 0
    xs = x.double().numpy()
    want = rotary.rotate(xs, position.numpy(), freq.numpy(), False, False, 1.0)
    tol = _tolerance(xs, want, freq.numpy(), False, 1.0, torch.finfo(x.dtype).eps)
    assert (np.abs(got - want) <= tol)[live].all()
    for D, n in ((256, 2), (32, 5)):
        Hkv, page, blocks = 1024, 3, 4
        kc, vc = dsv.kv4_cache(blocks, Hkv, page, D), dsv.kv4_cache(blocks, Hkv, page, D)
        g = _scales(5, Hkv)
        k = _rows(D, n, Hkv, D, dtype)
        slot = torch.tensor([11, 0, 4, 7, 2][:n])
        dsv.dspark_write_kv(k.cuda(), k.cuda(), slot.cuda(), kc, vc, g.cuda(), g.cuda())
        zero = np.zeros(kc.shape, np.uint8)
        np.testing.assert_array_equal(kc.cpu().numpy(), _expect(zero, page, slot, k, g))
        assert torch.equal(kc, vc)
        back = dsv.dspark_read_kv(slot.cuda(), kc, vc, g.cuda(), g.cuda(), D=D, dtype=torch.float32)
        c, s = cache4.quantise(k.float().numpy(), g.numpy())
        np.testing.assert_array_equal(back["k"].cpu().numpy(), cache4.values(c, s, g.numpy()).astype(np.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [([(20, 2), (0, 1)], 1024, 1, 64, 16), ([(9, 2)], 1024, 1024, 32, 4),
                                                ([(33, 1)], 1024, 128, 96, 16)])
def test_most_heads_of_attention(dsv, lens, Hq, Hkv, D, page, dtype):
    c, vals = _attend_case(Hkv, lens, Hq, Hkv, D, page, dtype, 0)
    out, code = _run_attend(dsv, c)
    assert code[0] == 0
    _check(out, _oracle(c, vals), vals, dtype, D)


@pytest.mark.gpu
def test_many_requests_of_one_key(dsv):
    """The shortest calls in great number: 5000 requests of one row, some without any."""
    r = np.random.default_rng(0)
    lens = [(int(r.integers(0, 3)), int(r.integers(0, 2))) for _ in range(5000)]
    for dtype in ("bf16", "f32"):
        c, vals = _attend_case(7, lens, 2, 1, 32, 1, dtype, 0)
        out, code = _run_attend(dsv, c)
        assert code[0] == 0
        _check(out, _oracle(c, vals), vals, dtype, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,heads,D,rot", [(700, 16, 128, 128), (1300, 17, 128, 64), (1301, 1, 16, 16), (1250, 7, 96, 64),
                                           (1219, 21, 96, 96), (1300, 8, 256, 256), (640, 9, 256, 128), (5, 32, 64, 64)])
def test_heads_about_a_blocks_groups(dsv, n, heads, D, rot, inter, dtype):
    """As many heads as a block has groups of threads, one more, and few; several rows a block, the last block not full."""
    x, position, freq = _case(n, n, heads, D, rot, dtype, 70000, 0)
    out = torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
    dsv.dspark_rotate(x.cuda(), position.cuda(), freq.cuda(), inter, True, out=out)
    xs, live = x.double().numpy(), position.numpy() >= 0
    want = rotary.rotate(xs, position.numpy(), freq.numpy(), inter, True, 1.0)
    tol = _tolerance(xs, want, freq.numpy(), inter, 1.0, torch.finfo(x.dtype).eps)
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= tol)[live].all() and (got[~live] == 7).all()
    y = x.cuda()
    dsv.dspark_rotate(y, position.cuda(), freq.cuda(), inter, True, out=y)
    assert torch.equal(y[position.cuda() >= 0], out[position.cuda() >= 0])
    assert torch.equal(y[position.cuda() < 0], x.cuda()[position.cuda() < 0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("most,Hq,Hkv,D", [(1, 2, 2, 32), (5, 8, 2, 64), (9, 4, 1, 128)])
def test_ragged_requests_in_number(dsv, most, Hq, Hkv, D, dtype):
    """More segments than blocks, of no keys to some units, whole ones and split ones in one block."""
    r = np.random.default_rng(most)
    lens = [(int(r.integers(0, 700)) if r.random() < 0.7 else int(r.integers(0, 3)), int(r.integers(0, most + 1)))
            for _ in range(400)]
    c, vals = _attend_case(most, lens, Hq, Hkv, D, 16, dtype, 0)
    out, code = _run_attend(dsv, c)
    assert code[0] == 0
    _check(out, _oracle(c, vals), vals, dtype, D)
