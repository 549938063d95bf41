"""Rotary positions on the GPU against the float64 oracle.

Error bound, fixed before the first run, with u = 2^-24.  The angle modulo a turn is exact to 2^-33 of one and
is rounded when it is an eighth of a turn at most: 0.8 u in radians.  Sine and cosine of it: 2 units in the
last place, 2 u below 1; the magnitude's product u; so a coefficient is off by 4 u m, a product of it with
x by 5 u m |x|, the sum's rounding u / 2 |y|:
  |y - exact| <= 5 u m (|x1| + |x2|) + u / 2 |y| + eps / 2 |y|.
"""
import numpy as np
import pytest
import torch

from oracle import rotary
from tests.test_gpu_target import _code, _gpu, _ws, dsv  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = dict(bf16=torch.bfloat16, f32=torch.float32)


def _case(seed, n, heads, D, rot, dtype, far, pad=3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads + pad, D), generator=g).to(TYPES[dtype])
    position = torch.randint(0, far, (n,), generator=g, dtype=torch.int32)
    if n > 2:
        position[n // 2] = -1
        position[n - 1] = far - 1
    freq = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()
    return x, position, freq


def _tolerance(x, want, freq, inter, m, eps):
    half, rot = len(freq), 2 * len(freq)
    a = np.abs(x)
    t = np.zeros_like(a)
    j1, j2 = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(half), np.arange(half, rot))
    t[..., j1] = t[..., j2] = 5 * U * abs(m) * (a[..., j1] + a[..., j2])
    t[..., :rot] += np.abs(want[..., :rot]) * (U / 2 + eps / 2)
    return t


def _check(got, x, position, freq, inter, back, m, dtype):
    x, position, freq = x.double().numpy(), position.numpy(), freq.numpy()
    want = rotary.rotate(x, position, freq, inter, back, m)
    live = position >= 0
    got = got.double().cpu().numpy()[live]
    tol = _tolerance(x[live], want[live], freq, inter, m, torch.finfo(TYPES[dtype]).eps)
    err = np.abs(got - want[live])
    assert np.isfinite(got).all() and (err <= tol).all(), float((err - tol).max())


SIZES = [(1, 1, 16, 16), (3, 2, 64, 64), (40, 12, 128, 64), (7, 5, 96, 96), (301, 3, 128, 128), (5, 40, 256, 256),
         (33, 1, 256, 16), (9, 2, 80, 48), (2, 70, 32, 32), (1500, 1, 64, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter,back,m,far", [(False, False, 1.0, 4096), (True, False, 1.2, 1000000),
                                              (False, True, 0.7, 2 ** 31 - 1), (True, True, 1.0, 300)])
@pytest.mark.parametrize("n,heads,D,rot", SIZES)
def test_rotate(dsv, n, heads, D, rot, inter, back, m, far, dtype):  # noqa: F811
    x, position, freq = _case(n + D, n, heads, D, rot, dtype, far)
    out = torch.full((n, heads + 1, D), 7.0, dtype=TYPES[dtype], device="cuda")
    ws = _ws()
    dsv.dspark_rotate(x.cuda()[:, 1:1 + heads], position.cuda(), freq.cuda(), inter, back, m, out=out[:, 1:], workspace=ws)
    assert _code(ws)[0] == 0
    _check(out[:, 1:], x[:, 1:1 + heads], position, freq, inter, back, m, dtype)
    assert (out[:, 0] == 7).all() and (out[position.cuda() < 0] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_rotate_in_place_and_slices_of_one_buffer(dsv, inter, dtype):  # noqa: F811
    x, position, freq = _case(5, 700, 6, 128, 96, dtype, 9000)
    want = dsv.dspark_rotate(x.cuda()[:, :4], position.cuda(), freq.cuda(), inter,
                             out=torch.zeros((700, 4, 128), dtype=TYPES[dtype], device="cuda"))
    y = x.cuda()
    before = y.clone()
    got = dsv.dspark_rotate(y[:, :4], position.cuda(), freq.cuda(), inter, out=y[:, :4])
    live = position.cuda() >= 0
    assert torch.equal(got[live], want[live]) and torch.equal(y[:, 4:], before[:, 4:])
    assert torch.equal(y[~live], before[~live])
    y = before.clone()
    dsv.dspark_rotate(y[:, :4], position.cuda(), freq.cuda(), inter, out=y[:, 4:8])
    assert torch.equal(y[:, 4:8][live], want[live]) and torch.equal(y[:, :4], before[:, :4])
    with pytest.raises(dsv.DSparkError):
        dsv.dspark_rotate(y[:, :4], position.cuda(), freq.cuda(), inter, out=y[:, 1:5])


def test_rotate_backwards_undoes_it(dsv):  # noqa: F811
    """The gradient of the sum of y dy with respect to x is dy rotated back; by differences in float32 it is the
    inverse that has to hold: 2 (5 u (|x1| + |x2|) + u |y|) <= 22 u of a pair's size."""
    x, position, freq = _case(6, 90, 3, 64, 64, "f32", 100000, pad=0)
    position = position.clamp(min=0)
    y = dsv.dspark_rotate(x.cuda(), position.cuda(), freq.cuda())
    z = dsv.dspark_rotate(y, position.cuda(), freq.cuda(), transposed=True).cpu()
    size = x[..., :32].abs() + x[..., 32:].abs()
    assert ((z - x).abs() <= 22 * U * torch.cat([size, size], -1)).all()
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).cuda()
    dx = dsv.dspark_rotate(dy, position.cuda(), freq.cuda(), transposed=True).double()
    # the map is linear: <R x, dy> = <x, R' dy>, each product off by 11 u of its terms at most
    left, right = (y.double() * dy.double()).sum((1, 2)), (x.cuda().double() * dx).sum((1, 2))
    terms = (x.cuda().abs().double().sum((1, 2)) * dy.abs().double().amax((1, 2))) * 4
    assert ((left - right).abs() <= 22 * U * terms).all()


def test_rotate_odd_frequencies(dsv):  # noqa: F811
    """Zero keeps, negative turns back, tiny ones and subnormal ones do next to nothing; those that are no frequencies
    give NaN, in their pairs alone."""
    x, position, _ = _case(7, 50, 2, 64, 64, "f32", 2 ** 31 - 1, pad=0)
    position = position.clamp(min=0)
    f = torch.zeros(32)
    f[1], f[2], f[3], f[4], f[5], f[6] = -0.3, 1e-30, 2.0 ** -140, 2.0 ** 25, 3.0, 6.0e7
    bad = f.clone()
    bad[7], bad[8], bad[9] = float("nan"), float("inf"), 1e9
    got = dsv.dspark_rotate(x.cuda(), position.cuda(), f.cuda())
    # far positions times large frequencies: the oracle's double angle is exact only to 2^-53 of itself
    g = f.clone()
    g[4] = g[6] = 0.0
    want = dsv.dspark_rotate(x.cuda(), position.cuda(), g.cuda())
    same = [i for i in range(64) if i % 32 not in (4, 6)]
    assert torch.equal(got[..., same], want[..., same])
    small = torch.arange(50, dtype=torch.int32) * 40
    _check(dsv.dspark_rotate(x.cuda(), small.cuda(), f.cuda()), x, small, f, False, False, 1.0, "f32")
    odd = dsv.dspark_rotate(x.cuda(), position.cuda(), bad.cuda())
    nan = [i for i in range(64) if i % 32 in (7, 8, 9)]
    keep = [i for i in range(64) if i not in nan]
    assert torch.isnan(odd[..., nan]).all() and torch.equal(odd[..., keep], got[..., keep])


def test_rotate_no_rows_streams_and_graph(dsv):  # noqa: F811
    x, position, freq = _case(8, 400, 4, 128, 128, "bf16", 5000, pad=0)
    X, P, F = x.cuda(), position.clamp(min=0).cuda(), freq.cuda()
    want = dsv.dspark_rotate(X, P, F)
    assert dsv.dspark_rotate(X[:0], P[:0], F).shape == (0, 4, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsv.dspark_rotate(X, P, F, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out, ws = torch.zeros_like(X), _ws()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsv.dspark_rotate(X, P, F, out=out, workspace=ws)
    X.copy_(X.flip(0))
    P.copy_(P.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want.flip(0))


def test_rotate_offsets_past_32_bits(dsv):  # noqa: F811
    """Rows far apart: the last ones start past element 2^32 of the buffer."""
    stride = 1 << 24
    buf = torch.empty(300 * stride, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((300, 2, 64), (stride, 64, 1))
    src, position, freq = _case(9, 300, 2, 64, 64, "bf16", 5000, pad=0)
    x.copy_(src.cuda())
    want = dsv.dspark_rotate(src.cuda(), position.clamp(min=0).cuda(), freq.cuda())
    got = dsv.dspark_rotate(x, position.clamp(min=0).cuda(), freq.cuda(), out=x)
    assert torch.equal(got, want)
