"""Paged attention where scores are far beyond what a float32 tells apart by one: 2^24 to 2^30 in units of log 2.

Every key's elements are alike and so are every query's, of so few bits that the sums of products are exact; the
keys have eight levels, so a row's weights are those of its highest level alone, equal among its keys and
nothing else: the scores between two levels differ by an eighteenth of the largest, by 2^19 at least.
  out = mean of the highest level's values, lse = the score + ln of their number.

Error bound, fixed before the first run, u = 2^-24.  Equal weights come from equal operations; the factors that join
warps and parts add 2^-20, the sums of n <= 64 equal weights 2 n u < 2^-16, the weights' own rounding 2^-11 (bf16
rows).  A score's float32 scale takes at most 6 roundings, its sum over D elements D (float32 rows):
  |out - exact| <= W (2^-15 + [bf16: 2^-11]) + |exact| eps / 2,  |lse - exact| <= (D + 12) u |exact|.
"""
import numpy as np
import pytest
import torch

from oracle import cache4
from tests import test_gpu_cache4 as four, test_gpu_target as wide
from tests.test_gpu_target import U, dsv  # noqa: F401

pytestmark = pytest.mark.gpu
KINDS = wide.KINDS + [("bf16", "e2m1"), ("f32", "e2m1")]
LEVELS = np.array([1.125, 1.25, 1.375, 1.5, 1.625, 1.75])


def _case(seed, lens, Hq, Hkv, D, page, dtype, cache):
    """A case of the caches' own tests whose keys and queries are replaced by constant rows; the keys' levels are the
    same in all heads."""
    r = np.random.default_rng(seed)
    if cache == "e2m1":
        c, vals = four._attend_case(seed, lens, Hq, Hkv, D, page, dtype, 0)
    else:
        c, vals = wide._attend_case(seed, lens, Hq, Hkv, D, page, dtype, cache, 0), None
    table = c["block_table"].cpu().numpy()
    code, scale, _ = cache4.layout(page, D)
    kc = c["k_cache"].cpu()
    for b, (n, m) in enumerate(lens):
        level = LEVELS[r.integers(0, len(LEVELS), n + m)]
        at = r.permutation(n + m)
        level[at[:4]], level[at[4:7]] = 1.875, 1.0
        for j, x in enumerate(level):
            blk, row = table[b, j // page], j % page
            if cache == "e2m1":
                kc[blk, :, row * code:(row + 1) * code] = 0x22               # ones
                kc[blk, :, page * code + row * scale:page * code + row * scale + D // 16] = cache4.e4m3_byte(x)
                vals[0][blk, :, row] = (np.float32(x) * c["k_scale"].cpu().numpy()).astype(np.float64)[:, None]
            else:
                kc[blk, :, row] = torch.tensor(x).to(kc.dtype)
    c["k_cache"] = kc.cuda()
    sign = torch.tensor(r.choice([1.0, -1.0, 1.5, -1.75], c["q"].shape[:2]))
    c["q"] = sign[..., None].expand(c["q"].shape).to(c["q"].dtype).contiguous().cuda()
    return c, vals


@pytest.mark.parametrize("size", [24.3, 25.2, 25.9, 26.6, 27.5, 28.2, 29.4])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ([(0, 7), (30, 1)], 4, 2, 64, 16), ([(300, 1), (9000, 1)], 8, 2, 128, 16), ([(150, 8), (700, 3)], 8, 2, 96, 24),
    ([(130, 17), (2500, 17)], 16, 4, 128, 16), ([(90, 4), (1000, 2)], 4, 1, 256, 8)])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_far_scores(dsv, dtype, cache, lens, Hq, Hkv, D, page, size):  # noqa: F811
    c, vals = _case(int(size), lens, Hq, Hkv, D, page, dtype, cache)
    largest = 1.75 * 1.875 * D * (1.0 if c["k_scale"] is None else float(c["k_scale"].max()))
    scale = 2.0 ** size / (largest * np.log2(np.e))
    if cache == "e2m1":
        out, code = four._run_attend(dsv, c, scale=scale)
        ref = four._oracle(c, vals, scale)
    else:
        out, code = wide._run_attend(dsv, c, scale=scale)
        ref = wide._oracle(c, scale)
    assert code[0] == 0
    bf16 = dtype == "bf16"
    tol = ref["weight"] * (2.0 ** -15 + (2.0 ** -11 if bf16 else 0.0)) + np.abs(ref["out"]) * torch.finfo(c["q"].dtype).eps / 2
    err = np.abs(out["out"].double().cpu().numpy() - ref["out"])
    assert np.isfinite(err).all(), int((~np.isfinite(err)).sum())
    assert (err <= tol + 1e-30).all(), float((err / (tol + 1e-30)).max())
    lerr = np.abs(out["lse"].double().cpu().numpy() - ref["lse"])
    assert (lerr <= (D + 12) * U * np.abs(ref["lse"])).all(), float((lerr / np.abs(ref["lse"]) / U).max())
