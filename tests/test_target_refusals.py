"""The calls of the target model's side refuse bad arguments on the host, before any launch:
through the C ABI with addresses that nothing may touch, and through the binding."""
import ctypes
import os

import pytest
import torch

P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
FAKE, WS, BIG = 0x1000, 0x10000, 1 << 40


@pytest.fixture(scope="module")
def lib():
    from serving_draft_verify_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    from serving_draft_verify_gb300 import _binding
    return _binding.load()


def _call(fn, defaults, **changes):
    assert set(changes) <= set(defaults), changes
    return fn(*{**defaults, **changes}.values())


def test_plan_rows(lib):
    d = dict(B=4, page=16, max_blocks=8, num_blocks=64, max_rows=32, len=FAKE, advance=None, rows=FAKE, held=FAKE,
             free_state=FAKE, free_ring=FAKE, block_table=FAKE, ld=8, len_out=FAKE, held_out=FAKE, free_out=FAKE,
             row_offset=FAKE, row_request=FAKE, position=FAKE, slot=FAKE, ws=WS, ws_bytes=BIG, stream=None)
    f = lib.dspark_plan_rows
    for bad in (dict(B=0), dict(B=65536), dict(page=0), dict(max_blocks=0), dict(num_blocks=0), dict(max_rows=-1),
                dict(max_rows=1 << 31), dict(ld=7), dict(len=None), dict(rows=None), dict(held=None),
                dict(free_state=None), dict(free_ring=None), dict(block_table=None), dict(len_out=None),
                dict(held_out=None), dict(free_out=None), dict(row_offset=None), dict(row_request=None),
                dict(position=None), dict(slot=None), dict(ws=None), dict(ws=WS + 16)):
        assert _call(f, d, **bad) == 1, bad
    assert _call(f, d, max_blocks=1 << 27, ld=1 << 27) == 2          # positions past 32 bits
    assert _call(f, d, B=65535, max_blocks=40000, ld=40000) == 2     # page sums past 32 bits
    assert _call(f, d, ws_bytes=256) == 3


def test_write_kv(lib):
    d = dict(rows=4, Hkv=8, D=128, page=16, num_blocks=64, dt=1, cache_dt=1, k=FAKE, k_stride=1024, v=FAKE,
             v_stride=1024, slot=FAKE, ks=None, vs=None, kc=FAKE, vc=FAKE, ws=WS, ws_bytes=BIG, stream=None)
    f = lib.dspark_write_kv
    for bad in (dict(rows=-1), dict(Hkv=0), dict(Hkv=1025), dict(D=0), dict(D=12), dict(D=264), dict(page=0),
                dict(num_blocks=0), dict(dt=2), dict(dt=7), dict(cache_dt=0), dict(cache_dt=7), dict(cache_dt=2),
                dict(cache_dt=2, ks=FAKE), dict(cache_dt=2, ks=FAKE, vs=FAKE, D=24), dict(k_stride=1000),
                dict(k_stride=1028), dict(v_stride=8), dict(v_stride=1025), dict(k=None), dict(v=None),
                dict(slot=None), dict(kc=None), dict(vc=None), dict(kc=FAKE + 8), dict(k=FAKE + 2), dict(ws=None),
                dict(ws=WS + 128)):
        assert _call(f, d, **bad) == 1, bad
    assert _call(f, d, ws_bytes=16) == 3


def test_paged_attention(lib):
    d = dict(B=2, rows=4, max_rows=4, Hq=32, Hkv=8, D=128, page=16, max_blocks=8, num_blocks=64, dt=1, cache_dt=1,
             q=FAKE, q_stride=4096, off=FAKE, len=FAKE, table=FAKE, ld=8, kc=FAKE, vc=FAKE, ks=None, vs=None,
             scale=0.1, window=0, out=FAKE, lse=None, ws=WS, ws_bytes=BIG, stream=None)
    f = lib.dspark_paged_attention
    nan, inf = float("nan"), float("inf")
    for bad in (dict(B=0), dict(B=65536), dict(rows=-1), dict(max_rows=0), dict(Hq=0), dict(Hkv=0), dict(Hq=33),
                dict(Hq=1032, Hkv=1032), dict(D=0), dict(D=20), dict(D=264), dict(page=0), dict(max_blocks=0),
                dict(num_blocks=0), dict(dt=2), dict(dt=7), dict(cache_dt=0), dict(cache_dt=2),
                dict(cache_dt=2, ks=FAKE, vs=FAKE, D=24), dict(q=None), dict(q=FAKE + 2), dict(q_stride=4095),
                dict(q_stride=4100), dict(off=None), dict(len=None), dict(table=None), dict(ld=7), dict(kc=None),
                dict(vc=None), dict(vc=FAKE + 4), dict(scale=nan), dict(scale=inf), dict(window=-1), dict(out=None),
                dict(ws=None), dict(ws=WS + 16)):
        assert _call(f, d, **bad) == 1, bad
    assert _call(f, d, max_blocks=1 << 27, ld=1 << 27) == 2
    assert _call(f, d, max_rows=1 << 30) == 2
    assert _call(f, d, ws_bytes=4096) == 3


def test_adjust_logits(lib):
    d = dict(B=2, R=8, V=64, dt=1, logits=0x100000, ell=None, history=FAKE, ld=16, prompt_len=None, history_len=FAKE,
             draft=None, rep=None, freq=None, pres=None, bias_token=None, bias_value=None, n_bias=0, mask_row=None,
             mask=None, n_mask=0, ld_mask=2, out=0x200000, ws=WS, ws_bytes=BIG, stream=None)
    f = lib.dspark_adjust_logits
    for bad in (dict(B=0), dict(B=65536), dict(R=0), dict(R=34), dict(V=0), dict(V=60), dict(dt=2), dict(dt=0, V=62),
                dict(logits=None), dict(out=None), dict(logits=0x100008), dict(out=0x200004), dict(history=None),
                dict(history_len=None), dict(history=None, history_len=None, prompt_len=FAKE), dict(ld=-1),
                dict(n_bias=-1), dict(n_bias=3), dict(n_bias=3, bias_token=FAKE), dict(mask_row=FAKE, n_mask=-1),
                dict(mask_row=FAKE, n_mask=1), dict(mask_row=FAKE, n_mask=1, mask=FAKE, ld_mask=1),
                dict(out=0x100000 + 1024), dict(out=0x100000 - 16), dict(ws=None), dict(ws=WS + 8)):
        assert _call(f, d, **bad) == 1, bad
    assert _call(f, d, n_bias=2048, bias_token=FAKE, bias_value=FAKE) == 2
    assert _call(f, d, ld=1048544) == 2
    assert _call(f, d, ws_bytes=16) == 3


def test_binding_refuses_host_tensors(lib):
    import serving_draft_verify_gb300 as dsv
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises((ValueError, TypeError)):
        dsv.dspark_plan_rows(i, i, i, i, i, torch.zeros((2, 4), dtype=torch.int32), 16, 8)
    c = torch.zeros((4, 2, 16, 64))
    x = torch.zeros((3, 2, 64))
    with pytest.raises((ValueError, TypeError)):
        dsv.dspark_write_kv(x, x, torch.zeros(3, dtype=torch.int64), c, c)
    with pytest.raises((ValueError, TypeError)):
        dsv.dspark_paged_attention(x, torch.zeros(3, dtype=torch.int32), i, torch.zeros((2, 4), dtype=torch.int32), c, c, 2)
    with pytest.raises((ValueError, TypeError)):
        dsv.dspark_adjust_logits(torch.zeros((1, 2, 64)))
