"""Plausible mistakes planted in the oracles of rotary positions and 4-bit caches (on the CPU, one at a time): the pins
have to catch each."""
import numpy as np
import pytest

from oracle import cache4, rotary
import tests.test_oracle_cache4 as T
import tests.test_rotary_frequencies as F


def _fails(fn, *args):
    try:
        fn(*args)
    except (AssertionError, ArithmeticError):
        return True
    return False


@pytest.fixture(scope="module")
def lib():
    return T.lib.__wrapped__()


def _edited(fn, old, new, names):
    """fn with a piece of its source replaced."""
    import inspect
    import textwrap
    src = textwrap.dedent(inspect.getsource(fn))
    assert src.count(old) == 1, (src.count(old), old)
    space = dict(names)
    exec(src.replace(old, new), space)
    return space[fn.__name__]


ROTATE = [
    ("sign of the sine", "magnitude * (x1 * c - x2 * s)", "magnitude * (x1 * c + x2 * s)"),
    ("second half from the wrong partner", "magnitude * (x2 * c + x1 * s)", "magnitude * (x2 * c + x2 * s)"),
    ("backwards ignored", "s = -s if transposed else s", "s = s"),
    ("pairs always apart", "(2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)", "(i, i + rot // 2)"),
    ("half of the head for half of the turned part", "(i, i + rot // 2)", "(i, i + x.shape[2] // 2)"),
    ("magnitude once", "magnitude * (x2 * c + x1 * s)", "(x2 * c + x1 * s)"),
    ("position off by one", "_cos_sin(position[n], f)", "_cos_sin(position[n] + 1, f)"),
    ("negative positions turned", "if position[n] < 0:", "if False:"),
]


@pytest.mark.parametrize("old,new", [r[1:] for r in ROTATE], ids=[r[0] for r in ROTATE])
def test_rotation(monkeypatch, old, new):
    monkeypatch.setattr(rotary, "rotate", _edited(rotary.rotate, old, new, vars(rotary)))
    assert any(_fails(T.test_rotation_is_a_complex_product, i) or _fails(T.test_transposed_rotation_is_the_gradient, i)
               for i in (False, True)) or _fails(T.test_scores_depend_on_distances)


FREQUENCIES = [
    ("exponent not doubled", "f = base ** (-2.0 * i / rot)", "f = base ** (-1.0 * i / rot)"),
    ("linear the wrong way", "return f / factor, 1.0", "return f * factor, 1.0"),
    ("base raised by the factor alone", "factor ** (rot / (rot - 2.0))", "factor"),
    ("bands the wrong way round", "f * keep + f / factor * (1 - keep), 1.0", "f * (1 - keep) + f / factor * keep, 1.0"),
    ("bands without a turn", "turns = original * f / (2 * np.pi)", "turns = original * f"),
    ("ramp the wrong way round", "keep = 1 - np.clip", "keep = np.clip"),
    ("ramp's ends exchanged", "np.floor(d(high))), min(rot - 1.0, np.ceil(d(low)))", "np.floor(d(low))), min(rot - 1.0, np.ceil(d(high)))"),
    ("no magnitude", "0.1 * np.log(factor) + 1.0", "1.0"),
]


@pytest.mark.parametrize("old,new", [r[1:] for r in FREQUENCIES], ids=[r[0] for r in FREQUENCIES])
def test_frequencies(monkeypatch, old, new):
    monkeypatch.setattr(rotary, "frequencies", _edited(rotary.frequencies, old, new, vars(rotary)))
    assert _fails(T.test_frequencies_closed_forms) or _fails(F.test_ramp_halfway)


CODES = [
    ("to_code", "ties down", "tie & (code % 2 == 1)", "tie & False"),
    ("to_code", "ties up", "tie & (code % 2 == 1)", "tie"),
    ("to_code", "no largest", "np.minimum(np.abs(np.asarray(y, np.float64)), 6.0)", "np.abs(np.asarray(y, np.float64)) % 7"),
    ("to_code", "no sign", "code + 8 * np.signbit(y)", "code"),
    ("e4m3_byte", "bias", "(e + 7) * 8", "(e + 8) * 8"),
    ("e4m3_byte", "subnormals", "if s < 2.0 ** -6:", "if False:"),
    ("e4m3_value", "subnormals", "e == 0, m * 2.0 ** -9", "e == 0, m * 2.0 ** -10"),
    ("quantise", "scale of the sum", "np.abs(blocks).max(-1)", "np.abs(blocks).sum(-1)"),
    ("quantise", "scale without the largest code", "one / (np.float32(6) * g)", "one / g"),
    ("quantise", "sign of the largest", "np.abs(blocks).max(-1)", "blocks.max(-1)"),
    ("quantise", "head's scale left out of the codes", "one / (s * g[:, None])", "one / s"),
    ("quantise", "blocks of 32", "blocks = x.reshape(*x.shape[:-1], -1, 16)",
     "blocks = np.where(np.arange(x.shape[-1]) < x.shape[-1] - 16, x, 0 * x).astype(np.float32).reshape(*x.shape[:-1], -1, 16)"),
    ("values", "head's scale left out", "e4m3_value(scale_bytes).astype(np.float32) * g.astype(np.float32)[:, None]",
     "e4m3_value(scale_bytes).astype(np.float32)"),
    ("values", "block scales interleaved", "np.repeat(s.astype(np.float64), 16, -1)", "np.tile(s.astype(np.float64), 16)"),
    ("put", "nibbles exchanged", "codes[0::2] | (codes[1::2] << 4)", "codes[1::2] | (codes[0::2] << 4)"),
    ("put", "scales before the codes' end", "at = page * code + r * scale", "at = page * code + r * (D // 16)"),
    ("get", "nibbles exchanged", "np.stack([c & 15, c >> 4], -1)", "np.stack([c >> 4, c & 15], -1)"),
    ("layout", "scales not rounded up", "-(-(D // 16) // 4) * 4", "D // 16"),
    ("layout", "page not rounded up", "-(-(page * (code + scale)) // 16) * 16", "page * (code + scale)"),
]


@pytest.mark.parametrize("name,old,new", [(r[0],) + r[2:] for r in CODES], ids=[f"{r[0]}: {r[1]}" for r in CODES])
def test_cache(monkeypatch, lib, name, old, new):
    monkeypatch.setattr(cache4, name, _edited(getattr(cache4, name), old, new, vars(cache4)))
    with np.errstate(all="ignore"):
        assert (_fails(T.test_codes_nearest_and_even) or _fails(T.test_scale_bytes) or _fails(T.test_blocks_of_zeros_infinities_and_nan)
                or any(_fails(T.test_quantised_values_are_near, g) for g in (1.0, 0.0021, 300.0))
                or any(_fails(T.test_layout, lib, *s) for s in ((1, 32), (5, 96), (16, 128), (7, 160))))
