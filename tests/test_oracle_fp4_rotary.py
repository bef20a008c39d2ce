"""Pins of the 4-bit codec, its pages, and the rotation's oracle; the
fixed-point angle arithmetic of the rotation kernel in Python integers."""
import itertools
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import e2m1, e4m3, rotary

# pi to 50 digits
PI = Fraction("3.14159265358979323846264338327950288419716939937510")


def test_codec_by_brute_force():
    sizes = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert e2m1.VALUES.tolist() == sizes + [-x for x in sizes]
    rng = np.random.default_rng(0)
    ties = [(a + b) / 2 for a, b in zip(sizes, sizes[1:])]
    xs = np.concatenate([rng.uniform(-8, 8, 4000), ties, np.nextafter(np.float32(ties), 9), np.nextafter(np.float32(ties), 0),
                         sizes, [7.0, 1e9, -1e9]]).astype(np.float32)
    for x in np.concatenate([xs, -xs]):
        c = int(e2m1.encode(x))
        d = [abs(abs(float(x)) - s) for s in sizes]
        near = [i for i in range(8) if d[i] == min(d)]
        assert (c & 7) == (near[0] if len(near) == 1 else next(i for i in near if i % 2 == 0)), x
        assert bool(c & 8) == bool(np.signbit(x))


def test_quantize_by_hand():
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [12.0, -6.0, 1.0, 0.4]
    codes, sb = e2m1.quantize(x, np.float32(0.5))
    # the block's largest value, 12, at 6 * 4.0 * 0.5; a block of zeros has scale and codes 0
    assert e4m3.decode(sb).tolist() == [[4.0, 0.0]]
    assert e2m1.decode(codes)[0, :4].tolist() == [6.0, -3.0, 0.5, 0.0]  # 12, 6, 1 and 0.4 over 2
    assert not codes[0, 4:].any()
    back = e2m1.dequantize(codes, sb) * 0.5
    assert back[0, :4].tolist() == [12.0, -6.0, 1.0, 0.0]


def test_value_times_block_scale_is_exact_in_float16():
    scales = e4m3.DECODE_TABLE[:0x7F]
    prod = np.outer(e2m1.VALUES, scales)
    assert np.array_equal(prod.astype(np.float16).astype(np.float64), prod)


@pytest.mark.parametrize("D", [64, 128])
def test_pages_place_every_byte_once(D):
    places = [e2m1.v_byte(t, j) for t in range(16) for j in range(D // 2)]
    assert sorted(places) == list(range(16 * D // 2))
    scales = [e2m1.v_scale_byte(t, i) for t in range(16) for i in range(D // 16)]
    assert sorted(scales) == list(range(D))
    rng = np.random.default_rng(1)
    k, v = (rng.integers(0, 16, (2, 3, 16, D), dtype=np.uint8) for _ in range(2))
    ks, vs = (rng.integers(0, 256, (2, 3, 16, D // 16), dtype=np.uint8) for _ in range(2))
    back = e2m1.from_pages(*e2m1.pages(k, ks, v, vs), D)
    assert all(np.array_equal(a, b) for a, b in zip(back, (k, ks, v, vs)))


def test_attend_by_brute_force():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((2, 8)), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    out, mag = e2m1.attend(q, k, v, 0.3)
    for i in range(2):
        w = [math.exp(0.3 * sum(a * b for a, b in zip(q[i], k[j]))) for j in range(5)]
        for d in range(8):
            assert out[i, d] == pytest.approx(sum(w[j] * v[j, d] for j in range(5)) / sum(w), abs=1e-12)
            assert mag[i, d] == pytest.approx(sum(w[j] * abs(v[j, d]) for j in range(5)) / sum(w), abs=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_closed_forms(interleaved):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 16))
    inv = np.float32([1.0, 0.5, 0.25, 0.01])
    zero = rotary.turn(x, np.zeros(4, int), inv, interleaved=interleaved)
    assert np.array_equal(zero, x)
    pos = np.array([0, 3, 100, -7])
    y = rotary.turn(x, pos, inv, interleaved=interleaved)
    assert np.array_equal(y[..., 8:], x[..., 8:])  # dims behind the pairs
    for i, t in itertools.product(range(4), range(4)):  # as complex numbers
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 4)
        z = (x[t, 1, a] + 1j * x[t, 1, b]) * complex(math.cos(pos[t] * float(inv[i])), math.sin(pos[t] * float(inv[i])))
        assert y[t, 1, a] == pytest.approx(z.real, abs=1e-12) and y[t, 1, b] == pytest.approx(z.imag, abs=1e-12)
    # a product of a query and a key depends on their distance alone
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    dots = [float((rotary.turn(q, [m + 5], inv, interleaved=interleaved) * rotary.turn(k, [m], inv, interleaved=interleaved)).sum())
            for m in (0, 1, 1000)]
    assert dots == pytest.approx([dots[0]] * 3, abs=1e-9)


def test_rotation_axes_and_norm():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 1, 8))
    inv = np.float32([1.0, 0.7, 0.3, 0.1])
    pos = np.array([[1, 2, 3], [10, 20, 30]])
    y = rotary.turn(x, pos, inv, pair_axis=[0, 1, 1, 0])
    for i, a in enumerate([0, 1, 1, 0]):
        one = rotary.turn(x, pos[a], inv)
        assert np.array_equal(y[..., [i, i + 4]], one[..., [i, i + 4]])
    w = rng.standard_normal(8)
    y = rotary.turn(x, None, None, weight=w, eps=0.5)
    for t in range(3):
        r = math.sqrt(sum(v * v for v in x[t, 0]) / 8 + 0.5)
        assert y[t, 0] == pytest.approx(x[t, 0] / r * w, abs=1e-12)


# ---- the kernel's angle: inv_freq / 2 pi in units of 2^-64 turns, times the position, mod 2^64
INV_TWO_PI = 0xA2F9836E4E441529


def _turns(inv_freq: np.float32, pos: int) -> int:
    u = int(np.float32(inv_freq).view(np.uint32))
    e = (u >> 23) & 0xFF
    m = (u & 0x7FFFFF) | (0x800000 if e else 0)
    f = ((m << 40) * INV_TWO_PI) >> 64
    shift = (e or 1) - 128
    x = 0 if shift <= -64 else f >> -shift if shift < 0 else (f << shift) % 2**64 if shift < 64 else 0
    x = -x if u >> 31 else x
    return (x * pos) % 2**64


def test_the_constant():
    assert INV_TWO_PI == int(2**66 / (2 * PI))


@pytest.mark.parametrize("inv_freq", [1.0, 0.86596, 1e-2, 500000.0 ** -0.984375, 1e-7, 3.7, 100.5, -0.3, 6.2831855, 0.0, 1e-40])
@pytest.mark.parametrize("pos", [0, 1, 17, 131071, 10**6 + 1, 2**31 - 1, -1, -(2**31)])
def test_fixed_point_angles(inv_freq, pos):
    inv = np.float32(inv_freq)
    exact = Fraction(float(inv)) * pos / (2 * PI)
    exact -= math.floor(exact)
    top = Fraction(_turns(inv, pos) >> 32, 2**32)  # what the kernel takes the sine of
    off = abs(top - exact)
    # the fraction's last place, 2^-64 (2^(e - 64) from inv_freq = 2^e, e >= 1, on), times the position; 2^-32 for the top half
    assert min(off, 1 - off) <= Fraction(1, 2**32) + Fraction(abs(pos), 2**64) * max(1, math.ceil(abs(float(inv))))
