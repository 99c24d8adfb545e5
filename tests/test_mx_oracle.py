"""The MXFP4 definitions in 64 bits against hand-computed blocks and a search in exact rationals; the packer."""
from fractions import Fraction

import numpy as np
import pytest

from block_quantized_weight_qmv_amd import qmv
from oracle import mx


def test_code_values():
    assert mx.code_values().tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_hand_block():
    # 2^-1 and 2^3, codes 0..15 twice each
    p = np.array([[126, 130]])
    code = np.concatenate([np.repeat(np.arange(16), 2), np.tile(np.arange(16), 2)])[None].astype(np.uint8)
    data = mx.mx4_pack(p, code)
    assert data.tolist() == [17 * i for i in range(16)] + [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2 + [126, 130]
    w = mx.mx4_decode64(data, 1, 64)[0]
    assert w[:8].tolist() == [0, 0, .25, .25, .5, .5, .75, .75]
    assert w[32:40].tolist() == [0, 4, 8, 12, 16, 24, 32, 48]
    data[-1] = 255
    assert np.isnan(mx.mx4_decode64(data, 1, 64)[0, 32:]).all()


def test_encoder_is_the_nearest_even():
    rng = np.random.default_rng(0)
    vals = [Fraction(v) for v in mx.code_values()[:8].tolist()]
    x = np.float32(rng.standard_normal((40, 32)) * np.exp2(rng.integers(-140, 100, (40, 1))))
    x[0, :8] = [8, 2.5, 5, 0.25, 0.75, 1.25, 1.75, 3.5]
    x[1, :4] = [7.99, 7, 6.5, -0.0]
    x[2] = 0
    p, code = mx.mx4_encode64(x.astype(np.float64))
    for r in range(len(x)):
        top = max(abs(Fraction(float(v))) for v in x[r])
        e = 0
        while top and top >= Fraction(8) * Fraction(2) ** (e - 127):
            e += 1
        assert p[r, 0] == e
        for k in range(32):
            m = abs(Fraction(float(x[r, k]))) / Fraction(2) ** (e - 127)
            best = min(range(8), key=lambda c: (abs(m - vals[c]), c % 2))
            assert code[r, k] & 7 == best, (r, k)
            assert code[r, k] >> 3 == np.signbit(x[r, k])


def test_encoder_on_nonfinite_blocks():
    x = np.ones((1, 96))
    x[0, 3], x[0, 40] = np.inf, np.nan
    p, code = mx.mx4_encode64(x)
    assert p.tolist() == [[255, 255, 125]] and not code[0, :64].any() and (code[0, 64:] == 6).all()


def test_packer_is_the_oracle():
    rng = np.random.default_rng(1)
    p, code = rng.integers(0, 256, (5, 3)), rng.integers(0, 16, (5, 96))
    assert np.array_equal(qmv.qmv_pack_mxfp4(p, code, 5, 96), mx.mx4_pack(p, code))
    assert qmv.qmv_packed_size("mxfp4", 5, 96) == 5 * 3 * 17 and qmv.qmv_block_size("mxfp4") == 32
    assert qmv.qmv_packed_size("mxfp4", 5, 48) == 0
    code[2, 7] = 16
    with pytest.raises(qmv.QmvError) as e:
        qmv.qmv_pack_mxfp4(p, code, 5, 96)
    assert e.value.status == -7


def test_groups_are_clamped():
    assert mx.groups([2, 5, 4, 9, 7], 8) == [(2, 5), (5, 5), (5, 8), (8, 8)]
    assert mx.groups([-3, -1, 2], 8) == [(0, 0), (0, 2)]


def test_norm_by_hand():
    x = np.array([[1.0, 2.0, 3.0, 6.0]])
    assert np.allclose(mx.norm64(x, "rms", eps=0.0), x / np.sqrt(12.5))
    assert np.allclose(mx.norm64(x, "layer", np.array([2.0]), np.array([1.0]), 0.5), (x - 3) / np.sqrt(4.0) * 2 + 1)
