"""The 8-bit oracle against independent statements of the format (CPU): torch's 8-bit types
for the codes, the definition of the scale by search, derivatives by differences; and the
binding's refusals that need no device."""
import ctypes

import numpy as np
import pytest
import torch

import muon_newton_schulz_06_b200 as mb
from muon_newton_schulz_06_b200 import build as mbuild
from oracle import fp8

TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_code_values_are_the_types(fmt):
    t = torch.arange(256, dtype=torch.uint8).view(TORCH[fmt]).double().numpy()
    np.testing.assert_array_equal(fp8.code_values(fmt), t)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_encode_rounds_like_the_type(fmt):
    rng = np.random.default_rng(0)
    pos = fp8.code_values(fmt)
    pos = np.sort(pos[np.isfinite(pos) & (pos >= 0)])
    mids = 0.5 * (pos[1:] + pos[:-1])                       # ties, exact in float32
    v = np.concatenate([pos, mids, np.nextafter(mids.astype(np.float32), np.float32(np.inf)).astype(np.float64),
                        rng.uniform(0, fp8.TOP[fmt], 4000), 2.0 ** rng.uniform(-20, 8, 4000), [0.0, np.nan]])
    v = np.concatenate([v, -v]).astype(np.float32).astype(np.float64)
    v = v[~(np.abs(v) > fp8.TOP[fmt])]
    want = torch.tensor(v, dtype=torch.float32).to(TORCH[fmt]).double().numpy()
    got = fp8.code_values(fmt)[fp8.encode(v, fmt)]
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(np.signbit(got[got == 0]), np.signbit(want[got == 0]))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_exponent_is_least(fmt):
    top = fp8.TOP[fmt]
    for a in [top, np.nextafter(np.float32(top), np.float32(np.inf)), 1.0, 0.875, 1e-30, 3e38, 0.3, 2.0 ** -20]:
        a = float(a)
        e = fp8.exponent(a, fmt)
        assert a <= top * 2.0 ** e and a > top * 2.0 ** (e - 1)
    assert fp8.exponent(0.0, fmt) == 0 and fp8.exponent(1e-45, fmt) == -127


@pytest.mark.parametrize("blocks", ["square", "row"])
def test_round_trip_error_is_half_a_step(blocks):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 300)) * np.exp(rng.standard_normal((1, 300)))
    codes, e = fp8.quantize(x, "e4m3", blocks)
    back = fp8.dequantize(codes, e, "e4m3", blocks)
    scale = np.exp2(fp8.expand(e, 200, 300, blocks))
    assert np.all(np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10))


def test_relu2_backward_is_the_derivative():
    u = np.linspace(-3, 3, 61)
    h = 1e-6
    num = (fp8.relu2(u + h) - fp8.relu2(u - h)) / (2 * h)
    np.testing.assert_allclose(fp8.relu2_backward(np.ones_like(u), fp8.relu2(u)), num, atol=2e-6)


# ----------------------------------------------------------------------------- refusals without a device

@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mb.load_library()


def test_null_handle(lib):
    for call in (lambda: lib.muon_fp8_quantize(None, None, None, 0, 0, None),
                 lambda: lib.muon_fp8_dequantize(None, None, None, 0, None),
                 lambda: lib.muon_fp8_act_backward(None, None, None, None, None, 0, 0, None),
                 lambda: lib.muon_fp8_matmul(None, None, 0, None),
                 lambda: lib.muon_selftest_fp8_timeout(None, 0, None),
                 lambda: lib.muon_fp8_profile_read(None, None, None)):
        assert call() == mb.MUON_ERR_INVALID_ARG


def test_structs_match_the_header():
    assert ctypes.sizeof(mb.muon_fp8_matrix) == 48
    assert ctypes.sizeof(mb.muon_dense) == 40
    assert ctypes.sizeof(mb.muon_fp8_product) == 288


def test_fp8_matrix_checks():
    m = mb.Fp8Matrix(200, 300, device="cpu")
    assert m.codes.shape == (200, 304) and m.scales.shape == (2, 3) and m.c.ld == 304
    m = mb.Fp8Matrix(200, 300, blocks="row", format="e5m2", device="cpu")
    assert m.scales.shape == (3, 200) and (m.c.format, m.c.blocks) == (1, 1)
    assert mb.Fp8Matrix(0, 5, device="cpu").shape == (0, 5)
    with pytest.raises(ValueError, match="format"):
        mb.Fp8Matrix(1, 1, format="e3m4", device="cpu")
    with pytest.raises(ValueError, match="blocks"):
        mb.Fp8Matrix(1, 1, blocks="column", device="cpu")
    with pytest.raises(ValueError, match=">= 0"):
        mb.Fp8Matrix(-1, 1, device="cpu")
    with pytest.raises(ValueError, match="both"):
        mb.Fp8Matrix(1, 1, codes=m.codes)
    with pytest.raises(TypeError, match="CUDA"):
        mb.Fp8Matrix(200, 300, codes=m.codes, scales=m.scales)


def test_binding_refuses():
    m = mb.Fp8Matrix(4, 4, device="cpu")
    w = torch.zeros(4, 4)
    with pytest.raises(TypeError, match="CUDA"):
        mb.muon_fp8_quantize(None, [w], [m])
    with pytest.raises(TypeError, match="Fp8Matrix"):
        mb.muon_fp8_dequantize(None, [w], [w])
    with pytest.raises(ValueError, match="length"):
        mb.muon_fp8_quantize(None, [w], [])
    with pytest.raises(ValueError, match="activation"):
        mb.muon_fp8_quantize(None, [w], [m], activation="gelu")
    with pytest.raises(ValueError, match="activation"):
        mb.muon_fp8_act_backward(None, [w], [m], [w], activation="gelu")
    with pytest.raises(TypeError, match="Fp8Matrix"):
        mb.muon_fp8_matmul(None, [mb.Fp8Product(w, m, m)])
    with pytest.raises(ValueError, match="epilogue"):
        mb.muon_fp8_matmul(None, [mb.Fp8Product(m, m, m, epilogue="gelu")])
    with pytest.raises(ValueError, match="saved"):
        mb.muon_fp8_matmul(None, [mb.Fp8Product(m, m, m, epilogue="relu2_backward")])
    with pytest.raises(ValueError, match="saved"):
        mb.muon_fp8_matmul(None, [mb.Fp8Product(m, m, m, saved=m)])
