"""Accuracy of float32 results over long contractions, whatever their size and their neighbours in
the list.

A contraction goes in parts of at most 4096, each at most n = 128 additions of 32 products. An
addition truncates by less than 2^-23 of the partial sum; after i of n random-sign steps that is
sqrt(i / n) of the part's result in the mean square, so a part is off by at most
2^-23 sqrt(sum i / n) = 2^-23 sqrt((n + 1) / 2) = 9.6e-7 of its result, and independent parts by the
same share of the whole. Joining P parts rounds to nearest, 2^-24 of a partial sum each time:
2^-24 sqrt((P + 1) / 2) in the same way, 1.75e-7 for 16 parts."""
import math

import pytest
import torch

import muon_newton_schulz_06_b200 as mb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    handle = mb.muon_init(0)
    yield handle
    mb.muon_destroy(handle)


def normal(h, rows, cols, g):
    m, v = mb.Fp8Matrix(rows, cols), torch.empty(rows, cols, device="cuda")
    mb.muon_fp8_quantize(h, [torch.randn(rows, cols, generator=g, device="cuda")], [m])
    mb.muon_fp8_dequantize(h, [m], [v])
    return m, v.double()


def check(d, va, vb):
    parts = math.ceil(va.shape[0] / 4096)
    want = va.t() @ vb
    err = ((d.double() - want).norm() / want.norm()).item()
    print(f"{tuple(d.shape)} x {va.shape[0]}: {err:.3e}")
    assert err <= 2.0 ** -23 * math.sqrt(129 / 2) + 2.0 ** -24 * math.sqrt((parts + 1) / 2)


@pytest.mark.parametrize("M,N,K", [(1280, 1280, 65536), (1536, 1536, 16384), (512, 384, 65536), (1000, 1100, 40000),
                                   (1280, 1152, 65001), (256, 256, 131072)])
def test_long_contraction_of_few_tiles(h, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(K)
    (a, va), (b, vb) = normal(h, K, M, g), normal(h, K, N, g)
    d = torch.empty(M, N, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_a=True)])
    check(d, va, vb)
    first = d.clone()
    c = torch.randn(M, N, generator=g, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_a=True, add=c)])
    assert torch.equal(d, first + c)                       # the same sum, one more addition
    for _ in range(5):
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_a=True)])
        assert torch.equal(d, first)


@pytest.mark.parametrize("other", ["bf16", "codes", "relu2"])
def test_long_contraction_beside_other_kinds(h, other):
    """Many tiles; the neighbour is a result that goes without parts."""
    g = torch.Generator(device="cuda").manual_seed(1)
    M, N, K = 2560, 2304, 16384
    (a, va), (b, vb) = normal(h, K, M, g), normal(h, K, N, g)
    d, alone = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    out = {"bf16": torch.empty(M, N, device="cuda", dtype=torch.bfloat16), "codes": mb.Fp8Matrix(M, N),
           "relu2": torch.empty(M, N, device="cuda")}[other]
    epi = "relu2" if other == "relu2" else "none"
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, out, trans_a=True, epilogue=epi), mb.Fp8Product(a, b, d, trans_a=True)])
    check(d, va, vb)
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, alone, trans_a=True)])
    assert torch.equal(d, alone)


@pytest.mark.parametrize("short", [128, 512])
def test_long_contraction_beside_a_short_one(h, short):
    """164 tiles of 128 x 128 in the list, 100 of them with the long contraction."""
    g = torch.Generator(device="cuda").manual_seed(2)
    (a, va), (b, vb) = normal(h, 16384, 1280, g), normal(h, 16384, 1280, g)
    (s, vs), (t, vt) = normal(h, short, 1024, g), normal(h, short, 1024, g)
    d, e = torch.empty(1280, 1280, device="cuda"), torch.empty(1024, 1024, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(s, t, e, trans_a=True), mb.Fp8Product(a, b, d, trans_a=True)])
    check(d, va, vb)
    check(e, vs, vt)
