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
from oracle import fp8
from test_fp8_blocks import codes, exps, values
from test_fp8_matmul import operands, roots

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


@pytest.mark.parametrize("M,N,K", [(300, 257, 52000), (640, 1290, 40000), (1100, 1300, 13000)])
def test_segments_beside_other_kinds_in_one_launch(h, M, N, K):
    """Few tiles: a float32 contraction summed in segments, in rows of any alignment and in place,
    beside 8-bit and bf16 results with their epilogues. Sums of small integers, exact in float32."""
    a, b, va, vb = operands(M, N, K, True, False, seed=K)
    want = torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda()
    assert want.abs().max() < 2 ** 19
    s, t, vs, vt = operands(100, 120, 300, False, True, seed=1)
    saved = roots(100, 120, "e4m3", "square", 2)
    c = torch.randint(-9, 10, (M, N), device="cuda").float()
    acc, big = c.clone(), torch.full((M, N + 7), 3.0, device="cuda")
    q, g = mb.Fp8Matrix(100, 120), torch.empty(100, 120, device="cuda", dtype=torch.bfloat16)
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, acc, trans_a=True, add=acc),
                           mb.Fp8Product(s, t, q, trans_b=True, epilogue="relu2"),
                           mb.Fp8Product(s, t, g, trans_b=True, epilogue="relu2_backward", saved=saved)])
    assert mb.muon_last_launch_count(h) == 1
    assert torch.equal(acc.double(), want + c.double())
    x, e = fp8.quantize(fp8.relu2(vs @ vt))
    assert (codes(q) == x).all() and (exps(q) == e).all()
    assert torch.equal(g.cpu(), torch.from_numpy(fp8.relu2_backward(vs @ vt, values(saved))).bfloat16())
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, big[:, 3:3 + N], trans_a=True, add=c)])
    assert torch.equal(big[:, 3:3 + N].double(), want + c.double())
    assert (big[:, :3] == 3).all() and (big[:, 3 + N:] == 3).all()
