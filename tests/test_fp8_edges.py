"""Products of many tiles whose last column of tiles is cut off: 8-bit results alone and beside
dense ones, three and more tiles per pair of CTAs, so that the two blocks of a tile finish at
different times.  Sums are exact (small integers, powers of two), so the codes have to be those of
the quantised exact result."""
import pytest
import torch

import muon_newton_schulz_06_b200 as mb
from test_fp8_matmul import operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    handle = mb.muon_init(0)
    yield handle
    mb.muon_destroy(handle)


def same(h, out, want):
    """out holds the codes and scales of want (float32, exact)."""
    ref = mb.Fp8Matrix(out.rows, out.cols, format=out.format, blocks=out.blocks)
    mb.muon_fp8_quantize(h, [want], [ref])
    n = out.cols
    return torch.equal(out.codes[:, :n], ref.codes[:, :n]) and torch.equal(out.scales, ref.scales)


@pytest.mark.parametrize("blocks", ["square", "row"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("M,N,K", [(12000, 1100, 100), (10100, 1290, 129), (22000, 400, 64)])
def test_blocks_cut_off_at_the_right_edge(h, M, N, K, add, blocks):
    a, b, va, vb = operands(M, N, K, False, True, seed=M)
    want = (torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda()).float()
    c = torch.randint(-9, 10, (M, N), device="cuda").float() if add else None
    want = want + c if add else want
    out = mb.Fp8Matrix(M, N, format="e5m2", blocks=blocks)
    for _ in range(20):
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, out, trans_b=True, add=c)])
    mb.muon_sync(h)                                      # no wait ran out
    assert same(h, out, want)


def test_eight_bit_results_between_dense_ones(h):
    """Tiles of every kind in turn in one launch: a dense tile makes no use of what an 8-bit one
    hands over."""
    prods, checks = [], []
    for i in range(8):
        M, N, K = 1500 + 128 * i, 1100 - 64 * i, 64 + 3 * i
        a, b, va, vb = operands(M, N, K, False, True, seed=i)
        want = (torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda()).float()
        out = mb.Fp8Matrix(M, N) if i % 2 else torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
        prods.append(mb.Fp8Product(a, b, out, trans_b=True))
        checks.append((out, want))
    for _ in range(20):
        mb.muon_fp8_matmul(h, prods)
    mb.muon_sync(h)
    for out, want in checks:
        assert same(h, out, want) if isinstance(out, mb.Fp8Matrix) else torch.equal(out, want.bfloat16())
