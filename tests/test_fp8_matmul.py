"""Block-scaled 8-bit products on the GPU against the float64 oracle.

Exact cases: codes are small integers and scales small powers of two, so that every partial
sum is an integer multiple of 2^-4 below 2^19 (K <= 8192): exact in float32 in any order,
and the result has to be equal bit for bit.

Rounded cases: fp32 accumulation of n = ceil(K / 32) + 12 additions (instruction steps, the
join of a split contraction, the addend), each within 2^-22 of the sum of magnitudes (twice a
truncation's step, for the alignment inside an instruction), then the rounding into the
output's type, half a step of it."""

import numpy as np
import pytest
import torch

import muon_newton_schulz_06_b200 as mb
from oracle import fp8
from test_fp8_blocks import codes, exps, values

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def h():
    handle = mb.muon_init(0)
    yield handle
    mb.muon_destroy(handle)


def small_ints(rows, cols, fmt, blocks, seed):
    """Integers -2 .. 2 under scales 2^-2 .. 2^2, as an Fp8Matrix."""
    rng = np.random.default_rng(seed)
    vals = fp8.code_values(fmt)
    table = np.array([int(np.flatnonzero(vals == v)[0]) for v in (-2, -1, 0, 1, 2)], dtype=np.uint8)
    m = mb.Fp8Matrix(rows, cols, format=fmt, blocks=blocks)
    m.codes.fill_(0x7f)                                   # padding holds NaN: it must never be read
    m.codes[:, :cols] = torch.from_numpy(table[rng.integers(0, 5, (rows, cols))]).cuda()
    m.scales.copy_(torch.from_numpy((127 + rng.integers(-2, 3, tuple(m.scales.shape))).astype(np.uint8)))
    return m


def operands(M, N, K, ta, tb, fa="e4m3", fb="e4m3", ba="square", bb="square", seed=0):
    a = small_ints(*((K, M) if ta else (M, K)), fa, ba, seed)
    b = small_ints(*((N, K) if tb else (K, N)), fb, bb, seed + 1)
    va, vb = values(a), values(b)
    return a, b, (va.T if ta else va), (vb.T if tb else vb)


SHAPES = [(1, 1, 1), (1, 128, 128), (5, 3, 130), (64, 512, 512), (128, 128, 128), (129, 257, 1000), (300, 200, 96),
          (257, 130, 4096), (1000, 777, 501), (16, 2048, 640), (700, 900, 33)]


@pytest.mark.parametrize("ta,tb", [(False, True), (False, False), (True, False), (True, True)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact(h, M, N, K, ta, tb):
    a, b, va, vb = operands(M, N, K, ta, tb, seed=M + N + K)
    d = torch.full((M, N), 7.0, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_a=ta, trans_b=tb)])
    mb.muon_sync(h)
    np.testing.assert_array_equal(d.double().cpu().numpy(), va @ vb)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("ba,bb", [("row", "square"), ("square", "row"), ("row", "row")])
def test_exact_formats_and_row_blocks(h, fa, fb, ba, bb):
    a, b, va, vb = operands(200, 333, 700, False, True, fa, fb, ba, bb, seed=4)
    d = torch.empty(200, 333, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True)])
    np.testing.assert_array_equal(d.double().cpu().numpy(), va @ vb)


def test_exact_many_tiles_and_long_contractions(h):
    """Persistent pairs of CTAs, two tiles per SM, and few tiles with a long K (split)."""
    for M, N, K in [(2600, 2700, 300), (4096, 2304, 768), (256, 256, 8192), (512, 384, 8100), (8192, 130, 128),
                    (1536, 2048, 300), (1, 40000, 129), (40000, 1, 129), (130, 1400, 2100), (2100, 2048, 2048)]:
        for ta, tb in [(False, True), (True, False)]:
            a, b, va, vb = operands(M, N, K, ta, tb, seed=K)
            d = torch.empty(M, N, device="cuda")
            mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_a=ta, trans_b=tb)])
            want = torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda()
            assert torch.equal(d.double(), want), (M, N, K, ta)


def test_extreme_scales(h):
    """Scales at the ends of the byte's range multiply to ordinary numbers; a scale of 255 is
    NaN for its block only."""
    M, N, K = 130, 140, 256
    a, b, _, _ = operands(M, N, K, False, True, seed=9)
    a.scales[0, 0], b.scales[0, 0], b.scales[1, 0] = 254, 1, 1         # 2^127 * 2^-126
    a.scales[1, 0] = 254
    d = torch.empty(M, N, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True)])
    np.testing.assert_array_equal(d.double().cpu().numpy(), values(a) @ values(b).T)
    a.scales[0, 1] = 255
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True)])
    assert d[:128].isnan().all() and not d[128:].isnan().any()


def test_nan_code_reaches_its_row_and_column_only(h):
    M, N, K = 200, 180, 300
    a, b, va, vb = operands(M, N, K, False, True, seed=11)
    a.codes[150, 299] = 0x7f
    d = torch.empty(M, N, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True)])
    nan = d.isnan()
    assert nan[150].all() and nan.sum() == N
    keep = [i for i in range(M) if i != 150]
    np.testing.assert_array_equal(d.double().cpu().numpy()[keep], (va @ vb)[keep])


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens", [33, 1000])
def test_rounded_realistic(h, out, tokens):
    rng = np.random.default_rng(5)
    M, N, K = tokens, 520, 1100
    x = torch.from_numpy(rng.standard_normal((M, K)) * np.exp(rng.standard_normal((1, K)))).float().cuda()
    w = torch.from_numpy(0.02 * rng.standard_normal((N, K))).float().cuda()
    a, b = mb.Fp8Matrix(M, K, blocks="row"), mb.Fp8Matrix(N, K)
    mb.muon_fp8_quantize(h, [x, w], [a, b])
    c = torch.from_numpy(rng.standard_normal((M, N))).to(DT[out]).cuda()
    d = torch.empty(M, N, dtype=DT[out], device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True, add=c)])
    want, mag = fp8.matmul(values(a), values(b).T, c.double().cpu().numpy())
    tol = (-(-K // 32) + 12) * 2.0 ** -22 * mag + torch.finfo(DT[out]).eps / 2 * np.abs(want) * 1.01
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_accumulates_in_place(h, out):
    a, b, va, vb = operands(300, 250, 2000, True, False, seed=2)
    g = torch.randint(-50, 50, (300, 250), device="cuda").to(DT[out])
    want = torch.from_numpy(g.double().cpu().numpy() + va @ vb)
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, g, trans_a=True, add=g)])
    assert torch.equal(g.double().cpu(), want.to(DT[out]).double())     # exact sum, one rounding


@pytest.mark.parametrize("blocks", ["square", "row"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (40, 70, 64), (130, 260, 500), (300, 520, 2048), (1024, 2048, 512)])
def test_eight_bit_results_are_exact(h, blocks, M, N, K):
    """Exact sums (and exact squares of them, below 2^24 after scaling) give the oracle's
    codes and exponents bit for bit, through each epilogue."""
    a, b, va, vb = operands(M, N, K, False, True, seed=M)
    want = va @ vb
    for epi in ("none", "relu2"):
        ref = fp8.relu2(want).astype(np.float32).astype(np.float64) if epi == "relu2" else want
        out = mb.Fp8Matrix(M, N, blocks=blocks, format="e5m2" if epi == "none" else "e4m3")
        out.codes.fill_(0xEE)
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, out, trans_b=True, epilogue=epi)])
        c, e = fp8.quantize(ref, out.format, blocks)
        np.testing.assert_array_equal(exps(out), e)
        np.testing.assert_array_equal(codes(out), c)
        assert (out.codes[:, N:] == 0xEE).all()
    # backward: saved values 0, 1, 4, 16 have exact roots
    saved = mb.Fp8Matrix(M, N, blocks=blocks)
    rng = np.random.default_rng(1)
    vals = fp8.code_values("e4m3")
    table = np.array([int(np.flatnonzero(vals == v)[0]) for v in (0, 1, 4, 16)], dtype=np.uint8)
    saved.codes[:, :N] = torch.from_numpy(table[rng.integers(0, 4, (M, N))]).cuda()
    saved.scales.copy_(torch.from_numpy((127 + 2 * rng.integers(-1, 2, tuple(saved.scales.shape))).astype(np.uint8)))
    ref = fp8.relu2_backward(want, values(saved))
    out = mb.Fp8Matrix(M, N, blocks=blocks)
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, out, trans_b=True, epilogue="relu2_backward", saved=saved)])
    c, e = fp8.quantize(ref, "e4m3", blocks)
    np.testing.assert_array_equal(exps(out), e)
    np.testing.assert_array_equal(values(out), fp8.dequantize(c, e, "e4m3", blocks))
    d = torch.empty(M, N, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True, epilogue="relu2_backward", saved=saved)])
    np.testing.assert_array_equal(d.double().cpu().numpy(), ref)


def quantized_equal(out, ref):
    c, e = fp8.quantize(ref, out.format, out.blocks)
    np.testing.assert_array_equal(exps(out), e)
    np.testing.assert_array_equal(values(out), fp8.dequantize(c, e, out.format, out.blocks))


BIG = (2350, 2195, 260)        # 342 tiles of 128 x 128: persistent pairs; nothing a multiple of 16


def roots(M, N, fmt, blocks, seed):
    """A checkpoint of 0, 1, 4, 16 under scales 2^-2, 1, 2^2: exact square roots."""
    saved = mb.Fp8Matrix(M, N, format=fmt, blocks=blocks)
    rng = np.random.default_rng(seed)
    vals = fp8.code_values(fmt)
    table = np.array([int(np.flatnonzero(vals == v)[0]) for v in (0, 1, 4, 16)], dtype=np.uint8)
    saved.codes[:, :N] = torch.from_numpy(table[rng.integers(0, 4, (M, N))]).cuda()
    saved.scales.copy_(torch.from_numpy((127 + 2 * rng.integers(-1, 2, tuple(saved.scales.shape))).astype(np.uint8)))
    return saved


@pytest.mark.parametrize("epi", ["none", "relu2", "relu2_backward"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("saved_fmt,saved_blocks", [("e4m3", "square"), ("e5m2", "row")])
def test_every_kind_of_result_of_many_tiles(h, epi, add, saved_fmt, saved_blocks):
    if epi != "relu2_backward" and saved_fmt == "e5m2":
        pytest.skip("no checkpoint in this epilogue")
    M, N, K = BIG
    a, b, va, vb = operands(M, N, K, False, True, seed=3)
    c = torch.randint(-9, 10, (M, N), device="cuda").float() if add else None
    base = va @ vb + (c.double().cpu().numpy() if add else 0.0)
    saved = roots(M, N, saved_fmt, saved_blocks, 5) if epi == "relu2_backward" else None
    ref = {"none": base, "relu2": fp8.relu2(base),
           "relu2_backward": fp8.relu2_backward(base, values(saved)) if saved else None}[epi]
    ref = ref.astype(np.float32).astype(np.float64)
    kw = dict(trans_b=True, epilogue=epi, saved=saved)
    for dt in ("bf16", "fp32"):
        for pitch, off in ((N, 0), (N + 13, 5), (N + 5, 0)):          # rows of every alignment
            big = torch.full((M, pitch), 3.0, dtype=DT[dt], device="cuda")
            d = big[:, off:off + N]
            cc = None
            if add:
                cc = c.to(DT[dt])
            mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, add=cc, **kw)])
            want = torch.from_numpy(ref).to(DT[dt])
            assert torch.equal(d.cpu(), want), (dt, pitch)
            rest = torch.cat([big[:, :off], big[:, off + N:]], dim=1)
            assert (rest == 3).all()
    for blocks in ("square", "row"):
        out = mb.Fp8Matrix(M, N, blocks=blocks)
        out.codes.fill_(0xEE)
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, out, add=c, **kw)])
        quantized_equal(out, ref)
        assert (out.codes[:, N:] == 0xEE).all()


@pytest.mark.parametrize("M,N,K", [(70, 135, 200), (70, 135, 4096), (300, 33, 200)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_few_tiles_in_rows_of_every_alignment(h, M, N, K, dt):
    """Result and addend in rows that start at any entry, whole and split contractions
    (sums exact in float32, rounded once)."""
    a, b, va, vb = operands(M, N, K, False, True, seed=M + K)
    for off in range(9):
        big = torch.full((M, N + 12), 3.0, dtype=DT[dt], device="cuda")
        c = torch.full((M, N + 14), float("nan"), dtype=DT[dt], device="cuda")
        add = c[:, 8 - off:8 - off + N]
        add.copy_(torch.randint(-9, 10, (M, N), device="cuda"))
        d = big[:, off:off + N]
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True, add=add)])
        want = torch.from_numpy((va @ vb + add.double().cpu().numpy()).astype(np.float32)).to(DT[dt])
        assert torch.equal(d.cpu(), want)
        assert (big[:, :off] == 3).all() and (big[:, off + N:] == 3).all()


@pytest.mark.parametrize("M,N,K", [(300, 520, 256), (200, 140, 4096), BIG])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("blocks", ["square", "row"])
def test_non_finite_sums_in_eight_bits(h, M, N, K, fmt, blocks):
    """Infinities and NaN do not reach the scale; they become the format's own."""
    a, b, va, vb = operands(M, N, K, False, True, seed=8)
    c = torch.zeros(M, N, device="cuda")
    c[0, 0], c[M - 1, N - 1], c[130, 131], c[150, :128] = float("inf"), float("nan"), -float("inf"), float("inf")
    ref = va @ vb + c.double().cpu().numpy()
    out = mb.Fp8Matrix(M, N, format=fmt, blocks=blocks)
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, out, trans_b=True, add=c)])
    quantized_equal(out, ref)
    # an 8-bit operand with a NaN entry: its row only
    a.codes[5, 7] = 0x7f
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, out, trans_b=True)])
    ref = va @ vb
    ref[5, :] = np.nan
    quantized_equal(out, ref)


def test_launches_of_mixed_kinds(h):
    """Results of different kinds in one persistent launch, more than one launch takes."""
    M, N, K = 1300, 1100, 200
    prods, checks = [], []
    for i in range(10):
        ta, tb = bool(i & 1), bool(i & 2)
        a, b, va, vb = operands(M, N, K + i, ta, tb, seed=i)
        want = va @ vb
        kw = dict(trans_a=ta, trans_b=tb)
        if i % 3 == 0:
            out = torch.empty(M, N, device="cuda")
        elif i % 3 == 1:
            out = mb.Fp8Matrix(M, N, format="e5m2")
        else:
            out = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
            kw["epilogue"], kw["saved"] = "relu2_backward", roots(M, N, "e4m3", "square", i)
            want = fp8.relu2_backward(want, values(kw["saved"]))
        prods.append(mb.Fp8Product(a, b, out, **kw))
        checks.append((out, want))
    mb.muon_fp8_matmul(h, prods)
    mb.muon_sync(h)
    for out, want in checks:
        if isinstance(out, mb.Fp8Matrix):
            quantized_equal(out, want)
        else:
            assert torch.equal(out.cpu(), torch.from_numpy(want).to(out.dtype))


@pytest.mark.parametrize("M,N,K", [(2600, 2700, 9001), (257, 300, 16000), (1500, 1400, 5000), (128, 128, 16000)])
def test_long_contractions_in_parts(h, M, N, K):
    """float32 results whose contraction is summed in parts: in segments of 4096 (many
    tiles), or in several accumulators; with and without an addend, in
    place, and in rows of odd alignment. Exact, as above (sums stay below 2^20 here)."""
    for ta, tb in ((False, True), (True, False)):
        a, b, va, vb = operands(M, N, K, ta, tb, seed=K)
        want = torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda()
        assert want.abs().max() < 2 ** 20
        c = torch.randint(-9, 10, (M, N), device="cuda").float()
        big = torch.full((M, N + 7), 3.0, device="cuda")
        d, acc = torch.empty(M, N, device="cuda"), c.clone()
        kw = dict(trans_a=ta, trans_b=tb)
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, **kw)])
        assert torch.equal(d.double(), want)
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, acc, add=acc, **kw)])
        assert torch.equal(acc.double(), want + c.double())
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, big[:, 3:3 + N], add=c, **kw)])
        assert torch.equal(big[:, 3:3 + N].double(), want + c.double())
        assert (big[:, :3] == 3).all() and (big[:, 3 + N:] == 3).all()
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, add=c, **kw), mb.Fp8Product(a, b, big[:, :N], **kw)])
        assert torch.equal(d.double(), want + c.double()) and torch.equal(big[:, :N].double(), want)


def test_accuracy_of_long_sums(h):
    """A contraction of 16384 in parts of 4096 (or less), each n = 128 additions of 32 products.
    An addition truncates by less than 2^-23 of the partial sum; after i of n random-sign steps
    that is sqrt(i / n) of the part's result in the mean square, so a part is off by at most
    2^-23 sqrt(sum i / n) = 2^-23 sqrt((n + 1) / 2) = 9.6e-7 of its result, and four independent
    parts by the same share of the whole (with 2^-24 for the rounding of their sum: 1.02e-6).
    Elementwise: n + 12 steps within 2^-22 of the sum of magnitudes, as for every product."""
    g = torch.Generator(device="cuda").manual_seed(0)
    for M, N in ((4096, 2560), (256, 256)):
        a, b = mb.Fp8Matrix(16384, M), mb.Fp8Matrix(16384, N)
        mb.muon_fp8_quantize(h, [torch.randn(16384, n, generator=g, device="cuda") for n in (M, N)], [a, b])
        va, vb = (torch.empty(16384, n, device="cuda") for n in (M, N))
        mb.muon_fp8_dequantize(h, [a, b], [va, vb])
        want = va.double().t() @ vb.double()
        d = torch.empty(M, N, device="cuda")
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_a=True)])
        err = (d.double() - want)
        assert err.norm() <= 1.02e-6 * want.norm()
        assert (err.abs() <= (128 + 12) * 2.0 ** -22 * (va.abs().double().t() @ vb.abs().double())).all()


def test_list_of_products_mixed(h):
    """Forms, shapes and destinations mixed in one call; more products than one launch takes;
    empty results and empty contractions among them."""
    prods, checks = [], []
    shapes = [(50, 60, 70), (1, 300, 128), (260, 20, 600), (128, 256, 0), (0, 40, 64), (40, 0, 64), (129, 129, 129)]
    for i in range(21):
        M, N, K = shapes[i % len(shapes)]
        ta, tb = bool(i & 1), bool(i & 2)
        a, b, va, vb = operands(M, N, K, ta, tb, seed=i)
        d = torch.full((M, N), 3.0, device="cuda")
        prods.append(mb.Fp8Product(a, b, d, trans_a=ta, trans_b=tb, add=d if i % 3 == 0 else None))
        checks.append((d, va @ vb + (3.0 if i % 3 == 0 else 0.0)))
    mb.muon_fp8_matmul(h, prods)
    assert mb.muon_last_launch_count(h) == 1      # 15 results with entries fit one launch
    for d, want in checks:
        np.testing.assert_array_equal(d.double().cpu().numpy(), want)
    more = []
    for i in range(35):
        a, b, va, vb = operands(33 + i, 20, 40 + i, False, True, seed=i)
        more.append((a, b, torch.empty(33 + i, 20, device="cuda"), va @ vb))
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True) for a, b, d, _ in more])
    for _, _, d, want in more:
        np.testing.assert_array_equal(d.double().cpu().numpy(), want)


def test_column_slices_as_results(h):
    """q, k and v written into one tensor; odd pitch and offset; the rest stays."""
    x, w1, vx, vw1 = operands(150, 130, 256, False, True, seed=1)
    w2 = small_ints(67, 256, "e4m3", "square", 77)
    big = torch.full((150, 211), 5.0, device="cuda", dtype=torch.float32)
    mb.muon_fp8_matmul(h, [mb.Fp8Product(x, w1, big[:, 1:131], trans_b=True),
                           mb.Fp8Product(x, w2, big[:, 131:198], trans_b=True)])
    got = big.double().cpu().numpy()
    np.testing.assert_array_equal(got[:, 1:131], vx @ vw1)
    np.testing.assert_array_equal(got[:, 131:198], vx @ values(w2).T)
    assert (got[:, 0] == 5).all() and (got[:, 198:] == 5).all()


def test_deterministic_and_capturable(h):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((4096, 256))).float().cuda()
    y = torch.from_numpy(rng.standard_normal((4096, 384))).float().cuda()
    a, b = mb.Fp8Matrix(4096, 256), mb.Fp8Matrix(4096, 384)
    handle = mb.muon_init(0)
    d = torch.empty(256, 384, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mb.muon_fp8_quantize(handle, [x, y], [a, b])
        mb.muon_fp8_matmul(handle, [mb.Fp8Product(a, b, d, trans_a=True)])
    g.replay()
    first = d.clone()
    for _ in range(20):
        d.zero_()
        g.replay()
        assert torch.equal(d, first)
    eager = torch.empty_like(d)
    mb.muon_fp8_matmul(handle, [mb.Fp8Product(a, b, eager, trans_a=True)])
    mb.muon_sync(handle)
    assert torch.equal(eager, first)
    # two streams at once, one handle
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(d) for _ in s]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, o in zip(s, outs):
            mb.muon_fp8_matmul(handle, [mb.Fp8Product(a, b, o, trans_a=True)], stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
    del g
    mb.muon_destroy(handle)


@pytest.mark.parametrize("ta,tb", [(False, True), (False, False), (True, False), (True, True)])
@pytest.mark.parametrize("M,N,K", [(2048, 512, 4200), (1000, 1400, 2100), (1013, 777, 4100), (130, 2200, 5000),
                                   (640, 1290, 4096), (1500, 1025, 8000)])
def test_exact_mid_sizes_with_long_contractions(h, M, N, K, ta, tb):
    """Results of 36 to 148 tiles of 128 x 128, contractions whole and split; dense epilogues,
    addends, rows of any alignment."""
    a, b, va, vb = operands(M, N, K, ta, tb, seed=M + K)
    base = torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda()
    kw = dict(trans_a=ta, trans_b=tb)
    for dt, pad, off in (("fp32", 0, 0), ("bf16", 0, 0), ("fp32", 7, 3), ("bf16", 7, 5)):
        c = torch.randint(-9, 10, (M, N), device="cuda").to(DT[dt])
        big = torch.full((M, N + pad), 3.0, dtype=DT[dt], device="cuda")
        d = big[:, off:off + N]
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, **kw)])
        assert torch.equal(d, base.float().to(DT[dt]))
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, add=c, epilogue="relu2", **kw)])
        assert torch.equal(d, (base + c.double()).float().relu().square().to(DT[dt]))
        acc = c.clone()                                                   # two in one launch, one in place
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, add=c, **kw), mb.Fp8Product(a, b, acc, add=acc, **kw)])
        assert torch.equal(d, (base + c.double()).float().to(DT[dt])) and torch.equal(d, acc)
        assert (big[:, :off] == 3).all() and (big[:, off + N:] == 3).all()


def test_many_products_of_one_operand(h):
    """One weight read by every item of a long list, each with a result of its own."""
    n = 20000
    w = small_ints(40, 160, "e4m3", "square", 1)
    x = small_ints(3, 160, "e4m3", "row", 2)
    y = torch.full((n, 3, 40), 7.0, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(x, w, y[i], trans_b=True) for i in range(n)])
    want = torch.from_numpy(values(x) @ values(w).T).float().cuda()
    assert (y == want).all()
    with pytest.raises(mb.MuonError, match="overlap"):                 # two of them to one result
        mb.muon_fp8_matmul(h, [mb.Fp8Product(x, w, y[i % (n - 1)], trans_b=True) for i in range(n)])


def far(m, pitch):
    """The same matrix with its rows `pitch` bytes apart (and scales of its own)."""
    buf = torch.empty(m.rows, pitch, dtype=torch.uint8, device="cuda")
    buf[:, :m.cols] = m.codes[:, :m.cols]
    return mb.Fp8Matrix(m.rows, m.cols, format=m.format, blocks=m.blocks, codes=buf[:, :m.cols], scales=m.scales.clone())


@pytest.mark.parametrize("N", [1500, 100])
def test_rows_past_32_bits(h, N):
    """Operand, checkpoint, addend and results whose last rows lie past 2^32 entries of their
    base: the same as with rows close together. Pairs (N = 1500) and a CTA per tile."""
    M, K, pitch = 4100, 256, 1 << 20
    a, b, _, _ = operands(M, N, K, False, True, seed=9)
    saved = small_ints(M, N, "e4m3", "row", 11)
    saved.codes.bitwise_and_(0x7f)                             # a checkpoint of relu^2 is not negative
    c = torch.randint(-9, 10, (M, N), device="cuda").bfloat16()
    want, want8 = torch.empty_like(c), mb.Fp8Matrix(M, N)
    kw = dict(trans_b=True, epilogue="relu2_backward")
    for out in (want, want8):
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, out, add=c, saved=saved, **kw)])
    a_far, saved_far, out8 = far(a, pitch), far(saved, pitch), far(want8, pitch)
    out8.codes.fill_(0)
    out8.scales.fill_(0)
    d = torch.empty(M, pitch, dtype=torch.bfloat16, device="cuda")[:, :N]
    d.copy_(c)
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a_far, b, out8, add=d, saved=saved_far, **kw)])
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a_far, b, d, add=d, saved=saved_far, **kw)])
    assert torch.equal(d, want)
    assert torch.equal(out8.codes[:, :N], want8.codes[:, :N]) and torch.equal(out8.scales, want8.scales)
    # the block passes, on the same matrices
    dy = torch.empty(M, pitch, dtype=torch.bfloat16, device="cuda")[:, :N]
    mb.muon_fp8_dequantize(h, [out8], [dy])
    near, du = torch.empty_like(c), torch.empty_like(c)
    mb.muon_fp8_dequantize(h, [want8], [near])
    assert torch.equal(dy, near)
    mb.muon_fp8_act_backward(h, [near], [saved], [du])
    mb.muon_fp8_act_backward(h, [dy], [saved_far], [d])
    assert torch.equal(d, du)
    mb.muon_fp8_quantize(h, [near, dy], [want8, out8])
    assert torch.equal(out8.codes[:, :N], want8.codes[:, :N]) and torch.equal(out8.scales, want8.scales)


def test_refusals(h):
    a, b = mb.Fp8Matrix(64, 128), mb.Fp8Matrix(96, 128)
    d = torch.zeros(64, 96, device="cuda")

    def refused(match, **kw):
        p = dict(a=a, b=b, out=d, trans_b=True)
        p.update(kw)
        with pytest.raises(mb.MuonError, match=match) as ei:
            mb.muon_fp8_matmul(h, [mb.Fp8Product(**p)])
        assert ei.value.code == mb.MUON_ERR_INVALID_ARG

    refused("op\\(A\\)", trans_b=False)
    refused("op\\(A\\)", trans_a=True)
    refused("the product 64 x 96", out=torch.zeros(64, 95, device="cuda"))
    refused("the product 64 x 96", out=mb.Fp8Matrix(64, 97))
    refused("c is", add=torch.zeros(63, 96, device="cuda"))
    refused("saved is", epilogue="relu2_backward", saved=mb.Fp8Matrix(64, 95))
    refused("square", a=mb.Fp8Matrix(128, 64, blocks="row"), trans_a=True)
    refused("square", b=mb.Fp8Matrix(128, 96, blocks="row"), trans_b=False)
    big = torch.zeros(64, 200, device="cuda")
    refused("overlap", out=big[:, :96], add=big[:, 1:97])
    sq = mb.Fp8Matrix(128, 128)
    refused("overlap", a=sq, b=sq, out=sq, trans_b=False)
    with pytest.raises(mb.MuonError, match="overlap"):
        mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True), mb.Fp8Product(a, b, d, trans_b=True)])
    # the same operands twice are fine
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, big[:, :96], trans_b=True),
                           mb.Fp8Product(a, b, big[:, 100:196], trans_b=True)])
    lib = mb.load_library()
    assert lib.muon_fp8_matmul(h, None, 1, None) == mb.MUON_ERR_INVALID_ARG
    raw = (mb.muon_fp8_product * 1)()
    raw[0].a, raw[0].b, raw[0].trans_b = a.c, b.c, 1
    assert lib.muon_fp8_matmul(h, raw, 1, None) == mb.MUON_ERR_INVALID_ARG          # no destination
    raw[0].d = mb.muon_dense(d.data_ptr(), 64, 96, 96, mb.MUON_F32)
    raw[0].epilogue = 9
    assert lib.muon_fp8_matmul(h, raw, 1, None) == mb.MUON_ERR_INVALID_ARG
    assert b"epilogue" in lib.muon_last_error(h)
    mb.muon_sync(h)
    # rows that no address space holds
    wide = mb.Fp8Matrix(512, 128)
    wide.c.ld = 1 << 39
    with pytest.raises(mb.MuonError, match="pitch"):
        mb.muon_fp8_dequantize(h, [wide], [torch.empty(512, 128, device="cuda")])
