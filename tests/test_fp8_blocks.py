"""Block passes of the 8-bit format on the GPU against the float64 oracle: quantise (with
relu^2), read back, activation gradient; refusals, strides, non-finite entries, capture."""
import numpy as np
import pytest
import torch

import muon_newton_schulz_06_b200 as mb
from oracle import fp8

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def h():
    handle = mb.muon_init(0)
    yield handle
    mb.muon_destroy(handle)


def exps(m: mb.Fp8Matrix) -> np.ndarray:
    e = m.scales.cpu().numpy().astype(np.int64) - 127
    return e if m.blocks == "square" else e.T


def codes(m: mb.Fp8Matrix) -> np.ndarray:
    return m.codes[:, :m.cols].cpu().numpy()


def values(m: mb.Fp8Matrix) -> np.ndarray:
    return fp8.dequantize(codes(m), exps(m), m.format, m.blocks)


def data(rows, cols, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2.0 * torch.randn(1, cols, generator=g))
    return x.to(DT[dtype])


SHAPES = [(1, 1), (1, 128), (3, 5), (16, 512), (127, 129), (128, 128), (129, 127), (200, 1000), (257, 384), (513, 40)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("blocks", ["square", "row"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_and_back_are_exact(h, fmt, blocks, dtype):
    """Scaling by a power of two is exact, so codes and exponents equal the oracle's; values
    have 4 significant bits and read back exactly."""
    xs = [data(r, c, 10 + i, dtype) for i, (r, c) in enumerate(SHAPES)]
    outs = [mb.Fp8Matrix(r, c, format=fmt, blocks=blocks) for r, c in SHAPES]
    mb.muon_fp8_quantize(h, [x.cuda() for x in xs], outs)          # one call for all
    back = [torch.empty(s, dtype=DT[dtype], device="cuda") for s in SHAPES]
    mb.muon_fp8_dequantize(h, outs, back)
    for x, m, b in zip(xs, outs, back):
        c, e = fp8.quantize(x.double().numpy(), fmt, blocks)
        np.testing.assert_array_equal(exps(m), e)
        np.testing.assert_array_equal(codes(m), c)
        np.testing.assert_array_equal(b.double().cpu().numpy(), values(m))


@pytest.mark.parametrize("blocks", ["square", "row"])
def test_quantize_relu2_bf16_is_exact(h, blocks):
    """A bf16 entry squared has 16 significant bits: exact in float32, rounded once."""
    x = data(300, 260, 3, "bf16")
    m = mb.Fp8Matrix(300, 260, blocks=blocks)
    mb.muon_fp8_quantize(h, [x.cuda()], [m], activation="relu2")
    c, e = fp8.quantize(fp8.relu2(x.double().numpy()), "e4m3", blocks)
    np.testing.assert_array_equal(exps(m), e)
    np.testing.assert_array_equal(codes(m), c)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("blocks", ["square", "row"])
def test_special_entries(h, fmt, blocks):
    x = torch.zeros(130, 260)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = float("nan"), float("inf"), -float("inf"), 3.0   # amax from finite entries
    x[5, :128] = float("inf")                                                              # no finite entry
    x[128, 200] = 1e-42                                                                    # subnormal amax
    x[129, 256] = 3.3e38
    x[129, 257] = -2.0 ** -126
    m = mb.Fp8Matrix(130, 260, format=fmt, blocks=blocks)
    mb.muon_fp8_quantize(h, [x.cuda()], [m])
    c, e = fp8.quantize(x.double().numpy(), fmt, blocks)
    np.testing.assert_array_equal(exps(m), e)
    np.testing.assert_array_equal(values(m), fp8.dequantize(c, e, fmt, blocks))
    # relu^2: NaN stays, -inf is cut off, +inf stays an infinity
    mb.muon_fp8_quantize(h, [x.cuda()], [m], activation="relu2")
    v = values(m)
    assert np.isnan(v[0, 0]) and v[0, 2] == 0
    assert np.isnan(v[0, 1]) if fmt == "e4m3" else np.isposinf(v[0, 1])


def test_scale_byte_255_reads_as_nan(h):
    m = mb.Fp8Matrix(2, 200)
    m.codes.fill_(0x38)
    m.scales.copy_(torch.tensor([[255, 0]], dtype=torch.uint8))
    out = torch.empty(2, 200, device="cuda")
    mb.muon_fp8_dequantize(h, [m], [out])
    assert out[:, :128].isnan().all() and (out[:, 128:] == 2.0 ** -127).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("blocks", ["square", "row"])
def test_act_backward(h, dtype, blocks):
    """du = 2 sqrt(h) dy: square root and product round once each in float32 (2 * 2^-24
    relative), then into the type: half a step of it, or half an 8-bit step."""
    shapes = [(1, 1), (77, 130), (256, 384)]
    us = [data(r, c, 20 + i, dtype) for i, (r, c) in enumerate(shapes)]
    dys = [1e-3 * data(r, c, 30 + i, dtype).float() for i, (r, c) in enumerate(shapes)]
    dys = [d.to(DT[dtype]) for d in dys]
    saved = [mb.Fp8Matrix(r, c, blocks=blocks) for r, c in shapes]
    mb.muon_fp8_quantize(h, [u.cuda() for u in us], saved, activation="relu2")
    dense = [torch.empty(s, dtype=DT[dtype], device="cuda") for s in shapes]
    mb.muon_fp8_act_backward(h, [d.cuda() for d in dys], saved, dense)
    quant = [mb.Fp8Matrix(r, c, format="e5m2", blocks=blocks) for r, c in shapes]
    mb.muon_fp8_act_backward(h, [d.cuda() for d in dys], saved, quant)
    inplace = [d.cuda() for d in dys]
    mb.muon_fp8_act_backward(h, inplace, saved, inplace)
    eps = torch.finfo(DT[dtype]).eps / 2
    for dy, s, d, q, ip in zip(dys, saved, dense, quant, inplace):
        want = fp8.relu2_backward(dy.double().numpy(), values(s))
        got = d.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= np.abs(want) * (eps + 2.0 ** -22) + 1e-40)
        assert torch.equal(d, ip)
        # 8-bit result: half a step of 2 fraction bits, 2^-3, or half the subnormal step
        scale = np.exp2(fp8.expand(exps(q), *q.shape, blocks))
        assert np.all(np.abs(values(q) - want) <= np.maximum(np.abs(want) * (2.0 ** -3 + 2.0 ** -22),
                                                             scale * 2.0 ** -17 * (1 + 2.0 ** -20)))
    # the identity's gradient is dy
    mb.muon_fp8_act_backward(h, [d.cuda() for d in dys], saved, dense, activation="none")
    for dy, d in zip(dys, dense):
        assert torch.equal(d.cpu(), dy)


def test_act_backward_matches_differences(h):
    """Against central differences of relu(u)^2, at values whose squares the format holds."""
    u = torch.tensor([[0.0, 0.5, 1.0, 2.0, 4.0, -1.0, -4.0, 8.0]]).double()
    m = mb.Fp8Matrix(1, 8)
    mb.muon_fp8_quantize(h, [u.float().cuda()], [m], activation="relu2")
    du = torch.empty(1, 8, device="cuda")
    mb.muon_fp8_act_backward(h, [torch.ones(1, 8, device="cuda")], [m], [du])
    eps = 2.0 ** -20
    num = (torch.relu(u + eps) ** 2 - torch.relu(u - eps) ** 2) / (2 * eps)
    torch.testing.assert_close(du.cpu().double(), num, rtol=0, atol=2 * eps)


def test_strided_rows_and_neighbours_left_alone(h):
    """Column slices with odd pitch and odd offsets; bytes outside rows x cols stay."""
    big = torch.full((70, 333), -7.0, device="cuda")
    x = data(70, 131, 5, "fp32")
    big[:, 3:134] = x.cuda()
    store = torch.full((70, 160), 0xEE, dtype=torch.uint8, device="cuda")
    m = mb.Fp8Matrix(70, 131, codes=store, scales=torch.empty(1, 2, dtype=torch.uint8, device="cuda"))
    mb.muon_fp8_quantize(h, [big[:, 3:134]], [m])
    c, e = fp8.quantize(x.double().numpy())
    np.testing.assert_array_equal(codes(m), c)
    assert (store[:, 131:] == 0xEE).all()
    out = torch.full((70, 201), 9.0, device="cuda", dtype=torch.bfloat16)
    mb.muon_fp8_dequantize(h, [m], [out[:, 7:138]])
    np.testing.assert_array_equal(out[:, 7:138].double().cpu().numpy(), values(m))
    assert (out[:, :7] == 9).all() and (out[:, 138:] == 9).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pitch", [301, 304])
def test_rows_of_every_alignment(h, dtype, pitch):
    """Rows that start at any entry, of widths around every edge, between NaN: the bits of the
    same matrices laid out alone, and nothing beside them written."""
    rows = 70
    widths = (1, 3, 7, 8, 9, 17, 127, 128, 129, 134, 135, 136, 137, 250, 256)
    cases = [(off, c) for off in range(9) for c in widths]
    xs, alone, near = [], [], []
    for i, (off, c) in enumerate(cases):
        base = torch.full((rows, pitch), float("nan"), dtype=DT[dtype], device="cuda")
        base[:, off:off + c] = data(rows, c, i, dtype).cuda()
        xs.append(base)
        near.append(base[:, off:off + c])
        alone.append(torch.zeros(rows, (c + 15) // 16 * 16, dtype=DT[dtype], device="cuda")[:, :c])
        alone[-1].copy_(near[-1])
    ms, refs = [[mb.Fp8Matrix(rows, c) for _, c in cases] for _ in range(2)]
    mb.muon_fp8_quantize(h, near, ms)
    mb.muon_fp8_quantize(h, alone, refs)
    for m, r in zip(ms, refs):
        assert torch.equal(m.codes[:, :m.cols], r.codes[:, :r.cols]) and torch.equal(m.scales, r.scales)
    mb.muon_fp8_act_backward(h, near, ms, near)
    mb.muon_fp8_act_backward(h, alone, refs, alone)
    for a, b in zip(near, alone):
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))      # the root of a negative entry is NaN
    mb.muon_fp8_dequantize(h, ms, near)
    for (off, c), base, m in zip(cases, xs, ms):
        assert torch.equal(base[:, off:off + c].double().cpu(), torch.from_numpy(values(m)))
        assert base[:, :off].isnan().all() and base[:, off + c:].isnan().all()


def test_empty_and_many(h):
    mb.muon_fp8_quantize(h, [], [])
    z = torch.empty(0, 64, device="cuda")
    mb.muon_fp8_quantize(h, [z], [mb.Fp8Matrix(0, 64)])
    mb.muon_fp8_dequantize(h, [mb.Fp8Matrix(5, 0)], [torch.empty(5, 0, device="cuda")])
    # more matrices than one launch takes
    xs = [data(1 + i % 7, 1 + i, i, "bf16") for i in range(200)]
    outs = [mb.Fp8Matrix(*x.shape) for x in xs]
    mb.muon_fp8_quantize(h, [x.cuda() for x in xs], outs)
    assert mb.muon_last_launch_count(h) == 3
    for x, m in zip(xs, outs):
        np.testing.assert_array_equal(codes(m), fp8.quantize(x.double().numpy())[0])


def test_large_offsets(h):
    """A matrix whose last entries lie past 2^31 elements of its base."""
    rows, ld = 70000, 40000                                    # 2.8e9 elements of pitch, few columns
    base = torch.empty(rows * ld // 8, dtype=torch.uint8, device="cuda")   # 350 MB of codes
    m = mb.Fp8Matrix(rows // 8, 130, codes=base.view(rows // 8, ld),
                     scales=torch.empty((rows // 8 + 127) // 128, 2, dtype=torch.uint8, device="cuda"))
    del base
    x = torch.zeros(rows, 24, dtype=torch.bfloat16, device="cuda")
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)      # 5.6 GB
    big[:, :24] = torch.arange(rows, device="cuda")[:, None] % 13
    x.copy_(big[:, :24])
    a, b = mb.Fp8Matrix(rows, 24), mb.Fp8Matrix(rows, 24)
    mb.muon_fp8_quantize(h, [big[:, :24], x], [a, b])
    assert torch.equal(a.codes[:, :24], b.codes[:, :24]) and torch.equal(a.scales, b.scales)
    assert m.c.ld == ld


def test_refusals(h):
    x = torch.zeros(64, 128, device="cuda")
    m = mb.Fp8Matrix(64, 128)

    def refused(match, call):
        with pytest.raises(mb.MuonError, match=match) as ei:
            call()
        assert ei.value.code == mb.MUON_ERR_INVALID_ARG

    refused("shape", lambda: mb.muon_fp8_quantize(h, [x[:63]], [m]))
    refused("shape", lambda: mb.muon_fp8_dequantize(h, [m], [x[:, :64]]))
    refused("overlap", lambda: mb.muon_fp8_quantize(h, [x, x], [m, m]))
    codes8 = torch.zeros(64 * 128 * 4, dtype=torch.uint8, device="cuda")
    over = mb.Fp8Matrix(64, 128, codes=codes8[:64 * 128].view(64, 128), scales=m.scales)
    refused("overlap", lambda: mb.muon_fp8_dequantize(h, [over], [codes8.view(torch.float32).view(64, 128)]))
    bad = mb.Fp8Matrix(64, 128, codes=codes8[1:1 + 64 * 128].view(64, 128), scales=m.scales)
    refused("16-byte", lambda: mb.muon_fp8_quantize(h, [x], [bad]))
    bad = mb.Fp8Matrix(64, 120, codes=codes8[:64 * 120].view(64, 120), scales=m.scales)
    refused("pitch", lambda: mb.muon_fp8_quantize(h, [x[:, :120]], [bad]))
    refused("row pitch", lambda: mb.muon_fp8_quantize(h, [x[:1].expand(64, 128)], [m]))
    pinned = torch.zeros(64, 128).pin_memory()
    raw = mb.muon_dense(pinned.data_ptr(), 64, 128, 128, mb.MUON_F32)
    lib = mb.load_library()
    import ctypes
    assert lib.muon_fp8_quantize(h, ctypes.byref(raw), ctypes.byref(m.c), 1, 0, None) == mb.MUON_ERR_INVALID_ARG
    assert b"device memory" in lib.muon_last_error(h)
    raw = mb.muon_dense(x.data_ptr(), 64, 128, 128, 7)
    assert lib.muon_fp8_quantize(h, ctypes.byref(raw), ctypes.byref(m.c), 1, 0, None) == mb.MUON_ERR_INVALID_ARG
    raw = mb.muon_dense(x.data_ptr(), 64, 128, 128, mb.MUON_F32)
    assert lib.muon_fp8_quantize(h, ctypes.byref(raw), ctypes.byref(m.c), 1, 9, None) == mb.MUON_ERR_INVALID_ARG
    assert lib.muon_fp8_quantize(h, ctypes.byref(raw), None, 1, 0, None) == mb.MUON_ERR_INVALID_ARG
    assert lib.muon_fp8_quantize(h, ctypes.byref(raw), ctypes.byref(m.c), -1, 0, None) == mb.MUON_ERR_INVALID_ARG
    # a gradient needs exactly one destination
    assert lib.muon_fp8_act_backward(h, ctypes.byref(raw), ctypes.byref(m.c), None, None, 1, 1, None) \
        == mb.MUON_ERR_INVALID_ARG
    out = torch.empty(64, 128, device="cuda")
    d = mb.muon_dense(out.data_ptr(), 64, 128, 128, mb.MUON_F32)
    m2 = mb.Fp8Matrix(64, 128)
    assert lib.muon_fp8_act_backward(h, ctypes.byref(raw), ctypes.byref(m.c), ctypes.byref(d), ctypes.byref(m2.c), 1,
                                     1, None) == mb.MUON_ERR_INVALID_ARG
    refused("overlap", lambda: mb.muon_fp8_act_backward(h, [x], [m], [m]))
    # the handle works on
    mb.muon_fp8_quantize(h, [x], [m])
    mb.muon_sync(h)


def test_first_call_can_be_captured_and_streams_may_overlap():
    x = data(300, 500, 8, "bf16").cuda()
    m, back = mb.Fp8Matrix(300, 500), torch.empty(300, 500, dtype=torch.bfloat16, device="cuda")
    handle = mb.muon_init(0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mb.muon_fp8_quantize(handle, [x], [m])
        mb.muon_fp8_dequantize(handle, [m], [back])
    for seed in (8, 9):
        x.copy_(data(300, 500, seed, "bf16"))
        g.replay()
        c, e = fp8.quantize(x.double().cpu().numpy())
        np.testing.assert_array_equal(codes(m), c)
        np.testing.assert_array_equal(back.double().cpu().numpy(), fp8.dequantize(c, e))
    # two streams, one handle
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    xs = [data(1000, 700, i, "bf16").cuda() for i in range(2)]
    ms = [mb.Fp8Matrix(1000, 700) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            mb.muon_fp8_quantize(handle, [xs[i]], [ms[i]], stream=s[i])
    torch.cuda.synchronize()
    for i in range(2):
        np.testing.assert_array_equal(codes(ms[i]), fp8.quantize(xs[i].double().cpu().numpy())[0])
    del g
    mb.muon_destroy(handle)


def test_profile_and_launch_count(h):
    x, m = torch.ones(64, 64, device="cuda"), mb.Fp8Matrix(64, 64)
    mb.muon_fp8_profile_read(h)
    mb.muon_profile_enable(h, True)
    mb.muon_fp8_quantize(h, [x], [m])
    assert mb.muon_last_launch_count(h) == 1
    mb.muon_profile_enable(h, False)
    r = mb.muon_fp8_profile_read(h)
    assert r["quantize"][1] == 1 and r["quantize"][0] > 0 and r["matmul"] == (0.0, 0)
    assert mb.muon_workspace_bytes(h) == 0
