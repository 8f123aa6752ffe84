"""Calls of the 8-bit operators around other work of their handle: captures after an optimizer
step, calls on several streams, lists whose products differ much, and arguments that have to be
refused before anything runs."""
import pytest
import torch

import muon_newton_schulz_06_b200 as mb
from test_fp8_blocks import values
from test_fp8_matmul import operands

pytestmark = pytest.mark.gpu


def step_args(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [torch.randn(256, 384, generator=g, device="cuda").bfloat16()]
    return w, [torch.randn(256, 384, generator=g, device="cuda").bfloat16()], [torch.zeros(256, 384, device="cuda")]


def test_capture_after_an_optimizer_step():
    """The step's status is still to be looked at when the capture begins."""
    opt = mb.Muon(0)
    w, g, m = step_args()
    x8, w8, y = mb.Fp8Matrix(256, 384), mb.Fp8Matrix(256, 384), torch.zeros(256, 256, device="cuda")
    opt.step(w, g, m, lr=0.02)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.fp8_quantize([g[0], w[0]], [x8, w8])
        opt.fp8_matmul([mb.Fp8Product(x8, w8, y, trans_b=True)])
    graph.replay()
    torch.cuda.synchronize()
    want = torch.from_numpy(values(x8)).cuda() @ torch.from_numpy(values(w8)).cuda().t()
    assert (y.double() - want).abs().max() <= 1e-5 * want.abs().max()
    mb.muon_sync(opt.handle)
    del graph
    opt.close()


def test_step_captured_after_a_step():
    w, g, m = step_args()
    opt, ref = mb.Muon(0), mb.Muon(0)
    rw, rm = [w[0].clone()], [m[0].clone()]
    for _ in range(2):
        ref.step(rw, g, rm, lr=0.02)
    mb.muon_sync(ref.handle)
    opt.step(w, g, m, lr=0.02)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(w, g, m, lr=0.02)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w[0], rw[0]) and torch.equal(m[0], rm[0])
    del graph
    opt.close()
    ref.close()


def test_time_out_of_a_step_is_kept_through_a_capture():
    opt = mb.Muon(0)
    x8, x = mb.Fp8Matrix(64, 64), torch.ones(64, 64, device="cuda")
    mb.muon_selftest_wait_timeout(opt.handle, 1_000_000)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.fp8_quantize([x], [x8])
    with pytest.raises(mb.MuonError) as ei:
        mb.muon_sync(opt.handle)
    assert ei.value.code == mb.MUON_ERR_TIMEOUT
    graph.replay()
    mb.muon_sync(opt.handle)
    torch.cuda.synchronize()
    assert (values(x8) == 1).all()
    del graph
    opt.close()


def slow_then_quick(opt):
    """A wait of half a second that runs out on one stream, then a call on another one."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    x, x8 = torch.ones(64, 64, device="cuda"), mb.Fp8Matrix(64, 64)
    opt.fp8_quantize([x], [x8])
    torch.cuda.synchronize()
    mb.muon_selftest_fp8_timeout(opt.handle, 500_000_000, stream=a)
    opt.fp8_quantize([x], [x8], stream=b)
    return a, b, x, x8


def test_sync_waits_for_every_stream():
    opt = mb.Muon(0)
    keep = slow_then_quick(opt)
    try:
        with pytest.raises(mb.MuonError) as ei:
            mb.muon_sync(opt.handle)
        assert ei.value.code == mb.MUON_ERR_TIMEOUT
    finally:
        torch.cuda.synchronize()
    # many streams, used in turn, some of them gone
    x, outs = keep[2], [mb.Fp8Matrix(64, 64) for _ in range(40)]
    for o in outs:
        opt.fp8_quantize([x], [o], stream=torch.cuda.Stream())
    mb.muon_sync(opt.handle)
    assert all((values(o) == 1).all() for o in outs)
    opt.close()


def test_destroy_waits_for_every_stream():
    opt = mb.Muon(0)
    keep = slow_then_quick(opt)
    with pytest.raises(mb.MuonError) as ei:
        mb.muon_destroy(opt.handle)
    opt.handle = None
    assert ei.value.code == mb.MUON_ERR_TIMEOUT
    torch.cuda.synchronize()
    del keep


def test_too_many_tiles_are_refused_before_the_first_launch():
    """Sixteen products that fit one launch, then one whose result has more tiles than a launch can
    count (a product of nothing: only its result has an address; it is never written)."""
    h = mb.muon_init(0)
    a, b, va, vb = operands(8, 16, 32, False, True, seed=1)
    arena = torch.full((17, 8, 16), 7.0, device="cuda")
    raw = (mb.muon_fp8_product * 17)()
    for i in range(16):
        raw[i].a, raw[i].b, raw[i].trans_b = a.c, b.c, 1
        raw[i].d = mb.muon_dense(arena[i].data_ptr(), 8, 16, 16, mb.MUON_F32)
    # the highest address of the call, so that its span holds no other buffer
    rows, cols = 1 << 18, 1 << 24
    top = max((t for t in (arena, torch.empty(1 << 20, device="cuda"), torch.empty(1 << 26, device="cuda"))),
              key=lambda t: t.data_ptr())
    raw[16].a.rows, raw[16].b.rows, raw[16].trans_b = rows, cols, 1
    raw[16].d = mb.muon_dense(arena[16].data_ptr() if top is arena else top.data_ptr(), rows, cols, cols, mb.MUON_BF16)
    if max(a.c.codes, b.c.codes, a.c.scales, b.c.scales) > raw[16].d.data:
        pytest.skip("the operands lie above every other buffer")
    lib = mb.load_library()
    st = torch.cuda.current_stream().cuda_stream
    assert lib.muon_fp8_matmul(h, raw, 17, st) == mb.MUON_ERR_UNSUPPORTED
    assert b"tiles" in lib.muon_last_error(h)
    torch.cuda.synchronize()
    assert (arena == 7).all()
    assert lib.muon_fp8_matmul(h, raw, 16, st) == mb.MUON_OK
    want = (torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda()).float()
    assert all(torch.equal(arena[i], want) for i in range(16))
    mb.muon_destroy(h)


def test_empty_contraction_beside_a_large_product():
    """A weight gradient over no tokens in the list of a large one: a launch of its own, and the
    large one keeps the launch that it has alone."""
    h = mb.muon_init(0)
    a, b, va, vb = operands(2560, 2304, 640, False, True, seed=2)
    e, f = mb.Fp8Matrix(300, 0), mb.Fp8Matrix(200, 0)
    d, alone = torch.empty(2560, 2304, device="cuda"), torch.empty(2560, 2304, device="cuda")
    z, c = torch.full((300, 200), 3.0, device="cuda"), torch.randn(300, 200, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(e, f, z, trans_b=True, add=c), mb.Fp8Product(a, b, d, trans_b=True)])
    assert mb.muon_last_launch_count(h) == 2
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, alone, trans_b=True)])
    assert mb.muon_last_launch_count(h) == 1
    assert torch.equal(z, c) and torch.equal(d, alone)
    assert torch.equal(d.double(), torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda())
    mb.muon_destroy(h)


@pytest.mark.parametrize("K", [640, 1920, 2176, 8000])
def test_short_contraction_beside_a_long_one(K):
    """164 tiles of 128 x 128 whose mean contraction lies on either side of the rule between two CTAs
    per SM and pairs."""
    h = mb.muon_init(0)
    a, b, va, vb = operands(1280, 1280, K, False, True, seed=K)
    s, t, vs, vt = operands(1000, 1024, 100, True, False, seed=1)
    d, e = (torch.empty(n, n2, device="cuda", dtype=torch.bfloat16) for n, n2 in ((1280, 1280), (1000, 1024)))
    mb.muon_fp8_matmul(h, [mb.Fp8Product(s, t, e, trans_a=True), mb.Fp8Product(a, b, d, trans_b=True)])
    assert mb.muon_last_launch_count(h) == 1
    for out, x, y in ((d, va, vb), (e, vs, vt)):
        assert torch.equal(out, (torch.from_numpy(x).cuda() @ torch.from_numpy(y).cuda()).bfloat16())
    mb.muon_destroy(h)


def test_addend_without_entries_is_refused():
    h = mb.muon_init(0)
    a, b, _, _ = operands(64, 96, 128, False, True)
    d = torch.full((64, 96), 7.0, device="cuda")
    for shape in ((0, 96), (64, 0), (0, 0)):
        with pytest.raises(mb.MuonError, match="c is") as ei:
            mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True, add=torch.empty(*shape, device="cuda"))])
        assert ei.value.code == mb.MUON_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (d == 7).all()
    # a result without entries takes one
    mb.muon_fp8_matmul(h, [mb.Fp8Product(mb.Fp8Matrix(0, 128), b, torch.empty(0, 96, device="cuda"), trans_b=True,
                                         add=torch.empty(0, 96, device="cuda"))])
    mb.muon_destroy(h)


def test_step_refuses_copies_that_overlap_before_stepping():
    opt = mb.Muon(0)
    ws = [torch.ones(64, 64, device="cuda") for _ in range(2)]
    gs, ms = [torch.ones_like(w) for w in ws], [torch.zeros_like(w) for w in ws]

    def refused(copies, params=ws):
        with pytest.raises(ValueError, match="overlap"):
            opt.step(params, gs[:len(params)], ms[:len(params)], lr=0.1, fp8_params=copies)
        torch.cuda.synchronize()
        assert all((w == 1).all() for w in ws) and all((m == 0).all() for m in ms)

    buf = torch.zeros(200, 64, dtype=torch.uint8, device="cuda")
    sc = [torch.zeros(1, 1, dtype=torch.uint8, device="cuda") for _ in range(2)]
    part = [mb.Fp8Matrix(64, 64, codes=buf[o:o + 64], scales=s) for o, s in zip((0, 32), sc)]
    refused(part)                                                             # codes
    refused([mb.Fp8Matrix(64, 64, codes=buf[o:o + 64], scales=sc[0]) for o in (0, 64)])    # one scale for two
    refused([mb.Fp8Matrix(64, 64, codes=buf[:64], scales=buf[2:3, :1])], ws[:1])            # scales in the codes
    over = ws[0].view(-1).view(torch.uint8)[:64 * 64].view(64, 64)
    refused([mb.Fp8Matrix(64, 64, codes=over, scales=sc[0])], ws[:1])         # over the weight
    # column slices of one buffer lie beside each other
    both = torch.zeros(64, 128, dtype=torch.uint8, device="cuda")
    ok = [mb.Fp8Matrix(64, 64, codes=both[:, o:o + 64], scales=s) for o, s in zip((0, 64), sc)]
    opt.step(ws, gs, ms, lr=0.1, fp8_params=ok)
    mb.muon_sync(opt.handle)
    ref = [mb.Fp8Matrix(64, 64) for _ in ws]
    opt.fp8_quantize(ws, ref)
    mb.muon_sync(opt.handle)
    for o, r in zip(ok, ref):
        assert torch.equal(o.codes, r.codes) and torch.equal(o.scales, r.scales)
    opt.close()


def test_single_rows_beside_column_slices():
    """One row of a tensor lies beside other columns of all its rows, and scales in the padding
    behind the codes."""
    opt = mb.Muon(0)
    big = torch.randn(20, 96, device="cuda")
    m = mb.Fp8Matrix(20, 32)
    one = mb.Fp8Matrix(1, 32)
    opt.fp8_quantize([big[:, 32:64]], [m])
    opt.fp8_quantize([big[7:8, 64:]], [one])
    want, keep = (torch.from_numpy(values(x)).float().cuda() for x in (m, one)), big.clone()
    opt.fp8_dequantize([m, one], [big[:, :32], big[7:8, 64:]])
    mb.muon_sync(opt.handle)
    keep[:, :32], keep[7:8, 64:] = want
    assert torch.equal(big, keep)
    with pytest.raises(mb.MuonError, match="overlap"):
        opt.fp8_dequantize([m, one], [big[:, :32], big[7:8, 31:63]])
    buf = torch.zeros(64, 80, dtype=torch.uint8, device="cuda")
    packed = mb.Fp8Matrix(64, 64, codes=buf[:, :64], scales=buf[5:6, 64:65])
    w, g, mo = torch.randn(64, 64, device="cuda"), torch.randn(64, 64, device="cuda"), torch.zeros(64, 64, device="cuda")
    opt.step([w], [g], [mo], lr=0.1, fp8_params=[packed])
    ref = mb.Fp8Matrix(64, 64)
    opt.fp8_quantize([w], [ref])
    mb.muon_sync(opt.handle)
    assert torch.equal(packed.codes[:, :64], ref.codes) and torch.equal(packed.scales, ref.scales)
    opt.close()
