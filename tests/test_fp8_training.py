"""The 8-bit operators as a training step uses them, around the optimizer step: forward and
backward pass of a relu^2 MLP, gradients into Muon, weights quantised again.

Every stage is checked against the float64 oracle from the 8-bit matrices that the stage
itself read, so no bound grows from stage to stage.  A product's accumulation error is taken
as in test_fp8_matmul.py (ceil(K / 32) + 12 additions, 2^-22 of the sum of magnitudes each)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import muon_newton_schulz_06_b200 as mb
from oracle import fp8
from test_fp8_blocks import codes, exps, values

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def acc(K):
    return (-(-K // 32) + 12) * 2.0 ** -22


def check_dense(t, a, b):
    want, mag = fp8.matmul(a, b)
    tol = acc(a.shape[1]) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)      # bf16: half a step
    assert np.all(np.abs(t.double().cpu().numpy() - want) <= tol)


def check_codes(m, want, err):
    """want +- err (elementwise, before the rounding) in 8 bits: half an e4m3 step more."""
    v = values(m)
    scale = np.exp2(fp8.expand(exps(m), m.rows, m.cols, m.blocks))
    tol = err + np.maximum((np.abs(want) + err) * 2.0 ** -4, scale * 2.0 ** -10)
    assert np.all(np.abs(v - want) <= tol)
    # the scale fits: codes use the format's top octave (above 448 / 2) unless the block is empty
    step = 128
    for i in range(0, m.rows, step):
        for j in range(0, m.cols, step):
            top = np.abs(v[i:i + step, j:j + step] / scale[i:i + step, j:j + step]).max()
            assert top == 0 or 224 <= top <= 448


@pytest.mark.parametrize("tokens,d,hidden", [(1, 64, 100), (300, 130, 520), (1024, 256, 1024)])
def test_mlp_step(tokens, d, hidden):
    gen = torch.Generator().manual_seed(tokens)
    w1 = (0.05 * torch.randn(hidden, d, generator=gen)).bfloat16().cuda()
    w2 = (0.05 * torch.randn(d, hidden, generator=gen)).bfloat16().cuda()
    x = torch.randn(tokens, d, generator=gen).bfloat16().cuda()
    dy = (1e-3 * torch.randn(tokens, d, generator=gen)).bfloat16().cuda()
    opt = mb.Muon(0)
    w1_8, w2_8 = mb.Fp8Matrix(hidden, d), mb.Fp8Matrix(d, hidden)
    x8, h8, dy8, du8 = (mb.Fp8Matrix(tokens, c) for c in (d, hidden, d, hidden))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw1, dw2 = torch.empty_like(w1), torch.empty_like(w2)
    opt.fp8_quantize([w1, w2], [w1_8, w2_8])

    def fwd_bwd():
        opt.fp8_quantize([x], [x8])
        opt.fp8_matmul([mb.Fp8Product(x8, w1_8, h8, trans_b=True, epilogue="relu2")])
        opt.fp8_matmul([mb.Fp8Product(h8, w2_8, y, trans_b=True)])
        opt.fp8_quantize([dy], [dy8])
        opt.fp8_matmul([mb.Fp8Product(dy8, w2_8, du8, epilogue="relu2_backward", saved=h8)])
        opt.fp8_matmul([mb.Fp8Product(dy8, h8, dw2, trans_a=True), mb.Fp8Product(du8, x8, dw1, trans_a=True)])
        opt.fp8_matmul([mb.Fp8Product(du8, w1_8, dx)])

    fwd_bwd()
    mb.muon_sync(opt.handle)
    for m, t in ((x8, x), (dy8, dy), (w1_8, w1), (w2_8, w2)):
        c, e = fp8.quantize(t.double().cpu().numpy())
        np.testing.assert_array_equal(codes(m), c)
        np.testing.assert_array_equal(exps(m), e)
    X, DY, W1, W2, H, DU = (values(m) for m in (x8, dy8, w1_8, w2_8, h8, du8))
    # h = relu(u)^2: an error of du_ in u moves it by (2 |u| + du_) du_, and rounding by 2^-24
    u, mag = fp8.matmul(X, W1.T)
    eu = acc(d) * mag
    check_codes(h8, fp8.relu2(u), (2 * np.abs(u) + eu) * eu + 2.0 ** -23 * u * u)
    g, mag = fp8.matmul(DY, W2)
    slope = 2 * np.sqrt(H)
    check_codes(du8, slope * g, slope * acc(d) * mag + 2.0 ** -22 * np.abs(slope * g))
    check_dense(y, H, W2.T)
    check_dense(dw2, DY.T, H)
    check_dense(dw1, DU.T, X)
    check_dense(dx, DU, W1)

    # the same pass captured into a graph, while the eager results live
    eager = [t.clone() for t in (y, dx, dw1, dw2)]
    g_ = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g_):
        fwd_bwd()
    for t in (y, dx, dw1, dw2):
        t.zero_()
    g_.replay()
    for t, e in zip((y, dx, dw1, dw2), eager):
        assert torch.equal(t, e)

    # the optimizer step takes the gradients; its 8-bit copies are those of the new weights
    ref, refm = [w1.clone(), w2.clone()], [torch.zeros(w.shape, device="cuda") for w in (w1, w2)]
    hd = mb.muon_init(0)
    mb.muon_step_ex(hd, ref, [dw1, dw2], refm, lr=0.02)
    mb.muon_sync(hd)
    mb.muon_destroy(hd)
    moms = [torch.zeros(w.shape, device="cuda") for w in (w1, w2)]
    opt.step([w1, w2], [dw1, dw2], moms, lr=0.02, fp8_params=[w1_8, w2_8])
    mb.muon_sync(opt.handle)
    for w, r, m in zip((w1, w2), ref, (w1_8, w2_8)):
        assert torch.equal(w, r)
        c, e = fp8.quantize(w.double().cpu().numpy())
        np.testing.assert_array_equal(codes(m), c)
        np.testing.assert_array_equal(exps(m), e)
    del g_
    opt.close()


def test_gradient_matches_differences():
    """dW of sum(y * r) through the 8-bit products against central differences of the same
    function of W, on operands that 8 bits hold exactly (the products are linear in W, so the
    differences are exact up to the float32 results)."""
    opt = mb.Muon(0)
    rng = np.random.default_rng(0)
    T, K, N = 37, 24, 19
    x = torch.from_numpy(rng.integers(-4, 5, (T, K))).float().cuda()
    w = torch.from_numpy(rng.integers(-4, 5, (N, K))).float().cuda()
    r = torch.from_numpy(rng.integers(-4, 5, (T, N))).float().cuda()
    x8, w8, r8 = mb.Fp8Matrix(T, K), mb.Fp8Matrix(N, K), mb.Fp8Matrix(T, N)
    opt.fp8_quantize([x, r], [x8, r8])

    def loss(wv):
        y = torch.empty(T, N, device="cuda")
        opt.fp8_quantize([wv], [w8])
        opt.fp8_matmul([mb.Fp8Product(x8, w8, y, trans_b=True)])
        return (y * r).double().sum().item()

    dw, dx = torch.empty(N, K, device="cuda"), torch.empty(T, K, device="cuda")
    opt.fp8_matmul([mb.Fp8Product(r8, x8, dw, trans_a=True)])
    opt.fp8_quantize([w], [w8])
    opt.fp8_matmul([mb.Fp8Product(r8, w8, dx)])
    for i, j in [(0, 0), (3, 7), (18, 23), (11, 2)]:
        up, dn = w.clone(), w.clone()
        up[i, j] += 1.0
        dn[i, j] -= 1.0
        assert (loss(up) - loss(dn)) / 2 == dw[i, j].item()
    torch.testing.assert_close(dx, r @ w, rtol=0, atol=0)
    opt.close()


def test_first_calls_of_a_process_can_be_captured():
    """Kernels that were never launched, and the handle's set-up, inside a capture."""
    code = """
import torch, muon_newton_schulz_06_b200 as mb
x = torch.randn(300, 256, device="cuda")
w = torch.randn(200, 256, device="cuda")
big = torch.randn(3000, 256, device="cuda")
y = torch.empty(300, 200, device="cuda")
z = torch.empty(3000, 3000, device="cuda", dtype=torch.bfloat16)
x8, w8, b8 = (mb.Fp8Matrix(*t.shape) for t in (x, w, big))
d = torch.empty(300, 256, device="cuda")
g = torch.cuda.CUDAGraph()
m = mb.Muon(0)
with torch.cuda.graph(g):
    m.fp8_quantize([x, w, big], [x8, w8, b8], activation="relu2")
    m.fp8_act_backward([x], [x8], [d])
    m.fp8_matmul([mb.Fp8Product(x8, w8, y, trans_b=True)])
    m.fp8_matmul([mb.Fp8Product(b8, b8, z, trans_b=True)])
g.replay()
torch.cuda.synchronize()
mb.muon_sync(m.handle)
a, b = (torch.empty_like(t) for t in (x, w))
m.fp8_dequantize([x8, w8], [a, b])
ref = a.double() @ b.double().t()
assert (y.double() - ref).abs().max() <= 1e-5 * ref.abs().max()
assert torch.equal(z, z.t()) and z.float().abs().sum() > 0
print("captured", flush=True)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_time_out_is_reported_and_cleared():
    opt = mb.Muon(0)
    mb.muon_selftest_fp8_timeout(opt.handle, 1_000_000)
    with pytest.raises(mb.MuonError, match="8-bit") as ei:
        mb.muon_sync(opt.handle)
    assert ei.value.code == mb.MUON_ERR_TIMEOUT
    mb.muon_sync(opt.handle)
    # a later call reports it too, before it enqueues anything; then the handle works on
    x, m = torch.ones(64, 64, device="cuda"), mb.Fp8Matrix(64, 64)
    m.codes.fill_(1)
    mb.muon_selftest_fp8_timeout(opt.handle, 1_000_000)
    torch.cuda.synchronize()
    with pytest.raises(mb.MuonError) as ei:
        opt.fp8_quantize([x], [m])
    assert ei.value.code == mb.MUON_ERR_TIMEOUT
    assert (m.codes == 1).all()
    opt.fp8_quantize([x], [m])
    assert (values(m) == 1).all()
    with pytest.raises(mb.MuonError):
        mb.muon_selftest_fp8_timeout(opt.handle, -1)
    opt.close()


def test_step_refuses_bad_copies_before_stepping():
    opt = mb.Muon(0)
    w = torch.ones(64, 64, device="cuda")
    g, m = torch.ones_like(w), torch.zeros_like(w)
    with pytest.raises(ValueError, match="fp8_params"):
        opt.step([w], [g], [m], lr=0.1, fp8_params=[])
    with pytest.raises(ValueError, match="fp8_params"):
        opt.step([w], [g], [m], lr=0.1, fp8_params=[mb.Fp8Matrix(64, 65)])
    with pytest.raises(TypeError, match="Fp8Matrix"):
        opt.step([w], [g], [m], lr=0.1, fp8_params=[w])
    w8 = mb.Fp8Matrix(64, 64)
    with pytest.raises(ValueError, match="twice"):
        opt.step([w, w.clone()], [g, g.clone()], [m, m.clone()], lr=0.1, fp8_params=[w8, w8])
    odd = torch.zeros(64 * 64 + 8, dtype=torch.uint8, device="cuda")[8:].view(64, 64)
    with pytest.raises(ValueError, match="aligned"):
        opt.step([w], [g], [m], lr=0.1, fp8_params=[mb.Fp8Matrix(64, 64, codes=odd, scales=w8.scales)])
    assert (w == 1).all() and (m == 0).all()
    opt.close()
