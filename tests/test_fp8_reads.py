"""The 8-bit operators read nothing outside their buffers. On the CPU: the scale loader of row
blocks, compiled for the host with its reads recorded, over every alignment, and the matrices'
ends. On the GPU: operands in buffers that end with their last entry."""
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "fp8_internal.h"
int main() {
  std::vector<unsigned char> mem(4096);
  for (size_t i = 0; i < mem.size(); ++i) mem[i] = (unsigned char)(i * 37 + 11);
  long reads = 0;
  for (int base = 64; base < 68; ++base)
    for (int rows = 128; rows < 140; ++rows)
      for (int nkb = 1; nkb < 4; ++nkb) {
        const uintptr_t lo = base, hi = base + rows * nkb;
        bool in = true;
        auto check = [&](uintptr_t a, int n) { in = in && a >= lo && a + n <= hi && a % n == 0; ++reads; };
        for (int kb = 0; kb < nkb; ++kb)
          for (int r = 0; r + 4 <= rows; r += 4) {
            const uintptr_t at = lo + (uintptr_t)kb * rows + r;
            const uint32_t got = muon::f8_read4(
                at, lo, hi,
                [&](uintptr_t a) {
                  check(a, 4);
                  return (uint32_t)mem[a] | (uint32_t)mem[a + 1] << 8 | (uint32_t)mem[a + 2] << 16 | (uint32_t)mem[a + 3] << 24;
                },
                [&](uintptr_t a) { check(a, 1); return (uint32_t)mem[a]; });
            for (int j = 0; j < 4; ++j)
              if (((got >> (8 * j)) & 255u) != mem[at + j]) { printf("value %d %d %d %d\n", base, rows, kb, r); return 1; }
            if (!in) { printf("outside %d %d %d %d\n", base, rows, kb, r); return 1; }
          }
      }
  printf("reads %ld\n", reads);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="the loader's header needs the CUDA headers")
def test_scale_words_stay_inside_the_scales(tmp_path):
    src, exe = tmp_path / "reads.cpp", tmp_path / "reads"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(shutil.which("nvcc")))), "include")
    csrc = os.path.join(ROOT, "muon_newton_schulz_06_b200", "csrc")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-w", "-I", cuda, "-I", csrc, "-o", str(exe), str(src)],
                   check=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "reads" in r.stdout, r.stdout


def tight(m, lead):
    """m with codes and scales in one buffer that ends with the scales' last byte; the scales
    start `lead` bytes past a multiple of 16."""
    import muon_newton_schulz_06_b200 as mb
    ld = m.codes.stride(0)
    n_codes, n = m.rows * ld, m.scales.numel()
    buf = torch.full((n_codes + lead + n,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN scales and codes around
    codes, scales = buf[:n_codes].view(m.rows, ld), buf[n_codes + lead:].view(m.scales.shape)
    codes[:, :m.cols] = m.codes[:, :m.cols]
    scales.copy_(m.scales)
    return mb.Fp8Matrix(m.rows, m.cols, format=m.format, blocks=m.blocks, codes=codes, scales=scales)


@pytest.mark.gpu
@pytest.mark.parametrize("lead", [0, 1, 2, 3])
@pytest.mark.parametrize("M,N,K", [(129, 257, 256), (128, 128, 128), (131, 130, 600), (2437, 2305, 200)])
def test_row_scales_at_any_address(M, N, K, lead):
    import muon_newton_schulz_06_b200 as mb
    from test_fp8_matmul import operands
    h = mb.muon_init(0)
    a, b, va, vb = operands(M, N, K, False, True, ba="row", bb="row", seed=M)
    d = torch.empty(M, N, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(tight(a, lead), tight(b, lead), d, trans_b=True)])
    mb.muon_sync(h)
    assert torch.equal(d.double(), torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda())
    mb.muon_destroy(h)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2305, 2319, 2177])
def test_checkpoint_that_ends_with_its_last_entry(N):
    """The slope epilogue into dense results, many tiles: the last row's codes are the last bytes
    of their buffer."""
    import muon_newton_schulz_06_b200 as mb
    from oracle import fp8
    from test_fp8_blocks import values
    from test_fp8_matmul import operands, roots
    h = mb.muon_init(0)
    M, K, ld = 2437, 200, (N + 15) // 16 * 16
    a, b, va, vb = operands(M, N, K, False, True, seed=N)
    whole = roots(M, N, "e4m3", "square", 3)
    buf = torch.empty((M - 1) * ld + N, dtype=torch.uint8, device="cuda")
    codes = buf.as_strided((M, N), (ld, 1))
    codes.copy_(whole.codes[:, :N])
    saved = mb.Fp8Matrix(M, N, codes=codes, scales=whole.scales)
    d = torch.empty(M, N, device="cuda")
    mb.muon_fp8_matmul(h, [mb.Fp8Product(a, b, d, trans_b=True, epilogue="relu2_backward", saved=saved)])
    mb.muon_sync(h)
    want = torch.from_numpy(fp8.relu2_backward(va @ vb, values(whole)))
    assert torch.equal(d.double().cpu(), want.float().double())
    mb.muon_destroy(h)
