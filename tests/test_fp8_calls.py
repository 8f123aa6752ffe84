"""Calls of the 8-bit operators around other work of their handle: captures after an optimizer
step, calls on several streams, lists whose products differ much, and arguments that have to be
refused before anything runs."""
import pytest
import torch

import muon_newton_schulz_06_b200 as mb
from test_fp8_matmul import operands

pytestmark = pytest.mark.gpu


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
