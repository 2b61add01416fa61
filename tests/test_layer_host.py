"""PoetxLayer's own checks and buffers, on the CPU (nothing is launched)."""
import pytest
import torch

import orthogonal_equivalence_cnp_b200 as P
from orthogonal_equivalence_cnp_b200.layer import PoetxLayer, make_desc


def _layer(mode="mem", **kw):
    return PoetxLayer(make_desc(256, 512, 64, 3, "bf16", mode), 8, device="cpu", **kw)


def test_four_permutation_comparator_needs_the_weight_that_quantize_releases():
    L = _layer()
    with pytest.raises(ValueError, match="un-absorbed"):
        L.fourperm_step(L.dX, L.Y)


def test_a_quantised_layer_takes_no_new_state():
    # Refused before anything is overwritten.
    L = _layer()
    L.mx4, L.W0p = True, None  # as quantize() leaves it
    n, k = 512 // 64, 256 // 64
    with pytest.raises(ValueError, match="quantised"):
        L.load_state(torch.zeros(512, 256).numpy(), torch.ones(n, 2016).numpy(), torch.ones(k, 2016).numpy(),
                     torch.arange(511, -1, -1).numpy(), torch.arange(255, -1, -1).numpy())
    assert not L.theta.any() and torch.equal(L.perm_L, torch.arange(512, dtype=torch.int32))


def test_moments_of_a_layer():
    with pytest.raises(ValueError, match="moments"):
        _layer(moments="int8")
    L = _layer()
    assert L.m.shape == L.theta.shape and L.v.shape == L.theta.shape and L.optimizer is None
    L = _layer(moments=None)
    assert L.m is None and L.v is None and L.optimizer is None
    with pytest.raises(ValueError, match="no moments"):
        L.optimizer_step(P.poetx_adamw_cfg(1e-4, 0.5, 0.9, 0.999, 1e-8, 0.0))
    assert L.t == 0


def test_workspace_from_outside():
    d = make_desc(256, 512, 64, 3, "bf16", "mem")
    need = PoetxLayer.workspace_bytes(d, 8)
    assert need == max(P.poetx_workspace_size(d, 8), 256) and _layer().ws.numel() == need
    ws = torch.empty(need + 64, dtype=torch.uint8)
    assert _layer(workspace=ws).ws is ws
    for bad in (torch.empty(need - 1, dtype=torch.uint8), torch.empty(need), torch.empty(2 * need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            _layer(workspace=bad)
    with pytest.raises(ValueError, match="is on"):
        _layer(workspace=torch.empty(need, dtype=torch.uint8, device="meta"))
