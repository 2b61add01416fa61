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
