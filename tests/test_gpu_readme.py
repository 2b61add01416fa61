"""The README's Python lines do what the README says of them."""
import os
import re

import numpy as np
import pytest
import torch

import orthogonal_equivalence_cnp_b200 as P
import poetx_inputs as I
from helpers import device_clean, rel, to_np

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _blocks():
    """The indented blocks of the README's section on Python."""
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    text = re.search(r"^## Using the layer from Python\n(.*?)(?=^## |\Z)", text, re.S | re.M).group(1)
    return [re.sub(r"^    ", "", b, flags=re.M) for b in re.findall(r"(?:^    .*\n|^\n(?=    ))+", text, re.M)]


def test_readme_blocks():
    blocks = [b for b in _blocks() if b.strip()]
    assert len(blocks) == 3
    s = I.small_shape(4096, 4096, 256, 3, 2048, "bf16", "mem", theta_std=0.005, w_std=0.02)
    inp = I.make_layer(s, 12)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.bfloat16)
    x = dev(inp.X[:5])
    y = torch.empty(5, 4096, dtype=torch.bfloat16, device="cuda")
    env = dict(W0=inp.W0, theta_R=inp.theta_R, theta_P=inp.theta_P, pi_L=inp.pi_L, pi_R=inp.pi_R, X=dev(inp.X), dY=dev(inp.dY),
               cfg=P.poetx_adamw_cfg(1e-4, 0.5, 0.9, 0.999, 1e-8, 0.0), step=1, n=5, x=x, y=y)
    exec(blocks[0], env)
    exec(blocks[1], env)
    L = env["L"]
    L.cnp()
    L.forward(env["X"])  # the layer before it is merged
    trained, pL, pR = L.Y[:5].clone(), L.perm_L.long(), L.perm_R.long()
    exec(blocks[2], env)
    torch.cuda.synchronize()
    device_clean()
    # The merged layer: theta is zero, its factors are the identity, so one rounding separates the two at most.
    L.cnp()
    L.forward(env["X"])
    assert rel(to_np(y), to_np(L.Y[:5])) <= 2.0 ** -8
    # And the layer as it was trained, but for the new quantisation: of a weight with normal values MX4 is off by under 0.15 of
    # its norm (a step of 1/2 at values up to 2, of 1 up to 4, 2 up to 6 scales, a twelfth of its square in the mean), an
    # independent error per weight, against both the old codes and the product.
    assert rel(to_np(y), to_np(trained)) <= 0.15
    # Other permutations, as the README's last line has them.
    perm = lambda k: torch.from_numpy(np.random.default_rng(k).permutation(4096).astype(np.int32)).cuda()
    L.merge(perm(1), perm(2))
    z = torch.empty_like(y)
    P.poetx_mx4_matmul(0, 5, 4096, 4096, x[:, L.perm_R.long()].contiguous(), L.W0q, L.W0s, z)
    L.cnp()
    L.forward(env["X"])
    y[:, L.perm_L.long()] = z
    assert rel(to_np(y), to_np(L.Y[:5])) <= 2.0 ** -8
