"""A wait of the many-token MX4 product that runs out: the block that misses its codes reports it, stores nothing of its
tile and lets its cluster store nothing of it, the other blocks' tiles are right, and the context stays usable."""
import pytest
import torch

import orthogonal_equivalence_cnp_b200 as P
from helpers import device_clean

pytestmark = pytest.mark.gpu


def _problem(n, d_in, d_out, adjoint, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randint(-2, 3, (n, d_out if adjoint else d_in), device="cuda", generator=g).to(torch.bfloat16)
    codes = torch.randint(0, 256, (d_out, d_in // 2), device="cuda", generator=g).to(torch.uint8)
    scales = torch.full((d_out, d_in // 32), 127, dtype=torch.uint8, device="cuda")
    lut = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    c = torch.stack([codes & 15, codes >> 4], 2).view(d_out, -1)
    W = torch.cat([lut, -lut])[c.long()]
    return X, codes, scales, (X.double() @ (W if adjoint else W.t())).to(torch.bfloat16)


# Small integers: every sum is exact, so a tile is right or it is not.  The shapes take 128 and 256 features a tile, K
# whole and split over a cluster.
@pytest.mark.parametrize("adjoint", [0, 1])
@pytest.mark.parametrize("n,d_in,d_out,features,split", [(1500, 2048, 2048, 256, False), (300, 1056, 1024, 128, False),
                                                         (64, 4096, 4096, 128, True), (700, 4096, 4096, 256, True)])
@pytest.mark.parametrize("steps", [0, 2])
def test_a_block_that_gives_up_stores_nothing(adjoint, n, d_in, d_out, features, split, steps):
    X, codes, scales, ref = _problem(n, d_in, d_out, adjoint, n)
    guard = 32768.0  # sixty times the spread of the results
    assert not (ref == guard).any().item()
    Y = torch.full_like(ref, guard)
    splits = P.poetx_test_mx4_give_up(adjoint, n, d_in, d_out, X, codes, scales, Y, steps, 5_000_000)
    st, detail = P.poetx_device_status()
    assert (splits > 1) == split
    assert P.STATUS[st] == "POETX_ERR_DEVICE_TIMEOUT" and detail >> 8 == 9, (st, hex(detail))
    # The first tile (features from 0 on, the first tokens) is left as it was; all else is right.
    left = Y == guard
    tokens = int(left[:, 0].sum())
    assert 0 < tokens <= min(n, 256)
    tile = torch.zeros_like(left)
    tile[:tokens, :features] = True
    assert torch.equal(left, tile) and torch.equal(Y[~tile], ref[~tile])
    # The same product right afterwards, on the same memory.
    P.poetx_mx4_matmul(adjoint, n, d_in, d_out, X, codes, scales, Y)
    torch.cuda.synchronize()
    device_clean()
    assert torch.equal(Y, ref)
