"""Waits of the tcgen05 products that run out: the block that misses a tile (or its block factor's Q) reports it and stores
nothing that it has not computed, the other blocks' tiles are right, and the context stays usable."""
import pytest
import torch

import orthogonal_equivalence_cnp_b200 as P
from helpers import device_clean

pytestmark = pytest.mark.gpu

M, N, K = 600, 512, 512
GUARD = 32768.0  # beyond every result: |D| <= K, |out2| <= 256 * 60 in practice


# Factors of -1, 0, 1 and scales of 2: every sum is exact in fp32, so a tile is right or it is not.
def _problem(kind):
    g = torch.Generator(device="cuda").manual_seed(kind)
    ints = lambda *shape: torch.randint(-1, 2, shape, device="cuda", generator=g)
    a, b, q = ints(M, K).to(torch.bfloat16), ints(N, K), ints(N, 256).to(torch.bfloat16)
    scale = torch.full((N,), 2.0, device="cuda") if kind == 3 else None
    D = a.double() @ b.double().t() * (2 if kind == 3 else 1)
    D = D.to(torch.bfloat16)
    out2 = torch.cat([D[:, i:i + 256].double() @ q[i:i + 256].double().t() for i in range(0, N, 256)], 1).to(torch.bfloat16)
    return a, b.to(torch.int8 if kind == 3 else torch.bfloat16), scale, q, D, out2


@pytest.mark.parametrize("kind,factor,steps", [(0, False, 0), (0, False, 5), (1, True, 0), (1, True, 6), (1, True, 8),
                                               (2, False, 0), (2, False, 7), (2, True, 3), (2, True, 8), (3, False, 4),
                                               (3, True, 2), (3, True, 8)])
def test_a_block_that_gives_up_stores_nothing(kind, factor, steps):
    a, b, scale, q, D, out2 = _problem(kind)
    d = torch.full_like(D, GUARD)
    o = torch.full_like(out2, GUARD) if factor else None
    P.poetx_test_gemm_give_up(kind, M, N, K, a, b, scale, q if factor else None, d, o, steps, 5_000_000)
    st, detail = P.poetx_device_status()
    assert P.STATUS[st] == "POETX_ERR_DEVICE_TIMEOUT" and detail >> 8 == 1, (st, hex(detail))
    rows, cols = (128 if kind < 2 else 256), (64 if kind == 0 else 256)
    tile = torch.zeros_like(D, dtype=torch.bool)
    tile[:rows, :cols] = True
    if factor:
        assert (o[tile] == GUARD).all().item() and torch.equal(o[~tile], out2[~tile])
    if steps == K // 64:  # D was there: all of it, or its half before Q was missed
        tile[:128] = False
    assert (d[tile] == GUARD).all().item() and torch.equal(d[~tile], D[~tile])
    # The same kernels right afterwards.
    y = torch.empty_like(D)
    P.poetx_test_gemm(P.POETX_BF16, M, N, K, 1, 1, a, M, K, K, 0, 0, 0, D[:, :K].contiguous(), M, K, K, 0, 0, 0, y,
                      P.POETX_BF16, N, 0, 0, 0, 1.0, 0.0, None, 0, 0, 0, 0)
    torch.cuda.synchronize()
    device_clean()
    assert torch.equal(y, (a.double() @ D[:N].double().t()).to(torch.bfloat16))
