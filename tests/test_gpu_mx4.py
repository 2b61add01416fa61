"""The 4-bit weight (MX4): quantisation, its product and adjoint, and the layer that runs on it.

Codes, scales and the values they stand for are exact functions of the input, so they are compared bit for
bit.  The product's factors are exact in float32 (2 by 8 significant bits), so with small integers in X and
scales near 1 every partial sum is an exact float32 number too, in any order: there Y must be the 64-bit
result rounded once.  With other values, each of the K products may be cut by 2^-23 of a partial sum, which is
at most S = sum |w x|, and Y is rounded once by half a step, 2^-8 of its value: |dY| <= 2^-8 |Y| + (K + 8) 2^-23 S (8: the
parts of a split sum).
"""
import numpy as np
import pytest
import torch

import oracle as O
import orthogonal_equivalence_cnp_b200 as P
import poetx_inputs as I
from helpers import TOL, device_clean, rel, to_np
from orthogonal_equivalence_cnp_b200.layer import PoetxLayer, make_desc
from orthogonal_equivalence_cnp_b200.optim import MultiAdamW

pytestmark = pytest.mark.gpu


def _u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _empty(rows, cols):
    return (torch.full((rows, cols // 2), 0xA5, dtype=torch.uint8, device="cuda"),
            torch.full((rows, cols // 32), 0x5A, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------------ the weight format
def _special(rows, cols, dtype, seed):
    rng = np.random.default_rng(seed)
    W = (rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 4, (rows, 1)))).astype(np.float32)
    ties = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, 0.24, 0.26, -6, 7.9, -0.0, 5.01], np.float32)
    for r, f in ((0, 1.0), (1, 2.0 ** -20), (2, 2.0 ** 60)):
        if r < rows:
            W[r, :16] = ties * np.float32(f)
            W[r, 16:32] = 0
    if rows > 8:
        W[3] = 0                                    # zero blocks: scale 0, signs kept
        W[3, 5] = -0.0
        W[4, 0], W[5, cols - 1], W[6, 1] = np.nan, np.inf, -np.inf
        W[7, :32] = np.float32(2.0 ** -133) * np.arange(-16, 16, dtype=np.float32)  # subnormal throughout
        W[8, :32] = np.float32(3.0e38)              # the largest magnitudes
        W[8, 0] = np.float32(2.0 ** 127)
    return I.round_to_bf16(W) if dtype == "bf16" else W


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (9, 32), (129, 96), (1000, 1056), (513, 4096)])
def test_quantize_and_back_bit_exact(dtype, rows, cols):
    W = _special(rows, cols, dtype, rows + cols)
    t = torch.from_numpy(W).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    codes, scales = _empty(rows, cols)
    P.poetx_mx4_quantize(P.POETX_BF16 if dtype == "bf16" else P.POETX_F32, rows, cols, t, codes, scales)
    back = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    P.poetx_mx4_dequantize(rows, cols, codes, scales, back)
    torch.cuda.synchronize()
    device_clean()
    c, s = O.mx4_quantize(W)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    ref = O.mx4_dequantize(c, s)
    assert np.array_equal(to_np(back), ref, equal_nan=True)
    assert np.array_equal(np.signbit(to_np(back))[np.isfinite(ref)], np.signbit(ref)[np.isfinite(ref)])


def test_every_code_at_every_scale_reads_back():
    # All 16 codes under all 256 scales, quantised weights never reaching the last two.
    codes = np.tile(np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2, np.uint8), (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    back = torch.empty(256, 32, dtype=torch.bfloat16, device="cuda")
    P.poetx_mx4_dequantize(256, 32, _u8(codes), _u8(scales), back)
    ref = O.mx4_dequantize(codes, scales)
    ref[np.abs(ref) >= 2.0 ** 128] *= np.inf
    got = to_np(back)
    assert np.array_equal(got, ref, equal_nan=True)
    assert np.array_equal(np.signbit(got[:255]), np.signbit(ref[:255]))


def test_quantize_offsets_past_32_bits():
    rows, cols = 70000, 32768  # 2.3e9 elements
    W = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = _special(16, cols, "bf16", 5)
    W[-16:] = torch.from_numpy(tail).cuda()
    codes, scales = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda"), torch.empty(
        rows, cols // 32, dtype=torch.uint8, device="cuda")
    P.poetx_mx4_quantize(P.POETX_BF16, rows, cols, W, codes, scales)
    c, s = O.mx4_quantize(tail)
    assert np.array_equal(codes[-16:].cpu().numpy(), c) and np.array_equal(scales[-16:].cpu().numpy(), s)
    assert not codes[:-16].any().item() and not scales[:-16].any().item()
    W.fill_(1.0)
    P.poetx_mx4_dequantize(rows, cols, codes, scales, W)
    assert np.array_equal(to_np(W[-16:]), O.mx4_dequantize(c, s), equal_nan=True)
    assert not W[:-16].any().item()


# ------------------------------------------------------------------------------ the product
def _matmul(adjoint, X, codes, scales, d_in, d_out, stream=None):
    """Y with guard rows behind the last token, which must be left as they were."""
    n, m = X.shape[0], d_in if adjoint else d_out
    buf = torch.full((n + 3, m), 1234.0, dtype=torch.bfloat16, device="cuda")
    P.poetx_mx4_matmul(adjoint, n, d_in, d_out, X, codes, scales, buf[:n], stream)
    torch.cuda.synchronize()
    device_clean()
    assert (buf[n:] == 1234).all().item()
    return buf[:n]


def _integer_problem(n, d_in, d_out, adjoint, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = d_out if adjoint else d_in
    X = torch.randint(-2, 3, (n, k), device="cuda", generator=g).to(torch.bfloat16)
    codes = torch.randint(0, 256, (d_out, d_in // 2), device="cuda", generator=g).to(torch.uint8)
    scales = torch.randint(126, 129, (d_out, d_in // 32), device="cuda", generator=g).to(torch.uint8)
    return X, codes, scales


def _weight64(codes, scales):
    lut = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    lut = torch.cat([lut, -lut])
    c = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    return lut[c.long()] * s


SHAPES = [(32, 8), (32, 128), (64, 136), (96, 1000), (1056, 264), (992, 256), (4096, 512), (320, 4096), (2080, 40),
          (32768, 24), (64, 32776)]
TOKENS = [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 127, 200, 257, 600]


@pytest.mark.parametrize("adjoint", [0, 1])
@pytest.mark.parametrize("d_in,d_out", SHAPES)
def test_products_of_small_integers_are_exact(adjoint, d_in, d_out):
    for n in TOKENS:
        X, codes, scales = _integer_problem(n, d_in, d_out, adjoint, n + d_in)
        Y = _matmul(adjoint, X, codes, scales, d_in, d_out)
        W = _weight64(codes, scales)
        ref = X.double() @ (W if adjoint else W.t())
        assert torch.equal(Y, ref.to(torch.bfloat16)), (n, (Y.double() - ref).abs().max().item())


@pytest.mark.parametrize("adjoint", [0, 1])
@pytest.mark.parametrize("n,d_in,d_out", [(600, 1056, 1000), (333, 4128, 1032), (1300, 2080, 3000), (2100, 4128, 4104),
                                          (700, 14368, 264), (640, 96, 14344)])
def test_large_products_whose_sides_fit_no_tile_are_exact(adjoint, n, d_in, d_out):
    X, codes, scales = _integer_problem(n, d_in, d_out, adjoint, n)
    Y = _matmul(adjoint, X, codes, scales, d_in, d_out)
    W = _weight64(codes, scales)
    ref = X.double() @ (W if adjoint else W.t())
    assert torch.equal(Y, ref.to(torch.bfloat16)), (Y.double() - ref).abs().max().item()


@pytest.mark.parametrize("adjoint", [0, 1])
@pytest.mark.parametrize("n,d_in,d_out", [(1, 4096, 14336), (5, 14336, 4096), (40, 4096, 4096), (300, 1056, 1000),
                                          (2048, 4096, 4096), (2500, 4096, 2056), (4097, 2048, 4096)])
def test_products_of_activations(adjoint, n, d_in, d_out):
    g = torch.Generator(device="cuda").manual_seed(n)
    k = d_out if adjoint else d_in
    X = torch.randn(n, k, device="cuda", generator=g)
    X = (X * (1 + 15 * (torch.rand(1, k, device="cuda", generator=g) < 0.01))).to(torch.bfloat16)
    W = torch.randn(d_out, d_in, device="cuda", generator=g) * 0.02
    codes, scales = _empty(d_out, d_in)
    P.poetx_mx4_quantize(P.POETX_F32, d_out, d_in, W, codes, scales)
    Y = _matmul(adjoint, X, codes, scales, d_in, d_out)
    W = _weight64(codes, scales)
    W = W if adjoint else W.t()
    ref, size = X.double() @ W, X.double().abs() @ W.abs()
    bound = 2.0 ** -8 * ref.abs() + (k + 8) * 2.0 ** -23 * size
    assert ((Y.double() - ref).abs() <= bound).all().item()
    # An elementwise bound that K makes wide, and a norm: one rounding, 2^-8 at most.
    assert (Y.double() - ref).norm().item() <= 2.0 ** -8 * ref.norm().item()
    again = _matmul(adjoint, X, codes, scales, d_in, d_out)
    assert torch.equal(Y, again)


@pytest.mark.parametrize("adjoint", [0, 1])
@pytest.mark.parametrize("n", [1, 12, 40, 300])
def test_nan_blocks_and_tokens_stay_where_they_are(adjoint, n):
    d_in, d_out = 320, 200
    X, codes, scales = _integer_problem(n, d_in, d_out, adjoint, 77 + n)
    scales[13, 4] = 255                       # row 13, columns 128..159
    clean = _matmul(adjoint, X, codes, torch.where(scales == 255, 127, scales), d_in, d_out)
    Y = _matmul(adjoint, X, codes, scales, d_in, d_out)
    hit = torch.zeros_like(Y, dtype=torch.bool)
    hit[:, 128:160] = True if adjoint else False
    if not adjoint:
        hit[:, 13] = True
    assert Y[hit].isnan().all().item() and torch.equal(Y[~hit], clean[~hit])
    # A token with an infinity and one with a NaN: no other row changes.
    scales[13, 4] = 127
    clean = _matmul(adjoint, X, codes, scales, d_in, d_out)
    X2 = X.clone()
    X2[0, 3] = float("nan")
    if n > 5:
        X2[5, 8] = float("inf")
    Y = _matmul(adjoint, X2, codes, scales, d_in, d_out)
    rows = torch.ones(n, dtype=torch.bool, device="cuda")
    rows[0] = False
    if n > 5:
        rows[5] = False
        W = _weight64(codes, scales)
        inf = X2[5:6].double() @ (W if adjoint else W.t())
        assert torch.equal(Y[5:6].double().nan_to_num(7.0, 1e300, -1e300), inf.to(torch.bfloat16).double().nan_to_num(7.0, 1e300, -1e300))
    assert Y[0].isnan().all().item() and torch.equal(Y[rows], clean[rows])


@pytest.mark.parametrize("adjoint", [0, 1])
@pytest.mark.parametrize("n", [3, 50])
def test_far_scales(adjoint, n):
    # Scales from the smallest to the largest that values reach: products and sums of one magnitude per block
    # of outputs, so that they are exact.
    d_in, d_out = 256, 64
    for e in (0, 1, 2, 100, 126, 127, 128, 129, 130, 200, 245):
        X, codes, scales = _integer_problem(n, d_in, d_out, adjoint, e)
        scales.fill_(e)
        # Partial results of float32's own range: units of 2^-128 and more are exact while they are not cut to
        # zero; X of 2^20 keeps the smallest scales' products normal.
        up = 2.0 ** 20 if e < 64 else 2.0 ** -20 if e > 200 else 1.0
        Y = _matmul(adjoint, (X * up), codes, scales, d_in, d_out)
        W = _weight64(codes, scales)
        ref = (X.double() * up) @ (W if adjoint else W.t())
        assert torch.equal(Y, ref.to(torch.bfloat16)), e


def test_product_offsets_past_32_bits():
    n, d_in, d_out = 160000, 64, 14336  # 2.3e9 outputs
    X, codes, scales = _integer_problem(n, d_in, d_out, 0, 3)
    Y = torch.empty(n, d_out, dtype=torch.bfloat16, device="cuda")
    P.poetx_mx4_matmul(0, n, d_in, d_out, X, codes, scales, Y)
    W = _weight64(codes, scales)
    rows = torch.tensor([0, 77777, 149796, 149797, n - 1], device="cuda")
    assert torch.equal(Y[rows], (X[rows].double() @ W.t()).to(torch.bfloat16))
    dX = torch.empty(n, d_in, dtype=torch.bfloat16, device="cuda")
    dY = (Y > 0).to(torch.bfloat16)
    P.poetx_mx4_matmul(1, n, d_in, d_out, dY, codes, scales, dX)
    assert torch.equal(dX[rows], (dY[rows].double() @ W).to(torch.bfloat16))
    device_clean()


@pytest.mark.parametrize("adjoint", [0, 1])
def test_more_token_tiles_than_a_grid_has_rows(adjoint):
    n, d_in, d_out = (1 << 20) + 5, 32, 8
    X, codes, scales = _integer_problem(n, d_in, d_out, adjoint, 4)
    W = _weight64(codes, scales)
    Y = _matmul(adjoint, X, codes, scales, d_in, d_out)
    assert torch.equal(Y, (X.double() @ (W if adjoint else W.t())).to(torch.bfloat16))


def test_products_on_streams_and_in_a_graph():
    cases = []
    for i, (adjoint, n, d_in, d_out) in enumerate([(0, 1, 4096, 1024), (0, 33, 1056, 1000), (1, 300, 1056, 1000),
                                                   (1, 2, 1024, 4096), (0, 700, 512, 2048)]):
        X, codes, scales = _integer_problem(n, d_in, d_out, adjoint, i)
        W = _weight64(codes, scales)
        Y = torch.zeros(n, d_in if adjoint else d_out, dtype=torch.bfloat16, device="cuda")
        cases.append((adjoint, n, d_in, d_out, X, codes, scales, Y,
                      (X.double() @ (W if adjoint else W.t())).to(torch.bfloat16)))

    def run(stream=None):
        for c in cases:
            P.poetx_mx4_matmul(*c[:8], stream)

    def check():
        for c in cases:
            assert torch.equal(c[7], c[8]), c[:4]
            c[7].zero_()

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for c, s in zip(cases, streams):  # all at once
        P.poetx_mx4_matmul(*c[:8], s)
    torch.cuda.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check()
    # New inputs in the captured buffers.
    for c in cases:
        c[4].neg_()
    graph.replay()
    torch.cuda.synchronize()
    for c in cases:
        assert torch.equal(c[7], -c[8])
    device_clean()


@pytest.mark.parametrize("n,d_in,d_out", [(3, 96, 40), (70, 256, 264), (300, 1056, 1000)])
def test_adjoint_is_the_transpose_of_the_forward_product(n, d_in, d_out):
    # <dY, X W^T> = <dY W, X>, and the derivative of <dY, Y(X)> along any direction: exact with numbers this small
    # (sparse -1, 0, 1 on both sides, codes of -1, 0, 1: every output an integer under 256, exact in bf16).
    g = torch.Generator(device="cuda").manual_seed(n)

    def sparse(rows, cols, p):
        return (torch.randint(-1, 2, (rows, cols), device="cuda", generator=g)
                * (torch.rand(rows, cols, device="cuda", generator=g) < p)).to(torch.bfloat16)

    nib = torch.tensor([0, 2, 10], device="cuda")[torch.randint(0, 3, (d_out, d_in), device="cuda", generator=g)]
    codes = (nib[:, 0::2] + 16 * nib[:, 1::2]).to(torch.uint8)
    scales = torch.full((d_out, d_in // 32), 127, dtype=torch.uint8, device="cuda")
    X, D, dY = sparse(n, d_in, 0.2), sparse(n, d_in, 0.2), sparse(n, d_out, 0.2)
    dX = _matmul(1, dY, codes, scales, d_in, d_out)
    assert dX.abs().max().item() <= 256
    f = lambda x: (dY.double() * _matmul(0, x, codes, scales, d_in, d_out).double()).sum().item()
    assert f(X) == (dX.double() * X.double()).sum().item()
    assert (f(X + D) - f(X - D)) / 2 == (dX.double() * D.double()).sum().item()


@pytest.mark.parametrize("adjoint", [0, 1])
@pytest.mark.parametrize("n,d_in,d_out", [(1, 96, 56), (9, 1056, 1000), (40, 1056, 1000), (300, 512, 264)])
def test_arrays_that_start_on_16_bytes_only(adjoint, n, d_in, d_out):
    X, codes, scales = _integer_problem(n, d_in, d_out, adjoint, 21)
    W = _weight64(codes, scales)
    ref = (X.double() @ (W if adjoint else W.t())).to(torch.bfloat16)

    def shifted(t):  # the same values 16 bytes into a buffer, with 16 bytes behind
        flat = torch.zeros(t.numel() * t.element_size() + 32, dtype=torch.uint8, device="cuda")
        assert flat.data_ptr() % 256 == 0
        v = flat[16:-16].view(t.dtype).view(t.shape)
        v.copy_(t)
        return flat, v

    bx, x = shifted(X)
    bc, c = shifted(codes)
    bs, sc = shifted(scales)
    by, y = shifted(torch.zeros_like(ref))
    by[:16] = by[-16:] = 77
    P.poetx_mx4_matmul(adjoint, n, d_in, d_out, x, c, sc, y)
    assert torch.equal(y, ref)
    assert (by[:16] == 77).all().item() and (by[-16:] == 77).all().item()
    bw, w = shifted(torch.zeros(d_out, d_in, dtype=torch.bfloat16, device="cuda"))
    bw[:16] = bw[-16:] = 77
    P.poetx_mx4_dequantize(d_out, d_in, c, sc, w)
    assert torch.equal(w, W.to(torch.bfloat16))
    P.poetx_mx4_quantize(P.POETX_BF16, d_out, d_in, w, c, sc)
    back = torch.empty(d_out, d_in, dtype=torch.bfloat16, device="cuda")
    P.poetx_mx4_dequantize(d_out, d_in, c, sc, back)
    assert torch.equal(back, w) and (bw[:16] == 77).all().item() and (bw[-16:] == 77).all().item()
    device_clean()


def test_same_buffers_from_two_graphs_and_threads():
    # Two graphs of the same call, replayed in turn and at once on two streams (same inputs, two outputs), and two host threads.
    import threading
    n, d_in, d_out = 100, 1056, 1000
    X, codes, scales = _integer_problem(n, d_in, d_out, 0, 8)
    ref = (X.double() @ _weight64(codes, scales).t()).to(torch.bfloat16)
    Ys = [torch.zeros(n, d_out, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    P.poetx_mx4_matmul(0, n, d_in, d_out, X, codes, scales, Ys[0])
    graphs = []
    for Y in Ys:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            P.poetx_mx4_matmul(0, n, d_in, d_out, X, codes, scales, Y)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in Ys]
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(Y, ref) for Y in Ys)

    failed = []

    def work(i):  # the first call of a thread is one that needs tensor maps
        try:
            for _ in range(50):
                P.poetx_mx4_matmul(0, n, d_in, d_out, X, codes, scales, Ys[i], streams[i])
        except Exception as e:
            failed.append(e)

    for Y in Ys:
        Y.zero_()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and all(torch.equal(Y, ref) for Y in Ys)
    device_clean()


@pytest.mark.parametrize("adjoint,n,d_in,d_out", [(1, 64, 4096, 14336), (0, 64, 4096, 4096), (1, 33, 1024, 14336),
                                                  (0, 500, 4096, 1024), (1, 2048, 4096, 4096), (0, 1, 4096, 4096)])
def test_products_with_cold_caches(adjoint, n, d_in, d_out):
    # Everything from HBM, the rings of tiles gone round many times: a tile given back before it is read, or read
    # before it has arrived, shows only with such latencies.
    X, codes, scales = _integer_problem(n, d_in, d_out, adjoint, 11)
    W = _weight64(codes, scales)
    ref = (X.double() @ (W if adjoint else W.t())).to(torch.bfloat16)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")  # larger than the L2 cache
    Y = torch.empty_like(ref)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(25):
        Y.zero_()
        flush.fill_(i)
        if i % 3 == 0:
            torch.cuda.synchronize()
        P.poetx_mx4_matmul(adjoint, n, d_in, d_out, X, codes, scales, Y)
        wrong += (Y != ref).sum()
    assert wrong.item() == 0
    device_clean()


def test_quantize_then_multiply_needs_no_wait():
    # Launched back to back on one stream: the product reads what the quantiser has just written.
    g = torch.Generator(device="cuda").manual_seed(4)
    codes, scales = _empty(4096, 4096)
    back = torch.empty(4096, 4096, dtype=torch.bfloat16, device="cuda")
    for i in range(4):
        W = (torch.randn(4096, 4096, device="cuda", generator=g) * 2.0 ** -i).to(torch.bfloat16)
        X = torch.eye(4096, device="cuda", dtype=torch.bfloat16)[i * 40:i * 40 + 37].contiguous()
        Y = torch.empty(37, 4096, dtype=torch.bfloat16, device="cuda")
        P.poetx_mx4_quantize(P.POETX_BF16, 4096, 4096, W, codes, scales)
        P.poetx_mx4_matmul(1, 37, 4096, 4096, X, codes, scales, Y)
        P.poetx_mx4_dequantize(4096, 4096, codes, scales, back)
        assert torch.equal(Y, back[i * 40:i * 40 + 37])


# -------------------------------------------------------------------------------- the layer
def _layer(inp, n=None):
    s = inp.shape
    L = PoetxLayer(make_desc(s.d_in, s.d_out, s.b, s.k, "bf16", "mem"), n or inp.X.shape[0])
    L.load_state(inp.W0, inp.theta_R, inp.theta_P, inp.pi_L, inp.pi_R)
    L.quantize("mx4")
    return L


def _oracle(inp, theta_R=None, theta_P=None, rows=None):
    s = inp.shape
    tR = inp.theta_R if theta_R is None else theta_R
    tP = inp.theta_P if theta_P is None else theta_P
    X, dY = (inp.X, inp.dY) if rows is None else (inp.X[rows], inp.dY[rows])
    codes, scales = O.mx4_quantize(O.absorb(inp.W0, inp.pi_L, inp.pi_R))
    W = O.mx4_dequantize(codes, scales)
    Y = O.forward_chain(X, W, O.cnp(tR, s.b, s.k), O.cnp(tP, s.b, s.k), inp.pi_L, inp.pi_R)[0]
    dX, gR, gP = O.backward_chain(X, dY, W, tR, tP, inp.pi_L, inp.pi_R, s.b, s.k)
    return dict(Y=Y, dX=dX, g_R=gR, g_P=gP, codes=codes, scales=scales)


@pytest.mark.parametrize("d_in,d_out,b,n", [(512, 768, 256, 300), (768, 512, 128, 200), (1024, 1024, 512, 129),
                                            (64, 192, 64, 1), (512, 512, 256, 600), (256, 1280, 64, 77)])
def test_layer_matches_oracle(d_in, d_out, b, n):
    s = I.small_shape(d_in, d_out, b, 3, n, "bf16", "mem", theta_std=0.005, w_std=0.02)
    inp = I.make_layer(s, 5 * d_in + d_out + b + n)
    L = _layer(inp)
    L.step(L.to_dev(inp.X), L.to_dev(inp.dY))
    torch.cuda.synchronize()
    device_clean()
    o = _oracle(inp)
    assert np.array_equal(L.W0q.cpu().numpy(), o["codes"]) and np.array_equal(L.W0s.cpu().numpy(), o["scales"])
    errs = {k: rel(to_np(t), o[k]) for k, t in (("Y", L.Y), ("dX", L.dX), ("g_R", L.g_R), ("g_P", L.g_P))}
    assert all(e <= TOL["bf16"] for e in errs.values()), errs


def test_full_size_layer_sampled():
    inp = I.make_workload("llama8b_up_4096x14336_b256_bf16_mem")
    rows = np.sort(np.random.default_rng(6).choice(inp.X.shape[0], 64, replace=False))
    dY = np.zeros_like(inp.dY)
    dY[rows] = inp.dY[rows]
    L = _layer(inp)
    L.step(L.to_dev(inp.X), L.to_dev(dY))
    torch.cuda.synchronize()
    device_clean()
    o = _oracle(inp, rows=rows)
    errs = {"Y": rel(to_np(L.Y)[rows], o["Y"]), "dX": rel(to_np(L.dX)[rows], o["dX"]),
            "g_R": rel(to_np(L.g_R), o["g_R"]), "g_P": rel(to_np(L.g_P), o["g_P"])}
    assert all(e <= TOL["bf16"] for e in errs.values()), errs


def test_theta_gradients_match_differences():
    # The layer's gradient along a random direction of theta against a difference of the oracle's loss
    # <dY, Y(theta)> in 64 bits (central, so off by the step's square).
    s = I.small_shape(256, 128, 64, 3, 40, "bf16", "mem", theta_std=0.01, w_std=0.02)
    inp = I.make_layer(s, 31)
    L = _layer(inp)
    L.step(L.to_dev(inp.X), L.to_dev(inp.dY))
    codes, scales = O.mx4_quantize(O.absorb(inp.W0, inp.pi_L, inp.pi_R))
    W = O.mx4_dequantize(codes, scales)
    gR, gP = to_np(L.g_R), to_np(L.g_P)
    # The gradient's own direction: its size is the product's, and errors elsewhere do not drown it.
    dR, dP = gR / np.linalg.norm(gR), gP / np.linalg.norm(gP)

    def loss(h, side):
        tR = inp.theta_R + (h * dR if side == "R" else 0)
        tP = inp.theta_P + (h * dP if side == "P" else 0)
        Y = O.forward_chain(inp.X, W, O.cnp(tR, s.b, s.k), O.cnp(tP, s.b, s.k), inp.pi_L, inp.pi_R)[0]
        return float((inp.dY.astype(np.float64) * Y).sum())

    for side, g in (("R", gR), ("P", gP)):
        diff = (loss(1e-3, side) - loss(-1e-3, side)) / 2e-3
        assert abs(diff - np.linalg.norm(g)) <= TOL["bf16"] * np.linalg.norm(g), side


@pytest.mark.parametrize("d_in,d_out,b", [(1024, 512, 256), (512, 768, 128)])
def test_merge(d_in, d_out, b):
    s = I.small_shape(d_in, d_out, b, 3, 64, "bf16", "mem", theta_std=0.005, w_std=0.02)
    inp = I.make_layer(s, 91 + b)
    pL2, pR2 = I.fresh_permutations(s, 91 + b)
    L = _layer(inp)
    L.cnp()
    # The same merge on the bf16 weight that the codes stand for, then quantised, must give the same codes.
    F = PoetxLayer(L.desc, 64)
    F.load_state(inp.W0, inp.theta_R, inp.theta_P, inp.pi_L, inp.pi_R)
    P.poetx_mx4_dequantize(d_out, d_in, L.W0q, L.W0s, F.W0p)
    F.cnp()
    new = torch.from_numpy(pL2).cuda(), torch.from_numpy(pR2).cuda()
    L.merge(*new)
    F.merge(*new)
    merged = to_np(F.W0p)
    torch.cuda.synchronize()
    device_clean()
    assert torch.count_nonzero(L.theta_R).item() == 0 and torch.count_nonzero(L.theta_P).item() == 0
    codes, scales = O.mx4_quantize(O.absorb(inp.W0, inp.pi_L, inp.pi_R))
    Wn = O.mx4_merge(codes, scales, inp.theta_R, inp.theta_P, inp.pi_L, inp.pi_R, pL2, pR2, b, 3)[0]
    assert rel(merged, Wn) <= TOL["bf16"]
    cn, sn = O.mx4_quantize(merged)
    assert np.array_equal(L.W0q.cpu().numpy(), cn) and np.array_equal(L.W0s.cpu().numpy(), sn)
    # The merged layer serves tokens as a plain product in the permuted basis: Y[:, pi_L] = X[:, pi_R] W0'^T.
    L.cnp()
    X = L.to_dev(inp.X)
    L.forward(X)
    Z = _matmul(0, X[:, new[1].long()].contiguous(), L.W0q, L.W0s, d_in, d_out)
    Y = torch.empty_like(Z)
    Y[:, new[0].long()] = Z
    assert rel(to_np(L.Y), to_np(Y)) <= TOL["bf16"]


def test_training_steps_with_8_bit_moments():
    # Three steps of the layer on its 4-bit weight with MultiAdamW on e4m3 moments, a captured graph of the
    # same step replayed for the second and third, against the oracle's steps.
    s = I.small_shape(512, 384, 128, 3, 96, "bf16", "mem", theta_std=0.005, w_std=0.02)
    inp = I.make_layer(s, 44)
    L = _layer(inp)
    X, dY = L.to_dev(inp.X), L.to_dev(inp.dY)
    opt = MultiAdamW.from_params([L.theta_R, L.theta_P], [L.g_R, L.g_P])
    cfg = P.poetx_adamw_cfg(1e-4, 0.5, 0.9, 0.999, 1e-8, 0.0)
    tR, tP = inp.theta_R.astype(np.float64), inp.theta_P.astype(np.float64)
    state = [[np.zeros(t.size), np.zeros(t.size)] for t in (tR, tP)]
    graph = None
    for t in (1, 2, 3):
        if graph is None:
            L.step(X, dY)
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                L.step(X, dY)
        else:
            graph.replay()
        o = _oracle(inp, tR, tP)
        for got, want in ((L.g_R, o["g_R"]), (L.g_P, o["g_P"]), (L.Y, o["Y"]), (L.dX, o["dX"])):
            assert rel(to_np(got), want) <= TOL["bf16"], t
        # The oracle's step on the layer's own gradients: the optimiser's part alone.
        for i, (x, g) in enumerate(((tR, L.g_R), (tP, L.g_P))):
            m, v = state[i]
            p, m, v = O.adamw_step(x.ravel(), to_np(g).ravel(), m, v, t, 1e-4, 0.5, 0.9, 0.999, 1e-8, 0.0)
            qm, um = O.e4m3_moments(m, False)
            qr, ur = O.e4m3_moments(np.sqrt(v), True)
            state[i] = [qm * np.repeat(um, 256)[:m.size], (qr * np.repeat(ur, 256)[:m.size]) ** 2]
            x[...] = p.reshape(x.shape)
        opt.step(cfg)
        # A code next to a rounding border may fall on the other side: half a step of m (2^-4) and of the root
        # (2^-4) of an update of at most lr per step, on few elements; the float32 steps by far less.
        for got, want, start in ((L.theta_R, tR, inp.theta_R), (L.theta_P, tP, inp.theta_P)):
            assert rel(to_np(got) - start, want.reshape(got.shape) - start) <= 2.0 ** -4, t
    device_clean()


def test_refusals_and_empty_calls():
    L = PoetxLayer(make_desc(512, 512, 256, 3, "bf16", "mem"), 8)
    L.W0p.zero_()
    L.quantize("mx4")
    assert L.W0p is None and not L.W0q.any().item() and not L.W0s.any().item()
    with pytest.raises(ValueError):
        L.quantize("mx4")
    with pytest.raises(ValueError):
        PoetxLayer(make_desc(512, 512, 256, 3, "bf16", "fast"), 8).quantize("mx4")
    P.poetx_mx4_forward(L.desc, 0, L.dX, L.W0q, L.W0s, L.perm_L, L.perm_R, L.Q_R, L.Q_P, L.Y, L.ws)
    P.poetx_mx4_matmul(0, 0, 512, 512, L.dX, L.W0q, L.W0s, L.Y)
    with pytest.raises(ValueError, match="W0q|codes"):
        P.poetx_mx4_matmul(0, 8, 1024, 512, torch.empty(8, 1024, dtype=torch.bfloat16, device="cuda"), L.W0q, L.W0s, L.Y)
    with pytest.raises(ValueError, match="X"):
        P.poetx_mx4_matmul(0, 9, 512, 512, L.dX, L.W0q, L.W0s, torch.empty(9, 512, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        P.poetx_mx4_matmul(0, 4, 512, 512, torch.empty(8, 512, dtype=torch.bfloat16, device="cuda")[::2], L.W0q, L.W0s, L.Y)
    device_clean()


@pytest.mark.parametrize("bits", ["mx4", "int8"])
def test_quantize_releases_every_bf16_weight(bits):
    d = 2048
    held = lambda: torch.cuda.memory_stats()["requested_bytes.all.current"]  # without the allocator's own rounding
    inp = I.make_layer(I.small_shape(d, d, 256, 3, 8, "bf16", "mem", theta_std=0.005, w_std=0.02), 3, with_activations=False)
    L = PoetxLayer(make_desc(d, d, 256, 3, "bf16", "mem"), 8)
    before = held() - 2 * d * d  # without W0'
    L.load_state(inp.W0, inp.theta_R, inp.theta_P, inp.pi_L, inp.pi_R)
    L.quantize(bits)
    assert held() - before == (d * d // 2 + d * d // 32 if bits == "mx4" else d * d + 4 * d)  # codes and scales
    assert L.W0 is None and L.W0p is None
    with pytest.raises(ValueError, match="un-absorbed"):
        L.fourperm_step(L.dX, L.Y)
    device_clean()


def test_moments_held_by_a_layer():
    desc = make_desc(2048, 2048, 256, 3, "bf16", "mem")
    held = lambda: torch.cuda.memory_stats()["requested_bytes.all.current"]
    sizes = {}
    for moments in ("f32", "e4m3", None):
        before = held()
        L = PoetxLayer(desc, 8, moments=moments)
        sizes[moments] = held() - before
        n = L.theta.numel()
        del L
    assert sizes["f32"] - sizes[None] == 8 * n and sizes["e4m3"] - sizes[None] == 2 * n + 8 * (n // 256)


@pytest.mark.parametrize("bits", ["mx4", "int8", None])
def test_train_step_with_8_bit_moments_and_merges(bits):
    # The layer's own schedule against the same calls made one by one with an optimiser from outside: the same bits.
    s = I.small_shape(512, 768, 256, 3, 64, "bf16", "mem", theta_std=0.005, w_std=0.02)
    inp = I.make_layer(s, 71)
    cfg = P.poetx_adamw_cfg(1e-3, 0.5, 0.9, 0.999, 1e-8, 0.01)
    perms = [I.fresh_permutations(s, 300 + i) for i in range(2)]
    layers = []
    for moments in ("e4m3", None):
        L = PoetxLayer(make_desc(512, 768, 256, 3, "bf16", "mem"), 64, moments=moments)
        L.load_state(inp.W0, inp.theta_R, inp.theta_P, inp.pi_L, inp.pi_R)
        if bits:
            L.quantize(bits)
        layers.append(L)
    A, B = layers
    X, dY = A.to_dev(inp.X), A.to_dev(inp.dY)
    queue = list(perms)
    for i in range(5):
        A.train_step(X, dY, cfg, reset_gap=2, new_perms=lambda: queue.pop(0), seed=i + 1)
        if i == 2:  # gradients moved into a buffer of several layers
            flat = torch.zeros(A.grad.numel() + 256, device="cuda")
            nbo = A.g_R.shape[0]
            A.grad = flat[256:].view(A.grad.shape)
            A.g_R, A.g_P = A.grad[:nbo], A.grad[nbo:]
    assert not queue and A.t == 1 and A.steps == 5
    opt = MultiAdamW.from_params([B.theta], [B.grad])
    for i in range(5):
        B.step(X, dY)
        opt.step(cfg, seed=i + 1)
        if i in (1, 3):
            B.cnp()
            B.merge(*(torch.from_numpy(p).cuda() for p in perms[i // 2]))
            opt.reset()
    torch.cuda.synchronize()
    device_clean()
    assert torch.equal(A.theta, B.theta) and A.theta.any().item()
    assert torch.equal(A.perm_L, B.perm_L) and torch.equal(A.perm_R, B.perm_R)
    for a, b in ((A.W0q, B.W0q), (A.W0s, B.W0s)) if bits else ((A.W0p, B.W0p),):
        assert torch.equal(a, b)
    x, y = A.optimizer.tensors[0], opt.tensors[0]
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in ((x.m, y.m), (x.v, y.v), (x.scale, y.scale)))


def test_layers_that_share_a_workspace():
    # Two layers of different sizes, steps and merges in turn: the same bits as with a workspace each, and what a
    # layer on MX4 with 8-bit moments and shared scratch holds is its codes, theta, gradient, moments and activations.
    shapes = [I.small_shape(512, 768, 256, 3, 64, "bf16", "mem", theta_std=0.005, w_std=0.02),
              I.small_shape(1024, 512, 128, 3, 96, "bf16", "mem", theta_std=0.005, w_std=0.02)]
    inps = [I.make_layer(s, 80 + i) for i, s in enumerate(shapes)]
    descs = [make_desc(s.d_in, s.d_out, s.b, 3, "bf16", "mem") for s in shapes]
    ws = torch.empty(max(PoetxLayer.workspace_bytes(d, s.n_tokens) for d, s in zip(descs, shapes)), dtype=torch.uint8,
                     device="cuda")
    cfg = P.poetx_adamw_cfg(1e-3, 0.5, 0.9, 0.999, 1e-8, 0.01)
    runs = []
    for shared in (None, ws):
        layers = []
        for inp, d, s in zip(inps, descs, shapes):
            before = torch.cuda.memory_stats()["requested_bytes.all.current"]
            L = PoetxLayer(d, s.n_tokens, moments="e4m3", workspace=shared)
            L.load_state(inp.W0, inp.theta_R, inp.theta_P, inp.pi_L, inp.pi_R)
            L.quantize("mx4")
            layers.append(L)
            if shared is not None:
                torch.cuda.synchronize()
                n, side = L.theta.numel(), d.d_in + d.d_out
                assert torch.cuda.memory_stats()["requested_bytes.all.current"] - before == (
                    d.d_in * d.d_out * 17 // 32 + 8 * n + 2 * n + 8 * ((n + 255) // 256) + 2 * s.n_tokens * side
                    + 2 * d.b * side + 4 * side)
        acts = [(L.to_dev(inp.X), L.to_dev(inp.dY)) for L, inp in zip(layers, inps)]
        for step in range(4):
            for i, (L, (X, dY)) in enumerate(zip(layers, acts)):
                L.train_step(X, dY, cfg, reset_gap=2, seed=step + 1,
                             new_perms=lambda: I.fresh_permutations(shapes[i], 500 + 10 * i + step))
        torch.cuda.synchronize()
        runs.append([t.clone() for L in layers for t in (L.theta, L.Y, L.dX, L.grad, L.W0q, L.W0s)])
        del layers, L
    device_clean()
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1187, 2080), (2411, 1056)])
def test_quantize_batches_that_end_inside_a_warp(dtype, rows, cols):
    # More pieces of eight than there are resident threads, and no whole number of warps of them.
    assert rows * cols // 8 > 256 * 8 * 148 and rows * cols // 8 % 32
    W = _special(rows, cols, dtype, rows)
    t = torch.from_numpy(W).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    codes, scales = _empty(rows, cols)
    P.poetx_mx4_quantize(P.POETX_BF16 if dtype == "bf16" else P.POETX_F32, rows, cols, t, codes, scales)
    back = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    P.poetx_mx4_dequantize(rows, cols, codes, scales, back)
    c, s = O.mx4_quantize(W)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(to_np(back), O.mx4_dequantize(c, s), equal_nan=True)
    device_clean()
