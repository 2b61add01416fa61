"""The 4-bit weight (MX4) and the many-tensor AdamW step as they are measured: inputs, one pass
through each in elementary torch operations or through the library, the work that a pass cannot do
without, and the same results in 64 bits.

MX4 is the OCP microscaled 4-bit format: e2m1 codes, one power-of-two scale (E8M0) for 32
consecutive columns of a row; codes are packed two to a byte, the even column in the low nibble.
AdamW keeps its moments in 32 bits, or in e4m3 with one pair of scales for 256 elements.
"""
import math

import torch

own = False

DEV = "cuda"
BLK = 32      # columns that share an MX4 scale
ABLK = 256    # elements that share a pair of moment scales
M32 = 0xFFFFFFFF
CFG = dict(lr=1e-3, gamma=0.5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


# ----------------------------------------------------------------------------------- the cases
def listed():
    return [
        # A frozen weight is quantised when a layer switches to MX4 and after every merge, and read
        # back for inspection or for the merge itself: the gate/up projection of an 8B layer.
        dict(name="mx4 quantize up", op="quant", rows=14336, cols=4096, dtype="bf16"),
        # A small fp32 weight whose sides fit no tile.
        dict(name="mx4 quantize ragged f32", op="quant", rows=1000, cols=1056, dtype="f32"),
        # Serving one token through a merged gate/up projection: every weight is read once.
        dict(name="mx4 forward 1 token", op="mm", n=1, d_in=4096, d_out=14336, adjoint=False),
        # A few sequences decoded together, sides that fit no tile.
        dict(name="mx4 forward 17 ragged", op="mm", n=17, d_in=1056, d_out=1000, adjoint=False),
        # The attention projection of the training step of the benchmark.
        dict(name="mx4 forward 2048", op="mm", n=2048, d_in=4096, d_out=4096, adjoint=False),
        # The gate/up projection over a whole batch of prompts: the largest product.
        dict(name="mx4 forward 8192 up", op="mm", n=8192, d_in=4096, d_out=14336, adjoint=False),
        # The adjoint dX = dY W of a short ragged sequence, and of the training step.
        dict(name="mx4 adjoint 300 ragged", op="mm", n=300, d_in=1056, d_out=1000, adjoint=True),
        dict(name="mx4 adjoint 2048", op="mm", n=2048, d_in=4096, d_out=4096, adjoint=True),
        # One linear's packed theta with a norm and a bias: launch latency counts.
        dict(name="adamw e4m3 one linear", op="adamw", sizes="1044480,4096,4095,1", state="e4m3", pdt="f32",
             gdt="f32", seed=7),
        # theta_R and theta_P of the seven linears of all 32 blocks of an 8B model, in one step.
        dict(name="adamw e4m3 stack", op="adamw", sizes="+".join(["522240,522240,522240,130560,522240,130560,522240,"
             "522240,522240,1827840,522240,1827840,1827840,522240"] * 32), state="e4m3", pdt="f32", gdt="f32",
             seed=11),
        # One block's tensors with 32-bit moments.
        dict(name="adamw f32 block", op="adamw", sizes="522240,522240,522240,130560,522240,130560,522240,522240,"
             "522240,1827840,522240,1827840,1827840,522240", state="f32", pdt="f32", gdt="f32", seed=0),
        # Embedding and head rows and norms held in bf16 (stochastic rounding), odd sizes.
        dict(name="adamw bf16 odd", op="adamw", sizes="8388613,4096,255,257,5000001", state="e4m3", pdt="bf16",
             gdt="bf16", seed=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "mm", "mm", "adamw"])
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 14336), cols=BLK * _log(rng, 1, 448), dtype=rng.choice(["bf16", "f32"]))
    if op == "mm":
        d_in, d_out = BLK * _log(rng, 1, 448), 8 * _log(rng, 1, 1792)
        n = min(_log(rng, 1, 8192), 8192 * 4096 * 14336 // (d_in * d_out))  # no more than the largest listed
        return dict(op=op, n=n, d_in=d_in, d_out=d_out, adjoint=rng.random() < 0.5)
    state = rng.choice(["e4m3", "e4m3", "f32"])
    pdt = rng.choice(["f32", "f32", "bf16"])
    sizes = [_log(rng, 1, 1000000) for _ in range(_log(rng, 1, 448))]
    return dict(op=op, sizes=",".join(map(str, sizes)), state=state, pdt=pdt, gdt=rng.choice([pdt, "f32"]),
                seed=rng.randrange(1, 1 << 40) if state == "e4m3" else 0)


def _sizes(case):
    return [int(s) for s in case["sizes"].replace("+", ",").split(",")]


# --------------------------------------------------------------------------------- the inputs
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _weight(g, rows, cols):
    """A trained weight's spread: normal, some rows larger, some blocks zero (pruned columns)."""
    W = torch.randn(rows, cols, device=DEV, generator=g) * 0.02
    W *= torch.exp2(torch.randint(-2, 3, (rows, 1), device=DEV, generator=g).float())
    zero = torch.rand(rows, cols // BLK, device=DEV, generator=g) < 0.002
    return (W.view(rows, cols // BLK, BLK) * (~zero).unsqueeze(2)).view(rows, cols)


def _rows_of_tokens(g, n, d):
    """Activations after a norm: normal, with a few channels that stand out."""
    out = 1 + 15 * (torch.rand(1, d, device=DEV, generator=g) < 0.01).float()
    return (torch.randn(n, d, device=DEV, generator=g) * out).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "quant":
        rows, cols = case["rows"], case["cols"]
        return dict(case, W=_weight(g, rows, cols).to(_dt(case["dtype"])),
                    codes=torch.empty(rows, cols // 2, dtype=torch.uint8, device=DEV),
                    scales=torch.empty(rows, cols // BLK, dtype=torch.uint8, device=DEV),
                    back=torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV))
    if case["op"] == "mm":
        n, di, do = case["n"], case["d_in"], case["d_out"]
        codes, scales = _mx4_codes(_weight(g, do, di))
        k, m = (do, di) if case["adjoint"] else (di, do)
        return dict(case, codes=codes, scales=scales, X=_rows_of_tokens(g, n, k),
                    Y=torch.empty(n, m, dtype=torch.bfloat16, device=DEV))
    # All tensors are views of flat buffers, each starting on a block of 256 elements, as gradient
    # buckets hold them; the few elements between them stay zero.
    sizes = _sizes(case)
    nb = [(s + ABLK - 1) // ABLK for s in sizes]
    first = torch.tensor([0] + nb, dtype=torch.int64).cumsum(0)
    total = int(first[-1])
    at = torch.arange(total, device=DEV) - torch.repeat_interleave(first[:-1], torch.tensor(nb)).to(DEV)
    length = torch.repeat_interleave(torch.tensor(sizes), torch.tensor(nb)).to(DEV)
    tensor = torch.repeat_interleave(torch.arange(len(sizes)), torch.tensor(nb)).to(DEV)
    live = (at * ABLK).unsqueeze(1) + torch.arange(ABLK, device=DEV) < length.unsqueeze(1)
    scale = torch.exp2(torch.randint(-14, -8, (total, 1), device=DEV, generator=g).float())

    def normal(spread):
        return torch.randn(total, ABLK, device=DEV, generator=g).mul_(spread).mul_(live)

    s = dict(case, t=200, at=at, tensor=tensor, p=normal(0.005).to(_dt(case["pdt"])),
             g=normal(scale).to(_dt(case["gdt"])))
    m, r = normal(scale * 0.3), normal(scale).abs_()
    if case["state"] == "f32":
        s.update(m=m, v=r.square_())
    else:
        um, ur = m.abs().amax(1) / 448, r.amax(1) / 448
        s["scale"] = torch.stack([um, ur], 1).contiguous()
        s["m"] = (m / um.clamp_min(1e-30).unsqueeze(1)).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["v"] = (r / ur.clamp_min(1e-30).unsqueeze(1)).clamp_(2.0 ** -9, 448).mul_(live).to(torch.float8_e4m3fn)
    if "scale" not in s:
        s["scale"] = None
    del live, m, r
    # What a user's program keeps between steps: the tensors and, with the library, its optimiser.
    starts = [int(f) * ABLK for f in first[:-1]]
    s["tensors"] = [dict(p=s["p"].view(-1)[a:a + z], g=s["g"].view(-1)[a:a + z], m=s["m"].view(-1)[a:a + z],
                         v=s["v"].view(-1)[a:a + z],
                         scale=None if s["scale"] is None else s["scale"][a // ABLK:a // ABLK + (z + ABLK - 1) // ABLK])
                    for a, z in zip(starts, sizes)]
    s["kept"] = {}
    return s


def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))  # the settings are 32-bit numbers


def _corrections(t):
    return 1 - _f32(CFG["beta1"]) ** t, 1 - _f32(CFG["beta2"]) ** t


# ------------------------------------------------------------------------------ the plain forms
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx4_codes(W):
    """Codes [rows, cols / 2] and scales [rows, cols / 32] (uint8) of a weight, in exact steps."""
    rows, cols = W.shape
    w = W.float().view(rows, cols // BLK, BLK)
    amax = w.abs().amax(2)
    _, ex = torch.frexp(amax)                      # amax = f * 2^ex, f in [1/2, 1)
    e = torch.where(amax > 0, (ex - 3 + 127).clamp(0, 254), torch.zeros_like(ex))
    fine = torch.isfinite(w).all(2)
    e = torch.where(fine, e, torch.full_like(e, 255))
    y = torch.ldexp(w, (127 - e).unsqueeze(2))     # a power of two: exact
    a = y.abs()
    # Midpoints between neighbours; a tie goes to the even code.
    c = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = torch.where(fine.unsqueeze(2), c + 8 * torch.signbit(w).int(), torch.zeros_like(c)).view(rows, cols)
    return (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8), e.to(torch.uint8)


def _mx4_values(codes, scales, dtype=torch.float32):
    """The weight that codes and scales stand for."""
    c = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1).long()
    lut = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), dtype=dtype, device=codes.device)
    s = torch.ldexp(torch.ones_like(scales, dtype=dtype), scales.int() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return (lut[c].view(codes.shape[0], -1, BLK) * s.unsqueeze(2)).view(codes.shape[0], -1)


def _hash(at, tensor, seed):
    """The 32 random bits of every element (int64), from (seed, tensor, element)."""
    lo, hi = seed & M32, (seed >> 32) & M32
    salt = (lo + (tensor + 1) * 0xBB67AE85 + hi * 0x3C6EF373) & M32
    i = (at * ABLK).unsqueeze(1) + torch.arange(ABLK, device=at.device)
    h = ((i & M32) * 0x9E3779B1 + salt.unsqueeze(1) + (i >> 32) * 0x6A09E667) & M32
    h = ((h ^ (h >> 16)) * 0x6A09E667) & M32
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & M32
    return h ^ (h >> 16)


def _e4m3_stochastic(y, rnd):
    """e4m3 of y (|y| <= 448) from 16 random bits: up with the probability of the part below."""
    a = y.abs()
    normal = ((a.view(torch.int32) + (rnd << 4).int()) & ~0xFFFFF).view(torch.float32)
    small = torch.floor(a * 512 + rnd.float() * (1 / 65536)) * (1 / 512)
    q = torch.where(a < 2.0 ** -6, small, normal).clamp_max(448)
    return torch.where(torch.signbit(y), -q, q)


def _adamw_plain(s):
    c, f32 = CFG, torch.float32
    at, tensor = s["at"], s["tensor"]
    b1, b2 = (torch.tensor(c[k], dtype=f32, device=DEV) for k in ("beta1", "beta2"))
    g = s["g"].float()
    if s["state"] == "f32":
        m, v = s["m"], s["v"]
    else:
        m = s["m"].float() * s["scale"][:, :1]
        r = s["v"].float() * s["scale"][:, 1:]
        v = r * r
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    r = torch.sqrt(v)
    bc1, bc2 = _corrections(s["t"])
    p = s["p"].float()
    p = p - c["lr"] * c["gamma"] * (c["weight_decay"] * p + (m * (1 / bc1)) / (r * (1 / math.sqrt(bc2)) + c["eps"]))
    h = _hash(at, tensor, s["seed"]) if s["seed"] else None
    if s["pdt"] == "bf16" and s["seed"]:
        h2 = (h * 0xBB67AE85) & M32
        p = ((p.view(torch.int32) + (h2 >> 16).int()) & ~0xFFFF).view(f32)
    s["p"].copy_(p)
    if s["state"] == "f32":
        s["m"].copy_(m)
        s["v"].copy_(v)
        return
    for x, name, k in ((m, "m", 0), (r, "v", 1)):
        top = x.abs().amax(1, keepdim=True)
        top = torch.where(top < 2.0 ** -100, torch.zeros_like(top), top)
        y = torch.where(top > 0, x * (448 / top), torch.zeros_like(x)).clamp_(-448, 448)
        q = _e4m3_stochastic(y, (h & 0xFFFF) if k == 0 else h >> 16) if s["seed"] else y
        q = q.to(torch.float8_e4m3fn)
        if k == 1:
            q = torch.where(x > 0, q.float().clamp_min(2.0 ** -9), q.float()).to(torch.float8_e4m3fn)
        s[name].copy_(q)
        s["scale"][:, k] = top[:, 0] / 448


# ------------------------------------------------------------------------------------- one pass
def run(s):
    if s["op"] == "quant":
        if own:
            import orthogonal_equivalence_cnp_b200 as P
            P.poetx_mx4_quantize(P.POETX_BF16 if s["dtype"] == "bf16" else P.POETX_F32, s["rows"], s["cols"], s["W"],
                                 s["codes"], s["scales"])
            P.poetx_mx4_dequantize(s["rows"], s["cols"], s["codes"], s["scales"], s["back"])
            return dict(values=s["back"], scales=s["scales"])
        codes, scales = _mx4_codes(s["W"])
        return dict(values=_mx4_values(codes, scales).to(torch.bfloat16), scales=scales)
    if s["op"] == "mm":
        if own:
            import orthogonal_equivalence_cnp_b200 as P
            P.poetx_mx4_matmul(s["adjoint"], s["n"], s["d_in"], s["d_out"], s["X"], s["codes"], s["scales"], s["Y"])
            return s["Y"]
        W = _mx4_values(s["codes"], s["scales"])
        return (s["X"].float() @ (W if s["adjoint"] else W.t())).to(torch.bfloat16)
    if own:
        opt = s["kept"].get("opt")
        if opt is None:
            from orthogonal_equivalence_cnp_b200 import poetx_adamw_cfg
            from orthogonal_equivalence_cnp_b200.optim import AdamWTensor, MultiAdamW
            opt = s["kept"]["opt"] = MultiAdamW(
                [AdamWTensor(t["p"], t["g"], t["m"], t["v"], t["scale"]) for t in s["tensors"]])
            s["kept"]["cfg"] = poetx_adamw_cfg(*(CFG[k] for k in ("lr", "gamma", "beta1", "beta2", "eps", "weight_decay")))
        opt.step(s["kept"]["cfg"], t=s["t"], seed=s["seed"])
    else:
        _adamw_plain(s)
    return dict(p=s["p"], m=s["m"], v=s["v"], scale=s["scale"])


def work(case):
    if case["op"] == "quant":
        e = case["rows"] * case["cols"]
        return dict(bytes=e * ((2 if case["dtype"] == "bf16" else 4) + 2 + 2 * (0.5 + 1 / BLK)), flops=3.0 * e)
    if case["op"] == "mm":
        n, di, do = case["n"], case["d_in"], case["d_out"]
        return dict(bytes=di * do * (0.5 + 1 / BLK) + 2.0 * n * (di + do), flops=2.0 * n * di * do)
    e = sum(_sizes(case))
    per = 2 * (2 if case["pdt"] == "bf16" else 4) + (2 if case["gdt"] == "bf16" else 4)
    per += 16 if case["state"] == "f32" else 4 + 16 / ABLK
    return dict(bytes=per * e, flops=20.0 * e)


# -------------------------------------------------------------------------------- in 64 bits
def _mx4_exact(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1).int()
    mag, man = (c & 7) >> 1, (c & 1).double()
    val = torch.where(mag == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2(mag.double() - 1))
    val = torch.where(c >= 8, -val, val).view(codes.shape[0], -1, BLK)
    return (val * torch.exp2(scales.double() - 127).unsqueeze(2)).view(codes.shape[0], -1)


def _round_exact(a, step, rnd):
    return torch.floor(a / step + rnd / 65536.0) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        # The nearest of the grid's values, a tie to the even code, found by trying all eight.
        w = s["W"].double().view(case["rows"], -1, BLK)
        amax = w.abs().amax(2)
        e = torch.where(amax > 0, torch.floor(torch.log2(amax.clamp_min(1e-300))) - 2, torch.full_like(amax, -127.0))
        y = w.abs() * torch.exp2(-e).unsqueeze(2)
        best, dist = torch.zeros_like(y), y.clone()
        for i, x in enumerate(_E2M1[1:], 1):
            d = (y - x).abs()
            take = (d < dist) | ((d == dist) & (i % 2 == 0))
            best, dist = torch.where(take, torch.full_like(y, x), best), torch.where(take, d, dist)
        v = torch.where(w < 0, -best, best) * torch.exp2(e).unsqueeze(2)
        return dict(values=v.view(case["rows"], case["cols"]), scales=None)
    if case["op"] == "mm":
        W = _mx4_exact(s["codes"], s["scales"])
        return s["X"].double() @ (W if case["adjoint"] else W.t())
    c, step = CFG, 1 << 17  # blocks of 256 elements at a time
    bc1, bc2 = _corrections(s["t"])
    out = {k: [] for k in ("p", "m", "v", "scale")}
    b1, b2 = _f32(c["beta1"]), _f32(c["beta2"])
    for i in range(0, s["p"].shape[0], step):
        cut = slice(i, i + step)
        g, m, v, p = (s[k][cut].double() for k in ("g", "m", "v", "p"))
        if case["state"] == "e4m3":
            m = s["m"][cut].float().double() * s["scale"][cut, :1].double()
            v = (s["v"][cut].float().double() * s["scale"][cut, 1:].double()) ** 2
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        up = (m / bc1) / (torch.sqrt(v / bc2) + c["eps"])
        p = p - c["lr"] * c["gamma"] * (c["weight_decay"] * p + up)
        h = _hash(s["at"][cut], s["tensor"][cut], case["seed"]) if case["seed"] else None
        if case["pdt"] == "bf16" and case["seed"]:
            a = p.abs().clamp_min(1e-37)
            grid = torch.exp2(torch.floor(torch.log2(a)) - 7)
            a = _round_exact(a, grid, (((h * 0xBB67AE85) & M32) >> 16).double())
            p = torch.where(p == 0, p, torch.where(p < 0, -a, a))
        out["p"].append(p)
        if case["state"] == "f32":
            out["m"].append(m)
            out["v"].append(v)
            continue
        tops = []
        for x, name, rnd in ((m, "m", None if h is None else h & 0xFFFF), (torch.sqrt(v), "v", None if h is None else h >> 16)):
            top = x.abs().amax(1, keepdim=True)
            tops.append(top / 448)
            a = torch.where(top > 0, x.abs() * 448 / top.clamp_min(1e-300), torch.zeros_like(x)).clamp_max(448)
            grid = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
            q = _round_exact(a, grid, rnd.double()) if rnd is not None else torch.round(a / grid) * grid
            q = q.clamp_max(448)
            if name == "v":
                q = torch.where(x > 0, q.clamp_min(2.0 ** -9), q)
            out[name].append(torch.where(x < 0, -q, q))
        out["scale"].append(torch.cat(tops, 1))
    # Codes are whole steps of e4m3, compared as those; 32-bit results in 64 bits.
    return {k: torch.cat(x) if x else None for k, x in out.items()}
