"""Layer operators on the GPU against their definitions in 64 bits.

Bounds, element by element, from the arithmetic (u: half an ulp of the output
type relative to a value, 2^-8 bf16, 2^-11 fp16, 2^-24 fp32):
 - a product accumulates exact 16-bit products in FP32, at most 16 per step,
   each step within 2^-22 of the sum of the magnitudes:
   e = (K/16 + 2) 2^-22 sum |a b|;
 - activations have slopes of at most 1.13, their derivatives of at most 0.8
   (ReLU is tested where z is exact), and the fast exponential, division and
   erfc are within 2^-18 of |z| + 1;
 - a 16-bit intermediate of a backward pass contributes u of its magnitude
   through the product that reads it;
 - fp16 results below 2^-14 round to multiples of 2^-24.
"""
import numpy as np
import pytest
import torch

import quantized_tensor_activation_gb300 as qta
from quantized_tensor_activation_gb300 import layer
from gpu_util import device

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
FAST = 2.0 ** -18


@pytest.fixture(scope="module")
def dev():
    return device()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, rows, cols, dt, std=1.0, ld=None, fill=float("nan")):
    """[rows, cols] inside a buffer with `ld` elements between rows; what lies between holds `fill`."""
    ld = cols if ld is None else ld
    buf = torch.full((rows, ld), fill, dtype=DT[dt], device="cuda")
    buf[:, :cols] = (torch.randn(rows, cols, generator=g, device="cuda") * std).to(DT[dt])
    return buf[:, :cols]


def outbuf(rows, cols, dt, ld=None, pad=0):
    """An output view in a buffer of a canary value; check with canary_ok."""
    ld = cols if ld is None else ld
    buf = torch.full((rows * ld + 2 * pad,), 77.0, dtype=DT[dt], device="cuda")
    return buf, buf[pad:pad + rows * ld].view(rows, ld)[:, :cols]


def canary_ok(buf, view):
    n = int((buf == 77.0).sum())
    inside = int((view == 77.0).sum())
    return n - inside == buf.numel() - view.numel()


def check(name, got, ref, bound):
    got, ref, bound = got.double(), ref.double(), bound.double()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    bad = (got - ref).abs() > bound
    if bad.any():
        i = int(torch.argmax(((got - ref).abs() / (bound + 1e-300)).reshape(-1)))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} out of bounds; worst at {i}: "
                             f"{got.reshape(-1)[i].item()} against {ref.reshape(-1)[i].item()}, "
                             f"bound {bound.reshape(-1)[i].item()}")


def done():
    torch.cuda.synchronize()
    assert qta.qta_device_error() == 0


# ---------------------------------------------------------------- 64-bit definitions
def act64(z, act):
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if act == "gelu_erf":
        P = torch.special.erfc(-z / np.sqrt(2)) / 2
        return z * P, P + z * torch.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    k = np.sqrt(2 / np.pi)   # (1 + tanh q)/2 as 1/(1 + e^-2q): no cancellation for q << 0
    p = torch.sigmoid(2 * k * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * (1 - p) * 2 * k * (1 + 3 * 0.044715 * z * z)


def prod(a, b, K):
    """a b^T in 64 bits and the accumulation bound."""
    a, b = a.double(), b.double()
    return a @ b.T, (K / 16 + 2) * 2.0 ** -22 * (a.abs() @ b.abs().T)


# ---------------------------------------------------------------- norm
NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (2, 33), (5, 250), (4, 256), (7, 1000), (3, 1024), (2, 4096), (2, 4109), (3, 5120),
               (2, 8192), (1, 8199), (2, 16384), (1, 40000), (700, 264),
               # all rows at once, several in a CTA
               (153, 4096), (305, 1116), (423, 1115), (200, 2441)]


def norm64(x, r, g, b, kind, eps):
    s = x.double() if r is None else x.double() + r.double()
    if kind == "layer":
        m = s.mean(1, keepdim=True)
        c = s - m
    else:
        m, c = None, s
    rs = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    xh = c * rs
    y = xh * g.double()
    if b is not None:
        y = y + b.double()
    return s, m, rs, xh, y


@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "fp32")])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("R,C", NORM_SHAPES)
def test_norm(dev, R, C, kind, dt, wdt):
    g = gen(R * 1000 + C)
    for res in (False, True):
        x, r = rand(g, R, C, dt, 2.0), rand(g, R, C, dt) if res else None
        if R > 1:
            x[0] = 0   # a padding token: nothing in it
            if res:
                r[0] = 0
        ga = 1 + 0.1 * rand(g, 1, C, wdt)[0]
        be = rand(g, 1, C, wdt)[0] if kind == "layer" else None
        yb, y = outbuf(R, C, dt, pad=8)
        sb, s = outbuf(R, C, dt, pad=8)
        mb, mean = outbuf(1, R, "fp32", pad=4)
        rb, rstd = outbuf(1, R, "fp32", pad=4)
        d = qta.norm_desc(R, C, dt, kind, 1e-5, wdt)
        qta.qta_norm(d, x, ga, y, beta=be, residual=r, sum_out=s, mean=mean[0] if kind == "layer" else None,
                     rstd=rstd[0])
        done()
        s64, m64, rs64, xh64, y64 = norm64(x, r, ga, be, kind, 1e-5)
        # sums of C terms in a tree of at most C/32 + 10 roundings
        e = (C / 32 + 12) * 2.0 ** -24
        mag = s64.abs().mean(1, keepdim=True)
        em = e * mag + 2.0 ** -24 * mag if kind == "layer" else torch.zeros_like(mag)
        # the centred values are off by em and a rounding of s, so rstd by about their share of the row's spread
        spread = 1 / rs64
        ers = (2 * e + 2.0 ** -21 + (em + 2.0 ** -23 * mag) / spread) * rs64
        if kind == "layer":
            check("mean", mean.T, m64, em + 2.0 ** -24 * m64.abs())
        check("rstd", rstd.T, rs64, ers)
        check("sum", s, s64, U[dt] * s64.abs() * 1.001 + TINY[dt])
        ey = ga.double().abs() * ((em + 2.0 ** -23 * s64.abs()) * rs64 + xh64.abs() * (ers / rs64 + 2.0 ** -21))
        check("y", y, y64, ey * 1.01 + U[dt] * (y64.abs() + ey) + 2.0 ** -23 * y64.abs() + TINY[dt])
        assert canary_ok(yb, y) and canary_ok(sb, s) and canary_ok(mb, mean) and canary_ok(rb, rstd)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("R,C", NORM_SHAPES + [(1021, 1000), (300, 4109), (257, 8192)])
def test_norm_bwd(dev, R, C, kind, dt):
    g = gen(R * 77 + C)
    for res in (False, True):
        s, dy = rand(g, R, C, dt, 2.0), rand(g, R, C, dt, 0.1)
        ds = rand(g, R, C, dt, 0.1) if res else None
        ga = 1 + 0.1 * rand(g, 1, C, dt)[0]
        _, m64, rs64, xh, _ = norm64(s, None, ga, None, kind, 1e-5)
        mean = m64[:, 0].float() if kind == "layer" else None
        rstd = rs64[:, 0].float()
        db_, dx = outbuf(R, C, dt, pad=8)
        gb, dg = outbuf(1, C, "fp32", pad=4)
        bb, db = outbuf(1, C, "fp32", pad=4)
        d = qta.norm_desc(R, C, dt, kind)
        ws = qta.alloc_workspace(qta.norm_bwd_workspace_bytes(d))
        qta.qta_norm_bwd(d, dy, s, ga, rstd, dx, dg[0], ws, mean=mean, dbeta=db[0] if kind == "layer" else None,
                         dsum=ds)
        done()
        # mean and rstd are inputs here, in 32 bits
        rs = rstd.double()[:, None]
        xh = (s.double() - (mean.double()[:, None] if mean is not None else 0)) * rs
        exh = 2.0 ** -23 * (xh.abs() + (s.double().abs() + (m64.abs() if m64 is not None else 0)) * rs)
        t = dy.double() * ga.double()
        mt = t.mean(1, keepdim=True) if kind == "layer" else 0 * rs
        mtx = (t * xh).mean(1, keepdim=True)
        dx64 = rs * (t - mt - xh * mtx) + (ds.double() if res else 0)
        e = (C / 32 + 12) * 2.0 ** -24
        emt = e * t.abs().mean(1, keepdim=True)
        emtx = e * (t * xh).abs().mean(1, keepdim=True) + (t.abs() * exh).mean(1, keepdim=True)
        edx = rs * (emt + xh.abs() * emtx + exh * mtx.abs() + 2.0 ** -22 * (t.abs() + mt.abs() + (xh * mtx).abs()))
        if res:
            edx = edx + 2.0 ** -23 * (ds.double().abs() + dx64.abs())
        check("dx", dx, dx64, edx * 1.01 + U[dt] * (dx64.abs() + edx) + TINY[dt])
        # column sums of R terms, each partial sum within R + 8 roundings of the magnitudes
        eg = (R + 8) * 2.0 ** -24
        col = (dy.double() * xh)
        check("dgamma", dg, col.sum(0, keepdim=True),
              eg * col.abs().sum(0, keepdim=True) + (dy.double().abs() * exh).sum(0, keepdim=True))
        if kind == "layer":
            check("dbeta", db, dy.double().sum(0, keepdim=True), eg * dy.double().abs().sum(0, keepdim=True))
        assert canary_ok(db_, dx) and canary_ok(gb, dg) and (kind == "rms" or canary_ok(bb, db))


# ---------------------------------------------------------------- linear
LIN_SHAPES = [  # rows, n_out, n_in
    (1, 8, 8), (1, 129, 64), (2, 64, 72), (3, 1000, 200), (6, 264, 520), (8, 8, 1096), (9, 128, 128), (16, 256, 64),
    (17, 200, 136), (31, 72, 2056), (33, 65, 64), (64, 128, 192), (127, 129, 264), (128, 128, 64), (129, 384, 72),
    (300, 344, 1024), (257, 513, 328), (1, 4096, 4096), (5, 2048, 4104), (1000, 40, 40),
    # more 128 x 128 tiles than SMs: pairs of CTAs, several tiles each, ragged ends, one contraction block, one column block
    (1700, 1800, 1504), (1701, 1801, 1496), (2049, 2312, 520), (5000, 600, 8), (20001, 8, 64), (24, 136, 2048),
    (32, 1000, 2056), (70, 1000, 4104), (500, 1100, 2056)]
ACTS = ["none", "relu", "silu", "gelu_tanh", "gelu_erf"]


@pytest.mark.parametrize("dt,odt,bdt", [("bf16", "bf16", "bf16"), ("fp16", "fp16", "fp16"), ("bf16", "fp32", "fp32"),
                                        ("fp16", "fp32", "fp16")])
@pytest.mark.parametrize("R,N,K", LIN_SHAPES)
def test_linear(dev, R, N, K, dt, odt, bdt):
    g = gen(R + 31 * N + 7 * K)
    for i, act in enumerate(ACTS):
        x, w = rand(g, R, K, dt), rand(g, N, K, dt, K ** -0.5)
        b = rand(g, 1, N, bdt)[0] if i % 2 == 0 else None
        r = rand(g, R, N, odt) if i % 3 != 1 else None
        yb, y = outbuf(R, N, odt, pad=8)
        qta.qta_linear(qta.linear_desc(R, N, K, dt, act, odt, bdt), x, w, y, bias=b, residual=r)
        done()
        z, e = prod(x, w, K)
        if b is not None:
            z = z + b.double()
            e = e + 2.0 ** -24 * z.abs()
        f, _ = act64(z, act)
        e = 1.13 * e + (0 if act in ("none", "relu") else FAST * (z.abs() + 1))
        y64 = f if r is None else f + r.double()
        check(act, y, y64, e * 1.01 + (U[odt] + 2.0 ** -24) * (y64.abs() + e) + TINY[odt])
        assert canary_ok(yb, y)


def bwd_bounds(dy, z, ez, act, dt):
    """dz in 64 bits, its bound before and after the rounding to dt."""
    _, df = act64(z, act)
    dz = dy.double() * df
    e = dy.double().abs() * (0.0 if act in ("none", "relu") else 1.0) * (0.8 * ez + FAST * (z.abs() + 1))
    e = e + 2.0 ** -23 * dz.abs()
    if act == "none":
        return dz, torch.zeros_like(dz), torch.zeros_like(dz)
    return dz, e, e + U[dt] * (dz.abs() + e) + TINY[dt]


def int_rand(g, rows, cols, dt):
    return torch.randint(-3, 4, (rows, cols), generator=g, device="cuda").to(DT[dt])


@pytest.mark.parametrize("dt,gdt", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32")])
@pytest.mark.parametrize("R,N,K", LIN_SHAPES)
def test_linear_bwd(dev, R, N, K, dt, gdt):
    g = gen(3 * R + 5 * N + K)
    N8 = (N + 7) // 8 * 8
    for i, act in enumerate(ACTS):
        if act == "relu":   # whole numbers: z is exact, and so is its sign
            x, w = int_rand(g, R, K, dt), int_rand(g, N, K, dt)
        else:
            x, w = rand(g, R, K, dt), rand(g, N, K, dt, K ** -0.5)
        b = rand(g, 1, N, dt)[0] if i % 2 == 0 else None
        dy = rand(g, R, N, dt, 0.1, ld=N8)
        dxb, dx = outbuf(R, K, dt, pad=8)
        dwb, dw = outbuf(N, K, gdt, pad=8)
        dbb, db = outbuf(1, N, "fp32", pad=4)
        d = qta.linear_desc(R, N, K, dt, act, grad_dtype=gdt)
        ws = qta.alloc_workspace(qta.linear_bwd_workspace_bytes(d))
        qta.qta_linear_bwd(d, dy, x, w, dx, dw, ws, bias=b, dbias=db[0])
        done()
        z, ez = prod(x, w, K)
        if b is not None:
            z = z + b.double()
            ez = ez + 2.0 ** -24 * z.abs()
        dz, e32, e16 = bwd_bounds(dy, z, ez, act, dt)
        dx64, ea = prod(dz, w.T, N)
        e = ea + e16 @ w.double().abs()
        check(act + " dx", dx, dx64, e * 1.01 + U[dt] * (dx64.abs() + e) + TINY[dt])
        dw64, ea = prod(dz.T, x.T, R)
        e = ea + e16.T @ x.double().abs()
        check(act + " dw", dw, dw64, e * 1.01 + U[gdt] * (dw64.abs() + e) + TINY[gdt])
        eb = (R + 8) * 2.0 ** -24 * dz.abs().sum(0, keepdim=True) + e32.sum(0, keepdim=True)
        check(act + " dbias", db, dz.sum(0, keepdim=True), eb)
        assert canary_ok(dxb, dx) and canary_ok(dwb, dw) and canary_ok(dbb, db)


# ---------------------------------------------------------------- gated feed-forward
FFN_SHAPES = [  # rows, hidden, width
    (1, 8, 8), (1, 520, 65), (2, 72, 64), (6, 5120, 3456), (9, 64, 136), (16, 256, 264), (17, 1000, 72), (40, 136, 200),
    (128, 64, 64), (129, 328, 130), (300, 1024, 344), (1, 4096, 1024), (24, 512, 1000), (32, 2056, 72),
    (1300, 1904, 904), (1281, 2000, 901), (10001, 64, 72), (12, 4104, 200), (24, 1032, 264), (70, 2056, 1000)]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("R,H,F", FFN_SHAPES)
def test_gated_ffn(dev, R, H, F, dt):
    g = gen(R + H + 3 * F)
    for act in ACTS:
        x, wg, wu = rand(g, R, H, dt), rand(g, F, H, dt, H ** -0.5), rand(g, F, H, dt, H ** -0.5)
        hb, h = outbuf(R, F, dt, pad=8)
        qta.qta_gated_ffn(qta.ffn_desc(R, H, F, dt, act), x, wg, wu, h)
        done()
        (gz, eg), (u, eu) = prod(x, wg, H), prod(x, wu, H)
        f, _ = act64(gz, act)
        ef = 1.13 * eg + (0 if act in ("none", "relu") else FAST * (gz.abs() + 1))
        h64 = f * u
        e = f.abs() * eu + u.abs() * ef + ef * eu
        check(act, h, h64, e * 1.01 + (U[dt] + 2.0 ** -23) * (h64.abs() + e) + TINY[dt])
        assert canary_ok(hb, h)


@pytest.mark.parametrize("dt,gdt", [("bf16", "bf16"), ("fp16", "fp16"), ("fp16", "fp32")])
@pytest.mark.parametrize("R,H,F", FFN_SHAPES)
def test_gated_ffn_bwd(dev, R, H, F, dt, gdt):
    g = gen(R + 2 * H + F)
    F8 = (F + 7) // 8 * 8
    for act in ACTS:
        if act == "relu":
            x, wg, wu = int_rand(g, R, H, dt), int_rand(g, F, H, dt), int_rand(g, F, H, dt)
            dh = rand(g, R, F, dt, 1e-3, ld=F8)
        else:
            x, wg, wu = rand(g, R, H, dt), rand(g, F, H, dt, H ** -0.5), rand(g, F, H, dt, H ** -0.5)
            dh = rand(g, R, F, dt, 0.1, ld=F8)
        dxb, dx = outbuf(R, H, dt, pad=8)
        dgb, dwg = outbuf(F, H, gdt, pad=8)
        dub, dwu = outbuf(F, H, gdt, pad=8)
        d = qta.ffn_desc(R, H, F, dt, act, gdt)
        ws = qta.alloc_workspace(qta.gated_ffn_bwd_workspace_bytes(d))
        qta.qta_gated_ffn_bwd(d, dh, x, wg, wu, dx, dwg, dwu, ws)
        done()
        (gz, eg), (u, eu) = prod(x, wg, H), prod(x, wu, H)
        f, df = act64(gz, act)
        a = dh.double().abs()
        smooth = 0.0 if act in ("none", "relu") else 1.0
        ef = 1.13 * eg + smooth * FAST * (gz.abs() + 1)
        edf = smooth * (0.8 * eg + FAST * (gz.abs() + 1))
        dg, du = dh.double() * u * df, dh.double() * f
        edg = a * (u.abs() * edf + df.abs() * eu + edf * eu)
        edu = a * ef
        edg = edg * 1.01 + (U[dt] + 2.0 ** -22) * (dg.abs() + edg) + TINY[dt]
        edu = edu * 1.01 + (U[dt] + 2.0 ** -22) * (du.abs() + edu) + TINY[dt]
        dx64 = dg @ wg.double() + du @ wu.double()
        e = (2 * F / 16 + 4) * 2.0 ** -22 * (dg.abs() @ wg.double().abs() + du.abs() @ wu.double().abs())
        e = e + edg @ wg.double().abs() + edu @ wu.double().abs()
        check(act + " dx", dx, dx64, e * 1.01 + U[dt] * (dx64.abs() + e) + TINY[dt])
        for name, m, em, got in (("dwg", dg, edg, dwg), ("dwu", du, edu, dwu)):
            ref, ea = prod(m.T, x.T, R)
            e = ea + em.T @ x.double().abs()
            check(act + " " + name, got, ref, e * 1.01 + U[gdt] * (ref.abs() + e) + TINY[gdt])
        assert canary_ok(dxb, dx) and canary_ok(dgb, dwg) and canary_ok(dub, dwu)


# ---------------------------------------------------------------- strides, aliases, non-finite values
def test_strided_matrices(dev):
    g = gen(5)
    R, N, K = 70, 203, 200
    x, w = rand(g, R, K, "bf16", ld=224), rand(g, N, K, "bf16", K ** -0.5, ld=208)   # NaN between the rows
    r = rand(g, R, N, "bf16", ld=211)
    yb, y = outbuf(R, N, "bf16", ld=205, pad=8)
    qta.qta_linear(qta.linear_desc(R, N, K, "bf16"), x, w, y, residual=r)
    done()
    z, e = prod(x, w, K)
    ref = z + r.double()
    check("y", y, ref, e * 1.01 + U["bf16"] * (ref.abs() + e) + 2.0 ** -23 * ref.abs())
    assert canary_ok(yb, y)
    # odd contraction lengths in padded rows, both directions, few and many rows
    for R in (2, 70):
        x, w = rand(g, R, 77, "fp16", ld=80), rand(g, 53, 77, "fp16", 0.1, ld=88)
        yb, y = outbuf(R, 53, "fp16", ld=64, pad=8)
        qta.qta_linear(qta.linear_desc(R, 53, 77, "fp16"), x, w, y)
        dy = rand(g, R, 53, "fp16", 0.1, ld=56)
        dxb, dx = outbuf(R, 77, "fp16", ld=81, pad=8)
        dwb, dw = outbuf(53, 77, "fp16", ld=79, pad=8)
        d = qta.linear_desc(R, 53, 77, "fp16")
        ws = qta.alloc_workspace(qta.linear_bwd_workspace_bytes(d))
        qta.qta_linear_bwd(d, dy, x, w, dx, dw, ws)
        done()
        for got, (ref, e) in ((y, prod(x, w, 77)), (dx, prod(dy, w.T, 53)), (dw, prod(dy.T, x.T, R))):
            check("odd", got, ref, e * 1.01 + U["fp16"] * (ref.abs() + e) + TINY["fp16"])
        assert canary_ok(yb, y) and canary_ok(dxb, dx) and canary_ok(dwb, dw)
    # two column slices of one buffer: gate and up projections stored side by side
    wgu = rand(g, 96, 2 * 128, "bf16", 0.1)
    x = rand(g, 33, 128, "bf16")
    hb, h = outbuf(33, 96, "bf16", ld=104)
    qta.qta_gated_ffn(qta.ffn_desc(33, 128, 96, "bf16"), x, wgu[:, :128], wgu[:, 128:], h)
    done()
    (gz, eg), (u, eu) = prod(x, wgu[:, :128], 128), prod(x, wgu[:, 128:], 128)
    f, _ = act64(gz, "silu")
    ef = 1.13 * eg + FAST * (gz.abs() + 1)
    e = f.abs() * eu + u.abs() * ef + ef * eu
    check("h", h, f * u, e * 1.01 + (U["bf16"] + 2.0 ** -23) * ((f * u).abs() + e))
    assert canary_ok(hb, h)


@pytest.mark.parametrize("off", [0, 1, 3])
def test_norm_strides_and_offsets(dev, off):
    """Rows that start anywhere: base offsets and row distances off every vector boundary."""
    g = gen(9)
    for R, C, lds in ((5, 1000, (1001, 1000, 1003, 1007)), (3, 4096, (4104, 4104, 4104, 4104)),
                      (4, 333, (340, 333, 350, 334))):
        def view(ld, dt="bf16"):
            b = torch.full((off + R * ld + 8,), float("nan"), dtype=DT[dt], device="cuda")
            return b, b[off:off + R * ld].view(R, ld)[:, :C]
        _, x = view(lds[0])
        _, r = view(lds[1])
        x.copy_(torch.randn(R, C, generator=g, device="cuda"))
        r.copy_(torch.randn(R, C, generator=g, device="cuda"))
        yb, y = view(lds[2])
        sb, s = view(lds[3])
        wb = torch.randn(2 * C + 2 * off, generator=g, device="cuda").bfloat16()
        ga, be = wb[off:off + C], wb[off + C:off + 2 * C]
        d = qta.norm_desc(R, C, "bf16")
        mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
        qta.qta_norm(d, x, ga, y, beta=be, residual=r, sum_out=s, mean=mean, rstd=rstd)
        done()
        s64, m64, rs64, xh64, y64 = norm64(x, r, ga, be, "layer", 1e-5)
        check("sum", s, s64, U["bf16"] * s64.abs() * 1.001)
        check("y", y, y64, U["bf16"] * y64.abs() * 1.001 + 1e-5 * (1 + ga.double().abs() * (1 + xh64.abs())))
        assert int(torch.isfinite(yb).sum()) == R * C and int(torch.isfinite(sb).sum()) == R * C
        dxb, dx = view(lds[2])
        dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
        ws = qta.alloc_workspace(qta.norm_bwd_workspace_bytes(d))
        qta.qta_norm_bwd(d, r, s, ga, rstd, dx, dg, ws, mean=mean, dbeta=db, dsum=x)
        done()
        rs, sm = rstd.double()[:, None], s.double()
        xh = (sm - mean.double()[:, None]) * rs
        t = r.double() * ga.double()
        ref = rs * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True)) + x.double()
        check("dx", dx, ref, U["bf16"] * ref.abs() * 1.001 + 2e-5 * (1 + t.abs() + xh.abs()) * (1 + rs))
        assert int(torch.isfinite(dxb).sum()) == R * C
        check("dgamma", dg, (r.double() * xh).sum(0), 1e-5 * (1 + (r.double() * xh).abs().sum(0)))
        check("dbeta", db, r.double().sum(0), 1e-5 * (1 + r.double().abs().sum(0)))


def test_linear_residual_in_place(dev):
    g = gen(6)
    for R in (1, 5, 200):
        x, w, r = rand(g, R, 256, "bf16"), rand(g, 264, 256, "bf16", 1 / 16), rand(g, R, 264, "bf16")
        y, a = torch.empty_like(r), r.clone()
        d = qta.linear_desc(R, 264, 256, "bf16")
        qta.qta_linear(d, x, w, y, residual=r)
        qta.qta_linear(d, x, w, a, residual=a)
        done()
        assert torch.equal(y, a)


@pytest.mark.parametrize("R", [3, 150])
def test_non_finite_values_stay_in_their_rows(dev, R):
    g = gen(7)
    x, w = rand(g, R, 136, "bf16"), rand(g, 72, 136, "bf16", 0.1)
    y, y2 = torch.empty(R, 72, dtype=torch.bfloat16, device="cuda"), torch.empty(R, 72, dtype=torch.bfloat16, device="cuda")
    d = qta.linear_desc(R, 72, 136, "bf16")
    qta.qta_linear(d, x, w, y)
    x2, w2 = x.clone(), w.clone()
    x2[1, 7] = float("nan")
    x2[2, 100] = float("inf")
    w2[5, 3] = float("-inf")
    qta.qta_linear(d, x2, w2, y2)
    done()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1] = keep[2] = False
    keep[:, 5] = False
    assert torch.equal(y[keep], y2[keep])
    assert torch.isnan(y2[1]).all() and not torch.isfinite(y2[2]).any() and not torch.isfinite(y2[:, 5]).any()
    # norm: a NaN spoils its own row only
    s = torch.empty(R, 136, dtype=torch.bfloat16, device="cuda")
    yn, yn2 = torch.empty_like(s), torch.empty_like(s)
    ga = torch.ones(136, dtype=torch.bfloat16, device="cuda")
    dn = qta.norm_desc(R, 136, "bf16")
    qta.qta_norm(dn, x, ga, yn)
    qta.qta_norm(dn, x2, ga, yn2)
    done()
    assert torch.isnan(yn2[1]).all() and torch.isnan(yn2[2]).all()
    assert torch.equal(yn[0], yn2[0]) and torch.equal(yn[3:], yn2[3:])


def test_activation_tails(dev):
    """Large arguments: no overflow, no cancellation where GELU and SiLU vanish."""
    z = torch.tensor([-1e4, -300.0, -100.0, -40.0, -9.0, -5.0, -1.0, -0.0, 0.0, 1e-4, 1.0, 5.0, 9.0, 100.0, 1e4, 3e4],
                     device="cuda")
    R = z.numel()
    x = torch.zeros(R, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = z.bfloat16()
    w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1
    zz = x[:, :1].double().expand(R, 8)
    for act in ACTS:
        y = torch.empty(R, 8, dtype=torch.float32, device="cuda")
        qta.qta_linear(qta.linear_desc(R, 8, 8, "bf16", act, out_dtype="fp32"), x, w, y)
        dy = torch.ones(R, 8, dtype=torch.bfloat16, device="cuda")
        d = qta.linear_desc(R, 8, 8, "bf16", act, grad_dtype="fp32")
        ws = qta.alloc_workspace(qta.linear_bwd_workspace_bytes(d))
        dx = torch.empty(R, 8, dtype=torch.bfloat16, device="cuda")
        qta.qta_linear_bwd(d, dy, x, w, dx, None, ws)
        done()
        f, df = act64(zz, act)
        # the exponentials keep their relative accuracy: an exponent E is off by at most E 2^-21 (its own roundings and
        # the fast exponential's E ulp); results below 2^-126 may be flushed
        E = {"gelu_tanh": 1.6 * zz.abs() + 0.0714 * zz.abs() ** 3, "gelu_erf": zz * zz / 2}.get(act, zz.abs())
        rel = 2.0 ** -17 + E.clamp(max=100) * 2.0 ** -21
        check(act, y, f, rel * f.abs() + 1e-37)
        ref = 8 * df[:, :1].expand(R, 8).clone()
        ref[:, 1:] = 0
        check(act + "'", dx, ref, (2.0 ** -7 + 16 * rel) * ref.abs() + 2.0 ** -17 * (zz.abs() < 50) + 1e-36)


def test_gradients_against_differences(dev):
    """The backward calls against central differences of the forward calls (FP32 outputs)."""
    g = gen(8)
    R, N, K = 24, 40, 48
    for act in ("silu", "gelu_tanh", "gelu_erf"):
        x, w, b = rand(g, R, K, "fp16"), rand(g, N, K, "fp16", K ** -0.5), rand(g, 1, N, "fp32")[0]
        dy = rand(g, R, N, "fp16")
        d = qta.linear_desc(R, N, K, "fp16", act, out_dtype="fp32", bias_dtype="fp32", grad_dtype="fp32")
        dx, dw = torch.empty_like(x), torch.empty(N, K, device="cuda")
        db = torch.empty(N, device="cuda")
        ws = qta.alloc_workspace(qta.linear_bwd_workspace_bytes(d))
        qta.qta_linear_bwd(d, dy, x, w, dx, dw, ws, bias=b, dbias=db)
        # along a random direction of every argument, steps that fp16 holds exactly
        vx = torch.randint(-1, 2, x.shape, generator=g, device="cuda").half() * 2 ** -4
        vw = torch.randint(-1, 2, w.shape, generator=g, device="cuda").half() * 2 ** -6
        vb = torch.randint(-1, 2, b.shape, generator=g, device="cuda").float() * 2 ** -4
        x0 = (x * 16).round() / 16
        w0 = (w * 64).round() / 64
        qta.qta_linear_bwd(d, dy, x0, w0, dx, dw, ws, bias=b, dbias=db)
        yp, ym = torch.empty(R, N, device="cuda"), torch.empty(R, N, device="cuda")
        for name, args_p, args_m, an in (
                ("x", (x0 + vx, w0, b), (x0 - vx, w0, b), (dx.double() * vx.double()).sum()),
                ("w", (x0, w0 + vw, b), (x0, w0 - vw, b), (dw.double() * vw.double()).sum()),
                ("b", (x0, w0, b + vb), (x0, w0, b - vb), (db.double() * vb.double()).sum())):
            qta.qta_linear(d, args_p[0], args_p[1], yp, bias=args_p[2])
            qta.qta_linear(d, args_m[0], args_m[1], ym, bias=args_m[2])
            done()
            num = ((yp.double() - ym.double()) / 2 * dy.double()).sum()
            # third-order term of the difference: |f'''| <= 2, |step of z| <= 48 * 2^-4 in x (3 sigma about 0.5)
            dz = {"x": (vx.double().abs() @ w0.double().abs().T), "w": (x0.double().abs() @ vw.double().abs().T),
                  "b": vb.double().abs()[None].expand(R, N)}[name]
            bound = (dy.double().abs() * (dz ** 3) / 3).sum() + 2.0 ** -10 * (dy.double().abs() * dz).sum()
            assert abs(num - an) <= bound, (act, name, num.item(), an.item(), bound.item())


# ---------------------------------------------------------------- empty, repeated, other streams, long offsets
def test_empty_batches(dev):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(16, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    d = qta.linear_desc(0, 16, 64, "bf16", "silu")
    qta.qta_linear(d, x, w, y)
    dw, db = torch.full((16, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((16,), 3.0, device="cuda")
    ws = qta.alloc_workspace(qta.linear_bwd_workspace_bytes(d))
    qta.qta_linear_bwd(d, y, x, w, x, dw, ws, dbias=db)
    f = qta.ffn_desc(0, 64, 16, "bf16")
    qta.qta_gated_ffn(f, x, w, w, y)
    dwg = torch.full((16, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    dwu = torch.full((16, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    qta.qta_gated_ffn_bwd(f, y, x, w, w, x, dwg, dwu, qta.alloc_workspace(qta.gated_ffn_bwd_workspace_bytes(f)))
    n = qta.norm_desc(0, 64, "bf16")
    e = torch.empty(0, device="cuda")
    qta.qta_norm(n, x, w[0], x, mean=e, rstd=e)
    dg, dbt = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    qta.qta_norm_bwd(n, x, x, w[0], e, x, dg, qta.alloc_workspace(qta.norm_bwd_workspace_bytes(n)), mean=e, dbeta=dbt)
    done()
    for t in (dw, db, dwg, dwu, dg, dbt):
        assert not t.any()


def test_partial_gradients(dev):
    """A gradient that is not asked for is not computed, and the others do not change."""
    g = gen(11)
    R, N, K = 140, 136, 200
    x, w, dy = rand(g, R, K, "bf16"), rand(g, N, K, "bf16", 0.1), rand(g, R, N, "bf16")
    for act in ("none", "silu"):
        d = qta.linear_desc(R, N, K, "bf16", act)
        ws = qta.alloc_workspace(qta.linear_bwd_workspace_bytes(d))
        full = [torch.empty(R, K, dtype=torch.bfloat16, device="cuda"),
                torch.empty(N, K, dtype=torch.bfloat16, device="cuda"), torch.empty(N, device="cuda")]
        qta.qta_linear_bwd(d, dy, x, w, full[0], full[1], ws, dbias=full[2])
        for keep in range(3):
            part = [torch.empty_like(t) if i == keep else None for i, t in enumerate(full)]
            qta.qta_linear_bwd(d, dy, x, w, part[0], part[1], ws, dbias=part[2])
            done()
            assert torch.equal(part[keep], full[keep])
    f = qta.ffn_desc(R, K, N, "bf16")
    wu = rand(g, N, K, "bf16", 0.1)
    ws = qta.alloc_workspace(qta.gated_ffn_bwd_workspace_bytes(f))
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    qta.qta_gated_ffn_bwd(f, dy, x, w, wu, dx, dwg, dwu, ws)
    dx2, dwg2, dwu2 = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    qta.qta_gated_ffn_bwd(f, dy, x, w, wu, dx2, None, None, ws)
    qta.qta_gated_ffn_bwd(f, dy, x, w, wu, None, dwg2, dwu2, ws)
    done()
    assert torch.equal(dx, dx2) and torch.equal(dwg, dwg2) and torch.equal(dwu, dwu2)


def test_repeatable_and_stream_ordered(dev):
    """The same bits on every call, on another stream too, with the inputs made on that stream just before."""
    g = gen(12)
    R, H, F = 700, 512, 392
    base = [rand(g, R, H, "bf16"), rand(g, F, H, "bf16", 0.05), rand(g, F, H, "bf16", 0.05), rand(g, R, F, "bf16")]

    def step(scale, stream):
        with torch.cuda.stream(stream):
            x, wg, wu, dh = [(t * scale) for t in base]
            out = [torch.empty(R, F, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x), torch.empty_like(wg),
                   torch.empty_like(wu), torch.empty_like(x), torch.empty(H, device="cuda"),
                   torch.empty(H, device="cuda"), torch.empty(R, device="cuda"), torch.empty(R, device="cuda")]
            f = qta.ffn_desc(R, H, F, "bf16")
            ws = qta.alloc_workspace(qta.gated_ffn_bwd_workspace_bytes(f))
            qta.qta_gated_ffn(f, x, wg, wu, out[0], stream=stream)
            qta.qta_gated_ffn_bwd(f, dh, x, wg, wu, out[1], out[2], out[3], ws, stream=stream)
            n = qta.norm_desc(R, H, "bf16")
            nws = qta.alloc_workspace(qta.norm_bwd_workspace_bytes(n))
            qta.qta_norm(n, x, wg[0], out[4], beta=wu[0], mean=out[7], rstd=out[8], stream=stream)
            qta.qta_norm_bwd(n, x, x, wg[0], out[8], out[4], out[5], nws, mean=out[7], dbeta=out[6], stream=stream)
        return out

    a = step(1.0, torch.cuda.current_stream())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        b = step(1.0, side)
        c = step(1.0, torch.cuda.current_stream())
        done()
        for p, q, r in zip(a, b, c):
            assert torch.equal(p, q) and torch.equal(p, r)


def test_row_offsets_past_32_bits(dev):
    """Rows further apart than 2^31 elements in all."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    g = gen(13)
    ld = (1 << 30) + 8
    buf = torch.empty(2 * ld + 256, dtype=torch.bfloat16, device="cuda")

    def far(cols, at=0):
        return buf.as_strided((3, cols), (ld, 1), at)

    x, w = far(64), rand(g, 72, 64, "bf16", 0.1)
    x.copy_(torch.randn(3, 64, generator=g, device="cuda"))
    y = far(72, 64)
    qta.qta_linear(qta.linear_desc(3, 72, 64, "bf16"), x, w, y)
    done()
    z, e = prod(x, w, 64)
    check("y", y, z, e * 1.01 + U["bf16"] * (z.abs() + e))
    wide = rand(g, 200, 64, "bf16")
    d = qta.linear_desc(3, 72, 64, "bf16", "silu")
    dx, dw = far(64, 136), torch.empty(72, 64, dtype=torch.bfloat16, device="cuda")
    qta.qta_linear_bwd(d, y, x, w, dx, dw, qta.alloc_workspace(qta.linear_bwd_workspace_bytes(d)))
    done()
    dz, _, e16 = bwd_bounds(y, z, e, "silu", "bf16")
    ref, ea = prod(dz, w.T, 72)
    eb = ea + e16 @ w.double().abs()
    check("dx", dx, ref, eb * 1.01 + U["bf16"] * (ref.abs() + eb))
    yn, ga = far(64, 200 - 64), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    qta.qta_norm(qta.norm_desc(3, 64, "bf16"), x, ga, yn)
    done()
    _, _, _, xh, y64 = norm64(x, None, ga, None, "layer", 1e-5)
    check("norm", yn, y64, U["bf16"] * y64.abs() + 1e-5)
    del wide


def test_wrapper_checks(dev):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    d = qta.linear_desc(4, 32, 64, "bf16")
    qta.qta_linear(d, x, w, y)
    with pytest.raises(ValueError):
        qta.qta_linear(d, x.half(), w, y)              # type
    with pytest.raises(ValueError):
        qta.qta_linear(d, x.cpu(), w, y)               # device
    with pytest.raises(ValueError):
        qta.qta_linear(d, x[:3], w, y)                 # shape
    with pytest.raises(ValueError):
        qta.qta_linear(d, x, w, y, bias=torch.zeros(31, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        qta.qta_linear(d, torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda").t(), w, y)   # stride along a row
    with pytest.raises(ValueError):
        qta.qta_linear(d, x[:1].expand(4, 64), w, y)   # rows on top of each other
    with pytest.raises(qta.QtaError) as e:
        qta.qta_linear(d, torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")[1:257].view(4, 64), w, y)
    assert e.value.status == qta.QTA_ERR_ALIGNMENT
    with pytest.raises(qta.QtaError) as e:
        qta.qta_linear(qta.linear_desc(4, 64, 64, "bf16"), x, torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda"), x)
    assert e.value.status == qta.QTA_ERR_INVALID_ARG
    da = qta.linear_desc(4, 32, 64, "bf16", "silu")
    with pytest.raises(ValueError):
        qta.qta_linear_bwd(da, y, x, w, None, None, torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        qta.linear_desc(4, 32, 64, "bf16", "swish")
    done()
