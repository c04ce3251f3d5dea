"""GPU parity of every kernel plan of the linear and gated calls (include/linear.h)
at the sizes where a plan can go wrong: last steps of every length, tiles that the
rows end in, odd operands that are packed first, few rows, both gradients in one
launch.  Small whole numbers, so that every sum is exact and the results are compared
bit for bit with 64-bit sums rounded once; each case names the plan it is meant for.
Activations at large and infinite arguments against their 64-bit definitions."""
import math

import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_linear import (ACTS, PARAM, T, U, act64, backward, forward, gated, gated_back, gen, h,
                             scratch, stream, strided, whole)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


def product64(x, w, kn=False):
    """Exact in float32 too: whole numbers, sums below 2^24 (float64 is slow here)."""
    return (x.float() @ (w.float() if kn else w.float().t())).double()


def plan(m, n, k, dtype, **kw):
    return cf.linear_describe_variant(cf.make_linear_problem(m, n, k, **kw), dtype)


# last steps of 8 .. 64 k, one to five steps, ends inside the last tile
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,tile", [
    (4096, 4096, 520, "tile256x256"), (4096, 4096, 584, "tile256x256"),
    (8192, 8192, 520, "tile256x256"), (8000, 1032, 1032, "tile256x256"),
    (7990, 1016, 2056, "tile256x128"), (8192, 1024, 1096, "tile256x128"),
    (2000, 4088, 1544, "tile256x128"), (3000, 1500, 264, "tile128x128"),
    (4050, 4104, 456, "tile128x128"), (8100, 4400, 200, "tile128x128"), (4000, 1000, 248, "tile"),
    (1000, 1000, 8, "tile64x64"), (1000, 1000, 72, "tile64x64"), (500, 520, 136, "tile64x64"),
    (70, 200, 192, "tile64x64"), (64, 256, 4096, "split"), (300, 520, 2056, "split")])
def test_tiles(m, n, k, tile, dtype, kn):
    assert tile in plan(m, n, k, dtype, w_layout="kn" if kn else "nk")
    g = gen(m + n + k)
    print(f"[tiles] {m} {n} {k} {dtype} kn={kn}", flush=True)
    x, w = whole(g, dtype, m, k), whole(g, dtype, *((k, n) if kn else (n, k)))
    b, r = whole(g, dtype, n, lo=-8, hi=9), whole(g, dtype, m, n, lo=-8, hi=9)
    want = product64(x, w, kn) + b.double()
    y, z = forward(dtype, x, w, b, r, act="relu", res="after", kn=kn, save=True)
    assert torch.equal(z, want.to(T[dtype]))
    assert torch.equal(y, (want.clamp(min=0) + r.double()).to(T[dtype]))
    y = forward(dtype, x, w, None, r, act="identity", res="before", kn=kn)
    assert torch.equal(y, (want - b.double() + r.double()).to(T[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,f,k,tile", [
    (4096, 2048, 520, "tile256x256"), (8000, 516, 1032, "tile256x256"), (4050, 2060, 328, "tile128x128"),
    (2000, 1021, 1544, "tile"), (700, 300, 72, "tile"), (64, 256, 4096, "split")])
def test_gated_tiles(m, f, k, tile, dtype):
    assert tile in cf.gated_describe_variant(cf.make_gated_problem(m, f, k), dtype)
    g = gen(m + f + k)
    print(f"[gated tiles] {m} {f} {k} {dtype}", flush=True)
    x, wg, wu = (whole(g, dtype, *s, lo=-1, hi=2) for s in ((m, k), (f, k), (f, k)))
    a, b = product64(x, wg), product64(x, wu)
    assert float(a.abs().max() * b.abs().max()) < 2 ** 24
    out, pg, pu = gated(dtype, x, wg, wu, act="relu", save=True, packed=True)
    assert torch.equal(pg, a.to(T[dtype])) and torch.equal(pu, b.to(T[dtype]))
    assert torch.equal(out, (a.clamp(min=0) * b).to(T[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m", [1, 3, 16, 17, 32])
@pytest.mark.parametrize("n,k", [(3, 8), (250, 64), (1000, 520), (1003, 1000), (2050, 1032),
                                 (4100, 264), (8200, 72), (1001, 777), (2049, 129), (4099, 65),
                                 (500, 9)])
def test_streamed(m, n, k, dtype):
    g = gen(m + n + k)
    x, w = whole(g, dtype, m, k), whole(g, dtype, n, k)
    b, r = whole(g, dtype, n, lo=-8, hi=9), whole(g, dtype, m, n, lo=-8, hi=9)
    want = product64(x, w) + b.double() + r.double()
    y, z = forward(dtype, x, w, b, r, act="relu", res="before", save=True)
    assert torch.equal(z, want.to(T[dtype])) and torch.equal(y, want.clamp(min=0).to(T[dtype]))
    # rows apart, from odd elements on, between NaN
    (_, xv), (_, wv), (_, rv) = (strided(t, 5, 3) for t in (x, w, r))
    ybuf, yv = strided(torch.zeros(m, n, dtype=T[dtype], device="cuda"), 3, 1)
    forward(dtype, xv, wv, b, rv, y=yv, act="relu", res="before")
    assert torch.equal(yv, want.clamp(min=0).to(T[dtype]))
    yv.zero_()
    assert int(torch.isnan(ybuf).sum()) == ybuf.numel() - m * n


def test_streamed_plans():
    """The sizes above reach every number of weight rows a workgroup."""
    names = {plan(m, n, k, "f16") for m in (1, 32) for n, k in ((250, 64), (2050, 1032), (4100, 264),
                                                                (8200, 72))}
    assert all("stream" in s for s in names)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,f,k", [(1, 1500, 520), (2, 5001, 264), (17, 700, 129), (32, 2100, 72),
                                   (5, 333, 9)])
def test_gated_streamed(m, f, k, dtype):
    assert "stream" in cf.gated_describe_variant(cf.make_gated_problem(m, f, k), dtype)
    g = gen(m + f + k)
    x, wg, wu = (whole(g, dtype, *s, lo=-1, hi=2) for s in ((m, k), (f, k), (f, k)))
    bg, bu = whole(g, dtype, f), whole(g, dtype, f)
    a, b = product64(x, wg) + bg.double(), product64(x, wu) + bu.double()
    out, pg, pu = gated(dtype, x, wg, wu, bg, bu, act="relu", save=True)
    assert torch.equal(pg, a.to(T[dtype])) and torch.equal(pu, b.to(T[dtype]))
    assert torch.equal(out, (a.clamp(min=0) * b).to(T[dtype]))


@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(4001, 4003, 1031), (3001, 3003, 2051)])
def test_packed_operands(m, n, k, dtype, kn):
    """Odd rows inside buffers of NaN, large enough that they are copied first."""
    kw = dict(w_layout="kn" if kn else "nk", ldx=k + 5, ldw=(n if kn else k) + 5)
    assert dtype == "f32" or ".pack" in plan(m, n, k, dtype, **kw)
    g = gen(m + n + k)
    print(f"[packed] {m} {n} {k} {dtype} kn={kn}", flush=True)
    x, w = whole(g, dtype, m, k), whole(g, dtype, *((k, n) if kn else (n, k)))
    (_, xv), (_, wv) = strided(x, 5, 1), strided(w, 5, 3)
    want = product64(x, w, kn)
    assert torch.equal(forward(dtype, xv, wv, kn=kn), want.to(T[dtype]))
    if not kn:
        half = n // 2
        w1, w2 = w[:half], w[half:2 * half]
        a, b = want[:, :half], want[:, half:2 * half]
        if float(a.abs().max() * b.abs().max()) < 2 ** 24:
            out = gated(dtype, xv, strided(w1, 5, 1)[1], strided(w2, 5, 1)[1], act="identity")
            assert torch.equal(out, (a * b).to(T[dtype]))


@pytest.mark.parametrize("act", ["identity", "relu"])
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,name", [
    (2048, 2048, 1024, "both"), (2000, 2056, 1000, "both"), (4096, 4096, 2048, "both.tile256x256"),
    (4000, 1992, 1992, "both"), (2001, 2003, 1031, ""), (520, 1032, 72, ""), (1001, 65, 2000, "")])
def test_both_gradients(m, n, k, name, dtype, kn, act):
    p = cf.make_linear_problem(m, n, k, act=act, w_layout="kn" if kn else "nk")
    assert name in cf.linear_backward_describe_variant(p, dtype)
    g = gen(m + n + k)
    print(f"[both] {m} {n} {k} {dtype} kn={kn} {act}", flush=True)
    x, w = whole(g, dtype, m, k), whole(g, dtype, *((k, n) if kn else (n, k)))
    z, dy = whole(g, dtype, m, n), whole(g, dtype, m, n)
    d = dy.double() * ((z > 0).double() if act == "relu" else 1.0)
    wd = w.float().t() if kn else w.float()
    dx64 = (d.float() @ wd).double()
    dw64 = (d.float().t() @ x.float()).double()
    for want in ("xwb", "x", "w"):
        dx, dw, db, _ = backward(dtype, x, w, z, dy, act=act, kn=kn, want=want)
        if dx is not None:
            assert torch.equal(dx, dx64.to(T[dtype]))
        if dw is not None:
            assert torch.equal(dw, (dw64.t() if kn else dw64).to(T[dtype]))
        if db is not None:
            assert torch.equal(db, d.sum(0).to(T[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,f,k,name", [(2048, 1408, 1024, "both"), (2000, 1401, 1000, "both"),
                                        (1501, 1003, 1031, ""), (4096, 5632, 2048, "both.tile256x256")])
def test_gated_both_gradients(m, f, k, name, dtype):
    assert name in cf.gated_backward_describe_variant(cf.make_gated_problem(m, f, k), dtype)
    g = gen(m + f + k)
    print(f"[gated both] {m} {f} {k} {dtype}", flush=True)
    x, wg, wu = (whole(g, dtype, *s) for s in ((m, k), (f, k), (f, k)))
    pg, pu, dh = (whole(g, dtype, m, f, lo=-1, hi=2) for _ in range(3))
    dg = dh.float() * pu.float() * (pg > 0).float()
    du = dh.float() * pg.float().clamp(min=0)
    dx, dwg, dwu, dbg, dbu = gated_back(dtype, x, wg, wu, pg, pu, dh, act="relu")
    assert torch.equal(dx, (dg @ wg.float() + du @ wu.float()).to(T[dtype]))
    assert torch.equal(dwg, (dg.t() @ x.float()).to(T[dtype]))
    assert torch.equal(dwu, (du.t() @ x.float()).to(T[dtype]))
    assert torch.equal(dbg, dg.sum(0).to(T[dtype])) and torch.equal(dbu, du.sum(0).to(T[dtype]))


@pytest.mark.parametrize("m,n,k", [(2100, 2100, 1032), (300, 300, 72), (8, 2100, 264)])
def test_views_from_odd_elements(m, n, k):
    """Strides of whole pieces, but every operand from an odd 16-bit element on."""
    g = gen(7)
    x, w, r = whole(g, "f16", m, k), whole(g, "f16", n, k), whole(g, "f16", m, n)
    (_, xv), (_, wv), (_, rv) = (strided(t, 8, 1) for t in (x, w, r))
    _, yv = strided(torch.zeros(m, n, dtype=torch.float16, device="cuda"), 8, 1)
    forward("f16", xv, wv, None, rv, y=yv, res="before")
    assert torch.equal(yv, (product64(x, w) + r.double()).to(torch.float16))


@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(4, 1000, 264), (300, 304, 200), (3000, 1504, 264),
                                   (4096, 4096, 520), (8192, 1024, 1096)])
def test_rows_at_multiples_of_four_bytes(m, n, k, dtype, kn):
    """Whole pieces in rows that start on multiples of 4 bytes only."""
    pad, off = (2, 6) if dtype == "f16" else (1, 3)
    g = gen(m + k)
    x, w = whole(g, dtype, m, k), whole(g, dtype, *((k, n) if kn else (n, k)))
    z, dy = whole(g, dtype, m, n), whole(g, dtype, m, n)
    (_, xv), (_, wv), (_, zv), (_, dyv) = (strided(t, pad, off) for t in (x, w, z, dy))
    assert torch.equal(forward(dtype, xv, wv, kn=kn), product64(x, w, kn).to(T[dtype]))
    if m > 4096 or n > 4000:
        return
    for act in ("identity", "relu"):
        d = dy.float() * ((z > 0).float() if act == "relu" else 1.0)
        dx, dw, _, _ = backward(dtype, xv, wv, zv, dyv, act=act, kn=kn, want="xw")
        assert torch.equal(dx, (d @ (w.float().t() if kn else w.float())).to(T[dtype]))
        want = d.t() @ x.float()
        assert torch.equal(dw, (want.t() if kn else want).to(T[dtype]))


def test_plan_rerun_is_bit_identical():
    g = torch.Generator(device="cuda").manual_seed(3)
    for m, n, k in ((4096, 4096, 264), (64, 256, 4096), (2001, 2003, 1031), (16, 1000, 2048)):
        x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
        w = torch.randn(n, k, generator=g, device="cuda").bfloat16()
        a = forward("bf16", x, w, act="gelu")
        assert torch.equal(a, forward("bf16", x, w, act="gelu"))


# ------------------------------------------------------------------- activations' ends

EXTREMES = [0.0, -0.0, 1e-8, -1e-8, 1e-4, -1e-4, 0.3, -0.3, 0.35, -0.35, 0.36, -0.36, 1.0, -1.0, 3.0,
            -3.0, 5.5, -5.5, 9.0, -9.0, 12.0, -12.0, 30.0, -30.0, 88.0, -88.0, 200.0, -200.0, 6e4, -6e4]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_activation_far_out(act, dtype):
    """y = act(x) through a product with one, k = 1: 16 float32 ulps of the argument and
    of the value, and one rounding; nothing overflows to NaN on the way."""
    x = torch.tensor(EXTREMES, dtype=T[dtype], device="cuda").view(-1, 1)
    one = torch.ones(1, 1, dtype=T[dtype], device="cuda")
    y = forward(dtype, x, one, act=act).double()
    v = x.double()
    want = act64(v, act)[0]
    err = 16 * U * (v.abs() + want.abs()) + h(dtype) * want.abs() + {"f32": 2.0 ** -126}.get(dtype, 2.0 ** -25)
    assert bool(((y - want).abs() <= err).all()), (y - want).abs().max()
    # slopes, through the gradient of a residual before the activation
    d = backward(dtype, x, one, x, torch.ones_like(x), act=act, res="before", want="r")[3].double()
    want = act64(v, act)[1]
    err = 16 * U * (1 + v.abs()) + h(dtype) * want.abs() + 2.0 ** -25
    assert not torch.isnan(d).any() and bool(((d - want).abs() <= err).all()), (d - want).abs().max()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ["identity", "relu", "tanh", "sigmoid", "silu", "gelu", "gelu_tanh"])
def test_activation_of_infinity_and_nan(act, dtype):
    x = torch.tensor([math.inf, math.nan, -math.inf], dtype=T[dtype], device="cuda").view(-1, 1)
    y = forward(dtype, x, torch.ones(1, 1, dtype=T[dtype], device="cuda"), act=act).flatten().tolist()
    assert y[0] == (1.0 if act in ("tanh", "sigmoid") else math.inf)
    if act == "relu":
        return  # max(x, 0) of a NaN is 0 where the comparison is false, as the convolution's
    assert math.isnan(y[1])
    low = {"identity": -math.inf, "tanh": -1.0, "sigmoid": 0.0}.get(act)
    assert y[2] == low if low is not None else (math.isnan(y[2]) or y[2] == 0.0)
