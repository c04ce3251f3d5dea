"""GPU parity of the layer norm (include/layer_norm.h), forward and backward, against a
plain implementation in 64 bits.

Bounds, per element, with u = 2^-24 and h = eps / 2 of the element type (one rounding
where a value is stored).  A row's sums run through at most D = 72 additions one after
the other: 32 elements of a thread, 6 steps of a wave, 16 waves, and 18 for the parts of
a long row; D u times the sum of the absolute terms bounds each.
 - s = r + drop(x) is off by es = 2 u (|drop(x)| + |r|);
 - mean by em = (D + 2) u mean|s| + mean(es);
 - the sum of squared distances q from the mean as it was computed: every distance is
   off by (es + em + u |s - mean|), so the variance by (D + 3) u var + 2 mean(|s - mean|
   (es + em)) + mean((es + em)^2) + 2 u var, and rstd = (var + eps)^-1/2 relatively by
   half of that over (var + eps), + 3 u;
 - y = (s - mean) rstd w + b: |w| (rstd (es + em) + |xhat| (er + 4 u)) + 2 u |y|, |b|;
 - backward, from the kept s, mean and rstd (exact inputs): xhat is off by 2 u |xhat|,
   the row sums by (D + 4) u of their absolute terms, every step of the formula by u
   of its terms; a column's sum of m terms by (m + 100) u of its absolute terms.
"""
import math

import numpy as np
import pytest

import convolution_forward_amd as cf
import mask_reference as mask

torch = pytest.importorskip("torch")

from test_gpu_linear import T, TINY, U, gen, h, strided, stream  # noqa: E402

pytestmark = pytest.mark.gpu

D = 72
SEED, OFFSET = 0x123456789ABCDEF1, (1 << 33) + 5


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


def close(name, got, want, err, half=0.0, tiny=0.0):
    d = (got.double() - want).abs()
    lim = err + half * (want.abs() + err) + tiny
    bad = ~((d <= lim) | (torch.isnan(want) & torch.isnan(got)))
    if bad.any():
        i = tuple(int(q) for q in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} out of bounds, first at "
                             f"{i}: {got[i].item()} for {want[i].item()}, error {d[i].item():.3g} "
                             f"bound {lim[i].item():.3g}")


def keep64(m, n, drop, step=0):
    """1 where kept, and the scale."""
    k = torch.from_numpy(mask.keeps(m, n, drop, SEED, OFFSET + step)).cuda().double()
    return k, mask.scale(drop)


def forward64(x, r, w, b, drop, eps, step=0):
    """y, s, mean, rstd in 64 bits, and their bounds before the final rounding."""
    x = x.double()
    v, es = x, torch.zeros_like(x)
    if mask.threshold(drop):
        keep, scale = keep64(*x.shape, drop, step)
        v = torch.where(keep > 0, x * scale, torch.zeros_like(x))
    if r is not None:
        es = 2 * U * (v.abs() + r.double().abs())
        v = v + r.double()
    elif mask.threshold(drop):
        es = U * v.abs()
    eps = float(np.float32(eps))
    mean = v.mean(1, keepdim=True)
    em = (D + 2) * U * v.abs().mean(1, keepdim=True) + es.mean(1, keepdim=True)
    d = v - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    off = es + em
    ev = (D + 5) * U * var + 2 * (d.abs() * off).mean(1, keepdim=True) + (off * off).mean(1, keepdim=True)
    er = 0.5 * ev / (var + eps) + 3 * U
    assert float(er.nan_to_num().max()) < 0.05  # the first-order bound holds
    xhat = d * rstd
    one = torch.ones_like(v)
    wd = one if w is None else w.double() * one
    y = xhat * wd + (0 if b is None else b.double())
    ey = wd.abs() * (rstd * off + xhat.abs() * (1.1 * er + 4 * U))
    ey = ey + 2 * U * (y.abs() + (xhat * wd).abs())
    return (y, v, mean[:, 0], rstd[:, 0]), (ey, es, em[:, 0], (1.1 * er * rstd)[:, 0])


def backward64(s, w, mean, rstd, dy, ds, drop, step=0):
    m, n = s.shape
    s, dy, mean, rstd = s.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    xhat = (s - mean) * rstd
    wd = torch.ones_like(s) if w is None else w.double() * torch.ones_like(s)
    g = dy * wd
    along, level = (g * xhat).mean(1, keepdim=True), g.mean(1, keepdim=True)
    d = rstd * (g - level - xhat * along)
    ea = (D + 6) * U * (g * xhat).abs().mean(1, keepdim=True)
    el = (D + 3) * U * g.abs().mean(1, keepdim=True)
    ed = rstd * (el + xhat.abs() * ea + 6 * U * (g.abs() + level.abs() + (xhat * along).abs()))
    if ds is not None:
        d = d + ds.double()
        ed = ed + U * (d.abs() + ds.double().abs())
    dx, ex = d, ed
    if mask.threshold(drop):
        keep, scale = keep64(m, n, drop, step)
        dx, ex = torch.where(keep > 0, d * scale, torch.zeros_like(d)), keep * scale * (ed + 2 * U * d.abs())
    ew = (m + 100) * U * (dy * xhat).abs().sum(0)
    eb = (m + 100) * U * dy.abs().sum(0)
    return (dx, d, (dy * xhat).sum(0), dy.sum(0)), (ex, ed, ew, eb)


def ws_of(size):
    return torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device="cuda")


def run_forward(dtype, x, r, w, b, *, drop=0.0, eps=1e-5, step=None, y=None, s=None, keep=True):
    m, n = x.shape
    empty = lambda: torch.full((m, n), float("nan"), dtype=T[dtype], device="cuda")  # noqa: E731
    y = empty() if y is None else y
    s = empty() if s is None and keep else s
    stats = [torch.full((m,), float("nan"), device="cuda") if keep else None for _ in range(2)]
    p = cf.make_layer_norm_problem(m, n, eps=eps, weight=w is not None, bias=b is not None,
                                   residual=r is not None, drop=drop, seed=SEED, offset=OFFSET,
                                   ldx=x.stride(0), ldr=0 if r is None else r.stride(0),
                                   ldy=y.stride(0), lds=0 if s is None else s.stride(0))
    size = cf.layer_norm_scratch_size(p, dtype)
    cf.layer_norm_forward(p, dtype, x, r, w, b, y, s, *stats, step, ws_of(size), size, stream())
    return y, s, *stats


def run_backward(dtype, s, w, mean, rstd, dy, ds, *, bias=True, residual=True, drop=0.0, step=None,
                 dx=None, dr=None, want="dx dr dw db"):
    m, n = s.shape
    empty = lambda *shape: torch.full(shape, float("nan"), dtype=T[dtype], device="cuda")  # noqa: E731
    if dx is None and "dx" in want:
        dx = empty(m, n)
    if dr is None and "dr" in want and residual:
        dr = empty(m, n)
    dw = empty(n) if w is not None and "dw" in want else None
    db = empty(n) if bias and "db" in want else None
    ld = lambda v: 0 if v is None else v.stride(0)  # noqa: E731
    p = cf.make_layer_norm_problem(m, n, weight=w is not None, bias=bias, residual=residual,
                                   drop=drop, seed=SEED, offset=OFFSET, lds=s.stride(0),
                                   ldy=dy.stride(0), ldds=ld(ds), lddx=ld(dx), lddr=ld(dr))
    size = cf.layer_norm_backward_scratch_size(p, dtype)
    cf.layer_norm_backward(p, dtype, s, w, mean, rstd, dy, ds, dx, dr, dw, db, step, ws_of(size),
                           size, stream())
    return dx, dr, dw, db


def rnd(g, dtype, *shape, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(T[dtype])


def inputs(dtype, m, n, seed=0):
    g = gen(seed)
    return (rnd(g, dtype, m, n), rnd(g, dtype, m, n, scale=2.0, shift=0.5),
            rnd(g, dtype, n, scale=0.3, shift=1.0), rnd(g, dtype, n, scale=0.3))


def check_forward(dtype, x, r, w, b, drop, got, eps=1e-5, step=0):
    want, err = forward64(x, r, w, b, drop, eps, step)
    close("y", got[0], want[0], err[0], h(dtype), TINY[dtype])
    if got[1] is not None:
        close("s", got[1], want[1], err[1], h(dtype), TINY[dtype])
    if got[2] is not None:
        close("mean", got[2], want[2], err[2], U, TINY["f32"])
        close("rstd", got[3], want[3], err[3], U)


# rows of one element to several parts; both sides of every plan's limits
SIZES = [(1, 1), (3, 2), (5, 7), (4, 8), (9, 15), (2, 511), (7, 512), (6, 520), (13, 1001),
         (5, 1032), (3, 2048), (4, 2049), (3, 4096), (2, 5000), (3, 8192), (2, 8200), (2, 16384),
         (3, 16391), (1, 32768), (2, 32769), (3, 50_001), (1, 100_000), (1000, 33), (257, 264)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n", SIZES)
def test_forward(dtype, m, n):
    x, r, w, b = inputs(dtype, m, n, seed=m * 31 + n)
    for res, drop in ((None, 0.0), (r, 0.0), (r, 0.3), (None, 0.5)):
        check_forward(dtype, x, res, w, b, drop, run_forward(dtype, x, res, w, b, drop=drop))
    check_forward(dtype, x, r, None, None, 0.0, run_forward(dtype, x, r, None, None, keep=False))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n", SIZES)
def test_backward(dtype, m, n):
    x, dy, w, b = inputs(dtype, m, n, seed=m * 17 + n)
    _, ds, _, _ = inputs(dtype, m, n, seed=1)
    f = x.float()
    mean = f.mean(1)
    rstd = ((f - mean[:, None]) ** 2).mean(1).add(1e-5).rsqrt()
    for extra, drop in ((None, 0.0), (ds, 0.3)):
        got = run_backward(dtype, x, w, mean, rstd, dy, extra, drop=drop)
        want, err = backward64(x, w, mean, rstd, dy, extra, drop)
        for name, a, v, e in zip(("dx", "dr", "dw", "db"), got, want, err):
            close(name, a, v, e, h(dtype), TINY[dtype])
    got = run_backward(dtype, x, None, mean, rstd, dy, ds, bias=False, residual=False)
    want, err = backward64(x, None, mean, rstd, dy, ds, 0.0)
    close("dx alone", got[0], want[0], err[0], h(dtype), TINY[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n", [(1024, 3), (1023, 5), (897, 66), (769, 130), (770, 1001),
                                 (513, 2047), (1024, 4096), (512, 8190), (40, 20_001), (300, 8193),
                                 (3, 100_003)])
def test_backward_of_few_rows(dtype, m, n):
    """Rows up to the limit of columns summed beside them, with columns left over; the
    same over dy."""
    assert cf.layer_norm_backward_describe_variant(cf.make_layer_norm_problem(m, n), dtype).endswith(".once")
    backward_of_many_rows(dtype, m, n)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n", [(1025, 9), (20_000, 50), (1100, 100), (9000, 250), (2100, 500),
                                 (5003, 1001), (1025, 2048), (1500, 2047), (2600, 4090), (1030, 5000),
                                 (800, 8192), (1100, 8193), (600, 20_001)])
def test_backward_of_several_rows_a_group(dtype, m, n):
    """Rows beyond that limit: partial rows of dw and db, joined; the same over dy."""
    assert "once" not in cf.layer_norm_backward_describe_variant(cf.make_layer_norm_problem(m, n), dtype)
    backward_of_many_rows(dtype, m, n)


def backward_of_many_rows(dtype, m, n):
    x, dy, w, b = inputs(dtype, m, n, seed=m + n)
    ds = inputs(dtype, m, n, seed=5)[0]
    f = x.float()
    mean = f.mean(1)
    rstd = ((f - mean[:, None]) ** 2).mean(1).add(1e-5).rsqrt()
    got = run_backward(dtype, x, w, mean, rstd, dy, ds, drop=0.3)
    want, err = backward64(x, w, mean, rstd, dy, ds, 0.3)
    for name, a, v, e in zip(("dx", "dr", "dw", "db"), got, want, err):
        close(name, a, v, e, h(dtype), TINY[dtype])
    over, other = dy.clone(), ds.clone()
    again = run_backward(dtype, x, w, mean, rstd, over, other, drop=0.3, dx=over, dr=other)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("n", [7, 40, 1001, 3000, 9001, 50_003])
def test_weight_or_bias_alone_from_odd_elements(dtype, n):
    """w without b and b without w, each from an odd element of a buffer."""
    m = 5
    x, dy, w, b = inputs(dtype, m, n)
    w, b = (torch.cat([t.new_full((1,), float("nan")), t])[1:] for t in (w, b))
    for one, two in ((w, None), (None, b)):
        got = run_forward(dtype, x, None, one, two)
        check_forward(dtype, x, None, one, two, 0.0, got)
        grads = run_backward(dtype, x, one, got[2], got[3], dy, None, bias=two is not None,
                             residual=False)
        want, err = backward64(x, one, got[2], got[3], dy, None, 0.0)
        close("dx", grads[0], want[0], err[0], h(dtype), TINY[dtype])
        at = 2 if two is None else 3
        close("dw or db", grads[at], want[at], err[at], h(dtype), TINY[dtype])
        assert grads[5 - at] is None


@pytest.mark.parametrize("n", [24, 1000, 3000, 9000, 20_000, 40_000])
def test_each_gradient_alone(n):
    x, dy, w, _ = inputs("f32", 6, n)
    mean, rstd = x.mean(1), x.var(1, correction=0).add(1e-5).rsqrt()
    whole = run_backward("f32", x, w, mean, rstd, dy, None, drop=0.2)
    for i, name in enumerate(("dx", "dr", "dw", "db")):
        one = run_backward("f32", x, w, mean, rstd, dy, None, drop=0.2, want=name)
        assert torch.equal(one[i], whole[i])
        assert all(v is None for j, v in enumerate(one) if j != i)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,pad,off", [(1001, 6, 1), (513, 7, 3), (4096, 8, 8), (2048, 3, 5),
                                       (17_000, 5, 1), (40_003, 2, 3)])
def test_strides_and_what_lies_between_rows(dtype, n, pad, off):
    """Every operand in rows of its own stride, off its 16 bytes; what is between and
    behind the rows stays as it was."""
    m = 5
    x, r, w, b = inputs(dtype, m, n)
    views = [strided(t, pad + 2 * i, off + i) for i, t in enumerate((x, r))]
    outs = [strided(torch.zeros_like(x), pad + 3 + i, off + 1 + i) for i in range(2)]
    got = run_forward(dtype, views[0][1], views[1][1], w, b, drop=0.2, y=outs[0][1], s=outs[1][1])
    check_forward(dtype, x, r, w, b, 0.2, got)
    for buf, v in outs:
        rim = torch.isnan(buf)
        assert int(rim.sum()) == buf.numel() - v.numel()  # the rims are NaN still
    mean, rstd = got[2], got[3]
    dy, ds = inputs(dtype, m, n, seed=3)[:2]
    ins = [strided(t.clone(), pad + i, off + i)[1] for i, t in enumerate((x, dy, ds))]
    outs = [strided(torch.zeros_like(x), pad + 3 + i, off + 1 + i) for i in range(2)]
    got = run_backward(dtype, ins[0], w, mean, rstd, ins[1], ins[2], drop=0.2, dx=outs[0][1], dr=outs[1][1])
    want, err = backward64(x, w, mean, rstd, dy, ds, 0.2)
    for name, a, v, e in zip(("dx", "dr", "dw", "db"), got, want, err):
        close(name, a, v, e, h(dtype), TINY[dtype])
    for buf, v in outs:
        assert int(torch.isnan(buf).sum()) == buf.numel() - v.numel()


def test_offsets():
    """Element offsets added to every pointer equal views of the buffers."""
    m, n = 6, 72
    x, r, w, b = inputs("f16", m, n)
    arena = torch.full((8, 1000), float("nan"), dtype=torch.float16, device="cuda")
    offs = (8, 3, 40, 5, 16, 1)
    for row, t, o in zip(arena, (x, r, w, b), offs):
        row[o:o + t.numel()] = t.reshape(-1)
    p = cf.make_layer_norm_problem(m, n, residual=True, offsets=offs)
    cf.layer_norm_forward(p, "f16", *arena[:6], stream=stream())
    y, s, _, _ = run_forward("f16", x, r, w, b)
    assert torch.equal(arena[4][16:16 + m * n].view(m, n), y)
    assert torch.equal(arena[5][1:1 + m * n].view(m, n), s)


@pytest.mark.parametrize("n", [40, 1000, 5000, 40_000])
def test_in_place(n):
    x, r, w, b = inputs("bf16", 7, n)
    y, s, mean, rstd = run_forward("bf16", x, r, w, b, drop=0.1)
    for which in range(2):
        a, c = x.clone(), r.clone()
        outs = (a, c) if which else (c, a)  # y over x and s over r, and the reverse
        got = run_forward("bf16", a, c, w, b, drop=0.1, y=outs[0], s=outs[1])
        assert torch.equal(got[0], y) and torch.equal(got[1], s)
    dy, ds = inputs("bf16", 7, n, seed=4)[:2]
    want = run_backward("bf16", s, w, mean, rstd, dy, ds, drop=0.1)
    for which in range(2):
        a, c = dy.clone(), ds.clone()
        outs = (a, c) if which else (c, a)
        got = run_backward("bf16", s, w, mean, rstd, a, c, drop=0.1, dx=outs[0], dr=outs[1])
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("n", [16, 700, 3000, 20_000, 60_000])
def test_far_from_zero(n):
    """A mean 4000 times the spread: a difference of squares would leave nothing of it.
    The values are multiples of 2^-10 below 2^3, so s is exact; the sums' bounds hold."""
    g = gen(n)
    x = (torch.randint(-8, 9, (3, n), generator=g, device="cuda") / 1024 + 7).float()
    w, b = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    got = run_forward("f32", x, None, w, b, eps=1e-12)
    d = x.double() - x.double().mean(1, keepdim=True)
    rstd = ((d * d).mean(1) + 1e-12) ** -0.5
    # mean is off by (D + 2) u 7 = 3.1e-5 at most, under a hundredth of the spread 0.0048, and
    # var by its square: 1% bounds rstd, where a difference of squares would be off by
    # 7^2 u over 2.3e-5, an eighth of the value for one rounding alone; y is off by rstd
    # times the mean's error, 0.0065
    assert float(((got[3].double() - rstd) / rstd).abs().max()) < 0.01
    assert float((got[0].double() - d * rstd[:, None]).abs().max()) < 0.05


@pytest.mark.parametrize("n", [9, 800, 5000, 70_000])
def test_equal_values_and_not_finite(n):
    x, r, w, b = inputs("f32", 5, n)
    x[1] = 3.25  # 13/4: sums of up to 2^20 of them are exact, and so is their quotient by n
    x[2, n // 2] = float("inf")
    x[3, 0] = float("nan")
    y, s, mean, rstd = run_forward("f32", x, None, w, b)
    assert torch.equal(y[1], b)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    for i in (0, 4):
        check_forward("f32", x[i:i + 1], None, w, b, 0.0, [v[i:i + 1] for v in (y, s, mean, rstd)])
    dy = r
    dx, _, dw, db = run_backward("f32", s, w, mean, rstd, dy, None)
    assert torch.isnan(dx[2]).all() and torch.isnan(dx[3]).all() and torch.isnan(dw).all()
    assert torch.isfinite(dx[0]).all() and torch.isfinite(dx[4]).all() and torch.isfinite(db).all()


def test_an_infinite_dropped_element_is_gone():
    """A dropped element is 0 whatever x holds: the row stays finite."""
    x, r, w, b = inputs("f32", 64, 40)
    keep = mask.keeps(64, 40, 0.5, SEED, OFFSET)
    x[torch.from_numpy(~keep).cuda()] = float("inf")
    check_forward("f32", torch.where(torch.isinf(x), torch.zeros_like(x), x), r, w, b, 0.5,
                  run_forward("f32", x, r, w, b, drop=0.5))
    check_forward("f32", torch.zeros_like(x), r, w, b, 0.0,
                  run_forward("f32", x, r, w, b, drop=1.0))  # all dropped


def test_no_rows():
    w, b = (torch.ones(300, dtype=torch.float16, device="cuda") for _ in range(2))
    p = cf.make_layer_norm_problem(0, 300)
    cf.layer_norm_forward(p, "f16", None, None, w, b, None, stream=stream())
    for n in (300, 5000, 40_000):
        dw, db = (torch.full((n,), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
        w = torch.ones(n, dtype=torch.float16, device="cuda")
        p = cf.make_layer_norm_problem(0, n)
        size = cf.layer_norm_backward_scratch_size(p, "f16")
        cf.layer_norm_backward(p, "f16", None, w, None, None, None, None, None, None, dw, db, None,
                               ws_of(size), size, stream())
        assert not dw.any() and not db.any()


@pytest.mark.parametrize("n", [24, 1500, 20_000])
def test_gradients_against_differences(n):
    """(L(v + t e) - L(v - t e)) / 2t of L = sum(y c) + sum(s k), in 64 bits, along random
    directions of x, r, w and b; the float32 gradients times the direction.  t = 1e-5:
    the third-order term is below 1e-8 of the value, rounding 1e-16 / 1e-5."""
    m, eps = 5, 1e-5
    x, r, w, b = inputs("f32", m, n)
    g = gen(9)
    c, k = rnd(g, "f32", m, n), rnd(g, "f32", m, n)
    keep, scale = keep64(m, n, 0.25)
    eps = float(np.float32(eps))

    def loss(x, r, w, b):
        s = r + keep * scale * x
        d = s - s.mean(1, keepdim=True)
        y = d * ((d * d).mean(1, keepdim=True) + eps) ** -0.5 * w + b
        return float((y * c.double()).sum() + (s * k.double()).sum())

    _, s, mean, rstd = run_forward("f32", x, r, w, b, drop=0.25)
    got = run_backward("f32", s, w, mean, rstd, c, k, drop=0.25)
    at = [t.double() for t in (x, r, w, b)]
    for i, (grad, v) in enumerate(zip(got, at)):
        e = torch.randn(v.shape, generator=g, device="cuda", dtype=torch.float64)
        ends = [loss(*(q + sign * 1e-5 * e if j == i else q for j, q in enumerate(at)))
                for sign in (1, -1)]
        want = (ends[0] - ends[1]) / 2e-5
        size = float((grad.double() * e).abs().sum())
        # float32 gradients: a few hundred roundings of their terms
        assert abs(float((grad.double() * e).sum()) - want) <= 500 * U * size + 1e-7 * abs(want) + 1e-6


@pytest.mark.parametrize("m,n", [(70, 600), (9, 4096), (3, 20_000), (4, 50_000),
                                 (1100, 264), (300, 20_000)])
def test_rerun_graph_and_streams(m, n):
    """Reruns are equal bit for bit; a captured forward and backward, replayed with new
    inputs and a step that moves on, equals the eager calls, also with eager work and a
    second captured call with a scratch of its own between the replays."""
    dtype = "bf16"
    x, r, w, b = inputs(dtype, m, n)
    dy = inputs(dtype, m, n, seed=2)[0]
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    new = lambda *shape, t=T[dtype]: torch.zeros(shape, dtype=t, device="cuda")  # noqa: E731
    y, s, dx, dr, dw, db = new(m, n), new(m, n), new(m, n), new(m, n), new(n), new(n)
    mean, rstd = new(m, t=torch.float32), new(m, t=torch.float32)
    p = cf.make_layer_norm_problem(m, n, residual=True, drop=0.2, seed=SEED, offset=OFFSET)
    size = [cf.layer_norm_scratch_size(p, dtype), cf.layer_norm_backward_scratch_size(p, dtype)]
    ws = [ws_of(v) for v in size]

    def call():
        cf.layer_norm_forward(p, dtype, x, r, w, b, y, s, mean, rstd, step, ws[0], size[0], stream())
        cf.layer_norm_backward(p, dtype, s, w, mean, rstd, dy, r, dx, dr, dw, db, step, ws[1],
                               size[1], stream())
        return [t.clone() for t in (y, s, mean, rstd, dx, dr, dw, db)]

    first = call()
    assert all(torch.equal(a, c) for a, c in zip(first, call()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cf.layer_norm_forward(p, dtype, x, r, w, b, y, s, mean, rstd, step, ws[0], size[0], stream())
        cf.layer_norm_backward(p, dtype, s, w, mean, rstd, dy, r, dx, dr, dw, db, step, ws[1],
                               size[1], stream())
        step.add_(1)
    for i in range(4):
        x.copy_(inputs(dtype, m, n, seed=20 + i)[0])
        step.fill_(100 + i)
        want = call()
        check_forward(dtype, x, r, w, b, 0.2, want[:4], step=100 + i)
        for t in (y, s, dx, dr, dw, db, mean, rstd):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, (y, s, mean, rstd, dx, dr, dw, db))), i
        assert int(step) == 101 + i
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step.fill_(103)
        got = call()
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))


def test_past_32_bits():
    """More than 2^31 elements: rows at both ends and in the middle."""
    m, n = 70_000, 32_768
    x = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    rows = [0, m // 2, m - 1]
    some, _, w, b = inputs("bf16", 3, n)
    for i, row in enumerate(rows):
        x[row] = some[i]
    y, _, mean, rstd = run_forward("bf16", x, None, w, b, y=torch.empty_like(x), s=x.new_empty(m, n))
    check_forward("bf16", some, None, w, b, 0.0, [y[rows], None, mean[rows], rstd[rows]])
    dy = torch.zeros_like(x)
    dy[rows[2]] = some[0]
    dx = y  # the forward's output is done with
    got = run_backward("bf16", x, w, mean, rstd, dy, None, residual=False, dx=dx)
    want, err = backward64(x[rows[2]:], w, mean[rows[2]:], rstd[rows[2]:], dy[rows[2]:], None, 0.0)
    close("dx", got[0][rows[2]:], want[0], err[0], h("bf16"), TINY["bf16"])
    close("dw", got[2], want[2], err[2] * 10, h("bf16"), TINY["bf16"])
