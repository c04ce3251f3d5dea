"""GPU parity of row quantization and the 8-bit linear layer (include/linear_int8.h).

Quantization is compared exactly: the largest |x|, two float32 divisions, a float32
product and a rounding to even are the same on the host.  The product's integer sums
are exact; with u = 2^-24 the value before the bias is off by 3 u of itself (the sum's
rounding to float32, the product of the scales, their product), bias and residual add
a u each, the activation passes errors on with its largest slope and adds 16 u of
argument and value, and the result is rounded once (h).  Scales that are powers of two
and small sums make every step exact: those are compared bit for bit."""
import numpy as np
import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_linear import (ACTS, PARAM, T, TINY, U, act64, act_error, close, gen, rnd,  # noqa: E402
                             scratch, strided, stream)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


# ---------------------------------------------------------------- quantization

def quantize(dtype, x, q=None):
    m, n = x.shape
    q = torch.full((m, n), 99, dtype=torch.int8, device="cuda") if q is None else q
    scale = torch.full((m,), -1.0, device="cuda")
    p = cf.make_quantize_problem(m, n, ldx=x.stride(0), ldq=q.stride(0))
    cf.quantize_rows(p, dtype, x, q, scale, stream())
    return q, scale


def quantized(x):
    """q and scale by the definition, in numpy's float32."""
    v = x.float().cpu().numpy()
    top = np.abs(v).max(1)  # NaN where there is one
    bad = ~np.isfinite(top)
    small = top < np.float32(2.0 ** -100)
    with np.errstate(all="ignore"):
        scale = np.where(small, np.float32(0), top / np.float32(127)).astype(np.float32)
        inv = np.where(small | bad, np.float32(0), np.float32(127) / top).astype(np.float32)
        q = np.rint(v * inv[:, None])
    q[bad] = 0
    scale[bad] = np.nan
    return torch.from_numpy(q.astype(np.int8)), torch.from_numpy(scale)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n", [(1, 1), (3, 5), (4, 8), (9, 511), (6, 520), (777, 1001), (5, 2048),
                                 (3, 4097), (2, 8192), (4, 8193), (2, 32768), (3, 32769),
                                 (2, 100_001), (1000, 24)])
def test_quantize(dtype, m, n):
    x = rnd(gen(m + n), dtype, m, n, scale=3.0)
    x[m // 2] = 0
    q, s = quantize(dtype, x)
    wq, wsc = quantized(x)
    assert torch.equal(s.cpu(), wsc) and torch.equal(q.cpu(), wq)


@pytest.mark.parametrize("n", [7, 300, 3000, 9000, 40_000])
def test_quantize_borders(n):
    """Ties, the smallest and largest values, rows that are not finite."""
    x = torch.zeros(9, n, device="cuda")
    x[0] = torch.arange(n, device="cuda") % 254 - 127 + 0.5  # halves, with 127 as the largest
    x[0, 0] = 127
    x[1] = 3e38
    x[2] = 1e-42  # subnormal
    x[3] = 2.0 ** -100
    x[4] = 2.0 ** -101
    x[5, n - 1] = float("inf")
    x[6, n // 2] = float("nan")
    x[7, 0] = -float("inf")
    x[8, n - 1] = -5.0
    q, s = quantize("f32", x)
    wq, wsc = quantized(x)
    assert torch.equal(q.cpu(), wq)
    assert torch.equal(s.cpu().nan_to_num(-7.0), wsc.nan_to_num(-7.0))
    assert int(torch.isnan(s).sum()) == 3 and float(s[4]) == 0.0 and float(s[3]) > 0.0
    assert int(q[8, n - 1]) == -127


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [5, 1001, 4099, 33_001])
def test_quantize_strides(dtype, n):
    """Rows of wider buffers at odd places; what lies between the rows stays."""
    x = rnd(gen(n), dtype, 6, n)
    _, xv = strided(x, 5, 3)
    buf = torch.full((6 * (n + 9) + 20,), 77, dtype=torch.int8, device="cuda")
    q = buf[7:7 + 6 * (n + 9)].view(6, n + 9)[:, :n]
    _, s = quantize(dtype, xv, q)
    wq, wsc = quantized(x)
    assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu(), wsc)
    q.fill_(77)
    assert bool((buf == 77).all())


def test_quantize_offsets_and_no_rows():
    x = rnd(gen(0), "bf16", 5, 33)
    arena = torch.zeros(400, dtype=torch.bfloat16, device="cuda")
    arena[3:168] = x.reshape(-1)
    q, s = torch.zeros(400, dtype=torch.int8, device="cuda"), torch.zeros(20, device="cuda")
    cf.quantize_rows(cf.make_quantize_problem(5, 33, offsets=(3, 11, 2)), "bf16", arena, q, s, stream())
    wq, wsc = quantized(x)
    assert torch.equal(q[11:176].view(5, 33).cpu(), wq) and torch.equal(s[2:7].cpu(), wsc)
    assert not q[:11].any() and not q[176:].any() and not s[:2].any() and not s[7:].any()
    assert cf.quantize_rows(cf.make_quantize_problem(0, 33), "bf16", None, None, None, stream()) == 0


# -------------------------------------------------------------- the 8-bit product

def whole8(g, m, k):
    return torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)


def forward(dtype, x, xs, w, ws, b=None, r=None, y=None, act="identity", res="none", use=None):
    m, k = x.shape
    n = w.shape[0]
    y = torch.full((m, n), float("nan"), dtype=T[dtype], device="cuda") if y is None else y
    a, be = PARAM.get(act, (0.0, 0.0))
    p = cf.make_linear_int8_problem(m, n, k, act=act, alpha=a, beta=be, bias=b is not None,
                                    residual=res, ldx=x.stride(0), ldw=w.stride(0),
                                    ldr=0 if r is None else r.stride(0), ldy=y.stride(0))
    size = cf.linear_int8_scratch_size(p, dtype)
    s = scratch(size)
    cf.linear_int8_forward(p, dtype, x, xs, w, ws, b, r, y, s, size, stream())
    if use is not None:
        use.append((p, s, size))
    return y


def forward64(x, xs, w, ws, b, r, act, res):
    """y and its bound before the final rounding."""
    acc = x.double() @ w.double().t()  # exact: whole numbers below 2^53
    z = acc * xs.double()[:, None] * ws.double()
    e = 3 * U * z.abs()
    if b is not None:
        z = z + b.double()
        e = e + U * z.abs()
    if res == "before":
        z = z + r.double()
        e = e + U * z.abs()
    y = act64(z, act)[0]
    e = act_error(z, y, e, act)
    if res == "after":
        y = y + r.double()
        e = e + U * y.abs()
    return y, e * (1 + 1e-5)


def operands(dtype, m, n, k, seed=0):
    g = gen(seed)
    x, w = whole8(g, m, k), whole8(g, n, k)
    xs = torch.rand(m, generator=g, device="cuda") * 0.02 + 0.001
    ws = torch.rand(n, generator=g, device="cuda") * 0.01 / k ** 0.5 + 0.0001
    return x, xs, w, ws, rnd(g, dtype, n), rnd(g, dtype, m, n)


# few rows (streamed), small and split tiles, large ones; whole and odd k
SIZES = [(1, 1, 1), (1, 8, 16), (3, 5, 7), (2, 33, 15), (1, 1000, 2048), (7, 100, 1531), (16, 256, 640),
         (17, 300, 512), (32, 64, 4096), (33, 1001, 240), (64, 256, 4096), (129, 130, 131),
         (200, 300, 1001), (300, 520, 384), (777, 1001, 1531), (1000, 768, 512), (2048, 1024, 256),
         (2100, 4096, 272)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_forward(dtype, m, n, k):
    x, xs, w, ws, b, r = operands(dtype, m, n, k, seed=m + n + k)
    for act, res, bias in (("identity", "none", False), ("gelu", "before", True), ("silu", "after", True)):
        got = forward(dtype, x, xs, w, ws, b if bias else None, None if res == "none" else r,
                      act=act, res=res)
        want, err = forward64(x, xs, w, ws, b if bias else None, r, act, res)
        close(f"{act} {res}", got, want, err, dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [5, 150])
def test_activations(act, m):
    x, xs, w, ws, b, r = operands("f16", m, 96, 200)
    for res in ("before", "after"):
        got = forward("f16", x, xs, w, ws, b, r, act=act, res=res)
        want, err = forward64(x, xs, w, ws, b, r, act, res)
        close(f"{act} {res}", got, want, err, "f16")


@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (20, 40, 1000), (128, 128, 512), (700, 513, 131),
                                   (2048, 2048, 128)])
def test_exact_in_float32(m, n, k):
    """Scales of powers of two and sums below 2^24: bit for bit, whatever the plan."""
    g = gen(k)
    x = torch.randint(-100, 101, (m, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    xs = 2.0 ** torch.randint(-6, 7, (m,), generator=g, device="cuda")
    ws = 2.0 ** torch.randint(-6, 7, (n,), generator=g, device="cuda")
    want = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    assert torch.equal(forward("f32", x, xs, w, ws).double(), want)


@pytest.mark.parametrize("m,n", [(1, 3), (17, 20), (40, 300), (300, 300)])
def test_longest_k(m, n):
    """-128 times -128 over the whole of k = 131071: 2^31 - 2^14, the largest sum."""
    k = 131071
    x = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    one = lambda q: torch.ones(q, device="cuda")  # noqa: E731
    y = forward("f32", x, one(m), w, one(n))
    assert bool((y == float(np.float32(128 * 128 * k))).all())
    w[:] = 127
    y = forward("f32", x, one(m), w, one(n))
    assert bool((y == float(np.float32(-128 * 127 * k))).all())


@pytest.mark.parametrize("m,n,k", [(3, 50, 200), (20, 70, 333), (100, 130, 1024), (600, 700, 500)])
def test_positions(m, n, k):
    """One element of x and of w apiece: every output is its own product or 0."""
    g = gen(m)
    x, w = (torch.zeros(q, k, dtype=torch.int8, device="cuda") for q in (m, n))
    ix, iw = (torch.randint(0, k, (q,), generator=g, device="cuda") for q in (m, n))
    iw[: min(m, n)] = ix[: min(m, n)]
    vx, vw = (torch.randint(1, 128, (q,), generator=g, device="cuda", dtype=torch.int8) for q in (m, n))
    x[torch.arange(m), ix] = vx
    w[torch.arange(n), iw] = vw
    want = (ix[:, None] == iw).double() * vx.double()[:, None] * vw.double()
    y = forward("f32", x, torch.ones(m, device="cuda"), w, torch.ones(n, device="cuda"))
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("m,n,k,pad,off", [(1, 100, 160, 16, 16), (9, 64, 333, 3, 1), (16, 40, 512, 1, 2),
                                           (40, 200, 1000, 5, 3), (130, 257, 640, 4, 4),
                                           (600, 520, 259, 7, 5), (300, 300, 512, 16, 8)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_what_lies_between_rows(dtype, m, n, k, pad, off):
    """Operands in rows of wider buffers at any byte, other values around them."""
    x, xs, w, ws, b, r = operands(dtype, m, n, k)

    def wide(t, pad, off):
        ld = t.shape[1] + pad
        buf = torch.full((off + t.shape[0] * ld + 64,), 113, dtype=t.dtype, device="cuda")
        v = buf[off:off + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
        v.copy_(t)
        return v

    _, rv = strided(r, pad, off)
    buf, y = strided(torch.zeros_like(r), pad + 1, off + 1)
    forward(dtype, wide(x, pad, off), xs, wide(w, pad + 2, off + 1), ws, b, rv, y=y, res="before")
    want, err = forward64(x, xs, w, ws, b, r, "identity", "before")
    close("strided", y, want, err, dtype)
    assert int(torch.isnan(buf).sum()) == buf.numel() - y.numel()


def test_offsets_in_place_and_no_rows():
    m, n, k = 5, 24, 48
    x, xs, w, ws, b, r = operands("f16", m, n, k)
    want = forward("f16", x, xs, w, ws, b, r, res="after")
    arenas = []
    offs = (7, 3, 5, 2, 9, 4, 6)
    for t, o in zip((x, xs, w, ws, b, r, torch.zeros_like(r)), offs):
        buf = torch.zeros(o + t.numel() + 40, dtype=t.dtype, device="cuda")
        buf[o:o + t.numel()] = t.reshape(-1)
        arenas.append(buf)
    p = cf.make_linear_int8_problem(m, n, k, bias=True, residual="after", offsets=offs)
    size = cf.linear_int8_scratch_size(p, "f16")
    cf.linear_int8_forward(p, "f16", *arenas, scratch(size), size, stream())
    assert torch.equal(arenas[6][6:6 + m * n].view(m, n), want)
    c = r.clone()
    assert torch.equal(forward("f16", x, xs, w, ws, b, c, y=c, res="after"), want)
    p = cf.make_linear_int8_problem(0, n, k)
    assert cf.linear_int8_forward(p, "f16", None, None, w, ws, None, None, None, stream=stream()) == 0


def test_scales_that_are_not_finite():
    """A NaN scale (a row that held a NaN) makes its row NaN and no other."""
    x, xs, w, ws, b, r = operands("bf16", 40, 60, 128)
    xs[7] = float("nan")
    x[7] = 0
    y = forward("bf16", x, xs, w, ws, b)
    assert torch.isnan(y[7]).all() and int(torch.isnan(y).sum()) == 60
    z = torch.zeros(3, 128, device="cuda", dtype=torch.bfloat16)
    z[1, 5] = float("inf")
    q, s = quantize("bf16", z)
    y = forward("bf16", q, s, w, ws)
    assert torch.isnan(y[1]).all() and not y[0].any() and not y[2].any()


def test_plans_agree():
    """The same rows alone (streamed), among a few (split) and among many (large tiles)
    give the same bits: integer sums do not depend on the plan."""
    x, xs, w, ws, b, _ = operands("f32", 2560, 2048, 2048)
    names = set()
    use = []
    big = forward("f32", x, xs, w, ws, b, use=use)
    for rows in (1, 5, 20, 33, 64, 200, 600):
        part = forward("f32", x[:rows], xs[:rows], w, ws, b, use=use)
        assert torch.equal(part, big[:rows]), rows
    for p, _, _ in use:
        names.add(cf.linear_int8_describe_variant(p, "f32").split(".")[2])
    assert len(names) >= 3, names


@pytest.mark.parametrize("m,n,k,plan", [
    (1, 5, 17, "stream16.r4"), (3, 1293, 17, "stream16.r8"), (1, 2284, 17, "stream16.r16"),
    (20, 4, 20, "stream32.r4"), (20, 1117, 18, "stream32.r8"), (24, 2585, 17, "stream32.r16"),
    (25, 4566, 20, "stream32.r32"), (35, 4, 1372, "split"), (1, 4, 4, "tile64x64"),
    (2497, 2749, 32, "tile128x128"), (2001, 2003, 1001, "tile128x128"),
    (1691, 4544, 1856, "tile256x128"), (2229, 3712, 1728, "tile256x256"),
    (2033, 9750, 1552, "cut"), (1900, 9750, 1552, "cut"), (1981, 4350, 1560, "tile256x256.pack"),
    (1202, 2505, 3846, "tile64x64.pack")])
def test_every_plan(m, n, k, plan):
    """Each kernel at sizes that the plan gives it, ends inside its tiles."""
    x, xs, w, ws, b, r = operands("bf16", m, n, k, seed=k)
    use = []
    got = forward("bf16", x, xs, w, ws, b, r, act="relu", res="before", use=use)
    name = cf.linear_int8_describe_variant(use[0][0], "bf16")
    assert plan in name, name
    want, err = forward64(x, xs, w, ws, b, r, "relu", "before")
    close(name, got, want, err, "bf16")


@pytest.mark.parametrize("m,n,k", [(4, 500, 1024), (64, 256, 4096), (50, 100, 1531), (1000, 1000, 777)])
def test_rerun_graph_and_streams(m, n, k):
    """The whole path, quantization and product: reruns and replays are equal."""
    g = gen(5)
    a = rnd(g, "bf16", m, k)
    w, ws = whole8(g, n, k), torch.rand(n, generator=g, device="cuda")
    q, s = torch.zeros(m, k, dtype=torch.int8, device="cuda"), torch.zeros(m, device="cuda")
    y = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    p, z = cf.make_linear_int8_problem(m, n, k, act="relu"), cf.make_quantize_problem(m, k)
    size = cf.linear_int8_scratch_size(p, "bf16")
    room = scratch(size)

    def call():
        cf.quantize_rows(z, "bf16", a, q, s, stream())
        cf.linear_int8_forward(p, "bf16", q, s, w, ws, None, None, y, room, size, stream())

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        a.copy_(rnd(gen(30 + i), "bf16", m, k))
        call()
        want = y.clone()
        y.zero_(), q.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        close("replay", y, *forward64(q, s, w, ws, None, None, "relu", "none"), "bf16")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(y, want)


def test_past_32_bits():
    """x and y of more than 2^31 elements; rows from both ends."""
    m, n, k = 70_000, 32_768, 32_768
    g = gen(1)
    x = torch.zeros(m, k, dtype=torch.int8, device="cuda")
    rows = [0, 40_000, m - 1]
    x[rows] = whole8(g, 3, k)
    w = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    some = [0, 17, n - 1]
    w[some] = whole8(g, 3, k)
    one = lambda q: torch.full((q,), 2.0 ** -16, device="cuda")  # noqa: E731
    y = forward("f16", x, one(m), w, one(n), y=torch.empty(m, n, dtype=torch.float16, device="cuda"))
    want = (x[rows].double() @ w[some].double().t()) * 2.0 ** -32
    got = y[rows][:, some].double()
    assert bool(((got - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -25).all())
    assert not y[1:1000].any() and not y[rows][:, 1:17].any()
