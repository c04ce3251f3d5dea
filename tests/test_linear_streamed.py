"""The streamed kernels of the linear and gated calls (include/linear.h), every one of
them: which plan a size gets (CPU), and small whole numbers through it, exactly."""
import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_linear import T, forward, gated, gen, strided, whole

# rows of x, outputs, the plan: 16 or 32 rows of x, weight rows of a workgroup
PLANS = [(1, 1000, "stream16.r4"), (16, 1300, "stream16.r8"), (3, 4001, "stream16.r16"),
         (17, 700, "stream32.r4"), (17, 1500, "stream32.r8"), (32, 2041, "stream32.r8"),
         (20, 2500, "stream32.r16"), (32, 5000, "stream32.r32")]


def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,name", PLANS)
@pytest.mark.parametrize("k,pad", [(200, 0), (201, 0), (200, 5)])
def test_plans(m, n, k, pad, name, dtype):
    p = cf.make_linear_problem(m, n, k, ldx=k + pad, ldw=k + pad)
    assert cf.linear_describe_variant(p, dtype) == f"linear.{dtype}.{name}"
    p = cf.make_gated_problem(m, n, k, ldx=k + pad, ldw=k + pad)
    assert cf.gated_describe_variant(p, dtype) == f"gated.{dtype}.{name}"


def test_every_streamed_plan_is_named():
    """Over many sizes no other streamed plan comes up than those above."""
    seen = set()
    for dtype in ("f16", "f32"):
        for m in (1, 2, 7, 16, 17, 25, 32):
            for n in [int(1.25 ** i) for i in range(4, 48)]:
                for k in (8, 65, 264, 1001, 4096, 9000):
                    p = cf.make_linear_problem(m, n, k)
                    seen.add(cf.linear_describe_variant(p, dtype).split(".", 2)[2])
                    p = cf.make_gated_problem(m, n, k)
                    seen.add(cf.gated_describe_variant(p, dtype).split(".", 2)[2])
    assert {s for s in seen if s.startswith("stream")} == {name for _, _, name in PLANS}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,name", PLANS)
@pytest.mark.parametrize("k,pad", [(200, 0), (201, 0), (200, 5)])
def test_linear(m, n, k, pad, name, dtype):
    device()
    g = gen(m + n + k)
    x, w = whole(g, dtype, m, k), whole(g, dtype, n, k)
    if pad:
        x, w = strided(x, pad, 3)[1], strided(w, pad, 1)[1]
    b, r = whole(g, dtype, n, lo=-8, hi=9), whole(g, dtype, m, n, lo=-8, hi=9)
    y, z = forward(dtype, x, w, b, r, act="relu", res="before", save=True)
    want = x.double() @ w.double().t() + b.double() + r.double()
    assert torch.equal(z, want.to(T[dtype])) and torch.equal(y, want.clamp(min=0).to(T[dtype]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,f,name", PLANS)
@pytest.mark.parametrize("k,pad", [(200, 0), (201, 0), (200, 5)])
def test_gated(m, f, k, pad, name, dtype):
    device()
    g = gen(m + f + k)
    x, wg, wu = (whole(g, dtype, *s, lo=-1, hi=2) for s in ((m, k), (f, k), (f, k)))
    if pad:
        x, wg, wu = strided(x, pad, 3)[1], strided(wg, pad, 1)[1], strided(wu, pad, 1)[1]
    bg, bu = whole(g, dtype, f), whole(g, dtype, f)
    a, b = x.double() @ wg.double().t() + bg.double(), x.double() @ wu.double().t() + bu.double()
    out, pg, pu = gated(dtype, x, wg, wu, bg, bu, act="relu", save=True)
    assert torch.equal(pg, a.to(T[dtype])) and torch.equal(pu, b.to(T[dtype]))
    assert torch.equal(out, (a.clamp(min=0) * b).to(T[dtype]))
