"""Two calls of the layer norm, the dropout or the 8-bit linear layer at once: each with its own
scratch and outputs, on streams of their own or captured into graphs of their own, they
give the bits that they give alone."""
import pytest

import convolution_forward_amd as cf

torch = pytest.importorskip("torch")

from test_gpu_layer_norm import OFFSET, SEED, T, inputs, ws_of  # noqa: E402
from test_gpu_linear import gen, rnd, stream  # noqa: E402
from test_gpu_linear_int8 import whole8  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cf.lib()


def nan(*shape, t=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=t, device="cuda")


class Norm:
    """A forward and a backward pass with dropout and residual."""

    def __init__(self, m, n, seed):
        self.size, self.seed = (m, n), seed
        self.x, self.r, self.w, self.b = inputs("bf16", m, n, seed=seed)
        self.dy = inputs("bf16", m, n, seed=seed + 50)[0]
        self.step = torch.full((1,), seed, dtype=torch.int64, device="cuda")
        self.out = [nan(m, n), nan(m, n), nan(m, t=torch.float32), nan(m, t=torch.float32),
                    nan(m, n), nan(m, n), nan(n), nan(n)]
        self.p = cf.make_layer_norm_problem(m, n, residual=True, drop=0.2, seed=SEED, offset=OFFSET)
        self.bytes = [cf.layer_norm_scratch_size(self.p, "bf16"),
                      cf.layer_norm_backward_scratch_size(self.p, "bf16")]
        self.room = [ws_of(v) for v in self.bytes]

    def renew(self, seed):
        self.x.copy_(inputs("bf16", *self.size, seed=seed + self.seed)[0])

    def call(self):
        y, s, mean, rstd, dx, dr, dw, db = self.out
        cf.layer_norm_forward(self.p, "bf16", self.x, self.r, self.w, self.b, y, s, mean, rstd,
                              self.step, self.room[0], self.bytes[0], stream())
        cf.layer_norm_backward(self.p, "bf16", s, self.w, mean, rstd, self.dy, self.r, dx, dr, dw, db,
                               self.step, self.room[1], self.bytes[1], stream())


class Drop:
    def __init__(self, m, n, seed):
        self.size, self.seed = (m, n), seed
        self.x, self.r = inputs("bf16", m, n, seed=seed)[:2]
        self.out = [nan(m, n), nan(m, n)]
        self.step = torch.full((1,), seed, dtype=torch.int64, device="cuda")
        self.p = cf.make_dropout_problem(m, n, 0.25, seed=SEED, residual=True)

    def renew(self, seed):
        self.x.copy_(inputs("bf16", *self.size, seed=seed + self.seed)[0])

    def call(self):
        cf.dropout_forward(self.p, "bf16", self.x, self.r, self.out[0], self.step, stream())
        cf.dropout_backward(self.p, "bf16", self.x, self.out[1], self.step, stream())


class Int8:
    """Rows to 8 bits and their product."""

    def __init__(self, m, n, k, seed):
        g = gen(seed)
        self.size, self.seed = (m, k), seed
        self.x, self.w = rnd(g, "bf16", m, k), whole8(g, n, k)
        self.ws = torch.rand(n, generator=g, device="cuda")
        self.q = torch.zeros(m, k, dtype=torch.int8, device="cuda")
        self.xs = nan(m, t=torch.float32)
        self.out = [nan(m, n)]
        self.z, self.p = cf.make_quantize_problem(m, k), cf.make_linear_int8_problem(m, n, k)
        self.bytes = cf.linear_int8_scratch_size(self.p, "bf16")
        self.room = ws_of(self.bytes)

    def renew(self, seed):
        self.x.copy_(rnd(gen(seed + self.seed), "bf16", *self.size))

    def call(self):
        cf.quantize_rows(self.z, "bf16", self.x, self.q, self.xs, stream())
        cf.linear_int8_forward(self.p, "bf16", self.q, self.xs, self.w, self.ws, None, None,
                               self.out[0], self.room, self.bytes, stream())


# a row in registers; long rows in parts; partial rows of dw and db; the backward's parts with
# and without columns beside them; planes of a split; packed rows
JOBS = [(Norm, (70, 600), ""), (Norm, (6, 50_000), "split13 split25.once"), (Norm, (4000, 264), "rows64x1 rows64x1"),
        (Norm, (1100, 2047), "rows256x1 rows256x1"), (Norm, (300, 40_000), "split10 split20"),
        (Drop, (900, 1001), ""), (Int8, (64, 256, 4096), "split"), (Int8, (50, 100, 1531), "split"),
        (Int8, (1981, 4350, 1560), "pack"), (Int8, (16, 2048, 2048), "stream")]


def pair(kind, size, plan):
    jobs = [kind(*size, seed=s) for s in (1, 2)]
    p = jobs[0].p
    if kind is Norm:
        names = (cf.layer_norm_describe_variant(p, "bf16"), cf.layer_norm_backward_describe_variant(p, "bf16"))
        for name, part in zip(names, plan.split()):
            assert name.endswith(part), names
    elif kind is Int8:
        assert plan in cf.linear_int8_describe_variant(p, "bf16")
    return jobs


def alone(jobs):
    """What each gives by itself; its outputs are NaN again afterwards."""
    want = []
    for j in jobs:
        j.call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in j.out])
        for t in j.out:
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    return want


def agree(jobs, want):
    return all(torch.equal(a, b) for j, w in zip(jobs, want) for a, b in zip(j.out, w))


@pytest.mark.parametrize("kind,size,plan", JOBS)
def test_two_streams(kind, size, plan):
    jobs = pair(kind, size, plan)
    want = alone(jobs)
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        for _ in range(8):  # nothing waits in between
            for j, s in zip(jobs, streams):
                with torch.cuda.stream(s):
                    j.call()
        torch.cuda.synchronize()
        assert agree(jobs, want)


@pytest.mark.parametrize("kind,size,plan", JOBS)
def test_two_graphs(kind, size, plan):
    jobs = pair(kind, size, plan)
    alone(jobs)
    graphs = []
    for j in jobs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            j.call()
    streams = [torch.cuda.Stream() for _ in jobs]
    eager = kind(*size, seed=3)
    for i in range(4):
        for j in jobs:
            j.renew(10 * (i + 1))
        want = alone(jobs)
        if i % 2:  # one after the other, with eager work in between
            graphs[0].replay()
            eager.call()
            graphs[1].replay()
        else:  # side by side
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert agree(jobs, want), i
