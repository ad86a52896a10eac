"""norm() and norm_backward() against plain 64-bit forms on the same inputs.

Tolerances are worst-case bounds, element by element.  With h the half step of
the storage type and u = 2^-24:
  * a sum over a row goes through at most 64 values in a lane, 6 exchanges and
    16 waves: D = 90 roundings, off by D u sum |terms| at most.
  * mu is off by em = D u mean |s|; d = s - mu by em + u |d|.  The squares around
    mu sum to an error of (D + 4) u of themselves, and 2 em |d| in each term;
    sum |d| <= C sqrt(var), so the variance is off by a relative
    ev = (D + 4) u + 2 em / sqrt(var + eps) + (em / sqrt(var + eps))^2, where
    the join of the waves' means adds as much again: twice that.
  * n = d rstd is off by en = (em + u |d|) rstd + |n| (ev / 2 + 4 u).
  * sums over M rows go through at most M + 16 roundings.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import binding, norm, norm_backward  # noqa: E402

from layers import DEV, HALF, IDS, TYPES, U32, generator, guarded, rand, replays, say, within  # noqa: E402

D = 90
EPS = 1e-5
KINDS = ["layer", "rms"]
SHAPES = [(1, 1), (1, 8), (3, 5), (2, 64), (5, 257), (7, 512), (4, 513), (33, 1001), (2, 2560), (3, 4096), (2, 4097),
          (2, 5120), (1, 8200), (2, 16384), (1, 32768), (1030, 600), (9001, 40), (8200, 520)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


class Plain:
    """The definition in 64 bits, and how far the kernels may be off."""

    def __init__(self, s, w, b, kind, eps=EPS, dy=None, dsum=None):
        h, C = HALF[s.dtype], s.shape[1]
        v = s.double()
        w = torch.ones(C, dtype=torch.float64, device=DEV) if w is None else w.double()
        b = torch.zeros(C, dtype=torch.float64, device=DEV) if b is None else b.double()
        layer = kind == "layer"
        self.mean = v.mean(1, keepdim=True) if layer else torch.zeros_like(v[:, :1])
        d = v - self.mean
        var = (d * d).mean(1, keepdim=True)
        dev = (var + eps).sqrt()
        self.rstd = 1 / dev
        em = D * U32 * v.abs().mean(1, keepdim=True) if layer else torch.zeros_like(dev)
        ev = 2 * ((D + 4) * U32 + 2 * em / dev + (em / dev) ** 2)
        self.mean_tol, self.rstd_tol = em + U32 * self.mean.abs(), self.rstd * (ev / 2 + 4 * U32)
        n = d * self.rstd
        en = (em + U32 * d.abs()) * self.rstd + n.abs() * (ev / 2 + 4 * U32)
        self.y = n * w + b
        self.y_tol = en * w.abs() + 2 * U32 * ((n * w).abs() + b.abs()) + h * self.y.abs() + 1e-40
        if dy is None:
            return
        g = dy.double()
        q = g * w
        mq = q.mean(1, keepdim=True) if layer else torch.zeros_like(dev)
        eq = (D + 2) * U32 * q.abs().mean(1, keepdim=True)
        sn = (q * n).mean(1, keepdim=True)
        esn = (q.abs() * en).mean(1, keepdim=True) + (D + 4) * U32 * (q * n).abs().mean(1, keepdim=True)
        inner = q - mq - n * sn
        self.dx = inner * self.rstd
        size = q.abs() + mq.abs() + (n * sn).abs()
        tol = self.rstd * (5 * U32 * size + eq + en * sn.abs() + n.abs() * esn) + self.dx.abs() * (ev / 2 + 6 * U32)
        if dsum is not None:
            self.dx = self.dx + dsum.double()
            tol = tol + U32 * dsum.double().abs()
        self.dx_tol = tol + (h + U32) * self.dx.abs() + 1e-40
        M = s.shape[0]
        self.dw, self.db = (g * n).sum(0), g.sum(0)
        self.dw_tol = (g.abs() * en).sum(0) + (M + 18) * U32 * (g * n).abs().sum(0) + h * self.dw.abs() + 1e-40
        self.db_tol = (M + 16) * U32 * g.abs().sum(0) + h * self.db.abs() + 1e-40


def inputs(M, C, dtype, seed=0, mean=0.3):
    gen = generator(seed + 7 * M + C)
    x = rand(gen, M, C, mean=mean, dtype=dtype)
    residual = rand(gen, M, C, sd=2.0, dtype=dtype)
    return (x, residual, rand(gen, C, sd=0.2, mean=1.0, dtype=dtype), rand(gen, C, sd=0.3, dtype=dtype),
            rand(gen, M, C, dtype=dtype), rand(gen, M, C, dtype=dtype))


def check(M, C, dtype, kind, residual, affine):
    x, r, w, b, dy, dsum = inputs(M, C, dtype)
    if not affine:
        w = b = None
    if not residual:
        r = dsum = None
    stat = torch.empty((M, 2), device=DEV)
    got = norm(x, w, b, residual=r, eps=EPS, kind=kind, stat=stat)
    y, s = got if residual else (got, x)
    if residual:
        assert torch.equal(s, (x.float() + r.float()).to(dtype))
    p = Plain(s, w, b, kind, dy=dy, dsum=dsum)
    within(y, p.y, p.y_tol, "y")
    within(stat[:, :1], p.mean, p.mean_tol, "mean")
    within(stat[:, 1:], p.rstd, p.rstd_tol, "rstd")
    dx, dw, db = norm_backward(dy, s, stat, w, dsum=dsum, kind=kind)
    within(dx, p.dx, p.dx_tol, "dx")
    within(dw, p.dw, p.dw_tol, "dweight")
    within(db, p.db, p.db_tol, "dbias")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,C", SHAPES)
def test_norm(M, C, kind, dtype):
    say(f"[case] norm M={M} C={C} {kind} {dtype}")
    check(M, C, dtype, kind, residual=True, affine=True)
    check(M, C, dtype, kind, residual=False, affine=M % 2 == 0)


@pytest.mark.parametrize("C", [40, 5120])
def test_mean_far_from_the_spread(C):
    """A mean 1000 times the spread costs the accuracy of the inputs' own
    last bits, not more."""
    gen = generator(3)
    x = rand(gen, 4, C, mean=1000.0)
    p = Plain(x, None, None, "layer")
    stat = torch.empty((4, 2), device=DEV)
    within(norm(x, stat=stat), p.y, p.y_tol, "y")
    within(stat[:, 1:], p.rstd, p.rstd_tol, "rstd")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rows_without_spread_and_rows_that_are_not_finite(dtype):
    x = torch.zeros((4, 600), dtype=dtype, device=DEV)
    x[1] = 3.0                      # exact in both types: the variance is exactly 0
    x[2, 5] = float("inf")
    b = torch.full((600,), 0.5, dtype=dtype, device=DEV)
    y = norm(x, None, b, kind="layer")
    assert torch.equal(y[:2], b.expand(2, 600)) and torch.equal(y[3], b)
    assert y[2].isnan().all()
    x[2, 5] = float("nan")
    y = norm(x, None, b, kind="rms")
    assert y[2].isnan().all() and y[[0, 1, 3]].isfinite().all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_sum_in_place_and_rows_at_element_alignment(dtype):
    M, C = 5, 1003
    x, r, w, b, dy, dsum = inputs(M, C, dtype, seed=9)
    want_y, want_s = norm(x, w, b, residual=r)
    for target in (0, 1):
        x2, r2 = x.clone(), r.clone()
        y, s = norm(x2, w, b, residual=r2, sum_out=(x2, r2)[target])
        assert s is (x2, r2)[target]
        assert torch.equal(y, want_y) and torch.equal(s, want_s)
        assert torch.equal((r2, x2)[target], (r, x)[target])
    stat = torch.empty((M, 2), device=DEV)
    norm(want_s, w, b, stat=stat)
    dx, dw, db = norm_backward(dy, want_s, stat, w, dsum=dsum)
    d2 = dsum.clone()
    got = norm_backward(dy, want_s, stat, w, dsum=d2, dx_out=d2)
    assert got[0] is d2 and torch.equal(d2, dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    # every array one element behind its allocation's start, outputs guarded
    shift = lambda t: guarded(t.shape, t.dtype, 1)[0].copy_(t)  # noqa: E731
    y, y_ok = guarded((M, C), dtype, 1)
    s, s_ok = guarded((M, C), dtype, 3)
    norm(shift(x), shift(w), shift(b), residual=shift(r), out=y, sum_out=s)
    assert torch.equal(y, want_y) and torch.equal(s, want_s) and y_ok() and s_ok()
    d, d_ok = guarded((M, C), dtype, 1)
    got = norm_backward(shift(dy), shift(want_s), stat, shift(w), dsum=shift(dsum), dx_out=d)
    assert torch.equal(d, dx) and torch.equal(got[1], dw) and d_ok()


def test_each_gradient_on_its_own():
    x, _, w, b, dy, dsum = inputs(40, 700, torch.bfloat16)
    stat = torch.empty((40, 2), device=DEV)
    norm(x, w, b, stat=stat)
    full = dict(zip(("dx", "dweight", "dbias"), norm_backward(dy, x, stat, w, dsum=dsum)))
    for need in ((), ("dx",), ("dweight",), ("dbias",), ("dweight", "dx")):
        got = dict(zip(("dx", "dweight", "dbias"), norm_backward(dy, x, stat, w, dsum=dsum, need=need)))
        for k, v in got.items():
            assert (v is None) == (k not in need)
            assert v is None or torch.equal(v, full[k]), k


def test_no_rows():
    x = torch.empty((0, 64), device=DEV)
    stat = torch.empty((0, 2), device=DEV)
    assert norm(x, stat=stat).shape == (0, 64)
    dx, dw, db = norm_backward(x, x, stat)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


@pytest.mark.parametrize("kind", KINDS)
def test_gradients_against_differences(kind):
    """Central differences of the 64-bit form of sum(y c), step 1e-6."""
    gen = generator(11)
    x, w, b, c = (rand(gen, 3, 37), rand(gen, 37, mean=1.0), rand(gen, 37), rand(gen, 3, 37))
    stat = torch.empty((3, 2), device=DEV)
    norm(x, w, b, kind=kind, stat=stat)
    dx, dw, db = norm_backward(c, x, stat, w, kind=kind)


    step = 1e-6
    for name, got, args, i in (("dx", dx, [x, w, b], 0), ("dw", dw, [x, w, b], 1), ("db", db, [x, w, b], 2)):
        for at in (0, 5, 36):
            up, down = [t.double() for t in args], [t.double() for t in args]
            up[i] = up[i].clone()
            down[i] = down[i].clone()
            up[i].view(-1)[at] += step
            down[i].view(-1)[at] -= step

            def plain(a):
                xx, ww, bb = a
                m = xx.mean(1, keepdim=True) if kind == "layer" else 0.0
                d = xx - m
                return float(((d / ((d * d).mean(1, keepdim=True) + EPS).sqrt() * ww + bb) * c.double()).sum())

            want = (plain(up) - plain(down)) / (2 * step)
            # the difference's own error: 2^-53 |f| / step, and step^2 of a third derivative of order 10
            assert abs(float(got.view(-1)[at]) - want) <= 1e-6 + 1e-5 * abs(want), (name, at)


@pytest.mark.parametrize("M,C", [(1, 2560), (300, 1001)])
def test_captured_replayed_and_on_another_stream(M, C):
    x, r, w, b, dy, dsum = inputs(M, C, torch.bfloat16)
    stat = torch.empty((M, 2), device=DEV)

    def call():
        y, s = norm(x, w, b, residual=r, stat=stat)
        return (y, s) + norm_backward(dy, s, stat, w, dsum=dsum)

    seeds = iter(range(100, 200))
    replays(call, [x, r, w, b, dy, dsum], lambda: inputs(M, C, torch.bfloat16, seed=next(seeds)), lambda o: o)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_same_inputs_same_bits():
    x, r, w, b, dy, dsum = inputs(5000, 520, torch.bfloat16)
    stat = torch.empty((5000, 2), device=DEV)
    first = None
    for _ in range(3):
        y, s = norm(x, w, b, residual=r, stat=stat)
        now = (y, s) + norm_backward(dy, s, stat, w, dsum=dsum)
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_refusals():
    x = torch.zeros((4, 64), device=DEV)
    stat = torch.empty((4, 2), device=DEV)
    for bad in (dict(kind="batch"), dict(weight=torch.zeros(63, device=DEV)), dict(residual=x[:2]),
                dict(sum_out=torch.empty_like(x)), dict(out=torch.empty((4, 64), device=DEV).t())):
        with pytest.raises(ValueError):
            norm(x, **bad)
    with pytest.raises(TypeError):
        norm(x.half())
    with pytest.raises(TypeError):
        norm(x, weight=torch.zeros(64, dtype=torch.bfloat16, device=DEV))
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(out=x)):
        with pytest.raises(binding.DSparkError):
            norm(x, **bad)
    with pytest.raises(binding.DSparkError):
        norm(torch.zeros((1, 32769), device=DEV))
    with pytest.raises(ValueError):
        norm_backward(x, x, stat, need=("dw",))
    with pytest.raises(ValueError):
        norm_backward(x, x, stat, need="dbias", dx_out=torch.empty_like(x))
    w = torch.ones(64, device=DEV, requires_grad=True)
    with pytest.raises(RuntimeError, match="autograd"):
        norm(x, w)
    with torch.no_grad():
        norm(x, w)
