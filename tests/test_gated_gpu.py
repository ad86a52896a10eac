"""gated_linear() and gated_linear_backward() against plain 64-bit forms on the
same inputs.

Tolerances are worst-case bounds, element by element.  With h the half step of
the storage type and u = 2^-24:
  * a sum of K products in fp32, in any order, is off by at most (K + 2) u
    sum |terms|; the matrix unit may truncate where IEEE rounds, which doubles
    u: E = 2 (K + 8) u sum |terms|.
  * act' and act'' of relu away from 0, gelu and silu are below 1.2, so an error
    e in z moves act(z), and act'(z), by at most 1.2 e; act and act' themselves
    are computed within 16 u (|z| + 1).
  * a result rounded to the type once is off by h times itself more, and dz,
    rounded to the type before its products, by h |dz| in every term.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import binding, gated_linear, gated_linear_backward  # noqa: E402

from layers import DEV, HALF, IDS, TYPES, U32, generator, guarded, rand, replays, say, within  # noqa: E402

ACTS = ["none", "relu", "gelu", "silu"]
SHAPES = [(1, 1, 1), (1, 17, 8), (2, 3, 5), (1, 130, 64), (3, 64, 200), (8, 256, 64), (16, 300, 129), (17, 33, 65),
          (31, 128, 72), (64, 256, 128), (77, 131, 1001), (129, 257, 192), (255, 520, 333), (300, 512, 256),
          (1, 4096, 520), (8, 2000, 2056), (513, 96, 40), (257, 1027, 136), (16, 5000, 64), (40, 64, 4096), (3, 50, 1001), (16, 33, 191),
          (1, 70, 4095), (5, 19, 127)]
NAMES = ("dx", "dwg", "dwu", "dbg", "dbu")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


def act64(act, z):
    """act and its slope."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    return z, torch.ones_like(z)


class Plain:
    def __init__(self, x, wg, wu, bg, bu, act, dy=None):
        half, u, K = HALF[x.dtype], U32, x.shape[1]
        wide = lambda t: t.double()  # noqa: E731
        e = 2 * (K + 8) * u
        self.z, tol = [], []
        for w, b in ((wg, bg), (wu, bu)):
            z, size = wide(x) @ wide(w).T, wide(x).abs() @ wide(w).abs().T
            if b is not None:
                z, size = z + wide(b), size + wide(b).abs()
            self.z.append(z)
            tol.append(e * size)
        g, v = self.z
        eg, ev = tol
        self.z_tol = [t + 1e-40 for t in tol]
        a, slope = act64(act, g)
        ea = 1.2 * eg + 16 * u * (g.abs() + 1)
        es = 1.2 * eg + 16 * u * (g.abs() + 1)
        if act == "relu":      # inputs whose sums round across the step are kept out by the caller
            es = torch.zeros_like(es)
        self.y = a * v
        self.y_tol = ea * v.abs() + a.abs() * ev + ea * ev + 2 * u * self.y.abs() + half * self.y.abs() + 1e-40
        if dy is None:
            return
        d = wide(dy)
        dg, du = d * v * slope, d * a
        tg = d.abs() * (ev * slope.abs() + v.abs() * es + ev * es) + 3 * u * dg.abs()
        tu = d.abs() * ea + 2 * u * du.abs()
        M, N = d.shape
        self.grads, self.tols = {}, {}

        def put(name, value, t):
            self.grads[name], self.tols[name] = value, t + half * value.abs() + 1e-40

        put("dbg", dg.sum(0), tg.sum(0) + (M + 8) * u * dg.abs().sum(0))
        put("dbu", du.sum(0), tu.sum(0) + (M + 8) * u * du.abs().sum(0))
        tg, tu = tg + half * dg.abs(), tu + half * du.abs()        # rounded before the products
        ag, au = wide(wg).abs(), wide(wu).abs()
        e = 2 * (2 * N + 8) * u
        put("dx", dg @ wide(wg) + du @ wide(wu), tg @ ag + tu @ au + e * ((dg.abs() + tg) @ ag + (du.abs() + tu) @ au))
        e, ax = 2 * (M + 8) * u, wide(x).abs()
        put("dwg", dg.T @ wide(x), tg.T @ ax + e * ((dg.abs() + tg).T @ ax))
        put("dwu", du.T @ wide(x), tu.T @ ax + e * ((du.abs() + tu).T @ ax))


def inputs(M, N, K, dtype, seed=0, bias=True):
    gen = generator(seed + M + 3 * N + 5 * K)
    sd = math.sqrt(2.0 / max(K, 1))
    x, wg, wu = rand(gen, M, K, dtype=dtype), rand(gen, N, K, sd=sd, dtype=dtype), rand(gen, N, K, sd=sd, dtype=dtype)
    bg, bu = (rand(gen, N, sd=0.5, dtype=dtype), rand(gen, N, sd=0.5, dtype=dtype)) if bias else (None, None)
    return x, wg, wu, bg, bu, rand(gen, M, N, dtype=dtype)


def check(M, N, K, dtype, act, bias):
    x, wg, wu, bg, bu, dy = inputs(M, N, K, dtype, bias=bias)
    out, ok = guarded((M, N), dtype, 3)
    pre, pre_ok = guarded((2, M, N), torch.float32, 1)
    y = gated_linear(x, wg, wu, bg, bu, act=act, pre=pre, out=out)
    assert y is out and ok() and pre_ok()
    if act == "relu":      # the gradient is that of the side of the step which the sums were rounded to
        dy = torch.where(pre[0].abs() > 1e-3, dy, torch.zeros_like(dy))
    p = Plain(x, wg, wu, bg, bu, act, dy)
    within(pre[0], p.z[0], p.z_tol[0], "zg")
    within(pre[1], p.z[1], p.z_tol[1], "zu")
    within(y, p.y, p.y_tol, "y")
    assert torch.equal(gated_linear(x, wg, wu, bg, bu, act=act), y)
    got = gated_linear_backward(dy, x, wg, wu, pre.clone(), act=act)
    for name, g in zip(NAMES, got):
        within(g, p.grads[name], p.tols[name], name)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_gated_linear(i, dtype):
    M, N, K = SHAPES[i]
    for act in {ACTS[i % 4], "silu"}:
        say(f"[case] gated {M} x {N} x {K} {act} {dtype}")
        check(M, N, K, dtype, act, bias=i % 3 != 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_activations(act, dtype):
    check(50, 70, 96, dtype, act, bias=True)
    check(5, 70, 96, dtype, act, bias=False)


@pytest.mark.parametrize("M,N,K", [(1500, 2056, 1096), (4000, 1032, 520), (2050, 1024, 1032), (2400, 10000, 2600),
                                   (2700, 2560, 5120), (4503, 2000, 4104)])
def test_large_tiles(M, N, K):
    say(f"[case] gated {M} x {N} x {K}")
    check(M, N, K, torch.bfloat16, "silu", bias=True)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(40, 0, 8), (0, 40, 8), (4, 40, 0), (40, 33, 0), (0, 12, 9)])
def test_empty(M, N, K, dtype):
    x, wg, wu, bg, bu, dy = inputs(M, N, K, dtype)
    pre = torch.empty((2, M, N), device=DEV)
    y = gated_linear(x, wg, wu, bg, bu, act="none", pre=pre)
    assert y.shape == (M, N)
    if M and N:      # no inputs: the biases alone
        within(y, (bg.double() * bu.double()).expand(M, N), HALF[dtype] * (bg.double() * bu.double()).abs().expand(M, N) +
               U32, "y")
    got = dict(zip(NAMES, gated_linear_backward(dy, x, wg, wu, pre, act="none")))
    for name in ("dx", "dwg", "dwu") + (() if M else ("dbg", "dbu")):
        assert not got[name].any(), name
    if K == 0:
        p = Plain(x, wg, wu, bg, bu, "none", dy)
        for name in ("dbg", "dbu"):
            within(got[name], p.grads[name], p.tols[name], name)


@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (40, 300, 128), (300, 264, 72), (40, 100, 99)])
def test_each_gradient_on_its_own(M, N, K):
    x, wg, wu, bg, bu, dy = inputs(M, N, K, torch.bfloat16)
    pre = torch.empty((2, M, N), device=DEV)
    gated_linear(x, wg, wu, bg, bu, pre=pre)
    full = dict(zip(NAMES, gated_linear_backward(dy, x, wg, wu, pre)))
    for need in ((), ("dx",), ("dwg",), ("dwu",), ("dbg",), ("dbu",), ("dx", "dbu")):
        got = dict(zip(NAMES, gated_linear_backward(dy, x, wg, wu, pre, need=need)))
        for k, v in got.items():
            assert (v is None) == (k not in need)
            # the bias sums' chunks are longer than those of a pass without them: the products see the same dz
            assert v is None or torch.equal(v, full[k]), k


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (40, 300, 129), (300, 264, 4104)])
def test_what_is_not_finite_stays_in_its_row(M, N, K, dtype):
    x, wg, wu, bg, bu, _ = inputs(M, N, K, dtype)
    want = gated_linear(x, wg, wu, bg, bu)
    for value in (float("inf"), float("nan")):
        bad = x.clone()
        bad[1, K - 1] = value
        y = gated_linear(bad, wg, wu, bg, bu)
        keep = [r for r in range(M) if r != 1]
        assert torch.equal(y[keep], want[keep]) and not y[1].isfinite().all()
    # an infinite gate weight in the last column: gelu and silu of -inf are 0 times it, so NaN; of +inf, infinite
    w = wg.clone()
    w[2, K - 1] = float("inf")
    y = gated_linear(x, w, wu, bg, bu)
    cols = [c for c in range(N) if c != 2]
    assert torch.equal(y[:, cols], want[:, cols]) and not y[:, 2].isfinite().all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (40, 300, 129), (100, 130, 4100), (20, 70, 1001), (300, 264, 1032)])
def test_workspace_of_the_stated_size_is_enough(M, N, K, dtype):
    x, wg, wu, bg, bu, dy = inputs(M, N, K, dtype)
    code = binding.DSPARK_BF16 if dtype is torch.bfloat16 else binding.DSPARK_F32
    pre = torch.empty((2, M, N), device=DEV)
    want = (gated_linear(x, wg, wu, bg, bu, pre=pre),) + tuple(gated_linear_backward(dy, x, wg, wu, pre))

    def exact(name):
        n = binding._bytes(name, M, N, K, code)
        whole = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=DEV)
        return whole[:n], whole[n:]

    ws, tail = exact("gated_linear")
    wb, tail_b = exact("gated_linear_backward")
    got = (gated_linear(x, wg, wu, bg, bu, workspace=ws),) + tuple(gated_linear_backward(dy, x, wg, wu, pre, workspace=wb))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (tail == 0xFF).all() and (tail_b == 0xFF).all()


def test_gradients_against_differences():
    """Central differences of the 64-bit form of sum(y c), step 1e-6."""
    M, N, K = 3, 5, 7
    x, wg, wu, bg, bu, c = inputs(M, N, K, torch.float32)
    for act in ("gelu", "silu"):
        pre = torch.empty((2, M, N), device=DEV)
        gated_linear(x, wg, wu, bg, bu, act=act, pre=pre)
        got = gated_linear_backward(c, x, wg, wu, pre, act=act)

        def f(a):
            xx, gg, uu, bb, vv = a
            return float((act64(act, xx @ gg.T + bb)[0] * (xx @ uu.T + vv) * c.double()).sum())

        args = [t.double() for t in (x, wg, wu, bg, bu)]
        for i, g in enumerate(got):
            for at in (0, args[i].numel() // 2, args[i].numel() - 1):
                sides = []
                for sign in (1, -1):
                    moved = [t.clone() for t in args]
                    moved[i].view(-1)[at] += sign * 1e-6
                    sides.append(f(moved))
                want = (sides[0] - sides[1]) / 2e-6
                assert abs(float(g.view(-1)[at]) - want) <= 1e-6 + 1e-5 * abs(want), (act, NAMES[i], at)


@pytest.mark.parametrize("M,N,K", [(1, 512, 256), (40, 100, 99), (300, 520, 1032)])
def test_captured_replayed_and_on_another_stream(M, N, K):
    made = inputs(M, N, K, torch.bfloat16)
    x, wg, wu, bg, bu, dy = made

    def call():
        pre = torch.empty((2, M, N), device=DEV)
        return (gated_linear(x, wg, wu, bg, bu, pre=pre),) + tuple(gated_linear_backward(dy, x, wg, wu, pre))

    seeds = iter(range(1000, 2000))
    replays(call, made, lambda: inputs(M, N, K, torch.bfloat16, seed=next(seeds)), lambda o: o)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(call(), want))


def test_refusals():
    x = torch.zeros((4, 64), device=DEV)
    w = torch.zeros((8, 64), device=DEV)
    pre = torch.zeros((2, 4, 8), device=DEV)
    dy = torch.zeros((4, 8), device=DEV)
    for bad in (dict(act="tanh"), dict(bg=torch.zeros(7, device=DEV)), dict(pre=pre[0]), dict(wu=w[:7]),
                dict(out=torch.empty((8, 4), device=DEV).t())):
        with pytest.raises(ValueError):
            gated_linear(**{**dict(x=x, wg=w, wu=w), **bad})
    with pytest.raises(TypeError):
        gated_linear(x, w, w.bfloat16())
    with pytest.raises(ValueError):
        gated_linear_backward(dy, x, w, w, pre, need=("dw",))
    with pytest.raises(ValueError):
        gated_linear_backward(dy, x, w, w, pre[:1])
    wide = torch.zeros((8, 65537), device=DEV)
    with pytest.raises(binding.DSparkError):
        gated_linear(wide[:4], wide, wide)
    with pytest.raises(binding.DSparkError):
        gated_linear(x, w, w, out=pre[0], pre=pre)
    with pytest.raises(RuntimeError, match="autograd"):
        gated_linear(x, w.clone().requires_grad_(), w)
