"""The linear layer, the heads' loss and their gradients against plain 64-bit
forms on the same inputs.

Tolerances are worst-case bounds, element by element.  With h the half step of
the storage type (bf16 2^-8, fp32 2^-24) and u = 2^-24:
  * a sum of K products in fp32, in any order, is off by at most (K + 2) u
    sum |terms|; products of bf16 values are exact in fp32.  The matrix unit may
    truncate where IEEE rounds, which doubles u: E = 2 (K + 8) u sum |terms|.
  * act' and act'' of relu away from 0, gelu and silu are below 1.2, so an
    error e in z moves act(z), and act'(z), by at most 1.2 e (relu's slope
    at 0 is kept out by the inputs); act itself is computed within
    16 u (|z| + 1).
  * a result rounded to the type once is off by h times itself more, and dz,
    rounded to the type before its products, by h |dz| in every term.
  * exp in fp32 is off by (|x| + 4) 2^-23 relatively.
"""
import ctypes
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import binding  # noqa: E402
from semi_ar_drafter_amd import (hidden_draft, linear, linear_backward, markov_draft, markov_loss,  # noqa: E402
                                 markov_loss_backward)

DEV = "cuda:0"
U32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ACTS = ["none", "relu", "gelu", "silu"]
TYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


def say(*a):
    print(*a, flush=True)


def rand(gen, *shape, sd=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device=DEV) * sd).to(dtype)


def within(got, want, tol, what):
    assert got.shape == want.shape, what
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got "
                             f"{float(got.flatten()[i])}, want {float(want.flatten()[i])} within "
                             f"{float(tol.flatten()[i])}")


# ---------------------------------------------------------------------------
# linear layer
# ---------------------------------------------------------------------------
SHAPES = [(1, 1, 1), (1, 17, 8), (2, 3, 5), (1, 130, 64), (3, 64, 200), (8, 1024, 64), (16, 300, 129), (17, 33, 65),
          (31, 128, 72), (64, 256, 128), (77, 131, 1001), (129, 257, 192), (255, 520, 333), (300, 512, 256),
          (1, 4096, 520), (8, 2000, 2056), (513, 96, 40), (257, 1027, 136)]


def act64(act, z):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(act, z):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def linear_inputs(M, N, K, dtype, act, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(1000 * seed + 7 * M + 3 * N + K)
    x, w = rand(gen, M, K, dtype=dtype), rand(gen, N, K, sd=(2.0 / max(K, 1)) ** 0.5, dtype=dtype)
    bias, res, dy = rand(gen, N, dtype=dtype), rand(gen, M, N, dtype=dtype), rand(gen, M, N, dtype=dtype)
    return x, w, bias, res, dy


def pre64(x, w, bias):
    z = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    return z, 2 * (x.shape[1] + 8) * U32 * size


def check_linear(x, w, bias, act, res, y, pre=None):
    h = HALF[x.dtype]
    z, e = pre64(x, w, bias)
    want = act64(act, z)
    tol = (1.2 if act != "none" else 1.0) * e + (16 * U32 * (z.abs() + 1) if act != "none" else 0)
    if res is not None:
        want = want + res.double()
        tol = tol + U32 * want.abs()
    within(y, want, tol + h * (want.abs() + tol) + 1e-38, "y")
    if pre is not None:
        within(pre, z, e + U32 * z.abs() + 1e-38, "pre")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dtype):
    for i, act in enumerate(ACTS):
        x, w, bias, res, _ = linear_inputs(M, N, K, dtype, act)
        b, r = (bias if i != 1 else None), (res if i % 2 else None)
        pre = torch.full((M, N), math.nan, device=DEV) if i >= 2 else None
        y = linear(x, w, bias=b, act=act, residual=r, pre=pre)
        torch.cuda.synchronize()
        check_linear(x, w, b, act, r, y, pre)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_backward(M, N, K, dtype):
    h = HALF[dtype]
    for act in ACTS:
        x, w, bias, _, dy = linear_inputs(M, N, K, dtype, act)
        z, e = pre64(x, w, bias)
        # the pre-activation is an input of the backward call: give it the 64-bit one, rounded to fp32,
        # and keep relu's step out of the way
        pre = None
        if act != "none":
            pre = z.float()
            if act == "relu":
                pre = torch.where(pre.abs() < 1e-3, torch.full_like(pre, 1e-3), pre)
            z = pre.double()
        dx, dw, db = linear_backward(dy, x, w, act=act, pre=pre)
        torch.cuda.synchronize()
        dz = dy.double() * slope64(act, z)
        # dz in fp32 (the slope within 16 u (|z| + 1)), then rounded to the type
        ez = (16 * U32 * (z.abs() + 1) * dy.double().abs() if act != "none" else 0) + 2 * U32 * dz.abs()
        er = ez + (h * (dz.abs() + ez) if act != "none" else 0)
        for got, want, size, err, n, what in (
                (dx, dz @ w.double(), dz.abs() @ w.double().abs(), er @ w.double().abs(), N, "dx"),
                (dw, dz.t() @ x.double(), dz.abs().t() @ x.double().abs(), er.t() @ x.double().abs(), M, "dw"),
                (db, dz.sum(0), dz.abs().sum(0), ez.sum(0), M, "dbias")):
            tol = err + 2 * (n + 8) * U32 * size
            within(got, want, tol + h * (want.abs() + tol) + 1e-38, f"{what} {act}")


def test_linear_empty():
    for dtype in TYPES:
        x, w, bias, res, dy = linear_inputs(5, 6, 0, dtype, "silu")
        y = linear(x, w, bias=bias, act="silu", residual=res)     # no inputs: z = bias
        check_linear(x, w, bias, "silu", res, y)
        e = torch.empty(0, 8, dtype=dtype, device=DEV)
        assert linear(e, torch.ones(4, 8, dtype=dtype, device=DEV)).shape == (0, 4)
        dx, dw, db = linear_backward(torch.empty(0, 4, dtype=dtype, device=DEV), e,
                                     torch.ones(4, 8, dtype=dtype, device=DEV))
        assert dx.shape == (0, 8) and not dw.any() and not db.any()
        dx, dw, db = linear_backward(torch.empty(3, 0, dtype=dtype, device=DEV),
                                     torch.ones(3, 8, dtype=dtype, device=DEV),
                                     torch.empty(0, 8, dtype=dtype, device=DEV))
        assert not dx.any() and dw.shape == (0, 8) and db.shape == (0,)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_linear_in_place_and_unaligned(dtype):
    """The residual added in place, and bias, residual and y that are aligned
    to their element only."""
    M, N, K = 37, 260, 136
    x, w, bias, res, _ = linear_inputs(M, N, K, dtype, "none")
    y = res.clone()
    assert linear(x, w, bias=bias, residual=y, out=y) is y
    check_linear(x, w, bias, "none", res, y)
    room = torch.empty(M * N + 1, dtype=dtype, device=DEV)[1:].view(M, N)
    off = torch.empty(N + 1, dtype=dtype, device=DEV)[1:]
    off.copy_(bias)
    r2 = torch.empty(M * N + 3, dtype=dtype, device=DEV)[3:].view(M, N)
    r2.copy_(res)
    pre = torch.empty(M * N + 1, device=DEV)[1:].view(M, N)
    linear(x, w, bias=off, act="gelu", residual=r2, out=room, pre=pre)
    check_linear(x, w, bias, "gelu", res, room, pre)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_linear_leaves_what_lies_behind(dtype):
    """Rows behind the last one of a larger buffer keep what they held."""
    for M, N, K in ((5, 100, 64), (130, 100, 64), (300, 300, 192)):
        x, w, bias, _, _ = linear_inputs(M, N, K, dtype, "none")
        room = torch.full((M + 300, N), 7.0, dtype=dtype, device=DEV)
        linear(x, w, bias=bias, out=room[:M])
        check_linear(x, w, bias, "none", None, room[:M])
        assert (room[M:] == 7.0).all()


def test_linear_infinities_stay_in_their_row():
    x, w, bias, _, _ = linear_inputs(40, 300, 200, torch.bfloat16, "none")
    clean = linear(x, w, bias=bias)
    x2 = x.clone()
    x2[7] = math.nan
    x2[9, 3] = math.inf
    y = linear(x2, w, bias=bias)
    keep = [i for i in range(40) if i not in (7, 9)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[9]).any()


def test_linear_gradients_against_differences():
    """fp32, a smooth loss sum(c y): for a change of size t along a direction
    the difference quotient is off by at most t^2 / 6 of the third derivative
    plus the rounding of two values of the loss over 2 t.  With |z| = O(1),
    third derivatives below 2, 24 outputs and t = 2^-7 the first is below
    24 * 2 * 6 * t^2 < 0.02 relative to changes of order 6 * 24; the loss is
    summed in 64 bits from fp32 outputs within 2^-19, 24 * 2^-19 / t < 0.006.
    0.05 holds both."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    for act in ("none", "gelu", "silu"):
        x, w, b = rand(gen, 4, 9, sd=0.3), rand(gen, 6, 9, sd=0.3), rand(gen, 6)
        c = rand(gen, 4, 6)
        pre = torch.empty(4, 6, device=DEV)
        linear(x, w, bias=b, act=act, pre=pre)
        grads = linear_backward(c, x, w, act=act, pre=pre if act != "none" else None)
        for i, g in enumerate(grads):
            v = rand(gen, *g.shape)
            v /= v.norm()
            t = 2.0 ** -7
            args = [x, w, b]
            vals = []
            for s in (t, -t):
                args2 = list(args)
                args2[i] = args[i] + s * v
                vals.append(float((linear(args2[0], args2[1], bias=args2[2], act=act).double() * c.double()).sum()))
            assert abs((vals[0] - vals[1]) / (2 * t) - float((g.double() * v.double()).sum())) < 0.05


# ---------------------------------------------------------------------------
# the heads' loss
# ---------------------------------------------------------------------------
LOSS = [  # N, V, d, r, base, ignored
    (1, 1, 1, 1, False, 0), (1, 7, 3, 2, True, 0), (2, 1024, 64, 16, False, 1), (5, 129, 0, 8, True, 2),
    (5, 130, 8, 0, False, 0), (3, 50, 0, 0, True, 1), (9, 1000, 40, 24, False, 3), (16, 515, 72, 9, True, 4),
    (33, 4096, 128, 32, False, 8), (77, 3001, 200, 40, True, 9), (130, 517, 72, 64, False, 0),
    (256, 2048, 256, 256, True, 60), (300, 5003, 104, 7, False, 77), (600, 1030, 333, 100, False, 599),
    (64, 900, 64, 64, True, 64), (520, 8200, 512, 128, False, 100)]


def loss_inputs(N, V, d, r, base, ignored, dtype, seed=0, tokens=None):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + N + 11 * V + 5 * d + r)
    s = {}
    if base:
        s["U"] = rand(gen, N, V, sd=2 ** 0.5, dtype=dtype)
    if d:
        s["h"], s["Wo"] = rand(gen, N, d, dtype=dtype), rand(gen, V, d, sd=(2.0 / d) ** 0.5, dtype=dtype)
    if r:
        s["prev"] = torch.randint(0, tokens or V, (N,), generator=gen, device=DEV, dtype=torch.int32)
        s["W1"], s["W2"] = rand(gen, V, r, sd=r ** -0.25, dtype=dtype), rand(gen, r, V, sd=r ** -0.25, dtype=dtype)
    label = torch.randint(0, V, (N,), generator=gen, device=DEV, dtype=torch.int32)
    drop = torch.randperm(N, generator=gen, device=DEV)[:ignored]
    label[drop] = torch.tensor([-1, V, -100, 2 ** 31 - 1], device=DEV, dtype=torch.int32)[
        torch.arange(ignored, device=DEV) % 4]
    g = torch.rand(N, generator=gen, device=DEV) / N
    return s, label, g


class Loss64:
    """The definitions in 64 bits, with the bounds of the errors that the
    operator's own arithmetic may add."""

    def __init__(self, s, label, g, dtype):
        self.h = HALF[dtype]
        V = next(t.shape[1] for t in (s.get("U"), s.get("W2"), s["Wo"].t() if "Wo" in s else None) if t is not None)
        d, r = (s["Wo"].shape[1] if "Wo" in s else 0), (s["W2"].shape[0] if "W2" in s else 0)
        used = (label >= 0) & (label < V)
        self.used, self.n = used, int(used.sum())
        z = torch.zeros(self.n, V, dtype=torch.float64, device=DEV)
        size = torch.zeros_like(z)
        self.E = self.X = None
        if "U" in s:
            u = s["U"][used].double()
            z, size = z + u, size + u.abs()
        if d:
            self.X, self.Wo = s["h"][used].double(), s["Wo"].double()
            z, size = z + self.X @ self.Wo.t(), size + self.X.abs() @ self.Wo.abs().t()
        if r:
            self.prev = s["prev"][used].long().clamp(0, V - 1)
            self.E, self.W2 = s["W1"].double()[self.prev], s["W2"].double()
            z, size = z + self.E @ self.W2, size + self.E.abs() @ self.W2.abs()
        self.V, self.d, self.r = V, d, r
        self.ez = torch.where(torch.isfinite(z), 2 * (d + r + 10) * U32 * size, 0.0)
        self.z, self.lse = z, torch.logsumexp(z, 1)
        self.y = label[used].long()
        at = self.y[:, None]
        self.nll = self.lse - z.gather(1, at)[:, 0]
        top = self.ez.amax(1)
        # the sum of exponentials: 1 part in 2^-23 (|x| + 4) each, weighted by the probabilities, and the
        # joining of at most V terms' partial sums in fp32 (in-lane, in-tile, over tiles: below 600 steps)
        p = torch.softmax(z, 1)
        x = torch.where(p > 0, (self.lse[:, None] - z).clamp(max=200), 0.0)
        self.elog = (p * ((x + 12) * 2 ** -23)).sum(1) + 600 * U32 + 2 * U32 * self.lse.abs() + 2 ** -22
        self.elog = self.elog + (p * self.ez).sum(1) * 1.01
        self.enll = self.elog + self.ez.gather(1, at)[:, 0] + U32 * (self.lse.abs() + self.nll.abs())
        self.top = top
        gu = g[used].double()[:, None]
        one = torch.zeros_like(p).scatter_(1, at, 1.0)
        self.dz = gu * (p - one)
        # exp(z - lse) with both off, and exp's own error; then the rounding to the type
        rel = self.ez + self.elog[:, None] + (x + 6) * 2 ** -23 + U32 * self.lse.abs()[:, None]
        e = gu.abs() * (p * rel * 1.01) + 4 * U32 * gu.abs() * one + 2 * U32 * self.dz.abs()
        self.er = e + self.h * (self.dz.abs() + e)

    def full(self, rows, n):
        out = torch.zeros((n,) + rows.shape[1:], dtype=torch.float64, device=DEV)
        out[self.used] = rows
        return out

    def grads(self, N):
        """{name: (value, tolerance)}"""
        out = {}

        def add(name, want, size, err, k):
            tol = err + 2 * (k + 8) * U32 * size
            out[name] = (want, tol + self.h * (want.abs() + tol) + 1e-38)

        dz, er = self.dz, self.er
        out["dU"] = (self.full(dz, N), self.full(er, N) + 1e-38)
        if self.d:
            add("dh", self.full(dz @ self.Wo, N), self.full(dz.abs() @ self.Wo.abs(), N),
                self.full(er @ self.Wo.abs(), N), self.V)
            add("dWo", dz.t() @ self.X, dz.abs().t() @ self.X.abs(), er.t() @ self.X.abs(), N)
        if self.r:
            add("dW2", self.E.t() @ dz, self.E.abs().t() @ dz.abs(), self.E.abs().t() @ er, N)
            put = lambda t: torch.zeros(self.V, self.r, dtype=torch.float64, device=DEV).index_add_(0, self.prev, t)  # noqa: E731
            add("dW1", put(dz @ self.W2.t()), put(dz.abs() @ self.W2.abs().t()), put(er @ self.W2.abs().t()),
                self.V + N)
        return out


def check_loss(s, label, g, dtype, need=None):
    N = label.numel()
    ref = Loss64(s, label, g, dtype)
    nll, lse = markov_loss(label, **s)
    grads = markov_loss_backward(g, lse, label, need=need, **s)
    torch.cuda.synchronize()
    assert not nll[~ref.used].any() and not lse[~ref.used].any()
    within(lse, ref.full(ref.lse, N), ref.full(ref.elog, N), "lse")
    within(nll, ref.full(ref.nll, N), ref.full(ref.enll, N), "nll")
    want = ref.grads(N)
    for k, got in grads.items():
        within(got, *want[k], k)
    return nll, lse, grads


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("N,V,d,r,base,ignored", LOSS)
def test_loss(N, V, d, r, base, ignored, dtype):
    s, label, g = loss_inputs(N, V, d, r, base, ignored, dtype)
    _, _, grads = check_loss(s, label, g, dtype)
    assert len(grads) == base + 2 * (d > 0) + 2 * (r > 0)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_loss_of_a_large_vocabulary_in_several_pieces(dtype):
    N, V = (4100, 70003) if dtype is torch.bfloat16 else (2100, 70003)
    say(f"[case] loss in pieces {N} {V}")
    s, label, g = loss_inputs(N, V, 64, 16, False, 100, dtype)
    check_loss(s, label, g, dtype)


@pytest.mark.parametrize("need", [["dW1"], ["dW2"], ["dh"], ["dWo"], ["dU"], [], ["dh", "dW2"]])
def test_loss_gradients_on_their_own(need):
    """Each gradient does not depend on which others are asked for."""
    s, label, g = loss_inputs(70, 1500, 136, 40, True, 10, torch.bfloat16)
    _, lse, every = check_loss(s, label, g, torch.bfloat16)
    some = markov_loss_backward(g, lse, label, need=need, **s)
    assert sorted(some) == sorted(need)
    for k in need:
        assert torch.equal(some[k], every[k])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_loss_same_previous_token(dtype):
    """Rows that share their previous token, and tokens outside the vocabulary
    (clamped): their gradients add up."""
    s, label, g = loss_inputs(150, 600, 32, 24, False, 20, dtype, tokens=3)
    s["prev"][5], s["prev"][6], s["prev"][7] = -4, 600, 2 ** 31 - 1
    check_loss(s, label, g, dtype)
    s["prev"].fill_(599)
    _, _, grads = check_loss(s, label, g, dtype)
    assert not grads["dW1"][:599].any()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_loss_ignored_rows_may_hold_anything(dtype):
    s, label, g = loss_inputs(140, 1100, 72, 16, True, 50, dtype)
    nll, lse, grads = check_loss(s, label, g, dtype)
    drop = (label < 0) | (label >= 1100)
    s["h"][drop] = math.nan
    s["U"][drop] = math.inf
    s["prev"][drop] = -2 ** 31
    g = g.clone()
    g[drop] = math.nan
    lse2 = lse.clone()
    lse2[drop] = math.nan
    n2, l2 = markov_loss(label, **s)
    g2 = markov_loss_backward(g, lse2, label, **s)
    assert torch.equal(n2, nll) and torch.equal(l2, lse)
    for k in grads:
        assert torch.equal(g2[k], grads[k]), k


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_loss_masked_tokens(dtype):
    """Base logits of -inf and of the type's lowest value: no probability, no
    gradient, also where a whole tile of the vocabulary is masked."""
    s, label, g = loss_inputs(40, 2000, 16, 8, True, 5, dtype)
    label.clamp_(max=99)
    s["U"][:, 100:1900] = -math.inf
    s["U"][::2, 1900:] = torch.finfo(dtype).min
    _, _, grads = check_loss(s, label, g, dtype, need=["dU", "dh", "dWo", "dW1", "dW2"])
    assert not grads["dU"][:, 100:1900].any() and not grads["dU"][::2, 1900:].any()
    assert not grads["dWo"][100:1900].any()


def test_loss_weights_of_zero_and_large_logits():
    s, label, g = loss_inputs(50, 700, 48, 8, False, 0, torch.bfloat16)
    s["h"] *= 30                      # logits of some hundreds: one token takes everything
    g[10:20] = 0
    _, _, grads = check_loss(s, label, g, torch.bfloat16)
    assert not grads["dh"][10:20].any()


def test_loss_no_rows():
    s, label, g = loss_inputs(0, 300, 16, 8, True, 0, torch.bfloat16)
    nll, lse = markov_loss(label, **s)
    assert nll.shape == lse.shape == (0,)
    grads = markov_loss_backward(g, lse, label, **s)
    for k in ("dWo", "dW1", "dW2"):
        assert not grads[k].any(), k
    assert grads["dU"].shape == (0, 300) and grads["dh"].shape == (0, 16)


def test_loss_gradients_against_differences():
    """fp32: (L(t) - L(-t)) / 2t against the gradient, L = sum g nll with sum g
    about 1/2.  nll is within 2^-18 here, so L's rounding adds at most
    2^-18 / 2t; the third derivative of a softmax's log-sum along a direction
    of unit length moves z by at most |row| < 4, so by less than 4^3 t^2 / 6.
    With t = 2^-6: 2^-13 + 0.0027 < 0.004."""
    s, label, g = loss_inputs(12, 90, 6, 4, True, 3, torch.float32)
    for k in ("h", "Wo", "W1", "W2"):
        s[k] *= 0.5
    _, lse = markov_loss(label, **s)
    grads = markov_loss_backward(g, lse, label, **s)
    gen = torch.Generator(device=DEV).manual_seed(17)
    t = 2.0 ** -6
    for k, grad in grads.items():
        v = rand(gen, *grad.shape)
        v /= v.norm()
        vals = []
        for sign in (t, -t):
            moved = dict(s)
            moved[k[1:]] = s[k[1:]] + sign * v
            vals.append(float((markov_loss(label, **moved)[0].double() * g.double()).sum()))
        assert abs((vals[0] - vals[1]) / (2 * t) - float((grad.double() * v.double()).sum())) < 0.004, k


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_workspace_of_the_stated_size_is_enough(dtype):
    """A workspace of exactly the stated size, in the middle of a larger
    buffer that keeps what it holds around it."""
    lib = binding.load()
    storage = 1 if dtype is torch.bfloat16 else 0

    def inside(nbytes):
        room = torch.full((nbytes + 1024,), 91, dtype=torch.uint8, device=DEV)
        off = 512 + (-(room.data_ptr() + 512)) % 256
        return room, room[off:off + nbytes], off

    def untouched(room, off, nbytes):
        return bool((room[:off] == 91).all()) and bool((room[off + nbytes:] == 91).all())

    for M, N, K in ((1, 40, 24), (5, 4100, 129), (70, 130, 1000), (300, 200, 4096), (333, 515, 333), (64, 64, 64)):
        x, w, bias, res, dy = linear_inputs(M, N, K, dtype, "gelu")
        pre = torch.empty(M, N, device=DEV)
        n = lib.dspark_linear_workspace_bytes(M, N, K, storage)
        room, ws, off = inside(n)
        y = linear(x, w, bias=bias, act="gelu", residual=res, pre=pre, workspace=ws if n else None)
        check_linear(x, w, bias, "gelu", res, y, pre)
        assert untouched(room, off, n)
        n = lib.dspark_linear_backward_workspace_bytes(M, N, K, storage)
        room, ws, off = inside(n)
        got = linear_backward(dy, x, w, act="gelu", pre=pre, workspace=ws)
        assert untouched(room, off, n)
        assert all(torch.equal(a, b) for a, b in zip(got, linear_backward(dy, x, w, act="gelu", pre=pre)))
    for N, V, d, r in ((1, 9, 5, 3), (20, 1001, 600, 17), (70, 3000, 129, 64), (300, 700, 64, 33)):
        s, label, g = loss_inputs(N, V, d, r, True, N // 5, dtype)
        nll, lse, grads = check_loss(s, label, g, dtype)
        n = lib.dspark_markov_loss_workspace_bytes(N, V, d, r, storage)
        room, ws, off = inside(n)
        again = markov_loss(label, workspace=ws, **s)
        assert torch.equal(again[0], nll) and torch.equal(again[1], lse) and untouched(room, off, n)
        n = lib.dspark_markov_loss_backward_workspace_bytes(N, V, d, r, storage)
        room, ws, off = inside(n)
        more = markov_loss_backward(g, lse, label, workspace=ws, **s)
        assert untouched(room, off, n) and all(torch.equal(more[k], grads[k]) for k in grads)


@pytest.mark.parametrize("M,N,K", [(4000, 4090, 1096), (1000, 4090, 4080)])
def test_linear_large_tiles(M, N, K):
    """Sizes that fill the compute units with the largest tile, ragged along
    every axis (the contraction too), in all three products."""
    x, w, bias, res, dy = linear_inputs(M, N, K, torch.bfloat16, "silu")
    y = linear(x, w, bias=bias, act="silu", residual=res)
    check_linear(x, w, bias, "silu", res, y)
    dx, dw, _ = linear_backward(dy, x, w)
    h = HALF[torch.bfloat16]
    for got, a, b, n, what in ((dx, dy.double(), w.double(), N, "dx"), (dw, dy.double().t(), x.double(), M, "dw")):
        want, tol = a @ b, 2 * (n + 8) * U32 * (a.abs() @ b.abs())
        within(got, want, tol + h * (want.abs() + tol) + 1e-38, what)


def test_loss_large_tiles():
    for base, d in ((False, 456), (True, 0)):
        s, label, g = loss_inputs(2040, 8190, d, 72, base, 100, torch.bfloat16)
        check_loss(s, label, g, torch.bfloat16)


def test_loss_of_many_rows():
    """More rows than one workgroup counts for itself, most of them ignored."""
    N = 9000
    s, label, g = loss_inputs(N, 300, 24, 16, False, 7000, torch.bfloat16, tokens=40)
    check_loss(s, label, g, torch.bfloat16)


def test_same_inputs_same_bits():
    s, label, g = loss_inputs(300, 5003, 104, 56, False, 20, torch.bfloat16)
    first = markov_loss(label, **s)
    grads = markov_loss_backward(g, first[1], label, **s)
    x, w, bias, res, dy = linear_inputs(70, 600, 500, torch.bfloat16, "none")
    y, back = linear(x, w, bias=bias), linear_backward(dy, x, w)
    for _ in range(3):
        again = markov_loss(label, **s)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
        g2 = markov_loss_backward(g, first[1], label, **s)
        assert all(torch.equal(g2[k], grads[k]) for k in grads)
        assert torch.equal(linear(x, w, bias=bias), y)
        assert all(torch.equal(a, b) for a, b in zip(linear_backward(dy, x, w), back))


# ---------------------------------------------------------------------------
# as they are used: streams, graphs, together with the drafting
# ---------------------------------------------------------------------------
def test_two_streams_at_once():
    a = loss_inputs(200, 3001, 96, 32, False, 10, torch.bfloat16, seed=1)
    b = loss_inputs(180, 2500, 128, 16, False, 30, torch.bfloat16, seed=2)
    want = [check_loss(*c, torch.bfloat16) for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (s, label, g), st in zip((a, b), streams):
            with torch.cuda.stream(st):
                nll, lse = markov_loss(label, **s)
                got.append((nll, lse, markov_loss_backward(g, lse, label, **s)))
        torch.cuda.synchronize()
        for (n1, l1, g1), (n2, l2, g2) in zip(want, got):
            assert torch.equal(n1, n2) and torch.equal(l1, l2) and all(torch.equal(g1[k], g2[k]) for k in g1)


def test_threads_on_one_stream():
    """Calls of several launches from threads that share a stream, and so its
    workspace, are not enqueued into each other."""
    import threading
    sets = [loss_inputs(60 + 40 * i, 1500 + 300 * i, 64, 24, False, 5, torch.bfloat16, seed=i) for i in range(4)]
    want = [check_loss(*c, torch.bfloat16) for c in sets]
    wrong = []

    def work(i):
        s, label, g = sets[i]
        for _ in range(20):
            nll, lse = markov_loss(label, **s)
            grads = markov_loss_backward(g, lse, label, **s)
            torch.cuda.synchronize()
            if not (torch.equal(nll, want[i][0]) and all(torch.equal(grads[k], want[i][2][k]) for k in grads)):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_captured_and_replayed():
    """Two graphs, captured one after the other, replayed with new inputs in
    place, with eager calls between the replays."""
    sets = [loss_inputs(90, 1203, 64, 24, False, 9, torch.bfloat16, seed=i) for i in range(4)]
    lin = [linear_inputs(40, 333, 136, torch.bfloat16, "gelu", seed=i) for i in range(4)]

    def work(s, label, g, x, w, bias, res, dy):
        nll, lse = markov_loss(label, **s)
        grads = markov_loss_backward(g, lse, label, **s)
        pre = torch.empty(40, 333, device=DEV)
        y = linear(x, w, bias=bias, act="gelu", residual=res, pre=pre)
        return [nll, lse, *grads.values(), y, *linear_backward(dy, x, w, act="gelu", pre=pre)]

    want = [work(*a, *b) for a, b in zip(sets, lin)]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        held = [{k: t.clone() for k, t in sets[0][0].items()}, sets[0][1].clone(), sets[0][2].clone()]
        lheld = [t.clone() for t in lin[0]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = work(*held, *lheld)
        graphs.append((graph, held, lheld, outs))
    for i in (1, 2, 3, 0, 2):
        for j, (graph, held, lheld, outs) in enumerate(graphs):
            n = (i + j) % 4
            for k, t in sets[n][0].items():
                held[0][k].copy_(t)
            held[1].copy_(sets[n][1])
            held[2].copy_(sets[n][2])
            for dst, src in zip(lheld, lin[n]):
                dst.copy_(src)
            graph.replay()
        eager = work(*sets[i], *lin[i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, want[i]))
        for j, (_, _, _, outs) in enumerate(graphs):
            for a, b in zip(outs, want[(i + j) % 4]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,r", [(torch.bfloat16, 32), (torch.float32, 16)], ids=IDS)
@pytest.mark.parametrize("B,gamma", [(1, 8), (3, 4), (40, 3)])
def test_draft_from_hidden_states_and_train_on_it(dtype, r, B, gamma):
    """hidden_draft is linear then markov_draft; the loss's logits are the
    drafting's: at the drafted tokens lse - nll is the drafted logit.  fp32
    logits differ by the rounding of U to its type (half a step of |U| < 16)
    and the sums' error."""
    V, d = 3000, 64
    gen = torch.Generator(device=DEV).manual_seed(B + gamma)
    h, Wo = rand(gen, B, gamma, d, dtype=dtype), rand(gen, V, d, sd=(2 / d) ** 0.5, dtype=dtype)
    W1, W2 = rand(gen, V, r, sd=r ** -0.25, dtype=dtype), rand(gen, r, V, sd=r ** -0.25, dtype=dtype)
    conf_w, sts_T = rand(gen, d + r, sd=0.05), torch.ones(gamma, device=DEV)
    anchor = torch.randint(0, V, (B,), generator=gen, device=DEV, dtype=torch.int32)
    U = torch.empty(B, gamma, V, dtype=dtype, device=DEV)
    got = hidden_draft(anchor, h, Wo, W1, W2, conf_w, 1.0, sts_T, U=U)
    U2 = linear(h.view(-1, d), Wo).view(B, gamma, V)
    want = markov_draft(anchor, U2, h, W1, W2, conf_w, 1.0, sts_T)
    torch.cuda.synchronize()
    assert torch.equal(U, U2) and all(torch.equal(a, b) for a, b in zip(got, want))
    tokens, logit = got[0], got[1]
    assert (tokens >= 0).all()
    prev = torch.cat([anchor[:, None], tokens[:, :-1]], 1).reshape(-1).contiguous()
    nll, lse = markov_loss(tokens.reshape(-1), h=h.view(-1, d), Wo=Wo, prev=prev, W1=W1, W2=W2)
    tol = 16 * HALF[dtype] + 2e-4
    assert float(((lse - nll) - logit.view(-1)).abs().max()) < tol
    # a bias that makes one token win everywhere reaches the drafting
    bias = torch.zeros(V, dtype=dtype, device=DEV)
    bias[1234] = 100
    assert (hidden_draft(anchor, h, Wo, W1, W2, conf_w, 1.0, sts_T, bias=bias)[0] == 1234).all()


def test_training_step_of_both_heads():
    """A step of training as a user writes it: gradients of the mean loss by
    the projection, its input layer and the Markov factors, end to end against
    autograd in 64 bits."""
    dtype, N, V, d, r = torch.float32, 48, 700, 40, 16
    s, label, g = loss_inputs(N, V, d, r, False, 6, dtype)
    gen = torch.Generator(device=DEV).manual_seed(5)
    x, w, b = rand(gen, N, 24), rand(gen, d, 24, sd=0.3), rand(gen, d, sd=0.1)
    pre = torch.empty(N, d, device=DEV)
    s["h"] = linear(x, w, bias=b, act="gelu", pre=pre)
    nll, lse = markov_loss(label, **s)
    grads = markov_loss_backward(g, lse, label, **s)
    dx, dw, db = linear_backward(grads["dh"], x, w, act="gelu", pre=pre)
    p = {k: t.double().requires_grad_() for k, t in dict(x=x, w=w, b=b, Wo=s["Wo"], W1=s["W1"], W2=s["W2"]).items()}
    hid = torch.nn.functional.gelu(p["x"] @ p["w"].t() + p["b"])
    z = hid @ p["Wo"].t() + p["W1"][s["prev"].long()] @ p["W2"]
    used = (label >= 0) & (label < V)
    each = torch.nn.functional.cross_entropy(z[used], label[used].long(), reduction="none")
    (each * g[used].double()).sum().backward()
    # every sum here has under 800 fp32 terms of like size, chained four deep: 4 * 800 u < 2e-4 of the norm
    for k, got in dict(x=dx, w=dw, b=db, Wo=grads["dWo"], W1=grads["dW1"], W2=grads["dW2"]).items():
        want = p[k].grad
        assert float((got.double() - want).norm()) < 2e-4 * float(want.norm()), k


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_refusals():
    x, w, bias, res, dy = linear_inputs(8, 24, 16, torch.bfloat16, "none")
    with pytest.raises(TypeError):
        linear(x.half(), w.half())
    with pytest.raises(TypeError):
        linear(x, w.float())
    with pytest.raises(ValueError):
        linear(x, w[:, :8].contiguous())
    with pytest.raises(ValueError):
        linear(x.t().contiguous().t(), w)          # not contiguous
    with pytest.raises(ValueError):
        linear(x.cpu(), w)
    with pytest.raises(ValueError):
        linear(x, w, act="tanh")
    with pytest.raises(ValueError):
        linear(x, w, bias=bias[:5])
    with pytest.raises(TypeError):
        linear(x, w, pre=torch.empty(8, 24, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        linear_backward(dy, x, w, act="gelu")
    with pytest.raises(ValueError):
        linear_backward(dy, x, w, need=("dz",))
    off = torch.empty(24 * 16 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(24, 16)
    with pytest.raises(binding.DSparkError, match="16-byte"):
        linear(x, off)
    with pytest.raises(binding.DSparkError, match="workspace"):
        linear_backward(dy, x, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    s, label, g = loss_inputs(8, 90, 16, 8, True, 0, torch.bfloat16)
    with pytest.raises(ValueError):
        markov_loss(label)
    with pytest.raises(ValueError):
        markov_loss(label, h=s["h"])
    with pytest.raises(ValueError):
        markov_loss(label, prev=s["prev"], W1=s["W1"])
    with pytest.raises(TypeError):
        markov_loss(label.long(), **s)
    with pytest.raises(TypeError):
        markov_loss(label, **{**s, "U": s["U"].float()})
    with pytest.raises(ValueError):
        markov_loss(label[:4].contiguous(), **s)
    _, lse = markov_loss(label, **s)
    with pytest.raises(ValueError):
        markov_loss_backward(g, lse, label, U=s["U"], need=["dh"])
    with pytest.raises(TypeError):
        markov_loss_backward(g.double(), lse, label, **s)
    with pytest.raises(binding.DSparkError, match="workspace"):
        markov_loss(label, workspace=torch.empty(16, dtype=torch.uint8, device=DEV), **s)
    with pytest.raises(ValueError):
        markov_loss(label, workspace=torch.empty(1 << 20, dtype=torch.uint8), **s)      # host memory
