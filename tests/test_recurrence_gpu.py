"""recurrence() and recurrence_backward() against plain 64-bit forms on the
same inputs.

Tolerances are worst-case bounds, element by element.  With h the half step of
the storage type and u = 2^-24:
  * a and 1 - a of a logit g are off by a relative ea = (2 |g| + 14) u: the
    exponential's argument and result, one addition, a reciprocal and a product
    (a given decay: ea = 0).
  * H[t] = |a| H[t-1] + |b| bounds |h| and every partial result of any way to
    join the rows; each row adds at most (ea + 6 u) (|a| H[t-1] + |b|) to the
    error, which the gates behind it shrink as they do the state:
    E[t] = |a| E[t-1] + (ea + 6 u) (|a| H[t-1] + |b|), and 8 u H[t] for joining.
  * the same backwards for d, with G and F.
  * products of these add up; a sum over T rows of S sequences goes through at
    most T / 8 + S + 256 roundings.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import RECURRENCE_BLOCK, binding, recurrence, recurrence_backward  # noqa: E402

from layers import DEV, HALF, IDS, TYPES, U32, generator, guarded, rand, replays, say, within  # noqa: E402

KINDS = ["sigmoid", "decay"]
LENGTHS = [[1], [2], [31], [32], [33], [64], [0, 0], [0, 1, 0], [1] * 5, [16] * 9, [7, 0, 130, 1, 0, 65], [300],
           [1000, 3], [5, 2047], [4100], [517] * 3, [0, 3000, 0, 1100, 129, 0]]
CHANNELS = [1, 2, 3, 64, 127, 128, 129, 257]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


class Plain:
    """Row after row in 64 bits on the CPU, with the bounds beside."""

    def __init__(self, lengths, x, gate, kind, h0, dh=None, dlast=None):
        half, u = HALF[x.dtype], U32
        T, C = x.shape
        S = len(lengths)
        cpu = lambda t, shape: torch.zeros(shape, dtype=torch.float64) if t is None else t.double().cpu()  # noqa: E731
        x, h0 = cpu(x, (T, C)), cpu(h0, (S, C))
        g = gate.double().cpu()
        if kind == "sigmoid":
            a, rest, ea = torch.sigmoid(g), torch.sigmoid(-g), (2 * g.abs() + 14) * u
            b = rest * x
        else:
            a, rest, ea, b = g.expand(T, C), None, torch.zeros((T, C), dtype=torch.float64), x
        new = lambda n=T: torch.zeros((n, C), dtype=torch.float64)  # noqa: E731
        h, H, E, before, Hb, Eb = (new() for _ in range(6))
        self.last, self.last_tol = h0.clone(), torch.zeros_like(h0)
        at = 0
        for s, n in enumerate(lengths):
            v, V, e = h0[s], h0[s].abs(), torch.zeros(C, dtype=torch.float64)
            for t in range(at, at + n):
                before[t], Hb[t], Eb[t] = v, V, e
                v = a[t] * v + b[t]
                e = a[t].abs() * e + (ea[t] + 6 * u) * (a[t].abs() * V + b[t].abs())
                V = a[t].abs() * V + b[t].abs()
                h[t], H[t], E[t] = v, V, e
            self.last[s], self.last_tol[s] = v, e + 9 * u * V
            at += n
        self.rows = at
        self.h, self.h_tol = h, E + 8 * u * H + half * h.abs() + 1e-40
        if dh is None:
            return
        dh, dlast = cpu(dh, (T, C)), cpu(dlast, (S, C))
        d, G, F = new(), new(), new()
        self.dh0, self.dh0_tol = dlast.clone(), torch.zeros_like(dlast)
        at = 0
        for s, n in enumerate(lengths):
            v, V, e = dlast[s], dlast[s].abs(), torch.zeros(C, dtype=torch.float64)   # what reaches the row before
            for t in range(at + n - 1, at - 1, -1):
                d[t], G[t], F[t] = dh[t] + v, dh[t].abs() + V, e + 3 * u * (dh[t].abs() + V)
                v, V = a[t] * d[t], a[t].abs() * G[t]
                e = a[t].abs() * F[t] + (ea[t] + 6 * u) * V
            if n:
                self.dh0[s], self.dh0_tol[s] = v, e + 9 * u * V
            at += n
        F = F + 8 * u * G
        Eb = Eb + 8 * u * Hb
        if kind == "sigmoid":
            self.dx = d * rest
            self.dx_tol = rest * (F + (ea + 3 * u) * d.abs()) + half * self.dx.abs() + 1e-40
            diff = before - x
            self.dgate = d * a * rest * diff
            self.dgate_tol = (a * rest * (F * diff.abs() + d.abs() * (Eb + 2 * u * (before.abs() + x.abs()))) +
                              self.dgate.abs() * (2 * ea + 8 * u) + half * self.dgate.abs() + 1e-40)
        else:
            self.dx, self.dx_tol = d, F + half * d.abs() + 1e-40
            self.dgate = (d * before)[:at].sum(0)
            self.dgate_tol = ((F * Hb + G * Eb)[:at].sum(0) +
                              (at / 8 + S + 256) * u * (G * Hb)[:at].sum(0) + 1e-40)


def inputs(lengths, C, dtype, kind, seed=0, behind=0):
    T, S = sum(lengths) + behind, len(lengths)
    gen = generator(1000 * seed + 31 * T + 7 * S + C)
    x, dh = rand(gen, T, C, dtype=dtype), rand(gen, T, C, dtype=dtype)
    if kind == "sigmoid":
        gate = rand(gen, T, C, sd=2.5, mean=1.5, dtype=dtype)
    else:      # both signs; one that forgets nothing, one that remembers nothing
        gate = rand(gen, C, sd=0.5).clamp(-0.999, 0.999)
        gate[0] = 1.0 if T < 200 else 0.999
        gate[-1] = 0.0 if C > 1 else gate[-1]
    h0, dlast = rand(gen, S, C), rand(gen, S, C)
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    offsets = torch.tensor(at, dtype=torch.int32, device=DEV)
    return x, gate, h0, offsets, dh, dlast


def kept(T, C):
    return torch.full((-(-T // RECURRENCE_BLOCK), C), float("nan"), device=DEV)


def check(lengths, C, dtype, kind, h0=True, behind=0, regular=False):
    x, gate, first, offsets, dh, dlast = inputs(lengths, C, dtype, kind, behind=behind)
    if not h0:
        first = dlast = None
    T, S = x.shape[0], len(lengths)
    p = Plain(lengths, x, gate, kind, first, dh, dlast)
    where = dict(sequences=S) if regular else dict(offsets=offsets)
    out, out_ok = guarded((T, C), dtype, 1)
    last, last_ok = guarded((S, C), torch.float32, 1)
    states = kept(T, C)
    h = recurrence(x, gate, kind, h0=first, last=last, states=states, out=out, **where)
    assert h is out and out_ok() and last_ok()
    n = p.rows
    within(h[:n].cpu(), p.h[:n], p.h_tol[:n], "h")
    assert (h[n:] == 7).all()                       # rows of no sequence are left alone
    within(last.cpu(), p.last, p.last_tol, "last")
    dx, dg, d0 = recurrence_backward(dh, x, gate, states, kind, h0=first, dlast=dlast, **where)
    within(dx[:n].cpu(), p.dx[:n], p.dx_tol[:n], "dx")
    if kind == "sigmoid":
        within(dg[:n].cpu(), p.dgate[:n], p.dgate_tol[:n], "dgate")
    else:
        within(dg.cpu(), p.dgate, p.dgate_tol, "dgate")
    within(d0.cpu(), p.dh0, p.dh0_tol, "dh0")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("i", range(len(LENGTHS)))
def test_recurrence(i, kind, dtype):
    lengths = LENGTHS[i]
    for C in {CHANNELS[i % len(CHANNELS)], CHANNELS[(3 * i + 5) % len(CHANNELS)]}:
        say(f"[case] recurrence {lengths} C={C} {kind} {dtype}")
        check(lengths, C, dtype, kind, h0=i % 3 != 1, behind=(0, 5, 77)[i % 3])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S,L,C", [(1, 1, 5), (300, 1, 130), (33, 16, 256), (3, 700, 64), (1, 9000, 2), (2, 64, 2560)])
def test_sequences_of_equal_length(S, L, C, kind, dtype):
    say(f"[case] recurrence {S} x {L} C={C} {kind} {dtype}")
    check([L] * S, C, dtype, kind, regular=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths", [[1] * 7, [40, 0, 9], [2500, 0, 1700]])
def test_states_in_place(lengths, kind):
    x, gate, h0, offsets, dh, dlast = inputs(lengths, 130, torch.bfloat16, kind)
    last, states = torch.empty_like(h0), kept(x.shape[0], 130)
    h = recurrence(x, gate, kind, offsets=offsets, h0=h0, last=last, states=states)
    state = h0.clone()
    assert torch.equal(recurrence(x, gate, kind, offsets=offsets, h0=state, last=state), h)
    assert torch.equal(state, last)


@pytest.mark.parametrize("kind", KINDS)
def test_steps_of_a_decoder_are_the_sequence(kind):
    """One row at a time from the state before: the sequence's outputs, bit for
    bit, where one wave goes through them."""
    S, L, C = 5, 12, 200
    x, gate, h0, _, _, _ = inputs([L] * S, C, torch.bfloat16, kind)
    whole = recurrence(x, gate, kind, h0=h0).view(S, L, C)
    state = h0.clone()
    for t in range(L):
        row = lambda v: v.view(S, L, C)[:, t].contiguous()  # noqa: E731
        h = recurrence(row(x), row(gate) if kind == "sigmoid" else gate, kind, h0=state, last=state)
        assert torch.equal(h, whole[:, t]), t


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("lengths", [[40, 30, 50], [900, 1300, 800]])
def test_what_is_not_finite_stays_in_its_sequence_and_channel(lengths, dtype):
    x, gate, h0, offsets, dh, dlast = inputs(lengths, 64, dtype, "sigmoid")
    clean = recurrence(x, gate, offsets=offsets, h0=h0)
    a, b = lengths[0], lengths[0] + lengths[1]
    for value in (float("nan"), float("inf"), float("-inf")):
        bad, bad0 = x.clone(), h0.clone()
        bad[a + 20, 3] = value
        bad0[0, 5] = value
        states, last = kept(x.shape[0], 64), torch.empty_like(h0)
        h = recurrence(bad, gate, offsets=offsets, h0=bad0, states=states, last=last)
        hit = torch.zeros_like(h, dtype=torch.bool)
        hit[a + 20:b, 3] = True
        hit[:a, 5] = True
        assert torch.equal(h[~hit], clean[~hit])
        assert not h[a + 20, 3].isfinite() and not h[0, 5].isfinite()
        assert last[2].isfinite().all()
        bad_dh = dh.clone()
        bad_dh[a + 20, 7] = value
        dx, dg, d0 = recurrence_backward(bad_dh, bad, gate, states, offsets=offsets, h0=bad0, dlast=dlast)
        assert dx[:a].isfinite().all() and dx[b:].isfinite().all() and dx[a + 21:b].isfinite().all()
        assert d0[0].isfinite().all() and d0[2].isfinite().all() and not dx[a + 20, 7].isfinite()
        assert dg[b:].isfinite().all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gates_at_their_ends(dtype):
    """Logits so far out that a or 1 - a is 0, or rounds to 1."""
    C = 4
    gate = torch.tensor([100.0, -100.0, float("inf"), float("-inf")], device=DEV).expand(80, C).to(dtype).contiguous()
    x = rand(generator(1), 80, C, dtype=dtype)
    h0 = rand(generator(2), 1, C)
    h = recurrence(x, gate, h0=h0)
    assert torch.equal(h[:, 0], h0[0, 0].to(dtype).expand(80)) and torch.equal(h[:, 2], h0[0, 2].to(dtype).expand(80))
    assert torch.equal(h[:, 1], x[:, 1]) and torch.equal(h[:, 3], x[:, 3])


def test_offsets_out_of_range_are_cut():
    """Nothing outside the arrays is read or written, whatever the offsets hold."""
    x, gate, h0, _, dh, dlast = inputs([50] * 4, 66, torch.bfloat16, "sigmoid")
    out, ok = guarded((200, 66), torch.bfloat16, 3)
    for bad in ([-5, 60, 1 << 30, 50, 200], [200, 100, 0, -(1 << 31), (1 << 31) - 1], [300, 300, 300, 300, 300]):
        offsets = torch.tensor(bad, dtype=torch.int64, device=DEV).to(torch.int32)
        states, last = kept(200, 66), torch.empty_like(h0)
        recurrence(x, gate, offsets=offsets, h0=h0, out=out, states=states, last=last)
        recurrence_backward(dh, x, gate, states, offsets=offsets, h0=h0, dlast=dlast)
        torch.cuda.synchronize()
        assert ok()


def test_no_rows_and_no_sequences():
    x = torch.empty((0, 6), device=DEV)
    h0 = rand(generator(1), 3, 6)
    last = torch.empty_like(h0)
    recurrence(x, x, h0=h0, last=last, states=kept(0, 6))
    assert torch.equal(last, h0)
    for kind, gate in (("sigmoid", x), ("decay", torch.ones(6, device=DEV))):
        dx, dg, d0 = recurrence_backward(x, x, gate, kept(0, 6), kind, h0=h0, dlast=h0)
        assert torch.equal(d0, h0) and not dg.any()
    y = torch.ones((4, 6), device=DEV)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(y, 7.0)
    recurrence(y, y, offsets=none, out=out)
    assert (out == 7).all()
    dx, dg, d0 = recurrence_backward(y, y, torch.ones(6, device=DEV), kept(4, 6), "decay", offsets=none)
    assert not dg.any() and d0.shape == (0, 6)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths", [[9, 50], [4000]])
def test_each_gradient_on_its_own(lengths, kind):
    x, gate, h0, offsets, dh, dlast = inputs(lengths, 70, torch.bfloat16, kind)
    states = kept(x.shape[0], 70)
    recurrence(x, gate, kind, offsets=offsets, h0=h0, states=states)
    names = ("dx", "dgate", "dh0")
    full = dict(zip(names, recurrence_backward(dh, x, gate, states, kind, offsets=offsets, h0=h0, dlast=dlast)))
    for need in ((), ("dx",), ("dgate",), ("dh0",), ("dh0", "dx")):
        got = dict(zip(names, recurrence_backward(dh, x, gate, states, kind, offsets=offsets, h0=h0, dlast=dlast,
                                                  need=need)))
        for k, v in got.items():
            assert (v is None) == (k not in need)
            assert v is None or torch.equal(v, full[k]), k


@pytest.mark.parametrize("kind", KINDS)
def test_gradients_against_differences(kind):
    """Central differences of the 64-bit form of sum(h c) + sum(last e), step
    1e-6: their own error is below 1e-9 for values of order 100."""
    lengths, C = [3, 0, 40], 2
    x, gate, h0, offsets, c, e = inputs(lengths, C, torch.float32, kind, seed=3)
    states = kept(43, C)
    recurrence(x, gate, kind, offsets=offsets, h0=h0, states=states)
    dx, dg, d0 = recurrence_backward(c, x, gate, states, kind, offsets=offsets, h0=h0, dlast=e)

    def f(xx, gg, hh):
        a = torch.sigmoid(gg) if kind == "sigmoid" else gg.expand(43, C)
        b = (1 - a) * xx if kind == "sigmoid" else xx
        total, at = 0.0, 0
        for s, n in enumerate(lengths):
            v = hh[s]
            for t in range(at, at + n):
                v = a[t] * v + b[t]
                total += float((v * c[t].double().cpu()).sum())
            total += float((v * e[s].double().cpu()).sum())
            at += n
        return total

    args = [t.double().cpu() for t in (x, gate, h0)]
    for got, i in ((dx, 0), (dg, 1), (d0, 2)):
        for at in {0, 1, 2, args[i].numel() // 2, args[i].numel() - 1} & set(range(args[i].numel())):
            sides = []
            for sign in (1, -1):
                moved = [t.clone() for t in args]
                moved[i].view(-1)[at] += sign * 1e-6
                sides.append(f(*moved))
            want = (sides[0] - sides[1]) / 2e-6
            assert abs(float(got.view(-1)[at]) - want) <= 1e-6 + 1e-5 * abs(want), (i, at)


@pytest.mark.parametrize("lengths", [[1] * 40, [16] * 30, [3000, 0, 2000]])
@pytest.mark.parametrize("kind", KINDS)
def test_captured_replayed_and_on_another_stream(lengths, kind):
    C = 192
    made = list(inputs(lengths, C, torch.bfloat16, kind))
    x, gate, h0, offsets, dh, dlast = made
    T = x.shape[0]

    def call():
        states, last = torch.empty((-(-T // RECURRENCE_BLOCK), C), device=DEV), torch.empty_like(h0)
        h = recurrence(x, gate, kind, offsets=offsets, h0=h0, last=last, states=states)
        return (h, last) + recurrence_backward(dh, x, gate, states, kind, offsets=offsets, h0=h0, dlast=dlast)

    seeds = iter(range(1, 100))
    replays(call, made, lambda: inputs(lengths, C, torch.bfloat16, kind, seed=next(seeds)), lambda o: o)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    again = call()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_refusals():
    x = torch.zeros((8, 6), device=DEV)
    at = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    decay = torch.ones(6, device=DEV)
    for bad in (dict(kind="tanh"), dict(sequences=3), dict(sequences=0), dict(offsets=at, sequences=2),
                dict(h0=torch.zeros((3, 6), device=DEV)), dict(h0=torch.zeros((2, 5), device=DEV)),
                dict(states=torch.zeros((2, 6), device=DEV)), dict(last=torch.zeros((2, 6), device=DEV)),
                dict(offsets=at[:0]), dict(offsets=at.view(1, 2)), dict(kind="decay"),
                dict(out=torch.empty((6, 8), device=DEV).t())):
        with pytest.raises(ValueError):
            recurrence(x, x, **bad)
    with pytest.raises(TypeError):
        recurrence(x, x, offsets=at.long())
    with pytest.raises(TypeError):
        recurrence(x, decay.bfloat16(), kind="decay")
    with pytest.raises(binding.DSparkError):
        recurrence(x, x.clone(), out=x)
    states = torch.zeros((1, 6), device=DEV)
    with pytest.raises(ValueError):
        recurrence_backward(x, x, x, states, need=("dg",))
    with pytest.raises(ValueError):
        recurrence_backward(x, x, x, states[:0])
    with pytest.raises(RuntimeError, match="autograd"):
        recurrence(x, x.clone().requires_grad_())
