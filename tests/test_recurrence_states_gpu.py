"""recurrence() and its gradient: the states' gradient in the place of its
input, states that are not finite, gates of zero."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import binding, recurrence, recurrence_backward  # noqa: E402

import test_recurrence_gpu as forms  # noqa: E402
from layers import DEV, IDS, TYPES, say  # noqa: E402

KINDS = ["sigmoid", "decay"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


def backward(x, gate, kind, offsets, h0, dh, dlast, states, dh0):
    """dspark_recurrence_backward itself, whose dh0 may be dlast: (dx, dgate)."""
    lib, (T, C), S = binding.load(), x.shape, len(dlast)
    dt = binding.DSPARK_BF16 if x.dtype == torch.bfloat16 else binding.DSPARK_F32
    k = binding.GATES[kind]
    need = binding._bytes("recurrence_backward", T, S, C, dt, k)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    dx, dg = torch.zeros_like(x), torch.zeros_like(gate)
    binding._check(lib.dspark_recurrence_backward(
        T, S, C, dt, k, offsets.data_ptr(), dh.data_ptr(), x.data_ptr(), gate.data_ptr(), h0.data_ptr(), dlast.data_ptr(),
        states.data_ptr(), dx.data_ptr(), dg.data_ptr(), dh0.data_ptr(), ws.data_ptr() if need else None, need,
        torch.cuda.current_stream().cuda_stream))
    return dx, dg


# sequences of two rows over the border of two blocks of 16: the first is one
# wave's last row, the second another wave's (or another tile's) first
ACROSS = [15, 2] + [62, 2] * 60 + [45]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths,C", [(ACROSS, 130), (ACROSS, 2050), ([17] * 40, 384), ([3, 0, 2000, 1, 900], 257),
                                       ([5] * 300, 130), ([1] * 33, 3)])
def test_gradient_of_the_states_in_place(lengths, C, kind, dtype):
    say(f"[case] states in place {len(lengths)} sequences C={C} {kind} {dtype}")
    x, gate, h0, offsets, dh, dlast = forms.inputs(lengths, C, dtype, kind)
    states = forms.kept(x.shape[0], C)
    recurrence(x, gate, kind, offsets=offsets, h0=h0, states=states)
    want = recurrence_backward(dh, x, gate, states, kind, offsets=offsets, h0=h0, dlast=dlast)
    p = forms.Plain(lengths, x, gate, kind, h0, dh, dlast) if C < 2000 else None
    for turn in range(3):
        place = dlast.clone()
        dx, dg = backward(x, gate, kind, offsets, h0, dh, place, states, place)
        assert torch.equal(place, want[2]) and torch.equal(dx, want[0]) and torch.equal(dg, want[1]), turn
    if p is not None:
        forms.within(place.cpu(), p.dh0, p.dh0_tol, "dh0")


# rows of sequences, and which of them the tests touch: by tiles, whose gates'
# product falls below the smallest fp32 value over their rows, and row by row
LONG = [([4000], 0), ([700, 0, 9000, 300], 2), ([2100, 5000], 0), ([100] * 400, 7)]


def gates_and(lengths, C, dtype, kind):
    x, gate, h0, offsets, dh, dlast = forms.inputs(lengths, C, dtype, kind)
    if kind == "decay":      # none that remembers nothing
        gate = torch.where(gate == 0, torch.full_like(gate, 0.4), gate)
    return x, gate, h0, offsets, dh, dlast


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths,at", LONG)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")], ids=["nan", "inf", "-inf"])
def test_a_state_that_is_not_finite_stays_so_to_its_sequences_end(value, lengths, at, kind, dtype):
    """h = a h + b with a > 0 and b finite: an infinity stays that infinity, NaN
    NaN, and nothing else changes; the gradient the same in the other order."""
    C = 70
    say(f"[case] {value} in {len(lengths)} sequences {kind} {dtype}")
    x, gate, h0, offsets, dh, dlast = gates_and(lengths, C, dtype, kind)
    if kind == "decay":
        gate = gate.abs()
    begin = sum(lengths[:at])
    end, S, T = begin + lengths[at], len(lengths), x.shape[0]
    clean_last, clean_states = torch.empty_like(h0), forms.kept(T, C)
    clean = recurrence(x, gate, kind, offsets=offsets, h0=h0, last=clean_last, states=clean_states)
    grads = recurrence_backward(dh, x, gate, clean_states, kind, offsets=offsets, h0=h0, dlast=dlast)
    same = (lambda t: t.isnan()) if value != value else (lambda t: t == value)  # noqa: E731
    for row in (begin, begin + 20):
        bad, bad0 = x.clone(), h0.clone()
        bad[row, 3] = value
        bad0[at, 5] = value
        last, states = torch.empty_like(h0), forms.kept(T, C)
        h = recurrence(bad, gate, kind, offsets=offsets, h0=bad0, last=last, states=states)
        hit, ends = torch.zeros_like(h, dtype=torch.bool), torch.zeros_like(last, dtype=torch.bool)
        hit[row:end, 3], hit[begin:end, 5], ends[at, 3], ends[at, 5] = True, True, True, True
        assert same(h[hit]).all() and same(last[ends]).all()
        assert torch.equal(h[~hit], clean[~hit]) and torch.equal(last[~ends], clean_last[~ends])
        # the states kept are those of h: the gradient of the gate reads them
        dgate = recurrence_backward(dh, bad, gate, states, kind, offsets=offsets, h0=bad0, dlast=dlast)[1]
        if kind == "sigmoid":
            touched = torch.zeros_like(hit)
            touched[row:end, 3], touched[begin:end, 5] = True, True
            assert not dgate[touched].isfinite().any() and torch.equal(dgate[~touched], grads[1][~touched])
        else:
            assert not dgate[3].isfinite() and not dgate[5].isfinite() and dgate[6:].isfinite().all()
    for row in (end - 1, end - 21):
        bad, bad_last = dh.clone(), dlast.clone()
        bad[row, 3] = value
        bad_last[at, 5] = value
        dx, dgate, dh0 = recurrence_backward(bad, x, gate, clean_states, kind, offsets=offsets, h0=h0, dlast=bad_last)
        hit, ends = torch.zeros_like(dx, dtype=torch.bool), torch.zeros_like(dh0, dtype=torch.bool)
        hit[begin:row + 1, 3], hit[begin:end, 5], ends[at, 3], ends[at, 5] = True, True, True, True
        assert same(dx[hit]).all() and same(dh0[ends]).all()
        assert torch.equal(dx[~hit], grads[0][~hit]) and torch.equal(dh0[~ends], grads[2][~ends])
        if kind == "sigmoid":
            assert not dgate[hit].isfinite().any() and torch.equal(dgate[~hit], grads[1][~hit])


@pytest.mark.parametrize("kind", KINDS)
def test_a_gate_of_zero_forgets_a_finite_state(kind):
    """Rows whose gate is 0 in the middle of tiles, and at their ends, whatever
    finite state came before; rows behind them are those of a sequence that
    begins there."""
    T, C = 3000, 130
    x, gate, _, _, _, _ = forms.inputs([T], C, torch.float32, kind)
    if kind == "decay":
        gate = torch.zeros_like(gate)
        assert torch.equal(recurrence(x, gate, kind, h0=torch.full((1, C), 1e30, device=DEV)), x)
        return
    cuts = [0, 5, 128, 1023, 1024, 2048, 2999]
    for c in cuts:
        gate[c] = float("-inf")
    first = torch.full((1, C), 1e30, device=DEV)
    h = recurrence(x, gate, h0=first)
    for a, b in zip(cuts, cuts[1:] + [T]):
        p = forms.Plain([b - a], x[a:b], gate[a:b], kind, None)
        forms.within(h[a:b].cpu(), p.h, p.h_tol, f"rows from {a}")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gates_keep_their_relative_accuracy(dtype):
    """a and 1 - a of a logit, each by itself: a state of 2^60 and no input
    leaves a 2^60, an input of 1 and no state 1 - a.  At worst one is off by 2 u
    for the exponential, 3 for its correction, 1 for the sum, 2 for the reciprocal
    and 1 for the product: 12 u are enough."""
    from layers import U32
    g = torch.arange(-86.0, 86.25, 0.25).to(dtype).unique()
    S = len(g)
    gate = g.view(S, 1).to(DEV).contiguous()
    want = torch.sigmoid(g.double())
    rest = torch.sigmoid(-g.double())
    for rows in (1, 700):                       # one wave's sequences; tiles
        x = torch.zeros((rows, S), device=DEV, dtype=dtype)
        h0, last = torch.full((1, S), 2.0 ** 60, device=DEV), torch.empty((1, S), device=DEV)
        logits = gate.view(1, S).expand(rows, S).contiguous()
        if rows > 1:                            # all but one row keep the state
            logits[1:] = float("inf")
        recurrence(x, logits, sequences=1, h0=h0, last=last)
        forms.within(last[0].cpu() * 2.0 ** -60, want, 12 * U32 * want, "a")
        x[0] = 1
        recurrence(x, logits, sequences=1, last=last)
        forms.within(last[0].cpu(), rest, 12 * U32 * rest, "1 - a")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_a_logit_of_minus_infinity_is_a_gate_of_zero(dtype):
    x = torch.zeros((40, 2), device=DEV, dtype=dtype)
    gate = torch.zeros_like(x)
    gate[0], gate[20] = float("-inf"), torch.finfo(dtype).min
    h0, last = torch.full((1, 2), 1e30, device=DEV), torch.empty((1, 2), device=DEV)
    assert not recurrence(x, gate, h0=h0, last=last).any() and not last.any()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("lengths", [[1500], [700, 0, 1400], [3, 40, 17] * 20])
def test_decays_above_one(lengths, dtype):
    """States that grow, up to 1.05^1500 = 6e31, with factors of both signs."""
    C = 130
    say(f"[case] growing states {lengths[:3]} {dtype}")
    x, gate, h0, offsets, dh, dlast = forms.inputs(lengths, C, dtype, "decay")
    gate = torch.linspace(0.99, 1.05, C, device=DEV)
    gate[::3] *= -1
    gate[7] = 1.0
    T, S = x.shape[0], len(lengths)
    states, last = forms.kept(T, C), torch.empty_like(h0)
    p = forms.Plain(lengths, x, gate, "decay", h0, dh, dlast)
    h = recurrence(x, gate, "decay", offsets=offsets, h0=h0, states=states, last=last)
    forms.within(h.cpu(), p.h, p.h_tol, "h")
    forms.within(last.cpu(), p.last, p.last_tol, "last")
    dx, dg, d0 = recurrence_backward(dh, x, gate, states, "decay", offsets=offsets, h0=h0, dlast=dlast)
    forms.within(dx.cpu(), p.dx, p.dx_tol, "dx")
    forms.within(d0.cpu(), p.dh0, p.dh0_tol, "dh0")
    small = gate.abs().cpu() < 1.02      # the other gradients' products of states leave fp32
    forms.within(dg.cpu()[small], p.dgate[small], p.dgate_tol[small], "dgate")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_a_largest_decay_over_many_tiles(dtype):
    """1.09 from a state of 0: zeros stay zeros whatever the product of the gates
    has become, and a state that begins late is what it is step by step."""
    T, C = 4000, 6
    x = torch.zeros((T, C), device=DEV, dtype=dtype)
    x[3300:, 1] = 1.0
    x[3990:, 2] = 1e-30
    gate = torch.full((C,), 1.09, device=DEV)
    h = recurrence(x, gate, "decay")
    assert not h[:, [0, 3, 4, 5]].any() and not h[:3300, 1].any() and not h[:3990, 2].any()
    for c, n in ((1, 700), (2, 10)):
        p = forms.Plain([n], x[-n:, c:c + 1], gate[:1], "decay", None)
        forms.within(h[-n:, c:c + 1].cpu(), p.h, p.h_tol, f"channel {c}")
