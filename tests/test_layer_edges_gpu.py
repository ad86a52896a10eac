"""norm, recurrence and gated_linear at their edges: arrays of more than 2^31
values, the stated limits, workspaces of the stated size, calls of two streams
and of threads at once."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import (RECURRENCE_BLOCK, binding, gated_linear, gated_linear_backward, norm,  # noqa: E402
                                 norm_backward, recurrence, recurrence_backward)

import test_gated_gpu as gated_forms  # noqa: E402
import test_norm_gpu as norm_forms  # noqa: E402
import test_recurrence_gpu as recurrence_forms  # noqa: E402
from layers import DEV, generator, rand, say, within  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()
    yield
    torch.cuda.empty_cache()


def many(gen, *shape, mean=0.0):
    """Normal values in bf16 without an array of them in fp32."""
    t = torch.empty(shape, dtype=BF16, device=DEV)
    for part in t.split(1 << 16):
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) + mean)
    return t


def test_norm_of_very_many_values():
    M, C = 1 << 20, 2304
    say(f"[case] norm {M} x {C}")
    gen = generator(1)
    x, dy, w = many(gen, M, C), many(gen, M, C), rand(gen, C, mean=1.0, dtype=BF16)
    stat = torch.empty((M, 2), device=DEV)
    y = norm(x, w, stat=stat)
    dx, dw, db = norm_backward(dy, x, stat, w)
    for rows in (slice(0, 3), slice(M // 2 + 1, M // 2 + 4), slice(M - 3, M)):
        p = norm_forms.Plain(x[rows], w, None, "layer", dy=dy[rows])
        within(y[rows], p.y, p.y_tol, "y")
        within(dx[rows], p.dx, p.dx_tol, "dx")
    want, size = torch.zeros(C, dtype=torch.float64, device=DEV), torch.zeros(C, dtype=torch.float64, device=DEV)
    for part in dy.split(1 << 16):
        want += part.double().sum(0)
        size += part.double().abs().sum(0)
    within(db, want, (M / 512 + 600) * 2.0 ** -24 * size + 2.0 ** -8 * want.abs(), "dbias")


def test_recurrence_of_very_many_values():
    S, L, C = 4096, 256, 2304
    T = S * L
    say(f"[case] recurrence {S} x {L} x {C}")
    gen = generator(2)
    x, gate, dh = many(gen, T, C), many(gen, T, C, mean=1.5), many(gen, T, C)
    h0, dlast = rand(gen, S, C), rand(gen, S, C)
    for where in (dict(sequences=S), dict(offsets=torch.arange(0, T + 1, L, dtype=torch.int32, device=DEV))):
        states, last = torch.empty((T // RECURRENCE_BLOCK, C), device=DEV), torch.empty_like(h0)
        h = recurrence(x, gate, h0=h0, states=states, last=last, **where)
        dx, dg, d0 = recurrence_backward(dh, x, gate, states, h0=h0, dlast=dlast, **where)
        for s in (0, S - 1):
            rows = slice(s * L, (s + 1) * L)
            p = recurrence_forms.Plain([L], x[rows], gate[rows], "sigmoid", h0[s:s + 1], dh[rows], dlast[s:s + 1])
            within(h[rows].cpu(), p.h, p.h_tol, "h")
            within(last[s:s + 1].cpu(), p.last, p.last_tol, "last")
            within(dx[rows].cpu(), p.dx, p.dx_tol, "dx")
            within(dg[rows].cpu(), p.dgate, p.dgate_tol, "dgate")
            within(d0[s:s + 1].cpu(), p.dh0, p.dh0_tol, "dh0")


def test_recurrence_of_one_very_long_sequence():
    """2^20 rows: every level of the words that the tiles pass on, and sums of
    a gradient over all of them."""
    T, C = 1 << 20, 130
    say(f"[case] recurrence {T} x {C}")
    gen = generator(3)
    x, dh = rand(gen, T, C, dtype=BF16), rand(gen, T, C, dtype=BF16)
    decay = 0.9 + 0.09 * torch.rand(C, generator=gen, device=DEV)
    states = torch.empty((T // RECURRENCE_BLOCK, C), device=DEV)
    h = recurrence(x, decay, "decay", states=states)
    # a state forgets: 0.99^4000 is 3e-18, so that the last rows do not know where the sequence began
    n = 5000
    p = recurrence_forms.Plain([n], x[-n:], decay, "decay", None)
    within(h[-500:].cpu(), p.h[-500:], p.h_tol[-500:] + 1e-15, "h")
    dx, dg, d0 = recurrence_backward(dh, x, decay, states, "decay")
    p = recurrence_forms.Plain([n], x[:n], decay, "decay", None, dh[:n])
    within(dx[:500].cpu(), p.dx[:500], p.dx_tol[:500] + 1e-15, "dx")
    # dgate from the kernel's own d (before rounding it is dx) and h, in 64 bits: rounded by 2^-8 each, over T rows
    before = torch.cat([torch.zeros((1, C), device=DEV, dtype=BF16), h[:-1]]).double()
    terms = dx.double() * before
    within(dg, terms.sum(0), (2 * 2.0 ** -8 + 2.0 ** -16) * terms.abs().sum(0), "dgate")


def test_gated_linear_of_very_many_values():
    M, N, K = 70000, 32768, 16
    say(f"[case] gated {M} x {N} x {K}")
    gen = generator(4)
    x, wg, wu = rand(gen, M, K, dtype=BF16), rand(gen, N, K, sd=0.3, dtype=BF16), rand(gen, N, K, sd=0.3, dtype=BF16)
    dy = many(gen, M, N)
    pre = torch.empty((2, M, N), device=DEV)
    y = gated_linear(x, wg, wu, pre=pre)
    dx, dwg, dwu, _, dbu = gated_linear_backward(dy, x, wg, wu, pre, need=("dx", "dwg", "dwu", "dbu"))
    for rows in (slice(0, 2), slice(M - 2, M)):
        p = gated_forms.Plain(x[rows], wg, wu, None, None, "silu", dy[rows])
        within(y[rows], p.y, p.y_tol, "y")
        within(dx[rows], p.grads["dx"], p.tols["dx"], "dx")
    for cols in (slice(0, 2), slice(N - 2, N)):
        p = gated_forms.Plain(x, wg[cols], wu[cols], None, None, "silu", dy[:, cols].contiguous())
        within(dwg[cols], p.grads["dwg"], p.tols["dwg"], "dwg")
        within(dwu[cols], p.grads["dwu"], p.tols["dwu"], "dwu")
        within(dbu[cols], p.grads["dbu"], p.tols["dbu"], "dbu")


def test_norm_at_its_limits():
    gen = generator(5)
    x = rand(gen, 1 << 20, 3, dtype=BF16)
    p = norm_forms.Plain(x, None, None, "layer")
    within(norm(x), p.y, p.y_tol, "y")
    for dtype in (BF16, torch.float32):
        norm_forms.check(600, 32768, dtype, "layer", residual=True, affine=True)     # shares of many rows


@pytest.mark.parametrize("kind", ["sigmoid", "decay"])
@pytest.mark.parametrize("lengths,C", [([3000, 0, 1100], 130), ([16] * 40, 257), ([1] * 30, 64)])
def test_workspace_of_the_stated_size_is_enough(lengths, C, kind):
    x, gate, h0, offsets, dh, dlast = recurrence_forms.inputs(lengths, C, BF16, kind)
    T, S = x.shape[0], len(lengths)
    states, last = recurrence_forms.kept(T, C), torch.empty_like(h0)
    want_h = recurrence(x, gate, kind, offsets=offsets, h0=h0, states=states, last=last)
    want = recurrence_backward(dh, x, gate, states, kind, offsets=offsets, h0=h0, dlast=dlast)

    def exact(name):
        n = binding._bytes(name, T, S, C, binding.DSPARK_BF16, binding.GATES[kind])
        whole = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=DEV)
        return whole[:n], whole[n:]

    ws, tail = exact("recurrence")
    wb, tail_b = exact("recurrence_backward")
    for _ in range(2):      # whatever the workspace holds, its last call's rest too
        h = recurrence(x, gate, kind, offsets=offsets, h0=h0, workspace=ws)
        got = recurrence_backward(dh, x, gate, states, kind, offsets=offsets, h0=h0, dlast=dlast, workspace=wb)
        assert torch.equal(h, want_h) and all(torch.equal(a, b) for a, b in zip(got, want))
        assert (tail == 0xFF).all() and (tail_b == 0xFF).all()


def test_two_streams_and_threads_at_once():
    """Calls of two streams overlap, each with a workspace of its own; calls of
    threads on one stream come one after the other."""
    made = [recurrence_forms.inputs([9000], 384, BF16, "sigmoid", seed=i) for i in range(2)]

    def call(i):
        x, gate, h0, offsets, dh, dlast = made[i]
        states, last = recurrence_forms.kept(9000, 384), torch.empty_like(h0)
        h = recurrence(x, gate, offsets=offsets, h0=h0, states=states, last=last)
        stat = torch.empty((9000, 2), device=DEV)
        return (h, last, norm(h, stat=stat)) + recurrence_backward(dh, x, gate, states, offsets=offsets, h0=h0, dlast=dlast) \
            + norm_backward(dh, h, stat)

    want = [call(0), call(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(call(i))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    results = {}

    def work(i):
        for k in range(8):
            results[i, k] = call(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(results) == 16
    for (i, _), got in results.items():
        assert all(torch.equal(p, q) for p, q in zip(got, want[i]))
