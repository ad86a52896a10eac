"""Sums over very many rows that a gradient makes, with values for which a lost
share or a careless order shows, and tiles of very many values."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import (RECURRENCE_BLOCK, binding, norm_backward, recurrence,  # noqa: E402
                                 recurrence_backward)

import test_recurrence_gpu as recurrence_forms  # noqa: E402
from layers import DEV, U32, say, within  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,C", [(512, 1001), (333, 900), (500, 250), (512, 3000)])
def test_small_terms_behind_large_ones_of_few_rows(M, C):
    """Eight rows of 1, one for each thread of a channel, then rows of a little
    under half a step of 1, each of which is lost where it is added to a 1 by
    itself.  With four sums to each of eight threads or more, of which the joins
    are at most 2 and 12, that is M / 32 + 14 roundings at most."""
    say(f"[case] sums of {M} x {C}")
    dy = torch.full((M, C), 0.99 * 2.0 ** -24, device=DEV)
    dy[:8] = 1.0
    x = torch.ones((M, C), device=DEV)
    stat = torch.tensor([0.0, 1.0], device=DEV).expand(M, 2).contiguous()
    _, dw, db = norm_backward(dy, x, stat, kind="rms", need=("dweight", "dbias"))
    want = dy.double().sum(0)
    tol = (M / 32 + 14) * U32 * want
    within(dw, want, tol, "dweight")
    within(db, want, tol, "dbias")


# ----------------------------------------------------------------------------
# sums of very many rows whose value is known exactly
# ----------------------------------------------------------------------------
def test_normalisation_gradients_of_a_million_rows():
    """dy of ones at some 150 random rows of each channel (fewer than 257, which
    bf16 holds), n of 1 and -1: counts, exactly.  A share that is lost misses
    ones in most of its 600 channels."""
    M, C = 1 << 20, 600
    say(f"[case] counts of {M} x {C}")
    gen = torch.Generator(device=DEV).manual_seed(3)
    for dtype in (torch.bfloat16, torch.float32):
        dy = (torch.rand((M, C), generator=gen, device=DEV) < 150 / M).to(dtype)
        x = (torch.randint(0, 2, (M, C), generator=gen, device=DEV, dtype=torch.int8) * 2 - 1).to(dtype)
        stat = torch.tensor([0.0, 1.0], device=DEV).expand(M, 2).contiguous()
        for need in (("dweight", "dbias"), ("dx", "dweight", "dbias")):
            _, dw, db = norm_backward(dy, x, stat, need=need)
            want = dy.sum(0, dtype=torch.float32)
            assert 50 < want.min() and want.max() < 257
            assert torch.equal(db.float(), want)
            assert torch.equal(dw.float(), torch.where(x > 0, dy, -dy).sum(0, dtype=torch.float32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[1 << 20], [300000, 0, 1, 500000, 248575], [256] * 4096, [1] * 40000],
                         ids=["one", "four", "many", "steps"])
def test_gradient_of_a_decay_over_a_million_rows(lengths, dtype):
    """A decay of 0 leaves d = dh and h = x, so that its gradient is the sum over
    the rows behind a sequence's first of dh[t] x[t - 1]: small whole numbers,
    whose sum of both signs stays below 2^24 at every step, exactly."""
    T, C, S = sum(lengths), 130, len(lengths)
    say(f"[case] gradient of a decay over {T} rows in {S} sequences")
    gen = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randint(1, 4, (T, C), generator=gen, device=DEV).to(dtype)
    dh = torch.randint(-1, 4, (T, C), generator=gen, device=DEV).to(dtype)
    h0 = torch.randint(1, 4, (S, C), generator=gen, device=DEV).float()
    offsets = torch.tensor([0] + lengths, device=DEV).cumsum(0).int()
    gate = torch.zeros(C, device=DEV)
    states = torch.empty((-(-T // RECURRENCE_BLOCK), C), device=DEV)
    h = recurrence(x, gate, "decay", offsets=offsets, h0=h0, states=states)
    assert torch.equal(h, x)
    dx, dg, dh0 = recurrence_backward(dh, x, gate, states, "decay", offsets=offsets, h0=h0)
    assert torch.equal(dx, dh) and not dh0[[n > 0 for n in lengths]].any()
    before = torch.cat([x[:1], x[:-1]]).double()
    full = torch.tensor(lengths, device=DEV) > 0
    before[offsets[:-1][full].long()] = h0[full].double()
    want = (dh.double() * before).sum(0)
    assert want.abs().max() < 2 ** 24
    assert torch.equal(dg.double(), want)


def test_tiles_of_more_than_2_31_values():
    """Long sequences, whose rows go by tiles: 2^20 rows of 2304, some of them a
    sequence of one row.  The first and last rows of every sequence against the
    64-bit form of 40 rows: with gates of at most 0.4 what lies further away
    adds less than 1e-14."""
    C = 2304
    lengths = [350000, 1, 0, 400000, 17]
    lengths.append((1 << 20) - sum(lengths))
    T, S = 1 << 20, len(lengths)
    say(f"[case] tiles of {T} x {C}")
    gen = torch.Generator(device=DEV).manual_seed(5)

    def many(mean=0.0, most=None):
        t = torch.empty((T, C), dtype=torch.bfloat16, device=DEV)
        for part in t.split(1 << 16):
            v = torch.randn(part.shape, generator=gen, device=DEV) + mean
            part.copy_(v if most is None else v.clamp(max=most))
        return t

    x, gate, dh = many(), many(-1.5, -0.41), many()
    h0, dlast = (torch.randn((S, C), generator=gen, device=DEV) for _ in range(2))
    offsets = torch.tensor([0] + lengths, device=DEV).cumsum(0).int()
    states, last = torch.empty((T // RECURRENCE_BLOCK, C), device=DEV), torch.empty_like(h0)
    h = recurrence(x, gate, offsets=offsets, h0=h0, states=states, last=last)
    dx, dg, d0 = recurrence_backward(dh, x, gate, states, offsets=offsets, h0=h0, dlast=dlast)
    n, keep, begin = 80, 40, 0
    for s, length in enumerate(lengths):
        end = begin + length
        if length <= n:
            p = recurrence_forms.Plain([length], x[begin:end], gate[begin:end], "sigmoid", h0[s:s + 1], dh[begin:end],
                                       dlast[s:s + 1])
            for got, name in ((h, "h"), (dx, "dx"), (dg, "dgate")):
                within(got[begin:end].cpu(), getattr(p, name), getattr(p, name + "_tol"), name)
            within(last[s:s + 1].cpu(), p.last, p.last_tol, "last")
            within(d0[s:s + 1].cpu(), p.dh0, p.dh0_tol, "dh0")
        else:
            a, b = slice(begin, begin + n), slice(end - n, end)
            p = recurrence_forms.Plain([n], x[a], gate[a], "sigmoid", h0[s:s + 1], dh[a], None)
            for got, name in ((h, "h"), (dx, "dx"), (dg, "dgate")):
                within(got[a][:keep].cpu(), getattr(p, name)[:keep], getattr(p, name + "_tol")[:keep] + 1e-12, name)
            within(d0[s:s + 1].cpu(), p.dh0, p.dh0_tol + 1e-12, "dh0")
            p = recurrence_forms.Plain([n], x[b], gate[b], "sigmoid", None, dh[b], dlast[s:s + 1])
            for got, name in ((h, "h"), (dx, "dx"), (dg, "dgate")):
                within(got[b][keep:].cpu(), getattr(p, name)[keep:], getattr(p, name + "_tol")[keep:] + 1e-12, name)
            within(last[s:s + 1].cpu(), p.last, p.last_tol + 1e-12, "last")
        begin = end
