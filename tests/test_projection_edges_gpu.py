"""The projection's operators at the edges: values that are not finite, empty
batches, the tails of the activations, the largest sizes.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import (binding, hidden_draft, linear, linear_backward, markov_draft,  # noqa: E402
                                 markov_loss, markov_loss_backward)

DEV = "cuda:0"
U32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step of the type
TYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


def rand(seed, *shape, sd=1.0, dtype=torch.float32):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=DEV) * sd).to(dtype)


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_nan_passes_every_activation(act, dtype):
    """A row of x that holds NaN gives a row of NaN, forward and backward (dx
    of that row, and every weight gradient: its rows sum over all of them)."""
    for M, N, K in ((3, 40, 64), (40, 300, 200)):
        x, w, b = rand(1, M, K, dtype=dtype), rand(2, N, K, sd=0.1, dtype=dtype), rand(3, N, dtype=dtype)
        dy = rand(4, M, N, dtype=dtype)
        pre = torch.empty(M, N, device=DEV)
        clean = linear(x, w, bias=b, act=act)
        x[1, 5] = math.nan
        y = linear(x, w, bias=b, act=act, pre=pre)
        rest = [i for i in range(M) if i != 1]
        assert torch.isnan(y[1]).all() and torch.equal(y[rest], clean[rest])
        if act == "none":
            continue
        dx, dw, db = linear_backward(dy, x, w, act=act, pre=pre)
        assert torch.isnan(dx[1]).all() and torch.isfinite(dx[rest]).all()
        assert torch.isnan(dw).all() and torch.isnan(db).all()


# Contractions whose last step is not whole, through every tile of the products: few and many rows, rows that are
# 16-byte aligned, copied, and staged as they are.
TAILS = [(2, 40, 72), (20, 300, 72), (40, 300, 200), (100, 300, 136), (300, 520, 200), (20, 300, 77), (40, 300, 201),
         (100, 300, 141), (300, 520, 333), (2000, 4090, 1096)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", TAILS)
def test_infinities_keep_their_sign(M, N, K, dtype):
    """One infinite factor in a sum of finite terms: the sum is infinite, with
    the sign of the other factor, also where it is the last of the contraction
    and what lies behind it is padding.  The other sums do not see it."""
    x, w, dy = rand(5, M, K, dtype=dtype), rand(6, N, K, sd=0.1, dtype=dtype), rand(7, M, N, dtype=dtype)
    y0, (dx0, dw0, _) = linear(x, w), linear_backward(dy, x, w)
    for k in (K - 1, (K - 1) // 64 * 64):
        v = w.clone()
        v[N - 1, k], v[0, k] = math.inf, -math.inf
        y = linear(x, v)
        assert torch.equal(y[:, N - 1].float(), torch.sign(x[:, k].float()) * math.inf)
        assert torch.equal(y[:, 0].float(), torch.sign(x[:, k].float()) * -math.inf)
        assert torch.equal(y[:, 1:N - 1], y0[:, 1:N - 1])
    # dx sums over the features, dw over the rows
    v, z = w.clone(), x.clone()
    v[N - 1, K - 1], z[M - 1, K - 1] = math.inf, -math.inf
    dx, dw, _ = linear_backward(dy, z, v)
    assert torch.equal(dx[:, K - 1].float(), torch.sign(dy[:, N - 1].float()) * math.inf)
    assert torch.equal(dw[:, K - 1].float(), torch.sign(dy[M - 1].float()) * -math.inf)
    assert torch.equal(dx[:, :K - 1], dx0[:, :K - 1]) and torch.equal(dw[:, :K - 1], dw0[:, :K - 1])


# ---------------------------------------------------------------------------
# empty batches
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("K", [8, 9, 72, 333])
def test_gradients_of_nothing_are_zero(K, dtype):
    """No rows: dw and dbias are zero; no features: dx is.  The other axis on
    both sides of the size from which unaligned rows are copied."""
    for n in (5, 256, 1030):
        empty = lambda *sh: torch.empty(sh, dtype=dtype, device=DEV)  # noqa: E731
        dx, dw, db = linear_backward(empty(0, n), empty(0, K), rand(1, n, K, dtype=dtype))
        assert dx.shape == (0, K) and dw.shape == (n, K) and not dw.any() and not db.any()
        dx, dw, db = linear_backward(empty(n, 0), rand(2, n, K, dtype=dtype), empty(0, K))
        assert dx.shape == (n, K) and not dx.any() and dw.shape == (0, K) and db.shape == (0,)


# ---------------------------------------------------------------------------
# the activations' tails
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_activations_to_their_own_scale(dtype):
    """gelu and silu keep the type's precision where they are small: z runs
    over [-13, 13] (gelu(-13) is 1e-37), as the product of 1 and w.  z is exact.
    Beside the half step of the result, 64 u z^2 + 64 u: exp(-z^2 / 2) is off
    by the rounding of its argument (z^2 u, and twice that for its scaling to
    base 2), silu's exp(-z) by less, and polynomial and quotient by a few u
    each; gelu's slope Phi + z phi loses a factor of 4 by cancellation at most
    outside [-1.2, -0.3], and there an absolute 4 u; so does silu's."""
    N = 6000
    w = torch.linspace(-13, 13, N, device=DEV).to(dtype)[:, None].contiguous()
    z = w[:, 0].double()
    x = torch.ones(1, 1, dtype=dtype, device=DEV)
    phi, Phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), 0.5 * torch.erfc(-z / math.sqrt(2))
    sig = torch.sigmoid(z)
    rel = 64 * U32 * (z * z + 1)
    for act, value, slope in (("gelu", z * Phi, Phi + z * phi), ("silu", z * sig, sig + z * sig * (1 - sig))):
        pre = torch.empty(1, N, device=DEV)
        y = linear(x, w, act=act, pre=pre)
        assert torch.equal(pre[0].double(), z)
        off = (y[0].double() - value).abs()
        assert (off <= (HALF[dtype] + rel) * value.abs() + 1e-38).all(), act
        _, _, db = linear_backward(torch.ones(1, N, dtype=dtype, device=DEV), x, w, act=act, pre=pre)
        off = (db.double() - slope).abs()
        near = 16 * U32 * ((z > -3) & (z < 0)).double()
        assert (off <= (HALF[dtype] + 4 * rel) * slope.abs() + near + 1e-38).all(), act + " slope"


# ---------------------------------------------------------------------------
# the largest sizes
# ---------------------------------------------------------------------------
def test_row_gradient_of_very_many_features():
    """Rows of dy so long that 256 of them take more than 2^32 bytes: every row
    of dx is its own row's product.  Row m of dy is 1 + m % 7 in the last 64
    features and zero elsewhere, w is 1 there: dx is 64 (1 + m % 7), exact."""
    M, N, K = 256, 8421504 + 64, 1024
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    dy, w = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV), torch.zeros(N, K, dtype=torch.bfloat16, device=DEV)
    row = 1 + torch.arange(M, device=DEV) % 7
    dy[:, -64:] = row[:, None].to(torch.bfloat16)
    w[-64:] = 1
    dx, _, _ = linear_backward(dy, torch.empty(M, K, dtype=torch.bfloat16, device=DEV), w, need=("dx",))
    assert torch.equal(dx.float(), (64.0 * row)[:, None].expand(M, K))


def test_sizes_that_an_int_does_not_hold_are_refused():
    """More than 2^31 - 1 rows or tokens (of nothing, which takes no memory):
    refused, not cut to 32 bits."""
    none = lambda *sh, dtype=torch.bfloat16: torch.empty(sh, dtype=dtype, device=DEV)  # noqa: E731
    ints, floats = none(1, dtype=torch.int32), none(0, dtype=torch.float32)
    for M in (1 << 31, (1 << 32) + 4):
        for call in (lambda: linear(none(M, 0), none(0, 0)), lambda: linear(none(0, 0), none(M, 0)),
                     lambda: linear_backward(none(M, 0), none(M, 0), none(0, 0)),
                     lambda: markov_loss(ints[:0], U=none(0, M)),
                     lambda: markov_loss_backward(floats, floats, ints[:0], U=none(0, M)),
                     lambda: hidden_draft(ints, none(1, 1, 0), none(M, 0), none(M, 0), none(0, M), floats, 0.0,
                                          torch.ones(1, device=DEV))):
            with pytest.raises(binding.DSparkError, match="over 2"):
                call()


# ---------------------------------------------------------------------------
# workspaces
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gradient_workspace_of_the_stated_size_is_enough(dtype):
    """Without an activation, with and without a copy of dy: a workspace of
    exactly the stated size, in the middle of a larger buffer that keeps what
    it holds around it, and the same gradients as with a larger one."""
    size = binding.load().dspark_linear_backward_act_workspace_bytes
    for M, N, K in ((64, 128, 64), (64, 128, 2050), (300, 512, 256), (2048, 64, 320), (77, 131, 1001), (5, 4100, 129)):
        x, w, dy = rand(1, M, K, dtype=dtype), rand(2, N, K, sd=0.1, dtype=dtype), rand(3, M, N, dtype=dtype)
        n = size(M, N, K, 1 if dtype is torch.bfloat16 else 0, 0)
        room = torch.full((n + 1024,), 91, dtype=torch.uint8, device=DEV)
        off = 512 + (-(room.data_ptr() + 512)) % 256
        got = linear_backward(dy, x, w, workspace=room[off:off + n])
        assert (room[:off] == 91).all() and (room[off + n:] == 91).all()
        more = torch.empty(n + (64 << 20), dtype=torch.uint8, device=DEV)
        assert all(torch.equal(a, b) for a, b in zip(got, linear_backward(dy, x, w, workspace=more)))


# ---------------------------------------------------------------------------
# as a program uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 4096, 64), (3, 40, 64), (16, 300, 129), (77, 1027, 1001), (300, 512, 4096)])
def test_residual_in_place_is_the_residual(M, N, K, dtype):
    """Added in place by every kernel (few rows, tiles, joined splits): the same
    bits as into another array."""
    x, w, b, res = rand(1, M, K, dtype=dtype), rand(2, N, K, sd=0.1, dtype=dtype), rand(3, N, dtype=dtype), rand(4, M, N, dtype=dtype)
    for act in ("none", "silu"):
        want = linear(x, w, bias=b, act=act, residual=res)
        y = res.clone()
        linear(x, w, bias=b, act=act, residual=y, out=y)
        assert torch.equal(y, want)


def test_two_graphs_replayed_at_once():
    """Graphs of the same calls on two streams, replayed together and beside
    eager calls: each has memory of its own."""
    sets = []
    for i in range(3):
        N, V, d, r = 100 + 30 * i, 3001, 72, 24
        s = dict(h=rand(10 * i, N, d, dtype=torch.bfloat16), Wo=rand(10 * i + 1, V, d, sd=0.2, dtype=torch.bfloat16),
                 prev=torch.arange(N, device=DEV, dtype=torch.int32) % 50,
                 W1=rand(10 * i + 2, V, r, sd=0.5, dtype=torch.bfloat16), W2=rand(10 * i + 3, r, V, sd=0.5, dtype=torch.bfloat16))
        label = (torch.arange(N, device=DEV, dtype=torch.int32) * 29) % (V + 200)
        x, w = rand(10 * i + 4, 77, 1001, dtype=torch.bfloat16), rand(10 * i + 5, 1027, 1001, sd=0.1, dtype=torch.bfloat16)
        sets.append((s, label, torch.ones(N, device=DEV) / N, x, w))

    def work(s, label, g, x, w):
        nll, lse = markov_loss(label, **s)
        return [nll, lse, *markov_loss_backward(g, lse, label, **s).values(), linear(x, w, act="gelu")]

    want = [[t.clone() for t in work(*a)] for a in sets]
    graphs = []
    for a in sets[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = work(*a)
        graphs.append((graph, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(6):
        for graph, outs, stream in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        eager = work(*sets[2])
        torch.cuda.synchronize()
        for got, ref in ((eager, want[2]), (graphs[0][1], want[0]), (graphs[1][1], want[1])):
            assert all(torch.equal(p, q) for p, q in zip(got, ref))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_base_logits_aligned_to_their_element_only(dtype):
    """U at an odd element of a larger array, with rows that would keep
    four-value alignment: the same bits as at an aligned address."""
    N, V = 70, 2000
    U, label, g = rand(1, N, V, dtype=dtype), torch.arange(N, device=DEV, dtype=torch.int32) * 17, torch.ones(N, device=DEV)
    label[5] = -1
    moved = torch.empty(N * V + 1, dtype=dtype, device=DEV)[1:].view(N, V)
    moved.copy_(U)
    out = [(a, b, markov_loss_backward(g, b, label, U=t)["dU"]) for t in (U, moved) for a, b in [markov_loss(label, U=t)]]
    assert all(torch.equal(p, q) for p, q in zip(*out)) and not out[0][2][5].any()


def test_many_rows_all_ignored():
    """No row has a label, above and below the number of rows that one launch
    counts for itself."""
    for N in (50, 9001):
        s = dict(h=rand(1, N, 24), Wo=rand(2, 300, 24), prev=torch.zeros(N, dtype=torch.int32, device=DEV),
                 W1=rand(3, 300, 8), W2=rand(4, 8, 300), U=rand(5, N, 300))
        s["h"].fill_(math.nan)
        label = torch.full((N,), 300, dtype=torch.int32, device=DEV)
        nll, lse = markov_loss(label, **s)
        grads = markov_loss_backward(torch.full((N,), math.nan, device=DEV), lse, label, **s)
        assert not nll.any() and not lse.any() and len(grads) == 5
        assert not any(t.any() for t in grads.values())


# ---------------------------------------------------------------------------
# autograd
# ---------------------------------------------------------------------------
def test_inputs_that_require_a_gradient_are_refused():
    """The operators record no graph, so they do not take a tensor whose
    gradient autograd would be asked for; without gradient mode they do."""
    x, w, b, res = rand(1, 8, 16), rand(2, 24, 16), rand(3, 24), rand(4, 8, 24)
    label = torch.zeros(8, dtype=torch.int32, device=DEV)
    s = dict(U=rand(5, 8, 90), h=rand(6, 8, 16), Wo=rand(7, 90, 16), prev=label, W1=rand(8, 90, 8), W2=rand(9, 8, 90))
    g = torch.ones(8, device=DEV)
    _, lse = markov_loss(label, **s)
    calls = [(lambda: linear(x, w, bias=b, residual=res), (x, w, b, res)),
             (lambda: linear_backward(res, x, w), (res, x, w)),
             (lambda: markov_loss(label, **s), [s[k] for k in s if k != "prev"]),
             (lambda: markov_loss_backward(g, lse, label, **s), [g] + [s[k] for k in s if k != "prev"])]
    for call, tensors in calls:
        call()
        for t in tensors:
            t.requires_grad_(True)
            with pytest.raises(RuntimeError, match="no graph"):
                call()
            with torch.no_grad():
                call()
            t.requires_grad_(False)


# ---------------------------------------------------------------------------
# drafting from hidden states
# ---------------------------------------------------------------------------
def hidden_inputs(B, gamma, V, d, r, dtype, seed=0):
    return (torch.randint(0, V, (B,), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV,
                          dtype=torch.int32),
            rand(seed + 1, B, gamma, d, dtype=dtype), rand(seed + 2, V, d, sd=(2 / d) ** 0.5, dtype=dtype),
            rand(seed + 3, V, r, sd=r ** -0.25, dtype=dtype), rand(seed + 4, r, V, sd=r ** -0.25, dtype=dtype),
            rand(seed + 5, d + r, sd=0.05), 1.0, torch.ones(gamma, device=DEV))


def test_hidden_draft_refusals():
    """What is not a device tensor of the right type and shape gets no further
    than the binding; neither does a workspace that is too small."""
    B, gamma, V, d, r = 3, 4, 500, 16, 32
    args = hidden_inputs(B, gamma, V, d, r, torch.bfloat16)
    good = [torch.empty(B, gamma, dtype=t, device=DEV) for t in (torch.int32,) + (torch.float32,) * 3]
    hidden_draft(*args, out=good)
    for i in range(4):
        for wrong, error in ((good[i].cpu(), ValueError), (good[i][:, :3].contiguous(), ValueError),
                             (good[i].half(), TypeError), (good[i].t().contiguous().t(), ValueError), (None, TypeError)):
            with pytest.raises(error):
                hidden_draft(*args, out=good[:i] + [wrong] + good[i + 1:])
    for wrong, error in ((torch.zeros(1 << 20, dtype=torch.uint8), ValueError),
                         (torch.zeros(1 << 20, device=DEV), TypeError),
                         (torch.zeros(64, dtype=torch.uint8, device=DEV), binding.DSparkError)):
        with pytest.raises(error):
            hidden_draft(*args, workspace=wrong)
    for mode in ("argmax", "Greedy", None):
        with pytest.raises(ValueError):
            hidden_draft(*args, mode=mode)


@pytest.mark.parametrize("B,gamma", [(2, 8), (40, 3)])
def test_hidden_draft_captured_and_replayed(B, gamma):
    """Two graphs, captured one after the other and replayed with new inputs in
    place, with eager calls between the replays."""
    V, d, r = 2000, 48, 32
    sets = [hidden_inputs(B, gamma, V, d, r, torch.bfloat16, seed=10 * i) for i in range(3)]

    def work(args):
        U = torch.empty(B, gamma, V, dtype=torch.bfloat16, device=DEV)
        return [U, *hidden_draft(*args, U=U)]

    want = [[t.clone() for t in work(a)] for a in sets]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        held = [t.clone() if isinstance(t, torch.Tensor) else t for t in sets[0]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = work(held)
        graphs.append((graph, held, outs))
    for i in (1, 2, 0, 1):
        for j, (graph, held, _) in enumerate(graphs):
            for dst, src in zip(held, sets[(i + j) % 3]):
                if isinstance(dst, torch.Tensor):
                    dst.copy_(src)
            graph.replay()
        eager = work(sets[i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, want[i]))
        for j, (_, _, outs) in enumerate(graphs):
            assert all(torch.equal(a, b) for a, b in zip(outs, want[(i + j) % 3]))


def test_linear_of_the_most_rows_and_of_the_most_features():
    """2^20 rows, and 2^24 features: values are small whole numbers, so every
    sum is exact in both types, and every row and feature is looked at."""
    for dtype in TYPES:
        for M, N, K in ((1 << 20, 40, 24), (3, 1 << 24, 8), (70, 1 << 24, 8)):
            x = (torch.arange(M * K, device=DEV) % 5 - 2).view(M, K)
            w = (torch.arange(N * K, device=DEV) % 3 - 1).view(N, K)
            dy = (torch.arange(M * N, device=DEV) % 7 == 0).view(M, N).to(dtype)
            xt, wt = x.to(dtype), w.to(dtype)
            y = linear(xt, wt)                       # |y| <= 48: exact in bf16
            assert torch.equal(y, (xt.float() @ wt.float().t()).to(dtype)), (M, N, K)
            del y
            # sums of up to 2^20 whole numbers below 2^22: exact in fp32, rounded once
            dx, dw, db = linear_backward(dy, xt, wt)
            dyf = dy.float()
            assert torch.equal(dx, (dyf @ wt.float()).to(dtype)), (M, N, K)
            assert torch.equal(dw, (dyf.t().contiguous() @ xt.float()).to(dtype)), (M, N, K)
            assert torch.equal(db, dyf.sum(0).to(dtype)), (M, N, K)
            del x, w, dy, xt, wt, dx, dw, db, dyf
            torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_loss_of_the_most_rows(dtype):
    """2^20 rows, a third of them ignored, over a tiny vocabulary whose tokens
    all occur often, against the definition in 64 bits.  With |z| < 8 and 16
    tokens lse and nll are sums of few terms: 64 u of values below 16.  dz is
    off by h and 64 u relative to g, dW1 sums about N / 16 rows of |dE| <= |g|
    |W2| 16 in fp32 in four interleaved sums, 2 (N / 64 + 64) u in all; dW2 and
    dWo sum N terms in fp32, 2 (N + 64) u of the sum of their sizes."""
    N, V, d, r = 1 << 20, 16, 8, 8
    h_, u = HALF[dtype], U32
    label = torch.randint(-8, V, (N,), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV, dtype=torch.int32)
    prev = torch.randint(0, V, (N,), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV, dtype=torch.int32)
    s = dict(h=rand(3, N, d, sd=0.5, dtype=dtype).clamp(-1, 1), Wo=rand(4, V, d, sd=0.5, dtype=dtype).clamp(-1, 1) / 2,
             prev=prev, W1=rand(5, V, r, sd=0.5, dtype=dtype).clamp(-1, 1) / 2,
             W2=rand(6, r, V, sd=0.5, dtype=dtype).clamp(-1, 1))
    g = torch.rand(N, generator=torch.Generator(device=DEV).manual_seed(7), device=DEV)
    nll, lse = markov_loss(label, **s)
    grads = markov_loss_backward(g, lse, label, **s)
    torch.cuda.synchronize()
    used = label >= 0
    hd, Wo, W1, W2 = (s[k].double() for k in ("h", "Wo", "W1", "W2"))
    E = W1[prev.long()]
    z = hd @ Wo.t() + E @ W2
    lse64 = torch.logsumexp(z, 1)
    y = label.long().clamp(min=0)[:, None]
    gu = torch.where(used, g.double(), 0.0)[:, None]
    dz = gu * (torch.softmax(z, 1) - torch.zeros_like(z).scatter_(1, y, 1.0))
    zero = torch.zeros_like(lse64)
    assert ((lse.double() - torch.where(used, lse64, zero)).abs() <= 64 * u * 16).all()
    assert ((nll.double() - torch.where(used, lse64 - z.gather(1, y)[:, 0], zero)).abs() <= 64 * u * 16).all()
    er = h_ * dz.abs() + 64 * u * gu
    E0 = torch.where(used[:, None], E, 0.0)
    put = lambda t: torch.zeros(V, r, dtype=torch.float64, device=DEV).index_add_(0, prev.long(), t)  # noqa: E731
    terms = 2 * (N + 64) * u
    for k, want, size, err, t in (
            ("dh", dz @ Wo, dz.abs() @ Wo.abs(), er @ Wo.abs(), 2 * (V + 8) * u),
            ("dWo", dz.t() @ hd, dz.abs().t() @ hd.abs(), er.t() @ hd.abs(), terms),
            ("dW2", E0.t() @ dz, E0.abs().t() @ dz.abs(), E0.abs().t() @ er, terms),
            ("dW1", put(dz @ W2.t()), put(dz.abs() @ W2.abs().t()), put(er @ W2.abs().t()), terms)):
        tol = err + t * size
        off = (grads[k].double() - want).abs()
        assert (off <= tol + h_ * (want.abs() + tol)).all(), k


def test_linear_of_unaligned_rows_that_are_very_many_values():
    """2^20 rows of 32771 values: their aligned copy is more 16-byte pieces
    than one launch has threads.  Two features in two places of each row: y is
    the sum of x there, whole numbers below 16, exact."""
    M, K = 1 << 20, 32771
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GB of free device memory")
    x, w = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV), torch.zeros(2, K, dtype=torch.bfloat16, device=DEV)
    at = torch.arange(M, device=DEV)
    x[:, 0], x[:, K - 1] = (at % 5).to(torch.bfloat16), (at % 7).to(torch.bfloat16)
    w[0, 0], w[0, K - 1], w[1, K - 1] = 1, 1, -1
    y = linear(x, w, workspace=torch.empty(binding.load().dspark_linear_workspace_bytes(M, 2, K, 1), dtype=torch.uint8,
                                           device=DEV)).float()
    assert torch.equal(y[:, 0], (at % 5 + at % 7).float()) and torch.equal(y[:, 1], -(at % 7).float())
    del x, y
    torch.cuda.empty_cache()


def test_loss_of_the_largest_vocabulary():
    """2^24 tokens: logits that are small whole numbers, so lse is known in
    closed form, and each row's label and gradient at both ends of the
    vocabulary."""
    N, V, r = 5, 1 << 24, 8
    W1 = torch.zeros(V, r, dtype=torch.bfloat16, device=DEV)
    W2 = torch.zeros(r, V, dtype=torch.bfloat16, device=DEV)
    prev = torch.tensor([0, 1, V - 1, V - 2, 77], dtype=torch.int32, device=DEV)
    label = torch.tensor([0, V - 1, V - 1, 5, V // 2], dtype=torch.int32, device=DEV)
    W1[prev.long(), 0] = torch.arange(1, 6, dtype=torch.bfloat16, device=DEV)
    W2[0, label.long()] = 4
    nll, lse = markov_loss(label, prev=prev, W1=W1, W2=W2)
    z = 4.0 * torch.arange(1, 6, dtype=torch.float64, device=DEV)
    hot = torch.unique(label).numel()                       # tokens whose logit is z, the others' is 0
    want = torch.log(hot * torch.exp(z) + (V - hot))
    # V equal terms summed in fp32 over lanes, tiles and threads: below 600 additions deep
    assert ((lse.double() - want).abs() <= 700 * U32 + 2 * U32 * want).all()
    assert ((nll.double() - (want - z)).abs() <= 700 * U32 + 4 * U32 * want).all()
    g = torch.ones(N, device=DEV)
    grads = markov_loss_backward(g, lse, label, prev=prev, W1=W1, W2=W2)
    p = torch.exp(z - want)
    # dW2[0, v] = sum_n W1[prev_n, 0] dz_n(v)
    e = torch.arange(1, 6, dtype=torch.float64, device=DEV)
    for n in range(N):
        v = int(label[n])
        ref = float((e * (p - (label == v).double())).sum())
        assert abs(float(grads["dW2"][0, v]) - ref) <= 3 * 2.0 ** -8 * float((e * (p + 1)).sum())
    cold = float((e * torch.exp(-want)).sum())
    assert abs(float(grads["dW2"][0, 3]) - cold) <= 3 * 2.0 ** -8 * cold
    # dW1[prev_n, 0] = 4 (sum over the hot tokens of p - 1); no other token has a gradient
    for n in range(N):
        ref = 4 * float(hot * p[n] - 1)
        assert abs(float(grads["dW1"][int(prev[n]), 0]) - ref) <= 3 * 2.0 ** -8 * 4 * float(hot * p[n] + 1)
    grads["dW1"][prev.long()] = 0
    assert not grads["dW1"].any() and not grads["dW2"][1:].any()


@pytest.mark.parametrize("mode", ["greedy", "gumbel"])
@pytest.mark.parametrize("dtype,r", [(torch.bfloat16, 64), (torch.float32, 32)], ids=IDS)
def test_hidden_draft_on_another_stream(dtype, r, mode):
    """Both samplings on a stream of their own, shapes in turn on one
    workspace: what linear and markov_draft give."""
    stream = torch.cuda.Stream()
    cases = [hidden_inputs(B, gamma, V, d, r, dtype, seed=B) for B, gamma, V, d in
             ((1, 1, 40, 8), (5, 3, 1203, 33), (20, 4, 3000, 64), (5, 3, 700, 16))]
    torch.cuda.synchronize()
    for _ in range(2):
        got = []
        with torch.cuda.stream(stream):
            for a in cases:
                got.append(hidden_draft(*a, mode=mode, seed=99))
        torch.cuda.synchronize()
        for a, out in zip(cases, got):
            anchor, h, Wo, W1, W2, cw, cb, T = a
            U = linear(h.view(-1, h.shape[2]), Wo).view(h.shape[0], h.shape[1], -1)
            want = markov_draft(anchor, U, h, W1, W2, cw, cb, T, mode=mode, seed=99)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, want)) and (out[0] >= 0).all()
