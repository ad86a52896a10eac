"""A recurrent backbone's layer, made of norm(), recurrence(), linear() and
gated_linear() as a program would: trained, run one token at a time and
captured into graphs; and the RNN head's state trained under the heads' loss."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import (RECURRENCE_BLOCK, binding, gated_linear, gated_linear_backward, linear,  # noqa: E402
                                 linear_backward, markov_loss, markov_loss_backward, norm, norm_backward, recurrence,
                                 recurrence_backward)

from layers import DEV, generator, rand, replays, say  # noqa: E402

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


def weights(d, f, dtype, seed=0):
    gen = generator(seed)
    sd = math.sqrt(1.0 / d)
    return dict(n1=rand(gen, d, sd=0.1, mean=1.0, dtype=dtype), n2=rand(gen, d, sd=0.1, mean=1.0, dtype=dtype),
                wx=rand(gen, d, d, sd=sd, dtype=dtype), wr=rand(gen, d, d, sd=sd, dtype=dtype),
                wo=rand(gen, d, d, sd=sd, dtype=dtype), wg=rand(gen, f, d, sd=sd, dtype=dtype),
                wu=rand(gen, f, d, sd=sd, dtype=dtype), wd=rand(gen, d, f, sd=math.sqrt(1.0 / f), dtype=dtype))


def forward(w, stream, h0, offsets=None, keep=None, last=None):
    """One layer on the residual stream [T, d]; `keep` (a dict) takes what the gradient needs."""
    T, d = stream.shape
    f32 = lambda *s: torch.empty(s, device=DEV) if keep is not None else None  # noqa: E731
    st1, st2, states = f32(T, 2), f32(T, 2), f32(-(-T // RECURRENCE_BLOCK), d)
    pre = f32(2, T, w["wg"].shape[0])
    y1 = norm(stream, w["n1"], kind="rms", eps=EPS, stat=st1)
    x, g = linear(y1, w["wx"]), linear(y1, w["wr"])
    h = recurrence(x, g, offsets=offsets, h0=h0, last=last, states=states)
    o = linear(h, w["wo"])
    y2, s = norm(o, w["n2"], residual=stream, kind="rms", eps=EPS, stat=st2)
    a = gated_linear(y2, w["wg"], w["wu"], pre=pre)
    out = linear(a, w["wd"], residual=s)
    if keep is not None:
        keep.update(st1=st1, st2=st2, states=states, pre=pre, y1=y1, x=x, g=g, h=h, s=s, y2=y2, a=a)
    return out


def backward(w, k, stream, h0, dout, offsets=None):
    grads = {}
    da, grads["wd"], _ = linear_backward(dout, k["a"], w["wd"], need=("dx", "dw"))
    dy2, grads["wg"], grads["wu"], _, _ = gated_linear_backward(da, k["y2"], w["wg"], w["wu"], k["pre"],
                                                               need=("dx", "dwg", "dwu"))
    ds, grads["n2"], _ = norm_backward(dy2, k["s"], k["st2"], w["n2"], dsum=dout, kind="rms", need=("dx", "dweight"))
    dh, grads["wo"], _ = linear_backward(ds, k["h"], w["wo"], need=("dx", "dw"))
    dx, dg, grads["h0"] = recurrence_backward(dh, k["x"], k["g"], k["states"], offsets=offsets, h0=h0)
    d1, grads["wx"], _ = linear_backward(dx, k["y1"], w["wx"], need=("dx", "dw"))
    d2, grads["wr"], _ = linear_backward(dg, k["y1"], w["wr"], need=("dx", "dw"))
    grads["stream"], grads["n1"], _ = norm_backward(d1 + d2, stream, k["st1"], w["n1"], dsum=ds, kind="rms",
                                                    need=("dx", "dweight"))
    return grads


def plain(w, stream, h0, lengths):
    """The layer in 64 bits, with autograd."""
    def rms(v, n):
        return v / ((v * v).mean(1, keepdim=True) + EPS).sqrt() * n

    y1 = rms(stream, w["n1"])
    x, a = y1 @ w["wx"].T, torch.sigmoid(y1 @ w["wr"].T)
    rows, at = [], 0
    for s, n in enumerate(lengths):
        v = h0[s]
        for t in range(at, at + n):
            v = a[t] * v + (1 - a[t]) * x[t]
            rows.append(v)
        at += n
    s = torch.stack(rows) @ w["wo"].T + stream
    y2 = rms(s, w["n2"])
    return torch.nn.functional.silu(y2 @ w["wg"].T) * (y2 @ w["wu"].T) @ w["wd"].T + s


def relative(got, want):
    return float((got.double() - want).norm() / want.norm().clamp(min=1e-30))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[5, 0, 40, 1], [16] * 6, [200]])
def test_layer_in_training(lengths, dtype):
    """Every gradient against autograd's of the 64-bit form.  In fp32 each of
    the layer's ten operators errs by at most 1e-5 of the norm (sums of 96 terms
    in fp32: 98 half steps of 2^-24 are 6e-6), in bf16 by two roundings of 2^-8
    at most: ten in a row, 1e-4 and 0.08."""
    d, f = 64, 96
    T, S = sum(lengths), len(lengths)
    say(f"[case] layer {lengths} {dtype}")
    w = weights(d, f, dtype)
    gen = generator(5)
    stream, h0, dout = rand(gen, T, d, dtype=dtype), rand(gen, S, d), rand(gen, T, d, dtype=dtype)
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    offsets = torch.tensor(at, dtype=torch.int32, device=DEV)
    keep = {}
    out = forward(w, stream, h0, offsets, keep)
    grads = backward(w, keep, stream, h0, dout, offsets)
    leaves = {k: v.double().requires_grad_() for k, v in {**w, "stream": stream, "h0": h0}.items()}
    ref = plain({k: leaves[k] for k in w}, leaves["stream"], leaves["h0"], lengths)
    want = dict(zip(leaves, torch.autograd.grad(ref, list(leaves.values()), dout.double())))
    tol = 1e-4 if dtype is torch.float32 else 0.08
    assert relative(out, ref.detach()) <= tol
    for name, g in want.items():
        assert relative(grads[name], g) <= tol, name


@pytest.mark.parametrize("T", [7, 150])
def test_layer_one_token_at_a_time(T):
    """A prompt, then tokens one by one with the state carried on: the same
    stream, to the roundings of the different kernels (each output of the layer
    is rounded to bf16 after at most seven operators that round by 2^-8)."""
    d, f, S, more = 128, 256, 3, 4
    w = weights(d, f, torch.bfloat16)
    stream = rand(generator(8), S, T + more, d, dtype=torch.bfloat16)
    state = torch.zeros((S, d), device=DEV)
    whole = forward(w, stream.view(-1, d), torch.zeros_like(state)).view(S, T + more, d)
    forward(w, stream[:, :T].reshape(-1, d), state, last=state)
    for t in range(T, T + more):
        out = forward(w, stream[:, t].contiguous(), state, last=state)
        assert relative(out, whole[:, t].double()) <= 7 * 2 ** -8, t


def test_layer_captured_with_its_gradients():
    d, f, S, L = 128, 200, 4, 60
    w = weights(d, f, torch.bfloat16)
    new = lambda seed: (rand(generator(seed), S * L, d, dtype=torch.bfloat16), rand(generator(seed + 1), S, d),  # noqa: E731
                        rand(generator(seed + 2), S * L, d, dtype=torch.bfloat16))
    stream, h0, dout = new(1)

    def step():
        keep = {}
        out = forward(w, stream, h0, keep=keep)
        g = backward(w, keep, stream, h0, dout)
        return [out] + [g[k] for k in sorted(g)]

    seeds = iter(range(10, 1000, 3))
    replays(step, [stream, h0, dout], lambda: new(next(seeds)), lambda o: o)


def test_two_graphs_replayed_at_once():
    """Graphs that hold the same calls have workspaces of their own."""
    C, T = 256, 3000
    gen = generator(3)
    cases = []
    for i in range(2):
        x, g, dh = (rand(gen, T, C, dtype=torch.bfloat16) for _ in range(3))
        w = rand(gen, 2, 77, C, sd=0.1, dtype=torch.bfloat16)

        def call(x=x, g=g, dh=dh, w=w):
            states = torch.empty((-(-T // RECURRENCE_BLOCK), C), device=DEV)
            h = recurrence(x, g, states=states)
            pre = torch.empty((2, 300, 77), device=DEV)
            y = gated_linear(h[:300], w[0], w[1], pre=pre)
            stat = torch.empty((T, 2), device=DEV)
            n = norm(h, stat=stat)
            return (h, y, n) + recurrence_backward(dh, x, g, states)[:2] + \
                tuple(gated_linear_backward(y, h[:300], w[0], w[1], pre)) + tuple(norm_backward(dh, h, stat))

        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = call()
        cases.append((graph, torch.cuda.Stream(), held, want, call))   # call: a graph does not keep its inputs
    for _ in range(5):
        for graph, stream, *_ in cases:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, held, want, _ in cases:
            assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_rnn_head_in_training(dtype):
    """The RNN head's state over every request's draft positions, under the
    loss of the logits U + s W2: the gradients of the decay, the embeddings'
    rows and W2 against autograd's of the 64-bit form."""
    B, gamma, V, r = 6, 8, 200, 32
    gen = generator(21)
    E = rand(gen, B * gamma, r, sd=0.5, dtype=dtype)                # W1[x_{k-1}]
    W2 = rand(gen, r, V, sd=0.5, dtype=dtype)
    U = rand(gen, B * gamma, V, dtype=dtype)
    decay = 0.2 + 0.7 * torch.rand(r, generator=gen, device=DEV)
    label = torch.randint(0, V, (B * gamma,), generator=gen, device=DEV, dtype=torch.int32)
    weight = torch.full((B * gamma,), 1.0 / (B * gamma), device=DEV)
    states = torch.empty((-(-B * gamma // RECURRENCE_BLOCK), r), device=DEV)
    s = recurrence(E, decay, "decay", sequences=B, states=states)
    Wo = W2.t().contiguous()
    nll, lse = markov_loss(label, U=U, h=s, Wo=Wo)
    g = markov_loss_backward(weight, lse, label, U=U, h=s, Wo=Wo, need=("dh", "dWo"))
    dE, ddecay, _ = recurrence_backward(g["dh"], E, decay, states, "decay", sequences=B, need=("dx", "dgate"))
    e, w2, a = (t.double().requires_grad_() for t in (E, W2, decay))
    rows, v = [], None
    for t in range(B * gamma):
        v = e[t] if t % gamma == 0 else a * v + e[t]
        rows.append(v)
    z = torch.stack(rows) @ w2 + U.double()
    loss = torch.nn.functional.cross_entropy(z, label.long())
    value = float(loss.detach())
    want = torch.autograd.grad(loss, (e, w2, a))
    # three roundings of the storage type (s, dz, the result) and the fp32 sums
    tol = 4 * 2.0 ** -8 if dtype is torch.bfloat16 else 1e-5
    assert abs(float((nll * weight).sum()) - value) <= tol * value
    for got, ref, name in ((dE, want[0], "dE"), (g["dWo"].t(), want[1], "dW2"), (ddecay, want[2], "ddecay")):
        assert relative(got, ref) <= tol, name
