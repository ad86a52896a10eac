"""Measured cases of a recurrent backbone's layer: ``norm`` (layer or
root-mean-square normalisation with the residual stream's sum), ``recurrence``
(a gated linear recurrence over packed sequences) and ``gated_linear`` (the
gated feed-forward projection), forward and backward.

Shapes are those of the package's workloads: hidden sizes 2560 to 5120, Markov
rank 256, requests x draft positions as rows; sequence lengths and feed-forward
widths are generic.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def norm_case(M, C, dtype="bf16", kind="layer", residual=False, train=False, **name):
    return dict(name, op="norm", M=M, C=C, dtype=dtype, kind=kind, residual=residual, train=train)


def gated_case(M, N, K, dtype="bf16", act="silu", bias=False, train=False, **name):
    return dict(name, op="gated", M=M, N=N, K=K, dtype=dtype, act=act, bias=bias, train=train)


def recurrence_case(T, S, C, dtype="bf16", kind="sigmoid", packed=False, train=False, **name):
    """T rows in S sequences: of T / S rows each, or (packed) of different lengths, some perhaps empty."""
    return dict(name, op="recurrence", T=T, S=S, C=C, dtype=dtype, kind=kind, packed=packed, train=train)


def listed():
    return [
        # one token's residual stream while serving: all latency
        norm_case(1, 2560, residual=True, name="norm-1-token"),
        # odd rows and channels of an fp32 model in training
        norm_case(333, 1001, dtype="f32", kind="rms", train=True, name="norm-f32-odd"),
        # 1024 requests x 16 positions in training, the largest batch of rows
        norm_case(16384, 5120, residual=True, train=True, name="norm-train-16384"),
        # one token's gate while serving: the weights are read once
        gated_case(1, 16384, 4096, name="gated-1-token"),
        # fp32 training of a small layer over one request's block
        gated_case(8, 256, 64, dtype="f32", act="gelu", bias=True, train=True, name="gated-f32-tiny"),
        # odd sizes in training: nothing is a multiple of a tile or of a 16-byte load
        gated_case(77, 1027, 1001, act="gelu", bias=True, train=True, name="gated-odd"),
        # a prompt of 2048 tokens
        gated_case(2048, 16384, 4096, name="gated-2048"),
        # 256 requests x 16 positions in training, the largest product
        gated_case(4096, 10240, 5120, train=True, name="gated-train-4096"),
        # one token of 256 requests while serving: the state goes one step on
        recurrence_case(256, 256, 2560, name="recurrence-step"),
        # the RNN head's state over 256 requests x 16 draft positions, in training
        recurrence_case(4096, 256, 256, kind="decay", train=True, name="recurrence-rnn-head"),
        # odd rows and channels of an fp32 model in training, three sequences
        recurrence_case(5003, 3, 1001, dtype="f32", packed=True, train=True, name="recurrence-f32-odd"),
        # a batch of 65536 tokens in a few long sequences in training
        recurrence_case(65536, 12, 2560, packed=True, train=True, name="recurrence-train-65536"),
    ]


def spread(rng, low, high):
    """A size between low and high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def rounded(rng, n, to):
    """n as it is (mostly odd), or on a multiple of `to`."""
    return n if n <= to or rng.random() < 0.4 else n // to * to


def draw(rng):
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    small = dtype == "f32"
    train = rng.random() < 0.6
    op = rng.choice(("norm", "gated", "recurrence"))
    if op == "norm":
        M = spread(rng, 1, 2048 if small else 16384)
        C = rounded(rng, spread(rng, 16, 5120), 64)
        return norm_case(M, C, dtype, rng.choice(("layer", "rms")), rng.random() < 0.5, train)
    if op == "gated":
        M = spread(rng, 1, 4096)
        most = 1 << (32 if small else 37)     # fp32 stays small
        K = rounded(rng, spread(rng, 16, 5120), 64)
        N = rounded(rng, min(spread(rng, 16, 16384), max(16, most // (M * K))), 64)
        # relu's step at zero is left out of training draws: a sum that rounds to the other side of zero is another gradient
        act = rng.choice([a for a in ACTS if a != "relu" or not train])
        return gated_case(M, N, K, dtype, act, rng.random() < 0.5, train)
    C = rounded(rng, spread(rng, 16, 5120), 64)
    T = spread(rng, 1, max(1, min(65536, (1 << (24 if small else 27)) // C)))
    S = spread(rng, 1, min(T, 512))
    packed = rng.random() < 0.6
    return recurrence_case(T if packed else T // S * S, S, C, dtype, rng.choice(("sigmoid", "decay")), packed, train)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, sd=1.0, mean=0.0, to=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * sd + mean).to(to)

    s = {"case": case}
    if case["op"] == "norm":
        M, C = case["M"], case["C"]
        # a residual stream: channels of different size and offset
        size = torch.exp(0.5 * torch.randn(C, generator=gen, device="cuda"))
        s["x"] = ((torch.randn((M, C), generator=gen, device="cuda") + 0.3) * size).to(dt)
        s["residual"] = normal(M, C, sd=3.0) if case["residual"] else None
        s["weight"] = normal(C, sd=0.2, mean=1.0)
        s["bias"] = normal(C, sd=0.2) if case["kind"] == "layer" else None
        s["dy"] = normal(M, C, sd=1.0 / M) if case["train"] else None
        # the stream's own gradient, past the normalisation
        s["dsum"] = normal(M, C, sd=1.0 / M) if case["train"] and case["residual"] else None
        return s
    if case["op"] == "gated":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = normal(M, K)
        s["wg"], s["wu"] = normal(N, K, sd=math.sqrt(2.0 / K)), normal(N, K, sd=math.sqrt(2.0 / K))
        s["bg"], s["bu"] = (normal(N, sd=0.5), normal(N, sd=0.5)) if case["bias"] else (None, None)
        s["dy"] = normal(M, N, sd=1.0 / M) if case["train"] else None
        return s
    T, S, C = case["T"], case["S"], case["C"]
    s["x"] = normal(T, C)
    s["h0"] = normal(S, C, to=torch.float32)
    if case["kind"] == "sigmoid":     # gates from 0.02 to 0.998: channels of short and of long memory
        s["gate"] = normal(T, C, sd=2.0, mean=2.0)
    else:
        s["gate"] = 0.5 + 0.499 * torch.rand(C, generator=gen, device="cuda")
    s["offsets"] = None
    if case["packed"]:
        cut = torch.randint(0, T + 1, (S - 1,), generator=gen, device="cuda", dtype=torch.int32).sort().values
        ends = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        s["offsets"] = torch.cat([ends[:1], cut, ends[1:]])
    s["dh"] = normal(T, C) if case["train"] else None
    s["dlast"] = normal(S, C, to=torch.float32) if case["train"] else None
    return s


def run(state):
    c = state["case"]
    return {"norm": run_norm, "gated": run_gated, "recurrence": run_recurrence}[c["op"]](state, c)


def run_norm(s, c):
    x, residual, weight, bias = s["x"], s["residual"], s["weight"], s["bias"]
    if own:
        from semi_ar_drafter_amd import norm, norm_backward
        stat = torch.empty((c["M"], 2), dtype=torch.float32, device=x.device) if c["train"] else None
        y = norm(x, weight, bias, residual=residual, eps=EPS, kind=c["kind"], stat=stat)
        y, total = y if c["residual"] else (y, x)
        out = {"y": y, "sum": total if c["residual"] else None}
        if c["train"]:
            out["dx"], out["dweight"], dbias = norm_backward(
                s["dy"], total, stat, weight, dsum=s["dsum"], kind=c["kind"],
                need=("dx", "dweight", "dbias") if bias is not None else ("dx", "dweight"))
            out["dbias"] = dbias
        return out
    total = (x.float() + residual.float()).to(x.dtype) if c["residual"] else x
    v = total.float()
    if c["kind"] == "layer":
        v = v - v.mean(1, keepdim=True)
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    v = v * rstd
    w = weight.float()
    y = v * w
    if bias is not None:
        y = y + bias.float()
    out = {"y": y.to(x.dtype), "sum": total if c["residual"] else None}
    if not c["train"]:
        return out
    dy = s["dy"].float()
    q = dy * w
    dx = q - v * (q * v).mean(1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - q.mean(1, keepdim=True)
    dx = dx * rstd
    if c["residual"]:
        dx = dx + s["dsum"].float()
    out["dx"] = dx.to(x.dtype)
    out["dweight"] = (dy * v).sum(0).to(x.dtype)
    out["dbias"] = dy.sum(0).to(x.dtype) if bias is not None else None
    return out


def run_gated(s, c):
    x, wg, wu, bg, bu = s["x"], s["wg"], s["wu"], s["bg"], s["bu"]
    if own:
        from semi_ar_drafter_amd import gated_linear, gated_linear_backward
        if not c["train"]:
            return gated_linear(x, wg, wu, bg=bg, bu=bu, act=c["act"])
        pre = torch.empty((2, c["M"], c["N"]), dtype=torch.float32, device=x.device)
        y = gated_linear(x, wg, wu, bg=bg, bu=bu, act=c["act"], pre=pre)
        names = ("dx", "dwg", "dwu", "dbg", "dbu")
        need = names if c["bias"] else names[:3]
        return dict(zip(("y",) + names, (y,) + tuple(gated_linear_backward(s["dy"], x, wg, wu, pre, act=c["act"], need=need))))
    xf, gf, uf = x.float(), wg.float(), wu.float()
    g, u = xf @ gf.t(), xf @ uf.t()
    if c["bias"]:
        g, u = g + bg.float(), u + bu.float()
    if c["act"] == "relu":
        a, slope = torch.clamp(g, min=0.0), (g > 0).float()
    elif c["act"] == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        a, slope = g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    elif c["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        a, slope = g * sig, sig * (1.0 + g * (1.0 - sig))
    else:
        a, slope = g, torch.ones_like(g)
    y = (a * u).to(x.dtype)
    if not c["train"]:
        return y
    dy = s["dy"].float()
    dg, du = dy * u * slope, dy * a
    return {"y": y, "dx": (dg @ gf + du @ uf).to(x.dtype), "dwg": (dg.t() @ xf).to(x.dtype), "dwu": (du.t() @ xf).to(x.dtype),
            "dbg": dg.sum(0).to(x.dtype) if c["bias"] else None, "dbu": du.sum(0).to(x.dtype) if c["bias"] else None}


def run_recurrence(s, c):
    x, gate, h0, offsets = s["x"], s["gate"], s["h0"], s["offsets"]
    T, S, C = c["T"], c["S"], c["C"]
    if own:
        from semi_ar_drafter_amd import RECURRENCE_BLOCK, recurrence, recurrence_backward
        last = torch.empty((S, C), dtype=torch.float32, device=x.device)
        states = torch.empty((-(-T // RECURRENCE_BLOCK), C), dtype=torch.float32, device=x.device) if c["train"] else None
        h = recurrence(x, gate, kind=c["kind"], offsets=offsets, h0=h0, last=last, states=states)
        out = {"h": h, "last": last}
        if c["train"]:
            out["dx"], out["dgate"], out["dh0"] = recurrence_backward(
                s["dh"], x, gate, states, kind=c["kind"], offsets=offsets, h0=h0, dlast=s["dlast"], need=("dx", "dgate", "dh0"))
        return out
    if offsets is None:
        offsets = torch.arange(0, T + 1, T // S, device=x.device)
    offsets = offsets.long()
    # a sequence's first and last row; an empty one adds nothing at the row that it names
    full = (offsets[1:] > offsets[:-1])
    first, end = offsets[:-1].clamp(max=T - 1), (offsets[1:] - 1).clamp(min=0)
    weight = full.float().unsqueeze(1)
    starts = torch.zeros((T, 1), device=x.device).index_add_(0, first, weight)
    ends = torch.zeros((T, 1), device=x.device).index_add_(0, end, weight)
    xf = x.float()
    if c["kind"] == "sigmoid":
        a = 1.0 / (1.0 + torch.exp(-gate.float()))
        b = xf / (1.0 + torch.exp(gate.float()))
    else:
        a = gate.unsqueeze(0).expand(T, C)
        b = xf
    h = scan(a * (1.0 - starts), b.index_add(0, first, a[first] * h0 * weight))
    out = {"h": h.to(x.dtype), "last": torch.where(full.unsqueeze(1), h[end], h0)}
    if not c["train"]:
        return out
    before = torch.cat([h[:1], h[:-1]]) * (1.0 - starts)      # the state that a row's gate multiplies
    before.index_add_(0, first, h0 * weight)
    del h
    dh = s["dh"].float().index_add_(0, end, s["dlast"] * weight) if x.dtype != torch.float32 else s["dh"].index_add(0, end, s["dlast"] * weight)
    after = torch.cat([a[1:], a[:1]]) * (1.0 - ends)
    d = scan(after.flip(0), dh.flip(0)).flip(0)
    if c["kind"] == "sigmoid":
        keep = 1.0 / (1.0 + torch.exp(gate.float()))           # 1 - a
        out["dx"], out["dgate"] = (d * keep).to(x.dtype), (d * (before - xf) * a * keep).to(x.dtype)
    else:
        out["dx"], out["dgate"] = d.to(x.dtype), (d * before).sum(0)
    out["dh0"] = torch.where(full.unsqueeze(1), (a * d)[first] if c["kind"] == "sigmoid" else a[first] * d[first], s["dlast"])
    return out


def scan(a, b):
    """h[t] = a[t] h[t - 1] + b[t] over the rows, doubling the distance."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["train"]
    if case["op"] == "norm":
        M, C, residual = case["M"], case["C"], case["residual"]
        vectors = 2 if case["kind"] == "layer" else 1
        # x, y and the stream's other part and sum; in training dy and dx, and the stream's gradient
        items = M * C * (2 + 2 * residual + (2 + residual) * train) + C * vectors * (1 + train)
        return {"bytes": items * e, "flops": M * C * (8 + 12 * train)}
    if case["op"] == "gated":
        M, N, K, bias = case["M"], case["N"], case["K"], case["bias"]
        items = M * K + 2 * N * K + M * N + 2 * N * bias
        if train:
            items += M * N + M * K + 2 * N * K + 2 * N * bias
        return {"bytes": items * e, "flops": 4 * M * N * K * (3 if train else 1)}
    T, S, C = case["T"], case["S"], case["C"]
    sigmoid = case["kind"] == "sigmoid"
    items = T * C * (2 + sigmoid + (2 + sigmoid) * train)      # x, gate, h; in training dh, dx and the gate's gradient
    vectors = 2 * S * C * (1 + train) + (0 if sigmoid else C * (1 + train))
    return {"bytes": items * e + 4 * vectors + 4 * (S + 1) * case["packed"], "flops": T * C * ((8 if sigmoid else 2) + (14 if sigmoid else 6) * train)}


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    return {"norm": exact_norm, "gated": exact_gated, "recurrence": exact_recurrence}[case["op"]](s, case)


def exact_norm(s, c):
    """The sum is rounded to its storage type before it is normalised: that is the operator's definition."""
    x64 = s["x"].double()
    total = x64 + s["residual"].double() if c["residual"] else x64
    out = {"y": None, "sum": total if c["residual"] else None}
    v = total.to(s["x"].dtype).double().requires_grad_(c["train"])
    w = s["weight"].double().requires_grad_(c["train"])
    b = s["bias"].double().requires_grad_(c["train"]) if s["bias"] is not None else None
    m = v.sum(1) / c["C"] if c["kind"] == "layer" else torch.zeros(c["M"], dtype=torch.float64, device=v.device)
    var = ((v - m[:, None]) ** 2).sum(1) / c["C"]
    y = torch.einsum("mc,m,c->mc", v - m[:, None], 1.0 / torch.sqrt(var + EPS), w)
    if b is not None:
        y = y + b[None, :]
    out["y"] = y.detach()
    if c["train"]:
        grads = torch.autograd.grad(y, [t for t in (v, w, b) if t is not None], s["dy"].double())
        out["dx"] = grads[0] + s["dsum"].double() if c["residual"] else grads[0]
        out["dweight"] = grads[1]
        out["dbias"] = grads[2] if b is not None else None
    return out


def exact_gated(s, c):
    M, N, K, train = c["M"], c["N"], c["K"], c["train"]
    f = {"none": lambda t: t + 0.0, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[c["act"]]
    weights = torch.cat([s["wg"], s["wu"]]).double()
    both = torch.cat([s["bg"], s["bu"]]).double() if c["bias"] else torch.zeros(2 * N, dtype=torch.float64, device="cuda")
    y = torch.empty((M, N), dtype=torch.float64, device="cuda")
    dx = torch.empty((M, K), dtype=torch.float64, device="cuda")
    dw, db = torch.zeros_like(weights), torch.zeros_like(both)
    for lo in range(0, M, 1024):
        rows = slice(lo, min(lo + 1024, M))
        x = s["x"][rows].double()
        pre = torch.addmm(both, x, weights.T).requires_grad_(train)
        out = f(pre[:, :N]) * pre[:, N:]
        y[rows] = out.detach()
        if train:
            (grad,) = torch.autograd.grad(out, pre, s["dy"][rows].double())
            dx[rows] = torch.mm(grad, weights)
            dw.addmm_(grad.T, x)
            db += grad.sum(0)
    if not train:
        return y
    return {"y": y, "dx": dx, "dwg": dw[:N], "dwu": dw[N:], "dbg": db[:N] if c["bias"] else None, "dbu": db[N:] if c["bias"] else None}


def exact_recurrence(s, c):
    """Row after row, there and back."""
    T, S, C, train = c["T"], c["S"], c["C"], c["train"]
    at = s["offsets"].tolist() if s["offsets"] is not None else list(range(0, T + 1, T // S))
    begins = {at[i]: i for i in range(S) if at[i + 1] > at[i]}
    finishes = {at[i + 1] - 1: i for i in range(S) if at[i + 1] > at[i]}
    x, h0 = s["x"].double(), s["h0"].double()
    sigmoid = c["kind"] == "sigmoid"
    if sigmoid:
        a = torch.sigmoid(s["gate"].double())
        b = torch.sigmoid(-s["gate"].double()) * x
    else:
        a = s["gate"].double().expand(T, C)
        b = x
    h, before = torch.empty_like(x), torch.empty_like(x) if train else None
    last = h0.clone()
    state = None
    for t in range(T):
        if t in begins:
            state = h0[begins[t]]
        if train:
            before[t] = state
        torch.addcmul(b[t], a[t], state, out=h[t])
        state = h[t]
        if t in finishes:
            last[finishes[t]] = state
    out = {"h": h, "last": last}
    if not train:
        return out
    d, dlast = s["dh"].double(), s["dlast"].double()
    dh0 = dlast.clone()
    for t in range(T - 1, -1, -1):
        if t in finishes:
            d[t] += dlast[finishes[t]]
        if t in begins:
            dh0[begins[t]] = a[t] * d[t]
        else:
            d[t - 1].addcmul_(a[t], d[t])
    if sigmoid:
        keep = torch.sigmoid(-s["gate"].double())
        out["dx"], out["dgate"] = d * keep, d * (before - x) * a * keep
    else:
        out["dx"], out["dgate"] = d, (d * before).sum(0)
    out["dh0"] = dh0
    return out
