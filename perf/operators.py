"""Measured cases of the vocabulary projection: ``linear`` (a matrix product
with bias, activation and residual) and ``markov_loss`` (softmax cross entropy
over the drafting heads' logits), forward and backward.

Shapes are those of the package's workloads: vocabularies 151936, 129280 and
1024, hidden sizes 2560 to 7168, Markov rank 256 (16 for the fp32 one),
requests x draft positions as rows.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def linear_case(M, N, K, dtype="bf16", act="none", bias=True, residual=False, train=False, **name):
    return dict(name, op="linear", M=M, N=N, K=K, dtype=dtype, act=act, bias=bias, residual=residual, train=train)


def loss_case(N, V, d, r, dtype="bf16", base=False, ignored=0, train=False, frozen=False, **name):
    """base: base logits U are given; ignored: rows without a label; frozen: no gradient for the output projection."""
    return dict(name, op="loss", N=N, V=V, d=d, r=r, dtype=dtype, base=base, ignored=ignored, train=train, frozen=frozen)


def listed():
    return [
        # fp32 layer over one small request's block: all latency
        linear_case(8, 1024, 64, dtype="f32", act="silu", residual=True, name="linear-f32-tiny"),
        # one token through a square backbone projection while serving
        linear_case(1, 4096, 4096, residual=True, name="linear-1-token"),
        # base logits of one request's eight draft positions: the projection's weights are read once
        linear_case(8, 151936, 2560, bias=False, name="linear-logits-8"),
        # odd sizes: nothing is a multiple of a tile or of a 16-byte load
        linear_case(77, 1027, 1001, act="relu", residual=True, name="linear-odd"),
        # base logits of 64 requests x 16 positions
        linear_case(1024, 151936, 4096, bias=False, name="linear-logits-1024"),
        # a backbone layer in training, 256 x 16 positions
        linear_case(4096, 5120, 5120, act="gelu", residual=True, train=True, name="linear-train"),
        # fp32 training of the small head
        loss_case(8, 1024, 64, 16, dtype="f32", ignored=1, train=True, name="loss-f32-tiny"),
        # scoring one request's block
        loss_case(8, 151936, 2560, 256, name="loss-score-8"),
        # evaluation over a batch, a fifth of its positions past the end of their sequences
        loss_case(1024, 129280, 4096, 256, ignored=205, name="loss-score-1024"),
        # odd rows, vocabulary, hidden size and rank, in training
        loss_case(333, 50021, 1000, 40, ignored=33, train=True, name="loss-train-odd"),
        # the Markov head alone on given base logits of a frozen backbone, 256 x 16 positions
        loss_case(4096, 151936, 0, 256, base=True, ignored=256, train=True, name="loss-train-markov"),
        # the whole projection trained, 256 x 16 positions
        loss_case(4096, 151936, 5120, 256, ignored=256, train=True, name="loss-train-4096"),
    ]


def spread(rng, low, high):
    """A size between low and high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def rounded(rng, n, to):
    """n as it is (mostly odd), or on a multiple of `to`."""
    return n if n <= to or rng.random() < 0.4 else n // to * to


def draw(rng):
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    train = rng.random() < 0.5
    if rng.random() < 0.5:
        M = spread(rng, 1, 4096)
        most = 1 << 33 if dtype == "bf16" else 1 << 30     # weights x rows, so that fp32 stays small
        K = rounded(rng, spread(rng, 16, 7168), 64)
        N = rounded(rng, min(spread(rng, 16, 151936), max(16, most // (M * K) * 64)), 64)
        # relu's step at zero is left out of training draws: a sum that rounds to the other side of zero is another gradient
        act = rng.choice([a for a in ACTS if a != "relu" or not train])
        return linear_case(M, N, K, dtype, act, rng.random() < 0.5, rng.random() < 0.5, train)
    N = spread(rng, 1, 4096 if dtype == "bf16" else 512)
    V = rounded(rng, spread(rng, 1000, 151936 if dtype == "bf16" else 30000), 64)
    d = rounded(rng, spread(rng, 16, 5120 if dtype == "bf16" else 1024), 64)
    r = rounded(rng, spread(rng, 8, 256), 8)
    base = rng.random() < 0.3
    return loss_case(N, V, 0 if base and rng.random() < 0.5 else d, r, dtype, base, rng.randrange(N // 4 + 1), train, rng.random() < 0.4)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, sd=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * sd).to(dt)

    s = {"case": case}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = normal(M, K)
        s["w"] = normal(N, K, sd=math.sqrt(2.0 / K))          # outputs of variance 2, as the base logits have
        s["bias"] = normal(N, sd=0.5) if case["bias"] else None
        s["residual"] = normal(M, N) if case["residual"] else None
        s["dy"] = normal(M, N, sd=1.0 / M) if case["train"] else None
        return s
    N, V, d, r = case["N"], case["V"], case["d"], case["r"]
    # tokens as text has them: few frequent, many rare, so that rows share previous tokens
    token = (V * torch.rand(N, generator=gen, device="cuda") ** 4).to(torch.int64).clamp(max=V - 1)
    label = (V * torch.rand(N, generator=gen, device="cuda") ** 2).to(torch.int64).clamp(max=V - 1)
    s["prev"] = token.to(torch.int32)
    s["W1"] = normal(V, r, sd=r ** -0.25)
    s["W2"] = normal(r, V, sd=r ** -0.25)                     # one Markov bias has unit variance
    s["U"] = s["h"] = s["Wo"] = None
    if d:
        s["Wo"] = normal(V, d, sd=math.sqrt(2.0 / d))
        # a hidden state that has learnt something: its label's logit is raised by 8
        s["h"] = (torch.randn((N, d), generator=gen, device="cuda") + 4.0 * s["Wo"][label].float()).to(dt)
    if case["base"]:
        s["U"] = normal(N, V, sd=math.sqrt(2.0))
        if not d:
            s["U"][torch.arange(N, device="cuda"), label] += 8.0
    drop = torch.randperm(N, generator=gen, device="cuda")[:case["ignored"]]
    label[drop] = -1
    s["label"] = label.to(torch.int32)
    # position-weighted mean: weights fall over the 16 positions of a block
    weight = 0.9 ** (torch.arange(N, device="cuda") % 16).float()
    s["g"] = weight / weight.sum()
    return s


def run(state):
    c = state["case"]
    if c["op"] == "linear":
        return run_linear(state, c)
    return run_loss(state, c)


def run_linear(s, c):
    x, w, bias, residual = s["x"], s["w"], s["bias"], s["residual"]
    if own:
        from semi_ar_drafter_amd import linear, linear_backward
        if not c["train"]:
            return linear(x, w, bias=bias, act=c["act"], residual=residual)
        pre = torch.empty((c["M"], c["N"]), dtype=torch.float32, device=x.device) if c["act"] != "none" else None
        y = linear(x, w, bias=bias, act=c["act"], residual=residual, pre=pre)
        dx, dw, dbias = linear_backward(s["dy"], x, w, act=c["act"], pre=pre, need=("dx", "dw", "dbias") if c["bias"] else ("dx", "dw"))
        return {"y": y, "dx": dx, "dw": dw, "dbias": dbias}
    xf, wf = x.float(), w.float()
    z = xf @ wf.t()
    if bias is not None:
        z = z + bias.float()
    if c["act"] == "relu":
        y = torch.clamp(z, min=0.0)
    elif c["act"] == "gelu":
        y = z * 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
    elif c["act"] == "silu":
        y = z * torch.sigmoid(z)
    else:
        y = z
    if residual is not None:
        y = y + residual.float()
    y = y.to(x.dtype)
    if not c["train"]:
        return y
    dz = s["dy"].float()
    if c["act"] == "relu":
        dz = torch.where(z > 0, dz, torch.zeros_like(dz))
    elif c["act"] == "gelu":
        dz = dz * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    elif c["act"] == "silu":
        sig = torch.sigmoid(z)
        dz = dz * sig * (1.0 + z * (1.0 - sig))
    return {"y": y, "dx": (dz @ wf).to(x.dtype), "dw": (dz.t() @ xf).to(x.dtype),
            "dbias": dz.sum(0).to(x.dtype) if bias is not None else None}


def run_loss(s, c):
    inputs = dict(U=s["U"], h=s["h"], Wo=s["Wo"], prev=s["prev"], W1=s["W1"], W2=s["W2"])
    if own:
        from semi_ar_drafter_amd import markov_loss, markov_loss_backward
        nll, lse = markov_loss(s["label"], **inputs)
        out = {"nll": nll, "lse": lse}
        if c["train"]:
            need = ["dW1", "dW2"] + (["dU"] if c["base"] and not c["frozen"] and not c["d"] else [])
            need += (["dh"] if c["frozen"] else ["dh", "dWo"]) if c["d"] else []
            out.update(markov_loss_backward(s["g"], lse, s["label"], need=need, **inputs))
        return out
    label, prev, dt = s["label"].long(), s["prev"].long(), s["W1"].dtype
    kept = label >= 0
    W2 = s["W2"].float()
    E = s["W1"][prev].float()
    z = E @ W2
    if c["d"]:
        h, Wo = s["h"].float(), s["Wo"].float()
        z += h @ Wo.t()
    if c["base"]:
        z += s["U"].float()
    top = z.max(1, keepdim=True).values
    p = torch.exp(z - top)
    total = p.sum(1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(1)
    at = label.clamp(min=0).unsqueeze(1)
    nll = lse - z.gather(1, at).squeeze(1)
    zero = torch.zeros_like(lse)
    out = {"nll": torch.where(kept, nll, zero), "lse": torch.where(kept, lse, zero)}
    if not c["train"]:
        return out
    del z
    p /= total
    p[torch.arange(c["N"], device=p.device), at.squeeze(1)] -= 1.0
    p *= torch.where(kept, s["g"], zero).unsqueeze(1)
    out["dW2"] = (E.t() @ p).to(dt)
    dE = p @ W2.t()
    out["dW1"] = torch.zeros(s["W1"].shape, device=p.device).index_add_(0, prev, dE).to(dt)
    if c["base"] and not c["frozen"] and not c["d"]:
        out["dU"] = p.to(dt)
    if c["d"]:
        out["dh"] = (p @ Wo).to(dt)
        if not c["frozen"]:
            out["dWo"] = (p.t() @ h).to(dt)
    return out


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        items = M * K + N * K + M * N + N * case["bias"] + M * N * case["residual"]
        if case["train"]:
            items += M * N + M * K + N * K + N * case["bias"]
        return {"bytes": items * e, "flops": 2 * M * N * K * (3 if case["train"] else 1)}
    N, V, d, r = case["N"], case["V"], case["d"], case["r"]
    rows = N - case["ignored"]
    items = rows * d + V * d + rows * r + r * V + (rows * V if case["base"] else 0)
    flops = 2 * rows * V * (d + r)
    if case["train"]:
        items += N * d + V * d * (not case["frozen"]) + 2 * V * r
        items += N * V * (case["base"] and not case["frozen"] and not d)
        flops += 2 * rows * V * (d + 2 * r + d * (not case["frozen"]))
    return {"bytes": items * e + 8 * N + 4 * N * (2 + case["train"]), "flops": flops}


def exact(case, seed):
    """The definitions in 64 bits, a block of rows at a time."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        return exact_linear(s, case)
    return exact_loss(s, case)


def exact_linear(s, c):
    w = s["w"].double()
    y = torch.empty((c["M"], c["N"]), dtype=torch.float64, device="cuda")
    out = {"y": y, "dx": torch.empty((c["M"], c["K"]), dtype=torch.float64, device="cuda"),
           "dw": torch.zeros((c["N"], c["K"]), dtype=torch.float64, device="cuda"),
           "dbias": torch.zeros(c["N"], dtype=torch.float64, device="cuda") if c["bias"] else None}
    for lo in range(0, c["M"], 1024):
        rows = slice(lo, min(lo + 1024, c["M"]))
        x = s["x"][rows].double()
        pre = torch.mm(x, w.T)
        if c["bias"]:
            pre += s["bias"].double()[None, :]
        pre.requires_grad_(c["train"])
        a = {"none": lambda t: t + 0.0, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[c["act"]](pre)
        y[rows] = a.detach() + (s["residual"][rows].double() if c["residual"] else 0.0)
        if c["train"]:
            (grad,) = torch.autograd.grad(a, pre, s["dy"][rows].double())
            out["dx"][rows] = torch.mm(grad, w)
            out["dw"] += torch.mm(grad.T, x)
            if c["bias"]:
                out["dbias"] += grad.sum(0)
    return out if c["train"] else y


def exact_loss(s, c):
    N, V, d, r, train = c["N"], c["V"], c["d"], c["r"], c["train"]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"nll": new(N), "lse": new(N)}
    W2, Wo = s["W2"].double(), s["Wo"].double() if d else None
    with_dU = c["base"] and not c["frozen"] and not d
    if train:
        out.update(dW1=new(V, r), dW2=new(r, V))
        if d:
            out["dh"] = new(N, d)
            if not c["frozen"]:
                out["dWo"] = new(V, d)
        if with_dU:
            out["dU"] = new(N, V)
    used = torch.nonzero(s["label"] >= 0).flatten()
    for idx in torch.split(used, 512):
        if not idx.numel():
            continue
        y, t = s["label"][idx].long(), s["prev"][idx].long()
        e = s["W1"][t].double()
        logits = torch.mm(e, W2)
        if d:
            x = s["h"][idx].double()
            logits.addmm_(x, Wo.T)
        if c["base"]:
            logits += s["U"][idx].double()
        lse = torch.logsumexp(logits, 1)
        out["lse"][idx] = lse
        out["nll"][idx] = lse - logits[torch.arange(len(idx), device="cuda"), y]
        if not train:
            continue
        grad = torch.exp(logits - lse[:, None])
        grad.scatter_add_(1, y[:, None], torch.full((len(idx), 1), -1.0, dtype=torch.float64, device="cuda"))
        grad *= s["g"][idx].double()[:, None]
        out["dW2"].addmm_(e.T, grad)
        out["dW1"].index_add_(0, t, torch.mm(grad, W2.T))
        if d:
            out["dh"][idx] = torch.mm(grad, Wo)
            if not c["frozen"]:
                out["dWo"].addmm_(grad.T, x)
        if with_dU:
            out["dU"][idx] = grad
    return out
