"""What the tests of a backbone's layer (norm, gated_linear, recurrence) share."""
import torch

DEV = "cuda:0"
U32 = 2.0 ** -24                                             # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


def say(*a):
    print(*a, flush=True)


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(gen, *shape, sd=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device=DEV) * sd + mean).to(dtype)


def within(got, want, tol, what):
    assert got.shape == want.shape, what
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got "
                             f"{float(got.flatten()[i])}, want {float(want.flatten()[i])} within "
                             f"{float(tol.flatten()[i])}")


def guarded(shape, dtype, offset=0):
    """A tensor inside a larger one, `offset` elements behind its start, and a
    function that says whether the memory around it is as it was."""
    n = 1
    for s in shape:
        n *= s
    whole = torch.full((n + offset + 64,), 7.0, dtype=dtype, device=DEV)

    def untouched():
        return bool((whole[:offset] == 7).all() and (whole[offset + n:] == 7).all())

    return whole[offset:offset + n].view(shape), untouched


def replays(call, inputs, fresh, outputs):
    """Captures call() into a graph and replays it on changing inputs, with
    eager work in between: every replay equals the eager call.  fresh() gives
    new values for `inputs`, in order; outputs() the tensors call() wrote."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for turn in range(4):
        for t, v in zip(inputs, fresh()):
            t.copy_(v)
        eager = [t.clone() for t in outputs(call())]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outputs(held), eager):
            assert torch.equal(a, b), f"replay {turn}"
