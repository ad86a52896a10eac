"""The projection's entry points (linear layer, heads' loss, their gradients,
drafting from hidden states) reject bad arguments on the host, before the GPU
is touched (CPU only: no call gets as far as a launch)."""
import ctypes
import os

import pytest

from semi_ar_drafter_amd import binding

OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = range(5)
P = ctypes.c_void_p(0x10000)        # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10008)     # 8-byte aligned only
NULL = ctypes.c_void_p(0)
BIG = ctypes.c_size_t(1 << 50)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from semi_ar_drafter_amd import build_lib
        build_lib.build(verbose=False)
    return binding.load()


def linear(lib, M=4, N=8, K=16, dt=1, x=P, w=P, bias=P, act=0, res=P, y=P, pre=P, ws=P, n=BIG):
    return lib.dspark_linear(M, N, K, dt, x, w, bias, act, res, y, pre, ws, n, NULL)


def linear_backward(lib, M=4, N=8, K=16, dt=1, dy=P, x=P, w=P, act=0, pre=P, dx=P, dw=P, db=P, ws=P, n=BIG):
    return lib.dspark_linear_backward(M, N, K, dt, dy, x, w, act, pre, dx, dw, db, ws, n, NULL)


def loss(lib, N=4, V=100, d=8, r=8, dt=1, label=P, U=P, h=P, Wo=P, prev=P, W1=P, W2=P, nll=P, lse=P, ws=P, n=BIG):
    return lib.dspark_markov_loss(N, V, d, r, dt, label, U, h, Wo, prev, W1, W2, nll, lse, ws, n, NULL)


def loss_backward(lib, N=4, V=100, d=8, r=8, dt=1, g=P, lse=P, label=P, U=P, h=P, Wo=P, prev=P, W1=P, W2=P, dU=P,
                  dh=P, dWo=P, dW1=P, dW2=P, ws=P, n=BIG):
    return lib.dspark_markov_loss_backward(N, V, d, r, dt, g, lse, label, U, h, Wo, prev, W1, W2, dU, dh, dWo, dW1,
                                           dW2, ws, n, NULL)


@pytest.mark.parametrize("call", [linear, linear_backward])
def test_linear_sizes_and_types(lib, call):
    for k in ("M", "N", "K"):
        assert call(lib, **{k: -1}) == INVALID
    assert call(lib, dt=2) == INVALID
    assert call(lib, act=4) == INVALID and call(lib, act=-1) == INVALID
    assert call(lib, M=(1 << 20) + 1) == UNSUPPORTED
    assert call(lib, N=(1 << 24) + 1) == UNSUPPORTED
    assert call(lib, K=65537) == UNSUPPORTED
    assert lib.dspark_last_error().decode()


def test_linear_pointers(lib):
    for k in ("x", "w", "y"):
        assert linear(lib, **{k: NULL}) == INVALID
    assert linear(lib, x=HALF) == INVALID and linear(lib, w=HALF) == INVALID
    for k in ("bias", "res", "y", "pre"):
        assert linear(lib, **{k: ODD}) == INVALID, k
    assert linear(lib, dt=0, bias=ctypes.c_void_p(0x10002)) == INVALID
    # empty batches are no-ops without any pointer
    none = dict(x=NULL, w=NULL, bias=NULL, res=NULL, y=NULL, pre=NULL, ws=NULL, n=ctypes.c_size_t(0))
    assert linear(lib, M=0, **none) == OK and linear(lib, N=0, **none) == OK


def test_linear_backward_pointers(lib):
    for k in ("dy", "x", "w"):
        assert linear_backward(lib, **{k: NULL}) == INVALID, k
        assert linear_backward(lib, **{k: HALF}) == INVALID, k
    assert linear_backward(lib, act=2, pre=NULL) == INVALID
    for k in ("dx", "dw", "db", "pre"):
        assert linear_backward(lib, **{k: ODD}) == INVALID, k
    need = lib.dspark_linear_backward_workspace_bytes(4, 8, 16, 1)
    assert need > 0 and need % 256 == 0
    assert linear_backward(lib, ws=NULL) == WORKSPACE
    assert linear_backward(lib, n=ctypes.c_size_t(need - 1)) == WORKSPACE
    assert linear_backward(lib, ws=ctypes.c_void_p(0x10040)) == WORKSPACE


@pytest.mark.parametrize("call", [loss, loss_backward])
def test_loss_arguments(lib, call):
    for k in ("N", "V", "d", "r"):
        assert call(lib, **{k: -1}) == INVALID
    assert call(lib, V=0) == INVALID
    assert call(lib, dt=5) == INVALID
    for k in ("label", "h", "Wo", "prev", "W1", "W2"):
        assert call(lib, **{k: NULL}) == INVALID, k
    for k in ("h", "Wo", "W1", "W2"):
        assert call(lib, **{k: HALF}) == INVALID, k
    for k in ("label", "prev", "U"):
        assert call(lib, **{k: ODD}) == INVALID, k
    assert call(lib, d=0) == INVALID and call(lib, r=0) == INVALID     # operands without a size
    gone = dict(d=0, h=NULL, Wo=NULL, r=0, prev=NULL, W1=NULL, W2=NULL)
    assert call(lib, U=NULL, **gone) == INVALID                        # no logits at all
    assert call(lib, N=(1 << 20) + 1) == UNSUPPORTED
    assert call(lib, V=(1 << 24) + 1) == UNSUPPORTED
    assert call(lib, d=65537) == UNSUPPORTED and call(lib, r=65537) == UNSUPPORTED
    assert call(lib, ws=NULL) == WORKSPACE
    assert call(lib, ws=ctypes.c_void_p(0x10040)) == WORKSPACE
    assert call(lib, n=ctypes.c_size_t(255)) == WORKSPACE
    assert lib.dspark_last_error().decode()


def test_loss_outputs(lib):
    assert loss(lib, nll=NULL) == INVALID and loss(lib, lse=NULL) == INVALID
    assert loss(lib, nll=ODD) == INVALID
    none = {k: NULL for k in ("label", "U", "h", "Wo", "prev", "W1", "W2", "nll", "lse", "ws")}
    assert loss(lib, N=0, d=0, r=0, **none, n=ctypes.c_size_t(0)) == OK


def test_loss_backward_outputs(lib):
    assert loss_backward(lib, g=NULL) == INVALID and loss_backward(lib, lse=NULL) == INVALID
    for k in ("dU", "dh", "dWo", "dW1", "dW2", "g", "lse"):
        assert loss_backward(lib, **{k: ODD}) == INVALID, k
    assert loss_backward(lib, U=NULL) == INVALID                       # dU without U
    assert loss_backward(lib, d=0, h=NULL, Wo=NULL) == INVALID         # dh, dWo without them
    assert loss_backward(lib, r=0, prev=NULL, W1=NULL, W2=NULL) == INVALID


def test_workspace_sizes(lib):
    assert lib.dspark_linear_workspace_bytes(0, 8, 8, 1) == 0
    assert lib.dspark_linear_workspace_bytes(8, 8, 8, 7) == 0
    assert lib.dspark_linear_backward_workspace_bytes(-1, 8, 8, 1) == 0
    assert lib.dspark_markov_loss_workspace_bytes(0, 100, 8, 8, 1) == 0
    assert lib.dspark_markov_loss_workspace_bytes(4, 0, 8, 8, 1) == 0
    assert lib.dspark_markov_loss_backward_workspace_bytes(4, 100, 65537, 8, 1) == 0
    for f in (lib.dspark_markov_loss_workspace_bytes, lib.dspark_markov_loss_backward_workspace_bytes):
        assert f(8, 1024, 64, 16, 0) % 256 == 0 and f(8, 1024, 64, 16, 0) > 0
    # the gradients of no rows at all still need a (small) workspace
    assert 0 < lib.dspark_markov_loss_backward_workspace_bytes(0, 1024, 64, 16, 1) < 1 << 24
    # nothing as large as the logits: 4096 rows over 151936 tokens would be 1.2e9 (bf16) or 2.5e9 bytes (fp32)
    assert lib.dspark_markov_loss_workspace_bytes(4096, 151936, 5120, 256, 1) < 2 ** 27
    assert lib.dspark_markov_loss_backward_workspace_bytes(4096, 151936, 5120, 256, 1) < 9 * 10 ** 8
    # sizes at the limits do not wrap
    assert lib.dspark_markov_loss_backward_workspace_bytes(1 << 20, 1 << 24, 65536, 65536, 1) > 1 << 38


def test_hidden_draft_validation(lib):
    need = lib.dspark_hidden_draft_workspace_bytes(4, 4, 1024, 32, 16, 1)
    assert need >= lib.dspark_draft_workspace_bytes(4, 4, 1024, 32)

    def call(B=4, g=4, V=1024, r=32, d=16, dt=1, mode=0, ws=P, n=need, **over):
        p = {k: P for k in ("anchor", "h", "Wo", "bias", "W1", "W2", "conf_w", "sts_T", "U", "tokens", "logit", "conf",
                            "surv")}
        p.update(over)
        return lib.dspark_hidden_draft(B, g, V, r, d, dt, p["anchor"], p["h"], p["Wo"], p["bias"], p["W1"], p["W2"],
                                       p["conf_w"], ctypes.c_float(1.0), p["sts_T"], mode, ctypes.c_uint64(0), p["U"],
                                       p["tokens"], p["logit"], p["conf"], p["surv"], ws, ctypes.c_size_t(n), NULL)

    assert call(B=-1) == INVALID and call(V=-1) == INVALID and call(dt=3) == INVALID and call(mode=9) == INVALID
    for k in ("anchor", "h", "W1", "W2", "conf_w", "sts_T", "U", "tokens", "logit", "conf", "surv"):
        assert call(**{k: NULL}) == INVALID, k
    assert call(g=65) == UNSUPPORTED
    assert call(r=48) == UNSUPPORTED
    assert call(B=1 << 15, g=64) == UNSUPPORTED
    assert call(ws=NULL) == WORKSPACE and call(n=100) == WORKSPACE
    assert call(ws=ctypes.c_void_p(0x10040)) == WORKSPACE
    assert call(B=0, anchor=NULL, U=NULL, ws=NULL, n=0) == OK
    assert lib.dspark_hidden_draft_workspace_bytes(0, 4, 1024, 32, 16, 1) == 0


def test_overlapping_outputs_are_refused(lib):
    """Every array at an address of its own is past this check; each output
    moved onto (or into) an input, or onto another output, is not.  Only
    calls that fail are made."""
    at = lambda i, off=0: ctypes.c_void_p(0x100000 * (i + 1) + off)  # noqa: E731
    lin = dict(x=at(0), w=at(1), bias=at(2), res=at(3), y=at(4), pre=at(5), ws=at(6))
    for out in ("y", "pre"):
        for other in ("x", "w", "bias"):
            assert linear(lib, **{**lin, out: lin[other]}) == INVALID, (out, other)
    assert linear(lib, **{**lin, "y": lin["pre"]}) == INVALID
    assert linear(lib, **{**lin, "y": at(0, 16)}) == INVALID             # inside x
    assert linear(lib, **{**lin, "y": at(3, 2)}) == INVALID              # the residual, shifted
    back = dict(dy=at(0), x=at(1), w=at(2), pre=at(3), dx=at(4), dw=at(5), db=at(6), ws=at(7))
    for out in ("dx", "dw", "db"):
        for other in ("dy", "x", "w", "pre"):
            assert linear_backward(lib, **{**back, "act": 2, out: back[other]}) == INVALID, (out, other)
    assert linear_backward(lib, **{**back, "dx": back["dw"]}) == INVALID
    ins = {k: at(i) for i, k in enumerate(("label", "U", "h", "Wo", "prev", "W1", "W2"))}
    assert loss(lib, **ins, nll=at(8), lse=at(8), ws=at(9)) == INVALID
    outs = {k: at(10 + i) for i, k in enumerate(("dU", "dh", "dWo", "dW1", "dW2"))}
    rest = dict(g=at(20), lse=at(21), ws=at(22))
    for out in outs:
        for other in ("U", "h", "Wo", "W1", "W2"):
            assert loss_backward(lib, **{**ins, **outs, **rest, out: ins[other]}) == INVALID, (out, other)
    assert loss_backward(lib, **{**ins, **outs, **rest, "dW1": outs["dWo"]}) == INVALID
    assert "overlaps" in lib.dspark_last_error().decode()
