"""Refusals of the projection's entry points, each for its own reason: every
array has an address of its own, so that a call is refused for what the test
changes and for nothing else (CPU only: no call gets as far as a launch)."""
import ctypes
import os

import pytest

from semi_ar_drafter_amd import binding

OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = range(5)
STEP = 1 << 24          # between the arrays' addresses, which are never dereferenced
BIG = 1 << 22           # workspace bytes: enough for every shape here
F32, BF16 = 0, 1


class Entry:
    """One entry point: its arguments in order, sizes and options with their
    values, arrays (named in `arrays`) at addresses of their own."""

    def __init__(self, name, order, arrays, **values):
        self.name, self.order = name, order.split()
        self.values = dict(values, stream=0, n=BIG)
        for i, a in enumerate(arrays.split()):
            self.values[a] = STEP * (i + 1)
        self.arrays = arrays.split()

    def __call__(self, lib, **over):
        assert set(over) <= set(self.values), over
        v = {**self.values, **over}
        f = getattr(lib, "dspark_" + self.name)
        args = [t(v[k]) if t is not ctypes.c_void_p else ctypes.c_void_p(v[k]) for k, t in zip(self.order, f.argtypes)]
        return f(*args)


LINEAR = Entry("linear", "M N K dt x w bias act res y pre ws n stream", "x w bias res y pre ws",
               M=70, N=130, K=1000, dt=BF16, act=0)      # a product that needs a workspace
LINEAR_BACKWARD = Entry("linear_backward", "M N K dt dy x w act pre dx dw db ws n stream",
                        "dy x w pre dx dw db ws", M=4, N=8, K=16, dt=BF16, act=2)
LOSS = Entry("markov_loss", "N V d r dt label U h Wo prev W1 W2 nll lse ws n stream",
             "label U h Wo prev W1 W2 nll lse ws", N=4, V=100, d=8, r=8, dt=BF16)
LOSS_BACKWARD = Entry("markov_loss_backward",
                      "N V d r dt g lse label U h Wo prev W1 W2 dU dh dWo dW1 dW2 ws n stream",
                      "g lse label U h Wo prev W1 W2 dU dh dWo dW1 dW2 ws", N=4, V=100, d=8, r=8, dt=BF16)
HIDDEN_DRAFT = Entry("hidden_draft",
                     "B gamma V r d dt anchor h Wo bias W1 W2 conf_w conf_b sts_T mode seed U tokens logit conf surv ws n "
                     "stream", "anchor h Wo bias W1 W2 conf_w sts_T U tokens logit conf surv ws",
                     B=4, gamma=4, V=1024, r=32, d=16, dt=BF16, conf_b=1.0, mode=0, seed=0)
OUTPUTS = {"linear": "y pre", "linear_backward": "dx dw db", "markov_loss": "nll lse",
           "markov_loss_backward": "dU dh dWo dW1 dW2", "hidden_draft": "U tokens logit conf surv"}
ENTRIES = [LINEAR, LINEAR_BACKWARD, LOSS, LOSS_BACKWARD, HIDDEN_DRAFT]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from semi_ar_drafter_amd import build_lib
        build_lib.build(verbose=False)
    return binding.load()


def refused(lib, entry, status, why, **over):
    assert entry(lib, **over) == status, (entry.name, over)
    assert why in lib.dspark_last_error().decode(), (entry.name, over, lib.dspark_last_error())


@pytest.mark.parametrize("entry", ENTRIES, ids=lambda e: e.name)
def test_every_output_that_overlaps_is_refused(lib, entry):
    """Each output, and the workspace, on another array, and each array inside
    the workspace."""
    outputs = OUTPUTS[entry.name].split() + ["ws"]
    for out in outputs:
        for other in entry.arrays:
            if other == out or (entry is LINEAR and (out, other) in (("y", "res"), ("res", "y"))):
                continue
            refused(lib, entry, INVALID, "overlaps", **{out: entry.values[other]})
    if entry is LINEAR:     # the residual in place is allowed, beside it is not
        refused(lib, entry, INVALID, "overlaps", y=entry.values["res"] + 2)
    size = [entry.values[k] for k in ("B gamma V r d dt" if entry is HIDDEN_DRAFT else "M N K dt" if "M" in entry.values
                                      else "N V d r dt").split()]
    need = getattr(lib, f"dspark_{entry.name}_workspace_bytes")(*size)
    assert 256 < need <= BIG
    for other in entry.arrays[:-1]:
        refused(lib, entry, INVALID, "overlaps", **{other: entry.values["ws"] + (need - 16) // 256 * 256})


def test_workspace_of_a_gradient_without_activation(lib):
    """dz = dy takes no memory of its own where dy can be read as it is: the
    output projection's gradient asks for little more than its bias sums."""
    act = lib.dspark_linear_backward_act_workspace_bytes
    for dt, elem in ((F32, 4), (BF16, 2)):
        M, N, K = 4096, 151936, 2560
        copy = M * N * elem
        assert act(M, N, K, dt, 0) < copy // 2
        for a in (1, 2, 3):
            assert act(M, N, K, dt, a) == act(M, N, K, dt, 0) + copy
        for size in ((M, N, K), (77, 1027, 1001), (1, 1, 1), (64, 128, 0), (0, 300, 9)):
            assert lib.dspark_linear_backward_workspace_bytes(*size, dt) == act(*size, dt, 1) >= act(*size, dt, 0)
    # sizes that are no whole steps are copied for bf16, not for fp32
    assert act(77, 1027, 1001, BF16, 0) == act(77, 1027, 1001, BF16, 2)
    assert act(77, 1027, 1001, F32, 0) < act(77, 1027, 1001, F32, 2)
    assert act(4, 8, 16, 7, 0) == act(-1, 8, 16, BF16, 0) == 0
    need = act(64, 128, 64, BF16, 0)
    refused(lib, LINEAR_BACKWARD, WORKSPACE, "smaller", M=64, N=128, K=64, act=0, n=need - 1)
    refused(lib, LINEAR_BACKWARD, WORKSPACE, "smaller", M=64, N=128, K=64, act=2, n=need)
