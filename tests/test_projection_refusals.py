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


SIZES = {"linear": "M N K", "linear_backward": "M N K", "markov_loss": "N V d r", "markov_loss_backward": "N V d r",
         "hidden_draft": "B gamma V r d"}
# limits that are one too many
LIMITS = {"linear": dict(M=1 << 20, N=1 << 24, K=1 << 16), "linear_backward": dict(M=1 << 20, N=1 << 24, K=1 << 16),
          "markov_loss": dict(N=1 << 20, V=1 << 24, d=1 << 16, r=1 << 16),
          "markov_loss_backward": dict(N=1 << 20, V=1 << 24, d=1 << 16, r=1 << 16),
          "hidden_draft": dict(gamma=64, V=1 << 24, d=1 << 16)}


@pytest.mark.parametrize("entry", ENTRIES, ids=lambda e: e.name)
def test_sizes_types_and_limits(lib, entry):
    for k in SIZES[entry.name].split():
        refused(lib, entry, INVALID, "negative size", **{k: -1})
    for dt in (-1, 2, 99):
        refused(lib, entry, INVALID, "unknown dtype", dt=dt)
    if "act" in entry.values:
        for act in (-1, 4):
            refused(lib, entry, INVALID, "unknown activation", act=act)
    for k, most in LIMITS[entry.name].items():
        refused(lib, entry, UNSUPPORTED, f"{k} >" if k not in "dr" or entry is HIDDEN_DRAFT else "d or r >", **{k: most + 1})
    if entry is HIDDEN_DRAFT:
        refused(lib, entry, INVALID, "sampling mode", mode=2)
        refused(lib, entry, INVALID, "positive", V=0)
        refused(lib, entry, UNSUPPORTED, "B * gamma", B=1 << 15, gamma=64)
        refused(lib, entry, UNSUPPORTED, "supports r", r=48)
    elif "V" in entry.values:
        refused(lib, entry, INVALID, "V must be positive", V=0)


# arrays that may be left out
OPTIONAL = {"linear": "bias res pre", "linear_backward": "dx dw db", "markov_loss": "U",
            "markov_loss_backward": "dU dh dWo dW1 dW2", "hidden_draft": "bias"}


@pytest.mark.parametrize("entry", ENTRIES, ids=lambda e: e.name)
def test_arrays_that_are_missing(lib, entry):
    for k in entry.arrays:
        if k in OPTIONAL[entry.name].split():
            continue
        if k == "ws":
            refused(lib, entry, WORKSPACE, "workspace missing", ws=0)
        elif k in ("Wo", "W2") and entry in (LOSS, LOSS_BACKWARD):
            refused(lib, entry, INVALID, "go with d > 0", **{k: 0})
        elif k == "U" and entry is LOSS_BACKWARD:
            refused(lib, entry, INVALID, "gradient of an input that is not there", U=0)
        elif k == "Wo" and entry is HIDDEN_DRAFT:
            continue        # looked at after the draft's own checks, which end at the device
        else:
            refused(lib, entry, INVALID, "null pointer", **{k: 0})
    if entry in (LOSS, LOSS_BACKWARD):
        refused(lib, entry, INVALID, "go with d > 0", d=0)
        refused(lib, entry, INVALID, "go with d > 0", r=0)
        refused(lib, entry, INVALID, "no logits", U=0, d=0, h=0, Wo=0, r=0, prev=0, W1=0, W2=0)
    if entry is LOSS_BACKWARD:
        refused(lib, entry, INVALID, "gradient of an input", d=0, h=0, Wo=0)
        refused(lib, entry, INVALID, "gradient of an input", r=0, prev=0, W1=0, W2=0)


@pytest.mark.parametrize("entry", ENTRIES, ids=lambda e: e.name)
def test_arrays_that_are_not_aligned(lib, entry):
    """Operands of the products to 16 bytes, everything else to its element,
    the workspace to 256 bytes."""
    wide = {"linear": "x w", "linear_backward": "dy x w", "markov_loss": "h Wo W1 W2",
            "markov_loss_backward": "h Wo W1 W2", "hidden_draft": "W1"}[entry.name].split()
    narrow = {"linear": "bias res y pre", "linear_backward": "pre dx dw db", "markov_loss": "label prev U nll lse",
              "markov_loss_backward": "label prev U g lse dU dh dWo dW1 dW2", "hidden_draft": "U"}[entry.name].split()
    for k in wide:
        refused(lib, entry, INVALID, "16-byte", **{k: entry.values[k] + 8})
    for dt in (BF16, F32):
        fp32 = dict(r=16) if entry is HIDDEN_DRAFT else {}
        for k in narrow:
            refused(lib, entry, INVALID, "misaligned", dt=dt, **fp32, **{k: entry.values[k] + 1})
    for k in narrow:
        if k in ("U", "bias", "res", "y", "dx", "dw", "db", "dU", "dh", "dWo", "dW1", "dW2"):
            refused(lib, entry, INVALID, "misaligned", dt=F32, **(dict(r=16) if entry is HIDDEN_DRAFT else {}),
                    **{k: entry.values[k] + 2})
    refused(lib, entry, WORKSPACE, "256-byte", ws=entry.values["ws"] + 64)


@pytest.mark.parametrize("entry", ENTRIES, ids=lambda e: e.name)
def test_a_workspace_that_is_short(lib, entry):
    size = [entry.values[k] for k in ("B gamma V r d dt" if entry is HIDDEN_DRAFT else "M N K dt" if "M" in entry.values
                                      else "N V d r dt").split()]
    need = getattr(lib, f"dspark_{entry.name}_workspace_bytes")(*size)
    for n in (0, 255, need - 1):
        refused(lib, entry, WORKSPACE, "smaller than", n=n)


def test_no_gradient_asked_for_enqueues_nothing(lib):
    """Here, where there is no device, a launch would be an error."""
    assert LINEAR_BACKWARD(lib, dx=0, dw=0, db=0) == OK
    assert LOSS_BACKWARD(lib, dU=0, dh=0, dWo=0, dW1=0, dW2=0) == OK
    # the checks are made all the same
    refused(lib, LINEAR_BACKWARD, WORKSPACE, "missing", dx=0, dw=0, db=0, ws=0)
    refused(lib, LOSS_BACKWARD, INVALID, "null pointer", dU=0, dh=0, dWo=0, dW1=0, dW2=0, g=0)


def test_more_logits_than_a_launch_holds_are_refused(lib):
    far = {a: (1 << 50) + (i << 44) for i, a in enumerate(LOSS.arrays)}
    for N, V in ((1 << 20, 1 << 18), (1 << 14, 1 << 24), ((1 << 20) - 127, (1 << 18) - 127), (1 << 20, 1 << 24)):
        refused(lib, LOSS, UNSUPPORTED, "N * V", N=N, V=V, **far)
    # one tile fewer is past this check
    refused(lib, LOSS, WORKSPACE, "smaller", N=1 << 20, V=(1 << 18) - 128, **far)
    refused(lib, LOSS, WORKSPACE, "smaller", N=1 << 20, V=151936, **far)
    # the gradient goes piece by piece
    far = {a: (1 << 50) + (i << 44) for i, a in enumerate(LOSS_BACKWARD.arrays)}
    refused(lib, LOSS_BACKWARD, WORKSPACE, "smaller", N=1 << 20, V=1 << 18, **far)
