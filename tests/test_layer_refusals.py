"""Refusals of norm, recurrence and gated_linear and of their gradients, each
for its own reason: every array has an address of its own, so that a call is
refused for what the test changes and for nothing else (CPU only: no call gets
as far as a launch)."""
import os

import pytest

from semi_ar_drafter_amd import binding

from test_projection_refusals import BF16, F32, INVALID, OK, UNSUPPORTED, WORKSPACE, Entry, refused

NAN = float("nan")
NORM = Entry("norm", "M C dt kind x residual w b eps sum y stat stream", "x residual w b sum y stat",
             M=4, C=64, dt=BF16, kind=0, eps=1e-5)
NORM_BACKWARD = Entry("norm_backward", "M C dt kind dy x stat w dsum dx dw db ws n stream",
                      "dy x stat w dsum dx dw db ws", M=1000, C=64, dt=BF16, kind=0)
RECURRENCE = Entry("recurrence", "T S C dt kind offsets x gate h0 h last states ws n stream",
                   "offsets x gate h0 h last states ws", T=600, S=2, C=20, dt=BF16, kind=0)
RECURRENCE_BACKWARD = Entry("recurrence_backward",
                            "T S C dt kind offsets dh x gate h0 dlast states dx dgate dh0 ws n stream",
                            "offsets dh x gate h0 dlast states dx dgate dh0 ws", T=600, S=2, C=20, dt=BF16, kind=0)
GATED = Entry("gated_linear", "M N K dt x wg wu bg bu act y pre ws n stream", "x wg wu bg bu y pre ws",
              M=70, N=65, K=1000, dt=BF16, act=3)
GATED_BACKWARD = Entry("gated_linear_backward", "M N K dt dy x wg wu act pre dx dwg dwu dbg dbu ws n stream",
                       "dy x wg wu pre dx dwg dwu dbg dbu ws", M=4, N=8, K=16, dt=BF16, act=3)
ENTRIES = [NORM, NORM_BACKWARD, RECURRENCE, RECURRENCE_BACKWARD, GATED, GATED_BACKWARD]
OUTPUTS = {"norm": "sum y stat", "norm_backward": "dx dw db ws", "recurrence": "h last states ws",
           "recurrence_backward": "dx dgate dh0 ws", "gated_linear": "y pre ws",
           "gated_linear_backward": "dx dwg dwu dbg dbu ws"}
# an output in the place of an input that the call allows
IN_PLACE = {("norm", "sum", "x"), ("norm", "sum", "residual"), ("norm_backward", "dx", "dsum"),
            ("recurrence", "last", "h0"), ("recurrence_backward", "dh0", "dlast")}
SIZES = {"norm": "M C", "norm_backward": "M C", "recurrence": "T S C", "recurrence_backward": "T S C",
         "gated_linear": "M N K", "gated_linear_backward": "M N K"}
IDS = [e.name for e in ENTRIES]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from semi_ar_drafter_amd import build_lib
        build_lib.build(verbose=False)
    return binding.load()


@pytest.mark.parametrize("entry", ENTRIES, ids=IDS)
def test_every_output_that_overlaps_is_refused(lib, entry):
    for out in OUTPUTS[entry.name].split():
        for other in entry.arrays:
            if other == out or (entry.name, out, other) in IN_PLACE or (entry.name, other, out) in IN_PLACE:
                continue
            refused(lib, entry, INVALID, "overlaps", **{out: entry.values[other]})
    for name, out, other in IN_PLACE:      # beside its place it is refused
        if name == entry.name:
            refused(lib, entry, INVALID, "overlaps", **{out: entry.values[other] + 8})


@pytest.mark.parametrize("entry", ENTRIES, ids=IDS)
def test_sizes_and_options(lib, entry):
    for k in SIZES[entry.name].split():
        refused(lib, entry, INVALID, "negative size", **{k: -1})
    refused(lib, entry, INVALID, "dtype", dt=2)
    refused(lib, entry, INVALID, "dtype", dt=-1)
    if "kind" in entry.values:
        for bad in (-1, 2):
            refused(lib, entry, INVALID, "unknown", kind=bad)
    if "act" in entry.values:
        for bad in (-1, 4):
            refused(lib, entry, INVALID, "activation", act=bad)


def test_limits(lib):
    for entry in (NORM, NORM_BACKWARD):
        refused(lib, entry, UNSUPPORTED, "M > 2^20", M=(1 << 20) + 1)
        refused(lib, entry, UNSUPPORTED, "C > 32768", C=32769)
    for entry in (RECURRENCE, RECURRENCE_BACKWARD):
        refused(lib, entry, UNSUPPORTED, "T > 2^24", T=(1 << 24) + 1)
        refused(lib, entry, UNSUPPORTED, "S > 2^20", S=(1 << 20) + 1)
        refused(lib, entry, UNSUPPORTED, "C > 65536", C=65537)
    for entry in (GATED, GATED_BACKWARD):
        refused(lib, entry, UNSUPPORTED, "M > 2^20", M=(1 << 20) + 1)
        refused(lib, entry, UNSUPPORTED, "N > 2^24", N=(1 << 24) + 1)
        refused(lib, entry, UNSUPPORTED, "K > 65536", K=65537)


def test_missing_arrays(lib):
    for entry, names in ((NORM, "x y"), (NORM_BACKWARD, "dy x stat"), (RECURRENCE, "x gate h"),
                         (RECURRENCE_BACKWARD, "dh x gate states"), (GATED, "x wg wu y"),
                         (GATED_BACKWARD, "dy x wg wu pre")):
        for k in names.split():
            refused(lib, entry, INVALID, "null pointer", **{k: 0})
    refused(lib, NORM, INVALID, "sum goes with residual", sum=0)
    refused(lib, NORM, INVALID, "sum goes with residual", residual=0)


def test_alignment(lib):
    for entry in ENTRIES:
        for k in entry.arrays:
            if k == "ws":
                continue
            refused(lib, entry, INVALID, "align", **{k: entry.values[k] + 1})
            if entry.values[k] and k in ("x", "dy", "wg", "wu") and entry in (GATED, GATED_BACKWARD):
                refused(lib, entry, INVALID, "16-byte", **{k: entry.values[k] + 8})
            if k in ("h0", "last", "states", "dlast", "dh0", "offsets", "pre"):
                refused(lib, entry, INVALID, "misaligned", **{k: entry.values[k] + 2})
    refused(lib, NORM, INVALID, "misaligned", stat=NORM.values["stat"] + 4)
    refused(lib, RECURRENCE, INVALID, "misaligned", kind=1, gate=RECURRENCE.values["gate"] + 2)
    refused(lib, RECURRENCE_BACKWARD, INVALID, "misaligned", kind=1, dgate=RECURRENCE_BACKWARD.values["dgate"] + 2)
    refused(lib, NORM, INVALID, "misaligned", dt=F32, w=NORM.values["w"] + 2)


def test_workspaces(lib):
    for entry in (NORM_BACKWARD, RECURRENCE, RECURRENCE_BACKWARD, GATED, GATED_BACKWARD):
        refused(lib, entry, WORKSPACE, "workspace", ws=0)
        refused(lib, entry, WORKSPACE, "aligned", ws=entry.values["ws"] + 64)
        sizes = [entry.values[k] for k in SIZES[entry.name].split()] + [BF16]
        if entry in (RECURRENCE, RECURRENCE_BACKWARD):
            sizes.append(0)
        need = getattr(lib, f"dspark_{entry.name}_workspace_bytes")(*sizes)
        assert need > 0 and need % 256 == 0
        refused(lib, entry, WORKSPACE, "workspace", n=need - 1)


def test_eps(lib):
    for eps in (-1e-9, NAN, float("inf")):
        refused(lib, NORM, INVALID, "eps", eps=eps)


def test_sequences_of_equal_length_divide_the_rows(lib):
    for entry in (RECURRENCE, RECURRENCE_BACKWARD):
        refused(lib, entry, INVALID, "divide", offsets=0, S=7)
        refused(lib, entry, INVALID, "divide", offsets=0, S=0)


def test_nothing_to_do_is_no_call(lib):
    """Empty sizes, and gradients that nobody asks for, are accepted without
    arrays."""
    none = {k: 0 for e in ENTRIES for k in e.arrays}
    pick = lambda e: {k: 0 for k in e.arrays}  # noqa: E731
    assert none
    for entry, sizes in ((NORM, dict(M=0)), (NORM, dict(C=0)), (GATED, dict(M=0)), (GATED, dict(N=0)),
                         (RECURRENCE, dict(C=0)), (RECURRENCE, dict(T=0, S=0)), (RECURRENCE, dict(T=0, S=3))):
        assert entry(lib, **pick(entry), **sizes, n=0) == OK, (entry.name, sizes)
    assert NORM_BACKWARD(lib, dx=0, dw=0, db=0) == OK
    assert RECURRENCE_BACKWARD(lib, dx=0, dgate=0, dh0=0) == OK
    assert GATED_BACKWARD(lib, dx=0, dwg=0, dwu=0, dbg=0, dbu=0) == OK


def test_workspace_sizes(lib):
    assert lib.dspark_norm_backward_workspace_bytes(0, 8, BF16) == 0
    assert lib.dspark_norm_backward_workspace_bytes(8, 8, 7) == 0
    assert lib.dspark_gated_linear_workspace_bytes(0, 8, 8, BF16) == 0
    assert lib.dspark_gated_linear_backward_workspace_bytes(-1, 8, 8, BF16) == 0
    assert lib.dspark_recurrence_workspace_bytes(8, 8, 8, BF16, 5) == 0
    assert lib.dspark_recurrence_workspace_bytes(256, 256, 2560, BF16, 0) == 0          # a decoder's step needs none
    # nothing of the order of the rows themselves
    assert lib.dspark_recurrence_backward_workspace_bytes(1 << 20, 1, 4096, BF16, 0) < (1 << 20) * 4096 // 4
    # sizes at the limits do not wrap
    assert lib.dspark_gated_linear_backward_workspace_bytes(1 << 20, 1 << 24, 65536, BF16) > 1 << 46
    assert lib.dspark_recurrence_backward_workspace_bytes(1 << 24, 1, 65536, F32, 1) > 1 << 36
