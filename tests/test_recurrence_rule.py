"""Which recurrences are split into tiles, told by whether they need a
workspace (CPU only)."""
import os

import pytest

from semi_ar_drafter_amd import binding


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from semi_ar_drafter_amd import build_lib
        build_lib.build(verbose=False)
    return binding.load()


def test_no_sequence_is_taken_to_be_longer_than_all_rows(lib):
    """One or two packed sequences: the longest is counted with the rows that
    there are, as one sequence without offsets is."""
    for S in (1, 2, 3):
        for T, tiles in ((14, False), (32, False), (40, False), (41, True), (64, True), (4000, True)):
            for dt in (binding.DSPARK_F32, binding.DSPARK_BF16):
                for name in ("recurrence", "recurrence_backward"):
                    n = getattr(lib, f"dspark_{name}_workspace_bytes")(T, S, 256, dt, 0)
                    assert (n > 0) == tiles, (name, T, S)


def test_many_short_sequences_go_row_by_row(lib):
    for T, S in ((256, 256), (4096, 256), (65536, 512), (1 << 24, 1 << 20)):
        assert lib.dspark_recurrence_workspace_bytes(T, S, 256, binding.DSPARK_BF16, 0) == 0
    assert lib.dspark_recurrence_workspace_bytes(65536, 200, 256, binding.DSPARK_BF16, 0) > 0
