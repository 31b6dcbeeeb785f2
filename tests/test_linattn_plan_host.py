"""What the linear attention's calls ask of their caller and refuse, by their
sizes (no GPU: sizes of workspaces, and calls that end before any launch)."""
import pytest

import selective_state_space_44_amd as ssm

STATE = 40 * 128 * 64 * 4   # one segment's states: 40 heads, 64 values, 128 keys


@pytest.fixture(scope="module")
def lib():
    return ssm.load_library()


def _fwd_bytes(lib, batch, tokens, nsplit, packed=1):
    return lib.ssm_linattn_fwd_workspace_bytes(batch, tokens, packed, 40, 8, 128, 64, 1, nsplit)


def test_given_segments_cut_packed_sequences_of_any_mean_length(lib):
    """One long sequence among many short ones: with segments asked for, its
    states between segments have their place, also where the mean is below a
    chunk of 64."""
    for batch in (2, 100, 201, 5000):
        assert _fwd_bytes(lib, batch, 10200, 1) < STATE
        assert _fwd_bytes(lib, batch, 10200, 8) >= 8 * STATE, batch
    # of one length: a chunk cannot be cut
    assert _fwd_bytes(lib, 200, 64, 8, packed=0) == 0
    assert _fwd_bytes(lib, 200, 65, 8, packed=0) > 0
