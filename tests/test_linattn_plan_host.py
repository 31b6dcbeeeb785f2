"""What the linear attention's calls ask of their caller and refuse, by their
sizes (no GPU: sizes of workspaces, and calls that end before any launch)."""
import pytest
import torch

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


def test_tokens_whose_last_chunk_ends_past_32_bits_are_refused(lib):
    """Walks number tokens in 32 bits, 64 at a time."""
    for packed in (0, 1):
        for over, ok in ((0, True), (1, False), (63, False), (64, False)):
            tokens = 2 ** 31 - 64 + over
            need = lib.ssm_linattn_fwd_workspace_bytes(1, tokens, packed, 1, 1, 8, 8, 1, 1)
            back = lib.ssm_linattn_bwd_workspace_bytes(1, tokens, packed, 1, 1, 8, 8, 1, 0, 1)
            assert (need >= 0, back >= 0) == (ok, ok), tokens


def test_workspaces_that_kernels_cannot_write_to_are_refused():
    """One on another device than the operands, or whose elements share memory."""
    gpu, cpu = torch.device("cuda", 0), torch.device("cpu")
    for bad, device in ((torch.empty(4096, dtype=torch.uint8), gpu),
                        (torch.empty(1, dtype=torch.uint8).expand(4096), cpu),
                        (torch.empty(64, 128, dtype=torch.uint8).t(), cpu), ("workspace", cpu)):
        with pytest.raises(ValueError, match="workspace"):
            ssm._workspace(1024, bad, device)
    ws = torch.empty(1024, dtype=torch.float32)
    assert ssm._workspace(1024, ws, cpu) == (ws.data_ptr(), 4096, ws)
    at, size, new = ssm._workspace(8192, ws, cpu)       # too small: another one
    assert size == 8192 and new is not ws and at == new.data_ptr()
