"""What the attend calls ask for as scratch (host only)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def L():
    import linear_attention_ssm_gdn_amd._lib as lib
    if not os.path.exists(lib.LIB_PATH):
        pytest.skip("libgdn.so not built")
    return lib


def size(L, dims, n_seqs, n_rows, backward):
    out = ctypes.c_size_t()
    assert L.load().gdnl_attend_workspace_bytes(ctypes.byref(L.GdnlDims(*dims, 1.0)), n_seqs, n_rows, backward, ctypes.byref(out)) == 0
    return out.value


def test_many_short_documents_need_no_states_for_each(L):
    """1024 documents of 64 rows, 32 heads of 128 x 128: 2 MB a document's states.
    At 512 workgroups' worth of borders there are 16, and per row and head 16 bytes."""
    state, rows = 32 * 128 * 128 * 4, 65536
    need = size(L, (16, 32, 128, 128, 1, 0), 1024, rows, 0)
    assert need <= 2 * 16 * state + 32 * rows * 16 + (1024 + 17) * (16 + 8 + 32 * 8) + 6 * 256
    assert size(L, (16, 32, 128, 128, 1, 0), 1, rows, 0) >= 2 * 16 * state  # one document is cut, and in place
