"""What the attend calls ask for as scratch (host only)."""
import ctypes
import os
import re

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


def test_a_backward_call_asks_for_states_of_sequences_that_it_reads(L):
    """`last`, the final states, beside a dg and a d_state, and `first`, the
    gradient of the initial ones, beside a dg and no d_state0: nothing else
    grows with the sequences but for their 16 + 8 + 32 * 8 bytes a slot."""
    dims, state = (16, 32, 128, 128, 1, 0), 32 * 128 * 128 * 4
    extra = lambda what: size(L, dims, 1024, 65536, what) - size(L, dims, 24, 65536, what)  # noqa: E731
    for dg in (0, L.GDNL_ASKS_DG):
        for ds in (0, L.GDNL_ASKS_D_STATE):
            for d0 in (0, L.GDNL_ASKS_D_STATE0):
                states = ((1 if ds else 0) + (0 if d0 else 1)) * 1000 * state if dg else 0
                assert states <= extra(L.GDNL_ASKS | dg | ds | d0) <= states + 1000 * 2048
    assert size(L, dims, 1024, 65536, 1) == size(L, dims, 1024, 65536, L.GDNL_ASKS | L.GDNL_ASKS_DG | L.GDNL_ASKS_D_STATE)
    out = ctypes.c_size_t()
    for what in (3, 8, 24, 32, -1, 16 + 8):
        assert L.load().gdnl_attend_workspace_bytes(ctypes.byref(L.GdnlDims(*dims, 1.0)), 4, 64, what, ctypes.byref(out)) == 1


def test_the_binding_has_the_headers_constants(L):
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdn_linear.h")
    with open(header) as f:
        defined = dict(re.findall(r"^#define (GDNL_\w+) (\d+)", f.read(), re.M))
    assert {"GDNL_TOKEN_ROWS", "GDNL_ASKS", "GDNL_ASKS_DG", "GDNL_ASKS_D_STATE", "GDNL_ASKS_D_STATE0"} <= set(defined)
    for name, value in defined.items():
        assert getattr(L, name) == int(value)


def test_the_limits_that_the_header_states(L):
    """At a limit a size is given, beyond it refused; row by row the call itself is."""
    so, out = L.load(), ctypes.c_size_t()
    ask = lambda dims, seqs, rows, back: so.gdnl_attend_workspace_bytes(ctypes.byref(L.GdnlDims(*dims, 1.0)), seqs, rows, back, ctypes.byref(out))  # noqa: E731
    narrow = (1, 1, 1, 1, 0, 0)
    assert ask(narrow, 1, (1 << 31) - 1025, 0) == 0 and ask(narrow, 1, (1 << 31) - 1024, 0) == 1
    assert ask((16, 32, 128, 128, 1, 0), 262000, 1 << 20, 0) == 0
    assert ask((1, 32, 4, 4, 1, 0), 262144, 0, 0) == 1
    for hv, d, status in ((1 << 24, 1, 1), (1 << 17, 128, 0), ((1 << 17) + 1, 128, 1)):  # h_v d_k at most 2^24
        assert ask((1, hv, d, 1, 0, 0), 1, 1, 0) == status
    fake, pool = 0x10000, L.GdnStatePool

    def forward(seqs, pages, max_len=8):
        d = L.GdnlDims(1, 32, 4, 4, 0, 0, 1.0)
        b = L.GdnBatch(fake, fake, None, seqs, max_len, 1)
        return so.gdnl_attend_forward(ctypes.byref(d), fake, 4, fake, 4, fake, 128, fake, 32, ctypes.byref(b), pool(fake, 512, pages),
                                      pool(fake, 512, pages), fake, 128, None, 0, None, None)

    assert forward(262144, 4) == 1      # 2^23 workgroups
    assert forward(1, 1 << 29) == 1     # pages
    assert forward(1, 4, 9) == 1        # in chunks: no workspace
