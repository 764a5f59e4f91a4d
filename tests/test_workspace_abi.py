"""Host-side refusals of workspaces that the kernels' vector accesses cannot use (no GPU: every
call here is refused before anything is enqueued)."""
import ctypes

import pytest

from block_causal_kv_gb300 import d2f

P = ctypes.c_void_p(256)  # an aligned pointer that is never dereferenced
BF16, F32 = 0, 1
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return d2f.load()


def attn_kv4(lib, ws, dt):
    return lib.d2f_block_attn_kv4(P, P, P, P, P, 8, P, P, P, None, 1, 16, 16, 64, 4, 2, 128, 16, 4, 0,
                                  0, dt, ctypes.c_float(0.1), ws, BIG, None, None)


def attn(lib, ws, dt):
    return lib.d2f_block_attn(P, P, P, P, P, P, 8, P, P, P, None, 1, 16, 16, 64, 4, 2, 128, 16, 4, dt,
                              ctypes.c_float(0.1), 3, ws, BIG, None, None)


def logprobs(lib, ws, dt):
    return lib.d2f_token_logprobs(P, 152064, dt, 152064, 1, None, P, 1, 2, P, None, P, P, ws, BIG,
                                  None, None)


def commit(lib, ws, dt):
    return lib.d2f_commit(P, 152064, dt, 152064, 16, None, P, P, P, P, P, 1, 16, 16, 7, None, None,
                          None, 4, ws, BIG, None, None)


@pytest.mark.parametrize("offset", [1, 2, 4, 8, 12])
@pytest.mark.parametrize("call,dt", [(attn_kv4, BF16), (attn_kv4, F32), (attn, F32),
                                     (logprobs, BF16), (logprobs, F32), (commit, BF16),
                                     (commit, F32)])
def test_a_workspace_off_16_bytes_is_refused(lib, call, dt, offset):
    assert call(lib, ctypes.c_void_p(256 + offset), dt) == 1
    assert "16-byte" in lib.d2f_last_error_string().decode()
