"""CPU tests of what a launch of linear attention, sampling and cache moves can hold: sizes whose grids pass 2^32 - 1 threads are
refused on the host, before any launch (the addresses here are never followed)."""
import ctypes

import selective_state_space_51_amd as S

L = S.lm_lib
OK, NULL, SHAPE, ALIGN, ALIAS, UNSUPPORTED, WORKSPACE = range(7)
A = lambda i: (i + 1) << 50  # arrays far from one another


def packed(tokens, nseq, longest, heads, dk, dv):
    ws = S.linear_attn_packed_workspace_bytes(tokens, nseq, longest, heads, dk, dv, 1)
    return L.linear_attn_packed_fwd(A(0), dk, A(1), dk, A(2), heads * dv, A(3), heads, 1.0, A(4), None, None, None, A(5), tokens, nseq,
                                    0, longest, heads, 1, dk, dv, 1, A(6), ws, None)


def step(rows, heads, dk, dv):
    return L.linear_attn_step(A(0), dk, A(1), dk, A(2), heads * dv, A(3), heads, 1.0, A(6), A(4), A(5), rows, 1, heads, 1, dk, dv, 1, None)


def test_linear_attention():
    most = ((1 << 32) - 1) // 256
    assert packed(1 << 24, most // 64 + 1, 64, 64, 16, 64) == UNSUPPORTED
    assert packed(1 << 24, most // 128 + 1, 64, 64, 16, 65) == UNSUPPORTED
    # in segments, beside many short sequences
    assert S.linear_attn_packed_workspace_bytes(1 << 24, most // 64 + 1, 1 << 23, 64, 16, 64, 1) > 0
    assert packed(1 << 24, most // 64 + 1, 1 << 23, 64, 16, 64) == UNSUPPORTED
    assert step(most // 64 + 1, 64, 16, 64) == UNSUPPORTED
    assert step(most // 128 + 1, 64, 16, 65) == UNSUPPORTED


def test_sampling():
    def sample(rows, vocab):
        return L.token_sample(A(0), vocab, A(1), None, 1.0, None, 0, None, 1.0, None, 0.0, A(2), A(3), A(4), rows, vocab, 1, None)
    assert sample(1 << 24, 250) == UNSUPPORTED
    assert sample(1 << 23, 250) == UNSUPPORTED
    assert sample(1, (1 << 21) + 1) == UNSUPPORTED


def test_cache_moves():
    def move(sizes, n):
        at = (ctypes.c_void_p * len(sizes))(*(A(i) for i in range(len(sizes))))
        return L.cache_entries_copy(at, (ctypes.c_int64 * len(sizes))(*sizes), len(sizes), A(100), A(101), n, 1 << 15, None)
    assert move([(1 << 32) + 1], 1) == UNSUPPORTED
    assert move([16], 16385) == UNSUPPORTED
