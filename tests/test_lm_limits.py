"""CPU tests of what a launch can hold: sizes whose grids pass 2^32 - 1 threads are refused on the host, before any launch
(the addresses here are never followed)."""
import selective_state_space_51_amd as S

L = S.lm_lib
OK, NULL, SHAPE, ALIGN, ALIAS, UNSUPPORTED, WORKSPACE = range(7)
A = lambda i: (i + 1) << 50  # arrays far from one another


def norm(rows, width):
    return L.add_rms_norm_fwd(A(0), width, A(1), A(2), 1e-5, 0, A(3), A(4), None, None, rows, width, 1, 0, None)


def test_norm_rows():
    most = (1 << 32) - 1
    assert norm(4 * (most // 256) + 1, 8) == UNSUPPORTED
    assert norm(most // 256 + 1, 2048) == UNSUPPORTED
    assert norm(most // 1024 + 1, 16384) == UNSUPPORTED


def test_logprobs_rows():
    def fwd(rows, vocab, ws=None, wsb=0):
        return L.token_logprobs_fwd(A(0), vocab, A(1), 1.0, 0, A(2), A(3), A(4), None, None, rows, vocab, 1, ws, wsb, None)

    def bwd(rows, vocab):
        return L.token_logprobs_bwd(A(0), vocab, A(1), A(2), A(3), A(4), None, 1.0, A(5), rows, vocab, 1, None)
    for call in (lambda r, v: fwd(r, v, A(6), 1 << 40), bwd):
        assert call(1 << 24, 250) == UNSUPPORTED
        assert call((1 << 23) + 1, 8193) == UNSUPPORTED
        assert call(1 << 30, 2) == UNSUPPORTED


def test_logprobs_scale():
    # the exponents are of base 2: a scale whose product with log2 e overflows would make every one of them NaN
    fwd = lambda scale: L.token_logprobs_fwd(A(0), 8, A(1), scale, 0, A(2), A(3), A(4), None, None, 0, 8, 1, None, 0, None)
    bwd = lambda scale: L.token_logprobs_bwd(A(0), 8, A(1), A(2), A(3), A(4), None, scale, A(5), 0, 8, 1, None)
    for call in (fwd, bwd):
        assert call(2.35e38) == OK and call(1e-38) == OK
        for scale in (2.4e38, 3.4e38):
            assert call(scale) == UNSUPPORTED


def test_packed_sequences():
    def conv(tokens, nseq, dim):
        return L.causal_conv1d_packed_fwd(A(0), dim, A(1), None, A(2), None, None, None, 0, A(3), tokens, nseq, 0, dim, 4, 1, None)

    def scan(tokens, nseq, longest, dim):
        ws = S.selscan_packed_workspace_bytes(tokens, nseq, longest, dim)
        return L.selscan_packed_fwd(A(0), A(1), A(2), A(3), A(4), 32, None, None, 0, None, 0, A(5), None, None, None, A(6), tokens,
                                    nseq, 0, longest, dim, 16, 1, A(7), ws, None)
    assert conv(1 << 29, 1 << 24, 2048) == UNSUPPORTED
    assert scan(1 << 20, 1 << 18, 4, 4096) == UNSUPPORTED
    # cut into segments (a few long ones among as many short ones)
    assert S.selscan_packed_workspace_bytes(1 << 30, 1 << 18, 1 << 29, 4096) > 0
    assert scan(1 << 30, 1 << 18, 1 << 29, 4096) == UNSUPPORTED


def test_tokens_are_counted_in_32_bits():
    # a walk in blocks, two of them ahead, must not pass 2^31
    def scan(tokens):
        return L.selscan_packed_fwd(A(0), A(1), A(2), A(3), A(4), 32, None, None, 0, None, 0, A(5), None, None, None, A(6), tokens,
                                    1, 0, 1, 4, 16, 1, None, 0, None)

    def step(rows):
        return L.selscan_step(A(0), A(1), A(2), A(3), A(4), 32, None, None, 0, None, 0, A(5), A(6), A(7), rows, 1, 4, 16, 1, None)

    def conv_step(rows):
        return L.causal_conv1d_step(A(0), 4, A(1), None, A(2), A(3), 0, A(4), rows, 1, 4, 4, 1, None)
    for call in (scan, step, conv_step):
        for n in ((1 << 31) - 1, (1 << 31) - (1 << 17) + 1):
            assert call(n) == UNSUPPORTED
    assert S.selscan_packed_workspace_bytes((1 << 31) - 1, 1, (1 << 31) - 1, 64) == 0


def test_step_channels_and_matrix_rows():
    def step(dim):
        return L.selscan_step(A(0), A(1), A(2), A(3), A(4), 32, None, None, 0, None, 0, A(5), A(6), A(7), 1, 1, dim, 16, 1, None)

    def w4(n):
        return L.w4_matvec(A(0), 32, A(1), A(2), None, None, A(3), 1, n, 32, 32, 1, None)
    assert step(1 << 30) == UNSUPPORTED
    assert w4((1 << 30) + 1) == UNSUPPORTED
