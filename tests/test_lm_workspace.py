"""CPU tests of the packed scan's workspace where the longest sequence is not known (max_seqlen None: any bound, the number of
tokens): what is kept of segments is kept of those that another follows, so short sequences take nothing."""
import selective_state_space_51_amd as S


def test_short_sequences_of_unknown_length():
    entry = lambda dim: dim * 17 * 4
    for nseq, each, dim in ((1000, 32, 4096), (5000, 4, 4096), (100_000, 3, 1536), (1, 4097, 1536)):
        tokens = nseq * each
        need = S.selscan_packed_workspace_bytes(tokens, nseq, tokens, dim)
        # segments that fill the units four times over, and of 16 tokens at least: no more of them than that, rounded up
        most = min(tokens // 16, 2 * 1024 // -(-dim // 64))
        assert 0 < need <= most * entry(dim)
        # ... and how many sequences there are does not count
        assert need == S.selscan_packed_workspace_bytes(tokens, 1, tokens, dim)
