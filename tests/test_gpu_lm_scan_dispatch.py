"""GPU tests of the packed scan's ways of dealing out its work that depend on how many sequences and channels there are:
whole sequences dealt to the compute units longest first (up to 64 of them, more than fill the units once), and segments
whose start states the second launch finds by walking the maps itself (up to 16 segments).  Sampled channels against the
fp64 oracle, sequence by sequence; bars as in the operator's other tests."""
import sys

import numpy as np
import pytest

import oracle
from tests import parity as PT
from tests import test_gpu_lm_scan as T

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def run(lens, dim, dtype, slots, carry, max_seqlen, zoh=False, seed=0):
    """Scans the sequences in a cache of len(lens) + 3 entries; checks every sequence and entry on sampled channels."""
    import torch

    import selective_state_space_51_amd as S
    n = len(lens)
    i = T.make(lens, dim, dtype, seed=seed, nslots=n + 3, bc_pad=4)
    old, h = i["h_state"], i["h_state"].clone()
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    ca = torch.tensor(carry, dtype=torch.bool, device="cuda")
    y = torch.full_like(i["u"], float("nan"))
    S.selscan_packed_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["cu"], h, D=i["D"], z=i["z"], delta_bias=i["bias"],
                         delta_softplus=True, zoh=zoh, slots=sl, carry=ca, max_seqlen=max_seqlen, y=y)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y.float()).all())
    ch = sorted(c for c in {0, 1, 17, 63, 64, dim // 2, dim - 65, dim - 2, dim - 1} if 0 <= c < dim)
    cd = torch.tensor(ch, device="cuda")
    pick = lambda t: T.f64(t[:, cd].contiguous())
    u, d, z, y5 = map(pick, (i["u"], i["delta"], i["z"], y))
    B, C, A, D, bias = T.f64(i["B"].contiguous()), T.f64(i["C"].contiguous()), T.f64(i["A"][cd]), T.f64(i["D"][cd]), T.f64(i["bias"][cd])
    cu = i["cu"].tolist()
    touched = set()
    for s in range(n):
        ok = 0 <= slots[s] < n + 3
        h0 = T.f64(old[slots[s]][cd]) if ok and carry[s] else np.zeros((len(ch), 16))
        k = slice(cu[s], cu[s + 1])
        last = h0
        if lens[s]:
            r, hl = oracle.selscan(u[k][None], d[k][None], A, B[k][None], C[k][None], D=D, z=z[k][None], delta_bias=bias,
                                   delta_softplus=True, zoh=zoh, h0=h0[None], return_h_last=True)
            T.check(("y", s), y5[k][None], r, PT.TOL[dtype])
            last = hl[0]
        if ok:
            touched.add(slots[s])
            T.check(("h", s), h[slots[s]][cd], last, PT.TOL["f32"])
    for s in set(range(n + 3)) - touched:
        assert torch.equal(h[s], old[s])


def order(n, seed):
    """Slots of n sequences in a cache of n + 3, one of them outside it, and which sequences go on from theirs."""
    rng = np.random.default_rng(seed)
    slots = rng.permutation(n + 3)[:n].tolist()
    if n > 2:
        slots[n // 2] = n + 3
        slots[n // 3] = -1
    return slots, (rng.random(n) < 0.5).tolist()


def lengths(kind, n, most, seed):
    rng = np.random.default_rng(seed)
    if kind == "equal":
        return [most] * n
    if kind == "empties":
        return [0 if s % 3 == 0 else int(v) for s, v in enumerate(rng.integers(1, most + 1, n))]
    return rng.integers(1, most + 1, n).tolist()


# (sequences, channels, longest): rounds of 256 / ceil(channels / 64); whole rounds, a last one that is short in a rising and
# in a falling place, 64 sequences, and more channel blocks than compute units
@pytest.mark.parametrize("kind", ["mixed", "equal", "empties"])
@pytest.mark.parametrize("n,dim,most", [(20, 1536, 300), (36, 1536, 200), (64, 1536, 100), (63, 2050, 120), (23, 4096, 150),
                                        (26, 4096, 90), (9, 16400, 40)])
def test_whole_sequences_dealt_out(n, dim, most, kind):
    import selective_state_space_51_amd as S
    dtype = "bf16" if n % 2 else "f32"
    lens = lengths(kind, n, most, seed=n)
    _say("dealt", n, dim, kind, dtype)
    longest = max(lens)
    if S.selscan_packed_workspace_bytes(sum(lens), n, longest, dim) > 0:
        longest = 1  # (a bound too low: whole sequences)
    assert S.selscan_packed_workspace_bytes(sum(lens), n, longest, dim) == 0
    assert 64 >= n > max(1, 256 // -(-dim // 64))
    slots, carry = order(n, n)
    run(lens, dim, dtype, slots, carry, longest, seed=n)


# lengths of up to 16 segments of 16 tokens, cut at their ends and inside
@pytest.mark.parametrize("zoh", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,dim", [((1, 7, 33, 120, 64, 5, 257, 18), 1536), ((200, 0, 70, 33), 200), ((16, 271, 32, 0, 17), 65),
                                      ((48, 80, 96, 255, 256, 1), 520), ((2000, 1800, 1900, 37), 4096)])
def test_segments_walked_by_the_second_launch(lens, dim, dtype, zoh):
    import selective_state_space_51_amd as S
    lens = list(lens)
    _say("walked", lens, dim, dtype, zoh)
    need = S.selscan_packed_workspace_bytes(sum(lens), len(lens), max(lens), dim)
    assert need > 0
    slots, carry = order(len(lens), dim)
    run(lens, dim, dtype, slots, carry, max(lens), zoh=zoh, seed=dim)


# nobody says how long the longest is: all tokens could be one sequence's.  Sequences shorter than a segment beside long ones,
# many of them in one segment's tokens; more sequences than segments with a join of its own, and fewer
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,short,long,dim", [(1000, 9, (700, 0, 301), 40), (5000, 3, (16, 17, 33), 24), (300, 40, (), 70),
                                              (40, 6, (3000, 1999), 200), (150, 30, (900,), 2100), (3, 400, (2, 16), 4096)])
def test_longest_length_not_given(n, short, long, dim, dtype):
    _say("unknown", n, short, long, dim, dtype)
    rng = np.random.default_rng(n)
    lens = rng.integers(0, short + 1, n).tolist()
    for v in long:
        lens.insert(int(rng.integers(0, len(lens) + 1)), v)
    slots, carry = order(len(lens), n)
    run(lens, dim, dtype, slots, carry, None, zoh=n == 300, seed=n)
