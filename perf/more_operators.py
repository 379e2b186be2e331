"""The operators that a program calls between a language model's layers and its next token, as cases to time.

Each case is one pass through one operator as a program calls it:

  prompt  packed prompts of different lengths through linear attention with a decay for each head,
          with the state of each prompt left in a cache
  step    one token for each of several running sequences through the same, the cache updated in place
  sample  the next token from logits: temperature, top-k, top-p and min-p, from given uniform numbers
  move    entries of all arrays of a model's cache copied, moved and freed at once

`own` selects between elementary torch operations and the framework's kernels.
"""
import math

import torch

own = False

CHUNK = 64  # tokens that the plain form takes side by side
WIDTH = 4  # taps of the convolution whose rows a cache holds
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lm():
    import selective_state_space_51_amd as S
    return S


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a batch of short chat turns arriving together, some continuing a conversation (carry); a small model, inner width 1536
        dict(name="prompt_turns", op="prompt", dtype="bf16", heads=24, groups=1, dk=64, dv=64, lens="1,7,33,120,64,5,257,18",
             carry=True, fused=True, decay="token", slots=12),
        # one document read alone, full precision, with a fixed decay for each head and queries and keys of their own
        dict(name="prompt_document", op="prompt", dtype="f32", heads=24, groups=24, dk=64, dv=64, lens="4097", carry=False,
             fused=False, decay="head", slots=1),
        # a full prefill batch of a large layer (inner width 4096): long and short prompts packed
        dict(name="prompt_batch", op="prompt", dtype="bf16", heads=64, groups=1, dk=128, dv=64,
             lens="4096,3001,2048,2000,1999,1777,1500,1411,1300,1111,1024,1000,999,900,802,701,640,512,300,255,128,77,9,1",
             carry=True, fused=True, decay="token", slots=32),
        # one user's next token: latency counts
        dict(name="step_one", op="step", dtype="bf16", heads=24, groups=1, dk=64, dv=64, rows=1, fused=True, decay="token", slots=4),
        # a full decode batch of a large layer
        dict(name="step_batch", op="step", dtype="bf16", heads=64, groups=1, dk=128, dv=64, rows=128, fused=True, decay="token",
             slots=144),
        # the next token of a few conversations with one setting for all
        dict(name="sample_turns", op="sample", dtype="bf16", vocab=50280, rows=3, pad=0, settings="shared", temperature=0.8,
             top_k=50, top_p=0.95, min_p=0.0),
        # a full decode batch, each row with its user's own settings (greedy ones and unlimited ones among them)
        dict(name="sample_batch", op="sample", dtype="bf16", vocab=50280, rows=256, pad=3, settings="rows", temperature=1.0,
             top_k=0, top_p=1.0, min_p=0.0),
        # nucleus sampling over a large vocabulary
        dict(name="sample_nucleus", op="sample", dtype="bf16", vocab=131072, rows=64, pad=0, settings="shared", temperature=1.0,
             top_k=0, top_p=0.9, min_p=0.0),
        # rollouts for policy-gradient training: the model's own distribution, nothing cut off
        dict(name="sample_rollout", op="sample", dtype="f32", vocab=32001, rows=1000, pad=0, settings="shared", temperature=1.0,
             top_k=0, top_p=1.0, min_p=0.0),
        # a prompt that was read once goes on as eight continuations: 24 layers' convolution rows and scan states
        dict(name="move_fork", op="move", layers=24, slots=16, moves=7, kind="fork", state="scan", dtype="bf16", dim=1536, dk=16, dv=1),
        # a large cache after its short sequences ended: the running ones move to the front, the rest is freed
        dict(name="move_compact", op="move", layers=4, slots=160, moves=60, kind="compact", state="heads", dtype="bf16", dim=4096,
             dk=128, dv=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly multiples of 8 as models have, sometimes odd ones."""
    w = _log(rng, lo, hi)
    return max(8, w // 8 * 8) if rng.random() < 0.75 else w


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "step", "step", "sample", "sample", "sample", "move"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("prompt", "step"):
        dk, dv = _width(rng, 16, 256), _width(rng, 16, 256)
        heads = _log(rng, 1, 64)
        groups = rng.choice([g for g in range(1, heads + 1) if heads % g == 0])
        both = dict(op=op, dtype=dtype, heads=heads, groups=groups, dk=dk, dv=dv, fused=rng.random() < 0.5,
                    decay=rng.choice(["token", "token", "head"]))
        each = heads * dk * dv
        if op == "step":
            rows = max(1, min(_log(rng, 1, 256), (1 << 26) // each))
            return dict(both, rows=rows, slots=rows + rng.randrange(9))
        lens, chunks = [], 0
        for _ in range(_log(rng, 1, 48)):
            n = _log(rng, 1, 4096) if rng.random() < 0.95 else 0
            more = -(-n // CHUNK)
            # what the chunks of the plain form hold, and what its sequences' states do
            if (chunks + more) * CHUNK * each <= 27591 * 64 * 128 * 64 and (chunks + more) * heads * 64 * max(dk, dv, 64) <= 1 << 28 and \
                    (len(lens) + 1) * each <= 1 << 25:
                lens.append(n)
                chunks += more
        lens = lens if sum(lens) else [17]
        return dict(both, lens=",".join(map(str, lens)), carry=rng.random() < 0.5, slots=len(lens) + rng.randrange(5))
    if op == "sample":
        vocab = _log(rng, 250, 131072)
        rows = max(1, min(_log(rng, 1, 1024), 32 * 1024 * 1024 // vocab))
        return dict(op=op, dtype=dtype, vocab=vocab, rows=rows, pad=rng.choice([0, 0, 1, vocab // 50]),
                    settings=rng.choice(["shared", "rows"]), temperature=rng.choice([0.6, 0.8, 1.0, 1.0, 1.3]),
                    top_k=rng.choice([0, 0, 1, 20, 50, 400]), top_p=rng.choice([1.0, 0.99, 0.95, 0.9, 0.5]),
                    min_p=rng.choice([0.0, 0.0, 0.02, 0.1]))
    slots = _log(rng, 2, 128)
    state = rng.choice(["scan", "heads"])
    dim = _width(rng, 64, 4096)
    dk, dv = (16, 1) if state == "scan" else (rng.choice([32, 64, 128]), 64)
    dim = max(64, dim // 64 * 64) if state == "heads" else dim
    layers = max(1, min(_log(rng, 1, 24), (1 << 27) // (slots * dim * dk)))
    kind = rng.choice(["fork", "compact"])
    return dict(op=op, layers=layers, slots=slots, moves=max(1, min(_log(rng, 1, 64), slots // 2)), kind=kind, state=state,
                dtype=dtype, dim=dim, dk=dk, dv=dv)


# ---------------------------------------------------------------------------------- prepare
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)
    ru = lambda *s: torch.rand(*s, generator=g, device=dev)
    st = {"case": case, "seed": seed}
    op = case["op"]
    if op in ("prompt", "step"):
        io = TORCH[case["dtype"]]
        H, G, dk, dv = case["heads"], case["groups"], case["dk"], case["dv"]
        if op == "prompt":
            lens = [int(v) for v in case["lens"].split(",")]
            rows, nseq = sum(lens), len(lens)
            st["cu"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
            st["lens"], st["max_len"] = lens, max(lens)
            carry = (ru(nseq) < 0.5) if case["carry"] else torch.zeros(nseq, dtype=torch.bool, device=dev)
            st["carry"] = carry.to(torch.uint8)
        else:
            rows = nseq = case["rows"]
        st["slot"] = torch.randperm(case["slots"], generator=g, device=dev)[:nseq].to(torch.int32)
        # queries, keys and values side by side as one projection leaves them, or apart
        if case["fused"]:
            p = rn(rows, 2 * G * dk + H * dv).to(io)
            parts = p[:, :G * dk], p[:, G * dk:2 * G * dk], p[:, 2 * G * dk:]
        else:
            parts = rn(rows, G * dk).to(io), rn(rows, G * dk).to(io), rn(rows, H * dv).to(io)
        st["q"], st["k"], st["v"] = (t.unflatten(1, (n, -1)) for t, n in zip(parts, (G, G, H)))
        rate = 1.0 + 15.0 * ru(H)
        if case["decay"] == "token":  # a step size between 1e-3 and 1e-1 for each token, times the head's rate
            st["decay"] = -torch.exp(ru(rows, H) * math.log(100.0) + math.log(1e-3)) * rate
        else:  # from about two tokens' memory to a thousand's
            st["decay"] = -torch.exp(ru(H) * math.log(500.0) + math.log(1e-3))
        st["scale"] = dk ** -0.5
        st["state"] = rn(case["slots"], H, dk, dv)
    elif op == "sample":
        rows, v = case["rows"], case["vocab"]
        logits = 2.5 * rn(rows, v)
        if case["pad"]:
            logits[:, v - case["pad"]:] = float("-inf")  # the vocabulary's padding columns
        st["logits"] = logits.to(TORCH[case["dtype"]])
        st["uniform"] = ru(rows)
        if case["settings"] == "rows":
            pick = lambda *s: torch.tensor(s, device=dev)[torch.randint(len(s), (rows,), generator=g, device=dev)]
            st["temperature"], st["top_k"] = pick(0.0, 0.6, 0.8, 1.0, 1.0, 1.3), pick(0, 0, 1, 20, 50, 200).to(torch.int32)
            st["top_p"], st["min_p"] = pick(1.0, 1.0, 0.95, 0.9, 0.5), pick(0.0, 0.0, 0.02, 0.1)
        else:
            for key in ("temperature", "top_k", "top_p", "min_p"):
                st[key] = case[key]
    else:
        slots, moves = case["slots"], case["moves"]
        dim, io = case["dim"], TORCH[case["dtype"]]
        caches = []
        for _ in range(case["layers"]):
            caches.append(rn(slots, WIDTH - 1, dim).to(io))
            caches.append(rn(slots, dim, case["dk"]) if case["state"] == "scan" else rn(slots, dim // case["dv"], case["dk"], case["dv"]))
        st["caches"] = caches
        order = torch.randperm(slots, generator=g, device=dev)
        if case["kind"] == "fork":  # one entry to several others, the last of them left empty for a new sequence
            st["dst"] = order[1:1 + moves].to(torch.int32)
            src = order[:1].repeat(st["dst"].numel())
            src[5:6] = -1
        else:  # running entries go to the front, which may hold running ones too; every fifth place is freed
            st["dst"] = torch.arange(moves, device=dev, dtype=torch.int32)
            src = order[:moves].clone()
            src[4::5] = -1
        st["src"] = src.to(torch.int32)
    return st


# ------------------------------------------------------------------------- plain operators
def _heads(t, heads):
    """[..., groups, n, d] -> [..., heads, n, d], each group's heads side by side."""
    return t.repeat_interleave(heads // t.shape[-3], -3)


def _plain_prompt(st):
    c = st["case"]
    io, H, dv = TORCH[c["dtype"]], c["heads"], c["dv"]
    dev = st["q"].device
    cu, slot, carry = st["cu"].long(), st["slot"].long(), st["carry"].bool()
    total, nseq = st["q"].shape[0], cu.numel() - 1
    counts = [-(-n // CHUNK) for n in st["lens"]]
    nc, deep = sum(counts), max(counts)
    # chunk j of a sequence holds its tokens from 64 j on
    count = (cu[1:] - cu[:-1] + CHUNK - 1) // CHUNK
    base = count.cumsum(0) - count
    ids = torch.arange(nc, device=dev)
    seq = (ids[:, None] >= (base + count)[None]).sum(1)
    row = cu[seq][:, None] + (ids - base[seq])[:, None] * CHUNK + torch.arange(CHUNK, device=dev)
    live = row < cu[seq + 1][:, None]
    row = row.clamp(max=total - 1)
    take = lambda t: torch.where(live[:, :, None, None], t.float()[row], torch.zeros((), device=dev)).transpose(1, 2)
    q, k, v = take(st["q"]), take(st["k"]), take(st["v"])  # [chunks, groups or heads, 64, d]
    g = st["decay"].double()
    g = g[row] if g.dim() == 2 else g.expand(nc, CHUNK, H)
    G = torch.where(live[:, :, None], g, torch.zeros((), device=dev, dtype=g.dtype)).cumsum(1).transpose(1, 2)  # [chunks, heads, 64]
    low = torch.ones(CHUNK, CHUNK, device=dev, dtype=torch.bool).tril()
    D = torch.where(low, G[..., :, None] - G[..., None, :], torch.full((), -math.inf, device=dev, dtype=G.dtype))
    w = _heads(q @ k.transpose(2, 3), H) * torch.exp(D).float()
    del D
    o = w @ v
    del w
    left = torch.exp(G[..., -1:] - G).float()[..., None]
    local = _heads(k, H).transpose(2, 3) @ (v * left)  # what each chunk adds to the state
    # the states from chunk to chunk, all sequences side by side
    S = torch.where(carry[:, None, None, None], st["state"][slot], torch.zeros((), device=dev))
    keep = torch.exp(G[..., -1]).float()[..., None, None]
    starts = torch.empty(nc + 1, *local.shape[1:], device=dev)  # (the last row: for sequences that have ended)
    for j in range(deep):
        on = j < count
        at = torch.where(on, base + j, nc)
        starts[at] = S
        at = at.clamp(max=nc - 1)
        S = torch.where(on[:, None, None, None], keep[at] * S + local[at], S)
    o = o + torch.exp(G).float()[..., None] * (_heads(q, H) @ starts[:nc])
    st["state"][slot] = S
    tok = torch.arange(total, device=dev)
    s = (tok[:, None] >= cu[None, 1:]).sum(1)
    pos = tok - cu[s]
    o = o.transpose(1, 2).reshape(nc * CHUNK, H, dv)[(base[s] + pos // CHUNK) * CHUNK + pos % CHUNK]
    return (st["scale"] * o).to(io), st["state"]


def _plain_step(st):
    c = st["case"]
    H, slot = c["heads"], st["slot"].long()
    q, k = (st[n].float().repeat_interleave(H // c["groups"], 1) for n in "qk")
    e = torch.exp(st["decay"].expand(c["rows"], H))[..., None, None]
    S = e * st["state"][slot] + k[..., :, None] * st["v"].float()[..., None, :]
    st["state"][slot] = S
    return (st["scale"] * (q[..., :, None] * S).sum(2)).to(TORCH[c["dtype"]]), st["state"]


def _settings(st, dtype):
    """Temperature, top-k, top-p and min-p of each row, [rows, 1]."""
    x = st["logits"]
    out = []
    for key, t in (("temperature", torch.float32), ("top_k", torch.int64), ("top_p", torch.float32), ("min_p", torch.float32)):
        v = st[key]
        v = v.to(t) if isinstance(v, torch.Tensor) else torch.full((x.shape[0],), v, device=x.device, dtype=t)
        out.append((v if key == "top_k" else v.to(dtype))[:, None])
    return out


def _plain_sample(st):
    """In 64 bits: whether a token stays, and which one a number falls on, turn on sums next to a border."""
    x = st["logits"].double()
    rows, n = x.shape
    T, k, p, m = _settings(st, torch.float64)
    greedy = T <= 0
    val, order = torch.sort(x, dim=1, descending=True, stable=True)
    best = val[:, :1]
    rank = torch.arange(n, device=x.device)[None]
    divisor = torch.where(greedy, torch.ones_like(T), T)
    w = torch.exp((val - best) / divisor)
    stays = (rank < torch.where(k <= 0, n, k)) & (val > -math.inf)
    w = torch.where(stays, w, torch.zeros_like(w))
    cum = w.cumsum(1)
    before = torch.cat([torch.zeros_like(best), cum[:, :-1]], 1)
    stays &= (p >= 1) | (before < p * cum[:, -1:])
    stays &= w >= m
    stays = torch.where(greedy, torch.zeros_like(stays), stays)
    stays[:, 0] = True
    kept = torch.zeros_like(stays).scatter_(1, order, stays)
    z = (x - best) / divisor
    cum = torch.where(kept, torch.exp(z), torch.zeros_like(z)).cumsum(1)
    token = (cum <= st["uniform"].double()[:, None] * cum[:, -1:]).sum(1, keepdim=True)
    last = torch.where(kept, rank, 0).amax(1, keepdim=True)
    token = torch.minimum(token, last)
    logprob = z.gather(1, token) - torch.log(cum[:, -1:])
    return token[:, 0], logprob[:, 0].float(), kept.sum(1).to(torch.int32)


def _plain_move(st):
    src, dst = st["src"].long(), st["dst"].long()
    for c in st["caches"]:
        rows = c[src.clamp(min=0)]
        rows[src < 0] = 0
        c[dst] = rows
    return st["caches"]


# -------------------------------------------------------------------------------------- run
def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        return {"prompt": _plain_prompt, "step": _plain_step, "sample": _plain_sample, "move": _plain_move}[op](st)
    S = _lm()
    if op == "prompt":
        o = S.linear_attn_packed_fwd(st["q"], st["k"], st["v"], st["decay"], st["cu"], st["state"], scale=st["scale"],
                                     slots=st["slot"], carry=st["carry"], max_seqlen=st["max_len"])
        return o, st["state"]
    if op == "step":
        return S.linear_attn_step(st["q"], st["k"], st["v"], st["decay"], st["state"], scale=st["scale"], slots=st["slot"]), st["state"]
    if op == "sample":
        return S.token_sample(st["logits"], st["uniform"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                              min_p=st["min_p"])
    S.cache_entries_copy(st["caches"], st["src"], st["dst"])
    return st["caches"]


# ------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    s = 2 if case["dtype"] == "bf16" else 4
    if op in ("prompt", "step"):
        H, G, dk, dv = case["heads"], case["groups"], case["dk"], case["dv"]
        rows = nseq = carried = case.get("rows", 0)
        if op == "prompt":
            lens = [int(v) for v in case["lens"].split(",")]
            rows, nseq = sum(lens), len(lens)
            carried = nseq / 2 if case["carry"] else 0
        # q, k, v in, o out, decays, states in and out; the recurrence: the state's update and its product with q
        b = rows * (2 * G * dk + 2 * H * dv) * s + (rows if case["decay"] == "token" else 1) * H * 4 + (nseq + carried) * H * dk * dv * 4
        return {"bytes": int(b), "flops": rows * H * dk * dv * 4}
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * s + 36 * case["rows"], "flops": 8 * n}
    n = min(case["moves"], case["slots"] - 1) if case["kind"] == "fork" else case["moves"]
    freed = int(n > 5) if case["kind"] == "fork" else n // 5
    entry = (WIDTH - 1) * case["dim"] * s + case["dim"] * case["dk"] * 4
    return {"bytes": (2 * n - freed) * entry * case["layers"], "flops": 0}


# ------------------------------------------------------------------------------------ exact
def _exact_heads(q, k, v, g, scale, S0):
    """One sequence as attention whose scores decay with distance, block of rows by block of rows: o and the last state."""
    L, H = v.shape[:2]
    if L == 0:
        return v.clone(), S0
    share = H // q.shape[1]
    q, k, v = q.permute(1, 0, 2), k.permute(1, 0, 2), v.permute(1, 0, 2)
    t = g.t().cumsum(1)  # [heads, L]
    outs = []
    for h in range(H):
        kh, vh, th = k[h // share], v[h], t[h]
        o = torch.exp(th)[:, None] * (q[h // share] @ S0[h])
        for a in range(0, L, 2048):
            b = min(L, a + 2048)
            far = th[a:b, None] - th[None, :b]
            late = torch.arange(b, device=v.device)[None] > torch.arange(a, b, device=v.device)[:, None]
            o[a:b] += ((q[h // share][a:b] @ kh[:b].t()) * torch.exp(far.masked_fill(late, -math.inf))) @ vh[:b]
        outs.append(o * scale)
    end = torch.stack([torch.exp(t[h, -1]) * S0[h] + (k[h // share] * torch.exp(t[h, -1] - t[h])[:, None]).t() @ v[h] for h in range(H)])
    return torch.stack(outs, 1), end


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = lambda t: t.double()
    if op == "prompt":
        state, outs, at = f64(st["state"]), [], 0
        for i, n in enumerate(st["lens"]):
            rows, slot = slice(at, at + n), int(st["slot"][i])
            S0 = state[slot] if bool(st["carry"][i]) else torch.zeros_like(state[slot])
            g = f64(st["decay"][rows] if st["decay"].dim() == 2 else st["decay"][None].repeat(n, 1))
            o, state[slot] = _exact_heads(f64(st["q"][rows]), f64(st["k"][rows]), f64(st["v"][rows]), g, st["scale"], S0)
            outs.append(o)
            at += n
        return torch.cat(outs), state
    if op == "step":
        state, outs = f64(st["state"]), []
        share = case["heads"] // case["groups"]
        for r in range(case["rows"]):
            slot = int(st["slot"][r])
            e = torch.exp(f64(st["decay"] if st["decay"].dim() == 1 else st["decay"][r]))
            k, q = (f64(st[n][r]).repeat_interleave(share, 0) for n in "kq")
            state[slot] = e[:, None, None] * state[slot] + torch.matmul(k[:, :, None], f64(st["v"][r])[:, None, :])
            outs.append(st["scale"] * torch.matmul(q[:, None, :], state[slot])[:, 0])
        return torch.stack(outs), state
    if op == "sample":
        T, k, p, m = _settings(st, torch.float64)
        tokens, logs, counts = [], [], []
        for r in range(case["rows"]):
            x = f64(st["logits"][r])
            if float(T[r]) <= 0:
                tokens.append(int((x == x.max()).nonzero()[0]))
                logs.append(0.0)
                counts.append(1)
                continue
            live = (x > -math.inf).nonzero()[:, 0]
            order = live[torch.sort(-x[live], dim=0, stable=True).indices]
            if int(k[r]) > 0:
                order = order[:int(k[r])]
            prob = torch.softmax(x[order] / T[r], 0)
            n = order.numel()
            if float(p[r]) < 1:
                n = 1 + int((prob.cumsum(0)[:-1] < p[r]).sum())
            n = max(1, min(n, int((prob >= m[r] * prob[0]).sum())))
            ids = torch.sort(order[:n]).values
            prob = torch.softmax(x[ids] / T[r], 0)
            at = min(n - 1, int(torch.searchsorted(prob.cumsum(0), st["uniform"][r].double()[None], right=True)))
            tokens.append(int(ids[at]))
            logs.append(float(torch.log_softmax(x[ids] / T[r], 0)[at]))
            counts.append(n)
        dev = st["logits"].device
        return (torch.tensor(tokens, device=dev), torch.tensor(logs, device=dev, dtype=torch.float64),
                torch.tensor(counts, device=dev, dtype=torch.int32))
    src, dst = st["src"].tolist(), st["dst"].tolist()
    news = []
    for c in st["caches"]:
        new = f64(c)
        for a, b in zip(src, dst):
            new[b] = f64(c[a]) if a >= 0 else 0.0
        news.append(new)
    return news
