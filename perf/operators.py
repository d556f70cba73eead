"""Operators of drafted-token decoding: what they compute, on which sizes, and
how a program calls them.

Three operators make one step of decoding with drafted tokens over a
key/value cache:

  attention  queries of a tree of drafted tokens against a sequence's cached
             keys and values and against the drafted tokens on their own path
             (a single token and a causal chunk of a prompt are trees too);
  verify     the walk through the tree that accepts or rejects each drafted
             token against the target's probabilities, from given uniform
             numbers, and draws the token that follows the accepted path;
  append     the keys and values of the accepted tokens stored into the caches
             of every layer.

With ``own`` false, ``run`` computes them in elementary torch operations; with
``own`` true it makes the calls of decoder_only_lm_b200.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "fp32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}


# ---------------------------------------------------------------------- cases
def listed():
    """The cases, smallest calls to largest, per operator."""
    return [
        # one sequence generating one token with GPT-2 124M's heads: latency
        dict(name="attn-1-token", op="attention", dtype=BF16, B=1, N=1, H=12, Hkv=12, D=64,
             lo=700, hi=700, ragged=False, tree=0),
        # the single-token step of a batch of 16 ragged sequences (124M heads)
        dict(name="attn-decode-16", op="attention", dtype=BF16, B=16, N=1, H=12, Hkv=12, D=64,
             lo=64, hi=1023, ragged=False, tree=0),
        # trees of up to 64 drafted tokens, 16 sequences, GPT-2 350M heads
        dict(name="attn-tree-16", op="attention", dtype=BF16, B=16, N=64, H=16, Hkv=16, D=64,
             lo=100, hi=1024, ragged=True, tree=8),
        # trees of 48 over long caches of very different lengths
        dict(name="attn-tree-long", op="attention", dtype=BF16, B=4, N=48, H=12, Hkv=12, D=64,
             lo=9001, hi=32768, ragged=False, tree=6),
        # shared key/value heads: 4 query heads read one cache head, 256 rows a head
        dict(name="attn-tree-shared", op="attention", dtype=BF16, B=8, N=64, H=32, Hkv=8, D=128,
             lo=1000, hi=8191, ragged=True, tree=7),
        # a 256-token chunk of a long prompt behind what is cached already
        dict(name="attn-chunk", op="attention", dtype=BF16, B=2, N=256, H=12, Hkv=12, D=64,
             lo=515, hi=4001, ragged=False, tree=0),
        # the fp32 mode: small odd trees
        dict(name="attn-tree-fp32", op="attention", dtype=F32, B=4, N=13, H=12, Hkv=12, D=64,
             lo=33, hi=1000, ragged=True, tree=5),
        # one sequence, a chain of 4 drafts from a smaller model, plain temperature
        dict(name="verify-chain-1", op="verify", B=1, N=5, V=50257, pad=47, draft=True,
             temperature=0.8, top_k=0, top_p=1.0, tree=0, ragged=False),
        # 16 sequences, trees of 64 proposed without probabilities, nucleus sampling
        dict(name="verify-tree-16", op="verify", B=16, N=64, V=50257, pad=47, draft=False,
             temperature=0.8, top_k=0, top_p=0.9, tree=6, ragged=True),
        # a large batch, small trees with the draft's probabilities, top-k and nucleus
        dict(name="verify-tree-64", op="verify", B=64, N=12, V=50257, pad=47, draft=True,
             temperature=1.0, top_k=200, top_p=0.95, tree=4, ragged=True),
        # the accepted tokens of one 124M sequence into 12 layers' caches
        dict(name="append-1", op="append", dtype=BF16, L=12, B=1, N=5, H=12, Hkv=12, D=64,
             Tc=1024, fill=1.0),
        # 16 sequences of 350M, accepted paths of trees of 64, 24 layers
        dict(name="append-16", op="append", dtype=BF16, L=24, B=16, N=64, H=16, Hkv=16, D=64,
             Tc=160, fill=0.4),
    ]


HEADS = [(12, 12, 64), (12, 12, 64), (16, 16, 64), (4, 4, 16), (8, 2, 32), (32, 8, 128),
         (6, 1, 64)]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["attention", "attention", "attention", "verify", "verify", "append"])
    if op == "attention":
        while True:
            dtype = rng.choice([BF16, BF16, BF16, F32])
            H, Hkv, D = rng.choice(HEADS)
            B, N = _log_int(rng, 1, 32), _log_int(rng, 1, 256)
            hi = _log_int(rng, 1, 32768)
            c = dict(op=op, dtype=dtype, B=B, N=N, H=H, Hkv=Hkv, D=D, lo=rng.randint(0, hi), hi=hi,
                     ragged=rng.random() < 0.5, tree=rng.choice([0, rng.randint(1, 12)]))
            w = work(c)
            scores = 4 * B * H * N * (hi + N)  # the plain form's score matrix
            if (w["bytes"] <= 2.0e8 and w["flops"] <= (3.0e10 if dtype == BF16 else 3.0e9) and
                    scores <= 1.5e9):
                return c
    if op == "verify":
        V = _log_int(rng, 300, 50257)
        draft = rng.random() < 0.5
        while True:
            B, N = _log_int(rng, 1, 64), _log_int(rng, 2, 64)
            if B * N <= 1024:
                break
        return dict(op=op, B=B, N=N, V=V, pad=rng.choice([0, 47, rng.randint(0, 200)]),
                    draft=draft, temperature=rng.choice([0.0, 0.8, 1.0, 1.2]),
                    top_k=rng.choice([0, 0, rng.randint(2, 200)]),
                    top_p=rng.choice([1.0, 0.9, 0.95]), tree=rng.choice([0, rng.randint(1, 8)]),
                    ragged=rng.random() < 0.5)
    while True:
        H, Hkv, D = rng.choice(HEADS)
        L, B, N = rng.randint(1, 24), _log_int(rng, 1, 32), _log_int(rng, 1, 256)
        Tc = N + _log_int(rng, 1, 1024)
        if L * B * Hkv * Tc * D <= 4.0e7 and L * B * N * (H + 2 * Hkv) * D <= 6.0e7:
            return dict(op=op, dtype=rng.choice([BF16, F32]), L=L, B=B, N=N, H=H, Hkv=Hkv, D=D,
                        Tc=Tc, fill=rng.choice([1.0, 0.4, 0.1]))


# ---------------------------------------------------------------------- layout of a case
def _spread(B, lo, hi):
    """B lengths over [lo, hi], the ends included, in a scattered order."""
    if B == 1:
        return [hi]
    order = sorted(range(B), key=lambda b: (b * 0.6180339887498949) % 1.0)
    out = [0] * B
    for r, b in enumerate(order):
        out[b] = lo + (hi - lo) * r // (B - 1)
    return out


def _counts(case):
    """Nodes of each sequence's tree: all N, or ragged from 1 up to N."""
    B, N = case["B"], case["N"]
    return _spread(B, max(1, N // 3), N) if case["ragged"] else [N] * B


def _parents(case):
    """parent[b][i] < i, node 0 the root: a chain (tree = 0), or a random tree
    of at most `tree` levels under the root."""
    B, N, depth = case["B"], case["N"], case["tree"]
    if depth == 0:
        return np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))
    rs = np.random.RandomState(1000 * depth + N)
    par = np.full((B, N), -1, np.int32)
    for b in range(B):
        level = [0]
        for i in range(1, N):
            # mostly below the newest nodes, sometimes anywhere
            cand = [j for j in range(i) if level[j] < depth]
            j = cand[-1 - min(len(cand) - 1, int(rs.geometric(0.35)) - 1)] if rs.rand() < 0.7 \
                else cand[rs.randint(len(cand))]
            par[b, i] = j
            level.append(level[j] + 1)
    return par


def _depths(par):
    d = np.zeros(par.shape, np.int64)
    for i in range(1, par.shape[1]):
        p = par[:, i]
        d[:, i] = np.where(p >= 0, d[np.arange(len(p)), np.maximum(p, 0)] + 1, 0)
    return d


def _append_path(case):
    """Accepted paths: increasing node ids from 0, as many as `fill` gives."""
    B, N = case["B"], case["N"]
    rs = np.random.RandomState(7 * B + N)
    path = np.full((B, N), -1, np.int32)
    n = np.zeros(B, np.int32)
    for b, top in enumerate(_spread(B, 1, max(1, int(case["fill"] * N)))):
        ids = np.concatenate([[0], 1 + np.sort(rs.permutation(N - 1)[:top - 1])])
        path[b, :top] = ids
        n[b] = top
    return path, n


def work(case):
    """Bytes and operations the operator cannot do without."""
    op = case["op"]
    if op == "attention":
        es = 2 if case["dtype"] == BF16 else 4
        H, Hkv, D = case["H"], case["Hkv"], case["D"]
        lens, cnt = _spread(case["B"], case["lo"], case["hi"]), _counts(case)
        dep = _depths(_parents(case))
        keys = sum(lens)
        nodes = sum(cnt)
        pairs = sum(n * l + int((dep[b, :n] + 1).sum())
                    for b, (l, n) in enumerate(zip(lens, cnt)))
        return {"bytes": es * (2 * keys * Hkv * D + nodes * (H + 2 * Hkv) * D + nodes * H * D) +
                4 * nodes * H, "flops": 4 * D * H * pairs}
    if op == "verify":
        # the rows that the walk has to look at: the root's, and one for every
        # accepted token (about 6 in 10 proposals are accepted with the draft's
        # probabilities or with several alternatives); leaves need no draft row
        d = int(_depths(_parents(case)).max())
        rows = sum(0.6 ** i for i in range(d + 1))
        rows += sum(0.6 ** i for i in range(d)) if case["draft"] else 0.0
        n = case["B"] * rows * case["V"]
        return {"bytes": int(4 * n), "flops": int(8 * n)}
    es = 2 if case["dtype"] == BF16 else 4
    _, n = _append_path(case)
    return {"bytes": int(n.sum()) * case["L"] * 4 * case["Hkv"] * case["D"] * es, "flops": 0}


# ---------------------------------------------------------------------- inputs
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    """What a program holds before the call: activations, caches, lengths, trees."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    s = dict(case=case)
    if case["op"] == "attention":
        dt = DTYPES[case["dtype"]]
        B, N, H, Hkv, D = (case[k] for k in ("B", "N", "H", "Hkv", "D"))
        Tc = case["hi"] + N  # room for the drafted tokens behind the longest sequence
        # queries a little larger than unit variance: peaked rows as trained heads have
        qkv = randn(B, N, (H + 2 * Hkv) * D)
        qkv[..., :H * D] *= 1.5
        s.update(qkv=qkv.to(dt), k=randn(B, Hkv, Tc, D, dtype=dt), v=randn(B, Hkv, Tc, D, dtype=dt),
                 lens=_i32(_spread(B, case["lo"], case["hi"])),
                 parent=_i32(_parents(case)) if case["tree"] else None,
                 counts=_i32(_counts(case)) if case["ragged"] else None)
        return s
    if case["op"] == "verify":
        B, N, V, pad = (case[k] for k in ("B", "N", "V", "pad"))
        # peaked rows; the draft's rows are the target's with an error, and the
        # drafted tokens come from them: drawn when the draft's probabilities
        # are known to the verification, its best ones in turn otherwise
        target = 4.0 * randn(B, N, V + pad)
        draft = target + 1.0 * randn(B, N, V + pad)
        par = _parents(case)
        tokens = torch.zeros((B, N), dtype=torch.int32, device="cuda")
        t = case["temperature"] if case["temperature"] > 0 else 1.0
        rank = np.zeros((B, N), np.int64)
        for b in range(B):
            seen = {}
            for i in range(1, N):
                rank[b, i] = seen.get(par[b, i], 0)
                seen[par[b, i]] = rank[b, i] + 1
        rank = torch.from_numpy(rank).cuda()
        rows = torch.arange(B, device="cuda")
        parent = _i32(par)
        for i in range(1, N):
            row = draft[rows, parent[:, i].long(), :V]
            if case["draft"] and case["temperature"] > 0:
                if case["top_k"]:
                    kth = torch.topk(row, min(case["top_k"], V), dim=1).values[:, -1:]
                    row = row.masked_fill(row < kth, float("-inf"))
                tokens[:, i] = torch.multinomial(torch.softmax(row / t, 1), 1,
                                                 generator=gen)[:, 0].int()
            else:
                best = torch.topk(row, min(8, V), dim=1).indices
                tokens[:, i] = best[rows, rank[:, i].clamp(max=min(8, V) - 1)].int()
        s.update(logits=target, draft=draft if case["draft"] else None, tokens=tokens,
                 parent=parent if case["tree"] else None,
                 counts=_i32(_counts(case)) if case["ragged"] else None,
                 uniform=torch.rand((B, N), generator=gen, device="cuda"))
        return s
    dt = DTYPES[case["dtype"]]
    L, B, N, H, Hkv, D, Tc = (case[k] for k in ("L", "B", "N", "H", "Hkv", "D", "Tc"))
    path, n = _append_path(case)
    s.update(qkv=randn(L, B, N, (H + 2 * Hkv) * D, dtype=dt),
             k=randn(L, B, Hkv, Tc, D, dtype=dt), v=randn(L, B, Hkv, Tc, D, dtype=dt),
             path=_i32(path), n_path=_i32(n),
             lens=_i32([l for l in _spread(B, 0, Tc - N)]))
    return s


# ---------------------------------------------------------------------- one pass
def run(state):
    """One pass through the state's operator; its outputs."""
    op = state["case"]["op"]
    if own:
        import decoder_only_lm_b200 as g
        c = state["case"]
        if op == "attention":
            return g.tree_attention(state["qkv"], state["k"], state["v"], state["lens"], c["H"],
                                    parent=state["parent"], counts=state["counts"])
        if op == "verify":
            return g.tree_verify(state["logits"], c["V"], state["tokens"], state["uniform"],
                                 temperature=c["temperature"], top_k=c["top_k"], top_p=c["top_p"],
                                 parent=state["parent"], draft_logits=state["draft"],
                                 counts=state["counts"])
        new_lens = g.kv_append(state["qkv"], state["k"], state["v"], state["lens"],
                               path=state["path"], n_path=state["n_path"])
        return state["k"], state["v"], new_lens
    return {"attention": _plain_attention, "verify": _plain_verify,
            "append": _plain_append}[op](state)


def _chain(B, N):
    return torch.arange(-1, N - 1, device="cuda", dtype=torch.int32).expand(B, N)


def _plain_attention(s):
    """out = softmax(q k^T / sqrt(D)) v over the cached positions t < lens[b]
    and the nodes on the query node's path to the root (itself included), and
    the log of the softmax's normaliser; rows of nodes >= counts[b] are 0."""
    c = s["case"]
    B, N, H, Hkv, D = (c[k] for k in ("B", "N", "H", "Hkv", "D"))
    G, Tc = H // Hkv, s["k"].shape[2]
    x = s["qkv"].float()
    q = x[..., :H * D].view(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, D)
    kn = x[..., H * D:(H + Hkv) * D].view(B, N, Hkv, D).transpose(1, 2)
    vn = x[..., (H + Hkv) * D:].view(B, N, Hkv, D).transpose(1, 2)
    parent = s["parent"] if s["parent"] is not None else _chain(B, N)
    counts = s["counts"] if s["counts"] is not None else torch.full((B,), N, device="cuda")
    # sees[b, i, j]: node j is on node i's path to the root, by doubling the
    # reach of (self or parent)
    ids = torch.arange(N, device="cuda")
    sees = ((ids[None, None] == parent[..., None]) | (ids[:, None] == ids)).float()
    for _ in range((N - 1).bit_length()):
        sees = ((sees @ sees) > 0).float()
    sees = sees > 0
    cached = torch.arange(Tc, device="cuda")[None] < s["lens"][:, None]
    scale = 1.0 / math.sqrt(D)
    sc = (q * scale) @ s["k"].float().transpose(2, 3)
    sc = sc.masked_fill(~cached[:, None, None], float("-inf"))
    sn = ((q * scale) @ kn.transpose(2, 3)).view(B, Hkv, G, N, N)
    sn = sn.masked_fill(~sees[:, None, None], float("-inf")).view(B, Hkv, G * N, N)
    m = torch.maximum(sc.amax(3), sn.amax(3))[..., None]
    pc, pn = torch.exp(sc - m), torch.exp(sn - m)
    z = pc.sum(3, keepdim=True) + pn.sum(3, keepdim=True)
    v = s["v"].float().masked_fill(~cached[:, None, :, None], 0.0)
    o = (pc @ v + pn @ vn) / z
    lse = (m + torch.log(z)).view(B, H, N)
    o = o.view(B, Hkv, G, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, H * D)
    live = torch.arange(N, device="cuda")[None] < counts[:, None]
    o = o.masked_fill(~live[..., None], 0.0).to(s["qkv"].dtype)
    return o, lse.masked_fill(~live[:, None], 0.0)


def _weights(z, temperature, top_k, top_p):
    """Integer weights (held in float64) of rows of logits: rint(2^36 p) with
    p = exp((z - max z) / temperature), zero outside the top-k and top-p cuts;
    ids ordered by logit, the smaller id first among equal ones."""
    z = z.double()
    z = torch.where(torch.isnan(z), float("-inf"), z)
    top = z.amax(1, keepdim=True)
    if temperature == 0.0:
        first = (z == top).to(torch.int32).argmax(1, keepdim=True)
        return torch.zeros_like(z).scatter_(1, first, 2.0 ** 36)
    p = torch.exp((z - top) / temperature)
    w = torch.round(torch.where(z == top, 1.0, p) * 2.0 ** 36)
    if top_k == 0 and top_p >= 1.0:
        return w
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    if top_k > 0:
        ws[:, top_k:] = 0.0
    cum = ws.cumsum(1)
    if top_p < 1.0:
        ws = torch.where(cum - ws < top_p * cum[:, -1:], ws, 0.0)
    return torch.zeros_like(w).scatter_(1, order, ws)


def _plain_verify(s):
    """Node by node in order (children have larger ids than their parents): a
    child of the node that the walk stands at is accepted when
    u * q(token) < p(token), with p what is left of the target's distribution
    after the rejected siblings; the walk ends with a draw from what is left."""
    c = s["case"]
    B, N, V = c["B"], c["N"], c["V"]
    T, top_p = float(np.float32(c["temperature"])), float(np.float32(c["top_p"]))
    parent = s["parent"] if s["parent"] is not None else _chain(B, N)
    counts = s["counts"] if s["counts"] is not None else torch.full((B,), N, device="cuda")
    rows = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    path = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    n = torch.ones(B, dtype=torch.long, device="cuda")
    u = s["uniform"].double().clamp(0.0, 1.0)
    W = _weights(s["logits"][:, 0, :V], T, c["top_k"], top_p)
    X = _weights(s["draft"][:, 0, :V], T, c["top_k"], top_p) if c["draft"] else None
    for i in range(1, N):
        child = (parent[:, i] == cur) & (i < counts)
        tok = s["tokens"][:, i].long()
        S = W.sum(1)
        wt = W[rows, tok]
        if c["draft"]:
            f = S / X.sum(1)
            lhs = u[:, i] * (X[rows, tok] * f)
            left = (W - torch.round(X * f[:, None])).clamp(min=0.0)
        else:
            lhs = u[:, i] * S
            left = W.clone()
            left[rows, tok] = 0.0
        yes = child & (lhs < wt)
        no = child & ~(lhs < wt) & (left.sum(1) > 0)
        W = torch.where(no[:, None], left, W)
        W = torch.where(yes[:, None], _weights(s["logits"][:, i, :V], T, c["top_k"], top_p), W)
        if c["draft"]:
            X = torch.where(yes[:, None], _weights(s["draft"][:, i, :V], T, c["top_k"], top_p), X)
        cur = torch.where(yes, i, cur)
        at = n.clamp(max=N - 1)
        path[rows, at] = torch.where(yes, i, path[rows, at].long()).int()
        n = n + yes.long()
    cum = W.cumsum(1)
    over = cum > u[:, :1] * cum[:, -1:]
    last = V - 1 - (W > 0).flip(1).to(torch.int32).argmax(1)
    nxt = torch.where(over.any(1), over.to(torch.int32).argmax(1), last)
    return path, n.int(), nxt.int()


def _plain_append(s):
    """cache row lens[b] + r of every layer and head = the key (value) of node
    path[b][r], r < n_path[b]; the new lengths."""
    c = s["case"]
    L, B, N, H, Hkv, D = (c[k] for k in ("L", "B", "N", "H", "Hkv", "D"))
    r = torch.arange(N, device="cuda")
    b, r = torch.nonzero(r[None] < s["n_path"][:, None], as_tuple=True)
    node = s["path"][b, r].long()
    slot = s["lens"][b].long() + r
    rows = s["qkv"][:, b, node]
    # indexed like this the rows come first: [rows, L, Hkv, D]
    s["k"][:, b, :, slot] = rows[..., H * D:(H + Hkv) * D].view(L, -1, Hkv, D).transpose(0, 1)
    s["v"][:, b, :, slot] = rows[..., (H + Hkv) * D:].view(L, -1, Hkv, D).transpose(0, 1)
    return s["k"], s["v"], s["lens"] + s["n_path"]


# ---------------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    """What run returns, from the definitions in 64 bits, one sequence at a time."""
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    if case["op"] == "verify":
        return _exact_verify(case, s)
    k, v = s["k"].double(), s["v"].double()
    path, n, lens = (s[x].tolist() for x in ("path", "n_path", "lens"))
    kd = case["Hkv"] * case["D"]
    x = s["qkv"].double()
    for b in range(case["B"]):
        for r in range(n[b]):
            row = x[:, b, path[b][r]]
            k[:, b, :, lens[b] + r] = row[:, -2 * kd:-kd].unflatten(1, (case["Hkv"], case["D"]))
            v[:, b, :, lens[b] + r] = row[:, -kd:].unflatten(1, (case["Hkv"], case["D"]))
    return k, v, torch.tensor([l + m for l, m in zip(lens, n)], dtype=torch.int32)


def _exact_attention(case, s):
    B, N, H, Hkv, D = (case[k] for k in ("B", "N", "H", "Hkv", "D"))
    out = torch.zeros((B, N, H * D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, H, N), dtype=torch.float64, device="cuda")
    par, cnt, lens = _parents(case), _counts(case), _spread(B, case["lo"], case["hi"])
    for b in range(B):
        n, l = cnt[b], lens[b]
        anc = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):
            j = i
            while j >= 0:
                anc[i, j] = True
                j = int(par[b, j])
        anc = torch.cat([torch.ones((n, l), dtype=torch.bool), anc], 1).cuda()
        x = s["qkv"][b, :n].double().view(n, H + 2 * Hkv, D)
        for h in range(H):
            hk = h * Hkv // H
            keys = torch.cat([s["k"][b, hk, :l].double(), x[:, H + hk]])
            vals = torch.cat([s["v"][b, hk, :l].double(), x[:, H + Hkv + hk]])
            a = torch.einsum("id,jd->ij", x[:, h], keys) / D ** 0.5
            a = torch.where(anc, a, float("-inf"))
            lse[b, h, :n] = torch.logsumexp(a, 1)
            out[b, :n, h * D:(h + 1) * D] = torch.softmax(a, 1) @ vals
    return out, lse


def _exact_weights(z, T, top_k, top_p):
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    V = len(z)
    w = np.zeros(V, np.int64)
    if T == 0.0:
        w[int(np.argmax(z))] = 2 ** 36
        return w
    with np.errstate(invalid="ignore"):
        p = np.where(z == z.max(), 1.0, np.exp((z - z.max()) / T))
    w = np.rint(p * 2.0 ** 36).astype(np.int64)
    if top_k == 0 and top_p >= 1.0:
        return w
    order = np.lexsort((np.arange(V), -z))
    if top_k:
        w[order[top_k:]] = 0
    if top_p < 1.0:
        c = np.cumsum(w[order])
        stop = int(np.argmax(c.astype(np.float64) >= top_p * float(c[-1])))
        w[order[stop + 1:]] = 0
    return w


def _exact_verify(case, s):
    B, N, V = case["B"], case["N"], case["V"]
    T, top_p = float(np.float32(case["temperature"])), float(np.float32(case["top_p"]))
    par, cnt = _parents(case), _counts(case)
    tokens, u = s["tokens"].cpu().numpy(), s["uniform"].cpu().numpy().astype(np.float64)
    path = np.full((B, N), -1, np.int32)
    n, nxt = np.zeros(B, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        cur, walk = 0, [0]
        while True:
            row = lambda t: _exact_weights(t[b, cur, :V].cpu().numpy(), T, case["top_k"], top_p)
            w = row(s["logits"])
            kids = [i for i in range(cur + 1, cnt[b]) if par[b, i] == cur]
            x = row(s["draft"]) if case["draft"] and kids else None
            moved = False
            for i in kids:
                tok = tokens[b, i]
                tot = float(w.sum())
                if x is None:
                    lhs = u[b, i] * tot
                    left = w.copy()
                    left[tok] = 0
                else:
                    f = tot / float(x.sum())
                    lhs = u[b, i] * (float(x[tok]) * f)
                    left = np.maximum(w - np.rint(x * f).astype(np.int64), 0)
                if lhs < float(w[tok]):
                    cur, moved = i, True
                    walk.append(i)
                    break
                if left.sum() > 0:
                    w = left
            if not moved:
                break
        cum = np.cumsum(w).astype(np.float64)
        over = np.nonzero(cum > u[b, 0] * cum[-1])[0]
        nxt[b] = over[0] if len(over) else np.nonzero(w)[0][-1]
        path[b, :len(walk)] = walk
        n[b] = len(walk)
    return path, n, nxt
