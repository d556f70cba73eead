"""Decoding with drafted tokens on the GPU: tree attention, verification and the
cache store against plain implementations in 64 bits, and together against
ordinary greedy generation."""
import numpy as np
import pytest

import synth
from tests import tree_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import torch
    assert torch.cuda.is_available()
    import decoder_only_lm_b200 as g
    return g


def cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Random activations, caches and trees; what the call returns is compared
    row by row with the plain implementation."""

    def __init__(self, dtype, B, N, H, Hkv, D, Tc, lens, seed=0, tree="random", counts=None,
                 pad=0, qscale=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.B, self.N, self.H, self.Hkv, self.D, self.Tc = B, N, H, Hkv, D, Tc
        W = (H + 2 * Hkv) * D
        buf = torch.from_numpy(rng.normal(size=(B, N, W + pad)).astype(np.float32))
        buf[..., :H * D] *= qscale
        self.buf = buf.cuda().to(self.dt)
        self.qkv = self.buf[..., :W]
        self.k = torch.from_numpy(rng.normal(size=(B, Hkv, Tc, D)).astype(np.float32)).cuda().to(self.dt)
        self.v = torch.from_numpy(rng.normal(size=(B, Hkv, Tc, D)).astype(np.float32)).cuda().to(self.dt)
        self.lens = np.asarray(lens, np.int32)
        self.counts = None if counts is None else np.asarray(counts, np.int32)
        if tree == "chain":
            self.par = None
        elif tree == "forest":
            self.par = np.stack([tree_ref.random_tree(rng, N, roots=min(N, 3)) for _ in range(B)])
        elif tree == "star":
            self.par = np.where(np.arange(N) == 0, -1, 0).astype(np.int32)[None].repeat(B, 0)
        else:
            self.par = np.stack([tree_ref.random_tree(rng, N, spread=N) for _ in range(B)])

    def args(self):
        return dict(parent=None if self.par is None else cuda(self.par),
                    counts=None if self.counts is None else cuda(self.counts))

    def call(self, g, **kw):
        return g.tree_attention(self.qkv, self.k, self.v, cuda(self.lens), self.H, **self.args(), **kw)

    def check(self, out, lse, seqs=None):
        """Rounding bounds.  With u = 2^-23 (twice the half step of fp32, for
        accumulation that truncates) and A = max sum |q k| / sqrt(D): a score is
        off by at most (D + 8) u A (products, sum, scale, log2 factor), p by
        twice that relative to the normalised value, sums over n keys by n u, and
        the running rescales and merges by a few u each (64 u).  bf16 adds half a
        step, 2^-8, of the probabilities' rounding and of the output's.  exp2f:
        2 ulp, in the 64."""
        out = out.double().cpu().numpy()
        lse = lse.double().cpu().numpy()
        H, Hkv, D = self.H, self.Hkv, self.D
        u = 2.0 ** -23
        bf = 2.0 ** -8 if self.out_is_bf16() else 0.0
        for b in range(self.B) if seqs is None else seqs:
            n = self.N if self.counts is None else int(self.counts[b])
            L = int(self.lens[b])
            if n == 0:
                continue
            x = self.qkv[b, :n].double().cpu().numpy()
            q = x[:, :H * D].reshape(n, H, D)
            k = x[:, H * D:(H + Hkv) * D].reshape(n, Hkv, D)
            v = x[:, (H + Hkv) * D:].reshape(n, Hkv, D)
            par = np.arange(-1, n - 1) if self.par is None else self.par[b, :n]
            o, ls, mag, A = tree_ref.attention(q, k, v, self.k[b, :, :L].double().cpu().numpy(),
                                               self.v[b, :, :L].double().cpu().numpy(), par)
            rel = 2 * (D + 8) * u * A + (L + n + 64) * u
            tol = (rel + bf) * mag + (bf + u) * (np.abs(o) + (rel + bf) * mag)
            err = np.abs(out[b, :n].reshape(n, H, D) - o)
            assert (err <= tol).all(), (b, float((err / tol).max()))
            err = np.abs(lse[b, :, :n] - ls)
            tol = (D + 8) * u * A + (L + n + 64) * u + 4 * u * np.abs(ls)
            assert (err <= tol).all(), (b, float((err / tol).max()))

    def out_is_bf16(self):
        import torch
        return self.dt == torch.bfloat16


HEADS = [(2, 2, 16), (4, 2, 32), (3, 3, 64), (8, 2, 64), (6, 1, 128), (4, 4, 128)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", HEADS)
@pytest.mark.parametrize("N,tree", [(1, "chain"), (2, "random"), (7, "random"), (17, "forest"),
                                    (33, "chain"), (64, "random")])
def test_attention_ragged(g, dtype, H, Hkv, D, N, tree):
    """Lengths around the tiles' borders, 0 and the whole cache among them;
    ragged node counts, 0 among them; rows beyond them stay as they were."""
    import torch
    lens = [0, 1, 63, 64, 65, 127, 200, 129, 256, 300]
    B, Tc = len(lens), 300
    rng = np.random.default_rng(N)
    counts = rng.integers(1, N + 1, size=B)
    counts[0], counts[4], counts[7] = N, 0, N
    c = Case(dtype, B, N, H, Hkv, D, Tc, lens, seed=H * D + N, tree=tree, counts=counts, pad=8)
    out = torch.full((B, N, H * D), 7.0, dtype=c.dt, device="cuda")
    lse = torch.full((B, H, N), 7.0, device="cuda")
    c.call(g, out=out, lse=lse)
    c.check(out, lse)
    for b in range(B):
        assert (out[b, counts[b]:] == 7).all() and (lse[b, :, counts[b]:] == 7).all()
    first = out.clone(), lse.clone()
    c.call(g, out=out, lse=lse)
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)  # repeatable
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,N,H,Hkv,D,lens,tree", [
    (1, 1, 12, 12, 64, [5000], "chain"),         # one row split over many CTAs
    (1, 5, 2, 1, 64, [9001], "random"),
    (2, 256, 2, 2, 64, [513, 0], "chain"),       # a whole chunk of a prompt, and the first one
    (2, 256, 4, 1, 64, [100, 1025], "random"),   # 1024 rows on one cache head
    (1, 130, 4, 2, 128, [700], "forest"),
    (3, 256, 1, 1, 16, [40, 2000, 0], "star"),
    (40, 3, 2, 2, 64, list(range(0, 400, 10)), "random"),  # more sequences than a warp scans at once
    (2, 64, 16, 2, 128, [1500, 77], "random"),
])
def test_attention_sizes(g, dtype, B, N, H, Hkv, D, lens, tree):
    c = Case(dtype, B, N, H, Hkv, D, max(max(lens), 1), lens, seed=N + D, tree=tree)
    c.check(*c.call(g))
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_many_pieces_a_cta(g, dtype, D):
    """Short segments, several of them in every CTA's run, each ending in a
    partly filled tile and the nodes' own."""
    lens = [(37 * b) % 911 for b in range(24)]
    c = Case(dtype, 24, 20, 24, 12, D, 911, lens, seed=D, tree="random",
             counts=[1 + (7 * b) % 20 for b in range(24)])
    c.check(*c.call(g))
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("N", [6, 40])
def test_attention_peaked_rows(g, dtype, D, N):
    """Scores of a large spread: running maxima that jump, probabilities that
    vanish."""
    c = Case(dtype, 3, N, 4, 2, D, 700, [700, 333, 64], seed=D, qscale=8.0)
    c.check(*c.call(g))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("N", [9, 70])
def test_attention_ignores_what_it_may_not_see(g, dtype, D, N):
    """Infinities and NaN behind the cached length, in nodes beyond the count
    and in nodes off the path stay out of every other row."""
    import torch
    lens, counts = [130, 0, 61], [N - 2, N, N - 1]
    c = Case(dtype, 3, N, 4, 2, D, 200, lens, seed=D + N, counts=counts, tree="random")
    clean = c.call(g)
    H, Hkv = c.H, c.Hkv
    bad = 3  # a node with no finite key or value, except for those below it
    for b in range(3):
        c.k[b, :, lens[b]:], c.v[b, :, lens[b]:] = float("nan"), float("inf")
        c.buf[b, counts[b]:] = float("nan")
        c.qkv[b, bad, H * D:(H + Hkv) * D] = float("inf")
        c.qkv[b, bad, (H + Hkv) * D:] = float("nan")
    out, lse = c.call(g)
    for b in range(3):
        below = tree_ref.ancestors(c.par[b])[:counts[b], bad]
        keep = torch.from_numpy(~below).cuda()
        assert torch.equal(out[b, :counts[b]][keep], clean[0][b, :counts[b]][keep])
        assert torch.equal(lse[b, :, :counts[b]][:, keep], clean[1][b, :, :counts[b]][:, keep])
        assert torch.isfinite(out[b, :counts[b]][keep]).all()
        # a node that sees the NaN values says so
        assert not torch.isfinite(out[b, bad]).any()
    assert g.device_error() == 0


def test_attention_far_offsets(g):
    """Sequences whose cache rows start past 2^31 elements."""
    import torch
    Hkv, Tc, D = 8, 1 << 20, 128
    c = Case("bf16", 3, 5, 8, 8, D, 1, [1, 1, 1], seed=1)
    c.Tc, c.lens = Tc, np.array([3, 130, 257], np.int32)
    c.k = torch.zeros((3, Hkv, Tc, D), dtype=torch.bfloat16, device="cuda")
    c.v = torch.zeros((3, Hkv, Tc, D), dtype=torch.bfloat16, device="cuda")
    c.k[:, :, :300] = torch.randn((3, Hkv, 300, D), device="cuda").bfloat16()
    c.v[:, :, :300] = torch.randn((3, Hkv, 300, D), device="cuda").bfloat16()
    out = c.call(g)
    c.check(*out)
    new = g.kv_append(c.qkv[None], c.k[None], c.v[None], cuda(c.lens))
    assert new.tolist() == [8, 135, 262]
    want = c.qkv[2, :, 8 * D:16 * D].view(5, 8, D).transpose(0, 1)
    assert torch.equal(c.k[2, :, 257:262], want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_bad_lengths_and_parents(g, dtype):
    """A length or count out of range leaves its sequence alone, a bad parent
    counts as -1, both are reported once."""
    import torch
    c = Case(dtype, 5, 6, 2, 2, 64, 100, [50, -1, 101, 20, 30], seed=3, counts=[6, 6, 6, 7, 6])
    c.par[4, 2], c.par[4, 3] = 5, -7
    out = torch.full((5, 6, 128), 7.0, dtype=c.dt, device="cuda")
    lse = torch.full((5, 2, 6), 7.0, device="cuda")
    c.call(g, out=out, lse=lse)
    assert g.device_error() == g.ERR_ARG
    assert (out[1:4] == 7).all() and (lse[1:4] == 7).all()
    c.par[4, 2], c.par[4, 3] = -1, -1
    c.check(out, lse, seqs=[0, 4])
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [1, 6, 64])
def test_attention_stream_and_graph(g, dtype, N):
    """On another stream, and captured once then replayed with other lengths,
    trees and contents."""
    import torch
    c = Case(dtype, 4, N, 4, 4, 64, 600, [10, 300, 599, 64], seed=5, counts=[N, 1, N, 1])
    want = c.call(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.call(g, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    lens, counts, par = cuda(c.lens), cuda(c.counts), cuda(c.par)
    out = torch.zeros_like(want[0])
    lse = torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.tree_attention(c.qkv, c.k, c.v, lens, 4, parent=par, counts=counts, out=out, lse=lse)
    graph.replay()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    d = Case(dtype, 4, N, 4, 4, 64, 600, [600, 0, 1, 331], seed=6, counts=[1, N, N, 0])
    c.qkv.copy_(d.qkv), c.k.copy_(d.k), c.v.copy_(d.v)
    lens.copy_(cuda(d.lens)), counts.copy_(cuda(d.counts)), par.copy_(cuda(d.par))
    graph.replay()
    d.check(out, lse)
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,H,Hkv,D", [(1, 4, 4, 64), (12, 4, 2, 64), (60, 4, 2, 128), (20, 2, 2, 16)])
def test_attention_calls_at_once(g, dtype, N, H, Hkv, D):
    """Calls on two streams at the same time, each with its own inputs."""
    import torch
    cases = [Case(dtype, 6, N, H, Hkv, D, 2000, [2000, 3, 900, 0, 64, 1500], seed=s) for s in (1, 2)]
    args = [dict(c.args()) for c in cases]
    lens = [cuda(c.lens) for c in cases]
    call = lambda i, **kw: g.tree_attention(cases[i].qkv, cases[i].k, cases[i].v, lens[i], H,
                                            **args[i], **kw)
    want = [call(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(i, stream=streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("N,G", [(1, 1), (3, 2), (40, 1)])
def test_attention_tiny_caches(g, dtype, D, N, G):
    """Caches of fewer rows than a tile, empty and full ones."""
    for Tc, lens in ((1, [1]), (3, [0]), (5, [5, 2])):
        c = Case(dtype, len(lens), N, G, 1, D, Tc, lens, seed=Tc + N)
        c.check(*c.call(g))
    assert g.device_error() == 0


def test_attention_matches_the_causal_forward(g):
    """A chain behind an empty cache is the causal attention of training."""
    import torch
    for dt, B, T, H, D in ((torch.float32, 2, 100, 3, 32), (torch.bfloat16, 2, 200, 4, 64)):
        qkv = torch.randn((B, T, 3 * H * D), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dt)
        a, la = g.attention_fwd(qkv, H)
        kc = torch.zeros((B, H, 1, D), dtype=dt, device="cuda")
        b, lb = g.tree_attention(qkv, kc, kc, torch.zeros(B, dtype=torch.int32, device="cuda"), H)
        # two bf16 outputs, each within half a step plus the rounding of its
        # probabilities (2^-8 of a mean of |v| that stays below 4)
        tol = 1e-5 if dt == torch.float32 else 4 * 2.0 ** -8 * 4
        assert (a.float() - b.float()).abs().max() <= tol
        assert (la - lb).abs().max() <= 1e-4


# ---------------------------------------------------------------- verification
SETTINGS = [(0.0, 0, 1.0), (1.0, 0, 1.0), (0.8, 0, 0.9), (1.0, 50, 1.0), (1.3, 40, 0.7),
            (0.5, 1, 0.9), (0.7, 0, 0.05), (2.0, 3000, 0.95)]


def check_verify(g, logits, tokens, par, u, T, k, p, draft=None, counts=None, pad=0):
    B, N, V = logits.shape
    padded = lambda a: None if a is None else cuda(
        np.concatenate([a, np.full((B, N, pad), 100, np.float32)], 2))
    got = g.tree_verify(padded(logits), V, cuda(tokens), cuda(u), T, k, p,
                        parent=None if par is None else cuda(par), draft_logits=padded(draft),
                        counts=None if counts is None else cuda(np.asarray(counts, np.int32)))
    path, n, nxt = (t.cpu().numpy() for t in got)
    for b in range(B):
        c = N if counts is None else counts[b]
        if c == 0:
            assert n[b] == 0 and nxt[b] == -1 and (path[b] == -1).all()
            continue
        pb = np.arange(-1, c - 1) if par is None else par[b, :c]
        want, nw = tree_ref.verify(logits[b, :c], None if draft is None else draft[b, :c],
                                   tokens[b, :c], pb, u[b, :c], T, k, p)
        assert path[b, :n[b]].tolist() == want and (path[b, n[b]:] == -1).all(), b
        assert nxt[b] == nw, b
    return path, n, nxt


def make_verify(seed, B, N, V, draft, scale=4.0, tree="random", T=1.0):
    """Peaked rows, drafts near them, drafted tokens that are often accepted."""
    rng = np.random.default_rng(seed)
    z = (scale * rng.normal(size=(B, N, V))).astype(np.float32)
    y = (z + rng.normal(size=z.shape)).astype(np.float32)
    par = None if tree == "chain" else np.stack([tree_ref.random_tree(rng, N) for _ in range(B)])
    tok = np.zeros((B, N), np.int32)
    for b in range(B):
        for i in range(1, N):
            row = y[b, i - 1 if par is None else max(par[b, i], 0)].astype(np.float64)
            e = np.exp((row - row.max()) / max(T, 0.3))
            tok[b, i] = rng.choice(V, p=e / e.sum())
    return z, (y if draft else None), tok, par, rng.random((B, N)).astype(np.float32)


@pytest.mark.parametrize("setting", SETTINGS)
@pytest.mark.parametrize("V,pad", [(50257, 47), (1000, 0), (37, 3)])
@pytest.mark.parametrize("draft", [False, True], ids=["guess", "draft"])
def test_verify_matches(g, setting, V, pad, draft):
    T, k, p = setting
    B, N = (3, 9) if V > 10000 else (12, 24)
    z, y, tok, par, u = make_verify(V + k, B, N, V, draft, T=T)
    counts = [N] * B
    counts[1], counts[2] = 1, 0
    _, n, _ = check_verify(g, z, tok, par, u, T, k, p, draft=y, counts=counts, pad=pad)
    assert g.device_error() == 0
    if V < 10000 and T <= 1:
        assert n.max() > 1  # some drafts are accepted (flat rows, T > 1, accept few guesses)


@pytest.mark.parametrize("draft", [False, True], ids=["guess", "draft"])
def test_verify_chain_and_sizes(g, draft):
    """Chains; vocabularies of one id, of fewer ids than CTAs, and the largest."""
    for V, B, N in ((1, 4, 5), (2, 9, 6), (5, 30, 16), (13, 30, 256), (65536, 1, 3)):
        z, y, tok, par, u = make_verify(V, B, N, V, draft, tree="chain", scale=1.0)
        check_verify(g, z, tok, par, u, 1.0, 0, 1.0, draft=y)
        check_verify(g, z, tok, par, u, 0.9, 3, 0.8, draft=y)
    z, y, tok, par, u = make_verify(3, 150, 8, 300, draft)
    check_verify(g, z, tok, par, u, 1.0, 0, 0.9, draft=y)
    assert g.device_error() == 0


@pytest.mark.parametrize("draft", [False, True], ids=["guess", "draft"])
@pytest.mark.parametrize("setting", [(0.0, 0, 1.0), (1.0, 0, 1.0), (1.0, 0, 0.5), (1.0, 700, 1.0),
                                     (0.7, 901, 0.33), (1.0, 1, 1.0), (1.0, 40, 1.0),
                                     (0.7, 256, 0.33)])
def test_verify_special_rows(g, draft, setting):
    """Equal logits in mass, NaN and infinities, the same token proposed twice,
    tokens out of range, numbers at the ends of [0, 1) and outside, a node that
    hangs on nothing."""
    T, k, p = setting
    B, N, V = 10, 12, 1500
    z, y, tok, par, u = make_verify(11, B, N, V, True, scale=2.0)
    z[0] = 0.0                                # all equal
    z[1, :, :700] = z[1, :, 700:701]          # many equal to one value
    z[2, :, 5:900] = -np.inf
    z[3, :, 3::2] = np.nan
    z[4, :, 17] = np.inf
    z[5, :, 17] = z[5, :, 20] = np.inf
    z[6] = -np.inf
    z[7, :, ::2], z[7, :, 1::2] = 0.0, -0.0   # equal, in spite of their signs
    y[0], y[7] = z[0], 0.0
    y[8] = z[8]                               # the draft is the target
    par[:, 1:6] = 0                           # five children of the root
    tok[:, 2] = tok[:, 1]
    tok[:, 4] = V
    tok[:, 5] = -3
    par[9, 6] = -1
    u[3], u[4], u[5] = 0.0, np.nextafter(np.float32(1), np.float32(0)), 1.0
    u[6], u[8] = 1.5, -0.5
    check_verify(g, z, tok, par, u, T, k, p, draft=y if draft else None)
    assert g.device_error() == 0


@pytest.mark.parametrize("draft", [False, True], ids=["guess", "draft"])
@pytest.mark.parametrize("k,p", [(0, 1.0), (0, 0.9), (40, 0.9)])
@pytest.mark.parametrize("T", [1e-30, 1e-7, 0.8, 1e20])
def test_verify_extreme_logits(g, draft, k, p, T):
    """Logits whose fp32 steps are coarser than the temperature, rows masked with
    the type's lowest value, temperatures at the ends of their range."""
    B, N, V = 8, 6, 1500
    z, y, tok, par, u = make_verify(13, B, N, V, True, scale=2.0)
    low = np.finfo(np.float32).min
    z[0] = low
    z[1, :, 9:] = low
    z[2] = low
    z[2, :, ::3] = -np.inf
    z[3] *= np.float32(1e9)
    z[4] += np.float32(1e6)
    z[5] = np.where(z[5] > 1, np.float32(3.3e38), np.float32(-3.3e38))
    z[6] *= np.float32(1e-38)
    y[:4], y[5] = z[:4], z[5]
    par[:, 1:4] = 0
    check_verify(g, z, tok, par, u, T, k, p, draft=y if draft else None)
    assert g.device_error() == 0


@pytest.mark.parametrize("draft", [False, True], ids=["guess", "draft"])
@pytest.mark.parametrize("V,k,p", [(2, 1, 1.0), (300, 256, 0.9), (257, 256, 1.0), (300, 257, 0.9),
                                   (5000, 1, 0.5), (5000, 255, 1.0), (5000, 256, 0.7),
                                   (5000, 257, 0.7), (65536, 200, 0.95)])
def test_verify_top_k(g, draft, V, k, p):
    """Kept lists of all lengths: the best ids in one place, equal logits across
    the cut (in few places and in many), and fewer ids that have a weight."""
    B, N = 7, 5
    z, y, tok, par, u = make_verify(V + k, B, N, V, True, scale=3.0)
    z[1] = -np.sort(-z[1], -1)                       # the first ids
    z[2] = np.round(z[2])                            # hundreds of equal ones
    z[3, :, ::2] = z[3].max(-1, keepdims=True)       # half of them equal and best
    z[4, :, 60:] = -np.inf
    z[5, :, :V - V // 9] = -3e38                     # a mask of low values
    y[1], y[3] = -np.sort(-y[1], -1), 0.0
    y[6] = z[6]
    par[:, 1:4] = 0
    check_verify(g, z, tok, par, u, 0.9, k, p, draft=y if draft else None, pad=3)
    assert g.device_error() == 0


@pytest.mark.parametrize("k,p", [(0, 1.0), (0, 0.9), (20, 0.9), (300, 1.0)])
def test_verify_calls_at_once_and_recorded(g, k, p):
    """Calls on two streams at the same time, and one recorded and replayed on
    other inputs, agree with calls alone."""
    import torch
    runs = []
    for seed in (21, 22):
        t = [cuda(x) for x in make_verify(seed, 40, 12, 2000, True)]
        runs.append((t, torch.cuda.Stream()))
    call = lambda t, **kw: g.tree_verify(t[0], 2000, t[2], t[4], 0.8, k, p, parent=t[3],
                                         draft_logits=t[1], **kw)
    want = [[x.clone() for x in call(t)] for t, _ in runs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [call(t, stream=s) for t, s in runs]
        torch.cuda.synchronize()
        for w, r in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(w, r))
    own = [x.clone() for x in runs[0][0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(own)
    for (t, _), w in zip(reversed(runs), reversed(want)):
        for x, y in zip(own, t):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(w, out))
    assert g.device_error() == 0


def test_verify_bad_counts_and_parents(g):
    z, y, tok, par, u = make_verify(2, 3, 6, 100, False)
    import torch
    par[2, 3] = 4  # not below its own index: never reached
    path, n, nxt = g.tree_verify(cuda(z), 100, cuda(tok), cuda(u), 1.0, 0, 1.0, parent=cuda(par),
                                 counts=cuda(np.array([-1, 7, 6], np.int32)))
    assert g.device_error() == g.ERR_ARG
    assert n.tolist()[:2] == [0, 0] and nxt.tolist()[:2] == [-1, -1] and (path[:2] == -1).all()
    want, nw = tree_ref.verify(z[2], None, tok[2], par[2], u[2], 1.0, 0, 1.0)
    assert path[2, :n[2]].tolist() == want and nxt[2] == nw
    assert g.device_error() == 0


def test_verify_keeps_the_target_distribution(g):
    """The first token after the root over many sequences, with children drawn
    from the draft: each id's share within five standard deviations of p."""
    import torch
    B, V, kids = 60000, 6, 3
    rng = np.random.default_rng(4)
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    z = torch.log(torch.tensor(p, dtype=torch.float32, device="cuda")).expand(B, kids + 1, V).contiguous()
    y = torch.log(torch.tensor(q, dtype=torch.float32, device="cuda")).expand(B, kids + 1, V).contiguous()
    tok = cuda(rng.choice(V, size=(B, kids + 1), p=q).astype(np.int32))
    par = cuda(np.tile(np.array([-1, 0, 0, 0], np.int32), (B, 1)))
    u = cuda(rng.random((B, kids + 1)).astype(np.float32))
    path, n, nxt = g.tree_verify(z, V, tok, u, 1.0, 0, 1.0, parent=par, draft_logits=y)
    first = torch.where(n > 1, tok.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], nxt)
    share = torch.bincount(first, minlength=V).cpu().numpy() / B
    assert (np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / B) + 1e-7).all(), (share, p)


def test_verify_stream_and_graph(g):
    import torch
    z, y, tok, par, u = make_verify(8, 4, 10, 3000, True)
    t = [cuda(a) for a in (z, y, tok, par, u)]
    want = g.tree_verify(t[0], 3000, t[2], t[4], 1.0, 0, 0.9, parent=t[3], draft_logits=t[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = g.tree_verify(t[0], 3000, t[2], t[4], 1.0, 0, 0.9, parent=t[3], draft_logits=t[1], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = g.tree_verify(t[0], 3000, t[2], t[4], 1.0, 0, 0.9, parent=t[3], draft_logits=t[1])
    z2, y2, tok2, par2, u2 = make_verify(9, 4, 10, 3000, True)
    for a, b in zip(t, (z2, y2, tok2, par2, u2)):
        a.copy_(cuda(b))
    graph.replay()
    for b in range(4):
        path, nw = tree_ref.verify(z2[b], y2[b], tok2[b], par2[b], u2[b], 1.0, 0, 0.9)
        assert out[0][b, :out[1][b]].tolist() == path and out[2][b] == nw


# ---------------------------------------------------------------- cache store
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("L,B,N,H,Hkv,D,Tc", [(1, 1, 1, 2, 2, 16, 4), (3, 5, 9, 4, 2, 64, 40),
                                              (2, 3, 256, 3, 1, 128, 300), (12, 2, 17, 12, 12, 64, 64)])
def test_append(g, dtype, L, B, N, H, Hkv, D, Tc):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator("cuda").manual_seed(N)
    W = (H + 2 * Hkv) * D
    qkv = torch.randn((L, B, N, W + 8), device="cuda", generator=gen).to(dt)[..., :W]
    k = torch.randn((L, B, Hkv, Tc, D), device="cuda", generator=gen).to(dt)
    v = torch.randn((L, B, Hkv, Tc, D), device="cuda", generator=gen).to(dt)
    rng = np.random.default_rng(N)
    n = rng.integers(0, N + 1, size=B).astype(np.int32)
    n[0] = N
    lens = np.array([rng.integers(0, Tc - n[b] + 1) for b in range(B)], np.int32)
    lens[-1] = Tc - n[-1]  # filled to the last row
    path = np.full((B, N), -1, np.int32)
    for b in range(B):
        path[b, :n[b]] = np.sort(rng.permutation(N)[:n[b]])
    for p, m in ((path, n), (None, n), (None, None)):
        if m is None and any(lens[b] + N > Tc for b in range(B)):
            continue
        wk, wv = k.clone(), v.clone()
        for b in range(B):
            for r in range(N if m is None else m[b]):
                row = qkv[:, b, r if p is None else int(p[b, r])]
                wk[:, b, :, lens[b] + r] = row[:, H * D:(H + Hkv) * D].view(L, Hkv, D)
                wv[:, b, :, lens[b] + r] = row[:, (H + Hkv) * D:].view(L, Hkv, D)
        new = g.kv_append(qkv, k, v, cuda(lens), path=None if p is None else cuda(p),
                          n_path=None if m is None else cuda(m))
        assert torch.equal(k, wk) and torch.equal(v, wv)
        assert new.tolist() == [int(lens[b] + (N if m is None else m[b])) for b in range(B)]
    assert g.device_error() == 0


def test_append_refuses_what_does_not_fit(g):
    import torch
    qkv = torch.randn((2, 4, 3, 192), device="cuda")
    k, v = torch.zeros((2, 4, 1, 8, 64), device="cuda"), torch.zeros((2, 4, 1, 8, 64), device="cuda")
    path = cuda(np.array([[0, 1, 2], [0, 1, 2], [0, 1, 2], [0, 3, -2]], np.int32))
    lens = cuda(np.array([6, -1, 2, 5], np.int32))
    new = g.kv_append(qkv, k, v, lens, path=path, n_path=cuda(np.array([3, 1, 4, 3], np.int32)))
    assert g.device_error() == g.ERR_ARG
    assert new.tolist() == [6, -1, 2, 8]
    assert (k[:, :3] == 0).all() and (v[:, :3] == 0).all()
    assert torch.equal(k[:, 3, 0, 5], qkv[:, 3, 0, 64:128])
    assert (k[:, 3, 0, 6:] == 0).all() and (k[:, 3, 0, :5] == 0).all()
    assert g.device_error() == 0


# ---------------------------------------------------------------- together
def test_decoding_with_drafts_matches_greedy_generation(g):
    """Greedy decoding with drafted trees through the op-level calls, over the
    weights of a model handle in fp32, against gpt2_generate_cached: the same
    tokens, in fewer steps.  The trees hold the right continuation with some
    tokens wrong, next to wrong siblings."""
    import torch
    L, Cc, H, V, max_T, B = 2, 64, 4, 512, 96, 3
    gm = g.GPT2(L, Cc, H, V, V, max_T, bf16=False, max_B=B, max_Tseq=max_T)
    named = synth.init_params(0, gm.shapes())
    for n in named:  # larger weights: greedy choices that differ from step to step
        named[n] = np.asarray(named[n], np.float32) * (8.0 if n.endswith(".w") and named[n].ndim == 2 else 1.0)
    gm.set_params(named)
    rng = np.random.default_rng(0)
    T0, n_new, D = 7, 60, Cc // H
    prompt = cuda(rng.integers(0, V, size=(B, T0)).astype(np.int32))
    want = gm.generate(prompt, n_new, temperature=0.0, cached=True).cpu().numpy()
    p = {n: cuda(np.asarray(a, np.float32)) for n, a in named.items()}

    def logits_of(tokens, parent, counts, lens, k, v, depth):
        """[B, N] node tokens through the model: logits and the layers' qkv."""
        N = tokens.shape[1]
        pos = (lens[:, None] + depth).clamp(max=max_T - 1).long()
        x = (p["wte"][tokens.long()] + p["wpe"][pos]).reshape(B * N, Cc).contiguous()
        rows = []
        for l in range(L):
            w = lambda s: p[f"h.{l}.{s}"]
            a = g.layernorm_fwd(x, w("ln1.w"), w("ln1.b"))[0]
            qkv = g.linear(g.LINEAR_BIAS, a, w("attn.qkv.w"), bias=w("attn.qkv.b")).view(B, N, 3 * Cc)
            rows.append(qkv)
            o, _ = g.tree_attention(qkv, k[l], v[l], lens, H, parent=parent, counts=counts)
            x = g.linear(g.LINEAR_RESIDUAL, o.view(B * N, Cc), w("attn.proj.w"), bias=w("attn.proj.b"), inp=x)
            a = g.layernorm_fwd(x, w("ln2.w"), w("ln2.b"))[0]
            h = g.linear(g.LINEAR_BIAS_GELU, a, w("mlp.fc.w"), bias=w("mlp.fc.b"))[0]
            x = g.linear(g.LINEAR_RESIDUAL, h, w("mlp.proj.w"), bias=w("mlp.proj.b"), inp=x)
        a = g.layernorm_fwd(x, p["lnf.w"], p["lnf.b"])[0]
        return g.matmul(a, p["wte"]).view(B, N, V), torch.stack(rows)

    k = torch.zeros((L, B, H, max_T, D), device="cuda")
    v = torch.zeros((L, B, H, max_T, D), device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    # the prompt but its last token, as one chunk
    chain = torch.arange(T0 - 1, device="cuda")
    _, rows = logits_of(prompt[:, :-1], None, None, lens, k, v, chain)
    lens = g.kv_append(rows, k, v, lens)
    have = [list(r) for r in prompt.cpu().numpy()]
    N, steps = 9, 0
    while min(len(h) for h in have) < T0 + n_new:
        steps += 1
        tok, par = np.zeros((B, N), np.int32), np.full((B, N), -1, np.int32)
        dep, cnt = np.zeros((B, N), np.int64), np.ones(B, np.int32)
        for b in range(B):
            tok[b, 0] = have[b][-1]
            if len(have[b]) >= T0 + n_new:
                cnt[b] = 0  # done: this sequence has no node
                continue
            spine, i = 0, 1
            while i < N:
                at = len(have[b]) + dep[b, spine]
                right = want[b, at] if at < T0 + n_new else 0
                # a wrong sibling first, then the right token (wrong now and then)
                tok[b, i], par[b, i], dep[b, i] = (right + 1) % V, spine, dep[b, spine] + 1
                if i + 1 < N:
                    tok[b, i + 1] = right if rng.random() < 0.8 else (right + 2) % V
                    par[b, i + 1], dep[b, i + 1] = spine, dep[b, spine] + 1
                    spine = i + 1
                i += 2
            room = T0 + n_new - len(have[b])  # the cache holds max_T positions
            cnt[b] = N if room > N else 1
        z, rows = logits_of(cuda(tok), cuda(par), cuda(cnt), lens, k, v, cuda(dep))
        u = torch.rand((B, N), device="cuda")
        path, n, nxt = g.tree_verify(z, V, cuda(tok), u, temperature=0.0, parent=cuda(par), counts=cuda(cnt))
        lens = g.kv_append(rows, k, v, lens, path=path, n_path=n)
        path, n, nxt = path.cpu().numpy(), n.cpu().numpy(), nxt.cpu().numpy()
        for b in range(B):
            if n[b]:
                have[b] += [int(tok[b, i]) for i in path[b, 1:n[b]]] + [int(nxt[b])]
    for b in range(B):
        assert have[b][:T0 + n_new] == want[b].tolist()
    assert steps < n_new  # several tokens a step
    assert g.device_error() == 0
    gm.close()


# ---------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("N", [1, 20, 48, 80])
@pytest.mark.parametrize("lens", [[700, 64, 1], [9000, 33, 95]])
def test_attention_infinite_cached_values(g, dtype, D, N, lens):
    """Infinite and NaN values in cache rows that every node sees: the same sums
    whatever the number of rows, an infinity of its sign, NaN for two signs or
    a NaN, and the other channels as without them."""
    c = Case(dtype, len(lens), N, 4, 4, D, max(lens), lens, seed=D + N)
    inf, nan = float("inf"), float("nan")
    clean = [t.clone() for t in c.call(g)]
    want = {}
    for b, L in enumerate(lens):
        # keys in either half of a tile, and the last one
        first, second, last = 5 % L, 40 % L, L - 1
        c.v[b, :, first, 2] = inf
        c.v[b, :, second, 3] = -inf
        c.v[b, :, first, 6] = c.v[b, :, last, 6] = inf
        c.v[b, :, last, 7] = nan
        want[b] = {2: inf, 3: -inf, 6: inf, 7: nan}
        if last != first:
            c.v[b, :, first, 9], c.v[b, :, last, 9] = inf, -inf
            want[b][9] = nan
    out, lse = c.call(g)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    for b in range(len(lens)):
        x = out[b].reshape(N, 4, D)
        y = clean[0][b].float().cpu().numpy().reshape(N, 4, D)
        for d, value in want[b].items():
            y[..., d] = value
        np.testing.assert_array_equal(x, y, err_msg=f"sequence {b}")
    np.testing.assert_array_equal(lse, clean[1].cpu().numpy())
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("N", [4, 9, 20, 40, 70])
def test_attention_node_with_infinite_values(g, dtype, D, N):
    """One infinite or NaN value of a node: rows that see it have it in that
    channel, and everything else is what it is with a finite value there."""
    c = Case(dtype, 3, N, 4, 2, D, 400, [300, 0, 77], seed=D + N, tree="random")
    out, lse = [t.clone() for t in c.call(g)]
    v = c.qkv[..., (c.H + c.Hkv) * D:].view(3, N, c.Hkv, D)
    want = out.float().view(3, N, c.H, D).cpu().numpy()
    see = np.stack([tree_ref.ancestors(par) for par in c.par])
    for node, channel, value in ((1, 5, float("inf")), (2, 6, -float("inf")), (N - 1, 0, float("nan"))):
        v[:, node, :, channel] = value
        for b in range(3):
            want[b, see[b, :, node], :, channel] = value
    got, got_lse = c.call(g)
    np.testing.assert_array_equal(got.float().view(3, N, c.H, D).cpu().numpy(), want)
    np.testing.assert_array_equal(got_lse.cpu().numpy(), lse.cpu().numpy())
    assert g.device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,B", [(1, 64), (12, 8), (80, 16)])
def test_attention_late_maximum(g, D, N, B):
    """A maximum in a tile's second half far above the first half's, where the
    values are: the probabilities of the first are rounded once (a second
    rounding takes about one sum in 500 out of check()'s bound)."""
    import torch
    c = Case("bf16", B, N, 4, 1, D, 130, [64 if b % 2 else 130 for b in range(B)], seed=D)
    q = c.qkv[..., :4 * D].view(B, N, 4, D)
    e = torch.eye(D, device="cuda")[:3].bfloat16()
    gen = torch.Generator("cuda").manual_seed(N)
    u = torch.rand((2, B, N, 4), device="cuda", generator=gen)
    q.zero_()
    q[..., 0], q[..., 1], q[..., 2] = 4 * u[0] + 0.1, 2 * u[1] + 4, 1
    # scores: key 0 of every sequence 0, key 1 a few bits below it, key 32 some 11
    # to 18 bits above, all others (the nodes too) 12 to 18 bits below
    c.k[:] = -100 * e[2]
    c.qkv[..., 4 * D:5 * D] = -100 * e[2]
    c.k[:, :, 0], c.k[:, :, 1], c.k[:, :, 32] = 0, -4 * e[0], (16 if D == 64 else 24) * e[1]
    c.v.zero_()
    c.qkv[..., 5 * D:] = 0
    c.v[:, :, 1] = 1 + torch.arange(D, device="cuda") / D
    c.check(*c.call(g))
    assert g.device_error() == 0


# ---------------------------------------------------------------- records of bad input
def test_bad_input_is_no_timeout(g):
    """What a call on drafted tokens finds out of range stays on record until it
    is asked for: calls on a handle neither fail for it nor clear it, and a wait
    that gives up is told apart from it."""
    import torch
    gm = g.GPT2(2, 64, 4, 512, 512, 64, bf16=True, max_B=2, max_Tseq=32)
    gm.set_params(synth.init_params(0, gm.shapes()))
    x = cuda(np.random.default_rng(0).integers(0, 512, size=(2, 32)).astype(np.int32))
    c = Case("bf16", 2, 6, 2, 2, 64, 100, [50, -1], seed=3)

    def attention():
        c.call(g)

    def parents():
        c.lens[1], c.par[1, 2] = 5, 4
        c.call(g)

    def verify():
        z, _, tok, par, u = make_verify(2, 1, 6, 100, False)
        g.tree_verify(cuda(z), 100, cuda(tok), cuda(u), parent=cuda(par), counts=cuda(np.array([9], np.int32)))

    def append():
        kv = torch.zeros((2, 1, 2, 2, 8, 64), device="cuda")
        g.kv_append(torch.zeros((1, 2, 3, 384), device="cuda"), kv[0], kv[1],
                    cuda(np.array([6, 0], np.int32)))

    for call in (attention, parents, verify, append):
        assert g.device_error() == 0
        call()
        assert np.isfinite(gm.forward_loss(x, x))
        gm.generate(x[:, :8].contiguous(), 3, temperature=0.0, cached=True)
        assert g.device_error() == g.ERR_ARG, call.__name__
        assert g.device_error() == 0
    c.lens[1] = -1
    attention()
    assert g.wait_selfcheck()
    assert g.device_error() == g.ERR_ARG
    assert g.device_error() == 0
    gm.close()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,D,B", [(1, 64, 5), (6, 16, 5), (6, 64, 5), (70, 64, 5), (40, 128, 40)])
@pytest.mark.parametrize("ragged", [False, True])
def test_attention_own_buffers_hold_zeros(g, dtype, N, D, B, ragged):
    """Rows without a node of the buffers that the call allocates are 0: beyond
    the counts, and of sequences whose length or count is out of range, also
    when no counts are given.  One buffer of the caller: its rows stay."""
    import torch
    lens = [50, -1, 101, 0, 30] * (B // 5)
    counts = [N, N, N, max(N - 3, 0), N + 1] * (B // 5) if ragged else None
    real = [N, 0, 0, max(N - 3, 0), 0] * (B // 5) if ragged else [N, 0, 0, N, N] * (B // 5)
    c = Case(dtype, B, N, 2, 2, D, 100, lens, seed=3, counts=counts)
    sizes = (B * N * 2 * D, c.dt), (B * 2 * N, torch.float32)

    def rows(out, lse, value, of_lse):
        for b in range(B):
            assert (out[b, real[b]:] == value).all() and (lse[b, :, real[b]:] == of_lse).all()

    # what the allocator gives out next is not 0
    old = [torch.full((n,), 7.0, dtype=t, device="cuda") for n, t in sizes for _ in range(3)]
    torch.cuda.synchronize()
    del old
    out, lse = c.call(g)
    rows(out, lse, 0, 0)
    assert g.device_error() == g.ERR_ARG
    good = [b for b in range(B) if real[b]]
    whole = c.counts
    c.counts = np.asarray(real, np.int32)
    c.check(out, lse, seqs=good)
    c.counts = whole
    mine = torch.full((B, N, 2 * D), 7.0, dtype=c.dt, device="cuda")
    got = c.call(g, out=mine)
    rows(mine, got[1], 7, 0)
    got = c.call(g, lse=torch.full((B, 2, N), 7.0, device="cuda"))
    rows(got[0], got[1], 0, 7)
    assert g.device_error() == g.ERR_ARG
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype,N", [("bf16", 40), ("bf16", 70), ("fp32", 5), ("fp32", 60)])
def test_attention_far_offsets_of_every_kernel(g, dtype, N):
    """Sequences whose cache rows start past 2^31 elements, in the kernels for
    more rows and for fp32."""
    import torch
    Hkv, Tc, D = 8, 1 << 20, 128
    c = Case(dtype, 3, N, 8, 8, D, 1, [1, 1, 1], seed=1)
    c.Tc, c.lens = Tc, np.array([3, 130, 257], np.int32)
    c.k = torch.empty((3, Hkv, Tc, D), dtype=c.dt, device="cuda")
    c.v = torch.empty((3, Hkv, Tc, D), dtype=c.dt, device="cuda")
    c.k[:, :, :300] = torch.randn((3, Hkv, 300, D), device="cuda").to(c.dt)
    c.v[:, :, :300] = torch.randn((3, Hkv, 300, D), device="cuda").to(c.dt)
    c.check(*c.call(g))
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("N", [1, 20, 48, 80])
def test_attention_infinite_keys(g, dtype, D, N):
    """An infinite key that every node sees: a score of -inf leaves its key out,
    one of +inf makes the row NaN, and other rows do not notice."""
    c = Case(dtype, 2, N, 4, 2, D, 700, [700, 90], seed=D + N)
    q = c.qkv[..., :c.H * D].view(2, N, c.H, D)
    q[..., 0] = 1 + q[..., 0].abs()
    q[:, ::2, :, 0] *= -1
    for b, key in ((0, 5), (0, 355), (1, 70)):
        c.k[b, :, key] = 0
        c.k[b, :, key, 0] = 1e30  # (far below all others for the rows with q < 0)
    out, lse = [t.clone() for t in c.call(g)]
    for b, key in ((0, 5), (0, 355), (1, 70)):
        c.k[b, :, key, 0] = float("inf")
    got, got_lse = c.call(g)
    want, want_lse = out.float().cpu().numpy(), lse.cpu().numpy()
    want[:, 1::2], want_lse[:, :, 1::2] = np.nan, np.nan
    np.testing.assert_array_equal(got.float().cpu().numpy(), want)
    np.testing.assert_array_equal(got_lse.cpu().numpy(), want_lse)
    assert g.device_error() == 0


@pytest.mark.parametrize("dtype,N", [("fp32", 7), ("bf16", 7), ("bf16", 64)])
def test_attention_recorded_with_own_buffers(g, dtype, N):
    """A recorded call that allocates its buffers: rows that have no node at a
    replay are 0, whatever an earlier one left there."""
    import torch
    c = Case(dtype, 4, N, 4, 4, 64, 300, [10, 300, 0, 64], seed=5, counts=[N] * 4)
    c.call(g)
    lens, counts, par = cuda(c.lens), cuda(c.counts), cuda(c.par)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = g.tree_attention(c.qkv, c.k, c.v, lens, 4, parent=par, counts=counts)
    for now in ([N] * 4, [1, 0, N, N - 2], [0] * 4, [N, 2, 1, 0]):
        c.counts = np.asarray(now, np.int32)
        counts.copy_(cuda(c.counts))
        graph.replay()
        c.check(out, lse)
        for b in range(4):
            assert (out[b, now[b]:] == 0).all() and (lse[b, :, now[b]:] == 0).all()
    assert g.device_error() == 0
