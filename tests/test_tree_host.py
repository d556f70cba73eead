"""Refusals of the calls on drafted tokens, all decided on the host before any
device call, and the rule of the verification on its plain implementation."""
import ctypes as C

import numpy as np
import pytest

from tests import tree_ref


@pytest.fixture(scope="module")
def g():
    import decoder_only_lm_b200 as g
    return g


P = C.c_void_p(4096)  # never dereferenced: the arguments are rejected first


def attention(g, **kw):
    a = dict(qkv=P, ld=192, k=P, v=P, lens=P, parent=None, counts=None, dtype=g.BF16, B=1, N=4, H=1,
             Hkv=1, D=64, Tc=16, out=P, ldo=64, lse=None, ws=P, wsb=1 << 40)
    a.update(kw)
    return g.lib.gpt2_tree_attention(a["qkv"], a["ld"], a["k"], a["v"], a["lens"], a["parent"],
                                     a["counts"], a["dtype"], a["B"], a["N"], a["H"], a["Hkv"],
                                     a["D"], a["Tc"], a["out"], a["ldo"], a["lse"], a["ws"],
                                     a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(qkv=None), dict(k=None), dict(v=None), dict(lens=None), dict(out=None), dict(ws=None),
    dict(dtype=7), dict(B=0), dict(N=0), dict(N=257), dict(H=3, Hkv=2), dict(Hkv=0), dict(D=48),
    dict(D=0), dict(Tc=0), dict(ld=191), dict(ld=196), dict(ldo=63), dict(ldo=68), dict(wsb=0),
    dict(qkv=C.c_void_p(4104)), dict(k=C.c_void_p(4098)), dict(out=C.c_void_p(4100)),
    dict(B=65536), dict(B=60000, N=256, H=256, Hkv=256, D=16, ld=12288, ldo=4096)])
def test_tree_attention_refuses(g, bad):
    assert attention(g, **bad) == g.ERR_ARG
    assert b"tree_attention" in g.lib.gpt2_last_error(None)


def test_tree_attention_workspace(g):
    ws = C.c_size_t()
    f = g.lib.gpt2_tree_attention_workspace
    for dt in (g.BF16, g.F32):
        for H, Hkv, D in ((12, 12, 64), (4, 4, 16), (32, 8, 128), (6, 1, 32)):
            assert f(4, 64, H, Hkv, D, dt, C.byref(ws)) == g.OK and 0 < ws.value <= 1 << 28
    assert f(4, 64, 12, 5, 64, g.BF16, C.byref(ws)) == g.ERR_ARG
    assert f(4, 64, 12, 12, 96, g.BF16, C.byref(ws)) == g.ERR_ARG
    assert f(4, 300, 12, 12, 64, g.BF16, C.byref(ws)) == g.ERR_ARG
    assert f(4, 64, 12, 12, 64, g.BF16, None) == g.ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(tokens=None), dict(uniform=None), dict(path=None), dict(n=None),
    dict(next=None), dict(B=0), dict(N=0), dict(N=257), dict(V=0), dict(V=65537, ld=1 << 20),
    dict(ld=99), dict(draft=P, ldd=99), dict(T=-0.5), dict(T=float("inf")), dict(T=float("nan")), dict(T=2e20),
    dict(k=-1), dict(p=0.0), dict(p=1.5), dict(p=float("nan"))])
def test_tree_verify_refuses(g, bad):
    a = dict(logits=P, ld=100, draft=None, ldd=0, tokens=P, uniform=P, B=1, N=4, V=100, T=1.0, k=0,
             p=1.0, path=P, n=P, next=P)
    a.update(bad)
    rc = g.lib.gpt2_tree_verify(a["logits"], a["ld"], a["draft"], a["ldd"], a["tokens"], None, None,
                                a["uniform"], a["B"], a["N"], a["V"], a["T"], a["k"], a["p"],
                                a["path"], a["n"], a["next"], None)
    assert rc == g.ERR_ARG and b"tree_verify" in g.lib.gpt2_last_error(None)


VERIFY_BUFFERS = ["logits", "draft", "tokens", "parent", "counts", "uniform", "path", "n", "next"]


@pytest.mark.parametrize("which,over", [(a, b) for a in ("path", "n", "next") for b in VERIFY_BUFFERS
                                        if a != b])
def test_tree_verify_refuses_outputs_over_its_arguments(g, which, over):
    """The CTAs of a sequence read while one of them writes: an output may not
    share memory with an input or another output."""
    at = {n: 1 << (20 + i) for i, n in enumerate(VERIFY_BUFFERS)}
    last = {"logits": 8 * 100 * 4, "draft": 8 * 100 * 4, "counts": 8, "n": 8, "next": 8}.get(over, 32) - 4
    for offset in (0, last):  # the first and the last element
        a = dict(at)
        a[which] = at[over] + offset
        a = {k: C.c_void_p(v) for k, v in a.items()}
        rc = g.lib.gpt2_tree_verify(a["logits"], 100, a["draft"], 100, a["tokens"], a["parent"],
                                    a["counts"], a["uniform"], 2, 4, 100, 1.0, 0, 1.0, a["path"],
                                    a["n"], a["next"], None)
        assert rc == g.ERR_ARG and b"tree_verify" in g.lib.gpt2_last_error(None)


@pytest.mark.parametrize("bad", [
    dict(qkv=None), dict(lens=None), dict(k=None), dict(v=None), dict(new=C.c_void_p(8192)),
    dict(dtype=3), dict(L=0), dict(L=65536), dict(B=0), dict(N=257), dict(D=20), dict(Tc=0),
    dict(ld=190), dict(ld=195), dict(qkv=C.c_void_p(4100)), dict(H=3, Hkv=2)])
def test_kv_append_refuses(g, bad):
    a = dict(qkv=P, ld=192, lens=C.c_void_p(8192), dtype=g.BF16, L=1, B=1, N=4, H=1, Hkv=1, D=64,
             Tc=16, k=P, v=P, new=None)
    a.update(bad)
    rc = g.lib.gpt2_kv_append(a["qkv"], a["ld"], a["lens"], None, None, a["dtype"], a["L"], a["B"],
                              a["N"], a["H"], a["Hkv"], a["D"], a["Tc"], a["k"], a["v"], a["new"],
                              None)
    assert rc == g.ERR_ARG and b"kv_append" in g.lib.gpt2_last_error(None)


@pytest.mark.parametrize("new", [8192, 8188, 8200, 12288, 12296, 12284, 16384, 16384 + 44, 16380])
def test_kv_append_refuses_lengths_over_its_inputs(g, new):
    """new_lens may not overlap lens, n_path or path, which other blocks read."""
    V = C.c_void_p
    rc = g.lib.gpt2_kv_append(P, 192, V(8192), V(16384), V(12288), g.BF16, 1, 3, 4, 1, 1, 64, 16, P, P,
                              V(new), None)
    assert rc == g.ERR_ARG and b"new_lens" in g.lib.gpt2_last_error(None)


def test_binding_checks_cpu_tensors(g):
    """Tensors that are not on a GPU, or do not fit together, are refused before
    any library call."""
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):
        g.tree_attention(z(1, 4, 192), z(1, 1, 8, 64), z(1, 1, 8, 64), z(1, dtype=torch.int32), 1)
    with pytest.raises(ValueError):
        g.tree_verify(z(1, 4, 10), 10, z(1, 4, dtype=torch.int32), z(1, 4))
    with pytest.raises(ValueError):
        g.kv_append(z(1, 1, 4, 192), z(1, 1, 1, 8, 64), z(1, 1, 1, 8, 64), z(1, dtype=torch.int32))


def test_row_spacing_of_views(g):
    """Views with evenly spaced rows give their spacing, others are refused
    (shapes only; the check itself does not look at the device)."""
    import torch

    class Fake:  # a tensor's shape and strides, said to be on a GPU
        is_cuda, device = True, "cuda:0"

        def __init__(self, t):
            self.shape, self.s, self.is_contiguous = t.shape, t.stride(), t.is_contiguous

        def dim(self):
            return len(self.shape)

        def stride(self, d=None):
            return self.s if d is None else self.s[d]

    rows = lambda t: g._node_rows("qkv", Fake(t), t.dim(), 1, 1, 64)
    full = torch.empty(2, 3, 5, 256)
    assert rows(full[..., :192]) == 256
    assert rows(full[:, :, :1, :192].contiguous()) == 192
    assert rows(full[:, :1, :1, :192][:1]) == 192  # one row: any spacing
    for bad in (full[:, :, :4, :192], full[:, :2, :, :192], full.transpose(1, 2)[..., :192],
                full[..., ::2][..., :64]):
        with pytest.raises(ValueError):
            rows(bad)
    one = torch.empty(2, 3, 1, 256)[..., :192]
    assert rows(one) == 256  # one node a sequence: the spacing of the sequences


def enumerate_verify(p, q, kids, V):
    """Distribution of the first token emitted after the root for the rule on
    probabilities: `kids` children drawn independently from q."""
    out = np.zeros(V)

    def step(w, k, mass):
        if k == 0:
            out[:] += mass * w / w.sum()
            return
        S = w.sum()
        rest = np.maximum(w - q * S, 0.0)
        rej = 0.0
        for t in range(V):
            a = min(1.0, w[t] / (q[t] * S)) if q[t] > 0 else 0.0
            out[t] += mass * q[t] * a
            rej += mass * q[t] * (1 - a)
        if rej > 1e-15:
            step(rest, k - 1, rej)
    step(np.asarray(p, float), kids, 1.0)
    return out


@pytest.mark.parametrize("kids", [1, 2, 3])
def test_the_rule_keeps_the_target_distribution(kids):
    rng = np.random.default_rng(kids)
    p, q = rng.dirichlet(np.ones(6)), rng.dirichlet(np.ones(6))
    # every product and sum of at most 6^3 terms of doubles: 1e-12 is far above
    # their rounding
    np.testing.assert_allclose(enumerate_verify(p, q, kids, 6), p, rtol=0, atol=1e-12)


def test_plain_verify_follows_its_definition():
    z = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.2, 0.7], [0.6, 0.3, 0.1]], np.float32))
    par = np.array([-1, 0, 1])
    tok = np.array([0, 1, 2])
    # p(1) = 0.25 accepted below it, p(2 | node 1) = 0.7; the last draw from row 2
    u = np.array([0.65, 0.2, 0.69], np.float32)
    assert tree_ref.verify(z, None, tok, par, u, 1.0, 0, 1.0) == ([0, 1, 2], 1)
    u[1] = 0.3  # rejected: what is left is 0.5 and 0.25 of ids 0 and 2
    assert tree_ref.verify(z, None, tok, par, u, 1.0, 0, 1.0) == ([0], 0)
    u[0] = 0.67
    assert tree_ref.verify(z, None, tok, par, u, 1.0, 0, 1.0) == ([0], 2)


def test_tree_attention_takes_zero_rows_with_either_type(g):
    """GPT2_ZERO_ROWS is added to a type; what is no type stays refused."""
    for dt in (7 + g.ZERO_ROWS, 2 * g.ZERO_ROWS):
        assert attention(g, dtype=dt) == g.ERR_ARG
        assert g.lib.gpt2_last_error(None) == b"tree_attention: bad dtype"
    for dt in (g.F32, g.BF16):  # (refused for the workspace, the last check)
        assert attention(g, dtype=dt + g.ZERO_ROWS, wsb=0) == g.ERR_ARG
        assert b"workspace" in g.lib.gpt2_last_error(None)


def test_tree_attention_limit_of_cache_rows(g):
    """A length plus a tile has to fit 32 bits: 2^31 - 65 rows of a cache at most."""
    for kw in (dict(Tc=2 ** 31 - 64), dict(Tc=2 ** 31 - 1), dict(B=2, Tc=2 ** 30 - 32)):
        assert attention(g, wsb=0, **kw) == g.ERR_ARG
        assert b"out of range" in g.lib.gpt2_last_error(None)
    assert attention(g, Tc=2 ** 31 - 65, wsb=0) == g.ERR_ARG
    assert b"workspace" in g.lib.gpt2_last_error(None)
