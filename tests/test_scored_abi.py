"""Argument checks of the scored router, its balance loss and backward, and of the 8-bit
checkpoint calls: every bad call answers with a status (or, in the binding, a ValueError)
before any CUDA work.  The oracle's gradient against differences.  No GPU is needed."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_layer_60_b200 as moe
from mixture_experts_layer_60_b200 import build as moe_build
from oracle import moe_scored as S

D = ctypes.c_void_p(256)                 # never dereferenced: validation fails first
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


def _route(L, u=D, E=D, dt=1, b=None, T=8, d=64, N=16, K=4, score=0, ng=1, tg=1, top=1, renorm=1,
           scale=1.0, idx=D, gate=D, counts=D, logits=None, ws=D, n=BIG):
    return L.moe_route_scored(u, E, dt, b, T, d, N, K, score, ng, tg, top, renorm, scale, idx, gate,
                              counts, logits, ws, n, None)


@pytest.mark.parametrize("want,kw", [
    (2, dict(dt=2)), (1, dict(T=-1)), (1, dict(K=0)), (2, dict(K=17)), (2, dict(N=1025)),
    (2, dict(d=96)), (2, dict(d=16448)), (2, dict(dt=0, d=8256)), (1, dict(score=2)),
    (1, dict(ng=3)), (1, dict(ng=64, N=64)), (1, dict(ng=4, tg=5)), (1, dict(ng=8, tg=1)),
    (1, dict(top=0)), (1, dict(top=3)), (1, dict(ng=16, tg=8, top=2)),
    (1, dict(scale=float("inf"))), (1, dict(scale=float("nan"))), (1, dict(E=None)),
    (1, dict(u=None)), (1, dict(counts=None)), (1, dict(idx=None)), (1, dict(gate=None)),
    (1, dict(u=ctypes.c_void_p(264))), (1, dict(ws=None)), (3, dict(n=64)),
    (1, dict(ws=ctypes.c_void_p(272))), (2, dict(T=1 << 28)),
])
def test_route_scored_argument_errors(L, want, kw):
    assert _route(L, **kw) == want
    assert b"moe_route_scored" in L.moe_last_error()


@pytest.mark.parametrize("want,kw", [
    (1, dict(T=-1)), (1, dict(K=0)), (2, dict(K=17)), (1, dict(score=-1)), (1, dict(n_seq=0)),
    (1, dict(n_seq=(1 << 20) + 1)), (1, dict(off=None, n_seq=2)), (1, dict(loss=None)),
    (1, dict(coef=None)), (1, dict(logits=None)), (1, dict(idx=None)),
    (1, dict(alpha=float("nan"))), (1, dict(ws=None)), (3, dict(n=8)),
    (1, dict(ws=ctypes.c_void_p(8))),
])
def test_balance_loss_argument_errors(L, want, kw):
    a = dict(logits=D, idx=D, off=D, n_seq=1, T=8, N=16, K=4, score=0, alpha=1.0, loss=D, coef=D,
             ws=D, n=BIG)
    a.update(kw)
    assert L.moe_balance_loss(a["logits"], a["idx"], a["off"], a["n_seq"], a["T"], a["N"], a["K"],
                              a["score"], a["alpha"], a["loss"], a["coef"], a["ws"], a["n"],
                              None) == want
    assert b"moe_balance_loss" in L.moe_last_error()


@pytest.mark.parametrize("want,kw", [
    (2, dict(dt=2)), (1, dict(T=-1)), (2, dict(N=1025)), (2, dict(d=96)), (1, dict(score=7)),
    (1, dict(dg=None)), (1, dict(coef=None, dl=D)), (1, dict(off=None, n_seq=3, coef=D)),
    (1, dict(n_seq=0)), (1, dict(scale=float("inf"))), (1, dict(E=None)), (1, dict(dE=None)),
    (1, dict(u=None)), (1, dict(du=None)), (1, dict(logits=None)), (1, dict(idx=None)),
    (1, dict(du=ctypes.c_void_p(260))), (1, dict(ws=None)), (3, dict(n=8)),
])
def test_route_scored_backward_argument_errors(L, want, kw):
    a = dict(u=D, E=D, dt=1, logits=D, idx=D, dg=D, off=None, n_seq=1, coef=None, dl=None, T=8,
             d=64, N=16, K=4, score=0, renorm=1, scale=1.0, base=None, dlg=None, du=D, dE=D, ws=D,
             n=BIG)
    a.update(kw)
    assert L.moe_route_scored_backward(
        a["u"], a["E"], a["dt"], a["logits"], a["idx"], a["dg"], a["off"], a["n_seq"], a["coef"],
        a["dl"], a["T"], a["d"], a["N"], a["K"], a["score"], a["renorm"], a["scale"], a["base"],
        a["dlg"], a["du"], a["dE"], a["ws"], a["n"], None) == want
    assert b"moe_route_scored_backward" in L.moe_last_error()


@pytest.mark.parametrize("want,kw", [
    (2, dict(dt=0)), (2, dict(dt=2)), (2, dict(d=64)), (2, dict(I=64)), (1, dict(G=0)),
    (2, dict(G=1025)), (1, dict(rows=-1)), (1, dict(x=None)), (1, dict(h=None)), (1, dict(q=None)),
    (1, dict(sc=None)), (1, dict(off=None)), (1, dict(q=ctypes.c_void_p(260))),
])
def test_save8_argument_errors(L, want, kw):
    a = dict(x=D, off=D, G=2, rows=8, d=128, I=128, dt=1, W=D, h=D, q=D, sc=D)
    a.update(kw)
    assert L.moe_expert_gate_up_save8(a["x"], a["off"], a["G"], a["rows"], a["d"], a["I"], a["dt"],
                                      a["W"], a["h"], a["q"], a["sc"], None) == want
    assert b"moe_expert_gate_up_save8" in L.moe_last_error()


@pytest.mark.parametrize("want,kw", [
    (2, dict(dt=0)), (2, dict(dt=2)), (2, dict(d=128)), (2, dict(I=128)), (1, dict(G=0)),
    (1, dict(x=None)), (1, dict(Wd=None)), (1, dict(q=None)), (1, dict(sc=None)),
    (1, dict(dy=None)), (1, dict(dx=None)), (1, dict(gu=None)), (1, dict(dn=None)),
    (1, dict(ws=None)), (3, dict(n=64)), (1, dict(ws=ctypes.c_void_p(128))),
])
def test_backward8_argument_errors(L, want, kw):
    a = dict(x=D, off=D, G=2, rows=8, d=256, I=256, dt=1, W=D, Wd=D, q=D, sc=D, dy=D, dx=D, gu=D,
             dn=D, ws=D, n=BIG)
    a.update(kw)
    assert L.moe_expert_ffn_backward8(
        a["x"], a["off"], a["G"], a["rows"], a["d"], a["I"], a["dt"], a["W"], a["Wd"], a["q"],
        a["sc"], a["dy"], a["dx"], a["gu"], a["dn"], a["ws"], a["n"], None) == want
    assert b"moe_expert_ffn_backward8" in L.moe_last_error()


def test_workspace_sizes(L):
    assert L.moe_route_scored_workspace_size(0, 64, 16) == 0
    assert L.moe_route_scored_workspace_size(8192, 7168, 256) >= 8192 * 256 * 4
    assert L.moe_balance_loss_workspace_size(8192, 256, 2) >= 2 * 256 * 8
    assert L.moe_balance_loss_workspace_size(8192, 256, 0) == 0
    assert L.moe_route_scored_backward_workspace_size(1, 8192, 7168, 256) >= 8192 * 256 * 4
    assert L.moe_expert_ffn_backward8_workspace_size(1, 100, 256, 256, 4) >= 100 * 3 * 256 * 2
    assert L.moe_expert_ffn_backward8_workspace_size(2, 100, 256, 256, 4) == 0


def test_binding_refuses_wrong_types_and_shapes():
    u, E = torch.zeros(4, 64), torch.zeros(8, 64)
    i, g, c = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(8, dtype=torch.int32)
    for bad in (dict(i=i.long()), dict(g=g.double()), dict(c=torch.zeros(9, dtype=torch.int32)),
                dict(E=E.bfloat16()), dict(E=torch.zeros(8, 128))):
        a = dict(E=E, i=i, g=g, c=c)
        a.update(bad)
        with pytest.raises(ValueError):
            moe.moe_route_scored(u, a["E"], None, 2, a["i"], a["g"], a["c"], None)
    with pytest.raises(ValueError):
        moe.moe_route_scored(u, E, None, 2, i, g, c, None)          # not on a device
    with pytest.raises(ValueError):
        moe.moe_balance_loss(torch.zeros(4, 8), i.long(), 1.0, torch.zeros(1), torch.zeros(1, 8), None)
    with pytest.raises(ValueError):
        moe.moe_route_scored_backward(u, E, torch.zeros(4, 8), i, g, u.bfloat16(), E.clone(), None)


@pytest.mark.parametrize("score", [S.SIGMOID, S.SOFTMAX])
@pytest.mark.parametrize("renorm", [True, False])
def test_oracle_gradient_matches_differences(score, renorm):
    rng = np.random.default_rng(3)
    T, N, K = 7, 10, 3
    x = rng.normal(size=(T, N))
    idx = S.select(S.keys(x, None, score), K)
    dg, off = rng.normal(size=(T, K)), [0, 4, 4, 6]
    dl = rng.normal(size=3)
    _, coef = S.balance(x, idx, off, 0.3, score)
    got = S.backward(x, idx, dg, off, coef, dl, score, renorm, 1.7)

    def f(v):
        return (dg * S.gates(v, idx, score, renorm, 1.7)).sum() + \
            (dl * S.balance(v, idx, off, 0.3, score)[0]).sum()
    for t in range(T):
        for e in range(N):
            p, m = x.copy(), x.copy()
            p[t, e] += 1e-5
            m[t, e] -= 1e-5
            assert abs((f(p) - f(m)) / 2e-5 - got[t, e]) <= 1e-8


def test_oracle_checkpoint_rounds_to_nearest():
    rng = np.random.default_rng(4)
    a = (rng.normal(size=(5, 256)) * np.exp(2 * rng.normal(size=(5, 256)))).astype(np.float32)
    q, sc = S.checkpoint(a)
    v = S.from_checkpoint(q, sc)
    step = np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * np.repeat(sc, 128, axis=1))
    assert (np.abs(v - a) <= step * (1 + 1e-6)).all()
    t = torch.from_numpy(np.linspace(-460, 460, 40001).astype(np.float32))
    assert np.array_equal(S.e4m3(t.numpy()),
                          t.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy())


def test_a_workspace_for_more_tokens_serves_fewer(L):
    for N in (16, 61, 256, 257, 1024):
        for size in (lambda T: L.moe_route_scored_workspace_size(T, 7168, N),
                     lambda T: L.moe_balance_loss_workspace_size(T, N, 9),
                     lambda T: L.moe_route_scored_backward_workspace_size(1, T, 7168, N),
                     lambda T: L.moe_route_scored_backward_workspace_size(0, T, 7168, N)):
            at = [size(T) for T in list(range(1, 700, 13)) + list(range(700, 20500, 97))]
            assert all(a <= b for a, b in zip(at, at[1:]))


def test_token_counts_past_the_index_range_are_refused(L):
    T = (1 << 30) + 1                                      # T * N_r still fits in 31 bits
    assert _route(L, T=T, N=1, K=1) == 2
    assert L.moe_balance_loss(D, D, None, 1, T, 1, 1, 0, 1.0, D, D, D, BIG, None) == 2
    assert b"moe_balance_loss" in L.moe_last_error()
