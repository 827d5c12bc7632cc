"""The scored router, its balance loss and its gradients, against the float64 oracle.

Tolerances are counted from the arithmetic before any run:
  selection   exact (the router decides close calls from float64 logits)
  logits      float32 tensor-core sums: L = 2.5e-6 max(4, max|x|), the bound the router's
              own listing of close calls rests on; float64 paths: half a float32 step
  gates       a logit error L moves a gate by at most 2 L of itself, and float32 scores
              cost at most eight roundings: 2 L + 8 * 2^-24, relative
              (a gate below 2^-126 lies on float32's grid of 2^-149: at most two roundings to
              it, scaled by gate_scale, 2^-149 (1 + gate_scale), are added)
  loss, coef  coef is rounded once (2^-24); the loss sums s' of at most 16 roundings: 2^-20
  d_logit     products of at most 16 float32 roundings of terms bounded by
              scale sum|d_gate| and max|q|: 2^-20 (2 scale sum|d_gate| + 2 max|q|)
  du, dE      from the router's own d_logit: float32 sums, 2^-18 sum|terms|; du then rounded
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_60_b200 as moe
from oracle import moe_scored as S
from tests.harness import f64

pytestmark = pytest.mark.gpu

SIG, SOFT = moe.MOE_SCORE_SIGMOID, moe.MOE_SCORE_SOFTMAX
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _inputs(T, d, N, dt, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    u = (torch.randn(T, d, generator=g, device="cuda") * scale).to(dt)
    E = (torch.randn(N, d, generator=g, device="cuda") * d ** -0.5).to(dt)
    b = (torch.rand(N, generator=g, device="cuda") * 2 - 1) * 0.01
    return u, E, b


def _route(u, E, b, K, logits=True, stream=None, **kw):
    T, d = u.shape
    N = E.shape[0]
    dev = u.device
    idx = torch.full((T, K), -7, dtype=torch.int32, device=dev)
    gate = torch.full((T, K), float("nan"), device=dev)
    counts = torch.full((N,), 12345, dtype=torch.int32, device=dev)
    lg = torch.full((T, N), float("nan"), device=dev) if logits else None
    ws = torch.full((max(256, moe.moe_route_scored_workspace_size(T, d, N)),), 255,
                    dtype=torch.uint8, device=dev)
    moe.moe_route_scored(u, E, b, K, idx, gate, counts, ws, logits=lg, stream=stream, **kw)
    return idx, gate, counts, lg, ws


def _logit_tol(x):
    return 2.5e-6 * max(4.0, np.abs(x).max()) if x.size else 0.0


def _check_route(u, E, b, K, score=SIG, n_groups=1, topk_groups=1, group_top=1, renorm=True,
                 gate_scale=1.0):
    idx, gate, counts, lg, _ = _route(u, E, b, K, score=score, n_groups=n_groups,
                                      topk_groups=topk_groups, group_top=group_top,
                                      renorm=renorm, gate_scale=gate_scale)
    torch.cuda.synchronize()
    x = f64(u) @ f64(E).T
    want = S.select(S.keys(x, None if b is None else b.cpu().numpy(), score), K, n_groups,
                    topk_groups, group_top)
    got = idx.cpu().numpy()
    bad = (got != want).any(axis=1)
    assert not bad.any(), f"{bad.sum()} tokens, first {np.nonzero(bad)[0][0]}: " \
        f"{got[bad][0]} != {want[bad][0]}"
    assert np.array_equal(counts.cpu().numpy(), np.bincount(want.reshape(-1), minlength=len(E)))
    L = _logit_tol(x)
    assert np.abs(f64(lg) - x).max() <= L
    g = S.gates(x, want, score, renorm, gate_scale)
    tol = (2 * L + 8 * 2.0 ** -24) * np.abs(g) + 2.0 ** -149 * (1 + gate_scale)
    assert (np.abs(f64(gate) - g) <= tol).all(), (np.abs(f64(gate) - g) / tol).max()
    return idx, gate, lg


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("T,d,N,K,kw", [
    (1, 64, 1, 1, {}),
    (1, 7168, 256, 8, dict(n_groups=8, topk_groups=4, group_top=2, gate_scale=2.5)),
    (3, 128, 5, 5, dict(renorm=False)),
    (8, 2048, 64, 6, dict(renorm=False, gate_scale=16.0)),
    (9, 320, 61, 6, {}),
    (33, 64, 31, 4, {}),
    (129, 192, 33, 3, dict(renorm=False)),
    (257, 256, 96, 8, dict(n_groups=8, topk_groups=3, group_top=2)),
    (300, 512, 160, 16, dict(n_groups=5, topk_groups=2, group_top=1, renorm=False)),
    (513, 1024, 256, 8, dict(n_groups=8, topk_groups=4, group_top=2)),
    (700, 320, 257, 9, {}),
    (260, 128, 1024, 40, dict(n_groups=32, topk_groups=16, group_top=2)),
    (64, 128, 700, 700, {}),
    (1037, 2048, 64, 6, {}),
])
def test_route_scored(dt, score, T, d, N, K, kw):
    u, E, b = _inputs(T, d, N, dt, 100 + T)
    _check_route(u, E, b, K, score, **kw)


@pytest.mark.parametrize("score", [SIG, SOFT])
def test_route_scored_training_batch(score):
    """The V3 shape at 8192 tokens: every token's selection, and no bias."""
    u, E, _ = _inputs(8192, 7168, 256, torch.bfloat16, 7)
    _check_route(u, E, None, 8, score, n_groups=8, topk_groups=4, group_top=2, gate_scale=2.5)
    _check_route(u, E, None, 8, score, renorm=False)


@pytest.mark.parametrize("T", [5, 600])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_route_scored_ties_padding_and_masked_experts(T, score):
    """Equal experts, tokens of zeros, experts barred by -inf and by the lowest float."""
    u, E, b = _inputs(T, 256, 64, torch.bfloat16, 3)
    E[10] = E[3]
    E[40] = E[3]
    b[10] = b[40] = b[3]
    u[T // 2:T // 2 + 2] = 0
    b[5] = -float("inf")
    b[6] = torch.finfo(torch.float32).min
    b[7] = 0.5
    for kw in (dict(), dict(renorm=False), dict(n_groups=4, topk_groups=2, group_top=2)):
        idx, gate, _ = _check_route(u, E, b, 6, score, **kw)
        assert not (idx == 5).any() and not (idx == 6).any()
    # every expert equal: the lowest ids, by index
    E[:] = E[3]
    idx, gate, _ = _check_route(u, E, None, 6, score)
    assert torch.equal(idx, torch.arange(6, dtype=torch.int32, device="cuda").expand(T, 6))
    # fewer open experts than K: the barred ones by index
    b = torch.full((64,), -float("inf"), device="cuda")
    b[20] = 0
    idx, gate, _ = _check_route(u, E, b, 3, score)
    assert torch.equal(idx[0].cpu(), torch.tensor([20, 0, 1], dtype=torch.int32))


@pytest.mark.parametrize("T", [4, 300])
def test_route_scored_underflowing_scores_stay_normalised(T):
    """Every selected sigmoid underflows, and softmax leaves the selected experts nothing."""
    d, N = 128, 32
    u = torch.full((T, d), 1.0, device="cuda").to(torch.bfloat16)
    E = torch.full((N, d), -2.0, device="cuda").to(torch.bfloat16)
    E[:, 0] -= (torch.arange(N, device="cuda") * 0.25).to(torch.bfloat16)
    idx, gate, _, _, _ = _route(u, E, None, 4, score=SIG)
    x = f64(u) @ f64(E).T
    g = S.gates(x, idx.cpu().numpy(), SIG, True, 1.0)
    assert np.abs(f64(gate) - g).max() <= 1e-5 and np.abs(f64(gate).sum(1) - 1).max() <= 1e-6
    # softmax: one expert takes everything, the bias selects others
    E = torch.full((N, d), -2.0, device="cuda").to(torch.bfloat16)
    E[0] = 2.0
    b = torch.zeros(N, device="cuda")
    b[8:12] = 5.0
    idx, gate, _, _, _ = _route(u, E, b, 4, score=SOFT)
    assert torch.equal(idx[0].cpu(), torch.tensor([8, 9, 10, 11], dtype=torch.int32))
    assert np.abs(f64(gate) - 0.25).max() <= 1e-6


@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_route_scored_nan_and_inf_stay_in_their_token(T, score):
    u, E, b = _inputs(T, 128, 40, torch.bfloat16, 9)
    clean = _route(u, E, b, 5, score=score)
    bad = u.clone()
    bad[1, 7] = float("nan")
    if T > 200:
        bad[150, 3] = float("inf")
        bad[151] = -float("inf")
    got = _route(bad, E, b, 5, score=score)
    keep = torch.isfinite(bad.float()).all(1)
    assert torch.equal(got[0][keep], clean[0][keep])
    assert torch.equal(got[1][keep], clean[1][keep])
    ids = got[0].cpu().numpy()
    assert ids.min() >= 0 and ids.max() < 40
    assert all(len(set(r)) == 5 for r in ids.tolist())
    assert int(got[2].sum()) == 5 * T


def test_route_scored_magnitudes():
    """Logits far larger and smaller than one: the selection stays the definition's."""
    for scale in (1e-3, 30.0):
        for score in (SIG, SOFT):
            u, E, b = _inputs(400, 512, 64, torch.bfloat16, 21, scale)
            _check_route(u, E, b, 6, score)


def test_route_scored_agrees_with_moe_route():
    """Sigmoid, renormalised, scale 1: moe_route's selection."""
    u, E, b = _inputs(1000, 1024, 128, torch.bfloat16, 5)
    idx, gate, counts, _, _ = _route(u, E, b, 8)
    i2, g2, c2 = torch.empty_like(idx), torch.empty_like(gate), torch.empty_like(counts)
    ws = torch.empty(moe.moe_route_workspace_size(1000, 128), dtype=torch.uint8, device="cuda")
    moe.moe_route(u, E, b, 8, i2, g2, c2, ws)
    assert torch.equal(idx, i2) and torch.equal(counts, c2)
    assert (gate - g2).abs().max() <= 1e-5


@pytest.mark.parametrize("T", [1, 4, 200, 3000])
def test_route_scored_repeats_streams_and_graphs(T):
    """Equal bits on every call, on another stream, and from a replayed graph whose inputs
    changed in place; no logits asked for changes nothing else."""
    u, E, b = _inputs(T, 512, 96, torch.bfloat16, 31)
    kw = dict(score=SOFT, n_groups=6, topk_groups=3, group_top=2, renorm=False)
    first = _route(u, E, b, 4, **kw)
    plain = _route(u, E, b, 4, logits=False, **kw)
    assert torch.equal(first[0], plain[0]) and torch.equal(first[1], plain[1])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        other = _route(u, E, b, 4, **kw)
    st.synchronize()
    for k in range(4):
        assert torch.equal(first[k], other[k])
    u2, _, _ = _inputs(T, 512, 96, torch.bfloat16, 32)
    want = _route(u2, E, b, 4, **kw)
    static = u.clone()
    idx, gate, counts, lg, ws = _route(static, E, b, 4, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_route_scored(static, E, b, 4, idx, gate, counts, ws, logits=lg, **kw)
    static.copy_(u2)
    for _ in range(2):
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for k, t in enumerate((idx, gate, counts, lg)):
            assert torch.equal(t, want[k])


def test_route_scored_no_tokens():
    u, E, b = _inputs(0, 128, 16, torch.bfloat16, 1)
    counts = torch.full((16,), 9, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 4, device="cuda")
    moe.moe_route_scored(u, E, b, 4, e.int(), e, counts, None)
    assert not counts.any()


# ------------------------------------------------------------------ balance loss

def _logits(T, N, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(T, N, generator=g, device="cuda") + 0.5 * torch.randn(N, generator=g,
                                                                         device="cuda")
    return x.to(dtype), g


def _balance(x, idx, off, n_seq, alpha, score):
    N = x.shape[1]
    loss = torch.full((n_seq,), float("nan"), device="cuda")
    coef = torch.full((n_seq, N), float("nan"), device="cuda")
    ws = torch.full((moe.moe_balance_loss_workspace_size(x.shape[0], N, n_seq),), 255,
                    dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss(x, idx, alpha, loss, coef, ws, score=score, seq_offsets=off)
    return loss, coef


SEQS = [
    (1, 1, 1, None),
    (37, 8, 3, [0, 0, 1, 36, 36]),
    (300, 61, 6, [5, 31, 32, 33, 33, 200, 290]),
    (1000, 256, 8, None),
    (4097, 96, 16, [0, 4096, 4096, 4097]),
    (513, 1024, 33, [0, 100, 512]),
    (64, 40, 2, [0, 0, 0]),
]


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("T,N,K,off", SEQS)
def test_balance_loss(score, T, N, K, off):
    x, g = _logits(T, N, 40 + T)
    idx = torch.topk(x, K, dim=1).indices.int()
    if T > 30:                                   # dropped slots and a repeated expert
        idx[3, 0] = -1
        idx[4, 0] = N + 5
        idx[7] = idx[7, 0]
    o = [0, T] if off is None else off
    ot = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    loss, coef = _balance(x, idx, ot, len(o) - 1, 1e-3, score)
    wl, wc = S.balance(f64(x), idx.cpu().numpy(), o, 1e-3, score)
    assert (np.abs(f64(coef) - wc) <= 2.0 ** -23 * np.abs(wc)).all()
    assert (np.abs(f64(loss) - wl) <= 2.0 ** -20 * np.abs(wl)).all()
    again = _balance(x, idx, ot, len(o) - 1, 1e-3, score)
    assert torch.equal(again[0], loss) and torch.equal(again[1], coef)
    assert moe.moe_device_status() == 0


def test_balance_loss_uniform_is_alpha():
    """Equal scores and equal loads: f_i = 1 and P_i = 1/N, so the loss is alpha."""
    T, N, K = 64, 16, 4
    x = torch.zeros(T, N, device="cuda")
    idx = ((torch.arange(T, device="cuda")[:, None] * K + torch.arange(K, device="cuda")) % N).int()
    for score in (SIG, SOFT):
        loss, coef = _balance(x, idx, None, 1, 0.01, score)
        assert abs(float(loss) - 0.01) <= 0.01 * 2.0 ** -20


def test_balance_loss_reports_bad_offsets():
    x, _ = _logits(100, 16, 3)
    idx = torch.topk(x, 2, dim=1).indices.int()
    off = torch.tensor([-5, 40, 30, 400], dtype=torch.int32, device="cuda")
    _balance(x, idx, off, 3, 1.0, SIG)
    assert moe.moe_device_status() == 16
    assert moe.moe_device_status() == 0


# ------------------------------------------------------------------ backward

def _bwd(u, E, x, idx, dg, score, renorm, scale, off=None, coef=None, dl=None, base=None,
         want_logit=True):
    T, d = u.shape
    N = E.shape[0]
    du = torch.full((T, d), float("nan"), device="cuda", dtype=u.dtype)
    dE = torch.full((N, d), float("nan"), device="cuda")
    dlg = torch.full((T, N), float("nan"), device="cuda") if want_logit else None
    dt = moe.MOE_F32 if u.dtype == torch.float32 else moe.MOE_BF16
    ws = torch.full((max(256, moe.moe_route_scored_backward_workspace_size(dt, T, d, N)),), 255,
                    dtype=torch.uint8, device="cuda")
    moe.moe_route_scored_backward(u, E, x, idx, dg, du, dE, ws, score=score, renorm=renorm,
                                  gate_scale=scale, seq_offsets=off, balance_coef=coef, d_loss=dl,
                                  du_base=base, d_logit=dlg)
    return du, dE, dlg


def _check_products(u, E, dlg, base, du, dE):
    dl, uu, ee = f64(dlg), f64(u), f64(E)
    b = 0 if base is None else f64(base)
    want = b + dl @ ee
    mag = np.abs(b) + np.abs(dl) @ np.abs(ee)
    tol = 2.0 ** -15 if u.dtype == torch.bfloat16 else 2.0 ** -18
    err = np.abs(f64(du) - want)
    assert (err <= HALF[u.dtype] * np.abs(want) * 1.01 + tol * mag).all(), (err - HALF[u.dtype] * np.abs(want)).max()
    want = dl.T @ uu
    mag = np.abs(dl).T @ np.abs(uu)
    assert (np.abs(f64(dE) - want) <= 2.0 ** -18 * mag).all()
    # the float32 gradient holds float32 accuracy over the whole, not only entry by entry
    assert np.linalg.norm(f64(dE) - want) <= 2.0 ** -18 * np.linalg.norm(want)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score,renorm", [(SIG, True), (SIG, False), (SOFT, True), (SOFT, False)])
@pytest.mark.parametrize("T,d,N,K,off", [
    (1, 64, 1, 1, None),
    (5, 128, 9, 3, [0, 2, 5]),
    (130, 320, 61, 6, [3, 3, 60, 125]),
    (257, 192, 33, 33, [0, 257]),
    (300, 512, 64, 6, None),
    (700, 256, 256, 8, [0, 128, 700]),
    (515, 64, 320, 4, [0, 100, 400]),
    (70, 128, 1024, 40, None),
])
def test_route_scored_backward(dt, score, renorm, T, d, N, K, off):
    u, E, _ = _inputs(T, d, N, dt, 60 + T)
    x, g = _logits(T, N, 61 + T)
    idx = torch.topk(x, K, dim=1).indices.int()
    if T > 100:
        idx[3, 0] = -1
        idx[4] = N + 1                           # every slot left out
        if K > 2:
            idx[7, 1] = idx[7, 0]                # the same expert twice, and three times
            idx[8, :3] = idx[8, 0]
    dg = torch.randn(T, K, generator=g, device="cuda") * 0.1
    o = [0, T] if off is None else off
    n = len(o) - 1
    ot = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    coef = torch.rand(n, N, generator=g, device="cuda") * 0.01
    dl = torch.rand(n, generator=g, device="cuda")
    base = torch.randn(T, d, generator=g, device="cuda").to(dt)
    for dgx, cx, dlx, bx in ((dg, coef, dl, base), (dg, None, None, None), (None, coef, None, base)):
        du, dE, dlg = _bwd(u, E, x, idx, dgx, score, renorm, 2.5, ot, cx, dlx, bx)
        want = S.backward(f64(x), idx.cpu().numpy(), None if dgx is None else f64(dgx), o,
                          None if cx is None else f64(cx), None if dlx is None else f64(dlx),
                          score, renorm, 2.5)
        mag = np.zeros((T, 1))
        if dgx is not None:
            mag = mag + 2 * 2.5 * np.abs(f64(dgx)).sum(1, keepdims=True)
        if cx is not None:
            mag = mag + 2 * f64(cx).max()
        assert (np.abs(f64(dlg) - want) <= 2.0 ** -20 * mag).all(), \
            (np.abs(f64(dlg) - want) / mag).max() * 2 ** 20
        _check_products(u, E, dlg, bx, du, dE)
        d2, e2, _ = _bwd(u, E, x, idx, dgx, score, renorm, 2.5, ot, cx, dlx, bx, want_logit=False)
        assert torch.equal(du, d2) and torch.equal(dE, e2)


def test_route_scored_backward_training_batch():
    """The V3 shape at 8192 tokens: the products in full against float64 on the GPU."""
    T, d, N, K = 8192, 7168, 256, 8
    u, E, _ = _inputs(T, d, N, torch.bfloat16, 8)
    x = (u.double() @ E.double().T).float()
    idx = torch.topk(x, K, dim=1).indices.int()
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    dg = torch.randn(T, K, generator=g, device="cuda") * 0.01
    base = (torch.randn(T, d, generator=g, device="cuda") * 0.01).to(torch.bfloat16)
    off = torch.tensor([0, 4096, 8000], dtype=torch.int32, device="cuda")
    coef = torch.rand(2, N, generator=g, device="cuda") * 1e-5
    du, dE, dlg = _bwd(u, E, x, idx, dg, SIG, True, 2.5, off, coef, None, base)
    want = base.double() + dlg.double() @ E.double()
    assert ((du.double() - want).norm() / want.norm()).item() <= 2.0 ** -8
    want = dlg.double().T @ u.double()
    assert ((dE.double() - want).norm() / want.norm()).item() <= 2.0 ** -18


def test_route_scored_backward_in_place_base_streams_and_graphs():
    T, d, N, K = 300, 256, 64, 6
    u, E, _ = _inputs(T, d, N, torch.bfloat16, 70)
    x, g = _logits(T, N, 71)
    idx = torch.topk(x, K, dim=1).indices.int()
    dg = torch.randn(T, K, generator=g, device="cuda")
    base = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    du, dE, dlg = _bwd(u, E, x, idx, dg, SOFT, True, 1.0, base=base)
    ws = torch.empty(moe.moe_route_scored_backward_workspace_size(moe.MOE_BF16, T, d, N),
                     dtype=torch.uint8, device="cuda")
    inout, dE2 = base.clone(), torch.empty_like(dE)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    moe.moe_route_scored_backward(u, E, x, idx, dg, inout, dE2, ws, score=SOFT, du_base=inout,
                                  stream=st)
    st.synchronize()
    assert torch.equal(inout, du) and torch.equal(dE2, dE)
    out, dE3 = torch.empty_like(du), torch.empty_like(dE)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_route_scored_backward(u, E, x, idx, dg, out, dE3, ws, score=SOFT, du_base=base)
    for _ in range(2):
        out.zero_()
        dE3.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, du) and torch.equal(dE3, dE)


def test_route_scored_backward_matches_differences():
    """The gradient of <d_gate, gate> + <d_loss, loss> through the forward calls themselves:
    central differences of the float64 definition at the GPU's selection."""
    T, N, K = 6, 12, 3
    x, g = _logits(T, N, 90)
    idx = torch.topk(x, K, dim=1).indices.int()
    dg = torch.randn(T, K, generator=g, device="cuda")
    u, E, _ = _inputs(T, 64, N, torch.float32, 91)
    ii, xx, dgg = idx.cpu().numpy(), f64(x), f64(dg)
    for score, renorm in ((SIG, True), (SIG, False), (SOFT, True), (SOFT, False)):
        loss, coef = _balance(x, idx, None, 1, 0.5, score)
        _, _, dlg = _bwd(u, E, x, idx, dg, score, renorm, 1.5, None, coef, None)

        def f(v):
            return (dgg * S.gates(v, ii, score, renorm, 1.5)).sum() \
                + S.balance(v, ii, [0, T], 0.5, score)[0].sum()
        num = np.zeros((T, N))
        for t in range(T):
            for e in range(N):
                p, m = xx.copy(), xx.copy()
                p[t, e] += 1e-5
                m[t, e] -= 1e-5
                num[t, e] = (f(p) - f(m)) / 2e-5
        # central differences: error of order 1e-10 of the third derivative, 1e-11 of rounding
        assert np.abs(f64(dlg) - num).max() <= 2.0 ** -20 * (3 * np.abs(dgg).sum(1).max() + 1) + 1e-8


def test_route_scored_backward_no_tokens():
    u, E, _ = _inputs(0, 128, 16, torch.bfloat16, 1)
    dE = torch.full((16, 128), 3.0, device="cuda")
    z = torch.empty(0, 16, device="cuda")
    moe.moe_route_scored_backward(u, E, z, z[:, :4].int(), z[:, :4].contiguous(), u.clone(), dE,
                                  None)
    assert not dE.any()


def test_route_scored_backward_float32_many_tokens():
    """More 64-token tiles than a grid's second dimension holds."""
    T, d, N, K = 65536 * 64 + 5, 64, 2, 1
    g = torch.Generator(device="cuda").manual_seed(5)
    u = torch.randn(T, d, generator=g, device="cuda")
    E = torch.randn(N, d, generator=g, device="cuda")
    logits = torch.randn(T, N, generator=g, device="cuda")
    idx = torch.randint(0, N, (T, K), generator=g, device="cuda", dtype=torch.int32)
    dg = torch.randn(T, K, generator=g, device="cuda")
    du, dE, dl = torch.empty_like(u), torch.empty(N, d, device="cuda"), torch.empty_like(logits)
    ws = torch.empty(max(1, moe.moe_route_scored_backward_workspace_size(moe.MOE_F32, T, d, N)),
                     dtype=torch.uint8, device="cuda")
    moe.moe_route_scored_backward(u, E, logits, idx, dg, du, dE, ws, renorm=False, d_logit=dl)
    for rows in (slice(0, 64), slice(T - 69, T)):
        a, e = dl[rows].double(), E.double()
        # two products and a sum in float32, each off by at most half a step of
        # the sum of the absolute values
        bound = 3 * 2.0 ** -24 * (a.abs() @ e.abs())
        assert ((du[rows].double() - a @ e).abs() <= bound).all()
    assert torch.isfinite(dE).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K,kw", [
    *[(20, 96, K, {}) for K in (1, 3, 4, 27, 28, 30, 31, 32, 33, 64, 95, 96)],
    (40, 66, 5, dict(n_groups=6, topk_groups=3, group_top=2)),       # groups of 11
    (40, 66, 22, dict(n_groups=3, topk_groups=1)),                   # as many as the group holds
    (40, 64, 3, dict(n_groups=32, topk_groups=2, group_top=2)),      # groups of two
    (2000, 66, 5, dict(n_groups=6, topk_groups=3, group_top=2)),
    (12, 1024, 1024, {}),
    (1100, 1024, 33, {}),
])
def test_route_scored_ranks_across_warps(dt, T, N, K, kw):
    """Slots around a warp's 32 keys, group sizes of no vector, the largest sizes."""
    u, E, b = _inputs(T, 128, N, dt, 900 + K + N)
    for score in (SIG, SOFT):
        _check_route(u, E, b, K, score, **kw)


@pytest.mark.parametrize("T", [6, 100, 1500])
def test_route_scored_equal_keys_across_warps(T):
    """Four distinct experts, each in every warp many times over: ties go by index."""
    u, E, _ = _inputs(T, 192, 256, torch.bfloat16, 12)
    E = E[torch.arange(256, device="cuda") % 4].contiguous()
    for kw in (dict(), dict(n_groups=8, topk_groups=3, group_top=2)):
        _check_route(u, E, None, 40, SIG, **kw)
        _check_route(u, E, None, 40, SOFT, renorm=False, **kw)


def test_route_scored_calls_at_once():
    """Calls on two streams, each with its own buffers, are those of one stream."""
    cases = [(_inputs(T, 512, 128, torch.bfloat16, 40 + T), score) for T, score in
             ((200, SIG), (1800, SOFT))]
    alone = [_route(*i[:2], i[2], 6, score=s) for i, s in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        both = []
        for (i, s), st in zip(cases, streams):
            with torch.cuda.stream(st):
                both.append(_route(*i[:2], i[2], 6, score=s))
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(x, y) for x, y in zip(a[:4], b[:4]))
