"""The scored router, its balance loss and gradients where float32 sums cancel, underflow or tie.

Tolerances are counted from the arithmetic before any run:
  selection   exact, against float64 logits
  loss        sums of s' of at most 16 float32 roundings: 2^-20
  d_logit     2^-20 (2 scale sum|d_gate| + 2 max|q|); where a token's renormalised gates
              have no gradient (one slot, or equal upstream values) only the balance
              term's share is left: 2^-20 * 2 max|q|
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_60_b200 as moe
from oracle import moe_scored as S
from tests.harness import f64

pytestmark = pytest.mark.gpu

SIG, SOFT = moe.MOE_SCORE_SIGMOID, moe.MOE_SCORE_SOFTMAX
BF = torch.bfloat16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(T, d, N, seed, dt=BF):
    g = _gen(seed)
    u = torch.randn(T, d, generator=g, device="cuda").to(dt)
    E = (torch.randn(N, d, generator=g, device="cuda") * d ** -0.5).to(dt)
    b = (torch.rand(N, generator=g, device="cuda") * 2 - 1) * 0.01
    return u, E, b


def _route(u, E, b, K, **kw):
    T, d = u.shape
    N = E.shape[0]
    idx = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    gate = torch.full((T, K), float("nan"), device="cuda")
    counts = torch.full((N,), 12345, dtype=torch.int32, device="cuda")
    ws = torch.full((max(256, moe.moe_route_scored_workspace_size(T, d, N)),), 255,
                    dtype=torch.uint8, device="cuda")
    moe.moe_route_scored(u, E, b, K, idx, gate, counts, ws, **kw)
    return idx, gate, counts


def _check_selection(u, E, b, K, score, n_groups=1, topk_groups=1, group_top=1, **kw):
    idx, gate, counts = _route(u, E, b, K, score=score, n_groups=n_groups,
                               topk_groups=topk_groups, group_top=group_top, **kw)
    x = f64(u) @ f64(E).T
    want = S.select(S.keys(x, None if b is None else b.cpu().numpy(), score), K, n_groups,
                    topk_groups, group_top)
    got = idx.cpu().numpy()
    bad = (got != want).any(axis=1)
    assert not bad.any(), f"{bad.sum()} of {len(bad)} tokens, first {np.nonzero(bad)[0][0]}: " \
        f"{got[bad][0]} != {want[bad][0]}"
    assert np.array_equal(counts.cpu().numpy(), np.bincount(want.reshape(-1), minlength=len(E)))
    assert torch.isfinite(gate).all()


# ------------------------------------------------------------------ underflow

def _underflow(T, N, K, seed, rows):
    """Logits of which the given rows lie far below every float32 sigmoid."""
    g = _gen(seed)
    x = torch.randn(T, N, generator=g, device="cuda")
    low = -90 - 210 * torch.rand(len(rows), 1, generator=g, device="cuda")
    x[rows] = low + 3 * torch.randn(len(rows), N, generator=g, device="cuda")
    return x, torch.topk(x, K, dim=1).indices.int(), g


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,N,K,rows", [(70, 32, 4, [3]), (9, 256, 8, list(range(9))),
                                        (130, 61, 6, [0, 64, 129])])
def test_backward_of_underflowing_sigmoids(renorm, T, N, K, rows):
    d = 128
    x, idx, g = _underflow(T, N, K, 5, rows)
    dg = torch.randn(T, K, generator=g, device="cuda") * 0.1
    coef = torch.rand(1, N, generator=g, device="cuda") * 0.01
    for dt in (BF, torch.float32):
        u, E, _ = _normal(T, d, N, 6, dt)
        for dgx, cx in ((dg, None), (dg, coef), (None, coef)):
            du = torch.full((T, d), float("nan"), dtype=dt, device="cuda")
            dE = torch.full((N, d), float("nan"), device="cuda")
            dl = torch.full((T, N), float("nan"), device="cuda")
            ws = torch.empty(moe.moe_route_scored_backward_workspace_size(
                moe.MOE_BF16 if dt == BF else moe.MOE_F32, T, d, N), dtype=torch.uint8,
                device="cuda")
            moe.moe_route_scored_backward(u, E, x, idx, dgx, du, dE, ws, score=SIG, renorm=renorm,
                                          gate_scale=2.5, balance_coef=cx, d_logit=dl)
            want = S.backward(f64(x), idx.cpu().numpy(), None if dgx is None else f64(dgx),
                              [0, T], None if cx is None else f64(cx), None, S.SIGMOID, renorm, 2.5)
            mag = np.zeros((T, 1))
            if dgx is not None:
                mag = mag + 2 * 2.5 * np.abs(f64(dgx)).sum(1, keepdims=True)
            if cx is not None:
                mag = mag + 2 * f64(cx).max()
            assert torch.isfinite(dl).all() and torch.isfinite(du).all() and torch.isfinite(dE).all()
            assert (np.abs(f64(dl) - want) <= 2.0 ** -20 * mag).all()


@pytest.mark.parametrize("T,N,K,off", [(300, 61, 6, None), (1000, 256, 8, [0, 10, 10, 700, 990]),
                                       (70, 600, 5, [0, 70])])
def test_balance_of_underflowing_sigmoids(T, N, K, off):
    x, idx, _ = _underflow(T, N, K, 7, [0, 9, 10, 69])
    o = [0, T] if off is None else off
    ot = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    n = len(o) - 1
    loss = torch.full((n,), float("nan"), device="cuda")
    coef = torch.full((n, N), float("nan"), device="cuda")
    ws = torch.empty(moe.moe_balance_loss_workspace_size(T, N, n), dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss(x, idx, 1e-3, loss, coef, ws, score=SIG, seq_offsets=ot)
    wl, wc = S.balance(f64(x), idx.cpu().numpy(), o, 1e-3, S.SIGMOID)
    assert (np.abs(f64(coef) - wc) <= 2.0 ** -23 * np.abs(wc)).all()
    assert (np.abs(f64(loss) - wl) <= 2.0 ** -20 * np.abs(wl)).all()


# ------------------------------------------------------------------ gradients that cancel

@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("T,N,K", [(1, 8, 1), (100, 300, 1), (1500, 64, 1), (64, 64, 2),
                                   (300, 96, 8), (33, 64, 40)])
def test_equal_gate_gradients_leave_the_balance_term_alone(score, T, N, K):
    """Renormalised gates sum to a constant: upstream values that are the same for all of a
    token's slots have no gradient, and one slot never has."""
    d = 64
    u, E, _ = _normal(T, d, N, 30 + T)
    g = _gen(31 + K)
    x = torch.randn(T, N, generator=g, device="cuda")
    idx = torch.topk(x, K, dim=1).indices.int()
    dg = torch.randn(T, 1, generator=g, device="cuda").expand(T, K).contiguous()
    coef = 0.01 * torch.rand(1, N, generator=g, device="cuda") / T
    du, dE = torch.empty_like(u), torch.empty(N, d, device="cuda")
    dl = torch.full((T, N), float("nan"), device="cuda")
    ws = torch.empty(moe.moe_route_scored_backward_workspace_size(moe.MOE_BF16, T, d, N),
                     dtype=torch.uint8, device="cuda")
    moe.moe_route_scored_backward(u, E, x, idx, dg, du, dE, ws, score=score, renorm=True,
                                  gate_scale=2.5, balance_coef=coef, d_logit=dl)
    want = S.backward(f64(x), idx.cpu().numpy(), None, [0, T], f64(coef), None, score, True, 2.5)
    assert (np.abs(f64(dl) - want) <= 2.0 ** -20 * 2 * f64(coef).max()).all()


# ------------------------------------------------------------------ sums that cancel

def _cancelling(kind, T, d, N, seed):
    u, E, b = _normal(T, d, N, seed)
    if kind.startswith("pair"):
        _, a, c0, c1 = kind.split("_")
        c0, c1 = int(c0), int(c1) % d
        u[:, c0], u[:, c1] = float(a), -float(a)
        E[:, c0] = E[:, c1] = 1.0
    elif kind == "mean":
        u = (u.float() + 30).to(BF)
        E = (E.float() - E.float().mean(1, keepdim=True)).to(BF)
    elif kind == "outliers":
        k = torch.randperm(d // 2, generator=_gen(seed), device="cuda")[:6]
        u[:, k] = 1000.0
        u[:, k + d // 2] = -1000.0
        E[:, k + d // 2] = E[:, k]
    elif kind == "coherent":
        # running sums rise over half of every 512 columns and come back
        g = _gen(seed + 1)
        u = (4 + 0.4 * torch.randn(T, d, generator=g, device="cuda")).to(BF)
        sign = 1 - 2.0 * (torch.arange(d, device="cuda") // 256 % 2)
        mag = 1 + 0.1 * torch.randn(N, d, generator=g, device="cuda")
        E = (sign * mag * d ** -0.5).to(BF)
    elif kind == "cuts":
        # values of about 1 that cancel from chunk to chunk; every other product lies below what
        # a float32 sum of that size keeps, and their sum tells the experts apart
        c = torch.arange(0, d, 256, device="cuda")[:d // 512 * 2]
        u[:] = 2.0 ** -12
        E[:] = (2.0 ** -13 * (0.5 + torch.randperm(N, device="cuda")[:, None] / N)).to(BF)
        E[:, c] = 1.0
        u[:, c[0::2]], u[:, c[1::2]] = 1.0078125, -1.0078125
        b = None
    elif kind == "vanish":
        # every float32 logit is 0, the exact ones are not: the small term meets a large sum
        e = E[:, 2].clone()
        u[:], E[:] = 0, 0
        u[:, 0], u[:, 20], u[:, 40] = 256.0, 2.0 ** -18, -256.0
        E[:, 0] = E[:, 40] = 1.0
        E[:, 20] = (e.float() * d ** 0.5).to(BF)
        b = None
    return u, E, b


KINDS = ["pair_64_3_4", "pair_64_0_511", "pair_256_5_-3", "pair_4096_0_1", "pair_4096_16_200",
         "mean", "outliers", "coherent", "cuts", "vanish"]


@pytest.mark.parametrize("T", [300, 1500])
@pytest.mark.parametrize("d,N,K", [(512, 64, 6), (7168, 256, 8), (2048, 96, 8)])
@pytest.mark.parametrize("kind", KINDS)
def test_selection_of_cancelling_rows(kind, d, N, K, T):
    u, E, b = _cancelling(kind, T, d, N, 17)
    _check_selection(u, E, b, K, SIG)
    _check_selection(u, E, b, K, SOFT, n_groups=8, topk_groups=4, group_top=2, renorm=False)


@pytest.mark.parametrize("T", [40, 1500])
def test_selection_of_rows_of_zeros_among_others(T):
    """Padding tokens tie everywhere; other rows whose logits are 0 in float32 do not."""
    u, E, _ = _cancelling("vanish", T, 512, 64, 3)
    u[::3] = 0
    u[1::3] = -0.0
    for score in (SIG, SOFT):
        _check_selection(u, E, None, 6, score)


@pytest.mark.parametrize("T", [300, 1500])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_selection_of_rows_of_nan(T, score):
    """Every key of a token with a NaN is NaN, and NaN keys are equal: the lowest ids, in the
    lowest groups."""
    u, E, b = _normal(T, 256, 64, 19)
    clean = _route(u, E, b, 6, score=score)[0]
    rows = [0, 7, T - 1]
    bad = u.clone()
    bad[rows[0]] = float("nan")
    bad[rows[1], 9] = float("nan")
    bad[rows[2], 200] = float("nan")
    for kw in (dict(), dict(n_groups=8, topk_groups=4, group_top=2)):
        idx = _route(bad, E, b, 6, score=score, **kw)[0]
        for r in rows:
            assert idx[r].tolist() == list(range(6)), idx[r]
        if not kw:
            keep = [t for t in range(T) if t not in rows]
            assert torch.equal(idx[keep], clean[keep])


@pytest.mark.parametrize("T", [40, 1300])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_selection_of_rows_past_every_bound(T, score):
    """|u| |E| so large that the float32 logits say nothing: every logit is made exact."""
    u, E, b = _cancelling("pair_65536_3_300", T, 512, 64, 41)
    clean, _, _ = _normal(T, 512, 64, 41)
    u[1::3] = clean[1::3]
    _check_selection(u, E, b, 6, score)
    _check_selection(u, E, b, 6, score, n_groups=8, topk_groups=4, group_top=2, renorm=False)


@pytest.mark.parametrize("T", [9, 300, 1300])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_special_rows_route_as_few_tokens_do(T, score):
    """Infinities of one or both signs, a NaN, huge and tiny rows: what the float64 path of a
    few tokens says, beside ordinary rows."""
    d, N, K = 256, 48, 5
    u, E, b = _normal(T, d, N, 43)
    u[1, 3] = float("inf")
    u[2, 3], u[2, 9] = float("inf"), -float("inf")
    u[3, 200] = float("nan")
    u[4] *= 1e18
    u[5] *= 1e-30
    u[6, :] = -float("inf")
    for kw in (dict(), dict(n_groups=6, topk_groups=3, group_top=2, renorm=False)):
        idx, gate, _ = _route(u, E, b, K, score=score, **kw)
        want, g, _ = _route(u[:8].contiguous(), E, b, K, score=score, **kw)
        assert torch.equal(idx[:8], want), (idx[:8], want)
        nan = torch.isnan(g)
        assert torch.equal(torch.isnan(gate[:8]), nan)
        # ordinary rows' gates come from float32 logits: 2 * 5e-6 |u| |E| of a gate
        assert ((gate[:8] - g).abs()[~nan] <= 4e-4 * g.abs()[~nan] + 1e-30).all()


@pytest.mark.parametrize("T", [5, 300, 1300])
def test_selection_among_scores_below_the_normal_range(T):
    """Sigmoids of logits near -95 are subnormal floats: a rounding of each still orders them."""
    u, E, _ = _normal(T, 512, 64, 47)
    u[:, 0] = 1.0
    E[:, 0] = -95.0
    _check_selection(u, E, None, 6, SIG)
    _check_selection(u, E, None, 6, SIG, n_groups=8, topk_groups=4, group_top=2)


@pytest.mark.parametrize("T", [300, 1300])
@pytest.mark.parametrize("scale", [4, 16, 64])
def test_selection_of_saturated_scores(T, scale):
    """Logits of many standard deviations: scores a few float32 steps below 1, and ties at 1."""
    for N, d, K in ((256, 1024, 8), (64, 512, 40)):
        u, E, b = _normal(T, d, N, 53)
        E = (E.float() * scale).to(BF)
        for score in (SIG, SOFT):
            _check_selection(u, E, b, K, score)
            _check_selection(u, E, None, min(K, 16), score, n_groups=8, topk_groups=4, group_top=2)


# ------------------------------------------------------------------ groups

@pytest.mark.parametrize("T", [64, 1300])
@pytest.mark.parametrize("group_top", [1, 2])
def test_softmax_group_scores_a_rounding_apart(T, group_top):
    """Copies of one token; the bias of one group is moved, a step of its key at a time, over the
    point where the group choice turns.  Other groups keep inexact keys near their best."""
    d, N, G, K = 7168, 32, 4, 2
    for seed in range(8):
        u, E, _ = _normal(1, d, N, 700 + seed)
        u = (u.float() * 3).to(BF)                             # scores of some tenths
        x = f64(u) @ f64(E).T
        s = S.scores(x, S.SOFTMAX).astype(np.float32)
        top = np.sort(s.reshape(G, -1), axis=1)[:, ::-1][:, :group_top].astype(np.float64)
        b = np.zeros(N, np.float32)
        b[0] = 4                                               # group 0 is always kept,
        b[8:24] = 1                                            # then group 1 or group 2
        # where their scores are equal, spread over the group's biases
        diff = (top[1].sum() - top[2].sum()) / group_top
        tokens = u.expand(T, d).contiguous()
        step = 2.0 ** -23
        for k in range(-8, 9):
            b[16:24] = np.float32(round((1.0 + diff) / step) * step) + np.float32(k * step)
            _check_selection(tokens, E, torch.from_numpy(b).cuda(), K, SOFT, n_groups=G,
                             topk_groups=2, group_top=group_top)


@pytest.mark.parametrize("T", [60, 1200])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_groups_beside_a_group_of_nan_or_infinite_keys(T, score):
    """A group that always comes first or last, by a bias of NaN or +-inf, leaves the choice
    among the others what it is."""
    N, G, K = 64, 8, 8
    u, E, b = _normal(T, 2048, N, 29)
    E[24:32] = E[8:16]                             # groups 1 and 3 tie for every token
    b[24:32] = b[8:16]
    clean = b.clone()
    x = f64(u) @ f64(E).T
    for group, value in ((0, float("nan")), (0, float("inf")), (5, -float("inf"))):
        b = clean.clone()
        b[group * 8 + 3] = value
        if value < 0:
            b[group * 8:group * 8 + 8] = value
        idx, _, _ = _route(u, E, b, K, score=score, n_groups=G, topk_groups=4, group_top=1)
        key = S.keys(x, b.cpu().numpy(), score)
        if value != value:
            key[:, group * 8 + 3] = np.inf         # NaN comes first
        want = S.select(key, K, G, 4, 1)
        assert np.array_equal(idx.cpu().numpy(), want)


@pytest.mark.parametrize("T", [1000, 1300])
def test_groups_of_large_biases_that_cancel(T):
    """A group's two keys near 8000 and -8000: a step of a key is 2^-11, a hundred times a
    logit's error.  Where the float32 logit puts a key on the other side of a rounding than the
    exact one, two groups that tie do not seem to."""
    N, G, d = 64, 32, 7168
    base = np.where(np.arange(N) % 2 == 0, 8000.0, -8000.0).astype(np.float32)
    seen_any = 0
    for seed in range(800, 804):
        u, E, _ = _normal(T, d, N, seed)
        lg = torch.empty(T, N, device="cuda")
        _route(u, E, None, 8, logits=lg)
        x = f64(u) @ f64(E).T
        exact, seen = S.keys(x, base, S.SIGMOID), S.keys(f64(lg), base, S.SIGMOID)
        for t, e in np.argwhere(exact != seen)[:6]:
            a = e // 2
            up = seen[t, e] > exact[t, e]
            if a == (0 if up else G - 1):
                continue
            seen_any += 1
            c = (a - 1 if up else a + 1)               # ties keep the lower group
            others = [g for g in range(G) if g not in (a, c)]
            b = base.copy()
            for k, g in enumerate(others):
                b[2 * g] += 100 if k < 15 else -100    # surely kept, surely not
            score = exact[t].reshape(G, 2).sum(1)
            b[2 * c] += score[a] - score[c]            # a whole number of steps: now they tie
            bt = torch.from_numpy(b).cuda()
            idx, _, _ = _route(u, E, bt, 16, n_groups=G, topk_groups=16, group_top=2)
            want = S.select(S.keys(x[t:t + 1], b, S.SIGMOID), 16, G, 16, 2)[0]
            assert np.array_equal(idx[t].cpu().numpy(), want), (t, e, a, c)
    assert seen_any
