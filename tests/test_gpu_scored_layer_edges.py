"""MoELayer and expert-parallel ranks with the scored router's choices: one rounding of du, streams,
memory kept by 8-bit checkpoints, the selection that the balance loss counts, FP8 and float32."""
from dataclasses import replace

import numpy as np
import pytest
import torch

import mixture_experts_layer_60_b200 as moe
from mixture_experts_layer_60_b200.configs import LayerConfig
from mixture_experts_layer_60_b200.layer import MoELayer
from mixture_experts_layer_60_b200.parallel_ep import EPGroupEmulated
from mixture_experts_layer_60_b200.synth import make_layer_inputs, step_u, upstream_grad
from oracle import moe_scored as S
from tests.harness import TOL, assert_close, f64

pytestmark = pytest.mark.gpu

BASE = LayerConfig("scored", T=150, d=256, N_r=16, K=3, N_s=1, I=256, dtype="bf16", seed=43,
                   bias="uniform")


@pytest.mark.parametrize("kw", [dict(), dict(group_top=2, gate_scale=2.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_expert_parallel_ranks_keep_the_group_limit(kw, dtype):
    cfg = replace(BASE, n_groups=4, topk_groups=2, dtype=dtype, **kw)
    w = make_layer_inputs(cfg, "cuda")
    us = [step_u(cfg, s, "cuda") for s in range(2)]
    us[1] = us[1][:33].contiguous()
    ep = EPGroupEmulated(cfg, w, 2, T_max=cfg.T)
    hs = [h.clone() for h in ep.forward(us)]
    torch.cuda.synchronize()
    for s, u in enumerate(us):
        one = MoELayer(cfg, w, T_max=u.shape[0])
        want = one.forward(u)
        assert torch.equal(ep.ranks[s].topk_idx[:u.shape[0]], one.topk_idx)
        assert torch.equal(hs[s], want)


def test_first_training_step_on_a_stream_of_its_own():
    """Buffers that a first step makes are ready on the step's stream, whatever the current one
    is busy with."""
    cfg = replace(BASE, score="softmax")
    w = make_layer_inputs(cfg, "cuda")
    dh = upstream_grad(cfg, "cuda")
    ref = MoELayer(cfg, w)
    ref.forward_train(w["u"])
    want = ref.backward(dh).clone()
    lay = MoELayer(cfg, w)
    st = torch.cuda.Stream()
    junk = [torch.full((cfg.T, cfg.K), float("nan"), device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    del junk                                       # their memory is handed out next
    torch.cuda._sleep(int(3e8))                    # the current stream is busy for a while
    lay.forward_train(w["u"], stream=st)
    got = lay.backward(dh, stream=st)
    st.synchronize()
    got = got.cpu()
    torch.cuda.synchronize()
    assert torch.equal(got, want.cpu())


def test_a_new_token_count_on_a_stream_of_its_own():
    """Nothing that the layer clears for a new token count is cleared after the step has used it."""
    cfg = replace(BASE, score="softmax")
    w = make_layer_inputs(cfg, "cuda")
    lay = MoELayer(cfg, w)
    u = w["u"][:70].contiguous()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(int(3e8))
    lay.forward(u, stream=st)
    torch.cuda.synchronize()
    assert int(lay.counts.sum()) == int(lay.offsets[-1]) == 70 * cfg.K


@pytest.mark.parametrize("kw", [dict(score="softmax"), dict(renorm=False, N_s=0),
                                dict(balance_alpha=0.05, N_s=2)])
def test_du_of_a_scored_layer_is_rounded_once(kw):
    """du is the sum of dh, the experts' and the router's parts, each of them bf16 (half a step,
    2^-8 of the value, lies in the router's), rounded once (2^-8) from float32 sums (2^-18)."""
    cfg = replace(BASE, **kw)
    w = make_layer_inputs(cfg, "cuda")
    lay = MoELayer(cfg, w)
    lay.forward_train(w["u"])
    dh = upstream_grad(cfg, "cuda")
    du = lay.backward(dh)
    T, N, d = cfg.T, cfg.N_r, cfg.d
    dl = torch.empty(T, N, device="cuda")
    bal = cfg.balance_alpha > 0
    moe.moe_route_scored_backward(w["u"], w["E"], lay.logits, lay.topk_idx, lay.d_gate,
                                  torch.empty_like(w["u"]), torch.empty(N, d, device="cuda"),
                                  lay.route_bwd_ws, score=lay.score, renorm=cfg.renorm,
                                  gate_scale=cfg.gate_scale,
                                  balance_coef=lay.balance_coef if bal else None, d_logit=dl)
    router = f64(dl) @ f64(w["E"])
    parts = [f64(dh), router] + [f64(lay.dx_s[j]) for j in range(cfg.N_s)] + \
        [f64(lay.dx_perm)[lay.inv_row.cpu().numpy()[:, k]] for k in range(cfg.K)]
    want, mag = sum(parts), sum(np.abs(p) for p in parts)
    tol = 2.0 ** -8 * (np.abs(want) + np.abs(router)) + 2.0 ** -15 * np.abs(f64(dl)) @ np.abs(f64(w["E"])) \
        + 2.0 ** -18 * mag
    err = np.abs(f64(du) - want)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size}, worst {(err / tol).max():.2f}"


@pytest.mark.parametrize("N_s", [0, 1, 2])
def test_checkpoint8_keeps_fewer_bytes(N_s):
    """What a layer holds after a training step: 2.06 I bytes of codes and scales a row instead
    of 4 I of pre-activations; the forward's h lies where the backward forms it again."""
    cfg = replace(BASE, T=2048, K=4, N_s=N_s, d=256, I=512)
    w = make_layer_inputs(cfg, "cuda")
    dh = upstream_grad(cfg, "cuda")
    held = {}
    for c8 in (False, True):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        lay = MoELayer(replace(cfg, checkpoint8=c8), w)
        lay.forward_train(w["u"])
        lay.backward(dh)
        torch.cuda.synchronize()
        held[c8] = torch.cuda.memory_allocated() - before
        del lay
    rows, I = cfg.T * (cfg.K + N_s), cfg.I
    want = rows * (4 * I - 2 * I - 2 * I / 32)     # bytes that the codes and scales free
    # buffers are handed out in blocks of 512 bytes and up to 2 MB
    assert held[False] - held[True] >= 0.9 * want, (held, want)


def test_checkpoint8_layer_changes_its_token_count():
    cfg = replace(BASE, checkpoint8=True, N_s=2)
    w = make_layer_inputs(cfg, "cuda")
    dh = upstream_grad(cfg, "cuda")
    lay = MoELayer(cfg, w)
    plain = MoELayer(replace(cfg, checkpoint8=False), w)
    for T in (150, 70, 150):
        u, g = w["u"][:T].contiguous(), dh[:T].contiguous()
        assert torch.equal(lay.forward(u), plain.forward(u))
        h = lay.forward_train(u).clone()
        assert torch.equal(h, plain.forward_train(u))
        first = lay.backward(g).clone()
        # inference in between with another token count, then the step again
        lay.forward(w["u"][:33].contiguous())
        assert torch.equal(lay.forward_train(u), h)
        assert torch.equal(lay.backward(g), first)


@pytest.mark.parametrize("kw", [dict(d=384), dict(I=384)])
def test_checkpoint8_refuses_its_shape_when_the_layer_is_made(kw):
    cfg = replace(BASE, checkpoint8=True, **kw)
    w = make_layer_inputs(cfg, "cuda")
    with pytest.raises(ValueError, match="256"):
        MoELayer(cfg, w)


@pytest.mark.parametrize("kw", [dict(), dict(score="softmax", renorm=False),
                                dict(n_groups=4, topk_groups=2, group_top=2)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_balance_loss_of_the_unbiased_choice(kw, dtype):
    """f_i counts the top K of the scores over all experts, whatever bias and groups route."""
    cfg = replace(BASE, balance_alpha=1.0, balance_unbiased=True, dtype=dtype, **kw)
    w = make_layer_inputs(cfg, "cuda")
    w["b"] = torch.linspace(0.4, -0.4, cfg.N_r, device="cuda")
    off = [0, 40, 40, 130]
    ot = torch.tensor(off, dtype=torch.int32, device="cuda")
    lay = MoELayer(cfg, w)
    routed = MoELayer(replace(cfg, balance_unbiased=False), w)
    h = lay.forward_train(w["u"], seq_offsets=ot).clone()
    assert torch.equal(h, routed.forward_train(w["u"], seq_offsets=ot)), "the loss routes nothing"
    assert torch.equal(lay.topk_idx, routed.topk_idx) and torch.equal(lay.counts, routed.counts)
    soft = cfg.score == "softmax"
    x = f64(w["u"]) @ f64(w["E"]).T
    idx = S.select(S.keys(x, None, S.SOFTMAX if soft else S.SIGMOID), cfg.K)
    want, coef = S.balance(x, idx, off, 1.0, S.SOFTMAX if soft else S.SIGMOID)
    # a score moves by at most its logit's error (5e-6 |u| |E|, some 1e-4 here)
    assert_close(f64(lay.balance), want, 2e-4, "balance loss")
    assert (np.abs(f64(lay.balance_coef) - coef) <= 2.0 ** -23 * coef).all()
    assert not torch.equal(lay.balance, routed.balance)
    # its gradient, without any of the gates'
    dh = torch.zeros_like(w["u"])
    lay.backward(dh)
    t = torch.from_numpy(x).requires_grad_()
    s = torch.softmax(t, 1) if soft else torch.sigmoid(t)
    sn = s / s.sum(1, keepdim=True)
    loss = sum((torch.from_numpy(coef[q]) * sn[a:b].sum(0)).sum()
               for q, (a, b) in enumerate(zip(off[:-1], off[1:])))
    loss.backward()
    assert_close(f64(lay.grad["E"]), t.grad.numpy().T @ f64(w["u"]), 2e-3, "dE")


VARIANTS = [dict(score="softmax"), dict(renorm=False, gate_scale=4.0, balance_alpha=0.02),
            dict(gate_scale=2.5, n_groups=4, topk_groups=2, group_top=2, N_s=0)]


@pytest.mark.parametrize("kw", VARIANTS)
@pytest.mark.parametrize("dtype", ["f32", "e4m3"])
def test_forward_of_other_types_with_the_scored_router(kw, dtype):
    """Selection by the definition; h' from the layer's own expert outputs, gates and load:
    float32 sums, rounded once."""
    cfg = replace(BASE, dtype=dtype, **kw)
    w = make_layer_inputs(cfg, "cuda")
    lay = MoELayer(cfg, w)
    h = lay.forward(w["u"])
    x = f64(w["u"]) @ f64(w["E"]).T
    score = S.SOFTMAX if cfg.score == "softmax" else S.SIGMOID
    want = S.select(S.keys(x, w["b"].cpu().numpy(), score), cfg.K, cfg.n_groups, cfg.topk_groups,
                    cfg.group_top)
    assert np.array_equal(lay.topk_idx.cpu().numpy(), want)
    assert np.array_equal(lay.counts.cpu().numpy(), np.bincount(want.reshape(-1), minlength=cfg.N_r))
    g = S.gates(x, want, score, cfg.renorm, cfg.gate_scale)
    # float32 layers route from float64 logits; bf16 inputs: 5e-6 |u| |E| of a logit, some 1e-4
    assert_close(f64(lay.topk_gate), g, 1e-6 if dtype == "f32" else 4e-4, "gates")
    rows = lay.inv_row.cpu().numpy()
    parts = [f64(w["u"])] + [f64(lay.y_shared[j]) for j in range(cfg.N_s)] + \
        [f64(lay.topk_gate)[:, k:k + 1] * f64(lay.y_perm)[rows[:, k]] for k in range(cfg.K)]
    mag = sum(np.abs(p) for p in parts)
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    assert (np.abs(f64(h) - sum(parts)) <= half * np.abs(sum(parts)) + 2.0 ** -20 * mag).all()


@pytest.mark.parametrize("kw", VARIANTS)
def test_training_step_of_an_fp8_layer_with_the_scored_router(kw):
    """The step's parts against each other: d_gate from the expert outputs, dE and the router's
    share of du from d_gate by the definition, du their sum."""
    cfg = replace(BASE, dtype="e4m3", **kw)
    w = make_layer_inputs(cfg, "cuda")
    lay = MoELayer(cfg, w)
    h = lay.forward_train(w["u"]).clone()
    assert torch.equal(h, MoELayer(cfg, w).forward(w["u"]))
    dh = upstream_grad(cfg, "cuda")
    du = lay.backward(dh)
    torch.cuda.synchronize()
    assert moe.moe_device_status() == 0
    rows, idx = lay.inv_row.cpu().numpy(), lay.topk_idx.cpu().numpy()
    y, g = f64(lay.y_perm), f64(dh)
    dots = np.stack([(y[rows[:, k]] * g).sum(1) for k in range(cfg.K)], 1)
    size = np.stack([np.abs(y[rows[:, k]] * g).sum(1) for k in range(cfg.K)], 1)
    assert (np.abs(f64(lay.d_gate) - dots) <= 2.0 ** -18 * size).all()
    score = S.SOFTMAX if cfg.score == "softmax" else S.SIGMOID
    bal = cfg.balance_alpha > 0
    x, T = f64(lay.logits), cfg.T
    dl = S.backward(x, idx, f64(lay.d_gate), [0, T], f64(lay.balance_coef) if bal else None, None,
                    score, cfg.renorm, cfg.gate_scale)
    E, u = f64(w["E"]), f64(w["u"])
    size = 2 * cfg.gate_scale * np.abs(f64(lay.d_gate)).sum(1, keepdims=True) + \
        (2 * f64(lay.balance_coef).max() if bal else 0)          # of d_logit, 2^-20 of it its error
    want = dl.T @ u
    err = np.abs(f64(lay.grad["E"]) - want)
    assert (err <= 2.0 ** -18 * (np.abs(dl).T @ np.abs(u)) + 2.0 ** -20 * (size * np.ones_like(dl)).T
            @ np.abs(u)).all()
    router = dl @ E
    parts = [g, router] + [f64(lay.dx_s[j]) for j in range(cfg.N_s)] + \
        [f64(lay.dx_perm)[rows[:, k]] for k in range(cfg.K)]
    mag = sum(np.abs(p) for p in parts)
    tol = 2.0 ** -8 * (np.abs(sum(parts)) + np.abs(router)) + 2.0 ** -18 * mag + \
        2.0 ** -15 * (np.abs(dl) + size) @ np.abs(E)
    assert (np.abs(f64(du) - sum(parts)) <= tol).all()
    for k in ("W_gate_up", "W_down"):
        assert torch.isfinite(lay.grad[k].float()).all()


@pytest.mark.parametrize("kw", VARIANTS)
def test_expert_parallel_float32_ranks_with_the_scored_router(kw):
    cfg = replace(BASE, dtype="f32", **kw)
    w = make_layer_inputs(cfg, "cuda")
    us = [step_u(cfg, s, "cuda") for s in range(2)]
    us[1] = us[1][:7].contiguous()
    hs = [h.clone() for h in EPGroupEmulated(cfg, w, 2, T_max=cfg.T).forward(us)]
    for s, u in enumerate(us):
        assert torch.equal(hs[s], MoELayer(cfg, w, T_max=u.shape[0]).forward(u))
