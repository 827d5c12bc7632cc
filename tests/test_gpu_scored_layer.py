"""MoELayer with the scored router, its balance loss and 8-bit checkpoints: a run of the calls
together (route, permute, experts, combine; their backward) against automatic differentiation of
the layer's equations in float64, the selection held at the GPU's."""
from dataclasses import replace

import numpy as np
import pytest
import torch

from mixture_experts_layer_60_b200 import moe_device_status
from mixture_experts_layer_60_b200.configs import LayerConfig
from mixture_experts_layer_60_b200.layer import MoELayer
from mixture_experts_layer_60_b200.parallel_ep import EPGroupEmulated
from mixture_experts_layer_60_b200.synth import make_layer_inputs, step_u, upstream_grad
from oracle import moe_scored as S
from tests.harness import TOL, assert_close, f64

pytestmark = pytest.mark.gpu
BF = TOL["bf16"]

BASE = LayerConfig("scored", T=150, d=256, N_r=16, K=3, N_s=1, I=256, dtype="bf16", seed=41,
                   bias="uniform")
VARIANTS = [
    dict(score="softmax"),
    dict(score="softmax", renorm=False, gate_scale=4.0, balance_alpha=0.02),
    dict(gate_scale=2.5, n_groups=4, topk_groups=2, group_top=2, balance_alpha=0.02),
    dict(renorm=False, N_s=0, K=1),
    dict(balance_alpha=0.05, N_s=2),
]


def _autograd(w, cfg, idx, dh, off, d_balance):
    """(h', balance, gradients) of the layer in float64."""
    t = {k: w[k].detach().cpu().double().requires_grad_() for k in
         ("u", "E", "W_gate_up", "W_down", "Ws_gate_up", "Ws_down")}
    u, I = t["u"], cfg.I
    x = u @ t["E"].T
    s = torch.sigmoid(x) if cfg.score == "sigmoid" else torch.softmax(x, 1)
    ids = torch.from_numpy(idx.astype(np.int64))
    g = s.gather(1, ids)
    g = cfg.gate_scale * (g / g.sum(1, keepdim=True) if cfg.renorm else g)

    def ffn(z, gu, dn):
        a = z @ gu.T
        return (torch.nn.functional.silu(a[:, :I]) * a[:, I:]) @ dn.T
    h = u
    for j in range(cfg.N_s):
        h = h + ffn(u, t["Ws_gate_up"][j], t["Ws_down"][j])
    for e in range(cfg.N_r):
        rows, k = (ids == e).nonzero(as_tuple=True)
        if len(rows):
            y = g[rows, k][:, None] * ffn(u[rows], t["W_gate_up"][e], t["W_down"][e])
            h = h.index_add(0, rows, y)
    total = (h * dh).sum()
    bal = []
    if cfg.balance_alpha > 0:
        sn = s / s.sum(1, keepdim=True)
        for q, (a, b) in enumerate(zip(off[:-1], off[1:])):
            f = torch.bincount(ids[a:b].reshape(-1), minlength=cfg.N_r) * cfg.N_r / (cfg.K * max(1, b - a))
            bal.append(cfg.balance_alpha * (f * sn[a:b].sum(0) / max(1, b - a)).sum())
            total = total + d_balance[q] * bal[-1]
    total.backward()
    return h.detach(), [float(b.detach()) for b in bal], {k: v.grad for k, v in t.items()}


@pytest.mark.parametrize("kw", VARIANTS)
def test_training_step_of_a_scored_layer(kw):
    cfg = replace(BASE, **kw)
    assert cfg.scored
    w = make_layer_inputs(cfg, "cuda")
    lay = MoELayer(cfg, w)
    off = [0, 40, 40, 130]                       # an empty sequence, rows behind the last
    ot = torch.tensor(off, dtype=torch.int32, device="cuda")
    d_bal = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    h = lay.forward_train(w["u"], seq_offsets=ot).clone()
    assert torch.equal(h, MoELayer(cfg, w).forward(w["u"])), "forward_train is the forward"
    dh = upstream_grad(cfg, "cuda")
    du = lay.backward(dh, d_balance=d_bal)
    torch.cuda.synchronize()
    assert moe_device_status() == 0
    idx = lay.topk_idx.cpu().numpy()
    want = S.select(S.keys(f64(w["u"]) @ f64(w["E"]).T, w["b"].cpu().numpy(),
                           S.SOFTMAX if cfg.score == "softmax" else S.SIGMOID),
                    cfg.K, cfg.n_groups, cfg.topk_groups, cfg.group_top)
    assert np.array_equal(idx, want)
    ref_h, bal, ref = _autograd(w, cfg, idx, dh.cpu().double(), off, d_bal.cpu().double())
    assert_close(f64(h), ref_h.numpy(), BF, "h'")
    if bal:
        # a score moves by at most a quarter of its logit's error (1e-5) over a score of order 1/2
        assert_close(f64(lay.balance), np.array(bal), 2e-5, "balance loss")
    assert_close(f64(du), ref["u"].numpy(), BF, "du")
    assert_close(f64(lay.grad["E"]), ref["E"].numpy(), BF, "dE")
    for k in ("W_gate_up", "W_down") + (("Ws_gate_up", "Ws_down") if cfg.N_s else ()):
        assert_close(f64(lay.grad[k]), ref[k].numpy(), BF, k)


def test_default_router_is_not_scored():
    assert not BASE.scored and replace(BASE, checkpoint8=True).scored is False


@pytest.mark.parametrize("kw", [dict(), dict(score="softmax", balance_alpha=0.01)])
def test_training_step_with_8_bit_checkpoints(kw):
    """The forward is the same; the gradients are those of pre-activations that moved by at most
    2^-4 of their value (2^-5 on average): every gradient within 2^-4 of the exact one in norm,
    and bit for bit what another step gives."""
    cfg = replace(BASE, **kw)
    w = make_layer_inputs(cfg, "cuda")
    full, kept = MoELayer(cfg, w), MoELayer(replace(cfg, checkpoint8=True), w)
    dh = upstream_grad(cfg, "cuda")
    assert torch.equal(full.forward_train(w["u"]), kept.forward_train(w["u"]))
    du, dk = full.backward(dh), kept.backward(dh)
    torch.cuda.synchronize()
    assert moe_device_status() == 0
    first = {k: v.clone() for k, v in kept.grad.items()}
    for name, a, b in [("du", du, dk)] + [(k, full.grad[k], kept.grad[k]) for k in full.grad]:
        err = ((a.double() - b.double()).norm() / a.double().norm()).item()
        assert err <= 2.0 ** -4, (name, err)
    dk = dk.clone()
    kept.forward_train(w["u"])
    assert torch.equal(kept.backward(dh), dk)
    for k, v in first.items():
        assert torch.equal(v, kept.grad[k]), k


def test_training_step_follows_the_stream_and_the_token_count():
    cfg = replace(BASE, score="softmax", balance_alpha=0.01, checkpoint8=True)
    w = make_layer_inputs(cfg, "cuda")
    lay = MoELayer(cfg, w)
    dh = upstream_grad(cfg, "cuda")
    h = lay.forward_train(w["u"]).clone()
    du = lay.backward(dh).clone()
    part = w["u"][:70].contiguous()
    lay.forward_train(part)
    lay.backward(dh[:70].contiguous())
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        h2 = lay.forward_train(w["u"]).clone()
        du2 = lay.backward(dh).clone()
    st.synchronize()
    assert torch.equal(h, h2) and torch.equal(du, du2)


def test_unknown_choices_are_refused():
    w = make_layer_inputs(BASE, "cuda")
    with pytest.raises(ValueError):
        MoELayer(replace(BASE, score="tanh"), w)
    with pytest.raises(ValueError):
        MoELayer(replace(BASE, dtype="e4m3", checkpoint8=True), w)


def test_expert_parallel_ranks_use_the_scored_router():
    cfg = replace(BASE, score="softmax", renorm=False, gate_scale=2.0, n_groups=4, topk_groups=2,
                  group_top=2)
    w = make_layer_inputs(cfg, "cuda")
    us = [step_u(cfg, s, "cuda") for s in range(2)]
    us[1] = us[1][:33].contiguous()
    hs = EPGroupEmulated(cfg, w, 2, T_max=cfg.T).forward(us)
    torch.cuda.synchronize()
    for s, u in enumerate(us):
        assert torch.equal(hs[s], MoELayer(cfg, w, T_max=u.shape[0]).forward(u))
