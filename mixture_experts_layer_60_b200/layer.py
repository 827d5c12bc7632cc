"""The DeepSeekMoE layer step built from the C-ABI calls.

MoELayer owns the layer's device state (centroids, bias, expert weights,
FP8 copies of them) and the per-step buffers, and runs one step as
    moe_route -> [moe_quantize_1x128] -> moe_permute
    -> gate/up and down of the routed experts (bf16: with the shared experts
       as extra groups of the same two launches; FP8 / f32: the shared
       experts' moe_expert_ffn after them) -> moe_combine [-> moe_bias_update]
on one CUDA stream.  For training (bf16 or FP8), forward_train keeps the
activations the backward needs and backward(dh) returns du and fills
self.grad with the gradients of E and of every expert weight.  A configuration
whose router differs from moe_route's (softmax scores, group scores of two
keys, raw or scaled gates, a balance loss) routes with moe_route_scored, and
its backward ends in moe_route_scored_backward; checkpoint8 keeps the gate/up
pre-activations in 8 bits between forward_train and backward.  Every step of the layer runs in libmoe's kernels; this
module only allocates buffers and sequences calls.
"""
from __future__ import annotations

import contextlib

import torch

from . import (MOE_BF16, MOE_E4M3, MOE_F32, MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX,
               moe_balance_loss, moe_balance_loss_workspace_size, moe_bias_update, moe_combine,
               moe_combine_backward,
               moe_expert_down, moe_expert_down_shared, moe_expert_ffn, moe_expert_ffn_backward,
               moe_expert_ffn_backward_workspace_size, moe_expert_ffn_workspace_size,
               moe_expert_ffn_backward8, moe_expert_ffn_backward8_workspace_size,
               moe_expert_gate_up, moe_expert_gate_up_save, moe_expert_gate_up_save8,
               moe_expert_gate_up_shared, moe_permute,
               moe_permute_workspace_size, moe_quantize_128x128, moe_quantize_1x128, moe_route,
               moe_route_grouped, moe_route_scored, moe_route_scored_backward,
               moe_route_scored_backward_workspace_size, moe_route_scored_workspace_size,
               moe_route_workspace_size, moe_router_weight_grad,
               moe_unpermute_backward)
from .configs import LayerConfig

GAMMA = 0.001


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _on(stream):
    """The stream of a step as PyTorch's current one: what a step's buffers are cleared or
    filled with comes before the step's kernels."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream")
                             else torch.cuda.ExternalStream(int(stream)))


class MoELayer:
    def __init__(self, cfg: LayerConfig, weights: dict, T_max: int | None = None, device="cuda"):
        self.cfg = cfg
        self.device = torch.device(device)
        self.T_max = cfg.T if T_max is None else T_max
        self.E = weights["E"]
        self.b = weights["b"].clone()
        self.fp8 = cfg.dtype == "e4m3"
        if cfg.score not in ("sigmoid", "softmax"):
            raise ValueError(f"unknown router score {cfg.score!r}")
        if cfg.checkpoint8 and cfg.dtype != "bf16":
            raise ValueError("8-bit activation checkpoints are implemented for bf16 layers")
        if cfg.checkpoint8 and (cfg.d % 256 or cfg.I % 256):
            raise ValueError(f"8-bit activation checkpoints need d={cfg.d} and I={cfg.I} to be "
                             "multiples of 256")
        self.score = MOE_SCORE_SOFTMAX if cfg.score == "softmax" else MOE_SCORE_SIGMOID
        if self.fp8:
            self.W = {k: self._quantise(weights[k]) for k in
                      ("W_gate_up", "W_down", "Ws_gate_up", "Ws_down")}
        else:
            self.W = {k: (weights[k], None) for k in ("W_gate_up", "W_down", "Ws_gate_up", "Ws_down")}
        self._alloc(self.T_max)

    # -- setup ---------------------------------------------------------------
    def _quantise(self, w):
        G, R, C = w.shape
        q = torch.empty(G, R, C, dtype=torch.uint8, device=self.device)
        s = torch.empty(G, R // 128, C // 128, dtype=torch.float32, device=self.device)
        moe_quantize_128x128(w, q, s)
        return q, s

    def _alloc(self, T):
        c, dev = self.cfg, self.device
        d, K, N_r, N_s = c.d, c.K, c.N_r, c.N_s
        R = T * K
        act = torch.float32 if c.dtype == "f32" else torch.bfloat16
        xdt = torch.uint8 if self.fp8 else act
        ffn_dt = {"f32": MOE_F32, "bf16": MOE_BF16, "e4m3": MOE_E4M3}[c.dtype]
        self.topk_idx = torch.empty(T, K, dtype=torch.int32, device=dev)
        self.topk_gate = torch.empty(T, K, dtype=torch.float32, device=dev)
        self.counts = torch.zeros(N_r, dtype=torch.int32, device=dev)
        self.route_ws = _ws(moe_route_scored_workspace_size(T, d, N_r) if c.scored
                            else moe_route_workspace_size(T, N_r), dev)
        self.perm_ws = _ws(moe_permute_workspace_size(T, N_r), dev)
        self.x_perm = torch.empty(R, d, dtype=xdt, device=dev)
        self.offsets = torch.zeros(N_r + 1, dtype=torch.int32, device=dev)
        self.perm_src = torch.empty(R, dtype=torch.int32, device=dev)
        self.inv_row = torch.empty(T, K, dtype=torch.int32, device=dev)
        # bf16: the shared experts run as extra groups of the routed launches,
        # their rows after the routed ones in the same h and y buffers
        self.merged_shared = (c.dtype == "bf16" and N_s > 0 and d % 256 == 0
                              and c.I % 128 == 0)
        self.y_all = torch.empty(R + N_s * T, d, dtype=act, device=dev)
        self.y_perm = self.y_all[:R]
        self.y_shared = self.y_all[R:].view(N_s, T, d)
        self.ffn_ws = _ws(moe_expert_ffn_workspace_size(ffn_dt, T, c.I), dev)
        hdt = torch.uint8 if self.fp8 else act
        self.h_all = torch.empty(R + (N_s * T if self.merged_shared else 0), c.I, dtype=hdt,
                                 device=dev)
        self.h_mid = self.h_all[:R]
        self.h_scale = torch.empty(R, c.I // 128, dtype=torch.float32, device=dev) if self.fp8 \
            else None
        self.h_out = torch.empty(T, d, dtype=act, device=dev)
        self.shared_offsets = torch.tensor([0, T], dtype=torch.int32, device=dev)
        if self.fp8:
            self.u_q = torch.empty(T, d, dtype=torch.uint8, device=dev)
            self.u_s = torch.empty(T, d // 128, dtype=torch.float32, device=dev)
            self.x_scale = torch.empty(R, d // 128, dtype=torch.float32, device=dev)
        self.T_alloc = T
        if c.checkpoint8:
            self.T_train = None                # h lies in a training step's workspace

    def _route(self, u, stream, logits=None):
        c = self.cfg
        out = (self.topk_idx, self.topk_gate, self.counts, self.route_ws)
        if c.scored:
            moe_route_scored(u, self.E, self.b, c.K, *out, score=self.score, n_groups=c.n_groups,
                             topk_groups=c.topk_groups, group_top=c.group_top, renorm=c.renorm,
                             gate_scale=c.gate_scale, logits=logits, stream=stream)
        elif c.n_groups > 1:
            moe_route_grouped(u, self.E, self.b, c.K, c.n_groups, c.topk_groups, *out, stream)
        else:
            moe_route(u, self.E, self.b, c.K, *out, stream)

    # -- one step ------------------------------------------------------------
    def forward(self, u: torch.Tensor, stream=None, gate_up_events=None,
                out: torch.Tensor | None = None, phase_events=None) -> torch.Tensor:
        """h' for the T tokens of u, written to `out` (default: the layer's own
        h_out buffer, overwritten by the next call).  gate_up_events=(start,
        end) records CUDA events around the routed gate/up GEMM launch on the
        same stream; phase_events, a dict name -> (start, end) for any of
        "route", "permute", "gate_up", "down", "shared", "combine", records
        events around those phases."""
        c = self.cfg
        T = u.shape[0]
        if T != self.T_alloc:
            with _on(stream):
                self._alloc(T)
        st = torch.cuda.current_stream() if stream is None else stream
        pe = phase_events or {}
        if gate_up_events:
            pe = dict(pe, gate_up=gate_up_events)

        def mark(name, i):
            if name in pe:
                pe[name][i].record(st)
        mark("route", 0)
        self._route(u, stream)
        mark("route", 1)
        mark("permute", 0)
        if self.fp8:
            moe_quantize_1x128(u, self.u_q, self.u_s, stream)
            moe_permute(self.u_q, self.topk_idx, c.N_r, self.x_perm, self.offsets, self.perm_src,
                        self.inv_row, self.perm_ws, u_scale=self.u_s, x_scale=self.x_scale,
                        stream=stream)
            x_sh, xs_sh = self.u_q, self.u_s
        else:
            moe_permute(u, self.topk_idx, c.N_r, self.x_perm, self.offsets, self.perm_src,
                        self.inv_row, self.perm_ws, stream=stream)
            x_sh, xs_sh = u, None
        mark("permute", 1)
        (wgu, sgu), (wdn, sdn) = self.W["W_gate_up"], self.W["W_down"]
        (wsgu, ssgu), (wsdn, ssdn) = self.W["Ws_gate_up"], self.W["Ws_down"]
        if self.merged_shared:
            # routed + shared experts: one gate/up launch, one down launch
            mark("gate_up", 0)
            moe_expert_gate_up_shared(self.x_perm, self.offsets, wgu, u, wsgu, self.h_all,
                                      stream=stream)
            mark("gate_up", 1)
            mark("down", 0)
            moe_expert_down_shared(self.h_all, self.offsets, wdn, wsdn, T * c.K, T, self.y_all,
                                   stream=stream)
            mark("down", 1)
        else:
            mark("gate_up", 0)
            moe_expert_gate_up(self.x_perm, self.offsets, wgu, self.h_mid,
                               x_scale=self.x_scale if self.fp8 else None, w_scale_gate_up=sgu,
                               h_scale=self.h_scale, stream=stream)
            mark("gate_up", 1)
            mark("down", 0)
            moe_expert_down(self.h_mid, self.offsets, wdn, self.y_perm, h_scale=self.h_scale,
                            w_scale_down=sdn, stream=stream)
            mark("down", 1)
            mark("shared", 0)
            for j in range(c.N_s):
                moe_expert_ffn(x_sh, self.shared_offsets, wsgu[j:j + 1], wsdn[j:j + 1],
                               self.y_shared[j], self.ffn_ws, x_scale=xs_sh,
                               w_scale_gate_up=None if ssgu is None else ssgu[j:j + 1],
                               w_scale_down=None if ssdn is None else ssdn[j:j + 1],
                               stream=stream)
            mark("shared", 1)
        u_res = u
        h = self.h_out if out is None else out
        mark("combine", 0)
        moe_combine(u_res, self.y_shared if c.N_s else None, self.y_perm, self.inv_row,
                    self.topk_gate, h, stream)
        mark("combine", 1)
        return h

    # -- training (bf16 / FP8): forward that keeps activations, then the backward
    def _alloc_train(self, T):
        c, dev = self.cfg, self.device
        R, bf = T * c.K, torch.bfloat16
        hdt = torch.uint8 if self.fp8 else bf
        dt = MOE_E4M3 if self.fp8 else MOE_BF16
        if c.checkpoint8:
            # pre-activations as E4M3 codes and a scale for each row and 128 columns
            pair = lambda rows: (torch.empty(rows, 2 * c.I, dtype=torch.uint8, device=dev),
                                 torch.empty(rows, 2 * c.I // 128, dtype=torch.float32, device=dev))
            self.a_gu, self.a_s = pair(R), [pair(T) for _ in range(c.N_s)]
            # the forward's h is not kept: it lies where the backward forms h again,
            # the last R rows of its workspace, the shared experts' behind it
            size = moe_expert_ffn_backward8_workspace_size
            at = size(dt, R, c.d, c.I, c.N_r) - 2 * R * c.I
            rows = R + c.N_s * T
            self.h_all = self.h_mid = None
            self.bwd_ws = _ws(max(at + 2 * rows * c.I, size(dt, T, c.d, c.I, 1)), dev)
            self.h_all = self.bwd_ws[at:at + 2 * rows * c.I].view(bf).view(rows, c.I)
            self.h_mid, self.h_s = self.h_all[:R], self.h_all[R:].view(c.N_s, T, c.I)
        else:
            self.a_gu = torch.empty(R, 2 * c.I, dtype=bf, device=dev)
            self.a_s = torch.empty(c.N_s, T, 2 * c.I, dtype=bf, device=dev)
            self.h_s = torch.empty(c.N_s, T, c.I, dtype=hdt, device=dev)
            size = moe_expert_ffn_backward_workspace_size
            self.bwd_ws = _ws(max(size(dt, R, c.d, c.I, c.N_r), size(dt, T, c.d, c.I, 1)), dev)
        self.h_s_scale = torch.empty(c.N_s, T, c.I // 128, dtype=torch.float32, device=dev) \
            if self.fp8 else None
        self.dy_perm = torch.empty(R, c.d, dtype=bf, device=dev)
        self.d_gate = torch.empty(T, c.K, dtype=torch.float32, device=dev)
        self.d_logit = torch.empty(T, c.K, dtype=torch.float32, device=dev)
        self.d_logit_perm = torch.empty(R, dtype=torch.float32, device=dev)
        self.dx_perm = torch.empty(R, c.d, dtype=bf, device=dev)
        # a scored router's own part of du lies behind the shared experts'
        self.dx_s = torch.empty(c.N_s + c.scored, T, c.d, dtype=bf, device=dev)
        self.du = torch.empty(T, c.d, dtype=bf, device=dev)
        if c.scored:
            rdt = MOE_F32 if self.E.dtype == torch.float32 else MOE_BF16
            self.logits = torch.empty(T, c.N_r, dtype=torch.float32, device=dev)
            self.ones = torch.ones(T, c.K, dtype=torch.float32, device=dev)
            if c.balance_unbiased:
                self.free_choice = (torch.empty(T, c.K, dtype=torch.int32, device=dev),
                                    torch.empty(T, c.K, dtype=torch.float32, device=dev),
                                    torch.empty(c.N_r, dtype=torch.int32, device=dev))
            self.route_bwd_ws = _ws(moe_route_scored_backward_workspace_size(rdt, T, c.d, c.N_r),
                                    dev)
        if not hasattr(self, "grad"):
            self.grad = {k: torch.empty(self.W[k][0].shape, dtype=bf, device=dev) for k in
                         ("W_gate_up", "W_down", "Ws_gate_up", "Ws_down")}
            self.grad["E"] = torch.empty(c.N_r, c.d, dtype=torch.float32, device=dev)
        self.T_train = T

    def _gate_up_save(self, x, offsets, wgu, h, keep, stream, x_scale=None, w_scale=None,
                      h_scale=None):
        if self.cfg.checkpoint8:
            moe_expert_gate_up_save8(x, offsets, wgu, h, *keep, stream=stream)
        else:
            moe_expert_gate_up_save(x, offsets, wgu, h, keep, x_scale=x_scale,
                                    w_scale_gate_up=w_scale, h_scale=h_scale, stream=stream)

    def forward_train(self, u: torch.Tensor, stream=None,
                      seq_offsets: torch.Tensor | None = None) -> torch.Tensor:
        """forward() that also keeps the gate/up pre-activations and h of the
        routed and shared experts for backward().  bf16 and FP8 layers.  With
        balance_alpha > 0, self.balance holds the balance loss of every
        sequence [seq_offsets[q], seq_offsets[q+1]) of the tokens (int32 on the
        device; default: one sequence of all of them); without a balance loss
        they are not looked at.  The loss counts the routed choice, or that of
        the unbiased scores (balance_unbiased)."""
        c = self.cfg
        if c.dtype not in ("bf16", "e4m3"):
            raise ValueError("the backward is implemented for bf16 and FP8 layers")
        T = u.shape[0]
        if T != self.T_alloc:
            with _on(stream):
                self._alloc(T)
        if getattr(self, "T_train", None) != T:
            with _on(stream):
                self._alloc_train(T)
        self._route(u, stream, getattr(self, "logits", None))
        (wgu, sgu), (wdn, sdn) = self.W["W_gate_up"], self.W["W_down"]
        (wsgu, ssgu), (wsdn, ssdn) = self.W["Ws_gate_up"], self.W["Ws_down"]
        sl = lambda t, j: None if t is None else t[j:j + 1]
        if self.fp8:
            moe_quantize_1x128(u, self.u_q, self.u_s, stream)
            moe_permute(self.u_q, self.topk_idx, c.N_r, self.x_perm, self.offsets, self.perm_src,
                        self.inv_row, self.perm_ws, u_scale=self.u_s, x_scale=self.x_scale,
                        stream=stream)
            x_sh, xs_sh = self.u_q, self.u_s
        else:
            moe_permute(u, self.topk_idx, c.N_r, self.x_perm, self.offsets, self.perm_src,
                        self.inv_row, self.perm_ws, stream=stream)
            x_sh, xs_sh = u, None
        self._gate_up_save(self.x_perm, self.offsets, wgu, self.h_mid, self.a_gu, stream,
                           self.x_scale if self.fp8 else None, sgu, self.h_scale)
        moe_expert_down(self.h_mid, self.offsets, wdn, self.y_perm, h_scale=self.h_scale,
                        w_scale_down=sdn, stream=stream)
        for j in range(c.N_s):
            hs_scale = None if self.h_s_scale is None else self.h_s_scale[j]
            self._gate_up_save(x_sh, self.shared_offsets, wsgu[j:j + 1], self.h_s[j], self.a_s[j],
                               stream, xs_sh, sl(ssgu, j), hs_scale)
            moe_expert_down(self.h_s[j], self.shared_offsets, wsdn[j:j + 1], self.y_shared[j],
                            h_scale=hs_scale, w_scale_down=sl(ssdn, j), stream=stream)
        moe_combine(u, self.y_shared if c.N_s else None, self.y_perm, self.inv_row,
                    self.topk_gate, self.h_out, stream)
        if c.balance_alpha > 0:
            self._balance(u, seq_offsets, stream)
        self._u = u
        return self.h_out

    def _balance(self, u, seq_offsets, stream):
        c, T = self.cfg, self.T_train
        idx = self.topk_idx
        if c.balance_unbiased:
            # the top K of the scores alone; gates and load of that choice are not used
            idx, gate, counts = self.free_choice
            moe_route_scored(u, self.E, None, c.K, idx, gate, counts, self.route_ws,
                             score=self.score, stream=stream)
        n = 1 if seq_offsets is None else seq_offsets.shape[0] - 1
        if getattr(self, "_balance_for", None) != (T, n):
            self.balance = torch.empty(n, dtype=torch.float32, device=self.device)
            self.balance_coef = torch.empty(n, c.N_r, dtype=torch.float32, device=self.device)
            self.balance_ws = _ws(moe_balance_loss_workspace_size(T, c.N_r, n), self.device)
            self._balance_for = (T, n)
        moe_balance_loss(self.logits, idx, c.balance_alpha, self.balance,
                         self.balance_coef, self.balance_ws, score=self.score,
                         seq_offsets=seq_offsets, stream=stream)
        self.seq_offsets = seq_offsets

    def _ffn_backward(self, x, offsets, wgu, wdn, keep, h, dy, dx, dwgu, dwdn, stream, x_rows=None,
                      sgu=None, sdn=None):
        if self.cfg.checkpoint8:
            moe_expert_ffn_backward8(x, offsets, wgu, wdn, *keep, dy, dx, dwgu, dwdn, self.bwd_ws,
                                     stream=stream)
        else:
            moe_expert_ffn_backward(x, offsets, wgu, wdn, keep, h, dy, dx, dwgu, dwdn, self.bwd_ws,
                                    x_rows=x_rows, w_scale_gate_up=sgu, w_scale_down=sdn,
                                    stream=stream)

    def backward(self, dh: torch.Tensor, stream=None, ffn_events=None,
                 d_balance: torch.Tensor | None = None) -> torch.Tensor:
        """Gradients for upstream dh = dL/dh' of the last forward_train:
        returns du (overwritten by the next call) and fills self.grad
        (E: float32; W_gate_up, W_down, Ws_gate_up, Ws_down: bf16).
        d_balance [n_seq] float32: dL/dself.balance (default 1 for every
        sequence) where the configuration has a balance loss.
        ffn_events=(start, end) records CUDA events around the routed expert
        FFN backward on the same stream."""
        c, g = self.cfg, self.grad
        u = self._u
        st = torch.cuda.current_stream() if stream is None else stream
        moe_combine_backward(dh, u, self.E, self.y_perm, self.inv_row, self.topk_idx,
                             self.topk_gate, self.dy_perm, self.d_gate, self.d_logit,
                             self.d_logit_perm, stream)
        if ffn_events:
            ffn_events[0].record(st)
        (wgu, sgu), (wdn, sdn) = self.W["W_gate_up"], self.W["W_down"]
        (wsgu, ssgu), (wsdn, ssdn) = self.W["Ws_gate_up"], self.W["Ws_down"]
        sl = lambda t, j: None if t is None else t[j:j + 1]
        if self.fp8:
            # the FP8 Wgrad re-quantises the layer input: rows of u through perm_src
            x_r, x_rows, h_r = u, self.perm_src, None
        else:
            x_r, x_rows, h_r = self.x_perm, None, self.h_mid
        self._ffn_backward(x_r, self.offsets, wgu, wdn, self.a_gu, h_r, self.dy_perm,
                           self.dx_perm, g["W_gate_up"], g["W_down"], stream, x_rows, sgu, sdn)
        if ffn_events:
            ffn_events[1].record(st)
        for j in range(c.N_s):
            self._ffn_backward(u, self.shared_offsets, wsgu[j:j + 1], wsdn[j:j + 1], self.a_s[j],
                               None if self.fp8 else self.h_s[j], dh, self.dx_s[j],
                               g["Ws_gate_up"][j:j + 1], g["Ws_down"][j:j + 1], stream, None,
                               sl(ssgu, j), sl(ssdn, j))
        if c.scored:
            # the router's own gradient, then residual, shared, routed and router
            # gradients in one sum (the combine with weights 1), rounded once
            bal = c.balance_alpha > 0
            moe_route_scored_backward(u, self.E, self.logits, self.topk_idx, self.d_gate,
                                      self.dx_s[c.N_s], g["E"], self.route_bwd_ws,
                                      score=self.score, renorm=c.renorm, gate_scale=c.gate_scale,
                                      seq_offsets=self.seq_offsets if bal else None,
                                      balance_coef=self.balance_coef if bal else None,
                                      d_loss=d_balance if bal else None, stream=stream)
            moe_combine(dh, self.dx_s, self.dx_perm, self.inv_row, self.ones, self.du, stream)
            return self.du
        moe_unpermute_backward(dh, self.dx_s if c.N_s else None, self.dx_perm, self.inv_row,
                               self.topk_idx, self.d_logit, self.E, self.du, stream)
        if self.fp8:
            moe_router_weight_grad(u, self.d_logit_perm, self.offsets, g["E"],
                                   x_rows=self.perm_src, stream=stream)
        else:
            moe_router_weight_grad(self.x_perm, self.d_logit_perm, self.offsets, g["E"],
                                   stream=stream)
        return self.du

    def bias_update(self, counts=None, T_total=None, stream=None):
        """b <- b -/+ gamma from the load of the last step (or from the given
        global counts / token total of data-parallel replicas)."""
        counts = self.counts if counts is None else counts
        T_total = self.T_alloc if T_total is None else T_total
        moe_bias_update(self.b, counts, T_total, self.cfg.K, GAMMA, stream)

    def step(self, u, stream=None, process_group=None):
        """One training-style step: forward, global load, bias update."""
        h = self.forward(u, stream)
        if process_group is not None:
            from .parallel_load import allreduce_load
            counts, T_total = allreduce_load(self.counts, u.shape[0], process_group)
            self.bias_update(counts, T_total, stream)
        else:
            self.bias_update(stream=stream)
        return h
