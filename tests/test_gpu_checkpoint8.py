"""The expert FFN's 8-bit activation checkpoint: packing, and the backward that reads it.

Tolerances are counted from the arithmetic: E4M3 is off by at most 2^-4 of a value or half its
smallest step (2^-10 of the scale); tensor-core sums by 2^-16 of sum|terms|; bf16 by 2^-8 of a
value, once where dA or h is rounded and once at the output."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_60_b200 as moe
from oracle import moe_scored as S
from tests.harness import f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _off(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def _save8(x, off, W, fill=77):
    R, I = x.shape[0], W.shape[1] // 2
    h = torch.full((R, I), float(fill), dtype=BF, device="cuda")
    q = torch.full((R, 2 * I), fill, dtype=torch.uint8, device="cuda")
    sc = torch.full((R, 2 * I // 128), float(fill), device="cuda")
    moe.moe_expert_gate_up_save8(x, off, W, h, q, sc)
    return h, q, sc


def _values(q):
    return q.view(torch.float8_e4m3fn).float()


SIZES = [[1], [0, 1, 15, 63, 64, 65, 130, 257, 17], [700], [31, 32, 33, 0, 0, 300, 16]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("d,I", [(256, 128), (512, 384), (128, 256)])
def test_save8_packs_the_preactivations(sizes, d, I):
    R, G = int(sum(sizes)), len(sizes)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(R, d, generator=g, device="cuda").to(BF)
    W = (torch.randn(G, 2 * I, d, generator=g, device="cuda") * d ** -0.5).to(BF)
    off = _off(sizes)
    h, q, sc = _save8(x, off, W)
    ref = torch.empty_like(h)
    moe.moe_expert_gate_up(x, off, W, ref)
    assert torch.equal(h, ref), "h is the plain gate/up's, bit for bit"
    o = off.tolist()
    for e in range(G):
        r = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            continue
        a = f64(x[r]) @ f64(W[e]).T
        mag = np.abs(f64(x[r])) @ np.abs(f64(W[e])).T
        amax = np.abs(a).reshape(len(a), -1, 128).max(2)
        acc = 2.0 ** -16 * mag.reshape(len(a), -1, 128).max(2)
        assert (np.abs(f64(sc[r]) * 448 - amax) <= acc + 2.0 ** -23 * amax).all()
        v = f64(_values(q[r])) * np.repeat(f64(sc[r]), 128, axis=1)
        tol = np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * np.repeat(f64(sc[r]), 128, axis=1))
        assert (np.abs(v - a) <= tol * 1.01 + 2.0 ** -15 * mag).all()
    h2, q2, s2 = _save8(x, off, W, 3)
    assert torch.equal(q, q2) and torch.equal(sc, s2) and torch.equal(h, h2)


def test_save8_codes_are_exact_for_exact_preactivations():
    """One-hot rows pick weight columns, so the pre-activations are the stored weights: scales
    and codes have to be the oracle's, all-zero tiles, ties and the largest values among them."""
    d, I = 256, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    W = torch.randn(1, 2 * I, d, generator=g, device="cuda") * \
        torch.exp(3 * torch.randn(1, 2 * I, d, generator=g, device="cuda"))
    W[0, 128:256, :9] = 0                         # an all-zero tile
    W[0, :128, 9] = (torch.arange(128, device="cuda") - 64) * 7.0      # amax 448: codes at ties
    W[0, 256:384, 10] = 2.0 ** -120               # tiny values
    W = W.to(BF)
    x = torch.eye(d, device="cuda").to(BF)
    h, q, sc = _save8(x, _off([d]), W)
    want_q, want_s = S.checkpoint(f64(W[0]).T)
    assert np.array_equal(sc.cpu().numpy(), want_s)
    assert np.array_equal(f64(_values(q)), want_q)


def test_save8_leaves_rows_outside_every_group():
    x = torch.randn(90, 256, device="cuda").to(BF)
    W = torch.randn(2, 256, 256, device="cuda").to(BF)
    off = torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda")
    h, q, sc = _save8(x, off, W)
    assert (h[70:] == 77).all() and (q[70:] == 77).all() and (sc[70:] == 77).all()
    off = torch.tensor([0, 40, 200], dtype=torch.int32, device="cuda")     # past the rows
    assert moe.moe_device_status() == 0
    _save8(x, off, W)
    assert moe.moe_device_status() == 16


def _backward8(x, off, Wgu, Wdn, q, sc, dy):
    R, d = x.shape
    G, two_i, _ = Wgu.shape
    out = [torch.full((R, d), float("nan"), dtype=BF, device="cuda"),
           torch.full_like(Wgu, float("nan")), torch.full_like(Wdn, float("nan"))]
    n = moe.moe_expert_ffn_backward8_workspace_size(moe.MOE_BF16, R, d, two_i // 2, G)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    moe.moe_expert_ffn_backward8(x, off, Wgu, Wdn, q, sc, dy, *out, ws)
    return out, ws


def _ffn(sizes, d, I, seed=8):
    R, G = int(sum(sizes)), len(sizes)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s, k=1.0: (torch.randn(*s, generator=g, device="cuda") * k).to(BF)
    return (rn(R, d), _off(sizes), rn(G, 2 * I, d, k=d ** -0.5), rn(G, d, I, k=I ** -0.5),
            rn(R, d, k=0.05))


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("d,I", [(512, 256), (256, 512)])
def test_backward8(sizes, d, I):
    x, off, Wgu, Wdn, dy = _ffn(sizes, d, I)
    h, q, sc = _save8(x, off, Wgu)
    (dx, dWgu, dWdn), _ = _backward8(x, off, Wgu, Wdn, q, sc, dy)
    a = S.from_checkpoint(f64(_values(q)), f64(sc))
    o = off.tolist()
    B8 = 2.0 ** -8
    for e in range(len(sizes)):
        r = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            assert not dWgu[e].any() and not dWdn[e].any(), "a group without rows"
            continue
        xs, dys, wg, wd = f64(x[r]), f64(dy[r]), f64(Wgu[e]), f64(Wdn[e])
        want = S.ffn_backward(xs, wg, wd, a[r], dys)
        # magnitudes of the sums: |dA| and |h| with their own sums' error
        sig = S.scores(a[r][:, :I], S.SIGMOID)
        dsl = np.abs(sig * (1 + a[r][:, :I] * (1 - sig)))
        dh, mdh = dys @ wd, np.abs(dys) @ np.abs(wd)
        fa = np.concatenate([np.abs(a[r][:, I:]) * dsl, np.abs(a[r][:, :I]) * sig], 1)
        two = lambda v: np.concatenate([v, v], 1)
        edA = B8 * two(np.abs(dh)) * fa + 2.0 ** -15 * two(mdh) * fa      # error of dA
        mA = two(np.abs(dh)) * fa
        hm = np.abs(a[r][:, :I] * sig * a[r][:, I:])
        for name, got, ref, tol in (
                ("dx", dx[r], want[0], edA @ np.abs(wg) + 2.0 ** -15 * mA @ np.abs(wg)),
                ("dWgu", dWgu[e], want[1], (edA + 2.0 ** -15 * mA).T @ np.abs(xs)),
                ("dWdn", dWdn[e], want[2], (B8 + 2.0 ** -15) * np.abs(dys).T @ hm)):
            err = np.abs(f64(got) - ref)
            assert (err <= B8 * np.abs(ref) + 1.01 * tol).all(), name
            # independent roundings: far inside the sum of their bounds
            assert np.linalg.norm(err) <= 2.0 ** -7 * np.linalg.norm(ref), name


def test_backward8_is_the_plain_backward_for_exact_checkpoints():
    """Scales that are powers of two leave pre-activations that bf16 holds: the gradients are
    moe_expert_ffn_backward's bit for bit."""
    sizes, d, I = [100, 0, 33, 260], 512, 256
    x, off, Wgu, Wdn, dy = _ffn(sizes, d, I, 9)
    R = x.shape[0]
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    sc = 2.0 ** torch.randint(-9, -6, (R, 2 * I // 128), generator=g, device="cuda").float()
    q = (torch.randn(R, 2 * I, generator=g, device="cuda") * 100).to(torch.float8_e4m3fn)
    a = (q.float().view(R, -1, 128) * sc[:, :, None]).view(R, 2 * I).to(BF)
    (dx, dWgu, dWdn), _ = _backward8(x, off, Wgu, Wdn, q, sc, dy)
    fa = a.float()
    h = (fa[:, :I] * torch.sigmoid(fa[:, :I]) * fa[:, I:]).to(BF)
    ref = [torch.empty_like(dx), torch.empty_like(dWgu), torch.empty_like(dWdn)]
    ws = torch.empty(moe.moe_expert_ffn_backward_workspace_size(moe.MOE_BF16, R, d, I, 4),
                     dtype=torch.uint8, device="cuda")
    moe.moe_expert_ffn_backward(x, off, Wgu, Wdn, a, h, dy, *ref, ws)
    assert torch.equal(dx, ref[0]) and torch.equal(dWgu, ref[1])


def test_backward8_keeps_groups_apart():
    """Rows of another group, and rows behind the last one, may hold anything: NaN there stays out
    of a group's gradients.  Rows outside every group are not written."""
    sizes, d, I = [37, 5, 0, 130, 1, 64], 256, 512
    x, off, Wgu, Wdn, dy = _ffn(sizes + [50], d, I, 12)
    off = off[:-1].contiguous()                   # the last 50 rows belong to no group
    Wgu, Wdn = Wgu[:-1].contiguous(), Wdn[:-1].contiguous()
    h, q, sc = _save8(x, off, Wgu, 0)
    (dx, dWgu, dWdn), _ = _backward8(x, off, Wgu, Wdn, q, sc, dy)
    n = int(off[-1])
    assert torch.isfinite(dWgu).all() and torch.isfinite(dWdn).all()
    assert torch.isnan(dx[n:]).all() and torch.isfinite(dx[:n]).all()
    bx, bdy, bsc = x.clone(), dy.clone(), sc.clone()
    for t in (bx, bdy, bsc):
        t[n:] = float("nan")                      # behind the last group
        t[37:42] = float("nan")                   # all of group 1
    (ex, egu, edn), _ = _backward8(bx, off, Wgu, Wdn, q, bsc, bdy)
    keep = [e for e in range(len(sizes)) if e != 1]
    assert torch.equal(egu[keep], dWgu[keep]) and torch.equal(edn[keep], dWdn[keep])
    assert torch.isnan(egu[1]).all() and torch.isnan(edn[1]).all()
    rows = [r for r in range(n) if not 37 <= r < 42]
    assert torch.equal(ex[rows], dx[rows])


def test_backward8_many_small_groups():
    """Groups of fewer rows than a stage, one after the other in the ring."""
    rng = np.random.default_rng(2)
    sizes = rng.integers(0, 20, 150).tolist()
    x, off, Wgu, Wdn, dy = _ffn(sizes, 256, 256, 13)
    h, q, sc = _save8(x, off, Wgu)
    (dx, dWgu, dWdn), _ = _backward8(x, off, Wgu, Wdn, q, sc, dy)
    a = S.from_checkpoint(f64(_values(q)), f64(sc))
    o = off.tolist()
    for e in range(len(sizes)):
        r = slice(o[e], o[e + 1])
        if sizes[e] == 0:
            assert not dWgu[e].any() and not dWdn[e].any()
            continue
        want = S.ffn_backward(f64(x[r]), f64(Wgu[e]), f64(Wdn[e]), a[r], f64(dy[r]))
        for got, ref in ((dx[r], want[0]), (dWgu[e], want[1]), (dWdn[e], want[2])):
            assert np.linalg.norm(f64(got) - ref) <= 2.0 ** -7 * np.linalg.norm(ref)


def test_checkpoint8_streams_and_graphs():
    sizes, d, I = [70, 5, 130], 256, 256
    x, off, Wgu, Wdn, dy = _ffn(sizes, d, I, 11)
    h, q, sc = _save8(x, off, Wgu)
    (dx, dWgu, dWdn), ws = _backward8(x, off, Wgu, Wdn, q, sc, dy)
    torch.cuda.synchronize()
    out = [torch.zeros_like(t) for t in (h, q, sc, dx, dWgu, dWdn)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_expert_gate_up_save8(x, off, Wgu, *out[:3])
        moe.moe_expert_ffn_backward8(x, off, Wgu, Wdn, out[1], out[2], dy, *out[3:], ws)
    for _ in range(2):
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, (h, q, sc, dx, dWgu, dWdn)):
            assert torch.equal(got, want)
    st = torch.cuda.Stream()
    out = [torch.zeros_like(t) for t in (h, q, sc)]
    torch.cuda.synchronize()
    moe.moe_expert_gate_up_save8(x, off, Wgu, *out, stream=st)
    st.synchronize()
    assert torch.equal(out[1], q) and torch.equal(out[0], h)


def test_checkpoint8_no_rows():
    x, off, Wgu, Wdn, dy = _ffn([0, 0], 256, 256)
    h, q, sc = _save8(x, off, Wgu)
    (dx, dWgu, dWdn), _ = _backward8(x, off, Wgu, Wdn, q, sc, dy)
    assert not dWgu.any() and not dWdn.any()
