"""GPU parity: per-head norm with rotation, forward and gradient, against the float64 oracle."""

import numpy as np
import pytest
import torch

import oracle
import linear_attention_sequence_causal_b200 as based
from sink_util import DT, HALF, assert_within, f64, fused, normal, scale_of, tol_y

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BASE = 10000.0
U32 = 2.0 ** -24


def _inputs(B, Hq, Hkv, N, d, dtype, seed):
    q, k = normal((B, Hq, N, d), dtype, seed), normal((B, Hkv, N, d), dtype, seed + 1)
    wq, wk = (1 + 0.1 * normal((d,), "f32", seed + 2 + i) for i in range(2))
    return q, k, wq, wk


def _positions(B, N, max_pos, seed):
    start = np.random.default_rng(seed).integers(0, max_pos - N + 1, B)
    return torch.from_numpy(start[:, None] + np.arange(N)[None, :])


def _forward_tol(out, size, d, dtype):
    # sum of squares (d roundings, halved by the root), root, two products, the table's and
    # the rotation's roundings: (d / 2 + 12) steps of the terms, then one rounding to the type
    return (d / 2 + 12) * U32 * size + HALF[dtype] * np.abs(out) + 1e-30


def _check(B, Hq, Hkv, N, d, rot, dtype, interleaved, weights=True, max_pos=4096, seed=0, views=False, shared=False):
    q, k, wq, wk = _inputs(B, Hq, Hkv, N, d, dtype, seed)
    if not weights:
        wq = wk = None
    pos = _positions(B, N, max_pos, seed)
    if shared:
        pos = pos[:1].expand(B, N)
    gpos = (pos[0] if shared else pos).contiguous().to(DEV)
    table = based.rope_table(max_pos, rot, BASE, device=DEV) if rot else None
    gq, gk = fused(q.to(DEV), k.to(DEV)) if views else (q.to(DEV), k.to(DEV))
    gw = [None if x is None else x.to(DEV) for x in (wq, wk)]
    qo, ko = based.qk_norm_rope(gq, gk, table, gpos if rot else None, *gw, eps=1e-5, interleaved=interleaved)
    dqo, dko = normal(q.shape, dtype, seed + 9), normal(k.shape, dtype, seed + 10)
    gdq, gdk = (x.to(DEV) for x in (dqo, dko))
    grads = based.qk_norm_rope_backward(gq, gk, table, gpos if rot else None, gdq, gdk, *gw, eps=1e-5,
                                        interleaved=interleaved)
    assert based.get_last_error() == 0
    ang = oracle.rope_angles(pos.numpy(), rot, BASE)
    rows = (B * N * Hq, B * N * Hkv)
    for x, w, o, g, dx, dw, n in ((q, wq, qo, dqo, grads[0], grads[2], rows[0]),
                                  (k, wk, ko, dko, grads[1], grads[3], rows[1])):
        w64 = np.ones(d) if w is None else f64(w)
        ref, size = oracle.norm_rope(f64(x), w64, ang, rot, 1e-5, interleaved)
        assert_within(o, ref, _forward_tol(ref, size, d, dtype), "out")
        rdx, rdw, sx, sw = oracle.norm_rope_backward(f64(x), w64, ang, f64(g), rot, 1e-5, interleaved)
        # xhat twice, the mean's d terms, the rotation
        assert_within(dx, rdx, (2 * d + 24) * U32 * sx + HALF[dtype] * np.abs(rdx) + 1e-30, "dx")
        assert_within(dw, rdw, (n + d / 2 + 16) * U32 * sw + 1e-30, "dweight")
    return (gq, gk, table, gpos, gw), (qo, ko), (gdq, gdk), grads


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,N,d,rot", [
    (1, 1, 1, 1, 16, 16), (2, 4, 2, 3, 32, 16), (1, 5, 1, 37, 48, 32), (2, 16, 16, 33, 64, 64), (3, 6, 3, 17, 80, 48),
    (2, 8, 2, 50, 128, 128), (1, 3, 3, 65, 128, 64), (1, 9, 1, 20, 192, 192), (2, 4, 4, 9, 256, 240), (1, 2, 1, 300, 64, 0),
])
def test_norm_rope(dtype, interleaved, B, Hq, Hkv, N, d, rot):
    _check(B, Hq, Hkv, N, d, rot, dtype, interleaved, seed=N + d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_views_shared_positions_and_no_weights(dtype):
    _check(3, 4, 2, 41, 64, 32, dtype, False, seed=1, views=True)
    _check(3, 4, 2, 41, 64, 64, dtype, False, seed=2, shared=True)
    _check(2, 4, 2, 41, 64, 64, dtype, True, seed=3, weights=False)


def test_many_tokens_fill_the_persistent_grid():
    _check(4, 8, 2, 2100, 64, 64, "bf16", False, seed=4)


def test_far_positions_keep_their_angle():
    """Angles of positions near a million, formed in fp64 by the table."""
    _check(1, 2, 1, 8, 64, 64, "f32", False, max_pos=1 << 20, seed=5)
    t = based.rope_table(1 << 20, 64, BASE, device=DEV)
    ang = oracle.rope_angles(np.arange((1 << 20) - 50, 1 << 20), 64, BASE)
    ref = np.stack([np.cos(ang), np.sin(ang)], -1)
    assert np.abs(f64(t[-50:]) - ref).max() <= U32 * 1.01 + 1e-9      # one rounding; the angle's own 2^-53 * 1e6


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place(dtype):
    (q, k, table, pos, w), (qo, ko), (dq, dk), grads = _check(2, 4, 2, 60, 64, 64, dtype, False, seed=6, views=True)
    based.qk_norm_rope_backward(q, k, table, pos, dq, dk, *w, eps=1e-5, dq=dq, dk=dk)
    assert torch.equal(dq, grads[0]) and torch.equal(dk, grads[1])
    based.qk_norm_rope(q, k, table, pos, *w, eps=1e-5, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_position_outside_the_table_is_reported():
    q, k, wq, wk = (x.to(DEV) for x in _inputs(2, 2, 1, 5, 64, "bf16", 7))
    table = based.rope_table(100, 64, device=DEV)
    pos = torch.tensor([[0, 1, 2, 3, 4], [98, 99, 100, -1, 1 << 40]], device=DEV)
    qo, ko = based.qk_norm_rope(q, k, table, pos, wq, wk)
    assert based.get_last_error() == 1
    assert based.get_last_error() == 0
    bad = torch.zeros(2, 5, dtype=torch.bool, device=DEV)
    bad[1, 2:] = True
    assert torch.equal(torch.isnan(qo), bad[:, None, :, None].expand_as(qo))
    assert torch.equal(torch.isnan(ko), bad[:, None, :, None].expand_as(ko))


def test_gradient_is_deterministic_and_captured():
    q, k, wq, wk = (x.to(DEV) for x in _inputs(2, 8, 2, 700, 128, "bf16", 8))
    table = based.rope_table(1024, 128, device=DEV)
    dqo, dko = normal(q.shape, "bf16", 9).to(DEV), normal(k.shape, "bf16", 10).to(DEV)
    step = lambda: based.qk_norm_rope_backward(q, k, table, None, dqo, dko, wq, wk)
    eager = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, held):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_step_from_projection_to_cache(dtype):
    """Norm + rotation, the prompt's attention and a generated token, chained as a layer runs them."""
    B, Hq, Hkv, N, d, w, sinks = 2, 4, 2, 140, 64, 50, 4
    q, k, wq, wk = _inputs(B, Hq, Hkv, N + 1, d, dtype, 11)
    v = normal(k.shape, dtype, 15)
    table = based.rope_table(512, d, BASE, device=DEV)
    gq, gk, gv = fused(*(x.to(DEV) for x in (q, k, v)))
    gw = (wq.to(DEV), wk.to(DEV))
    pq, pk = based.qk_norm_rope(gq[:, :, :N], gk[:, :, :N], table, None, *gw)
    y, _, kc, vc = based.swa_sink_prefill(pq, pk, gv[:, :, :N], w, sinks)
    at = torch.full((B, 1), N, device=DEV)
    tq, tk = based.qk_norm_rope(gq[:, :, N:], gk[:, :, N:], table, at, *gw)
    yt = based.swa_sink_decode(kc, vc, at[:, 0].contiguous(), tq[:, :, 0].contiguous(), tk[:, :, 0].contiguous(),
                               gv[:, :, N].contiguous(), w, sinks)
    assert based.get_last_error() == 0
    # The oracle takes the rotated tensors as they were rounded: each stage has its own bound.
    rq, rk = (torch.cat([a, b], 2) for a, b in ((pq, tq), (pk, tk)))
    ang = oracle.rope_angles(np.arange(N + 1)[None].repeat(B, 0), d, BASE)
    for x, wgt, got in ((q, wq, rq), (k, wk, rk)):
        ref, size = oracle.norm_rope(f64(x), f64(wgt), ang, d, 1e-6, False)
        assert_within(got, ref, _forward_tol(ref, size, d, dtype), "rotated")
    ref, _, mass = oracle.swa_sink(f64(rq), f64(rk), f64(v), w, sinks, scale_of(d))
    tol = tol_y(ref, mass, rq, rk, scale_of(d), dtype, w + sinks)
    assert_within(y, ref[:, :, :N], tol[:, :, :N], "prompt")
    assert_within(yt, ref[:, :, N], tol[:, :, N], "token")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_outputs_keep_to_their_buffers(dtype):
    q, k, wq, wk = (x.to(DEV) for x in _inputs(2, 3, 1, 37, 48, dtype, 12))
    table = based.rope_table(64, 32, device=DEV)

    def tailed(t):
        buf = torch.full((t.numel() + 512,), 3.0, dtype=t.dtype, device=DEV)
        return buf[:t.numel()].view(t.shape), buf[t.numel():]

    (qo, t0), (ko, t1), (dq, t2), (dk, t3) = (tailed(x) for x in (q, k, q, k))
    based.qk_norm_rope(q, k, table, None, wq, wk, q_out=qo, k_out=ko)
    n = based.lib().based_qk_norm_rope_backward_workspace(2, 3, 1, 37, 48, 0 if dtype == "f32" else 1)
    ws, t4 = tailed(torch.empty(n, dtype=torch.uint8, device=DEV))
    based.qk_norm_rope_backward(q, k, table, None, qo, ko, wq, wk, dq=dq, dk=dk, workspace=ws)
    assert based.get_last_error() == 0
    for t in (t0, t1, t2, t3, t4):
        assert torch.all(t == 3)
