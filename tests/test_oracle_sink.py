"""Pins of the oracle's sink-window attention and norm + rotation (CPU only)."""

import math

import numpy as np
import pytest
import torch

import oracle


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("w", [1, 3, 8])
def test_no_sinks_is_the_plain_window(w):
    q, k, v = (_rand(2, 2, 20, 8, seed=s) for s in range(3))
    y, _, _ = oracle.swa_sink(q, k, v, w, 0, 0.3)
    np.testing.assert_allclose(y, oracle.swa(q, k, v, w, 0.3), rtol=0, atol=1e-12)


def test_wide_window_is_causal_attention():
    q, k, v = (torch.from_numpy(_rand(2, 4, 17, 8, seed=s)) for s in range(3))
    ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True, scale=0.3).numpy()
    for w, sinks in ((17, 0), (99, 5), (1, 17)):
        y, _, _ = oracle.swa_sink(q.numpy(), k.numpy(), v.numpy(), w, sinks, 0.3)
        np.testing.assert_allclose(y, ref, rtol=0, atol=1e-12)


def test_visible_by_hand():
    # w = 2, one sink: token 3 sees 0 (sink), 2 and 3
    assert oracle.sink_visible(4, 2, 1).astype(int).tolist() == \
        [[1, 0, 0, 0], [1, 1, 0, 0], [1, 1, 1, 0], [1, 0, 1, 1]]


def test_grouped_heads_padding_and_lse():
    q, k, v = _rand(2, 4, 12, 8, seed=0), _rand(2, 2, 12, 8, seed=1), _rand(2, 2, 12, 8, seed=2)
    q[0, :, 7:] = k[0, :, 7:] = v[0, :, 7:] = np.nan
    y, lse, _ = oracle.swa_sink(q, k, v, 3, 2, 0.3, lengths=[7, 12])
    assert np.all(y[0, :, 7:] == 0) and np.all(np.isneginf(lse[0, :, 7:])) and np.all(np.isfinite(y))
    # row 6 of head 3 by hand: sinks 0, 1 and tokens 4, 5, 6 of key/value head 1
    js = [0, 1, 4, 5, 6]
    s = [0.3 * float(q[0, 3, 6] @ k[0, 1, j]) for j in js]
    e = [math.exp(x) for x in s]
    np.testing.assert_allclose(y[0, 3, 6], sum(x * v[0, 1, j] for x, j in zip(e, js)) / sum(e), atol=1e-12)
    assert abs(lse[0, 3, 6] - math.log(sum(e))) < 1e-12


def test_backward_against_autograd_and_differences():
    B, Hq, Hkv, N, d, w, sinks, sc = 1, 4, 2, 11, 4, 3, 2, 0.4
    q, k, v, dy = _rand(B, Hq, N, d, seed=0), _rand(B, Hkv, N, d, seed=1), _rand(B, Hkv, N, d, seed=2), \
        _rand(B, Hq, N, d, seed=3)
    got = oracle.swa_sink_backward(q, k, v, dy, w, sinks, sc)[:3]
    leaves = [torch.from_numpy(x).requires_grad_(True) for x in (q, k, v)]
    kk, vv = (x.repeat_interleave(Hq // Hkv, dim=1) for x in leaves[1:])
    mask = torch.from_numpy(~oracle.sink_visible(N, w, sinks))
    y = torch.softmax((leaves[0] @ kk.transpose(-1, -2) * sc).masked_fill(mask, -math.inf), -1) @ vv
    for g, ref in zip(got, torch.autograd.grad((y * torch.from_numpy(dy)).sum(), leaves)):
        np.testing.assert_allclose(g, ref.numpy(), atol=1e-12)
    f = lambda *a: float((oracle.swa_sink(*a, w, sinks, sc)[0] * dy).sum())
    rng = np.random.default_rng(9)
    for which in range(3):
        for _ in range(5):
            args = [x.copy() for x in (q, k, v)]
            idx = tuple(rng.integers(0, n) for n in args[which].shape)
            h = 1e-5
            args[which][idx] += h
            up = f(*args)
            args[which][idx] -= 2 * h
            assert abs((up - f(*args)) / (2 * h) - got[which][idx]) < 1e-7


def test_decode_continues_the_prompt():
    B, Hq, Hkv, N, d, w, sinks = 2, 4, 2, 23, 4, 5, 3
    q, k, v = _rand(B, Hq, N, d, seed=0), _rand(B, Hkv, N, d, seed=1), _rand(B, Hkv, N, d, seed=2)
    y, _, _ = oracle.swa_sink(q, k, v, w, sinks, 0.3)
    for prompt in (0, 1, 3, 9):
        kc, vc = (oracle.swa_sink_cache(x[:, :, :prompt], w, sinks) for x in (k, v))
        for t in range(prompt, N):
            yt, kc, vc, _ = oracle.swa_sink_decode_step(kc, vc, [t] * B, q[:, :, t], k[:, :, t], v[:, :, t], w, sinks,
                                                        0.3)
            np.testing.assert_allclose(yt, y[:, :, t], atol=1e-12)
        np.testing.assert_array_equal(kc, oracle.swa_sink_cache(k, w, sinks))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32])
def test_norm_rope_against_complex_rotation_and_autograd(rot, interleaved):
    x, wgt, g = _rand(2, 3, 5, 32, seed=0), 1 + 0.1 * _rand(32, seed=1), _rand(2, 3, 5, 32, seed=2)
    pos = np.array([[0, 1, 7, 100, 30000], [5, 6, 7, 8, 9]])
    ang = oracle.rope_angles(pos, rot, 10000.0)
    out, _ = oracle.norm_rope(x, wgt, ang, rot, 1e-6, interleaved)
    leaves = [torch.from_numpy(t).requires_grad_(True) for t in (x, wgt)]
    n = torch.nn.functional.rms_norm(leaves[0], (32,), eps=1e-6) * leaves[1]
    ph = torch.polar(torch.ones(()).double(), torch.from_numpy(ang))[:, None]
    a = n[..., :rot]
    if rot and interleaved:
        a = torch.view_as_real(torch.view_as_complex(a.reshape(2, 3, 5, rot // 2, 2).contiguous()) * ph).flatten(-2)
    elif rot:
        z = torch.complex(a[..., :rot // 2], a[..., rot // 2:]) * ph
        a = torch.cat([z.real, z.imag], -1)
    ref = torch.cat([a, n[..., rot:]], -1)
    np.testing.assert_allclose(out, ref.detach().numpy(), atol=1e-12)
    dx, dw, _, _ = oracle.norm_rope_backward(x, wgt, ang, g, rot, 1e-6, interleaved)
    rx, rw = torch.autograd.grad((ref * torch.from_numpy(g)).sum(), leaves)
    np.testing.assert_allclose(dx, rx.numpy(), atol=1e-12)
    np.testing.assert_allclose(dw, rw.numpy(), atol=1e-11)


def test_rotation_depends_on_distance_only():
    q, k = _rand(1, 1, 1, 16, seed=0), _rand(1, 1, 1, 16, seed=1)
    dots = []
    for p in (0, 11, 20000):
        a, b = (oracle.norm_rope(x, 1.0, oracle.rope_angles([[t]], 16, 10000.0), 16, 0.0, False)[0]
                for x, t in ((q, p + 5), (k, p)))
        dots.append(float((a * b).sum()))
    assert max(dots) - min(dots) < 1e-9
