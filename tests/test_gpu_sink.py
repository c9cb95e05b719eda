"""GPU parity: sliding-window attention with sink tokens (prompt, single tokens, gradient)
against the float64 oracle, element by element within bounds derived in sink_util."""

import numpy as np
import pytest
import torch

import oracle
import linear_attention_sequence_causal_b200 as based
from sink_util import DT, HALF, U, assert_within, f64, fused, normal, scale_of, score_error, token_major, tol_y

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _qkv(B, Hq, Hkv, N, d, dtype, seed):
    return (normal((B, Hq, N, d), dtype, 3 * seed), normal((B, Hkv, N, d), dtype, 3 * seed + 1),
            normal((B, Hkv, N, d), dtype, 3 * seed + 2))


def _check_prefill(q, k, v, w, sinks, dtype, scale=None, lengths=None, views=None, seen=None):
    """Runs the prompt on `views` (default: the tensors) and checks y, lse and the caches."""
    d = q.shape[-1]
    scale = scale_of(d) if scale is None else scale
    dq, dk, dv = views if views is not None else (x.to(DEV) for x in (q, k, v))
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int64, device=DEV)
    y, lse, kc, vc = based.swa_sink_prefill(dq, dk, dv, w, sinks, scale=scale, lengths=ln, want_lse=True)
    assert based.get_last_error() == 0
    ref, rlse, mass = oracle.swa_sink(f64(q), f64(k), f64(v), w, sinks, scale, lengths)
    keys = min(q.shape[2], w + sinks)
    assert_within(y, ref, tol_y(ref, mass, q, k, scale, dtype, keys), "y")
    real = np.isfinite(rlse)
    got = f64(lse)
    assert np.all(np.isneginf(got[~real]))
    # log of the sum: its relative error, and two roundings of the result
    tol = 2 * score_error(q, k, scale, dtype) + keys * U[dtype] + 2.0 ** -21 * (1 + np.abs(rlse[real]))
    assert np.all(np.abs(got[real] - rlse[real]) <= tol)
    for c, x in ((kc, k), (vc, v)):
        assert np.array_equal(f64(c), oracle.swa_sink_cache(f64(x), w, sinks, lengths))
    return y, lse


SHAPES = [
    # B, Hq, Hkv, N, w, sinks
    (1, 1, 1, 1, 1, 0), (1, 2, 1, 1, 7, 4), (2, 4, 2, 2, 1, 1), (1, 4, 4, 63, 5, 2), (2, 2, 2, 64, 64, 0),
    (1, 4, 1, 65, 64, 4), (1, 6, 2, 127, 16, 64), (2, 4, 2, 128, 128, 1), (1, 5, 1, 129, 127, 33),
    (1, 2, 2, 200, 129, 4), (1, 4, 2, 300, 64, 4), (1, 3, 3, 517, 200, 16), (2, 8, 2, 385, 1, 0),
    (1, 2, 1, 700, 1000, 4), (1, 4, 4, 640, 256, 0), (1, 16, 1, 260, 65, 3),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,N,w,sinks", SHAPES)
def test_prefill(dtype, d, B, Hq, Hkv, N, w, sinks):
    _check_prefill(*_qkv(B, Hq, Hkv, N, d, dtype, N + w), w, sinks, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 300, 1, 129], [128, 0, 0, 64], [257, 255, 256, 2]])
def test_prefill_padding_never_reaches_a_row(dtype, d, lengths):
    N = 300
    q, k, v = _qkv(4, 4, 2, N, d, dtype, 5)
    for b, n in enumerate(lengths):
        for x in (q, k, v):
            x[b, :, n:] = float("nan") if b % 2 else float("inf")
    _check_prefill(q, k, v, 40, 4, dtype, lengths=lengths)
    _check_prefill(q, k, v, 400, 0, dtype, lengths=lengths)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_reads_and_writes_views(dtype):
    q, k, v = _qkv(2, 4, 2, 197, 64, dtype, 8)
    views = [token_major(q.to(DEV))] + fused(k.to(DEV), v.to(DEV))
    y, _ = _check_prefill(q, k, v, 70, 3, dtype, views=views)
    out = torch.full((2, 199, 6, 64), 7.0, dtype=DT[dtype], device=DEV)
    based.swa_sink_prefill(*views, 70, 3, want_cache=False, y=out[:, 1:198, 1:5].transpose(1, 2))
    assert torch.equal(out[:, 1:198, 1:5].transpose(1, 2), y)
    out[:, 1:198, 1:5] = 7.0
    assert torch.all(out == 7.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_far_and_large_scores(dtype):
    q, k, v = _qkv(1, 2, 2, 400, 64, dtype, 11)
    _check_prefill(q * 4, k * 4, v, 90, 4, dtype, scale=0.5)      # scores of order 100
    _check_prefill(q, k, v, 90, 4, dtype, scale=0.0)              # the mean of the visible values
    ramp = torch.arange(400, dtype=torch.float32)[:, None] / 40   # a maximum that grows along the keys
    _check_prefill(q.abs(), (k.float().abs() * ramp).to(k.dtype), v, 300, 4, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("w,sinks,at", [(40, 4, 150), (900, 0, 101), (300, 16, 15), (64, 3, 3),
                                        (1100, 0, 50)])
def test_prefill_hidden_infinities_never_reach_a_row(dtype, d, w, sinks, at):
    """Token `at` holds infinities and NaN: the rows that do not see it are as if it held zeros."""
    N, scale = 1200, scale_of(d)
    q, k, v = _qkv(1, 2, 1, N, d, dtype, at)
    clean = (f64(k).copy(), f64(v).copy())
    for c in clean:
        c[:, :, at] = 0.0
    k[:, :, at], v[:, :, at, ::3], v[:, :, at, 1::3] = float("nan"), float("inf"), float("nan")
    y, lse, _, _ = based.swa_sink_prefill(*(x.to(DEV) for x in (q, k, v)), w, sinks, want_cache=False, want_lse=True)
    assert based.get_last_error() == 0
    hidden = ~oracle.sink_visible(N, w, sinks)[:, at]
    assert hidden.sum() == at + (0 if at < sinks else max(0, N - at - w))
    ref, rlse, mass = oracle.swa_sink(f64(q), *clean, w, sinks, scale)
    tol = tol_y(ref, mass, q, torch.from_numpy(clean[0]), scale, dtype, min(N, w + sinks))
    assert_within(f64(y)[:, :, hidden], ref[:, :, hidden], tol[:, :, hidden], "hidden rows")
    assert np.abs(f64(lse)[:, :, hidden] - rlse[:, :, hidden]).max() < 1e-3
    assert np.all(np.isnan(f64(y)[:, :, ~hidden]))                # a NaN score: the definition's NaN


@pytest.mark.parametrize("dtype,d,w", [("f32", 64, 100), ("bf16", 64, 100), ("bf16", 64, 5000), ("bf16", 128, 5000)])
def test_prefill_infinity_that_every_row_sees(dtype, d, w):
    """One infinite value in a sink: its channel is infinite in every row, the others are as ever."""
    N, scale = 2100, scale_of(d)
    q, k, v = _qkv(1, 4, 2, N, d, dtype, 77)
    clean = f64(v).copy()
    v[:, :, 1, 5] = float("inf")
    y, lse, _, _ = based.swa_sink_prefill(*(x.to(DEV) for x in (q, k, v)), w, 2, want_cache=False, want_lse=True)
    assert based.get_last_error() == 0
    got = f64(y)
    assert np.all(got[:, :, 1:, 5] == np.inf) and np.all(np.isfinite(got[:, :, 0]))
    ref, rlse, mass = oracle.swa_sink(f64(q), f64(k), clean, w, 2, scale)
    tol = tol_y(ref, mass, q, k, scale, dtype, min(N, w + 2))
    others = np.arange(d) != 5
    assert_within(got[..., others], ref[..., others], tol[..., others], "other channels")
    assert np.abs(f64(lse) - rlse).max() < 1e-3


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_longer(d):
    """Many tiles and heads: every role of the pipeline wraps its ring several times."""
    q, k, v = _qkv(2, 8, 2, 1500, d, "bf16", 21)
    _check_prefill(q, k, v, 500, 8, "bf16")
    _check_prefill(q, k, v, 5000, 0, "bf16")


def test_prefill_is_deterministic_and_runs_on_any_stream():
    q, k, v = (x.to(DEV) for x in _qkv(2, 4, 2, 777, 64, "bf16", 31))
    a = based.swa_sink_prefill(q, k, v, 100, 4)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = based.swa_sink_prefill(q, k, v, 100, 4)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b)


def test_length_out_of_range_is_reported():
    q, k, v = (x.to(DEV) for x in _qkv(3, 2, 2, 70, 64, "bf16", 33))
    ln = torch.tensor([-5, 1000, 70], device=DEV)
    y = based.swa_sink_prefill(q, k, v, 20, 2, lengths=ln)[0]
    assert based.get_last_error() == 1
    assert based.get_last_error() == 0
    full = based.swa_sink_prefill(q, k, v, 20, 2)[0]
    assert torch.all(y[0] == 0) and torch.equal(y[1:], full[1:])


# ------------------------------------------------------------------ decode

def _check_decode(B, Hq, Hkv, d, w, sinks, dtype, positions, seed=0, garbage=True):
    q, k, v = normal((B, Hq, d), dtype, seed), normal((B, Hkv, d), dtype, seed + 1), normal((B, Hkv, d), dtype, seed + 2)
    kc, vc = (normal((B, Hkv, sinks + w, d), dtype, seed + 3 + i) for i in range(2))
    ref, rk, rv, mass = oracle.swa_sink_decode_step(f64(kc), f64(vc), positions, f64(q), f64(k), f64(v), w, sinks,
                                                    scale_of(d))
    if garbage:                                      # slots not in use hold anything
        for b, t in enumerate(positions):
            kc[b, :, max(t + 1, 0):] = float("nan")
            vc[b, :, max(t + 1, 0):] = float("inf")
    before = (kc.clone(), vc.clone())
    gk, gv = kc.to(DEV), vc.to(DEV)
    y = based.swa_sink_decode(gk, gv, torch.tensor(positions, dtype=torch.int64, device=DEV), q.to(DEV), k.to(DEV),
                              v.to(DEV), w, sinks)
    assert based.get_last_error() == 0
    keys = min(w + sinks, max(positions) + 1)
    tol = tol_y(ref, mass, q, torch.from_numpy(np.nan_to_num(rk)), scale_of(d), dtype, keys)
    assert_within(y, ref, tol, "decode y")
    for got, old, new in ((gk, before[0], k), (gv, before[1], v)):
        want = old.clone()
        for b, t in enumerate(positions):
            if t >= 0:
                want[b, :, t if t < sinks else sinks + (t - sinks) % w] = new[b]
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=5.0, posinf=6.0), torch.nan_to_num(want, nan=5.0, posinf=6.0))
    return y


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,w,sinks,positions", [
    (1, 1, 1, 1, 0, [0]), (1, 2, 2, 1, 0, [1000]), (2, 4, 2, 7, 3, [0, 2]), (3, 4, 1, 16, 4, [3, 4, 19]),
    (4, 6, 2, 64, 4, [-1, 67, 68, 5000]), (2, 20, 1, 33, 1, [40, 7]), (3, 40, 2, 100, 64, [63, 64, 400]),
    (2, 16, 16, 64, 4, [10, 1 << 40]),
])
def test_decode(dtype, d, B, Hq, Hkv, w, sinks, positions):
    _check_decode(B, Hq, Hkv, d, w, sinks, dtype, positions, seed=w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,w,sinks,positions", [
    (1, 4, 1, 1000, 4, [1003]), (1, 4, 4, 5000, 16, [123456]), (2, 8, 2, 4099, 0, [4098, 17]),
    (1, 16, 4, 20000, 16, [19000]), (3, 2, 1, 2500, 1, [-1, 2500, 0]),
])
def test_decode_long_windows_split(dtype, B, Hq, Hkv, w, sinks, positions):
    _check_decode(B, Hq, Hkv, 128, w, sinks, dtype, positions, seed=w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("prompt", [1, 3, 30])
def test_decode_continues_the_prompt(dtype, prompt):
    B, Hq, Hkv, N, d, w, sinks = 2, 4, 2, 75, 64, 20, 4
    q, k, v = _qkv(B, Hq, Hkv, N, d, dtype, 41)
    lengths = [prompt, max(prompt - 2, 0)]
    g = [x.to(DEV) for x in (q, k, v)]
    _, _, kc, vc = based.swa_sink_prefill(*(x[:, :, :prompt] for x in g), w, sinks,
                                          lengths=torch.tensor(lengths, device=DEV))
    pos = torch.tensor(lengths, device=DEV)
    ref, _, mass = oracle.swa_sink(f64(q), f64(k), f64(v), w, sinks, scale_of(d))
    tol = tol_y(ref, mass, q, k, scale_of(d), dtype, w + sinks)
    steps = N - prompt
    for s in range(steps):
        rows = [n + s for n in lengths]
        qs, ks, vs = (torch.stack([x[b, :, rows[b]] for b in range(B)]) for x in g)
        y = f64(based.swa_sink_decode(kc, vc, pos, qs, ks, vs, w, sinks))
        for b in range(B):
            assert_within(y[b], ref[b, :, rows[b]], tol[b, :, rows[b]], f"step {s}, sequence {b}")
        pos += 1
    assert based.get_last_error() == 0


def test_decode_captured_and_replayed():
    """The position is read on the device: one captured step serves every later token."""
    B, Hq, Hkv, d, w, sinks, steps = 2, 8, 2, 128, 600, 4, 9
    kc, vc = (normal((B, Hkv, sinks + w, d), "bf16", 51 + i).to(DEV) for i in range(2))
    toks = [tuple(normal((B, h, d), "bf16", 60 + 3 * s + i).to(DEV) for i, h in enumerate((Hq, Hkv, Hkv)))
            for s in range(steps)]
    start = torch.tensor([598, 3], device=DEV)
    ek, ev, pos = kc.clone(), vc.clone(), start.clone()
    eager = []
    for q, k, v in toks:
        eager.append(based.swa_sink_decode(ek, ev, pos, q, k, v, w, sinks))
        pos += 1
    ins = [torch.empty_like(x) for x in toks[0]]
    pos, y = start.clone(), torch.empty_like(toks[0][0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        based.swa_sink_decode(kc, vc, pos, *ins, w, sinks, y=y)
        pos += 1
    pos.copy_(start)
    for s in range(steps):
        for dst, src in zip(ins, toks[s]):
            dst.copy_(src)
        graph.replay()
        assert torch.equal(y, eager[s]), s
    assert torch.equal(kc, ek) and torch.equal(vc, ev)


# ------------------------------------------------------------------ backward

def _check_backward(q, k, v, dy, w, sinks, dtype, lengths=None, views=None, scale=None):
    d = q.shape[-1]
    scale = scale_of(d) if scale is None else scale
    vq, vk, vv, vdy = views if views is not None else (x.to(DEV) for x in (q, k, v, dy))
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int64, device=DEV)
    y, lse, _, _ = based.swa_sink_prefill(vq, vk, vv, w, sinks, scale=scale, lengths=ln, want_cache=False, want_lse=True)
    got = based.swa_sink_backward(vq, vk, vv, y, lse, vdy, w, sinks, scale=scale, lengths=ln)
    assert based.get_last_error() == 0
    ref, _, mass = oracle.swa_sink(f64(q), f64(k), f64(v), w, sinks, scale, lengths)
    keys = min(q.shape[2], w + sinks)
    # The backward's delta = dy . y takes the forward's rounded y (bf16 with few keys sums p dP in
    # fp32 instead: p's own error stays); dy . v is a sum of d terms.
    few = dtype == "bf16" and w + sinks < 64
    ey = (2 * score_error(q, k, scale, dtype) * mass if few else tol_y(ref, mass, q, k, scale, dtype, keys)) + \
        (d + 4) * U[dtype] * 2 * float(np.abs(np.nan_to_num(f64(v), nan=0.0, posinf=0.0, neginf=0.0)).max())
    n_terms = q.shape[2] * (q.shape[1] // k.shape[1])
    rel = 2 * score_error(q, k, scale, dtype) + n_terms * U[dtype] + HALF[dtype]
    out = oracle.swa_sink_backward(f64(q), f64(k), f64(v), f64(dy), w, sinks, scale, lengths, ey, rel * (1 + 2.0 ** -6))
    for name, g, r, e in zip(("dq", "dk", "dv"), got, out[:3], out[3:]):
        assert_within(g, r, e + HALF[dtype] * np.abs(r) + 1e-30, name)
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,N,w,sinks", SHAPES)
def test_backward(dtype, d, B, Hq, Hkv, N, w, sinks):
    q, k, v = _qkv(B, Hq, Hkv, N, d, dtype, N + w)
    _check_backward(q, k, v, normal(q.shape, dtype, 7), w, sinks, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 300, 1, 129], [257, 255, 0, 2]])
def test_backward_padding_never_reaches_a_gradient(dtype, d, lengths):
    q, k, v = _qkv(4, 4, 2, 300, d, dtype, 5)
    dy = normal(q.shape, dtype, 9)
    for b, n in enumerate(lengths):
        for x in (q, k, v, dy):
            x[b, :, n:] = float("nan") if b % 2 else float("inf")
    _check_backward(q, k, v, dy, 40, 4, dtype, lengths=lengths)
    _check_backward(q, k, v, dy, 400, 0, dtype, lengths=lengths)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_views_and_given_outputs(dtype):
    q, k, v = _qkv(2, 4, 2, 230, 64, dtype, 8)
    dy = normal(q.shape, dtype, 10)
    views = fused(*(x.to(DEV) for x in (q, k, v))) + [token_major(dy.to(DEV))]
    dense = _check_backward(q, k, v, dy, 50, 5, dtype)
    got = _check_backward(q, k, v, dy, 50, 5, dtype, views=views)
    for a, b in zip(dense, got):
        assert torch.equal(a, b)
    out = torch.zeros((2, 230, 8, 64), dtype=DT[dtype], device=DEV)
    parts = [out[:, :, a:b].transpose(1, 2) for a, b in ((0, 4), (4, 6), (6, 8))]
    y, lse, _, _ = based.swa_sink_prefill(*views[:3], 50, 5, want_cache=False, want_lse=True)
    based.swa_sink_backward(*views[:3], y, lse, views[3], 50, 5, dq=parts[0], dk=parts[1], dv=parts[2])
    for a, b in zip(dense, parts):
        assert torch.equal(a, b)


def test_backward_equal_weights_and_large_scores():
    q, k, v = _qkv(1, 4, 2, 260, 64, "bf16", 91)
    dy = normal(q.shape, "bf16", 92)
    for w in (30, 100):
        dq, dk, _ = _check_backward(q, k, v, dy, w, 3, "bf16", scale=0.0)
        assert torch.all(dq == 0) and torch.all(dk == 0)
        _check_backward(q * 4, k * 4, v, dy, w, 3, "bf16", scale=0.5)


@pytest.mark.parametrize("d", [64, 128])
def test_backward_longer_and_deterministic(d):
    """Sink chunks beyond one, rings that wrap, and the same bits twice."""
    q, k, v = _qkv(1, 8, 2, 1100, d, "bf16", 61)
    dy = normal(q.shape, "bf16", 62)
    a = _check_backward(q, k, v, dy, 150, 10, "bf16")
    b = _check_backward(q, k, v, dy, 150, 10, "bf16")
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    _check_backward(q, k, v, dy, 3000, 0, "bf16")


def test_backward_captured():
    q, k, v = (x.to(DEV) for x in _qkv(1, 4, 2, 400, 64, "bf16", 71))
    dy = normal(q.shape, "bf16", 72).to(DEV)

    def step():
        y, lse, _, _ = based.swa_sink_prefill(q, k, v, 90, 4, want_cache=False, want_lse=True)
        return (y,) + based.swa_sink_backward(q, k, v, y, lse, dy, 90, 4)

    eager = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        held = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, held):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """fp32: the directional derivative of sum(dy * y) along random directions."""
    q, k, v = _qkv(1, 2, 1, 150, 64, "f32", 81)
    dy = normal(q.shape, "f32", 82)
    g = [f64(x) for x in _check_backward(q, k, v, dy, 40, 4, "f32")]
    f = lambda a: float((f64(dy) * oracle.swa_sink(*a, 40, 4, scale_of(64))[0]).sum())
    base = [f64(x) for x in (q, k, v)]
    for which in range(3):
        direction = np.random.default_rng(which).standard_normal(base[which].shape)
        hi, lo = list(base), list(base)
        hi[which], lo[which] = base[which] + 1e-4 * direction, base[which] - 1e-4 * direction
        num = (f(hi) - f(lo)) / 2e-4
        ana = float((g[which] * direction).sum())
        # central differences: O(h^2) of a third derivative of order 1e2 per term; fp32 gradients
        assert abs(num - ana) <= 1e-4 * np.sqrt((g[which] ** 2).sum()) * np.sqrt((direction ** 2).sum())


# ------------------------------------------------------------------ room around the outputs, waits that run out

def _tailed(shape, dtype, seed=0):
    """A dense tensor of this shape at the front of a buffer with a sentinel tail."""
    n = int(np.prod(shape))
    buf = torch.full((n + 1024,), 3.0, dtype=dtype, device=DEV)
    return buf[:n].view(shape), buf[n:]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,w,sinks,lengths", [(129, 40, 5, [129, 70]), (1, 3, 2, [1, 0]), (200, 900, 0, [3, 200])])
def test_outputs_keep_to_their_buffers(dtype, N, w, sinks, lengths):
    B, Hq, Hkv, d = 2, 4, 2, 64
    q, k, v = (x.to(DEV) for x in _qkv(B, Hq, Hkv, N, d, dtype, 95))
    dy = normal((B, Hq, N, d), dtype, 96).to(DEV)
    ln = torch.tensor(lengths, device=DEV)
    outs = {n: _tailed(sh, torch.float32 if n == "lse" else DT[dtype])
            for n, sh in dict(y=(B, Hq, N, d), lse=(B, Hq, N), k_cache=(B, Hkv, sinks + w, d),
                              v_cache=(B, Hkv, sinks + w, d)).items()}
    based.swa_sink_prefill(q, k, v, w, sinks, lengths=ln, **{n: o[0] for n, o in outs.items()})
    grads = {n: _tailed(sh, DT[dtype]) for n, sh in dict(dq=q.shape, dk=k.shape, dv=v.shape).items()}
    need = based.swa_sink_backward_workspace(B, Hq, Hkv, N, d, w, sinks, DT[dtype])
    ws, ws_tail = _tailed((need,), torch.uint8)
    based.swa_sink_backward(q, k, v, outs["y"][0], outs["lse"][0], dy, w, sinks, lengths=ln, workspace=ws,
                            **{n: g[0] for n, g in grads.items()})
    yd, yd_tail = _tailed((B, Hq, d), DT[dtype])
    based.swa_sink_decode(outs["k_cache"][0], outs["v_cache"][0], ln, q[:, :, 0].contiguous(), k[:, :, 0].contiguous(),
                          v[:, :, 0].contiguous(), w, sinks, y=yd)
    assert based.get_last_error() == 0
    for tail in [o[1] for o in outs.values()] + [g[1] for g in grads.values()] + [ws_tail, yd_tail]:
        assert torch.all(tail == 3)


@pytest.mark.parametrize("w", [40, 900, 1100])
@pytest.mark.parametrize("d", [64, 128])
def test_stalled_tensor_core_is_reported_and_the_context_stays_usable(monkeypatch, d, w):
    """No MMA is issued, so every wait for one runs out (after 2 s): a status, no fault."""
    q, k, v = (x.to(DEV) for x in _qkv(1, 2, 2, 300, d, "bf16", 97))
    dy = normal(q.shape, "bf16", 98).to(DEV)
    y, lse, _, _ = based.swa_sink_prefill(q, k, v, w, 4, want_cache=False, want_lse=True)
    good = based.swa_sink_backward(q, k, v, y, lse, dy, w, 4)
    assert based.get_last_error() == 0
    monkeypatch.setenv("BASED_DEBUG_SKIP_MMA", "1")
    based.swa_sink_prefill(q, k, v, w, 4, want_cache=False)
    assert based.get_last_error() == 4
    based.swa_sink_backward(q, k, v, y, lse, dy, w, 4)
    assert based.get_last_error() == 4
    monkeypatch.delenv("BASED_DEBUG_SKIP_MMA")
    assert torch.equal(based.swa_sink_prefill(q, k, v, w, 4, want_cache=False)[0], y)
    for a, b in zip(based.swa_sink_backward(q, k, v, y, lse, dy, w, 4), good):
        assert torch.equal(a, b)
    assert based.get_last_error() == 0


def test_calls_on_two_streams_at_once():
    """Prompts, gradients and decode steps that share SMs (and tensor memory) with each other."""
    sets = []
    for i, (d, w) in enumerate([(64, 40), (128, 300), (64, 900), (128, 64)]):
        q, k, v = (x.to(DEV) for x in _qkv(2, 4, 2, 900, d, "bf16", 100 + i))
        sets.append((q, k, v, normal(q.shape, "bf16", 110 + i).to(DEV), w))

    def work(q, k, v, dy, w):
        y, lse, kc, vc = based.swa_sink_prefill(q, k, v, w, 4, want_lse=True)
        pos = torch.full((2,), 900, device=DEV)
        t = [x[:, :, 5].contiguous() for x in (q, k, v)]
        return (y,) + based.swa_sink_backward(q, k, v, y, lse, dy, w, 4) + (based.swa_sink_decode(kc, vc, pos, *t, w, 4),)

    alone = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    together = [None] * len(sets)
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                together[i] = work(*sets[i])
    torch.cuda.synchronize()
    assert based.get_last_error() == 0
    for a, b in zip(alone, together):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


# ------------------------------------------------------------------ offsets past 32 bits

def test_decode_offsets_past_32_bits():
    """The last sequence's cache lies past 2^31 elements (4.8 GB each of K and V)."""
    B, Hkv, Hq, d, w, t = 72, 1, 4, 128, 1 << 18, 1000
    kc, vc = (torch.empty(B, Hkv, w, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v, q = (normal((h, t + 1, d), "bf16", 120 + h) for h in (1, 2, 5))
    v, q = v[:1], q[:Hq]
    kc[-1, :, :t], vc[-1, :, :t] = k[:, :t].to(DEV), v[:, :t].to(DEV)
    pos = torch.full((B,), -1, device=DEV)
    pos[-1] = t
    one = [torch.zeros(B, h, d, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv)]
    for x, y in zip(one, (q, k, v)):
        x[-1] = y[:, t].to(DEV)
    got = based.swa_sink_decode(kc, vc, pos, *one, w)
    assert based.get_last_error() == 0
    scale = scale_of(d)
    ref, _, mass = oracle.swa_sink(f64(q)[None], f64(k)[None], f64(v)[None], w, 0, scale)
    tol = tol_y(ref, mass, q, k, scale, "bf16", t + 1)
    assert_within(f64(got)[-1], ref[0, :, t], tol[0, :, t], "y")
    assert torch.all(got[:-1] == 0)
    assert torch.equal(kc[-1, 0, t].cpu(), k[0, t]) and torch.equal(vc[-1, 0, t].cpu(), v[0, t])


@pytest.mark.parametrize("d,w", [(64, 40), (128, 40), (64, 2000), (128, 2000)])
def test_strides_past_32_bits(d, w):
    """Sequences 2^31 elements apart give the bits of dense ones."""
    N, H = 200, 2
    gap = (1 << 31) + 1024

    def far(seed=None):
        big = torch.empty(gap + H * N * d, dtype=torch.bfloat16, device=DEV)
        x = big.as_strided((2, H, N, d), (gap, N * d, d, 1))
        if seed is not None:
            x.copy_(normal((2, H, N, d), "bf16", seed))
        return x

    q, k, v, dy, y = far(130), far(131), far(132), far(133), far()
    _, lse, _, _ = based.swa_sink_prefill(q, k, v, w, 3, want_cache=False, want_lse=True, y=y)
    dense = [x.contiguous() for x in (q, k, v)]
    yd, lsed, _, _ = based.swa_sink_prefill(*dense, w, 3, want_cache=False, want_lse=True)
    assert torch.equal(y, yd) and torch.equal(lse, lsed)
    grads = based.swa_sink_backward(q, k, v, y, lse, dy, w, 3, dq=far(), dk=far(), dv=far())
    for a, b in zip(grads, based.swa_sink_backward(*dense, yd, lsed, dy.contiguous(), w, 3)):
        assert torch.equal(a, b)
    assert based.get_last_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("w", [40, 1500])
def test_prompts_and_tokens_back_to_back_over_one_cache(dtype, w):
    """The cache's fill may start while the attention ends: it never overtakes an earlier reader."""
    B, Hq, Hkv, N, d = 2, 8, 2, 1000, 64
    sets = [[x.to(DEV) for x in _qkv(B, Hq, Hkv, N, d, dtype, 140 + i)] for i in range(3)]
    pos = torch.full((B,), N, device=DEV)
    kc, vc = (torch.empty(B, Hkv, 4 + w, d, dtype=DT[dtype], device=DEV) for _ in range(2))

    def run(q, k, v):
        y = based.swa_sink_prefill(q, k, v, w, 4, k_cache=kc, v_cache=vc)[0]
        return y, based.swa_sink_decode(kc, vc, pos, *(x[:, :, 7].contiguous() for x in (q, k, v)), w, 4)

    alone = []
    for s in sets:
        alone.append(run(*s))
        torch.cuda.synchronize()
    for _ in range(20):
        together = [run(*s) for s in sets]
    for a, b in zip(alone, together):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert based.get_last_error() == 0


@pytest.mark.parametrize("dtype,w", [("f32", 40), ("bf16", 40), ("bf16", 1500)])
def test_prompt_captured_and_replayed_beside_another(dtype, w):
    """Two graphs of a prompt and a token over their own caches, replayed at once on new inputs."""
    B, Hq, Hkv, N, d = 2, 4, 2, 700, 64
    pos = torch.full((B,), N, device=DEV)

    def run(q, k, v, kc, vc):
        y, lse, _, _ = based.swa_sink_prefill(q, k, v, w, 4, want_lse=True, k_cache=kc, v_cache=vc)
        return y, lse, based.swa_sink_decode(kc, vc, pos, *(x[:, :, 9].contiguous() for x in (q, k, v)), w, 4)

    graphs = []
    for i in range(2):
        x = [t.to(DEV) for t in _qkv(B, Hq, Hkv, N, d, dtype, 150 + i)]
        x += [torch.empty(B, Hkv, 4 + w, d, dtype=DT[dtype], device=DEV) for _ in range(2)]
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run(*x)
            with torch.cuda.graph(g, stream=s):
                out = run(*x)
        graphs.append((x, s, g, out))
    for seed in (160, 170):
        new = [[t.to(DEV) for t in _qkv(B, Hq, Hkv, N, d, dtype, seed + i)] for i in range(2)]
        for (x, s, g, _), n in zip(graphs, new):
            for a, b in zip(x, n):
                a.copy_(b)
        torch.cuda.synchronize()
        for _ in range(5):
            for _, s, g, _ in graphs:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for (x, _, _, out), n in zip(graphs, new):
            caches = [torch.empty_like(t) for t in x[3:]]
            for a, b in zip(out, run(*n, *caches)):
                assert torch.equal(a, b)
            assert torch.equal(x[3], caches[0]) and torch.equal(x[4], caches[1])
    assert based.get_last_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,N,w,sinks", [(1, 71, 1, 150, 20, 4), (1, 3, 1, 1400, 1100, 4), (1, 4, 2, 1290, 1200, 33)])
def test_odd_groups_and_windows_past_a_thousand(d, B, Hq, Hkv, N, w, sinks):
    q, k, v = _qkv(B, Hq, Hkv, N, d, "bf16", N)
    _check_prefill(q, k, v, w, sinks, "bf16", lengths=[N - 7])
    _check_backward(q, k, v, normal(q.shape, "bf16", 8), w, sinks, "bf16", lengths=[N - 7])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,N,w,sinks,lengths", [
    (4, 4, 1100, 64, 4, [1100, 300, 130]), (8, 2, 1500, 40, 33, [700, 90]), (2, 1, 900, 1, 64, [899, 0, 66, 129]),
])
def test_backward_of_short_sequences_in_a_long_batch(dtype, d, Hq, Hkv, N, w, sinks, lengths):
    """Many chunks of the sinks' pairs, some of them all padding in a sequence that has real tiles."""
    q, k, v = _qkv(len(lengths), Hq, Hkv, N, d, dtype, 180)
    _check_backward(q, k, v, normal(q.shape, dtype, 183), w, sinks, dtype, lengths=lengths)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("w,sinks", [(20, 2), (400, 0)])
def test_length_out_of_range_is_reported_by_the_backward(dtype, w, sinks):
    q, k, v = (x.to(DEV) for x in _qkv(3, 2, 2, 170, 64, dtype, 33))
    dy = normal(q.shape, dtype, 34).to(DEV)
    inside = torch.tensor([0, 170, 90], device=DEV)
    y, lse, _, _ = based.swa_sink_prefill(q, k, v, w, sinks, lengths=inside, want_cache=False, want_lse=True)
    want = based.swa_sink_backward(q, k, v, y, lse, dy, w, sinks, lengths=inside)
    assert based.get_last_error() == 0
    for bad in ([-5, 1000, 90], [-1 << 40, 170, 90], [0, 171, 90]):
        got = based.swa_sink_backward(q, k, v, y, lse, dy, w, sinks, lengths=torch.tensor(bad, device=DEV))
        assert based.get_last_error() == 1 and based.get_last_error() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_backward_padding_rows_are_zeros_beside_non_finite_tokens(dtype, d, value):
    """Real tokens next to the sequences' ends hold infinities and NaN; padding stays zero."""
    lengths = [3, 70, 150, 129]
    q, k, v = _qkv(4, 4, 2, 170, d, dtype, 190)
    dy = normal(q.shape, dtype, 193)
    for b, n in enumerate(lengths):
        for x in (q, k, v, dy):
            x[b, :, n - 1] = value
    ln = torch.tensor(lengths, device=DEV)
    q, k, v, dy = (x.to(DEV) for x in (q, k, v, dy))
    for w, sinks in ((40, 4), (400, 0)):
        y, lse, _, _ = based.swa_sink_prefill(q, k, v, w, sinks, lengths=ln, want_cache=False, want_lse=True)
        for x in (y,) + based.swa_sink_backward(q, k, v, y, lse, dy, w, sinks, lengths=ln):
            for b, n in enumerate(lengths):
                assert torch.all(x[b, :, n:] == 0)
    assert based.get_last_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_infinity_seen_by_rows_of_a_million_keys(d):
    """Rows computed again one by one take seconds there; no wait of the kernel's runs out over them."""
    N, at = 1 << 20, (1 << 20) - 300
    g = torch.Generator(device=DEV).manual_seed(200)
    q, k, v = (torch.randn(1, 1, N, d, generator=g, device=DEV).bfloat16() for _ in range(3))
    clean = based.swa_sink_prefill(q, k, v, N, 0, want_cache=False, want_lse=True)
    v[0, 0, at, 5] = float("inf")
    y, lse, _, _ = based.swa_sink_prefill(q, k, v, N, 0, want_cache=False, want_lse=True)
    assert based.get_last_error() == 0
    tile = at - at % 128                                     # its rows share a product with the infinity
    assert torch.equal(y[:, :, :tile], clean[0][:, :, :tile]) and torch.equal(lse[:, :, :tile], clean[1][:, :, :tile])
    assert torch.all(y[0, 0, at:, 5] == float("inf")) and torch.all(torch.isfinite(y[0, 0, tile:at]))
    # Both are within one rounding of y, the rounding of the weights and the scores' error (see
    # sink_util.tol_y) of the definition.
    rows = q[0, 0, tile:].double() @ k[0, 0].double().T * scale_of(d)
    rows.masked_fill_(torch.arange(N, device=DEV)[None] > torch.arange(tile, N, device=DEV)[:, None], float("-inf"))
    p = torch.softmax(rows, 1)
    vv = v[0, 0].double()
    vv[at, 5] = 0.0
    others = torch.arange(d, device=DEV) != 5
    mass, ref = (p @ vv.abs())[:, others], (p @ vv)[:, others]
    size = scale_of(d) * float(q.float().abs().max() * k.float().abs().sum(-1).max())
    rel = 2 * ((d + 4) * U["bf16"] * size + 2.0 ** -20) + N * U["f32"] + HALF["bf16"]
    tol = rel * (1 + 2.0 ** -6) * mass + HALF["bf16"] * ref.abs()
    for x in (y, clean[0]):
        assert torch.all((x[0, 0, tile:][:, others].double() - ref).abs() <= tol)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,w,sinks,positions", [
    (3, 8, 2, 7, 3, [2, 5, 30]), (2, 20, 1, 64, 4, [70, 40]), (1, 4, 1, 3000, 4, [5000]), (64, 4, 4, 300, 4, [299] * 64),
])
def test_decode_weights_keep_their_bits(d, B, Hq, Hkv, w, sinks, positions):
    """bf16: the weights enter the second product with 2^-15 of them lost, not 2^-8: cut off to
    bf16, the rest (below 2^-7 of a weight) rounded to bf16 (2^-8 of it)."""
    q, k, v = (normal((B, h, d), "bf16", 210 + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    kc, vc = (normal((B, Hkv, sinks + w, d), "bf16", 213 + i) for i in range(2))
    ref, rk, _, mass = oracle.swa_sink_decode_step(f64(kc), f64(vc), positions, f64(q), f64(k), f64(v), w, sinks, scale_of(d))
    y = based.swa_sink_decode(kc.to(DEV), vc.to(DEV), torch.tensor(positions, device=DEV), q.to(DEV), k.to(DEV), v.to(DEV), w,
                              sinks)
    assert based.get_last_error() == 0
    keys = min(w + sinks, max(positions) + 1)
    rel = 2 * score_error(q, torch.from_numpy(rk), scale_of(d), "bf16") + keys * U["bf16"] + 2.0 ** -15
    assert_within(y, ref, rel * (1 + 2.0 ** -6) * mass + HALF["bf16"] * np.abs(ref) + 1e-30, "decode y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,w", [(64, 90), (64, 1100), (128, 90), (128, 300)])
def test_small_scales_of_large_scores(dtype, d, w):
    """Scores of 1e35 under scales that make them of order 1, or under 0: equal weights."""
    q, k, v = _qkv(1, 2, 1, 260, d, dtype, 220)
    q, k = q * 1e17, k * 1e17
    dy = normal(q.shape, dtype, 223)
    for scale in (2e-35, 0.0):
        _check_prefill(q, k, v, w, 3, dtype, scale=scale)
        _check_backward(q, k, v, dy, w, 3, dtype, scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,N,w,sinks,lengths", [
    (64, 300, 1100, 5, [300, 129]), (64, 1290, 1100, 0, [1290, 1]), (64, 1290, 1030, 64, [1283, 1100]), (64, 1026, 800, 5, [1026, 0]),
    (128, 129, 40, 5, [129, 70]), (128, 300, 250, 64, [300, 2]), (128, 1, 900, 2, [1, 0]), (128, 700, 200, 0, [3, 700]),
])
def test_outputs_of_every_kernel_keep_to_their_buffers(dtype, d, N, w, sinks, lengths):
    """The wide prompt kernel, whose rows are stored one by one, and all of d = 128."""
    B, Hq, Hkv = 2, 6, 2
    q, k, v = (x.to(DEV) for x in _qkv(B, Hq, Hkv, N, d, dtype, 230))
    dy = normal((B, Hq, N, d), dtype, 233).to(DEV)
    ln = torch.tensor(lengths, device=DEV)
    outs = {n: _tailed(sh, torch.float32 if n == "lse" else DT[dtype])
            for n, sh in dict(y=(B, Hq, N, d), lse=(B, Hq, N), k_cache=(B, Hkv, sinks + w, d),
                              v_cache=(B, Hkv, sinks + w, d)).items()}
    based.swa_sink_prefill(q, k, v, w, sinks, lengths=ln, **{n: o[0] for n, o in outs.items()})
    grads = {n: _tailed(sh, DT[dtype]) for n, sh in dict(dq=q.shape, dk=k.shape, dv=v.shape).items()}
    need = based.swa_sink_backward_workspace(B, Hq, Hkv, N, d, w, sinks, DT[dtype])
    ws, ws_tail = _tailed((need,), torch.uint8)
    based.swa_sink_backward(q, k, v, outs["y"][0], outs["lse"][0], dy, w, sinks, lengths=ln, workspace=ws,
                            **{n: g[0] for n, g in grads.items()})
    yd, yd_tail = _tailed((B, Hq, d), DT[dtype])
    based.swa_sink_decode(outs["k_cache"][0], outs["v_cache"][0], ln, *(x[:, :, 0].contiguous() for x in (q, k, v)), w, sinks,
                          y=yd)
    assert based.get_last_error() == 0
    for tail in [o[1] for o in outs.values()] + [g[1] for g in grads.values()] + [ws_tail, yd_tail]:
        assert torch.all(tail == 3)


@pytest.mark.parametrize("lengths", [[0, 1100, 1, 129], [128, 1050, 0, 64], [257, 255, 1024, 2]])
@pytest.mark.parametrize("d,w,sinks", [(64, 1100, 0), (64, 1030, 7), (128, 193, 7)])
def test_padding_never_reaches_a_row_of_the_wide_kernel(d, w, sinks, lengths):
    q, k, v = _qkv(4, 4, 2, 1100, d, "bf16", 240)
    dy = normal(q.shape, "bf16", 243)
    for b, n in enumerate(lengths):
        for x in (q, k, v, dy):
            x[b, :, n:] = float("nan") if b % 2 else float("inf")
    _check_prefill(q, k, v, w, sinks, "bf16", lengths=lengths)
    _check_backward(q, k, v, dy, w, sinks, "bf16", lengths=lengths)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1)])
def test_wide_kernel_reports_a_stalled_tensor_core(monkeypatch, Hq, Hkv):
    q, k, v = (x.to(DEV) for x in _qkv(1, Hq, Hkv, 1100, 64, "bf16", 97))
    y = based.swa_sink_prefill(q, k, v, 2000, 4, want_cache=False)[0]
    assert based.get_last_error() == 0
    monkeypatch.setenv("BASED_DEBUG_SKIP_MMA", "1")
    based.swa_sink_prefill(q, k, v, 2000, 4, want_cache=False)
    assert based.get_last_error() == 4
    monkeypatch.delenv("BASED_DEBUG_SKIP_MMA")
    assert torch.equal(based.swa_sink_prefill(q, k, v, 2000, 4, want_cache=False)[0], y)
    assert based.get_last_error() == 0


@pytest.mark.parametrize("d,N", [(64, 768), (64, 769), (64, 1025), (128, 192), (128, 193), (128, 300)])
def test_prompts_at_the_border_of_the_two_kernels(d, N):
    """The border is at min(w, N): windows just inside it, at it and past it."""
    q, k, v = _qkv(1, 4, 2, N, d, "bf16", 260)
    for w in (191, 192, 193) if d == 128 else (767, 768, 769, N // 2 + 256, N // 2 + 257, 5000):
        _check_prefill(q, k, v, w, 4, "bf16")


def test_wide_kernels_on_two_streams_at_once():
    sets = [[x.to(DEV) for x in _qkv(2, 4, 2, 1500, d, "bf16", 250 + i)] + [w]
            for i, (d, w) in enumerate([(64, 1100), (128, 300), (64, 1300), (64, 1100)])]

    def work(q, k, v, w):
        return based.swa_sink_prefill(q, k, v, w, 4, want_lse=True)

    alone = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        together = []
        for s, x in zip(streams, sets):
            with torch.cuda.stream(s):
                together.append(work(*x))
    torch.cuda.synchronize()
    assert based.get_last_error() == 0
    for a, b in zip(alone, together):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def _check_hidden(dtype, d, Hq, Hkv, N, w, sinks, at, bad, value, lengths=None):
    """Token `at` of the tensors `bad` is non-finite: gradients that no pair with it enters are as if
    it held zeros. Returns the gradients and which queries and keys are such."""
    scale = scale_of(d)
    B = 1 if lengths is None else len(lengths)
    t = dict(zip("qkv", _qkv(B, Hq, Hkv, N, d, dtype, at)))
    t["g"] = normal(t["q"].shape, dtype, at + 1)
    clean = {n: f64(x).copy() for n, x in t.items()}
    for n in bad:
        clean[n][:, :, at] = 0.0
        t[n][:, :, at] = value
    g = {n: x.to(DEV) for n, x in t.items()}
    ln = None if lengths is None else torch.tensor(lengths, device=DEV)
    y, lse, _, _ = based.swa_sink_prefill(g["q"], g["k"], g["v"], w, sinks, lengths=ln, want_cache=False, want_lse=True)
    got = based.swa_sink_backward(g["q"], g["k"], g["v"], y, lse, g["g"], w, sinks, lengths=ln)
    assert based.get_last_error() == 0
    see = oracle.sink_visible(N, w, sinks)
    spoilt = np.zeros(N, dtype=bool)                              # queries
    if set("kv") & set(bad):
        spoilt |= see[:, at]
    if set("qg") & set(bad):
        spoilt[at] = True
    keys = ~see[spoilt].any(axis=0)                               # keys that no such query sees
    cq, ck = torch.from_numpy(clean["q"]), torch.from_numpy(clean["k"])
    ref, _, mass = oracle.swa_sink(clean["q"], clean["k"], clean["v"], w, sinks, scale, lengths)
    count = min(N, w + sinks)
    err = score_error(cq, ck, scale, dtype)
    ey = (2 * err * mass if dtype == "bf16" and w + sinks < 64 else tol_y(ref, mass, cq, ck, scale, dtype, count)) + \
        (d + 4) * U[dtype] * 2 * float(np.abs(clean["v"]).max())
    rel = 2 * err + N * (Hq // Hkv) * U[dtype] + HALF[dtype]
    out = oracle.swa_sink_backward(*(clean[n] for n in "qkvg"), w, sinks, scale, lengths, ey, rel * (1 + 2.0 ** -6))
    for name, x, r, e, rows in zip(("dq", "dk", "dv"), got, out[:3], out[3:], (~spoilt, keys, keys)):
        assert_within(f64(x)[:, :, rows], r[:, :, rows], (e + HALF[dtype] * np.abs(r) + 1e-30)[:, :, rows], name)
    return got, ~spoilt, keys


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad,value", [("k", float("nan")), ("v", float("inf")), ("q", float("inf")), ("g", float("nan")),
                                       ("qkvg", float("nan"))])
@pytest.mark.parametrize("Hq,Hkv,N,w,sinks,at", [(2, 1, 600, 40, 4, 150), (1, 1, 900, 100, 0, 130), (4, 2, 500, 300, 16, 450),
                                                 (2, 2, 700, 64, 33, 699)])
def test_backward_hidden_non_finite_tokens_reach_no_gradient(dtype, d, bad, value, Hq, Hkv, N, w, sinks, at):
    got, queries, keys = _check_hidden(dtype, d, Hq, Hkv, N, w, sinks, at, bad, value)
    assert queries.sum() > N // 3 and keys.any()
    if "k" in bad:                                                # a NaN score: the definition's NaN
        assert torch.all(torch.isnan(got[0][:, :, torch.from_numpy(~queries).to(DEV)]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_hidden_non_finite_tokens_in_a_padded_batch(dtype, d):
    for at, bad in ((200, "qkvg"), (650, "v"), (2, "q")):
        _check_hidden(dtype, d, 4, 2, 1100, 64, 4, at, bad, float("inf"), lengths=[1100, 700, 203])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("w,sinks,at", [(100, 4, 20), (65, 1, 63), (300, 16, 16), (100, 4, 300)])
def test_hidden_infinities_beside_the_sinks_and_beside_visible_ones(dtype, d, w, sinks, at):
    """Token `at` shares the first keys' block with the sinks; a sink's own value is infinite in one
    channel, which every row shows there and nowhere else."""
    N, scale = 700, scale_of(d)
    q, k, v = _qkv(1, 2, 1, N, d, dtype, at)
    clean = (f64(k).copy(), f64(v).copy())
    for c in clean:
        c[:, :, at] = 0.0
    k[:, :, at] = v[:, :, at] = float("inf")
    v[:, :, 0, 7] = float("inf")
    clean[1][:, :, 0, 7] = 0.0
    y, lse, _, _ = based.swa_sink_prefill(*(x.to(DEV) for x in (q, k, v)), w, sinks, want_cache=False, want_lse=True)
    hidden = ~oracle.sink_visible(N, w, sinks)[:, at]
    assert hidden.sum() > 100
    ref, rlse, mass = oracle.swa_sink(f64(q), *clean, w, sinks, scale)
    tol = tol_y(ref, mass, q, torch.from_numpy(clean[0]), scale, dtype, w + sinks)
    other = np.arange(d) != 7
    got = f64(y)
    assert_within(got[:, :, hidden][..., other], ref[:, :, hidden][..., other], tol[:, :, hidden][..., other], "hidden rows")
    assert np.all(got[:, :, hidden, 7] == np.inf)
    assert np.abs(f64(lse)[:, :, hidden] - rlse[:, :, hidden]).max() < 1e-3
    assert based.get_last_error() == 0
    _check_hidden(dtype, d, 2, 1, N, w, sinks, at, "k", float("inf"))
    _check_hidden(dtype, d, 2, 1, N, w, sinks, at, "qg", float("nan"))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("w", [1, 20, 1100])
def test_nothing_behind_a_sequence_is_looked_at(dtype, d, w):
    """An infinite sink spoils every row; what lies behind the tensors' last token, or behind a
    length, changes no bit of any result."""
    B, N, H = 2, 1200 if w > 1000 else 200, 2
    lengths = torch.tensor([N, N - 50], device=DEV)
    base = [normal((B, N + 200, H, d), dtype, 270 + i).to(DEV) for i in range(4)]
    for x in base[1:3]:
        x[:, 0, :, 5] = float("inf") if x is base[2] else 0.0
    base[0][:, :, :, 5] = 0.0

    def run(fill):
        t = []
        for x in base:
            x = x.clone()
            x[:, N:] = fill
            x[1, N - 50:] = fill
            t.append(x[:, :N].transpose(1, 2))
        q, k, v, dy = t
        out = []
        for ln in (lengths, None):
            if ln is None:
                q, k, v, dy = (x[:1] for x in t)
            y, lse, _, _ = based.swa_sink_prefill(q, k, v, w, 1, lengths=ln, want_cache=False, want_lse=True)
            out += [y, lse, *based.swa_sink_backward(q, k, v, y, lse, dy, w, 1, lengths=ln)]
        assert based.get_last_error() == 0
        return out

    clean, dirty = run(0.0), run(float("nan"))
    for a, b in zip(clean, dirty):
        assert torch.equal(torch.nan_to_num(a.float(), nan=7e30), torch.nan_to_num(b.float(), nan=7e30))
    for y in (clean[0], clean[5]):
        assert torch.all(y[0, :, :, 5] == float("inf")) and torch.all(torch.isfinite(y[0, ..., 6:]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,w,sinks,positions", [
    (2, 4, 2, 7, 3, [30, 5]), (1, 20, 1, 64, 4, [70]), (2, 4, 1, 1, 1, [9, 1]), (1, 8, 2, 3000, 4, [5000]), (1, 5, 5, 40, 0, [0]),
])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_decode_shows_a_visible_infinity_as_it_is(dtype, d, B, Hq, Hkv, w, sinks, positions, value):
    """One value in use is not finite: so is its channel in every head that reads it, no other."""
    q, k, v = (normal((B, h, d), dtype, 280 + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    kc, vc = (normal((B, Hkv, sinks + w, d), dtype, 283 + i) for i in range(2))
    vc[:, :, 0, 5] = v[:, :, 5] = 0.0
    ref, rk, _, mass = oracle.swa_sink_decode_step(f64(kc), f64(vc), positions, f64(q), f64(k), f64(v), w, sinks, scale_of(d))
    tol = tol_y(ref, mass, q, torch.from_numpy(rk), scale_of(d), dtype, min(w + sinks, max(positions) + 1))
    for x in (vc[:, :, 0], v):                               # a slot in use that is not the token's own; the token
        x[:, :, 5] = value
        y = f64(based.swa_sink_decode(kc.to(DEV), vc.to(DEV), torch.tensor(positions, device=DEV), q.to(DEV), k.to(DEV),
                                      v.to(DEV), w, sinks))
        assert based.get_last_error() == 0
        x[:, :, 5] = 0.0
        spoilt = y[..., 5]
        if x is v or min(positions) > 0:
            assert np.all(np.isnan(spoilt) if np.isnan(value) else spoilt == value)
        other = np.arange(d) != 5
        assert_within(y[..., other], ref[..., other], tol[..., other], "other channels")


@pytest.mark.parametrize("w", [1156, 1157])
def test_prompts_at_the_border_with_many_tiles(w):
    """450 tiles, enough for three per SM: the border is at N / 2 + 256."""
    _check_prefill(*_qkv(1, 30, 2, 1800, 64, "bf16", 290), w, 4, "bf16")
