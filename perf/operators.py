"""Measured cases of the sliding-window attention with sink tokens and of the query/key
norm with rotary positions.

Five operators, each through the package's public calls:

* prefill: causal softmax attention over a prompt, a query seeing the last ``w`` tokens
  (itself included) and the first ``sinks`` tokens; the generation cache is filled too;
* decode: one token per sequence over that cache (``sinks`` fixed slots, then a ring of ``w``);
* train: the same attention forward and backward (y, dq, dk, dv);
* rope: per-head RMS norm of queries and keys with the rotation by position, in one pass;
* rope_grad: its gradient (both inputs and both norm weights).

``own`` selects what ``run`` calls: elementary torch operations in 32 bits, or the package.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROPE_BASE = 10000.0
EPS = 1e-6


def listed():
    attn = dict(ragged=False, far=False)
    rope = dict(interleaved=False, max_pos=32768)
    return [
        # A prompt batch of the 360M-shaped model: its 16 heads of 64, the library's window of 64.
        dict(attn, name="prefill_base", op="prefill", B=8, Hq=16, Hkv=16, N=2048, d=64, w=64, sinks=4, dtype="bf16"),
        # Long prompts, shared key/value heads of 128 and a window of a thousand tokens: matrix-bound.
        dict(attn, name="prefill_long", op="prefill", B=2, Hq=16, Hkv=4, N=16384, d=128, w=1024, sinks=4,
             dtype="bf16"),
        # A padded batch of uneven prompts (one empty) at odd sizes, in full precision.
        dict(attn, name="prefill_ragged", op="prefill", B=5, Hq=8, Hkv=2, N=1337, d=64, w=200, sinks=7, dtype="f32",
             ragged=True),
        # One user's next token on the small window: latency only.
        dict(attn, name="decode_one", op="decode", B=1, Hq=16, Hkv=16, N=1, d=64, w=64, sinks=4, dtype="bf16"),
        # A serving batch, some sequences still filling their ring: the cache read bounds it.
        dict(attn, name="decode_batch", op="decode", B=64, Hq=16, Hkv=4, N=1, d=128, w=1024, sinks=4, dtype="bf16"),
        # One sequence with a long window: few rows, a long axis.
        dict(attn, name="decode_far", op="decode", B=1, Hq=16, Hkv=4, N=1, d=128, w=32768, sinks=16, dtype="bf16",
             far=True),
        # Training on the 360M shape.
        dict(attn, name="train_base", op="train", B=8, Hq=16, Hkv=16, N=2048, d=64, w=64, sinks=4, dtype="bf16"),
        # Training on long sequences with shared heads of 128.
        dict(attn, name="train_long", op="train", B=2, Hq=16, Hkv=4, N=8192, d=128, w=1024, sinks=4, dtype="bf16"),
        # Norm and rotation before the attention of the 360M shape: one pass over memory.
        dict(rope, name="rope_base", op="rope", B=8, Hq=16, Hkv=16, N=2048, d=64, rot=64, dtype="bf16"),
        # The same for one generated token of a serving batch: latency.
        dict(rope, name="rope_step", op="rope", B=64, Hq=16, Hkv=4, N=1, d=128, rot=128, dtype="bf16"),
        # Its gradient in training.
        dict(rope, name="rope_grad_base", op="rope_grad", B=8, Hq=16, Hkv=16, N=2048, d=64, rot=64, dtype="bf16"),
        # The gradient at odd lengths, half of each head rotated as neighbouring pairs, full precision.
        dict(rope, name="rope_grad_odd", op="rope_grad", B=3, Hq=8, Hkv=2, N=1531, d=128, rot=64, dtype="f32",
             interleaved=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case: the same operators, sizes spread over the whole range, odd ones among them."""
    limit = {}
    for c in listed():
        wk = work(c)
        old = limit.get(c["op"], (0, 0))
        limit[c["op"]] = (max(old[0], wk["bytes"]), max(old[1], wk["flops"]))
    while True:
        op = rng.choice(["prefill", "decode", "train", "rope", "rope_grad"])
        Hq, Hkv = rng.choice([(16, 16), (16, 4), (16, 1), (8, 8), (8, 2), (6, 3), (5, 1), (1, 1)])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if op in ("rope", "rope_grad"):
            d = rng.choice([16, 32, 64, 64, 96, 128, 128, 256])
            rot = d if rng.random() < 0.6 else 16 * rng.randint(1, d // 16)
            case = dict(op=op, B=_log_int(rng, 1, 64), Hq=Hq, Hkv=Hkv, N=_log_int(rng, 1, 16384), d=d, rot=rot,
                        dtype=dtype, interleaved=rng.random() < 0.4, max_pos=32768)
        else:
            d = rng.choice([64, 128])
            sinks = rng.choice([0, 1, 4, 4, 16, 33, 64])
            if op == "decode":
                case = dict(op=op, B=_log_int(rng, 1, 256), Hq=Hq, Hkv=Hkv, N=1, d=d, w=_log_int(rng, 1, 32768),
                            sinks=sinks, dtype=dtype, ragged=rng.random() < 0.5, far=rng.random() < 0.5)
            else:
                case = dict(op=op, B=_log_int(rng, 1, 16), Hq=Hq, Hkv=Hkv, N=_log_int(rng, 1, 16384), d=d,
                            w=_log_int(rng, 1, 4096), sinks=sinks, dtype=dtype, ragged=rng.random() < 0.4, far=False)
                if dtype == "f32" and work(case)["flops"] > 2e10:
                    continue
        wk = work(case)
        if wk["bytes"] <= limit[op][0] and wk["flops"] <= limit[op][1]:
            return case


# ------------------------------------------------------------------ inputs

def _lengths(case, rng):
    """Tokens per sequence of a padded batch: one full, one empty where there are several."""
    B, N = case["B"], case["N"]
    n = [rng.randint(1, N) for _ in range(B)]
    if B > 2:
        n[rng.randrange(B)] = 0
    n[rng.randrange(B)] = N
    return n


def _positions(case, rng):
    """Tokens each sequence has seen: a young one, ones that filled the ring, -1 for an idle row."""
    B, w, s = case["B"], case["w"], case["sinks"]
    if case["far"]:
        return [w + s + rng.randint(0, 1 << 20) for _ in range(B)]
    t = [rng.randint(0, 3 * (w + s)) for _ in range(B)]
    if case["ragged"] and B > 1:
        t[rng.randrange(B)] = -1
    return t


def prepare(case, seed):
    import random
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = random.Random(seed)
    dt = DT[case["dtype"]]
    B, Hq, Hkv, N, d = (case[k] for k in ("B", "Hq", "Hkv", "N", "d"))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    # The projections' outputs, token-major; keys and values come from one fused projection.
    qp = normal(B, N, Hq, d)
    kvp = normal(B, N, 2 * Hkv, d)
    st = dict(case)
    st["q"] = qp.transpose(1, 2)
    st["k"] = kvp[:, :, :Hkv].transpose(1, 2)
    st["v"] = kvp[:, :, Hkv:].transpose(1, 2)
    op = case["op"]
    if op in ("prefill", "train"):
        st["scale"] = 1.0 / math.sqrt(d)
        st["lengths"] = torch.tensor(_lengths(case, rng), dtype=torch.int64, device=dev) if case["ragged"] else None
        if op == "train":
            st["dy"] = normal(B, N, Hq, d).transpose(1, 2)
    elif op == "decode":
        st["scale"] = 1.0 / math.sqrt(d)
        st["q"], st["k"], st["v"] = (st[n][:, :, 0].contiguous() for n in "qkv")
        slots = case["sinks"] + case["w"]
        st["k_cache"] = normal(B, Hkv, slots, d)
        st["v_cache"] = normal(B, Hkv, slots, d)
        st["positions"] = torch.tensor(_positions(case, rng), dtype=torch.int64, device=dev)
    else:
        rot, mp = case["rot"], case["max_pos"]
        start = torch.tensor([rng.randint(0, mp - N) for _ in range(B)], dtype=torch.int64, device=dev)
        st["positions"] = start[:, None] + torch.arange(N, device=dev)
        inv = ROPE_BASE ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=dev) / rot)
        ang = torch.arange(mp, dtype=torch.float64, device=dev)[:, None] * inv
        # cos and sin of every position, as such a program keeps them: [max_pos, rot / 2, 2]
        st["table"] = torch.stack([ang.cos(), ang.sin()], dim=-1).float().contiguous()
        st["wq"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=dev)
        st["wk"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=dev)
        if op == "rope_grad":
            st["dqr"] = normal(B, Hq, N, d)
            st["dkr"] = normal(B, Hkv, N, d)
    return st


# ------------------------------------------------------------------ the plain forms

def _blocks(N, w, sinks, rows):
    """Row blocks with the key columns they can see: (r0, r1, column indices)."""
    for r0 in range(0, N, rows):
        r1 = min(N, r0 + rows)
        c0 = max(0, r0 - w + 1)
        yield r0, r1, list(range(min(sinks, c0))), c0


def _block_scores(st, q, k, r0, r1, cols, w, sinks):
    i = torch.arange(r0, r1, device=q.device)[:, None]
    j = cols[None, :]
    keep = (j <= i) & ((j > i - w) | (j < sinks))
    s = torch.matmul(q[:, :, :, r0:r1], k[:, :, None, cols].transpose(-1, -2)) * st["scale"]
    return torch.where(keep, s, torch.full_like(s, float("-inf")))


def _plain_attention(st, want_grad):
    q, k, v = (st[n].float() for n in "qkv")
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    w, sinks, dt = st["w"], st["sinks"], DT[st["dtype"]]
    q = q.reshape(B, Hkv, Hq // Hkv, N, d)
    y = torch.zeros_like(q)
    rows = max(64, min(1024, N))
    pad = None
    if st["lengths"] is not None:
        pad = torch.arange(N, device=q.device)[None, :] >= st["lengths"][:, None]          # [B, N]
    if want_grad:
        dy = st["dy"].float().reshape(B, Hkv, Hq // Hkv, N, d)
        if pad is not None:
            dy = dy.masked_fill(pad[:, None, None, :, None], 0.0)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for r0, r1, first, c0 in _blocks(N, w, sinks, rows):
        cols = torch.cat([torch.arange(len(first), device=q.device), torch.arange(c0, r1, device=q.device)])
        s = _block_scores(st, q, k, r0, r1, cols, w, sinks)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        yb = torch.matmul(p, v[:, :, None, cols])
        y[:, :, :, r0:r1] = yb
        if want_grad:
            g = dy[:, :, :, r0:r1]
            dp = torch.matmul(g, v[:, :, None, cols].transpose(-1, -2))
            ds = p * (dp - (g * yb).sum(-1, keepdim=True)) * st["scale"]
            dq[:, :, :, r0:r1] = torch.matmul(ds, k[:, :, None, cols])
            dk.index_add_(2, cols, torch.matmul(ds.transpose(-1, -2), q[:, :, :, r0:r1]).sum(2))
            dv.index_add_(2, cols, torch.matmul(p.transpose(-1, -2), g).sum(2))
    y = y.reshape(B, Hq, N, d)
    if pad is not None:
        y = y.masked_fill(pad[:, None, :, None], 0.0)
    if not want_grad:
        return y.to(dt)
    return {"y": y.to(dt), "dq": dq.reshape(B, Hq, N, d).to(dt), "dk": dk.to(dt), "dv": dv.to(dt)}


def _plain_cache(st, x):
    """The generation cache after the prompt: sink slots, then the ring; zeros where no token went."""
    B, Hkv, N, d = x.shape
    w, sinks = st["w"], st["sinks"]
    n = st["lengths"] if st["lengths"] is not None else torch.full((B,), N, dtype=torch.int64, device=x.device)
    ring = torch.arange(w, device=x.device)[None, :]
    last = n[:, None] - 1 - sinks - ring
    tok = ring + sinks + w * torch.div(last, w, rounding_mode="floor")
    tok = torch.where(last >= 0, tok, torch.full_like(tok, -1))
    sink = torch.arange(sinks, device=x.device)[None, :].expand(B, sinks)
    sink = torch.where(sink < n[:, None], sink, torch.full_like(sink, -1))
    tok = torch.cat([sink, tok], 1)
    idx = tok.clamp(min=0)[:, None, :, None].expand(B, Hkv, sinks + w, d)
    return torch.where((tok >= 0)[:, None, :, None], x.gather(2, idx), torch.zeros((), dtype=x.dtype, device=x.device))


def _plain_decode(st):
    kc, vc, q, t = st["k_cache"], st["v_cache"], st["q"], st["positions"]
    B, Hkv, slots, d = kc.shape
    w, sinks = st["w"], st["sinks"]
    slot = torch.where(t < sinks, t, sinks + torch.remainder(t - sinks, w))
    live = t >= 0
    here = (torch.arange(slots, device=q.device)[None, :] == slot[:, None]) & live[:, None]      # [B, slots]
    kc.copy_(torch.where(here[:, None, :, None], st["k"][:, :, None, :], kc))
    vc.copy_(torch.where(here[:, None, :, None], st["v"][:, :, None, :], vc))
    seen = torch.arange(slots, device=q.device)[None, :] <= t[:, None]        # a full ring shows every slot
    qf = q.float().reshape(B, Hkv, -1, d)
    s = torch.matmul(qf, kc.float().transpose(-1, -2)) * st["scale"]
    s = torch.where(seen[:, None, None, :], s, torch.full_like(s, float("-inf")))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    y = torch.matmul(torch.where(seen[:, None, None, :], p, torch.zeros_like(p)), vc.float())
    y = torch.where(live[:, None, None, None], y, torch.zeros_like(y))
    return {"y": y.reshape(q.shape).to(q.dtype), "k_cache": kc, "v_cache": vc}


def _rotate(x, c, s, rot, interleaved):
    """Rotate the first `rot` channels by (c, s) [B, 1, N, rot / 2]."""
    h, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = h[..., 0::2], h[..., 1::2]
        r = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    else:
        a, b = h[..., : rot // 2], h[..., rot // 2:]
        r = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _plain_rope(st, grad):
    cs = st["table"][st["positions"]][:, None]                                # [B, 1, N, rot / 2, 2]
    c, s = cs[..., 0], cs[..., 1]
    out = []
    wgrad = []
    for x, wgt, dr in ((st["q"], st["wq"], st.get("dqr")), (st["k"], st["wk"], st.get("dkr"))):
        xf = x.float()
        r = 1.0 / torch.sqrt((xf * xf).mean(-1, keepdim=True) + EPS)
        xh = xf * r
        if not grad:
            out.append(_rotate(xh * wgt, c, s, st["rot"], st["interleaved"]).to(x.dtype))
            continue
        dn = _rotate(dr.float(), c, -s, st["rot"], st["interleaved"])
        wgrad.append((dn * xh).sum((0, 1, 2)))
        dh = dn * wgt
        out.append((r * (dh - xh * (dh * xh).mean(-1, keepdim=True))).to(x.dtype))
    return tuple(out + wgrad)


# ------------------------------------------------------------------ one pass

def run(state):
    st = state
    op = st["op"]
    if own:
        import linear_attention_sequence_causal_b200 as based
        if op == "prefill":
            y, _, kc, vc = based.swa_sink_prefill(st["q"], st["k"], st["v"], st["w"], st["sinks"], scale=st["scale"],
                                                  lengths=st["lengths"])
            return {"y": y, "k_cache": kc, "v_cache": vc}
        if op == "decode":
            y = based.swa_sink_decode(st["k_cache"], st["v_cache"], st["positions"], st["q"], st["k"], st["v"],
                                      st["w"], st["sinks"], scale=st["scale"])
            return {"y": y, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        if op == "train":
            y, lse, _, _ = based.swa_sink_prefill(st["q"], st["k"], st["v"], st["w"], st["sinks"], scale=st["scale"],
                                                  lengths=st["lengths"], want_cache=False, want_lse=True)
            dq, dk, dv = based.swa_sink_backward(st["q"], st["k"], st["v"], y, lse, st["dy"], st["w"], st["sinks"],
                                                 scale=st["scale"], lengths=st["lengths"])
            return {"y": y, "dq": dq, "dk": dk, "dv": dv}
        if op == "rope":
            return based.qk_norm_rope(st["q"], st["k"], st["table"], st["positions"], q_weight=st["wq"],
                                      k_weight=st["wk"], eps=EPS, interleaved=st["interleaved"])
        return based.qk_norm_rope_backward(st["q"], st["k"], st["table"], st["positions"], st["dqr"], st["dkr"],
                                           q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
                                           interleaved=st["interleaved"])
    if op == "prefill":
        y = _plain_attention(st, False)
        return {"y": y, "k_cache": _plain_cache(st, st["k"]), "v_cache": _plain_cache(st, st["v"])}
    if op == "decode":
        return _plain_decode(st)
    if op == "train":
        return _plain_attention(st, True)
    return _plain_rope(st, op == "rope_grad")


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs(N, w, sinks):
    """Query-key pairs of one head over a sequence of N tokens."""
    def tri(n):
        return n * (n + 1) // 2
    band = tri(min(N, w)) + max(0, N - w) * w
    # sink j is outside the window of queries i >= j + w
    return band + sum(max(0, N - w - j) for j in range(min(sinks, N)))


def work(case):
    B, Hq, Hkv, N, d = (case[k] for k in ("B", "Hq", "Hkv", "N", "d"))
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    qb, kb = B * Hq * N * d * e, B * Hkv * N * d * e
    if op == "prefill" or op == "train":
        # Ragged batches are counted at half their padded length on average.
        frac = 0.5 if case["ragged"] else 1.0
        flops = 4 * d * _pairs(N, case["w"], case["sinks"]) * B * Hq * frac
        if op == "prefill":
            cache = 2 * B * Hkv * (case["w"] + case["sinks"]) * d * e
            return {"bytes": qb * (1 + frac) + 2 * kb * frac + cache, "flops": flops}
        return {"bytes": qb * (2 + 2 * frac) + kb * (2 + 2 * frac), "flops": flops * 3.5}
    if op == "decode":
        slots = case["w"] + case["sinks"]
        # Without a full ring the drawn positions (0 .. 3 slots) show 5/6 of it on average.
        frac = 1.0 if case["far"] else 5.0 / 6.0
        return {"bytes": 2 * B * Hkv * slots * d * e * frac + 2 * qb + 4 * kb,
                "flops": 4 * B * Hq * slots * d * frac}
    table = min(case["max_pos"], B * N) * case["rot"] * 4
    if op == "rope":
        return {"bytes": 2 * (qb + kb) + table + B * N * 8 + 8 * d, "flops": 9 * B * (Hq + Hkv) * N * d}
    return {"bytes": 3 * (qb + kb) + table + B * N * 8 + 16 * d, "flops": 16 * B * (Hq + Hkv) * N * d}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_head(q, k, v, w, sinks, scale):
    """softmax over the visible keys of one head, [N, d] each, dense mask."""
    N = q.shape[0]
    i = torch.arange(N, device=q.device).unsqueeze(1)
    j = torch.arange(N, device=q.device).unsqueeze(0)
    hidden = (j > i) | ((j <= i - w) & (j >= sinks))
    return torch.softmax((q @ k.t() * scale).masked_fill(hidden, -math.inf), dim=1) @ v


def _exact_cache(case, x, n):
    out = torch.zeros((x.shape[0], case["sinks"] + case["w"], x.shape[2]), dtype=torch.float64, device=x.device)
    for t in list(range(min(n, case["sinks"]))) + list(range(max(case["sinks"], n - case["w"]), n)):
        out[:, t if t < case["sinks"] else case["sinks"] + (t - case["sinks"]) % case["w"]] = x[:, t]
    return out


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    B, Hq, Hkv, N, d = (case[k] for k in ("B", "Hq", "Hkv", "N", "d"))
    G = Hq // Hkv
    q, k, v = (st[n].double() for n in "qkv")
    if op in ("prefill", "train"):
        grad = op == "train"
        if N > 12000 and B * Hq > 64:
            return None
        lens = [N] * B if st["lengths"] is None else st["lengths"].tolist()
        y = torch.zeros_like(q)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for b, n in enumerate(lens):
            for h in range(Hq if n else 0):
                qh, kh, vh = (x[b, hh, :n].clone().requires_grad_(grad) for x, hh in ((q, h), (k, h // G), (v, h // G)))
                yh = _exact_head(qh, kh, vh, case["w"], case["sinks"], st["scale"])
                y[b, h, :n] = yh.detach()
                if grad:
                    yh.backward(st["dy"][b, h, :n].double())
                    dq[b, h, :n] = qh.grad
                    dk[b, h // G, :n] += kh.grad
                    dv[b, h // G, :n] += vh.grad
                del yh
        if grad:
            return {"y": y, "dq": dq, "dk": dk, "dv": dv}
        caches = [torch.stack([_exact_cache(case, x[b], n) for b, n in enumerate(lens)]) for x in (k, v)]
        return {"y": y, "k_cache": caches[0], "v_cache": caches[1]}
    if op == "decode":
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        y = torch.zeros_like(q)
        for b, t in enumerate(st["positions"].tolist()):
            if t < 0:
                continue
            sl = t if t < case["sinks"] else case["sinks"] + (t - case["sinks"]) % case["w"]
            kc[b, :, sl], vc[b, :, sl] = k[b], v[b]
            n = min(t + 1, case["sinks"] + case["w"])
            for h in range(Hq):
                a = torch.softmax(kc[b, h // G, :n] @ q[b, h] * st["scale"], 0)
                y[b, h] = a @ vc[b, h // G, :n]
        return {"y": y, "k_cache": kc, "v_cache": vc}
    rot = case["rot"]
    f = torch.exp(torch.arange(0, rot, 2, dtype=torch.float64, device=q.device) * (-math.log(ROPE_BASE) / rot))
    phase = torch.polar(torch.ones((), dtype=torch.float64, device=q.device),
                        st["positions"].double().unsqueeze(-1) * f).unsqueeze(1)            # [B, 1, N, rot / 2]

    def forward(x, wgt):
        n = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * wgt
        a = n[..., :rot]
        if case["interleaved"]:
            z = torch.view_as_complex(a.reshape(*a.shape[:-1], rot // 2, 2).contiguous()) * phase
            a = torch.view_as_real(z).reshape(a.shape)
        else:
            z = torch.complex(a[..., : rot // 2], a[..., rot // 2:]) * phase
            a = torch.cat([z.real, z.imag], -1)
        return torch.cat([a, n[..., rot:]], -1)

    wq, wk = st["wq"].double(), st["wk"].double()
    if op == "rope":
        return forward(q, wq), forward(k, wk)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, wq, wk)]
    loss = (forward(leaves[0], leaves[2]) * st["dqr"].double()).sum() \
        + (forward(leaves[1], leaves[3]) * st["dkr"].double()).sum()
    return tuple(torch.autograd.grad(loss, leaves))
