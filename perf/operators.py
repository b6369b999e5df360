"""Workloads of the selective state space operators and the block norm.

Each case is one operator on inputs of a real call: the causal convolution and the
selective scan over packed prompts, the decode step of both for a batch of requests,
and the norms around a block.  ``run`` makes the library's calls where ``own`` is
true; elsewhere it evaluates the same formulas with elementary torch operations.

The formulas, with head h reading group h % n_groups (r = n_heads / n_groups heads per group):

* conv:  y[t][c] = act(bias[c] + sum_j w[c][j] X[t - (K - 1) + j][c]), the rows before a
  sequence's first taken from its slot of ``hist`` (zeros for a new sequence); ``hist``
  then holds the last K - 1 rows.
* scan:  dt = softplus(a + dt_bias), S <- exp(-exp(A_log) dt) S + dt B x^T,
  y = (S^T C + D x) silu(z), S [state_dim][head_dim] per head, from and back to its slot.
* step:  the convolution and the scan of one token for each request.
* norm:  r <- r + scale gate RMSNorm(b; w_post), y = RMSNorm(r; w_pre).
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_CHUNK = 128


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------- the cases


def _conv(name, dtype, tokens, seqs, channels, width, bias, pad, fresh):
    return {"name": name, "op": "conv", "dtype": dtype, "tokens": tokens, "seqs": seqs, "channels": channels,
            "width": width, "bias": bias, "pad": pad, "fresh": fresh}


def _scan(name, dtype, tokens, seqs, heads, groups, head_dim, state_dim, gate, pad, fresh):
    return {"name": name, "op": "scan", "dtype": dtype, "tokens": tokens, "seqs": seqs, "heads": heads,
            "groups": groups, "head_dim": head_dim, "state_dim": state_dim, "gate": gate, "pad": pad, "fresh": fresh}


def _step(name, dtype, batch, heads, groups, head_dim, state_dim, width, gate):
    return {"name": name, "op": "step", "dtype": dtype, "batch": batch, "heads": heads, "groups": groups,
            "head_dim": head_dim, "state_dim": state_dim, "width": width, "gate": gate}


def _norm(name, dtype, stream, tokens, dim, post, gate):
    return {"name": name, "op": "norm", "dtype": dtype, "stream": stream, "tokens": tokens, "dim": dim, "post": post,
            "gate": gate}


def listed():
    return [
        # one 2048-token call of a prompt, the packed row of 48 heads and 2 x 16 groups of 128
        _conv("conv bf16 2048x10240", "bf16", 2048, 1, 10240, 4, True, 0, False),
        # a long FP32 batch of several prompts, some of them new
        _conv("conv fp32 16383x10240, 7 seqs", "fp32", 16383, 7, 10240, 4, False, 9, True),
        # a few prompt tokens in FP32: latency and the launch count
        _scan("scan fp32 77, 1 seq", "fp32", 77, 1, 48, 16, 128, 128, True, 0, False),
        # one 2048-token call of a prompt, its state carried
        _scan("scan bf16 2048, 1 seq", "bf16", 2048, 1, 48, 16, 128, 128, True, 0, False),
        # a batch of prompts of ragged lengths, packed and padded
        _scan("scan fp16 16375, 24 seqs", "fp16", 16375, 24, 48, 16, 128, 128, True, 25, True),
        # one whole long prompt
        _scan("scan bf16 32768, 1 seq", "bf16", 32768, 1, 48, 16, 128, 128, True, 0, True),
        # decode: one request, a usual batch, a large batch with FP32 activations
        _step("step bf16 batch 1", "bf16", 1, 48, 16, 128, 128, 4, True),
        _step("step bf16 batch 64", "bf16", 64, 48, 16, 128, 128, 4, True),
        _step("step fp32 batch 250", "fp32", 250, 48, 16, 128, 128, 4, False),
        # the norms between two blocks: one decode token, a prompt, a ragged prompt in FP16
        _norm("norm bf16 1x6144", "bf16", "bf16", 1, 6144, True, "row"),
        _norm("norm bf16 8192x6144", "bf16", "fp32", 8192, 6144, True, "token"),
        _norm("norm fp16 4099x2048", "fp16", "fp16", 4099, 2048, False, "none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "conv":
        tokens = _log(rng, 1, 16000)
        c = _conv("", dtype, tokens, min(tokens, _log(rng, 1, 64)), 8 * _log(rng, 8, 1280), rng.choice([2, 3, 4, 4]),
                  rng.random() < 0.5, rng.choice([0, 0, 5]), rng.random() < 0.5)
    elif op == "scan":
        tokens = _log(rng, 1, 4000 if dtype == "fp32" else 24000)
        groups = rng.choice([1, 2, 4, 8, 16])
        c = _scan("", dtype, tokens, min(tokens, _log(rng, 1, 48)), groups * rng.choice([1, 2, 3]), groups,
                  rng.choice([64, 128, 128]), rng.choice([64, 128, 128]), rng.random() < 0.5, rng.choice([0, 0, 5]),
                  rng.random() < 0.5)
    elif op == "step":
        groups = rng.choice([1, 2, 4, 8, 16])
        c = _step("", dtype, _log(rng, 1, 240), groups * rng.choice([1, 2, 3]), groups, rng.choice([64, 128, 128]),
                  rng.choice([64, 128, 128]), rng.choice([2, 3, 4, 4]), rng.random() < 0.5)
    else:
        c = _norm("", dtype, rng.choice([dtype, "fp32"]), _log(rng, 1, 8000), 2 * _log(rng, 64, 4096),
                  rng.random() < 0.5, rng.choice(["none", "row", "token"]))
    del c["name"]
    return c


def _lengths(case):
    """The packed sequences' lengths: a spread of sizes that sums to `tokens` (from the case alone)."""
    n, total = case["seqs"], case["tokens"]
    if n == 1:
        return [total]
    rng = random.Random(1000 * n + total)
    w = [math.exp(rng.uniform(-1.5, 1.5)) for _ in range(n)]
    lens = [max(1, int(total * x / sum(w))) for x in w]
    while sum(lens) > total:
        lens[lens.index(max(lens))] -= 1
    lens[rng.randrange(n)] += total - sum(lens)
    return lens


def _slots_of(n, seed):
    """n different slots of a pool of n + 2, in no order."""
    rng = random.Random(seed)
    return rng.sample(range(n + 2), n)


def prepare(case, seed):
    dev, ty = _dev(), _TYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float32) * (hi - lo) + lo

    s = {"case": case}
    if case["op"] in ("conv", "scan"):
        n, lens = case["seqs"], _lengths(case)
        s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=dev)
        s["slots"] = torch.tensor(_slots_of(n, seed), dtype=torch.int32, device=dev)
        s["has"] = torch.tensor([not (case["fresh"] and i % 2 == 0) for i in range(n)], dtype=torch.bool, device=dev)
        s["chunks"] = sum(-(-m // _CHUNK) for m in lens)
        rows = case["tokens"] + case["pad"]
    if case["op"] == "conv":
        c, k = case["channels"], case["width"]
        s["x"] = normal(rows, c, dtype=ty)
        s["w"] = uniform(-0.5, 0.5, c, k)
        s["bias"] = 0.1 * normal(c) if case["bias"] else None
        s["hist"] = normal(n + 2, k - 1, c, dtype=ty)
        s["out"] = torch.zeros((rows, c), dtype=ty, device=dev)
        return s
    if case["op"] == "norm":
        t, d = case["tokens"], case["dim"]
        s["b"] = normal(t, d, dtype=ty)
        s["r"] = (2 * normal(t, d)).to(_TYPES[case["stream"]])
        s["w_pre"] = 1 + 0.1 * normal(d)
        s["w_post"] = 1 + 0.1 * normal(d) if case["post"] else None
        s["gate"] = None if case["gate"] == "none" else normal(1 if case["gate"] == "row" else t, d, dtype=ty)
        return s
    h, g, p, m = case["heads"], case["groups"], case["head_dim"], case["state_dim"]
    s["A_log"] = torch.log(uniform(1.0, 16.0, h))
    s["dt_bias"] = torch.log(torch.expm1(torch.exp(uniform(math.log(1e-3), math.log(0.1), h))))
    s["D"] = 1 + 0.1 * normal(h)
    cw = h * p + 2 * g * m
    if case["op"] == "scan":
        # the convolution's output: x, B and C side by side in one row
        s["xbc"] = normal(rows, cw, dtype=ty)
        s["a"] = normal(rows, h, dtype=ty)
        s["z"] = normal(rows, h, p, dtype=ty) if case["gate"] else None
        s["states"] = 0.1 * normal(n + 2, h, m, p)
        s["out"] = torch.zeros((rows, h, p), dtype=ty, device=dev)
        return s
    n = case["batch"]
    s["slots"] = torch.tensor(_slots_of(n, seed), dtype=torch.int32, device=dev)
    s["xbc"] = normal(n, cw, dtype=ty)
    s["a"] = normal(n, h, dtype=ty)
    s["z"] = normal(n, h, p, dtype=ty) if case["gate"] else None
    s["w"] = uniform(-0.5, 0.5, cw, case["width"])
    s["bias"] = 0.1 * normal(cw)
    s["hist"] = normal(n + 2, case["width"] - 1, cw, dtype=ty)
    s["states"] = 0.1 * normal(n + 2, h, m, p)
    return s


def _parts(case, xbc):
    """x [rows][heads][head_dim], B and C [rows][groups][state_dim], as views of the packed row."""
    h, g, p, m = case["heads"], case["groups"], case["head_dim"], case["state_dim"]
    x, b, c = xbc.split([h * p, g * m, g * m], dim=-1)
    return x.unflatten(-1, (h, p)), b.unflatten(-1, (g, m)), c.unflatten(-1, (g, m))


# ---------------------------------------------------------------- one pass


def run(s):
    return {"conv": _run_conv, "scan": _run_scan, "step": _run_step, "norm": _run_norm}[s["case"]["op"]](s)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _run_conv(s):
    case = s["case"]
    if own:
        from linear_attention_recurrence_gb300 import gdn

        y = gdn.gdn_ssm_conv(s["x"], s["w"], bias=s["bias"], hist=s["hist"], cu_seqlens=s["cu"], slots=s["slots"],
                             has_state=s["has"], out=s["out"])
        return {"y": y, "hist": s["hist"]}
    k, t, cu = case["width"], case["tokens"], s["cu"].long()
    x, hist, slots = s["x"][:t], s["hist"], s["slots"].long()
    lens = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device=cu.device), lens, output_size=t)
    # row `at` of (history, sequence) for every token and tap: the history's rows are -(K-1) .. -1
    taps = torch.arange(k, device=cu.device) - (k - 1)
    at = (torch.arange(t, device=cu.device) - cu[seq])[:, None] + taps
    rows = _rows_of(x, hist, slots, s["has"], cu, seq[:, None], at, k)
    y = torch.einsum("tkc,ck->tc", rows, s["w"])
    if s["bias"] is not None:
        y = y + s["bias"]
    s["out"][:t] = _silu(y).to(x.dtype)
    last = lens[:, None] + torch.arange(k - 1, device=cu.device) - (k - 1)
    new = _rows_of(x, hist, slots, s["has"], cu, torch.arange(case["seqs"], device=cu.device)[:, None], last, k)
    hist[slots] = new.to(hist.dtype)
    return {"y": s["out"], "hist": hist}


def _rows_of(x, hist, slots, has, cu, seq, at, k):
    """Row `at` of sequence `seq`, in FP32; negative rows come from its history (zeros if it has none)."""
    old = hist[slots[seq], (at + k - 1).clamp(0, k - 2)].float() * has[seq][..., None]
    new = x[(cu[seq] + at).clamp(0, x.shape[0] - 1)].float()
    return torch.where((at < 0)[..., None], old, new)


def _run_scan(s):
    case = s["case"]
    if own:
        from linear_attention_recurrence_gb300 import gdn

        x, b, c = _parts(case, s["xbc"])
        y = gdn.gdn_ssm_scan(x, s["a"], b, c, s["A_log"], s["dt_bias"], s["states"], D=s["D"], z=s["z"],
                             cu_seqlens=s["cu"], slots=s["slots"], has_state=s["has"], out=s["out"])
        return {"y": y, "states": s["states"]}
    h, g, p, m, n, t = (case[k] for k in ("heads", "groups", "head_dim", "state_dim", "seqs", "tokens"))
    r, nc, cu, dev = h // g, s["chunks"], s["cu"].long(), s["cu"].device
    lens = cu[1:] - cu[:-1]
    per = (lens + _CHUNK - 1) // _CHUNK
    seq = torch.repeat_interleave(torch.arange(n, device=dev), per, output_size=nc)
    first = (torch.cumsum(per, 0) - per)[seq]
    tok = (cu[seq] + (torch.arange(nc, device=dev) - first) * _CHUNK)[:, None] + torch.arange(_CHUNK, device=dev)
    live = tok < cu[seq + 1][:, None]
    tok = tok.clamp(max=t - 1)
    x, b, c = (v[tok].float() * live[:, :, None, None] for v in _parts(case, s["xbc"]))
    # gates in 64 bits: their running sums over a long sequence are large
    dt = _softplus(s["a"][tok].double() + s["dt_bias"].double()) * live[..., None]  # [nc][L][h]
    gam = torch.cumsum(-torch.exp(s["A_log"].double()) * dt, 1).transpose(1, 2)  # [nc][h][L]
    dt = dt.float().transpose(1, 2)
    xh = x.unflatten(2, (r, g)).permute(0, 2, 3, 1, 4)  # [nc][r][g][L][p]
    bg, cg = b.transpose(1, 2), c.transpose(1, 2)  # [nc][g][L][m]
    low = torch.ones((_CHUNK, _CHUNK), dtype=torch.bool, device=dev).tril()
    decay = torch.exp(torch.where(low, (gam[..., :, None] - gam[..., None, :]), -math.inf).float())
    mix = (cg @ bg.transpose(-1, -2))[:, None] * (decay * dt[..., None, :]).unflatten(1, (r, g))
    y = mix @ xh
    del decay, mix
    # each chunk's own contribution to the state after it, then the states before every chunk
    end = (torch.exp((gam[..., -1:] - gam).float()) * dt).unflatten(1, (r, g))
    part = bg.transpose(-1, -2)[:, None] @ (xh * end[..., None])  # [nc][r][g][m][p]
    part = part.flatten(1, 2).transpose(0, 1).flatten(2)  # [h][nc][m p]
    total = torch.cumsum(gam[..., -1], 0).transpose(0, 1)  # [h][nc], through each chunk
    before = total - gam[..., -1].transpose(0, 1)
    base = before.gather(1, first[None].expand(h, nc))  # before each chunk's sequence
    own_state = s["states"][s["slots"].long()] * s["has"][:, None, None, None]
    start = own_state.transpose(0, 1).flatten(2)  # [h][n][m p]
    idx = torch.arange(nc, device=dev)
    same = (seq[:, None] == seq[None, :]) & (idx[:, None] > idx[None, :])
    carry = torch.exp(torch.where(same, before[:, :, None] - total[:, None, :], -math.inf).float())
    prev = carry @ part + torch.exp((before - base).float())[..., None] * start[:, seq]
    prev = prev.unflatten(2, (m, p)).transpose(0, 1).unflatten(1, (r, g))  # [nc][r][g][m][p]
    y = y + torch.exp(gam.float()).unflatten(1, (r, g))[..., None] * (cg[:, None] @ prev)
    del prev, carry
    y = y.permute(0, 3, 1, 2, 4).flatten(2, 3) + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"][tok].float())
    s["out"][tok[live]] = y[live].to(s["out"].dtype)
    # the states after every sequence (every one has a token)
    last = torch.cumsum(per, 0) - 1
    mine = seq[None, :] == torch.arange(n, device=dev)[:, None]
    weight = torch.exp(torch.where(mine, total[:, last][:, :, None] - total[:, None, :], -math.inf).float())
    after = weight @ part + torch.exp((total[:, last] - base[:, last]).float())[..., None] * start
    s["states"][s["slots"].long()] = after.unflatten(2, (m, p)).transpose(0, 1)
    return {"y": s["out"], "states": s["states"]}


def _run_step(s):
    case = s["case"]
    if own:
        from linear_attention_recurrence_gb300 import gdn

        y = gdn.gdn_ssm_step(s["xbc"], s["a"], s["w"], s["A_log"], s["dt_bias"], s["hist"], s["states"],
                             conv_bias=s["bias"], D=s["D"], z=s["z"], slots=s["slots"])
        return {"y": y, "hist": s["hist"], "states": s["states"]}
    h, g = case["heads"], case["groups"]
    slots, new = s["slots"].long(), s["xbc"][:, None]
    rows = torch.cat([s["hist"][slots], new], 1)
    u = _silu(torch.einsum("nkc,ck->nc", rows.float(), s["w"]) + s["bias"])
    s["hist"][slots] = rows[:, 1:]
    x, b, c = _parts(case, u)
    dt = _softplus(s["a"].float() + s["dt_bias"])
    keep = torch.exp(-torch.exp(s["A_log"]) * dt)
    of = torch.arange(h, device=u.device) % g
    st = s["states"][slots] * keep[..., None, None] + (dt[..., None] * b[:, of])[..., :, None] * x[..., None, :]
    s["states"][slots] = st
    y = (st * c[:, of][..., None]).sum(2) + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"y": y.to(s["xbc"].dtype), "hist": s["hist"], "states": s["states"]}


_EPS, _SCALE = 1e-6, 0.7


def _run_norm(s):
    case = s["case"]
    if own:
        from linear_attention_recurrence_gb300 import gdn

        r, y = gdn.gdn_block_norm(s["b"], s["r"], s["w_pre"], w_post=s["w_post"], gate=s["gate"], gate_sigmoid=True,
                                  scale=_SCALE, eps=_EPS, residual_out=torch.empty_like(s["r"]))
        return {"residual": r, "y": y}
    u = s["b"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + _EPS) * s["w_post"]
    if s["gate"] is not None:
        u = u / (1 + torch.exp(-s["gate"].float()))
    r = s["r"].float() + _SCALE * u
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + _EPS) * s["w_pre"]
    return {"residual": r.to(s["r"].dtype), "y": y.to(_TYPES[case["dtype"]])}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "conv":
        t, c, k, n = case["tokens"], case["channels"], case["width"], case["seqs"]
        kept = sum(1 for i in range(n) if not (case["fresh"] and i % 2 == 0))
        return {"bytes": 2 * t * c * e + c * (k + case["bias"]) * 4 + (kept + n) * (k - 1) * c * e,
                "flops": t * c * (2 * k + 4)}
    if case["op"] == "norm":
        t, d, er = case["tokens"], case["dim"], _BYTES[case["stream"]]
        gate = {"none": 0, "row": d, "token": t * d}[case["gate"]]
        return {"bytes": 2 * t * d * (e + er) + gate * e + 4 * d * (1 + case["post"]), "flops": 10 * t * d}
    h, g, p, m = case["heads"], case["groups"], case["head_dim"], case["state_dim"]
    state = 4 * h * p * m
    if case["op"] == "step":
        n, k, cw = case["batch"], case["width"], h * p + 2 * g * m
        return {"bytes": n * (2 * state + e * (cw * (2 * k - 1) + h + h * p * (1 + case["gate"]))) + 4 * cw * (k + 1),
                "flops": n * (6 * h * p * m + 2 * k * cw)}
    t, n = case["tokens"], case["seqs"]
    kept = sum(1 for i in range(n) if not (case["fresh"] and i % 2 == 0))
    return {"bytes": e * t * (h * p * (2 + case["gate"]) + 2 * g * m + h) + state * (n + kept),
            "flops": 6 * t * h * p * m}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    """The definition, token by token, in 64 bits."""
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "step": _exact_step, "norm": _exact_norm}[case["op"]](s)


def _exact_conv(s):
    case, k = s["case"], s["case"]["width"]
    y, hist, cu, slots = s["out"].double(), s["hist"].double(), s["cu"].tolist(), s["slots"].tolist()
    for i, slot in enumerate(slots):
        old = hist[slot] if bool(s["has"][i]) else torch.zeros_like(hist[slot])
        ext = torch.cat([old, s["x"][cu[i]:cu[i + 1]].double()])
        acc = sum(s["w"][:, j].double() * ext[j:ext.shape[0] - (k - 1) + j] for j in range(k))
        acc = acc if s["bias"] is None else acc + s["bias"].double()
        y[cu[i]:cu[i + 1]] = acc * torch.sigmoid(acc)
        hist[slot] = ext[ext.shape[0] - (k - 1):]
    return {"y": y, "hist": hist}


def _recur(case, x, b, c, a, st, s):
    """One token of every sequence: (y, the new states), x [n][h][p], b, c [n][g][m], st [n][h][m][p]."""
    h, g = case["heads"], case["groups"]
    dt = torch.logaddexp(a + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device=a.device))
    keep = torch.exp(-torch.exp(s["A_log"].double()) * dt)
    b, c = b.repeat(1, h // g, 1), c.repeat(1, h // g, 1)  # head h reads group h % g
    st = torch.baddbmm((st * keep[..., None, None]).flatten(0, 1), b.flatten(0, 1)[:, :, None],
                       (dt[..., None] * x).flatten(0, 1)[:, None, :]).view_as(st)
    y = torch.bmm(c.flatten(0, 1)[:, None, :], st.flatten(0, 1)).view_as(x) + s["D"].double()[:, None] * x
    return y, st


def _exact_scan(s):
    case = s["case"]
    lens = _lengths(case)
    work_of_it = max(lens) * (100e-6 + len(lens) * case["heads"] * case["head_dim"] * case["state_dim"] * 1.2e-11)
    if work_of_it > 20:
        return None
    order = sorted(range(len(lens)), key=lambda i: -lens[i])  # the longest first: the live ones are a prefix
    cu = [sum(lens[:i]) for i in order]
    x, b, c = _parts(case, s["xbc"])
    st = s["states"].double()[s["slots"].long()] * s["has"].double()[:, None, None, None]
    st = st[torch.tensor(order, device=st.device)]
    y = s["out"].double()
    base = torch.tensor(cu, device=y.device)
    for t in range(max(lens)):
        n = sum(1 for i in order if lens[i] > t)
        at = base[:n] + t
        v, st[:n] = _recur(case, x[at].double(), b[at].double(), c[at].double(), s["a"][at].double(), st[:n], s)
        if s["z"] is not None:
            z = s["z"][at].double()
            v = v * z * torch.sigmoid(z)
        y[at] = v
    states = s["states"].double()
    states[s["slots"].long()[torch.tensor(order, device=st.device)]] = st
    return {"y": y, "states": states}


def _exact_step(s):
    case, k = s["case"], s["case"]["width"]
    slots = s["slots"].long()
    hist, states = s["hist"].double(), s["states"].double()
    acc = s["bias"].double() + s["xbc"].double() * s["w"][:, k - 1].double()
    for j in range(k - 1):
        acc = acc + hist[slots, j] * s["w"][:, j].double()
    u = acc * torch.sigmoid(acc)
    x, b, c = _parts(case, u)
    y, st = _recur(case, x, b, c, s["a"].double(), states[slots], s)
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z * torch.sigmoid(z)
    states[slots] = st
    hist[slots] = torch.cat([hist[slots][:, 1:], s["xbc"].double()[:, None]], 1)
    return {"y": y, "hist": hist, "states": states}


def _exact_norm(s):
    b, r = s["b"].double(), s["r"].double()
    if s["w_post"] is not None:
        b = b / torch.sqrt(b.square().mean(-1, keepdim=True) + _EPS) * s["w_post"].double()
    if s["gate"] is not None:
        b = b * torch.sigmoid(s["gate"].double())
    r = r + _SCALE * b
    return {"residual": r, "y": r / torch.sqrt(r.square().mean(-1, keepdim=True) + _EPS) * s["w_pre"].double()}
