"""Measured cases of the operators that a training or prompt step needs around a TSP layer.

* attention: causal attention over a packed batch (sequences of different lengths, back to back
  on one token axis), with grouped query heads: prompts (forward only) and training (forward and
  backward).
* norm: the residual's addition and a root-mean-square norm in one pass, with a bf16 output, an
  8-bit (e4m3) output with scales, and its backward.
* clip: the global norm of many gradient tensors, and their scaling to a largest norm.

`run` computes them in elementary torch operations where `own` is false, and through
folded_tensor_sequence_tsp_gb300 where it is true.
"""
import math
import random

import torch

own = False

LOG2E = 1.4426950408889634
E4M3_MAX = 448.0
EPS = 1e-5


# --------------------------------------------------------------------------- cases

def _ragged(rng, total, longest):
    """Lengths of a packed batch, spread over their logarithm, of `total` tokens in all."""
    out, left = [], total
    while left:
        n = min(left, max(1, int(round(math.exp(rng.uniform(0.0, math.log(longest)))))))
        out.append(n)
        left -= n
    return ",".join(str(n) for n in out)


def listed():
    r = random.Random(2024)
    return [
        # a handful of short prompts answered at once: latency, one to three tiles each
        {"name": "prompt_short", "op": "attention", "train": False, "heads": 16, "kv_heads": 4, "dim": 64,
         "lengths": "1,5,64,130,17", "pad": 7},
        # an ordinary packed batch of prompts, each of its own length
        {"name": "prompt_packed", "op": "attention", "train": False, "heads": 32, "kv_heads": 8, "dim": 128,
         "lengths": _ragged(r, 16384, 6000), "pad": 0},
        # one long document beside two short ones
        {"name": "prompt_long", "op": "attention", "train": False, "heads": 32, "kv_heads": 8, "dim": 128,
         "lengths": "32768,1,999", "pad": 0},
        # a small model's training step: as many key as query heads
        {"name": "train_short", "op": "attention", "train": True, "heads": 16, "kv_heads": 16, "dim": 64,
         "lengths": "300,1,129,570", "pad": 24},
        # an ordinary packed training batch with grouped heads
        {"name": "train_packed", "op": "attention", "train": True, "heads": 32, "kv_heads": 8, "dim": 128,
         "lengths": _ragged(r, 8192, 4000), "pad": 0},
        # long-context training: one sequence fills the batch but for its padding
        {"name": "train_long", "op": "attention", "train": True, "heads": 32, "kv_heads": 4, "dim": 128,
         "lengths": "16381", "pad": 3},
        # a few tokens through a small model's norm
        {"name": "norm_few", "op": "norm", "rows": 8, "width": 1024, "residual": "bf16", "out": "bf16", "group": 0},
        # a long sequence with the residual stream kept in fp32, as the layer keeps h
        {"name": "norm_fp32_stream", "op": "norm", "rows": 16384, "width": 4096, "residual": "fp32", "out": "bf16", "group": 0},
        # the same with an 8-bit output in blocks of 128 columns, for products in 8 bits
        {"name": "norm_e4m3", "op": "norm", "rows": 16384, "width": 4096, "residual": "bf16", "out": "e4m3", "group": 128},
        # the backward of the norm between two blocks of a training step
        {"name": "norm_backward", "op": "norm_backward", "rows": 16384, "width": 4096, "residual": "bf16"},
        # a small model's gradients: many tensors, most of them small
        {"name": "clip_small", "op": "clip", "sizes": "65536x8,176128x6,256x9,1x3,1021x2", "dtype": "mixed", "max_norm": 1.0},
        # the fp32 weight gradients of one 7B-shaped layer
        {"name": "clip_layer", "op": "clip", "sizes": "16777216x4,45088768x3,4096x2", "dtype": "fp32", "max_norm": 1.0},
    ]


_HEADS = [(4, 4, 64), (4, 2, 64), (16, 4, 64), (16, 16, 64), (6, 2, 64), (14, 2, 64), (5, 1, 64),
          (8, 1, 128), (12, 4, 128), (16, 16, 128), (32, 8, 128), (32, 4, 128)]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "norm", "norm", "norm_backward", "clip"])
    if op == "attention":
        heads, kv, dim = rng.choice(_HEADS)
        train = rng.random() < 0.5
        total = _log_int(rng, 16, 12000)
        longest = _log_int(rng, 2, total)
        return {"op": op, "train": train, "heads": heads, "kv_heads": kv, "dim": dim,
                "lengths": _ragged(rng, total, longest) + rng.choice(["", ",0", ",1"]), "pad": rng.choice([0, 0, 1, 50])}
    if op == "norm":
        out = rng.choice(["bf16", "e4m3"])
        return {"op": op, "rows": _log_int(rng, 1, 16384), "width": rng.choice([256, 1000, 1001, 1024, 2048, 4096, 4095, 5120]),
                "residual": rng.choice(["none", "bf16", "fp32"]), "out": out,
                "group": rng.choice([0, 128]) if out == "e4m3" else 0}
    if op == "norm_backward":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "width": rng.choice([256, 1000, 1001, 1024, 2048, 4096, 4095, 5120]),
                "residual": rng.choice(["none", "bf16", "fp32"])}
    kinds = [(_log_int(rng, 1, 3_000_000), rng.randint(1, 10)) for _ in range(rng.randint(1, 6))]
    return {"op": op, "sizes": ",".join("%dx%d" % k for k in kinds), "dtype": rng.choice(["fp32", "bf16", "mixed"]),
            "max_norm": rng.choice([0.5, 1.0, 1e9])}


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def _sizes(case):
    out = []
    for part in case["sizes"].split(","):
        n, count = part.split("x")
        out += [int(n)] * int(count)
    return out


def _dtypes(case):
    kind = case["dtype"]
    return [torch.bfloat16 if kind == "bf16" or (kind == "mixed" and i % 2) else torch.float32
            for i in range(len(_sizes(case)))]


def work(case):
    if case["op"] == "attention":
        L, h, kv, d = _lengths(case), case["heads"], case["kv_heads"], case["dim"]
        n = sum(L)
        product = d * h * sum(x * (x + 1) for x in L)  # 2 d per visible pair, of which there are L (L + 1) / 2
        qo, kvb, lse = 2 * n * h * d, 2 * n * kv * d, 4 * n * h
        if not case["train"]:
            return {"bytes": 2 * qo + 2 * kvb, "flops": 2 * product}
        # forward: two products; backward: five. q, k, v, dout in; o, lse, dq, dk, dv out
        return {"bytes": 2 * qo + 2 * kvb + 2 * qo + 2 * kvb + lse, "flops": 7 * product}
    if case["op"] == "clip":
        b = sum(n * t.itemsize for n, t in zip(_sizes(case), _dtypes(case)))
        return {"bytes": 2 * b, "flops": 3 * sum(_sizes(case))}
    rows, w = case["rows"], case["width"]
    stream = {"none": 0, "bf16": 2, "fp32": 4}[case["residual"]]
    if case["op"] == "norm":
        groups = -(-w // case["group"]) if case["group"] else 1
        y = 2 * w if case["out"] == "bf16" else w + 4 * groups
        return {"bytes": rows * (2 * w + 2 * stream * w + y) + 2 * w, "flops": 5 * rows * w}
    # h, dy and the stream's gradient in, dx out; the weight and its fp32 gradient
    hb = stream or 2
    return {"bytes": rows * w * (hb + 2 + stream + (stream or 2)) + 6 * w, "flops": 10 * rows * w}


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "attention":
        L, h, kv, d = _lengths(case), case["heads"], case["kv_heads"], case["dim"]
        starts = [0]
        for n in L:
            starts.append(starts[-1] + n)
        rows = starts[-1] + case["pad"]
        # q, k and v as a fused projection leaves them: column ranges of one buffer
        qkv = normal(rows, (h + 2 * kv) * d).bfloat16()
        s["q"] = qkv[:, :h * d].unflatten(1, (h, d))
        s["k"] = qkv[:, h * d:(h + kv) * d].unflatten(1, (kv, d))
        s["v"] = qkv[:, (h + kv) * d:].unflatten(1, (kv, d))
        s["starts_host"] = starts
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        # rows behind the last sequence belong to the caller: zeros here, and they stay so
        s["o"] = torch.zeros(rows, h, d, dtype=torch.bfloat16, device="cuda")
        if case["train"]:
            s["do"] = normal(rows, h, d).bfloat16()
            s["lse"] = torch.zeros(h, rows, device="cuda")
            for name, n in (("dq", h), ("dk", kv), ("dv", kv)):
                s[name] = torch.zeros(rows, n, d, dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "clip":
        sizes, types = _sizes(case), _dtypes(case)
        # gradients of different layers differ by orders of magnitude
        s["grads"] = [(normal(n) * 10.0 ** (-(i % 5))).to(t) for i, (n, t) in enumerate(zip(sizes, types))]
        s["outs"] = [torch.empty_like(x) for x in s["grads"]]
        return s
    rows, w = case["rows"], case["width"]
    wide = torch.exp(0.7 * normal(w))  # channels of a residual stream differ in size
    kind = {"none": None, "bf16": torch.bfloat16, "fp32": torch.float32}[case["residual"]]
    s["w"] = (1 + 0.2 * normal(w)).bfloat16()
    if case["op"] == "norm":
        s["x"] = (normal(rows, w) * wide).bfloat16()
        s["r"] = None if kind is None else (3 * normal(rows, w) * wide).to(kind)
    else:
        s["h"] = (3 * normal(rows, w) * wide).to(kind or torch.bfloat16)
        s["dy"] = normal(rows, w).bfloat16()
        s["dh"] = None if kind is None else normal(rows, w).to(kind)
    return s


# --------------------------------------------------------------------------- plain forms

CHUNK = 1024  # query rows whose scores are held at a time


def _plain_attention(s):
    """softmax(q k^T / sqrt(d)) v over the keys of the same sequence up to the query's own."""
    case, starts = s["case"], s["starts_host"]
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    G, n = h // kv, starts[-1]
    scale = 1.0 / math.sqrt(d)
    pos = torch.arange(n, device="cuda")
    seq_start = s["starts"].long()[torch.searchsorted(s["starts"].long(), pos, right=True) - 1]
    # [kv heads][tokens][...]
    k = s["k"][:n].float().transpose(0, 1)
    v = s["v"][:n].float().transpose(0, 1)
    q = s["q"][:n].float().unflatten(1, (kv, G)).permute(1, 2, 0, 3)  # [kv][G][tokens][d]
    if case["train"]:
        do = s["do"][:n].float().unflatten(1, (kv, G)).permute(1, 2, 0, 3)
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for r0 in range(0, n, CHUNK):
        r1 = min(n, r0 + CHUNK)
        k0 = max(x for x in starts if x <= r0)  # the first key that these rows see
        kc, vc = k[:, None, k0:r1], v[:, None, k0:r1]
        sc = (q[:, :, r0:r1] @ kc.transpose(-1, -2)) * scale
        keys, rows = pos[k0:r1][None, :], pos[r0:r1][:, None]
        sc = sc.masked_fill((keys > rows) | (keys < seq_start[r0:r1][:, None]), -math.inf)
        m = sc.amax(-1, keepdim=True)
        p = torch.exp(sc - m)
        l = p.sum(-1, keepdim=True)
        p = p / l
        o = p @ vc
        s["o"][r0:r1] = o.permute(2, 0, 1, 3).flatten(1, 2).bfloat16()
        if case["train"]:
            s["lse"][:, r0:r1] = ((m + torch.log(l)) * LOG2E).flatten(0, 1)[..., 0]
            g = do[:, :, r0:r1]
            dv[:, k0:r1] += (p.transpose(-1, -2) @ g).sum(1)
            ds = p * (g @ vc.transpose(-1, -2) - (g * o).sum(-1, keepdim=True))
            s["dq"][r0:r1] = ((ds @ kc) * scale).permute(2, 0, 1, 3).flatten(1, 2).bfloat16()
            dk[:, k0:r1] += (ds.transpose(-1, -2) @ q[:, :, r0:r1]).sum(1) * scale
    if not case["train"]:
        return s["o"]
    s["dk"][:n] = dk.transpose(0, 1).bfloat16()
    s["dv"][:n] = dv.transpose(0, 1).bfloat16()
    return {"o": s["o"], "lse": s["lse"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _plain_norm(s):
    case = s["case"]
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
    out = {} if s["r"] is None else {"h": h.to(s["r"].dtype)}
    if case["out"] == "bf16":
        out["y"] = y.bfloat16()
        return out
    rows, w = y.shape
    group = case["group"] or w
    groups = -(-w // group)
    padded = torch.nn.functional.pad(y, (0, groups * group - w)).unflatten(1, (groups, group))
    top = padded.abs().amax(-1)
    scales = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    q = (padded / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :w]
    out["y"] = q.to(torch.float8_e4m3fn)
    out["scales"] = scales
    return out


def _plain_norm_backward(s):
    h, w = s["h"].float(), s["w"].float()
    dy = s["dy"].float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    xhat = h * rstd
    g = dy * w
    dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    kind = torch.bfloat16
    if s["dh"] is not None:
        dx, kind = dx + s["dh"].float(), s["dh"].dtype
    return {"dx": dx.to(kind), "dw": (dy * xhat).sum(0)}


def _plain_clip(s):
    total = torch.stack([x.float().square().sum() for x in s["grads"]]).sum()
    norm = total.sqrt()
    factor = torch.clamp(s["case"]["max_norm"] / (norm + 1e-6), max=1.0)
    for x, y in zip(s["grads"], s["outs"]):
        y.copy_((x.float() * factor).to(y.dtype))
    return {"norm": norm, "outs": s["outs"]}


# --------------------------------------------------------------------------- the framework's operators

_handles = {}


def _handle(key, make):
    """The operator object that a program makes once for its shapes and keeps."""
    if key not in _handles:
        _handles[key] = make()
    return _handles[key]


def _own(s):
    import folded_tensor_sequence_tsp_gb300 as tsp
    case = s["case"]
    if case["op"] == "attention":
        rows, seqs = s["q"].shape[0], s["starts"].numel() - 1
        key = ("attention", rows, seqs, case["heads"], case["kv_heads"], case["dim"])
        op = _handle(key, lambda: tsp.TSPPackedAttention(*key[1:]))
        if not case["train"]:
            return op.forward(s["q"], s["k"], s["v"], s["starts"], out=s["o"])
        o, lse = op.forward_train(s["q"], s["k"], s["v"], s["starts"], out=s["o"], lse=s["lse"])
        dq, dk, dv = op.backward(s["q"], s["k"], s["v"], s["starts"], o, lse, s["do"], dq=s["dq"], dk=s["dk"], dv=s["dv"])
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if case["op"] == "clip":
        op = _handle(("clip", len(s["grads"])), lambda: tsp.TSPGradClip(len(s["grads"])))
        return {"norm": op.clip(s["grads"], case["max_norm"], outs=s["outs"]), "outs": s["outs"]}
    op = _handle(("norm", case["rows"], case["width"]), lambda: tsp.TSPRMSNorm(case["rows"], case["width"], eps=EPS))
    if case["op"] == "norm_backward":
        dx, dw = op.backward(s["h"], s["w"], s["dy"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if case["out"] == "bf16":
        y, h = op.forward(s["x"], s["w"], residual=s["r"])
        return {"y": y} if h is None else {"y": y, "h": h}
    y, scales, h = op.forward_e4m3(s["x"], s["w"], residual=s["r"], group=case["group"])
    out = {"y": y, "scales": scales}
    return out if h is None else {**out, "h": h}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "attention":
        return _plain_attention(state)
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_backward":
        return _plain_norm_backward(state)
    return _plain_clip(state)


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    if case["op"] == "clip":
        if sum(_sizes(case)) > 50_000_000:
            return None
        flat = torch.cat([x.double().reshape(-1) for x in s["grads"]])
        norm = torch.linalg.vector_norm(flat)
        factor = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm, "outs": [x.double() * factor for x in s["grads"]]}
    if case["op"] == "norm":
        h = s["x"].double() if s["r"] is None else torch.add(s["x"].double(), s["r"].double())
        y = h / torch.sqrt(torch.linalg.vecdot(h, h) / case["width"] + EPS).unsqueeze(-1) * s["w"].double()
        out = {} if s["r"] is None else {"h": h}
        if case["out"] == "bf16":
            return {**out, "y": y}
        group = case["group"] or case["width"]
        tops = torch.stack([part.abs().max(dim=1).values for part in torch.split(y, group, dim=1)], dim=1)
        scales = torch.where(tops > 0, tops / E4M3_MAX, 1.0)
        wide = torch.repeat_interleave(scales, group, dim=1)[:, :case["width"]]
        return {**out, "y": y / wide, "scales": scales}
    # the backward, by differentiating the definition
    h = s["h"].double().requires_grad_()
    w = s["w"].double().requires_grad_()
    y = h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + EPS) * w
    dx, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
    return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dw": dw}


def _exact_attention(case, s):
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    G, L = h // kv, _lengths(case)
    if 4 * d * h * sum(x * x for x in L) * (4 if case["train"] else 1) > 4e12:
        return None
    rows = s["q"].shape[0]
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = new(rows, h, d), new(h, rows)
    dq, dk, dv = new(rows, h, d), new(rows, kv, d), new(rows, kv, d)
    for start, n in zip(s["starts_host"], L):
        at = slice(start, start + n)
        hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for j in range(kv if n else 0):
            mine = slice(j * G, (j + 1) * G)
            q = s["q"][at, mine].double().requires_grad_(case["train"])
            k = s["k"][at, j].double().requires_grad_(case["train"])
            v = s["v"][at, j].double().requires_grad_(case["train"])
            logits = torch.einsum("igd,jd->gij", q, k) / math.sqrt(d)
            logits = logits.masked_fill(hidden, -math.inf)
            out = torch.einsum("gij,jd->igd", torch.softmax(logits, dim=-1), v)
            o[at, mine] = out.detach()
            if case["train"]:
                lse[mine, at] = torch.logsumexp(logits.detach(), dim=-1) / math.log(2.0)
                a, b, c = torch.autograd.grad(out, (q, k, v), s["do"][at, mine].double())
                dq[at, mine], dk[at, j], dv[at, j] = a, b, c
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if case["train"] else o
