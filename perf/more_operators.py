"""Measured cases of what a training step in 8 bits needs next to the layer's own operators.

* quantize: e4m3 values with an fp32 scale for each block of 128, from bf16 or fp32: rows (128
  columns of one row), the transpose of the same matrix quantised along its rows' axis, and
  weights (128 x 128 tiles, both layouts).
* linear: the product of such activations with such weights, from a token to a long prompt.
* linear_train: forward and backward of a linear layer in 8 bits: y, dx and the fp32 dw.
* adamw: one AdamW step over many tensors, with states in 32 bits or in e4m3 with block scales,
  clipped by a gradient norm that is on the device.

`run` computes them in elementary torch operations where `own` is false, and through
folded_tensor_sequence_tsp_gb300 where it is true.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
BLOCK = 128
LR, BETAS, EPS, DECAY = 3e-4, (0.9, 0.95), 1e-8, 0.1
SEED = 77  # of the stochastic rounding


# --------------------------------------------------------------------------- cases

_LAYER = "16777216x4,45088768x3,4096x2"  # the weights of one 7B-shaped layer and its norms


def listed():
    return [
        # a few tokens' activations in front of a product: latency
        {"name": "quantize_few", "op": "quantize", "rows": 8, "width": 4096, "source": "bf16", "block": 1, "both": False},
        # a training step's activations: along the rows for y and dx, along the tokens for dw
        {"name": "quantize_activations", "op": "quantize", "rows": 16384, "width": 4096, "source": "bf16", "block": 1, "both": True},
        # fp32 master weights after an update, in both layouts
        {"name": "quantize_weight", "op": "quantize", "rows": 11008, "width": 4096, "source": "fp32", "block": 128, "both": True},
        # one new token each of four sequences, from the norm's 8-bit output
        {"name": "linear_token", "op": "linear", "tokens": 4, "inner": 4096, "outer": 11008, "source": "e4m3"},
        # one new token each of a batch of sequences, from bf16
        {"name": "linear_batch", "op": "linear", "tokens": 48, "inner": 11008, "outer": 4096, "source": "bf16"},
        # a prompt of no round length through odd widths
        {"name": "linear_ragged", "op": "linear", "tokens": 1999, "inner": 1000, "outer": 2815, "source": "bf16"},
        # a long prompt through a 7B-shaped layer's widest product
        {"name": "linear_prompt", "op": "linear", "tokens": 16384, "inner": 4096, "outer": 11008, "source": "e4m3"},
        # a small model's training step
        {"name": "train_small", "op": "linear_train", "tokens": 1000, "inner": 1024, "outer": 2816},
        # a 7B-shaped layer's training step
        {"name": "train_layer", "op": "linear_train", "tokens": 8192, "inner": 4096, "outer": 11008},
        # a small model's step: many tensors, most of them small, of both types
        {"name": "adamw_small", "op": "adamw", "sizes": "65536x8,176128x6,256x9,1x3,1021x2", "params": "mixed", "bits": 32},
        # one 7B-shaped layer: bf16 weights beside fp32 masters, fp32 gradients, fp32 states
        {"name": "adamw_layer", "op": "adamw", "sizes": _LAYER, "params": "master", "bits": 32},
        # the same with 8-bit states
        {"name": "adamw_layer_8bit", "op": "adamw", "sizes": _LAYER, "params": "master", "bits": 8},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_WIDTHS = [64, 256, 688, 1000, 1001, 1024, 2816, 4096, 5120]


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "linear_train", "linear_train", "adamw", "adamw"])
    if op == "quantize":
        block = rng.choice([1, 1, 128])
        return {"op": op, "rows": _log_int(rng, 1, 16384), "width": rng.choice(_WIDTHS + [_log_int(rng, 1, 8192)]),
                "source": rng.choice(["bf16", "fp32"]), "block": block, "both": rng.random() < 0.6}
    if op == "linear":
        source = rng.choice(["bf16", "e4m3"])
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "inner": rng.choice(_WIDTHS), "outer": rng.choice(_WIDTHS),
                "source": source}
    if op == "linear_train":
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "inner": rng.choice(_WIDTHS), "outer": rng.choice(_WIDTHS)}
    kinds = [(_log_int(rng, 1, 3_000_000), rng.randint(1, 10)) for _ in range(rng.randint(1, 6))]
    return {"op": op, "sizes": ",".join("%dx%d" % k for k in kinds),
            "params": rng.choice(["fp32", "bf16", "master", "mixed"]), "bits": rng.choice([8, 32])}


def _sizes(case):
    out = []
    for part in case["sizes"].split(","):
        n, count = part.split("x")
        out += [int(n)] * int(count)
    return out


def _kinds(case):
    """fp32 (fp32 weight and gradient), bf16 (both bf16) or master (bf16 weight, fp32 master and
    gradient) for every tensor."""
    kind = case["params"]
    return [("fp32", "bf16", "master")[i % 3] if kind == "mixed" else kind for i in range(len(_sizes(case)))]


def _up(n, to):
    return -(-n // to) * to


def work(case):
    if case["op"] == "adamw":
        each = {"fp32": 4 + 4 + 4, "bf16": 2 + 2 + 2, "master": 4 + 4 + 4 + 2}  # gradient in, weights in and out
        states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        n = [(k, s) for k, s in zip(_kinds(case), _sizes(case))]
        return {"bytes": sum(s * (each[k] + states) for k, s in n), "flops": 14 * sum(s for _, s in n)}
    if case["op"] == "quantize":
        r, w = case["rows"], case["width"]
        out = r * w + 4 * (r if case["block"] == 1 else -(-r // BLOCK)) * -(-w // BLOCK)
        out_t = r * w + 4 * (w if case["block"] == 1 else -(-w // BLOCK)) * -(-r // BLOCK)
        return {"bytes": r * w * (2 if case["source"] == "bf16" else 4) + out + (out_t if case["both"] else 0),
                "flops": 4 * r * w}
    m, k, n = case["tokens"], case["inner"], case["outer"]
    weight = n * k + 4 * -(-n // BLOCK) * -(-k // BLOCK)
    if case["op"] == "linear":
        x = 2 * m * k if case["source"] == "bf16" else m * k + 4 * m * -(-k // BLOCK)
        return {"bytes": x + weight + 2 * m * n, "flops": 2 * m * n * k}
    # x, dy and the weight in both layouts in; y, dx and the fp32 dw out
    return {"bytes": 4 * m * k + 4 * m * n + 2 * weight + 4 * n * k, "flops": 6 * m * n * k}


# --------------------------------------------------------------------------- inputs

def _block_scale(top):
    """The scale of a block from its largest magnitude: that over 448, never below the smallest
    normal number, 1 for a block of zeros."""
    # by a tensor: torch multiplies by the reciprocal of a plain number
    return torch.where(top > 0, (top / torch.full_like(top, E4M3_MAX)).clamp_min(2.0 ** -126), torch.ones_like(top))


def _rows8(x):
    """(e4m3 [rows, width], scales [rows, ceil(width / 128)]) of an fp32 matrix."""
    rows, w = x.shape
    g = torch.nn.functional.pad(x, (0, _up(w, BLOCK) - w)).unflatten(1, (-1, BLOCK))
    scales = _block_scale(g.abs().amax(-1))
    return (g / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :w].to(E4M3), scales


def _tiles8(x):
    """(e4m3 [rows, width], scales [ceil(rows / 128), ceil(width / 128)])."""
    rows, w = x.shape
    g = torch.nn.functional.pad(x, (0, _up(w, BLOCK) - w, 0, _up(rows, BLOCK) - rows))
    g = g.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))  # [row tiles, 128, column tiles, 128]
    scales = _block_scale(g.abs().amax((1, 3)))
    q = (g / scales[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(2).flatten(0, 1)
    return q[:rows, :w].to(E4M3), scales


def _dense16(q):
    """The e4m3 matrix in rows of a multiple of 16 bytes, as products read them."""
    rows, w = q.shape
    buf = torch.zeros(rows, _up(w, 16), dtype=torch.uint8, device=q.device)
    buf[:, :w] = q.view(torch.uint8)
    return buf.view(E4M3)[:, :w]


def _flat(sizes, dtype, step=BLOCK):
    """One buffer and its tensors: each starts on a block of its own, as a program that keeps a
    kind of state in one allocation has them."""
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _up(n, step))
    flat = torch.zeros(starts[-1], device="cuda", dtype=dtype)
    return flat, [flat[a:a + n] for a, n in zip(starts, sizes)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "adamw":
        return _prepare_adamw(case, s, normal)
    if case["op"] == "quantize":
        rows, w = case["rows"], case["width"]
        x = normal(rows, w)
        if case["block"] == 1:  # channels of an activation differ in size
            x = x * torch.exp(0.7 * normal(w))
        else:
            x = x * 0.02
        s["x"] = x if case["source"] == "fp32" else x.bfloat16()
        b = case["block"]
        new = lambda r, c: torch.zeros(r, _up(c, 16), dtype=E4M3, device="cuda")[:, :c]  # noqa: E731
        s["y"], s["scales"] = new(rows, w), torch.zeros(-(-rows // b), -(-w // BLOCK), device="cuda")
        s["yt"] = s["scales_t"] = None
        if case["both"]:
            s["yt"], s["scales_t"] = new(w, rows), torch.zeros(-(-w // b), -(-rows // BLOCK), device="cuda")
        return s
    m, k, n = case["tokens"], case["inner"], case["outer"]
    w8, ws = _tiles8(0.02 * normal(n, k))
    x = normal(m, k) * torch.exp(0.7 * normal(k))
    # the weight as quantize leaves it, in both layouts for training
    s["weight"] = (_dense16(w8), ws)
    if case["op"] == "linear_train":
        s["weight"] += (_dense16(w8.view(torch.uint8).t().contiguous().view(E4M3)), ws.t().contiguous())
        # gradients of the outputs are small, and some channels matter more than others
        s["dy"] = (1e-4 * normal(m, n) * torch.exp(0.7 * normal(n))).bfloat16()
    if case.get("source") == "e4m3":
        x8, s["x_scales"] = _rows8(x)
        s["x"] = _dense16(x8)
    else:
        s["x"] = x.bfloat16()
    return s


def _prepare_adamw(case, s, normal):
    sizes, kinds, bits = _sizes(case), _kinds(case), case["bits"]
    kind_sizes = lambda *names: [n if k in names else 0 for n, k in zip(sizes, kinds)]  # noqa: E731
    p32, s["p32"] = _flat(kind_sizes("fp32", "master"), torch.float32)
    p16, s["p16"] = _flat(kind_sizes("bf16", "master"), torch.bfloat16)
    s["out"] = {"p32": p32, "p16": p16}
    # gradients of different layers differ by orders of magnitude
    s["grads"] = []
    for i, (n, k) in enumerate(zip(sizes, kinds)):
        w, grad = 0.02 * normal(n), normal(n) * 10.0 ** (-(i % 5) - 1)
        s["p32"][i].copy_(w[:s["p32"][i].numel()])
        s["p16"][i].copy_(w[:s["p16"][i].numel()])
        s["grads"].append(grad.bfloat16() if k == "bf16" else grad)
    s["norm"] = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
    s["max_norm"] = 1.0
    # states of a run that is under way, of the clipped gradients' sizes
    clipped = min(1.0, s["max_norm"] / (float(s["norm"]) + 1e-6))
    kind = torch.float32 if bits == 32 else E4M3
    m, s["m"] = _flat(sizes, kind)
    v, s["v"] = _flat(sizes, kind)
    s["out"] |= {"m": m, "v": v}
    if bits == 8:
        ms, s["m_scales"] = _flat([-(-n // BLOCK) for n in sizes], torch.float32, 1)
        vs, s["v_scales"] = _flat([-(-n // BLOCK) for n in sizes], torch.float32, 1)
        s["out"] |= {"m_scales": ms, "v_scales": vs}
    for i, n in enumerate(sizes):
        size = clipped * 10.0 ** (-(i % 5) - 1)
        m32, v32 = 0.3 * size * normal(n), (size * (0.3 + 0.7 * normal(n).abs())).square()
        if bits == 32:
            s["m"][i].copy_(m32)
            s["v"][i].copy_(v32)
        else:
            for name, value in (("m", m32), ("v", v32)):
                q, scales = _rows8(value[None])
                s[name][i].copy_(q[0])
                s[name + "_scales"][i].copy_(scales[0])
    s["t"] = 100  # steps before this one
    if own:  # the optimizer that a program makes once and keeps, here resumed with its states
        import folded_tensor_sequence_tsp_gb300 as tsp
        masters = [a if k == "master" else None for a, k in zip(s["p32"], kinds)]
        params = [a if k == "fp32" else b for a, b, k in zip(s["p32"], s["p16"], kinds)]
        s["optimizer"] = tsp.TSPAdamW(params, masters=masters, betas=BETAS, eps=EPS, weight_decay=DECAY,
                                      state_bits=bits, seed=SEED)
        s["optimizer"].resume(s["t"], s["m"], s["v"], s.get("m_scales"), s.get("v_scales"))
    return s


# --------------------------------------------------------------------------- plain forms

def _wide(q, scales, block):
    """The fp32 values that an e4m3 matrix with its block scales stands for."""
    rows, w = q.shape
    s = scales.repeat_interleave(BLOCK, 1)[:, :w]
    if block == BLOCK:
        s = s.repeat_interleave(BLOCK, 0)[:rows]
    return q.float() * s


def _plain_quantize(s):
    x, make = s["x"].float(), _rows8 if s["case"]["block"] == 1 else _tiles8
    y, scales = make(x)
    out = {"y": y, "scales": scales}
    if s["case"]["both"]:
        out["yt"], out["scales_t"] = make(x.t())
    return out


def _plain_linear(s):
    x = _wide(s["x"], s["x_scales"], 1) if s["case"]["source"] == "e4m3" else _wide(*_rows8(s["x"].float()), 1)
    return (x @ _wide(*s["weight"], BLOCK).t()).bfloat16()


def _plain_linear_train(s):
    x, dy, w = s["x"].float(), s["dy"].float(), _wide(*s["weight"][:2], BLOCK)
    y = _wide(*_rows8(x), 1) @ w.t()
    dx = _wide(*_rows8(dy), 1) @ w
    dw = _wide(*_rows8(dy.t()), 1) @ _wide(*_rows8(x.t()), 1).t()
    return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw}


_LOW = 0xFFFFFFFF


def _mix(x):
    """32 scrambled bits of a 32-bit number (held in 64)."""
    x = ((x ^ (x >> 16)) * 0x7A35E9B5) & _LOW
    x = ((x ^ (x >> 15)) * 0x68E31DA5) & _LOW
    return x ^ (x >> 16)


def _random(n, t, tensor, stream):
    """32 random bits for each of a tensor's n elements: a function of the seed, the step, the
    tensor's place in the list, the element and the stream (0 the states, 1 a bf16 weight)."""
    key = _mix(_mix(_mix((SEED + t) & _LOW) + tensor & _LOW) + stream & _LOW)
    return _mix(torch.arange(n, device="cuda") ^ key)


def _stochastic8(q, r16):
    """|q| <= 448 rounded to a neighbouring e4m3 value, up with the probability of its distance
    from the lower one; r16: 16 random bits for each."""
    a = q.abs()
    normal = ((a.view(torch.int32) + (r16 << 4)) & ~0xFFFFF).view(torch.float32)
    small = torch.floor(a * 512 + r16.float() / 65536) / 512
    return torch.where(a >= 2.0 ** -6, normal, small).clamp_max(E4M3_MAX).copysign(q)


def _states8(x, r16, keep):
    """Codes and scales of a state, in blocks of 128. keep: what is not zero stays so."""
    n = x.numel()
    g = torch.nn.functional.pad(x, (0, _up(n, BLOCK) - n)).unflatten(0, (-1, BLOCK))
    r = torch.nn.functional.pad(r16, (0, _up(n, BLOCK) - n)).unflatten(0, (-1, BLOCK))
    scales = _block_scale(g.abs().amax(-1))
    q = _stochastic8((g * (1.0 / scales)[:, None]).clamp(-E4M3_MAX, E4M3_MAX), r)
    if keep:
        q = torch.where(g > 0, q.clamp_min(2.0 ** -9), q)
    return q.flatten()[:n].to(E4M3), scales


def _plain_adamw(s):
    s["t"] += 1
    t, bits, (b1, b2) = s["t"], s["case"]["bits"], BETAS
    rate, root = LR / (1 - b1 ** t), 1 / math.sqrt(1 - b2 ** t)
    factor = torch.clamp(s["max_norm"] / (s["norm"] + 1e-6), max=1.0)
    for i, kind in enumerate(_kinds(s["case"])):
        g = s["grads"][i].float() * factor
        n = g.numel()
        m, v = s["m"][i].float(), s["v"][i].float()
        if bits == 8:
            m = m * s["m_scales"][i].repeat_interleave(BLOCK)[:n]
            v = v * s["v_scales"][i].repeat_interleave(BLOCK)[:n]
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * (g * g)
        p = s["p16"][i].float() if kind == "bf16" else s["p32"][i]
        p = p - (LR * DECAY * p + rate * m / (v.sqrt() * root + EPS))
        if kind == "bf16":
            r = _random(n, t, i, 1).to(torch.int32) & 0xFFFF
            s["p16"][i].copy_(((p.view(torch.int32) + r) & ~0xFFFF).view(torch.float32))
        else:
            s["p32"][i].copy_(p)
        if kind == "master":
            s["p16"][i].copy_(p)
        if bits == 8:
            r = _random(n, t, i, 0)
            q, scales = _states8(m, (r & 0xFFFF).to(torch.int32), False)
            s["m"][i].copy_(q)
            s["m_scales"][i].copy_(scales)
            m = q
            v, scales = _states8(v, (r >> 16).to(torch.int32), True)
            s["v_scales"][i].copy_(scales)
        s["m"][i].copy_(m)
        s["v"][i].copy_(v)
    return s["out"]


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
    if case["op"] == "quantize":
        tsp.tsp_quantize_e4m3(s["x"], s["y"], s["scales"], s["yt"], s["scales_t"], block=case["block"])
        return {k: s[k] for k in ("y", "scales", "yt", "scales_t") if s[k] is not None}
    if case["op"] == "adamw":
        s["optimizer"].step(s["grads"], LR, norm=s["norm"], max_norm=s["max_norm"])
        return s["out"]
    sizes = (case["tokens"], case["outer"], case["inner"])
    op = _handle(sizes, lambda: tsp.TSPLinearE4M3(*sizes))
    if case["op"] == "linear":
        return op.forward(s["x"], s["weight"], scales=s.get("x_scales"))
    y, saved = op.forward_train(s["x"], s["weight"])
    dx, dw = op.backward(saved, s["dy"], s["weight"])
    return {"y": y, "dx": dx, "dw": dw}


def run(state):
    if own:
        return _own(state)
    return {"quantize": _plain_quantize, "linear": _plain_linear, "linear_train": _plain_linear_train,
            "adamw": _plain_adamw}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- 64 bits

def _exact_codes(x, tile):
    """The definition: fp32 scales, quotients by them rounded to fp32 and then to e4m3, each step
    rounded once from its exact value (a quotient in 64 bits is off by far less than what an
    fp32 rounding could notice)."""
    x = x.double()
    rows, w = x.shape
    tops = torch.stack([part.abs().amax(1) for part in torch.split(x, BLOCK, dim=1)], 1)
    if tile:
        tops = torch.stack([part.amax(0) for part in torch.split(tops, BLOCK, dim=0)], 0)
    scales = torch.where(tops > 0, torch.clamp((tops / 448).float(), min=2.0 ** -126), torch.ones((), device="cuda"))
    wide = torch.repeat_interleave(scales.double(), BLOCK, dim=1)[:, :w]
    if tile:
        wide = torch.repeat_interleave(wide, BLOCK, dim=0)[:rows]
    codes = torch.clamp((x / wide).float(), -448, 448).to(E4M3)
    return codes, scales, codes.double() * wide


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    if case["op"] == "quantize":
        tile = case["block"] == BLOCK
        y, scales, _ = _exact_codes(s["x"], tile)
        out = {"y": y.double(), "scales": scales.double()}
        if case["both"]:
            yt, scales_t, _ = _exact_codes(s["x"].t(), tile)
            out |= {"yt": yt.double(), "scales_t": scales_t.double()}
        return out
    w8, ws = s["weight"][:2]
    w = w8.double() * torch.kron(ws.double(), torch.ones(BLOCK, BLOCK, dtype=torch.float64, device="cuda"))[:w8.shape[0], :w8.shape[1]]
    if case["op"] == "linear":
        x = s["x"]
        if case["source"] == "e4m3":
            x = x.double() * torch.repeat_interleave(s["x_scales"].double(), BLOCK, dim=1)[:, :x.shape[1]]
        else:
            x = _exact_codes(x, False)[2]
        return torch.einsum("mk,nk->mn", x, w)
    x, dy = s["x"], s["dy"]
    return {"y": torch.einsum("mk,nk->mn", _exact_codes(x, False)[2], w),
            "dx": torch.einsum("mn,nk->mk", _exact_codes(dy, False)[2], w),
            "dw": torch.einsum("nm,km->nk", _exact_codes(dy.t(), False)[2], _exact_codes(x.t(), False)[2])}


def _exact_adamw(case, s):
    """The weights and, with 32 bits, the states from the update rule in 64 bits. With 8 bits the
    scales, and the states as quotients by them (their rounding is by random numbers); a bf16 weight
    without a master before its rounding."""
    t, (b1, b2) = s["t"] + 1, BETAS
    factor = min(1.0, s["max_norm"] / (float(s["norm"]) + 1e-6))
    out = {name: torch.zeros(x.shape, dtype=torch.float64, device="cuda") for name, x in s["out"].items()}

    def place(name, i, value):
        like, flat = s[name][i], s["out"][name]
        start = (like.data_ptr() - flat.data_ptr()) // flat.element_size()
        out[name][start:start + like.numel()] = value

    for i, kind in enumerate(_kinds(case)):
        g = s["grads"][i].double() * factor
        m, v = s["m"][i].double(), s["v"][i].double()
        if case["bits"] == 8:
            m = m * torch.repeat_interleave(s["m_scales"][i].double(), BLOCK)[:m.numel()]
            v = v * torch.repeat_interleave(s["v_scales"][i].double(), BLOCK)[:v.numel()]
        m, v = torch.lerp(g, m, b1), torch.lerp(g.square(), v, b2)
        p = (s["p16"] if kind == "bf16" else s["p32"])[i].double()
        p = p * (1 - LR * DECAY) - LR * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + EPS)
        if kind != "bf16":
            place("p32", i, p)
        if kind != "fp32":
            place("p16", i, p)
        for name, x in (("m", m), ("v", v)):
            if case["bits"] == 8:
                tops = torch.stack([part.abs().max() for part in torch.split(x, BLOCK)]) if x.numel() < 100_000 else \
                    torch.nn.functional.pad(x.abs(), (0, -x.numel() % BLOCK)).view(-1, BLOCK).max(1).values
                scales = torch.where(tops > 0, tops / 448, 1.0)
                place(name + "_scales", i, scales)
                x = x / torch.repeat_interleave(scales, BLOCK)[:x.numel()]
            place(name, i, x)
    return out
