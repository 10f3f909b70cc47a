"""Cases for timing the operators of a MoE block that surround its routed experts:

  norm_pre, norm_pre_backward     the norm that makes the block's input from the residual stream
  norm_post, norm_post_backward   the block's output: norm, sigmoid gate, residual and branch scale, and the next
                                  block's norm in the same pass
  balance                         per-expert counts and the router's balance loss, and the loss's gradient
  q4                              4-bit matrix-vector products with group scales, alone or as a SwiGLU pair

With `own` false, run() computes them from elementary torch operations in 32 bits, rounded once at the end; with
`own` true it calls vector_quantized_moe_b200.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _norm_pre(name, T, H, h="bf16", w="bf16", offset=0.0, pad=0, back=False):
    return {"name": name, "op": "norm_pre_backward" if back else "norm_pre", "T": T, "H": H, "h": h, "w": w,
            "offset": offset, "pad": pad}


def _norm_post(name, T, H, h="bf16", y="f32", w="bf16", gate="none", post=True, following=True, res_scale=1.0,
               out_scale=1.0, offset=0.0, pad=0, back=False):
    return {"name": name, "op": "norm_post_backward" if back else "norm_post", "T": T, "H": H, "h": h, "y": y, "w": w,
            "gate": gate, "post": post, "following": following, "res_scale": res_scale, "out_scale": out_scale,
            "offset": offset, "pad": pad}


def _balance(name, T, E, k, padding=0.0):
    return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "padding": padding}


def _q4(name, T, rows, cols, group, biased=False, pair=False, y="bf16"):
    return {"name": name, "op": "q4", "T": T, "rows": rows, "cols": cols, "group": group, "biased": biased,
            "pair": pair, "y": y}


def listed():
    return [
        # one token of a decode step enters a block of hidden size 4096
        _norm_pre("pre_T1_h4096", 1, 4096),
        # training: the gradient of that norm over a batch of 4096 tokens, hidden 6144
        _norm_pre("pre_backward_T4096_h6144", 4096, 6144, back=True),
        # 16 decoded tokens leave a block: fp32 output of the experts, a gate logit a token, the next block's norm
        _norm_post("post_T16_h6144_token_gate", 16, 6144, gate="token"),
        # a prompt of 4096 tokens: scaled residual, no gate, weights stored as w - 1
        _norm_post("post_T4096_h4096_scaled", 4096, 4096, y="bf16", res_scale=1.25, out_scale=0.5, offset=1.0),
        # training: the gradient of the block's output, an odd number of tokens, a gate for each channel
        _norm_post("post_backward_T2047_h4096_channel_gate", 2047, 4096, gate="channel", back=True),
        # the router's statistics over one small batch of 512 experts, 10 a token
        _balance("balance_T16_e512_k10", 16, 512, 10),
        # a training batch with an eighth of padding, 256 experts, 8 a token
        _balance("balance_T4096_e256_k8_padded", 4096, 256, 8, padding=0.125),
        # a large global batch on one GPU
        _balance("balance_T32768_e512_k10", 32768, 512, 10),
        # one token through a small projection
        _q4("q4_T1_512x1024_g64", 1, 512, 1024, 64),
        # one token through a square projection of hidden 6144, affine groups of 64 with offsets
        _q4("q4_T1_6144x6144_g64_biased", 1, 6144, 6144, 64, biased=True),
        # a shared expert's gate and up for 16 tokens, ragged row count, groups of 32
        _q4("q4_pair_T16_2040x6144_g32", 16, 2040, 6144, 32, pair=True),
        # 8 tokens through an output head
        _q4("q4_T8_131072x4096_g128", 8, 131072, 4096, 128, y="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_pre", "norm_pre_backward", "norm_post", "norm_post_backward", "balance", "q4", "q4"])
    if op.startswith("norm"):
        H = _log(rng, 64, 8192)
        H = H if rng.random() < 0.3 else max(64, H // 8 * 8)
        T = _log(rng, 1, max(1, min(4096, 4096 * 4096 // H)))
        c = {"op": op, "T": T, "H": H, "h": rng.choice(["bf16", "bf16", "f32"]), "w": rng.choice(["bf16", "f32"]),
             "offset": rng.choice([0.0, 1.0]), "pad": rng.choice([0, 0, 5, 64])}
        if op.startswith("norm_post"):
            c.update(y=rng.choice(["f32", "bf16"]), gate=rng.choice(["none", "token", "channel"]),
                     post=rng.random() < 0.75, following=rng.random() < 0.75,
                     res_scale=rng.choice([1.0, 1.0, 0.75]), out_scale=rng.choice([1.0, 1.0, 0.5]))
        return c
    if op == "balance":
        E = _log(rng, 8, 1024)
        return {"op": op, "T": _log(rng, 1, min(32768, 32768 * 512 // E)), "E": E, "k": rng.randint(1, min(E, 10)),
                "padding": rng.choice([0.0, 0.0, 0.25])}
    group = rng.choice([32, 64, 128])
    cols = max(group, _log(rng, 128, 16384) // group * group)
    rows = _log(rng, 16, min(131072, 65536 * 4096 // cols))
    return {"op": op, "T": _log(rng, 1, 32 if rows * cols <= 1 << 26 else 8), "rows": rows, "cols": cols, "group": group,
            "biased": rng.random() < 0.5, "pair": rows * cols <= 1 << 26 and rng.random() < 0.4,
            "y": rng.choice(["bf16", "f32"])}


# ---------------------------------------------------------------- inputs

def _rows(T, H, dtype, g, pad, scale=1.0):
    """A [T, H] array, a window of a wider one where pad > 0."""
    return (torch.randn((T, H + pad), generator=g, device="cuda") * scale).to(dtype)[:, :H]


def _weight(c, g):
    w = 1.0 - c["offset"] + 0.2 * torch.randn(c["H"], generator=g, device="cuda")
    return w.to(TYPES[c["w"]])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    if op.startswith("norm"):
        T, H, pad, ht = c["T"], c["H"], c["pad"], TYPES[c["h"]]
        # a residual stream: unit rows with a few large channels
        chan = 1.0 + 15.0 * (torch.rand(H, generator=g, device="cuda") < 0.01)
        s["h"] = (torch.randn((T, H + pad), generator=g, device="cuda")[:, :H] * chan).to(ht)
        if pad:
            wide = torch.zeros((T, H + pad), dtype=ht, device="cuda")
            wide[:, :H] = s["h"]
            s["h"] = wide[:, :H]
        if op.startswith("norm_pre"):
            s["w"] = _weight(c, g)
            if op.endswith("backward"):
                s["dx"] = _rows(T, H, BF16, g, pad)
                s["dres"] = _rows(T, H, ht, g, pad)
        else:
            s["y"] = _rows(T, H, TYPES[c["y"]], g, pad, 0.3)
            s["gate"] = None
            if c["gate"] != "none":
                s["gate"] = _rows(T, 1 if c["gate"] == "token" else H, BF16, g, 0, 1.5)
            s["post"] = _weight(c, g) if c["post"] else None
            s["next"] = _weight(c, g) if c["following"] else None
            if op.endswith("backward"):
                s["dh"] = _rows(T, H, ht, g, pad)
                s["dx"] = _rows(T, H, BF16, g, pad) if c["following"] else None
    elif op == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        # router logits with popular and unpopular experts
        s["logits"] = (torch.randn((T, E), generator=g, device="cuda")
                       + 0.7 * torch.randn(E, generator=g, device="cuda"))
        s["ids"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
        s["mask"] = None
        if c["padding"]:
            s["mask"] = torch.rand(T, generator=g, device="cuda") >= c["padding"]
        s["dloss"] = torch.rand((), generator=g, device="cuda") + 0.5
        s["coef"] = 0.01
    else:
        s["x"] = _rows(c["T"], c["cols"], BF16, g, 0)
        s["m"] = [_q4_weights(c, g) for _ in range(2 if c["pair"] else 1)]
    if own:
        import vector_quantized_moe_b200 as vq
        s["vq"] = vq
        if op.startswith("norm_pre"):
            s["norm"] = vq.Norm(s["w"], EPS, c["offset"])
        elif op.startswith("norm_post"):
            s["norms"] = [None if w is None else vq.Norm(w, EPS, c["offset"]) for w in (s["post"], s["next"])]
        elif op == "q4":
            s["m"] = [vq.Q4Module.from_rows(*m, group=c["group"]) for m in s["m"]]
    return s


def _q4_weights(c, g):
    """Codes as 32-bit words [rows, cols / 8] (the lowest 4 bits first), fp16 scales, and fp16 offsets or None."""
    rows, cols, n = c["rows"], c["cols"], c["cols"] // c["group"]
    words = torch.randint(-2**31, 2**31, (rows, cols // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    scales = ((0.5 + 1.5 * torch.rand((rows, n), generator=g, device="cuda")) / (6.0 * math.sqrt(cols))).to(torch.float16)
    biases = None
    if c["biased"]:
        biases = (-scales.float() * (7.5 + torch.randn((rows, n), generator=g, device="cuda"))).to(torch.float16)
    return words, scales, biases


# ---------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    c, vq = s["case"], s["vq"]
    op = c["op"]
    if op == "norm_pre":
        return {"x": vq.norm_pre(s["norm"], s["h"])}
    if op == "norm_pre_backward":
        dh, dw = vq.norm_pre_backward(s["norm"], s["h"], s["dx"], s["dres"])
        return {"dh": dh, "dw": dw}
    if op == "norm_post":
        h, x = vq.norm_post(s["y"], s["h"], s["norms"][0], s["gate"], c["res_scale"], c["out_scale"], s["norms"][1])
        return {"h": h, "x": x}
    if op == "norm_post_backward":
        dy, dgate, dh, dpost, dnext = vq.norm_post_backward(s["y"], s["h"], s["dh"], s["dx"], s["norms"][0], s["gate"],
                                                            c["res_scale"], c["out_scale"], s["norms"][1])
        return {"dy": dy, "dgate": dgate, "dh": dh, "dpost": dpost, "dnext": dnext}
    if op == "balance":
        loss, counts, probs = vq.balance_loss(s["logits"], s["ids"], s["mask"], s["coef"])
        dlogits = vq.balance_loss_backward(s["logits"], counts, c["k"], s["dloss"], s["mask"], s["coef"])
        return {"loss": loss, "counts": counts, "probs": probs, "dlogits": dlogits}
    return {"y": vq.q4_gemv(s["m"][0], s["x"], s["m"][1] if c["pair"] else None, TYPES[c["y"]])}


def _run_plain(s):
    op = s["case"]["op"]
    return {"norm_pre": _plain_pre, "norm_pre_backward": _plain_pre_backward, "norm_post": _plain_post,
            "norm_post_backward": _plain_post_backward, "balance": _plain_balance, "q4": _plain_q4}[op](s)


def _rstd(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)


def _norm_grad(v, r, dn):
    """Gradient at v of v * r(v), r = rsqrt(mean(v^2) + eps), for the gradient dn."""
    return r * dn - v * (r * r * r * (dn * v).mean(1, keepdim=True))


def _plain_pre(s):
    h = s["h"].float()
    return {"x": (h * _rstd(h) * (s["w"].float() + s["case"]["offset"])).to(BF16)}


def _plain_pre_backward(s):
    h, dx = s["h"].float(), s["dx"].float()
    r = _rstd(h)
    dh = _norm_grad(h, r, dx * (s["w"].float() + s["case"]["offset"])) + s["dres"].float()
    return {"dh": dh.to(s["h"].dtype), "dw": (dx * h * r).sum(0)}


def _plain_post(s):
    c = s["case"]
    u = s["y"].float()
    if s["post"] is not None:
        u = u * _rstd(u) * (s["post"].float() + c["offset"])
    if s["gate"] is not None:
        u = u / (1.0 + torch.exp(-s["gate"].float()))
    h = (c["res_scale"] * s["h"].float() + c["out_scale"] * u).to(s["h"].dtype)
    x = None
    if s["next"] is not None:      # the norm of the row as it is stored
        v = h.float()
        x = (v * _rstd(v) * (s["next"].float() + c["offset"])).to(BF16)
    return {"h": h, "x": x}


def _plain_post_backward(s):
    c = s["case"]
    y, dH = s["y"].float(), s["dh"].float()
    dpost = dnext = dgate = None
    if s["next"] is not None:
        h, dx = s["h"].float(), s["dx"].float()
        r = _rstd(h)
        dH = dH + _norm_grad(h, r, dx * (s["next"].float() + c["offset"]))
        dnext = (dx * h * r).sum(0)
    du = c["out_scale"] * dH
    u, n, r = y, None, None
    if s["post"] is not None:
        w = s["post"].float() + c["offset"]
        r = _rstd(y)
        n = y * r
        u = n * w
    if s["gate"] is not None:
        z = s["gate"].float()
        on, off = 1.0 / (1.0 + torch.exp(-z)), 1.0 / (1.0 + torch.exp(z))
        dgate = du * u
        dgate = ((dgate.sum(1, keepdim=True) if c["gate"] == "token" else dgate) * on * off).to(s["gate"].dtype)
        du = du * on
    dy = du
    if s["post"] is not None:
        dpost = (du * n).sum(0)
        dy = _norm_grad(y, r, du * w)
    return {"dy": dy.to(s["y"].dtype), "dgate": dgate, "dh": (c["res_scale"] * dH).to(s["h"].dtype), "dpost": dpost,
            "dnext": dnext}


def _plain_balance(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    m = torch.ones(T, device="cuda") if s["mask"] is None else s["mask"].float()
    pairs = torch.zeros(E, dtype=torch.int32, device="cuda")
    pairs.index_add_(0, s["ids"].reshape(-1), m.to(torch.int32).repeat_interleave(k))
    valid = m.sum()
    per = 1.0 / valid.clamp(min=1.0)
    e = torch.exp(s["logits"] - s["logits"].max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True)
    probs = (p * m[:, None]).sum(0) * per
    d = pairs.float() * (E * per / k)           # E * share of the pairs
    loss = s["coef"] * (d * probs).sum()
    dlogits = (s["dloss"] * s["coef"] * per) * m[:, None] * p * (d - (p * d).sum(1, keepdim=True))
    return {"loss": loss, "counts": torch.cat([pairs, valid.to(torch.int32)[None]]), "probs": probs, "dlogits": dlogits}


def _dequantised(c, m):
    words, scales, biases = m
    q = ((words[:, :, None] >> torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)) & 15).float()
    q = q.reshape(c["rows"], -1, c["group"])
    sc = scales.float()[:, :, None]
    w = sc * (q - 8.0) if biases is None else sc * q + biases.float()[:, :, None]
    return w.reshape(c["rows"], c["cols"])


def _plain_q4(s):
    c = s["case"]
    x = s["x"].float()
    y = x @ _dequantised(c, s["m"][0]).T
    if c["pair"]:
        y = y / (1.0 + torch.exp(-y)) * (x @ _dequantised(c, s["m"][1]).T)
    return {"y": y.to(TYPES[c["y"]])}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f32": 4}
    if op.startswith("norm"):
        n, H = c["T"] * c["H"], c["H"]
        hb, wb = size[c["h"]], size[c["w"]]
        if op == "norm_pre":
            return {"bytes": n * (hb + 2) + H * wb, "flops": 4 * n}
        if op == "norm_pre_backward":
            return {"bytes": n * (3 * hb + 2) + H * (wb + 4), "flops": 12 * n}
        yb = size[c["y"]]
        z = {"none": 0, "token": 2 * c["T"], "channel": 2 * n}[c["gate"]]
        norms = c["post"] + c["following"]
        if op == "norm_post":
            return {"bytes": n * (yb + 2 * hb + 2 * c["following"]) + z + norms * H * wb, "flops": 10 * n}
        return {"bytes": n * (2 * yb + 2 * hb + (hb + 2) * c["following"]) + 2 * z + norms * H * (wb + 4),
                "flops": 30 * n}
    if op == "balance":
        n = c["T"] * c["E"]
        # the logits are read once and the gradient written once; counts and sums stay on the chip
        return {"bytes": 8 * n + 4 * c["T"] * c["k"] + 8 * c["E"] + (c["T"] if c["padding"] else 0), "flops": 10 * n}
    n = c["rows"] * c["cols"] * (2 if c["pair"] else 1)
    return {"bytes": n // 2 + n // c["group"] * (4 if c["biased"] else 2) + 2 * c["T"] * c["cols"]
            + c["T"] * c["rows"] * size[c["y"]], "flops": 2 * c["T"] * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def _n64(v, w, offset):
    return v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS) * (w + offset)


def _back64(f, inputs, grads):
    """Gradients of sum(outputs * grads) at `inputs`, by differentiating the definition."""
    leaves = [None if v is None else v.double().requires_grad_() for v in inputs]
    outs = f(*leaves)
    total = sum((o * d.double()).sum() for o, d in zip(outs, grads) if d is not None)
    got = torch.autograd.grad(total, [v for v in leaves if v is not None], allow_unused=True)
    got = iter(got)
    return [None if v is None else next(got) for v in leaves]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, op = case, case["op"]
    if op == "norm_pre":
        return {"x": _n64(s["h"].double(), s["w"].double(), c["offset"])}
    if op == "norm_pre_backward":
        dh, dw = _back64(lambda h, w: (_n64(h, w, c["offset"]), h), (s["h"], s["w"]), (s["dx"], s["dres"]))
        return {"dh": dh, "dw": dw}

    def branch(y, w, z):
        u = y if w is None else _n64(y, w, c["offset"])
        return c["out_scale"] * (u if z is None else u * torch.sigmoid(z))

    dbl = lambda v: None if v is None else v.double()  # noqa: E731
    if op == "norm_post":
        h = (c["res_scale"] * s["h"].double() + branch(dbl(s["y"]), dbl(s["post"]), dbl(s["gate"])))
        stored = h.to(s["h"].dtype).double()
        return {"h": h, "x": None if s["next"] is None else _n64(stored, s["next"].double(), c["offset"])}
    if op == "norm_post_backward":
        # the stored row is the saved one: first the gradient at it, then through the branch
        dH, dnext = s["dh"].double(), None
        if s["next"] is not None:
            dn, dnext = _back64(lambda h, w: (_n64(h, w, c["offset"]),), (s["h"], s["next"]), (s["dx"],))
            dH = dH + dn
        dy, dpost, dgate = _back64(lambda y, w, z: (branch(y, w, z),), (s["y"], s["post"], s["gate"]), (dH,))
        return {"dy": dy, "dgate": dgate, "dh": c["res_scale"] * dH, "dpost": dpost, "dnext": dnext}
    if op == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        live = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
        n = int(live.sum())
        counts = torch.bincount(s["ids"][live].reshape(-1).long(), minlength=E)
        if n == 0:
            zero = torch.zeros(E, dtype=torch.float64, device="cuda")
            return {"loss": zero[0], "counts": torch.cat([counts, live.sum()[None]]), "probs": zero,
                    "dlogits": torch.zeros((T, E), dtype=torch.float64, device="cuda")}
        share = counts.double() / (n * k)
        logits = s["logits"].double().requires_grad_()
        probs = torch.softmax(logits, 1)[live].sum(0) / n
        loss = s["coef"] * E * (share * probs).sum()
        d, = torch.autograd.grad(loss, logits, s["dloss"].double())
        return {"loss": loss.detach(), "counts": torch.cat([counts, live.sum()[None]]), "probs": probs.detach(),
                "dlogits": d}
    x = s["x"].double()

    def product(m):
        words, scales, biases = m
        out = torch.empty((c["T"], c["rows"]), dtype=torch.float64, device="cuda")
        step = max(1, (1 << 27) // c["cols"])
        for r in range(0, c["rows"], step):
            part = words[r:r + step].long() & 0xFFFFFFFF
            q = torch.stack([(part // 16 ** i) % 16 for i in range(8)], 2).reshape(part.shape[0], c["cols"]).double()
            sc = scales[r:r + step].double().repeat_interleave(c["group"], 1)
            b = -8.0 * sc if biases is None else biases[r:r + step].double().repeat_interleave(c["group"], 1)
            out[:, r:r + step] = x @ (q * sc + b).T
        return out

    y = product(s["m"][0])
    if c["pair"]:
        y = y * torch.sigmoid(y) * product(s["m"][1])
    return {"y": y}
