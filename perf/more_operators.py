"""Measured cases of a training step's further operators: the router with sigmoid or softmax scores, balance bias and
expert groups; the RMS norms around a block fused with its gate and residual; the gated activation between an expert's
two matrix products with its quantisation; and the AdamW step over many tensors with states in 32 or 8 bits.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, in 64 where a value's side of a
border counts, rounded once at the end), or, where ``own`` is set, through this package's calls.  ``exact`` computes the
definition in 64 bits.
"""

import math
import random

import torch

own = False

EPS = 1e-6                                   # the norms
BETA1, BETA2, ADAM_EPS = 0.9, 0.95, 1e-8     # AdamW
CLIP_EPS = 1e-6                              # added to the gradient norm before the division
DECAY = 0.1
ROUTE_SCALE = 2.5                            # the routed experts' weights together
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}

# How large a drawn case may be; the largest listed one moves about 3 GB.
MOST_BYTES = 1.2e9


def listed():
    return [
        # a decode batch's router: 256 experts in 8 groups, the best 4 groups stay: latency
        {"name": "route_decode", "op": "route", "dir": "fwd", "T": 64, "E": 256, "k": 8, "groups": 8, "kept": 4,
         "score": "sigmoid", "bias": True, "x": "f32", "renorm": True, "masked": False},
        # a large training batch of the same router, bf16 logits, some padding tokens
        {"name": "route_large", "op": "route", "dir": "fwd", "T": 65536, "E": 256, "k": 8, "groups": 8, "kept": 4,
         "score": "sigmoid", "bias": True, "x": "bf16", "renorm": True, "masked": True},
        # its gradient, softmax scores, odd numbers of tokens and experts
        {"name": "route_grad", "op": "route", "dir": "bwd", "T": 16383, "E": 160, "k": 6, "groups": 8, "kept": 3,
         "score": "softmax", "bias": True, "x": "f32", "renorm": False, "masked": False},
        # a decode batch between two blocks: the residual joined, the next block's norm: latency
        {"name": "norm_decode", "op": "norm", "dir": "fwd", "M": 64, "N": 7168, "stream": "bf16", "block": "bf16",
         "w": "bf16", "f": True, "post": False, "gate": False},
        # an odd width (no 16-byte rows) and an odd number of rows in 32 bits, with every part
        {"name": "norm_odd_f32", "op": "norm", "dir": "fwd", "M": 1021, "N": 4099, "stream": "f32", "block": "f32",
         "w": "f32", "f": True, "post": True, "gate": True},
        # a training batch's gradient, residual stream in 32 bits, block in bf16, norms on both sides and a gate
        {"name": "norm_grad", "op": "norm", "dir": "bwd", "M": 8192, "N": 7168, "stream": "f32", "block": "bf16",
         "w": "f32", "f": True, "post": True, "gate": True},
        # a decode batch's expert rows between their two matrix products, a capacity per expert: latency
        {"name": "glu_decode", "op": "glu", "dir": "fwd", "E": 32, "M": 64, "F": 2048, "masked": True, "h": False},
        # a training batch's routed rows, quantised for the second product and kept for the gradient
        {"name": "glu_train", "op": "glu", "dir": "fwd", "E": 1, "M": 33024, "F": 4096, "masked": False, "h": True},
        # the gradient of another batch's, an odd number of rows
        {"name": "glu_grad", "op": "glu", "dir": "bwd", "E": 1, "M": 8577, "F": 7168, "masked": False, "h": True},
        # many small odd tensors of both types, as views into flat buffers (few of them aligned)
        {"name": "adamw_many_odd", "op": "adamw", "dir": "upd", "bits": 32, "tensors": 150, "total": 1500000,
         "p": "mixed", "g": "same", "master": False, "flat": True, "sizes": 2, "clip": True},
        # an expert layer's weights in 32 bits with bf16 gradients
        {"name": "adamw_layer", "op": "adamw", "dir": "upd", "bits": 32, "tensors": 7, "total": 8 * 2048 * 7168,
         "p": "f32", "g": "bf16", "master": False, "flat": False, "sizes": 1, "clip": True},
        # a larger one's weights in bf16 with their 32-bit copies and states in 8 bits
        {"name": "adamw_layer_8bit", "op": "adamw", "dir": "upd", "bits": 8, "tensors": 7, "total": 8 * 2048 * 7168,
         "p": "bf16", "g": "bf16", "master": True, "flat": False, "sizes": 1, "clip": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["route", "route", "norm", "norm", "glu", "glu", "adamw", "adamw"])
        if op == "route":
            groups = rng.choice([1, 1, 2, 4, 8, rng.randint(1, 12)])
            per = rng.choice([4, 8, 16, 32, 64, _log(rng, 2, 64)])
            e = groups * per
            kept = rng.randint(1, groups)
            c = {"op": op, "dir": rng.choice(["fwd", "fwd", "bwd"]), "T": _log(rng, 1, 65536), "E": e,
                 "k": rng.randint(1, min(8, kept * per)), "groups": groups, "kept": kept,
                 "score": rng.choice(["sigmoid", "sigmoid", "softmax"]), "bias": rng.random() < 0.7,
                 "x": rng.choice(["f32", "bf16"]), "renorm": rng.random() < 0.7, "masked": rng.random() < 0.4}
            if e < 4 or e > 512:
                continue
        elif op == "norm":
            n = rng.choice([_log(rng, 64, 16384), 8 * _log(rng, 8, 2048), 128 * _log(rng, 2, 96)])
            stream = rng.choice(["bf16", "f32"])
            f = rng.random() < 0.85
            c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "M": _log(rng, 1, 16384), "N": n, "stream": stream,
                 "block": "bf16" if stream == "bf16" else rng.choice(["bf16", "f32"]), "w": rng.choice(["bf16", "f32"]),
                 "f": f, "post": f and rng.random() < 0.5, "gate": f and rng.random() < 0.5}
        elif op == "glu":
            masked = rng.random() < 0.4
            c = {"op": op, "dir": "fwd" if masked else rng.choice(["fwd", "bwd"]),
                 "E": _log(rng, 1, 64) if masked else 1, "M": _log(rng, 1, 512) if masked else _log(rng, 1, 32768),
                 "F": 128 * _log(rng, 1, 64), "masked": masked, "h": not masked and rng.random() < 0.5}
        else:
            flat = rng.random() < 0.4
            p = rng.choice(["bf16", "f32", "mixed"])
            c = {"op": op, "dir": "upd", "bits": rng.choice([8, 32]), "tensors": _log(rng, 1, 300 if flat else 20),
                 "total": _log(rng, 1000, 40_000_000), "p": p, "g": rng.choice(["same", "bf16", "f32"]),
                 "master": p == "bf16" and rng.random() < 0.5, "flat": flat, "sizes": rng.randrange(1 << 20),
                 "clip": rng.random() < 0.6}
        if work(c)["bytes"] <= MOST_BYTES:
            return c


def _adam_tensors(c):
    """Each tensor's number of values, its type, its gradient's and its place in the flat state buffers, and their
    length: by the case alone.  A tensor's states start on a multiple of 128 values."""
    r = random.Random(c["sizes"])
    share = [math.exp(r.gauss(0.0, 2.0)) for _ in range(c["tensors"])]
    whole = sum(share)
    got, at = [], 0
    for s in share:
        n = max(1, int(c["total"] * s / whole))
        p = c["p"] if c["p"] != "mixed" else r.choice(["bf16", "f32"])
        got.append((n, p, p if c["g"] == "same" else c["g"], at))
        at += (n + 127) // 128 * 128
    return got, at


def work(c):
    """Bytes and operations that one pass cannot do without."""
    if c["op"] == "route":
        t, e, k, x = c["T"], c["E"], c["k"], SIZE[c["x"]]
        mask = t if c["masked"] else 0
        if c["dir"] == "fwd":
            return {"bytes": t * e * x + 8 * t * k + 8 * e + mask, "flops": 8 * t * e}
        read = t * e * x if c["score"] == "softmax" else t * k * x  # the sigmoid's needs the chosen logits alone
        return {"bytes": read + t * e * x + 8 * t * k + mask, "flops": 8 * t * e}
    if c["op"] == "norm":
        m, n, x, y, w = c["M"], c["N"], SIZE[c["stream"]], SIZE[c["block"]], SIZE[c["w"]]
        weights = 1 + c["post"] + c["gate"]
        if c["dir"] == "fwd":
            moved = x + y + ((x + y) if c["f"] else 0)
            return {"bytes": m * n * moved + weights * n * w + 4 * m * (1 + c["post"]), "flops": 10 * m * n}
        reads_f = c["f"] and (c["post"] or c["gate"])
        moved = 3 * x + y + (y if c["f"] else 0) + (y if reads_f else 0)
        return {"bytes": m * n * moved + weights * n * (w + 4) + 4 * m * (1 + c["post"]), "flops": 20 * m * n}
    if c["op"] == "glu":
        rows = int(_counts(c).sum()) if c["masked"] else c["M"]
        f = c["F"]
        if c["dir"] == "fwd":
            return {"bytes": rows * f * (4 + 1 + (2 if c["h"] else 0)) + rows * f // 32, "flops": 10 * rows * f}
        return {"bytes": rows * f * (2 + 4 + 4 + (2 if c["h"] else 0)), "flops": 20 * rows * f}
    tensors, _ = _adam_tensors(c)
    state = 16 if c["bits"] == 32 else 4 + 4 * 4 / 128
    moved = sum(n * (state + SIZE[g] + ((8 + SIZE[p]) if c["master"] else 2 * SIZE[p])) for n, p, g, _ in tensors)
    return {"bytes": moved, "flops": 15 * sum(t[0] for t in tensors)}


def _counts(c):
    """The masked layout's valid rows an expert: by the case alone (uniform; the first expert none, the second all)."""
    r = random.Random(c["E"] * 1000003 + c["M"])
    n = [r.randint(0, c["M"]) for _ in range(c["E"])]
    if c["E"] > 2:
        n[0], n[1] = 0, c["M"]
    return torch.tensor(n, dtype=torch.int32)


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=DEV) * std + mean).to(dtype)

    s = dict(c)
    if c["op"] == "route":
        t, e, k = c["T"], c["E"], c["k"]
        skew = torch.randn(e, generator=gen, device=DEV) * 0.5  # some experts are liked better
        s["logits"] = (torch.randn((t, e), generator=gen, device=DEV) + skew).to(DT[c["x"]])
        spread = 0.05 if c["score"] == "sigmoid" else 0.3 / e
        s["bias_"] = normal(e, std=spread) if c["bias"] else None  # what balances them, in steps of training
        s["mask"] = (torch.arange(t, device=DEV) % 100) < 93 if c["masked"] else None
        if c["dir"] == "bwd":
            any_order = torch.argsort(torch.rand((t, e), generator=gen, device=DEV), dim=1)
            s["ids"] = any_order[:, :k].to(torch.int32).contiguous()
            s["dweights"] = normal(t, k, std=0.1)
    elif c["op"] == "norm":
        m, n = c["M"], c["N"]
        scale = torch.ones(n, device=DEV)
        scale[torch.randperm(n, generator=gen, device=DEV)[: max(1, n // 100)]] = 20.0  # outlier channels
        st, bl, wt = DT[c["stream"]], DT[c["block"]], DT[c["w"]]
        s["x_"] = (torch.randn((m, n), generator=gen, device=DEV) * scale).to(st)
        s["f_"] = normal(m, n, std=0.7, dtype=bl) if c["f"] else None
        s["weight"] = normal(n, std=0.2, mean=1.0, dtype=wt)
        s["post_"] = normal(n, std=0.2, mean=1.0, dtype=wt) if c["post"] else None
        s["gate_"] = normal(n, std=0.1, mean=0.5, dtype=wt) if c["gate"] else None
        s["scale"] = 0.75 if c["f"] else 1.0
        if c["dir"] == "bwd":  # x_ is the stream after the block here
            s["dy"] = normal(m, n, std=0.02, dtype=bl)
            s["dh"] = normal(m, n, std=0.02, dtype=st)
            s["rstd"] = 1.0 / torch.sqrt(s["x_"].float().square().mean(1) + EPS)
            s["rstd_f"] = 1.0 / torch.sqrt(s["f_"].float().square().mean(1) + EPS) if c["post"] else None
    elif c["op"] == "glu":
        e, m, f = c["E"], c["M"], c["F"]
        shape = (e, m, 2 * f) if c["masked"] else (m, 2 * f)
        s["gu"] = torch.randn(shape, generator=gen, device=DEV).mul_(1.5).to(torch.bfloat16)
        if c["masked"]:
            s["counts"] = _counts(c).to(DEV)
            # a serving program's buffers: what lies behind an expert's rows stays
            s["q"] = torch.zeros((e, m, f), dtype=torch.uint8, device=DEV)
            s["sA"] = torch.zeros((f // 128, (e * m + 3) // 4 * 4), device=DEV)
        if c["dir"] == "bwd":
            s["dh"] = normal(m, f, std=0.02, dtype=torch.bfloat16)
    else:
        tensors, length = _adam_tensors(c)

        def buffers(kind, fill):
            if not c["flat"]:
                return [fill(t[0], DT[t[kind]]) for t in tensors]
            kinds = sorted({t[kind] for t in tensors})
            flat = {k: fill(sum(t[0] for t in tensors if t[kind] == k), DT[k]) for k in kinds}
            at, views = {k: 0 for k in flat}, []
            for t in tensors:
                views.append(flat[t[kind]][at[t[kind]]: at[t[kind]] + t[0]])
                at[t[kind]] += t[0]
            return views

        s["params"] = buffers(1, lambda n, d: normal(n, std=0.02, dtype=d))
        s["grads"] = buffers(2, lambda n, d: normal(n, std=0.01, dtype=d))
        s["step"] = torch.full((1,), 100, dtype=torch.int64, device=DEV)
        s["norm"] = torch.sqrt(sum(g.float().square().sum() for g in s["grads"])).reshape(1)
        s["max_norm"] = 0.37 * 0.01 * math.sqrt(sum(t[0] for t in tensors))  # well below the norm: it clips
        used = torch.zeros(length, device=DEV)
        [used[t[3]: t[3] + t[0]].fill_(1.0) for t in tensors]
        m0 = normal(length, std=0.002).mul_(used)
        v0 = normal(length, std=0.01).square_().add_(1e-6).mul_(used)
        if c["bits"] == 32:
            s["m"], s["v"] = m0, v0
        else:
            s["m"], s["ms"] = _codes(m0, torch.zeros((), dtype=torch.int64, device=DEV), 0)
            s["v"], s["vs"] = _codes(v0.sqrt_(), torch.zeros((), dtype=torch.int64, device=DEV), 0)
        s["places"] = [(t[3], t[0]) for t in tensors]
        s["masters"] = None
        if c["master"]:
            s["masters"] = torch.zeros(length, device=DEV)
            [s["masters"][at: at + n].copy_(p) for (at, n), p in zip(s["places"], s["params"])]
        if own:  # a training program's tensors stay where they are: it lists them once
            import moe_grouped_gemm_block_gb300 as g

            cut = lambda flat: None if flat is None else [flat[at: at + n] for at, n in s["places"]]  # noqa: E731
            blocks = lambda flat: [flat[at // 128: (at + n + 127) // 128] for at, n in s["places"]]  # noqa: E731
            more = {"m_scales": blocks(s["ms"]), "v_scales": blocks(s["vs"])} if c["bits"] == 8 else {}
            s["list"] = g.AdamWList(s["params"], s["grads"], masters=cut(s["masters"]), state_bits=c["bits"],
                                    weight_decay=DECAY, m=cut(s["m"]), v=cut(s["v"]), step=s["step"], **more)
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_grouped_gemm_block_gb300 as g

    if s["op"] == "route":
        if s["dir"] == "fwd":
            ids, w, counts = g.moe_route(s["logits"], s["k"], bias=s["bias_"], score=s["score"], groups=s["groups"],
                                         topk_groups=s["kept"], renormalize=s["renorm"], scale=ROUTE_SCALE,
                                         token_mask=s["mask"])
            return {"ids": ids, "weights": w, "counts": counts}
        return {"dlogits": g.moe_route_backward(s["logits"], s["ids"], s["dweights"], score=s["score"],
                                                renormalize=s["renorm"], scale=ROUTE_SCALE, token_mask=s["mask"])}
    if s["op"] == "norm":
        if s["dir"] == "fwd":
            h, y, rstd, rstd_f = g.residual_rms_norm(s["x_"], s["f_"], s["weight"], gate=s["gate_"], scale=s["scale"],
                                                     post_norm=s["post"], post_weight=s["post_"], eps=EPS,
                                                     out_dtype=DT[s["block"]])
            return {"h": h if s["f"] else None, "y": y, "rstd": rstd, "rstd_f": rstd_f}
        dx, df, dw, dgate, dpost = g.residual_rms_norm_backward(
            s["dy"], s["dh"], s["x_"], s["f_"], s["rstd"], s["rstd_f"], s["weight"], gate=s["gate_"], scale=s["scale"],
            post_norm=s["post"], post_weight=s["post_"])
        return {"dx": dx, "df": df, "dweight": dw, "dgate": dgate, "dpost": dpost}
    if s["op"] == "glu":
        if s["masked"]:
            g.fp8_swiglu_quantize_1x128_masked(s["gu"], s["q"], s["sA"], s["counts"])
            return {"q": s["q"].view(torch.float8_e4m3fn), "sA": s["sA"]}
        if s["dir"] == "fwd":
            q, sA, h = g.swiglu_quantize_1x128(s["gu"], ld_sa=(s["M"] + 3) // 4 * 4, keep=s["h"])
            return {"q": q.view(torch.float8_e4m3fn), "sA": sA[:, : s["M"]], "h": h}
        dgu, h = g.swiglu_backward(s["dh"], s["gu"], keep=s["h"])
        return {"dgu": dgu, "h": h}
    g.adamw_step(s["list"], 1e-3, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, norm=s["norm"] if s["clip"] else None,
                 max_norm=s["max_norm"], norm_eps=CLIP_EPS)
    return _adam_result(s)


def _adam_result(s):
    """Everything that the step writes: the parameters (the tensors, or the flat buffers that they are views of), their
    32-bit copies, the states (in 8 bits: the codes' values and the blocks' scales) and the count of steps."""
    p = {str(t.dtype): t._base for t in s["params"]} if s["flat"] else {"params": s["params"]}
    got = {**p, "masters": s["masters"], "step": s["step"]}
    if s["bits"] == 32:
        return {**got, "m": s["m"], "v": s["v"]}
    e4m3 = torch.float8_e4m3fn
    return {**got, "m": s["m"].view(e4m3), "ms": s["ms"], "v": s["v"].view(e4m3), "vs": s["vs"]}


# ------------------------------------------------------------------ the plain forms

def _plain(s):
    return {"route": _plain_route, "norm": _plain_norm, "glu": _plain_glu, "adamw": _plain_adamw}[s["op"]](s)


def _scores(logits, kind):
    """Scores of the experts; an expert whose logit is -inf has none."""
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    top = logits.max(1, keepdim=True).values
    e = torch.exp(logits - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    logits, k = s["logits"], s["k"]
    t, e = logits.shape
    real = torch.ones(t, dtype=torch.bool, device=logits.device) if s["mask"] is None else s["mask"]
    score = _scores(logits.float(), s["score"])
    if s["dir"] == "fwd":
        # the choice is made in 64 bits: two scores may be near one another
        fine = _scores(logits.double(), s["score"])
        choice = fine if s["bias_"] is None else fine + s["bias_"].double()
        per = e // s["groups"]
        best = choice.reshape(t, s["groups"], per).sort(2, descending=True).values[:, :, : min(2, per)].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : s["kept"]]
        out = torch.ones((t, s["groups"]), dtype=torch.bool, device=logits.device).scatter_(1, kept, False)
        order = logits.double() if s["bias_"] is None else choice  # (the scores order as the logits do)
        order = order.masked_fill(out[:, :, None].expand(t, s["groups"], per).reshape(t, e), -math.inf)
        ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
        w = score.gather(1, ids)
        if s["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = w * (ROUTE_SCALE * real.float())[:, None]
        counts = torch.zeros(e, dtype=torch.int32, device=logits.device).index_add_(
            0, ids.reshape(-1), real.to(torch.int32)[:, None].expand(t, k).reshape(-1))
        return {"ids": ids.to(torch.int32), "weights": w, "counts": counts}
    ids = s["ids"].long()
    dw = s["dweights"] * ROUTE_SCALE
    if s["renorm"]:
        sel = score.gather(1, ids)
        total = sel.sum(1, keepdim=True)
        dw = (dw - (dw * sel / total).sum(1, keepdim=True)) / total
    ds = torch.zeros((t, e), device=logits.device).scatter_add_(1, ids, dw)
    if s["score"] == "sigmoid":
        dl = ds * score * (1.0 - score)
    else:
        dl = score * (ds - (ds * score).sum(1, keepdim=True))
    return {"dlogits": (dl * real[:, None]).to(logits.dtype)}


def _plain_norm(s):
    x, w = s["x_"].float(), s["weight"].float()
    n = x.shape[1]
    f = None if s["f_"] is None else s["f_"].float()
    a = s["scale"] if s["gate_"] is None else s["scale"] * s["gate_"].float()
    st, bl = DT[s["stream"]], DT[s["block"]]
    if s["dir"] == "fwd":
        rstd_f = None
        if f is not None:
            if s["post"]:
                rstd_f = 1.0 / torch.sqrt((f * f).sum(1) / n + EPS)
                f = f * rstd_f[:, None] * s["post_"].float()
            x = x + a * f
        rstd = 1.0 / torch.sqrt((x * x).sum(1) / n + EPS)
        return {"h": x.to(st) if s["f"] else None, "y": (x * rstd[:, None] * w).to(bl), "rstd": rstd, "rstd_f": rstd_f}
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    hat = x * rstd
    g = dy * w
    dx = s["dh"].float() + rstd * (g - hat * ((g * hat).sum(1, keepdim=True) / n))
    got = {"dx": dx.to(st), "dweight": (dy * hat).sum(0)}
    if f is None:
        return got
    g = dx * a
    if s["post"]:
        rstd_f = s["rstd_f"][:, None]
        f = f * rstd_f
        g = g * s["post_"].float()
        got["df"] = (rstd_f * (g - f * ((g * f).sum(1, keepdim=True) / n))).to(bl)
        got["dpost"] = (dx * f).sum(0) * a
    else:
        got["df"] = g.expand_as(dx).to(bl)
    if s["gate"]:
        got["dgate"] = (dx * f).sum(0) * (s["scale"] * s["post_"].float() if s["post"] else s["scale"])
    return got


def _plain_glu(s):
    f = s["F"]
    gate, up = s["gu"][..., :f].float(), s["gu"][..., f:].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    h = gate * sig * up
    if s["dir"] == "bwd":
        dh = s["dh"].float()
        dg = dh * up * sig * (1.0 + gate * (1.0 - sig))
        dgu = torch.cat([dg, dh * gate * sig], 1)
        return {"dgu": dgu.to(torch.bfloat16), "h": h.to(torch.bfloat16) if s["h"] else None}
    rows = h.reshape(-1, f // 128, 128)
    top = rows.abs().amax(2)
    scale = top / 448.0
    q = (rows / torch.where(top > 0, scale, torch.ones_like(scale))[..., None]).to(torch.float8_e4m3fn).reshape(h.shape)
    sA = scale.t().contiguous()
    if not s["masked"]:
        return {"q": q, "sA": sA, "h": h.to(torch.bfloat16) if s["h"] else None}
    valid = torch.arange(s["M"], device=h.device)[None, :] < s["counts"][:, None]
    q = torch.where(valid[..., None], q.view(torch.uint8), s["q"])
    old = s["sA"].clone()
    old[:, : valid.numel()] = torch.where(valid.reshape(1, -1), sA, old[:, : valid.numel()])
    return {"q": q.view(torch.float8_e4m3fn), "sA": old}


def _codes(x, step, salt):
    """x in blocks of 128 -> (e4m3 bytes, the blocks' scales): |x| 448 / amax is taken up or down to a neighbouring e4m3
    value, up where its place between them and a number that goes by position and step are 1 or more together; what is
    not 0 gives no 0 where salt is set (the second moments' roots)."""
    n = x.numel()
    pad = (n + 127) // 128 * 128
    b = torch.nn.functional.pad(x, (0, pad - n)).reshape(-1, 128)
    top = b.abs().amax(1)
    live = top >= 2.0 ** -60
    inv = torch.where(live, 448.0 / top, torch.zeros_like(top))
    scale = torch.where(live, top / 448.0, torch.zeros_like(top))
    y = (b.abs() * inv[:, None]).double()
    place = torch.arange(pad, device=x.device).reshape(-1, 128)
    u = (place * 0xC13FA9A9 + step * 0x91E10DA5 + salt) & 0xFFFFFFFF
    u = (u >> 12).double() / 2 ** 20
    unit = torch.exp2(torch.frexp(y.clamp(min=2.0 ** -6)).exponent.double() - 4)
    c = torch.clamp(torch.floor(y / unit + u) * unit, max=448.0)
    if salt:
        c = torch.where((b > 0) & live[:, None], c.clamp(min=2.0 ** -9), c)
    c = torch.where(b < 0, -c, c).float().to(torch.float8_e4m3fn)
    return c.view(torch.uint8).reshape(-1)[:n].contiguous(), scale.float()


def _values(codes, scales):
    """What 8-bit states stand for."""
    n = codes.numel()
    return (codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128)[:n])


def _plain_adamw(s):
    s["step"] += 1
    t = s["step"].double()
    c1, c2 = (1.0 - BETA1 ** t).float(), (1.0 - BETA2 ** t).float()
    coef = torch.clamp(s["max_norm"] / (s["norm"] + CLIP_EPS), max=1.0) if s["clip"] else torch.ones_like(s["norm"])
    [_plain_adamw_tensor(s, i, coef, c1, c2) for i in range(s["tensors"])]
    return _adam_result(s)


def _plain_adamw_tensor(s, i, coef, c1, c2):
    at, n = s["places"][i]
    cut, blocks = slice(at, at + n), slice(at // 128, (at + n + 127) // 128)
    g = s["grads"][i].float() * coef
    p = s["params"][i].float() if s["masters"] is None else s["masters"][cut]
    if s["bits"] == 32:
        m = BETA1 * s["m"][cut] + (1.0 - BETA1) * g
        v = BETA2 * s["v"][cut] + (1.0 - BETA2) * g * g
        root = torch.sqrt(v)
        s["m"][cut], s["v"][cut] = m, v
    else:
        m = BETA1 * _values(s["m"][cut], s["ms"][blocks]) + (1.0 - BETA1) * g
        v = BETA2 * _values(s["v"][cut], s["vs"][blocks]).square() + (1.0 - BETA2) * g * g
        root = torch.sqrt(v)
        s["m"][cut], s["ms"][blocks] = _codes(m, s["step"], 0)
        s["v"][cut], s["vs"][blocks] = _codes(root, s["step"], 1 << 31)
    p = p * (1.0 - 1e-3 * DECAY) - 1e-3 * (m / c1) / (root / torch.sqrt(c2) + ADAM_EPS)
    s["params"][i].copy_(p)
    if s["masters"] is not None:
        s["masters"][cut] = p


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    return {"route": _exact_route, "norm": _exact_norm, "glu": _exact_glu, "adamw": _exact_adamw}[c["op"]](c, s)


def _exact_route(c, s):
    logits, k, e = s["logits"].double(), c["k"], c["E"]
    t = c["T"]
    real = torch.ones(t, device=DEV, dtype=torch.float64) if s["mask"] is None else s["mask"].double()
    with torch.enable_grad():
        leaf = logits.requires_grad_()
        score = torch.sigmoid(leaf) if c["score"] == "sigmoid" else torch.softmax(leaf, dim=1)
        if c["dir"] == "bwd":  # by differentiating the definition
            w = score.gather(1, s["ids"].long())
            if c["renorm"]:
                w = w / w.sum(1, keepdim=True)
            goal = (w * (ROUTE_SCALE * real)[:, None] * s["dweights"].double()).sum()
            return {"dlogits": torch.autograd.grad(goal, leaf)[0]}
    score = score.detach()
    choice = score if s["bias_"] is None else score + s["bias_"].double()
    per = e // c["groups"]

    def take(left, count):  # the largest that is left, the lowest place of equal ones
        got, place = [], torch.arange(left.shape[1], device=DEV)
        for _ in range(count):
            best = left.max(1, keepdim=True).values
            i = torch.where(left == best, place, torch.full_like(place, left.shape[1])).min(1, keepdim=True).values
            got.append(i)
            left = left.scatter(1, i, -math.inf)
        return torch.cat(got, 1)

    first, second = choice.reshape(t, -1, per).max(2).values, 0.0
    if per > 1:
        second = choice.reshape(t, -1, per).topk(2, dim=2).values[:, :, 1]
    kept = take(first + second, c["kept"])
    open_ = torch.zeros((t, c["groups"]), device=DEV, dtype=torch.bool).scatter_(1, kept, True)
    open_ = open_.repeat_interleave(per, dim=1)
    by = s["logits"].double() if s["bias_"] is None else choice
    ids = take(torch.where(open_, by, torch.full_like(by, -math.inf)), k)
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": None, "weights": w * (ROUTE_SCALE * real)[:, None], "counts": None}


def _exact_norm(c, s):
    w = s["weight"].double()
    x = s["x_"].double()
    f = s["f_"].double() if c["f"] else None
    gate = s["gate_"].double() if c["gate"] else torch.ones_like(w)
    post = s["post_"].double() if c["post"] else torch.ones_like(w)
    if c["dir"] == "fwd":
        rstd_f = None
        if f is not None:
            if c["post"]:
                rstd_f = (f.square().mean(1) + EPS).rsqrt()
                f = f * rstd_f[:, None]
            x = x + f * (post * gate * s["scale"])
        rstd = (x.square().mean(1) + EPS).rsqrt()
        return {"h": x if c["f"] else None, "y": x * rstd[:, None] * w, "rstd": rstd, "rstd_f": rstd_f}
    n = c["N"]
    rstd, dy = s["rstd"].double()[:, None], s["dy"].double()
    x *= rstd
    inner = ((dy * w) * x).sum(1, keepdim=True) / n
    dx = s["dh"].double() + rstd * (dy * w - x * inner)
    got = {"dx": dx, "dweight": (dy * x).sum(0)}
    if f is None:
        return got
    if c["post"]:
        f *= s["rstd_f"].double()[:, None]
    both = s["scale"] * (dx * f).sum(0)
    inner = (dx * (s["scale"] * gate * post) * f).sum(1, keepdim=True) / n
    got["df"] = dx * (s["scale"] * gate * post)
    if c["post"]:
        got["df"] = (got["df"] - f * inner) * s["rstd_f"].double()[:, None]
        got["dpost"] = both * gate
    if c["gate"]:
        got["dgate"] = both * post
    return got


def _exact_glu(c, s):
    f = c["F"]
    gate, up = s["gu"][..., :f].double(), s["gu"][..., f:].double()
    if c["dir"] == "bwd":
        sig = torch.sigmoid(gate)
        dh = s["dh"].double()
        dgu = torch.empty(s["gu"].shape, dtype=torch.float64, device=DEV)
        dgu[:, :f] = dh * up * (sig + gate * sig * torch.sigmoid(-gate))
        dgu[:, f:] = dh * gate * sig
        return {"dgu": dgu, "h": gate * sig * up if c["h"] else None}
    h = gate * torch.sigmoid(gate) * up
    rows = h.reshape(-1, 128)
    scale = rows.abs().amax(1, keepdim=True) / 448.0
    q = (rows / scale).reshape(h.shape)  # what the codes are the rounding of
    sA = scale.reshape(-1, f // 128).t()
    if not c["masked"]:
        return {"q": q, "sA": sA, "h": h if c["h"] else None}
    valid = torch.arange(c["M"], device=DEV)[None, :] < s["counts"][:, None]
    full = torch.zeros(s["sA"].shape, dtype=torch.float64, device=DEV)
    full[:, : valid.numel()] = sA * valid.reshape(1, -1)
    return {"q": q * valid[..., None], "sA": full}


def _exact_adamw(c, s):
    t = 101
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"]))
    coef = min(1.0, s["max_norm"] / (norm + CLIP_EPS)) if c["clip"] else 1.0
    root2 = math.sqrt(1.0 - BETA2 ** t)
    got = {k: torch.zeros(s["m"].shape, dtype=torch.float64, device=DEV) for k in ("m", "v")}
    if c["bits"] == 8:
        got |= {k: torch.zeros(s["ms"].shape, dtype=torch.float64, device=DEV) for k in ("ms", "vs")}
    if c["master"]:
        got["masters"] = torch.zeros(s["m"].shape, dtype=torch.float64, device=DEV)
    params = []
    for i, (at, n) in enumerate(s["places"]):
        cut, blocks = slice(at, at + n), slice(at // 128, (at + n + 127) // 128)
        g = s["grads"][i].double() * coef
        if c["bits"] == 32:
            m, v = s["m"][cut].double(), s["v"][cut].double()
        else:
            block = torch.arange(n, device=DEV) // 128
            m = s["m"][cut].view(torch.float8_e4m3fn).double() * s["ms"][blocks].double()[block]
            v = (s["v"][cut].view(torch.float8_e4m3fn).double() * s["vs"][blocks].double()[block]).square()
        m = torch.lerp(g, m, BETA1)
        v = torch.lerp(g.square(), v, BETA2)
        p = (s["masters"][cut] if c["master"] else s["params"][i]).double()
        p = p - 1e-3 * (DECAY * p + m / (1.0 - BETA1 ** t) / (v.sqrt() / root2 + ADAM_EPS))
        params.append(p)
        if c["master"]:
            got["masters"][cut] = p
        if c["bits"] == 32:
            got["m"][cut], got["v"][cut] = m, v
            continue
        for name, x in (("m", m), ("v", v.sqrt())):  # the values that the codes are near to, and the scales
            top = torch.zeros(blocks.stop - blocks.start, dtype=torch.float64, device=DEV).scatter_reduce_(
                0, block, x.abs(), "amax")
            got[name + "s"][blocks] = top / 448.0
            got[name][cut] = x * 448.0 / top[block]
    got["step"] = None
    if not c["flat"]:
        return {**got, "params": params}
    kinds = [str(t.dtype) for t in s["params"]]
    return {**got, **{k: torch.cat([p for p, kk in zip(params, kinds) if kk == k]) for k in set(kinds)}}
