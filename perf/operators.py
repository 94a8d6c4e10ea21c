"""Measured cases of the MoE block's training operators: layer norm, the router's gate with its balance loss, the
combine of the experts' rows, each with its gradient, and the global gradient norm with clipping.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once at the end), or,
where ``own`` is set, through this package's calls.  ``exact`` computes the definition in 64 bits.
"""

import math
import random

import torch

own = False

EPS = 1e-5        # layer norm
CLIP_EPS = 1e-6   # added to the norm before the division
LOSS_COEF = 0.01  # balance loss
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}

# How large a drawn case may be: the listed ones' largest moves about 1.34 GB.
MOST_BYTES = 1.0e9


def listed():
    return [
        # a decode batch's rows through the norm, at the block's width: latency
        {"name": "norm_decode", "op": "norm", "dir": "fwd", "M": 64, "N": 7168, "x": "bf16", "y": "bf16", "w": "bf16"},
        # an odd row length (no 16-byte rows) and an odd number of rows, all in 32 bits
        {"name": "norm_odd_f32", "op": "norm", "dir": "fwd", "M": 1021, "N": 4099, "x": "f32", "y": "f32", "w": "f32"},
        # a training batch's gradient at the MoE block's width
        {"name": "norm_grad", "op": "norm", "dir": "bwd", "M": 4096, "N": 7168, "x": "bf16", "y": "bf16", "w": "bf16"},
        # a large batch whose residual stream is kept in 32 bits and whose block works in bf16
        {"name": "norm_grad_large", "op": "norm", "dir": "bwd", "M": 16384, "N": 8192, "x": "f32", "y": "bf16", "w": "f32"},
        # a decode batch's router, 32 experts: latency
        {"name": "gate_decode", "op": "gate", "dir": "fwd", "T": 64, "E": 32, "k": 2, "x": "f32", "renorm": True, "masked": False},
        # a large batch with many experts and some padding tokens; bf16 logits tie often
        {"name": "gate_large", "op": "gate", "dir": "fwd", "T": 65536, "E": 256, "k": 8, "x": "bf16", "renorm": True, "masked": True},
        # a training batch's router gradient, top-2 of 8 experts, odd number of tokens
        {"name": "gate_grad", "op": "gate", "dir": "bwd", "T": 4095, "E": 8, "k": 2, "x": "f32", "renorm": False, "masked": False},
        # a decode batch's expert rows brought back to their tokens: latency
        {"name": "combine_decode", "op": "combine", "dir": "fwd", "T": 64, "E": 32, "k": 8, "N": 7168, "y": "bf16", "residual": False, "drop": 0.0},
        # a training batch, top-2 of 8 experts, added to a residual stream in 32 bits
        {"name": "combine_train", "op": "combine", "dir": "fwd", "T": 4096, "E": 8, "k": 2, "N": 4096, "y": "f32", "residual": True, "drop": 0.0},
        # its gradient with more experts, an odd number of tokens and entries dropped by a capacity
        {"name": "combine_grad", "op": "combine", "dir": "bwd", "T": 4001, "E": 32, "k": 4, "N": 7168, "y": "bf16", "residual": False, "drop": 0.03},
        # the gradients of a MoE layer: a few large bf16 tensors and small ones, 470 MB
        {"name": "clip_layer", "op": "clip", "dir": "upd", "tensors": 14, "total": 8 * 4096 * 7168, "x": "bf16", "flat": False, "sizes": 1},
        # many small odd tensors of both types, as views into flat buffers (few of them aligned)
        {"name": "clip_many_odd", "op": "clip", "dir": "upd", "tensors": 150, "total": 1500000, "x": "mixed", "flat": True, "sizes": 2},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; never 3072."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + 1 if v == 3072 else v


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm", "gate", "gate", "combine", "combine", "clip"])
        if op == "norm":
            n = rng.choice([_log(rng, 64, 16384), 8 * _log(rng, 8, 2048), 128 * _log(rng, 2, 96)])
            x = rng.choice(["bf16", "bf16", "f32"])
            c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "M": _log(rng, 1, 16384), "N": n, "x": x,
                 "y": "bf16" if x == "bf16" else rng.choice(["bf16", "f32"]), "w": rng.choice(["bf16", "f32"])}
        elif op == "gate":
            e = rng.choice([8, 16, 32, 64, 128, 256, _log(rng, 4, 512)])
            c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "T": _log(rng, 1, 65536), "E": e,
                 "k": rng.randint(1, min(8, e)), "x": rng.choice(["f32", "bf16"]), "renorm": rng.random() < 0.5,
                 "masked": rng.random() < 0.5}
        elif op == "combine":
            e = rng.choice([4, 8, 16, 32, 64, 128, _log(rng, 2, 128)])
            c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "T": _log(rng, 1, 8192), "E": e,
                 "k": rng.randint(1, min(8, e)), "N": rng.choice([16 * _log(rng, 4, 512), 128 * _log(rng, 2, 64)]),
                 "y": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.5, "drop": rng.choice([0.0, 0.0, 0.05])}
            c["residual"] = c["residual"] and c["dir"] == "fwd"
        else:
            flat = rng.random() < 0.4
            c = {"op": op, "dir": "upd", "tensors": _log(rng, 1, 300 if flat else 60), "total": _log(rng, 1000, 200_000_000),
                 "x": rng.choice(["bf16", "f32", "mixed"]), "flat": flat, "sizes": rng.randrange(1 << 20)}
        if c.get("N") != 3072 and work(c)["bytes"] <= MOST_BYTES:
            return c


def _capacity(c):
    """Rows of the routed layout: every expert's group padded to 128 rows."""
    return (c["T"] * c["k"] + 127 * c["E"] + 127) // 128 * 128


def _clip_sizes(c):
    """The tensors' numbers of values and types: by the case alone."""
    r = random.Random(c["sizes"])
    share = [math.exp(r.gauss(0.0, 2.0)) for _ in range(c["tensors"])]
    whole = sum(share)
    sizes = [max(1, int(c["total"] * s / whole)) for s in share]
    kinds = [c["x"] if c["x"] != "mixed" else r.choice(["bf16", "f32"]) for _ in sizes]
    return [(n + 1 if n == 3072 else n, k) for n, k in zip(sizes, kinds)]


def work(c):
    """Bytes and operations that one pass cannot do without."""
    if c["op"] == "norm":
        m, n, x, y, w = c["M"], c["N"], SIZE[c["x"]], SIZE[c["y"]], SIZE[c["w"]]
        if c["dir"] == "fwd":
            return {"bytes": m * n * (x + y) + 2 * n * w + 8 * m, "flops": 8 * m * n}
        return {"bytes": m * n * (2 * x + y) + n * w + 8 * n + 8 * m, "flops": 16 * m * n}
    if c["op"] == "gate":
        t, e, k, x = c["T"], c["E"], c["k"], SIZE[c["x"]]
        mask = t if c["masked"] else 0
        if c["dir"] == "fwd":
            return {"bytes": t * e * x + 8 * t * k + 4 * e + 4 + mask, "flops": 6 * t * e}
        return {"bytes": 2 * t * e * x + 8 * t * k + 4 * e + 4 + mask, "flops": 10 * t * e}
    if c["op"] == "combine":
        t, k, n, y = c["T"], c["k"], c["N"], SIZE[c["y"]]
        rows = t * k * (1.0 - c["drop"])
        if c["dir"] == "fwd":
            return {"bytes": rows * n * 2 + t * n * y * (2 if c["residual"] else 1) + 8 * t * k, "flops": 2 * rows * n}
        return {"bytes": t * n * y + rows * n * 2 + _capacity(c) * n * 2 + 12 * t * k + 4 * _capacity(c), "flops": 3 * rows * n}
    total = sum(n * SIZE[k] for n, k in _clip_sizes(c))
    return {"bytes": 2 * total, "flops": 3 * sum(n for n, _ in _clip_sizes(c))}


def _layout(ids, e, cap):
    """The routed layout of expert choices ids [T, k] (-1: dropped): each expert's rows in the order of the tokens,
    padded to 128.  Returns the row of each entry (-1: dropped) and the token of each row (-1: padding)."""
    t, k = ids.shape
    flat = ids.reshape(-1).long()
    kept = flat >= 0
    key = torch.where(kept, flat, torch.full_like(flat, e))
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(e + 1, dtype=torch.long, device=ids.device).index_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(count, 0) - count                   # first place of each expert in the sorted order
    padded = (count[:e] + 127) // 128 * 128
    start = torch.cumsum(padded, 0) - padded                 # first row of each expert
    start = torch.cat([start, start.new_zeros(1)])
    sorted_key = key[order]
    row = start[sorted_key] + torch.arange(t * k, device=ids.device) - first[sorted_key]
    row = torch.where(sorted_key < e, row, torch.full_like(row, -1))
    entry_row = torch.empty_like(row)
    entry_row[order] = row
    row_token = torch.full((cap + 1,), -1, dtype=torch.int32, device=ids.device)
    at = torch.where(row >= 0, row, torch.full_like(row, cap))  # dropped entries land in a place of their own
    row_token[at] = torch.where(row >= 0, order // k, torch.full_like(order, -1)).to(torch.int32)
    return entry_row.reshape(t, k).to(torch.int32), row_token[:cap].contiguous()


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=DEV) * std + mean).to(dtype)

    s = dict(c)
    if c["op"] == "norm":
        m, n = c["M"], c["N"]
        scale = torch.ones(n, device=DEV)
        cols = torch.randperm(n, generator=gen, device=DEV)[: max(1, n // 100)]
        scale[cols] = 20.0  # outlier channels, as activations have them
        s["x_"] = ((torch.randn((m, n), generator=gen, device=DEV) + 0.3) * scale).to(DT[c["x"]])
        s["weight"] = normal(n, std=0.2, mean=1.0, dtype=DT[c["w"]])
        s["bias"] = normal(n, std=0.1, dtype=DT[c["w"]])
        if c["dir"] == "bwd":
            s["dy"] = normal(m, n, std=0.02, dtype=DT[c["y"]])
            xf = s["x_"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
    elif c["op"] == "gate":
        t, e, k = c["T"], c["E"], c["k"]
        skew = torch.randn(e, generator=gen, device=DEV) * 0.7  # some experts are liked better
        s["logits"] = (torch.randn((t, e), generator=gen, device=DEV) + skew).to(DT[c["x"]])
        s["mask"] = None
        if c["masked"]:  # the last tokens of each stretch of 100 are padding
            s["mask"] = (torch.arange(t, device=DEV) % 100) < 93
        if c["dir"] == "bwd":
            lf = s["logits"].float()
            s["ids"] = torch.sort(lf, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
            ones = torch.ones(t, dtype=torch.int32, device=DEV) if s["mask"] is None else s["mask"].to(torch.int32)
            s["counts"] = torch.zeros(e, dtype=torch.int32, device=DEV).index_add_(
                0, s["ids"].reshape(-1).long(), ones[:, None].expand(t, k).reshape(-1))
            s["dweights"] = normal(t, k, std=0.1)
            s["dloss"] = torch.ones(1, device=DEV)
    elif c["op"] == "combine":
        t, e, k, n = c["T"], c["E"], c["k"], c["N"]
        skew = torch.randn(e, generator=gen, device=DEV) * 0.7
        logits = torch.randn((t, e), generator=gen, device=DEV) + skew
        top = torch.sort(logits, dim=1, descending=True, stable=True)
        ids = top.indices[:, :k].to(torch.int32)
        ids = torch.where(torch.rand((t, k), generator=gen, device=DEV) < c["drop"], torch.full_like(ids, -1), ids)
        s["weights"] = torch.softmax(top.values[:, :k], dim=1).contiguous()
        cap = _capacity(c)
        s["entry_row"], s["row_token"] = _layout(ids, e, cap)
        s["D"] = normal(cap, n, dtype=torch.bfloat16)
        s["res"] = normal(t, n, dtype=DT[c["y"]]) if c["residual"] else None
        if c["dir"] == "bwd":
            s["dout"] = normal(t, n, std=0.02, dtype=DT[c["y"]])
    else:
        kinds = _clip_sizes(c)

        def buffers(fill):
            if not c["flat"]:
                return [fill(n, DT[k]) for n, k in kinds]
            flat = {k: fill(sum(n for n, kk in kinds if kk == k), DT[k]) for k in sorted({k for _, k in kinds})}
            at, views = {k: 0 for k in flat}, []
            for n, k in kinds:
                views.append(flat[k][at[k]: at[k] + n])
                at[k] += n
            return views

        s["grads"] = buffers(lambda n, d: normal(n, std=0.01, dtype=d))
        s["out"] = buffers(lambda n, d: torch.empty(n, dtype=d, device=DEV))
        s["max_norm"] = 0.37 * 0.01 * math.sqrt(sum(n for n, _ in kinds))  # well below the norm: every pass clips
        if own:  # a training program's gradients stay where they are: it lists them once
            import moe_grouped_gemm_block_gb300 as g

            s["list"] = g.GradList(s["grads"], s["out"])
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_grouped_gemm_block_gb300 as g

    if s["op"] == "norm":
        if s["dir"] == "fwd":
            y, mean, rstd = g.layer_norm(s["x_"], s["weight"], s["bias"], eps=EPS, out_dtype=DT[s["y"]])
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = g.layer_norm_backward(s["dy"], s["x_"], s["weight"], s["mean"], s["rstd"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if s["op"] == "gate":
        if s["dir"] == "fwd":
            ids, w, counts, loss = g.moe_gate(s["logits"], s["k"], renormalize=s["renorm"], loss_coef=LOSS_COEF,
                                              token_mask=s["mask"])
            return {"ids": ids, "weights": w, "counts": counts, "loss": loss}
        return {"dlogits": g.moe_gate_backward(s["logits"], s["ids"], s["counts"], s["dweights"], s["dloss"],
                                               renormalize=s["renorm"], loss_coef=LOSS_COEF, token_mask=s["mask"])}
    if s["op"] == "combine":
        if s["dir"] == "fwd":
            return {"out": g.moe_combine(s["D"], s["entry_row"], s["weights"], residual=s["res"], out_dtype=DT[s["y"]])}
        dD, dw = g.moe_combine_backward(s["dout"], s["D"], s["entry_row"], s["row_token"], s["weights"])
        return {"dD": dD, "dweights": dw}
    norm = g.clip_grad_norm(s["list"], s["max_norm"], eps=CLIP_EPS)
    return _clip_result(s, norm)


def _clip_result(s, norm):
    """The norm and the clipped gradients: the tensors themselves, or the flat buffers that they are views of."""
    if s["flat"]:
        return {"norm": norm, **{str(t.dtype): t._base for t in s["out"]}}
    return {"norm": norm, "grads": s["out"]}


def _plain(s):
    if s["op"] == "norm":
        x = s["x_"].float()
        n = x.shape[1]
        w, b = s["weight"].float(), s["bias"].float()
        if s["dir"] == "fwd":
            mean = x.sum(1) / n
            d = x - mean[:, None]
            rstd = 1.0 / torch.sqrt((d * d).sum(1) / n + EPS)
            return {"y": (d * rstd[:, None] * w + b).to(DT[s["y"]]), "mean": mean, "rstd": rstd}
        dy = s["dy"].float()
        h = (x - s["mean"][:, None]) * s["rstd"][:, None]
        gw = dy * w
        c1 = gw.sum(1, keepdim=True) / n
        c2 = (gw * h).sum(1, keepdim=True) / n
        dx = (gw - c1 - h * c2) * s["rstd"][:, None]
        return {"dx": dx.to(DT[s["x"]]), "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}
    if s["op"] == "gate":
        lf = s["logits"].float()
        t, e = lf.shape
        k = s["k"]
        valid = torch.ones(t, device=lf.device) if s["mask"] is None else s["mask"].float()
        tv = valid.sum().clamp(min=1.0)
        ex = torch.exp(lf - lf.max(1, keepdim=True).values)
        p = ex / ex.sum(1, keepdim=True)
        if s["dir"] == "fwd":
            ids = torch.sort(lf, dim=1, descending=True, stable=True).indices[:, :k]
            w = p.gather(1, ids)
            if s["renorm"]:
                w = w / w.sum(1, keepdim=True)
            w = w * valid[:, None]
            counts = torch.zeros(e, dtype=torch.int32, device=lf.device).index_add_(
                0, ids.reshape(-1), valid.to(torch.int32)[:, None].expand(t, k).reshape(-1))
            mean_p = (p * valid[:, None]).sum(0) / tv
            loss = LOSS_COEF * e * (counts.float() / (k * tv) * mean_p).sum()
            return {"ids": ids.to(torch.int32), "weights": w, "counts": counts, "loss": loss.reshape(1)}
        ids = s["ids"].long()
        dw = s["dweights"]
        if s["renorm"]:
            sel = p.gather(1, ids)
            total = sel.sum(1, keepdim=True)
            dw = (dw - (dw * sel / total).sum(1, keepdim=True)) / total
        gp = (s["dloss"] * (LOSS_COEF * e) * s["counts"].float() / (k * tv * tv))[None, :].expand(t, e)
        gp = gp.scatter_add(1, ids, dw)
        dl = p * (gp - (gp * p).sum(1, keepdim=True)) * valid[:, None]
        return {"dlogits": dl.to(s["logits"].dtype)}
    if s["op"] == "combine":
        rows = s["entry_row"].long()
        kept = (rows >= 0)[..., None]
        picked = s["D"][rows.clamp(min=0)].float() * kept
        if s["dir"] == "fwd":
            out = (picked * s["weights"][..., None]).sum(1)
            if s["res"] is not None:
                out = out + s["res"].float()
            return {"out": out.to(DT[s["y"]])}
        dout = s["dout"].float()
        dw = (picked * dout[:, None, :]).sum(2)
        cap, n = s["D"].shape
        dD = torch.zeros((cap + 1, n), device=dout.device)
        dD[torch.where(rows >= 0, rows, torch.full_like(rows, cap))] = dout[:, None, :] * s["weights"][..., None]
        return {"dD": dD[:cap].to(torch.bfloat16), "dweights": dw}
    norm = torch.sqrt(torch.stack([t.float().square().sum() for t in s["grads"]]).sum()).reshape(1)
    coef = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
    [o.copy_(t.float() * coef) for t, o in zip(s["grads"], s["out"])]
    return _clip_result(s, norm)


def exact(c, seed):
    """The definitions in 64 bits."""
    s = prepare(c, seed)
    if c["op"] == "norm":
        x, w, b = s["x_"].double(), s["weight"].double(), s["bias"].double()
        if c["dir"] == "fwd":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            std = torch.sqrt(var + EPS)
            return {"y": (x - mean[:, None]) / std[:, None] * w + b, "mean": mean, "rstd": 1 / std}
        dy, mean, rstd = s["dy"].double(), s["mean"].double(), s["rstd"].double()
        x -= mean[:, None]
        x *= rstd[:, None]                         # the normalised rows
        dw, db = (dy * x).sum(0), dy.sum(0)
        dy *= w
        inner = (dy * x).sum(1, keepdim=True) / c["N"]
        x *= inner
        dy -= dy.mean(1, keepdim=True)
        return {"dx": (dy - x) * rstd[:, None], "dweight": dw, "dbias": db}
    if c["op"] == "gate":
        logits, e, k = s["logits"].double(), c["E"], c["k"]
        real = torch.ones(c["T"], dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
        tv = max(1, int(real.sum()))
        p = torch.softmax(logits, dim=1)
        if c["dir"] == "fwd":
            w, ids = [], []
            left = logits.clone()
            place = torch.arange(e, device=DEV)
            for _ in range(k):  # the largest that is left, the lowest index of equal ones
                best = left.max(1, keepdim=True).values
                i = torch.where(left == best, place, torch.full_like(place, e)).min(1, keepdim=True).values
                ids.append(i)
                w.append(p.gather(1, i))
                left.scatter_(1, i, -math.inf)
            w, ids = torch.cat(w, 1), torch.cat(ids, 1)
            if c["renorm"]:
                w = w / w.sum(1, keepdim=True)
            w[~real] = 0
            counts = torch.bincount(ids[real].reshape(-1), minlength=e).double()
            loss = LOSS_COEF * e * (counts / (k * tv)).dot(p[real].sum(0) / tv)
            return {"ids": None, "weights": w, "counts": None, "loss": loss.reshape(1)}
        with torch.enable_grad():  # by differentiating the definition
            leaf = logits.requires_grad_()
            q = torch.softmax(leaf, dim=1)
            w = q.gather(1, s["ids"].long())
            if c["renorm"]:
                w = w / w.sum(1, keepdim=True)
            loss = LOSS_COEF * e * (s["counts"].double() / (k * tv)).dot(q[real].sum(0) / tv)
            goal = (w[real] * s["dweights"].double()[real]).sum() + s["dloss"].double()[0] * loss
            return {"dlogits": torch.autograd.grad(goal, leaf)[0]}
    if c["op"] == "combine":
        rows, w = s["entry_row"].long(), s["weights"].double()
        t, n, cap = c["T"], c["N"], s["D"].shape[0]
        if c["dir"] == "fwd":
            out = torch.zeros((t, n), dtype=torch.float64, device=DEV) if s["res"] is None else s["res"].double()
            for j in range(c["k"]):
                has = rows[:, j] >= 0
                out[has] += w[has, j, None] * s["D"][rows[has, j]].double()
            return {"out": out}
        dout = s["dout"].double()
        dD = torch.zeros((cap, n), dtype=torch.float64, device=DEV)
        dw = torch.zeros_like(w)
        for j in range(c["k"]):
            has = rows[:, j] >= 0
            dD[rows[has, j]] = w[has, j, None] * dout[has]
            dw[has, j] = (dout[has] * s["D"][rows[has, j]].double()).sum(1)
        return {"dD": dD, "dweights": dw}
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in s["grads"]))
    coef = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
    done = torch.tensor([norm], dtype=torch.float64, device=DEV)
    if c["flat"]:
        base = {t.dtype: t._base for t in s["grads"]}
        return {"norm": done, **{str(d): t.double() * coef for d, t in base.items()}}
    return {"norm": done, "grads": [t.double() * coef for t in s["grads"]]}
