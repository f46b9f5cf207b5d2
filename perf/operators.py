"""Cases and plain forms of the expert-training operators.

One expert layer of a training step: the tokens are normalised (layer norm),
sent to their experts and quantized in 1x128 blocks in the order the experts
read them (grouped quantization), multiplied by each expert's FP8 weights
(grouped GEMM: fprop and dgrad over ragged rows, wgrad over ragged
contractions), and the gradients of the step are clipped by their global norm.
Serving runs the first three on a handful of tokens.

``own`` chooses the side: False computes every operator from elementary torch
operations in 32 bits (64 where noted), True calls the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

E4M3, E5M2 = 0, 1
FP8 = (torch.float8_e4m3fn, torch.float8_e5m2)
FP8_MAX = (448.0, 57344.0)
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-5


# ----------------------------------------------------------------- cases --
def listed():
    return [
        # a batch of 8192 tokens sent to two of eight experts each: the E4M3
        # rows of fprop and the token-contiguous copy that wgrad reads
        dict(name="quantize_train", op="quantize", dtype="bf16", tokens=8192, topk=2, groups=8, cols=4096, fmt=E4M3,
             columns=True, skew=0.3),
        # one serving step of 37 sequences over 64 experts: rows only
        dict(name="quantize_serve", op="quantize", dtype="bf16", tokens=37, topk=6, groups=64, cols=2048, fmt=E4M3,
             columns=False, skew=0.5),
        # four sequences generating: eight rows, most experts idle or on one row
        dict(name="gemm_decode", op="gemm", fa=E4M3, fb=E4M3, rows=8, groups=8, n=14336, k=4096, out="bf16",
             skew=0.3),
        # the up projection of a training batch over eight large experts
        dict(name="gemm_fprop", op="gemm", fa=E4M3, fb=E4M3, rows=16384, groups=8, n=14336, k=4096, out="bf16",
             skew=0.3),
        # the gradient of the activations of 64 small experts, an odd number of
        # tokens spread unevenly
        dict(name="gemm_dgrad_fine", op="gemm", fa=E5M2, fb=E4M3, rows=24594, groups=64, n=2048, k=1408, out="bf16",
             skew=1.0),
        # weight gradients of eight large experts, fp32
        dict(name="wgrad_large", op="wgrad", fa=E5M2, fb=E4M3, rows=8192, groups=8, m=14336, n=4096, out="f32",
             skew=0.3),
        # weight gradients of 64 small experts, reduced over the replicas in bf16
        dict(name="wgrad_fine", op="wgrad", fa=E5M2, fb=E4M3, rows=24594, groups=64, m=1408, n=2048, out="bf16",
             skew=1.0),
        # one token of a generating sequence
        dict(name="layernorm_one", op="layernorm", dtype="bf16", params="bf16", rows=1, cols=4096),
        # odd sizes in fp32
        dict(name="layernorm_odd", op="layernorm", dtype="f32", params="f32", rows=2051, cols=5003),
        # the backward pass of a training batch, with the gradients of gain and bias
        dict(name="layernorm_backward", op="layernorm_backward", dtype="bf16", params="f32", rows=16384, cols=4096),
        # the fp32 gradients of eight experts with their router and norms
        dict(name="clip_experts", op="clip", dtype="f32", small="f32", big=8, rows=14336, cols=2048, little=20,
             width=4096, max_norm=1.0),
        # a small model's: many short bf16 tensors
        dict(name="clip_small", op="clip", dtype="bf16", small="f32", big=12, rows=255, cols=129, little=36, width=257,
             max_norm=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _blocks_of_128(rng, hi):
    """A multiple of 128 from 512 to about 128 hi (multiples of 24 blocks move up by one)."""
    n = _log(rng, 4, hi)
    return 128 * (n + 1 if n % 24 == 0 else n)


def draw(rng):
    op = rng.choice(["quantize", "quantize", "gemm", "gemm", "gemm", "wgrad", "wgrad", "layernorm",
                     "layernorm_backward", "clip"])
    most = {"quantize": work(listed()[0])["bytes"], "gemm": work(listed()[3])["flops"],
            "wgrad": work(listed()[5])["flops"], "layernorm": 4 * work(listed()[8])["bytes"],
            "layernorm_backward": work(listed()[9])["bytes"], "clip": work(listed()[10])["bytes"]}[op]
    while True:
        groups, skew = _log(rng, 1, 128), rng.choice([0.0, 0.3, 1.0])
        if op == "quantize":
            groups = max(groups, 2)
            case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), tokens=_log(rng, 1, 8192),
                        topk=rng.choice([1, 2, min(6, groups)]), groups=groups, cols=_blocks_of_128(rng, 56),
                        fmt=rng.choice([E4M3, E5M2]), columns=rng.choice([True, False]), skew=skew)
        elif op == "gemm":
            case = dict(op=op, fa=rng.choice([E4M3, E5M2]), fb=E4M3, rows=_log(rng, 1, 32768), groups=groups,
                        n=_blocks_of_128(rng, 112), k=_blocks_of_128(rng, 56), out="bf16", skew=skew)
            if case["groups"] * case["n"] * case["k"] > 8 * 14336 * 4096:
                continue
        elif op == "wgrad":
            case = dict(op=op, fa=E5M2, fb=E4M3, rows=_log(rng, 64, 32768), groups=groups, m=_blocks_of_128(rng, 112),
                        n=_blocks_of_128(rng, 56), out=rng.choice(["f32", "bf16"]), skew=skew)
            if case["groups"] * case["m"] * case["n"] > 8 * 14336 * 4096:
                continue
        elif op == "clip":
            case = dict(op=op, dtype=rng.choice(["bf16", "f32"]), small=rng.choice(["bf16", "f32"]),
                        big=rng.randint(1, 16), rows=_log(rng, 64, 14336), cols=_log(rng, 64, 4096),
                        little=rng.randint(0, 40), width=_log(rng, 1, 8192), max_norm=rng.choice([0.5, 1.0, 1e9]))
        else:
            case = dict(op=op, dtype=rng.choice(["bf16", "f32"]), params=rng.choice(["same", "f32"]),
                        rows=_log(rng, 1, 32768), cols=_log(rng, 64, 16384))
            if case["params"] == "same":
                case["params"] = case["dtype"]
        if 3072 in case.values():
            continue
        w = work(case)
        # no more than the largest listed case of its kind, in bytes and in operations
        if op in ("gemm", "wgrad"):
            big = work(listed()[3 if op == "gemm" else 5])
            if w["flops"] <= most and w["bytes"] <= big["bytes"]:
                return case
        elif w["bytes"] <= most:
            return case


def work(case):
    op = case["op"]
    if op == "quantize":
        t, d = case["tokens"] * case["topk"], case["cols"]
        codes = t * d + 4 * t * (d // 128)
        return {"bytes": min(t, case["tokens"]) * d * BYTES[case["dtype"]] + codes * (2 if case["columns"] else 1),
                "flops": 0}
    if op == "gemm":
        t, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
        live = min(g, t)  # an expert without rows is not read
        return {"bytes": t * k + live * n * k + t * n * BYTES[case["out"]], "flops": 2 * t * n * k}
    if op == "wgrad":
        t, g, m, n = case["rows"], case["groups"], case["m"], case["n"]
        return {"bytes": t * (m + n) + g * m * n * BYTES[case["out"]], "flops": 2 * t * m * n}
    if op == "clip":
        total = case["big"] * case["rows"] * case["cols"] * BYTES[case["dtype"]] + \
            case["little"] * case["width"] * BYTES[case["small"]]
        return {"bytes": 2 * total, "flops": 0}
    cells = case["rows"] * case["cols"]
    if op == "layernorm":
        return {"bytes": 2 * cells * BYTES[case["dtype"]] + 2 * case["cols"] * BYTES[case["params"]], "flops": 0}
    return {"bytes": 3 * cells * BYTES[case["dtype"]] + 3 * case["cols"] * BYTES[case["params"]], "flops": 0}


# ---------------------------------------------------------------- inputs --
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 11)


def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32) * std


def _routing(case, seed, tokens, topk):
    """Experts of each token: the router's logits, some experts liked more
    (skew), the topk largest.  Returns the token of each grouped row and the
    experts' row counts."""
    rng = np.random.default_rng(int(seed) + 1)
    groups = case["groups"]
    like = rng.standard_normal(groups) * case["skew"]
    score = like + rng.gumbel(size=(tokens, groups))
    expert = np.argsort(-score, axis=1)[:, :topk].reshape(-1)
    order = np.argsort(expert, kind="stable")
    return (order // topk).astype(np.int32), np.bincount(expert, minlength=groups)


def _offsets(sizes):
    return np.concatenate([[0], np.cumsum(sizes)])


def _padded(sizes):
    """Offsets of the groups in the token-contiguous copies: whole blocks of 128."""
    return _offsets((np.asarray(sizes) + 127) // 128 * 128)


def _blocks(x, fmt):
    """FP8 values and scales of blocks along the last axis of x [..., 128]."""
    s = x.abs().amax(-1, keepdim=True).clamp_min(1e-12) / FP8_MAX[fmt]
    return (x * (1.0 / s)).to(FP8[fmt]), s


def _codes(x, fmt):
    """1x128 blocks along the last axis of a 2-D tensor: codes and scales."""
    q, s = _blocks(x.view(x.shape[0], -1, 128), fmt)
    return q.view(torch.uint8).view(x.shape), s.squeeze(-1).contiguous()


def _weights(gen, groups, n, k, fmt):
    """Expert weights in 128x128 blocks: codes [groups][n][k], scales."""
    w = _normal(gen, groups, n // 128, 128, k // 128, 128, std=0.02)
    s = w.abs().amax((2, 4), keepdim=True) / FP8_MAX[fmt]
    q = (w * (1.0 / s)).to(FP8[fmt]).view(torch.uint8).view(groups, n, k)
    return q, s.view(groups, n // 128, k // 128).contiguous()


def _activations(gen, rows, cols, std=1.0):
    """Activations with a few heavy channels."""
    heavy = torch.ones(cols, device=DEV)
    heavy[torch.randint(0, cols, (max(1, cols // 100),), generator=gen, device=DEV)] = 8.0
    return _normal(gen, rows, cols, std=std) * heavy


def _padded_rows(x, sizes):
    """x's grouped rows at the padded offsets, zeros between."""
    pad, off = _padded(sizes), _offsets(sizes)
    at = np.concatenate([np.arange(n) + pad[g] for g, n in enumerate(sizes)] + [np.zeros(0, np.int64)])
    out = torch.zeros(max(int(pad[-1]), 128), x.shape[1], device=DEV)
    out[torch.from_numpy(at.astype(np.int64)).to(DEV)] = x[: int(off[-1])]
    return out


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    state = dict(case=case)
    if op == "quantize":
        index, sizes = _routing(case, seed, case["tokens"], case["topk"])
        t, d, tp = len(index), case["cols"], max(int(_padded(sizes)[-1]), 128)
        state.update(x=_activations(gen, case["tokens"], d).to(DT[case["dtype"]]),
                     index=torch.from_numpy(index).to(DEV),
                     offsets=torch.from_numpy(_offsets(sizes).astype(np.int32)).to(DEV),
                     q_row=torch.empty(t, d, dtype=torch.uint8, device=DEV),
                     s_row=torch.empty(t, d // 128, device=DEV))
        if case["columns"]:
            state.update(q_col=torch.empty(d, tp, dtype=torch.uint8, device=DEV),
                         s_col=torch.empty(d, tp // 128, device=DEV))
    elif op == "gemm":
        t, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
        _, sizes = _routing(case, seed, t, 1)
        state["sizes"] = [int(v) for v in sizes]
        state["offsets"] = torch.from_numpy(_offsets(sizes).astype(np.int32)).to(DEV)
        x = _activations(gen, t, k) if case["fa"] == E4M3 else _normal(gen, t, k, std=1e-3)
        state["a"], state["sa"] = _codes(x, case["fa"])
        state["b"], state["sb"] = _weights(gen, g, n, k, case["fb"])
        state["c"] = torch.empty(t, n, dtype=DT[case["out"]], device=DEV)
    elif op == "wgrad":
        t, g, m, n = case["rows"], case["groups"], case["m"], case["n"]
        _, sizes = _routing(case, seed, t, 1)
        state["sizes"] = [int(v) for v in sizes]
        state["offsets"] = torch.from_numpy(_offsets(sizes).astype(np.int32)).to(DEV)
        dy = _padded_rows(_normal(gen, t, m, std=1e-3), sizes)
        x = _padded_rows(_activations(gen, t, n), sizes)
        state["a"], state["sa"] = _codes(dy.t().contiguous(), case["fa"])
        state["b"], state["sb"] = _codes(x.t().contiguous(), case["fb"])
        state["c"] = torch.empty(g, m, n, dtype=DT[case["out"]], device=DEV)
    elif op == "clip":
        big = [_normal(gen, case["rows"], case["cols"], std=1e-3).to(DT[case["dtype"]]) for _ in range(case["big"])]
        little = [_normal(gen, case["width"], std=1e-2).to(DT[case["small"]]) for _ in range(case["little"])]
        state["grads"] = big + little
        state["out"] = [torch.empty_like(t) for t in state["grads"]]
        state["norm"], state["coef"] = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    else:
        r, c, dt, pt = case["rows"], case["cols"], DT[case["dtype"]], DT[case["params"]]
        state["x"] = (_activations(gen, r, c) + _normal(gen, c)).to(dt)
        state["gamma"] = (1.0 + _normal(gen, c, std=0.1)).to(pt)
        state["beta"] = _normal(gen, c, std=0.1).to(pt)
        state["mean"], state["rstd"] = torch.empty(r, device=DEV), torch.empty(r, device=DEV)
        if op == "layernorm":
            state["y"] = torch.empty_like(state["x"])
        else:
            x = state["x"].float()
            mean = x.mean(1)
            state["mean"] = mean
            state["rstd"] = torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS)
            state["dy"] = _normal(gen, r, c, std=1e-3).to(dt)
            state["dx"] = torch.empty_like(state["x"])
            state["dgamma"], state["dbeta"] = torch.empty_like(state["gamma"]), torch.empty_like(state["gamma"])
    if op == "layernorm_backward":
        # the workspace that a program keeps for its largest layer
        state["workspace"] = torch.empty(1 << 24, dtype=torch.float32, device=DEV)
    return state


# ----------------------------------------------------------- plain forms --
def _group_of(offsets, rows):
    """Group of each grouped row, its place in the group, and the padded offsets."""
    off = offsets.long()
    t = torch.arange(rows, device=DEV)
    g = torch.searchsorted(off[1:].contiguous(), t, right=True)
    padded = torch.cumsum((off[1:] - off[:-1] + 127) // 128 * 128, 0)
    padded = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), padded])
    return g, t - off[g], padded


def _plain_quantize(s):
    case, index = s["case"], s["index"].long()
    x = s["x"].float()[index]
    rows, cols = x.shape
    q, sc = _blocks(x.view(rows, cols // 128, 128), case["fmt"])
    out = dict(q_row=q.view(rows, cols), s_row=sc.squeeze(-1))
    if case["columns"]:
        g, place, padded = _group_of(s["offsets"], rows)
        tp = s["q_col"].shape[1]
        laid = torch.zeros(tp, cols, device=DEV)
        laid[padded[g] + place] = x
        q, sc = _blocks(laid.t().contiguous().view(cols, tp // 128, 128), case["fmt"])
        out.update(q_col=q.view(cols, tp), s_col=sc.squeeze(-1))
    return out


def _value(codes, fmt):
    return codes.view(FP8[fmt]).float()


def _plain_gemm(s):
    case = s["case"]
    groups, n, k = s["b"].shape
    rows = s["a"].shape[0]
    a = (_value(s["a"], case["fa"]).view(rows, k // 128, 128) * s["sa"][:, :, None]).view(rows, k)
    b = _value(s["b"], case["fb"]).view(groups, n // 128, 128, k // 128, 128)
    b = (b * s["sb"][:, :, None, :, None]).view(groups, n, k)
    # every group's rows in a batch of their largest size
    most = max(s["sizes"])
    g, place, _ = _group_of(s["offsets"], rows)
    batch = torch.zeros(groups * most, k, device=DEV)
    batch[g * most + place] = a
    c = torch.bmm(b, batch.view(groups, most, k).transpose(1, 2).contiguous())
    return c.transpose(1, 2).reshape(groups * most, n)[g * most + place].to(DT[case["out"]])


def _plain_wgrad(s):
    case = s["case"]
    tp, groups = s["a"].shape[1], case["groups"]
    a = (_value(s["a"], case["fa"]).view(-1, tp // 128, 128) * s["sa"][:, :, None]).view(-1, tp)
    b = (_value(s["b"], case["fb"]).view(-1, tp // 128, 128) * s["sb"][:, :, None]).view(-1, tp)
    _, _, padded = _group_of(s["offsets"], case["rows"])
    most = (max(s["sizes"]) + 127) // 128 * 128
    at = padded[:-1, None] + torch.arange(most, device=DEV)
    held = (at < padded[1:, None]).float()
    at = at.clamp_max(tp - 1).view(-1)
    a = a[:, at].view(-1, groups, most) * held
    b = b[:, at].view(-1, groups, most) * held
    return torch.bmm(a.permute(1, 0, 2).contiguous(), b.permute(1, 2, 0).contiguous()).to(DT[case["out"]])


def _plain_layernorm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt(xc.square().mean(1, keepdim=True) + EPS)
    y = xc * rstd * s["gamma"].float() + s["beta"].float()
    return dict(y=y.to(s["x"].dtype), mean=mean.view(-1), rstd=rstd.view(-1))


def _plain_layernorm_backward(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float()
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * rstd
    return dict(dx=dx.to(s["x"].dtype),
                dgamma=(dy * xh).sum(0).to(s["gamma"].dtype), dbeta=dy.sum(0).to(s["gamma"].dtype))


def _plain_clip(s):
    # squares summed in 64 bits: a long sum
    total = torch.stack([t.double().square().sum() for t in s["grads"]]).sum()
    norm = total.sqrt().float()
    coef = (s["case"]["max_norm"] / (norm + 1e-6)).clamp_max(1.0)
    return dict(out=[(t.float() * coef).to(t.dtype) for t in s["grads"]], norm=norm.view(1), coef=coef.view(1))


PLAIN = dict(quantize=_plain_quantize, gemm=_plain_gemm, wgrad=_plain_wgrad, layernorm=_plain_layernorm,
             layernorm_backward=_plain_layernorm_backward, clip=_plain_clip)


# --------------------------------------------------------- the library's --
def _own(s):
    import fp8_scaled_quantization_reduce_amd as fq

    case = s["case"]
    op = case["op"]
    if op == "quantize":
        fq.fp8_quantize_grouped(s["x"], s["offsets"], case["fmt"], row_index=s["index"], q_row=s["q_row"],
                                s_row=s["s_row"], q_col=s.get("q_col"), s_col=s.get("s_col"))
        out = dict(q_row=s["q_row"].view(FP8[case["fmt"]]), s_row=s["s_row"])
        if case["columns"]:
            out.update(q_col=s["q_col"].view(FP8[case["fmt"]]), s_col=s["s_col"])
        return out
    if op == "gemm":
        fq.fp8_grouped_gemm(s["a"], case["fa"], s["sa"], s["b"], case["fb"], s["sb"], s["offsets"], s["c"])
        return s["c"]
    if op == "wgrad":
        fq.fp8_grouped_gemm_wgrad(s["a"], case["fa"], s["sa"], s["b"], case["fb"], s["sb"], s["offsets"], s["c"])
        return s["c"]
    if op == "layernorm":
        fq.fp8q_layernorm(s["x"], s["gamma"], s["beta"], EPS, s["y"], s["mean"], s["rstd"])
        return dict(y=s["y"], mean=s["mean"], rstd=s["rstd"])
    if op == "layernorm_backward":
        fq.fp8q_layernorm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"],
                                   s["dbeta"], s["workspace"])
        return dict(dx=s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"])
    fq.fp8q_grad_norm_clip(s["grads"], case["max_norm"], s["norm"], s["coef"], out=s["out"])
    return dict(out=s["out"], norm=s["norm"], coef=s["coef"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------ in 64 bits --
def exact(case, seed):
    """The operators' definitions, group by group and in float64."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "quantize":
        # codes are whole values, compared as such; the scales are quotients
        x, fmax = s["x"].to(f64), FP8_MAX[case["fmt"]]
        rows = torch.stack([x[i] for i in s["index"].tolist()]) if len(s["index"]) < 64 else x[s["index"].long()]
        floor = float(np.float32(1e-12))
        blocks = rows.abs().reshape(rows.shape[0], -1, 128).max(2).values
        out = dict(q_row=None, s_row=blocks.clamp_min(floor) / fmax)
        if case["columns"]:
            off = s["offsets"].tolist()
            parts = []
            for a, b in zip(off, off[1:]):
                for first in range(a, b, 128):
                    parts.append(rows[first:min(first + 128, b)].abs().max(0).values)
            sc = torch.stack(parts, 1) if parts else torch.zeros(case["cols"], 1, dtype=f64, device=DEV)
            out.update(q_col=None, s_col=sc.clamp_min(floor) / fmax)
        return out
    if op == "gemm":
        off = s["offsets"].tolist()
        c = torch.zeros(case["rows"], case["n"], dtype=f64, device=DEV)
        for e in range(case["groups"]):
            if off[e + 1] > off[e]:
                a = s["a"][off[e]:off[e + 1]].view(FP8[case["fa"]]).to(f64)
                a = a * s["sa"][off[e]:off[e + 1]].to(f64).repeat_interleave(128, 1)
                w = s["b"][e].view(FP8[case["fb"]]).to(f64)
                w = w * s["sb"][e].to(f64).repeat_interleave(128, 0).repeat_interleave(128, 1)
                c[off[e]:off[e + 1]] = a @ w.t().contiguous()
        return c
    if op == "wgrad":
        pad = _padded(s["sizes"])
        c = torch.zeros(case["groups"], case["m"], case["n"], dtype=f64, device=DEV)
        for e in range(case["groups"]):
            lo, hi = int(pad[e]), int(pad[e + 1])
            if hi > lo:
                a = s["a"][:, lo:hi].view(FP8[case["fa"]]).to(f64)
                a = a * s["sa"][:, lo // 128:hi // 128].to(f64).repeat_interleave(128, 1)
                b = s["b"][:, lo:hi].view(FP8[case["fb"]]).to(f64)
                b = b * s["sb"][:, lo // 128:hi // 128].to(f64).repeat_interleave(128, 1)
                c[e] = a @ b.t().contiguous()
        return c
    if op == "clip":
        norm = math.sqrt(sum(float((t.to(f64) ** 2).sum()) for t in s["grads"]))
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        one = torch.ones(1, dtype=f64, device=DEV)
        return dict(out=[t.to(f64) * coef for t in s["grads"]], norm=one * norm, coef=one * coef)
    x, gamma = s["x"].to(f64), s["gamma"].to(f64)
    if op == "layernorm":
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = (x - mean[:, None]) * rstd[:, None] * gamma + s["beta"].to(f64)
        return dict(y=y, mean=mean, rstd=rstd)
    dy, mean, rstd = s["dy"].to(f64), s["mean"].to(f64)[:, None], s["rstd"].to(f64)[:, None]
    xh = (x - mean) * rstd
    n = case["cols"]
    g = dy * gamma
    dx = rstd / n * (n * g - g.sum(1, keepdim=True) - xh * (g * xh).sum(1, keepdim=True))
    return dict(dx=dx, dgamma=(dy * xh).sum(0), dbeta=dy.sum(0))
