"""What is measured of the operators that a served layer has beside its routed experts.

Four operators: the selection of experts from router logits (``op`` "route":
sigmoid or softmax scores, a bias for balance, groups, renormalised gates), the
quantisation of rows to E4M3 with one scale for each block of 128 columns (``op``
"quant"), the product with 8-bit weights that have one scale for each block of
128 x 128 (``op`` "product"), and the shared expert, a gated feed-forward layer of
such products (``op`` "shared").
"""
import math

import torch

own = False


def _route(name, T, E, k, scores, groups=1, top=1, bias=True, bf16=False, out=0, renorm=True):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "scores": scores, "groups": groups, "top": top, "bias": bias, "bf16": bf16, "out": out, "renorm": renorm}


def listed():
    return [
        # one decoded token of a model whose 256 experts are chosen by groups
        _route("route_T1_E256", 1, 256, 6, "sigmoid", groups=8, top=4),
        # an odd batch, few experts, plain softmax gates, logits as a bf16 product leaves them, one expert out of service
        _route("route_T777_E24_softmax", 777, 24, 3, "softmax", bias=False, bf16=True, out=1, renorm=False),
        # a full prefill chunk
        _route("route_T8192_E256", 8192, 256, 6, "sigmoid", groups=8, top=4),
        # one decoded token's row
        {"name": "quant_T1_d4096", "op": "quant", "T": 1, "d": 4096, "wide": False},
        # a full chunk's rows
        {"name": "quant_T8192_d4096", "op": "quant", "T": 8192, "d": 4096, "wide": False},
        # one decoded token through a dense projection
        {"name": "product_M1_N4096_K4096", "op": "product", "M": 1, "N": 4096, "K": 4096, "codes": False, "wide": False},
        # a decode batch, rows quantised already, 32-bit sums for a residual
        {"name": "product_M32_N2048_K4096", "op": "product", "M": 32, "N": 2048, "K": 4096, "codes": True, "wide": True},
        # odd: rows and columns that fill no tile
        {"name": "product_M777_N1416_K1152", "op": "product", "M": 777, "N": 1416, "K": 1152, "codes": False, "wide": True},
        # a full chunk
        {"name": "product_M8192_N4096_K4096", "op": "product", "M": 8192, "N": 4096, "K": 4096, "codes": True, "wide": False},
        # the shared expert for one decoded token, for the 401-token prompt and for a full chunk
        {"name": "shared_T1_d4096_f2048", "op": "shared", "T": 1, "d": 4096, "f": 2048, "codes": False},
        {"name": "shared_T401_d4096_f2048", "op": "shared", "T": 401, "d": 4096, "f": 2048, "codes": False},
        {"name": "shared_T8192_d4096_f2048", "op": "shared", "T": 8192, "d": 4096, "f": 2048, "codes": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, T = rng.choice(["route", "quant", "product", "product", "shared", "shared"]), _log_int(rng, 1, 8192)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        per = _log_int(rng, 8, 256 // groups)
        top = rng.randint(1, groups)
        case = _route("", T, groups * per, rng.randint(1, min(8, top * per)), rng.choice(["sigmoid", "softmax"]), groups, top,
                      rng.random() < 0.6, rng.random() < 0.3, rng.choice([0, 0, 1, 5]), rng.random() < 0.7)
        del case["name"]
        return case
    if op == "quant":
        return {"op": op, "T": T, "d": 128 * rng.randint(1, 32), "wide": rng.random() < 0.4}
    if op == "product":
        return {"op": op, "M": T, "N": _log_int(rng, 64, 4096), "K": 128 * rng.randint(1, 32), "codes": rng.random() < 0.5, "wide": rng.random() < 0.5}
    return {"op": op, "T": T, "d": 128 * rng.randint(4, 32), "f": 128 * rng.randint(2, 16), "codes": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def _weights(gen, N, K):
    """E4M3 codes [N, K] of normal weights of deviation 0.02 and fp32 scales [ceil(N / 128), K / 128], blocks of unequal size."""
    nb = -(-N // 128)
    z = torch.randn(nb, 128, K // 128, 128, generator=gen, device="cuda") * torch.exp(0.5 * torch.randn(nb, 1, K // 128, 1, generator=gen, device="cuda"))
    s = 0.02 * z.abs().amax((1, 3), keepdim=True) / 448
    q = (0.02 * z / s).to(torch.float8_e4m3fn).view(torch.uint8).view(nb * 128, K)[:N].contiguous()
    return q, s.view(nb, K // 128)


def _rows(gen, T, d):
    """Normed rows with a few channels far larger than the rest."""
    x = torch.randn(T, d, generator=gen, device="cuda")
    x[:, :: max(1, d // 4)] *= 20
    return x


def _codes(x):
    """E4M3 values and scales of rows, block by block."""
    v = x.float().view(x.shape[0], -1, 128)
    top = v.abs().amax(-1, keepdim=True)
    s = torch.where(top == 0, 1.0, top / torch.full_like(top, 448))  # a quotient: by a number torch would multiply with the inverse
    return (v / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(x.shape), s.squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        z = torch.randn(T, E, generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
        z[:, torch.randperm(E, generator=gen, device="cuda")[: min(case["out"], E // case["groups"] - 1)]] = -math.inf
        s["logits"] = z.to(torch.bfloat16) if case["bf16"] else z
        s["bias"] = 0.1 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
        s["scale"] = 2.5 if case["renorm"] else 1.0
    elif case["op"] == "quant":
        x = _rows(gen, case["T"], case["d"])
        s["x"] = x if case["wide"] else x.to(torch.bfloat16)
    else:
        d, f = (case["K"], case["N"]) if case["op"] == "product" else (case["d"], case["f"])
        s["x"] = _rows(gen, case["M"] if case["op"] == "product" else case["T"], d).to(torch.bfloat16)
        if case["codes"]:
            q, sc = _codes(s["x"])
            s["x"] = (q.view(torch.uint8), sc)
        s["w"] = [_weights(gen, f, d)] if case["op"] == "product" else [_weights(gen, f, d), _weights(gen, f, d), _weights(gen, d, f)]
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    c = s["case"]
    if own:
        import routed_expert_prefill_amd as rep

        if c["op"] == "route":
            return rep.route_select(s["logits"], c["k"], scores=c["scores"], bias=s["bias"], groups=c["groups"], top_groups=c["top"], renormalise=c["renorm"], scale=s["scale"])
        if c["op"] == "quant":
            q, sc = rep.quant_blocks_fp8(s["x"])
            return q.view(torch.float8_e4m3fn), sc
        if c["op"] == "product":
            return rep.matmul_fp8(s["x"], *s["w"][0], out_dtype=torch.float32 if c["wide"] else torch.bfloat16)
        (wg, sg), (wu, su), (wd, sd) = s["w"]
        # bf16 rows: one code of h that falls the other way is more than 32 bits hide
        return rep.shared_ffn(s["x"], wg, wu, wd, sg, su, sd, out_dtype=torch.bfloat16)
    if c["op"] == "route":
        return _plain_route(s)
    if c["op"] == "quant":
        return _codes(s["x"])
    x = _values(*((s["x"][0].view(torch.float8_e4m3fn), s["x"][1]) if c["codes"] else _codes(s["x"])))
    if c["op"] == "product":
        return (x @ _matrix(*s["w"][0]).T).to(torch.float32 if c["wide"] else torch.bfloat16)
    g, u = x @ _matrix(*s["w"][0]).T, x @ _matrix(*s["w"][1]).T
    return (_values(*_codes(g / (1 + torch.exp(-g)) * u)) @ _matrix(*s["w"][2]).T).to(torch.bfloat16)


def _values(q, s):
    return (q.float().view(*s.shape, 128) * s[..., None]).view(q.shape)


def _matrix(q, s):
    wide = s.repeat_interleave(128, 0)[: q.shape[0]]
    return (q.view(torch.float8_e4m3fn).float().view(*wide.shape, 128) * wide[..., None]).view(q.shape)


def _plain_route(s):
    c = s["case"]
    z, k, G = s["logits"].double(), c["k"], c["groups"]  # 64 bits: neighbours in the order may lie close
    gone = z == -math.inf
    e = torch.exp(z - z.amax(-1, keepdim=True))
    score = torch.where(gone, 0.0, e / e.sum(-1, keepdim=True) if c["scores"] == "softmax" else 1 / (1 + torch.exp(-z)))
    choice = torch.where(gone, -math.inf, score if s["bias"] is None else score + s["bias"].double())
    if G > 1:
        # a group counts with its two largest choices
        two = choice.view(-1, G, c["E"] // G).topk(2, -1).values
        of_group = torch.where(two[..., 1] == -math.inf, two[..., 0], two.sum(-1))
        kept = torch.sort(of_group, dim=-1, descending=True, stable=True).indices[:, : c["top"]]
        keep = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(keep.repeat_interleave(c["E"] // G, 1), choice, -math.inf)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :k]
    # a route beyond the experts that are left weighs nothing
    w = torch.where(choice.gather(1, ids) == -math.inf, 0.0, score.gather(1, ids))
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    return ids.int(), (w * s["scale"]).float()


# ------------------------------------------------------------------ what a pass cannot do without, and its value in 64 bits


def work(case):
    if case["op"] == "route":
        n = case["T"] * case["E"]
        return {"bytes": n * (2 if case["bf16"] else 4) + (4 * case["E"] if case["bias"] else 0) + 8 * case["T"] * case["k"], "flops": 20 * n}
    if case["op"] == "quant":
        n = case["T"] * case["d"]
        return {"bytes": n * (4 if case["wide"] else 2) + n + n // 32, "flops": 4 * n}
    x_bytes = 1 + 1 / 32 if case["codes"] else 2
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * x_bytes + N * K + 4 * -(-N // 128) * (K // 128) + M * N * (4 if case["wide"] else 2), "flops": 2 * M * N * K}
    T, d, f = case["T"], case["d"], case["f"]
    return {"bytes": T * d * (x_bytes + 2) + 3 * d * f * (1 + 4 / 128 ** 2), "flops": 6 * T * d * f}


def _nearest(v):
    """Nearest E4M3 value, ties to even, of values in 64 bits: 8 steps to a power of two, 2^-9 at the least, 448 at the most."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _blocks_exact(x, narrow):
    """Values of codes and scales by their definition; narrow: scale and quotient are 32-bit numbers by definition, as the inputs are."""
    v = x.double().view(x.shape[0], -1, 128)
    top = v.abs().amax(-1)
    s = top / 448
    s[top == 0] = 1
    if narrow:
        s = s.float().double()
    t = v / s[..., None]
    return _nearest(t.float().double() if narrow else t), s


def _product_exact(q, s, w, ws):
    """Block after block of the columns, in 64 bits; q [M, blocks, 128]."""
    out = torch.zeros(q.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    wv = w.view(torch.float8_e4m3fn).double()
    of_row = torch.arange(w.shape[0], device="cuda") // 128
    for b in range(q.shape[1]):
        out += (q[:, b] @ wv[:, 128 * b:128 * (b + 1)].T) * s[:, b, None] * ws.double()[of_row, b]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _route_exact(s)
    if case["op"] == "quant":
        q, sc = _blocks_exact(s["x"], True)
        return q.view(s["x"].shape), sc
    if case["codes"]:
        q, sc = s["x"]
        q, sc = q.view(torch.float8_e4m3fn).double().view(*sc.shape, 128), sc.double()
    else:
        q, sc = _blocks_exact(s["x"], True)
    first = _product_exact(q, sc, *s["w"][0])
    if case["op"] == "product":
        return first
    h = first * torch.sigmoid(first) * _product_exact(q, sc, *s["w"][1])
    return _product_exact(*_blocks_exact(h, False), *s["w"][2])


def _route_exact(s):
    """Expert by expert in the order of the choice, on the host."""
    import numpy as np

    c = s["case"]
    z = s["logits"].double().cpu().numpy()
    T, E = z.shape
    with np.errstate(over="ignore"):
        p = np.exp(z - z.max(1, keepdims=True))
        score = p / p.sum(1, keepdims=True) if c["scores"] == "softmax" else 1 / (1 + np.exp(-z))
    score[np.isneginf(z)] = 0
    choice = score + (0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    choice[np.isneginf(z)] = -np.inf
    G = c["groups"]
    if G > 1:
        best = -np.sort(-choice.reshape(T, G, E // G), axis=2)[:, :, :2]
        best[..., 1][np.isneginf(best[..., 1])] = 0
        order = np.argsort(-best.sum(2), axis=1, kind="stable")
        for j in range(c["top"], G):
            choice.reshape(T, G, E // G)[np.arange(T), order[:, j]] = -np.inf
    ids = np.argsort(-choice, axis=1, kind="stable")[:, :c["k"]]
    w = np.where(np.isneginf(np.take_along_axis(choice, ids, 1)), 0, np.take_along_axis(score, ids, 1))
    if c["renorm"]:
        w = w / np.maximum(w.sum(1, keepdims=True), np.finfo(np.float64).tiny)
    return torch.from_numpy(ids.astype(np.int32)), torch.from_numpy(w * s["scale"])
