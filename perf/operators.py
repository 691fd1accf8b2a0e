"""What is measured of the routed-expert layer's newer operators.

Three operators, as one layer of a served model runs them: the residual's
addition with the root-mean-square norm ahead of the layer (``op`` "norm"),
and the routed experts with 4-bit weights (``op`` "experts"), which for a few
tokens are matrix-vector products and for a prompt ragged products grouped by
expert.  4-bit weights are OCP MXFP4: E2M1 codes, two to a byte with the
earlier column in the low half, and one E8M0 scale for each 32 columns.
"""
import math

import numpy as np
import torch

own = False

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
GATHER_ROUTES = 64  # the plain form gathers the weights of each route up to here, and pads rows by expert above


def listed():
    return [
        # one decoded token ahead of its expert layer
        {"name": "norm_T1_d4096", "op": "norm", "T": 1, "d": 4096, "fp8": False, "wide": False},
        # the 401-token prompt, codes for the experts beside bf16 rows for the router
        {"name": "norm_T401_d4096_fp8", "op": "norm", "T": 401, "d": 4096, "fp8": True, "wide": False},
        # an odd row count and width, the residual kept in 32 bits
        {"name": "norm_T1999_d1416_wide", "op": "norm", "T": 1999, "d": 1416, "fp8": True, "wide": True},
        # a full prefill chunk
        {"name": "norm_T8192_d4096_fp8", "op": "norm", "T": 8192, "d": 4096, "fp8": True, "wide": False},
        # the smallest layer of the tests, one token: launches count
        {"name": "token_T1_d512_f256_E16", "op": "experts", "T": 1, "k": 6, "E": 16, "d": 512, "f": 256, "mask": 0.0, "bias": 0.0, "shared": False},
        # one decoded token, with the shared expert's rows
        {"name": "token_T1_d4096_f2048_E256", "op": "experts", "T": 1, "k": 6, "E": 256, "d": 4096, "f": 2048, "mask": 0.0, "bias": 0.0, "shared": True},
        # four sequences decoding together, some routes another owner's
        {"name": "token_T4_d4096_f2048_E256", "op": "experts", "T": 4, "k": 6, "E": 256, "d": 4096, "f": 2048, "mask": 0.05, "bias": 0.0, "shared": False},
        # a wider decode batch: about 135 experts with one or two rows
        {"name": "batch_T32_d4096_f2048_E256", "op": "experts", "T": 32, "k": 6, "E": 256, "d": 4096, "f": 2048, "mask": 0.05, "bias": 0.0, "shared": False},
        # odd: few experts, widths that fill no tile, many masked routes
        {"name": "odd_T777_d1152_f640_E24", "op": "experts", "T": 777, "k": 3, "E": 24, "d": 1152, "f": 640, "mask": 0.4, "bias": 0.5, "shared": True},
        # the 401-token prompt: every expert's weights for about nine rows each
        {"name": "prompt_T401_d4096_f2048_E256", "op": "experts", "T": 401, "k": 6, "E": 256, "d": 4096, "f": 2048, "mask": 0.05, "bias": 0.0, "shared": False},
        # 2048 tokens, a router with favourites
        {"name": "prompt_T2048_d4096_f2048_E256", "op": "experts", "T": 2048, "k": 6, "E": 256, "d": 4096, "f": 2048, "mask": 0.05, "bias": 0.5, "shared": False},
        # a full prefill chunk: about 190 rows an expert
        {"name": "prompt_T8192_d4096_f2048_E256", "op": "experts", "T": 8192, "k": 6, "E": 256, "d": 4096, "f": 2048, "mask": 0.05, "bias": 0.0, "shared": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.3:
        return {"op": "norm", "T": _log_int(rng, 1, 8192), "d": 8 * _log_int(rng, 16, 512), "fp8": rng.random() < 0.6, "wide": rng.random() < 0.4}
    # few tokens and prompts alike often
    T = _log_int(rng, 1, 10) if rng.random() < 0.4 else _log_int(rng, 11, 6000)
    E = _log_int(rng, 4, 256)
    return {"op": "experts", "T": T, "k": rng.randint(1, min(6, E)), "E": E, "d": 128 * rng.randint(4, 32), "f": 128 * rng.randint(2, 16),
            "mask": rng.choice([0.0, 0.05, 0.4]), "bias": rng.choice([0.0, 0.5]), "shared": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs


def _routing(case, seed):
    """ids, gates and mask of a softmax router over normal logits, on the host."""
    g = np.random.default_rng([seed, 17])
    T, k, E = case["T"], case["k"], case["E"]
    z = g.standard_normal((T, E)) + case["bias"] * g.standard_normal(E)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    p = np.exp(np.take_along_axis(z, ids, 1))
    return ids, (p / p.sum(1, keepdims=True)).astype(np.float32), (g.random((T, k)) >= case["mask"]).astype(np.uint8)


def _mxfp4_weights(gen, E, rows, cols):
    """Codes [E, rows, cols/2] and scales [E, rows, cols/32] of normal weights of deviation 0.02."""
    codes = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, rows, cols // 32, dtype=torch.uint8, device="cuda")
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    per = max(1, min(E, (1 << 27) // (rows * cols)))
    for e in range(0, E, per):
        n = min(per, E - e)
        w = torch.randn(n, rows, cols // 32, 32, generator=gen, device="cuda") * 0.02
        ex = torch.floor(torch.log2(w.abs().amax(-1, keepdim=True).clamp_min(1e-30))) - 2
        w /= torch.exp2(ex)
        c = torch.bucketize(w.abs(), mids, out_int32=True).to(torch.uint8) | (w < 0).to(torch.uint8) << 3
        c = c.view(n, rows, cols // 2, 2)
        codes[e:e + n] = c[..., 0] | c[..., 1] << 4
        scales[e:e + n] = (ex.view(n, rows, cols // 32) + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, d = case["T"], case["d"]
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    if case["op"] == "norm":
        # a residual stream with a few channels far larger than the rest
        res = torch.randn(T, d, generator=gen, device="cuda") * 2
        res[:, :: max(1, d // 4)] *= 50
        weight = 1 + 0.1 * torch.randn(d, generator=gen, device="cuda")
        return {"case": case, "x": x, "residual": res if case["wide"] else res.to(torch.bfloat16), "weight": weight.to(torch.bfloat16), "eps": 1e-6}
    k, E, f = case["k"], case["E"], case["f"]
    ids, gates, mask = _routing(case, seed)
    s = {"case": case, "x": x, "ids": torch.from_numpy(ids).cuda(), "gates": torch.from_numpy(gates).cuda(), "mask": torch.from_numpy(mask).cuda()}
    s["most"] = int(np.bincount(ids[mask != 0], minlength=E).max())  # the plan of the plain form: rows of the fullest expert
    s["pairs"] = torch.tensor([[v if c < 8 else -v for c in (b & 15, b >> 4) for v in (E2M1[c & 7],)] for b in range(256)], device="cuda")
    s["shared"] = torch.randn(T, d, generator=gen, device="cuda") if case["shared"] else None
    s["wg"], s["sg"] = _mxfp4_weights(gen, E, f, d)
    s["wu"], s["su"] = _mxfp4_weights(gen, E, f, d)
    s["wd"], s["sd"] = _mxfp4_weights(gen, E, d, f)
    if own:  # the layer object that a program keeps: it holds workspaces and outputs
        import routed_expert_prefill_amd as rep

        s["layer"] = rep.MoEPrefill(T, k, E, d, f, weights="mxfp4", out_dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if s["case"]["op"] == "norm":
        return _run_norm(s)
    if own:
        return s["layer"](s["x"], s["ids"], s["gates"], s["mask"], s["wg"], s["wu"], s["wd"], s["sg"], s["su"], s["sd"], shared=s["shared"])
    return _plain_experts(s)


def _run_norm(s):
    fp8 = s["case"]["fp8"]
    if own:
        import routed_expert_prefill_amd as rep

        y, res, q, sc = rep.add_rmsnorm(s["x"], s["weight"], eps=s["eps"], residual=s["residual"], want_fp8=fp8)
        return {"y": y, "residual": res, "q": q.view(torch.float8_e4m3fn), "s": sc} if fp8 else {"y": y, "residual": res}
    v = s["residual"].float() + s["x"].float()
    n = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    out = {"y": n.to(torch.bfloat16), "residual": v.to(s["residual"].dtype)}
    if fp8:
        top = n.abs().amax(-1)
        sc = torch.where(top == 0, torch.ones_like(top), top / 448)
        out["q"], out["s"] = (n / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), sc
    return out


def _weights(s, w, sc, which=None):
    """fp32 weights of MXFP4 codes and scales, of all experts or of the given ones."""
    w, sc = (s[w], s[sc]) if which is None else (s[w][which], s[sc][which])
    v = s["pairs"][w.int()].view(*sc.shape, 32) * (sc.int() << 23).view(torch.float32)[..., None]
    return v.view(*w.shape[:-1], -1)


def _plain_experts(s):
    ids, mask, x = s["ids"].view(-1), s["mask"].view(-1) != 0, s["x"].float()
    T, k, E, d = (s["case"][n] for n in ("T", "k", "E", "d"))
    token = torch.arange(T * k, device="cuda") // k
    if T * k <= GATHER_ROUTES:
        rows, which, at = x[token][:, None], ids, torch.arange(T * k, device="cuda")
    else:  # rows in the order of their experts, each expert's padded to the fullest one's
        key = torch.where(mask, ids, E).long()
        order = torch.argsort(key, stable=True)
        first = torch.searchsorted(key[order], torch.arange(E + 1, device="cuda"))
        rank = torch.empty_like(order)
        rank[order] = torch.arange(T * k, device="cuda") - first[key[order]]
        at = torch.where(mask, key * s["most"] + rank, E * s["most"])
        place = torch.zeros(E * s["most"] + 1, dtype=torch.long, device="cuda")
        place[at] = token
        rows, which = x[place[:-1]].view(E, s["most"], d), None
        at = at.clamp_max(E * s["most"] - 1)
    g = torch.bmm(rows, _weights(s, "wg", "sg", which).transpose(1, 2))
    u = torch.bmm(rows, _weights(s, "wu", "su", which).transpose(1, 2))
    y = torch.bmm(g / (1 + torch.exp(-g)) * u, _weights(s, "wd", "sd", which).transpose(1, 2))
    y = torch.where(mask[:, None], y.view(-1, d)[at] * s["gates"].view(-1, 1), 0.0)
    out = y.view(T, k, d).sum(1)
    return (out if s["shared"] is None else out + s["shared"]).to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without, and its value in 64 bits


def work(case):
    T, d = case["T"], case["d"]
    if case["op"] == "norm":
        wide = 4 if case["wide"] else 2
        return {"bytes": T * d * (2 + wide + wide + 2 + (1 if case["fp8"] else 0)) + 2 * d + (4 * T if case["fp8"] else 0), "flops": 6 * T * d}
    ids, _, mask = _routing(case, 0)
    active = ids[mask != 0]
    used, rows, f = len(np.unique(active)), len(active), case["f"]
    return {"bytes": used * 3 * d * f * (1 / 2 + 1 / 32) + T * d * (2 + 2 + (4 if case["shared"] else 0)) + ids.size * 9, "flops": rows * 6 * d * f}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        v = s["x"].double() + s["residual"].double()
        n = v / torch.sqrt(v.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].double()
        out = {"y": n, "residual": v}
        if case["fp8"]:
            top = n.abs().amax(-1, keepdim=True)
            sc = torch.where(top == 0, torch.ones_like(top), top / 448)
            # to the nearest of 8 steps a power of two, 2^-9 at the least
            q = n / sc
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
            out["q"], out["s"] = torch.round(q / step) * step, sc.view(-1)
        return out
    T, k, E, d = (case[n] for n in ("T", "k", "E", "d"))
    value = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device="cuda")

    def weight(name, e):
        c, sc = s["w" + name][e], s["s" + name][e]
        v = torch.stack([value[(c & 15).long()], value[(c >> 4).long()]], -1).view(c.shape[0], -1, 32)
        return (v * torch.exp2(sc.double() - 127)[..., None]).view(c.shape[0], -1)

    out = torch.zeros(T, d, dtype=torch.float64, device="cuda") if s["shared"] is None else s["shared"].double()
    x, active = s["x"].double(), s["mask"] != 0
    for e in torch.unique(s["ids"][active]).tolist():
        t, j = torch.nonzero((s["ids"] == e) & active, as_tuple=True)
        g, u = x[t] @ weight("g", e).T, x[t] @ weight("u", e).T
        out.index_add_(0, t, (g * torch.sigmoid(g) * u) @ weight("d", e).T * s["gates"][t, j].double()[:, None])
    return out
