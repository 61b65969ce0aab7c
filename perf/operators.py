"""The layer operators next to the codec, as measured work: residual add + layer / RMS norm, linear layers
with a fused epilogue, and the gated feed-forward block, each forward and backward.

Shapes are one tensor-parallel rank's share of a layer: `rows` tokens, `hidden` channels of the activation
that travels between layers, `width` the rank's share of the feed-forward width."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one new token of one sequence: the residual add and norm between two layers, latency alone
        dict(name="norm_token", op="norm", rows=1, hidden=8192, kind="layer", dtype="fp16", residual=True),
        # GPT-style micro-batch (2 x 4096 tokens): residual add + layer norm after the all-reduce
        dict(name="norm_gpt", op="norm", rows=8192, hidden=4096, kind="layer", dtype="bf16", residual=True),
        # a ragged batch in single precision, hidden size away from powers of two
        dict(name="norm_bwd_ragged", op="norm_bwd", rows=1021, hidden=1000, kind="layer", dtype="fp32", residual=False),
        # Qwen-style training step: RMS norm's backward with the gradient that arrives through the residual
        dict(name="norm_bwd_qwen", op="norm_bwd", rows=8192, hidden=5120, kind="rms", dtype="bf16", residual=True),
        # one new token through a row-parallel down projection (8 ranks), residual added in the epilogue
        dict(name="linear_token", op="linear", rows=1, hidden=8192, width=3584, down=True, act="none", bias=False,
             residual=True, dtype="fp16"),
        # GPT-style row-parallel output of one of 8 ranks: bias and residual in the epilogue
        dict(name="linear_gpt", op="linear", rows=8192, hidden=4096, width=2048, down=True, act="none", bias=True,
             residual=True, dtype="bf16"),
        # a short ragged batch trained through a column-parallel layer with GELU, sizes off every tile
        dict(name="linear_bwd_ragged", op="linear_bwd", rows=1021, hidden=1000, width=1096, down=False,
             act="gelu_erf", bias=True, dtype="fp16"),
        # GPT-style column-parallel layer with GELU, training step of one of 8 ranks
        dict(name="linear_bwd_gpt", op="linear_bwd", rows=8192, hidden=4096, width=2048, down=False, act="gelu_tanh",
             bias=True, dtype="bf16"),
        # a small decoding batch (one token of each of 6 sequences) through a Qwen-style gated block, 4 ranks
        dict(name="ffn_tokens", op="ffn", rows=6, hidden=5120, width=3456, act="silu", dtype="bf16"),
        # prefill of 8192 tokens through the gated block that feeds a down projection, 8 ranks
        dict(name="ffn_prefill", op="ffn", rows=8192, hidden=8192, width=3584, act="silu", dtype="fp16"),
        # one short sequence trained through a small gated block with GELU
        dict(name="ffn_bwd_short", op="ffn_bwd", rows=300, hidden=1024, width=344, act="gelu_erf", dtype="fp16"),
        # Qwen-style training step of the gated block on one of 4 ranks: the largest work here
        dict(name="ffn_bwd_qwen", op="ffn_bwd", rows=8192, hidden=5120, width=3456, act="silu", dtype="bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_bwd", "linear", "linear_bwd", "ffn", "ffn_bwd"])
    c = dict(op=op, rows=spread(1, 8192))
    if op in ("norm", "norm_bwd"):
        # norms take any number of channels
        c.update(hidden=spread(250, 8192), kind=rng.choice(["layer", "rms"]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                 residual=rng.random() < 0.7)
        return c
    # products read 16-byte vectors along the channels: sizes in steps of 8
    c.update(hidden=8 * spread(32, 1024), width=8 * spread(16, 448), dtype=rng.choice(["bf16", "fp16"]))
    if op in ("ffn", "ffn_bwd"):
        c["act"] = rng.choice(["silu", "gelu_tanh", "gelu_erf"])
    else:
        c.update(down=rng.random() < 0.5, act=rng.choice(["none", "none", "relu", "gelu_tanh", "gelu_erf", "silu"]),
                 bias=rng.random() < 0.5)
        if op == "linear":
            c["residual"] = rng.random() < 0.5
        elif c["act"] == "relu":
            # a pre-activation within rounding of zero turns one row's whole term of the bias gradient on or off
            c["bias"] = False
    most = work(listed()[-1])["flops"]
    if work(c)["flops"] > most:
        c["rows"] = max(1, int(c["rows"] * most / work(c)["flops"]))
    return c


def _sizes(case):
    """(n_out, n_in) of a linear case: the down projection ends in `hidden`, the others start from it."""
    return (case["hidden"], case["width"]) if case["down"] else (case["width"], case["hidden"])


def work(case):
    R, H, op = case["rows"], case["hidden"], case["op"]
    es = 4 if case["dtype"] == "fp32" else 2
    if op == "norm":
        t = 4 if case["residual"] else 2
        layer = case["kind"] == "layer"
        return {"bytes": t * R * H * es + (2 if layer else 1) * (H * es + R * 4), "flops": 8.0 * R * H}
    if op == "norm_bwd":
        t = 4 if case["residual"] else 3
        layer = case["kind"] == "layer"
        return {"bytes": t * R * H * es + H * es + (2 if layer else 1) * (H * 4 + R * 4), "flops": 12.0 * R * H}
    if op == "linear":
        N, K = _sizes(case)
        b = (R * K + N * K + R * N) * es + (N * es if case["bias"] else 0) + (R * N * es if case["residual"] else 0)
        return {"bytes": b, "flops": 2.0 * R * N * K}
    if op == "linear_bwd":
        N, K = _sizes(case)
        b = (R * N + 2 * R * K + 2 * N * K) * es + (N * es + N * 4 if case["bias"] else 0)
        # with an activation the pre-activation is a product of its own
        return {"bytes": b, "flops": (4.0 if case["act"] == "none" else 6.0) * R * N * K}
    F = case["width"]
    if op == "ffn":
        return {"bytes": (R * H + 2 * F * H + R * F) * es, "flops": 4.0 * R * F * H}
    return {"bytes": (R * F + 2 * R * H + 4 * F * H) * es, "flops": 12.0 * R * F * H}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]
    R, H, op = case["rows"], case["hidden"], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    def empty(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        layer = case["kind"] == "layer"
        gain = torch.ones(H, device="cuda")
        gain[torch.randperm(H, generator=gen, device="cuda")[: max(1, H // 200)]] = 20.0   # outlier channels
        s["gamma"] = (1.0 + normal(H, std=0.1)).to(dt)
        if op == "norm":
            s["x"] = (normal(R, H, std=0.5) * gain + 0.1).to(dt)
            s["residual"] = normal(R, H).to(dt) if case["residual"] else None
            s["beta"] = normal(H, std=0.1).to(dt) if layer else None
            s["y"] = empty(R, H)
            s["sum"] = empty(R, H) if case["residual"] else None
            s["mean"] = empty(R, dtype=torch.float32) if layer else None
            s["rstd"] = empty(R, dtype=torch.float32)
        else:
            s["x"] = (normal(R, H) * gain + 0.1).to(dt)
            s["dy"] = normal(R, H, std=1e-2).to(dt)
            s["dsum"] = normal(R, H, std=1e-2).to(dt) if case["residual"] else None
            x = s["x"].float()
            s["mean"] = x.mean(1) if layer else None   # what the forward pass kept
            c = x - s["mean"][:, None] if layer else x
            s["rstd"] = torch.rsqrt((c * c).mean(1) + EPS)
            s["dx"] = empty(R, H)
            s["dgamma"] = empty(H, dtype=torch.float32)
            s["dbeta"] = empty(H, dtype=torch.float32) if layer else None
    elif op in ("linear", "linear_bwd"):
        N, K = _sizes(case)
        s["x"] = normal(R, K).to(dt)
        s["w"] = normal(N, K, std=K ** -0.5).to(dt)
        s["bias"] = normal(N, std=0.1).to(dt) if case["bias"] else None
        if op == "linear":
            s["residual"] = normal(R, N).to(dt) if case["residual"] else None
            s["y"] = empty(R, N)
        else:
            s["dy"] = normal(R, N, std=1e-2).to(dt)
            s["dx"], s["dw"] = empty(R, K), empty(N, K)
            s["dbias"] = empty(N, dtype=torch.float32) if case["bias"] else None
    else:
        F = case["width"]
        s["x"] = normal(R, H).to(dt)
        s["wg"] = normal(F, H, std=H ** -0.5).to(dt)
        s["wu"] = normal(F, H, std=H ** -0.5).to(dt)
        if op == "ffn":
            s["h"] = empty(R, F)
        else:
            s["dh"] = normal(R, F, std=1e-2).to(dt)
            s["dx"], s["dwg"], s["dwu"] = empty(R, H), empty(F, H), empty(F, H)
    return s


def run(state):
    return (_own if own else _plain)(state)


# ---------------------------------------------------------------- the plain forms
def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_erf":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu_erf":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    k = (2.0 / math.pi) ** 0.5
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DT[case["dtype"]]
    f = {k: v.float() for k, v in s.items() if torch.is_tensor(v)}
    layer = case.get("kind") == "layer"
    if op == "norm":
        t = f["x"] + f["residual"] if case["residual"] else f["x"]
        mean = t.mean(1) if layer else None
        c = t - mean[:, None] if layer else t
        rstd = 1.0 / torch.sqrt((c * c).mean(1) + EPS)
        y = c * rstd[:, None] * f["gamma"]
        y = y + f["beta"] if layer else y
        return {"y": y.to(dt), "sum": t.to(dt) if case["residual"] else None, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        xh = (f["x"] - f["mean"][:, None] if layer else f["x"]) * f["rstd"][:, None]
        t = f["dy"] * f["gamma"]
        d = t - xh * (t * xh).mean(1, keepdim=True)
        d = d - t.mean(1, keepdim=True) if layer else d
        d = d * f["rstd"][:, None]
        d = d + f["dsum"] if case["residual"] else d
        return {"dx": d.to(dt), "dgamma": (f["dy"] * xh).sum(0), "dbeta": f["dy"].sum(0) if layer else None}
    if op in ("linear", "linear_bwd"):
        z = None
        if op == "linear" or case["act"] != "none":
            z = f["x"] @ f["w"].T
            z = z + f["bias"] if case["bias"] else z
        if op == "linear":
            y = _act(z, case["act"])
            y = y + f["residual"] if case["residual"] else y
            return {"y": y.to(dt)}
        dz = f["dy"] if case["act"] == "none" else f["dy"] * _act_grad(z, case["act"])
        return {"dx": (dz @ f["w"]).to(dt), "dw": (dz.T @ f["x"]).to(dt), "dbias": dz.sum(0) if case["bias"] else None}
    g, u = f["x"] @ f["wg"].T, f["x"] @ f["wu"].T
    if op == "ffn":
        return {"h": (_act(g, case["act"]) * u).to(dt)}
    du = f["dh"] * _act(g, case["act"])
    dg = f["dh"] * u * _act_grad(g, case["act"])
    return {"dx": (dg @ f["wg"] + du @ f["wu"]).to(dt), "dwg": (dg.T @ f["x"]).to(dt), "dwu": (du.T @ f["x"]).to(dt)}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import quantized_tensor_activation_gb300 as qta

    case = s["case"]
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        d = qta.norm_desc(case["rows"], case["hidden"], case["dtype"], kind=case["kind"], eps=EPS)
        if op == "norm":
            qta.qta_norm(d, s["x"], s["gamma"], s["y"], beta=s["beta"], residual=s["residual"], sum_out=s["sum"],
                         mean=s["mean"], rstd=s["rstd"])
            return {"y": s["y"], "sum": s["sum"], "mean": s["mean"], "rstd": s["rstd"]}
        if "ws" not in s:   # a training program keeps its workspace
            s["ws"] = qta.alloc_workspace(qta.norm_bwd_workspace_bytes(d))
        qta.qta_norm_bwd(d, s["dy"], s["x"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], s["ws"], mean=s["mean"],
                         dbeta=s["dbeta"], dsum=s["dsum"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op in ("linear", "linear_bwd"):
        N, K = _sizes(case)
        d = qta.linear_desc(case["rows"], N, K, case["dtype"], act=case["act"])
        if op == "linear":
            qta.qta_linear(d, s["x"], s["w"], s["y"], bias=s["bias"], residual=s["residual"])
            return {"y": s["y"]}
        if "ws" not in s:
            s["ws"] = qta.alloc_workspace(qta.linear_bwd_workspace_bytes(d))
        qta.qta_linear_bwd(d, s["dy"], s["x"], s["w"], s["dx"], s["dw"], s["ws"], bias=s["bias"], dbias=s["dbias"])
        return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}
    d = qta.ffn_desc(case["rows"], case["hidden"], case["width"], case["dtype"], act=case["act"])
    if op == "ffn":
        qta.qta_gated_ffn(d, s["x"], s["wg"], s["wu"], s["h"])
        return {"h": s["h"]}
    if "ws" not in s:
        s["ws"] = qta.alloc_workspace(qta.gated_ffn_bwd_workspace_bytes(d))
    qta.qta_gated_ffn_bwd(d, s["dh"], s["x"], s["wg"], s["wu"], s["dx"], s["dwg"], s["dwu"], s["ws"])
    return {"dx": s["dx"], "dwg": s["dwg"], "dwu": s["dwu"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v)}
    op, act = case["op"], case.get("act")

    if op == "norm":
        a = d["x"] if d.get("residual") is None else d["x"] + d["residual"]
        if case["kind"] == "layer":
            var, mean = torch.var_mean(a, dim=1, correction=0)
            rstd = (var + EPS).rsqrt()
            y = torch.addcmul(d["beta"], (a - mean.unsqueeze(1)) * rstd.unsqueeze(1), d["gamma"])
        else:
            mean, rstd = None, (a.pow(2).mean(dim=1) + EPS).rsqrt()
            y = a * rstd.unsqueeze(1) * d["gamma"]
        return {"y": y, "sum": a if "residual" in d else None, "mean": mean, "rstd": rstd}

    if op == "norm_bwd":
        # y_j = gamma_j (x_j - m) r with r = (mean (x - m)^2 + eps)^(-1/2): the vector-Jacobian product of a row is
        # r [ t - <t> - xh <t xh> ], <.> the mean over the channels (without <t> where m = 0 by definition)
        r = d["rstd"].unsqueeze(1)
        centred = d["x"] - d["mean"].unsqueeze(1) if "mean" in d else d["x"]
        xh = centred * r
        t = d["gamma"] * d["dy"]
        H = case["hidden"]
        dx = r * (t - xh * ((t * xh).sum(dim=1, keepdim=True) / H))
        if "mean" in d:
            dx = dx - r * (t.sum(dim=1, keepdim=True) / H)
        if "dsum" in d:
            dx = dx + d["dsum"]
        return {"dx": dx, "dgamma": torch.einsum("rh,rh->h", d["dy"], xh),
                "dbeta": d["dy"].sum(dim=0) if "mean" in d else None}

    def fun(z):   # value and derivative
        if act == "none":
            return z, z * 0 + 1
        if act == "relu":
            return z.clamp(min=0), z.gt(0).double()
        if act == "silu":
            p = torch.sigmoid(z)
            return z * p, p + z * p * (1 - p)
        if act == "gelu_erf":   # z Phi(z), Phi + z phi
            Phi = torch.special.ndtr(z)
            return z * Phi, Phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        a, b = math.sqrt(2 / math.pi), 0.044715   # z sigmoid(2 q), q = a (z + b z^3)
        p = torch.sigmoid(2 * a * (z + b * z ** 3))
        return z * p, p + z * p * (1 - p) * 2 * a * (1 + 3 * b * z * z)

    if op in ("linear", "linear_bwd"):
        z = torch.einsum("rk,nk->rn", d["x"], d["w"])
        if "bias" in d:
            z = z + d["bias"]
        v, dv = fun(z)
        if op == "linear":
            return {"y": v + d["residual"] if "residual" in d else v}
        dz = d["dy"] * dv
        return {"dx": torch.einsum("rn,nk->rk", dz, d["w"]), "dw": torch.einsum("rn,rk->nk", dz, d["x"]),
                "dbias": dz.sum(dim=0) if "bias" in d else None}
    g = torch.einsum("rk,nk->rn", d["x"], d["wg"])
    u = torch.einsum("rk,nk->rn", d["x"], d["wu"])
    v, dv = fun(g)
    if op == "ffn":
        return {"h": v * u}
    dg, du = d["dh"] * u * dv, d["dh"] * v
    return {"dx": torch.einsum("rn,nk->rk", dg, d["wg"]) + torch.einsum("rn,nk->rk", du, d["wu"]),
            "dwg": torch.einsum("rn,rk->nk", dg, d["x"]), "dwu": torch.einsum("rn,rk->nk", du, d["x"])}
