"""The operators of the expert layer's training step, as cases to be measured:
products grouped by expert (forward, input gradient, weight gradient), the
SwiGLU with its activations kept in 8 bits for the backward pass, and the
movement of rows between token order and expert order.

`run` computes a case in plain torch operations (`own` false) or by the
framework's entry points (`own` true); `exact` computes it in 64 bits.
"""
import math

import torch

own = False

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ----------------------------------------------------------------- cases --
# T tokens choose K of E experts each (zipf: skew of the experts' popularity,
# 0 = even), which gives T*K rows in expert order.  `slack` rows behind the
# last expert belong to nobody and stay as they were.  N and C are an expert's
# output and input features, F its intermediate width, H the hidden width.
def listed():
    return [
        # one new token of the 64-expert model through its gate/up projections: latency of one call
        dict(name="mm_ocr_T1", op="mm", T=1, K=6, E=64, zipf=0.0, slack=0, N=1792, C=1280, out="bf16"),
        # a training batch on one of eight ranks of the 256-expert model, skewed experts
        dict(name="mm_dsv3_rank_T2048", op="mm", T=2048, K=8, E=32, zipf=1.1, slack=0, N=4096, C=7168, out="bf16"),
        # gradient into the intermediate, an odd number of tokens in a buffer with room to spare, kept in fp32
        dict(name="dgrad_ocr_down_T2047", op="dgrad", T=2047, K=6, E=64, zipf=0.0, slack=100, N=1280, C=896, out="fp32"),
        # gradient into the hidden rows of the rank's gate/up projections
        dict(name="dgrad_dsv3_rank_T2048", op="dgrad", T=2048, K=8, E=32, zipf=0.0, slack=0, N=4096, C=7168, out="bf16"),
        # weight gradient of all 64 experts, about 192 rows each
        dict(name="wgrad_ocr_T2048", op="wgrad", T=2048, K=6, E=64, zipf=0.0, slack=0, N=1792, C=1280, out="bf16", base=False),
        # a second micro-batch's weight gradient added to the first's in fp32, skewed experts
        dict(name="wgrad_dsv3_down_base", op="wgrad", T=2048, K=8, E=32, zipf=1.1, slack=0, N=7168, C=2048, out="fp32", base=True),
        # forward activation with the checkpoint written, a prompt of 2048 tokens
        dict(name="ckpt_ocr_T2048", op="ckpt", rows=12288, slack=0, F=896, weights=True),
        # the same at the largest batch of the 256-expert shape
        dict(name="ckpt_dsv3_T8192", op="ckpt", rows=65536, slack=0, F=2048, weights=True),
        # backward from the checkpoint: a few tokens (latency), then the largest batch
        dict(name="ckpt_bwd_ocr_T16", op="ckpt_bwd", rows=96, slack=32, F=896, weights=True),
        dict(name="ckpt_bwd_dsv3_T8192", op="ckpt_bwd", rows=65536, slack=0, F=2048, weights=True),
        # hidden rows kept in 8 bits, restored into expert order for the weight gradient
        dict(name="permute_fp8_dsv3_T2047", op="permute", T=2047, K=8, E=256, zipf=1.1, H=7168, fp8=True, dropped=0.0),
        # expert rows summed back to the tokens with the residual, and the router weights' gradient
        dict(name="unpermute_ocr_T2048", op="unpermute", T=2048, K=6, E=64, zipf=0.0, H=1280, y="bf16", residual=True, dropped=0.02),
    ]


_MOST = None   # cost of the largest listed case


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["mm", "dgrad", "wgrad", "ckpt", "ckpt_bwd", "permute", "unpermute"])
    if op in ("ckpt", "ckpt_bwd"):
        return dict(op=op, rows=_log_int(rng, 1, 65536), slack=rng.choice([0, 0, 1, 77]),
                    F=128 * _log_int(rng, 1, 32), weights=rng.random() < 0.7)
    E = _log_int(rng, 1, 256)
    c = dict(op=op, T=_log_int(rng, 1, 8192), K=rng.randint(1, min(8, E)), E=E,
             zipf=rng.choice([0.0, 0.0, 1.1]))
    if op == "permute":
        fp8 = rng.random() < 0.5
        return dict(c, H=128 * _log_int(rng, 1, 64) if fp8 else 8 * _log_int(rng, 8, 1024), fp8=fp8,
                    dropped=rng.choice([0.0, 0.1]))
    if op == "unpermute":
        return dict(c, H=8 * _log_int(rng, 8, 1024), y=rng.choice(["bf16", "fp32"]),
                    residual=rng.random() < 0.5, dropped=rng.choice([0.0, 0.1]))
    c.update(slack=rng.choice([0, 0, 1, 100]), N=8 * _log_int(rng, 8, 896), C=8 * _log_int(rng, 8, 896),
             out=rng.choice(["bf16", "fp32"]))
    if op == "wgrad":
        c["base"] = c["out"] == "fp32" and rng.random() < 0.5
    return c


def draw(rng):
    global _MOST
    if _MOST is None:
        _MOST = max(_cost(c) for c in listed())
    while True:
        c = _draw(rng)
        if _cost(c) <= _MOST:
            return c


def _touched(case):
    """Expected number of experts with at least one row."""
    E, K, T = case["E"], case["K"], case["T"]
    p = [(e + 1) ** -case["zipf"] for e in range(E)]
    s = sum(p)
    return sum(1.0 - (1.0 - min(1.0, K * v / s)) ** T for v in p)


def work(case):
    op = case["op"]
    if op in ("mm", "dgrad", "wgrad"):
        R, N, C, E = case["T"] * case["K"], case["N"], case["C"], case["E"]
        ob = 2 if case["out"] == "bf16" else 4
        flops = 2.0 * R * N * C
        if op == "wgrad":
            return {"bytes": 2.0 * R * (N + C) + E * N * C * ob * (2 if case["base"] else 1), "flops": flops}
        i, o = (C, N) if op == "mm" else (N, C)
        return {"bytes": 2.0 * R * i + 2.0 * _touched(case) * N * C + ob * R * o, "flops": flops}
    if op == "ckpt":      # gate and up in; h, two codes and their scales out
        R, F = case["rows"], case["F"]
        return {"bytes": R * (4.0 * F + 2 * F + 2 * F + 8 * (F // 128) + 4), "flops": 12.0 * R * F}
    if op == "ckpt_bwd":  # codes, scales and the gradient in; both gradients, h and the row's dot product out
        R, F = case["rows"], case["F"]
        return {"bytes": R * (2.0 * F + 8 * (F // 128) + 2 * F + 4 * F + 2 * F + 8), "flops": 24.0 * R * F}
    T, K, H = case["T"], case["K"], case["H"]
    if op == "permute":
        src = T * (H + 4 * (H // 128)) if case["fp8"] else 2 * T * H
        return {"bytes": src + 2.0 * T * K * H + 12.0 * T * K, "flops": 1.0 * T * K * H}
    yb = 2 if case["y"] == "bf16" else 4
    return {"bytes": yb * T * K * H + 2.0 * T * H * (2 if case["residual"] else 1) + 12.0 * T * K,
            "flops": 1.0 * T * K * H}


# ---------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=BF, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _routing(g, case):
    """[T,K] expert ids, best first, of softmax routing on random logits."""
    T, K, E = case["T"], case["K"], case["E"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    if case["zipf"]:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1
        logits = logits - case["zipf"] * rank.log()
    return torch.topk(logits, K, dim=1).indices


def _expert_order(idx, E):
    """offsets [E+1] and the position in expert order of each slot; ids outside [0,E) have none (-1)."""
    flat = idx.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    inv = torch.empty_like(order)
    inv[order] = torch.arange(order.numel(), device=order.device)
    inv = torch.where(key < E, inv, torch.full_like(inv, -1))
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, inv.to(torch.int32).view(idx.shape)


def _to_e4m3(v):
    """Codes and power-of-two scales per 128 values: the smallest 2^k that keeps max/2^k within 448."""
    blk = v.float().reshape(*v.shape[:-1], v.shape[-1] // 128, 128)
    amax = blk.abs().amax(-1)
    k = torch.where(amax > 0, torch.ceil(torch.log2(amax.double().clamp_min(1e-300) / 448)), torch.zeros_like(amax).double())
    k = k.clamp(-127, 127)
    codes = (blk.double() * torch.exp2(-k).unsqueeze(-1)).float().to(F8)
    return codes.reshape(v.shape), torch.exp2(k).float()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("mm", "dgrad", "wgrad"):
        E, N, C = case["E"], case["N"], case["C"]
        offsets, _ = _expert_order(_routing(g, case), E)
        rows = case["T"] * case["K"] + case["slack"]
        s["offsets"] = offsets
        ends = offsets.tolist()
        s["groups"] = [(e, ends[e], ends[e + 1]) for e in range(E)]   # known on the host to the plain form only
        dt = BF if case["out"] == "bf16" else F32
        if op in ("mm", "wgrad"):
            s["x"] = _randn(g, rows, C)
        if op in ("dgrad", "wgrad"):
            s["dy"] = _randn(g, rows, N, std=0.1)
        if op in ("mm", "dgrad"):
            s["w"] = _randn(g, E, N, C, std=0.02)
            s["out"] = torch.zeros(rows, N if op == "mm" else C, dtype=dt, device="cuda")
        else:
            s["base"] = _randn(g, E, N, C, dtype=F32) if case["base"] else None
            s["out"] = torch.zeros(E, N, C, dtype=dt, device="cuda")
        s["workspace"] = torch.zeros(8192, dtype=torch.uint8, device="cuda")
        return s
    if op in ("ckpt", "ckpt_bwd"):
        R, F = case["rows"], case["F"]
        total = R + case["slack"]
        gu = _randn(g, total, 2 * F, std=1.2)
        s["weights"] = torch.rand(total, generator=g, device="cuda") if case["weights"] else None
        s["n_rows"] = torch.tensor([R], dtype=torch.int32, device="cuda") if case["slack"] else None
        s["h"] = torch.zeros(total, F, dtype=BF, device="cuda")
        if op == "ckpt":
            s["gate_up"] = gu
            s["codes"] = torch.zeros(total, 2 * F, dtype=torch.uint8, device="cuda")
            s["scale"] = torch.zeros(total, 2 * F // 128, device="cuda")
        else:
            s["codes"], s["scale"] = _to_e4m3(gu)
            s["dh"] = _randn(g, total, F, std=0.1)
            s["dgate_up"] = torch.zeros(total, 2 * F, dtype=BF, device="cuda")
            s["dweights"] = torch.zeros(total, device="cuda")
        return s
    T, K, E, H = case["T"], case["K"], case["E"], case["H"]
    idx = _routing(g, case)
    if case["dropped"]:   # slots sent to no expert of this layer (another rank's, or over capacity)
        idx = torch.where(torch.rand(T, K, generator=g, device="cuda") < case["dropped"], torch.full_like(idx, -1), idx)
    _, s["inv"] = _expert_order(idx, E)
    if op == "permute":
        x = _randn(g, T, H)
        s["x"], s["x_scale"] = _to_e4m3(x) if case["fp8"] else (x, None)
        s["weights"] = torch.rand(T, K, generator=g, device="cuda")
        s["out"] = torch.zeros(T * K, H, dtype=BF, device="cuda")
        s["row_weights"] = torch.zeros(T * K, device="cuda")
    else:
        s["y"] = _randn(g, T * K, H, dtype=BF if case["y"] == "bf16" else F32)
        s["residual"] = _randn(g, T, H) if case["residual"] else None
        s["drow"] = _randn(g, T * K, dtype=F32)
    return s


# ------------------------------------------------------------------- run --
def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import mixture_experts_routed_expert_b200 as moe
    op = s["op"]
    if op == "mm":
        return moe.moe_grouped_mm(s["x"], s["offsets"], s["w"], out=s["out"], workspace=s["workspace"])
    if op == "dgrad":
        return moe.moe_grouped_mm_dgrad(s["dy"], s["offsets"], s["w"], out=s["out"], workspace=s["workspace"])
    if op == "wgrad":
        return moe.moe_grouped_mm_wgrad(s["dy"], s["x"], s["offsets"], base=s["base"], out=s["out"],
                                        workspace=s["workspace"])
    if op == "ckpt":
        h, codes, scale = moe.moe_swiglu_checkpoint(s["gate_up"], row_weights=s["weights"], n_rows=s["n_rows"],
                                                    h=s["h"], codes=s["codes"], scale=s["scale"])
        return h, codes.view(F8), scale
    if op == "ckpt_bwd":
        return moe.moe_swiglu_checkpoint_backward(s["codes"], s["scale"], s["dh"], row_weights=s["weights"],
                                                  n_rows=s["n_rows"], dgate_up=s["dgate_up"], h=s["h"],
                                                  drow_weights=s["dweights"])
    if op == "permute":
        return moe.moe_permute_rows(s["x"], s["inv"], top_k_weights=s["weights"], x_scale=s["x_scale"],
                                    out=s["out"], row_weights=s["row_weights"])
    return moe.moe_unpermute_rows(s["y"], s["inv"], residual=s["residual"], drow_weights=s["drow"])


# The grouped products go expert by expert, one matrix product each: a batch
# padded to the longest expert would multiply several times the rows.
def _plain_mm(s):
    for e, a, b in s["groups"]:
        if b > a:
            s["out"][a:b] = s["x"][a:b].float() @ s["w"][e].float().t()
    return s["out"]


def _plain_dgrad(s):
    for e, a, b in s["groups"]:
        if b > a:
            s["out"][a:b] = s["dy"][a:b].float() @ s["w"][e].float()
    return s["out"]


def _plain_wgrad(s):
    for e, a, b in s["groups"]:
        d = s["dy"][a:b].float().t() @ s["x"][a:b].float()   # zeros for an expert without rows
        s["out"][e] = d if s["base"] is None else s["base"][e] + d
    return s["out"]


def _plain_ckpt(s):
    R, F = s["case"]["rows"], s["case"]["F"]
    v = s["gate_up"][:R].float()
    gate, up = v[:, :F], v[:, F:]
    h = gate / (1 + torch.exp(-gate)) * up
    if s["weights"] is not None:
        h = h * s["weights"][:R, None]
    s["h"][:R] = h
    codes, s["scale"][:R] = _to_e4m3(s["gate_up"][:R])
    s["codes"][:R] = codes.view(torch.uint8)
    return s["h"], s["codes"].view(F8), s["scale"]


def _plain_ckpt_bwd(s):
    R, F = s["case"]["rows"], s["case"]["F"]
    v = (s["codes"][:R].float().view(R, -1, 128) * s["scale"][:R, :, None]).view(R, 2 * F)
    gate, up, dh = v[:, :F], v[:, F:], s["dh"][:R].float()
    sig = 1 / (1 + torch.exp(-gate))
    h = gate * sig * up
    s["dweights"][:R] = (dh * h).sum(1)
    if s["weights"] is not None:
        h, dh = h * s["weights"][:R, None], dh * s["weights"][:R, None]
    s["h"][:R] = h
    s["dgate_up"][:R, :F] = dh * up * (sig * (1 + gate * (1 - sig)))
    s["dgate_up"][:R, F:] = dh * gate * sig
    return s["dgate_up"], s["h"], s["dweights"]


def _plain_permute(s):
    T, K, H = s["case"]["T"], s["case"]["K"], s["case"]["H"]
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = (x.view(T, -1, 128) * s["x_scale"][:, :, None]).view(T, H)
    at = s["inv"].reshape(-1).long()
    kept = at >= 0
    slots = torch.arange(T * K, device=at.device)[kept]
    s["out"][at[kept]] = x.to(BF)[slots // K]
    s["row_weights"][at[kept]] = s["weights"].reshape(-1)[slots]
    return s["out"], s["row_weights"]


def _plain_unpermute(s):
    inv = s["inv"].long()
    kept = inv >= 0
    rows = s["y"].float()[inv.clamp_min(0)] * kept[:, :, None]
    out = rows.sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(BF), s["drow"][inv.clamp_min(0)] * kept


_PLAIN = {"mm": _plain_mm, "dgrad": _plain_dgrad, "wgrad": _plain_wgrad, "ckpt": _plain_ckpt,
          "ckpt_bwd": _plain_ckpt_bwd, "permute": _plain_permute, "unpermute": _plain_unpermute}


# ----------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[s["op"]](s, case)


def _exact_products(s, case):
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    if s["op"] == "wgrad" and s["base"] is not None:
        out += s["base"]
    bounds = s["offsets"].long()
    for e in torch.nonzero(bounds[1:] > bounds[:-1]).flatten().tolist():
        r = slice(int(bounds[e]), int(bounds[e + 1]))
        if s["op"] == "mm":
            out[r] = torch.einsum("rc,nc->rn", s["x"][r].double(), s["w"][e].double())
        elif s["op"] == "dgrad":
            out[r] = torch.einsum("rn,nc->rc", s["dy"][r].double(), s["w"][e].double())
        else:
            out[e] += torch.einsum("rn,rc->nc", s["dy"][r].double(), s["x"][r].double())
    return out


def _e4m3_nearest(v):
    """The E4M3 value nearest to each |v| <= 448 (ties to the even mantissa), in 64 bits."""
    m, e = torch.frexp(v)                                   # |m| in [0.5, 1)
    step = torch.exp2((e - 4).clamp_min(-9).double())       # three bits below the leading one; 2^-9 below the normals
    return torch.round(v / step) * step


def _exact_ckpt(s, case):
    R, F = case["rows"], case["F"]
    h = torch.zeros(s["h"].shape, dtype=torch.float64, device="cuda")
    codes = torch.zeros(s["codes"].shape, dtype=torch.float64, device="cuda")
    scale = torch.zeros(s["scale"].shape, dtype=torch.float64, device="cuda")
    for a in range(0, R, 8192):
        r = slice(a, min(R, a + 8192))
        v = s["gate_up"][r].double()
        g, u = v.split(F, 1)
        w = 1.0 if s["weights"] is None else s["weights"][r].double()[:, None]
        h[r] = w * (g * torch.sigmoid(g)) * u
        blk = v.unflatten(1, (-1, 128))
        m, e = torch.frexp(blk.abs().amax(2))               # max = m 2^e; 448 = 0.875 * 2^9
        k = torch.where(m == 0, torch.zeros_like(e), e - 9 + (m > 0.875)).clamp(-127, 127)
        scale[r] = torch.exp2(k.double())
        codes[r] = _e4m3_nearest(blk / scale[r][:, :, None]).flatten(1)
    return h, codes, scale


def _exact_ckpt_bwd(s, case):
    R, F = case["rows"], case["F"]
    dgu = torch.zeros(s["dgate_up"].shape, dtype=torch.float64, device="cuda")
    h = torch.zeros(s["h"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["dweights"].shape, dtype=torch.float64, device="cuda")
    for a in range(0, R, 8192):
        r = slice(a, min(R, a + 8192))
        v = s["codes"][r].double().unflatten(1, (-1, 128)) * s["scale"][r].double().unsqueeze(2)
        g, u = v.flatten(1).split(F, 1)
        w = torch.ones(1, 1, dtype=torch.float64, device="cuda") if s["weights"] is None else s["weights"][r].double()[:, None]
        p = torch.sigmoid(g)
        a_, d = g * p, s["dh"][r].double()
        dw[r] = torch.einsum("rf,rf->r", d, a_ * u)
        h[r] = w * a_ * u
        dgu[r] = torch.cat([w * d * u * (p + a_ * torch.sigmoid(-g)), w * d * a_], 1)
    return dgu, h, dw


def _exact_permute(s, case):
    T, K, H = case["T"], case["K"], case["H"]
    out = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    rw = torch.zeros(T * K, dtype=torch.float64, device="cuda")
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double().repeat_interleave(128, 1)
    for k in range(K):
        p = s["inv"][:, k].long()
        t = torch.nonzero(p >= 0).flatten()
        out.index_copy_(0, p[t], x[t])
        rw.index_copy_(0, p[t], s["weights"][t, k].double())
    return out, rw


def _exact_unpermute(s, case):
    T, K, H = case["T"], case["K"], case["H"]
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda") if s["residual"] is None else s["residual"].double()
    dw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for k in range(K):
        p = s["inv"][:, k].long()
        t = torch.nonzero(p >= 0).flatten()
        out.index_add_(0, t, s["y"][p[t]].double())
        dw[t, k] = s["drow"][p[t]].double()
    return out, dw


_EXACT = {"mm": _exact_products, "dgrad": _exact_products, "wgrad": _exact_products, "ckpt": _exact_ckpt,
          "ckpt_bwd": _exact_ckpt_bwd, "permute": _exact_permute, "unpermute": _exact_unpermute}
