"""A decoder block of experts served in FP8, as it is measured: routing of tokens to experts, the experts' products over
ragged rows (up with SwiGLU and a quantized output, down in bf16), and the residual norm around the block (gated sum of the
experts' rows, residual, RMSNorm, FP8 codes for the next product).

Each case is one call. `run` computes it in plain torch operations, or with the library's kernels where `own` is set.
FP8: E4M3 codes with one fp32 scale per row and 128 columns (activations) or per 128 x 128 block (weights);
value = code value * scale, scale = max(amax, 1e-12) / 448.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
FLT_MAX = 3.4028234663852886e38


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One user, one token: the router's latency alone.
        dict(name="route_token", op="route", T=1, E=64, k=8, score="softmax", renorm=True, bias=False, G=1, top=1, best=1, dtype="f32", pad=0),
        # A decode step of a fixed size of 77 rows, 13 of them padding: sigmoid scores, a balancing bias, groups of experts.
        dict(name="route_batch", op="route", T=77, E=256, k=8, score="sigmoid", renorm=True, bias=True, G=8, top=4, best=2, dtype="bf16", pad=13),
        # A long prompt: 16 thousand tokens.
        dict(name="route_prompt", op="route", T=16384, E=128, k=8, score="softmax", renorm=True, bias=False, G=1, top=1, best=1, dtype="f32", pad=0),
        # The same with the balancing bias and groups.
        dict(name="route_prompt_groups", op="route", T=8000, E=256, k=8, score="sigmoid", renorm=True, bias=True, G=8, top=4, best=2, dtype="f32", pad=0),
        # Up projections of one token: eight experts' weights are read, for one row each.
        dict(name="up_token", op="up", T=1, E=64, k=8, H=2048, I=1024, skew=0.0),
        # Up projections of a decode batch: all experts, about eight rows each, some with many.
        dict(name="up_batch", op="up", T=64, E=64, k=8, H=2048, I=1024, skew=0.7),
        # Up projections of a long prompt.
        dict(name="up_prompt", op="up", T=8192, E=64, k=8, H=2048, I=1024, skew=0.3),
        # Down projections of an odd batch.
        dict(name="down_batch", op="down", T=77, E=64, k=8, H=2048, I=1024, skew=0.7),
        # Down projections of a prompt with few large experts (the MLP shape of this repository's prefill workload).
        dict(name="down_prompt", op="down", T=4001, E=8, k=2, H=4096, I=14336, skew=0.3),
        # The norm in front of a block, one token: attention's output into the residual, codes for the next product.
        dict(name="norm_token", op="norm", T=1, H=4096, k=0, post=False, alpha=1.0, dtype="bf16"),
        # A prompt's experts gathered by their gates into the residual, and the next block's norm.
        dict(name="norm_experts_prompt", op="norm", T=8192, H=2048, k=8, post=False, alpha=1.0, dtype="bf16"),
        # A prompt through a block with norms on both sides and a scaled residual, kept in fp32.
        dict(name="norm_both_prompt", op="norm", T=5000, H=4096, k=0, post=True, alpha=0.22, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "up", "down", "norm"])
    if kind == "route":
        E = rng.choice([8, 16, 40, 60, 64, 96, 128, 160, 256, 384])
        G = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
        top = rng.randint(1, G)
        k = min(rng.choice([1, 2, 4, 6, 8]), top * (E // G))
        T = _log(rng, 1, 16384)
        return dict(op="route", T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), renorm=rng.choice([True, False]),
                    bias=rng.choice([True, False]), G=G, top=top, best=min(E // G, rng.choice([1, 2])),
                    dtype=rng.choice(["f32", "bf16"]), pad=rng.choice([0, T // 5]))
    if kind == "norm":
        k = rng.choice([0, 1, 2, 4, 8])
        H = 128 * _log(rng, 1, 64)
        return dict(op="norm", T=_log(rng, 1, max(1, min(16384, (1 << 27) // (H * max(1, k))))), H=H, k=k, post=rng.choice([True, False]),
                    alpha=rng.choice([1.0, 0.5]), dtype=rng.choice(["bf16", "f32"]))
    E = rng.choice([4, 8, 16, 32, 64, 128])
    k = min(rng.choice([1, 2, 4, 6, 8]), E)
    H, I = 128 * _log(rng, 2, 32), 128 * _log(rng, 1, 32)
    while E * H * I > 1.2e8:
        H, I = max(128, H // 256 * 128), max(128, I // 256 * 128)
    T = _log(rng, 1, max(1, min(8192, int(4e11 / (4.0 * k * H * I)))))
    return dict(op=kind, T=T, E=E, k=k, H=H, I=I, skew=rng.choice([0.0, 0.3, 0.7]))


def _used(c):
    """Experts that have rows, as expected of tokens that choose k of E."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])


def work(c):
    T, op = c["T"], c["op"]
    if op == "route":
        n = T * c["E"]
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + 16 * T * c["k"] + 4 * c["E"] * (2 if c["bias"] else 1) + 4, "flops": 8 * n}
    if op == "norm":
        n, size = T * c["H"], 2 if c["dtype"] == "bf16" else 4
        rows = n * max(1, c["k"])
        gammas = c["H"] * size * (2 if c["post"] else 1)
        return {"bytes": 2 * n * size + 2 * rows + 2 * n + n + n // 32 + 8 * T * c["k"] + gammas, "flops": 2 * rows + 8 * n}
    R, H, I = T * c["k"], c["H"], c["I"]
    if op == "up":
        return {"bytes": _used(c) * 2 * I * H * (1 + 4 / 16384) + T * H * (1 + 4 / 128) + 4 * R + R * I * (1 + 4 / 128),
                "flops": 4 * R * H * I}
    return {"bytes": _used(c) * I * H * (1 + 4 / 16384) + R * I * (1 + 4 / 128) + 2 * R * H, "flops": 2 * R * H * I}


# ------------------------------------------------------------------ inputs

def _over_448(amax):
    """The scale of an amax: a division of tensors, since one by a Python number multiplies by its reciprocal."""
    return amax.clamp(min=1e-12) / torch.full_like(amax, 448.0)


def _quantize_rows(x):
    """Codes and scales of the last dimension's groups of 128."""
    g = x.unflatten(-1, (-1, 128))
    s = _over_448(g.abs().amax(dim=-1))
    return (g / s[..., None]).clamp(-448, 448).to(F8).flatten(-2), s


def _weights(E, N, K, g):
    """E weights [N, K] in 128 x 128 blocks: codes and scales."""
    w = torch.randn((E, N // 128, 128, K // 128, 128), generator=g, device="cuda").mul_(0.02)
    s = _over_448(w.abs().amax(dim=(2, 4)))
    codes = w.div_(s[:, :, None, :, None]).clamp_(-448, 448).to(F8).view(torch.uint8)
    return codes.view(E, N, K), s


def _plan(ids, E):
    """Rows by expert, within an expert by token: offsets [E + 1], row_token [T k], token_row [T, k]; ids of -1 have no row."""
    T, k = ids.shape
    flat = torch.where(ids >= 0, ids, E).reshape(-1).long()
    order = torch.sort(flat, stable=True)[1]
    count = torch.zeros(E + 1, dtype=torch.long, device="cuda").index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.zeros(E + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum(count[:E], 0)
    at = torch.arange(T * k, device="cuda")
    row_token = torch.where(at < offsets[E], order // k, -1)
    token_row = torch.empty_like(at).scatter_(0, order, at)
    token_row = torch.where(flat < E, token_row, -1).view(T, k)
    return offsets.to(torch.int32), row_token.to(torch.int32), token_row.to(torch.int32)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    T, op = c["T"], c["op"]
    st = dict(case=c)
    if op == "route":
        logits = randn(T, c["E"]) * 1.5 + 0.5 * randn(1, c["E"])
        st["logits"] = logits.to(torch.bfloat16) if c["dtype"] == "bf16" else logits
        st["bias"] = 0.05 * randn(c["E"]) if c["bias"] else None
        st["n"] = torch.tensor([T - c["pad"]], dtype=torch.int32, device="cuda") if c["pad"] else None
        return st
    if op == "norm":
        H, k = c["H"], c["k"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        big = torch.ones(H, device="cuda")
        big[:: max(1, H // 20)] = 20.0                         # a few channels of a residual stream are far larger than the others
        st["x"] = (randn(T, H) * big).to(dt)
        st["gamma"] = (1.0 + 0.1 * randn(H)).to(dt)
        st["gamma_y"] = (1.0 + 0.1 * randn(H)).to(dt) if c["post"] else None
        rows = T * max(1, k)
        st["y"] = randn(rows, H).to(torch.bfloat16)
        st["rows"] = st["gates"] = None
        if k:
            rank = torch.randperm(rows, generator=g, device="cuda").view(T, k)     # every token's rows lie somewhere else
            st["rows"] = rank.to(torch.int32)
            st["gates"] = torch.softmax(randn(T, k), dim=1)
        return st
    E, k, H, I = c["E"], c["k"], c["H"], c["I"]
    likes = randn(T, E) + c["skew"] * randn(1, E)              # some experts are liked by many tokens
    ids = torch.topk(likes, k, dim=1)[1]
    st["offsets"], row_token, _ = _plan(ids, E)
    st["most"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
    if op == "up":
        x = randn(T, H)
        x[:, :: max(1, H // 20)] *= 20.0
        st["row_token"] = row_token
        st["w"], st["ws"] = _weights(E, 2 * I, H, g)           # gate rows, then up rows
    else:
        x = randn(T * k, I)
        st["row_token"] = None                                 # the rows lie in the experts' order already
        st["w"], st["ws"] = _weights(E, H, I, g)
    a, st["as"] = _quantize_rows(x)
    st["a"] = a.view(torch.uint8)
    return st


# ------------------------------------------------------------------ the plain forms

def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    l = s["logits"].double()
    l = torch.where(torch.isnan(l), -math.inf, l).clamp(max=FLT_MAX)
    if s["n"] is not None:
        l = torch.where(torch.arange(T, device="cuda")[:, None] < s["n"], l, -math.inf)
    if c["score"] == "softmax":
        m = l.amax(dim=1, keepdim=True).clamp(min=-FLT_MAX)
        p = torch.exp(l - m)
        p = p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
        logp = l - m
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
        logp = torch.where(l < 0, l, 0.0) - torch.log1p(torch.exp(-l.abs()))
    rank, key, closed = l, p, l == -math.inf
    if s["bias"] is not None:
        b = s["bias"].double()
        rank = key = p + torch.where(torch.isnan(b), -math.inf, b)
        closed = closed | (key == -math.inf)
    rank = torch.where(closed, -math.inf, rank)
    if G > 1:
        best = torch.sort(torch.where(closed, -math.inf, key).view(T, G, E // G), dim=2, descending=True)[0][:, :, :c["best"]]
        group = torch.where(best[:, :, 0] > -math.inf, torch.where(best > -math.inf, best, 0.0).sum(dim=2), -math.inf)
        first = torch.sort(group, dim=1, descending=True, stable=True)[1][:, :c["top"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device="cuda").scatter_(1, first, True)
        rank = torch.where(keep.repeat_interleave(E // G, dim=1), rank, -math.inf)
    value, ids = torch.sort(rank, dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    there = value > -math.inf
    if c["renorm"]:
        lp = torch.where(there, logp.gather(1, ids), -math.inf)
        w = torch.exp(lp - lp.amax(dim=1, keepdim=True).clamp(min=-FLT_MAX))
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    else:
        w = p.gather(1, ids)
    ids = torch.where(there, ids, -1)
    offsets, row_token, token_row = _plan(ids, E)
    return {"ids": ids.to(torch.int32), "weights": torch.where(there, w, 0.0).float(), "offsets": offsets, "row_token": row_token,
            "token_row": token_row}


def _plain_product(s):
    """P [R, N] in fp32: the experts' rows side by side, padded to the longest."""
    a = (s["a"].view(F8).float().unflatten(-1, (-1, 128)) * s["as"][..., None]).flatten(-2)
    E, N, K = s["w"].shape
    w = s["w"].view(F8).float().view(E, N // 128, 128, K // 128, 128) * s["ws"][:, :, None, :, None]
    off = s["offsets"].long()
    R = s["row_token"].numel() if s["row_token"] is not None else a.shape[0]
    row = (off[:-1, None] + torch.arange(s["most"], device="cuda")[None, :]).clamp(max=R - 1)
    x = a[s["row_token"].long()[row]] if s["row_token"] is not None else a[row]
    y = torch.bmm(x, w.view(E, N, K).transpose(1, 2))
    r = torch.arange(R, device="cuda")
    e = torch.searchsorted(off, r, right=True) - 1
    return y[e, r - off[e]]


def _plain_norm(s):
    c = s["case"]
    rms = lambda v: torch.sqrt(v.square().mean(dim=1, keepdim=True) + 1e-6)  # noqa: E731
    z = s["y"].float()
    if c["k"]:
        z = (z[s["rows"].long()] * s["gates"][:, :, None]).sum(dim=1)
    if s["gamma_y"] is not None:
        z = z / rms(z) * s["gamma_y"].float()
    r = s["x"].float() + c["alpha"] * z
    n = r / rms(r) * s["gamma"].float()
    codes, scales = _quantize_rows(n)
    return {"x": r.to(s["x"].dtype), "normed": n.to(torch.bfloat16), "codes": codes, "scales": scales}


# ------------------------------------------------------------------ one pass

def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        import bit_quantized_linear_quantizers_gb300 as qz
        if op == "route":
            if "work" not in s:                      # a program makes its workspace once
                s["work"] = qz.Workspace()
            score = qz.SCORE_SOFTMAX if c["score"] == "softmax" else qz.SCORE_SIGMOID
            ids, w, offsets, row_token, token_row = qz.qz_moe_route(
                s["logits"], c["k"], score=score, renormalize=c["renorm"], bias=s["bias"], groups=c["G"], top_groups=c["top"],
                group_best=c["best"], n_tokens=s["n"], ws=s["work"])
            return {"ids": ids, "weights": w, "offsets": offsets, "row_token": row_token, "token_row": token_row}
        if op == "up":
            codes, scales = qz.qz_moe_gemm_fp8_swiglu(s["a"], s["as"], s["w"], s["ws"], s["offsets"], s["row_token"])
            return {"codes": codes.view(F8), "scales": scales}
        if op == "down":
            return qz.qz_moe_gemm_fp8(s["a"], s["as"], s["w"], s["ws"], s["offsets"])
        x, n, codes, scales = qz.qz_residual_rmsnorm(s["x"], s["gamma"], y=s["y"], token_row=s["rows"], weights=s["gates"],
                                                     alpha=c["alpha"], gamma_y=s["gamma_y"], eps=1e-6, normed=True, fp8=True)
        return {"x": x, "normed": n, "codes": codes.view(F8), "scales": scales}
    if op == "route":
        return _plain_route(s)
    if op == "norm":
        return _plain_norm(s)
    p = _plain_product(s)
    if op == "down":
        return p.to(torch.bfloat16)
    gate, up = p.chunk(2, dim=1)
    codes, scales = _quantize_rows(gate / (1.0 + torch.exp(-gate)) * up)
    return {"codes": codes, "scales": scales}


# ------------------------------------------------------------------ the definition, in 64 bits

def _e4m3(x):
    """Nearest E4M3 value (ties to even), saturating at 448: 4 significant bits down to 2^-6, steps of 2^-9 below."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 1
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_codes(x):
    R, N = x.shape
    s = x.view(R, N // 128, 128).abs().amax(dim=2).clamp(min=1e-12) / 448.0
    return _e4m3(x / s.repeat_interleave(128, dim=1)), s


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "route":
        # the gates of the experts that a sort of (key, index) pairs chooses, token by token on the host
        if c["T"] * c["E"] > 300000:
            return None
        n = c["T"] if s["n"] is None else int(s["n"])
        bias = [0.0] * c["E"] if s["bias"] is None else s["bias"].double().tolist()
        w = torch.zeros((c["T"], c["k"]), dtype=torch.float64)
        for t, row in enumerate(s["logits"].double().tolist()[:n]):
            if c["score"] == "softmax":
                top = max(row)
                total = math.fsum(math.exp(v - top) for v in row)
                p = [math.exp(v - top) / total for v in row]
            else:
                p = [1.0 / (1.0 + math.exp(-v)) for v in row]
            key = [a + b for a, b in zip(p, bias)]
            size = c["E"] // c["G"]
            value = [sum(sorted(key[g * size:(g + 1) * size])[-c["best"]:]) for g in range(c["G"])]
            keep = sorted(range(c["G"]), key=lambda g: (-value[g], g))[:c["top"]]
            ids = sorted((e for g in keep for e in range(g * size, (g + 1) * size)), key=lambda e: (-key[e], e))[:c["k"]]
            total = math.fsum(p[e] for e in ids) if c["renorm"] else 1.0
            w[t] = torch.tensor([p[e] / total for e in ids], dtype=torch.float64)
        return {"ids": None, "weights": w.cuda(), "offsets": None, "row_token": None, "token_row": None}
    if op == "norm":
        x, H = s["x"].double(), c["H"]
        y = s["y"].double()
        z = y if not c["k"] else torch.zeros_like(x)
        for j in range(c["k"]):
            z = torch.addcmul(z, s["gates"][:, j:j + 1].double(), y.index_select(0, s["rows"][:, j].long()))
        if c["post"]:
            z = z * torch.rsqrt((z * z).sum(dim=1, keepdim=True) / H + 1e-6) * s["gamma_y"].double()
        r = x + c["alpha"] * z
        n = r * torch.rsqrt((r * r).sum(dim=1, keepdim=True) / H + 1e-6) * s["gamma"].double()
        codes, scales = _exact_codes(n)
        return {"x": r, "normed": n, "codes": codes, "scales": scales}
    off = s["offsets"].tolist()
    parts = []
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        at = s["row_token"][lo:hi].long() if op == "up" else torch.arange(lo, hi, device="cuda")
        a = s["a"].view(F8)[at].double() * s["as"][at].double().repeat_interleave(128, dim=1)
        ws = s["ws"][e].double().repeat_interleave(128, dim=0).repeat_interleave(128, dim=1)
        p = a @ (s["w"][e].view(F8).double() * ws).T
        if op == "up":
            gate, up = p[:, :c["I"]], p[:, c["I"]:]
            p = gate * torch.sigmoid(gate) * up
        parts.append(p)
    p = torch.cat(parts)
    if op == "down":
        return p
    codes, scales = _exact_codes(p)
    return {"codes": codes, "scales": scales}
