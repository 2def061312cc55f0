"""What the layer norms around the layer and the experts' weight update are measured on: cases,
inputs, and their plain forms.

Operators: the layer norm with the residual sum before it (``moe_layer_norm``) and its gradient
(``moe_layer_norm_backward``), Newton-Schulz orthogonalisation of the experts' matrices
(``moe_orthogonalize``) and the update step around it (``moe_muon_update``). ``run`` computes a
case in elementary torch operations in 32 bits (a matrix's norm in 64), rounded once at the end,
or (``own``) through the framework's entry points. ``exact`` computes it in 64 bits: the norms
with their gradient by differentiation, the orthogonalisation matrix by matrix from its short
side.
"""
import math

import torch

own = False

BF16, FP32 = "bf16", "fp32"
TYPES = {BF16: torch.bfloat16, FP32: torch.float32}
SIZE = {BF16: 2, FP32: 4}
DEV = "cuda"
EPS = 1e-5                             # of the norms
A, B, C = 3.4445, -4.7750, 2.0315      # the iteration's coefficients
STEPS = 5
ORTH_EPS = 1e-7


# ---- the cases -----------------------------------------------------------------------
def listed():
    return [
        # before the layer: one decoding step of 8 tokens
        _norm("norm_decode", T=8, d=4096, y=False),
        # after the layer and before the next block, at the Mixtral width: residual sum and norm
        _norm("norm_mixtral", T=16384, d=4096, y=True),
        # a short ragged step of the fine-grained layer in fp32
        _norm("norm_short_fp32", T=37, d=2048, y=True, dtype=FP32),
        # the gradient: mid-size with the residual's gradient, an odd token count in fp32, and
        # the Mixtral width with the layer output's gradient as well
        _norm("norm_back_mid", T=4096, d=1024, y=False, back=True),
        _norm("norm_back_fine_fp32", T=8191, d=2048, y=False, back=True, dtype=FP32),
        _norm("norm_back_mixtral", T=16384, d=4096, y=True, back=True),
        # the tiny layer's gate matrices in fp32
        _orth("orth_tiny_fp32", E=8, m=64, n=128, dtype=FP32),
        # the mid-size layer's gate matrices, and the gate matrices (tall) of 64 fine-grained experts
        _orth("orth_mid", E=8, m=1024, n=4096),
        _orth("orth_fine", E=64, m=2048, n=1408),
        # a step on a few odd matrices in fp32, on the mid-size layer's down matrices (tall),
        # and on the Mixtral-size layer's gate matrices
        _orth("muon_odd_fp32", E=5, m=201, n=333, dtype=FP32, update=True),
        _orth("muon_mid", E=8, m=4096, n=1024, update=True),
        _orth("muon_mixtral", E=8, m=4096, n=14336, update=True),
    ]


def _norm(name, *, T, d, y, back=False, dtype=BF16):
    return dict(name=name, op="norm", T=T, d=d, y=y, back=back, dtype=dtype)


def _orth(name, *, E, m, n, update=False, dtype=BF16, nesterov=True):
    return dict(name=name, op="orth", E=E, m=m, n=n, update=update, dtype=dtype, nesterov=nesterov)


def draw(rng):
    """One more case: sizes log-uniform over the listed range, odd token counts and odd matrices
    among them, no more work than the largest listed case of its operator."""
    def size(lo, hi, step=1):
        v = lo * (hi / lo) ** rng.random()
        return max(lo, min(hi, int(v / step) * step))

    dtype = FP32 if rng.random() < 0.3 else BF16
    if rng.random() < 0.5:
        d = size(64, 8192, 8)
        return _norm("", T=min(size(1, 32768), 16384 * 4096 // d), d=d, y=rng.random() < 0.5,
                     back=rng.random() < 0.5, dtype=dtype)
    E = rng.choice([1, 2, 5, 8, 16, 64])
    odd = rng.random() < 0.4
    m, n = size(16, 4096, 1 if odd else 8), size(16, 8192, 1 if odd else 8)
    if dtype == FP32:
        m, n = min(m, 2048), min(n, 2048)
    if rng.random() < 0.5:
        m, n = n, m
    while E > 1 and E * min(m, n) ** 2 * max(m, n) > 8 * 2048 ** 2 * 4096:
        E //= 2
    return _orth("", E=E, m=m, n=n, update=rng.random() < 0.5, dtype=dtype, nesterov=rng.random() < 0.7)


def work(case):
    c = dict(case)
    b = SIZE[c["dtype"]]
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        if not c["back"]:
            per = 2 * b + ((4 + b) if c["y"] else 0)     # x, u; y and out
        else:
            per = 4 * b + (b if c["y"] else 0)           # out, d_u, d_out, dx; dy
        return {"bytes": T * d * per + 8 * T + 8 * d, "flops": 10.0 * T * d}
    E, s, l = c["E"], min(c["m"], c["n"]), max(c["m"], c["n"])
    # symmetric products by their half; two steps may share a Gram matrix, where that is less
    one, two = 3.0 * s * s * l + 1.0 * s ** 3, 3.0 * s * s * l + 5.0 * s ** 3
    flops = (STEPS // 2) * min(two, 2 * one) + (STEPS % 2) * one
    per = 2 * b + 8 + b if c["update"] else 2 * b
    return {"bytes": E * s * l * per, "flops": E * flops}


# ---- inputs --------------------------------------------------------------------------
def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = TYPES[c["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype).mul_(std)

    s = {"case": c}
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        # a residual stream: channels of different scales, rows with a mean
        scale = torch.exp(normal(d, std=0.5, dtype=torch.float32))
        s["x"] = (normal(T, d, dtype=torch.float32) * scale + normal(T, 1, dtype=torch.float32)).to(dt)
        s["gamma"] = 1 + normal(d, std=0.1, dtype=torch.float32)
        s["beta"] = normal(d, std=0.1, dtype=torch.float32)
        s["y"] = normal(T, d, std=0.5, dtype=torch.float32) if c["y"] and not c["back"] else None
        s["scale"] = 0.75 if c["y"] else 1.0
        if c["back"]:  # what the forward pass left
            s["d_u"], s["d_out"] = normal(T, d, std=0.1), normal(T, d, std=0.1)
            v = s["x"].double()
            s["mean"] = v.mean(1).float()
            s["rstd"] = (v.var(1, correction=0) + EPS).rsqrt().float()
        return s
    E, m, n = c["E"], c["m"], c["n"]
    # a gradient: directions that many tokens share, of falling weight, and every token's own
    rank = max(1, min(m, n) // 8)
    weight = torch.arange(1, rank + 1, device=DEV, dtype=torch.float32).rsqrt()
    g = torch.bmm(normal(E, m, rank, dtype=torch.float32) * weight, normal(E, rank, n, dtype=torch.float32))
    for e in range(E):
        g[e] += normal(m, n, dtype=torch.float32)
    s["g"] = g.mul_(1e-3).to(dt)
    del g
    if c["update"]:
        s["w"] = normal(E, m, n, std=0.02)
        s["momentum"] = normal(E, m, n, std=5e-3, dtype=torch.float32)
        s["lr"], s["mu"], s["decay"] = 0.02, 0.95, 0.1
        s["update_scale"] = math.sqrt(max(1.0, n / m))
    return s


# ---- one pass ------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if c["op"] == "norm":
        return (_run_norm_backward if c["back"] else _run_norm)(s, c)
    return (_run_update if c["update"] else _run_orth)(s, c)


def _run_norm(s, c):
    if own:
        import sparse_mixture_experts_sum_amd as moe
        r = moe.moe_layer_norm(s["x"], s["gamma"], s["beta"], y=s["y"], residual_scale=s["scale"], eps=EPS)
        return {n: r[n] for n in ("u", "mean", "rstd") + (("out",) if c["y"] else ())}
    dt, r = TYPES[c["dtype"]], {}
    out = s["x"]
    if c["y"]:
        r["out"] = out = (s["scale"] * s["x"].float() + s["y"]).to(dt)
    v = out.float()
    r["mean"] = v.mean(1)
    z = v - r["mean"][:, None]
    r["rstd"] = ((z * z).mean(1) + EPS).rsqrt()
    r["u"] = (z * r["rstd"][:, None] * s["gamma"] + s["beta"]).to(dt)
    return r


def _run_norm_backward(s, c):
    if own:
        import sparse_mixture_experts_sum_amd as moe
        r = moe.moe_layer_norm_backward(s["x"], s["d_u"], s["mean"], s["rstd"], s["gamma"], d_out=s["d_out"],
                                        residual_scale=s["scale"], want_dy=c["y"])
        return {n: r[n] for n in ("dx", "dgamma", "dbeta") + (("dy",) if c["y"] else ())}
    dt = TYPES[c["dtype"]]
    d_u, rstd = s["d_u"].float(), s["rstd"][:, None]
    z = (s["x"].float() - s["mean"][:, None]) * rstd
    dz = d_u * s["gamma"]
    D = s["d_out"].float() + rstd * (dz - dz.mean(1, keepdim=True) - z * (dz * z).mean(1, keepdim=True))
    r = {"dx": (s["scale"] * D).to(dt), "dgamma": (d_u * z).sum(0), "dbeta": d_u.sum(0)}
    if c["y"]:
        r["dy"] = D.to(dt)
    return r


def _newton_schulz(g):
    """[E, m, n] fp32 -> fp32."""
    norm = g.double().square().sum((1, 2)).sqrt()
    tall = g.shape[1] > g.shape[2]
    x = (g / (norm + ORTH_EPS)[:, None, None].float())
    if tall:
        x = x.transpose(1, 2).contiguous()
    for _ in range(STEPS):
        gram = torch.bmm(x, x.transpose(1, 2))
        x = A * x + torch.bmm(B * gram + C * torch.bmm(gram, gram), x)
    return x.transpose(1, 2) if tall else x


def _run_orth(s, c):
    if own:
        import sparse_mixture_experts_sum_amd as moe
        return moe.moe_orthogonalize(s["g"], steps=STEPS, coefficients=(A, B, C), eps=ORTH_EPS)
    return _newton_schulz(s["g"].float()).to(TYPES[c["dtype"]])


def _run_update(s, c):
    """In place, as an optimiser's step is: the weights and the momentum."""
    if own:
        import sparse_mixture_experts_sum_amd as moe
        moe.moe_muon_update(s["w"], s["g"], s["momentum"], lr=s["lr"], momentum=s["mu"], nesterov=c["nesterov"],
                            weight_decay=s["decay"], scale=s["update_scale"], steps=STEPS, coefficients=(A, B, C),
                            eps=ORTH_EPS)
        return {"w": s["w"], "m": s["momentum"]}
    g, m = s["g"].float(), s["momentum"]
    m.mul_(s["mu"]).add_(g)
    u = g + s["mu"] * m if c["nesterov"] else m
    o = _newton_schulz(u)
    w = (1 - s["lr"] * s["decay"]) * s["w"].float() - s["lr"] * s["update_scale"] * o
    s["w"].copy_(w)
    return {"w": s["w"], "m": m}


# ---- the definition in 64 bits -------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        d = {n: v.double() if isinstance(v, torch.Tensor) else v for n, v in s.items()}
        r = {}
        if not c["back"]:
            out = d["x"]
            if c["y"]:
                r["out"] = s["scale"] * d["x"] + d["y"]
                out = r["out"].to(TYPES[c["dtype"]]).double()
            r["mean"], var = out.mean(1), out.var(1, correction=0)
            r["rstd"] = 1 / (var + EPS).sqrt()
            r["u"] = (out - r["mean"][:, None]) / (var + EPS).sqrt()[:, None] * d["gamma"] + d["beta"]
            return r
        x, gamma, beta = (d[n].requires_grad_() for n in ("x", "gamma", "beta"))
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        u = (x - mean) / (var + EPS).sqrt() * gamma + beta
        dx, r["dgamma"], r["dbeta"] = torch.autograd.grad(u, (x, gamma, beta), d["d_u"])
        r["dx"] = s["scale"] * (d["d_out"] + dx)
        if c["y"]:
            r["dy"] = d["d_out"] + dx
        return r

    def orth(g):
        """One matrix, [long, short] times polynomials of its [short, short] Gram matrix."""
        x = g.t() if g.shape[0] < g.shape[1] else g
        x = x / (torch.linalg.vector_norm(g) + ORTH_EPS)
        eye = torch.eye(x.shape[1], dtype=torch.float64, device=DEV)
        for _ in range(STEPS):
            gram = x.t() @ x
            x = x @ (A * eye + gram @ (B * eye + C * gram))
        return x.t() if g.shape[0] < g.shape[1] else x

    w, m = [], []
    for e in range(c["E"]):
        g = s["g"][e].double()
        if not c["update"]:
            w.append(orth(g))
            continue
        m.append(s["mu"] * s["momentum"][e].double() + g)
        u = g + s["mu"] * m[-1] if c["nesterov"] else m[-1]
        w.append((1 - s["lr"] * s["decay"]) * s["w"][e].double() - s["lr"] * s["update_scale"] * orth(u))
    return {"w": torch.stack(w), "m": torch.stack(m)} if c["update"] else torch.stack(w)
