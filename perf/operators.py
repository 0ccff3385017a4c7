"""Operators around the POET-X linear, as cases to measure: what a training step does before and
after the layer.

  ln_fwd   layer norm of the rows that the layer reads, y = (x - mean) rstd gamma + beta
  ln_bwd   its gradient: dx and, summed over the rows, dgamma and dbeta
  ns       an update orthogonalised by Newton-Schulz products: X <- X / (|X|_F + eps), then
           X <- a X + (b A + c A^2) X with A = X X^T, `steps` times
  ns_q     the same for updates of the packed skew parameters q, one b x b block each

`run` computes the operators in their plain form, in 32 bits with one rounding at the end, or
(own = True) through the library.
"""
import math

import torch

own = False

MUON = (3.4445, -4.7750, 2.0315)   # the quintic's coefficients (a, b, c) in common use
STEPS = 5
NS_EPS = 1e-7
LN_EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token on its way through a 4096-wide model: nothing but latency
        {"name": "ln_fwd_token", "op": "ln_fwd", "rows": 1, "m": 4096, "dtype": "bf16",
         "w": "f32"},
        # the input of an 8B up_proj step: 16384 tokens
        {"name": "ln_fwd_8b", "op": "ln_fwd", "rows": 16384, "m": 4096, "dtype": "bf16",
         "w": "f32"},
        # an fp32 model of odd width, rows that no tile divides
        {"name": "ln_fwd_odd", "op": "ln_fwd", "rows": 1777, "m": 1023, "dtype": "f32",
         "w": "f32"},
        # the tiny fp32 workload's 256 tokens of width 512
        {"name": "ln_bwd_tiny", "op": "ln_bwd", "rows": 256, "m": 512, "dtype": "f32",
         "w": "f32"},
        # a 13B layer's step: 8192 tokens of width 5120
        {"name": "ln_bwd_13b", "op": "ln_bwd", "rows": 8192, "m": 5120, "dtype": "bf16",
         "w": "f32"},
        # bf16 rows of odd width, bf16 weights
        {"name": "ln_bwd_odd", "op": "ln_bwd", "rows": 4099, "m": 509, "dtype": "bf16",
         "w": "bf16"},
        # the update of an 8B k or v projection (4096 x 1024, taller than wide)
        {"name": "ns_8b_kv", "op": "ns", "batch": 1, "m": 4096, "n": 1024, "dtype": "bf16"},
        # the update of an 8B up projection, the largest
        {"name": "ns_8b_up", "op": "ns", "batch": 1, "m": 4096, "n": 14336, "dtype": "bf16"},
        # a 1.3B model's attention projection, kept and updated in fp32
        {"name": "ns_1p3b_f32", "op": "ns", "batch": 1, "m": 2048, "n": 2048, "dtype": "f32"},
        # a stack of odd-sized fp32 matrices
        {"name": "ns_odd_f32", "op": "ns", "batch": 3, "m": 1000, "n": 333, "dtype": "f32"},
        # dq of an 8B up_proj: 8 + 28 blocks of b = 512
        {"name": "ns_q_8b_up", "op": "ns_q", "batch": 36, "b": 512},
        # dq of the tiny workload: 8 + 8 blocks of b = 64
        {"name": "ns_q_tiny", "op": "ns_q", "batch": 16, "b": 64},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _flops_cap():
    return 2.0 * 5 * (1.5 * 4096 * 4096 * 14336 + 0.5 * 4096 ** 3)


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ns", "ns_q"])
    if op in ("ln_fwd", "ln_bwd"):
        # (rows of two features have a gradient of almost nothing but rounding)
        m = _log_int(rng, 4, 16384)
        if rng.random() < 0.5 and m >= 8:
            m = m // 8 * 8
        rows = _log_int(rng, 1, max(1, min(65536, 8192 * 5120 // m)))
        return {"op": op, "rows": rows, "m": m, "dtype": rng.choice(["f32", "bf16"]),
                "w": rng.choice(["f32", "bf16"])}
    if op == "ns":
        while True:
            case = {"op": op, "batch": _log_int(rng, 1, 32), "m": _log_int(rng, 1, 8192),
                    "n": _log_int(rng, 1, 8192), "dtype": rng.choice(["f32", "bf16"])}
            if rng.random() < 0.5:
                case["m"], case["n"] = -(-case["m"] // 8) * 8, -(-case["n"] // 8) * 8
            # fp32 results are three times the work of bf16 ones
            if work(case)["flops"] * (3 if case["dtype"] == "f32" else 1) <= _flops_cap():
                return case
    b = rng.choice([2, 7, 32, 64, 100, 128, 200, 256, 384, 500, 512, 777, 1024])
    most = max(1, int(_flops_cap() / 3 / (2.0 * STEPS * 1.5 * b ** 3)))
    return {"op": op, "batch": _log_int(rng, 1, min(256, most)), "b": b}


def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        t, m = case["rows"], case["m"]
        e, w = (2 if case["dtype"] == "bf16" else 4), (2 if case["w"] == "bf16" else 4)
        if op == "ln_fwd":   # x and the weights in; y, mean and rstd out
            return {"bytes": 2 * t * m * e + 2 * m * w + 8 * t, "flops": 8 * t * m}
        # x, dy, gamma and the row statistics in; dx, dgamma and dbeta out
        return {"bytes": 3 * t * m * e + m * w + 8 * t + 8 * m, "flops": 14 * t * m}
    if op == "ns":
        r, k, nb = min(case["m"], case["n"]), max(case["m"], case["n"]), case["batch"]
        e = 2 if case["dtype"] == "bf16" else 4
        # A = X X^T and A A are symmetric: half of each has to be computed
        macs = nb * STEPS * (0.5 * r * r * k + 0.5 * r ** 3 + r * r * k)
        return {"bytes": 2 * nb * r * k * e, "flops": int(2 * macs)}
    b, nb = case["b"], case["batch"]
    # X is skew: half of the third product is enough too
    return {"bytes": 2 * nb * (b * (b - 1) // 2) * 4, "flops": int(2 * nb * STEPS * 1.5 * b ** 3)}


# ------------------------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _update_like(g, batch, m, n):
    """Updates as an optimiser sees them: a few strong directions of falling weight over a
    full-rank background, about 1e-3 in size."""
    p = max(1, min(m, n) // 16)
    fall = 1.0 / (1.0 + torch.arange(p, device="cuda", dtype=torch.float32))
    left = _randn(g, batch, m, p) * fall
    x = torch.baddbmm(_randn(g, batch, m, n), left, _randn(g, batch, p, n), beta=0.3)
    return x.mul_(1e-3)


def _stream_like(g, t, m):
    """Rows of a residual stream: features of different scale and offset, a few of them large."""
    scale = 0.5 + torch.rand(m, generator=g, device="cuda")
    scale[torch.randint(0, m, (max(1, m // 512),), generator=g, device="cuda")] *= 8.0
    return _randn(g, t, m) * scale + 0.3 * _randn(g, m)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        t, m, dt, wt = case["rows"], case["m"], DTYPES[case["dtype"]], DTYPES[case["w"]]
        st = {"op": op, "x": _stream_like(g, t, m).to(dt),
              "gamma": (1.0 + 0.1 * _randn(g, m)).to(wt), "beta": (0.1 * _randn(g, m)).to(wt)}
        if op == "ln_fwd":
            st["y"] = torch.empty_like(st["x"])
            st["mean"] = torch.empty(t, device="cuda")
            st["rstd"] = torch.empty(t, device="cuda")
            return st
        # the backward's caller holds what the forward left: the rows' mean and rstd
        x64 = st["x"].double()
        mean = x64.mean(1)
        st["mean"] = mean.float()
        st["rstd"] = ((x64 - mean[:, None]).square().mean(1) + LN_EPS).rsqrt().float()
        st["dy"] = (_randn(g, t, m) * 1e-2).to(dt)
        st["dx"] = torch.empty_like(st["x"])
        st["dgamma"] = torch.empty(m, device="cuda")
        st["dbeta"] = torch.empty(m, device="cuda")
        if own:
            from orthogonal_equivalence_build_b200 import poetx
            st["ws"] = torch.empty(max(16, poetx.layer_norm_bwd_workspace_bytes(t, m)),
                                   dtype=torch.uint8, device="cuda")
        return st
    if op == "ns":
        x = _update_like(g, case["batch"], case["m"], case["n"]).to(DTYPES[case["dtype"]])
        st = {"op": op, "x": x, "out": torch.empty_like(x)}
        if own:
            from orthogonal_equivalence_build_b200 import poetx
            st["ws"] = torch.empty(max(16, poetx.orthogonalize_workspace_bytes(x, st["out"])),
                                   dtype=torch.uint8, device="cuda")
        return st
    b, nb = case["b"], case["batch"]
    full = _update_like(g, nb, b, b)
    iu = torch.triu_indices(b, b, 1, device="cuda")
    u = (full - full.transpose(1, 2))[:, iu[0], iu[1]].contiguous()
    st = {"op": op, "b": b, "u": u, "out": torch.empty_like(u), "iu": iu}
    if own:
        from orthogonal_equivalence_build_b200 import poetx
        st["ws"] = torch.empty(max(16, poetx.orthogonalize_q_workspace_bytes(nb, b)),
                               dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------------- one pass
def _plain_ns(x):
    """X [batch, r, k] fp32 with r <= k or not: the Newton-Schulz iterates on the smaller side."""
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    a, b, c = MUON
    for _ in range(STEPS):
        s = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * s + c * torch.bmm(s, s), x)
    return x.transpose(1, 2) if tall else x


def run(state):
    op = state["op"]
    if own:
        return _run_own(state)
    if op == "ln_fwd":
        x = state["x"].float()
        mean = x.mean(1)
        xc = x - mean[:, None]
        rstd = (xc.square().mean(1) + LN_EPS).rsqrt()
        y = xc * rstd[:, None] * state["gamma"].float() + state["beta"].float()
        return {"y": y.to(state["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        rstd = state["rstd"][:, None]
        xh = (state["x"].float() - state["mean"][:, None]) * rstd
        dy = state["dy"].float()
        g = dy * state["gamma"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return {"dx": dx.to(state["x"].dtype), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
    if op == "ns":
        return _plain_ns(state["x"].float()).to(state["x"].dtype)
    nb, b, iu = state["u"].shape[0], state["b"], state["iu"]
    x = torch.zeros(nb, b, b, device=state["u"].device)
    x[:, iu[0], iu[1]] = state["u"]
    return _plain_ns(x - x.transpose(1, 2))[:, iu[0], iu[1]]


def _run_own(state):
    from orthogonal_equivalence_build_b200 import poetx
    op = state["op"]
    if op == "ln_fwd":
        poetx.layer_norm_fwd(state["x"], state["gamma"], state["beta"], state["y"],
                             state["mean"], state["rstd"], eps=LN_EPS)
        return {"y": state["y"], "mean": state["mean"], "rstd": state["rstd"]}
    if op == "ln_bwd":
        poetx.layer_norm_bwd(state["x"], state["dy"], state["gamma"], state["mean"],
                             state["rstd"], state["dx"], state["dgamma"], state["dbeta"],
                             workspace=state["ws"])
        return {"dx": state["dx"], "dgamma": state["dgamma"], "dbeta": state["dbeta"]}
    if op == "ns":
        poetx.orthogonalize(state["x"], state["out"], steps=STEPS, coeffs=MUON, eps=NS_EPS,
                            workspace=state["ws"])
        return state["out"]
    poetx.orthogonalize_q(state["u"], state["b"], state["out"], steps=STEPS, coeffs=MUON,
                          eps=NS_EPS, workspace=state["ws"])
    return state["out"]


# ------------------------------------------------------------------- the definition in 64 bits
def _exact_ns(x):
    """One matrix in 64 bits: X p(X^T X), the polynomial on the larger side, by Horner's rule."""
    tall = x.shape[0] > x.shape[1]
    y = x.double()
    y = y / (torch.linalg.vector_norm(y) + NS_EPS)
    if tall:
        y = y.T.contiguous()
    a, b, c = MUON
    for _ in range(STEPS):
        gram = y.T @ y
        inner = y * b + c * (y @ gram)
        y = a * y + inner @ gram
    return y.T.contiguous() if tall else y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "ln_fwd":
        x = st["x"].double()
        mean = x.sum(1) / case["m"]
        var = (x - mean[:, None]).pow(2).sum(1) / case["m"]
        rstd = 1.0 / torch.sqrt(var + LN_EPS)
        y = torch.addcmul(st["beta"].double(), (x - mean[:, None]) * rstd[:, None],
                          st["gamma"].double())
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        x, dy, gamma = st["x"].double(), st["dy"].double(), st["gamma"].double()
        mean, rstd, m = st["mean"].double(), st["rstd"].double(), case["m"]
        xc = x - mean[:, None]
        c1 = (dy @ gamma) / m
        c2 = ((dy * xc) @ gamma) * rstd / m
        dx = (dy * gamma - c1[:, None]) * rstd[:, None] - xc * (c2 * rstd.square())[:, None]
        return {"dx": dx, "dgamma": (dy * xc).T @ rstd, "dbeta": dy.sum(0)}
    if op == "ns":
        return torch.stack([_exact_ns(x) for x in st["x"]])
    iu, b = st["iu"], case["b"]
    out = torch.empty_like(st["u"], dtype=torch.float64)
    for i, u in enumerate(st["u"]):
        x = torch.zeros(b, b, dtype=torch.float64, device=u.device)
        x[iu[0], iu[1]] = u.double()
        x[iu[1], iu[0]] = -u.double()
        out[i] = _exact_ns(x)[iu[0], iu[1]]
    return out
