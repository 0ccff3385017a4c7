"""Layer norm, the POET-X linear, both gradients and the orthogonalised update of q as one training
step, against the same step in 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
import poetx_workloads as W

try:
    from orthogonal_equivalence_build_b200 import poetx
except ImportError:  # pragma: no cover
    poetx = None

MUON = (3.4445, -4.7750, 2.0315)


def step64(h, gamma, beta, w0m, pr, pp, q_r, q_p, b, dy, eps):
    mean = h.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((h - mean) ** 2).mean(1, keepdims=True) + eps)
    xh = (h - mean) * rstd
    ref = O.linear_bwd(xh * gamma + beta, dy, w0m, pr, pp, O.cnp(q_r, b), O.cnp(q_p, b), q_r, q_p, b)
    g = ref["dX"] * gamma
    dh = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    out = dict(y=ref["Y"], dh=dh, dgamma=(ref["dX"] * xh).sum(0), dbeta=ref["dX"].sum(0))
    return dict(out, dq_r=ref["dq_r"], dq_p=ref["dq_p"])


def updated64(q, dq, b, lr):
    iu = np.triu_indices(b, 1)
    new = np.array(q, np.float64)
    for i, d in enumerate(dq):
        X = np.zeros((b, b))
        X[iu] = d
        X = X - X.T
        X /= np.linalg.norm(X) + 1e-7
        for _ in range(5):
            A = X @ X.T
            X = MUON[0] * X + (MUON[1] * A + MUON[2] * A @ A) @ X
        new[i] -= lr * X[iu]
    return new


def step_gpu(layer, h, gamma, beta, dy, lr, o):
    poetx.layer_norm_fwd(h, gamma, beta, o["x"], o["mean"], o["rstd"])
    poetx.layer_cnp_build(layer, workspace=o["ws"])
    poetx.linear_fwd(layer, o["x"], o["y"], o["saved"], workspace=o["ws"])
    poetx.linear_bwd(layer, o["x"], dy, o["saved"], o["dx"], o["dq_r"], o["dq_p"],
                     workspace=o["ws"])
    poetx.layer_norm_bwd(h, o["dx"], gamma, o["mean"], o["rstd"], o["dh"], o["dgamma"], o["dbeta"],
                         workspace=o["ws"])
    for side, q in (("r", layer.q_r), ("p", layer.q_p)):
        up = o["up_" + side]
        poetx.orthogonalize_q(o["dq_" + side], layer.b, up, scale=lr, workspace=o["ws"])
        q.sub_(up)


def make(dt, m, n, b, T, dev="cuda"):
    wl = W.WORKLOADS["llama1p3b_attn"]
    p = W.layer_params(wl, m=m, n=n, b=b)
    a = W.layer_acts(wl, m=m, n=n, tokens=T)
    rng = np.random.default_rng(3)
    gamma, beta = 1 + 0.1 * rng.standard_normal(m), 0.1 * rng.standard_normal(m)
    t = lambda v, d: torch.from_numpy(np.ascontiguousarray(v)).to(d).to(dev)
    w0m = t(p["W0"][p["perm_r"]][:, p["perm_p"]], dt)
    layer = poetx.PoetxLinear(w0m, t(p["perm_r"], torch.int32), t(p["perm_p"], torch.int32),
                              t(p["q_r"], torch.float32), t(p["q_p"], torch.float32), b)
    h, dy = t(3.0 * a["X"] + 1.0, dt), t(a["dY"], dt)
    o = dict(x=torch.empty_like(h), y=torch.empty_like(dy), saved=torch.empty_like(dy),
             dx=torch.empty_like(h), dh=torch.empty_like(h))
    for k, s in (("mean", T), ("rstd", T), ("dgamma", m), ("dbeta", m)):
        o[k] = torch.empty(s, device=dev)
    o["dq_r"], o["dq_p"] = torch.empty_like(layer.q_r), torch.empty_like(layer.q_p)
    o["up_r"], o["up_p"] = torch.empty_like(layer.q_r), torch.empty_like(layer.q_p)
    need = max(poetx.layer_cnp_workspace_bytes(layer), poetx.fwd_workspace_bytes(layer, T),
               poetx.bwd_workspace_bytes(layer, T), poetx.layer_norm_bwd_workspace_bytes(T, m),
               poetx.orthogonalize_q_workspace_bytes(m // b, b),
               poetx.orthogonalize_q_workspace_bytes(n // b, b))
    o["ws"] = torch.empty(need, dtype=torch.uint8, device=dev)
    return p, layer, h, t(gamma, torch.float32), t(beta, torch.float32), dy, o


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
def test_training_step(dt, captured):
    m, n, b, T, lr = 256, 384, 128, 193, 1e-3
    p, layer, h, gamma, beta, dy, o = make(dt, m, n, b, T)
    q0 = [layer.q_r.clone(), layer.q_p.clone()]
    f = lambda t: t.double().cpu().numpy()
    want = step64(f(h), f(gamma), f(beta), f(layer.w0m), p["perm_r"], p["perm_p"], f(q0[0]),
                  f(q0[1]), b, f(dy), 1e-5)
    step_gpu(layer, h, gamma, beta, dy, lr, o)   # also the warm-up of the captured run
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step_gpu(layer, h, gamma, beta, dy, lr, o)
        layer.q_r.copy_(q0[0])
        layer.q_p.copy_(q0[1])
        graph.replay()
    torch.cuda.synchronize()
    poetx.device_status()
    # the layer's own bars: 1e-2 of the largest value for bf16, 1e-5 for fp32 (twice that through
    # the norm's gradient)
    tol = 1e-2 if dt == torch.bfloat16 else 2e-5
    for k in ("y", "dh", "dgamma", "dbeta", "dq_r", "dq_p"):
        err = np.abs(f(o[k]) - want[k]).max() / np.abs(want[k]).max()
        assert err <= tol, (k, err)
    # q against the update of the dq that the GPU found: dq's parts are off by 2^-21 of |X_0|_F = 1,
    # lifted by at most 3.4445^5 = 485, against a result of norm ~ sqrt(b): 2e-5; q's own rounding,
    # 2^-24 of 0.005, against lr / sqrt(b): 4e-6
    for side, q, old in (("r", layer.q_r, q0[0]), ("p", layer.q_p, q0[1])):
        new = updated64(f(old), f(o["dq_" + side]), b, lr)
        err = np.linalg.norm(f(q) - new) / np.linalg.norm(new - f(old))
        assert err <= 1e-4, (side, err)
