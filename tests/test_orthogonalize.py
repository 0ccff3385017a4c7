"""Newton-Schulz orthogonalisation (poetx_orthogonalize, poetx_orthogonalize_q) against the
recurrence in 64 bits.

The tolerance of a case is a first-order bound on the Frobenius error, worked out per case from
the exact iterates. With u_x, u_g and u_m the relative rounding errors of X, of the X that the
Gram product reads and of A, H and B, one step X -> B X, B = a I + A H, A = X X^T, H = b I + c A,
adds to the propagated error
    |X|_2 (u_m |B|_F + |H|_2 dA + |A|_2 dH),   dA = u_m |A|_F + 2 u_g |X|_2 |X|_F + acc,
    dH = u_m |H|_F + |c| (2 u_g |X|_2 |X|_F + acc),
and an error already in X grows by at most the largest divided difference of the odd polynomial
p(s) = a s + b s^3 + c s^5 over the singular values, (p_i - p_j) / (s_i - s_j) and
(p_i + p_j) / (s_i + s_j). fp32 results: parts of 22 bits, and the dropped lo lo product is
2^-22 of the full one: u = 2^-21 throughout. bf16 results: fp16 operands, u = 2^-11 (half a step),
X in two parts in every update but the last. acc: fp32 accumulation, K / 16 + 16 additions of half
a step, 2^-24 each (tensor cores may truncate: 2^-23), of the sum of magnitudes, at most
|X|_F^2. The result is rounded once: 2^-8 (bf16) or 2^-24 (fp32) of its norm.
"""
import ctypes

import numpy as np
import pytest
import torch

try:
    from orthogonal_equivalence_build_b200 import poetx
except ImportError:  # pragma: no cover
    poetx = None

MUON = (3.4445, -4.7750, 2.0315)
CONV = (1.875, -1.25, 0.375)
gpu = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def newton_schulz64(x, coeffs, eps, scale=1.0):
    """(result, iterates) of one matrix in 64 bits."""
    X = x / (np.sqrt((x * x).sum()) + eps)
    its = [X]
    for a, b, c in coeffs:
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
        its.append(X)
    return scale * X, its


def bound(its, coeffs, out_bf16, scale):
    err = 0.0
    s = np.linalg.svd(its[0], compute_uv=False)   # of X_t; the next ones are |p(s)|
    for t, (a, b, c) in enumerate(coeffs):
        X = its[t]
        if X.shape[0] > X.shape[1]:
            X = X.T
        r, k = X.shape
        last = t + 1 == len(coeffs)
        if out_bf16:
            u_m = u_g = 2.0 ** -11
            u_x = 2.0 ** -11 if last else 2.0 ** -21
        else:
            u_m = u_g = u_x = 2.0 ** -21
        A = X @ X.T
        H = b * np.eye(r) + c * A
        B = a * np.eye(r) + A @ H
        x2, a2, h2 = s.max(), s.max() ** 2, np.abs(b + c * s ** 2).max()   # spectral norms
        nf = np.linalg.norm
        acc = (k / 16 + 16) * 2.0 ** -23 * nf(X) ** 2
        acc_r = (r / 16 + 16) * 2.0 ** -23
        gram = 2 * u_g * x2 * nf(X) + acc
        dA = u_m * nf(A) + gram
        dH = u_m * nf(H) + abs(c) * gram
        dB = u_m * nf(B) + h2 * dA + a2 * dH + acc_r * nf(A) * nf(H)
        p = a * s + b * s ** 3 + c * s ** 5
        dp = a + 3 * b * s ** 2 + 5 * c * s ** 4
        ds, sm = s[:, None] - s[None, :], s[:, None] + s[None, :]
        close = np.abs(ds) < 1e-9
        div = np.where(close, dp[:, None], (p[:, None] - p[None, :]) / np.where(close, 1.0, ds))
        gain = max(np.abs(div).max(),
                   np.abs((p[:, None] + p[None, :]) / np.maximum(sm, 1e-30)).max(), abs(a))
        err = gain * (err + u_x * nf(X)) + x2 * dB + acc_r * nf(B) * nf(X)
        s = np.abs(p)
    X = its[-1]
    return abs(scale) * (err + (2.0 ** -8 if out_bf16 else 2.0 ** -24) * np.linalg.norm(X))


def spectrum_matrix(rng, m, n, lo=0.2):
    """m x n with singular values spread over [lo, 1] (before the normalisation)."""
    r = min(m, n)
    u = np.linalg.qr(rng.standard_normal((m, r)))[0]
    v = np.linalg.qr(rng.standard_normal((n, r)))[0]
    return (u * np.linspace(1.0, lo, r)) @ v.T


def check(x, out, coeffs, eps=1e-7, scale=1.0):
    """x, out: device stacks [batch, m, n]."""
    x64 = x.double().cpu().numpy()
    got = out.double().cpu().numpy()
    for g in range(x64.shape[0]):
        want, its = newton_schulz64(x64[g], coeffs, eps, scale)
        tol = bound(its, coeffs, out.dtype == torch.bfloat16, scale)
        err = np.linalg.norm(got[g] - want)
        assert err <= tol, (g, err, tol)


def run(x, coeffs, out_dtype, **kw):
    out = torch.full(x.shape, 777.0, dtype=out_dtype, device=x.device)
    poetx.orthogonalize(x, out, steps=len(coeffs), coeffs=coeffs, **kw)
    torch.cuda.synchronize()
    poetx.device_status()
    return out


SHAPES = [(1, 1, 1), (1, 1, 7), (2, 5, 3), (1, 64, 64), (3, 65, 130), (2, 130, 65),
          (1, 128, 300), (1, 257, 257), (2, 300, 1000), (1, 1000, 333), (4, 512, 512),
          (40, 256, 256), (38, 200, 521), (2, 1100, 1300), (12, 700, 640),
          (2, 1800, 1700), (3, 1500, 1550)]


@gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("xt,ot", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"),
                                   ("bf16", "f32")])
def test_matches_the_recurrence(shape, xt, ot):
    rng = np.random.default_rng(sum(shape))
    x = np.stack([spectrum_matrix(rng, *shape[1:]) for _ in range(shape[0])])
    x = torch.from_numpy(x).to(DT[xt]).cuda()
    check(x, run(x, [MUON] * 5, DT[ot]), [MUON] * 5)


@gpu
@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_step_counts_and_scale(steps, ot):
    rng = np.random.default_rng(steps)
    x = torch.from_numpy(np.stack([spectrum_matrix(rng, 96, 200) for _ in range(2)])).float().cuda()
    check(x, run(x, [MUON] * steps, DT[ot], scale=-0.37), [MUON] * steps, scale=-0.37)


@gpu
@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_coefficients_per_step(ot):
    # the second set lifts singular values of 1 to 2; the third brings them back
    rng = np.random.default_rng(5)
    coeffs = [MUON, (2.0, 1.0, -1.0), (0.5, 0.0, 0.0), CONV]
    x = torch.from_numpy(spectrum_matrix(rng, 150, 90)[None]).float().cuda()
    check(x, run(x, coeffs, DT[ot]), coeffs)


@gpu
def test_converges_to_the_polar_factor():
    rng = np.random.default_rng(6)
    x = spectrum_matrix(rng, 120, 120)
    u, _, vt = np.linalg.svd(x)
    out = run(torch.from_numpy(x[None]).float().cuda(), [CONV] * 16, torch.float32)
    assert np.abs(out[0].double().cpu().numpy() - u @ vt).max() < 1e-4


@gpu
@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_strong_directions_over_a_weak_background(ot):
    # singular values from 1 down to about 3e-3: what rounding X to one part would drown
    rng = np.random.default_rng(7)
    x = rng.standard_normal((192, 8)) @ rng.standard_normal((8, 320)) + \
        0.1 * rng.standard_normal((192, 320))
    x = torch.from_numpy(x[None]).float().cuda()
    out = run(x, [MUON] * 5, DT[ot])
    want, its = newton_schulz64(x[0].double().cpu().numpy(), [MUON] * 5, 1e-7)
    err = np.linalg.norm(out[0].double().cpu().numpy() - want) / np.linalg.norm(want)
    # X_0's parts are off by at most 2^-21 of |X_0|_F = 1, which five steps lift by at most
    # 3.4445^5 = 485, against a result of norm ~ 12: 2e-5. bf16: the same for X, and for A, H and
    # B one part each in the last step, 2^-11 of factors below 5, with the result's own 2^-8
    assert err < (2e-5 if ot == "f32" else 2.0 ** -8 + 3 * 5 * 2.0 ** -11)
    check(x, out, [MUON] * 5)


@gpu
@pytest.mark.parametrize("factor", [1e30, 1e-30])
def test_norm_over_the_whole_exponent_range(factor):
    rng = np.random.default_rng(8)
    x = torch.from_numpy(spectrum_matrix(rng, 40, 70)[None] * factor).float().cuda()
    check(x, run(x, [MUON] * 5, torch.float32, eps=0.0), [MUON] * 5, eps=0.0)


@gpu
def test_zero_and_nonfinite_matrices_stay_apart():
    rng = np.random.default_rng(9)
    x = torch.from_numpy(np.stack([spectrum_matrix(rng, 70, 100) for _ in range(4)])).float().cuda()
    x[1] = 0
    x[2, 3, 5] = float("nan")
    for out_t in (torch.float32, torch.bfloat16):
        out = run(x, [MUON] * 5, out_t)
        assert torch.equal(out[1], torch.zeros_like(out[1]))
        assert torch.isnan(out[2]).all()
        check(x[[0, 3]], out[[0, 3]], [MUON] * 5)
    y = x.clone()
    y[2, 3, 5] = float("inf")
    out = run(y, [MUON] * 5, torch.float32)
    assert torch.isnan(out[2]).all()
    check(y[[0, 3]], out[[0, 3]], [MUON] * 5)


@gpu
def test_in_place_two_dimensional_and_same_bits():
    rng = np.random.default_rng(10)
    x = torch.from_numpy(spectrum_matrix(rng, 333, 170)).float().cuda()
    a, b = torch.empty_like(x), x.clone()
    poetx.orthogonalize(x, a)
    poetx.orthogonalize(b, b)
    assert torch.equal(a, b)
    check(x[None], a[None], [MUON] * 5)


@gpu
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 70, 41), (3, 170, 141), (3, 1500, 1601)])
def test_writes_only_its_output_and_workspace(shape, xt):
    x = torch.randn(*shape, device="cuda").to(DT[xt])
    need = poetx.orthogonalize_workspace_bytes(x, x)
    buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = buf[256:256 + need]
    obuf = torch.full((x.numel() + 128,), 3.0, dtype=x.dtype, device="cuda")
    out = obuf[64:64 + x.numel()].view_as(x)
    poetx.orthogonalize(x, out, workspace=ws)
    torch.cuda.synchronize()
    assert (buf[:256] == 0x5A).all() and (buf[256 + need:] == 0x5A).all()
    assert (obuf[:64] == 3).all() and (obuf[64 + x.numel():] == 3).all()
    ref = torch.empty_like(x)
    poetx.orthogonalize(x, ref)
    assert torch.equal(out, ref)


def unpack(u, b):
    X = np.zeros((u.shape[0], b, b))
    iu = np.triu_indices(b, 1)
    X[:, iu[0], iu[1]] = u
    return X - X.transpose(0, 2, 1)


@gpu
@pytest.mark.parametrize("nb,b", [(1, 2), (3, 3), (5, 7), (16, 64), (2, 100), (3, 128), (4, 200),
                                  (40, 256), (9, 512), (1, 777), (2, 1024), (12, 777),
                                  (16, 1000)])
def test_packed_blocks(nb, b):
    rng = np.random.default_rng(b)
    u = torch.from_numpy(rng.standard_normal((nb, b * (b - 1) // 2)) * 1e-3).float().cuda()
    out = torch.full_like(u, 777.0)
    poetx.orthogonalize_q(u, b, out, scale=0.2)
    torch.cuda.synchronize()
    poetx.device_status()
    X = unpack(u.double().cpu().numpy(), b)
    got = unpack(out.double().cpu().numpy(), b)
    for g in range(0, nb, max(1, nb // 4)):
        want, its = newton_schulz64(X[g], [MUON] * 5, 1e-7, 0.2)
        err, tol = np.linalg.norm(got[g] - want), bound(its, [MUON] * 5, False, 0.2)
        assert err <= tol, (g, err, tol)
    # the packed form is the dense one on the unpacked blocks
    dense = torch.from_numpy(X).float().cuda()
    dout = torch.empty_like(dense)
    poetx.orthogonalize(dense, dout, scale=0.2)
    d = (dout.double().cpu().numpy() - got)
    assert np.linalg.norm(d[0]) <= 2 * bound(newton_schulz64(X[0], [MUON] * 5, 1e-7)[1],
                                             [MUON] * 5, False, 0.2)


@gpu
def test_packed_in_place_zero_and_nan_blocks():
    u = torch.randn(4, 100 * 99 // 2, device="cuda")
    u[1] = 0
    u[2, 17] = float("nan")
    out = torch.empty_like(u)
    poetx.orthogonalize_q(u, 100, out)
    v = u.clone()
    poetx.orthogonalize_q(v, 100, v)
    assert torch.equal(out[1], torch.zeros_like(out[1])) and torch.isnan(out[2]).all()
    assert torch.equal(v[[0, 1, 3]], out[[0, 1, 3]])


@gpu
def test_graph_replay_and_other_stream():
    x = torch.randn(2, 300, 520, device="cuda", dtype=torch.bfloat16)
    ref, out = torch.empty_like(x), torch.empty_like(x)
    poetx.orthogonalize(x, ref)
    ws = torch.empty(poetx.orthogonalize_workspace_bytes(x, out), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    poetx.orthogonalize(x, out, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        poetx.orthogonalize(x, out, workspace=ws)
    y = torch.randn_like(x)
    x.copy_(y)
    poetx.orthogonalize(y, ref)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    poetx.device_status()


@gpu
def test_graphs_that_share_a_workspace():
    xs = [torch.randn(300, 520, device="cuda"), torch.randn(700, 640, device="cuda")]
    refs, outs = ([torch.empty_like(x) for x in xs] for _ in range(2))
    for x, r in zip(xs, refs):
        poetx.orthogonalize(x, r)
    ws = torch.empty(max(poetx.orthogonalize_workspace_bytes(x, x) for x in xs),
                     dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in xs]
    for g, x, o in zip(graphs, xs, outs):
        with torch.cuda.graph(g):
            poetx.orthogonalize(x, o, workspace=ws)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            assert torch.equal(o, r)
    poetx.device_status()


@gpu
def test_an_input_written_by_the_launch_before():
    """A chain of calls whose inputs the call before has just written, with no wait in between."""
    x = torch.randn(4, 100 * 99 // 2, device="cuda")
    a, b = x.clone(), x.clone()
    for _ in range(20):
        poetx.orthogonalize_q(a, 100, a)
        poetx.orthogonalize_q(b, 100, b)
        torch.cuda.synchronize()
    c = x.clone()
    for _ in range(20):
        poetx.orthogonalize_q(c, 100, c)
    assert torch.equal(a, c) and torch.equal(b, c)
    y = torch.randn(2, 300, 520, device="cuda")
    d, e = y.clone(), y.clone()
    for _ in range(10):
        poetx.orthogonalize(d, d)
        torch.cuda.synchronize()
    for _ in range(10):
        poetx.orthogonalize(e, e)
    assert torch.equal(d, e)


@gpu
def test_two_streams_at_once():
    xs = [torch.randn(512, 640, device="cuda") for _ in range(2)]
    refs = [torch.empty_like(x) for x in xs]
    for x, r in zip(xs, refs):
        poetx.orthogonalize(x, r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [torch.empty_like(x) for x in xs]
    for _ in range(4):
        for x, o, s in zip(xs, outs, streams):
            poetx.orthogonalize(x, o, stream=s)
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)
    poetx.device_status()


# ----------------------------------------------------------------------------- refusals (CPU)
def _call(x=0x10000, xt=0, batch=1, m=64, n=64, coeffs=MUON, steps=1, eps=1e-7, scale=1.0,
          out=0x20000, ot=0, ws=None, wsb=0):
    c = None if coeffs is None else (ctypes.c_float * (3 * max(1, steps)))(*(coeffs * max(1, steps)))
    return poetx.lib.poetx_orthogonalize(x, xt, batch, m, n, c, steps, eps, scale, out, ot, ws,
                                         wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(batch=-1), 1), (dict(m=-1), 1), (dict(n=-3), 1),
    (dict(coeffs=None), 1), (dict(steps=0), 1), (dict(steps=-2), 1), (dict(steps=65), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(scale=float("inf")), 1), (dict(coeffs=(float("nan"), 0.0, 0.0)), 1),
    (dict(coeffs=(100.0, 0.0, 0.0), steps=5), 1),      # singular values grow without bound
    (dict(m=65537), 2), (dict(n=70000), 2), (dict(batch=65536), 2),
    (dict(batch=65535, m=65536, n=65536), 2),
    (dict(xt=7), 4), (dict(ot=-1), 4), (dict(x=0x10008), 3), (dict(out=0x20004), 3),
    (dict(m=200), 8), (dict(m=200, ws=0x30000, wsb=1024), 8), (dict(out=0x10000, ot=1), 1),
])
def test_refusals(kw, status):
    assert _call(**kw) == status


def test_workspace_alignment_and_empty_calls():
    need = poetx.lib.poetx_orthogonalize_workspace_bytes(1, 200, 64, 1)
    assert need > 0 and poetx.lib.poetx_orthogonalize_workspace_bytes(1, 128, 128, 1) == 0
    assert _call(m=200, ws=0x30008, wsb=need) == 3
    for kw in (dict(batch=0), dict(m=0), dict(n=0)):
        assert _call(x=None, out=None, **kw) == 0
    assert poetx.lib.poetx_orthogonalize_workspace_bytes(1, 0, 64, 1) == 0
    assert poetx.lib.poetx_orthogonalize_workspace_bytes(1, 64, 64, 0) == 0
    assert poetx.lib.poetx_orthogonalize_workspace_bytes(-1, 64, 64, 5) == 0
    assert poetx.lib.poetx_orthogonalize_workspace_bytes(65535, 65536, 65536, 5) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(b=1), 1), (dict(b=1025), 2), (dict(nb=-1), 1), (dict(nb=65536), 2), (dict(u=None), 1),
    (dict(out=None), 1), (dict(u=0x10004), 3), (dict(steps=0), 1), (dict(b=200), 8), (dict(nb=0), 0),
])
def test_packed_refusals(kw, status):
    a = dict(u=0x10000, nb=2, b=64, steps=1, out=0x20000)
    a.update(kw)
    c = (ctypes.c_float * 3)(*MUON)
    st = poetx.lib.poetx_orthogonalize_q(a["u"], a["nb"], a["b"], c, a["steps"], 1e-7, 1.0,
                                         a["out"], None, 0, None)
    assert st == status


def test_binding_refusals():
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="CUDA"):
        poetx.orthogonalize(x, torch.zeros(4, 6))
    with pytest.raises(ValueError, match="shape"):
        poetx.orthogonalize(x, torch.zeros(6, 4))
    with pytest.raises(ValueError, match="batch"):
        poetx.orthogonalize(torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="coeffs"):
        poetx.orthogonalize(x, x, steps=3, coeffs=[MUON, MUON])
    with pytest.raises(ValueError, match="fp32"):
        poetx.orthogonalize_q(torch.zeros(1, 6).half(), 4, torch.zeros(1, 6).half())
    with pytest.raises(ValueError, match="nblocks"):
        poetx.orthogonalize_q(torch.zeros(1, 5), 4, torch.zeros(1, 5))
