"""Layer norm and its gradient (poetx_layer_norm_fwd, poetx_layer_norm_bwd) against the formulas in
64 bits.

Tolerances, element by element, with u = 2^-24 and `adds` the longest chain of fp32 additions that
a row sum can take (a warp per row at least: m / 32 + 32): a sum is off by at most adds u of the sum
of its magnitudes. x - mean is off by e_x = 4 u (|x - first mean| + spread of the mean's error)
after the correction of the first mean; rstd, products and the final scaling add a few u each.
Outputs round once: half a step is 2^-8 (bf16) or 2^-24 (fp32) of the value.
"""
import ctypes

import numpy as np
import pytest
import torch

try:
    from orthogonal_equivalence_build_b200 import poetx
except ImportError:  # pragma: no cover
    poetx = None

gpu = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def out_u(dt):
    return 2.0 ** -8 if dt == "bf16" else 2.0 ** -24


def make(T, m, dt, wt, seed=0, offset=0.5):
    rng = np.random.default_rng(1000 * seed + T + 7 * m)
    x = rng.standard_normal((T, m)) * (0.5 + rng.random(m)) + offset * rng.standard_normal((T, 1))
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).to(DT[d]).cuda()
    return (t(x, dt), t(rng.standard_normal((T, m)), dt), t(1 + 0.2 * rng.standard_normal(m), wt),
            t(0.2 * rng.standard_normal(m), wt))


def f64(t):
    return t.double().cpu().numpy()


def fwd64(x, gamma, beta, eps):
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / np.sqrt((xc * xc).mean(1) + eps)
    xh = xc * rstd[:, None]
    return xh * gamma + beta, mean, rstd, xh


def check_fwd(x, gamma, beta, y, mean, rstd, dt, eps):
    x, m = f64(x), x.shape[1]
    g = np.ones(m) if gamma is None else f64(gamma)
    b = np.zeros(m) if beta is None else f64(beta)
    want, wm, wr, xh = fwd64(x, g, b, eps)
    adds = m / 32 + 32
    absx, absd = np.abs(x).mean(1), np.abs(x - wm[:, None]).mean(1)
    # the first mean's error stays in neither d - dm nor the variance; dm's own is adds u of the
    # deviations (with the first mean's error, adds u mean|x|, added to each)
    e_mean = adds * U * (absd + adds * U * absx) + 2 * U * np.abs(wm)
    if mean is not None:
        assert (np.abs(f64(mean) - wm) <= e_mean + U * absx).all()
    e_r = (2 * adds + 8) * U
    if rstd is not None:
        assert (np.abs(f64(rstd) - wr) <= e_r * wr).all()
    e_xh = wr[:, None] * (adds * U * (absd + adds * U * absx)[:, None] + 4 * U * np.abs(x - wm[:, None])
                          + 2 * U * np.abs(x - wm[:, None]).max(1, keepdims=True)
                          + U * np.abs(wm)[:, None] * 2) + np.abs(xh) * (e_r + 4 * U)
    tol = e_xh * np.abs(g) + 2 * U * (np.abs(xh * g) + np.abs(b)) + out_u(dt) * np.abs(want)
    err = np.abs(f64(y) - want)
    assert (err <= tol).all(), (err - tol).max()


def bwd64(x, dy, gamma, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    c1, c2 = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    return rstd[:, None] * (g - c1 - xh * c2), (dy * xh).sum(0), dy.sum(0), xh, g, c1, c2


def check_bwd(x, dy, gamma, mean, rstd, dx, dgamma, dbeta, dt):
    x, dy, mean, rstd = f64(x), f64(dy), f64(mean), f64(rstd)
    T, m = x.shape
    gm = np.ones(m) if gamma is None else f64(gamma)
    wdx, wdg, wdb, xh, g, c1, c2 = bwd64(x, dy, gm, mean, rstd)
    adds = m / 32 + 32
    e_x = 2 * U * np.abs(x - mean[:, None]) * rstd[:, None] + 2 * U * np.abs(xh)
    e_c1 = (adds + 2) * U * np.abs(g).mean(1, keepdims=True)
    e_c2 = (adds + 4) * U * np.abs(g * xh).mean(1, keepdims=True) + \
        (np.abs(g) * e_x).mean(1, keepdims=True)
    tol = rstd[:, None] * (4 * U * np.abs(g) + e_c1 + np.abs(xh) * e_c2 + e_x * np.abs(c2) +
                           4 * U * (np.abs(c1) + np.abs(xh * c2)))
    if dx is not None:
        err = np.abs(f64(dx) - wdx)
        tol = tol + out_u(dt) * np.abs(wdx)
        assert (err <= tol).all(), (err - tol).max()
    # column sums: at most 600 additions in a row (ranges of rows, then the ranges)
    adds_t = min(T, 600) + 8
    if dgamma is not None:
        tol = (adds_t * U * np.abs(dy * xh) + np.abs(dy) * e_x).sum(0) + U * np.abs(wdg)
        assert (np.abs(f64(dgamma) - wdg) <= tol).all()
    if dbeta is not None:
        assert (np.abs(f64(dbeta) - wdb) <= adds_t * U * np.abs(dy).sum(0)).all()


def run_fwd(x, gamma, beta, eps=1e-5):
    T = x.shape[0]
    y = torch.full_like(x, 777.0)
    mean, rstd = (torch.full((T,), 777.0, device="cuda") for _ in range(2))
    poetx.layer_norm_fwd(x, gamma, beta, y, mean, rstd, eps=eps)
    return y, mean, rstd


def run_bwd(x, dy, gamma, mean, rstd):
    m = x.shape[1]
    dx = torch.full_like(x, 777.0)
    dg, db = (torch.full((m,), 777.0, device="cuda") for _ in range(2))
    poetx.layer_norm_bwd(x, dy, gamma, mean, rstd, dx, dg, db)
    return dx, dg, db


SHAPES = [(1, 1), (3, 1), (1, 2), (2, 3), (1, 7), (5, 8), (1, 64), (300, 31), (33, 100), (129, 512),
          (7, 513), (64, 1000), (257, 1023), (5, 1024), (40, 1032), (3, 2047), (9, 2048), (2, 4096),
          (700, 4096), (3, 4100), (17, 5120), (3, 8191), (5, 8192), (2, 14336), (4, 16384),
          (2, 16391), (3, 20000), (2, 40001), (6000, 24), (4099, 509), (1500, 264)]


@gpu
@pytest.mark.parametrize("dt,wt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"),
                                   ("f32", "bf16")])
@pytest.mark.parametrize("T,m", SHAPES)
def test_forward_and_backward(T, m, dt, wt):
    x, dy, gamma, beta = make(T, m, dt, wt)
    y, mean, rstd = run_fwd(x, gamma, beta)
    check_fwd(x, gamma, beta, y, mean, rstd, dt, 1e-5)
    dx, dg, db = run_bwd(x, dy, gamma, mean, rstd)
    check_bwd(x, dy, gamma, mean, rstd, dx, dg, db, dt)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("m", [200, 1016, 2040, 4088, 8184, 13312, 16384])
def test_rows_that_fill_the_gpu(m, dt):
    """Enough elements (9.7M of bf16, 4.9M of fp32) for several rows per warp or set of threads; the
    last group of rows is not full."""
    T = (9_800_000 if dt == "bf16" else 4_900_000) // m | 1
    x, dy, gamma, beta = make(T, m, dt, "f32")
    y, mean, rstd = run_fwd(x, gamma, beta)
    check_fwd(x, gamma, beta, y, mean, rstd, dt, 1e-5)
    dx, dg, db = run_bwd(x, dy, gamma, mean, rstd)
    check_bwd(x, dy, gamma, mean, rstd, dx, dg, db, dt)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,m", [(50, 96), (20, 515), (9, 2560), (2, 17000)])
def test_optional_arguments(T, m, dt):
    x, dy, gamma, beta = make(T, m, dt, "f32")
    y = torch.empty_like(x)
    for g, b in ((None, None), (gamma, None), (None, beta)):
        poetx.layer_norm_fwd(x, g, b, y)
        check_fwd(x, g, b, y, None, None, dt, 1e-5)
    y, mean, rstd = run_fwd(x, gamma, beta)
    full = run_bwd(x, dy, gamma, mean, rstd)
    dx, dg, db = torch.empty_like(x), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    poetx.layer_norm_bwd(x, dy, gamma, mean, rstd, dx)
    assert torch.equal(dx, full[0])
    poetx.layer_norm_bwd(x, dy, gamma, mean, rstd, None, dg)
    poetx.layer_norm_bwd(x, dy, gamma, mean, rstd, None, None, db)
    assert torch.equal(dg, full[1]) and torch.equal(db, full[2])
    dx, dg, db = run_bwd(x, dy, None, mean, rstd)
    check_bwd(x, dy, None, mean, rstd, dx, dg, db, dt)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,m", [(70, 256), (33, 1021), (19, 4096), (3, 18000)])
def test_in_place(T, m, dt):
    x, dy, gamma, beta = make(T, m, dt, "f32")
    y, mean, rstd = run_fwd(x, gamma, beta)
    z = x.clone()
    poetx.layer_norm_fwd(z, gamma, beta, z)
    assert torch.equal(z, y)
    want = run_bwd(x, dy, gamma, mean, rstd)
    for which in (0, 1):
        a, d = x.clone(), dy.clone()
        out = (a, d)[which]
        dg, db = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
        poetx.layer_norm_bwd(a, d, gamma, mean, rstd, out, dg, db)
        assert torch.equal(out, want[0])
        assert torch.equal(dg, want[1]) and torch.equal(db, want[2])


@gpu
@pytest.mark.parametrize("m", [100, 1024, 4096, 4099])
def test_rows_with_a_large_offset(m):
    x, dy, gamma, beta = make(40, m, "f32", "f32", seed=3, offset=3000.0)
    y, mean, rstd = run_fwd(x, gamma, beta)
    check_fwd(x, gamma, beta, y, mean, rstd, "f32", 1e-5)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("m", [64, 333, 4096, 17000])
def test_constant_rows_and_nonfinite_rows(m, dt):
    x, dy, gamma, beta = make(6, m, dt, "f32")
    x[1] = 0.0
    x[2] = 2.5
    x[3, m // 2] = float("nan")
    x[4, 0] = float("inf")
    y, mean, rstd = run_fwd(x, gamma, beta)
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    assert torch.isnan(rstd[3]) and torch.isnan(rstd[4])
    keep = [0, 1, 2, 5]
    check_fwd(x[keep], gamma, beta, y[keep], mean[keep], rstd[keep], dt, 1e-5)
    assert torch.equal(y[1], beta.to(x.dtype))
    dx, dg, db = run_bwd(x, dy, gamma, mean, rstd)
    assert torch.isnan(dx[3]).all() and torch.isnan(dg).all()
    check_bwd(x[keep], dy[keep], gamma, mean[keep], rstd[keep], dx[keep], None, None, dt)


@gpu
def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    dg, db = torch.full((64,), 5.0, device="cuda"), torch.full((64,), 5.0, device="cuda")
    s = torch.empty(0, device="cuda")
    poetx.layer_norm_fwd(x, w, w, torch.empty_like(x), s, s)
    poetx.layer_norm_bwd(x, x, w, s, s, torch.empty_like(x), dg, db)
    assert (dg == 0).all() and (db == 0).all()


@gpu
@pytest.mark.parametrize("T,m", [(6, 48), (3, 129), (2, 1024)])
def test_gradient_against_differences(T, m):
    """Directional differences of L = sum(w y), summed in 64 bits from the fp32 y of the forward.
    h = 2^-7: the truncation error is h^2 / 6 of the third derivative (~6 |L'| here), 6e-5; y's
    rounding, 2^-22 sqrt(T m) |w y| / h, 2e-5 sqrt(T m)."""
    x, w, gamma, beta = make(T, m, "f32", "f32", seed=4)
    y, mean, rstd = run_fwd(x, gamma, beta)
    dx, dg, db = run_bwd(x, w, gamma, mean, rstd)
    h = 2.0 ** -7
    rng = np.random.default_rng(5)

    def loss(x_, g_, b_):
        return float((f64(run_fwd(x_, g_, b_)[0]) * f64(w)).sum())

    for grad, make_args, shape in (
            (dx, lambda d: (x + d, gamma, beta), (T, m)),
            (dg, lambda d: (x, gamma + d, beta), (m,)),
            (db, lambda d: (x, gamma, beta + d), (m,))):
        d = rng.standard_normal(shape)
        d = torch.from_numpy(d / np.linalg.norm(d)).float().cuda()
        diff = (loss(*make_args(h * d)) - loss(*make_args(-h * d))) / (2 * h)
        want = float((f64(grad) * f64(d)).sum())
        assert abs(diff - want) <= 1e-4 * np.linalg.norm(f64(grad)) + 2e-5 * np.sqrt(T * m)


@gpu
@pytest.mark.parametrize("T,m,dt", [(37, 200, "f32"), (13, 515, "bf16"), (300, 4096, "bf16"),
                                    (2, 16999, "f32")])
def test_writes_only_its_outputs(T, m, dt):
    x, dy, gamma, beta = make(T, m, dt, "f32")

    def guarded(n, dtype):
        buf = torch.full((n + 128,), 3.0, dtype=dtype, device="cuda")
        return buf, buf[64:64 + n]

    bufs = [guarded(T * m, x.dtype), guarded(T, torch.float32), guarded(T, torch.float32),
            guarded(T * m, x.dtype), guarded(m, torch.float32), guarded(m, torch.float32)]
    y, mean, rstd, dx, dg, db = (b[1] for b in bufs)
    need = poetx.layer_norm_bwd_workspace_bytes(T, m)
    wbuf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    poetx.layer_norm_fwd(x, gamma, beta, y.view(T, m), mean, rstd)
    poetx.layer_norm_bwd(x, dy, gamma, mean, rstd, dx.view(T, m), dg, db,
                         workspace=wbuf[256:256 + need])
    torch.cuda.synchronize()
    for buf, v in bufs:
        assert (buf[:64] == 3).all() and (buf[64 + v.numel():] == 3).all()
    assert (wbuf[:256] == 0x5A).all() and (wbuf[256 + need:] == 0x5A).all()
    check_bwd(x, dy, gamma, mean, rstd, dx.view(T, m), dg, db, dt)


@gpu
def test_graph_replay_and_other_stream():
    x, dy, gamma, beta = make(257, 1024, "bf16", "f32")
    y, mean, rstd = run_fwd(x, gamma, beta)
    want = run_bwd(x, dy, gamma, mean, rstd)
    outs = [torch.empty_like(t) for t in (y, mean, rstd, *want)]
    ws = torch.empty(poetx.layer_norm_bwd_workspace_bytes(257, 1024), dtype=torch.uint8,
                     device="cuda")

    def step(stream=None):
        poetx.layer_norm_fwd(x, gamma, beta, *outs[:3], stream=stream)
        poetx.layer_norm_bwd(x, dy, gamma, outs[1], outs[2], *outs[3:], workspace=ws,
                             stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    for o, w in zip(outs, (y, mean, rstd, *want)):
        assert torch.equal(o, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, (y, mean, rstd, *want)):
            assert torch.equal(o, w)


@gpu
@pytest.mark.parametrize("m", [512, 1021, 8192, 12000])
def test_inputs_written_by_the_launch_before(m):
    """Forward and backward in place, over and over: every launch reads what the one before wrote."""
    x, dy, gamma, beta = make(301, m, "f32", "f32")
    mean, rstd = torch.empty(301, device="cuda"), torch.empty(301, device="cuda")
    dg, db = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")

    def chain(wait):
        a, d = x.clone(), dy.clone()
        torch.cuda.synchronize()
        for _ in range(10):
            poetx.layer_norm_fwd(a, gamma, beta, a, mean, rstd)
            if wait:
                torch.cuda.synchronize()
            poetx.layer_norm_bwd(a, d, gamma, mean, rstd, d, dg, db)
            if wait:
                torch.cuda.synchronize()
        return a, d, mean.clone(), rstd.clone(), dg.clone(), db.clone()

    for got, want in zip(chain(False), chain(True)):
        assert torch.equal(got, want)


# ----------------------------------------------------------------------------- refusals (CPU)
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(T=-1), 1), (dict(m=-1), 1), (dict(eps=-1e-5), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(m=(1 << 20) + 1), 2),
    (dict(dt=2), 4), (dict(wd=-1), 4), (dict(x=0x10002), 3), (dict(gamma=0x20004), 3),
    (dict(beta=0x20008), 3), (dict(y=0x30001), 3), (dict(mean=0x40004), 3), (dict(rstd=0x40004), 3),
    (dict(T=0, x=None, y=None), 0), (dict(m=0), 0), (dict(T=1 << 62, m=4), 2),
])
def test_forward_refusals(kw, status):
    a = dict(x=0x10000, T=4, m=64, dt=0, gamma=0x20000, beta=0x28000, wd=0, eps=1e-5, y=0x30000,
             mean=0x40000, rstd=0x50000)
    a.update(kw)
    assert poetx.lib.poetx_layer_norm_fwd(a["x"], a["T"], a["m"], a["dt"], a["gamma"], a["beta"],
                                          a["wd"], a["eps"], a["y"], a["mean"], a["rstd"],
                                          None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(dy=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1),
    (dict(T=-1), 1), (dict(m=-5), 1), (dict(m=(1 << 20) + 1), 2), (dict(dt=9), 4), (dict(wd=9), 4),
    (dict(x=0x10004), 3), (dict(dy=0x18004), 3), (dict(dx=0x30004), 3), (dict(dgamma=0x60004), 3),
    (dict(dbeta=0x60008), 3), (dict(gamma=0x20001), 3), (dict(), 8),
    (dict(ws=0x90000, wsb=4), 8), (dict(ws=0x90004, wsb=1 << 30), 3),
    (dict(dx=None, dgamma=None, dbeta=None), 0), (dict(m=0), 0), (dict(T=1 << 49, m=4), 2),
])
def test_backward_refusals(kw, status):
    a = dict(x=0x10000, dy=0x18000, T=4, m=64, dt=0, gamma=0x20000, wd=0, mean=0x40000,
             rstd=0x50000, dx=0x30000, dgamma=0x60000, dbeta=0x70000, ws=None, wsb=0)
    a.update(kw)
    assert poetx.lib.poetx_layer_norm_bwd(a["x"], a["dy"], a["T"], a["m"], a["dt"], a["gamma"],
                                          a["wd"], a["mean"], a["rstd"], a["dx"], a["dgamma"],
                                          a["dbeta"], a["ws"], a["wsb"], None) == status


def test_workspace_query():
    q = poetx.lib.poetx_layer_norm_bwd_workspace_bytes
    assert q(0, 64) == 0 and q(64, 0) == 0 and q(-1, 64) == 0 and q(4, (1 << 20) + 1) == 0
    assert q(1, 1) > 0 and q(1 << 40, 4096) < 1 << 30


def test_binding_refusals():
    x, w, s = torch.zeros(4, 6), torch.ones(6), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        poetx.layer_norm_fwd(x, w, w, torch.zeros(4, 6))
    with pytest.raises(ValueError, match="y must be"):
        poetx.layer_norm_fwd(x, w, w, torch.zeros(4, 7))
    with pytest.raises(ValueError, match="y must be"):
        poetx.layer_norm_fwd(x, w, w, torch.zeros(4, 6).bfloat16())
    with pytest.raises(ValueError, match="gamma"):
        poetx.layer_norm_fwd(x, torch.ones(5), w, torch.zeros(4, 6))
    with pytest.raises(ValueError, match="one dtype"):
        poetx.layer_norm_fwd(x, w.bfloat16(), w, torch.zeros(4, 6))
    with pytest.raises(ValueError, match="mean"):
        poetx.layer_norm_fwd(x, w, w, torch.zeros(4, 6), torch.zeros(5))
    with pytest.raises(ValueError, match="dgamma"):
        poetx.layer_norm_bwd(x, x, w, s, s, x, w.bfloat16())
    with pytest.raises(ValueError, match="T, m"):
        poetx.layer_norm_fwd(torch.zeros(6), w, w, torch.zeros(6))
