"""Layer norm of rows whose offset is large against their spread, against the formula in 64 bits.

With first = fl(sum x / m), d = x - first and dm = sum d / m the result is ((x - first) - dm) rstd gamma
+ beta, so nothing in it is off by an ulp of the offset. With u = 2^-24 and `adds` the longest chain of
fp32 additions that a row sum can take (m / 32 + 32; a thread of 256 for the widest rows: m / 256 + 16, less):
  first is off by e_first = (adds + 1) u mean|x|, and |d| <= |x - mean| + e_first;
  dm is off by e_dm = (adds + 1) u (mean|x - mean| + e_first), or by u sqrt(var) where it is dropped;
  x - first and its difference from dm round to u of themselves: 2 u (|x - mean| + e_first + max);
  rstd is off by a relative (2 adds + 8) u, the products and the sum by 3 u more.
mean = fl(first + dm) is off by e_dm and half a step, u |mean|.
A layer norm without dm is off by e_first itself: an ulp or so of the offset.
"""
import numpy as np
import pytest
import torch

try:
    from orthogonal_equivalence_build_b200 import poetx
except ImportError:  # pragma: no cover
    poetx = None

gpu = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def rows(T, m, dt, offset, seed=0):
    g = torch.Generator().manual_seed(seed + T + 7 * m)
    x = torch.randn(T, m, generator=g, dtype=torch.float64) + \
        offset * (1.0 + 0.1 * torch.randn(T, 1, generator=g, dtype=torch.float64))
    w = [(1 + 0.2 * torch.randn(m, generator=g)), 0.2 * torch.randn(m, generator=g)]
    return x.to(DT[dt]), w[0], w[1]


def limits(x, gamma, beta, dt):
    """(y, limit), (mean, limit), (rstd, limit) in 64 bits."""
    x, gamma, beta = x.double().numpy(), gamma.double().numpy(), beta.double().numpy()
    m = x.shape[1]
    mean = x.mean(1, keepdims=True)
    d = np.abs(x - mean)
    var = (d * d).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + EPS)
    adds = m / 32 + 32
    e_first = (adds + 1) * U * np.abs(x).mean(1, keepdims=True)
    e_dm = (adds + 1) * U * (d.mean(1, keepdims=True) + e_first) + U * np.sqrt(var)
    e_r = (2 * adds + 8) * U
    e_xh = rstd * (e_dm + 4 * U * (d + e_first)) + d * rstd * (e_r + 3 * U)
    want = (x - mean) * rstd * gamma + beta
    tol = e_xh * np.abs(gamma) + 3 * U * (d * rstd * np.abs(gamma) + np.abs(beta)) + \
        HALF_STEP[dt] * np.abs(want)
    return (want, tol), (mean[:, 0], (e_dm + U * np.abs(mean))[:, 0]), (rstd[:, 0], e_r * rstd[:, 0])


def inside(got, want_tol):
    want, tol = want_tol
    return bool((np.abs(got.double().cpu().numpy() - want) <= tol).all())


def in_fp32(x, gamma, beta, corrected):
    """The kernels' formula in numpy's fp32, with or without the first mean's correction."""
    x = x.float().numpy()
    m = np.float32(x.shape[1])
    # (a plain running sum per row: a chain of m additions would pass the kernels' own, so 32 of them)
    lanes = np.zeros((x.shape[0], 32), np.float32)
    for c in range(0, x.shape[1], 32):
        piece = x[:, c:c + 32]
        lanes[:, :piece.shape[1]] += piece
    first = (lanes.sum(1, dtype=np.float32) / m)[:, None]
    d = x - first
    dm = d.mean(1, keepdims=True, dtype=np.float32) if corrected else np.float32(0)
    var = (d * d).mean(1, keepdims=True, dtype=np.float32) - dm * dm
    y = (d - dm) * (np.float32(1) / np.sqrt(var + np.float32(EPS))) * gamma.numpy() + beta.numpy()
    return torch.from_numpy(y)


WIDTHS = [100, 1023, 1024, 4096, 4099, 8192, 16384, 20000]


@pytest.mark.parametrize("m", WIDTHS)
def test_the_limit_sees_a_missing_correction(m):
    x, gamma, beta = rows(40, m, "f32", 3000.0)
    y = limits(x, gamma, beta, "f32")[0]
    assert inside(in_fp32(x, gamma, beta, True), y)
    assert not inside(in_fp32(x, gamma, beta, False), y)


@gpu
@pytest.mark.parametrize("dt,offset", [("f32", 3000.0), ("f32", -200.0), ("bf16", 60.0)])
@pytest.mark.parametrize("T,m", [(40, m) for m in WIDTHS] + [(1, 4096), (20000, 256), (5000, 1024),
                                                             (3000, 4096), (40, 2047), (40, 5120)])
def test_rows_with_an_offset(T, m, dt, offset):
    x, gamma, beta = rows(T, m, dt, offset)
    y = torch.full_like(x, 777.0, device="cuda")
    mean, rstd = (torch.full((T,), 777.0, device="cuda") for _ in range(2))
    poetx.layer_norm_fwd(x.cuda(), gamma.cuda(), beta.cuda(), y, mean, rstd, eps=EPS)
    torch.cuda.synchronize()
    for got, want in zip((y, mean, rstd), limits(x, gamma, beta, dt)):
        assert inside(got, want)


@gpu
@pytest.mark.parametrize("m", [4096, 4099, 20000])
def test_more_than_two_to_the_31_values(m):
    T = 2 ** 31 // m + 700
    x, dy = (torch.empty(T, m, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i in range(0, T, 50000):
        for t in (x, dy):
            t[i:i + 50000] = torch.randn(min(50000, T - i), m, device="cuda")
    gamma, beta = 1 + 0.2 * torch.randn(m, device="cuda"), 0.2 * torch.randn(m, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dgamma, dbeta = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    poetx.layer_norm_fwd(x, gamma, beta, y, mean, rstd, eps=EPS)
    poetx.layer_norm_bwd(x, dy, gamma, mean, rstd, dx, dgamma, dbeta)
    torch.cuda.synchronize()
    poetx.device_status()
    # the first rows, and those around and behind element 2^31
    pick = torch.cat([torch.arange(50), torch.arange(2 ** 31 // m - 50, 2 ** 31 // m + 50),
                      torch.arange(T - 50, T)]).cuda()
    for got, want in zip((y[pick], mean[pick], rstd[pick]),
                         limits(x[pick].cpu(), gamma.cpu(), beta.cpu(), "bf16")):
        assert inside(got, want)
    # the same rows alone
    part, dg, db = torch.empty_like(x[pick]), torch.empty_like(dgamma), torch.empty_like(dbeta)
    poetx.layer_norm_bwd(x[pick], dy[pick], gamma, mean[pick], rstd[pick], part, dg, db)
    assert torch.equal(part, dx[pick])
    # column sums in 64 bits, each thread's share of the rows in fp32: at most T / 148 additions in a row
    want, size = (torch.zeros(m, dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(0, T, 20000):
        d = dy[i:i + 20000].double()
        want += d.sum(0)
        size += d.abs().sum(0)
    assert ((dbeta.double() - want).abs() <= (T / 148 + 200) * U * size).all()
