"""How near the Newton-Schulz results come to the recurrence in 64 bits, element by element.

Limits, with rms the root mean square of the exact result. The recurrence on the operands' parts and
scales, worked out in 64 bits on the CPU for Gaussian matrices (5 steps, 60 matrices of a small shape, a
few of a large one) before any output's rounding:

  three part products (operands of 22 bits):   at most 8e-7 in norm, an element 3.5e-6 rms off
  plain fp32 products (numpy), to compare:     at most 2.2e-6 in norm, an element 2.4e-5 rms off

The accumulators' fp32 sums come on top, at plain fp32's level. So for three part products THREE = 6e-5
(an element, in rms) and THREE_NORM = 7e-6 (in norm): about three times plain fp32's. One lost part or
cross product is a relative 2^-12 or more of what it belongs to: 5e-4 to 2e-2 rms. The output's rounding
adds half a step of the element: 2^-8 of it for bf16, 2^-24 for fp32.
"""
import pytest
import torch

try:
    from orthogonal_equivalence_build_b200 import poetx
except ImportError:  # pragma: no cover
    poetx = None

gpu = pytest.mark.gpu
MUON = (3.4445, -4.7750, 2.0315)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
THREE, THREE_NORM = 6e-5, 7e-6


def exact(x, coeffs, eps=1e-7, scale=1.0):
    """The recurrence for a stack, in 64 bits."""
    X = x.double()
    if X.shape[1] > X.shape[2]:
        return exact(x.transpose(1, 2), coeffs, eps, scale).transpose(1, 2)
    X = X / (X.flatten(1).norm(dim=1)[:, None, None] + eps)
    for a, b, c in coeffs:
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return scale * X


def gaussian(shape, dt, seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g).to(DT[dt]).cuda()


def run(x, out_t, coeffs=(MUON,) * 5, **kw):
    out = torch.full(x.shape, 777.0, dtype=out_t, device=x.device)
    poetx.orthogonalize(x, out, steps=len(coeffs), coeffs=list(coeffs), **kw)
    torch.cuda.synchronize()
    poetx.device_status()
    return out


def check_three(got, want):
    """Stacks: every element, and every matrix in norm (fp32 results)."""
    err = (got.double() - want).abs()
    rms = want.square().mean((1, 2), keepdim=True).sqrt()
    half = HALF_STEP[got.dtype]
    over = err - (half * (1 + half) * want.abs() + THREE * rms)
    assert over.max() <= 0, (over / rms).max().item()
    if got.dtype == torch.float32:
        assert ((err.flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)) <= THREE_NORM).all()


# ------------------------------------------------------------------------- bf16 results, few rows
@gpu
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(60, 1, 1), (60, 1, 7), (60, 2, 30), (60, 30, 2), (60, 5, 9),
                                   (60, 8, 40), (20, 16, 16), (20, 64, 64), (10, 100, 120),
                                   (10, 128, 128), (1, 3, 2000), (20, 8, 300), (4, 300, 8),
                                   (3, 64, 700), (3, 700, 65), (3, 100, 500), (2, 128, 700)])
def test_bf16_results_of_few_rows_round_once(shape, xt):
    # few singular values do not average the operands' rounding: with one part per operand 2 x 30 came out
    # up to 6e-3 off in norm, against 1.7e-3 of the output's own rounding
    x = gaussian(shape, xt)
    check_three(run(x, torch.bfloat16), exact(x, [MUON] * 5))


@gpu
def test_bf16_results_of_coinciding_singular_values_round_once():
    # a multiple of an orthogonal matrix: every direction is off by the same amount
    for r in (2, 3, 7, 33, 65, 97, 128):
        x = torch.eye(r, 140, device="cuda")[None]
        check_three(run(x, torch.bfloat16), exact(x, [MUON] * 5))
        check_three(run(x[:, :, :r].contiguous(), torch.bfloat16), exact(x[:, :, :r], [MUON] * 5))


# ------------------------------------------------------------------ schedules that shrink and grow
# Linear steps only scale X, so the limits hold however small it gets; (0, b, 0) cubes the singular
# values and then B = b A alone carries the result.
@gpu
@pytest.mark.parametrize("shape", [(2, 200, 300), (3, 60, 100), (2, 320, 150)])
@pytest.mark.parametrize("coeffs", [
    [(0.01, 0.0, 0.0)] * 4, [(0.001, 0.0, 0.0)] * 4,
    [(0.001, 0.0, 0.0)] * 4 + [(1000.0, 0.0, 0.0)] * 4 + [MUON],
    [(1e-6, 0.0, 0.0), (1e5, 0.0, 0.0), (0.3, -0.2, 0.1)], [(0.0, 0.02, 0.0), (40.0, 0.0, 0.0)],
    [(0.0, 0.0, 1e-4)], [(1e-4, -3e-4, 1e-4), (0.0, 1e3, 0.0)],
    [(1e-9, 0.0, 0.0), (1e13, 0.0, 0.0), (1e-4, 0.0, 0.0)],   # (a factor of B that is large by itself)
], ids=range(8))
def test_schedules_that_shrink_the_singular_values(shape, coeffs):
    x = gaussian(shape, "f32")
    check_three(run(x, torch.float32, coeffs), exact(x, coeffs))


@gpu
@pytest.mark.parametrize("shape", [(2, 60, 100), (2, 200, 300)])
def test_coefficients_of_zero_give_zeros(shape):
    x = gaussian(shape, "f32")
    for out_t in (torch.float32, torch.bfloat16):
        out = run(x, out_t, [MUON, (0.0, 0.0, 0.0), MUON])
        assert torch.equal(out, torch.zeros_like(out))


# ------------------------------------------------------------------------ the caller's scale
@gpu
@pytest.mark.parametrize("shape", [(2, 200, 300), (2, 300, 200), (3, 60, 100)])
@pytest.mark.parametrize("scale", [1e-36, 1e-34, -1e-30, 1e30, 3e37])
def test_scales_near_the_ends_of_fp32(shape, scale):
    x = gaussian(shape, "f32")
    scale = torch.tensor(scale, dtype=torch.float32).item()
    check_three(run(x, torch.float32, scale=scale), exact(x, [MUON] * 5, scale=scale))
    if min(shape[1:]) <= 128 and abs(scale) > 1e-35:   # (bf16's smallest steps are 9e-41)
        check_three(run(x, torch.bfloat16, scale=scale), exact(x, [MUON] * 5, scale=scale))


@gpu
@pytest.mark.parametrize("scale", [1e-36, 1e-30, 3e37])
@pytest.mark.parametrize("b", [64, 200])
def test_packed_scales_near_the_ends_of_fp32(b, scale):
    scale = torch.tensor(scale, dtype=torch.float32).item()
    x = gaussian((2, b, b), "f32")
    x = x - x.transpose(1, 2)
    iu = torch.triu_indices(b, b, 1, device="cuda")
    u = x[:, iu[0], iu[1]].contiguous()
    out = torch.empty_like(u)
    poetx.orthogonalize_q(u, b, out, scale=scale)
    got = torch.zeros_like(x)
    got[:, iu[0], iu[1]] = out
    check_three(got - got.transpose(1, 2), exact(x, [MUON] * 5, scale=scale))


# ------------------------------------------------------------------------- norms below eps
# X_0 is then small, and so may be everything after it; a result's elements are held to the same limits.
@gpu
@pytest.mark.parametrize("shape", [(6, 60, 100), (6, 200, 300), (6, 300, 150), (6, 24, 24)])
@pytest.mark.parametrize("eps", [1e-7, 0.5])
def test_norms_far_below_eps(shape, eps):
    x = gaussian(shape, "f32")
    for i, factor in enumerate((1e3, 1.0, 1e-3, 1e-6, 1e-10, 1e-20)):   # of eps, one matrix each
        x[i] *= factor * eps / x[i].norm()
    eps = torch.tensor(eps, dtype=torch.float32).item()
    want = exact(x, [MUON] * 5, eps)
    check_three(run(x, torch.float32, eps=eps), want)
    if min(shape[1:]) <= 128:
        check_three(run(x, torch.bfloat16, eps=eps), want)


@gpu
def test_norms_far_below_eps_that_grow_to_one():
    # (1.875, -1.25, 0.375) lifts what is small by 1.875 a step and ends at the polar factor
    x = gaussian((3, 60, 100), "f32")
    for i, factor in enumerate((1.0, 1e-6, 1e-10)):
        x[i] *= factor * 1e-7 / x[i].norm()
    eps = torch.tensor(1e-7, dtype=torch.float32).item()
    coeffs = [(1.875, -1.25, 0.375)] * 48
    check_three(run(x, torch.float32, coeffs), exact(x, coeffs, eps))


@gpu
@pytest.mark.parametrize("b", [64, 200])
def test_packed_norms_far_below_eps(b):
    x = gaussian((4, b, b), "f32")
    x = x - x.transpose(1, 2)
    for i, factor in enumerate((1.0, 1e-3, 1e-6, 1e-10)):
        x[i] *= factor * 1e-7 / x[i].norm()
    iu = torch.triu_indices(b, b, 1, device="cuda")
    u = x[:, iu[0], iu[1]].contiguous()
    out = torch.empty_like(u)
    poetx.orthogonalize_q(u, b, out)
    got = torch.zeros_like(x)
    got[:, iu[0], iu[1]] = out
    eps = torch.tensor(1e-7, dtype=torch.float32).item()
    check_three(got - got.transpose(1, 2), exact(x, [MUON] * 5, eps))


# ------------------------------------------------- every tile shape, layout and type, piece by piece
# bf16 results of more than 128 rows come from partly single fp16 operands. The same emulation gives, before
# the output's rounding, at most 1.15e-3 in norm and an element 8.5e-3 rms off (129 to 1100 rows). So an
# element may be off by 2e-2 rms besides its own half step, and a matrix or a piece of 32 x 64 (what a warp
# of the epilogue stores, as worked on) in norm by 1.2e-3 and the rounding's 2^-8 / sqrt(3): 4e-3. fp32
# results: THREE, THREE_NORM, and three times that for a piece of a few thousand elements.
LARGE, LARGE_NORM = 2e-2, 4e-3


def check_pieces(got, want, few=False):
    """got [batch, r, k] as worked on (r <= k); few: bf16 from three part products."""
    err = got.double() - want
    rms = want.square().mean((1, 2), keepdim=True).sqrt()
    f32 = got.dtype == torch.float32
    half, most = HALF_STEP[got.dtype], THREE if f32 or few else LARGE
    over = err.abs() - (half * (1 + half) * want.abs() + most * rms)
    assert over.max() <= 0, (over / rms).max().item()
    norm = lambda t: t.flatten(1).norm(dim=1)
    assert (norm(err) <= (THREE_NORM if f32 else LARGE_NORM) * norm(want)).all()
    b, r, k = want.shape
    cut = lambda t: t[:, :r // 32 * 32, :k // 64 * 64].reshape(b, r // 32, 32, k // 64, 64)
    if r >= 32 and k >= 64:
        e, w = (cut(t).square().sum((2, 4)).sqrt() for t in (err, want))
        limit = 3 * THREE_NORM if f32 else LARGE_NORM
        assert (e <= limit * w).all(), (e / w).max().item()


def planted():
    g = torch.Generator().manual_seed(3)
    want = exact(torch.randn(1, 200, 320, generator=g), [MUON] * 5)
    zero, one_part = want.clone(), want.clone()
    zero[0, 64:96, 128:192] = 0
    one_part[0, 64:96, 128:192] = one_part[0, 64:96, 128:192].half().double()
    return want, zero, one_part


def test_the_limits_see_a_lost_piece_and_a_lost_part():
    want, zero, one_part = planted()
    for t in (torch.float32, torch.bfloat16):
        check_pieces(want.to(t), want)
        with pytest.raises(AssertionError):
            check_pieces(zero.to(t), want)
    with pytest.raises(AssertionError):
        check_pieces(one_part.float(), want)


# in the order of the tiles that sizes lead to: pairs of 256 x 256, 128 x 128 of half of the symmetric
# products, 128 x 128 of all, 128 x 64; tall ones are stored transposed, odd ones without vectors
STACKS = [(3, 1500, 1550), (2, 1800, 1700), (8, 1000, 1003), (5, 1101, 1000), (1, 2305, 2303),
          (1, 2048, 2048), (12, 700, 640), (60, 300, 700), (40, 333, 300), (6, 1024, 521),
          (40, 250, 300), (40, 256, 256), (41, 300, 193), (2, 513, 2100),
          (1, 1000, 333), (2, 300, 1001), (1, 129, 200), (1, 4096, 160), (3, 512, 512)]


@gpu
@pytest.mark.parametrize("shape", STACKS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("xt,ot", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"),
                                   ("bf16", "f32")])
def test_every_piece_of_a_stack(shape, xt, ot):
    x = gaussian(shape, xt)
    got, want = run(x, DT[ot]), exact(x, [MUON] * 5)
    if shape[1] > shape[2]:
        got, want = got.transpose(1, 2), want.transpose(1, 2)
    check_pieces(got, want)


@gpu
@pytest.mark.parametrize("nb,b", [(5, 64), (3, 128), (1, 129), (4, 200), (40, 256), (9, 512), (1, 777),
                                  (2, 1024), (12, 777), (36, 512), (16, 1000), (30, 1024)])
def test_every_piece_of_packed_blocks(nb, b):
    x = gaussian((nb, b, b), "f32")
    x = x - x.transpose(1, 2)
    iu = torch.triu_indices(b, b, 1, device="cuda")
    u = x[:, iu[0], iu[1]].contiguous()
    out = torch.full_like(u, 777.0)
    poetx.orthogonalize_q(u, b, out)
    torch.cuda.synchronize()
    poetx.device_status()
    got = torch.zeros_like(x)
    got[:, iu[0], iu[1]] = out
    check_pieces(got - got.transpose(1, 2), exact(x, [MUON] * 5))


@gpu
@pytest.mark.parametrize("shape", [(2, 96, 200), (2, 400, 200), (3, 1000, 1100)])
@pytest.mark.parametrize("ot", ["f32", "bf16"])
@pytest.mark.parametrize("steps", [1, 2, 3, 8, 12])
def test_step_counts_piece_by_piece(steps, ot, shape):
    # (1.875, -1.25, 0.375) brings errors of the singular values down again, whatever the number of steps
    coeffs = [(1.875, -1.25, 0.375)] * steps
    x = gaussian(shape, "f32")
    got, want = run(x, DT[ot], coeffs, scale=-0.5), exact(x, coeffs, scale=-0.5)
    if shape[1] > shape[2]:
        got, want = got.transpose(1, 2), want.transpose(1, 2)
    check_pieces(got, want, few=min(shape[1:]) <= 128)


# --------------------------------------------------------------------------- shapes at the ends
@gpu
@pytest.mark.parametrize("shape", [(500, 129, 1), (500, 1, 130), (3, 2, 5000), (2, 5000, 2),
                                   (1, 1, 65536), (1, 65536, 1), (2, 40, 20000), (65535, 2, 3),
                                   (2000, 33, 140)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_thin_matrices_and_long_stacks(shape, ot):
    x = gaussian(shape, "bf16")
    check_three(run(x, DT[ot]), exact(x, [MUON] * 5))


@gpu
@pytest.mark.parametrize("shape", [(5, 400, 190), (40, 300, 250), (12, 700, 640), (8, 1000, 1003)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_zero_and_nonfinite_matrices_of_every_tile_shape(shape, ot):
    x = gaussian(shape, "f32")
    want = exact(x, [MUON] * 5)
    x[1] = 0
    x[2, 3, 5] = float("nan")
    x[3, shape[1] - 1, shape[2] - 1] = -float("inf")
    out = run(x, DT[ot])
    assert torch.equal(out[1], torch.zeros_like(out[1]))
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
    pick = [0] + list(range(4, shape[0]))
    got, want = out[pick], want[pick]
    if shape[1] > shape[2]:
        got, want = got.transpose(1, 2), want.transpose(1, 2)
    check_pieces(got, want)
    # without eps, zeros are 0 / 0
    assert torch.isnan(run(x[:2].contiguous(), DT[ot], eps=0.0)[1]).all()


@gpu
@pytest.mark.parametrize("b", [200, 512])
def test_nonfinite_and_zero_packed_blocks_of_many_rows(b):
    g = torch.Generator().manual_seed(b)
    u = torch.randn(5, b * (b - 1) // 2, generator=g).cuda()
    clean, out = torch.empty_like(u), torch.empty_like(u)
    poetx.orthogonalize_q(u, b, clean)
    u[1] = 0
    u[2, 17] = float("nan")
    u[3, -1] = float("inf")
    poetx.orthogonalize_q(u, b, out)
    assert torch.equal(out[[0, 4]], clean[[0, 4]])
    assert torch.equal(out[1], torch.zeros_like(out[1]))
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()


@gpu
@pytest.mark.parametrize("shape", [(4, 200, 300), (4, 640, 400)])
@pytest.mark.parametrize("factor,coeffs", [(1e-3, [MUON] * 5), (1e-10, [MUON] * 5),
                                           (1e3, [(0.001, 0.0, 0.0)] * 3),
                                           (1e-6, [(0.01, 0.0, 0.0), (300.0, 0.0, 0.0), MUON])])
def test_small_iterates_of_large_bf16_results(shape, factor, coeffs):
    x = gaussian(shape, "f32")
    x *= factor * 1e-7 / x.flatten(1).norm(dim=1)[:, None, None]
    eps = torch.tensor(1e-7, dtype=torch.float32).item()
    got, want = run(x, torch.bfloat16, coeffs), exact(x, coeffs, eps)
    if shape[1] > shape[2]:
        got, want = got.transpose(1, 2), want.transpose(1, 2)
    check_pieces(got, want)


@gpu
@pytest.mark.parametrize("shape,xt", [((1100, 1000, 2000), "bf16"), ((1100, 2003, 1000), "f32")])
def test_stacks_of_more_than_two_to_the_31_values(shape, xt):
    x = torch.empty(shape, dtype=DT[xt], device="cuda")
    for i in range(0, shape[0], 100):
        x[i:i + 100] = torch.randn(min(100, shape[0] - i), *shape[1:], device="cuda")
    assert x.numel() > 2 ** 31
    pick = [0, 1, shape[0] // 2, shape[0] - 1]
    want = exact(x[pick], [MUON] * 5)
    got = run(x, DT[xt])[pick]
    if shape[1] > shape[2]:
        got, want = got.transpose(1, 2), want.transpose(1, 2)
    check_pieces(got, want)


@gpu
def test_large_bf16_results_of_few_directions():
    # One direction by itself, on the parts and scales in 64 bits: at most 2.1e-2 off over a million singular
    # values in [1/256, 1], and 1.03e-2 for the values 1 / sqrt(q) of q equal ones.
    x = torch.zeros(40, 300, 500, device="cuda")
    for i, q in enumerate(list(range(1, 30)) + [50, 64, 100, 128, 150, 200, 222, 256, 270, 299, 300]):
        x[i, :q, :q] = torch.eye(q, device="cuda")
    got, want = run(x.bfloat16(), torch.bfloat16).double(), exact(x, [MUON] * 5)
    assert ((got - want).abs() <= (2.2e-2 + 2.0 ** -8) * want.abs()).all()
    got = run(x.bfloat16(), torch.float32).double()   # three part products
    assert ((got - want).abs() <= THREE * want.abs()).all()
