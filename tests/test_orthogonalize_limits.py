"""The documented limits of poetx_orthogonalize and poetx_orthogonalize_q, from both sides, on the CPU:
what is inside them is refused for its missing workspace only (8), what is outside for its sizes (2) or
coefficients (1), and the workspace query answers 0 there."""
import ctypes

import pytest

try:
    from orthogonal_equivalence_build_b200 import poetx
except ImportError:  # pragma: no cover
    poetx = None

MUON = (3.4445, -4.7750, 2.0315)
INVALID, SHAPE, WORKSPACE = 1, 2, 8


def dense(batch, m, n, rows):
    c = (ctypes.c_float * (3 * len(rows)))(*[v for r in rows for v in r])
    return poetx.lib.poetx_orthogonalize(0x10000, 0, batch, m, n, c, len(rows), 1e-7, 1.0, 0x20000, 0,
                                         None, 0, None)


def packed(nb, b, rows):
    c = (ctypes.c_float * (3 * len(rows)))(*[v for r in rows for v in r])
    return poetx.lib.poetx_orthogonalize_q(0x10000, nb, b, c, len(rows), 1e-7, 1.0, 0x20000, None, 0,
                                           None)


# 3 steps batch ceil(m / 128) ceil(n / 128) up to 2^27 - 1: steps that fit
@pytest.mark.parametrize("batch,m,n,steps", [(65535, 1024, 1024, 10), (65535, 1000, 900, 10),
                                             (512, 4096, 14336, 24), (65535, 2048, 300, 14)])
def test_products_that_the_tile_counters_hold(batch, m, n, steps):
    tiles = 3 * batch * -(-m // 128) * -(-n // 128)
    assert tiles * steps < 2 ** 27 <= tiles * (steps + 1)
    query = poetx.lib.poetx_orthogonalize_workspace_bytes
    assert dense(batch, m, n, [MUON] * steps) == WORKSPACE and query(batch, m, n, steps) > 0
    assert dense(batch, m, n, [MUON] * (steps + 1)) == SHAPE and query(batch, m, n, steps + 1) == 0


def test_the_largest_sizes():
    assert dense(1, 65536, 65536, [MUON] * 64) == WORKSPACE
    assert dense(65535, 129, 1, [MUON] * 64) == WORKSPACE
    for args in ((1, 65537, 1), (1, 1, 65537), (65536, 1, 1)):
        assert dense(*args, [MUON]) == SHAPE


def test_packed_blocks_that_the_tile_counters_hold():
    query = poetx.lib.poetx_orthogonalize_q_workspace_bytes
    assert packed(65535, 1024, [MUON] * 10) == WORKSPACE and query(65535, 1024, 10) > 0
    assert packed(65535, 1024, [MUON] * 11) == SHAPE and query(65535, 1024, 11) == 0


def test_coefficients_within_the_bound_on_singular_values():
    assert dense(1, 200, 64, [(9.7e5, 0.0, 0.0)]) == WORKSPACE
    assert dense(1, 200, 64, [(1.1e6, 0.0, 0.0)]) == INVALID
    # 2 % a step
    assert dense(1, 200, 64, [(1.0, 0.0, 0.0)] * 63 + [(2.8e5, 0.0, 0.0)]) == WORKSPACE
    assert dense(1, 200, 64, [(1.0, 0.0, 0.0)] * 63 + [(2.9e5, 0.0, 0.0)]) == INVALID
    # what B is by itself has no bound
    assert dense(1, 200, 64, [(1e-9, 0.0, 0.0), (1e13, 0.0, 0.0)]) == WORKSPACE
    assert dense(1, 200, 64, [(1e-30, 0.0, 0.0), (3e34, 0.0, 0.0)]) == WORKSPACE


def test_binding_passes_on_no_other_number_of_steps():
    # ctypes keeps the low 32 bits of a number: 2^32 + 5 steps would be five
    torch = pytest.importorskip("torch")
    x, u = torch.zeros(200, 64), torch.zeros(1, 200 * 199 // 2)
    for steps in (2 ** 32 + 5, 2 ** 31, -2 ** 32 + 5):
        for call in (lambda: poetx.orthogonalize_workspace_bytes(x, x, steps),
                     lambda: poetx.orthogonalize_q_workspace_bytes(1, 200, steps),
                     lambda: poetx.orthogonalize(x, torch.empty_like(x), steps=steps),
                     lambda: poetx.orthogonalize_q(u, 200, torch.empty_like(u), steps=steps)):
            with pytest.raises(ValueError, match="steps"):
                call()
    # what the library refuses by itself needs no array of that size
    assert len(poetx._coeff_array(MUON, 2 ** 31 - 1)) <= 3 * 65
    assert poetx.orthogonalize_workspace_bytes(x, x, 65) == 0


def test_a_workspace_serves_every_number_of_steps_beyond_one():
    for args in ((1, 200, 64), (3, 1000, 333), (36, 512, 512)):
        two = poetx.lib.poetx_orthogonalize_workspace_bytes(*args, 2)
        assert all(poetx.lib.poetx_orthogonalize_workspace_bytes(*args, s) == two for s in (5, 8, 64))
