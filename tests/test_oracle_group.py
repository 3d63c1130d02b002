"""Pins of the expert-grouped oracle: the dispatch against a sort, the products
against loops over single elements, every gradient against central differences
of its forward function, the 4-bit layout against the library's packer."""

import numpy as np
import pytest

from oracle import group as OG


def test_plan_is_a_stable_sort():
    rng = np.random.default_rng(0)
    idx = rng.integers(-2, 9, (40, 3))
    offsets, pairs, pos = OG.plan(idx, 7)
    flat = idx.reshape(-1)
    held = np.flatnonzero((flat >= 0) & (flat < 7))
    want = held[np.argsort(flat[held], kind="stable")]
    n = len(want)
    assert offsets[-1] == n and np.array_equal(pairs[:n], want) and np.all(pairs[n:] == -1)
    assert np.array_equal(pos[want], np.arange(n))
    assert np.all(pos[flat == -1] == -1) and np.all(pos[(flat < -1) | (flat >= 7)] == -2)
    assert np.array_equal(np.diff(offsets), np.bincount(flat[held], minlength=7))


def test_products_by_element():
    rng = np.random.default_rng(1)
    offsets = [0, 2, 2, 5]
    x, w = rng.standard_normal((6, 4)), rng.standard_normal((3, 3, 4))
    y = OG.matmul(x, offsets, w, 6)
    group = [0, 0, 2, 2, 2]
    for i in range(5):
        for n in range(3):
            assert np.isclose(y[i, n], sum(x[i, k] * w[group[i], n, k] for k in range(4)))
    assert np.all(np.isnan(y[5]))
    dw = OG.wgrad(y[:5], x[:5], offsets, 3)
    assert np.all(dw[1] == 0)
    assert np.isclose(dw[2][1, 3], sum(y[i, 1] * x[i, 3] for i in (2, 3, 4)))
    assert OG.groups_of([3, 1, 9, 4], 6) == [(0, 3, 3), (1, 1, 6), (2, 6, 6)]
    assert np.array_equal(OG.gathered(np.arange(6.0).reshape(3, 2), [5, -1, 0, 6], 2), [[4, 5], [0, 0], [0, 1], [0, 0]])


def differences(f, at, eps=1e-6):
    g = np.zeros_like(at)
    for i in np.ndindex(at.shape):
        hi, lo = at.copy(), at.copy()
        hi[i] += eps
        lo[i] -= eps
        g[i] = (f(hi) - f(lo)) / (2 * eps)
    return g


def test_gradients_against_differences():
    """Loss = sum(c * output) for a fixed c; central differences of step 1e-6 are good to about 1e-9."""
    rng = np.random.default_rng(2)
    offsets, rows = [0, 1, 1, 4], 4
    x, w = rng.standard_normal((rows, 5)), rng.standard_normal((3, 6, 5))
    c = rng.standard_normal((rows, 6))
    tol = dict(rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(OG.matmul_t(c, offsets, w, rows),
                               differences(lambda v: np.sum(c * OG.matmul(v, offsets, w, rows)), x), **tol)
    np.testing.assert_allclose(OG.wgrad(c, x, offsets, 3),
                               differences(lambda v: np.sum(c * OG.matmul(x, offsets, v, rows)), w), **tol)
    pre, ch = 3 * rng.standard_normal((rows, 6)), rng.standard_normal((rows, 3))
    np.testing.assert_allclose(OG.swiglu_grad(ch, pre), differences(lambda v: np.sum(ch * OG.swiglu(v)), pre), **tol)
    o, wts = rng.standard_normal((4, 6)), rng.standard_normal((2, 2))
    pos, cy = np.array([2, 0, -1, 3]), rng.standard_normal((2, 6))
    d_o, d_w = OG.combine_grad(cy, o, pos, wts, 2)
    np.testing.assert_allclose(np.nan_to_num(d_o),
                               differences(lambda v: np.sum(cy * OG.combine(v, pos, wts, 2, 2)), o), **tol)
    np.testing.assert_allclose(d_w, differences(lambda v: np.sum(cy * OG.combine(o, pos, v, 2, 2)), wts), **tol)
    assert np.all(np.isnan(OG.combine(o, [4, 0, -2, 1], wts, 2, 2)))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("n,k,group", [(16, 128, 32), (5, 96, 32), (33, 320, 64), (17, 384, 128)])
def test_q4_packer_matches_the_layout(n, k, group, zeros):
    from bit_moe_expert_02_amd import _lib as L
    rng = np.random.default_rng(n + k)
    w = (rng.standard_normal((n, k)) * 0.02).astype(np.float32)
    w[0, :group] = 0.0                                   # a group without a scale
    w[-1, -group:] = 1e-9                                # a scale that underflows to 0
    w[1, 0] = 3.0
    codes, scales, zr = OG.q4_quantise(w, group, zeros)
    got = L.q4_pack(w, group, zeros, nthreads=3)
    for a, b in zip(got, OG.q4_layout(codes, scales, zr, group)):
        assert (a is None) == (b is None) and (a is None or np.array_equal(a, b))
    back = L.q4_unpack(*got, n, k, group, nthreads=2)
    assert np.array_equal(back.astype(np.float64), OG.q4_values(codes, scales, zr, group))
