"""Pins of the plain references that the 4-bit and SwiGLU kernels are compared
with: hand-worked values, closed properties, and differences for the gradient.
No GPU."""
import numpy as np
import pytest

import lowbit_ref as ref


def test_e2m1_rounding_by_hand():
    v = np.array([0.24, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6.0, 100.0])
    want = [0, 0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, 6]
    assert list(ref.E2M1[ref.nearest(ref.E2M1, v)]) == want


def test_fp8_tables():
    assert ref.FP8[ref.E4M3][-1] == 448 and ref.FP8[ref.E4M3][1] == 2.0 ** -9
    assert ref.FP8[ref.E5M2][-1] == 57344 and ref.FP8[ref.E5M2][1] == 2.0 ** -16


def test_mx_block_by_hand():
    x = np.zeros((1, 40))
    x[0, :4] = [7.0, -1.0, 0.5, 0.25]     # amax 7: 2^2, so 2^0; 7 saturates at 6
    x[0, 32:34] = [0.015625, -0.01]       # the short block: 2^-6, so 2^-8
    c, s = ref.fp4_quant(x, ref.MX)
    assert list(s[0]) == [127, 119]
    assert list(c[0, :4]) == [7, 8 | 2, 1, 0] and list(c[0, 32:34]) == [6, 8 | 5]   # 4, and -2.56 to -3


def test_nv_block_by_hand():
    x = np.zeros((1, 17))
    x[0, :3] = [12.0, -3.0, 1.0]          # amax / 6 = 2: s = 2, quotients 6, -1.5, 0.5
    x[0, 16] = 1e-9                       # s rounds to 0: codes 0
    c, s = ref.fp4_quant(x, ref.NV)
    assert ref.scale_values(s, ref.NV)[0, 0] == 2.0 and s[0, 1] == 0
    assert list(c[0, :3]) == [7, 8 | 3, 1] and c[0, 16] == 0


@pytest.mark.parametrize("kind", [ref.MX, ref.NV])
def test_values_quantize_to_themselves(kind):
    # NV: a block's own largest code has to be 6, or its scale would change
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (5, 64)).astype(np.uint8)
    codes[:, ::16] = 7
    scales = rng.integers(100 if kind == ref.MX else 0x20, 140 if kind == ref.MX else 0x70,
                          (5, 64 // ref.BLOCK[kind])).astype(np.uint8)
    v = ref.fp4_values(codes, scales, kind)
    c, s = ref.fp4_quant(v, kind)
    assert np.array_equal(s, scales) and np.array_equal(ref.fp4_values(c, s, kind), v)


def test_tensor_scale_is_the_least_power_of_two():
    for a in (2688.0, 2700.0, 1e-6, 3e4):
        t = ref.tensor_scale(np.array([a, -a / 2]))
        assert a <= 2688 * t and a > 2688 * t / 2
    assert ref.tensor_scale(np.zeros(3)) == 1.0


def test_scale_tiles_are_a_permutation():
    for kind in (ref.MX, ref.NV):
        rows, k = 300, 700
        nb = -(-k // ref.BLOCK[kind])
        r, j = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
        at = ref.scale_offset(r, j, k, kind)
        assert len(np.unique(at)) == at.size and at.max() < ref.tile_scales(np.zeros((rows, nb)), k, kind).size


def test_pack_round_trip():
    c = np.random.default_rng(1).integers(0, 16, (3, 37)).astype(np.uint8)
    assert np.array_equal(ref.unpack(ref.pack(c), 37), c)


@pytest.mark.parametrize("fmt", [ref.E4M3, ref.E5M2])
def test_round_up_scale_is_tight(fmt):
    top = 448.0 if fmt == ref.E4M3 else 57344.0
    a = np.exp(np.random.default_rng(2).uniform(-60, 60, 2000))
    s = np.exp2(ref.ue8m0(a, fmt).astype(float))
    assert (a <= top * s).all() and (a > top * s / 2).all()
    assert (ref.ue8m0(np.array([top, top * 2, top * 1.001]), fmt) == [0, 1, 1]).all()


def test_gradients_are_the_slopes_of_the_forward():
    rng = np.random.default_rng(3)
    g, u = rng.normal(0, 3, 500), rng.normal(0, 2, 500)
    dg, du = ref.swiglu_grads(g, u, np.ones(500))
    eps = 1e-5
    ng = (ref.swiglu(g + eps, u) - ref.swiglu(g - eps, u)) / (2 * eps)
    nu = (ref.swiglu(g, u + eps) - ref.swiglu(g, u - eps)) / (2 * eps)
    # third derivatives are below 1: eps^2 / 6 of them, and cancellation 1e-16 * |h| / eps
    assert np.abs(dg - ng).max() < 1e-8 and np.abs(du - nu).max() < 1e-8
