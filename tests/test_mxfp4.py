"""CPU checks of MXFP4: the oracle against the definition by hand, and the refusals of the C ABI
and of the binding (nothing here launches a kernel)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import mxfp4 as O


@pytest.fixture(scope="module")
def F():
    import nvfp4_precision_optimizer_b200 as F
    F._lib.lib()
    return F


def test_oracle_blocks_by_hand():
    # amax 7: floor rule 2^0 (7 saturates at 6), ceil rule 2^1 (7 / 2 = 3.5 is a tie: the even code 4)
    x = np.zeros((1, 33))
    x[0, :6] = [7.0, -0.25, 0.75, 2.5, 5.0, -0.0]
    x[0, 32] = 2.0 ** -140
    c, s = O.quantize(x)
    assert c[0, :6].tolist() == [7, 8, 2, 4, 6, 8] and s[0].tolist() == [127, 0]
    assert O.values(c, s)[0, :5].tolist() == [6.0, -0.0, 1.0, 2.0, 4.0]
    c, s = O.quantize(x, "ceil")
    assert c[0, :6].tolist() == [6, 8, 1, 2, 4, 8] and s[0].tolist() == [128, 0]
    # a block with NaN or Inf is NaN as a whole, its neighbour is not
    x[0, 3] = np.inf
    c, s = O.quantize(x)
    assert s[0].tolist() == [255, 0] and not c[0, :32].any() and np.isnan(O.values(c, s)[0, :32]).all()


def test_oracle_stochastic_rounding_is_unbiased_and_uses_the_stated_draws():
    assert O.draws(1, 4, 0)[0].tolist() == [(0xE220A8397B1DCDAF >> s) & 0xFFFF for s in (0, 16, 32, 48)]
    x = np.full((4096, 32), 2.75)
    x[:, 0] = 6.0
    c, s = O.quantize(x, "floor", seed=5)
    v = O.values(c, s)[:, 1:]
    assert set(np.unique(v)) == {2.0, 3.0}
    # the mean of n draws of variance 3/16 lies within 5 sqrt(3 / 16 n) of 2.75
    assert abs(v.mean() - 2.75) < 5 * np.sqrt(3 / 16 / v.size)


def _fake():
    ws = ctypes.create_string_buffer(1024)
    return ws, (ctypes.addressof(ws) + 255) // 256 * 256


def test_quantize_refusals(F):
    q, p = F._lib.lib().fs4_mxfp4_quantize, 1 << 20
    far = [p * 4 ** i for i in range(1, 6)]
    good = [far[0], 1, 5, 7, 7, far[1], far[2], far[3], far[4], 0, 0, None]

    def with_(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return q(*a)

    assert with_(_0=None) == -1
    assert with_(_5=None) == -1 and with_(_8=None) == -1                       # half a view
    assert with_(_5=None, _6=None, _7=None, _8=None) == -1                     # no view
    assert with_(_1=3) == -1 and with_(_1=-1) == -1                            # unknown type
    assert with_(_9=1 << 8) == -1 and with_(_9=F._lib.FS4_MX_ACCUMULATE) == -1  # unknown flags
    assert with_(_2=0) == -2 and with_(_3=0) == -2 and with_(_2=-4) == -2 and with_(_3=(1 << 31) + 1) == -2
    assert with_(_4=6) == -1 and with_(_4=1 << 62) == -1                       # leading dimension
    assert with_(_5=far[1] + 8) == -1 and with_(_0=far[0] + 1) == -1           # alignment
    assert with_(_7=far[1]) == -3 and with_(_5=far[0]) == -3                   # overlap


def test_dequantize_and_product_refusals(F):
    lib, p = F._lib.lib(), 1 << 20
    ws, wsp = _fake()
    far = [p * 4 ** i for i in range(1, 7)]
    d = lib.fs4_mxfp4_dequantize
    assert d(None, far[1], 4, 8, far[2], 0, 8, 0, None) == -1
    assert d(far[0], far[1], 4, 8, far[2], 0, 7, 0, None) == -1
    assert d(far[0], far[1], 4, 8, far[2], 9, 8, 0, None) == -1
    assert d(far[0], far[1], 0, 8, far[2], 0, 8, 0, None) == -2
    assert d(far[0], far[1], 4, 8, far[0], 0, 8, 0, None) == -3
    assert d(far[0], far[1], 4, 8, far[2], 0, 8, F._lib.FS4_MX_STOCHASTIC, None) == -1
    good = [far[0], far[1], far[2], far[3], 5, 6, 7, far[4], 0, 6, 0, wsp, 256, None]

    def gemm(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.fs4_mxfp4_gemm(*a)

    for i in (0, 1, 2, 3, 7):
        assert gemm(**{f"_{i}": None}) == -1
    for i in (4, 5, 6):
        assert gemm(**{f"_{i}": 0}) == -2 and gemm(**{f"_{i}": (1 << 20) + 1}) == -2
    assert gemm(_9=5) == -1 and gemm(_8=7) == -1 and gemm(_10=1) == -1 and gemm(_0=far[0] + 4) == -1
    assert gemm(_7=far[0]) == -3 and gemm(_7=wsp) == -3
    assert gemm(_11=None) == -4 and gemm(_11=wsp + 64) == -4 and gemm(_12=255) == -4
    need = lib.fs4_mxfp4_linear_workspace_size(5, 7)
    assert need == 256 + 128 * 256 // 32 * 17
    assert lib.fs4_mxfp4_linear_workspace_size(0, 7) == 0
    lin = [far[0], 1, 5, 7, 7, far[1], far[2], 6, far[3], 1, 6, 0, far[4], need, None]

    def linear(**kw):
        a = list(lin)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.fs4_mxfp4_linear(*a)

    assert linear(_0=None) == -1 and linear(_5=None) == -1 and linear(_8=None) == -1 and linear(_1=5) == -1
    assert linear(_2=0) == -2 and linear(_7=0) == -2 and linear(_4=6) == -1 and linear(_10=5) == -1
    assert linear(_13=need - 1) == -4 and linear(_12=far[4] + 16) == -4
    assert linear(_8=far[0]) == -3 and linear(_12=far[0]) == -3 and linear(_8=far[4] + 512) == -3
    assert linear(_11=F._lib.FS4_MX_STOCHASTIC) == -1


def test_binding_refuses_before_it_calls(F):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        F.mxfp4_quantize(x)
    with pytest.raises(ValueError, match="CUDA"):
        F.mxfp4_linear(x, (x, x), 4)
    with pytest.raises(ValueError, match="scale_rule"):
        F._mx_scale_flag("round")


def test_tiled_sizes(F):
    assert F.mxfp4_tiled_shape(1, 1) == (128 * 128, 128 * 8)
    assert F.mxfp4_tiled_shape(129, 257) == (256 * 256, 256 * 16)
    c, s = O.pack_tiled(*O.quantize(np.ones((129, 257))))
    assert (len(c), len(s)) == F.mxfp4_tiled_shape(129, 257)


def test_linear_with_a_status_word_of_its_own_refusals(F):
    lib, p = F._lib.lib(), 1 << 20
    far = [p * 4 ** i for i in range(1, 8)]
    need = lib.fs4_mxfp4_linear_workspace_size(5, 7)
    good = [far[0], 1, 5, 7, 7, far[1], far[2], 6, far[3], 1, 6, 0, far[4], need, far[5], None]

    def linear(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.fs4_mxfp4_linear_ex(*a)

    assert linear(_14=None) == -4 and linear(_14=far[5] + 128) == -4 and linear(_13=need - 1) == -4
    assert linear(_14=far[4] + 256) == -3 and linear(_14=far[0]) == -3 and linear(_14=far[1]) == -3
    assert linear(_14=far[2]) == -3 and linear(_14=far[3]) == -3 and linear(_8=far[4] + 512) == -3
    assert F.device_status() == 0                       # no call was made, and no device is needed


def test_stall_flag_is_the_products_alone(F):
    lib, p = F._lib.lib(), 1 << 20
    far = [p * 4 ** i for i in range(1, 7)]
    stall = F.FS4_TEST_STALL
    assert lib.fs4_mxfp4_quantize(far[0], 1, 5, 7, 7, far[1], far[2], None, None, stall, 0, None) == -1
    assert lib.fs4_mxfp4_dequantize(far[0], far[1], 4, 8, far[2], 0, 8, stall, None) == -1
    gemm = lambda flags: lib.fs4_mxfp4_gemm(*far[:4], 5, 6, 7, far[4], 0, 6, flags, None, 256, None)  # noqa: E731
    assert gemm(stall) == -4 and gemm(stall | 128) == -4 and gemm(stall | 1) == -1
    linear = lambda flags: lib.fs4_mxfp4_linear(far[0], 1, 5, 7, 7, far[1], far[2], 6, far[3], 1, 6, flags, None, 0, None)  # noqa: E731
    assert linear(stall) == -4 and linear(stall | 32 | 128) == -4 and linear(stall | 2) == -1
