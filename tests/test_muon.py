"""CPU checks of the Muon step: the oracle on closed forms, refusals and planning of the C ABI."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import muon as O


@pytest.fixture(scope="module")
def F():
    import nvfp4_precision_optimizer_b200 as F
    F._lib.lib()
    return F


def test_oracle_acts_on_singular_values():
    rng = np.random.default_rng(0)
    q1, _ = np.linalg.qr(rng.standard_normal((12, 7)))
    q2, _ = np.linalg.qr(rng.standard_normal((7, 7)))
    s = np.linspace(0.1, 2.0, 7)
    want = s / np.sqrt((s * s).sum())
    for a, b, c in [O.MUON, (1.5, -0.5, 0.0)] * 3:
        want = a * want + b * want ** 3 + c * want ** 5
    got = O.orthogonalize(q1 * s @ q2.T, 6, [O.MUON, (1.5, -0.5, 0.0)] * 3)
    np.testing.assert_allclose(got, q1 * want @ q2.T, atol=1e-7)


def test_diagonals_out_of_the_operands_is_the_same_iteration():
    """A^2 and a X + B X with the diagonals taken out and added back, as the kernels do."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((6, 9))
    A = x @ x.T
    d = np.diag(A)
    A0 = A - np.diag(d)
    np.testing.assert_allclose(A0 @ A0 + A0 * (d[:, None] + d[None]) + np.diag(d * d), A @ A)
    e = np.diag(A @ A)
    np.testing.assert_allclose((2.0 + e)[:, None] * x + (A @ A - np.diag(e)) @ x, 2.0 * x + A @ A @ x)


def _desc(F, base, rows=32, cols=48, step=True, **kw):
    d = F._lib.MuonDesc(base, base + (1 << 28), base + (2 << 28) if step else None, rows, cols, cols, cols, cols, 0, 1, 0, 1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_refusals(F):
    lib = F._lib.lib()
    one = (ctypes.c_float * 3)(*O.MUON)
    size = lambda *s: F.muon_workspace_size(list(s))  # noqa: E731
    need, ws, base = size((32, 48)), 1 << 40, 1 << 32

    def step(count=1, K=5, coeffs=one, nc=1, lr=1e-3, beta=0.9, wd=0.0, flags=1, w=ws, nbytes=need, descs=None, **kw):
        arr = (F._lib.MuonDesc * 1)(_desc(F, base, **kw)) if descs is None else descs
        return lib.fs4_muon_step(count, arr, K, coeffs, nc, lr, beta, wd, flags, w, nbytes, None)

    for bad in (dict(w=None), dict(g=None), dict(m=None), dict(ld_w=47), dict(ld_g=1), dict(ld_m=0), dict(w_dtype=3), dict(g_dtype=-1),
                dict(m_dtype=9), dict(scale=float("nan")), dict(ld_w=1 << 62)):
        if bad == dict(w=None):
            arr = (F._lib.MuonDesc * 1)(_desc(F, base))
            arr[0].w = None
            assert step(descs=arr) == -1
            continue
        assert step(**bad) == -1, bad
    assert step(rows=0) == -2 and step(cols=65537, ld_w=65537, ld_g=65537, ld_m=65537) == -2
    assert step(count=0) == -2 and step(count=225) == -2 and step(K=0) == -2 and step(K=33) == -2
    assert step(nc=2) == -1 and step(coeffs=(ctypes.c_float * 3)(17.0, 0, 0)) == -1
    assert step(coeffs=(ctypes.c_float * 3)(float("nan"), 0, 0)) == -1
    assert step(lr=-1.0) == -1 and step(lr=float("inf")) == -1 and step(beta=1.0) == -1 and step(beta=-0.1) == -1
    assert step(wd=float("nan")) == -1 and step(flags=2) == -1
    assert step(w=None) == -4 and step(w=ws + 128) == -4 and step(nbytes=need - 1) == -4
    assert step(w=base - need // 256 * 256 + 1024) == -3                       # workspace over the weights
    arr = (F._lib.MuonDesc * 1)(_desc(F, base))
    arr[0].g = arr[0].w
    assert step(descs=arr) == -3
    arr = (F._lib.MuonDesc * 2)(_desc(F, base), _desc(F, base + (5 << 28)))
    arr[1].w = arr[0].m
    assert lib.fs4_muon_step(2, arr, 5, one, 1, 1e-3, 0.9, 0.0, 1, ws, size((32, 48), (32, 48)), None) == -3
    arr = (F._lib.MuonDesc * 1)(_desc(F, base))                                 # a momentum where none belongs
    assert lib.fs4_muon_orthogonalize(1, arr, 5, one, 1, ws, need, None) == -1


def test_workspace_sizes(F):
    assert F.muon_workspace_size([(0, 4)]) == 0 and F.muon_workspace_size([(4, 65537)]) == 0
    assert F.muon_workspace_size([(16, 16)] * 225) == 0
    a, b = F.muon_workspace_size([(300, 1000)]), F.muon_workspace_size([(1000, 300)])
    # X in three FP16 parts, A in two and B in one, and two diagonals, on sizes padded to 256,
    # beside the table of matrices, the partial sums and, for a small call, at most 296 partial
    # tiles of 32 KB
    floor = 6 * 512 * 1024 + 6 * 512 * 512 + 8 * 512
    assert floor < a <= floor + (1 << 16) + 296 * 32768 and floor < b <= floor + (1 << 16) + 296 * 32768
    big, block = F.muon_workspace_size([(4096, 4096)] * 3), 12 * 4096 * 4096 + 8 * 4096
    assert 3 * block < big <= 3 * block + (1 << 17)


def test_binding_refusals(F):
    with pytest.raises(ValueError, match="coeffs"):
        F._muon_coeffs([(1, 2, 3)] * 4, 5)
    with pytest.raises(ValueError, match="one length"):
        F.muon_step([torch.zeros(2, 2)], [], [], 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        F.muon_orthogonalize([torch.zeros(2, 2)])
    assert F.muon_orthogonalize([]) == []
    assert F._muon_scale("spectral", 8, 2) == 2.0 and F._muon_scale("spectral", 2, 8) == 1.0
    assert F._muon_scale("rms", 25, 4) == 1.0 and F._muon_scale(3, 1, 1) == 3.0


def test_coefficient_ranges(F):
    """|a| <= 16 and |b s + c s^2| <= 255 on [0, 1]: accepted triples get as far as the workspace."""
    size = F.muon_workspace_size([(32, 48)])

    def call(*triples):
        d = (F._lib.MuonDesc * 1)(_desc(F, 1 << 32, step=False))
        flat = [v for t in triples for v in t]
        return F._lib.lib().fs4_muon_orthogonalize(1, d, len(triples), (ctypes.c_float * len(flat))(*flat), len(triples),
                                                   1 << 40, size - 1, None)

    steep = (8.16, -22.5, 15.9)
    for ok in (O.MUON, steep, (16.0, 16.0, 16.0), (-16.0, 0.0, 255.0), (1.0, 1000.0, -1000.0), (0.0, -255.0, 0.0), (1.0, -31.0, 1.0)):
        assert call(ok) == -4 and call(steep, ok) == -4, ok
    for bad in ((16.5, 0, 0), (1, 256, 0), (1, 0, -256), (1, 1100, -1100), (1, float("inf"), 0), (1, 0, float("nan")),
                (1, 3e38, -3e38), (float("-inf"), 0, 0)):
        assert call(bad) == -1 and call(steep, bad) == -1, bad


def test_rates_outside_fp32_are_refused(F):
    one, size = (ctypes.c_float * 3)(*O.MUON), F.muon_workspace_size([(32, 48)])

    def step(lr, wd):
        d = (F._lib.MuonDesc * 1)(_desc(F, 1 << 32))
        return F._lib.lib().fs4_muon_step(1, d, 5, one, 1, lr, 0.9, wd, 0, 1 << 40, size - 1, None)

    assert step(3e38, 0.0) == -4 and step(1e30, 1e8) == -4 and step(0.0, 1e300) == -4 and step(1e-3, -5.0) == -4
    for lr, wd in ((1e39, 0.0), (1e30, 1e9), (1e30, -1e9), (1e300, 1e300), (float("nan"), 0.0), (0.0, float("inf"))):
        assert step(lr, wd) == -1, (lr, wd)


def test_column_slices_overlap_where_they_share_a_byte(F):
    """Weights, gradients and momenta of two matrices as slices of one buffer."""
    lib, one = F._lib.lib(), (ctypes.c_float * 3)(*O.MUON)
    need, base, ws = F.muon_workspace_size([(32, 48)] * 2), 1 << 32, 1 << 40

    def step(offset, cols=(48, 48), ld=(400, 400), what="w", rows=(32, 32), space=ws):
        """Matrix 1's `what` starts `offset` bytes after matrix 0's w."""
        arr = (F._lib.MuonDesc * 2)(_desc(F, base), _desc(F, base + (5 << 28)))
        for d, c, r in zip(arr, cols, rows):
            d.cols, d.rows = c, r
        arr[0].ld_w = ld[0]
        setattr(arr[1], what, base + offset)
        setattr(arr[1], "ld_" + what, ld[1])
        setattr(arr[1], what + "_dtype", 0)
        return lib.fs4_muon_step(2, arr, 5, one, 1, 1e-3, 0.9, 0.0, 1, space, need, None)

    for what in "wgm":
        for shared in (47 * 4, 48 * 4 - 4, 1600 - 47 * 4, 1600 * 31, 0, -47 * 4, -1600 + 47 * 4, 1600 * 3 + 4):
            assert step(shared, what=what) == -3, (what, shared)
        assert step(48 * 4, ld=(400, 408), what=what) == -3             # another pitch
    assert step(360 * 4) == -3                                          # the second's rows reach the first's next ones
    assert step(48 * 4, space=base + 512) == -3                         # a workspace over the gaps
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would launch on these addresses")
    for what in "wgm":
        for apart in (48 * 4, 1600 - 48 * 4, 1600 * 31 + 48 * 4, -48 * 4, -1600 + 48 * 4, 1600 * 40):
            assert step(apart, what=what) in (-5, -6), (what, apart)    # as far as the device check
    assert step(48 * 4, rows=(32, 1), ld=(400, 48)) in (-5, -6)         # one row has no pitch


def test_stall_flag_of_the_step(F):
    one, size = (ctypes.c_float * 3)(*O.MUON), F.muon_workspace_size([(32, 48)])
    d = (F._lib.MuonDesc * 1)(_desc(F, 1 << 32))
    step = lambda flags: F._lib.lib().fs4_muon_step(1, d, 5, one, 1, 0.1, 0.9, 0.0, flags, 1 << 40, size - 1, None)  # noqa: E731
    assert step(F.FS4_TEST_STALL) == -4 and step(F.FS4_TEST_STALL | 1) == -4 and step(F.FS4_TEST_STALL | 2) == -1
