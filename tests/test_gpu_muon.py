"""The Muon step on the GPU against the 64-bit oracle.

The contract is accuracy to BF16: at most 2^-9 (Frobenius, relative) from the exact iteration
before the output's own rounding, which adds at most half a step of its type."""
import itertools

import numpy as np
import pytest
import torch

from oracle import mxfp4 as MX
from oracle import muon as O

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NEAR = 2.0 ** -9
SHAPES = [(1, 1), (1, 40), (40, 1), (2, 3), (16, 16), (31, 33), (128, 256), (257, 255), (300, 1111), (1030, 129), (513, 520), (33, 8190),
          (129, 4100), (2050, 70), (1100, 1300)]


def half_step(t):
    return torch.finfo(t).eps / 2


def make(m, n, dtype=torch.float32, seed=0, rank=None):
    g = torch.Generator().manual_seed(7919 * m + n + seed)
    x = torch.randn(m, n, generator=g)
    if rank:
        x = 0.05 * x + torch.randn(m, rank, generator=g) @ torch.randn(rank, n, generator=g)
    return (0.02 * x).to(dtype)


def np64(t):
    return t.detach().cpu().double().numpy()


def far(got, want):
    return np.linalg.norm(np64(got) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_orthogonalize_against_float64(fs4, shape, kind):
    G = make(*shape, TYPES[kind])
    want = O.orthogonalize(np64(G))
    ws = torch.empty(fs4.muon_workspace_size([shape]), dtype=torch.uint8, device="cuda")
    for t in TYPES.values():
        out = fs4.muon_orthogonalize([G.cuda()], dtype=t, workspace=ws)[0]
        assert out.dtype == t and out.shape == G.shape
        assert far(out, want) <= NEAR + half_step(t)
        assert fs4.device_status(ws) == 0


@pytest.mark.parametrize("rank", (1, 16, 64))
@pytest.mark.parametrize("shape", [(200, 200), (256, 700), (900, 300)], ids=str)
def test_orthogonalize_low_rank(fs4, shape, rank):
    G = make(*shape, rank=rank)
    assert far(fs4.muon_orthogonalize([G.cuda()], dtype=torch.float32)[0], O.orthogonalize(np64(G))) <= NEAR


def test_products_one_iteration_at_a_time(fs4):
    """Each term of the polynomial on its own, over several 256-blocks in each direction."""
    G = make(600, 1300)
    for coeffs in ((1.0, 0.0, 0.0), (0.0, 1.0, 0.0), (0.0, 0.0, 1.0), (0.5, -2.0, 1.0)):
        want = O.orthogonalize(np64(G), 1, coeffs)
        got = fs4.muon_orthogonalize([G.cuda()], K=1, coeffs=coeffs, dtype=torch.float32)[0]
        # operands rounded to FP16 enter the result at most five times (X once, or A0 twice and X)
        assert far(got, want) <= (2.0 ** -20 if coeffs[1:] == (0.0, 0.0) else 5 * 2.0 ** -12), coeffs
    per = [O.MUON, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)]
    assert far(fs4.muon_orthogonalize([G.cuda()], K=3, coeffs=per, dtype=torch.float32)[0], O.orthogonalize(np64(G), 3, per)) <= NEAR


def test_many_iterations_reach_the_polar_factor(fs4):
    G = make(300, 500)
    u, _, vt = np.linalg.svd(np64(G), full_matrices=False)
    got = fs4.muon_orthogonalize([G.cuda()], K=20, coeffs=(1.875, -1.25, 0.375), dtype=torch.float32)[0]
    assert far(got, u @ vt) <= NEAR


def test_batch_is_each_matrix_alone_bit_for_bit(fs4):
    Gs = [make(*s, t).cuda() for s, t in zip(SHAPES, [torch.float32, torch.bfloat16, torch.float16] * 4)]
    batch = fs4.muon_orthogonalize(Gs)
    again = fs4.muon_orthogonalize(Gs)
    for G, b, a in zip(Gs, batch, again):
        assert torch.equal(b, a) and torch.equal(b, fs4.muon_orthogonalize([G])[0])


def test_strided_inputs_and_outputs(fs4):
    big = make(400, 900, torch.bfloat16).cuda()
    for G in (big[3:300, 5:705], big[::2, 8:520], big[:, :17], big[5:6]):
        want = fs4.muon_orthogonalize([G.contiguous()])[0]
        wide = torch.full((G.shape[0], G.shape[1] + 9), 3.0, dtype=torch.bfloat16, device="cuda")
        fs4.muon_orthogonalize([G], outs=[wide[:, 4:-5]])
        assert torch.equal(wide[:, 4:-5], want) and (wide[:, :4] == 3).all() and (wide[:, -5:] == 3).all()


@pytest.mark.parametrize("shape", [(1, 300), (20, 77), (77, 20), (300, 411), (411, 300), (1500, 1900), (1900, 1501)], ids=str)
def test_rows_past_the_weights_and_momenta_stay_as_they_are(fs4, shape):
    m, n = shape
    G = make(m, n).cuda()
    W, M = (torch.full((m + 3, n), 5.0, device="cuda") for _ in range(2))
    w, v = torch.full((m, n), 5.0, device="cuda"), torch.full((m, n), 5.0, device="cuda")
    fs4.muon_step([W[1:m + 1]], [G], [M[1:m + 1]], lr=0.1, weight_decay=0.1)
    fs4.muon_step([w], [G], [v], lr=0.1, weight_decay=0.1)
    for big, one in ((W, w), (M, v)):
        assert torch.equal(big[1:m + 1], one) and (big[0] == 5).all() and (big[m + 1:] == 5).all()


def test_zero_tiny_and_huge_updates(fs4):
    G = make(60, 90)
    want = fs4.muon_orthogonalize([G.cuda()])[0]
    assert not fs4.muon_orthogonalize([torch.zeros(60, 90, device="cuda")])[0].any()
    for scale in (2.0 ** 60, 2.0 ** 100):
        assert torch.equal(fs4.muon_orthogonalize([G.cuda() * scale])[0], fs4.muon_orthogonalize([G.cuda() * 2.0 ** 30])[0])
    assert far(want, np64(fs4.muon_orthogonalize([G.cuda() * 2.0 ** 30])[0])) <= 2 * NEAR
    # the 1e-7 beside a small norm
    assert far(fs4.muon_orthogonalize([G.cuda() * 1e-8], dtype=torch.float32)[0], O.orthogonalize(np64(G * 1e-8))) <= NEAR


def test_nonfinite_matrix_is_reported_and_harms_no_other(fs4):
    shapes = [(40, 70), (300, 200), (64, 64)]
    Gs = [make(*s).cuda() for s in shapes]
    want = fs4.muon_orthogonalize(Gs)
    for bad in (float("nan"), float("inf")):
        Gs[1][299, 3] = bad
        ws = torch.empty(fs4.muon_workspace_size(shapes), dtype=torch.uint8, device="cuda")
        got = fs4.muon_orthogonalize(Gs, workspace=ws)
        assert fs4.device_status(ws) == -7
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and not got[1].any()
        w = [torch.ones(s, device="cuda") for s in shapes]
        m = [torch.zeros(s, device="cuda") for s in shapes]
        fs4.muon_step(w, Gs, m, lr=0.5, weight_decay=0.5, workspace=ws)
        assert fs4.device_status(ws) == -7 and (w[1] == 0.75).all() and not (w[0] == 0.75).all()
    fs4.muon_orthogonalize([Gs[0]], workspace=ws)
    assert fs4.device_status(ws) == 0
    # a diverging iteration is reported too
    fs4.muon_orthogonalize([Gs[0]], K=8, coeffs=(16.0, 16.0, 16.0), workspace=ws)
    assert fs4.device_status(ws) == -7


@pytest.mark.parametrize("nesterov", (False, True))
@pytest.mark.parametrize("types", [("f32", "f32", "f32"), ("f32", "bf16", "f32"), ("bf16", "bf16", "bf16"), ("f16", "f16", "f16"),
                                   ("bf16", "f32", "f16")], ids=str)
def test_step_against_float64(fs4, types, nesterov):
    tw, tg, tm = (TYPES[t] for t in types)
    shapes = [(96, 200), (333, 77), (1, 65), (512, 512)]
    lr, beta, wd = 0.02, 0.9, 0.1
    W, G, M = ([make(*s, t, k).mul(f).cuda() for s in shapes] for t, k, f in ((tw, 1, 2.0), (tg, 2, 1.0), (tm, 3, 0.5)))
    W0, G0, M0 = ([np64(t) for t in ts] for ts in (W, G, M))
    ws = torch.empty(fs4.muon_workspace_size(shapes), dtype=torch.uint8, device="cuda")
    fs4.muon_step(W, G, M, lr=lr, beta=beta, nesterov=nesterov, weight_decay=wd, workspace=ws)
    assert fs4.device_status(ws) == 0
    for w, m, w0, g0, m0 in zip(W, M, W0, G0, M0):
        new = beta * m0 + (1 - beta) * g0
        # beta and 1 - beta rounded, one product and one fused sum: four roundings
        size = beta * np.abs(m0) + (1 - beta) * np.abs(g0)
        tiny = float(torch.finfo(tm).smallest_normal) * float(torch.finfo(tm).eps)
        assert (np.abs(np64(m) - new) <= 4 * 2.0 ** -24 * size + half_step(tm) * (np.abs(new) + 4 * 2.0 ** -24 * size) + tiny).all()
        kept = np64(m)
        x = O.orthogonalize(beta * kept + (1 - beta) * g0 if nesterov else kept)
        step = lr * 0.2 * max(w0.shape) ** 0.5 * x
        want = (1 - lr * wd) * w0 - step
        error = np.linalg.norm(np64(w) - want)
        assert error <= (NEAR + 2.0 ** -22) * np.linalg.norm(step) + (half_step(tw) + 2.0 ** -22) * np.linalg.norm(want)


def test_step_scales(fs4):
    for shape in ((30, 120), (120, 30)):
        G = make(*shape).cuda()
        x = fs4.muon_orthogonalize([G], dtype=torch.float32)[0]
        for scale, f in (("spectral", max(1.0, shape[0] / shape[1]) ** 0.5), ("rms", 0.2 * 120 ** 0.5), (3.0, 3.0)):
            w, m = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
            fs4.muon_step([w], [G], [m], lr=0.25, beta=0.0, nesterov=False, scale=scale)
            assert far(w, np64(x) * -0.25 * f) <= 2.0 ** -20


def test_streams_and_graphs(fs4):
    shapes = [(100, 300), (520, 64)]
    G = [make(*s, torch.bfloat16).cuda() for s in shapes]
    want = fs4.muon_orthogonalize(G)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = [fs4.muon_orthogonalize(G, stream=s) for s in (side, None, side)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in runs for a, b in zip(r, want))
    W, M = ([torch.zeros(s, device="cuda") for s in shapes] for _ in range(2))
    W2, M2 = ([t.clone() for t in ts] for ts in (W, M))
    ws = torch.zeros(fs4.muon_workspace_size(shapes), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs4.muon_step(W, G, M, lr=0.1, workspace=ws)
    for _ in range(3):
        graph.replay()
        fs4.muon_step(W2, G, M2, lr=0.1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(W + M, W2 + M2))


def test_two_steps_at_once_with_workspaces_of_their_own(fs4):
    """Steps of both kernel kinds on two streams, none waiting for the other."""
    shapes = [(900, 1400), (64, 200), (20, 900), (2048, 2304)]
    Gs = [make(*s, torch.bfloat16).cuda() for s in shapes]
    want = [fs4.muon_orthogonalize([G])[0] for G in Gs]
    spaces = [torch.empty(fs4.muon_workspace_size([s]), dtype=torch.uint8, device="cuda") for s in shapes]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for G, ws, st in zip(Gs, spaces, streams):
            outs.append(fs4.muon_orthogonalize([G], workspace=ws, stream=st)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % len(shapes)]) for i, o in enumerate(outs))
    assert all(fs4.device_status(ws) == 0 for ws in spaces)


def test_large_batch_takes_the_whole_table(fs4):
    """More matrices than the small parameter block holds, thin and wide ones mixed."""
    shapes = [(1 + 37 * i % 90, 1 + 53 * i % 310) for i in range(224)]
    Gs = [make(*s).cuda() for s in shapes]
    outs = fs4.muon_orthogonalize(Gs, K=3)
    for i in (0, 7, 100, 150, 223):
        assert torch.equal(outs[i], fs4.muon_orthogonalize([Gs[i]], K=3)[0])
        assert far(outs[i], O.orthogonalize(np64(Gs[i]), 3)) <= NEAR + half_step(torch.bfloat16)
    with pytest.raises(fs4.Fs4Error):
        fs4.muon_orthogonalize(Gs + Gs[:1])


def test_refusals_on_device(fs4):
    G, W = torch.zeros(8, 16, device="cuda"), torch.zeros(8, 16, device="cuda")
    with pytest.raises(ValueError):
        fs4.muon_orthogonalize([G.t()[:, :3].t().t()])
    with pytest.raises(ValueError):
        fs4.muon_orthogonalize([G], outs=[torch.zeros(8, 15, device="cuda")])
    with pytest.raises(ValueError):
        fs4.muon_step([W], [G[:, :8]], [torch.zeros(8, 16, device="cuda")], 0.1)
    with pytest.raises(fs4.Fs4Error):
        fs4.muon_orthogonalize([G], workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fs4.Fs4Error):
        fs4.muon_step([W], [G], [W], 0.1)                      # momentum and weights in one place
    with pytest.raises(fs4.Fs4Error):
        fs4.muon_orthogonalize([G], outs=[G])
    with pytest.raises(fs4.Fs4Error):
        fs4.muon_step([W], [G], [torch.zeros(8, 16, device="cuda")], 0.1, beta=1.5)


def test_training_step_in_four_bits(fs4):
    """One linear layer: quantise, forward, both gradients, Muon, quantise the new weights."""
    T, n_in, n_out, lr = 160, 130, 270, 0.05
    x, dy = make(T, n_in, torch.bfloat16, 1).mul(50).cuda(), make(T, n_out, torch.bfloat16, 2).mul(50).cuda()
    w = make(n_out, n_in, torch.float32, 3).cuda()
    m, dw = torch.zeros_like(w), torch.zeros_like(w)
    W0 = np64(w)
    xr, xc = fs4.mxfp4_quantize_both(x, tiled=True)
    wr, wc = fs4.mxfp4_quantize_both(w, tiled=True)
    gr, gc = fs4.mxfp4_quantize_both(dy, tiled=True, seed=1)
    y = fs4.mxfp4_linear(x, wr, n_out)
    dx = fs4.mxfp4_gemm(gr, wc, T, n_in, n_out)
    fs4.mxfp4_gemm(gc, xc, n_out, n_in, T, out=dw, accumulate=True)
    fs4.muon_step([w], [dw], [m], lr=lr)
    wr2, _ = fs4.mxfp4_quantize_both(w, tiled=True)

    val = lambda t, seed=None: MX.values(*MX.quantize(t, "floor", seed))  # noqa: E731
    X, G = np64(x), np64(dy)
    step = torch.finfo(torch.bfloat16).eps / 2 + 2.0 ** -15
    assert far(y, val(X) @ val(W0).T) <= step
    assert far(dx, val(G, 1) @ val(W0.T).T) <= step
    want = val(G.T, 1 ^ MX.COLUMN_SEED) @ val(X.T).T
    assert far(dw, want) <= T * 2.0 ** -23 * 4
    moved = W0 - lr * 0.2 * max(w.shape) ** 0.5 * O.orthogonalize(want)
    assert np.linalg.norm(np64(w) - moved) <= (NEAR + 2.0 ** -15) * np.linalg.norm(moved - W0) + 2.0 ** -23 * np.linalg.norm(moved)
    codes, scales = MX.pack_tiled(*MX.quantize(np64(w)))
    assert np.array_equal(wr2[0].cpu().numpy(), codes) and np.array_equal(wr2[1].cpu().numpy(), scales)


def dominated(m, n, kind, noise):
    """One or few dominant directions over `noise` times as much noise an element."""
    g = torch.Generator().manual_seed(31 * m + n)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    if kind == "few rows":
        x = noise * rand(m, n)
        x[:5] += rand(5, 1) @ rand(1, n)
        return x
    if kind == "one row above all":          # three quarters of the direction in one row
        u = rand(m, 1)
        u[0] = 0
        u *= 0.5 / u.norm()
        u[0] = 0.75 ** 0.5
        return (u @ rand(1, n) + noise * rand(m, n) * m ** -0.5)
    if kind == "fading rows":
        return 0.6 ** torch.arange(m, dtype=torch.float64)[:, None] @ rand(1, n) + noise * rand(m, n)
    return rand(m, 4 if kind == "rank 4" else 1) @ rand(4 if kind == "rank 4" else 1, n) + noise * rand(m, n)


@pytest.mark.parametrize("noise", (1e-2, 1e-3, 1e-4))
@pytest.mark.parametrize("kind", ("rank 1", "rank 4", "few rows", "one row above all", "fading rows"))
@pytest.mark.parametrize("shape", [(40, 300), (64, 64), (128, 128), (411, 300), (2000, 1400)], ids=str)
def test_dominant_directions_leave_the_small_ones_exact(fs4, shape, kind, noise):
    """The iteration raises small singular values up to a^5 = 485 times, and so an error that
    the dominant ones leave among them.  The contract's bound, on both kernels."""
    G = dominated(*shape, kind, noise).float()
    got = fs4.muon_orthogonalize([G.cuda()], dtype=torch.float32)[0]
    if G.numel() < 1 << 20:
        assert far(got, O.orthogonalize(np64(G))) <= NEAR
    else:
        x = G.cuda().double()
        x = x.T / (x.norm() + 1e-7)
        for _ in range(5):
            a = x @ x.T
            x = O.MUON[0] * x + (O.MUON[1] * a + O.MUON[2] * (a @ a)) @ x
        assert far(got, np64(x.T)) <= NEAR


@pytest.mark.parametrize("shape", [(64, 64), (200, 200), (300, 40)], ids=str)
def test_converging_iterations_keep_small_directions(fs4, shape):
    G = dominated(*shape, "rank 1", 1e-3).float()
    per = (1.875, -1.25, 0.375)
    got = fs4.muon_orthogonalize([G.cuda()], K=20, coeffs=per, dtype=torch.float32)[0]
    assert far(got, O.orthogonalize(np64(G), 20, per)) <= NEAR


@pytest.mark.parametrize("shape", [(20, 90), (1, 33), (90, 64), (300, 411)], ids=str)
def test_updates_near_the_largest_fp32_values(fs4, shape):
    """1 / ||U|| is not a normal FP32 number from a norm of 2^126 on; a power of two on U is exact."""
    G = make(*shape)
    G = G / G.abs().max()
    want = fs4.muon_orthogonalize([G.cuda() * 2.0 ** 20], dtype=torch.float32)[0]
    for scale in (2.0 ** 110, 2.0 ** 124, 2.0 ** 127):
        got = fs4.muon_orthogonalize([(G * scale).cuda()], dtype=torch.float32)[0]
        # T or X_0 is rounded to FP32 once, wherever the power of two is
        assert far(got, np64(want)) <= 2.0 ** -20, scale
        w = torch.zeros(shape, device="cuda")
        m = torch.zeros(shape, device="cuda")
        fs4.muon_step([w], [(G * scale).cuda()], [m], lr=1.0, beta=0.0, nesterov=False, scale=1.0)
        assert torch.equal(w, -got)


@pytest.mark.parametrize("shape", [(64, 64), (200, 310), (1500, 1900), (20, 500)], ids=str)
def test_steep_first_triples(fs4, shape):
    """A schedule whose first triples have large b and c, as those that converge fastest do.  It
    raises small singular values 1000 times, where the Muon triple raises them 485 times: twice
    the bound."""
    per = [(8.16, -22.5, 15.9), (4.1, -2.95, 0.545), (3.95, -2.91, 0.552), (3.3, -2.49, 0.51), (2.3, -1.67, 0.42)]
    ws = torch.empty(fs4.muon_workspace_size([shape]), dtype=torch.uint8, device="cuda")
    G = make(*shape)
    got = fs4.muon_orthogonalize([G.cuda()], coeffs=per, dtype=torch.float32, workspace=ws)[0]
    assert far(got, O.orthogonalize(np64(G), 5, per)) <= 2 * NEAR and fs4.device_status(ws) == 0


def test_iterates_that_leave_the_operands_range_are_reported(fs4):
    """One element of 16 in X (a = 16 on a matrix of one element), and a B over 255."""
    G = torch.zeros(64, 64, device="cuda")
    G[3, 5] = 2.0
    ones = torch.ones(64, 64, device="cuda")
    for x, per in ((G, [(16.0, 0.0, 0.0), (1.0, 0.0, 0.0)]), (ones, [(16.0, 16.0, 16.0), (16.0, 16.0, 16.0)])):
        ws = torch.empty(fs4.muon_workspace_size([(64, 64)]), dtype=torch.uint8, device="cuda")
        fs4.muon_orthogonalize([x], K=len(per), coeffs=per, workspace=ws)
        assert fs4.device_status(ws) == -7


@pytest.mark.parametrize("shapes", [[(300, 40), (300, 200), (300, 7)], [(20, 33), (20, 31)], [(1300, 1024), (1300, 1400)]], ids=str)
def test_slices_of_one_buffer_step_as_matrices_of_their_own(fs4, shapes):
    """Projections stored side by side, gradients and momenta too, at odd offsets."""
    rows, total = shapes[0][0], sum(n for _, n in shapes)
    buffers = [make(rows, total + 3, t, k).cuda() for t, k in ((torch.float32, 1), (torch.bfloat16, 2), (torch.float32, 3))]
    at = [1 + sum(n for _, n in shapes[:i]) for i in range(len(shapes))]
    cut = lambda b: [b[:, c:c + n] for c, (_, n) in zip(at, shapes)]  # noqa: E731
    alone = [[t.clone() for t in cut(b)] for b in buffers]
    edges = [b[:, [0, -2, -1]].clone() for b in buffers]
    fs4.muon_step(*map(cut, buffers), lr=0.1, weight_decay=0.1)
    fs4.muon_step(*alone, lr=0.1, weight_decay=0.1)
    for b, ts, e in zip(buffers, alone, edges):
        assert torch.equal(b[:, [0, -2, -1]], e)
        for x, y in zip(cut(b), ts):
            # rows off 16 bytes add their squares up in another order: X_0 may differ by a step of
            # FP32, which moves one in 2^12 of its elements by 2^-11 in the operands
            assert far(x, np64(y)) <= 2.0 ** -15
    assert all(torch.equal(x, y) for b, ts in zip(buffers[1:], alone[1:]) for x, y in zip(cut(b), ts))
    with pytest.raises(fs4.Fs4Error):
        fs4.muon_step([buffers[0][:, :9], buffers[0][:, 8:20]], [g[:, :w] for g, w in zip(cut(buffers[1])[:1] * 2, (9, 12))],
                      [torch.zeros(rows, w, device="cuda") for w in (9, 12)], lr=0.1)


def test_status_of_calls_without_a_workspace(fs4):
    fs4.device_status()                           # what earlier calls left
    good, bad = make(40, 70).cuda(), make(300, 200).cuda()
    bad[299, 3] = float("nan")
    fs4.muon_orthogonalize([good])
    assert fs4.device_status() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        fs4.muon_orthogonalize([bad, good], stream=stream)
        fs4.muon_orthogonalize([good], stream=stream)              # does not hide it
        assert fs4.device_status() == -7 and fs4.device_status() == 0
        fs4.muon_step([torch.zeros_like(bad)], [bad], [torch.zeros_like(bad)], lr=0.1, stream=stream)
        assert fs4.device_status() == -7 and fs4.device_status() == 0
    ws = torch.empty(fs4.muon_workspace_size([bad.shape]), dtype=torch.uint8, device="cuda")
    fs4.muon_orthogonalize([bad], workspace=ws)
    assert fs4.device_status(ws) == -7 and fs4.device_status() == 0


def test_calls_without_a_workspace_in_graphs(fs4):
    """Captured on a stream that made no such call before, and on one that did."""
    G = make(64, 100).cuda()
    w = fs4.mxfp4_quantize(make(64, 100).cuda(), tiled=True)
    want, y = fs4.muon_orthogonalize([G])[0], fs4.mxfp4_linear(G, w, 64)
    p = fs4.mxfp4_gemm(w, w, 64, 64, 100)
    fs4.device_status()
    for warm in (False, True):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        if warm:
            fs4.mxfp4_gemm(w, w, 64, 64, 100, stream=stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = [fs4.muon_orthogonalize([G])[0], fs4.mxfp4_linear(G, w, 64), fs4.mxfp4_gemm(w, w, 64, 64, 100)]
        for _ in range(2):
            for o in outs:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, (want, y, p)))
        assert fs4.device_status() == 0
        if warm:
            kept = G.clone()
            G[3, 3] = float("inf")
            graph.replay()
            assert fs4.device_status() == -7
            G.copy_(kept)


@pytest.mark.parametrize("shapes", [[(64, 200)], [(64, 4096), (20, 30), (200, 300)], [(1500, 1900)], [(20, 700), (600, 2100), (1300, 900)]], ids=str)
def test_wait_that_runs_out_is_reported(fs4, shapes):
    """FS4_TEST_STALL on both kernels, with Gram products split along K and thin matrices among the
    others: the call ends, the status word tells, and the next call in the workspace is right."""
    import time
    ws = torch.zeros(fs4.muon_workspace_size(shapes), dtype=torch.uint8, device="cuda")
    G = [make(*s, torch.bfloat16).cuda() for s in shapes]
    W, M, W2, M2 = ([torch.zeros(s, device="cuda") for s in shapes] for _ in range(4))
    t0 = time.time()
    fs4.muon_step([torch.zeros_like(w) for w in W], G, [torch.zeros_like(m) for m in M], lr=0.1, workspace=ws,
                  flags=fs4.FS4_TEST_STALL)
    assert fs4.device_status(ws) == -8
    assert time.time() - t0 < 60.0
    fs4.muon_step(W, G, M, lr=0.1, workspace=ws)
    assert fs4.device_status(ws) == 0
    fs4.muon_step(W2, G, M2, lr=0.1)
    assert all(torch.equal(a, b) for a, b in zip(W + M, W2 + M2))


def takes_pairs(fs4, shapes):
    """Whether a call runs on CTA pairs: a small call's workspace also holds partial tiles of 32 KB, two at
    least, beside the table (27 KB) and the partial sums (under 10 KB a matrix) of all calls."""
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    blocks = sum(6 * up(m) * up(n) + 6 * up(min(m, n)) ** 2 for m, n in shapes if min(m, n) > 32)
    return fs4.muon_workspace_size(shapes) - blocks < (1 << 16) + 9600 * len(shapes)


def exact64(G, K=5, coeffs=O.MUON):
    """oracle.muon.orthogonalize on the GPU."""
    x = G.cuda().double()
    tall = x.shape[0] > x.shape[1]
    x = (x.T if tall else x) / (x.norm() + 1e-7)
    for k in range(K):
        a, b, c = coeffs[k] if hasattr(coeffs[0], "__len__") else coeffs
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return np64(x.T if tall else x)


LARGE = [(1500, 1900), (1900, 1501), (770, 9000), (2100, 2300), (4200, 2305)]      # 3 to 10 blocks of 256 rows


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_pairs_against_float64(fs4, shape, kind):
    assert takes_pairs(fs4, [shape]) and not takes_pairs(fs4, [(300, 1111)])
    G = make(*shape, TYPES[kind]).cuda()
    want = exact64(G)
    ws = torch.empty(fs4.muon_workspace_size([shape]), dtype=torch.uint8, device="cuda")
    for t in TYPES.values():
        wide = torch.full((shape[0], shape[1] + 9), 3.0, dtype=t, device="cuda")
        out = wide[:, 4:-5] if t is TYPES[kind] else torch.empty(shape, dtype=t, device="cuda")
        fs4.muon_orthogonalize([G], outs=[out], workspace=ws)
        assert far(out, want) <= NEAR + half_step(t) and fs4.device_status(ws) == 0
        assert (wide[:, :4] == 3).all() and (wide[:, -5:] == 3).all()


@pytest.mark.parametrize("shape", [(1500, 1900), (2305, 2100)], ids=str)
def test_pairs_products_one_iteration_at_a_time(fs4, shape):
    assert takes_pairs(fs4, [shape])
    G = make(*shape)
    top = float(torch.linalg.matrix_norm(G.cuda().double(), 2) / G.double().norm())
    for coeffs in ((1.0, 0.0, 0.0), (0.0, 1.0, 0.0), (0.0, 0.0, 1.0), (0.5, -2.0, 1.0)):
        got = fs4.muon_orthogonalize([G.cuda()], K=1, coeffs=coeffs, dtype=torch.float32)[0]
        want = exact64(G, 1, coeffs)
        # as in test_products_one_iteration_at_a_time, and an absolute part: the operands hold 2^8 A and
        # 2^8 B in FP16, whose subnormal numbers (here most of A^2) are off by up to 2^-25.  With
        # |dA|, |dB| <= 2^-33 an element, ||dB X|| <= m 2^-33 s for the largest singular value s of X,
        # and a change of A by dA moves A^2 X by at most 2 s^2 m 2^-33 s, b A X by |b| m 2^-33 s
        small = min(shape) * 2.0 ** -33 * top * (1 + abs(coeffs[1]) + 2 * abs(coeffs[2]) * top ** 2) / np.linalg.norm(want)
        assert far(got, want) <= (2.0 ** -20 if coeffs[1:] == (0.0, 0.0) else 5 * 2.0 ** -12 + small), coeffs
    per = [O.MUON, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)]
    assert far(fs4.muon_orthogonalize([G.cuda()], K=3, coeffs=per, dtype=torch.float32)[0], exact64(G, 3, per)) <= NEAR


@pytest.mark.parametrize("nesterov", (False, True))
@pytest.mark.parametrize("types", [("f32", "bf16", "f32"), ("bf16", "f32", "f16")], ids=str)
def test_pairs_step_against_float64(fs4, types, nesterov):
    """Several matrices of three and more blocks, thin and small ones among them: the direction
    itself (from zero weights) and the whole step."""
    tw, tg, tm = (TYPES[t] for t in types)
    shapes = [(800, 1100), (20, 300), (1300, 900), (33, 64), (2100, 2200)]
    assert takes_pairs(fs4, shapes)
    lr, beta, wd = 0.02, 0.9, 0.1
    for start in (0.0, 2.0):
        W, G, M = ([make(*s, t, k).mul(f).cuda() for s in shapes] for t, k, f in ((tw, 1, start), (tg, 2, 1.0), (tm, 3, 0.5)))
        W0, G0, M0 = ([np64(t) for t in ts] for ts in (W, G, M))
        fs4.muon_step(W, G, M, lr=lr, beta=beta, nesterov=nesterov, weight_decay=wd)
        for w, m, w0, g0, m0 in zip(W, M, W0, G0, M0):
            # the bounds of test_step_against_float64
            new, size = beta * m0 + (1 - beta) * g0, beta * np.abs(m0) + (1 - beta) * np.abs(g0)
            tiny = float(torch.finfo(tm).smallest_normal) * float(torch.finfo(tm).eps)
            assert (np.abs(np64(m) - new) <= 4 * 2.0 ** -24 * size + half_step(tm) * (np.abs(new) + 4 * 2.0 ** -24 * size) + tiny).all()
            kept = np64(m)
            step = lr * 0.2 * max(w0.shape) ** 0.5 * exact64(torch.from_numpy(beta * kept + (1 - beta) * g0 if nesterov else kept))
            want = (1 - lr * wd) * w0 - step
            assert np.linalg.norm(np64(w) - want) <= (NEAR + 2.0 ** -22) * np.linalg.norm(step) + (half_step(tw) + 2.0 ** -22) * np.linalg.norm(want)


def test_batch_of_all_shapes_stays_within_the_bound(fs4):
    """The call as a whole chooses kernel and splits, so bits may differ from each matrix alone;
    the bound does not, and the same call repeats bit for bit."""
    types = [TYPES[k] for _, k in zip(SHAPES, itertools.cycle(TYPES))]
    Gs = [make(*s, t).cuda() for s, t in zip(SHAPES, types)]
    assert takes_pairs(fs4, SHAPES) and not any(takes_pairs(fs4, [s]) for s in SHAPES if min(s) > 32)
    batch, again = fs4.muon_orthogonalize(Gs), fs4.muon_orthogonalize(Gs)
    for G, b, a in zip(Gs, batch, again):
        alone = fs4.muon_orthogonalize([G])[0]
        want = O.orthogonalize(np64(G))
        assert torch.equal(b, a) and far(b, want) <= NEAR + half_step(torch.bfloat16) and far(alone, want) <= NEAR + half_step(torch.bfloat16)


@pytest.mark.parametrize("shape", [(60, 90), (20, 90), (1500, 1900)], ids=str)
def test_updates_far_below_the_norms_floor(fs4, shape):
    """||U|| of 1e-11 and less beside 1e-7: the iteration is a^5 = 485 times X_0, whose elements are kept
    to 2^-37, and those of later iterates too: 485 (1 + 1/a + ...) < 700 such errors an element."""
    for scale in (1e-12, 1e-14, 1e-17, 1e-25):
        G = make(*shape) * scale
        want = exact64(G)
        got = np64(fs4.muon_orthogonalize([G.cuda()], dtype=torch.float32)[0])
        assert np.linalg.norm(got - want) <= NEAR * np.linalg.norm(want) + 700 * 2.0 ** -37 * want.size ** 0.5


def test_two_graphs_take_turns_in_one_workspace(fs4):
    """Captured steps on different shapes, replayed in turn on one stream."""
    sets = [[(100, 300), (20, 50)], [(1500, 1400)]]
    ws = torch.zeros(max(fs4.muon_workspace_size(s) for s in sets), dtype=torch.uint8, device="cuda")
    G = [[make(*s, torch.bfloat16).cuda() for s in shapes] for shapes in sets]
    W, M, W2, M2 = ([[torch.zeros(s, device="cuda") for s in shapes] for shapes in sets] for _ in range(4))
    graphs = []
    for w, g, m in zip(W, G, M):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fs4.muon_step(w, g, m, lr=0.1, workspace=ws)
    for _ in range(3):
        for graph, w, g, m in zip(graphs, W2, G, M2):
            graph.replay()
            fs4.muon_step(w, g, m, lr=0.1)
    torch.cuda.synchronize()
    for a, b in zip(W + M, W2 + M2):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("width", (24, 60, 1100))
def test_slices_past_32_bit_offsets(fs4, width):
    """Weights, gradient and momentum as slices of one buffer of 2.7e9 elements."""
    rows, total = 65_500, 41_000
    buffer = torch.zeros(rows, total, dtype=torch.bfloat16, device="cuda")
    cut = [buffer[:, c:c + width] for c in (8, 16_001, total - width - 3)]
    for t, k, f in zip(cut, (1, 2, 3), (2.0, 1.0, 0.5)):
        t.copy_(make(rows, width, torch.bfloat16, k).mul(f))
    alone = [t.clone() for t in cut]
    last = [t[-1].clone() for t in cut]
    fs4.muon_step(*[[t] for t in cut], lr=0.1, weight_decay=0.1)
    fs4.muon_step(*[[t] for t in alone], lr=0.1, weight_decay=0.1)
    assert torch.equal(cut[2], alone[2]) and torch.equal(cut[1][-1], last[1])
    # the bound of test_slices_of_one_buffer_step_as_matrices_of_their_own, and a step of BF16 at ties
    assert far(cut[0], np64(alone[0])) <= 2.0 ** -9 and not torch.equal(cut[0][-1], last[0])
    assert (cut[0][-300:].float() - alone[0][-300:].float()).abs().max() <= 2.0 ** -7 * alone[0].float().abs().max()
    for t in cut:
        t.zero_()
    assert not buffer.any()
