"""MXFP4 on the GPU against the 64-bit oracle: quantisation byte for byte, products within a
derived bound.

Bound of a product: a code times a code and its power of two are exact, so the only error before
the one rounding of the output is FP32 accumulation of K terms, at most K 2^-23 sum |a b|."""
import numpy as np
import pytest
import torch

from oracle import mxfp4 as O

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in TYPES.values()}
SHAPES = [(1, 1), (1, 33), (3, 64), (31, 31), (33, 257), (128, 256), (129, 130), (200, 515), (257, 96)]


def make(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(1000 * rows + cols + seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float())
    return x.to(dtype)


def np64(t):
    return t.detach().cpu().double().numpy()


def same(view, want, tiled):
    codes, scales = (O.pack_tiled if tiled else O.pack_plain)(*want)
    np.testing.assert_array_equal(view[1].cpu().numpy(), scales)
    np.testing.assert_array_equal(view[0].cpu().numpy(), codes)


@pytest.mark.parametrize("tiled", (False, True), ids=("plain", "tiled"))
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_matches_the_oracle(fs4, shape, kind, tiled):
    x = make(*shape, TYPES[kind])
    for rule in ("floor", "ceil"):
        for seed in (None, 77):
            row = O.quantize(np64(x), rule, seed)
            col = O.quantize(np64(x).T, rule, None if seed is None else seed ^ O.COLUMN_SEED)
            kw = dict(tiled=tiled, scale_rule=rule, seed=seed)
            both = fs4.mxfp4_quantize_both(x.cuda(), **kw)
            same(both[0], row, tiled)
            same(both[1], col, tiled)
            same(fs4.mxfp4_quantize(x.cuda(), **kw), row, tiled)
            same(fs4.mxfp4_quantize(x.cuda(), axis=fs4.FS4_AXIS_COL, **kw), col, tiled)


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_extremes(fs4, kind):
    """Zeros of either sign, subnormals, the largest values, ties, and blocks with NaN or Inf."""
    t = TYPES[kind]
    f = torch.finfo(t)
    x = torch.zeros(6, 96, dtype=t)
    x[0, 5] = -0.0
    x[1, :6] = torch.tensor([f.max, -f.max, f.tiny, f.smallest_normal, f.max / 4, -f.max / 16]).to(t)
    x[2, 32:40] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]).to(t)
    x[3, 64:67] = torch.tensor([f.tiny / 4, -f.tiny / 2, f.tiny / 8]).to(t)
    x[4, 3], x[4, 40], x[5, 95] = float("nan"), float("inf"), float("-inf")
    for seed, rule in ((None, "floor"), (3, "floor"), (None, "ceil"), (3, "ceil")):
        row, col = fs4.mxfp4_quantize_both(x.cuda(), seed=seed, scale_rule=rule)
        same(row, O.quantize(np64(x), rule, seed), False)
        same(col, O.quantize(np64(x).T, rule, None if seed is None else seed ^ O.COLUMN_SEED), False)
        y = fs4.mxfp4_dequantize(*row, 6, 96, dtype=t).cpu()
        want = O.values(*O.quantize(np64(x), rule, seed))
        with np.errstate(over="ignore"):
            assert torch.equal(torch.nan_to_num(y, nan=1.5), torch.nan_to_num(torch.from_numpy(want).to(t), nan=1.5))
            assert (torch.isnan(y).numpy() == np.isnan(want)).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dequantize_reads_back_every_layout(fs4, shape, kind):
    x = make(*shape, torch.float32)
    want = torch.from_numpy(O.values(*O.quantize(np64(x)))).to(TYPES[kind])
    for tiled in (False, True):
        view = fs4.mxfp4_quantize(x.cuda(), tiled=tiled)
        assert torch.equal(fs4.mxfp4_dequantize(*view, *shape, tiled=tiled, dtype=TYPES[kind]).cpu(), want)
        wide = torch.full((shape[0], shape[1] + 3), 7.0, dtype=TYPES[kind], device="cuda")
        fs4.mxfp4_dequantize(*view, *shape, tiled=tiled, out=wide[:, 1:-2])
        assert torch.equal(wide[:, 1:-2].cpu(), want) and (wide[:, 0] == 7).all() and (wide[:, -2:] == 7).all()


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_strided_and_unaligned_input(fs4, kind):
    big = make(70, 300, TYPES[kind]).cuda()
    for x in (big[3:60, 1:258], big[::2, 8:200], big[:, 5:6], big[4:5]):
        plain = x.cpu().contiguous()
        row, col = fs4.mxfp4_quantize_both(x)
        same(row, O.quantize(np64(plain)), False)
        same(col, O.quantize(np64(plain).T), False)


def test_quantize_past_32_bit_offsets(fs4):
    """2.2e9 elements: the last rows come out as they do on their own."""
    rows, cols = 67_000, 33_000
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(cols, device="cuda").remainder(97) - 48.0)
    x[-256:] = torch.randn(256, cols, device="cuda").bfloat16()
    codes, scales = fs4.mxfp4_quantize(x)
    part = fs4.mxfp4_quantize(x[-200:].contiguous())
    assert torch.equal(codes[-200:], part[0]) and torch.equal(scales[-200:], part[1])
    y = fs4.mxfp4_dequantize(codes, scales, rows, cols, dtype=torch.bfloat16)
    assert torch.equal(y[-200:], fs4.mxfp4_dequantize(*part, 200, cols, dtype=torch.bfloat16))


def operand(fs4, rows, k, seed):
    x = make(rows, k, torch.float32, seed).clamp(-300, 300)
    return fs4.mxfp4_quantize(x.cuda(), tiled=True), O.values(*O.quantize(np64(x)))


PRODUCTS = [(1, 1, 1), (1, 16, 32), (1, 300, 700), (7, 129, 257), (16, 128, 2048), (17, 520, 300), (33, 65, 64), (64, 1000, 1536),
            (65, 40, 515), (128, 128, 256), (130, 257, 1000), (300, 16, 2100), (513, 300, 130), (256, 512, 4096), (700, 1100, 96),
            (1790, 1300, 300), (513, 3600, 520), (4100, 1030, 130), (2048, 1280, 2048)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("size", PRODUCTS, ids=str)
def test_gemm_against_float64(fs4, size, kind):
    M, N, K = size
    t = TYPES[kind]
    (a, av), (b, bv) = operand(fs4, M, K, 1), operand(fs4, N, K, 2)
    scale = 2.0 ** -8          # keeps the FP16 products finite; exact
    av = av * scale
    a = (a[0], torch.where(a[1] == 0, a[1], a[1] - 8))
    want = av @ bv.T
    bound = K * 2.0 ** -23 * (np.abs(av) @ np.abs(bv).T)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = np64(fs4.mxfp4_gemm(a, b, M, N, K, dtype=t, workspace=ws))
    tiny = float(torch.finfo(t).smallest_normal) * float(torch.finfo(t).eps)
    assert (np.abs(got - want) <= bound + HALF_STEP[t] * (np.abs(want) + bound) + tiny).all()
    # added to D in place, in a strided D whose other columns stay as they are
    wide = torch.randn(M, N + 5, device="cuda").to(t)
    before = wide.clone()
    fs4.mxfp4_gemm(a, b, M, N, K, out=wide[:, 2:-3], accumulate=True, workspace=ws)
    total = want + np64(before[:, 2:-3])
    assert (np.abs(np64(wide[:, 2:-3]) - total) <= bound + 2.0 ** -24 * np.abs(total) + HALF_STEP[t] * (np.abs(total) + bound) + tiny).all()
    assert torch.equal(wide[:, :2], before[:, :2]) and torch.equal(wide[:, -3:], before[:, -3:])
    assert fs4.device_status(ws) == 0


@pytest.mark.parametrize("size", [(1, 200, 512), (17, 130, 300), (140, 150, 300), (1300, 1500, 256), (1300, 1501, 256)], ids=str)
def test_rows_and_columns_past_the_product_stay_as_they_are(fs4, size):
    M, N, K = size
    (a, _), (b, _) = operand(fs4, M, K, 1), operand(fs4, N, K, 2)
    want = fs4.mxfp4_gemm(a, b, M, N, K)
    big = torch.full((M + 3, N), 5.0, dtype=torch.bfloat16, device="cuda")
    fs4.mxfp4_gemm(a, b, M, N, K, out=big[1:M + 1])
    assert torch.equal(big[1:M + 1], want) and (big[0] == 5).all() and (big[M + 1:] == 5).all()


@pytest.mark.parametrize("size", [(1, 256, 512), (40, 130, 300), (300, 140, 300), (1500, 1400, 300)], ids=str)
def test_gemm_nan_blocks_reach_their_rows_and_no_others(fs4, size):
    M, N, K = size
    x = make(M, K, torch.float32)
    w = make(N, K, torch.float32, 1)
    x[M // 2, 7] = float("inf")
    w[N // 3, K - 1] = float("nan")
    y = fs4.mxfp4_gemm(fs4.mxfp4_quantize(x.cuda(), tiled=True), fs4.mxfp4_quantize(w.cuda(), tiled=True), M, N, K, dtype=torch.float32)
    want = torch.zeros(M, N, dtype=torch.bool)
    want[M // 2], want[:, N // 3] = True, True
    assert torch.equal(torch.isnan(y).cpu(), want)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("size", [(1, 200, 513), (9, 64, 4096), (16, 300, 33), (33, 48, 700), (140, 260, 384)], ids=str)
def test_linear_is_quantise_then_product(fs4, size, kind):
    M, N, K = size
    x = make(M, K + 3, TYPES[kind]).cuda()[:, 1:-2]
    w = fs4.mxfp4_quantize(make(N, K, torch.float32, 3).cuda() / 64, tiled=True)
    for rule in ("floor", "ceil"):
        want = fs4.mxfp4_gemm(fs4.mxfp4_quantize(x, tiled=True, scale_rule=rule), w, M, N, K, dtype=TYPES[kind])
        assert torch.equal(fs4.mxfp4_linear(x, w, N, scale_rule=rule), want)
    ws = torch.zeros(fs4.mxfp4_linear_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    d = torch.ones(M, N, device="cuda")
    fs4.mxfp4_linear(x, w, N, out=d, accumulate=True, workspace=ws)
    f32 = fs4.mxfp4_linear(x, w, N, dtype=torch.float32, workspace=ws)
    assert torch.equal(d, f32 + 1.0) and fs4.device_status(ws) == 0
    x[M - 1, 0] = float("nan")
    y = fs4.mxfp4_linear(x, w, N)
    assert torch.isnan(y[M - 1]).all() and not torch.isnan(y[:M - 1]).any()


def test_calls_repeat_bit_for_bit_on_streams_and_in_graphs(fs4):
    x = make(20, 2048, torch.bfloat16).cuda()
    w = fs4.mxfp4_quantize(make(400, 2048, torch.float32, 4).cuda(), tiled=True)
    want = fs4.mxfp4_linear(x, w, 400)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [fs4.mxfp4_linear(x, w, 400, stream=s) for s in (side, None, side, None)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    ws = torch.zeros(fs4.mxfp4_linear_workspace_size(20, 2048), dtype=torch.uint8, device="cuda")
    out = torch.zeros(20, 400, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs4.mxfp4_linear(x, w, 400, out=out, workspace=ws)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, fs4.mxfp4_linear(x, w, 400))


def test_products_at_once_share_a_status_word(fs4):
    """Large and small products on two streams with one workspace, which only holds the status."""
    (a, _), (b, _) = operand(fs4, 1300, 512, 1), operand(fs4, 1500, 512, 2)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = [fs4.mxfp4_gemm(a, b, M, 1500, 512) for M in (1300, 3, 100)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [(i, fs4.mxfp4_gemm(a, b, M, 1500, 512, workspace=ws, stream=s)) for _ in range(5) for s in (side, None)
            for i, M in enumerate((1300, 3, 100))]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in outs) and fs4.device_status(ws) == 0


def test_linear_follows_its_operands_producers_without_a_sync(fs4):
    """Each call's x is written by the launch before it, in one workspace for all."""
    w = fs4.mxfp4_quantize(make(600, 1024, torch.float32, 4).cuda(), tiled=True)
    for M in (1, 5, 40, 1500):
        base = make(M, 1024, torch.bfloat16).cuda()
        want = [fs4.mxfp4_linear((base * k), w, 600) for k in range(8)]
        torch.cuda.synchronize()
        ws = torch.zeros(fs4.mxfp4_linear_workspace_size(M, 1024), dtype=torch.uint8, device="cuda")
        x, outs = torch.empty_like(base), []
        for k in range(8):
            torch.mul(base, k, out=x)
            outs.append(fs4.mxfp4_linear(x, w, 600, workspace=ws))
        torch.cuda.synchronize()
        assert all(torch.equal(o, t) for o, t in zip(outs, want))


def test_three_products_of_a_linear_layer(fs4):
    """y = x W^T, dx = dy W, dW += dy^T x on quantised operands, against the oracle's operands."""
    T, n_in, n_out = 200, 300, 170
    x, w, dy = make(T, n_in, torch.bfloat16).cuda(), make(n_out, n_in, torch.float32, 1).cuda(), make(T, n_out, torch.bfloat16, 2).cuda()
    xr, xc = fs4.mxfp4_quantize_both(x, tiled=True)
    wr, wc = fs4.mxfp4_quantize_both(w, tiled=True)
    gr, gc = fs4.mxfp4_quantize_both(dy, tiled=True, seed=9)
    val = lambda t, seed=None: O.values(*O.quantize(t, "floor", seed))  # noqa: E731
    X, W, G = np64(x), np64(w), np64(dy)
    dw = torch.ones(n_out, n_in, device="cuda")
    for got, left, right, k, plus in (
            (fs4.mxfp4_gemm(xr, wr, T, n_out, n_in, dtype=torch.float32), val(X), val(W), n_in, 0.0),
            (fs4.mxfp4_gemm(gr, wc, T, n_in, n_out, dtype=torch.float32), val(G, 9), val(W.T), n_out, 0.0),
            (fs4.mxfp4_gemm(gc, xc, n_out, n_in, T, out=dw, accumulate=True), val(G.T, 9 ^ O.COLUMN_SEED), val(X.T), T, 1.0)):
        want = left @ right.T + plus
        bound = (k + 2) * 2.0 ** -23 * (np.abs(left) @ np.abs(right).T + plus)
        assert (np.abs(np64(got) - want) <= bound).all()


def test_refusals_on_device(fs4):
    x = torch.zeros(8, 64, device="cuda")
    view = fs4.mxfp4_quantize(x, tiled=True)
    with pytest.raises(ValueError):
        fs4.mxfp4_quantize(x.t())
    with pytest.raises(ValueError):
        fs4.mxfp4_quantize(x.double())
    with pytest.raises(ValueError):
        fs4.mxfp4_quantize(x[0])
    with pytest.raises(ValueError):
        fs4.mxfp4_gemm(view, view, 129, 8, 64)                   # more rows than the operand has
    with pytest.raises(ValueError):
        fs4.mxfp4_gemm(view, view, 8, 8, 64, accumulate=True)
    with pytest.raises(ValueError):
        fs4.mxfp4_gemm(view, view, 8, 8, 64, out=torch.zeros(8, 9, device="cuda"))
    with pytest.raises(ValueError):
        fs4.mxfp4_dequantize(view[0][:10], view[1], 8, 64, tiled=True)
    with pytest.raises(ValueError):
        fs4.mxfp4_linear(x, view, 8, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fs4.Fs4Error):
        fs4.mxfp4_dequantize(view[0][:8192].view(-1), view[0][8192:], 8, 64, out=view[0].view(torch.float32)[:512].view(8, 64))


@pytest.mark.parametrize("M", (3, 40, 600))
def test_linear_between_slices_of_one_buffer(fs4, M):
    """x and D side by side in one buffer."""
    N, K = 520, 640
    w = fs4.mxfp4_quantize(make(N, K, torch.float32, 3).cuda() / 64, tiled=True)
    x = make(M, K, torch.bfloat16).cuda()
    want = fs4.mxfp4_linear(x, w, N)
    buffer = torch.full((M, 4 + K + N + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    buffer[:, 4:4 + K] = x
    fs4.mxfp4_linear(buffer[:, 4:4 + K], w, N, out=buffer[:, 4 + K:4 + K + N])
    assert torch.equal(buffer[:, 4 + K:4 + K + N], want) and torch.equal(buffer[:, 4:4 + K], x)
    assert (buffer[:, :4] == 5).all() and (buffer[:, -3:] == 5).all()
    with pytest.raises(fs4.Fs4Error):
        fs4.mxfp4_linear(buffer[:, 4:4 + K], w, N, out=buffer[:, 3 + K:3 + K + N])


@pytest.mark.parametrize("tiled", (False, True), ids=("plain", "tiled"))
def test_no_rows_give_empty_views(fs4, tiled):
    for rows, cols in ((0, 96), (5, 0), (0, 0)):
        x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
        for seed in (None, 3):
            row, col = fs4.mxfp4_quantize_both(x, tiled=tiled, seed=seed)
            for view, (r, c) in ((row, (rows, cols)), (col, (cols, rows)), (fs4.mxfp4_quantize(x, tiled=tiled), (rows, cols)),
                                 (fs4.mxfp4_quantize(x, axis=fs4.FS4_AXIS_COL, tiled=tiled), (cols, rows))):
                assert all(t.numel() == 0 and t.dtype is torch.uint8 and t.is_cuda for t in view)
                y = fs4.mxfp4_dequantize(*view, r, c, tiled=tiled, dtype=torch.float16)
                assert y.shape == (r, c) and y.dtype is torch.float16
    with pytest.raises(ValueError):
        fs4.mxfp4_quantize(torch.zeros(0, 4, device="cuda"), scale_rule="nearest")


def test_an_expert_without_tokens_trains_like_the_others(fs4):
    """y, dx and dW of a linear layer for token counts with a zero among them."""
    n_in, n_out = 96, 160
    wr, wc = fs4.mxfp4_quantize_both(make(n_out, n_in, torch.float32).cuda(), tiled=True)
    for tokens in (0, 3):
        x, dy = make(tokens, n_in, torch.bfloat16, 1).cuda(), make(tokens, n_out, torch.bfloat16, 2).cuda()
        _, xc = fs4.mxfp4_quantize_both(x, tiled=True)
        gr, gc = fs4.mxfp4_quantize_both(dy, tiled=True)
        assert fs4.mxfp4_linear(x, wr, n_out).shape == (tokens, n_out)
        assert fs4.mxfp4_linear(x, wr, n_out, dtype=torch.float32).dtype is torch.float32
        assert fs4.mxfp4_gemm(gr, wc, tokens, n_in, n_out).shape == (tokens, n_in)
        dw = torch.full((n_out, n_in), 2.0, device="cuda")
        fs4.mxfp4_gemm(gc, xc, n_out, n_in, tokens, out=dw, accumulate=True)
        assert (dw == 2).all() == (tokens == 0)
        fs4.mxfp4_gemm(gc, xc, n_out, n_in, tokens, out=dw)
        assert dw.any() == (tokens > 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    empty = torch.zeros(0, dtype=torch.uint8, device="cuda")
    y = fs4.mxfp4_gemm((empty, empty), (empty, empty), 7, 9, 0, stream=side)
    side.synchronize()
    assert y.shape == (7, 9) and not y.any()
    with pytest.raises(ValueError):
        fs4.mxfp4_gemm((empty, empty), (empty, empty), 7, 9, 1)


def test_linears_at_once_with_workspaces_of_their_own(fs4):
    """Any row count may keep Q(x) in its workspace: calls on two streams, none waiting for the other."""
    N, K = 700, 4096
    w = fs4.mxfp4_quantize(make(N, K, torch.float32, 3).cuda() / 64, tiled=True)
    rows = (1, 3, 16, 17, 32, 33, 200)
    xs = [make(M, K, torch.bfloat16, s).cuda() for s in (0, 1) for M in rows]
    want = [fs4.mxfp4_linear(x, w, N) for x in xs]
    spaces = [torch.zeros(fs4.mxfp4_linear_workspace_size(max(rows), K), dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for i in range(len(rows)):
            for s in range(2):
                k = s * len(rows) + i
                outs.append((k, fs4.mxfp4_linear(xs[k], w, N, workspace=spaces[s], stream=streams[s])))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[k]) for k, o in outs)
    assert all(fs4.device_status(ws) == 0 for ws in spaces)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("size", [(141, 1000, 700), (500, 130, 2100), (1500, 1400, 300), (1025, 1501, 2304), (2300, 2048, 96)], ids=str)
def test_linear_of_many_rows_against_float64(fs4, size, kind):
    """The tile and the pair kernel behind the launch that quantises their operand."""
    M, N, K = size
    t = TYPES[kind]
    x = (make(M, K + 2, t) / 64).cuda()[:, 1:-1]
    wv = make(N, K, torch.float32, 3) / 64
    w = fs4.mxfp4_quantize(wv.cuda(), tiled=True)
    ws = torch.zeros(fs4.mxfp4_linear_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    got = fs4.mxfp4_linear(x, w, N, workspace=ws)
    assert torch.equal(got, fs4.mxfp4_gemm(fs4.mxfp4_quantize(x, tiled=True), w, M, N, K, dtype=t))
    a, b = O.values(*O.quantize(np64(x))), O.values(*O.quantize(np64(wv)))
    want, bound = a @ b.T, K * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
    tiny = float(torch.finfo(t).smallest_normal) * float(torch.finfo(t).eps)
    assert (np.abs(np64(got) - want) <= bound + HALF_STEP[t] * (np.abs(want) + bound) + tiny).all()
    d = torch.full((M, N), 1.0, device="cuda")
    fs4.mxfp4_linear(x, w, N, out=d, accumulate=True, workspace=ws)
    assert (np.abs(np64(d) - want - 1) <= bound + 2.0 ** -23 * (np.abs(want) + bound + 1)).all()
    assert fs4.device_status(ws) == 0


@pytest.mark.parametrize("size", [(40, 130, 300), (64, 256, 4096), (140, 150, 300), (1300, 1500, 512)], ids=str)
def test_gemm_wait_that_runs_out_is_reported(fs4, size):
    """FS4_TEST_STALL: the MMA issuers wait on a barrier nothing arrives on, give up and the call
    ends; the next one is right."""
    import time
    M, N, K = size
    (a, _), (b, _) = operand(fs4, M, K, 1), operand(fs4, N, K, 2)
    want = fs4.mxfp4_gemm(a, b, M, N, K)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    fs4.device_status()
    t0 = time.time()
    for space in (ws, None):
        fs4.mxfp4_gemm(a, b, M, N, K, workspace=space, flags=fs4.FS4_TEST_STALL)
        assert fs4.device_status(space) == -8
    assert time.time() - t0 < 60.0
    ws.zero_()
    assert torch.equal(fs4.mxfp4_gemm(a, b, M, N, K, workspace=ws), want)
    assert torch.equal(fs4.mxfp4_gemm(a, b, M, N, K), want)
    assert fs4.device_status(ws) == 0 and fs4.device_status() == 0


@pytest.mark.parametrize("size", [(1, 200, 512), (40, 200, 512), (1500, 1300, 300)], ids=str)
def test_linear_wait_that_runs_out_is_reported(fs4, size):
    M, N, K = size
    x = make(M, K, torch.bfloat16).cuda()
    w = fs4.mxfp4_quantize(make(N, K, torch.float32, 3).cuda() / 64, tiled=True)
    want = fs4.mxfp4_linear(x, w, N)
    ws = torch.zeros(fs4.mxfp4_linear_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    fs4.device_status()
    for space in (ws, None):
        fs4.mxfp4_linear(x, w, N, workspace=space, flags=fs4.FS4_TEST_STALL)
        assert fs4.device_status(space) == -8
    ws.zero_()
    assert torch.equal(fs4.mxfp4_linear(x, w, N, workspace=ws), want) and torch.equal(fs4.mxfp4_linear(x, w, N), want)
    assert fs4.device_status(ws) == 0 and fs4.device_status() == 0


def test_elements_next_to_the_largest_fp32_value(fs4):
    """The ceil rule's scale is 2^126 there: 1.75 2^127 is the tie between the codes 3 and 4, and 4 is 2^128."""
    x = torch.zeros(1, 32, device="cuda")
    for top, floor, ceil in ((1.5, 1.5, 1.5), (1.74, 1.5, 1.5), (1.75, 1.5, float("inf")), (1.99, 1.5, float("inf"))):
        x[0, 0] = top * 2.0 ** 127
        for rule, want in (("floor", floor), ("ceil", ceil)):
            view = fs4.mxfp4_quantize(x, scale_rule=rule)
            same(view, O.quantize(np64(x), rule), False)
            y = fs4.mxfp4_dequantize(*view, 1, 32)
            assert y[0, 0].item() == want * 2.0 ** 127 and not y[0, 1:].any(), (top, rule)


def test_strided_operands_past_32_bit_offsets(fs4):
    """x, D and the values read back as slices of one buffer of 2.7e9 elements."""
    rows, total, N, K = 66_000, 41_000, 130, 260
    buffer = torch.zeros(rows, total, dtype=torch.bfloat16, device="cuda")
    x, d, y = buffer[:, 5:5 + K], buffer[:, 20_000:20_000 + N], buffer[:, total - K:]
    x.copy_(make(rows, K, torch.bfloat16))
    w = fs4.mxfp4_quantize(make(N, K, torch.float32, 3).cuda() / 64, tiled=True)
    alone = x.clone()
    want = fs4.mxfp4_linear(alone, w, N)
    fs4.mxfp4_linear(x, w, N, out=d)
    assert torch.equal(d, want)
    a = fs4.mxfp4_quantize(x, tiled=True)
    fs4.mxfp4_gemm(a, w, rows, N, K, out=d, accumulate=True)
    assert torch.equal(d[-300:], fs4.mxfp4_gemm(a, w, rows, N, K, out=want, accumulate=True)[-300:]) and torch.equal(d, want)
    for layout in (False, True):
        view = fs4.mxfp4_quantize(x, tiled=layout)
        fs4.mxfp4_dequantize(*view, rows, K, tiled=layout, out=y)
        assert torch.equal(y, fs4.mxfp4_dequantize(*fs4.mxfp4_quantize(alone, tiled=layout), rows, K, tiled=layout, dtype=torch.bfloat16))
    assert torch.equal(x, alone)
    for t in (x, d, y):
        t.zero_()
    assert not buffer.any()


@pytest.mark.parametrize("size", [(1 << 20, 16, 33), (1, 1 << 20, 33), (33, 16, 1 << 20), (300, 300, 1 << 20), (1 << 20, 300, 64),
                                  (140, 1 << 20, 96), (1, 16, 1 << 20)], ids=str)
def test_largest_rows_columns_and_terms(fs4, size):
    M, N, K = size
    g = torch.Generator("cuda").manual_seed(M + N + K)
    x, w = (torch.randn(r, K, generator=g, device="cuda", dtype=torch.float32) for r in (M, N))
    a, b = fs4.mxfp4_quantize(x, tiled=True), fs4.mxfp4_quantize(w, tiled=True)
    av, bv = (fs4.mxfp4_dequantize(*q, r, K, tiled=True).double() for q, r in ((a, M), (b, N)))
    want, bound = av @ bv.T, K * 2.0 ** -23 * (av.abs() @ bv.abs().T)
    ws = torch.zeros(fs4.mxfp4_linear_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    got = fs4.mxfp4_gemm(a, b, M, N, K, dtype=torch.float32, workspace=ws)
    assert ((got.double() - want).abs() <= bound).all()
    assert torch.equal(fs4.mxfp4_linear(x, b, N, workspace=ws), got) and fs4.device_status(ws) == 0


def test_one_row_and_one_column_of_2_to_31_elements(fs4):
    n = 1 << 31
    x = torch.empty(1, n, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(1 << 16, device="cuda", dtype=torch.int32).remainder(97).sub(48).repeat(n >> 16)[None])
    tail = slice(n - 4096, n)
    codes, scales = fs4.mxfp4_quantize(x)
    part = fs4.mxfp4_quantize(x[:, tail].contiguous())
    assert torch.equal(codes[0, -2048:], part[0][0]) and torch.equal(scales[0, -128:], part[1][0])
    y = fs4.mxfp4_dequantize(codes, scales, 1, n, dtype=torch.bfloat16)
    assert torch.equal(y[:, tail], fs4.mxfp4_dequantize(*part, 1, 4096, dtype=torch.bfloat16))
    del codes, scales, y
    # as a column its row view has one element a row, and its column view is the row view above
    z = x.view(n, 1)
    codes, scales = fs4.mxfp4_quantize(z)
    few = fs4.mxfp4_quantize(z[tail].contiguous())
    assert torch.equal(codes[tail], few[0]) and torch.equal(scales[tail], few[1])
    y = fs4.mxfp4_dequantize(codes, scales, n, 1, dtype=torch.bfloat16)
    assert torch.equal(y[tail], fs4.mxfp4_dequantize(*few, 4096, 1, dtype=torch.bfloat16))
    del codes, scales, y
    codes, scales = fs4.mxfp4_quantize(z, axis=fs4.FS4_AXIS_COL)
    assert torch.equal(codes[0, -2048:], part[0][0]) and torch.equal(scales[0, -128:], part[1][0])


def test_calls_from_several_host_threads(fs4):
    """Each thread on a stream of its own, products of all kernels and Muon steps among them."""
    import threading
    ops = {k: operand(fs4, 1400, 700, k)[0] for k in (1, 2)}
    x = make(1400, 700, torch.bfloat16).cuda()
    G = [make(300, 411, torch.bfloat16, 5).cuda(), make(1300, 1500, torch.bfloat16, 6).cuda(), make(20, 700, torch.bfloat16, 7).cuda()]

    def work(i, stream=None):
        rows = (1, 9, 100, 1400)[i % 4]
        return [fs4.mxfp4_linear(x[:rows], ops[1], 1400, stream=stream), fs4.mxfp4_gemm(ops[1], ops[2], 1400, 1400 - 400 * (i % 3), 700, stream=stream),
                fs4.muon_orthogonalize(G[i % 3:i % 3 + 1], stream=stream)[0], fs4.mxfp4_quantize(x[:rows], seed=i, stream=stream)[0]]

    want = [work(i) for i in range(12)]
    torch.cuda.synchronize()
    got, errors = {}, []

    def thread(t):
        try:
            stream = torch.cuda.Stream()
            for i in range(12):
                got[t, i] = work(i, stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(t,)) for t in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and len(got) == 72
    assert all(torch.equal(a, b) for (_, i), outs in got.items() for a, b in zip(outs, want[i]))
    assert fs4.device_status() == 0
