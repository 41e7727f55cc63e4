"""Layer norm and dropout on the GPU against plain 64-bit forms.

Tolerances.  u = 2^-24 is fp32's half step.  A row sum adds at most 64 terms in a thread
and joins threads in at most 15 steps, so its error is below 80 u times the sum of the
magnitudes; a mean is off by at most 80 u max|h|.  (h - mean) rstd w + b then is off by
at most 80 u rstd max|h| |w| for the mean, the same relative size for rstd (half of the
variance's 160 u) and a few u for the operations: 256 u (rstd max|h| + |z|) |w| + 4 u |b|
covers them.  Every output adds half a step of its own type.
"""
import threading

import numpy as np
import pytest
import torch

import block_oracle as B
import sparse_attention_video_tile_b200 as sta

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_video_tile_b200.build import build
    build()
    sta.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def _np(t):
    return t.double().cpu().numpy()


def _rand(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def _subnormal(dtype):
    # below the smallest normal number a rounding is off by half of the smallest subnormal
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def _close(got, want, tol, what):
    got, want = np.asarray(got), np.asarray(want)
    assert np.all(np.isfinite(got)), f"{what}: non-finite"
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) / tol):.3g} of the bound"


SHAPES = [(1, 1), (3, 1), (1, 7), (5, 8), (33, 9), (2, 31), (129, 64), (40, 100), (7, 128), (300, 128), (64, 129),
          (6, 255), (5, 256), (9, 511), (3, 512), (4, 837), (2, 1024), (3, 1153), (17, 1536), (2, 1999), (3, 2048),
          (2, 4100), (2, 8192), (1, 8191), (3, 6000)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dtype):
    dt = TYPES[dtype]
    # the whole product of options on a rotation over the shapes
    i = SHAPES.index((rows, cols)) + list(TYPES).index(dtype)
    wdt = torch.float32 if i % 2 else dt
    residual, p, bias = i % 3 != 0, (0.0, 0.3)[(i // 2) % 2], i % 4 != 1
    x = _rand((rows, cols), dt, 1, 1.5, 3.0)
    w, b = _rand((cols,), wdt, 2, 0.3, 1.0), (_rand((cols,), wdt, 3) if bias else None)
    r = _rand((rows, cols), dt, 4) if residual else None
    seed, off = 0x123456789ABCDEF + i, 0xFEDCBA987 + i
    rng = torch.tensor([seed, off], device="cuda")
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, h, mean, rstd = sta.sta_layer_norm_forward(cu(x), cu(w), cu(b), 1e-5, residual=cu(r), dropout_p=p, rng=rng)
    hx = _np(x)
    hb = np.zeros_like(hx)
    if p > 0:
        hx = hx * B.dropout_factor(rows, cols, p, seed, off)
        hb = hb + 2 * U * np.abs(hx)        # the factor and the product in fp32
    if residual:
        hx = hx + _np(r)
        hb = hb + U * np.abs(hx)
    wn, bn = _np(w), (_np(b) if bias else 0.0)
    want, m, s = B.layer_norm(hx, wn, bn, 1e-5)
    big = np.abs(hx).max(1)
    _close(_np(mean), m, 100 * U * big + 1e-30, "mean")
    # the variance is off by 80 u of itself and by the square of the mean's error
    relv = 256 * U + (100 * U * big * s) ** 2 + 4 * U * big * s
    _close(_np(rstd), s, relv * s, "rstd")
    z = np.abs(hx - m[:, None]) * s[:, None]
    tol = (256 * U * (s * big)[:, None] + relv[:, None] * z + 4 * U * z) * np.abs(wn) + 4 * U * np.abs(bn)
    tol = tol + half_step(dt) * (np.abs(want) + tol) + _subnormal(dt)
    _close(_np(y), want, tol, "y")
    if residual or p > 0:
        _close(_np(h), hx, hb + half_step(dt) * (np.abs(hx) + hb) + _subnormal(dt), "h")
    else:
        assert h is None


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES + [(2000, 24), (1500, 128), (700, 1536), (400, 837)])
def test_backward(rows, cols, dtype):
    dt = TYPES[dtype]
    i = rows + cols + list(TYPES).index(dtype)
    wdt = torch.float32 if i % 2 else dt
    extra, p = i % 3 != 0, (0.0, 0.25)[(i // 2) % 2] if rows * cols < 200000 else 0.0
    h, dy = _rand((rows, cols), dt, 1, 1.5, 0.5), _rand((rows, cols), dt, 2)
    w = _rand((cols,), wdt, 3, 0.3, 1.0)
    dh = _rand((rows, cols), dt, 4) if extra else None
    hx = _np(h)
    _, m, s = B.layer_norm(hx, 1.0, 0.0, 1e-5)
    mean, rstd = torch.from_numpy(m).float(), torch.from_numpy(s).float()
    seed, off = 77 + i, 5
    rng = torch.tensor([seed, off], device="cuda")
    dx, dres, dw, db = sta.sta_layer_norm_backward(dy.cuda(), h.cuda(), mean.cuda(), rstd.cuda(), w.cuda(),
                                                   None if dh is None else dh.cuda(), True, p, rng)
    m, s = _np(mean), _np(rstd)
    wn = _np(w)
    want, wdw, wdb = B.layer_norm_backward(_np(dy), hx, m, s, wn)
    z = np.abs(hx - m[:, None]) * s[:, None]
    ez = 2 * U * z + U * (np.abs(m) * s)[:, None]
    g = np.abs(_np(dy) * wn)
    gm, gz = g.mean(1, keepdims=True), (g * z).mean(1, keepdims=True)
    # the two means are off by 80 u of the magnitudes' means
    tol = s[:, None] * (4 * U * g + 90 * U * gm + z * 90 * U * gz + ez * gz + z * (g * ez).mean(1, keepdims=True) + 4 * U * z * gz)
    if extra:
        want = want + _np(dh)
        tol = tol + 2 * U * np.abs(want)
    _close(_np(dres), want, tol + half_step(dt) * (np.abs(want) + tol) + _subnormal(dt), "dresidual")
    if p > 0:
        f = B.dropout_factor(rows, cols, p, seed, off)
        t2 = tol * f + 2 * U * np.abs(want * f)
        _close(_np(dx), want * f, t2 + half_step(dt) * (np.abs(want * f) + t2) + _subnormal(dt), "dx")
    # column sums: a thread adds the rows of one of the parts, then threads, warps and parts in order:
    # below rows + 64 additions one after the other
    steps = rows + 64
    sw, sb = (np.abs(_np(dy)) * (z + ez)).sum(0), np.abs(_np(dy)).sum(0)
    t = (np.abs(_np(dy)) * ez).sum(0) + steps * U * sw
    _close(_np(dw), wdw, t + half_step(wdt) * (np.abs(wdw) + t) + _subnormal(wdt), "dweight")
    t = steps * U * sb
    _close(_np(db), wdb, t + half_step(wdt) * (np.abs(wdb) + t) + _subnormal(wdt), "dbias")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols,p", [(1, 1, 0.5), (3, 5, 0.5), (9, 8, 0.1), (4, 13, 0.9), (31, 49, 0.25), (2, 1001, 0.5),
                                         (5, 2048, 0.1), (7, 7, 0.0), (6, 16, 1.0), (3, 17, 1.0), (1000, 3, 0.3)])
def test_dropout(rows, cols, p, dtype):
    dt = TYPES[dtype]
    x = _rand((rows, cols), dt, 5)
    seed, off = (1 << 62) + 12345, -7     # the whole 64 bits count
    y = sta.sta_dropout_forward(x.cuda(), p, torch.tensor([seed, off], device="cuda"))
    f = B.dropout_factor(rows, cols, p, seed, off & 0xFFFFFFFFFFFFFFFF)
    want = _np(x) * f
    got = _np(y)
    assert np.array_equal(got == 0, want == 0)
    tol = 2 * U * np.abs(want)
    _close(got, want, tol + half_step(dt) * (np.abs(want) + tol) + _subnormal(dt), "dropout")


def test_dropped_values_leave_zeros():
    x = torch.full((64, 40), float("inf"), device="cuda")
    x[1] = float("nan")
    rng = torch.tensor([3, 4], device="cuda")
    y = sta.sta_dropout_forward(x, 0.5, rng).cpu()
    f = torch.from_numpy(B.dropout_factor(64, 40, 0.5, 3, 4))
    assert torch.equal(y[f == 0], torch.zeros(int((f == 0).sum())))
    assert not torch.isfinite(y[f != 0]).any()


def test_counter_passes_32_bits():
    """More than 2^32 counter blocks, one per row: the counter's high word is used."""
    rows = 2 ** 32 + 5
    x = torch.ones(rows, 1, device="cuda", dtype=torch.bfloat16)
    y = sta.sta_dropout_forward(x, 0.5, torch.tensor([11, 22], device="cuda"))
    for first in (2 ** 31 - 4, rows - 12):
        got = y[first:first + 12].float().cpu().numpy()
        for i in range(12):
            n = first + i
            w = B.philox((n & 0xFFFFFFFF, n >> 32, 22, 0), (11, 0))
            assert got[i, 0] == (2.0 if (w[0] & 0xFFFF) >= 32768 else 0.0), n


def test_rows_and_columns_past_the_array_stay():
    """Nothing is written outside the outputs (odd sizes, every type)."""
    for dt in TYPES.values():
        for rows, cols in ((3, 9), (5, 128), (2, 837), (1, 8190)):
            n = rows * cols
            buf = torch.full((n + 64,), 7.0, device="cuda", dtype=dt)
            x = _rand((rows, cols), dt, 6).cuda()
            y = buf[:n].view(rows, cols)
            sta.sta_layer_norm_fwd(x, None, None, y)
            assert torch.equal(buf[n:], torch.full((64,), 7.0, device="cuda", dtype=dt))
            sta.sta_dropout(x, y, 0.5, torch.tensor([1, 2], device="cuda"))
            assert torch.equal(buf[n:], torch.full((64,), 7.0, device="cuda", dtype=dt))


def test_no_rows():
    x = torch.empty(0, 16, device="cuda")
    y, _, mean, _ = sta.sta_layer_norm_forward(x)
    assert y.shape == (0, 16) and mean.shape == (0,)
    w = torch.ones(16, device="cuda")
    _, _, dw, db = sta.sta_layer_norm_backward(x, x, mean, mean, w)
    assert torch.equal(dw, torch.zeros_like(dw)) and torch.equal(db, torch.zeros_like(db))
    sta.sta_dropout_forward(x, 0.5, torch.tensor([1, 2], device="cuda"))


def test_constant_row_and_nonfinite_rows_stay_apart():
    x = _rand((5, 64), torch.float32, 8)
    x[1] = 2.5
    x[2, 3] = float("inf")
    x[3, 4] = float("nan")
    y, _, mean, rstd = sta.sta_layer_norm_forward(x.cuda(), eps=1e-5)
    y = y.cpu()
    assert torch.equal(y[1], torch.zeros(64))
    assert rstd[1].item() == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    assert not torch.isfinite(y[2]).any() and not torch.isfinite(y[3]).any()
    want, _, _ = B.layer_norm(x[[0, 4]].double().numpy(), 1.0, 0.0, 1e-5)
    assert np.abs(y[[0, 4]].double().numpy() - want).max() < 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cols", [3, 7, 24, 37, 121, 257, 600, 837, 1153, 1999, 3000, 5000, 8190])
def test_constant_rows_are_the_bias(cols, dtype):
    """A row of one 16-bit value at any width: its sum is exact in fp32 (8 or 11 bits times at most
    13), the mean is that value, and y is the bias, not a rounding of the mean times 1 / sqrt(eps)."""
    dt = TYPES[dtype]
    x = _rand((40, 1), dt, 9, 200.0).expand(40, cols).contiguous().cuda()
    b = _rand((cols,), dt, 10).cuda()
    y, _, mean, rstd = sta.sta_layer_norm_forward(x, None, b, 1e-5)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(y, b.expand(40, cols))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=2.0 ** -20, atol=0)
    x[3, 0] = float("inf")
    _, _, mean, rstd = sta.sta_layer_norm_forward(x, None, b, 1e-5)
    assert mean[3] == float("inf") and torch.isnan(rstd[3]) and torch.isfinite(mean[4:]).all()


def test_deterministic_and_on_another_stream():
    h, dy = (_rand((5000, 300), torch.bfloat16, i).cuda() for i in (1, 2))
    w = _rand((300,), torch.float32, 3).cuda()
    _, _, mean, rstd = sta.sta_layer_norm_forward(h, w)
    torch.cuda.synchronize()
    first = sta.sta_layer_norm_backward(dy, h, mean, rstd, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = sta.sta_layer_norm_backward(dy, h, mean, rstd, w, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_graph_replay_reads_the_generator_state_anew():
    x = _rand((64, 256), torch.float32, 1).cuda()
    rng = torch.tensor([5, 0], device="cuda")
    y = torch.empty_like(x)
    sta.sta_dropout(x, y, 0.5, rng)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sta.sta_dropout(x, y, 0.5, rng)
    for off in (0, 9):
        rng[1] = off
        g.replay()
        torch.cuda.synchronize()
        f = B.dropout_factor(64, 256, 0.5, 5, off)
        assert np.array_equal(_np(y) == 0, f == 0)


@pytest.mark.parametrize("cols", [1536, 3000, 4096, 837])
def test_threads_with_unequal_calls_of_one_kernel(cols):
    """Calls from several threads that need unequal amounts of shared memory of the same kernels:
    with and without a residual (a gradient that reaches h), and at two widths of an instance.
    They go to the C entry points with ready arguments, which leaves the interpreter's lock, so
    that host code runs at the same time."""
    lib, rows, rounds = sta.load_library(), 16, 3000
    jobs, keep = [], []
    for i in range(8):
        c = cols - 8 * (i // 4)
        x, r = (_rand((rows, c), torch.bfloat16, 10 * i + j).cuda() for j in (1, 2))
        st = torch.cuda.Stream()
        y, _, mean, rstd = sta.sta_layer_norm_forward(x, residual=r if i % 2 else None)
        dx = sta.sta_layer_norm_backward(x, x, mean, rstd, None, r if i % 2 else None, False)[0]
        out = [torch.empty_like(x) for _ in range(2)]
        p = lambda t: t.data_ptr()  # noqa: E731
        res, raw = (p(r) if i % 2 else None), st.cuda_stream
        keep.append((x, r, y, mean, rstd, dx, out, st))
        if i % 4 < 2:
            jobs.append((lib.sta_layer_norm_fwd, (p(x), res, None, None, p(out[0]), None, None, None, rows, c, 0, 0, 1e-5, 0.0,
                                                  None, raw)))
        else:
            jobs.append((lib.sta_layer_norm_bwd, (p(x), p(x), p(mean), p(rstd), None, res, p(out[1]), None, None, None, rows, c,
                                                  0, 0, 0.0, None, None, 0, raw)))
    torch.cuda.synchronize()
    refused = []

    def work(fn, args):
        for _ in range(rounds):
            status = fn(*args)
            if status != sta.STA_OK:
                refused.append((status, lib.sta_last_cuda_error()))
                return

    ts = [threading.Thread(target=work, args=j) for j in jobs]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    assert not refused, refused
    for i, (_, _, y, _, _, dx, out, _) in enumerate(keep):
        assert torch.equal(out[0], y) if i % 4 < 2 else torch.equal(out[1], dx)
