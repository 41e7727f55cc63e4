"""Differential attention, layer norm and dropout together, and the calls around them that
the single tests do not make: graphs, streams, threads, guards, non-finite values, tensors
past 2^31 elements."""
import math
import threading

import numpy as np
import pytest
import torch

import block_oracle as B
import sparse_attention_video_tile_b200 as sta
from sparse_attention_video_tile_b200 import autograd as A

pytestmark = pytest.mark.gpu

GRID, TILE = (5, 9, 14), (2, 8, 8)
WINDOWS = [(1, 1, 1), (3, 2, 2), (2, 1, 2)]


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
    assert sta.sta_check_device_status() == sta.STA_OK


def inputs(seed=0, batch=2, heads=3, d=64, grid=GRID):
    g = torch.Generator().manual_seed(seed)
    L = math.prod(grid)
    q, k, v, do = (torch.randn(batch, heads, L, d, generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    return q, k, v, do, (torch.rand(heads, generator=g) * 0.6 + 0.2).cuda()


def backward(q, k, v, lam, saved, do, windows=WINDOWS, scale=0.18, grid=GRID, tile=TILE, **kw):
    grads = [torch.full_like(x, float("nan")) for x in (q, k, v, lam)]
    sta.sta_diff_attention_bwd(q, k, v, lam, *saved, do, *grads, grid, tile, windows, scale, **kw)
    return grads


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_block_runs_as_its_parts():
    """Attention, head norm and dropout through one call equal the explicit calls, bit for
    bit, forward and backward; so does the residual norm behind them."""
    q, k, v, do, lam = inputs()
    w = torch.randn(64, device="cuda") * 0.2 + 0.8
    b = torch.randn(64, device="cuda") * 0.1
    rng, rng2 = torch.tensor([5, 6], device="cuda"), torch.tensor([5, 7], device="cuda")
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v, lam, w, b)]
    out = A.sta_diff_attention(*leaves[:4], GRID, TILE, WINDOWS, 0.18, norm_weight=leaves[4], norm_bias=leaves[5],
                               dropout_p=0.25, rng=rng)
    res = torch.randn(2, 3, 630, 64, device="cuda").bfloat16().requires_grad_(True)
    y, h = A.sta_layer_norm(out, residual=res, dropout_p=0.1, rng=rng2)
    dh = torch.randn(2, 3, 630, 64, device="cuda").bfloat16()
    rng.zero_()     # the masks belong to the calls, not to what the state becomes
    got = torch.autograd.grad((y, h), leaves + [res], (do, dh))
    rng = torch.tensor([5, 6], device="cuda")

    o, o2, lse = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
    n, _, m, s = sta.sta_layer_norm_forward(o, w, b)
    dr = sta.sta_dropout_forward(n, 0.25, rng)
    y2, h2, m2, s2 = sta.sta_layer_norm_forward(dr, residual=res.detach(), dropout_p=0.1, rng=rng2)
    assert torch.equal(out, dr) and torch.equal(y, y2) and torch.equal(h, h2)
    dx, dres, _, _ = sta.sta_layer_norm_backward(do, h2, m2, s2, None, dh, False, 0.1, rng2)
    dn = sta.sta_dropout_forward(dx, 0.25, rng)
    dattn, _, dw, db = sta.sta_layer_norm_backward(dn, o, m, s, w)
    want = backward(q, k, v, lam, (o, o2, lse), dattn) + [dw, db, dres]
    assert same(got, want)


def test_block_against_the_definition():
    """The chain's output in 64 bits: the attention's elementwise bound carried through the
    norm (its derivative at the exact row), with half a step of bf16 where a result is stored."""
    q, k, v, _, lam = inputs(1)
    w, b = torch.rand(64, device="cuda") + 0.5, torch.randn(64, device="cuda") * 0.1
    rng = torch.tensor([9, 1], device="cuda")
    y = A.sta_diff_attention(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, norm_weight=w, norm_bias=b, dropout_p=0.25, rng=rng)
    f = B.dropout_factor(2 * 3 * 630, 64, 0.25, 9, 1).reshape(2, 3, 630, 64)
    y = y.double().cpu().numpy()
    wn, bn = w.double().cpu().numpy(), b.double().cpu().numpy()
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    for h in range(3):
        mask = B.diff_mask(GRID, TILE, WINDOWS[h])
        for i in range(2):
            o, _, _, bo, _ = B.diff_head(d(q[i, h]), d(k[i, h]), d(v[i, h]), float(lam[h]), mask, 0.18)
            want, m, s = B.layer_norm(o, wn, bn, 1e-5)
            z = np.abs(o - m[:, None]) * s[:, None]
            # d(z_c) = rstd (e_c - mean e - z_c mean(z e)); twice it covers the second order (the
            # errors are below a tenth of a row's spread)
            e = 2 * s[:, None] * (bo + bo.mean(1, keepdims=True) + z * (z * bo).mean(1, keepdims=True)) * np.abs(wn) + 1e-5
            e = e + B.BF16 * (np.abs(want) + e)
            e = e * f[i, h] + B.BF16 * f[i, h] * (np.abs(want) + e)
            assert np.all(np.abs(y[i, h] - want * f[i, h]) <= e + 1e-12)


def test_strided_and_half_precision_gradients_reach_the_leaves():
    """Views that are not contiguous, and a gradient of another type, go through."""
    q, k, v, do, lam = inputs(2)
    qt = q.transpose(1, 2).contiguous().transpose(1, 2).requires_grad_(True)     # [B, heads, L, d], strided
    out = A.sta_diff_attention(qt, k, v, lam, GRID, TILE, WINDOWS, 0.18)
    (g,) = torch.autograd.grad(out, qt, do.float())
    saved = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
    assert torch.equal(out, saved[0]) and torch.equal(g, backward(q, k, v, lam, saved, do)[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slices_that_start_off_a_16_byte_boundary(dtype):
    """Rows of an odd width, sliced and joined again: the slices and the gradients that reach
    them are contiguous and start anywhere.  The same values as aligned copies give."""
    g = torch.Generator().manual_seed(5)
    base, res, up = (torch.randn(9, 37, generator=g).to(dtype).cuda() for _ in range(3))
    flat = torch.randn(1 + 2 * 37, generator=g).to(dtype).cuda()
    rng = torch.tensor([3, 4], device="cuda")

    def step(copy):
        f = (lambda t: t.clone()) if copy else (lambda t: t)
        x, r, w = (t.clone().requires_grad_() for t in (base, res, flat))
        parts = []
        for rows in (slice(0, 4), slice(4, 9)):
            y, h = A.sta_layer_norm(f(x[rows]), f(w[1:38]), f(w[38:]), 1e-5, f(r[rows]), 0.25, rng)
            parts.append(A.sta_dropout(f(y[1:]), 0.5, rng) + h[1:])
        out = torch.cat(parts)
        return (out,) + torch.autograd.grad(out, (x, r, w), up[:out.shape[0]])

    for a, b in zip(step(False), step(True)):
        assert torch.equal(a, b)


def test_without_gradients_nothing_is_saved():
    q, k, v, _, lam = inputs(2)
    want = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18)
    assert torch.equal(A.sta_diff_attention(q, k, v, lam, GRID, TILE, WINDOWS, 0.18), want)
    with torch.no_grad():
        q.requires_grad_(True)
        out = A.sta_diff_attention(q, k, v, lam, GRID, TILE, WINDOWS, 0.18)
    assert torch.equal(out, want) and not out.requires_grad


@pytest.mark.parametrize("p", [0.0, 0.25])
def test_norm_gradients_by_either_output(p):
    """Through y alone, h alone and both: the first two add up to the third within roundings,
    and an unused h is worth a zero gradient, bit for bit."""
    g = torch.Generator().manual_seed(3)
    t = [torch.randn(9, 40, generator=g).cuda().requires_grad_() for _ in range(2)]
    w, b = (torch.randn(40, generator=g).cuda().requires_grad_() for _ in range(2))
    dy, dh = (torch.randn(9, 40, generator=g).cuda() for _ in range(2))
    rng = torch.tensor([1, 2], device="cuda")
    grads = lambda *o: torch.autograd.grad(*o, retain_graph=True, allow_unused=True)  # noqa: E731
    y, h = A.sta_layer_norm(t[0], w, b, residual=t[1], dropout_p=p, rng=rng)
    leaves = (*t, w, b)
    by_y, by_h, by_both = grads(y, leaves, dy), grads(h, leaves, dh), grads((y, h), leaves, (dy, dh))
    assert same(by_y, grads((y, h), leaves, (dy, torch.zeros_like(dh))))
    for u, v, s in zip(by_y, by_h, by_both):
        assert torch.allclose(u + v, s, rtol=0, atol=2.0 ** -20 * float(s.abs().max() + v.abs().max()))
    assert not by_h[2].any() and not by_h[3].any()


def test_second_derivative_raises():
    q, k, v, do, lam = inputs(2)
    q.requires_grad_(True)
    out = A.sta_diff_attention(q, k, v, lam, GRID, TILE, WINDOWS, 0.18)
    (g,) = torch.autograd.grad(out, q, do, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.float().sum(), q)


def test_token_major_equals_head_major():
    q, k, v, do, lam = inputs(3)
    hm = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
    t = [x.transpose(1, 2).contiguous() for x in (q, k, v, do)]
    tm = sta.sta_diff_forward(*t[:3], lam, GRID, TILE, WINDOWS, 0.18, token_major=True, save=True)
    assert torch.equal(tm[0].transpose(1, 2), hm[0]) and torch.equal(tm[1].transpose(1, 2), hm[1]) and torch.equal(tm[2], hm[2])
    a = backward(q, k, v, lam, hm, do)
    b = backward(*t[:3], lam, tm, t[3], token_major=True)
    assert all(torch.equal(y.transpose(1, 2), x) for x, y in zip(a[:3], b[:3])) and torch.equal(a[3], b[3])


def test_deterministic():
    q, k, v, do, lam = inputs(4, d=128)
    saved = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
    first = backward(q, k, v, lam, saved, do)
    for _ in range(3):
        again = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
        assert same(again, saved) and same(backward(q, k, v, lam, saved, do), first)


def test_captured_and_replayed():
    """Forward and backward in one graph, replayed on new inputs, beside an eager call."""
    q, k, v, do, lam = inputs(5)
    saved = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)     # before any capture
    backward(q, k, v, lam, saved, do)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s2 = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
        g2 = backward(q, k, v, lam, s2, do)
    for seed in (6, 7):
        new = inputs(seed)
        for dst, src in zip((q, k, v, do, lam), new):
            dst.copy_(src)
        g.replay()
        eager = sta.sta_diff_forward(*new[:3], new[4], GRID, TILE, WINDOWS, 0.18, save=True)
        eg = backward(*new[:3], new[4], eager, new[3])
        torch.cuda.synchronize()
        assert same(s2, eager) and same(g2, eg)


def test_training_step_captured_and_replayed():
    """Forward and gradients of the whole block through autograd in one graph: attention, head norm,
    dropout, the residual norm, replayed on new inputs and a new generator state."""
    static = [x.requires_grad_(i != 3) for i, x in enumerate(inputs(30))]
    w = torch.randn(64, device="cuda").requires_grad_()
    rng = torch.tensor([3, 1], device="cuda")

    def step(q, k, v, do, lam):
        a = A.sta_diff_attention(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, norm_weight=w, dropout_p=0.25, rng=rng)
        y, h = A.sta_layer_norm(a, residual=q, dropout_p=0.1, rng=rng)
        return [y.detach(), h.detach()] + list(torch.autograd.grad(y, (q, k, v, lam, w), do))

    side = torch.cuda.Stream()      # warm up off the default stream, as captures want it
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(*static)
    for seed in (31, 32):
        with torch.no_grad():
            for dst, src in zip(static, inputs(seed)):
                dst.copy_(src)
            rng[1] = seed
        g.replay()
        torch.cuda.synchronize()
        assert same(got, step(*static)), seed


def test_two_streams_at_once():
    sets = [inputs(8 + i, d=128) for i in range(2)]
    want = []
    for q, k, v, do, lam in sets:
        s = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
        want.append((s, backward(q, k, v, lam, s, do)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for (q, k, v, do, lam), st in zip(sets, streams):
        s = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True, stream=st)
        with torch.cuda.stream(st):
            grads = [torch.empty_like(x) for x in (q, k, v, lam)]
        sta.sta_diff_attention_bwd(q, k, v, lam, *s, do, *grads, GRID, TILE, WINDOWS, 0.18, stream=st.cuda_stream)
        got.append((s, grads))
    torch.cuda.synchronize()
    for (s, gr), (s2, g2) in zip(want, got):
        assert same(s, s2) and same(gr, g2)


def test_from_threads_that_have_not_used_the_device():
    q, k, v, do, lam = inputs(11)
    saved = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
    want = backward(q, k, v, lam, saved, do)
    torch.cuda.synchronize()
    results, errors = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                a = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
                results[i] = (a, backward(q, k, v, lam, a, do))
            s.synchronize()
        except Exception as e:   # noqa: BLE001 - reported below
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors
    assert all(same(a, saved) and same(g, want) for a, g in results)


def test_nothing_outside_the_outputs_is_written():
    q, k, v, do, lam = inputs(12)
    need_b = sta.sta_diff_attention_bwd_workspace(q, GRID, TILE, WINDOWS)

    def guarded(numel, dtype):
        buf = torch.full((numel + 256,), 3.0, device="cuda", dtype=dtype)
        return buf, buf[:numel]

    bufs = {n: guarded(q.numel(), torch.bfloat16) for n in ("out", "out2", "dq", "dk", "dv")}
    bufs["lse"] = guarded(2 * q.numel() // 64, torch.float32)
    bufs["dlam"] = guarded(3, torch.float32)
    t = {n: b[1].view(q.shape if n not in ("lse", "dlam") else ((2, 2, 3, 630) if n == "lse" else (3,))) for n, b in bufs.items()}
    ws = torch.full((need_b + 256,), 7, device="cuda", dtype=torch.uint8)
    ins = [x.clone() for x in (q, k, v, do, lam)]
    sta.sta_diff_attention_fwd(q, k, v, lam, t["out"], GRID, TILE, WINDOWS, 0.18, t["out2"], t["lse"])
    sta.sta_diff_attention_bwd(q, k, v, lam, t["out"], t["out2"], t["lse"], do, t["dq"], t["dk"], t["dv"], t["dlam"], GRID, TILE,
                               WINDOWS, 0.18, workspace=ws[:need_b])
    torch.cuda.synchronize()
    for n, (buf, view) in bufs.items():
        assert torch.equal(buf[view.numel():], torch.full((256,), 3.0, device="cuda", dtype=buf.dtype)), n
        assert torch.isfinite(view).all(), n
    assert torch.equal(ws[need_b:], torch.full((256,), 7, device="cuda", dtype=torch.uint8))
    assert same(ins, (q, k, v, do, lam))
    with pytest.raises(sta.StaError, match="SCRATCH"):
        sta.sta_diff_attention_bwd(q, k, v, lam, t["out"], t["out2"], t["lse"], do, t["dq"], t["dk"], t["dv"], t["dlam"], GRID,
                                   TILE, WINDOWS, 0.18, workspace=ws[:need_b - 1])


def test_nonfinite_keys_reach_their_window_only():
    """A NaN or infinite key, value or query touches the rows whose windows hold it, no other."""
    q, k, v, _, lam = inputs(13, batch=1, heads=1)
    win, masks = [(1, 1, 1)], B.diff_mask(GRID, TILE, (1, 1, 1))
    clean = sta.sta_diff_forward(q, k, v, lam[:1], GRID, TILE, win, 0.18)
    for t, val in ((k, float("nan")), (k, float("inf")), (v, float("nan")), (v, float("-inf"))):
        x = t.clone()
        x[0, 0, 300, 5] = val
        args = (q, x, v) if t is k else (q, k, x)
        o = sta.sta_diff_forward(*args, lam[:1], GRID, TILE, win, 0.18)[0, 0]
        hit = torch.from_numpy(masks[:, 300]).cuda()
        assert torch.equal(o[~hit], clean[0, 0][~hit])
        bad = ~torch.isfinite(o[hit])
        assert bad[:, 5].all() if t is v else bad.all(1).float().mean() > 0.4   # an infinite key: about half the scores are -inf
    x = q.clone()
    x[0, 0, 7] = float("nan")
    o = sta.sta_diff_forward(x, k, v, lam[:1], GRID, TILE, win, 0.18)[0, 0]
    assert torch.isnan(o[7]).all() and torch.equal(o[8:], clean[0, 0, 8:])


def test_very_low_and_very_high_scores():
    """Scores far outside the exponential's range in either direction: the running maximum
    carries them (one query scores -2000 with every key, one +2000 with a late one)."""
    q, k, v, _, lam = inputs(14, batch=1, heads=1)
    q[0, 0, 3] = 0
    q[0, 0, 3, 0], q[0, 0, 3, 32] = -100.0, -100.0
    q[0, 0, 4] = 0
    q[0, 0, 4, 1], q[0, 0, 4, 33] = 100.0, 100.0
    k[0, 0, :, 0], k[0, 0, :, 32] = 100.0, 100.0
    k[0, 0, 600, 1], k[0, 0, 600, 33] = 100.0, 100.0
    win = [(3, 2, 2)]
    out = sta.sta_diff_forward(q, k, v, lam[:1], GRID, TILE, win, 0.18, save=True)
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, want2, lse, bo, bo2 = B.diff_head(d(q[0, 0]), d(k[0, 0]), d(v[0, 0]), float(lam[0]), B.diff_mask(GRID, TILE, win[0]), 0.18)
    assert torch.isfinite(out[0]).all()
    got, gl = d(out[0][0, 0]), d(out[2][:, 0, 0])
    # fp32 scores near 2^11 are off by 2^-13 and more after the scaling: 2^-9 of P covers it
    slack = 2.0 ** -9 * (1 + abs(float(lam[0]))) * np.abs(d(v[0, 0])).max()
    for r in (3, 4):
        assert np.all(np.abs(got[r] - want[r]) <= bo[r] + slack)
        assert np.all(np.abs(gl[:, r] - lse[:, r]) <= 2.0 ** -9)


def test_large_values_under_a_late_maximum():
    """Values of 2^90 and a row whose last key scores 50 (in log2) above the rest: the sums before
    the division must not be held against the first keys' maximum, and the order of the keys
    must not matter."""
    q, k, v, _, lam = inputs(16, batch=1, heads=1)
    v = (v.float() * 2.0 ** 90).bfloat16()
    q[0, 0, 3] = 0
    q[0, 0, 3, 0], q[0, 0, 3, 32] = 12.0, 12.0
    win = [(3, 2, 2)]
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    for key in (600, 1):
        k[0, 0, :, 0], k[0, 0, :, 32] = 0, 0
        k[0, 0, key, 0], k[0, 0, key, 32] = 16.0, 16.0
        out, out2, _ = sta.sta_diff_forward(q, k, v, lam[:1], GRID, TILE, win, 0.18, save=True)
        want, want2, _, bo, bo2 = B.diff_head(d(q[0, 0]), d(k[0, 0]), d(v[0, 0]), float(lam[0]), B.diff_mask(GRID, TILE, win[0]),
                                              0.18)
        assert torch.isfinite(out).all() and torch.isfinite(out2).all(), key
        assert np.all(np.abs(d(out[0, 0]) - want) <= bo) and np.all(np.abs(d(out2[0, 0]) - want2) <= bo2), key


def test_lambda_zero_negative_and_large():
    q, k, v, do, _ = inputs(15)
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    lam = torch.tensor([0.0, -0.75, 3.0], device="cuda")
    saved = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
    grads = backward(q, k, v, lam, saved, do)
    for h in range(3):
        mask = B.diff_mask(GRID, TILE, WINDOWS[h])
        dl = bl = 0.0
        for b in range(2):
            want, _, _, bo, _ = B.diff_head(d(q[b, h]), d(k[b, h]), d(v[b, h]), float(lam[h]), mask, 0.18)
            assert np.all(np.abs(d(saved[0][b, h]) - want) <= bo)
            w, bd = B.diff_head_backward(d(q[b, h]), d(k[b, h]), d(v[b, h]), float(lam[h]), d(do[b, h]), mask, 0.18)
            for g, x, y in zip(grads, w[:3], bd[:3]):
                assert np.all(np.abs(d(g[b, h]) - x) <= y)
            dl, bl = dl + w[3], bl + bd[3]
        assert abs(float(grads[3][h]) - dl) <= bl
    assert not grads[0][:, 0, :, 32:].any()    # lambda 0: the second map has no gradient


def test_lambda_far_above_one():
    """The stated accuracy at |lambda| = 30 and 100: the bound on the first map's dq and dk holds D_1's
    term that grows with |lambda|; the second map's grows as these gradients themselves do."""
    q, k, v, do, _ = inputs(17)
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    lam = torch.tensor([30.0, -100.0, 0.5], device="cuda")
    saved = sta.sta_diff_forward(q, k, v, lam, GRID, TILE, WINDOWS, 0.18, save=True)
    grads = backward(q, k, v, lam, saved, do)
    for h in range(3):
        mask = B.diff_mask(GRID, TILE, WINDOWS[h])
        dl = bl = 0.0
        for b in range(2):
            want, _, _, bo, _ = B.diff_head(d(q[b, h]), d(k[b, h]), d(v[b, h]), float(lam[h]), mask, 0.18)
            assert np.all(np.abs(d(saved[0][b, h]) - want) <= bo)
            w, bd = B.diff_head_backward(d(q[b, h]), d(k[b, h]), d(v[b, h]), float(lam[h]), d(do[b, h]), mask, 0.18)
            for g, x, y in zip(grads, w[:3], bd[:3]):
                assert np.all(np.abs(d(g[b, h]) - x) <= y)
            dl, bl = dl + w[3], bl + bd[3]
        assert abs(float(grads[3][h]) - dl) <= bl


def test_empty_batch():
    q = torch.empty(0, 2, 630, 64, device="cuda", dtype=torch.bfloat16)
    lam = torch.rand(2, device="cuda")
    o, o2, lse = sta.sta_diff_forward(q, q, q, lam, GRID, TILE, WINDOWS[:2], 0.18, save=True)
    assert o.shape == q.shape and lse.shape == (2, 0, 2, 630)
    ws = torch.empty(16, device="cuda")
    g = [torch.empty_like(q) for _ in range(3)]
    dl = torch.full_like(lam, float("nan"))
    sta.sta_diff_attention_bwd(q, q, q, lam, o, o2, lse, q, *g, dl, GRID, TILE, WINDOWS[:2], 0.18, workspace=ws)
    assert torch.equal(dl, torch.zeros_like(dl))


def test_tensors_past_two_to_the_31_elements():
    """The last heads of tensors of 2.3e9 elements equal the same heads alone."""
    grid, tile, heads, d = (48, 96, 160), (6, 8, 8), 25, 128
    L = math.prod(grid)
    win = [(1, 1, 1)] * heads
    q, k, v, do = (torch.empty(1, heads, L, d, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (q, k, v, do):
        for h in range(heads):
            t[0, h] = torch.randn(L, d, device="cuda", generator=g)
    assert q.numel() > 2 ** 31
    lam = torch.full((heads,), 0.4, device="cuda")
    saved = sta.sta_diff_forward(q, k, v, lam, grid, tile, win, 0.125, save=True)
    grads = [torch.empty_like(x) for x in (q, k, v, lam)]
    sta.sta_diff_attention_bwd(q, k, v, lam, *saved, do, *grads, grid, tile, win, 0.125)
    for h in (0, heads - 1):
        part = [x[:, h:h + 1].contiguous() for x in (q, k, v, do)]
        s1 = sta.sta_diff_forward(*part[:3], lam[:1], grid, tile, win[:1], 0.125, save=True)
        g1 = [torch.empty_like(x) for x in (*part[:3], lam[:1])]
        sta.sta_diff_attention_bwd(*part[:3], lam[:1], *s1, part[3], *g1, grid, tile, win[:1], 0.125)
        assert torch.equal(saved[0][:, h], s1[0][:, 0]) and torch.equal(saved[2][:, :, h], s1[2][:, :, 0])
        assert all(torch.equal(a[:, h], b[:, 0]) for a, b in zip(grads[:3], g1[:3]))
        assert torch.equal(grads[3][h], g1[3][0])
