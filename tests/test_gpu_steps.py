"""The pipelined loops of the norm and attention kernels over several steps each: every launch
shape of the norm with enough rows that each warp or block takes four or more steps and a
remainder, and padded attention with more items than SMs, against plain 64-bit forms.

The norm's forms are torch operations in 64 bits on the device; the bounds are those of
test_gpu_norm.py (row sums below 80 additions of fp32), with the column sums' additions counted from
the launch: a thread adds its rows of a part, then come at most 5 shuffles, 8 warps, 10 parts and 5
shuffles.
"""
import math

import numpy as np
import pytest
import torch

import block_oracle as B
import sparse_attention_video_tile_b200 as sta

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


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


def keep_factor(rows, cols, p, seed, off):
    """0 or 65536 / (65536 - threshold) of every element, on the device (block_oracle's
    dropout_factor, all counters at once)."""
    m = 0xFFFFFFFF
    thr = int(math.floor(p * 65536.0 + 0.5))
    blocks = -(-cols // 8)
    n = torch.arange(rows * blocks, device="cuda", dtype=torch.int64)
    c = [n & m, n >> 32, torch.full_like(n, off & m), torch.full_like(n, (off >> 32) & m)]
    k0, k1 = seed & m, (seed >> 32) & m

    def mul(a, b):   # high and low words of a 32 x 32 bit product, in 64-bit integers
        low = a * (b & 0xFFFF)
        return ((a * (b >> 16) + (low >> 16)) >> 16) & m, (a * b) & m

    for _ in range(10):
        (h0, l0), (h1, l1) = mul(0xD2511F53, c[0]), mul(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    keep = torch.stack([w >= thr for x in c for w in (x & 0xFFFF, x >> 16)], -1).view(rows, blocks * 8)[:, :cols]
    return keep.double() * (65536.0 / (65536 - thr))


def half(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps


def close(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    bad = (got - want).abs() > tol
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}, worst "
                             f"{float(((got - want).abs() / tol).max()):.3g} of the bound")


def randn(shape, dt, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dt)


def rows_of(cols):
    """Rows for four steps and more: a grid's step takes at most 4.9 M elements (148 SMs x 8 blocks of
    256 threads that hold 16 columns each; threads that hold more leave room for fewer blocks), and
    at 1 to 8 columns 64 rows a warp, 606 208 rows."""
    return max(20_000_000 // cols, 0 if cols > 8 else 2_430_000) + 5


def test_the_vectorised_mask_is_the_oracles():
    for rows, cols, off in ((9, 21, 5), (3, 64, -7)):
        want = B.dropout_factor(rows, cols, 0.3, (1 << 62) + 9, off & 0xFFFFFFFFFFFFFFFF)
        assert np.array_equal(keep_factor(rows, cols, 0.3, (1 << 62) + 9, off & 0xFFFFFFFFFFFFFFFF).cpu().numpy(), want)


# a width in every branch of the launch's choice, whole chunks of eight and not
WIDTHS = [8, 32, 64, 128, 256, 512, 1024, 1536, 2048, 4096, 5120, 8192,
          5, 31, 57, 121, 249, 505, 1017, 1153, 2001, 4001, 5001, 8191]


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", WIDTHS)
def test_norm_forward(cols, dtype, full):
    """full: residual, dropout, fp32 parameters; else the norm alone."""
    dt, rows = TYPES[dtype], rows_of(cols)
    p, seed, off = (0.3 if full else 0.0), 0x123456789ABCDEF + cols, 0xFEDCBA987
    wdt = torch.float32 if full else dt
    x, w, b = randn((rows, cols), dt, 1, 1.5, 3.0), randn((cols,), wdt, 2, 0.3, 1.0), randn((cols,), wdt, 3)
    res = randn((rows, cols), dt, 4) if full else None
    y, h, mean, rstd = sta.sta_layer_norm_forward(x, w, b, 1e-5, residual=res, dropout_p=p,
                                                  rng=torch.tensor([seed, off], device="cuda"))
    wd, bd = w.double(), b.double()
    step = max(1, 10_000_000 // cols)
    keep = keep_factor(rows, cols, p, seed, off) if full else None
    for r in range(0, rows, step):
        part = slice(r, r + step)
        hx = x[part].double()
        hb = torch.zeros_like(hx)
        if full:
            hx = hx * keep[part]
            hb = 2 * U * hx.abs()
            hx = hx + res[part].double()
            hb = hb + U * hx.abs()
        m = hx.mean(1, keepdim=True)
        s = 1.0 / torch.sqrt((hx - m).square().mean(1, keepdim=True) + 1e-5)
        big = hx.abs().amax(1, keepdim=True)
        close(mean[part], m[:, 0], 100 * U * big[:, 0] + 1e-30, "mean")
        relv = 256 * U + (100 * U * big * s) ** 2 + 4 * U * big * s
        close(rstd[part], s[:, 0], (relv * s)[:, 0], "rstd")
        z = (hx - m) * s
        want = z * wd + bd
        tol = (256 * U * s * big + (relv + 4 * U) * z.abs()) * wd.abs() + 4 * U * bd.abs()
        if full:   # the error of h in what y is made of (in fp32, before its store)
            tol = tol + s * (hb + hb.mean(1, keepdim=True) + z.abs() * (z.abs() * hb).mean(1, keepdim=True)) * wd.abs()
        close(y[part], want, tol + half(dt) * (want.abs() + tol) + tiny(dt), "y")
        if full:
            close(h[part], hx, hb + half(dt) * (hx.abs() + hb) + tiny(dt), "h")


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", WIDTHS)
def test_norm_backward(cols, dtype, full):
    dt, rows = TYPES[dtype], rows_of(cols)
    p, seed, off = (0.25 if full else 0.0), 99 + cols, 7
    wdt = torch.float32 if full else dt
    h, dy = randn((rows, cols), dt, 1, 1.5, 0.5), randn((rows, cols), dt, 2)
    w = randn((cols,), wdt, 3, 0.3, 1.0)
    dh = randn((rows, cols), dt, 4) if full else None
    _, _, mean, rstd = sta.sta_layer_norm_forward(h)
    dx, dres, dw, db = sta.sta_layer_norm_backward(dy, h, mean, rstd, w, dh, True, p, torch.tensor([seed, off], device="cuda"))
    n8 = -(-cols // 8)
    tpr = next((t for n, t in ((1, 1), (4, 2), (8, 4), (16, 8), (32, 16)) if n8 <= n), 32)
    block = n8 > (128 if cols % 8 == 0 else 64)
    adds = rows // (148 * (1 if block else 256 // tpr)) + 2 + 5 + 8 + 10 + 5
    wd = w.double()
    keep = keep_factor(rows, cols, p, seed, off) if full else None
    sums = [torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(5)]
    step = max(1, 10_000_000 // cols)
    for r in range(0, rows, step):
        part = slice(r, r + step)
        m, s, y = mean[part, None].double(), rstd[part, None].double(), dy[part].double()
        z = (h[part].double() - m) * s
        ez = 2 * U * z.abs() + U * m.abs() * s
        g = y * wd
        want = s * (g - g.mean(1, keepdim=True) - z * (g * z).mean(1, keepdim=True))
        for t, v in zip(sums, (y * z, y, y.abs() * ez, y.abs() * (z.abs() + ez), y.abs())):
            t += v.sum(0)
        g, z = g.abs(), z.abs()
        gm, gz = g.mean(1, keepdim=True), (g * z).mean(1, keepdim=True)
        tol = s * (4 * U * g + 90 * U * gm + z * 90 * U * gz + ez * gz + z * (g * ez).mean(1, keepdim=True) + 4 * U * z * gz)
        if full:
            want = want + dh[part].double()
            tol = tol + 2 * U * want.abs()
        close(dres[part], want, tol + half(dt) * (want.abs() + tol) + tiny(dt), "dresidual")
        if full:
            f = keep[part]
            t2 = tol * f + 2 * U * (want * f).abs()
            close(dx[part], want * f, t2 + half(dt) * ((want * f).abs() + t2) + tiny(dt), "dx")
    t = sums[2] + adds * U * sums[3]
    close(dw, sums[0], t + half(wdt) * (sums[0].abs() + t) + tiny(wdt), "dweight")
    t = adds * U * sums[4]
    close(db, sums[1], t + half(wdt) * (sums[1].abs() + t) + tiny(wdt), "dbias")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(300001, 7), (40000, 1536), (20003, 1153), (90001, 20), (1500000, 1), (3001, 8191)])
def test_dropout(rows, cols, dtype):
    dt = TYPES[dtype]
    x = randn((rows, cols), dt, 1)
    y = sta.sta_dropout_forward(x, 0.25, torch.tensor([5, 6], device="cuda"))
    want = x.double() * keep_factor(rows, cols, 0.25, 5, 6)
    assert torch.equal(y == 0, want == 0)
    tol = 2 * U * want.abs()
    close(y, want, tol + half(dt) * (want.abs() + tol) + tiny(dt), "dropout")


@pytest.mark.parametrize("cols", [1536, 1153])
def test_norm_past_two_to_the_31_elements(cols):
    """The last rows of arrays of 2.2e9 elements equal the same rows alone, forward and backward, and
    the mask there is dropout's own."""
    rows = 2_200_000_000 // cols
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for t in (x, r):
        for i in range(0, rows, 1 << 17):
            part = t[i:i + (1 << 17)]
            part.copy_(torch.randn(part.shape, device="cuda", generator=g))
    assert x.numel() > 2 ** 31
    w, rng = randn((cols,), torch.float32, 3, 0.3, 1.0), torch.tensor([5, 6], device="cuda")
    y, h, mean, rstd = sta.sta_layer_norm_forward(x, w, residual=r)
    dx = sta.sta_layer_norm_backward(r, h, mean, rstd, w, dh=x)[0]
    tails = [slice(0, 512), slice(rows - rows % 8 - 512, rows)]   # start on a 16-byte boundary
    for part in tails:
        y1, h1, m1, s1 = sta.sta_layer_norm_forward(x[part].clone(), w, residual=r[part].clone())
        assert torch.equal(y[part], y1) and torch.equal(h[part], h1)
        assert torch.equal(mean[part], m1) and torch.equal(rstd[part], s1)
        assert torch.equal(dx[part], sta.sta_layer_norm_backward(r[part].clone(), h1, m1, s1, w, dh=x[part].clone())[0])
    del y, dx
    masked = sta.sta_dropout_forward(x, 0.5, rng)
    _, h, mean, rstd = sta.sta_layer_norm_forward(x, dropout_p=0.5, rng=rng)
    assert torch.equal(h, masked)
    dx, dres, _, _ = sta.sta_layer_norm_backward(r, h, mean, rstd, w, dropout_p=0.5, rng=rng)
    dropped = sta.sta_dropout_forward(torch.ones_like(x), 0.5, rng) == 0
    for part in tails:
        assert torch.equal(dx[part] == 0, dropped[part] | (dres[part] == 0))


# ------------------------------------------------------------------ padded attention, several items a CTA

# batch, heads, d, grid, tile, windows of the heads in turn; items: batch x heads x 128-row blocks
ITEMS = {
    "slab_tiles_d64": (1, 22, 64, (3, 19, 21), (2, 8, 8), [(1, 1, 1), (2, 3, 3), (1, 2, 1), (2, 1, 2)]),     # 396
    "slab_tiles": (2, 11, 128, (3, 19, 21), (2, 8, 8), [(2, 3, 3), (1, 1, 1), (1, 1, 2)]),                  # 396
    "short_last_tile_d64": (2, 13, 64, (7, 9, 10), (6, 8, 8), [(2, 2, 2), (1, 1, 1), (2, 1, 2)]),           # 416
    "short_last_tile": (1, 26, 128, (7, 9, 10), (6, 8, 8), [(1, 2, 2), (2, 2, 1), (1, 1, 1)]),              # 416
}


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("case", list(ITEMS))
def test_padded_attention(case, token_major):
    """More than two items for every SM: a CTA's second and third item reuse its Q buffers, rings,
    accumulators and row sums."""
    batch, heads, dim, grid, tile, some = ITEMS[case]
    windows = [some[i % len(some)] for i in range(heads)]
    g = torch.Generator().manual_seed(21)
    q, k, v, do = (torch.randn(batch, heads, math.prod(grid), dim, generator=g).to(torch.bfloat16) for _ in range(4))
    lam = torch.rand(heads, generator=g) * 1.2 - 0.2
    scale = 1.0 / math.sqrt(dim // 2)
    put = lambda x: (x.transpose(1, 2) if token_major else x).contiguous().cuda()  # noqa: E731
    back = lambda x: (x.transpose(1, 2) if token_major else x).double().cpu().numpy()  # noqa: E731
    dev, lam_c = [put(x) for x in (q, k, v)], lam.cuda()
    saved = sta.sta_diff_forward(*dev, lam_c, grid, tile, windows, token_major=token_major, save=True)
    grads = [torch.full_like(x, float("nan")) for x in (*dev, lam_c)]
    sta.sta_diff_attention_bwd(*dev, lam_c, *saved, put(do), *grads, grid, tile, windows, scale, token_major=token_major)
    out, out2, lse, dl = back(saved[0]), back(saved[1]), saved[2].double().cpu().numpy(), grads[3].double().cpu().numpy()
    got = [back(x) for x in grads[:3]]
    n = lambda x: x.double().numpy()  # noqa: E731
    within = lambda a, b, t: np.all(np.abs(a - b) <= t)  # noqa: E731 - False for a NaN
    masks = {w: B.diff_mask(grid, tile, w) for w in set(windows)}
    for h in range(heads):
        wl = bl = 0.0
        for b in range(batch):
            args = [n(x[b, h]) for x in (q, k, v)]
            o, o2, ls, bo, bo2 = B.diff_head(*args, float(lam[h]), masks[windows[h]], scale)
            assert within(out[b, h], o, bo) and within(out2[b, h], o2, bo2), (b, h)
            assert within(lse[:, b, h], ls, 2.0 ** -15 + 2.0 ** -22 * np.abs(ls)), (b, h)
            w, bd = B.diff_head_backward(*args, float(lam[h]), n(do[b, h]), masks[windows[h]], scale)
            for name, x, y, t in zip(("dq", "dk", "dv"), got, w, bd):
                assert within(x[b, h], y, t), (name, b, h)
            wl, bl = wl + w[3], bl + bd[3]
        assert abs(dl[h] - wl) <= bl, ("dlambda", h)
