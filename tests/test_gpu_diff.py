"""Differential attention on the GPU against the plain 64-bit form, element by element
within the bounds that block_oracle derives from the kernels' roundings."""
import math

import numpy as np
import pytest
import torch

import block_oracle as B
import sparse_attention_video_tile_b200 as sta
from sparse_attention_video_tile_b200 import autograd as A

pytestmark = pytest.mark.gpu


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


# batch, heads, d, grid, tile, windows
CASES = {
    "one_token": (1, 1, 128, (1, 1, 1), (6, 8, 8), [(1, 1, 1)]),
    "two_tokens_d64": (2, 2, 64, (1, 1, 2), (2, 8, 8), [(1, 1, 1), (3, 3, 3)]),
    "one_tile": (1, 2, 128, (2, 8, 8), (2, 8, 8), [(1, 1, 1), (2, 2, 2)]),
    "clip_d64": (1, 2, 64, (4, 16, 16), (2, 8, 8), [(1, 1, 1), (2, 2, 2)]),
    "windows": (1, 4, 128, (6, 24, 40), (6, 8, 8), [(1, 3, 3), (1, 2, 4), (1, 1, 5), (3, 1, 1)]),
    "image": (2, 2, 128, (1, 32, 64), (1, 8, 16), [(1, 3, 3), (1, 2, 2)]),
    "padded": (1, 3, 128, (7, 11, 13), (6, 8, 8), [(1, 1, 1), (2, 2, 2), (1, 2, 1)]),
    "padded_d64": (2, 3, 64, (5, 9, 14), (2, 8, 8), [(1, 1, 1), (3, 2, 2), (2, 1, 2)]),
    "pad_slabs": (1, 2, 128, (9, 8, 9), (8, 8, 8), [(1, 1, 1), (2, 1, 2)]),
    "short_last_tile": (1, 1, 64, (13, 4, 5), (12, 4, 8), [(2, 1, 1)]),
    "long_tiles": (1, 2, 128, (3, 5, 130), (1, 1, 128), [(2, 3, 2), (1, 1, 1)]),
    "tall_tiles": (1, 1, 128, (300, 1, 2), (128, 1, 1), [(2, 1, 2)]),
    "many_items": (1, 9, 64, (8, 24, 32), (2, 8, 8), [(1, 1, 1), (3, 3, 3), (1, 3, 1)] * 3),
}


def make(case, seed=0, scale_q=1.0):
    batch, heads, d, grid, tile, windows = CASES[case]
    g = torch.Generator().manual_seed(seed)
    L = math.prod(grid)
    q, k, v, do = (torch.randn(batch, heads, L, d, generator=g).to(torch.bfloat16) for _ in range(4))
    q = (q.float() * scale_q).to(torch.bfloat16)
    lam = torch.rand(heads, generator=g) * 1.2 - 0.2
    return q, k, v, do, lam, grid, tile, windows


def place(x, token_major):
    return (x.transpose(1, 2) if token_major else x).contiguous().cuda()


def back(x, token_major):
    x = x.transpose(1, 2) if token_major else x
    return x.double().cpu().numpy()


def check(got, want, bound, what):
    assert np.all(np.isfinite(got)), f"{what}: non-finite"
    ratio = np.abs(got - want) / bound
    assert ratio.max() <= 1.0, f"{what}: {int((ratio > 1).sum())} of {ratio.size} off, worst {ratio.max():.3g} of the bound"


def d(x):
    return x.double().numpy()


def check_forward(case, q, k, v, lam, grid, tile, windows, scale, out, out2, lse, token_major):
    out, out2 = back(out, token_major), back(out2, token_major)
    for h in range(q.shape[1]):
        mask = B.diff_mask(grid, tile, windows[h])
        for b in range(q.shape[0]):
            want, want2, wl, bo, bo2 = B.diff_head(d(q[b, h]), d(k[b, h]), d(v[b, h]), float(lam[h]), mask, scale)
            check(out[b, h], want, bo, f"{case} out")
            check(out2[b, h], want2, bo2, f"{case} out2")
            # scores in fp32 (at most 64 products, each row's magnitudes below 2^7), sum of exponentials to 2^-20
            check(lse[:, b, h].double().cpu().numpy(), wl, 2.0 ** -15 + 2.0 ** -22 * np.abs(wl), f"{case} lse")


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("case", list(CASES))
def test_forward(case, token_major):
    q, k, v, _, lam, grid, tile, windows = make(case)
    scale = 1.0 / math.sqrt(q.shape[-1] // 2)
    dev = [place(x, token_major) for x in (q, k, v)]
    r = sta.sta_diff_forward(*dev, lam.cuda(), grid, tile, windows, token_major=token_major, save=True)
    assert sta.sta_check_device_status() == sta.STA_OK
    check_forward(case, q, k, v, lam, grid, tile, windows, scale, *r, token_major)
    alone = sta.sta_diff_forward(*dev, lam.cuda(), grid, tile, windows, token_major=token_major)
    assert torch.equal(alone, r[0])


@pytest.mark.parametrize("case", ["windows", "padded_d64"])
def test_forward_large_scores(case):
    """Scores of tens: the running maximum rises block by block and O is rescaled."""
    q, k, v, _, lam, grid, tile, windows = make(case, 3, 12.0)
    scale = 1.0 / math.sqrt(q.shape[-1] // 2)
    r = sta.sta_diff_forward(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), grid, tile, windows, save=True)
    out, out2, lse = back(r[0], False), back(r[1], False), r[2].double().cpu().numpy()
    for h in range(q.shape[1]):
        mask = B.diff_mask(grid, tile, windows[h])
        for b in range(q.shape[0]):
            want, want2, wl, bo, bo2 = B.diff_head(d(q[b, h]), d(k[b, h]), d(v[b, h]), float(lam[h]), mask, scale)
            check(out[b, h], want, bo, "out")
            check(out2[b, h], want2, bo2, "out2")
            # |scores| reach 2^10 in the dot product: 64 u of that
            check(lse[:, b, h], wl, 2.0 ** -12 + 2.0 ** -22 * np.abs(wl), "lse")


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("case", list(CASES))
def test_backward(case, token_major):
    q, k, v, do, lam, grid, tile, windows = make(case, 1)
    scale = 1.0 / math.sqrt(q.shape[-1] // 2)
    leaves = [place(x, token_major).requires_grad_(True) for x in (q, k, v)]
    lam_c = lam.cuda().requires_grad_(True)
    out = A.sta_diff_attention(*leaves, lam_c, grid, tile, windows, token_major=token_major)
    grads = torch.autograd.grad(out, leaves + [lam_c], place(do, token_major))
    assert sta.sta_check_device_status() == sta.STA_OK
    got = [back(x, token_major) for x in grads[:3]]
    for h in range(q.shape[1]):
        mask = B.diff_mask(grid, tile, windows[h])
        dl, bl = 0.0, 0.0
        for b in range(q.shape[0]):
            w, bd = B.diff_head_backward(d(q[b, h]), d(k[b, h]), d(v[b, h]), float(lam[h]), d(do[b, h]), mask, scale)
            for name, x, y, z in zip(("dq", "dk", "dv"), got, w, bd):
                check(x[b, h], y, z, f"{case} {name}")
            dl, bl = dl + w[3], bl + bd[3]
        assert abs(float(grads[3][h]) - dl) <= bl, f"{case} dlam {float(grads[3][h])} {dl} {bl}"
