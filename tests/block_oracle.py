"""Plain 64-bit forms of differential attention, layer norm and dropout, for the tests.

Differential attention is two masked softmax attentions of the oracle (its mask, forward
and backward, each pinned in oracle_pins.py), put together by the operator's definition.
Beside each result stands an elementwise bound on what the kernels' roundings may add.
"""
import math

import numpy as np

import oracle.sta_oracle as O

BF16 = 2.0 ** -8     # half a step, relative
F32 = 2.0 ** -24


def diff_mask(grid, tile, window):
    c = O.raster_coords(grid)
    return O.sta_mask(c, c, grid, tile, window, pad=True)


def _softmax(q, k, mask, scale):
    s = scale * (q @ k.T)
    s = np.where(mask, s, -np.inf)
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    return p / l, (m + np.log(l))[:, 0]


def diff_head(q, k, v, lam, mask, scale):
    """out, out2, lse [2, L] of one head, and a bound on the kernel's error of out and out2."""
    h = q.shape[1] // 2
    p1, l1 = _softmax(q[:, :h], k[:, :h], mask, scale)
    p2, l2 = _softmax(q[:, h:], k[:, h:], mask, scale)
    out2 = p2 @ v
    out = p1 @ v - lam * out2
    av = np.abs(v)
    # P rounded to bf16 (half a step of each element); fp32 scores, exponentials (approximate to
    # 2^-22) and sums: 2^-14 of the same sums covers them; then the output's own rounding
    b2 = (BF16 + 2.0 ** -14) * (p2 @ av)
    b1 = (BF16 + 2.0 ** -14) * (p1 @ av) + abs(lam) * b2
    return out, out2, np.stack([l1, l2]), b1 + BF16 * (np.abs(out) + b1) + 1e-30, b2 + BF16 * (np.abs(out2) + b2) + 1e-30


def diff_head_backward(q, k, v, lam, do, mask, scale):
    """dq, dk, dv, dlam of one head and bounds on the kernels' errors of the same."""
    h = q.shape[1] // 2
    out, out2, _, bo, bo2 = diff_head(q, k, v, lam, mask, scale)
    dp = do @ v.T
    pc = np.zeros(mask.shape)
    dq, dk = np.zeros_like(q), np.zeros_like(k)
    bq, bk = np.zeros_like(q), np.zeros_like(k)
    ado = np.abs(do)
    # D_2 from the stored out2, D_1 from out and out2 (both bf16, with the forward's own error)
    e2 = (ado * bo2).sum(1)
    e1 = (ado * bo).sum(1) + abs(lam) * e2
    small = 2.0 ** -13    # fp32: the rebuilt P (lse and scores to 2^-15 absolute), dP, sums
    for m, (sl, w, e) in enumerate(((slice(0, h), 1.0, e1), (slice(h, 2 * h), -lam, e2))):
        p, _ = _softmax(q[:, sl], k[:, sl], mask, scale)
        pc += w * p
        d = (p * dp).sum(1, keepdims=True)
        ds = w * p * (dp - d)
        # error of dS before its rounding, then the rounding
        eds = abs(w) * p * (e[:, None] + small * (np.abs(dp) + np.abs(d) + (ado @ np.abs(v).T)))
        eds = eds + BF16 * (np.abs(ds) + eds)
        dq[:, sl] = scale * ds @ k[:, sl]
        dk[:, sl] = scale * ds.T @ q[:, sl]
        bq[:, sl] = scale * eds @ np.abs(k[:, sl])
        bk[:, sl] = scale * eds.T @ np.abs(q[:, sl])
        if m == 1:
            dlam = -float((p * dp).sum())
            # P_2 and dP in fp32; sums of rows x keys terms in fp32, by threads and then in order
            blam = small * float((p * (np.abs(dp) + ado @ np.abs(v).T)).sum())
            apc = np.abs(pc) + small * (np.abs(pc) + 2 * abs(w) * p)
    dv = pc.T @ do
    bv = (BF16 * apc + small * (np.abs(pc) + 2 * abs(lam) * 1.0 * mask * p)).T @ ado
    rnd = lambda x, b: b + BF16 * (np.abs(x) + b) + 1e-30  # noqa: E731
    return (dq, dk, dv, dlam), (rnd(dq, bq), rnd(dk, bk), rnd(dv, bv), blam + 1e-30)


# ------------------------------------------------------------------ dropout and layer norm

def philox(counter, key):
    """Philox 4x32-10 on Python integers: counter (c0, c1, c2, c3), key (k0, k1)."""
    c, (k0, k1) = list(counter), key
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k0, b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k1, a & 0xFFFFFFFF]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def dropout_factor(rows, cols, p, seed, offset):
    """0 or 65536 / (65536 - threshold) for every element."""
    thr = int(math.floor(p * 65536.0 + 0.5))
    fac = 65536.0 / (65536 - thr) if thr < 65536 else 0.0
    blocks = -(-cols // 8)
    out = np.zeros((rows, blocks * 8))
    key = (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)
    for r in range(rows):
        for b in range(blocks):
            n = r * blocks + b
            w = philox((n & 0xFFFFFFFF, n >> 32, offset & 0xFFFFFFFF, (offset >> 32) & 0xFFFFFFFF), key)
            for i in range(4):
                out[r, 8 * b + 2 * i] = fac if (w[i] & 0xFFFF) >= thr else 0.0
                out[r, 8 * b + 2 * i + 1] = fac if (w[i] >> 16) >= thr else 0.0
    return out[:, :cols]


def layer_norm(h, w, b, eps):
    mean = h.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((h - mean) ** 2).mean(1, keepdims=True) + eps)
    return (h - mean) * rstd * w + b, mean[:, 0], rstd[:, 0]


def layer_norm_backward(dy, h, mean, rstd, w):
    z = (h - mean[:, None]) * rstd[:, None]
    g = dy * w
    dh = rstd[:, None] * (g - g.mean(1, keepdims=True) - z * (g * z).mean(1, keepdims=True))
    return dh, (dy * z).sum(0), dy.sum(0)
