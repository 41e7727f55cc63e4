"""The differential tile attention block's operators, as cases that can be timed.

Three operators that a training step of a video transformer runs side by side:

* ``diff``: differential attention over sliding tile windows.  q, k, v are bf16 in
  raster order, [B, heads, L, d] or token-major [B, L, heads, d]; the first d/2
  columns of q and k belong to the first softmax map, the last d/2 to the second:
  out = (softmax(s Q1 K1^T) - lambda softmax(s Q2 K2^T)) V over each query tile's
  window of key tiles.  ``train`` cases run forward and backward.
* ``norm``: layer norm over the last dimension, optionally of
  h = residual + dropout(x), and its backward pass with the weight's and the bias's
  gradient.
* ``dropout``: dropout whose mask is a function of (seed, offset, row, column):
  element (r, c) of a [rows, cols] array takes 16-bit word c mod 8 of the Philox
  4x32-10 block with counter (r * ceil(cols / 8) + c div 8, offset) and key seed,
  and is kept where that word is at least round(65536 p).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a short low-resolution clip: one small launch, where latency counts
        {"name": "diff_fwd_clip", "op": "diff", "train": False, "save": False, "batch": 1, "heads": 2, "d": 64,
         "grid": "4,16,16", "tile": "2,8,8", "windows": "1,1,1;2,2,2", "token_major": False},
        # a latent that is no tile multiple, windows set per head, with what the backward keeps
        {"name": "diff_fwd_padded", "op": "diff", "train": False, "save": True, "batch": 1, "heads": 6, "d": 128,
         "grid": "11,22,37", "tile": "6,8,8", "windows": "1,3,3;2,3,3;1,1,5;2,2,4;1,3,3;2,3,5", "token_major": True},
        # the 720P, five-second latent with every head (the largest forward)
        {"name": "diff_fwd_video", "op": "diff", "train": False, "save": False, "batch": 1, "heads": 24, "d": 128,
         "grid": "30,48,80", "tile": "6,8,8", "windows": "3,3,3", "token_major": False},
        # training on two small odd-sized clips from a [B, L, heads * d] projection
        {"name": "diff_train_padded", "op": "diff", "train": True, "save": True, "batch": 2, "heads": 3, "d": 64,
         "grid": "5,9,14", "tile": "2,8,8", "windows": "1,1,1;3,2,2;2,1,2", "token_major": True},
        # training on the 720P latent, a shard of six heads (as when heads are split over GPUs)
        {"name": "diff_train_video", "op": "diff", "train": True, "save": True, "batch": 1, "heads": 6, "d": 128,
         "grid": "30,48,80", "tile": "6,8,8", "windows": "3,3,3", "token_major": False},
        # the norm of every head's output row: very many short rows
        {"name": "norm_fwd_heads", "op": "norm", "back": False, "rows": 115200 * 12, "cols": 128, "dtype": "bf16",
         "wdtype": "fp32", "residual": False, "p": 0.0, "bias": True},
        # residual stream + dropout of the attention branch, then the norm before the next projection
        {"name": "norm_fwd_block", "op": "norm", "back": False, "rows": 57600, "cols": 1536, "dtype": "bf16",
         "wdtype": "fp32", "residual": True, "p": 0.1, "bias": True},
        # a few conditioning tokens of an odd width
        {"name": "norm_fwd_ragged", "op": "norm", "back": False, "rows": 257, "cols": 1153, "dtype": "fp16",
         "wdtype": "fp16", "residual": True, "p": 0.0, "bias": False},
        # the backward of norm_fwd_block
        {"name": "norm_bwd_block", "op": "norm", "back": True, "rows": 57600, "cols": 1536, "dtype": "bf16",
         "wdtype": "fp32", "residual": True, "p": 0.1, "bias": True},
        # the backward of a small full-precision norm of an odd width
        {"name": "norm_bwd_ragged", "op": "norm", "back": True, "rows": 1000, "cols": 837, "dtype": "fp32",
         "wdtype": "fp32", "residual": False, "p": 0.0, "bias": True},
        # dropout of a whole latent's activations
        {"name": "dropout_video", "op": "dropout", "rows": 115200, "cols": 1536, "dtype": "bf16", "p": 0.1},
        # dropout of a small full-precision array of an odd width
        {"name": "dropout_ragged", "op": "dropout", "rows": 77, "cols": 1001, "dtype": "fp32", "p": 0.5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


# tiles that split into 128-row slabs of whole frames
_TILES = ((6, 8, 8), (2, 8, 8), (1, 8, 16), (4, 4, 8), (8, 4, 4), (1, 16, 8), (4, 8, 8))


def draw(rng):
    op = rng.choice(("diff", "diff", "norm", "norm", "dropout"))
    if op == "diff":
        train = rng.random() < 0.5
        d = rng.choice((64, 128))
        tile = rng.choice(_TILES)
        while True:
            grid = (_log_int(rng, 1, 30), _log_int(rng, 4, 48), _log_int(rng, 4, 80))
            batch, heads = rng.choice((1, 1, 2, 3)), rng.randint(1, 12)
            n = [-(-a // b) for a, b in zip(grid, tile)]
            wins = [tuple(rng.randint(1, 5 if x > 3 else 3) for x in n) for _ in range(heads)]
            case = {"op": "diff", "train": train, "save": train or rng.random() < 0.5, "batch": batch, "heads": heads,
                    "d": d, "grid": ",".join(map(str, grid)), "tile": ",".join(map(str, tile)),
                    "windows": ";".join(",".join(map(str, w)) for w in wins), "token_major": rng.random() < 0.5}
            # plain indexing walks tile by tile: keep the walk, and the products, within the listed cases'
            if attended(case) * d <= 4e11 and math.prod(n) * len(set(wins)) <= 2400:
                return case
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    cols = rng.choice((64, 128, 1536, 2048)) if rng.random() < 0.4 else _log_int(rng, 1, 8192)
    rows = _log_int(rng, 1, min(400000, 80000000 // cols))
    if op == "dropout":
        return {"op": "dropout", "rows": rows, "cols": cols, "dtype": dtype, "p": rng.choice((0.0, 0.1, 0.25, 0.5))}
    residual = rng.random() < 0.5
    return {"op": "norm", "back": rng.random() < 0.5, "rows": rows, "cols": cols, "dtype": dtype,
            "wdtype": rng.choice((dtype, "fp32")), "residual": residual,
            "p": rng.choice((0.0, 0.1, 0.3)) if residual else 0.0, "bias": rng.random() < 0.7}


def _ints(s):
    return tuple(int(x) for x in s.split(","))


def _windows(case):
    w = [_ints(x) for x in case["windows"].split(";")]
    return w * case["heads"] if len(w) == 1 else w


def attended(case):
    """(query, key) pairs of real tokens that a diff case attends, over batch and heads."""
    grid, tile = _ints(case["grid"]), _ints(case["tile"])
    total = 0
    for win in _windows(case):
        prod = 1
        for g, t, w in zip(grid, tile, win):
            n = -(-g // t)
            w = min(w, n)
            size = [min(t, g - a * t) for a in range(n)]
            s = [min(max(a - w // 2, 0), n - w) for a in range(n)]
            prod *= sum(size[a] * sum(size[s[a]:s[a] + w]) for a in range(n))
        total += prod
    return total * case["batch"]


def work(case):
    if case["op"] == "diff":
        L = math.prod(_ints(case["grid"]))
        elems = case["batch"] * case["heads"] * L * case["d"]
        rows = case["batch"] * case["heads"] * L
        pairs = attended(case)
        if case["train"]:   # q, k, v, dout read; out, dq, dk, dv written
            return {"bytes": 8 * elems * 2, "flops": 14 * case["d"] * pairs}
        extra = elems * 2 + rows * 8 if case["save"] else 0
        return {"bytes": 4 * elems * 2 + extra, "flops": 4 * case["d"] * pairs}
    size = DTYPES[case["dtype"]].itemsize
    n = case["rows"] * case["cols"]
    if case["op"] == "dropout":
        return {"bytes": 2 * n * size, "flops": 2 * n}
    wb = DTYPES[case["wdtype"]].itemsize * case["cols"] * (2 if case["bias"] else 1)
    if case["back"]:
        # dy, h (and the residual stream's gradient) read; dx (and the residual's gradient) written
        arrays = 3 + (1 if case["residual"] else 0) + (1 if case["p"] > 0 else 0)
        return {"bytes": arrays * n * size + 2 * wb + case["rows"] * 8, "flops": 12 * n}
    arrays = 2 + (2 if case["residual"] else 0)
    return {"bytes": arrays * n * size + wb + case["rows"] * 8, "flops": 8 * n}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, dtype):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    st = {"case": case}
    if case["op"] == "diff":
        B, H, d = case["batch"], case["heads"], case["d"]
        grid, tile = _ints(case["grid"]), _ints(case["tile"])
        L = math.prod(grid)
        shape = (B, L, H, d) if case["token_major"] else (B, H, L, d)
        for name in ("q", "k", "v") + (("dout",) if case["train"] else ()):
            st[name] = randn(*shape, dtype=torch.bfloat16)
        # the learned subtraction weight starts between 0.2 and 0.8 in the layers of such a model
        st["lam"] = 0.2 + 0.6 * torch.rand(H, generator=g, device="cuda")
        st.update(grid=grid, tile=tile, windows=_windows(case), scale=1.0 / math.sqrt(d // 2))
        if case["train"]:
            for name in ("q", "k", "v", "lam"):
                st[name].requires_grad_(True)
        return st
    rows, cols, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
    st["x"] = randn(rows, cols, dtype=dtype)
    gc = torch.Generator().manual_seed(seed)
    st["rng"] = torch.randint(0, 1 << 62, (2,), generator=gc, dtype=torch.int64).cuda()
    if case["op"] == "dropout":
        return st
    wd = DTYPES[case["wdtype"]]
    st["weight"] = (1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(wd)
    st["bias"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(wd) if case["bias"] else None
    st["eps"] = 1e-5
    if not case["back"]:
        # activations are not centred: a mean of its own for each row
        st["x"] = (st["x"].float() * 1.5 + randn(rows, 1, dtype=torch.float32)).to(dtype)
        st["residual"] = randn(rows, cols, dtype=dtype) if case["residual"] else None
        return st
    # backward: the normalised array, its statistics and the gradients that arrive
    h = (st.pop("x").float() * 1.5 + randn(rows, 1, dtype=torch.float32)).to(dtype)
    st["h"] = h
    step = max(1, (1 << 27) // cols)
    mean = torch.empty(rows, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    for r in range(0, rows, step):
        x = h[r:r + step].double()
        m = x.mean(1)
        mean[r:r + step] = m.float()
        rstd[r:r + step] = (1.0 / torch.sqrt((x - m[:, None]).square().mean(1) + st["eps"])).float()
    st["mean"], st["rstd"] = mean, rstd
    st["dy"] = randn(rows, cols, dtype=dtype)
    st["dh"] = randn(rows, cols, dtype=dtype) if case["residual"] else None
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if case["op"] == "diff":
        return _run_diff_own(st) if own else _run_diff_plain(st)
    if case["op"] == "norm":
        return _run_norm_own(st) if own else _run_norm_plain(st)
    return _run_dropout_own(st) if own else (_dropout_plain(st["x"].float(), case["p"], st["rng"]).to(st["x"].dtype),)


def _run_diff_own(st):
    import sparse_attention_video_tile_b200 as sta
    from sparse_attention_video_tile_b200 import autograd as A
    case = st["case"]
    args = (st["q"], st["k"], st["v"], st["lam"], st["grid"], st["tile"], st["windows"])
    if case["train"]:
        out = A.sta_diff_attention(*args, scale=st["scale"], token_major=case["token_major"])
        grads = torch.autograd.grad(out, (st["q"], st["k"], st["v"], st["lam"]), st["dout"])
        return (out.detach(),) + tuple(grads)
    r = sta.sta_diff_forward(*args, scale=st["scale"], token_major=case["token_major"], save=case["save"])
    return r if case["save"] else (r,)


def _run_norm_own(st):
    import sparse_attention_video_tile_b200 as sta
    case = st["case"]
    if not case["back"]:
        y, h, mean, rstd = sta.sta_layer_norm_forward(st["x"], st["weight"], st["bias"], st["eps"],
                                                      residual=st["residual"], dropout_p=case["p"],
                                                      rng=st["rng"] if case["p"] > 0 else None)
        return (y, h, mean, rstd) if case["residual"] else (y, mean, rstd)
    dx, dres, dw, db = sta.sta_layer_norm_backward(st["dy"], st["h"], st["mean"], st["rstd"], st["weight"],
                                                   dh=st["dh"], bias=case["bias"], dropout_p=case["p"],
                                                   rng=st["rng"] if case["p"] > 0 else None)
    out = (dx,) + ((dres,) if case["p"] > 0 else ()) + (dw,) + ((db,) if case["bias"] else ())
    return out


def _run_dropout_own(st):
    import sparse_attention_video_tile_b200 as sta
    return (sta.sta_dropout_forward(st["x"], st["case"]["p"], st["rng"]),)


# ------------------------------------------------------------------ plain forms: dropout and layer norm

def _philox_words(rng, first_row, rows, blocks):
    """16-bit words [rows, blocks * 8] of rows first_row .. first_row + rows - 1 (int64 arithmetic)."""
    m = 0xFFFFFFFF
    seed, off = rng[0], rng[1]
    n = (torch.arange(first_row, first_row + rows, device=rng.device, dtype=torch.int64)[:, None] * blocks +
         torch.arange(blocks, device=rng.device, dtype=torch.int64)[None, :])
    c = [n & m, (n >> 32) & m, (off & m).expand_as(n), ((off >> 32) & m).expand_as(n)]
    k0, k1 = seed & m, (seed >> 32) & m

    def mulhilo(a, b):
        lo16, hi16 = b & 0xFFFF, b >> 16
        low = a * lo16
        hi = (a * hi16 + (low >> 16)) >> 16
        return hi & m, (a * b) & m

    for _ in range(10):
        h0, l0 = mulhilo(0xD2511F53, c[0])
        h1, l1 = mulhilo(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    words = torch.stack([w for x in c for w in (x & 0xFFFF, x >> 16)], dim=-1)
    return words.reshape(rows, blocks * 8)


def _dropout_plain(x, p, rng):
    rows, cols = x.shape
    thr = int(math.floor(p * 65536.0 + 0.5))
    out = torch.empty_like(x)
    blocks = -(-cols // 8)
    step = max(1, (1 << 25) // cols)
    scale = 65536.0 / (65536 - thr) if thr < 65536 else 0.0
    for r in range(0, rows, step):
        n = min(step, rows - r)
        keep = _philox_words(rng, r, n, blocks)[:, :cols] >= thr
        out[r:r + n] = torch.where(keep, x[r:r + n] * scale, torch.zeros((), device=x.device))
    return out


def _run_norm_plain(st):
    case, w, b = st["case"], st["weight"].float(), st["bias"]
    dtype = DTYPES[case["dtype"]]
    if not case["back"]:
        h = st["x"].float()
        if case["p"] > 0:
            h = _dropout_plain(h, case["p"], st["rng"])
        if case["residual"]:
            h = h + st["residual"].float()
        mean = h.mean(1)
        cen = h - mean[:, None]
        rstd = 1.0 / torch.sqrt((cen * cen).mean(1) + st["eps"])
        y = cen * rstd[:, None] * w
        if b is not None:
            y = y + b.float()
        y = y.to(dtype)
        return (y, h.to(dtype), mean, rstd) if case["residual"] else (y, mean, rstd)
    dy, h = st["dy"].float(), st["h"].float()
    xhat = (h - st["mean"][:, None]) * st["rstd"][:, None]
    gy = dy * w
    c1 = gy.mean(1, keepdim=True)
    c2 = (gy * xhat).mean(1, keepdim=True)
    dh = (gy - c1 - xhat * c2) * st["rstd"][:, None]
    if st["dh"] is not None:
        dh = dh + st["dh"].float()
    dw = (dy * xhat).sum(0).to(DTYPES[case["wdtype"]])
    outs = (dh.to(dtype),) if case["p"] == 0 else (_dropout_plain(dh, case["p"], st["rng"]).to(dtype), dh.to(dtype))
    outs = outs + (dw,)
    if case["bias"]:
        outs = outs + (dy.sum(0).to(DTYPES[case["wdtype"]]),)
    return outs


# ------------------------------------------------------------------ plain form: differential attention

class _Tiles:
    """Raster <-> tiles of the padded latent, windows and validity, in plain indexing."""

    def __init__(self, case, device):
        self.grid, self.tile = _ints(case["grid"]), _ints(case["tile"])
        self.n = [-(-a // b) for a, b in zip(self.grid, self.tile)]
        self.token_major = case["token_major"]
        pad = [n * t for n, t in zip(self.n, self.tile)]
        T, H, W = self.grid
        idx = torch.full(pad, -1, dtype=torch.int64, device=device)
        idx[:T, :H, :W] = torch.arange(T * H * W, device=device).reshape(T, H, W)
        (nt, nh, nw), (tt, th, tw) = self.n, self.tile
        idx = idx.reshape(nt, tt, nh, th, nw, tw).permute(0, 2, 4, 1, 3, 5)
        self.idx = idx.reshape(nt * nh * nw, tt * th * tw)      # raster token of (tile, local), -1 for pads
        self.valid = self.idx >= 0

    def tiles(self, x):
        """[B, heads, tiles, ntile, d] fp32, pad tokens zero."""
        x = x.detach()
        x = x.permute(0, 2, 1, 3) if self.token_major else x
        t = x[:, :, self.idx.clamp(min=0)].float()
        return t * self.valid[None, None, :, :, None]

    def raster(self, t):
        """Back to raster order and the case's layout (t: [B, heads, tiles, ntile, ...])."""
        B, H = t.shape[:2]
        flat = t.reshape(B, H, -1, *t.shape[4:])
        v = self.valid.reshape(-1)
        out = torch.empty((B, H, math.prod(self.grid)) + tuple(t.shape[4:]), dtype=t.dtype, device=t.device)
        out[:, :, self.idx.reshape(-1)[v]] = flat[:, :, v]
        return out

    def keys(self, qt, win):
        (nt, nh, nw) = self.n
        a = (qt // (nh * nw), (qt // nw) % nh, qt % nw)
        r = []
        for x, w, n in zip(a, win, self.n):
            w = min(w, n)
            s = min(max(x - w // 2, 0), n - w)
            r.append(range(s, s + w))
        return [(i * nh + j) * nw + k for i in r[0] for j in r[1] for k in r[2]]


def _maps(qx, kx, scale, valid):
    """The two softmax maps and their log-sum-exps; qx [.., n, d], kx [.., m, d]."""
    half = qx.shape[-1] // 2
    probs, lses = [], []
    for m in range(2):
        s = torch.matmul(qx[..., m * half:(m + 1) * half], kx[..., m * half:(m + 1) * half].transpose(-1, -2))
        s *= scale
        if valid is not None:
            s.masked_fill_(~valid, float("-inf"))
        mx = s.amax(-1, keepdim=True)
        s = torch.exp_(s.sub_(mx))
        tot = s.sum(-1, keepdim=True)
        probs.append(s.div_(tot))
        lses.append((mx + torch.log(tot)).squeeze(-1))
    return probs, lses


def _run_diff_plain(st):
    case = st["case"]
    tl = _Tiles(case, st["q"].device)
    q, k, v = (tl.tiles(st[x]) for x in ("q", "k", "v"))
    B, H, nT, ntile, d = q.shape
    lam = st["lam"].detach().float()
    half = d // 2
    out, out2 = torch.empty_like(v), torch.empty_like(v)
    lse = torch.empty((2, B, H, nT, ntile), device=q.device)
    groups = {}
    for h, w in enumerate(st["windows"]):
        groups.setdefault(tuple(w), []).append(h)
    train = case["train"]
    if train:
        do = tl.tiles(st["dout"])
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
        dlam = torch.zeros(H, device=q.device)
    padded = not bool(tl.valid.all()) if any(g % t for g, t in zip(tl.grid, tl.tile)) else False
    for win, heads in groups.items():
        hs = torch.tensor(heads, device=q.device)
        lm = lam[hs][None, :, None, None]
        qg, kg, vg = q[:, hs], k[:, hs], v[:, hs]
        if train:
            dog, dkg, dvg, dqg = do[:, hs], torch.zeros_like(kg), torch.zeros_like(kg), torch.zeros_like(kg)
        og, o2g = torch.empty_like(vg), torch.empty_like(vg)
        lg = torch.empty((2,) + tuple(og.shape[:4]), device=q.device)
        for qt in range(nT):
            kt = tl.keys(qt, win)
            kx = kg[:, :, kt].flatten(2, 3)
            vx = vg[:, :, kt].flatten(2, 3)
            (p1, p2), (l1, l2) = _maps(qg[:, :, qt], kx, st["scale"], tl.valid[kt].reshape(-1) if padded else None)
            lg[0, :, :, qt], lg[1, :, :, qt] = l1, l2
            o2 = torch.matmul(p2, vx)
            o2g[:, :, qt] = o2
            og[:, :, qt] = torch.matmul(p1, vx) - lm * o2
            if train:
                dox = dog[:, :, qt]
                dp = torch.matmul(dox, vx.transpose(-1, -2))
                dvg[:, :, kt] += torch.matmul((p1 - lm * p2).transpose(-1, -2), dox).unflatten(2, (len(kt), ntile))
                d1 = (p1 * dp).sum(-1, keepdim=True)
                d2 = (p2 * dp).sum(-1, keepdim=True)
                dlam[hs] -= d2.sum(dim=(0, 2, 3))
                ds1 = p1 * (dp - d1) * st["scale"]
                ds2 = p2 * (dp - d2) * (-lm * st["scale"])
                qx = qg[:, :, qt]
                dqg[:, :, qt] = torch.cat((torch.matmul(ds1, kx[..., :half]), torch.matmul(ds2, kx[..., half:])), -1)
                dkx = torch.cat((torch.matmul(ds1.transpose(-1, -2), qx[..., :half]),
                                 torch.matmul(ds2.transpose(-1, -2), qx[..., half:])), -1)
                dkg[:, :, kt] += dkx.unflatten(2, (len(kt), ntile))
        out[:, hs], out2[:, hs], lse[:, :, hs] = og, o2g, lg
        if train:
            dq[:, hs], dk[:, hs], dv[:, hs] = dqg, dkg, dvg

    def back(t):
        r = tl.raster(t).to(torch.bfloat16)
        return r.permute(0, 2, 1, 3).contiguous() if tl.token_major else r

    if train:
        return back(out), back(dq), back(dk), back(dv), dlam
    if not case["save"]:
        return (back(out),)
    return back(out), back(out2), torch.stack([tl.raster(lse[0]), tl.raster(lse[1])])


# ------------------------------------------------------------------ definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "diff":
        return _exact_diff(case, st)
    if case["op"] == "norm":
        return _exact_norm(case, st)
    return (st["x"].double() * _exact_keep(case["rows"], case["cols"], case["p"], st["rng"]),)


def _exact_keep(rows, cols, p, rng):
    """The dropout factor of every element: 0 or 65536 / (65536 - threshold), fp64."""
    seed, off = (int(x) for x in rng.tolist())
    thr = int(math.floor(p * 65536.0 + 0.5))
    blocks = (cols + 7) // 8
    fac = 65536.0 / (65536 - thr) if thr < 65536 else 0.0
    out = torch.empty((rows, cols), dtype=torch.float64, device="cuda")
    u32 = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    step = max(1, (1 << 24) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        ctr = np.arange(r * blocks, (r + n) * blocks, dtype=np.uint64)
        x0, x1 = ctr & u32, ctr >> sh
        x2, x3 = np.full_like(ctr, off & 0xFFFFFFFF), np.full_like(ctr, (off >> 32) & 0xFFFFFFFF)
        ka, kb = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
        for _ in range(10):
            a = x0 * np.uint64(0xD2511F53)
            b = x2 * np.uint64(0xCD9E8D57)
            x0, x1, x2, x3 = (b >> sh) ^ x1 ^ np.uint64(ka), b & u32, (a >> sh) ^ x3 ^ np.uint64(kb), a & u32
            ka, kb = (ka + 0x9E3779B9) & 0xFFFFFFFF, (kb + 0xBB67AE85) & 0xFFFFFFFF
        quad = np.stack((x0, x1, x2, x3), axis=1).astype("<u4")
        words = quad.view("<u2").reshape(n, blocks * 8)[:, :cols]
        out[r:r + n] = torch.from_numpy((words >= thr).astype(np.uint8)).cuda().double() * fac
    return out


def _exact_norm(case, st):
    w = st["weight"].double()
    fac = _exact_keep(case["rows"], case["cols"], case["p"], st["rng"]) if case["p"] > 0 else None
    if not case["back"]:
        h = st["x"].double()
        if fac is not None:
            h = h * fac
        if st["residual"] is not None:
            h = h + st["residual"].double()
        var, mean = torch.var_mean(h, dim=1, unbiased=False)
        rstd = (var + st["eps"]).rsqrt()
        y = (h - mean[:, None]) * rstd[:, None] * w + (st["bias"].double() if st["bias"] is not None else 0.0)
        return (y, h, mean, rstd) if case["residual"] else (y, mean, rstd)
    # the vector-Jacobian product of the normalisation at the given statistics
    rs = st["rstd"].double()[:, None]
    z = (st["h"].double() - st["mean"].double()[:, None]) * rs
    dy = st["dy"].double()
    u = dy * w
    n = case["cols"]
    grad = rs / n * (n * u - u.sum(1, keepdim=True) - z * (u * z).sum(1, keepdim=True))
    if st["dh"] is not None:
        grad = grad + st["dh"].double()
    outs = (grad,) if fac is None else (grad * fac, grad)
    outs = outs + ((dy * z).sum(0),)
    return outs + (dy.sum(0),) if case["bias"] else outs


def _exact_diff(case, st):
    """Masked softmax over raster tokens: every query tile's keys are the tokens whose tile
    coordinates lie in its window; gradients by automatic differentiation of that."""
    dev = st["q"].device
    grid, tile, d = st["grid"], st["tile"], case["d"]
    T, H, W = grid
    tok = torch.arange(T * H * W, device=dev)
    coord = (tok // (H * W) // tile[0], tok // W % H // tile[1], tok % W // tile[2])
    n = [-(-a // b) for a, b in zip(grid, tile)]
    heads_first = (lambda x: x.transpose(1, 2)) if case["token_major"] else (lambda x: x)
    q, k, v = (heads_first(st[x].detach()).double() for x in ("q", "k", "v"))
    lam = st["lam"].detach().double()
    out, out2 = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros((2,) + tuple(q.shape[:3]), dtype=torch.float64, device=dev)
    if case["train"]:
        dout = heads_first(st["dout"]).double()
        gq, gk, gv, gl = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(lam)
    by_win = {}
    for h, w in enumerate(st["windows"]):
        by_win.setdefault(tuple(w), []).append(h)
    for win, hl in by_win.items():
        for at in range(n[0]):
            for ah in range(n[1]):
                for aw in range(n[2]):
                    here = torch.ones_like(tok, dtype=torch.bool)
                    seen = torch.ones_like(tok, dtype=torch.bool)
                    for c, a, w, m in zip(coord, (at, ah, aw), win, n):
                        w = min(w, m)
                        lo = min(max(a - w // 2, 0), m - w)
                        here &= c == a
                        seen &= (c >= lo) & (c < lo + w)
                    qi, ki = here.nonzero()[:, 0], seen.nonzero()[:, 0]
                    for h0 in range(0, len(hl), 4):
                        hs = hl[h0:h0 + 4]
                        hsel = torch.tensor(hs, device=dev)[:, None]
                        leaf = [q[:, hsel, qi], k[:, hsel, ki], v[:, hsel, ki], lam[hs]]
                        if case["train"]:
                            leaf = [x.requires_grad_(True) for x in leaf]
                        qx, kx, vx, lx = leaf
                        s = [st["scale"] * (a @ b.transpose(-1, -2)) for a, b in
                             zip(qx.split(d // 2, -1), kx.split(d // 2, -1))]
                        ls = [torch.logsumexp(x, -1) for x in s]
                        p = [torch.exp(x - y[..., None]) for x, y in zip(s, ls)]
                        o2 = p[1] @ vx
                        o = p[0] @ vx - lx[None, :, None, None] * o2
                        out[:, hsel, qi], out2[:, hsel, qi] = o.detach(), o2.detach()
                        for m in range(2):
                            lse[m][:, hsel, qi] = ls[m].detach()
                        if case["train"]:
                            g = torch.autograd.grad(o, leaf, dout[:, hsel, qi])
                            gq[:, hsel, qi] += g[0]
                            gk[:, hsel, ki] += g[1]
                            gv[:, hsel, ki] += g[2]
                            gl[hs] += g[3]
    if case["train"]:
        return tuple(heads_first(x) for x in (out, gq, gk, gv)) + (gl,)
    return (heads_first(out), heads_first(out2), lse) if case["save"] else (heads_first(out),)
