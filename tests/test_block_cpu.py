"""Argument checks of differential attention, layer norm and dropout that need no GPU
(they return before any device call), the host-side sizes, and the 64-bit forms that the
GPU tests compare with, pinned to published values, closed forms and autograd."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_oracle as B
import oracle.sta_oracle as O
import sparse_attention_video_tile_b200 as sta
from sparse_attention_video_tile_b200 import sta_dim3

NULL, ALIGN, ALIAS, SHAPE, WINDOW, HEADDIM, ARG, SCRATCH = 1, 2, 3, 4, 5, 6, 10, 11
BASE = 0x7F0000000000   # addresses that nothing dereferences
STEP = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_video_tile_b200.build import build
    build()
    return sta.load_library()


def addr(i):
    return BASE + i * STEP


def _on_gpu():
    return torch.cuda.is_available()


# ------------------------------------------------------------------ differential attention

def diff_args(back, **change):
    a = dict(batch=1, heads=2, d=128, token_major=0, grid=(6, 16, 16), tile=(6, 8, 8), windows=[(1, 1, 1), (1, 2, 2)],
             scale=0.125, ws=1 << 28)
    names = (["q", "k", "v", "lam", "out", "out2", "lse", "dout", "dq", "dk", "dv", "dlam", "work"] if back else
             ["q", "k", "v", "lam", "out", "out2", "lse"])
    a.update({n: addr(i) for i, n in enumerate(names)})
    a.update(change)
    w = a["windows"]
    win = None
    if w is not None:
        win = (sta_dim3 * max(1, len(w)))(*[sta_dim3(*x) for x in w])
    ptrs = [a[n] for n in names if n != "work"]
    return (*ptrs, a["batch"], a["heads"], a["d"], a["token_major"], sta_dim3(*a["grid"]), sta_dim3(*a["tile"]), win,
            a["scale"], *((a["work"], a["ws"]) if back else ()), None)


DIFF_REFUSALS = [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(lam=None), NULL), (dict(out=None), NULL),
    (dict(windows=None), NULL), (dict(q=addr(0) + 8), ALIGN), (dict(out=addr(4) + 2), ALIGN), (dict(lse=addr(6) + 1), ALIGN),
    (dict(lam=addr(3) + 2), ALIGN), (dict(d=96), HEADDIM), (dict(d=256), HEADDIM), (dict(batch=-1), ARG),
    (dict(heads=-1), ARG), (dict(heads=257, windows=[(1, 1, 1)] * 257), ARG), (dict(token_major=2), ARG),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(scale=1e-45), ARG), (dict(windows=[(1, 1, 1), (1, 0, 1)]), WINDOW), (dict(grid=(0, 16, 16)), SHAPE),
    (dict(grid=(6, -1, 16)), SHAPE), (dict(tile=(6, 8, 0)), SHAPE), (dict(tile=(6, 5, 5)), SHAPE),
    (dict(tile=(3, 8, 8)), SHAPE), (dict(tile=(1, 16, 16)), SHAPE), (dict(grid=(1 << 30, 16, 16)), SHAPE),
    (dict(tile=(1 << 30, 8, 8)), SHAPE), (dict(grid=(1 << 20, 1 << 12, 1 << 12)), SHAPE),
    (dict(batch=1 << 24, heads=2), SHAPE), (dict(out=addr(0)), ALIAS), (dict(out=addr(1) + 256), ALIAS),
]


@pytest.mark.parametrize("change,status", DIFF_REFUSALS)
@pytest.mark.parametrize("back", [False, True])
def test_diff_refusals(lib, back, change, status):
    if back and change.get("out") in (addr(0), addr(1) + 256):
        change = dict(dq=change["out"])   # out is an input of the backward
    fn = lib.sta_diff_attention_bwd if back else lib.sta_diff_attention_fwd
    assert fn(*diff_args(back, **change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dv=None), NULL), (dict(dlam=None), NULL), (dict(lse=None), NULL),
    (dict(out2=None), NULL), (dict(dout=None), NULL), (dict(work=None), NULL), (dict(ws=1000), SCRATCH),
    (dict(work=addr(12) + 8), ALIGN), (dict(dlam=addr(11) + 1), ALIGN), (dict(dv=addr(7)), ALIAS), (dict(dk=addr(8)), ALIAS),
    (dict(work=addr(2)), ALIAS), (dict(dlam=addr(3)), ALIAS)])
def test_diff_backward_refusals(lib, change, status):
    assert lib.sta_diff_attention_bwd(*diff_args(True, **change)) == status


def test_diff_empty_batch_is_a_no_op(lib):
    none = dict(q=None, k=None, v=None, lam=None, out=None, out2=None, lse=None, work=None, ws=0)
    assert lib.sta_diff_attention_fwd(*diff_args(False, batch=0, **none)) == sta.STA_OK
    assert lib.sta_diff_attention_fwd(*diff_args(False, heads=0, windows=[], **none)) == sta.STA_OK
    assert lib.sta_diff_attention_bwd(*diff_args(True, heads=0, windows=[], dout=None, dq=None, dk=None, dv=None, dlam=None,
                                                 **none)) == sta.STA_OK


@pytest.mark.skipif(_on_gpu(), reason="the valid call would run")
def test_valid_calls_fail_loudly_without_a_gpu(lib):
    assert lib.sta_diff_attention_fwd(*diff_args(False)) in (7, 8)
    assert lib.sta_diff_attention_bwd(*diff_args(True)) in (7, 8)
    assert lib.sta_layer_norm_fwd(*norm_args()) in (7, 8)
    assert lib.sta_layer_norm_bwd(*norm_bwd_args()) in (7, 8)
    assert lib.sta_dropout(addr(0), addr(1), 4, 8, 0, 0.5, addr(2), None) in (7, 8)


def test_diff_workspace_sizes(lib):
    q = torch.empty(2, 3, 6 * 16 * 20, 64)
    n = sta.sta_diff_attention_bwd_workspace(q, (6, 16, 20), (6, 8, 8), [(1, 1, 1)] * 3)
    rows = 2 * 3 * 6 * 16 * 24     # of the padded latent
    parts = 2 * 3 * (2 * 3 * 3)    # 128-row blocks
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    assert n == 4 * up(rows * 64 * 2) + up(rows * 16) + up(parts * 16)
    with pytest.raises(sta.StaError):
        sta.sta_diff_attention_bwd_workspace(q, (6, 16, 20), (6, 5, 5), [(1, 1, 1)] * 3)


def test_diff_binding_checks_before_the_library(lib):
    q = torch.empty(1, 2, 1536, 128, dtype=torch.bfloat16)
    lam = torch.empty(2)
    g, t, w = (6, 16, 16), (6, 8, 8), [(1, 1, 1)] * 2
    with pytest.raises(ValueError, match="CUDA"):
        sta.sta_diff_forward(q, q, q, lam, g, t, w)
    with pytest.raises(ValueError, match="window per head"):
        sta.sta_diff_forward(q, q, q, lam, g, t, w[:1])
    with pytest.raises(ValueError, match="T\\*H\\*W"):
        sta.sta_diff_forward(q, q, q, lam, (6, 16, 15), t, w)
    with pytest.raises(ValueError, match="must be \\[batch"):
        sta.sta_diff_forward(q[0], q, q, lam, g, t, w)


# ------------------------------------------------------------------ layer norm and dropout

def norm_args(**change):
    a = dict(x=addr(0), res=addr(1), w=addr(2), b=addr(3), y=addr(4), h=addr(5), mean=addr(6), rstd=addr(7), rows=4, cols=64,
             dtype=0, pdtype=2, eps=1e-5, p=0.1, rng=addr(8))
    a.update(change)
    return (a["x"], a["res"], a["w"], a["b"], a["y"], a["h"], a["mean"], a["rstd"], a["rows"], a["cols"], a["dtype"],
            a["pdtype"], a["eps"], a["p"], a["rng"], None)


def norm_bwd_args(**change):
    a = dict(dy=addr(0), h=addr(1), mean=addr(2), rstd=addr(3), w=addr(4), dh=addr(5), dx=addr(6), dres=addr(7), dw=addr(8),
             db=addr(9), rows=4, cols=64, dtype=0, pdtype=2, p=0.1, rng=addr(10), work=addr(11), ws=1 << 20)
    a.update(change)
    return (a["dy"], a["h"], a["mean"], a["rstd"], a["w"], a["dh"], a["dx"], a["dres"], a["dw"], a["db"], a["rows"],
            a["cols"], a["dtype"], a["pdtype"], a["p"], a["rng"], a["work"], a["ws"], None)


COMMON = [
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=-8), SHAPE), (dict(cols=8193), SHAPE),
    (dict(rows=1 << 40), SHAPE), (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(dtype=0, pdtype=1), ARG),
    (dict(p=-0.1), ARG), (dict(p=1.5), ARG), (dict(p=float("nan")), ARG), (dict(rng=None), NULL), (dict(rng=addr(8) + 4), ALIGN),
]


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(x=addr(0) + 2), ALIGN), (dict(w=addr(2) + 4), ALIGN), (dict(mean=addr(6) + 2), ALIGN),
    (dict(y=addr(0)), ALIAS), (dict(h=addr(1) + 16), ALIAS), (dict(h=addr(4)), ALIAS), (dict(mean=addr(7)), ALIAS),
    (dict(y=addr(3)), ALIAS)])
def test_layer_norm_refusals(lib, change, status):
    assert lib.sta_layer_norm_fwd(*norm_args(**change)) == status


@pytest.mark.parametrize("change,status", COMMON[:-1] + [
    (dict(dy=None), NULL), (dict(h=None), NULL), (dict(mean=None), NULL), (dict(dx=None, dres=None), NULL),
    (dict(work=None), NULL), (dict(ws=16), SCRATCH), (dict(dx=addr(6) + 8), ALIGN), (dict(work=addr(11) + 8), ALIGN),
    (dict(dx=addr(0)), ALIAS), (dict(dres=addr(6)), ALIAS), (dict(dw=addr(4)), ALIAS), (dict(work=addr(5)), ALIAS)])
def test_layer_norm_backward_refusals(lib, change, status):
    assert lib.sta_layer_norm_bwd(*norm_bwd_args(**change)) == status


@pytest.mark.parametrize("args,status", [
    ((None, addr(1), 4, 8, 0, 0.5, addr(2), None), NULL), ((addr(0), None, 4, 8, 0, 0.5, addr(2), None), NULL),
    ((addr(0), addr(1), 4, 8, 0, 0.5, None, None), NULL), ((addr(0), addr(1) + 8, 4, 8, 0, 0.5, addr(2), None), ALIGN),
    ((addr(0), addr(0) + 32, 4, 8, 0, 0.5, addr(2), None), ALIAS), ((addr(0), addr(0), 4, 8, 0, 0.5, addr(2), None), ALIAS),
    ((addr(0), addr(1), -4, 8, 0, 0.5, addr(2), None), SHAPE), ((addr(0), addr(1), 4, 0, 0, 0.5, addr(2), None), SHAPE),
    ((addr(0), addr(1), 4, 8, 7, 0.5, addr(2), None), ARG), ((addr(0), addr(1), 4, 8, 0, 1.01, addr(2), None), ARG)])
def test_dropout_refusals(lib, args, status):
    assert lib.sta_dropout(*args) == status


def test_layer_norm_workspace(lib):
    assert sta.sta_layer_norm_bwd_workspace(0, 16) == 0
    assert sta.sta_layer_norm_bwd_workspace(1, 16) >= 2 * 16 * 4
    with pytest.raises(sta.StaError):
        sta.sta_layer_norm_bwd_workspace(4, 8193)


def test_norm_binding_checks(lib):
    x = torch.empty(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        sta.sta_layer_norm_forward(x)
    with pytest.raises(TypeError, match="bfloat16"):
        sta.sta_layer_norm_fwd(x.double(), None, None, x.double())
    with pytest.raises(TypeError):
        sta.sta_dropout_forward(x.numpy(), 0.5, None)
    from sparse_attention_video_tile_b200 import autograd as A
    with pytest.raises(ValueError, match="rng"):
        A.sta_layer_norm(x, dropout_p=0.5)
    with pytest.raises(ValueError, match="rng"):
        A.sta_dropout(x, 0.5, None)
    assert A.sta_dropout(x, 0.0, None) is x


def test_geometry_follows_values_that_change():
    """The grid, tile and windows of a call are kept by value: a tensor that holds a number may
    hold another one in the next call."""
    from sparse_attention_video_tile_b200 import block
    n, w = torch.tensor(4), torch.tensor([[1, 2, 3], [3, 2, 1]])
    grid, windows = (n, 16, 16), [tuple(r) for r in w]
    dims = lambda d: (d.t, d.h, d.w)  # noqa: E731
    for a, b in ((4, 1), (7, 2)):
        n.fill_(a)
        w[0, 0] = b
        g, _, ws = block._geometry(grid, (2, 8, 8), windows)
        assert dims(g) == (a, 16, 16) and [dims(x) for x in ws] == [(b, 2, 3), (3, 2, 1)]
    plain = block._geometry([4, 16, 16], (2, 8, 8), [[1, 2, 3]])
    assert block._geometry((4, 16, 16), [2, 8, 8], ((1, 2, 3),)) is plain
    assert block._geometry((np.int64(4), 16, 16), (2, 8, 8), np.array([[1, 2, 3]])) is plain
    for i in range(200):
        block._geometry((4, 16, 16 + i), (2, 8, 8), [(1, 2, 3)])
    assert len(block._GEOMETRIES) <= 64


class Recorder:
    """Stands in for the binding under the autograd functions: keeps the calls' arguments and
    returns tensors of the right shapes."""

    def __init__(self, monkeypatch):
        from sparse_attention_video_tile_b200 import autograd as A
        self.A, self.forward, self.backward = A, [], []
        monkeypatch.setattr(A, "sta_diff_forward", self.diff_forward)
        monkeypatch.setattr(A, "sta_diff_attention_bwd", self.diff_backward)

    def diff_forward(self, q, k, v, lam, *args, save=False, **kw):
        self.forward.append((args, save))
        return (q * 1, q * 1, torch.zeros(2, *q.shape[:3])) if save else q * 1

    def diff_backward(self, *args, **kw):
        self.backward.append(args[12:])
        for g in args[8:12]:
            g.zero_()


def test_backward_uses_the_numbers_of_its_forward(monkeypatch):
    rec = Recorder(monkeypatch)
    q = torch.zeros(1, 1, 1024, 64, dtype=torch.bfloat16, requires_grad=True)
    n = torch.tensor(4)
    out = rec.A.sta_diff_attention(q, q, q, torch.zeros(1), (n, 16, 16), (2, 8, 8), [(n, 1, 1)])
    n.fill_(7)
    out.sum().backward()
    assert rec.forward[0][0][:3] == rec.backward[0][:3] == ((4, 16, 16), (2, 8, 8), [(4, 1, 1)])


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode, torch.enable_grad])
@pytest.mark.parametrize("leaf", [None, 0, 3])
def test_saves_only_for_a_backward(monkeypatch, mode, leaf):
    """out2 and the log-sum-exps are written where gradients are on and something requires one."""
    rec = Recorder(monkeypatch)
    t = [torch.zeros(1, 1, 1024, 64, dtype=torch.bfloat16) for _ in range(3)] + [torch.zeros(1)]
    if leaf is not None:
        t[leaf].requires_grad_(True)
    want = leaf is not None and mode is torch.enable_grad
    with mode():
        out = rec.A.sta_diff_attention(*t, (4, 16, 16), (2, 8, 8), [(1, 1, 1)])
    assert rec.forward[0][1] is want and out.requires_grad is want


@pytest.mark.parametrize("use", ["y", "h", "both"])
def test_the_gradient_of_an_unused_output_is_not_made(monkeypatch, use):
    """h = residual + dropout(x) is returned and often dropped: its gradient then stays None,
    instead of zeros that the kernel reads."""
    from sparse_attention_video_tile_b200 import autograd as A
    seen = []
    monkeypatch.setattr(A, "sta_layer_norm_forward",
                        lambda x, w, b, eps, r, p, rng: (x * 1, x * 1, torch.zeros(4), torch.ones(4)))

    def bwd(dy, h, mean, rstd, weight, dx, dres, dw, db, dh, p, rng):
        seen.append((dy, dh))
        dx.zero_()

    monkeypatch.setattr(A, "sta_layer_norm_bwd", bwd)
    x, r = (torch.randn(4, 8, requires_grad=True) for _ in range(2))
    y, h = A.sta_layer_norm(x, residual=r)
    sum({"y": [y], "h": [h], "both": [y, h]}[use]).sum().backward()
    dy, dh = seen[0]
    assert (dh is None) is (use == "y")
    assert torch.equal(dy, torch.zeros(4, 8) if use == "h" else torch.ones(4, 8))
    assert x.grad is not None and r.grad is not None


@pytest.mark.parametrize("p", [-0.1, 1.5, float("nan")])
def test_a_probability_outside_its_range_is_refused(monkeypatch, p):
    """By name and in every call, not taken as no dropout."""
    rec = Recorder(monkeypatch)
    q = torch.zeros(1, 1, 1024, 64, dtype=torch.bfloat16)
    for rng in (None, torch.zeros(2, dtype=torch.int64)):
        for call in (lambda: rec.A.sta_diff_attention(q, q, q, torch.zeros(1), (4, 16, 16), (2, 8, 8), [(1, 1, 1)],
                                                      dropout_p=p, rng=rng),
                     lambda: rec.A.sta_dropout(q, p, rng), lambda: rec.A.sta_layer_norm(q, dropout_p=p, rng=rng)):
            with pytest.raises(ValueError, match="dropout_p"):
                call()
    assert not rec.forward
    with pytest.raises(ValueError, match="rng"):
        rec.A.sta_dropout(q, 0.5, [1, 2])


def test_a_stream_of_another_device_is_refused():
    """Its kernels would run on that device and read this one's memory."""
    from types import SimpleNamespace

    from sparse_attention_video_tile_b200 import block

    class OnGpu(torch.Tensor):
        device = torch.device("cuda", 0)

    x = torch.zeros(2, 8).as_subclass(OnGpu)
    stream = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="the stream is on cuda:1"):
        block._On(stream, x, None).__enter__()


def test_sizes_past_32_bits_are_refused_not_cut(lib):
    """The library takes columns, heads, d, grids and windows as 32-bit numbers; a larger size
    must not arrive as its low half (2^32 + 8 columns as 8)."""
    x = torch.empty(2 ** 32 + 8, dtype=torch.bfloat16, device="meta")
    rng = torch.zeros(2, dtype=torch.int64)
    stat = torch.empty(1, device="meta")
    for call in (lambda: sta.sta_dropout(x, x, 0.5, rng), lambda: sta.sta_dropout_forward(x, 0.5, rng),
                 lambda: sta.sta_layer_norm_forward(x), lambda: sta.sta_layer_norm_fwd(x, None, None, x),
                 lambda: sta.sta_layer_norm_bwd(x, x, stat, stat, None, x),
                 lambda: sta.sta_layer_norm_backward(x, x, stat, stat)):
        with pytest.raises(ValueError, match="columns"):
            call()
    for rows, cols in ((1, 2 ** 32 + 8), (2 ** 64 + 1, 8), (1, -2 ** 32 + 8)):
        with pytest.raises(sta.StaError):
            sta.sta_layer_norm_bwd_workspace(rows, cols)
    q = torch.empty(1, 1, 1, 2 ** 32 + 64, dtype=torch.bfloat16, device="meta")
    lam = torch.empty(1, device="meta")
    with pytest.raises(ValueError, match="below 2\\^31"):
        sta.sta_diff_forward(q, q, q, lam, (1, 1, 1), (6, 8, 8), [(1, 1, 1)])
    small = torch.empty(1, 1, 384, 64, dtype=torch.bfloat16, device="meta")
    for windows in ([(2 ** 32 + 1, 1, 1)], [(1, -2 ** 31 - 1, 1)]):
        with pytest.raises(ValueError, match="32 bits"):
            sta.sta_diff_forward(small, small, small, lam, (6, 8, 8), (6, 8, 8), windows)
    with pytest.raises(ValueError, match="32 bits"):
        sta.sta_attended_pairs(1, 1, (2 ** 32 + 6, 8, 8), (6, 8, 8), [(1, 1, 1)])


def test_package_imports_without_the_block_module():
    with pytest.raises(AttributeError):
        sta.sta_no_such_operator


# ------------------------------------------------------------------ the 64-bit forms

def test_philox_known_answers():
    """The generator's published known-answer vectors."""
    f = 0xFFFFFFFF
    assert B.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert B.philox((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert B.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_factor_keeps_the_expectation():
    f = B.dropout_factor(200, 96, 0.25, 12, 34)
    assert set(np.unique(f)) == {0.0, 65536 / (65536 - 16384)}
    kept = (f > 0).mean()
    assert abs(kept - 0.75) < 5 * math.sqrt(0.75 * 0.25 / f.size)
    # rows start new blocks: the mask of a row does not depend on the number of rows
    assert np.array_equal(f[:7], B.dropout_factor(7, 96, 0.25, 12, 34))


def _head(seed, n, d):
    r = np.random.default_rng(seed)
    return [r.standard_normal((n, d)) for _ in range(4)]


@pytest.mark.parametrize("lam", [0.0, 0.35, -0.4, 1.7])
def test_diff_forms_match_autograd_and_differences(lam):
    grid, tile, win = (3, 5, 6), (2, 4, 4), (1, 2, 1)
    n, d, scale = 90, 8, 0.7
    q, k, v, do = _head(3, n, d)
    mask = B.diff_mask(grid, tile, win)
    out, out2, lse, _, _ = B.diff_head(q, k, v, lam, mask, scale)
    leaf = [torch.from_numpy(x).requires_grad_(True) for x in (q, k, v)] + [torch.tensor(lam, dtype=torch.float64, requires_grad=True)]
    tm = torch.from_numpy(mask)
    p = [torch.softmax((scale * leaf[0][:, s] @ leaf[1][:, s].T).masked_fill(~tm, -torch.inf), 1) for s in
         (slice(0, 4), slice(4, 8))]
    o = (p[0] - leaf[3] * p[1]) @ leaf[2]
    assert np.allclose(o.detach().numpy(), out, atol=1e-12)
    assert np.allclose((p[1] @ leaf[2]).detach().numpy(), out2, atol=1e-12)
    got, _ = B.diff_head_backward(q, k, v, lam, do, mask, scale)
    want = torch.autograd.grad(o, leaf, torch.from_numpy(do))
    for a, b in zip(got, want):
        assert np.allclose(a, b.numpy(), atol=1e-11)
    # central differences of sum(out * do)
    r = np.random.default_rng(9)
    e = 1e-5
    for i, x in enumerate((q, k, v)):
        u = r.standard_normal(x.shape)
        args = [q, k, v]
        vals = []
        for s in (e, -e):
            args[i] = x + s * u
            vals.append((B.diff_head(*args, lam, mask, scale)[0] * do).sum())
        assert (vals[0] - vals[1]) / (2 * e) == pytest.approx((got[i] * u).sum(), rel=1e-6)
    vals = [(B.diff_head(q, k, v, lam + s, mask, scale)[0] * do).sum() for s in (e, -e)]
    assert (vals[0] - vals[1]) / (2 * e) == pytest.approx(got[3], rel=1e-6)


def test_diff_forms_reduce_to_the_oracle():
    """lambda = 0: the first map's attention; equal maps: (1 - lambda) times it."""
    grid, tile, win = (2, 6, 5), (2, 4, 4), (1, 1, 2)
    q, k, v, _ = _head(5, 60, 8)
    mask = B.diff_mask(grid, tile, win)
    first = O.masked_softmax_attention(q[:, :4], k[:, :4], v, mask, 0.6)
    assert np.allclose(B.diff_head(q, k, v, 0.0, mask, 0.6)[0], first, atol=1e-12)
    qq, kk = np.concatenate([q[:, :4]] * 2, 1), np.concatenate([k[:, :4]] * 2, 1)
    assert np.allclose(B.diff_head(qq, kk, v, 0.25, mask, 0.6)[0], 0.75 * first, atol=1e-12)


def test_layer_norm_forms_match_autograd():
    r = np.random.default_rng(1)
    h, dy, w, b = r.standard_normal((7, 13)) * 2 + 1, r.standard_normal((7, 13)), r.standard_normal(13), r.standard_normal(13)
    y, mean, rstd = B.layer_norm(h, w, b, 1e-3)
    t = [torch.from_numpy(x).requires_grad_(True) for x in (h, w, b)]
    o = torch.nn.functional.layer_norm(t[0], (13,), t[1], t[2], 1e-3)
    assert np.allclose(o.detach().numpy(), y, atol=1e-12)
    for a, g in zip(B.layer_norm_backward(dy, h, mean, rstd, w), torch.autograd.grad(o, t, torch.from_numpy(dy))):
        assert np.allclose(a, g.numpy(), atol=1e-11)
