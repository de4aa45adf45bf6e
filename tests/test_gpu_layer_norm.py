"""Layer norm with dropout and the residual add, its backward pass, and dropout
on the GPU, against the formulas in 64 bits (needs a GB300)."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api

import residual_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def placed(t, order):
    """The values in memory order: packed rows, rows of a wider buffer on
    16-byte boundaries, rows that start one element past one with an odd stride,
    or one row for all."""
    rows, cols = t.shape
    if order == "packed":
        return t
    if order == "same":
        return t[:1].expand(rows, cols)
    width, at = ((cols + 7) // 8 * 8 + 16, 8) if order == "view" else ((cols + 4) | 1, 1)
    buf = torch.full((rows, width), float("nan"), dtype=t.dtype, device=DEV)
    buf[:, at:at + cols] = t
    return buf[:, at:at + cols]


def values(g, rows, cols, dtype, order="packed", offset=0.3):
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x = x * torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV)) + offset * torch.randn(cols, generator=g, device=DEV)
    return placed(x.to(dtype), order)


class Framed:
    """An output inside a larger buffer of sevens: what lies around it stays."""

    def __init__(self, rows, cols, dtype, odd):
        self.at, width = (3, (cols + 10) | 1) if odd else (8, (cols + 7) // 8 * 8 + 16)
        self.buf = torch.full((rows + 2, width), 7.0, dtype=dtype, device=DEV)
        self.t = self.buf[1:1 + rows, self.at:self.at + cols]

    def kept(self):
        rows, cols = self.t.shape
        left = self.buf.clone()
        left[1:1 + rows, self.at:self.at + cols] = 7.0
        assert bool((left == 7.0).all()), "written outside the output"


def vector(g, n, mean=0.0, std=0.1):
    return mean + std * torch.randn(n, generator=g, device=DEV)


# Widths on both sides of every change of kernel, of a team's lanes and of the
# 8 columns of a group; more rows than a launch has teams; one row.
SIZES = [(1, 1), (5, 2), (3, 7), (37, 8), (70, 9), (20001, 16), (33, 40), (513, 255), (9001, 256), (7, 257), (3000, 504),
         (41, 512), (6, 513), (2001, 1000), (5, 1024), (9, 1025), (700, 2048), (5, 2049), (1, 4096), (1300, 4096),
         (3, 4097), (11, 8192), (310, 8193), (5, 14336), (312, 16384), (3, 16385), (4, 20011)]
ORDERS = ["packed", "view", "odd"]


def forms(cases):
    """Each size with a type, order and options that change from one to the next."""
    out = []
    for i, (rows, cols) in enumerate(cases):
        for dtype in (BF, F32):
            j = i + (dtype is F32)
            out.append((rows, cols, dtype, ORDERS[j % 3], (i // 2 + j) % 2 == 0, (0.0, 0.1, 0.5)[(i + 2 * j) % 3]))
    return out


# The widest rows a team holds, by words: the most shared memory a block takes.
CASES = forms(SIZES) + [(40, 16383, dtype, "odd", True, 0.1) for dtype in (BF, F32)]
IDS = lambda c: "%dx%d-%s-%s-%s-p%g" % (c[0], c[1], str(c[2])[6:], c[3], "res" if c[4] else "x", c[5])  # noqa: E731


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_layer_norm(case):
    rows, cols, dtype, order, has_residual, p = case
    g = gen(rows * 31 + cols)
    x = values(g, rows, cols, dtype, order)
    residual = values(g, rows, cols, dtype, "same" if order == "view" else order) if has_residual else None
    w, b = (vector(g, cols, 1.0), vector(g, cols)) if cols % 3 else (None, None)
    rng = api.Dropout(p, seed=2 ** 63 + cols, step=2 ** 32 + rows, device=DEV) if p else None
    summed = has_residual or p > 0
    out, total = Framed(rows, cols, dtype, order == "odd"), Framed(rows, cols, dtype, order == "odd")
    mean, rstd = torch.full((rows + 1,), 7.0, device=DEV), torch.full((rows + 1,), 7.0, device=DEV)
    api.layer_norm(x, weight=w, bias=b, eps=1e-5, out=out.t, residual=residual, dropout=rng, site=cols,
                   sum_out=total.t if summed else None, mean=mean[:rows], rstd=rstd[:rows])
    mask = R.Mask(rng, rows, cols, cols)
    h, dh = R.summed(x, residual, mask)
    want = R.norm(h, dh, w, b, 1e-5)
    R.close(out.t, *want["y"], dtype, "y")
    R.close(mean[:rows], *want["mean"], F32, "mean")
    R.close(rstd[:rows], *want["rstd"], F32, "rstd")
    if summed:
        R.close(total.t, h, dh, dtype, "sum")
    else:
        assert bool((total.t == 7.0).all())
    out.kept(), total.kept()
    assert float(mean[rows]) == 7.0 and float(rstd[rows]) == 7.0


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_layer_norm_backward(case):
    rows, cols, dtype, order, has_add, p = case
    g = gen(rows * 37 + cols)
    x, dy = values(g, rows, cols, dtype, order), values(g, rows, cols, dtype, order, 0.0)
    add = values(g, rows, cols, dtype, "same" if order == "view" else order, 0.0) if has_add else None
    w = vector(g, cols, 1.0) if cols % 3 else None
    x64 = x.double()
    mean, rstd = x64.mean(1).float(), (x64.var(1, unbiased=False) + 1e-5).rsqrt().float()
    rng = api.Dropout(p, seed=cols, step=rows, device=DEV) if p else None
    dx, dr = Framed(rows, cols, dtype, order == "odd"), Framed(rows, cols, dtype, order == "odd")
    dw, db = torch.full((cols,), 7.0, device=DEV), torch.full((cols,), 7.0, device=DEV)
    ws = torch.full((api.layer_norm_workspace(cols) // 4,), float("nan"), device=DEV)
    api.layer_norm_backward(dy, x, mean, rstd, weight=w, dx=dx.t, dw=dw, db=db, add=add, dropout=rng, site=5,
                            d_residual=dr.t if p else None, workspace=ws)
    want = R.norm_backward(dy, x, mean, rstd, w, add, R.Mask(rng, rows, cols, 5))
    R.close(dx.t, *want["dx"], dtype, "dx")
    if p:
        R.close(dr.t, *want["d_residual"], dtype, "d_residual")
    R.close(dw, *want["dw"], F32, "dw")
    R.close(db, *want["db"], F32, "db")
    dx.kept(), dr.kept()


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_dropout(case):
    rows, cols, dtype, order, has_residual, p = case
    g = gen(rows * 41 + cols)
    x = values(g, rows, cols, dtype, order)
    residual = values(g, rows, cols, dtype, "same" if order == "view" else order) if has_residual else None
    rng = api.Dropout(p, seed=cols, step=rows, device=DEV)
    out = Framed(rows, cols, dtype, order == "odd")
    api.dropout(x, rng, out=out.t, residual=residual, site=2 ** 32 - 1)
    mask = R.Mask(rng, rows, cols, 2 ** 32 - 1)
    R.close(out.t, *R.summed(x, residual, mask), dtype, "dropout")
    if residual is None:  # the very elements, not near ones
        assert bool((out.t.cpu() != 0)[wide_nonzero(x)].eq(mask.keep[wide_nonzero(x)]).all())
    out.kept()


def wide_nonzero(x):
    return x.cpu() != 0


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("rows,cols", [(4, 40), (3, 600), (2, 4096), (2, 16392)])
def test_everything_dropped(rows, cols, backward):
    """p = 1 leaves rows of zeros (variance 0) or the residual alone, and no gradient; NaN and infinity are
    dropped as any value."""
    g = gen(rows)
    rng = api.Dropout(1.0, device=DEV)
    x = torch.full((rows, cols), float("nan"), device=DEV)
    x[0] = float("inf")
    w, b = vector(g, cols, 1.0), vector(g, cols)
    out, total = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    api.layer_norm(x, weight=w, bias=b, eps=0.25, out=out, dropout=rng, sum_out=total, mean=mean, rstd=rstd)
    assert torch.equal(out, b.expand(rows, cols)) and not total.any() and not mean.any() and bool((rstd == 2.0).all())
    residual = values(g, rows, cols, F32)
    api.layer_norm(x, weight=w, bias=b, eps=0.25, out=out, residual=residual, dropout=rng, sum_out=total)
    assert torch.equal(total, residual)
    R.close(out, *R.norm(R.wide(residual), torch.zeros(rows, cols).double(), w, b, 0.25)["y"], F32, "y")
    if backward:
        dx, dr = torch.empty_like(x), torch.empty_like(x)
        api.layer_norm_backward(residual, out, mean, rstd, weight=w, dx=dx, d_residual=dr, dropout=rng)
        assert not dx.any() and bool(dr.any())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [24, 700, 4096, 16400])
def test_what_is_dropped_does_not_matter(cols, dtype):
    """NaN and infinities where the mask drops, and rows that hold one where it keeps."""
    rows = 6
    g = gen(cols)
    rng = api.Dropout(0.5, seed=3, device=DEV)
    keep = R.Mask(rng, rows, cols).keep.to(DEV)
    clean = values(g, rows, cols, dtype)
    x = torch.where(keep, clean, torch.full_like(clean, float("nan")))
    x[1] = torch.where(keep[1], clean[1], torch.full_like(clean[1], float("-inf")))
    outs = []
    for t in (clean, x):
        out, total, mean, rstd = torch.empty_like(t), torch.empty_like(t), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        api.layer_norm(t, out=out, dropout=rng, sum_out=total, mean=mean, rstd=rstd)
        plain = torch.empty_like(t)
        api.dropout(t, rng, out=plain)
        assert torch.equal(plain, total)
        outs.append((out, total, mean, rstd))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    # kept: its row is NaN, the others are as before
    for bad in (float("nan"), float("inf")):
        y = clean.clone()
        y[2, int(keep[2].nonzero()[0])] = bad
        out, rstd = torch.empty_like(y), torch.empty(rows, device=DEV)
        api.layer_norm(y, out=out, dropout=rng, rstd=rstd)
        assert bool(out[2].isnan().all()) and bool(rstd[2].isnan())
        rest = [0, 1, 3, 4, 5]
        assert torch.equal(out[rest], outs[0][0][rest]) and torch.equal(rstd[rest], outs[0][3][rest])


@pytest.mark.parametrize("cols", [8, 640, 4096, 8192, 16400])
def test_far_from_zero(cols):
    """Rows whose mean is a thousand times their spread and more, one value repeated, and tiny values."""
    g = gen(cols)
    x = torch.randn(5, cols, generator=g, device=DEV) + torch.tensor([1000.0, -3e4, 0.0, 0.0, 0.0], device=DEV)[:, None]
    x[2] = 0.1
    x[3] = 1e-30 * x[3]
    out, mean, rstd = torch.empty_like(x), torch.empty(5, device=DEV), torch.empty(5, device=DEV)
    api.layer_norm(x, eps=1e-5, out=out, mean=mean, rstd=rstd)
    h = R.wide(x)
    want = R.norm(h, torch.zeros_like(h), None, None, 1e-5)
    for t, name in ((out, "y"), (mean, "mean"), (rstd, "rstd")):
        R.close(t, *want[name], F32, name)


@pytest.mark.parametrize("cols", [40, 1000, 4096, 16400])
def test_weights_that_start_anywhere(cols):
    """Weights one value past an aligned address."""
    g, rows = gen(cols), 700
    x, dy = values(g, rows, cols, BF), values(g, rows, cols, BF)
    w, b = (torch.cat([v[:1], v])[1:] for v in (vector(g, cols, 1.0), vector(g, cols)))
    assert w.data_ptr() % 16 and b.data_ptr() % 16
    ws = torch.empty(api.layer_norm_workspace(cols), dtype=torch.uint8, device=DEV)
    out, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    api.layer_norm(x, weight=w, bias=b, out=out, mean=mean, rstd=rstd)
    api.layer_norm_backward(dy, x, mean, rstd, weight=w, dx=dx, dw=dw, db=db, workspace=ws)
    mask = R.Mask(None, rows, cols)
    R.close(out, *R.norm(R.wide(x), torch.zeros(rows, cols).double(), w, b, 1e-5)["y"], BF, "y")
    want = R.norm_backward(dy, x, mean, rstd, w, None, mask)
    R.close(dx, *want["dx"], BF, "dx")
    R.close(dw, *want["dw"], F32, "dw")
    R.close(db, *want["db"], F32, "db")


def all_outputs(rows, cols, dtype, g):
    x, residual, dy, add = (values(g, rows, cols, dtype) for _ in range(4))
    w, b = vector(g, cols, 1.0), vector(g, cols)
    rng = api.Dropout(0.1, seed=11, device=DEV)
    ws = torch.empty(api.layer_norm_workspace(cols), dtype=torch.uint8, device=DEV)

    def run(out, total, dx, dr, stream=None):
        mean, rstd, dw, db = (torch.empty(n, device=DEV) for n in (rows, rows, cols, cols))
        api.layer_norm(x, weight=w, bias=b, out=out, residual=residual, dropout=rng, site=1, sum_out=total, mean=mean,
                       rstd=rstd, stream=stream)
        api.layer_norm_backward(dy, total, mean, rstd, weight=w, dx=dx, dw=dw, db=db, add=add, dropout=rng, site=1,
                                d_residual=dr, workspace=ws, stream=stream)
        return out, total, mean, rstd, dx, dr, dw, db

    return run, (x, residual, dy, add), rng


@pytest.mark.parametrize("rows,cols,dtype", [(300, 200, BF), (2500, 4096, BF), (50, 1000, F32), (20, 16392, BF),
                                             (3001, 17, F32), (300, 253, BF), (400, 1001, F32), (700, 4095, BF),
                                             (9, 16383, F32), (20, 16389, BF)])
def test_same_bits_every_time_in_place_and_on_a_stream(rows, cols, dtype):
    run, (x, residual, dy, add), _ = all_outputs(rows, cols, dtype, gen(5))
    fresh = lambda: [torch.empty_like(x) for _ in range(4)]  # noqa: E731
    first = run(*fresh())
    again = run(*fresh())
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    third = run(*fresh(), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, third))
    # y over x, the sum over the residual, dx over dy, the residual's gradient over `add`
    placed_ = run(x, residual, dy, add)
    assert all(torch.equal(a, b) for a, b in zip(first, placed_))


@pytest.mark.parametrize("rows,cols,dtype", [(64, 200, BF), (900, 4096, BF), (333, 1001, F32), (7, 16392, F32)])
def test_two_at_once(rows, cols, dtype):
    """Forward and backward passes on two streams, each with a workspace of its own, and a third on the caller's."""
    runs = [all_outputs(rows, cols, dtype, gen(seed)) for seed in (21, 22, 23)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), None]
    fresh = lambda x: [torch.empty_like(x) for _ in range(4)]  # noqa: E731
    want = [run(*fresh(x)) for run, (x, *_), _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(*fresh(x), stream=s) for (run, (x, *_), _), s in zip(runs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


def test_captured_and_replayed():
    """A graph of forward and backward whose step counts on: each replay has its own mask, the eager call's."""
    rows, cols = 70, 1032
    run, (x, *_), rng = all_outputs(rows, cols, BF, gen(6))
    bufs = [torch.empty_like(x) for _ in range(4)]
    rng.step[0] = 5
    want = []
    for _ in range(3):
        want.append([t.clone() for t in run(*bufs)])
        rng.advance()
    assert not torch.equal(want[0][1], want[1][1])
    rng.step[0] = 5
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = run(*bufs)
        rng.advance()
    assert int(rng.step) == 5
    for step in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want[step])), step
    assert int(rng.step) == 8


def test_first_call_inside_a_capture():
    """No kernel's first call needs anything that a capture forbids: sizes no other test uses."""
    cols = 6152
    x = values(gen(1), 9, cols, F32)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, dw = (torch.empty(n, device=DEV) for n in (9, 9, cols))
    ws = torch.empty(api.layer_norm_workspace(cols), dtype=torch.uint8, device=DEV)
    rng = api.Dropout(0.3, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.layer_norm(x, out=out, mean=mean, rstd=rstd, dropout=rng)
        api.layer_norm_backward(out, x, mean, rstd, dx=dx, dw=dw, workspace=ws)
    graph.replay()
    h, dh = R.summed(x, None, R.Mask(rng, 9, cols))
    R.close(out, *R.norm(h, dh, None, None, 1e-5)["y"], F32, "y")


@pytest.mark.parametrize("rows,cols", [(0, 64), (0, 5000), (4, 64)])
def test_nothing_to_do(rows, cols):
    """No rows: the weights' gradients are zero; no output wanted: nothing happens."""
    x = torch.empty(rows, cols, device=DEV, dtype=BF)
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    dw, db = torch.full((cols,), 7.0, device=DEV), torch.full((cols,), 7.0, device=DEV)
    if rows == 0:
        api.layer_norm(x, out=x, mean=mean, rstd=rstd)
        api.dropout(x, api.Dropout(0.5, device=DEV), out=x)
        api.layer_norm_backward(x, x, mean, rstd, dx=x, dw=dw, db=db)
        assert not dw.any() and not db.any()
    else:
        api.layer_norm_backward(x, x, mean, rstd)


@pytest.mark.parametrize("cols", [64, 1000, 4096, 16392])
@pytest.mark.parametrize("wanted", ["dx", "dr", "dw", "db", "dw db", "dx db"])
def test_backward_outputs_left_out(cols, wanted):
    """Each output is the same whichever of the others are asked for."""
    rows = 33
    run, (x, _, dy, add), rng = all_outputs(rows, cols, BF, gen(7))
    full = run(*[torch.empty_like(x) for _ in range(4)])
    total, mean, rstd = full[1], full[2], full[3]
    w = vector(gen(8), cols, 1.0)
    ws = torch.empty(api.layer_norm_workspace(cols), dtype=torch.uint8, device=DEV)

    def call(names):
        made = {n: torch.empty_like(x) if n in ("dx", "dr") else torch.empty(cols, device=DEV) for n in names}
        api.layer_norm_backward(dy, total, mean, rstd, weight=w, dx=made.get("dx"), d_residual=made.get("dr"),
                                dw=made.get("dw"), db=made.get("db"), add=add, dropout=rng, site=1,
                                workspace=ws if "dw" in made or "db" in made else None)
        return made

    everything, some = call(["dx", "dr", "dw", "db"]), call(wanted.split())
    assert all(torch.equal(everything[n], t) for n, t in some.items())


def test_shapes_of_more_dimensions():
    g = gen(9)
    flat = values(g, 30, 136, BF)
    x = flat.view(2, 3, 5, 136)
    out, want = torch.empty_like(x), torch.empty_like(flat)
    rng = api.Dropout(0.2, device=DEV)
    api.layer_norm(flat, out=want, dropout=rng)
    api.layer_norm(x, out=out, dropout=rng, mean=torch.empty(2, 3, 5, device=DEV))
    assert torch.equal(out.view(30, 136), want)
    one = flat[0]
    got = torch.empty_like(one)
    api.layer_norm(one, out=got, dropout=rng)
    assert torch.equal(got, want[0])
    # part of each row: the leading dimensions are still evenly spaced
    wide = torch.zeros(2, 3, 5, 200, device=DEV, dtype=BF)
    wide[..., 8:144] = x
    api.layer_norm(wide[..., 8:144], out=out, dropout=rng)
    assert torch.equal(out.view(30, 136), want)


@pytest.mark.parametrize("cols", [104, 4096, 16392])
def test_rows_past_32_bits(cols):
    """Row strides that take elements past 2^32."""
    rows, ld = 3, 2 ** 31 + 8
    buf = torch.empty((rows - 1) * ld + cols, dtype=BF, device=DEV)
    far = buf.as_strided((rows, cols), (ld, 1))
    x = values(gen(3), rows, cols, BF)
    far.copy_(x)
    rng = api.Dropout(0.5, device=DEV)
    out, dropped = torch.empty_like(x), torch.empty_like(x)
    api.layer_norm(x, out=out, dropout=rng)
    api.dropout(x, rng, out=dropped)
    api.layer_norm(far, out=far, dropout=rng)
    assert torch.equal(far, out)
    far.copy_(x)
    api.dropout(far, rng, out=far)
    assert torch.equal(far, dropped)
    mean, rstd = x.float().mean(1), x.float().var(1, unbiased=False).rsqrt()
    dx = torch.empty_like(x)
    api.layer_norm_backward(out, x, mean, rstd, dx=dx)
    far.copy_(out)
    api.layer_norm_backward(far, x, mean, rstd, dx=far)
    assert torch.equal(far, dx)


def test_gradient_against_differences():
    """The kernels' dx, d_residual, dw and db along random directions, against central differences of the
    formula in 64 bits."""
    rows, cols = 7, 120
    g = gen(10)
    x, residual, dy = (values(g, rows, cols, F32) for _ in range(3))
    w, b = vector(g, cols, 1.0), vector(g, cols)
    rng = api.Dropout(0.3, seed=5, device=DEV)
    out, total = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, dw, db = (torch.empty(n, device=DEV) for n in (rows, rows, cols, cols))
    api.layer_norm(x, weight=w, bias=b, out=out, residual=residual, dropout=rng, sum_out=total, mean=mean, rstd=rstd)
    dx, dr = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(api.layer_norm_workspace(cols), dtype=torch.uint8, device=DEV)
    api.layer_norm_backward(dy, total, mean, rstd, weight=w, dx=dx, d_residual=dr, dw=dw, db=db, dropout=rng, workspace=ws)
    mask = R.Mask(rng, rows, cols)
    args = [R.wide(x), R.wide(residual), w.cpu().double(), b.cpu().double()]

    def loss(x_, r_, w_, b_):
        h = mask(x_) + r_
        c = h - h.mean(1, keepdim=True)
        return float(((c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * w_ + b_) * R.wide(dy)).sum())

    cpu = torch.Generator().manual_seed(1)
    for i, grad in enumerate((dx, dr, dw, db)):
        v = torch.randn(args[i].shape, generator=cpu, dtype=torch.float64)
        e = 1e-5
        moved = [list(args), list(args)]
        moved[0][i], moved[1][i] = args[i] + e * v, args[i] - e * v
        difference = (loss(*moved[0]) - loss(*moved[1])) / (2 * e)
        along = float((grad.cpu().double() * v).sum())
        # third derivatives: e^2 times a few; rounding of the loss: 1e-16 |loss| / e; the kernel's fp32
        size = float((grad.cpu().double() * v).abs().sum())
        assert abs(along - difference) <= 1e-5 * size + 1e-6, (i, along, difference)
