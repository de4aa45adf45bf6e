"""Layer norm, its backward pass and dropout over every combination of type,
memory order, residual and probability at the widths of each kernel, with weights,
against the formulas in 64 bits; and sums of dw and db that have no rounding (needs
a GB300)."""
import itertools

import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api

import residual_ref as R
from test_gpu_layer_norm import BF, DEV, F32, Framed, gen, values, vector

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


# Lanes of a warp, warps that hold a row, rows read again; widths on and off a
# warp's columns, of one piece count and the next.
NARROW, HELD, LONG = (9, 40, 253, 256), (600, 768, 1000, 1280, 1800, 3000, 4095, 4096, 5000, 8200, 12300, 16384), (16392,)
SMALL = [(310 if (p == 0.1) != residual else 37, cols, dtype, order, residual, p)
         for cols, dtype, order, residual, p in itertools.product(NARROW + HELD + LONG, (BF, F32), ("packed", "odd"),
                                                                  (False, True), (0.0, 0.1, 0.5))]
# More rows than 16 to an SM, which stage the weights and share a block among
# several teams; a number of them that leaves every block's last round part empty.
ROWS = 2437
MANY = [(ROWS, cols, dtype, order, residual, p)
        for cols in (504, 600, 768, 1000, 1024, 1280, 2048, 3000, 4000, 4096) for dtype in (BF, F32)
        for order, residual, p in (("packed", True, 0.1), ("packed", False, 0.0), ("view", True, 0.0), ("view", False, 0.1))]
MANY += [(ROWS, cols, dtype, "odd", residual, p) for cols in (600, 1003, 4096) for dtype in (BF, F32)
         for residual, p in ((True, 0.1), (False, 0.0), (True, 0.0))]
MANY += [(20001, cols, dtype, "packed", True, p) for cols in (16, 64, 200) for dtype in (BF, F32) for p in (0.0, 0.1)]
MANY += [(ROWS, cols, BF, "packed", residual, 0.1) for cols in (2304, 2560, 2816) for residual in (False, True)]
# more than 64 rows to an SM: a team fewer to a block where `add` is read too
MANY += [(9800, cols, BF, "packed", True, p) for cols in (3040, 4088, 4096) for p in (0.0, 0.1)]
MANY += [(700, cols, BF, "packed", True, 0.1) for cols in (8192, 14336, 16392)]
CASES = SMALL + MANY
IDS = lambda c: "%dx%d-%s-%s-%s-p%g" % (c[0], c[1], str(c[2])[6:], c[3], "res" if c[4] else "x", c[5])  # noqa: E731


def same(order, residual):
    """The residual's order: one row for all beside rows of a wider buffer."""
    return "same" if order == "view" and residual else order


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_layer_norm(case):
    rows, cols, dtype, order, has_residual, p = case
    g = gen(rows + 7 * cols)
    x = values(g, rows, cols, dtype, order)
    residual = values(g, rows, cols, dtype, same(order, True)) if has_residual else None
    w, b = vector(g, cols, 1.0), vector(g, cols)
    rng = api.Dropout(p, seed=cols, step=rows, device=DEV) if p else None
    summed = has_residual or p > 0
    odd = order == "odd"
    out, total = Framed(rows, cols, dtype, odd), Framed(rows, cols, dtype, odd)
    mean, rstd = torch.full((rows + 1,), 7.0, device=DEV), torch.full((rows + 1,), 7.0, device=DEV)
    api.layer_norm(x, weight=w, bias=b, eps=1e-5, out=out.t, residual=residual, dropout=rng, site=1,
                   sum_out=total.t if summed else None, mean=mean[:rows], rstd=rstd[:rows])
    h, dh = R.summed(x, residual, R.Mask(rng, rows, cols, 1))
    want = R.norm(h, dh, w, b, 1e-5)
    R.close(out.t, *want["y"], dtype, "y")
    R.close(mean[:rows], *want["mean"], F32, "mean")
    R.close(rstd[:rows], *want["rstd"], F32, "rstd")
    if summed:
        R.close(total.t, h, dh, dtype, "sum")
    out.kept(), total.kept()
    assert float(mean[rows]) == 7.0 and float(rstd[rows]) == 7.0


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_layer_norm_backward(case):
    rows, cols, dtype, order, has_add, p = case
    g = gen(rows + 11 * cols)
    x, dy = values(g, rows, cols, dtype, order), values(g, rows, cols, dtype, order, 0.0)
    add = values(g, rows, cols, dtype, same(order, True), 0.0) if has_add else None
    w = vector(g, cols, 1.0)
    x64 = x.double()
    mean, rstd = x64.mean(1).float(), (x64.var(1, unbiased=False) + 1e-5).rsqrt().float()
    rng = api.Dropout(p, seed=cols, step=rows, device=DEV) if p else None
    odd = order == "odd"
    dx, dr = Framed(rows, cols, dtype, odd), Framed(rows, cols, dtype, odd)
    dw, db = torch.full((cols + 1,), 7.0, device=DEV), torch.full((cols + 1,), 7.0, device=DEV)
    ws = torch.full((api.layer_norm_workspace(cols) // 4,), float("nan"), device=DEV)
    api.layer_norm_backward(dy, x, mean, rstd, weight=w, dx=dx.t, dw=dw[:cols], db=db[:cols], add=add, dropout=rng,
                            site=5, d_residual=dr.t if p else None, workspace=ws)
    want = R.norm_backward(dy, x, mean, rstd, w, add, R.Mask(rng, rows, cols, 5))
    R.close(dx.t, *want["dx"], dtype, "dx")
    if p:
        R.close(dr.t, *want["d_residual"], dtype, "d_residual")
    R.close(dw[:cols], *want["dw"], F32, "dw")
    R.close(db[:cols], *want["db"], F32, "db")
    dx.kept(), dr.kept()
    assert float(dw[cols]) == 7.0 and float(db[cols]) == 7.0


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_dropout(case):
    rows, cols, dtype, order, has_residual, p = case
    g = gen(rows + 13 * cols)
    x = values(g, rows, cols, dtype, order)
    residual = values(g, rows, cols, dtype, same(order, True)) if has_residual else None
    rng = api.Dropout(p, seed=cols, step=rows, device=DEV)
    out = Framed(rows, cols, dtype, order == "odd")
    api.dropout(x, rng, out=out.t, residual=residual, site=2 ** 32 - 1)
    mask = R.Mask(rng, rows, cols, 2 ** 32 - 1)
    R.close(out.t, *R.summed(x, residual, mask), dtype, "dropout")
    if residual is None:  # the very elements, not near ones
        nonzero = x.cpu() != 0
        assert bool((out.t.cpu() != 0).eq(mask.keep)[nonzero].all())
    out.kept()


# ---------------------------------------------------------------- sums without rounding

# One row and every number around a round of one and two blocks to each of 152
# SMs, of 16 rows to an SM, of a block's teams and of the rows a team takes at once.
COUNTS = [1, 2, 151, 152, 153, 303, 304, 305, 306, 455, 608, 609, 1217, 2431, 2432, 2433, 4865, 9001]


@pytest.mark.parametrize("order", ["packed", "odd"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", [8, 40, 256, 300, 768, 1000, 1032, 1280, 3000, 4096, 6152, 8200, 14336, 16392])
def test_every_row_counts_once(cols, dtype, order):
    """dw and db of integers over powers of two, with mean 0 and rstd 1 given: every product is a multiple of 1/32 of
    at most 3/16, and 9001 of them add up to less than 2^16 / 32, so all partial sums are exact in fp32's 24 bits in
    any order.  A row left out or taken twice changes the result."""
    g = gen(cols)
    most = COUNTS[-1] if cols <= 4096 else 2433
    ints = lambda lo, hi, by: (torch.randint(lo, hi + 1, (most, cols), generator=g, device=DEV) / by).to(dtype)  # noqa: E731
    dy, x = ints(-3, 3, 4), ints(-2, 2, 8)
    if order == "odd":
        framed = [Framed(most, cols, dtype, True) for _ in range(2)]
        for f, t in zip(framed, (dy, x)):
            f.t.copy_(t)
        dy, x = (f.t for f in framed)
    mean, rstd = torch.zeros(most, device=DEV), torch.ones(most, device=DEV)
    w = vector(g, cols, 1.0)
    rng = api.Dropout(0.1, device=DEV)
    ws = torch.full((api.layer_norm_workspace(cols) // 4,), float("nan"), device=DEV)
    for rows in [n for n in COUNTS if n <= most]:
        a, b = dy[:rows], x[:rows]
        want = (a.double() * b.double()).sum(0).float(), a.double().sum(0).float()
        dx = torch.empty(rows, cols, dtype=dtype, device=DEV)
        for options in (dict(dx=dx), dict(dx=dx, dropout=rng, add=a), {}):
            dw, db = torch.full((cols,), 7.0, device=DEV), torch.full((cols,), 7.0, device=DEV)
            api.layer_norm_backward(a, b, mean[:rows], rstd[:rows], weight=w, dw=dw, db=db, workspace=ws, **options)
            assert torch.equal(dw, want[0]) and torch.equal(db, want[1]), (rows, sorted(options))


# ---------------------------------------------------------------- weights and orders of their own

@pytest.mark.parametrize("given", ["w", "b"])
@pytest.mark.parametrize("rows,cols", [(37, 40), (37, 1000), (ROWS, 1000), (ROWS, 4096), (3, 16392)])
def test_one_of_weight_and_bias(rows, cols, given):
    g = gen(cols)
    x, dy = values(g, rows, cols, BF), values(g, rows, cols, BF, offset=0.0)
    w, b = (vector(g, cols, 1.0), None) if given == "w" else (None, vector(g, cols))
    out, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    api.layer_norm(x, weight=w, bias=b, out=out, mean=mean, rstd=rstd)
    api.layer_norm_backward(dy, x, mean, rstd, weight=w, dx=dx)
    R.close(out, *R.norm(R.wide(x), torch.zeros(rows, cols).double(), w, b, 1e-5)["y"], BF, "y")
    R.close(dx, *R.norm_backward(dy, x, mean, rstd, w, None, R.Mask(None, rows, cols))["dx"], BF, "dx")


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("rows,cols", [(37, 40), (37, 1000), (ROWS, 1000), (ROWS, 4096), (3, 16392)])
def test_weights_that_start_anywhere(rows, cols, p):
    """Weights one value past an aligned address, beside rows that are on one."""
    g = gen(cols)
    x, dy = values(g, rows, cols, BF), values(g, rows, cols, BF, offset=0.0)
    w, b = (torch.cat([v[:1], v])[1:] for v in (vector(g, cols, 1.0), vector(g, cols)))
    assert w.data_ptr() % 16 and b.data_ptr() % 16
    rng = api.Dropout(p, seed=4, device=DEV) if p else None
    mask = R.Mask(rng, rows, cols)
    out, total, dx = torch.empty_like(x), torch.empty_like(x) if p else None, torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    api.layer_norm(x, weight=w, bias=b, out=out, dropout=rng, sum_out=total, mean=mean, rstd=rstd)
    h = total if p else x
    api.layer_norm_backward(dy, h, mean, rstd, weight=w, dx=dx, dw=dw, db=db, dropout=rng,
                            workspace=torch.empty(api.layer_norm_workspace(cols), dtype=torch.uint8, device=DEV))
    R.close(out, *R.norm(*R.summed(x, None, mask), w, b, 1e-5)["y"], BF, "y")
    want = R.norm_backward(dy, h, mean, rstd, w, None, mask)
    for t, name, dtype in ((dx, "dx", BF), (dw, "dw", F32), (db, "db", F32)):
        R.close(t, *want[name], dtype, name)


@pytest.mark.parametrize("which", ["x", "residual", "out", "sum"])
@pytest.mark.parametrize("cols", [200, 1000, 4096, 16392])
def test_one_tensor_that_starts_anywhere(cols, which):
    """The others are on 16 bytes."""
    rows = 311
    g = gen(cols)
    order = lambda name: "odd" if name == which else "packed"  # noqa: E731
    x, residual = values(g, rows, cols, BF, order("x")), values(g, rows, cols, BF, order("residual"))
    w, b = vector(g, cols, 1.0), vector(g, cols)
    rng = api.Dropout(0.1, seed=6, device=DEV)
    out, total = Framed(rows, cols, BF, which == "out"), Framed(rows, cols, BF, which == "sum")
    api.layer_norm(x, weight=w, bias=b, out=out.t, residual=residual, dropout=rng, sum_out=total.t)
    h, dh = R.summed(x, residual, R.Mask(rng, rows, cols))
    R.close(out.t, *R.norm(h, dh, w, b, 1e-5)["y"], BF, "y")
    R.close(total.t, h, dh, BF, "sum")
    dropped = Framed(rows, cols, BF, which == "out")
    api.dropout(x, rng, out=dropped.t, residual=residual)
    R.close(dropped.t, h, dh, BF, "dropout")
    out.kept(), total.kept(), dropped.kept()


@pytest.mark.parametrize("cols", [16, 300, 4096, 16392])
def test_one_row_for_all(cols):
    """Expanded inputs: row stride 0."""
    rows = 400
    g = gen(cols)
    x, dy, add = (values(g, 1, cols, BF).expand(rows, cols) for _ in range(3))
    w, b = vector(g, cols, 1.0), vector(g, cols)
    rng = api.Dropout(0.1, seed=8, device=DEV)
    out, total, dx, dr = (torch.empty(rows, cols, dtype=BF, device=DEV) for _ in range(4))
    mean, rstd, dw, db = (torch.empty(n, device=DEV) for n in (rows, rows, cols, cols))
    ws = torch.empty(api.layer_norm_workspace(cols), dtype=torch.uint8, device=DEV)
    api.layer_norm(x, weight=w, bias=b, out=out, dropout=rng, sum_out=total, mean=mean, rstd=rstd)
    mask = R.Mask(rng, rows, cols)
    h, dh = R.summed(x, None, mask)
    R.close(out, *R.norm(h, dh, w, b, 1e-5)["y"], BF, "y")
    api.layer_norm_backward(dy, total, mean, rstd, weight=w, dx=dx, d_residual=dr, dw=dw, db=db, add=add, dropout=rng,
                            workspace=ws)
    want = R.norm_backward(dy, total, mean, rstd, w, add, mask)
    for t, name, dtype in ((dx, "dx", BF), (dr, "d_residual", BF), (dw, "dw", F32), (db, "db", F32)):
        R.close(t, *want[name], dtype, name)


@pytest.mark.parametrize("cols", [64, 1000, 4096, 16392])
@pytest.mark.parametrize("wanted", ["dx", "dr", "dw", "db", "dx db"])
def test_backward_outputs_left_out_of_many_rows(cols, wanted):
    """Each output is right whichever of the others are asked for."""
    rows = ROWS if cols <= 4096 else 307
    g = gen(cols)
    x, dy, add = (values(g, rows, cols, BF, offset=0.0) for _ in range(3))
    w = vector(g, cols, 1.0)
    rng = api.Dropout(0.1, device=DEV)
    mean, rstd = x.double().mean(1).float(), (x.double().var(1, unbiased=False) + 1e-5).rsqrt().float()
    ws = torch.empty(api.layer_norm_workspace(cols), dtype=torch.uint8, device=DEV)
    made = {n: torch.empty_like(x) if n in ("dx", "dr") else torch.empty(cols, device=DEV) for n in wanted.split()}
    api.layer_norm_backward(dy, x, mean, rstd, weight=w, dx=made.get("dx"), d_residual=made.get("dr"), dw=made.get("dw"),
                            db=made.get("db"), add=add, dropout=rng, site=1,
                            workspace=ws if "dw" in made or "db" in made else None)
    want = R.norm_backward(dy, x, mean, rstd, w, add, R.Mask(rng, rows, cols, 1))
    for name, t in made.items():
        R.close(t, *want["d_residual" if name == "dr" else name], BF if name in ("dx", "dr") else F32, name)
