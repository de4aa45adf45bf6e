"""Cases of the operators on the residual stream between a block's GEMMs: layer
norm with the dropout and residual add in front of it in the same pass, its
backward pass with the weight's and bias's gradients, dropout with a mask that
is drawn anew from a counter wherever it is needed, and projections that apply
it to their output tile.

``own`` false: plain torch formulas in fp32 (long sums in fp64).  ``own`` true:
the package's entry points on the same inputs.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one generated token: launch latency
        dict(name="norm_one_token", op="norm", rows=1, cols=4096, type="bf16", order="packed", residual=False, p=0.0,
             sums=False, stats=False),
        # a decode step of 64 sequences: the block's output added to the residual stream and normalised
        dict(name="norm_add_decode_64", op="norm", rows=64, cols=4096, type="bf16", order="packed", residual=True,
             p=0.0, sums=True, stats=False),
        # a training batch of 16384 tokens: dropout, residual add, norm, with what the backward pass needs
        dict(name="norm_add_dropout_train", op="norm", rows=16384, cols=4096, type="bf16", order="packed",
             residual=True, p=0.1, sums=True, stats=True),
        # odd sizes in fp32, rows of a wider buffer
        dict(name="norm_f32_ragged", op="norm", rows=1777, cols=1003, type="f32", order="view", residual=False, p=0.0,
             sums=False, stats=True),
        # the backward pass of the training batch: gradients of both branches, of weight and bias
        dict(name="norm_backward_train", op="norm_backward", rows=16384, cols=4096, type="bf16", order="packed",
             add=True, p=0.1),
        # wide rows (the feed-forward width of the GEMM workloads), fewer of them
        dict(name="norm_backward_wide", op="norm_backward", rows=2048, cols=14336, type="bf16", order="packed",
             add=True, p=0.0),
        # a short fp32 step of odd length
        dict(name="norm_backward_f32", op="norm_backward", rows=333, cols=1000, type="f32", order="packed", add=False,
             p=0.0),
        # dropout behind the activation of a feed-forward layer (its backward pass is the same call)
        dict(name="dropout_hidden", op="dropout", rows=8192, cols=14336, type="bf16", order="packed", residual=False,
             p=0.1),
        # a small fp32 call of odd width with the residual add
        dict(name="dropout_f32_odd", op="dropout", rows=77, cols=1003, type="f32", order="packed", residual=True,
             p=0.25),
        # output projection of 8192 tokens: bias, dropout and the residual add on the output tile
        dict(name="project_residual", op="project", form="residual", m=8192, n=4096, k=4096, b_layout="nk", p=0.1),
        # feed-forward backward: the gradient through dropout and GELU, and the bias's gradient, on the tile
        dict(name="project_gelu_backward", op="project", form="gelu_backward", m=8192, n=16384, k=4096,
             b_layout="nk", p=0.1),
        # feed-forward forward with odd row count and K, weights stored K x N
        dict(name="project_gelu_odd", op="project", form="gelu", m=1003, n=4104, k=2056, b_layout="kn", p=0.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "norm_backward", "norm_backward", "norm_backward", "dropout", "project",
                     "project"])
    p = rng.choice([0.05, 0.1, 0.1, 0.2, 0.5])
    if op == "project":
        return dict(op=op, form=rng.choice(["residual", "gelu_backward", "gelu"]), m=_log(rng, 1, 8192),
                    n=8 * _log(rng, 8, 2048), k=8 * _log(rng, 8, 512), b_layout=rng.choice(["kn", "nk"]), p=p)
    type_ = rng.choice(["bf16", "bf16", "bf16", "f32"])
    cols = _log(rng, 16, 16384)
    if rng.random() < 0.7:
        cols = max(16, cols // 8 * 8)
    most = 16384 * 4096 // (cols * (2 if type_ == "f32" else 1))
    rows = _log(rng, 1, max(1, min(65536, most)))
    c = dict(op=op, rows=rows, cols=cols, type=type_, order=rng.choice(["packed", "packed", "view"]))
    if op == "dropout":
        c.update(residual=rng.random() < 0.5, p=p)
    elif op == "norm":
        residual = rng.random() < 0.6
        c.update(residual=residual, p=p if residual and rng.random() < 0.6 else 0.0, sums=residual,
                 stats=rng.random() < 0.6)
    else:
        c.update(add=rng.random() < 0.6, p=p if rng.random() < 0.5 else 0.0)
    return c


# ---------------------------------------------------------------- inputs

def _stream(case, g):
    """rows x cols values as a residual stream holds them: channels with a size and an offset of their own."""
    n = case["cols"]
    x = torch.randn(case["rows"], n, generator=g, device=DEV)
    x = x * torch.exp(0.5 * torch.randn(n, generator=g, device=DEV)) + 0.3 * torch.randn(n, generator=g, device=DEV)
    return _placed(case, x.to(TYPES[case["type"]]))


def _placed(case, x):
    """Packed rows, or the rows of a wider buffer."""
    if case["order"] == "packed":
        return x
    wide = torch.zeros(x.shape[0], (x.shape[1] + 8) // 8 * 8 + 64, device=DEV, dtype=x.dtype)
    wide[:, 16:16 + x.shape[1]] = x
    return wide[:, 16:16 + x.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    st = dict(case=case, site=seed % 89, step=seed % 1013,
              seed=(seed * 6364136223846793005 + 1442695040888963407) % 2 ** 63)
    if case["op"] == "project":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"] = normal(m, k).bfloat16()
        st["w"] = (normal(*((n, k) if case["b_layout"] == "nk" else (k, n))) * 0.02).bfloat16()
        if case["form"] != "gelu_backward":
            st["bias"] = normal(n) * 0.1
        if case["form"] != "gelu":  # the residual stream, or what the activation's forward pass read
            st["aux"] = normal(m, n).bfloat16()
    else:
        t, n = TYPES[case["type"]], case["cols"]
        st["x"] = _stream(case, g)
        if case.get("residual"):
            st["residual"] = _stream(case, g)
        if case["op"] != "dropout":
            st["w"], st["b"] = 1.0 + 0.1 * normal(n), 0.1 * normal(n)
        if case["op"] == "norm_backward":  # dy, and the statistics the forward pass kept
            st["dy"] = _placed(case, normal(case["rows"], n).to(t))
            if case["add"]:
                st["add"] = _placed(case, normal(case["rows"], n).to(t))
            x = st["x"].double()
            st["mean"] = x.mean(-1).float()
            st["rstd"] = torch.rsqrt(x.var(-1, unbiased=False) + EPS).float()
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    from gemm_epilogue_transformer_smem_gb300 import api
    case = st["case"]
    st["rng"] = None
    if case["p"]:
        st["rng"] = api.Dropout(case["p"], seed=st["seed"], step=st["step"], device=DEV)
    if case["op"] == "project":
        program = {"residual": ["bias", "dropout", "residual", "store_bf16"],
                   "gelu": ["bias", "gelu_tanh", "dropout", "store_bf16"],
                   "gelu_backward": ["dropout", "gelu_tanh_grad", "store_bf16", "col_sum"]}[case["form"]]
        st["plan"] = api.Plan(case["m"], case["n"], case["k"], program, b_layout=case["b_layout"], dropout=st["rng"])
        st["out"] = api.allocate_outputs(st["plan"], DEV)
        return
    empty = lambda: torch.empty(case["rows"], case["cols"], device=DEV, dtype=TYPES[case["type"]])  # noqa: E731
    vector = lambda n: torch.empty(n, device=DEV)  # noqa: E731
    st["out"] = empty()
    if case["op"] == "norm":
        st["sum"] = empty() if case["sums"] else None
        st["mean"], st["rstd"] = (vector(case["rows"]), vector(case["rows"])) if case["stats"] else (None, None)
    if case["op"] == "norm_backward":
        st["d_residual"] = empty() if case["p"] else None
        st["dw"], st["db"] = vector(case["cols"]), vector(case["cols"])
        st["workspace"] = torch.empty(api.layer_norm_workspace(case["cols"]), dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------- plain form

def _threshold(case):
    """Of the 65536 values a 16-bit number has, those that drop an element."""
    return round(case["p"] * 65536)


def _philox(counter, key):
    """Philox 4x32-10 (Salmon, Moraes, Dror, Shaw 2011): four 32-bit words of each counter, words in int64."""
    low = 0xFFFFFFFF
    a, b, c, d = counter
    k0, k1 = key
    for _ in range(10):
        x, y = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (y >> 32) & low ^ b ^ k0, y & low, (x >> 32) & low ^ d ^ k1, x & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return a, b, c, d


def _kept(st, rows, cols):
    """True where an element stays: one counter for 8 neighbouring columns of a row, 16 bits to each."""
    groups = (cols + 7) // 8
    a = torch.arange(groups, device=DEV).expand(rows, groups)
    b = torch.arange(rows, device=DEV)[:, None].expand(rows, groups)
    words = _philox((a, b, torch.full_like(a, st["site"]), torch.full_like(a, st["step"])),
                    (st["seed"] & 0xFFFFFFFF, st["seed"] >> 32))
    numbers = torch.stack([half for w in words for half in (w & 0xFFFF, w >> 16)], -1)
    return numbers.reshape(rows, groups * 8)[:, :cols] >= _threshold(st["case"])


def _drop(st, x):
    """Dropout of an fp32 matrix."""
    if not st["case"]["p"]:
        return x
    scale = 65536 / (65536 - _threshold(st["case"]))
    return torch.where(_kept(st, *x.shape), x * scale, torch.zeros_like(x))


GELU_A, GELU_B = math.sqrt(2 / math.pi), 0.044715


def _gelu(x):
    return 0.5 * x * (1 + torch.tanh(GELU_A * (x + GELU_B * x * x * x)))


def _gelu_grad(x):
    t = torch.tanh(GELU_A * (x + GELU_B * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * GELU_A * (1 + 3 * GELU_B * x * x)


def run(st):
    case = st["case"]
    if own:
        return _run_own(st)
    if case["op"] == "project":
        w = st["w"].float()
        y = st["x"].float() @ (w.t() if case["b_layout"] == "nk" else w)
        if case["form"] == "residual":
            return (_drop(st, y + st["bias"]) + st["aux"].float()).bfloat16()
        if case["form"] == "gelu":
            return _drop(st, _gelu(y + st["bias"])).bfloat16()
        y = _drop(st, y) * _gelu_grad(st["aux"].float())
        return y.bfloat16(), y.double().sum(0).float()
    t, x = TYPES[case["type"]], st["x"].float()
    if case["op"] == "norm_backward":
        n = (x - st["mean"][:, None]) * st["rstd"][:, None]
        dy = st["dy"].float()
        a = dy * st["w"]
        g = st["rstd"][:, None] * (a - a.mean(-1, keepdim=True) - n * (a * n).mean(-1, keepdim=True))
        if case["add"]:
            g = g + st["add"].float()
        weights = (dy * n).double().sum(0).float(), dy.double().sum(0).float()
        return ((_drop(st, g).to(t), g.to(t)) if case["p"] else (g.to(t),)) + weights
    h = _drop(st, x)
    if case["residual"]:
        h = h + st["residual"].float()
    if case["op"] == "dropout":
        return h.to(t)
    mean = h.mean(-1, keepdim=True)
    c = h - mean
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    out = [(c * rstd * st["w"] + st["b"]).to(t)]
    if case["sums"]:
        out.append(h.to(t))
    if case["stats"]:
        out += [mean[:, 0], rstd[:, 0]]
    return out


# ---------------------------------------------------------------- the package's operators

def _run_own(st):
    from gemm_epilogue_transformer_smem_gb300 import api
    case = st["case"]
    if case["op"] == "project":
        aux = st.get("aux")
        backward = case["form"] == "gelu_backward"
        st["plan"].run(st["x"], st["w"], bias=st.get("bias"), residual=None if backward else aux,
                       preact=aux if backward else None, C=st["out"].C, col_out=st["out"].col_out, site=st["site"],
                       workspace=st["out"].workspace)
        return (st["out"].C, st["out"].col_out) if backward else st["out"].C
    if case["op"] == "dropout":
        api.dropout(st["x"], st["rng"], out=st["out"], residual=st.get("residual"), site=st["site"])
        return st["out"]
    if case["op"] == "norm":
        api.layer_norm(st["x"], weight=st["w"], bias=st["b"], eps=EPS, out=st["out"], residual=st.get("residual"),
                       dropout=st["rng"], site=st["site"], sum_out=st["sum"], mean=st["mean"], rstd=st["rstd"])
        return [t for t in (st["out"], st["sum"], st["mean"], st["rstd"]) if t is not None]
    api.layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], weight=st["w"], dx=st["out"],
                            d_residual=st["d_residual"], dw=st["dw"], db=st["db"], add=st.get("add"),
                            dropout=st["rng"], site=st["site"], workspace=st["workspace"])
    return tuple(t for t in (st["out"], st["d_residual"], st["dw"], st["db"]) if t is not None)


# ---------------------------------------------------------------- in 64 bits

def _product(x, constant):
    """High and low 32-bit words of x * constant, from products of 16-bit halves."""
    x1, x0 = x // 65536, x % 65536
    c1, c0 = divmod(constant, 65536)
    middle = x1 * c0 + (x0 * c0) // 65536
    other = x0 * c1 + middle % 65536
    return x1 * c1 + middle // 65536 + other // 65536, (other % 65536) * 65536 + (x0 * c0) % 65536


def _factors(st, rows, cols):
    """0 or 65536 / (65536 - t) for every element, fp64."""
    case = st["case"]
    groups = -(-cols // 8)
    index = torch.arange(rows * groups, device=DEV, dtype=torch.int64)
    word = [index % groups, index // groups, torch.zeros_like(index) + st["site"], torch.zeros_like(index) + st["step"]]
    key = [st["seed"] % 2 ** 32, st["seed"] // 2 ** 32]
    for i in range(10):
        high0, low0 = _product(word[0], 0xD2511F53)
        high2, low2 = _product(word[2], 0xCD9E8D57)
        word = [torch.bitwise_xor(torch.bitwise_xor(high2, word[1]), (key[0] + i * 0x9E3779B9) % 2 ** 32), low2,
                torch.bitwise_xor(torch.bitwise_xor(high0, word[3]), (key[1] + i * 0xBB67AE85) % 2 ** 32), low0]
    t = int(math.floor(case["p"] * 65536 + 0.5))
    f = torch.empty(rows, groups, 8, dtype=torch.float64, device=DEV)
    for j in range(8):
        number = word[j // 2].reshape(rows, groups) // (65536 if j % 2 else 1) % 65536
        f[:, :, j] = (number >= t).double() * (65536.0 / (65536.0 - t))
    return f.reshape(rows, groups * 8)[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    shape = (case["m"], case["n"]) if case["op"] == "project" else (case["rows"], case["cols"])
    f = _factors(st, *shape) if case["p"] else 1.0
    if case["op"] == "project":
        y = torch.mm(st["x"].double(), st["w"].double().T if case["b_layout"] == "nk" else st["w"].double())
        if case["form"] == "residual":
            return (y + st["bias"].double()).mul_(f).add_(st["aux"].double())
        z = y + st["bias"].double() if case["form"] == "gelu" else st["aux"].double()
        s = torch.sigmoid(2.0 * GELU_A * (z + GELU_B * z ** 3))  # (1 + tanh(u)) / 2
        if case["form"] == "gelu":
            return z * s * f
        y = y * f * (s + 2.0 * GELU_A * z * s * (1.0 - s) * (1.0 + 3.0 * GELU_B * z ** 2))
        return y, y.sum(0)
    x = st["x"].double()
    if case["op"] == "norm_backward":
        r = st["rstd"].double()[:, None]
        n = (x - st["mean"].double()[:, None]) * r
        dy = st["dy"].double()
        a = dy * st["w"].double()
        along = torch.sum(a * n, 1, keepdim=True) / case["cols"]
        g = r * (a - torch.sum(a, 1, keepdim=True) / case["cols"] - n * along)
        if case["add"]:
            g = g + st["add"].double()
        return ((g * f, g) if case["p"] else (g,)) + (torch.sum(dy * n, 0), torch.sum(dy, 0))
    h = x * f
    if case["residual"]:
        h = h + st["residual"].double()
    if case["op"] == "dropout":
        return h
    mean = torch.sum(h, 1, keepdim=True) / case["cols"]
    size = torch.sqrt(torch.sum((h - mean) ** 2, 1, keepdim=True) / case["cols"] + EPS)
    out = [(h - mean) / size * st["w"].double() + st["b"].double()]
    if case["sums"]:
        out.append(h)
    if case["stats"]:
        out += [mean[:, 0], 1.0 / size[:, 0]]
    return out


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "project":
        m, n, k = case["m"], case["n"], case["k"]
        outer = 2 if case["form"] == "gelu" else 4  # C, and the residual or pre-activation
        return {"bytes": 2 * (m * k + k * n) + outer * m * n + 4 * n, "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "dropout":
        return {"bytes": (2 + case["residual"]) * rows * cols * size, "flops": 2 * rows * cols}
    if case["op"] == "norm":
        passes = 2 + case["residual"] + case["sums"]
        return {"bytes": passes * rows * cols * size + 8 * cols + (8 * rows if case["stats"] else 0),
                "flops": 8 * rows * cols}
    passes = 3 + case["add"] + (1 if case["p"] else 0)
    return {"bytes": passes * rows * cols * size + 8 * rows + 12 * cols, "flops": 14 * rows * cols}
