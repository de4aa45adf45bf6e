"""Cases of the query / key operators: rotary positions, the RMS norm of each
head with the rotation in the same pass (and its backward pass), and the
projection that applies both to its output tile.

``own`` false: plain torch formulas in fp32 (angles in fp64).  ``own`` true:
the package's entry points on the same inputs.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one generated token of one sequence, far into a long context: launch latency
        dict(name="rotary_one_token", op="rotary", batch=1, tokens=1, hq=32, hk=8, d=128, rot=128, layout="half",
             type="bf16", order="packed", base=500000.0, scaling="by_parts", far=131072, pos="int64", inverse=False),
        # a prompt of 8192 tokens, q and k read out of the packed projection output, scaled for a long context
        dict(name="rotary_prompt", op="rotary", batch=1, tokens=8192, hq=32, hk=8, d=128, rot=128, layout="half",
             type="bf16", order="packed", base=10000.0, scaling="by_parts", far=65536, pos="int32", inverse=False),
        # gradients of a long training batch: the inverse rotation, interleaved pairs
        dict(name="rotary_backward_long", op="rotary", batch=8, tokens=8192, hq=32, hk=8, d=128, rot=128,
             layout="interleaved", type="bf16", order="bshd", base=10000.0, scaling="none", far=0, pos="int64",
             inverse=True),
        # part of an 80-wide head rotated, odd length, heads outside tokens, fp32
        dict(name="rotary_part_f32", op="rotary", batch=3, tokens=1001, hq=12, hk=12, d=80, rot=32, layout="half",
             type="f32", order="bhsd", base=10000.0, scaling="linear", far=4096, pos="int32", inverse=False),
        # a decode step of 64 sequences at positions of their own
        dict(name="norm_decode_64", op="norm", batch=64, tokens=1, hq=32, hk=8, d=128, rot=128, layout="half",
             type="bf16", order="packed", base=1000000.0, scaling="none", far=40960, pos="int32", inverse=False),
        # the largest token count of the GEMM workloads: queries and keys of 16384 tokens
        dict(name="norm_prompt", op="norm", batch=2, tokens=8192, hq=32, hk=8, d=128, rot=128, layout="half",
             type="bf16", order="packed", base=1000000.0, scaling="none", far=0, pos="int64", inverse=False),
        # wide heads, a quarter of them rotated as interleaved pairs, a ragged number of tokens
        dict(name="norm_wide_ragged", op="norm", batch=1, tokens=1777, hq=10, hk=2, d=256, rot=64,
             layout="interleaved", type="bf16", order="bshd", base=10000.0, scaling="ntk", far=32768, pos="int64",
             inverse=False),
        # training: gradients of 16384 tokens and of both norm weights
        dict(name="norm_backward_train", op="norm_backward", batch=2, tokens=8192, hq=32, hk=8, d=128, rot=128,
             layout="half", type="bf16", order="packed", base=1000000.0, scaling="none", far=0, pos="int64",
             inverse=False),
        # a short fp32 step with 64-wide heads, heads outside tokens, odd length
        dict(name="norm_backward_f32", op="norm_backward", batch=3, tokens=333, hq=14, hk=2, d=64, rot=64,
             layout="interleaved", type="f32", order="bhsd", base=10000.0, scaling="none", far=1024, pos="int32",
             inverse=False),
        # q, k and v of an 8192-token prompt from one GEMM, norm and rotation on the output tile
        dict(name="project_prompt", op="project", m=8192, k=4096, hq=32, hk=8, d=128, rot=128, layout="half",
             b_layout="nk", norm=True, bias=False, base=1000000.0, scaling="none", far=32768, pos="int32"),
        # the same projection for a decode step of 64 tokens: reading the weights bounds it
        dict(name="project_decode_64", op="project", m=64, k=4096, hq=32, hk=8, d=128, rot=128, layout="half",
             b_layout="nk", norm=True, bias=False, base=1000000.0, scaling="none", far=40960, pos="int32"),
        # odd row count and K, 64-wide heads, bias and rotation without a norm, weights stored K x N
        dict(name="project_bias_odd", op="project", m=1003, k=2056, hq=14, hk=2, d=64, rot=64, layout="interleaved",
             b_layout="kn", norm=False, bias=True, base=10000.0, scaling="linear", far=8192, pos="int64"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "norm", "norm", "norm_backward", "project", "project"])
    c = dict(op=op, layout=rng.choice(["half", "interleaved"]), base=rng.choice([10000.0, 500000.0, 1000000.0]),
             scaling=rng.choice(["none", "none", "linear", "ntk", "by_parts"]), pos=rng.choice(["int32", "int64"]),
             far=_log(rng, 1, 1000000))
    groups = rng.choice([1, 2, 3, 4, 5, 8])
    hk = _log(rng, 1, 12)
    hq = min(64, groups * hk)
    if op == "project":
        d = rng.choice([64, 128, 256])
        hk = min(hk, 1024 // d)
        hq = min(hq, 4096 // d)
        rot = d if rng.random() < 0.7 else d // 2 if d > 64 or c["layout"] == "interleaved" else d
        m, k = _log(rng, 1, 8192), 8 * _log(rng, 8, 512)
        c.update(m=m, k=k, hq=hq, hk=hk, d=d, rot=rot, b_layout=rng.choice(["kn", "nk"]),
                 norm=rng.random() < 0.6, bias=rng.random() < 0.4)
        return c
    d = rng.choice([32, 40, 64, 64, 72, 80, 96, 128, 128, 128, 192, 256])
    rot = rng.choice([d, d, d // 2 // 4 * 4, d // 4 // 4 * 4])
    type_ = rng.choice(["bf16", "bf16", "bf16", "f32"])
    batch = _log(rng, 1, 64)
    most = 8 * 8192 * 40 * 128 // (batch * (hq + hk) * d * (2 if type_ == "f32" else 1))
    tokens = _log(rng, 1, max(1, min(65536, most // 2)))
    c.update(batch=batch, tokens=tokens, hq=hq, hk=hk, d=d, rot=max(4, rot), type=type_,
             order=rng.choice(["packed", "bshd", "bhsd"]), inverse=op == "rotary" and rng.random() < 0.4)
    return c


# ---------------------------------------------------------------- inputs

FACTOR, ORIGINAL, LOW, HIGH = 8.0, 8192.0, 1.0, 32.0  # of the long-context scalings


def _scaling(case):
    return {"none": None, "linear": dict(kind="linear", factor=FACTOR), "ntk": dict(kind="ntk", factor=FACTOR),
            "by_parts": dict(kind="by_parts", factor=FACTOR, original_length=ORIGINAL, low=LOW, high=HIGH,
                             amplitude=1.0 + 0.1 * math.log(FACTOR))}[case["scaling"]]


def _amplitude(case):
    return 1.0 + 0.1 * math.log(FACTOR) if case["scaling"] == "by_parts" else 1.0


def _positions(case, batch, tokens, g):
    """far 0: every sequence counts from 0; else each starts somewhere below `far`."""
    at = torch.arange(tokens, device=DEV).expand(batch, tokens)
    if case["far"]:
        at = at + torch.randint(0, case["far"], (batch, 1), generator=g, device=DEV)
    return at.to(torch.int32 if case["pos"] == "int32" else torch.int64).contiguous()


def _heads(case, g, spread):
    """q and k (batch, tokens, heads, d) of the case's memory order.  Channels
    of a projection's output differ in size: each has a scale of its own."""
    b, s, hq, hk, d = (case[n] for n in ("batch", "tokens", "hq", "hk", "d"))
    t = TYPES[case["type"]]

    def values(shape, heads_at):
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
        scale = [1] * len(shape)
        scale[heads_at], scale[-1] = shape[heads_at], d
        return (x * torch.exp(spread * torch.randn(scale, generator=g, device=DEV))).to(t)

    if case["order"] == "packed":  # the projection's output holds q, k and v heads side by side
        qkv = values((b, s, hq + 2 * hk, d), 2)
        return qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    if case["order"] == "bshd":
        return values((b, s, hq, d), 2), values((b, s, hk, d), 2)
    return values((b, hq, s, d), 1).transpose(1, 2), values((b, hk, s, d), 1).transpose(1, 2)


def _empty(case, heads):
    b, s, d, t = case["batch"], case["tokens"], case["d"], TYPES[case["type"]]
    if case["order"] == "bhsd":
        return torch.empty(b, heads, s, d, device=DEV, dtype=t).transpose(1, 2)
    return torch.empty(b, s, heads, d, device=DEV, dtype=t)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "project":
        m, k, d = case["m"], case["k"], case["d"]
        n = (case["hq"] + 2 * case["hk"]) * d
        normal = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
        st["x"] = normal(m, k).bfloat16()
        st["w"] = (normal(*((n, k) if case["b_layout"] == "nk" else (k, n))) * 0.02).bfloat16()
        st["bias"] = normal(n) * 0.1 if case["bias"] else None
        st["positions"] = torch.randint(0, case["far"], (m,), generator=g, device=DEV,
                                        dtype=torch.int32 if case["pos"] == "int32" else torch.int64)
        st["scale"] = None
        if case["norm"]:  # one factor per column: q's and k's norm weights for each head, 1 for v
            wq, wk = 1.0 + 0.1 * normal(d), 1.0 + 0.1 * normal(d)
            st["scale"] = torch.cat([wq.repeat(case["hq"]), wk.repeat(case["hk"]),
                                     torch.ones(case["hk"] * d, device=DEV)])
    else:
        st["q"], st["k"] = _heads(case, g, 0.5)
        st["positions"] = _positions(case, case["batch"], case["tokens"], g)
        st["q_out"], st["k_out"] = _empty(case, case["hq"]), _empty(case, case["hk"])
        if case["op"] != "rotary":
            st["wq"], st["wk"] = (1.0 + 0.1 * torch.randn(case["d"], generator=g, device=DEV) for _ in range(2))
        if case["op"] == "norm_backward":
            st["dyq"], st["dyk"] = (torch.randn(t.shape, generator=g, device=DEV).to(t.dtype) for t in (st["q"], st["k"]))
            st["dwq"], st["dwk"] = torch.empty(case["d"], device=DEV), torch.empty(case["d"], device=DEV)
    if own:
        from gemm_epilogue_transformer_smem_gb300 import api
        st["rope"] = api.Rotary(case["d"], case["rot"], base=case["base"], layout=case["layout"],
                                scaling=_scaling(case), device=DEV)
        if case["op"] == "project":
            program = (["bias"] if case["bias"] else []) + (["head_rms:%g" % EPS, "col_scale"] if case["norm"] else [])
            st["plan"] = api.Plan(m, n, k, program + ["rotary", "store_bf16"], b_layout=case["b_layout"],
                                  rotary=st["rope"], head_cols=(case["hq"] + case["hk"]) * d)
            st["out"] = api.allocate_outputs(st["plan"], DEV)
        if case["op"] == "norm_backward":
            st["workspace"] = torch.empty(api.qk_norm_rotary_workspace(case["d"]), dtype=torch.uint8, device=DEV)
    else:
        st["freq"] = _frequencies(case).to(DEV)
    return st


# ---------------------------------------------------------------- plain form

def _frequencies(case):
    """Radians per position of each pair, fp64."""
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64)
    base = case["base"]
    if case["scaling"] == "ntk":
        base = base * FACTOR ** (case["rot"] / (case["rot"] - 2))
    f = base ** (-i / case["rot"])
    if case["scaling"] == "linear":
        f = f / FACTOR
    if case["scaling"] == "by_parts":  # fast pairs keep their frequency, slow ones are interpolated
        turns = ORIGINAL * f / (2 * math.pi)
        keep = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = f * keep + f / FACTOR * (1 - keep)
    return f


def _cos_sin(st):
    """fp32 factors (..., 1, rot / 2) of every position, from fp64 angles."""
    angle = (st["positions"].double().unsqueeze(-1) * st["freq"]).unsqueeze(-2)
    a = _amplitude(st["case"])
    return (torch.cos(angle) * a).float(), (torch.sin(angle) * a).float()


def _rotate(x, c, s, case):
    """x (..., heads, d) fp32 with its first `rot` dimensions rotated pair by pair."""
    rot = case["rot"]
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _norm_backward(dy, x, w, c, s, case):
    g = _rotate(dy, c, -s, case)  # the rotation's transpose
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xn = x * r
    gw = g * w
    return r * (gw - xn * (gw * xn).mean(-1, keepdim=True)), (g * xn).double().sum((0, 1, 2)).float()


def run(st):
    case = st["case"]
    if own:
        return _run_own(st)
    c, s = _cos_sin(st)
    if case["op"] == "project":
        w = st["w"].float()
        y = st["x"].float() @ (w.t() if case["b_layout"] == "nk" else w)
        if case["bias"]:
            y = y + st["bias"]
        y = y.view(case["m"], -1, case["d"])
        n = case["hq"] + case["hk"]
        heads = y[:, :n]
        if case["norm"]:
            heads = _norm(heads, st["scale"].view(-1, case["d"])[:n])
        return torch.cat([_rotate(heads, c, s, case), y[:, n:]], 1).view(case["m"], -1).bfloat16()
    q, k, t = st["q"].float(), st["k"].float(), TYPES[case["type"]]
    if case["op"] == "rotary":
        s = -s if case["inverse"] else s
        return _rotate(q, c, s, case).to(t), _rotate(k, c, s, case).to(t)
    if case["op"] == "norm":
        return _rotate(_norm(q, st["wq"]), c, s, case).to(t), _rotate(_norm(k, st["wk"]), c, s, case).to(t)
    dq, dwq = _norm_backward(st["dyq"].float(), q, st["wq"], c, s, case)
    dk, dwk = _norm_backward(st["dyk"].float(), k, st["wk"], c, s, case)
    return dq.to(t), dk.to(t), dwq, dwk


# ---------------------------------------------------------------- the package's operators

def _run_own(st):
    from gemm_epilogue_transformer_smem_gb300 import api
    case = st["case"]
    if case["op"] == "project":
        st["plan"].run(st["x"], st["w"], bias=st["bias"], col_scale=st["scale"], positions=st["positions"],
                       C=st["out"].C, workspace=st["out"].workspace)
        return st["out"].C
    if case["op"] == "rotary":
        api.rotary(st["q"], st["k"], st["rope"], st["positions"], q_out=st["q_out"], k_out=st["k_out"],
                   inverse=case["inverse"])
        return st["q_out"], st["k_out"]
    if case["op"] == "norm":
        api.qk_norm_rotary(st["q"], st["k"], st["rope"], st["positions"], q_weight=st["wq"], k_weight=st["wk"],
                           eps=EPS, q_out=st["q_out"], k_out=st["k_out"])
        return st["q_out"], st["k_out"]
    api.qk_norm_rotary_backward(st["dyq"], st["dyk"], st["q"], st["k"], st["rope"], st["positions"],
                                q_weight=st["wq"], k_weight=st["wk"], eps=EPS, dq=st["q_out"], dk=st["k_out"],
                                dwq=st["dwq"], dwk=st["dwk"], workspace=st["workspace"])
    return st["q_out"], st["k_out"], st["dwq"], st["dwk"]


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """From the definition, in fp64: a rotated pair is a complex number times
    amplitude * exp(i position frequency)."""
    st = prepare(case, seed)
    rot, d = case["rot"], case["d"]
    base = case["base"] * (FACTOR ** (rot / (rot - 2.0)) if case["scaling"] == "ntk" else 1.0)
    freq = []
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(base))
        if case["scaling"] == "linear":
            f /= FACTOR
        if case["scaling"] == "by_parts":
            keep = min(1.0, max(0.0, (ORIGINAL * f / (2.0 * math.pi) - LOW) / (HIGH - LOW)))
            f = f * (keep + (1.0 - keep) / FACTOR)
        freq.append(f)
    angle = st["positions"].to(torch.float64)[..., None] * torch.tensor(freq, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full_like(angle, _amplitude(case)), angle)[..., None, :]

    def turned(x, by):
        y = x.clone()
        first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half" else \
            (slice(0, rot, 2), slice(1, rot, 2))
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * by
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def unit(x):
        return x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / d + EPS)

    if case["op"] == "project":
        w = st["w"].double()
        y = torch.mm(st["x"].double(), w.T if case["b_layout"] == "nk" else w)
        if case["bias"]:
            y += st["bias"].double()
        y = y.reshape(case["m"], -1, d)
        n = case["hq"] + case["hk"]
        if case["norm"]:
            y[:, :n] = unit(y[:, :n]) * st["scale"].double().reshape(-1, d)[:n]
        y[:, :n] = turned(y[:, :n], turn)
        return y.reshape(case["m"], -1)
    q, k = st["q"].double(), st["k"].double()
    if case["op"] == "rotary":
        by = turn.conj() if case["inverse"] else turn
        return turned(q, by), turned(k, by)
    if case["op"] == "norm":
        return turned(unit(q) * st["wq"].double(), turn), turned(unit(k) * st["wk"].double(), turn)

    def gradients(dy, x, w):
        g = turned(dy, turn.conj())
        n = unit(x)
        size = torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / d + EPS)
        gw = g * w
        return (gw - n * torch.sum(gw * n, -1, keepdim=True) / d) / size, (g * n).reshape(-1, d).sum(0)

    dq, dwq = gradients(st["dyq"].double(), q, st["wq"].double())
    dk, dwk = gradients(st["dyk"].double(), k, st["wk"].double())
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "project":
        m, k, n = case["m"], case["k"], (case["hq"] + 2 * case["hk"]) * case["d"]
        return {"bytes": 2 * (m * k + k * n + m * n), "flops": 2 * m * n * k}
    tokens, heads, d = case["batch"] * case["tokens"], case["hq"] + case["hk"], case["d"]
    size = 2 if case["type"] == "bf16" else 4
    passes = 3 if case["op"] == "norm_backward" else 2  # x and dy in, dx out; or x in, y out
    flops = {"rotary": 3 * case["rot"], "norm": 3 * case["rot"] + 4 * d, "norm_backward": 3 * case["rot"] + 11 * d}
    return {"bytes": passes * tokens * heads * d * size + tokens * (4 if case["pos"] == "int32" else 8),
            "flops": tokens * heads * flops[case["op"]]}
