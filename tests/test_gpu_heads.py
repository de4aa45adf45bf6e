"""Rotary positions, the head norm with the rotation and its backward on the
GPU, against the formulas in 64 bits (needs a GB300)."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api

import heads_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
BY_PARTS = dict(kind="by_parts", factor=8.0, original_length=256.0, amplitude=1.25)


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype=BF, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def tensors(g, b, s, hq, hk, d, dtype, order):
    """q and k (batch, tokens, heads, d) in memory order: the heads of a packed
    q|k|v projection, tokens outside heads, heads outside tokens, or a view
    that starts one element past an aligned address with odd strides."""
    if order == "packed":
        qkv = normal(g, b, s, hq + 2 * hk, d, dtype=dtype)
        return qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    if order == "bshd":
        return normal(g, b, s, hq, d, dtype=dtype), normal(g, b, s, hk, d, dtype=dtype)
    if order == "bhsd":
        return (normal(g, b, hq, s, d, dtype=dtype).transpose(1, 2), normal(g, b, hk, s, d, dtype=dtype).transpose(1, 2))
    return normal(g, b, s, hq, d + 3, dtype=dtype)[..., 1:d + 1], normal(g, b, s, hk, d + 1, dtype=dtype)[..., 1:]


def framed(t):
    """An output shaped like t inside a larger buffer filled with 7, and the
    buffer: what lies around the output must stay 7."""
    b, s, h, d = t.shape
    buf = torch.full((b, s + 1, h + 1, d + 8), 7.0, dtype=t.dtype, device=DEV)
    return buf[:, :s, :h, :d], buf


def frame_kept(buf, out):
    b, s, h, d = out.shape
    left = buf.clone()
    left[:, :s, :h, :d] = 7.0
    assert bool((left == 7.0).all()), "written outside the output"


# type, layout, d, rot, hq, hk, batch, tokens, order, far: sizes where a lane
# group is part full, a chunk has no partner, pairs end inside a chunk, a
# warp's last heads are missing; one token and one head; wide and single accesses
CASES = [
    (BF, "half", 128, 128, 32, 8, 1, 1, "packed", 131072),
    (BF, "half", 128, 128, 32, 8, 2, 37, "packed", 0),
    (BF, "interleaved", 128, 128, 5, 1, 3, 7, "bhsd", 1000),
    (BF, "half", 64, 64, 3, 3, 2, 19, "bshd", 77),
    (BF, "half", 96, 96, 7, 1, 1, 33, "bshd", 12345),
    (BF, "half", 80, 32, 12, 12, 2, 21, "bhsd", 4096),
    (BF, "interleaved", 80, 20, 4, 2, 1, 40, "bshd", 4096),
    (BF, "half", 80, 20, 4, 2, 1, 40, "packed", 4096),
    (BF, "half", 72, 36, 3, 2, 2, 11, "bshd", 9),
    (BF, "interleaved", 72, 72, 3, 2, 2, 11, "odd", 9),
    (BF, "half", 256, 64, 10, 2, 1, 50, "bshd", 32768),
    (BF, "interleaved", 512, 512, 2, 1, 1, 5, "bshd", 10),
    (BF, "half", 512, 128, 2, 1, 1, 5, "odd", 10),
    (BF, "half", 8, 4, 1, 1, 1, 3, "bshd", 5),
    (BF, "interleaved", 2, 2, 3, 1, 2, 9, "bshd", 100),
    (BF, "half", 128, 128, 65, 9, 1, 3, "odd", 100),
    (F32, "half", 128, 128, 32, 8, 1, 3, "packed", 1000000),
    (F32, "interleaved", 64, 64, 14, 2, 3, 33, "bhsd", 1024),
    (F32, "half", 80, 32, 12, 12, 1, 101, "bhsd", 4096),
    (F32, "half", 40, 40, 3, 1, 2, 5, "bshd", 64),
    (F32, "half", 88, 24, 3, 1, 2, 5, "odd", 64),
    (F32, "interleaved", 256, 30, 2, 2, 1, 13, "bshd", 64),
]
IDS = ["%s-%s-d%d-r%d-h%d+%d-%dx%d-%s" % (str(c[0])[6:], c[1], *c[2:8], c[8]) for c in CASES]


def setup(case, seed, scaling=None):
    dtype, layout, d, rot, hq, hk, b, s, order, far = case
    g = gen(seed)
    q, k = tensors(g, b, s, hq, hk, d, dtype, order)
    start = torch.randint(0, far + 1, (b, 1), generator=g, device=DEV) if far else torch.zeros(b, 1, device=DEV, dtype=torch.int64)
    pos = torch.arange(s, device=DEV) + start
    rope = api.Rotary(d, rot, layout=layout, scaling=scaling, device=DEV)
    ang = R.Angles(pos.cpu(), rot, layout, (scaling or {}).get("amplitude", 1.0), scaling=scaling)
    return g, q, k, pos, rope, ang


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(case, inverse):
    dtype = case[0]
    _, q, k, pos, rope, ang = setup(case, 1, BY_PARTS)
    (qo, qb), (ko, kb) = framed(q), framed(k)
    api.rotary(q, k, rope, pos.int() if inverse else pos, q_out=qo, k_out=ko, inverse=inverse)
    torch.cuda.synchronize()
    for x, y, buf in ((q, qo, qb), (k, ko, kb)):
        x64 = x.double().cpu()
        R.check(y, ang.rotate(x64, inverse), ang.spread(x64), dtype, 2.0 ** -19)
        frame_kept(buf, y)


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("weights", [True, False])
def test_qk_norm_rotary(case, weights):
    dtype, d = case[0], case[2]
    g, q, k, pos, rope, ang = setup(case, 2)
    wq, wk = (1.0 + 0.2 * normal(g, d, dtype=F32), 1.0 + 0.2 * normal(g, d, dtype=F32)) if weights else (None, None)
    (qo, qb), (ko, kb) = framed(q), framed(k)
    api.qk_norm_rotary(q, k, rope, pos, q_weight=wq, k_weight=wk, eps=1e-5, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    for x, w, y, buf in ((q, wq, qo, qb), (k, wk, ko, kb)):
        n = R.norm(x.double().cpu(), None if w is None else w.double().cpu(), 1e-5)
        R.check(y, ang.rotate(n), ang.spread(n), dtype, 2.0 ** -18)
        frame_kept(buf, y)


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("weights", [True, False])
def test_qk_norm_rotary_backward(case, weights):
    dtype, d = case[0], case[2]
    g, q, k, pos, rope, ang = setup(case, 3, BY_PARTS if weights else None)
    wq, wk = (1.0 + 0.2 * normal(g, d, dtype=F32), 1.0 + 0.2 * normal(g, d, dtype=F32)) if weights else (None, None)
    dyq, dyk = normal(g, *q.shape, dtype=dtype), normal(g, *k.shape, dtype=dtype)
    (dq, qb), (dk, kb) = framed(q), framed(k)
    dwq, dwk = torch.full((d,), 7.0, device=DEV), torch.full((d,), 7.0, device=DEV)
    ws = torch.full((api.qk_norm_rotary_workspace(d),), 0xFF, dtype=torch.uint8, device=DEV)
    api.qk_norm_rotary_backward(dyq, dyk, q, k, rope, pos, q_weight=wq, k_weight=wk, eps=1e-5, dq=dq, dk=dk,
                                dwq=dwq, dwk=dwk, workspace=ws)
    torch.cuda.synchronize()
    for x, dy, w, dx, dw, buf in ((q, dyq, wq, dq, dwq, qb), (k, dyk, wk, dk, dwk, kb)):
        want, want_dw, mag, mag_dw = R.backward(dy.double().cpu(), x.double().cpu(),
                                                None if w is None else w.double().cpu(), 1e-5, ang)
        R.check(dx, want, mag, dtype, 2.0 ** -17)
        rows = x.numel() // d
        R.check(dw, want_dw, mag_dw, F32, 2.0 ** -18 + rows * 2.0 ** -24)
        frame_kept(buf, dx)


def test_many_tokens_wrap_the_grid():
    """More tokens than one wave of warps: every warp takes several, and the
    weight gradients add up over all of them."""
    d, b, s = 64, 3, 20001
    g = gen(4)
    q, k = tensors(g, b, s, 3, 2, d, BF, "packed")
    dyq, dyk = normal(g, *q.shape), normal(g, *k.shape)
    rope = api.Rotary(d, device=DEV)
    pos = torch.arange(s, device=DEV).expand(b, s)
    ang = R.Angles(torch.arange(s).reshape(1, s), d, "half")
    wq, wk = 1.0 + 0.2 * normal(g, d, dtype=F32), 1.0 + 0.2 * normal(g, d, dtype=F32)
    y, yk, dq, dk = (torch.empty(t.shape, dtype=BF, device=DEV) for t in (q, k, q, k))
    dwq, dwk = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(api.qk_norm_rotary_workspace(d), dtype=torch.uint8, device=DEV)
    api.qk_norm_rotary(q, k, rope, pos[0], q_weight=wq, k_weight=wk, q_out=y, k_out=yk)
    api.qk_norm_rotary_backward(dyq, dyk, q, k, rope, None, q_weight=wq, k_weight=wk, dq=dq, dk=dk, dwq=dwq, dwk=dwk,
                                workspace=ws)
    torch.cuda.synchronize()
    for x, dy, w, out, dx, dw in ((q, dyq, wq, y, dq, dwq), (k, dyk, wk, yk, dk, dwk)):
        n = R.norm(x.double().cpu(), w.double().cpu(), 1e-6)
        R.check(out, ang.rotate(n), ang.spread(n), BF, 2.0 ** -18)
        want, want_dw, mag, mag_dw = R.backward(dy.double().cpu(), x.double().cpu(), w.double().cpu(), 1e-6, ang)
        R.check(dx, want, mag, BF, 2.0 ** -17)
        R.check(dw, want_dw, mag_dw, F32, 2.0 ** -18 + x.numel() // d * 2.0 ** -24)


def test_backward_repeats_bit_for_bit():
    d = 128
    g = gen(5)
    q, k = tensors(g, 2, 1500, 8, 2, d, BF, "packed")
    dyq, dyk = normal(g, *q.shape), normal(g, *k.shape)
    rope = api.Rotary(d, device=DEV)
    ws = torch.empty(api.qk_norm_rotary_workspace(d), dtype=torch.uint8, device=DEV)
    got = []
    for _ in range(5):
        dq, dk = torch.empty_like(dyq), torch.empty_like(dyk)
        dwq, dwk = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
        api.qk_norm_rotary_backward(dyq, dyk, q, k, rope, None, dq=dq, dk=dk, dwq=dwq, dwk=dwk, workspace=ws)
        got.append((dq, dk, dwq, dwk))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got[1:] for a, b in zip(got[0], r))


@pytest.mark.parametrize("rot", [128, 32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_equals_out_of_place(layout, rot):
    d = 128
    g = gen(6)
    qkv = normal(g, 1, 45, 12, d)
    q, k = qkv[:, :, :8], qkv[:, :, 8:10]
    rope = api.Rotary(d, rot, layout=layout, device=DEV)
    w = 1.0 + 0.1 * normal(g, d, dtype=F32)
    for op in ("rotary", "norm"):
        buf = qkv.clone()
        qi, ki = buf[:, :, :8], buf[:, :, 8:10]
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        if op == "rotary":
            api.rotary(q, k, rope, q_out=qo, k_out=ko)
            api.rotary(qi, ki, rope, q_out=qi, k_out=ki)
        else:
            api.qk_norm_rotary(q, k, rope, q_weight=w, q_out=qo, k_out=ko)
            api.qk_norm_rotary(qi, ki, rope, q_weight=w, q_out=qi, k_out=ki)
        torch.cuda.synchronize()
        assert torch.equal(qi, qo) and torch.equal(ki, ko)
        assert torch.equal(buf[:, :, 10:], qkv[:, :, 10:]), "v must stay as it was"
    # the backward over its own inputs, and over the gradients
    dyq, dyk = normal(g, *q.shape), normal(g, *k.shape)
    want = torch.empty_like(dyq), torch.empty_like(dyk)
    api.qk_norm_rotary_backward(dyq, dyk, q, k, rope, q_weight=w, dq=want[0], dk=want[1])
    buf, dyq2 = qkv.clone(), dyq.clone()
    api.qk_norm_rotary_backward(dyq2, dyk, buf[:, :, :8], buf[:, :, 8:10], rope, q_weight=w, dq=dyq2, dk=buf[:, :, 8:10])
    torch.cuda.synchronize()
    assert torch.equal(dyq2, want[0]) and torch.equal(buf[:, :, 8:10], want[1])


def test_one_of_q_and_k_alone_and_missing_outputs():
    d, rope = 64, api.Rotary(64, device=DEV)
    g = gen(7)
    q, k = tensors(g, 1, 30, 4, 2, d, BF, "bshd")
    both = torch.empty_like(q), torch.empty_like(k)
    alone = torch.empty_like(q), torch.empty_like(k)
    api.rotary(q, k, rope, q_out=both[0], k_out=both[1])
    api.rotary(q, None, rope, q_out=alone[0])
    api.rotary(None, k[0], rope, k_out=alone[1][0])  # (tokens, heads, d)
    torch.cuda.synchronize()
    assert torch.equal(both[0], alone[0]) and torch.equal(both[1], alone[1])
    dyq, dyk = normal(g, *q.shape), normal(g, *k.shape)
    ws = torch.empty(api.qk_norm_rotary_workspace(d), dtype=torch.uint8, device=DEV)
    dq, dwq, dwk, dw2 = torch.empty_like(q), *(torch.empty(d, device=DEV) for _ in range(3))
    api.qk_norm_rotary_backward(dyq, dyk, q, k, rope, dq=dq, dwq=dwq, dwk=dwk, workspace=ws)
    api.qk_norm_rotary_backward(None, dyk, None, k, rope, dwk=dw2, workspace=ws)  # a weight's gradient alone
    torch.cuda.synchronize()
    ang = R.Angles(torch.arange(30).reshape(1, 30), d, "half")
    for x, dy, dw in ((q, dyq, dwq), (k, dyk, dwk), (k, dyk, dw2)):
        _, want, _, mag = R.backward(dy.double().cpu(), x.double().cpu(), None, 1e-6, ang)
        R.check(dw, want, mag, F32, 2.0 ** -18 + x.numel() // d * 2.0 ** -24)


def test_no_rows():
    d, rope = 64, api.Rotary(64, device=DEV)
    empty = torch.empty(2, 0, 4, d, dtype=BF, device=DEV)
    api.rotary(empty, empty, rope, q_out=empty, k_out=empty)
    api.qk_norm_rotary(empty, None, rope, torch.empty(2, 0, dtype=torch.int32, device=DEV), q_out=empty)
    dw = torch.full((d,), 7.0, device=DEV)
    api.qk_norm_rotary_backward(empty, None, empty, None, rope, dq=empty, dwq=dw)
    no_heads = torch.empty(2, 3, 0, d, dtype=BF, device=DEV)
    api.rotary(no_heads, None, rope, q_out=no_heads)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_gradient_of_no_heads(dtype):
    """The gradient of a weight that no head used is zero, also where nothing
    else is asked for."""
    d, rope = 64, api.Rotary(64, device=DEV)
    x = torch.randn(2, 3, 4, d, device=DEV).to(dtype)
    dy = torch.randn(2, 3, 4, d, device=DEV).to(dtype)
    none = torch.empty(2, 3, 0, d, dtype=dtype, device=DEV)
    ws = torch.empty(api.qk_norm_rotary_workspace(d), dtype=torch.uint8, device=DEV)
    dwq, dwk, dwq2 = (torch.full((d,), 7.0, device=DEV) for _ in range(3))
    api.qk_norm_rotary_backward(none, dy, none, x, rope, dwq=dwq, workspace=ws)
    api.qk_norm_rotary_backward(dy, None, x, None, rope, dwk=dwk)
    dk = torch.empty_like(x)
    api.qk_norm_rotary_backward(none, dy, none, x, rope, dk=dk, dwq=dwq2, workspace=ws)
    want = torch.empty_like(x)
    api.qk_norm_rotary_backward(dy, None, x, None, rope, dq=want)
    torch.cuda.synchronize()
    for dw in (dwq, dwk, dwq2):
        assert bool((dw == 0).all())
    assert torch.equal(dk, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_positions_far_negative_and_shared(dtype):
    """Phases are exact for any 64-bit position; int32 and int64 agree; one row
    of positions serves a batch."""
    d = 64
    rope = api.Rotary(d, base=500000.0, device=DEV)
    x = normal(gen(8), 2, 9, 3, d, dtype=dtype)
    pos = torch.tensor([0, 1, -1, -77777, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 5, 123456789], device=DEV)
    far = torch.tensor([2 ** 40 + 12345, 2 ** 62 + 1, -2 ** 63, 2 ** 63 - 1, 0, 7, -2 ** 45, 3, 10 ** 12], device=DEV)
    outs = [torch.empty_like(x) for _ in range(4)]
    api.rotary(x, None, rope, pos, q_out=outs[0])
    api.rotary(x, None, rope, pos.int(), q_out=outs[1])
    api.rotary(x, None, rope, pos.expand(2, 9), q_out=outs[2])
    api.rotary(x, None, rope, far, q_out=outs[3])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    x64 = x.double().cpu()
    for p, y in ((pos, outs[0]), (far, outs[3])):
        ang = R.Angles(p.cpu().reshape(1, 9), d, "half", base=500000.0)
        R.check(y, ang.rotate(x64), ang.spread(x64), dtype, 2.0 ** -19)


def test_broadcast_inputs():
    """Inputs may repeat in memory (stride 0); outputs may not."""
    d, rope = 64, api.Rotary(64, device=DEV)
    one = normal(gen(9), 1, 1, 1, d)
    x = one.expand(2, 5, 3, d)
    y, want = torch.empty(2, 5, 3, d, dtype=BF, device=DEV), torch.empty(2, 5, 3, d, dtype=BF, device=DEV)
    api.rotary(x, None, rope, q_out=y)
    api.rotary(x.contiguous(), None, rope, q_out=want)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    with pytest.raises(Exception, match="overlap"):
        api.rotary(y, None, rope, q_out=x)


def test_zero_rows_and_bad_values_stay_in_their_head():
    d = 64
    rope = api.Rotary(d, device=DEV)
    x = normal(gen(10), 1, 6, 5, d)
    clean = torch.empty_like(x)
    api.qk_norm_rotary(x, None, rope, q_out=clean)
    bad = x.clone()
    bad[0, 1, 2] = 0.0
    bad[0, 3, 4, 7] = float("inf")
    bad[0, 4, 0, 9] = float("nan")
    y = torch.empty_like(x)
    dy = normal(gen(11), *x.shape)
    dx, dx0 = torch.empty_like(x), torch.empty_like(x)
    api.qk_norm_rotary(bad, None, rope, q_out=y)
    api.qk_norm_rotary_backward(dy, None, x, None, rope, dq=dx0)
    api.qk_norm_rotary_backward(dy, None, bad, None, rope, dq=dx)
    torch.cuda.synchronize()
    hit = torch.zeros(6, 5, dtype=torch.bool, device=DEV)
    hit[1, 2] = hit[3, 4] = hit[4, 0] = True
    assert torch.equal(y[0][~hit], clean[0][~hit]) and torch.equal(dx[0][~hit], dx0[0][~hit])
    assert bool((y[0, 1, 2] == 0).all())                 # 0 / sqrt(eps)
    assert bool(torch.isnan(y[0, 4, 0]).all())
    # a zero row's gradient is g w / sqrt(eps)
    ang = R.Angles(torch.arange(6).reshape(1, 6), d, "half")
    want, _, mag, _ = R.backward(dy.double().cpu(), bad.double().cpu(), None, 1e-6, ang)
    R.check(dx[0, 1, 2], want[0, 1, 2], mag[0, 1, 2], BF, 2.0 ** -17)


def test_missing_heads_add_nothing_with_zero_eps():
    """eps = 0 makes 1 / sqrt(0) of a lane group past the last head; the
    weights' gradients must not see it."""
    d = 64
    g = gen(12)
    q, k = tensors(g, 1, 20, 3, 1, d, BF, "bshd")
    dyq, dyk = normal(g, *q.shape), normal(g, *k.shape)
    dwq, dwk = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(api.qk_norm_rotary_workspace(d), dtype=torch.uint8, device=DEV)
    api.qk_norm_rotary_backward(dyq, dyk, q, k, api.Rotary(d, device=DEV), eps=0.0, dwq=dwq, dwk=dwk, workspace=ws)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(dwq).all()) and bool(torch.isfinite(dwk).all())


def test_strides_past_32_bits():
    """Tokens 2^30 + 8 elements apart: offsets past 2^31."""
    d, s = 128, 4
    step = 2 ** 30 + 8
    buf = torch.empty(step * (s - 1) + 2 * d, dtype=BF, device=DEV)
    x = normal(gen(13), s, 2, d)
    view = buf.as_strided((s, 2, d), (step, d, 1))
    view.copy_(x)
    rope = api.Rotary(d, device=DEV)
    want = torch.empty_like(x)
    api.qk_norm_rotary(x, None, rope, q_out=want)
    api.qk_norm_rotary(view, None, rope, q_out=view)
    torch.cuda.synchronize()
    assert torch.equal(view.contiguous(), want)


def test_streams_and_graphs():
    """A captured call replays on the values its tensors hold by then; two
    graphs with a workspace each run at once on two streams."""
    d = 128
    g = gen(14)
    rope = api.Rotary(d, device=DEV)

    class Step:
        def __init__(self):
            self.q, self.k = tensors(g, 1, 700, 8, 2, d, BF, "packed")
            self.dyq, self.dyk = normal(g, *self.q.shape), normal(g, *self.k.shape)
            self.pos = torch.arange(700, device=DEV, dtype=torch.int32).reshape(1, 700)
            self.y, self.yk, self.dq, self.dk = (torch.empty_like(t) for t in (self.dyq, self.dyk, self.dyq, self.dyk))
            self.dwq, self.dwk = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
            self.ws = torch.empty(api.qk_norm_rotary_workspace(d), dtype=torch.uint8, device=DEV)

        def run(self, **kw):
            api.qk_norm_rotary(self.q, self.k, rope, self.pos, q_out=self.y, k_out=self.yk, **kw)
            api.qk_norm_rotary_backward(self.dyq, self.dyk, self.q, self.k, rope, self.pos, dq=self.dq, dk=self.dk,
                                        dwq=self.dwq, dwk=self.dwk, workspace=self.ws, **kw)

        def results(self):
            return [t.clone() for t in (self.y, self.yk, self.dq, self.dk, self.dwq, self.dwk)]

    steps = [Step(), Step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    steps[0].run(stream=side)
    torch.cuda.synchronize()
    graphs = []
    for st in steps:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            st.run()
        graphs.append(gr)
    for st in steps:  # new values and positions before the replay
        st.q.copy_(normal(g, *st.q.shape))
        st.pos.add_(1000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for st in steps:
        replayed = st.results()
        st.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, st.results()))


def test_refuses_host_tensors():
    rope = api.Rotary(64, device="cpu")
    x = torch.zeros(1, 2, 3, 64, dtype=BF)
    with pytest.raises(ValueError, match="CUDA"):
        api.rotary(x, None, rope, q_out=x)
    with pytest.raises(ValueError, match="steps are on"):
        api.rotary(x.cuda(), None, rope, q_out=x.cuda())


def test_strides_of_single_steps_do_not_matter():
    """One sequence of one token: the strides of those dimensions are never
    used, whatever they are."""
    d, rope = 64, api.Rotary(64, device=DEV)
    x = normal(gen(15), 1, 1, 3, d)
    odd = x.as_strided((1, 1, 3, d), (7, 5, d, 1))
    want, got = torch.empty_like(x), torch.empty_like(x)
    api.rotary(x, None, rope, q_out=want)
    api.rotary(odd, None, rope, q_out=got.as_strided((1, 1, 3, d), (1, 3, d, 1)))
    torch.cuda.synchronize()
    assert torch.equal(want, got)


def test_few_tokens_share_and_many_tokens_fill_the_grid_alike():
    """A token's result does not depend on how many tokens go with it."""
    d, rope = 96, api.Rotary(96, device=DEV)
    x = normal(gen(16), 5000, 7, d)
    pos = torch.arange(5000, device=DEV, dtype=torch.int32) * 3
    w = 1.0 + 0.1 * normal(gen(17), d, dtype=F32)
    full = torch.empty_like(x)
    api.qk_norm_rotary(x, None, rope, pos, q_weight=w, q_out=full)
    for a, b in ((0, 1), (17, 20), (4000, 4999), (4999, 5000)):
        part = torch.empty(b - a, 7, d, dtype=BF, device=DEV)
        api.qk_norm_rotary(x[a:b], None, rope, pos[a:b], q_weight=w, q_out=part)
        torch.cuda.synchronize()
        assert torch.equal(part, full[a:b])


FIRST_CALL_IN_A_CAPTURE = """
import torch
from gemm_epilogue_transformer_smem_gb300 import api
d = 64
q, dy = (torch.randn(1, 50, 4, d, device="cuda").bfloat16() for _ in range(2))
rope, ws = api.Rotary(d), torch.empty(api.qk_norm_rotary_workspace(d), dtype=torch.uint8, device="cuda")
y, y2, dq = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
dw = torch.empty(d, device="cuda")
plan = api.Plan(48, 256, 512, ["head_rms", "rotary", "store_bf16"], b_layout="nk", rotary=rope, head_cols=128)
x, w = torch.randn(48, 512, device="cuda").bfloat16(), torch.randn(256, 512, device="cuda").bfloat16()
out = api.allocate_outputs(plan, "cuda")

def step():
    api.rotary(q, None, rope, q_out=y)
    api.qk_norm_rotary(q, None, rope, q_out=y2)
    api.qk_norm_rotary_backward(dy, None, q, None, rope, dq=dq, dwq=dw, workspace=ws)
    plan.run(x, w, C=out.C, workspace=out.workspace)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (y, y2, dq, dw, out.C)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (y, y2, dq, dw, out.C)))
print("ok")
"""


def test_first_call_of_a_process_inside_a_capture():
    """Nothing a first call sets up is in the way of a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE], cwd=root, capture_output=True, text=True,
                       timeout=300, env=dict(os.environ, PYTHONPATH=root))
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]


def test_frequencies_follow_their_tensor():
    """A copy of the frequencies, or ones put in their place, are the ones used."""
    import copy
    d = 64
    x = normal(gen(18), 1, 20, 2, d)
    rope, other = api.Rotary(d, device=DEV), api.Rotary(d, base=500.0, device=DEV)
    want, got = torch.empty_like(x), torch.empty_like(x)
    api.rotary(x, None, other, q_out=want)
    twin = copy.deepcopy(rope)
    del rope
    twin.steps = other.steps.clone()
    api.rotary(x, None, twin, q_out=got)
    torch.cuda.synchronize()
    assert torch.equal(want, got)
