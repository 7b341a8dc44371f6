"""Norms and rotary positions of queries and keys against their definitions in 64 bits.

Tolerances.  The norm's factor carries the error of a sum of D squares (a chain of 16 and 3 or 2 exchanges: at most 20 steps
of 2^-24, halved by the root), of rsqrt (2 units) and of two products; a cosine or sine that of its argument (an angle of at
most half a turn, rounded to 24 bits: pi * 2^-25) and of the function (2 units); the rotation two products and a sum.  Together
less than 30 * 2^-24 of |a| + |b| for a pair (a, b): bound 2^-19.  Gradients of the inputs chain two of these and a mean of D
products: 2^-17 of the terms' magnitudes.  A weight's gradient is a sum over rows: each term carries 2^-19, a lane adds up at most
2000 of them here in 2^-24 steps that grow with the sum, 2^-13 at worst and 2^-18 in practice, where errors of either sign
cancel; bound 2^-16 of the sum of magnitudes.  An output's own rounding: half a step, 2^-8 (bf16).
"""
import math

import pytest
import torch

import block_sparse_flash_ra_gb300 as ra

F4, F8, BF = torch.float4_e2m1fn_x2, torch.float8_e4m3fn, torch.bfloat16
gpu = pytest.mark.gpu
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_flash_ra_gb300 import _build
    _build.build()
    yield
    if torch.cuda.is_available():
        torch.cuda.synchronize()
        assert ra.ra_get_device_status() == ra.RA_OK


# ------------------------------------------------------------- definitions in 64 bits
def frequencies(rot, base=10000.0, **kw):
    return torch.tensor([base ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)


def turn(x, pos, f, interleaved, amplitude=1.0, size=False):
    """x (B, L, H, D), pos (B, L); size: |a| + |b| of each value's pair instead."""
    n = 2 * f.numel()
    ang = (pos.double()[..., None] * f)[:, :, None]
    c, s = amplitude * torch.cos(ang), amplitude * torch.sin(ang)
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if interleaved else (x[..., :n // 2], x[..., n // 2:n])
    y0, y1 = (amplitude * (a.abs() + b.abs()),) * 2 if size else (a * c - b * s, b * c + a * s)
    y = torch.stack([y0, y1], -1).flatten(-2) if interleaved else torch.cat([y0, y1], -1)
    return torch.cat([y, x[..., n:].abs() if size else x[..., n:]], -1)


def norm(x, w, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def forward64(x, pos, f, interleaved, amplitude=1.0, w=None, eps=None):
    u = norm(x, w, eps) if eps is not None else x
    return turn(u, pos, f, interleaved, amplitude) if f is not None else u


def bound64(x, f, interleaved, amplitude=1.0, w=None, eps=None):
    u = norm(x, w, eps) if eps is not None else x
    size = turn(u, torch.zeros(x.shape[:2]), f, interleaved, amplitude, size=True) if f is not None else u.abs()
    return 2.0 ** -19 * size


def close(got, want, slack, what=""):
    """got against fp64 `want`, `slack` elementwise, and the output type's own rounding."""
    step = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    far = (got.cpu().double() - want).abs() - (slack + step * want.abs() + 1e-38)
    assert (far <= 0).all(), f"{what}: {far.max()}"  # (a NaN is not)


def inputs(B, L, Hq, Hkv, D, dtype, seed=0, fused=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, L, Hq + 2 * Hkv, D), generator=g) * torch.exp(2 * torch.randn((B, L, Hq + 2 * Hkv, 1), generator=g))
    x = x.to(dtype)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype) for _ in range(2)]
    return x, x.cuda(), w


SHAPES = [(1, 1, 1, 1, 64), (3, 37, 6, 3, 128), (2, 130, 4, 2, 64), (64, 1, 32, 8, 128), (1, 1000, 16, 16, 128), (5, 3, 33, 1, 64),
          (1, 9, 200, 1, 128), (3, 1700, 1, 2, 64)]


# ------------------------------------------------------------- forward
@gpu
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rot,interleaved", [("D", False), ("D", True), (16, False), (48, True), (48, False), (0, False)])
@pytest.mark.parametrize("B,L,Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("eps", [None, 1e-5])
def test_forward_and_backward(B, L, Hq, Hkv, D, rot, interleaved, dtype, eps):
    rot = D if rot == "D" else rot
    if rot == 0 and eps is None:
        pytest.skip("nothing to do")
    x, xd, w = inputs(B, L, Hq, Hkv, D, dtype, seed=B * L + rot)
    q, k = xd[:, :, :Hq], xd[:, :, Hq:Hq + Hkv]  # slices of a wider tensor
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-5, 200000, (B, L), generator=g, dtype=torch.int32)
    amp = 1.25 if rot else 1.0
    rope = ra.make_rope(rot, interleaved=interleaved, amplitude=amp) if rot else None
    f = frequencies(rot) if rot else None
    kw = dict(eps=eps, q_weight=w[0].cuda(), k_weight=w[1].cuda()) if eps else {}
    p = ra.make_qk_params(q, k, rope=rope, pos=pos.cuda(), **kw)
    outs = ra.qk_forward(p, q, k)
    dy = [torch.randn((B, L, h, D), generator=g).to(dtype) for h in (Hq, Hkv)]
    before = xd.clone()
    grads = ra.qk_backward(p, q if eps else None, k if eps else None, dy[0].cuda(), dy[1].cuda())
    again = ra.qk_backward(p, q if eps else None, k if eps else None, dy[0].cuda(), dy[1].cuda())
    assert torch.equal(before, xd)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(grads, again))
    for i, (lo, hi) in enumerate(((0, Hq), (Hq, Hq + Hkv))):
        x64 = x[:, :, lo:hi].double().requires_grad_()
        w64 = w[i].double().requires_grad_()
        y = forward64(x64, pos, f, interleaved, amp, w64, eps)
        assert outs[i].is_contiguous() and outs[i].dtype == dtype
        close(outs[i], y.detach(), bound64(x64.detach(), f, interleaved, amp, w[i].double(), eps), "forward")
        y.backward(dy[i].double())
        back = turn(dy[i].double(), pos, f, interleaved, amp, size=True) if rot else dy[i].double().abs()
        if not eps:
            close(grads[i], x64.grad, 2.0 ** -19 * back, "dx")
            assert grads[2 + i] is None
            continue
        r = torch.rsqrt(x64.detach().square().mean(-1, keepdim=True) + eps)
        z, a = (x64.detach() * r).abs(), back * w[i].double().abs()
        close(grads[i], x64.grad, 2.0 ** -17 * r * (a + z * (a * z).mean(-1, keepdim=True)), "dx")
        close(grads[2 + i], w64.grad, 2.0 ** -16 * (back * z).sum((0, 1, 2)), "dw")


def test_the_definition_against_differences():
    """The gradients that the others are held to are those of the formula (autograd in 64 bits), and agree with differences."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn((1, 2, 2, 64), generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(64, generator=g, dtype=torch.float64, requires_grad=True)
    pos = torch.tensor([[3, 900]])
    assert torch.autograd.gradcheck(lambda x, w: forward64(x, pos, frequencies(32), True, 1.5, w, 1e-5), (x, w))
    assert torch.autograd.gradcheck(lambda x, w: forward64(x, pos, frequencies(64), False, 1.0, w, 1e-5), (x, w))


@gpu
def test_gradients_against_differences():
    """The kernel's own forward in fp32, moved by h along a direction, against its gradient.  The loss is a sum of some 2000
    products of order one: its difference carries 2^-19 * 2000 / 2h = 0.02 at worst and the curvature's h^2."""
    x, xd, w = inputs(1, 4, 2, 1, 128, torch.float32, seed=5)
    g = torch.Generator().manual_seed(6)
    xs = [torch.randn((1, 4, h, 128), generator=g).cuda() for h in (2, 1)]
    ws = [t.cuda() for t in w]
    rope, h = ra.make_rope(96), 2.0 ** -5
    dy = [torch.randn(t.shape, generator=g).cuda() for t in xs]

    def loss(q, k, wq, wk):
        p = ra.make_qk_params(q, k, rope=rope, eps=1e-5, q_weight=wq, k_weight=wk)
        return sum((o.double() * d.double()).sum() for o, d in zip(ra.qk_forward(p, q, k), dy))

    at = [*xs, *ws]
    p = ra.make_qk_params(*xs, rope=rope, eps=1e-5, q_weight=ws[0], k_weight=ws[1])
    grads = ra.qk_backward(p, *xs, *dy)
    for i in range(4):
        d = torch.randn(at[i].shape, generator=g).cuda()
        d /= d.norm()
        two = [loss(*(t + s * h * d if j == i else t for j, t in enumerate(at))) for s in (1, -1)]
        assert abs(float((two[0] - two[1]) / (2 * h) - (grads[i].double() * d.double()).sum())) < 0.05


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_keep_their_angles(interleaved):
    """fp32 values of one, positions to both ends of 32 bits: the turn is exact, so the outputs are within 2^-21 of cos +- sin.
    (The frequency itself is a double: 2^-53 of up to 2^31 radians is 2^-22.)"""
    pos = torch.tensor([[0, 1, -1, 1 << 20, 123456789, (1 << 31) - 1, -(1 << 31)]], dtype=torch.int32)
    x = torch.ones((1, 7, 1, 128))
    rope = ra.make_rope(128, interleaved=interleaved)
    p = ra.make_qk_params(x.cuda(), rope=rope, pos=pos.cuda())
    got = ra.qk_forward(p, x.cuda())[0].cpu().double()
    assert (got - turn(x.double(), pos, frequencies(128), interleaved)).abs().max() <= 2.0 ** -20


@gpu
def test_positions_from_start_and_prefix_and_changed_in_place():
    x, xd, _ = inputs(3, 5, 4, 2, 128, torch.float32)
    q = xd[:, :, :4]
    start = torch.tensor([0, 70000, 5], dtype=torch.int32).cuda()
    prefix = torch.tensor([1000], dtype=torch.int32).cuda()
    p = ra.make_qk_params(q, rope=ra.make_rope(64), start=start, prefix_len=prefix)
    for more in (0, 17):
        start += more
        pos = torch.arange(5) + start.cpu()[:, None] + 1000
        close(ra.qk_forward(p, q)[0], turn(x[:, :, :4].double(), pos, frequencies(64), False),
              bound64(x[:, :, :4].double(), frequencies(64), False))
    p = ra.make_qk_params(q, rope=ra.make_rope(64))
    close(ra.qk_forward(p, q)[0], turn(x[:, :, :4].double(), torch.arange(5).expand(3, 5), frequencies(64), False),
          bound64(x[:, :, :4].double(), frequencies(64), False))


@gpu
def test_in_place_and_into_slices():
    x, xd, w = inputs(2, 50, 6, 3, 128, BF)
    q, k = xd[:, :, :6], xd[:, :, 6:9]
    kw = dict(rope=ra.make_rope(128), eps=1e-6, q_weight=w[0].cuda(), k_weight=w[1].cuda())
    p = ra.make_qk_params(q, k, **kw)
    want = ra.qk_forward(p, q, k)
    dy = [torch.randn_like(t) for t in want]
    grads = ra.qk_backward(p, q, k, *dy)
    fused = torch.full_like(xd, 7.0)  # gradients as slices of the fused projection's
    ra.qk_backward(p, q, k, *dy, dq=fused[:, :, :6], dk=fused[:, :, 6:9])
    assert torch.equal(fused[:, :, :6], grads[0]) and torch.equal(fused[:, :, 6:9], grads[1]) and (fused[:, :, 9:] == 7).all()
    d2 = [t.clone() for t in dy]
    ra.qk_backward(p, q, k, *d2, dq=d2[0], dk=d2[1])
    assert torch.equal(d2[0], grads[0]) and torch.equal(d2[1], grads[1])
    y = xd.clone()
    ra.qk_backward(p, y[:, :, :6], y[:, :, 6:9], *dy, dq=y[:, :, :6], dk=y[:, :, 6:9])
    assert torch.equal(y[:, :, :6], grads[0]) and torch.equal(y[:, :, 6:9], grads[1])
    y = xd.clone()
    ra.qk_forward(p, y[:, :, :6], y[:, :, 6:9], q_out=y[:, :, :6], k_out=y[:, :, 6:9])
    assert torch.equal(y[:, :, :6], want[0]) and torch.equal(y[:, :, 6:9], want[1]) and torch.equal(y[:, :, 9:], xd[:, :, 9:])
    # keys alone, queries alone, other weight types, none
    assert torch.equal(ra.qk_forward(ra.make_qk_params(None, k, rope=kw["rope"], eps=1e-6, k_weight=w[1].float().cuda()), None, k)[1],
                       want[1])
    assert ra.qk_forward(ra.make_qk_params(q, rope=kw["rope"], eps=1e-6), q)[1] is None


@gpu
def test_norm_of_zeros_infinities_and_nan():
    x = torch.zeros((1, 4, 2, 128))
    x[0, 1, 0, 5], x[0, 2, 1, 7], x[0, 3, 0] = math.inf, math.nan, 1e25  # the last one's squares overflow
    p = ra.make_qk_params(x.cuda(), eps=1e-6, rope=ra.make_rope(128))
    y = ra.qk_forward(p, x.cuda())[0].cpu()
    assert (y[0, 0] == 0).all() and (y[0, 1, 1] == 0).all() and (y[0, 2, 0] == 0).all() and (y[0, 3] == 0).all()
    assert torch.isnan(y[0, 1, 0]).any() and torch.isnan(y[0, 2, 1]).all()
    dx, _, dw, _ = ra.qk_backward(p, x.cuda(), None, torch.ones((1, 4, 2, 128)).cuda())
    assert torch.isfinite(dx[0, 0]).all() and torch.isfinite(dx[0, 1, 1]).all()


@gpu
def test_empty_batches():
    q = torch.empty((0, 5, 4, 128), dtype=BF, device="cuda")
    p = ra.make_qk_params(q, rope=ra.make_rope(128), eps=1e-6)
    assert ra.qk_forward(p, q)[0].shape == q.shape
    dq, dk, dw, dwk = ra.qk_backward(p, q, None, q)
    assert dq.shape == q.shape and dk is None and (dw == 0).all() and dwk is None


@gpu
@pytest.mark.parametrize("eps", [None, 1e-6])
def test_captured_and_on_other_streams(eps):
    x, xd, w = inputs(2, 33, 4, 2, 128, BF)
    q, k = xd[:, :, :4], xd[:, :, 4:6]
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    kw = dict(eps=eps, q_weight=w[0].cuda(), k_weight=w[1].cuda()) if eps else {}
    p = ra.make_qk_params(q, k, rope=ra.make_rope(128), start=start, **kw)
    dy = [torch.randn_like(t) for t in ra.qk_forward(p, q, k)]

    def both(stream=None):
        return (*ra.qk_forward(p, q, k, stream=stream), *ra.qk_backward(p, q, k, *dy, stream=stream))

    both()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for s in (0, 12345):
        start.fill_(s)
        torch.cuda.synchronize()
        graph.replay()
        other = both(side)
        side.synchronize()
        want = both()
        torch.cuda.synchronize()
        for a, b, c in zip(out, other, want):
            assert c is None or (torch.equal(a, c) and torch.equal(b, c))


# ------------------------------------------------------------- a long tensor
@gpu
def test_offsets_beyond_32_bits():
    """2^31 elements and more between the first token and the last (bf16, strided): sampled rows."""
    B, L, Hq, D = 1, 1 << 16, 4, 128
    wide = torch.zeros((B, L, 270, D), dtype=BF, device="cuda")  # 2.26e9 elements
    q = wide[:, :, 100:104]
    q.normal_()
    p = ra.make_qk_params(q, rope=ra.make_rope(128), eps=1e-6)
    y = ra.qk_forward(p, q)[0]
    dx = ra.qk_backward(p, q, None, y, dq=wide[:, :, 200:204])[0]
    at = torch.tensor([0, 5, 40000, L - 1])
    x64 = q[:, at].cpu().double()
    close(y[:, at], forward64(x64, at[None], frequencies(128), False, 1.0, torch.ones(D).double(), 1e-6),
          bound64(x64, frequencies(128), False, 1.0, torch.ones(D).double(), 1e-6))
    assert (wide[:, :, 104:200] == 0).all() and torch.isfinite(dx).all()


# ------------------------------------------------------------- scaled frequencies
def test_frequencies_of_the_scalings():
    """Against their definitions, in double; stored as fractions of a turn."""
    def stored(**kw):
        r = ra.make_rope(64, 10000.0, device="cpu", **kw)
        t = [x % 2 ** 64 / 2 ** 64 for x in r._keep.tolist()]
        return torch.tensor(t, dtype=torch.float64) * 2 * math.pi, r.amplitude
    f = frequencies(64)
    near = lambda a, b: torch.allclose(a, b, rtol=1e-14, atol=1e-17)  # noqa: E731
    assert near(stored()[0], f) and stored()[1] == 1.0
    assert near(stored(scaling="linear", factor=4.0)[0], f / 4)
    ntk, _ = stored(scaling="ntk", factor=8.0)
    assert near(ntk[:1], f[:1]) and near(ntk[-1:], f[-1:] / 8)
    turns = 8192 * f / (2 * math.pi)
    bands, a = stored(scaling="bands", factor=8.0, trained_length=8192)
    assert near(bands[turns > 4], f[turns > 4]) and near(bands[turns < 1], f[turns < 1] / 8) and a == 1.0
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and (bands[mid] < f[mid]).all() and (bands[mid] > f[mid] / 8).all()
    yarn, a = stored(scaling="yarn", factor=16.0, trained_length=8192)
    assert near(yarn[turns > 40], f[turns > 40]) and near(yarn[turns < 0.7], f[turns < 0.7] / 16)
    assert abs(a - (0.1 * math.log(16) + 1)) < 1e-7
    own = ra.make_rope(16, frequencies=[0.5] * 8, amplitude=2.0, device="cpu")
    assert own.amplitude == 2.0 and abs(own._keep[0].item() / 2 ** 64 * 2 * math.pi - 0.5) < 1e-15


# ------------------------------------------------------------- entering the cache
def value_of(cache, at, which):
    """The values at a page place (page, offset) of all heads, fp64, and the scales' exponents."""
    pages, exps = ((cache.k_pages, cache.k_exps), (cache.v_pages, cache.v_exps))[which]
    page, off = at
    if cache.dtype == ra.RA_BF16:
        return pages[page, :, off].cpu().double(), None
    e = exps[page, :, off].cpu().double() - 127
    if cache.dtype == ra.RA_E4M3:
        return pages[page, :, off].cpu().double() * torch.pow(2.0, e)[..., None], e
    b = pages.view(torch.uint8)[page, :, off].cpu().long()
    c = torch.stack([b % 16, b // 16], -1).flatten(-2)
    v = E2M1[c % 8] * torch.where(c >= 8, -1.0, 1.0)
    return (v.unflatten(-1, (-1, 32)) * torch.pow(2.0, e)[..., None]).flatten(-2), e


def check_quantised(cache, val, e, x, slack):
    """Cached values against what they were made of (x, off by up to `slack`)."""
    if cache.dtype == ra.RA_BF16:
        assert ((val - x).abs() <= slack + 2.0 ** -8 * x.abs() + 1e-38).all()
        return
    top, width = (448.0, x.shape[-1]) if cache.dtype == ra.RA_E4M3 else (6.0, 32)
    xb, vb, sb = (t.unflatten(-1, (-1, width)) for t in (x, val, slack))
    s = torch.pow(2.0, e).view(xb.shape[:-1])[..., None]
    amax, room = xb.abs().amax(-1, keepdim=True), sb.amax(-1, keepdim=True)
    assert (amax <= top * s + room).all() and ((amax > top * s / 2 - room) | (s == 2.0 ** -110)).all()
    y = xb.abs() / s
    if cache.dtype == ra.RA_E4M3:
        half = torch.pow(2.0, torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 4)
    else:
        half = torch.where(y <= 2, 0.25, torch.where(y <= 4, 0.5, 1.0))
    assert ((vb - xb).abs() <= half * s * (1 + 1e-9) + sb).all()


@gpu
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("kind", [BF, F8, F4])
@pytest.mark.parametrize("rot,interleaved,eps", [("D", False, 1e-6), ("D", True, 1e-6), (16, False, None), (48, True, 1e-6), (32, False, 1e-6)])
@pytest.mark.parametrize("B,L,Hq,Hkv,D,page", [(1, 1, 1, 1, 64, 16), (3, 37, 6, 3, 128, 16), (2, 130, 4, 2, 64, 128), (64, 1, 32, 8, 128, 64)])
def test_enter(B, L, Hq, Hkv, D, page, rot, interleaved, eps, kind, dtype):
    rot = D if rot == "D" else rot
    x, xd, w = inputs(B, L, Hq, Hkv, D, dtype, seed=rot + B)
    q, k, v = xd[:, :, :Hq], xd[:, :, Hq:Hq + Hkv], xd[:, :, Hq + Hkv:]
    g = torch.Generator().manual_seed(B)
    start = torch.tensor([(11 * b) % 40 for b in range(B)], dtype=torch.int32)
    count = torch.tensor([L - (b * 7) % (L + 1) if b else L for b in range(B)], dtype=torch.int32)
    width = -(-(40 + L) // page)
    table = torch.randperm(B * width + 2, generator=g)[:B * width].to(torch.int32).view(B, width)
    rope = ra.make_rope(rot, interleaved=interleaved)
    kw = dict(eps=eps, q_weight=w[0].cuda(), k_weight=w[1].cuda()) if eps else {}
    prefix = torch.tensor([777], dtype=torch.int32)
    p = ra.make_qk_params(q, k, rope=rope, start=start.cuda(), prefix_len=prefix.cuda(), **kw)
    caches = [ra.new_kv_cache(B * width + 2, page, Hkv, D, kind) for _ in range(2)]
    for c in caches:
        for t in (c.k_pages, c.v_pages, c.k_exps, c.v_exps):
            if t is not None:
                t.view(torch.uint8).fill_(0x11)
    out = torch.full((B, L, Hq, D), 7.0, dtype=dtype, device="cuda")
    assert ra.qk_enter(p, caches[0], q, k, v, table.cuda(), count=count.cuda(), out=out) is out
    # values, and untouched places, as kv_write leaves them; keys likewise where nothing happens to them
    ra.kv_write(caches[1], k, v, table.cuda(), start.cuda(), count.cuda())
    assert torch.equal(caches[0].v_pages.view(torch.uint8), caches[1].v_pages.view(torch.uint8))
    assert kind == BF or torch.equal(caches[0].v_exps, caches[1].v_exps)
    plain = ra.make_qk_params(q, k, start=start.cuda())
    ra.qk_enter(plain, caches[1], q, k, v, table.cuda(), count=count.cuda())
    third = ra.new_kv_cache(B * width + 2, page, Hkv, D, kind)
    for t in (third.k_pages, third.v_pages, third.k_exps, third.v_exps):
        if t is not None:
            t.view(torch.uint8).fill_(0x11)
    ra.kv_write(third, k, v, table.cuda(), start.cuda(), count.cuda())
    assert torch.equal(caches[1].k_pages.view(torch.uint8), third.k_pages.view(torch.uint8))
    assert kind == BF or torch.equal(caches[1].k_exps, third.k_exps)
    pos = torch.arange(L) + start[:, None] + 777
    f = frequencies(rot)
    w64 = [t.double() for t in w]
    y = [forward64(x[:, :, lo:hi].double(), pos, f, interleaved, 1.0, w64[i], eps) for i, (lo, hi) in enumerate(((0, Hq), (Hq, Hq + Hkv)))]
    slack = [bound64(x[:, :, lo:hi].double(), f, interleaved, 1.0, w64[i], eps) for i, (lo, hi) in enumerate(((0, Hq), (Hq, Hq + Hkv)))]
    touched = torch.zeros(caches[0].k_pages.shape[:3], dtype=torch.bool)
    for b in range(B):
        n = int(count[b])
        close(out[b, :n], y[0][b, :n], slack[0][b, :n], "q")
        assert (out[b, n:] == 7).all()
        for i in range(n):
            t = int(start[b]) + i
            at = (int(table[b, t // page]), t % page)
            touched[at[0], :, at[1]] = True
            if i % 9 == 0 or i == n - 1:
                val, e = value_of(caches[0], at, 0)
                check_quantised(caches[0], val, e, y[1][b, i], slack[1][b, i])
    assert (caches[0].k_pages.view(torch.uint8)[~touched.cuda()] == 0x11).all()
    assert kind == BF or (caches[0].k_exps[~touched.cuda()] == 0x11).all()


@gpu
@pytest.mark.parametrize("kind", [BF, F8, F4])
def test_enter_takes_several_tokens_at_a_time(kind):
    """Enough tokens that a CTA has eight: counts that end inside its eight, at their edge and before any; keys alone."""
    B, L, Hkv, D, page = 4, 700, 2, 128, 64
    x, xd, w = inputs(B, L, 3, Hkv, D, BF, seed=77)
    q, k, v = xd[:, :, :3], xd[:, :, 3:5], xd[:, :, 5:]
    start = torch.tensor([0, 5, 64, 3], dtype=torch.int32).cuda()
    count = torch.tensor([L, 0, 333, 8], dtype=torch.int32).cuda()
    table = torch.randperm(60, generator=torch.Generator().manual_seed(1))[:52].to(torch.int32).view(B, 13).cuda()
    kw = dict(rope=ra.make_rope(D), eps=1e-6, q_weight=w[0].cuda(), k_weight=w[1].cuda(), start=start)
    p = ra.make_qk_params(q, k, **kw)
    want_q, want_k = ra.qk_forward(p, q, k)
    out = torch.full((B, L, 3, D), 7.0, dtype=BF, device="cuda")
    caches = [ra.new_kv_cache(60, page, Hkv, D, kind) for _ in range(2)]
    ra.qk_enter(p, caches[0], q, k, v, table, count=count, out=out)
    assert ra.qk_enter(ra.make_qk_params(None, k, **{**kw, "q_weight": None}), caches[1], None, k, v, table, count=count) is None
    for a, b in ((caches[0].k_pages, caches[1].k_pages), (caches[0].v_pages, caches[1].v_pages), (caches[0].k_exps, caches[1].k_exps),
                 (caches[0].v_exps, caches[1].v_exps)):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    kk, vv = ra.kv_read(caches[0], table, start + count, 705)
    for b in range(B):
        n, s = int(count[b]), int(start[b])
        assert torch.equal(out[b, :n], want_q[b, :n]) and (out[b, n:] == 7).all()
        if kind == BF:
            assert torch.equal(kk[b, s:s + n], want_k[b, :n]) and torch.equal(vv[b, s:s + n], v[b, :n])
        assert (kk[b, :s] == 0).all() and (kk[b, s + n:] == 0).all()


@gpu
def test_enter_skips_and_reports_tokens_without_a_place():
    x, xd, _ = inputs(2, 4, 2, 2, 64, BF)
    q, k, v = xd[:, :, :2], xd[:, :, 2:4], xd[:, :, 4:]
    table = torch.tensor([[0], [99]], dtype=torch.int32).cuda()  # a page that the cache does not have
    c = ra.new_kv_cache(2, 16, 2, 64, F4)
    p = ra.make_qk_params(q, k, start=torch.tensor([14, 0], dtype=torch.int32).cuda())  # 14, 15, and two behind the table
    out = ra.qk_enter(p, c, q, k, v, table)
    assert ra.ra_get_device_status() == ra.RA_ERR_INVALID_ARG
    assert torch.equal(out, q) and (c.k_exps[0, :, 14:] != 0).all() and (c.k_exps[0, :, :14] == 0).all() and (c.k_exps[1] == 0).all()
    ra.qk_enter(p, c, q, k, v, torch.zeros_like(table), count=torch.tensor([2, 9], dtype=torch.int32).cuda())  # 9 of 4 tokens
    assert ra.ra_get_device_status() == ra.RA_ERR_INVALID_ARG
    assert ra.ra_get_device_status() == ra.RA_OK


# ------------------------------------------------------------- refusals (no GPU needed)
def _c_params(**kw):
    d = dict(B=2, L=3, Hq=4, Hkv=2, D=128, dtype=ra.RA_BF16, rope=ra.RaRope(128, 0, 1.0, 4096), eps=1e-6,
             weight_dtype=ra.RA_FP32, q_weight=None, k_weight=None, pos=None, start=4096, prefix_len=None)
    d.update(kw)
    return ra.RaQkParams(**d)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), ra.RA_ERR_INVALID_ARG), (dict(Hq=0, Hkv=0), ra.RA_ERR_INVALID_ARG), (dict(D=96), ra.RA_ERR_UNSUPPORTED),
    (dict(dtype=2), ra.RA_ERR_INVALID_ARG), (dict(rope=ra.RaRope(24, 0, 1.0, 4096)), ra.RA_ERR_UNSUPPORTED),
    (dict(rope=ra.RaRope(256, 0, 1.0, 4096)), ra.RA_ERR_UNSUPPORTED), (dict(rope=ra.RaRope(64, 0, 1.0, None)), ra.RA_ERR_INVALID_ARG),
    (dict(rope=ra.RaRope(64, 0, math.nan, 4096)), ra.RA_ERR_INVALID_ARG), (dict(eps=-1.0), ra.RA_ERR_INVALID_ARG),
    (dict(eps=math.nan), ra.RA_ERR_INVALID_ARG), (dict(eps=0.0, q_weight=4096), ra.RA_ERR_INVALID_ARG),
    (dict(weight_dtype=5), ra.RA_ERR_INVALID_ARG), (dict(q_weight=4100), ra.RA_ERR_INVALID_ARG),
    (dict(B=1 << 20, L=1 << 12), ra.RA_ERR_UNSUPPORTED), (dict(pos=4098), ra.RA_ERR_INVALID_ARG),
    (dict(Hq=1 << 17), ra.RA_ERR_UNSUPPORTED),
])
def test_bad_params_are_refused(bad, code):
    p = _c_params(**bad)
    with pytest.raises(ra.RaError) as e:
        ra.ra_qk_fwd(p, 1 << 20, 512, 1 << 24, 256, 1 << 25, 512, 1 << 26, 256, stream=0)
    assert e.value.code == code
    assert ra.ra_qk_bwd_workspace_size(p) == 0


def test_overlaps_and_strides_are_refused():
    p, M = _c_params(), 1 << 20

    def refused(*a):
        with pytest.raises(ra.RaError) as e:
            ra.ra_qk_fwd(p, *a, stream=0)
        assert e.value.code == ra.RA_ERR_INVALID_ARG
        return str(e.value)

    assert "stride" in refused(M, 256, 2 * M, 256, 3 * M, 512, 4 * M, 256)  # narrower than the row
    assert "aligned" in refused(M + 8, 512, 2 * M, 256, 3 * M, 512, 4 * M, 256)
    assert "aligned" in refused(M, 516, 2 * M, 256, 3 * M, 512, 4 * M, 256)
    assert "NULL" in refused(None, 512, 2 * M, 256, 3 * M, 512, 4 * M, 256)
    assert "overlap" in refused(M, 512, 2 * M, 256, M + 256, 512, 4 * M, 256)  # shifted onto its input
    assert "overlap" in refused(M, 512, 2 * M, 256, 2 * M, 512, 4 * M, 256)  # q_out on k
    assert "overlap" in refused(M, 512, 2 * M, 256, 3 * M, 512, 3 * M + 512, 256)  # the outputs on each other
    assert "overlap" in refused(M, 768, M + 1024, 768, M, 512, 4 * M, 256)  # in place with another stride
    with pytest.raises(ra.RaError) as e:
        ra.ra_qk_bwd(p, M, 512, 2 * M, 256, 3 * M, 512, 4 * M, 256, 5 * M, 512, 6 * M, 256, 7 * M, 8 * M, None, stream=0)
    assert e.value.code == ra.RA_ERR_WORKSPACE
    c = ra.RaKvCache(4, 16, 3, 128, ra.RA_BF16, M, M, None, None)
    with pytest.raises(ra.RaError):  # other kv heads
        ra.ra_qk_enter(p, c, M, 512, 2 * M, 256, 3 * M, 256, 4 * M, 512, 4096, 1, stream=0)
    c = ra.RaKvCache(4, 16, 2, 128, ra.RA_BF16, M, M, None, None)
    with pytest.raises(ra.RaError, match="start"):
        ra.ra_qk_enter(_c_params(start=None), c, M, 512, 2 * M, 256, 3 * M, 256, 4 * M, 512, 4096, 1, stream=0)


def test_helpers_refuse():
    q, k = torch.zeros((2, 3, 4, 128)), torch.zeros((2, 3, 2, 128))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    rope = ra.make_rope(64, device="cpu")
    for kw, err in ((dict(pos=i32(2)), ValueError), (dict(pos=torch.zeros((2, 3))), TypeError), (dict(start=i32(3)), ValueError),
                    (dict(q_weight=torch.ones(128)), ValueError), (dict(eps=0.0), ValueError), (dict(eps=1e-50), ValueError),
                    (dict(eps=1e-6, q_weight=torch.ones(64)), ValueError), (dict(prefix_len=i32(2)), ValueError),
                    (dict(eps=1e-6, q_weight=torch.ones(128), k_weight=torch.ones(128, dtype=BF)), TypeError)):
        with pytest.raises(err):
            ra.make_qk_params(q, k, rope=rope, **kw)
    with pytest.raises(ValueError):
        ra.make_qk_params(None, None)
    with pytest.raises(TypeError):
        ra.make_qk_params(q.half(), k.half())
    with pytest.raises(TypeError):
        ra.make_qk_params(q, k.to(BF))
    with pytest.raises(ValueError):
        ra.make_qk_params(q, k[:, :2])
    with pytest.raises(ValueError):
        ra.make_qk_params(torch.zeros((2, 3, 4, 64)), rope=ra.make_rope(128, device="cpu"))
    for kw in (dict(rot=20), dict(rot=0), dict(rot=64, scaling="other"), dict(rot=64, scaling="yarn", factor=2.0),
               dict(rot=64, base=0.5), dict(rot=64, factor=0.5), dict(rot=64, frequencies=[1.0]), dict(rot=16, frequencies=[math.inf] * 8)):
        with pytest.raises(ValueError):
            ra.make_rope(device="cpu", **kw)


@gpu
def test_helpers_refuse_on_the_device():
    x, xd, _ = inputs(2, 3, 4, 2, 128, BF)
    q, k, v = xd[:, :, :4], xd[:, :, 4:6], xd[:, :, 6:]
    p = ra.make_qk_params(q, k, rope=ra.make_rope(64))
    for a in ((q, None), (q, k.float()), (q[:, :2], k[:, :2]), (q, v.transpose(2, 3).contiguous().transpose(2, 3)), (q.cpu(), k)):
        with pytest.raises(ValueError):
            ra.qk_forward(p, *a)
    with pytest.raises(ra.RaError):
        ra.qk_forward(p, q, k, q_out=xd[:, :, 1:5])
    c = ra.new_kv_cache(4, 16, 2, 128, F4)
    table = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    with pytest.raises(ra.RaError, match="start"):
        ra.qk_enter(p, c, q, k, v, table)
    with pytest.raises(ValueError):
        ra.qk_enter(p, c, q, k, v, table[:1])
    with pytest.raises(ValueError):
        ra.qk_enter(ra.make_qk_params(q), c, q, None, v, table)
