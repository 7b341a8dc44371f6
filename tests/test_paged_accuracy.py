"""The attention over a paged cache against 64 bits, with bounds relative to what an output is made of.

An output element is o = sum p_j v_j.  Its error is held to the store's rounding, 2^-8 |o| in bf16, and to a share of
sum p_j |v_j|, which stays small where the values' signs cancel."""
import math

import pytest
import torch

import block_sparse_flash_ra_gb300 as ra
from tests.test_paged import KERNELS, F8, Pool, check_attention, each_cache, each_kernel, each_type, queries

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_flash_ra_gb300 import _build
    _build.build()
    yield
    if torch.cuda.is_available():
        torch.cuda.synchronize()
        assert ra.ra_get_device_status() == ra.RA_OK


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def put(pool, which, b, rows):
    """Sets the cached rows of sequence b (None: the prefix) from its first token on; rows (n, D) or (n, Hkv, D) of values
    that the cache holds exactly."""
    at = pool.places(b)[:rows.shape[0]]
    at = torch.tensor([p for p, _, _ in at]), slice(None), torch.tensor([o for _, _, o in at])
    pages, exps = ((pool.cache.k_pages, pool.cache.k_exps), (pool.cache.v_pages, pool.cache.v_exps))[which]
    x = (rows if rows.dim() == 3 else rows[:, None]).double().expand(pool.val[which][at].shape)
    pool.val[which][at] = x
    if exps is None:
        y = x.to(torch.bfloat16)
        assert torch.equal(y.double(), x)
        pages[at] = y.cuda()
    else:
        e = torch.ceil(torch.log2(x.abs().amax(-1).clamp(min=2.0 ** -100) / 448))
        codes = (x * torch.pow(2.0, -e)[..., None]).float().to(F8)
        assert torch.equal(codes.double() * torch.pow(2.0, e)[..., None], x)
        pages.view(torch.uint8)[at] = codes.view(torch.uint8).cuda()
        exps[at] = (e + 127).to(torch.uint8).cuda()


def grid(x):
    """The nearest values of four bits, at most 2^12 below a row's largest: both kinds of cache hold them."""
    m, e = torch.frexp(x)
    y = torch.ldexp(torch.round(m * 16) / 16, e)
    return torch.where(y.abs() < 2.0 ** -12 * y.abs().amax(-1, keepdim=True), 0.0, y)


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def forward(pool, q, scale, **kw):
    p = ra.make_paged_params(pool.cache, q.cuda(), pool.table.cuda(), i32(pool.lens), scale=scale,
                             prefix_table=pool.prefix.cuda() if pool.prefix_len else None,
                             prefix_len=i32([pool.prefix_len]) if pool.prefix_len else None, **kw)
    return [x.cpu().double() for x in ra.paged_forward(p, q.cuda(), pool.cache)]


def allowed(p, v, o, dtype, share, key=0.0, weight=0.0, value=0.0, quiet=0.0):
    """What outputs o = sum p_j v_j may be off by; p (Hq, n, keys), v (keys, Hq, D), o (n, Hq, D).  The store's rounding;
    `share` of sum p |v|; of each key's contribution what is below `key` of the row's largest, p_j max|v_j|, or below
    `quiet` of its largest weight times the loudest value; of each weight what is below `weight` of the row's largest;
    and `value` of the loudest value for each value."""
    row, most = v.abs().amax(-1).T[:, None], p.amax(-1, keepdim=True)
    part, loud = p * row, row.amax(-1, keepdim=True)
    lost = torch.minimum(part, torch.maximum(key * part.amax(-1, keepdim=True), quiet * most * loud))
    lost = lost + torch.minimum(p, weight * most) * row + value * p * loud
    mass = torch.einsum("hij,jhd->ihd", p, v.abs())
    return torch.finfo(dtype).eps / 2 * o.abs() + share * mass + lost.sum(-1).T[..., None]


def errors(pool, q, got, scale, b=0, sinks=None, causal=True, device="cpu", **bound):
    """The largest error of outputs `got` (..., n, Hq, D) of sequence b's queries, in units of what is allowed."""
    q, got, (k, v) = *(t.to(device) for t in (q, got)), (t.to(device) for t in pool.dense(b))
    n, Hq, _ = q.shape
    k, v = (t.repeat_interleave(Hq // t.shape[1], 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q.double(), k) * scale
    if causal:
        i, j = torch.arange(n, device=device)[:, None], torch.arange(k.shape[0], device=device) - pool.prefix_len
        s = s.masked_fill((j > i + pool.lens[b] - n) & (j >= 0), -math.inf)
    whole = s if sinks is None else torch.cat([s, sinks.double()[:, None, None].expand(Hq, n, 1)], -1)
    p = torch.exp(s - torch.logsumexp(whole, -1, keepdim=True))
    o = torch.einsum("hij,jhd->ihd", p, v)
    return float(((got - o).abs() / allowed(p, v, o, q.dtype, **bound).clamp(min=1e-300)).max())


# The bounds of each kernel.
# share, what a weight may be off by, relative to itself; the logits are off by 2^-13 (the bound of their sum's logarithm in
# the other tests).  few8: half a step of f16, 2^-11, and of the third e4m3 term, 2^-12.  few16: two bf16 terms, 2^-16.
# rows8: half a step of f16.  rows16: half a step of bf16, 2^-8.  fp32: the logits.
# key: few8: half of the last step of the third term, 2^-9 / 2^10, at a largest contribution of 2^4.
# quiet: few8: a reference takes no value row for quieter than 2^-30 of the loudest (weights would grow beyond fp32
# otherwise), so the same of 2^-30 of the two's product.
# weight: rows8: half of the last step of f16, 2^-24, at a largest weight of 2^2 at least, and again where a reference
# moved after the weight was stored.
# value: rows8: the same, at a largest value of 2^7 (e4m3's 448 less a binade for a scale that is a power of two).
BOUNDS = {"few8": dict(share=2.0 ** -11 + 2.0 ** -12 + 2.0 ** -13, key=2.0 ** -24, quiet=2.0 ** -54),
          "few16": dict(share=2.0 ** -12), "rows8": dict(share=2.0 ** -11 + 2.0 ** -13, weight=2.0 ** -26, value=2.0 ** -32),
          "rows16": dict(share=2.0 ** -8 + 2.0 ** -12), "fp32": dict(share=2.0 ** -13)}


def kernel(rows, D, cache, dtype):
    return "fp32" if dtype == torch.float32 else ("rows" if D == 128 and rows > 32 else "few") + ("8" if cache == F8 else "16")


def bounds(name, cache, dtype, batch=0):
    """Those of a call of this shape; batch: of one whose prefix is attended for so many sequences too."""
    Hq, Hkv, Lq, D = SHAPES[name]
    of = [BOUNDS[kernel(Hq // Hkv * Lq * m, D, cache, dtype)] for m in (1, batch) if m]
    return {x: max(b.get(x, 0.0) for b in of) for x in ("share", "key", "quiet", "weight", "value")}


SHAPES = dict(KERNELS, rows8_8=(8, 1, 1, 128), rows16_2=(32, 2, 1, 128))
# rows per kv head and head size of calls that the few-row kernel takes
FEW = {"rows8": (8, 128), "rows16": (16, 128), "rows24": (24, 128), "rows32": (32, 128), "d64": (4, 64), "d64_12": (12, 64)}


@gpu
@each_cache
@pytest.mark.parametrize("name", FEW)
def test_references_that_rise_with_every_tile(name, cache):
    """Each tile's logits pass the reference by more than is let pass (2^4 of a weight with an 8-bit cache, 2^16 with a
    16-bit one, whose values fall as the weights grow): O is rescaled between its products again and again."""
    G, D = FEW[name]
    tile, tiles, step = (128 * 128 // D, 12, 5) if cache == F8 else (128 * 128 // D, 2, 61)
    pool = Pool([tile * tiles, tile * tiles - 37], Hkv=2, D=D, page=64, dtype=cache, seed=5)
    g = torch.Generator().manual_seed(6)
    for b, n in enumerate(pool.lens):
        at = torch.arange(n) // tile
        put(pool, 0, b, at[:, None].expand(n, D).float())
        put(pool, 1, b, grid(torch.randn((n, D), generator=g)) * (1 if cache == F8 else torch.pow(2.0, step * (1.0 - at))[:, None]))
    q = torch.ones((2, 1, 2 * G, D), dtype=torch.bfloat16)
    scale = f32(step * math.log(2) / D)
    out, _ = forward(pool, q, scale)
    for b in (0, 1):
        assert errors(pool, q[b], out[b], scale, b, share=2.0 ** -10) <= 1



def dominated(D, cache, loud, small=9, n=5000, seed=80):
    """One sequence: a key that outweighs the others, a value row 2^loud as large that has no weight, and n keys of equal
    weight with values around 1.  The first key's values are 2^-small: the output is the others' sum where they are."""
    pool = Pool([n], Hkv=1, D=D, page=64, dtype=cache, seed=seed)
    g = torch.Generator().manual_seed(seed)
    k, v = torch.zeros((n, D)), grid(torch.randn((n, D), generator=g) + 1)
    k[0], k[1] = 1.0, -8.0
    v[0], v[1] = v[0] * 2.0 ** -small, v[1] * 2.0 ** loud
    put(pool, 0, 0, k)
    put(pool, 1, 0, v)
    return pool


@gpu
@each_type
@each_cache
@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("low,loud,small", [(18, 0, 9), (20, 6, 9), (22, 0, 9), (23, 6, 9), (18, 3, 0), (20, 30, 12), (16, -9, 40)])
def test_small_weights_of_many_keys(low, loud, small, name, cache, dtype):
    """5000 weights 2^-low of the largest, in CTAs that have whole sequences: together they are what comes out."""
    Hq, Hkv, Lq, D = SHAPES[name]
    pool = dominated(D, cache, loud, small)
    B = 304
    pool.table, pool.lens = pool.table.expand(B, -1).contiguous(), pool.lens * B
    q = (1 - torch.arange(Hq // Hkv * Lq) % 4 / 16).view(Lq, -1, 1).expand(B, Lq, Hq // Hkv, D).to(dtype)
    scale = f32(low * math.log(2) / D)
    out, _ = forward(pool, q.contiguous(), scale, causal=False)
    assert errors(pool, q[0], out, scale, causal=False, **bounds(name, cache, dtype)) <= 1


def terms(y, n, rest):
    """y as n terms of e4m3 out of f16, each the rest of the ones before it times `rest`: what they stand for."""
    h, total = y.to(torch.float16), 0
    for k in range(n):
        c = h.float().to(F8)
        total = total + c.double() / rest ** k
        h = (h - c.to(torch.float16)) * rest
    return total


@pytest.mark.parametrize("how,fine", [((3, 32, 16), True), ((2, 32, 16), False), ((1, 32, 16), False), ((3, 16, 16), False)])
def test_the_bounds_tell_lost_terms(how, fine, monkeypatch):
    """Weights split as the few-row kernel does it, with its three terms and with fewer, or with less room below."""
    n, rest, at = how
    monkeypatch.setattr(torch.Tensor, "cuda", lambda self, *a, **kw: self)
    worst = 0.0
    for low, loud in ((18, 0), (20, 6), (22, 0), (23, 6), (None, 0)):
        if low is None:
            pool, scale = Pool([7], Hkv=1, page=64, dtype=F8, seed=81), 128 ** -0.5
            q = torch.randn((1, 64, 128), generator=torch.Generator().manual_seed(82)).to(torch.bfloat16)
        else:
            pool, scale = dominated(128, F8, loud), low * math.log(2) / 128
            q = torch.ones((1, 1, 128), dtype=torch.bfloat16)
        k, v = pool.dense(0)
        s = torch.einsum("ihd,jhd->hij", q.double(), k.expand(-1, q.shape[1], -1)) * scale
        p = torch.exp(s - s.amax(-1, keepdim=True))
        size = torch.pow(2.0, pool.cache.v_exps[pool.table[0, 0].long() if low is None else pool.table[0].long()].double() - 127)
        size = size.view(-1)[:k.shape[0]]
        by = (p * size if rest == 32 else size.expand_as(p)).amax(-1, keepdim=True)  # the reference: contributions, or values
        y = terms((p * size / by * at).float(), n, rest) / at * by / size
        o = torch.einsum("hij,jd->ihd", y / p.sum(-1, keepdim=True), v[:, 0]).to(torch.bfloat16)
        worst = max(worst, errors(pool, q, o.double(), scale, **BOUNDS["few8"]))
    assert (worst <= 1) == fine


@gpu
@each_type
@each_cache
@each_kernel
@pytest.mark.parametrize("prefix", [0, 3, 150])
def test_outputs_relative_to_what_they_are_made_of(prefix, name, cache, dtype):
    """Lengths of a few keys, where one weight's bits show, and of a few tiles, alone and behind a prefix."""
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([1, 2, 3, 5, 9, 17, 40, 129, 300], Hkv=Hkv, D=D, page=32, dtype=cache, seed=83, prefix=prefix)
    q = (2 * queries(name, 9, torch.float32, 84)).to(dtype)
    scale = f32(D ** -0.5)
    out, _ = forward(pool, q, scale, causal=False)
    for b in range(9):
        assert errors(pool, q[b], out[b], scale, b=b, causal=False, **bounds(name, cache, dtype, 9 if prefix else 0)) <= 1




@gpu
@each_type
@each_cache
@pytest.mark.parametrize("name", ["d64_80", "rows8_8", "rows80", "rows320"])
def test_causal_rows_relative_to_what_they_are_made_of(name, cache, dtype):
    """Rows that see their first key in one part of a tile or another: where one does, its neighbours' references move
    too, after some of their weights were stored."""
    _, Hkv, Lq, D = SHAPES[name]
    pool = Pool([Lq + n for n in (-1, 0, 20, 25, 30, 55, 90, 400)], Hkv=Hkv, D=D, page=32, dtype=cache, seed=89)
    q = (2 * torch.randn((8, Lq, SHAPES[name][0], D), generator=torch.Generator().manual_seed(90))).to(dtype)
    scale = f32(D ** -0.5)
    out, _ = forward(pool, q, scale)
    for b in range(8):
        n = min(Lq, pool.lens[b])  # rows before a sequence's first key see nothing
        assert (out[b, :Lq - n] == 0).all()
        assert not n or errors(pool, q[b, Lq - n:], out[b, Lq - n:], scale, b=b, **bounds(name, cache, dtype)) <= 1



@gpu
@each_type
@each_cache
@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("at", [40, 100, 200])
def test_weights_that_were_there_before_the_reference_moved(at, name, cache, dtype):
    """One key with loud values and a weight of 2^-25, then one that outweighs it and has small values."""
    Hq, Hkv, Lq, D = SHAPES[name]
    pool = Pool([250], Hkv=1, D=D, page=64, dtype=cache, seed=91)
    g = torch.Generator().manual_seed(91)
    k, v = torch.full((250, D), -8.0), grid(torch.randn((250, D), generator=g))
    k[0], k[at] = 0.0, 1.0
    v[0], v[at] = v[0] * 2.0 ** 12, v[at] * 2.0 ** -15
    put(pool, 0, 0, k)
    put(pool, 1, 0, v)
    q = torch.ones((1, Lq, Hq // Hkv, D)).to(dtype)
    scale = f32(25 * math.log(2) / D)
    out, _ = forward(pool, q, scale, causal=False)
    assert errors(pool, q[0], out[0], scale, causal=False, **bounds(name, cache, dtype)) <= 1


@gpu
@each_cache
@pytest.mark.parametrize("prefix", [0, 680])
def test_loud_keys_for_many_rows(prefix, cache):
    """Keys and values whose size differs between tokens: references move by any amount, and not only at a row's own
    largest key, since 32 rows move theirs together."""
    Hq, Hkv, Lq, B, D = 64, 2, 20, 5, 128
    pool = Pool([672, 1434, 1333, 90, 20], Hkv=Hkv, D=D, page=128, dtype=cache, seed=92, prefix=prefix)
    g = torch.Generator().manual_seed(92)
    for b in [None] * bool(prefix) + list(range(B)):
        n = prefix if b is None else pool.lens[b]
        for which, most in ((0, 2), (1, 3)):
            e = torch.randint(-most, most + 1, (n, Hkv, 1), generator=g)
            put(pool, which, b, grid(torch.randn((n, Hkv, D), generator=g)) * torch.pow(2.0, e))
    q = (3 * torch.randn((B, Lq, Hq, D), generator=g)).to(torch.bfloat16)
    scale = f32(D ** -0.5)
    out, _ = forward(pool, q, scale)
    for b in range(B):
        assert errors(pool, q[b], out[b], scale, b=b, device="cuda", **BOUNDS[kernel(999, D, cache, torch.bfloat16)]) <= 1



@gpu
@each_type
@each_cache
@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("far", [20, 26, 28])
def test_values_far_below_the_loudest(far, name, cache, dtype):
    """The one key that counts has values 2^-far of those of another."""
    Hq, Hkv, Lq, D = SHAPES[name]
    pool = Pool([130], Hkv=1, D=D, page=64, dtype=cache, seed=93)
    g = torch.Generator().manual_seed(93)
    k, v = torch.full((130, D), -8.0), grid(torch.randn((130, D), generator=g))
    k[3] = 1.0
    v[70] *= 2.0 ** far
    put(pool, 0, 0, k)
    put(pool, 1, 0, v)
    q = torch.ones((1, Lq, Hq // Hkv, D)).to(dtype)
    scale = f32(100 * math.log(2) / D)
    out, _ = forward(pool, q, scale, causal=False)
    assert errors(pool, q[0], out[0], scale, causal=False, **bounds(name, cache, dtype)) <= 1


@gpu
@each_type
@each_cache
@pytest.mark.parametrize("name", SHAPES)
def test_large_values_under_rising_logits(name, cache, dtype):
    """Values around 2^90 and logits that rise by 50 bits twice in a CTA's share: a product of the two does not fit fp32."""
    Hq, Hkv, Lq, D = SHAPES[name]
    pool = Pool([700], Hkv=1, D=D, page=64, dtype=cache, seed=94)
    g = torch.Generator().manual_seed(94)
    put(pool, 0, 0, (torch.arange(700) // 300)[:, None].expand(700, D).float())
    put(pool, 1, 0, grid(torch.randn((700, D), generator=g)) * 2.0 ** 90)
    pool.table, pool.lens = pool.table.expand(304, -1).contiguous(), pool.lens * 304
    q = torch.ones((304, Lq, Hq // Hkv, D)).to(dtype)
    scale = f32(50 * math.log(2) / D)
    out, _ = forward(pool, q, scale, causal=False)
    assert errors(pool, q[0], out, scale, causal=False, **bounds(name, cache, dtype)) <= 1


@gpu
@each_type
@each_cache
@pytest.mark.parametrize("name", ["d64", "rows8", "rows20", "rows80", "rows320"])
def test_long_contexts(name, cache, dtype):
    """65537 and 40001 tokens, causal, behind a short prefix and alone."""
    _, _, _, D = SHAPES[name]
    for prefix in (0, 77):
        pool = Pool([65537, 40001], Hkv=1, D=D, page=128, dtype=cache, seed=85, prefix=prefix)
        q = queries(name, 2, dtype, 86)
        scale = f32(D ** -0.5)
        out, _ = forward(pool, q, scale)
        for b in (0, 1):
            assert errors(pool, q[b], out[b], scale, b=b, device="cuda", **bounds(name, cache, dtype, 2 if prefix else 0)) <= 1


@gpu
@each_cache
@pytest.mark.parametrize("prefix", [0, 100])
def test_captured_behind_other_streams_and_copies(prefix, cache):
    """A call in a graph whose node follows a copy from the host and work of two other streams."""
    pool = Pool([300, 77], Hkv=2, page=32, dtype=cache, seed=87, prefix=prefix)
    host = queries("rows8", 2, torch.bfloat16, 88).repeat(1, 1, 4, 1).pin_memory()
    q, lens = torch.zeros(host.shape, dtype=host.dtype, device="cuda"), i32([300, 77])
    kv_len, more = torch.zeros_like(lens), torch.zeros_like(lens)
    p = ra.make_paged_params(pool.cache, q, pool.table.cuda(), kv_len, scale=0.1, prefix_table=pool.prefix.cuda() if prefix else None,
                             prefix_len=i32([prefix]) if prefix else None)
    want_p = ra.make_paged_params(pool.cache, q, pool.table.cuda(), lens, scale=0.1, prefix_table=pool.prefix.cuda() if prefix else None,
                                  prefix_len=i32([prefix]) if prefix else None)
    want = ra.paged_forward(want_p, host.cuda(), pool.cache)
    out, lse = torch.zeros_like(q), torch.zeros((2, 8, 1), device="cuda")
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        for s, x in zip(side, (kv_len, more)):
            s.wait_stream(here)
            with torch.cuda.stream(s):
                x.copy_(lens)
        q.copy_(host, non_blocking=True)
        for s in side:
            here.wait_stream(s)
        ra.paged_forward(p, q, pool.cache, out=out, lse=lse)
    for _ in range(3):
        for x in (q, kv_len, more, out, lse):
            x.zero_()
        graph.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(more, lens)


@gpu
@each_type
@each_cache
@each_kernel
def test_sinks_of_minus_infinity(name, cache, dtype):
    """A head without a sink among heads that have one: as if it had none, for rows that see nothing too (out 0, lse -inf;
    the others' lse is the sink)."""
    Hq, Hkv, _, D = KERNELS[name]
    sinks = torch.randn(Hq, generator=torch.Generator().manual_seed(70))
    sinks[::2] = -math.inf
    q = queries(name, 4, dtype, 71)
    pool = Pool([0, 300, 1, 40], Hkv=Hkv, D=D, page=32, dtype=cache, seed=72)
    check_attention(pool, q, sinks=sinks)
    # with partial results joined: an empty prefix
    kw = dict(scale=D ** -0.5, sinks=sinks.cuda())
    p = ra.make_paged_params(pool.cache, q.cuda(), pool.table.cuda(), i32(pool.lens), **kw)
    want, want_lse = ra.paged_forward(p, q.cuda(), pool.cache)
    p = ra.make_paged_params(pool.cache, q.cuda(), pool.table.cuda(), i32(pool.lens), prefix_table=i32([0]), prefix_len=i32([0]), **kw)
    got, lse = ra.paged_forward(p, q.cuda(), pool.cache)
    dead = want_lse == -math.inf
    assert dead.any() and torch.equal(lse[dead], want_lse[dead]) and (got.transpose(1, 2)[dead] == 0).all()
    # the same partial results, joined or stored: a rounding or two in fp32, one more step of bf16 at most
    assert (lse[~dead] - want_lse[~dead]).abs().max() <= 1e-5
    assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -7 if dtype == torch.bfloat16 else 2.0 ** -20, atol=2e-6)


# ------------------------------------------------------------- the helpers' checks (no GPU needed)
def host_cache(**kw):
    return ra.new_kv_cache(3, 16, 2, 64, torch.bfloat16, device="cpu", **kw)


def test_params_belong_to_the_device_of_their_tables(monkeypatch):
    """Params serve another cache of the same sizes on the same device only: their tables lie there."""
    c, twin, away = host_cache(), host_cache(), host_cache()
    q, i = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16), lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    p = ra.make_paged_params(c, q, i(1, 1), i(1), scale=1.0)
    # a cache and a query of another GPU, as the checks see them
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    away = ra.make_kv_cache(away.k_pages, away.v_pages)
    assert away._index == 1 and away._sizes != c._sizes and twin._sizes == c._sizes
    called = []
    monkeypatch.setattr(ra, "_on", lambda *a: called.append(a))
    monkeypatch.setattr(ra, "_here", lambda index: False)
    with pytest.raises(ValueError, match="params were made for"):
        ra.paged_forward(p, q, away)
    assert not called


def test_a_cache_is_made_where_it_was_asked_for(monkeypatch):
    """Device 0 is a device, not the lack of one."""
    asked, zeros = [], torch.zeros

    def fake(*a, device=None, **kw):
        asked.append(device)
        return zeros(*a, **kw)

    monkeypatch.setattr(torch, "zeros", fake)
    for device, want in ((0, 0), (None, "cuda"), ("cuda:1", "cuda:1")):
        asked.clear()
        ra.new_kv_cache(1, 16, 1, 64, device=device)
        assert asked == [want] * 4


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Work on it would run on that device, with this one's tensors."""
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 7

    class Device:
        def __init__(self, device):
            self.device = device

        __enter__ = __exit__ = lambda self, *a: None

    ran = []
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "stream", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    with pytest.raises(ValueError, match="stream"):
        ra._on(torch.device("cuda", 0), Stream(), ran.append)
    assert not ran
    ra._on(torch.device("cuda", 1), Stream(), ran.append)
    assert ran == [7]


@gpu
@pytest.mark.parametrize("first", ["page", "wait"])
def test_one_report_does_not_hide_another(first):
    """A wait that ran out and a page out of range: the wait's code, since results are missing then, and both in words."""
    c = ra.new_kv_cache(1, 16, 1, 64)
    x, out = torch.ones((1, 1, 1, 64), device="cuda"), i32([-1])

    def page():
        ra.kv_write(c, x, x, i32([[5]]), i32([0]))

    def wait():
        ra.ra_selftest_wait_timeout(2_000_000, out)

    assert ra.ra_get_device_status() == ra.RA_OK
    for report in (page, wait) if first == "page" else (wait, page):
        report()
        torch.cuda.synchronize()
    assert ra.ra_get_device_status() == ra.RA_ERR_TIMEOUT and "page" in ra.ra_last_error()
    assert ra.ra_get_device_status() == ra.RA_OK
    page()
    assert ra.ra_get_device_status() == ra.RA_ERR_INVALID_ARG and "wait" not in ra.ra_last_error()
    wait()
    assert ra.ra_get_device_status() == ra.RA_ERR_TIMEOUT and "page" not in ra.ra_last_error()
