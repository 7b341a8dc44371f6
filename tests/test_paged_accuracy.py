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


def errors(pool, b, q, got, scale, share, floor=0.0, sinks=None, causal=True):
    """The largest error of sequence b's outputs, in units of what is allowed: 2^-8 |o| + share sum p |v|, and `floor` of
    the largest contribution p_j max|v_j| for each key."""
    k, v = pool.dense(b)
    n, Hq, _ = q.shape
    k, v = (t.repeat_interleave(Hq // t.shape[1], 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q.double(), k) * scale
    if causal:
        j = torch.arange(k.shape[0]) - pool.prefix_len
        s = s.masked_fill((j > torch.arange(n)[:, None] + pool.lens[b] - n) & (j >= 0), -math.inf)
    whole = s if sinks is None else torch.cat([s, sinks.double()[:, None, None].expand(Hq, n, 1)], -1)
    p = torch.exp(s - torch.logsumexp(whole, -1, keepdim=True))
    o = torch.einsum("hij,jhd->ihd", p, v)
    mass = torch.einsum("hij,jhd->ihd", p, v.abs())
    top = (p * v.abs().amax(-1).T[:, None]).amax(-1).T[..., None]
    allowed = (2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -23) * o.abs() + share * mass + floor * k.shape[0] * top
    return float(((got - o).abs() / allowed).max())


# rows per kv head and head size of calls that the few-row kernel takes
FEW = {"rows8": (8, 128), "rows16": (16, 128), "rows24": (24, 128), "rows32": (32, 128), "d64": (4, 64), "d64_12": (12, 64)}


@gpu
@each_cache
@pytest.mark.parametrize("name", FEW)
def test_references_that_rise_with_every_tile(name, cache):
    """Each tile's logits pass the reference by more than is let pass (2^4 of a weight with an 8-bit cache, 2^60 with a
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
        assert errors(pool, b, q[b], out[b], scale, 2.0 ** -10) <= 1


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
