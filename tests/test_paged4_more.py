"""Attention over a cache in 4 bits: the keys' powers of two.  Against the definition in 64 bits, with the bounds of
tests/test_paged_accuracy.py."""
import math

import pytest
import torch

import block_sparse_flash_ra_gb300 as ra
from tests import test_paged as tp
from tests import test_paged_accuracy as ta
from tests.test_paged import KERNELS, each_kernel, each_type
from tests.test_paged4 import BF, Pool, bounds, i32

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_flash_ra_gb300 import _build
    _build.build()
    yield
    if torch.cuda.is_available():
        torch.cuda.synchronize()
        assert ra.ra_get_device_status() == ra.RA_OK


# ------------------------------------------------------------- keys' scales
@gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (4, 1, 64), (12, 1, 64), (8, 2, 128), (8, 1, 128), (16, 1, 128), (24, 1, 128), (32, 1, 128), (80, 1, 128)])
def test_keys_scales_that_change_with_every_tile(Hq, Hkv, D):
    """Every other tile's keys are 2^-12 as large: a scale of the tile before or behind moves logits by much more than the bound.
    The same bits every time, on two streams at once."""
    tile = 128 * 128 // D
    pool = Pool([13 * tile, 4 * tile + 37, tile - 1], Hkv=Hkv, D=D, page=64, seed=11, spread=0.3)
    for b in range(3):
        for t, at in enumerate(pool.places(b)):
            if t // tile % 2:
                pool.scale(0, at, -12)
    q = torch.randn((3, 1, Hq, D), generator=torch.Generator().manual_seed(12)).to(BF)
    scale = ta.f32(D ** -0.5)
    out, lse = ta.forward(pool, q, scale, causal=False)
    for b in range(3):
        assert ta.errors(pool, q[b], out[b], scale, b=b, causal=False, **ta.BOUNDS[ta.kernel(Hq // Hkv, D, tp.F8, BF)]) <= 1
    p = ra.make_paged_params(pool.cache, q.cuda(), pool.table.cuda(), i32(pool.lens), scale=scale, causal=False)
    qd, streams, got = q.cuda(), [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(50):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(ra.paged_forward(p, qd, pool.cache))
    torch.cuda.synchronize()
    for o, e in got:
        assert torch.equal(o.cpu().double(), out) and torch.equal(e.cpu().double(), lse)


# ------------------------------------------------------------- keys without a value
@gpu
@each_type
@pytest.mark.parametrize("Hq,Hkv,Lq,D", [(1, 1, 3, 128), (4, 2, 4, 128), (8, 1, 4, 128), (8, 1, 10, 128), (1, 1, 2, 64), (4, 2, 2, 64), (2, 1, 3, 64),
                                         (2, 1, 5, 64), (3, 1, 4, 64), (8, 1, 5, 64)])
def test_a_key_without_a_value_does_not_reach_rows_before_it(Hq, Hkv, Lq, D, dtype):
    """The drafts' own last tokens hold key blocks of NaN, at places of either parity: queries before them see none of it, those
    behind nothing else."""
    lens = [130, 41, 300, Lq, 259]
    pool = Pool(lens, Hkv=Hkv, D=D, page=16, seed=37, spread=0.5)
    gone = [(0, 1, 1), (1, 1, 0), (2, 2, 1), (2, 2, 0), (3, 1, 0), (4, 2, 1)]  # sequence, tokens from its end, block
    for b, back, x in gone:
        page, _, at = pool.places(b)[lens[b] - back]
        pool.val[0][page, :, at, 32 * x:32 * x + 32] = 0
        pool.cache.k_exps[page, :, at, x] = 255
        pool.cache.k_pages.view(torch.uint8)[page, :, at, 16 * x:16 * x + 16] = 0x5a  # whatever its codes are
    q = torch.randn((5, Lq, Hq, D), generator=torch.Generator().manual_seed(38)).to(dtype)
    scale = ta.f32(D ** -0.5)
    out, lse = ta.forward(pool, q, scale)
    bound = ta.BOUNDS[ta.kernel(Hq // Hkv * Lq, D, tp.F8, dtype)]
    for b in range(5):
        sees = torch.arange(Lq) >= Lq - max(back for s, back, _ in gone if s == b)
        assert torch.isnan(out[b, sees]).all() and torch.isnan(lse[b][:, sees]).all()
        assert torch.isfinite(out[b, ~sees]).all() and torch.isfinite(lse[b][:, ~sees]).all()
        k, v = (t.repeat_interleave(Hq // Hkv, 1) for t in pool.dense(b))
        s = torch.einsum("ihd,jhd->hij", q[b].double(), k) * scale
        s = s.masked_fill(torch.arange(lens[b]) > torch.arange(Lq)[:, None] + lens[b] - Lq, -math.inf)
        p = torch.softmax(s, -1)
        o = torch.einsum("hij,jhd->ihd", p, v)
        near = (out[b] - o).abs() <= ta.allowed(p, v, o, dtype, **bound)
        assert (near | sees[:, None, None]).all()


@gpu
@each_type
@pytest.mark.parametrize("Hq", [1, 4, 8, 16])
def test_pairs_of_keys_without_a_value_behind_a_length(Hq, dtype):
    """D = 64: an odd length ends inside a pair of tokens, whose other one is NaN in keys and values; and one token of a prefix is."""
    pool = Pool([7, 65, 64, 301], Hkv=1, D=64, page=16, seed=39, prefix=33)
    for b in (0, 1, 3, None):
        pages, n = (pool.prefix, 33) if b is None else (pool.table[b], pool.lens[b])
        at = (int(pages[n // 16]), slice(None), n % 16)
        pool.cache.k_exps[at], pool.cache.v_exps[at] = 255, 255
    q = torch.randn((4, 1, Hq, 64), generator=torch.Generator().manual_seed(40)).to(dtype)
    tp.check_attention(pool, q)
    page, _, at = pool.places(None)[4]
    pool.cache.k_exps[page, :, at, 1] = 255
    out, lse = ta.forward(pool, q, 0.125)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


# ------------------------------------------------------------- sizes of keys
@gpu
@each_type
@each_kernel
@pytest.mark.parametrize("keys,queries", [(116, -112), (116, 0), (60, -60), (-95, 0), (-108, 108)])
def test_keys_at_the_ends_of_their_range(keys, queries, name, dtype):
    """Keys around 2^116 or 2^-108, with queries or a scale that make the logits what they are without: up to 20 or so, as all
    products are positive."""
    Hq, Hkv, Lq, D = KERNELS[name]
    pool = Pool([300, 40], Hkv=Hkv, D=D, page=32, seed=61, spread=0.3)
    pool.cache.k_pages.view(torch.uint8).bitwise_and_(0x77)
    pool.cache.k_exps += keys
    pool.val[0] = pool.val[0].abs() * 2.0 ** keys
    q = (torch.randn((2, Lq, Hq, D), generator=torch.Generator().manual_seed(62)).abs() * 2.0 ** queries).to(dtype)
    scale = ta.f32(D ** -0.5 * 2.0 ** -(keys + queries))
    out, lse = ta.forward(pool, q, scale, causal=False)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for b in (0, 1):
        assert ta.errors(pool, q[b], out[b], scale, b=b, causal=False, **bounds(name, dtype)) <= 1


@gpu
@each_type
@each_kernel
@pytest.mark.parametrize("order", ["turns", "fixed"])
def test_key_blocks_far_apart(order, name, dtype):
    """The blocks of a key 2^0, 2^-7, 2^-14 and 2^-20 as large, in an order that turns from token to token; or by steps of 2^3 in
    one order, with queries the other way round, so that all blocks of a logit count alike.  No kernel rounds a key: the bounds
    are those of the weights."""
    Hq, Hkv, Lq, D = KERNELS[name]
    pool = Pool([300, 40], Hkv=Hkv, D=D, page=32, seed=21, spread=0.0)
    g = torch.Generator().manual_seed(22)
    x = torch.arange(D // 32)
    q = torch.randn((2, Lq, Hq, D), generator=torch.Generator().manual_seed(23))
    for b, n in enumerate(pool.lens):
        e = torch.tensor([0.0, -7.0, -14.0, -20.0])[(x + torch.arange(n)[:, None]) % 4] if order == "turns" else -3.0 * x.expand(n, -1)
        pool.put(0, b, torch.randn((n, D), generator=g) * torch.pow(2.0, e).repeat_interleave(32, -1))
    if order == "fixed":
        q = q * torch.pow(2.0, 3.0 * x).repeat_interleave(32)
    q = q.to(dtype)
    scale = ta.f32(D ** -0.5)
    out, _ = ta.forward(pool, q, scale, causal=False)
    for b in (0, 1):
        assert ta.errors(pool, q[b], out[b], scale, b=b, causal=False, **bounds(name, dtype)) <= 1
