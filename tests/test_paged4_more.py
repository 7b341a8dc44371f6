"""Attention over a cache in 4 bits: the keys' powers of two.  Against the definition in 64 bits, with the bounds of
tests/test_paged_accuracy.py."""
import pytest
import torch

import block_sparse_flash_ra_gb300 as ra
from tests import test_paged as tp
from tests import test_paged_accuracy as ta
from tests.test_paged4 import BF, Pool, i32

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
