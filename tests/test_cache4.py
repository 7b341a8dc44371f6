"""The cache in 4 bits against its definition: codes and scales exactly, values read back exactly."""
import math

import pytest
import torch

import block_sparse_flash_ra_gb300 as ra

F4, BF = torch.float4_e2m1fn_x2, torch.bfloat16
gpu = pytest.mark.gpu
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_flash_ra_gb300 import _build
    _build.build()
    yield
    if torch.cuda.is_available():
        torch.cuda.synchronize()
        assert ra.ra_get_device_status() == ra.RA_OK


def quantise(x):
    """fp64 (..., D) -> the codes' values, exponent bytes (..., D / 32)."""
    x = x.unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax / 6)
    e = torch.where(amax == 0, -110, torch.where(m > 0.5, e, e - 1)).clamp(min=-110)
    good = torch.isfinite(amax)
    e = torch.where(good, e, 128)
    y = x.abs() / torch.pow(2.0, e.double())[..., None]
    near = (y[..., None] - VALUES).abs()
    # the nearest; of two, the one with an even code
    code = torch.argmin(near * 16 + (torch.arange(8) % 2) * 1e-9, -1)
    v = torch.where(x < 0, -VALUES[code], VALUES[code])
    return torch.where(good[..., None], v, 0.0).flatten(-2), (e + 127).to(torch.uint8)


def pack(v):
    """Codes' values (..., D) -> bytes (..., D / 2)."""
    c = torch.searchsorted(VALUES, v.abs().contiguous()) + 8 * (v < 0)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def unpack(b):
    c = torch.stack([b.long() & 15, b.long() >> 4], -1).flatten(-2)
    return VALUES[c & 7] * torch.where(c >= 8, -1.0, 1.0)


def dense(codes, exps):
    s = torch.pow(2.0, exps.double() - 127)
    return (codes.unflatten(-1, (-1, 32)) * torch.where(exps == 255, math.nan, s)[..., None]).flatten(-2)


def test_the_definition_itself():
    x = torch.tensor([6.0, 5.0, 2.5, 3.5, 0.25, 0.75, -1.25, 1.75, -5.1] + [0.0] * 23, dtype=torch.float64)
    v, e = quantise(x)
    assert v[:9].tolist() == [6, 4, 2, 4, 0, 1, -1, 2, -6] and e.tolist() == [127]
    assert quantise(x * 1.01)[1].tolist() == [128] and quantise(x * 2.0 ** -60)[1].tolist() == [67]
    assert torch.equal(unpack(pack(v)), v)


@gpu
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("B,L,Hkv,D,page", [(1, 1, 1, 64, 16), (3, 37, 3, 128, 16), (2, 130, 2, 64, 128), (5, 1, 8, 128, 64)])
def test_write_then_read(B, L, Hkv, D, page, dtype):
    g = torch.Generator().manual_seed(B * L)
    start = [(11 * b) % 40 for b in range(B)]
    count = [L - (b * 7) % (L + 1) if b else L for b in range(B)]
    width = -(-(max(start) + L) // page)
    n = B * width + 2
    table = torch.randperm(n, generator=g)[:B * width].to(torch.int32).view(B, width)
    x = torch.randn((B, L, 2 * Hkv + 1, D), generator=g) * torch.exp(3 * torch.randn((B, L, 2 * Hkv + 1, D // 32), generator=g)
                                                                     ).repeat_interleave(32, -1)
    x[0, 0, 1, :32] = 0.0  # a block of zeros
    x[-1, -1, 1, 3] = 6.0 * 4  # the largest magnitude at a border
    x[0, -1, 1 + Hkv, 32:64] *= 2.0 ** -115  # below the least scale
    x = x.to(dtype)
    fused = x.cuda()
    c = ra.new_kv_cache(n, page, Hkv, D, F4)
    assert c.k_pages.shape == (n, Hkv, page, D // 2) and c.k_exps.shape == (n, Hkv, page, D // 32)
    for t in (c.k_pages, c.v_pages, c.k_exps, c.v_exps):
        t.view(torch.uint8).fill_(0x5a)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    ra.kv_write(c, fused[:, :, 1:1 + Hkv], fused[:, :, 1 + Hkv:], table.cuda(), i32(start), i32(count))
    got = ra.kv_read(c, table.cuda(), i32([s + m for s, m in zip(start, count)]), max(start) + L + 3, torch.float32)
    for which, (pages, exps) in enumerate(((c.k_pages, c.k_exps), (c.v_pages, c.v_exps))):
        codes, e = quantise(x[:, :, 1 + which * Hkv:1 + (which + 1) * Hkv].double())
        want_pages, want_exps = torch.full(pages.shape, 0x5a, dtype=torch.uint8), torch.full(exps.shape, 0x5a, dtype=torch.uint8)
        for b in range(B):
            for i in range(count[b]):
                t = start[b] + i
                at = (int(table[b, t // page]), slice(None), t % page)
                want_pages[at], want_exps[at] = pack(codes[b, i]), e[b, i]
            old = dense(unpack(want_pages), want_exps)  # what lies before `start` reads back, too
            for t in range(start[b] + count[b]):
                assert torch.equal(got[which][b, t].cpu().double(), old[int(table[b, t // page]), :, t % page])
            assert (got[which][b, start[b] + count[b]:] == 0).all()
        assert torch.equal(exps.cpu(), want_exps)
        assert torch.equal(unpack(pages.view(torch.uint8).cpu()), unpack(want_pages))  # (a zero's sign may be either)
    half = ra.kv_read(c, table.cuda(), i32([s + m for s, m in zip(start, count)]), max(start) + L + 3, BF)
    assert torch.equal(half[0].float(), got[0]) and torch.equal(half[1].float(), got[1])  # two bits of a code fit


@gpu
def test_every_code_scale_and_a_block_without_a_value():
    """All 16 codes under all scales read back as their values; an infinity or a NaN takes its own block only."""
    c = ra.new_kv_cache(4, 64, 1, 128, F4)
    codes = torch.arange(256, dtype=torch.uint8).view(4, 64)
    c.k_pages.view(torch.uint8).copy_(codes.cuda()[:, None, :].expand(4, 64, 64).reshape(4, 1, 64, 64))
    exps = torch.arange(256, dtype=torch.uint8).view(4, 1, 64, 1).expand(4, 1, 64, 4).contiguous()
    c.k_exps.copy_(exps.cuda())
    c.v_exps.fill_(127)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    k, _ = ra.kv_read(c, table, torch.tensor([256], dtype=torch.int32).cuda(), 256, torch.float32)
    want = dense(unpack(c.k_pages.view(torch.uint8).cpu()), exps).permute(0, 2, 1, 3).reshape(256, 1, 128)
    want = want.float()  # beyond fp32's range: infinities
    assert torch.equal(torch.isnan(k[0].cpu()), torch.isnan(want)) and torch.equal(k[0].cpu().nan_to_num(3.0, 4.0, 5.0), want.nan_to_num(3.0, 4.0, 5.0))
    x = torch.ones((1, 2, 1, 128), dtype=BF)
    x[0, 0, 0, 40], x[0, 1, 0, 127] = math.nan, -math.inf
    ra.kv_write(c, x.cuda(), x.cuda(), table, torch.zeros(1, dtype=torch.int32).cuda())
    k, _ = ra.kv_read(c, table, torch.tensor([2], dtype=torch.int32).cuda(), 2)
    want = torch.ones((2, 128))
    want[0, 32:64], want[1, 96:] = math.nan, math.nan
    assert torch.equal(torch.isnan(k[0, :, 0].cpu()), torch.isnan(want)) and (k[0, :, 0].cpu().nan_to_num(1.0) == 1).all()


def test_refusals():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    k = u8(4, 2, 16, 64).view(F4)
    c = ra.make_kv_cache(k, k.clone(), u8(4, 2, 16, 4), u8(4, 2, 16, 4))
    assert (c.D, c.dtype) == (128, ra.RA_E2M1)
    for exps in ((None, None), (u8(4, 2, 16), u8(4, 2, 16)), (u8(4, 2, 16, 4), None)):
        with pytest.raises(ValueError):
            ra.make_kv_cache(k, k.clone(), *exps)
    with pytest.raises(TypeError):
        ra.make_kv_cache(k.view(torch.uint8), k.view(torch.uint8), u8(4, 2, 16, 4), u8(4, 2, 16, 4))
    big = u8(4 * 2 * 16 * 64 + 32)
    odd = big[(16 - big.data_ptr()) % 32:][:4 * 2 * 16 * 64].view(4, 2, 16, 64)  # 16 bytes beside a multiple of 32
    c = ra.make_kv_cache(odd.view(F4), k, u8(4, 2, 16, 4), u8(4, 2, 16, 4))
    with pytest.raises(ra.RaError, match="32-byte"):
        ra.ra_kv_read(c, 4096, 1, 4096, 1, 1, 1 << 20, 1 << 21, ra.RA_BF16, stream=0)
    with pytest.raises(ra.RaError):
        ra.ra_kv_read(ra.RaKvCache(4, 16, 2, 128, ra.RA_E2M1, 4096, 8192, None, None), 4096, 1, 4096, 1, 1, 1 << 20, 1 << 21, ra.RA_BF16, stream=0)
