"""Attention over a cache in 4 bits against the definition in 64 bits: every kernel, its masks and edges.

Bounds are those of an 8-bit cache (tests/test_paged.py, tests/test_paged_accuracy.py): the codes are widened to e4m3 or f16
with a common power of two, exactly for blocks down to 2^-14 of a row's largest (few rows), or 2^-24 of a tile's (many).  Below,
a few-row call's values are off by half a step of e4m3's least, 2^-10, where the row's largest is at least 3 * 2^6: 2^-17 of it."""
import math

import pytest
import torch

import block_sparse_flash_ra_gb300 as ra
from tests import test_paged as tp
from tests import test_paged_accuracy as ta
from tests.test_cache4 import dense, pack, quantise, unpack
from tests.test_paged import CASES, KERNELS, check_attention, each_kernel, each_type, queries

F4, BF = torch.float4_e2m1fn_x2, torch.bfloat16
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


class Pool(tp.Pool):
    """A 4-bit cache with random contents everywhere; blocks of different size in a row."""

    def __init__(self, lens, *, spread=1.0, **kw):
        super().__init__(lens, dtype=BF, **kw)
        g = torch.Generator().manual_seed(kw.get("seed", 0) + 1000)
        q = []
        for t in self.val:
            t = t * torch.exp(spread * torch.randn(t.shape[:-1] + (t.shape[-1] // 32, 1), generator=g)).expand(*t.shape[:-1], -1, 32).flatten(-2)
            q.append(quantise(t))
        self.val = [dense(v, e) for v, e in q]
        self.cache = ra.make_kv_cache(*(pack(v).cuda().view(F4) for v, _ in q), *(e.cuda() for _, e in q))

    def scale(self, which, at, e):
        self.val[which][at] *= 2.0 ** e
        (self.cache.k_exps, self.cache.v_exps)[which][at] += e

    def put(self, which, b, rows):
        """Sets the cached rows of sequence b (None: the prefix) from its first token on; (n, D) or (n, Hkv, D)."""
        at = self.places(b)[:rows.shape[0]]
        at = torch.tensor([p for p, _, _ in at]), slice(None), torch.tensor([o for _, _, o in at])
        x = (rows if rows.dim() == 3 else rows[:, None]).double().expand(self.val[which][at].shape)
        codes, e = quantise(x)
        self.val[which][at] = dense(codes, e)
        pages, exps = ((self.cache.k_pages, self.cache.k_exps), (self.cache.v_pages, self.cache.v_exps))[which]
        pages.view(torch.uint8)[at], exps[at] = pack(codes).cuda(), e.cuda()


def bounds(name, dtype, batch=0):
    return ta.bounds(name, tp.F8, dtype, batch)


# ------------------------------------------------------------- sizes and masks
@gpu
@each_type
@pytest.mark.parametrize("name", CASES)
def test_attention(name, dtype):
    c = dict(dict(Hkv=2, D=128, page=16, Lq=1, prefix=0, sinks=False), **CASES[name])
    pool = Pool(c["lens"], Hkv=c["Hkv"], D=c["D"], page=c["page"], seed=len(name), prefix=c["prefix"])
    g = torch.Generator().manual_seed(len(name) + 1)
    # (blocks up to e^3 as large as 1: logits stay below 64 with queries of this size)
    q = (0.3 * torch.randn((len(c["lens"]), c["Lq"], c["Hq"], c["D"]), generator=g)).to(dtype)
    sinks = torch.randn(c["Hq"], generator=g) if c["sinks"] else None
    check_attention(pool, q, causal=c.get("causal", True), cap=c.get("cap", 0.0), q_len=c.get("q_len"), sinks=sinks)


@gpu
@each_type
@each_kernel
@pytest.mark.parametrize("prefix", [0, 3, 150])
def test_outputs_relative_to_what_they_are_made_of(prefix, name, dtype):
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([1, 2, 3, 5, 9, 17, 40, 129, 300], Hkv=Hkv, D=D, page=32, seed=83, prefix=prefix, spread=0.5)
    q = queries(name, 9, torch.float32, 84).to(dtype)
    scale = ta.f32(D ** -0.5)
    out, _ = ta.forward(pool, q, scale, causal=False)
    for b in range(9):
        assert ta.errors(pool, q[b], out[b], scale, b=b, causal=False, **bounds(name, dtype, 9 if prefix else 0)) <= 1


@gpu
@each_type
@pytest.mark.parametrize("name", ["d64_80", "rows8_8", "rows80", "rows320"])
def test_causal_rows_relative_to_what_they_are_made_of(name, dtype):
    _, Hkv, Lq, D = ta.SHAPES[name]
    pool = Pool([Lq + n for n in (-1, 0, 20, 25, 30, 55, 90, 400)], Hkv=Hkv, D=D, page=32, seed=89, spread=0.5)
    q = torch.randn((8, Lq, ta.SHAPES[name][0], D), generator=torch.Generator().manual_seed(90)).to(dtype)
    scale = ta.f32(D ** -0.5)
    out, _ = ta.forward(pool, q, scale)
    for b in range(8):
        n = min(Lq, pool.lens[b])
        assert (out[b, :Lq - n] == 0).all()
        assert not n or ta.errors(pool, q[b, Lq - n:], out[b, Lq - n:], scale, b=b, **bounds(name, dtype)) <= 1


@gpu
@each_type
@pytest.mark.parametrize("name", ["d64", "rows8", "rows16", "rows20", "rows32", "rows80", "rows320"])
def test_long_contexts(name, dtype):
    _, _, _, D = ta.SHAPES[name]
    for prefix in (0, 77):
        pool = Pool([65537, 40001], Hkv=1, D=D, page=128, seed=85, prefix=prefix, spread=0.5)
        q = (0.5 * queries(name, 2, torch.float32, 86)).to(dtype)
        scale = ta.f32(D ** -0.5)
        out, _ = ta.forward(pool, q, scale)
        for b in (0, 1):
            assert ta.errors(pool, q[b], out[b], scale, b=b, device="cuda", **bounds(name, dtype, 2 if prefix else 0)) <= 1


# ------------------------------------------------------------- scales
@gpu
@each_type
@each_kernel
@pytest.mark.parametrize("which", [0, 1])
def test_blocks_far_apart_in_a_row(which, name, dtype):
    """The blocks of a row 2^0, 2^-7, 2^-14 and 2^-20 as large, in an order that turns from token to token."""
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([300, 40], Hkv=Hkv, D=D, page=32, seed=21, spread=0.0)
    g = torch.Generator().manual_seed(22)
    for b, n in enumerate(pool.lens):
        e = torch.tensor([0.0, -7.0, -14.0, -20.0])[(torch.arange(D // 32) + torch.arange(n)[:, None]) % 4]
        pool.put(which, b, torch.randn((n, D), generator=g) * torch.pow(2.0, e).repeat_interleave(32, -1))
    q = queries(name, 2, torch.float32, 23).to(dtype)
    scale = ta.f32(D ** -0.5)
    out, _ = ta.forward(pool, q, scale, causal=False)
    more = bounds(name, dtype)
    # keys: 32 products of the quiet block, off by 2^-17 of a key's largest, 2^-10 of a logit at most here; values: of p max|v|
    more["share"] += 2.0 ** -10 if which == 0 else 0.0
    more["key"] = max(more["key"], 0.0)
    for b in (0, 1):
        k, v = pool.dense(b)
        got, lim = out[b], dict(more)
        G = q.shape[2] // Hkv
        s = torch.einsum("ihd,jhd->hij", q[b].double(), k.repeat_interleave(G, 1)) * scale
        p = torch.softmax(s, -1)
        vv = v.repeat_interleave(G, 1)
        o = torch.einsum("hij,jhd->ihd", p, vv)
        extra = 2.0 ** -17 * torch.einsum("hij,jh->ih", p, vv.abs().amax(-1))[..., None] if which else 0.0
        tol = ta.allowed(p, vv, o, q.dtype, **lim) + extra
        assert ((got - o).abs() <= tol).all()


@gpu
@each_type
@each_kernel
@pytest.mark.parametrize("way", ["up", "down"])
def test_scales_that_change_along_a_sequence(way, name, dtype):
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([700, 90, 0], Hkv=Hkv, D=D, page=32, seed=31, prefix=333, spread=0.3)
    for b in (None, 0, 1):
        at = pool.places(b)
        for t in range(len(at)):
            x = t if way == "up" else len(at) - 1 - t
            pool.scale(1, at[t], 18 * x // len(at))
            pool.scale(0, at[t], 3 * x // len(at))
    check_attention(pool, queries(name, 3, dtype, 32))


@gpu
@each_type
@each_kernel
def test_scales_at_the_ends_of_their_range(name, dtype):
    """Bytes from 0 on: values around 2^-127 weigh as much as any, and blocks of the least scale beside them."""
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([40], Hkv=Hkv, D=D, page=16, seed=41, spread=0.3)
    up = 100  # what is compared is 2^100 as large: an output of 2^-125 has lost bits in bf16 and fp32
    for e in (0, 1, 5, 6, 7, 20):
        pool.cache.v_exps.copy_(e + torch.arange(D // 32, device="cuda") % 2)
        val = unpack(pool.cache.v_pages.view(torch.uint8).cpu())
        pool.val[1] = dense(val, pool.cache.v_exps.cpu())
        q = queries(name, 1, torch.float32, 42).to(dtype)
        out, _ = ta.forward(pool, q, ta.f32(D ** -0.5), causal=False)
        k, v = pool.dense(0)
        o, _ = tp.attention(q[0].double(), k, v, scale=D ** -0.5, visible=torch.ones((q.shape[1], 40), dtype=torch.bool))
        assert ((out[0] - o) * 2.0 ** up).abs().max() <= 2 ** -7 * float((v * 2.0 ** up).abs().max()) + 2.0 ** (up - 133)


@gpu
@pytest.mark.parametrize("name", ta.FEW)
def test_references_that_rise_with_every_tile(name):
    G, D = ta.FEW[name]
    tile, tiles, step = 128 * 128 // D, 12, 5
    pool = Pool([tile * tiles, tile * tiles - 37], Hkv=2, D=D, page=64, seed=5)
    g = torch.Generator().manual_seed(6)
    rise = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 8, 12, 16, 24])  # what the codes hold
    for b, n in enumerate(pool.lens):
        pool.put(0, b, rise[torch.arange(n) // tile][:, None].expand(n, D))
        pool.put(1, b, torch.randn((n, D), generator=g))
    q = torch.ones((2, 1, 2 * G, D), dtype=BF)
    scale = ta.f32(2 * step * math.log(2) / D)
    out, _ = ta.forward(pool, q, scale)
    for b in (0, 1):
        assert ta.errors(pool, q[b], out[b], scale, b, share=2.0 ** -10) <= 1


@gpu
@each_type
@pytest.mark.parametrize("name", ta.SHAPES)
@pytest.mark.parametrize("low,loud,small", [(18, 0, 9), (22, 0, 9), (23, 6, 9), (20, 20, 12), (16, -9, 20)])
def test_small_weights_of_many_keys(low, loud, small, name, dtype):
    """5000 weights 2^-low of the largest: together they are what comes out."""
    Hq, Hkv, Lq, D = ta.SHAPES[name]
    n, B = 5000, 304
    pool = Pool([n], Hkv=1, D=D, page=64, seed=80)
    g = torch.Generator().manual_seed(80)
    k, v = torch.zeros((n, D)), torch.randn((n, D), generator=g) + 1
    k[0], k[1] = 1.0, -8.0
    v[0], v[1] = v[0] * 2.0 ** -small, v[1] * 2.0 ** loud
    pool.put(0, 0, k)
    pool.put(1, 0, v)
    pool.table, pool.lens = pool.table.expand(B, -1).contiguous(), pool.lens * B
    q = (1 - torch.arange(Hq // Hkv * Lq) % 4 / 16).view(Lq, -1, 1).expand(B, Lq, Hq // Hkv, D).to(dtype)
    scale = ta.f32(low * math.log(2) / D)
    out, _ = ta.forward(pool, q.contiguous(), scale, causal=False)
    assert ta.errors(pool, q[0], out, scale, causal=False, **bounds(name, dtype)) <= 1


@gpu
@each_type
@pytest.mark.parametrize("name", ta.SHAPES)
@pytest.mark.parametrize("far", [20, 26])
def test_values_far_below_the_loudest(far, name, dtype):
    """The one key that counts has values 2^-far of those of another."""
    Hq, Hkv, Lq, D = ta.SHAPES[name]
    pool = Pool([130], Hkv=1, D=D, page=64, seed=93)
    g = torch.Generator().manual_seed(93)
    k, v = torch.full((130, D), -8.0), torch.randn((130, D), generator=g)
    k[3] = 1.0
    v[70] *= 2.0 ** far
    pool.put(0, 0, k)
    pool.put(1, 0, v)
    q = torch.ones((1, Lq, Hq // Hkv, D)).to(dtype)
    scale = ta.f32(100 * math.log(2) / D)
    out, _ = ta.forward(pool, q, scale, causal=False)
    # the other keys' weights are 2^-900: none in fp32, so where the key that counts has a value of 0 so has the output,
    # and 64 bits 2^-900 times theirs; relative to that no output could be right, so the others' values do not count here
    v = pool.val[1][[x for x in pool.places(0)][3]][0]
    assert (out[0][..., v == 0] == 0).all()
    pool.val[1][:, :, :, v == 0] = 0
    assert ta.errors(pool, q[0], out[0], scale, causal=False, **bounds(name, dtype)) <= 1


# ------------------------------------------------------------- what must not count
@gpu
@each_type
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,B", [(2, 2), (16, 9), (24, 3), (48, 3)])
def test_what_lies_behind_a_length_does_not_count(Hq, B, D, dtype):
    lens = [(29 * b + 5) % 70 for b in range(B)]
    pool = Pool(lens, Hkv=1, D=D, page=32, seed=3, prefix=40 if D == 128 else 41, width=6)
    for b in range(B + 1):
        pages, n = (pool.table[b], lens[b]) if b < B else (pool.prefix, pool.prefix_len)
        for t in range(n, -(-n // 32) * 32):
            at = (int(pages[t // 32]), slice(None), t % 32)
            for x, e in ((pool.cache.k_pages, pool.cache.k_exps), (pool.cache.v_pages, pool.cache.v_exps)):
                x.view(torch.uint8)[at] = 0x7f if t % 2 else 0xff
                e[at] = 255 if t % 3 else 254
    q = (0.5 * torch.randn((B, 1, Hq, D), generator=torch.Generator().manual_seed(4))).to(dtype)
    check_attention(pool, q)


@gpu
@each_type
@each_kernel
def test_a_block_without_a_value_reaches_its_own_values(name, dtype):
    """A value block of NaN reaches its 32 values of the rows that see it; a key's, all of them."""
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([40, 40, 40], Hkv=Hkv, D=D, page=16, seed=5)
    for which, b in ((1, 1), (0, 2)):
        exps = (pool.cache.k_exps, pool.cache.v_exps)[which]
        exps[int(pool.table[b, 0]), :, 3, 1] = 255
        (pool.cache.k_pages, pool.cache.v_pages)[which].view(torch.uint8)[int(pool.table[b, 0]), :, 3, 16:32] = 0
    q = queries(name, 3, dtype, 6)
    out, lse = ta.forward(pool, q, 0.1, causal=False)
    assert torch.isfinite(out[0]).all() and torch.isfinite(lse[:2]).all()
    bad = torch.zeros(D, dtype=torch.bool)
    bad[32:64] = True
    assert torch.isnan(out[1][..., bad]).all() and torch.isfinite(out[1][..., ~bad]).all()
    assert torch.isnan(out[2]).all() and torch.isnan(lse[2]).all()


@gpu
@each_type
@pytest.mark.parametrize("Hq,Hkv,Lq,D", [(1, 1, 3, 128), (2, 2, 4, 128), (4, 2, 4, 128), (2, 1, 7, 128), (4, 1, 6, 128), (8, 1, 4, 128), (8, 1, 10, 128),
                                         (16, 1, 18, 128), (1, 1, 2, 64), (4, 2, 2, 64), (3, 1, 4, 64), (8, 1, 5, 64)])
def test_a_block_without_a_value_does_not_reach_rows_before_it(Hq, Hkv, Lq, D, dtype):
    """The drafts' own last tokens hold value blocks of NaN: queries before them see none of it, those behind all."""
    lens = [130, 41, 300, Lq]
    pool = Pool(lens, Hkv=Hkv, D=D, page=16, seed=37, spread=0.5)
    gone = [(0, 2, 1), (1, 1, 0), (1, 2, 1), (2, 1, 1), (2, 1, 0), (3, 2, 0)]  # sequence, tokens from its end, block
    for b, back, x in gone:
        page, _, at = pool.places(b)[lens[b] - back]
        pool.val[1][page, :, at, 32 * x:32 * x + 32] = 0
        pool.cache.v_exps[page, :, at, x] = 255
        pool.cache.v_pages.view(torch.uint8)[page, :, at, 16 * x:16 * x + 16] = 0
    q = torch.randn((4, Lq, Hq, D), generator=torch.Generator().manual_seed(38)).to(dtype)
    scale = ta.f32(D ** -0.5)
    out, lse = ta.forward(pool, q, scale)
    assert torch.isfinite(lse).all()
    bound = ta.BOUNDS["fp32" if dtype == torch.float32 else "rows8" if D == 128 and Lq * Hq // Hkv > 32 else "few8"]
    for b in range(4):
        sees = torch.zeros((Lq, Hq, D), dtype=torch.bool)
        for _, back, x in [g for g in gone if g[0] == b]:
            sees[Lq - back:, :, 32 * x:32 * x + 32] = True  # query i sees tokens up to Lq - 1 - i from the end
        assert torch.equal(torch.isnan(out[b].cpu()), sees)
        k, v = (t.repeat_interleave(Hq // Hkv, 1) for t in pool.dense(b))
        s = torch.einsum("ihd,jhd->hij", q[b].double(), k) * scale
        s = s.masked_fill(torch.arange(lens[b]) > torch.arange(Lq)[:, None] + lens[b] - Lq, -math.inf)
        p = torch.softmax(s, -1)
        o = torch.einsum("hij,jhd->ihd", p, v)
        near = (out[b].cpu() - o).abs() <= ta.allowed(p, v, o, dtype, **bound)
        assert (near | sees).all()


@gpu
@each_type
@pytest.mark.parametrize("Hq,Hkv,Lq,D,B,prefix", [(2, 1, 2, 128, 4000, 0), (4, 2, 4, 128, 2000, 0), (4, 1, 8, 128, 2000, 70), (8, 1, 10, 128, 2000, 0),
                                                  (16, 1, 18, 128, 2000, 0), (2, 1, 3, 64, 4000, 0), (8, 1, 20, 64, 700, 0), (8, 1, 4, 128, 3, 0), (4, 2, 2, 64, 3, 40)])
def test_blocks_without_values_of_many_sequences(Hq, Hkv, Lq, D, B, prefix, dtype):
    """Some of many sequences have them, anywhere, and one of three tokens of a prefix: the rows that see them and no others."""
    g = torch.Generator().manual_seed(39)
    lens = [Lq + int(x) for x in torch.randint(0, 40 if B > 3 else 3000, (B,), generator=g)]
    page, n = 16, [-(-x // 16) for x in lens]
    of = -(-prefix // page)
    cache = ra.new_kv_cache(sum(n) + of, page, Hkv, D, F4)
    for codes, exps in ((cache.k_pages, cache.k_exps), (cache.v_pages, cache.v_exps)):
        codes.view(torch.uint8).copy_(torch.randint(0, 256, codes.shape, generator=g, dtype=torch.uint8))
        exps.copy_(torch.randint(124, 127, exps.shape, generator=g, dtype=torch.uint8))
    table, at = torch.zeros((B, max(n)), dtype=torch.int32), of
    for b in range(B):
        table[b, :n[b]] = torch.arange(at, at + n[b])
        at += n[b]
    # first[b, x]: the first token without a value in block x, or 2^30
    first = torch.full((B, D // 32), 1 << 30)
    picked = torch.randperm(B, generator=g)[:max(B // 3, 2)].tolist()
    gone = []
    for b in picked:
        for _ in range(2):
            t, x = max(lens[b] - 1 - int(torch.randint(0, Lq + 3, (1,), generator=g)), 0), int(torch.randint(0, D // 32, (1,), generator=g))
            first[b, x] = min(int(first[b, x]), t)
            gone.append((int(table[b, t // page]), t % page, x))
    if prefix:
        first[:, 1] = -1
        gone.append((1, 2, 1))
    i = [torch.tensor(v) for v in zip(*gone)]
    where = (i[0].cuda(), slice(None), i[1].cuda())
    q = torch.randn((B, Lq, Hq, D), generator=g).to(dtype).cuda()
    p = ra.make_paged_params(cache, q, table.cuda(), i32(lens), scale=0.05, prefix_table=i32(list(range(of))) if prefix else None,
                             prefix_len=i32([prefix]) if prefix else None)
    got = []
    for e in (0, 255):
        codes = cache.v_pages.view(torch.uint8).view(*cache.v_pages.shape[:3], D // 32, 16)
        codes[where + (i[2].cuda(),)] = 0
        cache.v_exps[where + (i[2].cuda(),)] = e
        got.append(ra.paged_forward(p, q, cache)[0].cpu().float().view(B, Lq, Hq, D // 32, 32))
    sees = first[:, None] <= torch.tensor(lens)[:, None, None] - Lq + torch.arange(Lq)[None, :, None]
    assert torch.isfinite(got[0]).all()
    assert torch.equal(torch.isnan(got[1]), sees[:, :, None, :, None].expand(got[1].shape))
    # each is off by half a step of its type and 2^-10 of values of 6 * 2^-1 at the most
    off = torch.where(torch.isnan(got[1]), 0.0, (got[1] - got[0]).abs())
    assert float(off.max()) <= 2 * 3.0 * (torch.finfo(dtype).eps / 2 + 2.0 ** -10)


@gpu
@each_type
@each_kernel
def test_pages_out_of_range(name, dtype):
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([300, 130, 64], Hkv=Hkv, D=D, page=32, seed=33, prefix=200)
    table, prefix = pool.table.clone(), pool.prefix.clone()
    for b, i, number in ((0, 0, -1), (0, 5, pool.n), (1, 4, 2 ** 31 - 1), (2, 1, -2 ** 31), (None, 2, 1 << 20), (None, 6, -5)):
        pages, given = (pool.prefix, prefix) if b is None else (pool.table[b], table[b])
        for w in (0, 1):
            pool.val[w][int(pages[i])] = 0
        given[i] = number
    pool.given = table, prefix
    check_attention(pool, (0.5 * queries(name, 3, torch.float32, 34)).to(dtype))
    assert ra.ra_get_device_status() == ra.RA_ERR_INVALID_ARG
    assert ra.ra_get_device_status() == ra.RA_OK


@gpu
@each_type
@each_kernel
def test_sinks_of_minus_infinity(name, dtype):
    Hq, Hkv, Lq, D = KERNELS[name]
    pool = Pool([0, 50], Hkv=Hkv, D=D, page=16, seed=7)
    q = (0.5 * queries(name, 2, torch.float32, 8)).to(dtype)
    out, lse = ta.forward(pool, q, 0.1, sinks=torch.full((Hq,), -math.inf).cuda(), causal=False)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and torch.isfinite(out[1]).all()


# ------------------------------------------------------------- large caches, graphs, streams
@gpu
@each_type
@pytest.mark.parametrize("Hq,Lq", [(8, 1), (80, 8)])
def test_offsets_beyond_32_bits(Hq, Lq, dtype):
    """A cache of 4.4 GB of codes per tensor: the same tokens in its first and in its last pages."""
    page, n = 128, 68000
    c = ra.new_kv_cache(n, page, 8, 128, F4)
    g = torch.Generator().manual_seed(41)
    low = torch.arange(6, dtype=torch.int32).view(2, 3)
    lens = [3 * page - 5, page + 1]
    k, v = (torch.randn((2, 3 * page, 8, 128), generator=g).to(dtype).cuda() for _ in range(2))
    q = torch.randn((2, Lq, Hq, 128), generator=g).to(dtype).cuda()
    got = []
    for table in (low.cuda(), (n - 1 - low).cuda()):
        ra.kv_write(c, k, v, table, i32([0, 0]), i32(lens))
        p = ra.make_paged_params(c, q, table, i32(lens), scale=0.1, prefix_table=table[0, :2].contiguous(), prefix_len=i32([page + 3]))
        got.append(ra.kv_read(c, table, i32(lens), 3 * page) + ra.paged_forward(p, q, c))
    assert c.k_pages.view(torch.uint8)[n - 1].sum() > 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


@gpu
@each_kernel
def test_a_graph_serves_lengths_that_change(name):
    Hq, Hkv, Lq, D = KERNELS[name]
    pool = Pool([400, 90, 64], Hkv=Hkv, D=D, page=32, seed=43, prefix=333)
    kv, q_len, plen = i32([1, 90, 0]), i32([Lq, Lq, Lq]), i32([0])
    q = (0.5 * queries(name, 3, torch.float32, 44)).to(BF).cuda()
    p = ra.make_paged_params(pool.cache, q, pool.table.cuda(), kv, scale=D ** -0.5, q_len=q_len, prefix_table=pool.prefix.cuda(),
                             prefix_len=plen)
    ws = torch.empty(ra.ra_attn_paged_workspace_size(pool.cache, p), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((3, Hq, Lq), device="cuda")
    ra.paged_forward(p, q, pool.cache, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.paged_forward(p, q, pool.cache, out=out, lse=lse, ws=ws)
    for lens, n_q, prefix in (([1, 90, 0], Lq, 0), ([400, 3, 64], Lq, 333), ([0, 0, 0], Lq, 0), ([0, 0, 0], Lq, 16), ([129, 90, 1], 0, 200),
                              ([257, 1, 64], 1, 128)):
        kv.copy_(i32(lens))
        q_len.fill_(n_q)
        plen.fill_(prefix)
        out.fill_(7)
        lse.fill_(9)
        graph.replay()
        want = ra.paged_forward(p, q, pool.cache, out=torch.full_like(out, 7), lse=torch.full_like(lse, 9))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        pool.lens, pool.prefix_len = lens, prefix
        if prefix == 0:
            check_attention(pool, q.cpu(), q_len=[n_q] * 3)


@gpu
def test_calls_on_several_streams():
    jobs = []
    for i, name in enumerate(KERNELS):
        _, Hkv, _, D = KERNELS[name]
        pool = Pool([(97 * b + 11 * i) % 600 for b in range(24)], Hkv=Hkv, D=D, page=32, seed=50 + i, prefix=300)
        q = queries(name, 24, BF, 60 + i).cuda()
        p = ra.make_paged_params(pool.cache, q, pool.table.cuda(), i32(pool.lens), scale=D ** -0.5,
                                 prefix_table=pool.prefix.cuda(), prefix_len=i32([300]))
        jobs.append((torch.cuda.Stream(), p, q, pool.cache, ra.paged_forward(p, q, pool.cache)))
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for s, p, q, c, _ in jobs:
            with torch.cuda.stream(s):
                got.append(ra.paged_forward(p, q, c))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        want = jobs[i % len(jobs)][4]
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------- together, as a server uses them
@gpu
@pytest.mark.parametrize("kind", [F4, torch.float8_e4m3fn, BF], ids=["e2m1", "e4m3", "c16"])
def test_tokens_enter_and_are_attended(kind):
    """Projections' outputs are normalised, rotated and put into the cache, and attended: a prompt, then tokens one at a time
    in a captured step.  Against the attention in 64 bits over what the cache holds."""
    B, Hq, Hkv, D, page, L, steps = 3, 8, 2, 128, 32, 70, 5
    g = torch.Generator().manual_seed(11)
    cache = ra.new_kv_cache(16, page, Hkv, D, kind)
    table = torch.randperm(16, generator=g)[:12].to(torch.int32).view(B, 4).cuda()
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(BF).cuda() for _ in range(2))
    rope = ra.make_rope(64, 500000.0, scaling="yarn", factor=4.0, trained_length=4096)
    start, kv_len = i32([0, 0, 0]), i32([0, 0, 0])
    count = i32([70, 33, 1])
    kw = dict(rope=rope, eps=1e-6, q_weight=wq, k_weight=wk, start=start)

    def reference(out, q, n):
        lens = kv_len.tolist()
        k, v = ra.kv_read(cache, table, kv_len, max(lens), torch.float32)
        for b in range(B):
            m = n[b]
            i, j = torch.arange(m)[:, None], torch.arange(lens[b])
            o, _ = tp.attention(q[b, :m].cpu().double(), k[b, :lens[b]].cpu().double(), v[b, :lens[b]].cpu().double(), scale=D ** -0.5,
                                visible=j <= i + lens[b] - m)
            assert (out[b, :m].cpu().double() - o).abs().max() <= 2 ** -7 * float(v[b].abs().max())

    x = torch.randn((B, L, Hq + 2 * Hkv, D), generator=g).to(BF).cuda()
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    params = ra.make_qk_params(q, k, **kw)
    out = ra.qk_enter(params, cache, q, k, v, table, count=count)
    kv_len += count
    pp = ra.make_paged_params(cache, out, table, kv_len, scale=D ** -0.5, q_len=count)
    reference(ra.paged_forward(pp, out, cache)[0], out, count.tolist())
    start.copy_(kv_len)

    x = torch.empty((B, 1, Hq + 2 * Hkv, D), dtype=BF, device="cuda")
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    params = ra.make_qk_params(q, k, **kw)
    turned, y, lse = torch.empty((B, 1, Hq, D), dtype=BF, device="cuda"), torch.empty((B, 1, Hq, D), dtype=BF, device="cuda"), None
    pp = ra.make_paged_params(cache, turned, table, kv_len, scale=D ** -0.5)
    ws = torch.empty(ra.ra_attn_paged_workspace_size(cache, pp), dtype=torch.uint8, device="cuda")
    lse = torch.empty((B, Hq, 1), device="cuda")

    def step():
        ra.qk_enter(params, cache, q, k, v, table, out=turned)
        kv_len.add_(1)
        ra.paged_forward(pp, turned, cache, out=y, lse=lse, ws=ws)
        start.add_(1)

    state = [t.clone() for t in (start, kv_len)]
    x.normal_()
    step()  # a first run outside the graph
    for t, s in zip((start, kv_len), state):
        t.copy_(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((start, kv_len), state):
        t.copy_(s)
    for _ in range(steps):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        reference(y, turned, [1] * B)
        want = ra.qk_forward(ra.make_qk_params(q, k, rope=rope, eps=1e-6, q_weight=wq, k_weight=wk, start=start - 1), q, k)
        assert torch.equal(turned, want[0])
        kk, _ = ra.kv_read(cache, table, kv_len, int(kv_len.max()))
        if kind == BF:
            for b in range(B):
                assert torch.equal(kk[b, int(kv_len[b]) - 1], want[1][b, 0])


@gpu
def test_a_layer_is_trained():
    """Norm, rotation and the dense attention, forward and backward, against autograd in 64 bits."""
    B, L, Hq, Hkv, D = 1, 256, 4, 2, 64
    g = torch.Generator().manual_seed(12)
    q, k, v, do = (torch.randn((B, L, h, D), generator=g) for h in (Hq, Hkv, Hkv, Hq))
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    rope = ra.make_rope(D)
    p = ra.make_qk_params(q.cuda(), k.cuda(), rope=rope, eps=1e-6, q_weight=wq.cuda(), k_weight=wk.cuda())
    tq, tk = ra.qk_forward(p, q.cuda(), k.cuda())
    ap = ra.make_params(tq, tk, scale=D ** -0.5, causal=True)
    mask = ra.build_mask(ap)
    out, lse = ra.forward(ap, tq, tk, v.cuda(), mask)
    dq, dk, _, _ = ra.backward(ap, tq, tk, v.cuda(), out, lse, do.cuda(), mask)
    grads = ra.qk_backward(p, q.cuda(), k.cuda(), dq, dk)
    from tests.test_qk import forward64, frequencies
    leaves = [t.double().requires_grad_() for t in (q, k, wq, wk)]
    pos = torch.arange(L)[None]
    a, b = (forward64(x, pos, frequencies(D), False, 1.0, w, 1e-6)[0] for x, w in ((leaves[0], leaves[2]), (leaves[1], leaves[3])))
    s = torch.einsum("ihd,jhd->hij", a, b.repeat_interleave(2, 1)) * D ** -0.5
    s = s.masked_fill(torch.arange(L) > torch.arange(L)[:, None], -math.inf)
    o = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v[0].double().repeat_interleave(2, 1))
    o.backward(do[0].double())
    for got, leaf in zip(grads, leaves):
        # the dense backward's products read bf16 copies: 2^-8 of each factor, 1e-2 of the norm in its own tests
        assert (got.cpu().double() - leaf.grad).norm() <= 1e-2 * leaf.grad.norm()
