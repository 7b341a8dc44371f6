"""The paged cache and the attention over it against the definitions in 64 bits.

Tolerances.  An e4m3 code is off by half a step, 2^-4 relative (2^-10 of 2^e below the normal range); reading back is
exact, up to the output type's own rounding (bf16: 2^-8).  Attention: an output is a mean of values with weights that
sum to 1.  fp32 arithmetic: a logit of D products is off by about D * 2^-24 of sum |q k| * scale, at most 2^-17 * 64 for
the inputs here (|s| <= sum |q k| scale < 64), so weights and lse are off by 5e-4 at worst and about 1e-5 in practice;
bounds: lse 1e-4, out 1e-4 of the largest value.  bf16 outputs and 16-bit weights add half a step each: 2^-8 of the
row's largest value for the output's rounding and 2^-8 of a mean of values for the weights', 2^-7 together.
"""
import math

import pytest
import torch

import block_sparse_flash_ra_gb300 as ra

F8 = torch.float8_e4m3fn
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_flash_ra_gb300 import _build
    _build.build()
    yield
    if torch.cuda.is_available():
        torch.cuda.synchronize()
        assert ra.ra_get_device_status() == ra.RA_OK


# ------------------------------------------------------------- definitions in 64 bits
def e4m3(y):
    """fp64 -> nearest e4m3 value (ties to even)."""
    step = torch.pow(2.0, torch.floor(torch.log2(y.abs())).clamp(min=-6) - 3)
    return torch.round(y / step) * step


def quantise(x):
    """fp64 rows -> (codes' values, exponent byte)."""
    amax = x.abs().amax(-1)
    e = torch.ceil(torch.log2(amax / 448)).clamp(min=-110)
    good = torch.isfinite(amax)
    e = torch.where(good, e, 128.0)
    codes = e4m3(x / torch.pow(2.0, e)[..., None])
    return torch.where(good[..., None], codes, 0.0), (e + 127).to(torch.uint8)


def attention(q, k, v, *, scale, visible, cap=0.0, sinks=None):
    """q (n, Hq, D), k / v (m, Hkv, D), visible (n, m) -> out (n, Hq, D), lse (Hq, n); fp64."""
    n, Hq, D = q.shape
    k, v = (t.repeat_interleave(Hq // t.shape[1], 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, k) * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    s = s.masked_fill(~visible, -math.inf)
    if sinks is not None:
        s = torch.cat([s, sinks[:, None, None].expand(Hq, n, 1)], -1)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else s.new_full((Hq, n), -math.inf)
    p = torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[..., None])[..., :k.shape[0]]
    v = torch.where(visible.any(0)[:, None, None], v, 0.0)  # values that no row sees do not count
    return torch.einsum("hij,jhd->ihd", p, v), lse


class Pool:
    """A cache with random contents everywhere, and shuffled tables for given lengths."""

    def __init__(self, lens, *, Hkv=2, D=128, page=16, dtype=F8, seed=0, spare=3, prefix=0, width=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        n_prefix = -(-prefix // page)
        self.n = sum(need) + n_prefix + spare
        order = torch.randperm(self.n, generator=g)
        self.table = torch.full((len(lens), width or max([1] + need)), -7, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.prefix = order[at:at + n_prefix].to(torch.int32)
        self.page, self.lens, self.prefix_len = page, list(lens), prefix
        self.given = None  # the tables that a call gets, where they differ
        x = [torch.randn((self.n, Hkv, page, D), generator=g) * torch.exp(torch.randn((self.n, Hkv, page, 1), generator=g) * 0.3)
             for _ in range(2)]
        if dtype == F8:
            q = [quantise(t.double()) for t in x]
            self.val = [c * torch.pow(2.0, e.double() - 127)[..., None] for c, e in q]
            self.cache = ra.make_kv_cache(*(c.float().to(F8).cuda() for c, _ in q), *(e.cuda() for _, e in q))
        else:
            x = [t.to(torch.bfloat16) for t in x]
            self.val = [t.double() for t in x]
            self.cache = ra.make_kv_cache(*(t.cuda() for t in x))

    def places(self, b):
        """(page, offset) of sequence b's tokens, or of the prefix's for b = None."""
        pages, n = (self.prefix, self.prefix_len) if b is None else (self.table[b], self.lens[b])
        return [(int(pages[t // self.page]), slice(None), t % self.page) for t in range(n)]

    def scale(self, which, at, e):
        """Multiplies a token's row by 2^e."""
        self.val[which][at] *= 2.0 ** e
        pages, exps = ((self.cache.k_pages, self.cache.k_exps), (self.cache.v_pages, self.cache.v_exps))[which]
        if exps is None:
            pages[at] = self.val[which][at].to(torch.bfloat16).cuda()
        else:
            exps[at] += e

    def rows(self, which, pages, n):
        t = self.val[which][pages.long()]  # pages, Hkv, page, D
        return t.permute(0, 2, 1, 3).reshape(-1, t.shape[1], t.shape[3])[:n]

    def dense(self, b):
        used = self.table[b, :-(-self.lens[b] // self.page)]
        return [torch.cat([self.rows(w, self.prefix, self.prefix_len), self.rows(w, used, self.lens[b])]) for w in (0, 1)]


def check_attention(pool, q, *, causal=True, cap=0.0, q_len=None, sinks=None, seed=0, out=None, lse=None):
    B, Lq, Hq, D = q.shape
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    lens = torch.tensor(pool.lens, dtype=torch.int32)
    p = ra.make_paged_params(
        pool.cache, q.cuda(), (pool.given or (pool.table, pool.prefix))[0].cuda(), lens.cuda(), scale=D ** -0.5, causal=causal,
        soft_cap=cap, q_len=dev(None if q_len is None else torch.tensor(q_len, dtype=torch.int32)), sinks=dev(sinks),
        prefix_table=dev((pool.given or (pool.table, pool.prefix))[1]) if pool.prefix_len else None,
        prefix_len=torch.tensor([pool.prefix_len], dtype=torch.int32).cuda() if pool.prefix_len else None)
    ws = torch.full((ra.ra_attn_paged_workspace_size(pool.cache, p),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0).cuda()
    lse = torch.full((B, Hq, Lq), 9.0, device="cuda")
    ra.paged_forward(p, q.cuda(), pool.cache, out=out, lse=lse, ws=ws)
    again = ra.paged_forward(p, q.cuda(), pool.cache)
    out, lse = out.cpu(), lse.cpu()
    for b in range(B):
        n = Lq if q_len is None else q_len[b]
        assert torch.equal(again[0].cpu()[b, :n], out[b, :n]) and torch.equal(again[1].cpu()[b, :, :n], lse[b, :, :n])
        assert (out[b, n:] == 7).all() and (lse[b, :, n:] == 9).all(), "rows behind the last query were written"
        if n == 0:
            continue
        k, v = pool.dense(b)
        j = torch.arange(k.shape[0]) - pool.prefix_len
        last = torch.arange(n)[:, None] + (pool.lens[b] - n) if causal else torch.full((n, 1), 1 << 40)
        vis = (j <= last) | (j < 0)
        o, e = attention(q[b, :n].double(), k, v, scale=D ** -0.5, visible=vis, cap=cap,
                         sinks=None if sinks is None else sinks.double())
        got_o, got_e = out[b, :n].double(), lse[b, :, :n].double()
        fin = torch.isfinite(e)
        assert torch.equal(fin, torch.isfinite(got_e)) and torch.equal(e[~fin], got_e[~fin])
        if fin.any():
            assert (got_e[fin] - e[fin]).abs().max() <= 1e-4
        tol = (1e-4 if q.dtype == torch.float32 else 2 ** -7) * max(1.0, float(v.abs().max()) if v.numel() else 1.0)
        assert (got_o - o).abs().max() <= tol


# ------------------------------------------------------------- write and read
@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cache", [F8, torch.bfloat16])
@pytest.mark.parametrize("B,L,Hkv,D,page", [(1, 1, 1, 64, 16), (3, 37, 3, 128, 16), (2, 130, 2, 64, 128), (5, 1, 8, 128, 64)])
def test_write_then_read(B, L, Hkv, D, page, cache, dtype):
    g = torch.Generator().manual_seed(B * L)
    start = [(11 * b) % 40 for b in range(B)]
    count = [L - (b * 7) % (L + 1) if b else L for b in range(B)]
    width = -(-(max(start) + L) // page)
    n = B * width + 2
    table = torch.randperm(n, generator=g)[:B * width].to(torch.int32).view(B, width)
    fused = torch.randn((B, L, 2 * Hkv + 1, D), generator=g) * torch.exp(3 * torch.randn((B, L, 2 * Hkv + 1, 1), generator=g))
    fused[0, 0, 1] = 0.0  # a row of zeros
    fused[-1, -1, 1, 3] = 448.0 * 4
    fused = fused.to(dtype).cuda()
    c = ra.new_kv_cache(n, page, Hkv, D, cache)
    before = torch.randint(0, 255, (n, Hkv, page, D), generator=g, dtype=torch.uint8) % 0x70
    for t in (c.k_pages, c.v_pages):
        t.view(torch.uint8)[..., :D].copy_(before.cuda())
    old = c.k_pages.clone().view(torch.uint8)
    k, v = fused[:, :, 1:1 + Hkv], fused[:, :, 1 + Hkv:]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    ra.kv_write(c, k, v, table.cuda(), i32(start), i32(count))
    touched = torch.zeros((n, Hkv, page), dtype=torch.bool)
    for src, pages, exps in ((k, c.k_pages, c.k_exps), (v, c.v_pages, c.v_exps)):
        pages = pages.cpu()
        for b in range(B):
            for i in range(count[b]):
                at = (int(table[b, (start[b] + i) // page]), slice(None), (start[b] + i) % page)
                touched[at] = True
                x = src[b, i].cpu().double()
                if cache == F8:
                    want, e = quantise(x)
                    assert torch.equal(exps.cpu()[at], e)
                    assert torch.equal(pages[at].double(), want)
                else:
                    assert torch.equal(pages[at], x.float().to(torch.bfloat16))
    same = c.k_pages.view(torch.uint8).cpu().view(n, Hkv, page, -1) == old.cpu().view(n, Hkv, page, -1)
    assert same[~touched].all(), "bytes outside the written tokens changed"
    # a dense copy, rows behind the length zero
    reach = max(start) + L + 3
    lens = [start[b] + count[b] for b in range(B)]
    for out_dt in (torch.bfloat16, torch.float32):
        kk, vv = ra.kv_read(c, table.cuda(), i32(lens), reach, out_dt)
        for got, pages, exps in ((kk, c.k_pages, c.k_exps), (vv, c.v_pages, c.v_exps)):
            val = pages.cpu().double()
            if cache == F8:
                val = val * torch.pow(2.0, exps.cpu().double() - 127)[..., None]
            for b in range(B):
                t = val[table[b].long()].permute(0, 2, 1, 3).reshape(-1, Hkv, D)[:lens[b]]
                assert torch.equal(got[b, :lens[b]].cpu(), t.to(out_dt))
                assert (got[b, lens[b]:] == 0).all()


@gpu
def test_quantised_row_extremes():
    c = ra.new_kv_cache(1, 16, 1, 64)
    x = torch.zeros((1, 12, 1, 64))
    x[0, 1, 0, 5] = float("inf")
    x[0, 2, 0, 5] = float("nan")
    x[0, 3] = 1e-45                     # far below the smallest scale: codes of 0
    x[0, 4, 0, :2] = torch.tensor([448.0, -448.0])
    x[0, 5, 0, :2] = torch.tensor([448.0001, 1.0])
    x[0, 6] = 3.4028234e38              # rounds up to 2^128: an infinity when it is read
    x[0, 7, 0, 0], x[0, 7, 0, 1] = 256.0, 2.0 ** -10     # at half the smallest step: ties to 0
    x[0, 8, 0, 0], x[0, 8, 0, 1] = 256.0, 3 * 2.0 ** -11  # above it
    x[0, 9] = -2.0 ** -110
    x[0, 10, 0, 0] = float("-inf")
    x[0, 11, 0, 63] = 1e30
    one = torch.zeros(1, dtype=torch.int32).cuda()
    ra.kv_write(c, x.cuda(), (-x).cuda(), torch.zeros((1, 1), dtype=torch.int32).cuda(), one)
    e = c.k_exps[0, 0].cpu()
    codes = c.k_pages[0, 0].cpu().double()
    assert e.tolist()[:3] == [17, 255, 255] and e[10] == 255 and e[3] == 17 and e[4] == 127 and e[5] == 128
    assert (codes[[0, 1, 2, 3, 10]] == 0).all()
    assert codes[4, 0] == 448 and codes[4, 1] == -448 and codes[5, 0] == 224
    assert codes[7, 1] == 0 and codes[8, 1] == 2.0 ** -9
    assert (codes[9] == -1).all() and e[9] == 17
    k, v = ra.kv_read(c, torch.zeros((1, 1), dtype=torch.int32).cuda(), one + 12, 16, torch.float32)
    k, v = k[0, :, 0].cpu(), v[0, :, 0].cpu()
    assert torch.isnan(k[[1, 2, 10]]).all() and torch.isinf(k[6]).all() and (k[12:] == 0).all()
    good = [0, 3, 4, 5, 7, 8, 9, 11]
    assert torch.equal(k[good], -v[good])
    assert abs(float(k[11, 63]) - 1e30) <= 2 ** -4 * 1e30


@gpu
def test_out_of_range_places_are_skipped_and_reported():
    c = ra.new_kv_cache(4, 16, 1, 64, torch.bfloat16)
    c.k_pages.fill_(5.0)
    x = torch.ones((2, 40, 1, 64), dtype=torch.bfloat16).cuda()
    table = torch.tensor([[0, 9, 1], [2, -1, 3]], dtype=torch.int32).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    ra.kv_write(c, x, x, table, i32([-3, 20]))
    assert ra.ra_get_device_status() == ra.RA_ERR_INVALID_ARG
    got = c.k_pages[:, 0, :, 0].cpu()
    want = torch.full((4, 16), 5.0)
    want[0] = 1.0               # positions -3 .. 36 of sequence 0: pages 0, 9 (bad), 1
    want[1, :5] = 1.0
    want[3] = 1.0               # positions 20 .. 59 of sequence 1: page -1 (bad), 3, past the table
    assert torch.equal(got.float(), want)
    k, _ = ra.kv_read(c, table, i32([48, 99]), 64)
    assert ra.ra_get_device_status() == ra.RA_ERR_INVALID_ARG
    assert (k[0, 16:32] == 0).all() and (k[1, 16:32] == 0).all() and (k[1, 48:] == 0).all() and (k[0, :16] == 1).all()
    q = torch.ones((2, 1, 1, 64), dtype=torch.bfloat16).cuda()
    p = ra.make_paged_params(c, q, table, i32([48, -1]), scale=1.0)
    o, lse = ra.paged_forward(p, q, c)
    assert ra.ra_get_device_status() == ra.RA_ERR_INVALID_ARG
    assert torch.isfinite(o).all() and lse[1, 0, 0] == -math.inf and (o[1] == 0).all()
    assert ra.ra_get_device_status() == ra.RA_OK


# ------------------------------------------------------------- attention
CASES = {
    "one_key": dict(lens=[1], Hq=2),
    "one_key_d64": dict(lens=[1, 0, 2, 3], Hq=2, D=64),
    "tile_edges_d64": dict(lens=[255, 256, 257, 511, 513, 128, 127], Hq=16, D=64, page=128),
    "long_split_d64": dict(lens=[9001], Hq=8, D=64, page=64),
    "chunk_d64": dict(lens=[200, 151], Hq=4, Lq=150, D=64),
    "draft_ragged_d64": dict(lens=[70, 3, 129, 20], Hq=4, Lq=5, q_len=[5, 1, 0, 4], D=64, sinks=True),
    "nothing_cached": dict(lens=[0, 5, 0], Hq=2),
    "page_edges": dict(lens=[15, 16, 17, 31, 32, 33], Hq=4),
    "page128": dict(lens=[127, 128, 129, 300], Hq=4, page=128),
    "page64_d64": dict(lens=[63, 64, 65, 200], Hq=6, D=64, page=64, Hkv=3),
    "page32_mha": dict(lens=[100, 1, 257], Hq=5, Hkv=5, page=32),
    "mqa32": dict(lens=[513, 40], Hq=32, Hkv=1, page=32),
    "group17": dict(lens=[130], Hq=17, Hkv=1),
    "long_split": dict(lens=[5000], Hq=8, page=64),
    "many_short": dict(lens=[(37 * b) % 91 for b in range(150)], Hq=4),
    # several segments to a CTA, for each size of row block; blocks of one tile and of two
    "many_short_16": dict(lens=[(37 * b) % 91 for b in range(330)], Hq=16, Hkv=1),
    "many_short_24": dict(lens=[(29 * b) % 140 for b in range(330)], Hq=24, Hkv=1, page=32),
    "many_short_12_d64": dict(lens=[(29 * b) % 280 for b in range(330)], Hq=12, Hkv=1, D=64, page=32),
    "many_short_32": dict(lens=[(31 * b) % 140 for b in range(330)], Hq=32, Hkv=1, page=32),
    "many_short_64": dict(lens=[(37 * b) % 191 for b in range(200)], Hq=8, Lq=16),
    "many_short_200": dict(lens=[60 + (37 * b) % 91 for b in range(110)], Hq=8, Lq=50),
    "many_short_d64": dict(lens=[(37 * b) % 91 for b in range(200)], Hq=24, Hkv=2, D=64),
    "many_700": dict(lens=[(37 * b) % 23 for b in range(700)], Hq=2, Hkv=1),
    "many_behind_a_prefix": dict(lens=[(37 * b) % 23 for b in range(300)], Hq=2, Hkv=1, prefix=100, q_len=[b % 2 for b in range(300)]),
    "many_few_rows": dict(lens=[(37 * b) % 23 for b in range(140)], Hq=1, Hkv=1, D=64, sinks=True),
    "long_40_rows": dict(lens=[3100, 2500, 1], Hq=8, Lq=10, page=128),
    "draft": dict(lens=[70, 3, 129, 0], Hq=4, Lq=5),
    "draft_full": dict(lens=[70, 3, 129], Hq=4, Lq=3, causal=False),
    "draft_ragged": dict(lens=[70, 3, 129, 20], Hq=4, Lq=5, q_len=[5, 1, 0, 4]),
    "chunk": dict(lens=[200, 150], Hq=4, Lq=150),
    "cap_sinks": dict(lens=[300, 0, 64], Hq=8, cap=5.0, sinks=True),
    "prefix": dict(lens=[33, 0, 1, 100], Hq=4, prefix=75),
    "prefix_only": dict(lens=[0, 0], Hq=4, prefix=16),
    "prefix_d64_sinks": dict(lens=[20, 5, 40], Hq=4, D=64, Lq=3, prefix=130, sinks=True, cap=30.0, page=32),
    "prefix_rows": dict(lens=[(13 * b) % 50 for b in range(40)], Hq=8, prefix=300, page=64),
    "prefix_many_rows": dict(lens=[b % 7 for b in range(70)], Hq=16, Lq=2, prefix=1000, page=128, q_len=[b % 3 for b in range(70)]),
    "prefix_long": dict(lens=[9, 2], Hq=16, prefix=4097, page=128),
    "no_queries": dict(lens=[30, 2], Hq=4, Lq=2, prefix=20, q_len=[0, 0]),
    "rows_cap": dict(lens=[300, 140], Hq=8, Lq=40, cap=3.0, sinks=True),
    "rows_large_cap": dict(lens=[300, 140], Hq=8, Lq=70, Hkv=1, cap=50.0),
    "prefix_rows_cap": dict(lens=[(13 * b) % 50 for b in range(70)], Hq=16, prefix=300, page=64, cap=20.0, Hkv=4),
}


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cache", [F8, torch.bfloat16], ids=["e4m3", "c16"])
@pytest.mark.parametrize("name", CASES)
def test_attention(name, cache, dtype):
    c = dict(dict(Hkv=2, D=128, page=16, Lq=1, prefix=0, sinks=False), **CASES[name])
    pool = Pool(c["lens"], Hkv=c["Hkv"], D=c["D"], page=c["page"], dtype=cache, seed=len(name), prefix=c["prefix"])
    g = torch.Generator().manual_seed(len(name) + 1)
    q = torch.randn((len(c["lens"]), c["Lq"], c["Hq"], c["D"]), generator=g).to(dtype)
    sinks = torch.randn(c["Hq"], generator=g) if c["sinks"] else None
    check_attention(pool, q, causal=c.get("causal", True), cap=c.get("cap", 0.0), q_len=c.get("q_len"), sinks=sinks)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cache", [F8, torch.bfloat16], ids=["e4m3", "c16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,B", [(2, 2), (16, 9)])
def test_what_lies_behind_a_length_does_not_count(Hq, B, D, cache, dtype):
    """Keys and values past a sequence's end hold NaN and infinities; a page past it has no number."""
    lens = [(29 * b + 5) % 70 for b in range(B)]
    pool = Pool(lens, Hkv=1, D=D, page=32, dtype=cache, seed=3, prefix=40 if D == 128 else 41, width=6)
    bad = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38])
    for b in range(B + 1):
        pages, n = (pool.table[b], lens[b]) if b < B else (pool.prefix, pool.prefix_len)
        for t in range(n, -(-n // 32) * 32):
            at = (int(pages[t // 32]), slice(None), t % 32)
            for w, (x, e) in enumerate(((pool.cache.k_pages, pool.cache.k_exps), (pool.cache.v_pages, pool.cache.v_exps))):
                if cache == F8:
                    x.view(torch.uint8)[at] = 0x7f if t % 2 else 0xff
                    e[at] = 255 if t % 3 else 0
                else:
                    x[at] = bad[(t + w) % 4].to(torch.bfloat16)
    q = torch.randn((B, 1, Hq, D), generator=torch.Generator().manual_seed(4)).to(dtype)
    check_attention(pool, q)


@gpu
def test_a_row_without_a_value_reaches_the_rows_that_see_it():
    pool = Pool([40, 40], Hkv=1, seed=5)
    pool.cache.v_exps[int(pool.table[1, 0]), 0, 3] = 255
    q = torch.randn((2, 1, 2, 128), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    p = ra.make_paged_params(pool.cache, q, pool.table.cuda(), torch.tensor([40, 40], dtype=torch.int32).cuda(), scale=0.1)
    out, lse = ra.paged_forward(p, q, pool.cache)
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all() and torch.isfinite(lse).all()


@gpu
def test_large_logits_keep_their_weights():
    """Logits of some hundreds, where a softmax without its running maximum overflows."""
    pool = Pool([700], Hkv=1, page=64, dtype=torch.bfloat16, seed=8)
    q = 40 * torch.randn((1, 1, 4, 128), generator=torch.Generator().manual_seed(9))
    k, v = pool.dense(0)
    p = ra.make_paged_params(pool.cache, q.cuda(), pool.table.cuda(), torch.tensor([700], dtype=torch.int32).cuda(), scale=1.0)
    for dt in (torch.float32, torch.bfloat16):
        qd = q.to(dt)
        p = ra.make_paged_params(pool.cache, qd.cuda(), pool.table.cuda(), torch.tensor([700], dtype=torch.int32).cuda(), scale=1.0)
        out, lse = ra.paged_forward(p, qd.cuda(), pool.cache)
        o, e = attention(qd[0].double(), k, v, scale=1.0, visible=torch.ones((1, 700), dtype=torch.bool))
        # |s| is up to a few thousand: 2^-24 * 128 terms * sum |q k| ~ 8000 / 11 -> 1e-2 of a nat at worst
        assert (lse[0].cpu().double() - e).abs().max() <= 1e-2
        assert (out[0].cpu().double() - o).abs().max() <= 2e-2 * float(v.abs().max())


# heads, kv heads, query tokens and head size of a call that each kernel takes: rows per kv head decide
KERNELS = {"d64": (4, 1, 1, 64), "d64_8": (8, 1, 1, 64), "d64_12": (12, 1, 1, 64), "d64_16": (16, 1, 1, 64),
           "d64_80": (8, 1, 10, 64), "rows8": (2, 1, 1, 128), "rows16": (16, 1, 1, 128), "rows20": (20, 1, 1, 128),
           "rows32": (32, 1, 1, 128), "rows80": (8, 1, 10, 128), "rows320": (8, 1, 40, 128)}
each_kernel = pytest.mark.parametrize("name", KERNELS)
each_cache = pytest.mark.parametrize("cache", [F8, torch.bfloat16], ids=["e4m3", "c16"])
each_type = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


def queries(name, B, dtype, seed):
    Hq, _, Lq, D = KERNELS[name]
    return torch.randn((B, Lq, Hq, D), generator=torch.Generator().manual_seed(seed)).to(dtype)


@gpu
@each_type
@each_cache
@each_kernel
@pytest.mark.parametrize("way", ["up", "down"])
def test_scales_that_change_along_a_sequence(way, name, cache, dtype):
    """Values whose size runs over 2^18 within a sequence, keys over 2^3: references and common exponents move inside a
    tile and between tiles."""
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([700, 90, 0], Hkv=Hkv, D=D, page=32, dtype=cache, seed=31, prefix=333)
    for b in (None, 0, 1):
        at = pool.places(b)
        for t in range(len(at)):
            x = t if way == "up" else len(at) - 1 - t
            pool.scale(1, at[t], 18 * x // len(at))
            pool.scale(0, at[t], 3 * x // len(at))
    check_attention(pool, queries(name, 3, dtype, 32))


@gpu
@each_cache
def test_row_blocks_of_one_and_of_two_tiles_in_turn(cache):
    """320 rows per kv head are a block of 256 and one of 64: a CTA with many segments has runs of either, and values
    whose size differs between sequences."""
    pool = Pool([250 + (37 * b) % 300 for b in range(80)], Hkv=4, page=64, dtype=cache, seed=39)
    for b in range(80):
        for at in pool.places(b):
            pool.scale(1, at, (5 * b) % 12)
    check_attention(pool, torch.randn((80, 40, 32, 128), generator=torch.Generator().manual_seed(40)).to(torch.bfloat16))


@gpu
@each_type
@each_cache
@each_kernel
def test_pages_out_of_range(name, cache, dtype):
    """Their keys and values read as zeros, whatever the number, and the call reports them."""
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([300, 130, 64], Hkv=Hkv, D=D, page=32, dtype=cache, seed=33, prefix=200)
    table, prefix = pool.table.clone(), pool.prefix.clone()
    for b, i, number in ((0, 0, -1), (0, 5, pool.n), (1, 4, 2 ** 31 - 1), (2, 1, -2 ** 31), (None, 2, 1 << 20), (None, 6, -5)):
        pages, given = (pool.prefix, prefix) if b is None else (pool.table[b], table[b])
        for w in (0, 1):
            pool.val[w][int(pages[i])] = 0
        given[i] = number
    pool.given = table, prefix
    check_attention(pool, queries(name, 3, dtype, 34))
    assert ra.ra_get_device_status() == ra.RA_ERR_INVALID_ARG
    assert ra.ra_get_device_status() == ra.RA_OK


@gpu
@each_type
@each_cache
@each_kernel
def test_queries_that_are_not_finite(name, cache, dtype):
    """A row with a NaN or an infinity is NaN; a row of zeros is a mean; the other rows are what they should be (to the
    bounds above: rows of a block may move their references together, so not bit by bit)."""
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([200, 75], Hkv=Hkv, D=D, page=16, dtype=cache, seed=35, prefix=60)
    q = queries(name, 2, dtype, 36)
    q[0, -1, 1] = 0
    check_attention(pool, q)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    p = ra.make_paged_params(pool.cache, q.cuda(), pool.table.cuda(), i32(pool.lens), scale=D ** -0.5,
                             prefix_table=pool.prefix.cuda(), prefix_len=i32([60]))
    want, want_lse = ra.paged_forward(p, q.cuda(), pool.cache)
    q[0, 0, 0, 5] = float("nan")
    q[1, -1, 1, 7] = float("inf")
    q[1, -1, 1, 8] = float("-inf")
    got, lse = ra.paged_forward(p, q.cuda(), pool.cache)
    bad = torch.zeros(q.shape[:3], dtype=torch.bool)
    bad[0, 0, 0] = bad[1, -1, 1] = True
    assert torch.isnan(got.cpu()[bad]).all() and torch.isnan(lse.cpu().transpose(1, 2)[bad]).all()
    most = max(float(v.abs().max()) for v in (pool.dense(0)[1], pool.dense(1)[1]))
    assert (got - want).cpu().float()[~bad].abs().max() <= 2 * (1e-4 if dtype == torch.float32 else 2 ** -7) * most
    assert (lse - want_lse).cpu().transpose(1, 2)[~bad].abs().max() <= 2e-4


@gpu
@each_type
@each_cache
@each_kernel
def test_lse_of_small_capped_logits(name, cache, dtype):
    """One key: lse is the capped logit itself.  Without cancellation (q, k > 0) its relative error is at most
    D * 2^-23 (products accumulated with truncation), 3.4e-7 for the series of tanh, a few 2^-24, and 2^-23 absolute where
    the logit meets its reference: 2e-5 relative at logits of 0.05 and above."""
    _, Hkv, _, D = KERNELS[name]
    pool = Pool([1, 1], Hkv=Hkv, D=D, dtype=cache, seed=37)
    at = [pool.places(b)[0] for b in (0, 1)]
    for a in at:
        x = pool.val[0][a].abs()
        pool.val[0][a] = x
        if cache == F8:
            pool.cache.k_pages.view(torch.uint8)[a] &= 0x7f
        else:
            pool.cache.k_pages[a] = x.to(torch.bfloat16).cuda()
    q = (queries(name, 2, torch.float32, 38).abs() * 0.05).to(dtype)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    p = ra.make_paged_params(pool.cache, q.cuda(), pool.table.cuda(), i32([1, 1]), scale=D ** -0.5, soft_cap=50.0, causal=False)
    _, lse = ra.paged_forward(p, q.cuda(), pool.cache)
    for b in (0, 1):
        s = torch.einsum("ihd,hd->hi", q[b].double(), pool.val[0][at[b]].repeat_interleave(q.shape[2] // Hkv, 0)) * D ** -0.5
        assert s.min() > 0.05
        want = 50 * torch.tanh(s / 50)
        assert ((lse[b].cpu().double() - want) / want).abs().max() <= 2e-5


@gpu
@each_type
@pytest.mark.parametrize("cache,page,n", [(F8, 128, 34000), (torch.bfloat16, 64, 34000)], ids=["e4m3", "c16"])
@pytest.mark.parametrize("Hq,Lq", [(8, 1), (80, 8)])
def test_offsets_beyond_32_bits(Hq, Lq, cache, page, n, dtype):
    """A cache of 4.4 GB per tensor: the same tokens in its first and in its last pages."""
    c = ra.new_kv_cache(n, page, 8, 128, cache)
    g = torch.Generator().manual_seed(41)
    low = torch.arange(6, dtype=torch.int32).view(2, 3)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    lens = [3 * page - 5, page + 1]
    k, v = (torch.randn((2, 3 * page, 8, 128), generator=g).to(dtype).cuda() for _ in range(2))
    q = torch.randn((2, Lq, Hq, 128), generator=g).to(dtype).cuda()
    got = []
    for table in (low.cuda(), (n - 1 - low).cuda()):
        ra.kv_write(c, k, v, table, i32([0, 0]), i32(lens))
        p = ra.make_paged_params(c, q, table, i32(lens), scale=0.1, prefix_table=table[0, :2].contiguous(), prefix_len=i32([page + 3]))
        got.append(ra.kv_read(c, table, i32(lens), 3 * page) + ra.paged_forward(p, q, c))
    assert c.k_pages[n - 1].float().abs().sum() > 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


@gpu
@each_cache
@each_kernel
def test_a_graph_serves_lengths_that_change(name, cache):
    Hq, Hkv, Lq, D = KERNELS[name]
    pool = Pool([400, 90, 64], Hkv=Hkv, D=D, page=32, dtype=cache, seed=43, prefix=333)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    kv, q_len, plen = i32([1, 90, 0]), i32([Lq, Lq, Lq]), i32([0])
    q = queries(name, 3, torch.bfloat16, 44).cuda()
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
@each_cache
def test_calls_on_several_streams(cache):
    """Calls of all kernels at once, each with its own workspace, give what they give alone."""
    jobs = []
    for i, name in enumerate(KERNELS):
        _, Hkv, _, D = KERNELS[name]
        pool = Pool([(97 * b + 11 * i) % 600 for b in range(24)], Hkv=Hkv, D=D, page=32, dtype=cache, seed=50 + i, prefix=300)
        q = queries(name, 24, torch.bfloat16, 60 + i).cuda()
        p = ra.make_paged_params(pool.cache, q, pool.table.cuda(), torch.tensor(pool.lens, dtype=torch.int32).cuda(), scale=D ** -0.5,
                                 prefix_table=pool.prefix.cuda(), prefix_len=torch.tensor([300], dtype=torch.int32).cuda())
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
@pytest.mark.parametrize("cache", [F8, torch.bfloat16], ids=["e4m3", "c16"])
def test_prefill_then_decode(cache):
    """A prompt attended densely while its keys enter the cache, a shared prefix, decoding steps in a captured graph,
    and the whole history read back: every step equals dense attention over what the cache holds."""
    g = torch.Generator().manual_seed(12)
    B, Hq, Hkv, D, page, P, L, steps = 3, 8, 2, 128, 32, 128, 128, 5
    c = ra.new_kv_cache(64, page, Hkv, D, cache)
    order = torch.randperm(64, generator=g).to(torch.int32)
    prefix, table = order[:4].cuda(), order[4:4 + 3 * 6].view(3, 6).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    new = lambda n, h: torch.randn((B, n, h, D), generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    pk, pv = new(P, Hkv)[:1], new(P, Hkv)[:1]
    ra.kv_write(c, pk, pv, prefix[None], i32([0]))
    k, v = new(L, Hkv), new(L, Hkv)
    lens = [128, 77, 1]
    ra.kv_write(c, k, v, table, i32([0] * B), i32(lens))
    kv_len, plen = i32(lens), i32([P])
    # the cached prefix through the dense path: its keys read back and attended by a dense call
    rk, rv = ra.kv_read(c, prefix[None].contiguous(), plen, P)
    qd = new(P, Hq)[:1]
    params = ra.make_params(qd, rk, scale=D ** -0.5, causal=True)
    dense, dense_lse = ra.forward(params, qd, rk, rv, ra.build_mask(params))
    again = ra.make_paged_params(c, qd, prefix[None].contiguous(), plen, scale=D ** -0.5)
    paged, paged_lse = ra.paged_forward(again, qd, c)
    assert (dense.float() - paged.float()).abs().max() <= 2e-2 and (dense_lse - paged_lse).abs().max() <= 1e-3

    q, nk, nv = new(1, Hq), new(1, Hkv), new(1, Hkv)
    p = ra.make_paged_params(c, q, table, kv_len, scale=D ** -0.5, prefix_table=prefix, prefix_len=plen)
    ws = torch.empty(ra.ra_attn_paged_workspace_size(c, p), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")

    def step():
        ra.kv_write(c, nk, nv, table, kv_len)
        kv_len.add_(1)
        ra.paged_forward(p, q, c, out=out, lse=lse, ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(steps):
        for x in (q, nk, nv):
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        if t:
            graph.replay()
        else:
            step()
        hk, hv = ra.kv_read(c, table, kv_len, 6 * page, torch.float32)
        for b in range(B):
            n = lens[b] + 2 + t
            assert int(kv_len[b]) == n
            kk, vv = (torch.cat([ra.kv_read(c, prefix[None].contiguous(), plen, P, torch.float32)[w][0], h[b, :n]]).cpu().double()
                      for w, h in ((0, hk), (1, hv)))
            o, e = attention(q[b].cpu().double(), kk, vv, scale=D ** -0.5, visible=torch.ones((1, P + n), dtype=torch.bool))
            assert (out[b].cpu().double() - o).abs().max() <= 2 ** -7 * float(vv.abs().max())
            assert (lse[b].cpu().double() - e).abs().max() <= 1e-4


@gpu
def test_another_stream():
    pool = Pool([300, 40], Hkv=2, seed=21)
    q = torch.randn((2, 1, 4, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    p = ra.make_paged_params(pool.cache, q, pool.table.cuda(), torch.tensor([300, 40], dtype=torch.int32).cuda(), scale=0.1)
    want = ra.paged_forward(p, q, pool.cache)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for which in (s, s.cuda_stream):
        got = ra.paged_forward(p, q, pool.cache, stream=which)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------- refusals (no GPU needed)
def _c_cache(**kw):
    d = dict(n_pages=4, page_size=16, Hkv=2, D=128, dtype=ra.RA_E4M3, k=256, v=256, k_exp=256, v_exp=256)
    d.update(kw)
    return ra.RaKvCache(*d.values())


def _c_params(**kw):
    d = dict(B=2, Lq=1, Hq=4, dtype=ra.RA_BF16, scale=0.1, soft_cap=0.0, causal=1, max_pages=2, prefix_pages=0,
             page_table=256, kv_len=256, q_len=None, prefix_table=None, prefix_len=None, sinks=None)
    d.update(kw)
    return ra.RaPagedParams(*d.values())


@pytest.mark.parametrize("bad,code", [
    (dict(n_pages=0), -1), (dict(page_size=24), -1), (dict(page_size=256), -1), (dict(D=96), -2), (dict(dtype=ra.RA_FP32), -1),
    (dict(k=None), -1), (dict(k=264), -1), (dict(k_exp=None), -1), (dict(v_exp=257), -1), (dict(dtype=ra.RA_BF16), -1),
    (dict(n_pages=1 << 30, Hkv=4), -2),
])
def test_bad_caches_are_refused(bad, code):
    import ctypes
    L, c, p = ra.lib(), _c_cache(**bad), _c_params()
    by = ctypes.byref
    assert L.ra_kv_write(by(c), 256, 256, ra.RA_BF16, 1, 1, 256, 256, 256, 1, 256, None, None) == code
    assert ra.ra_last_error()
    assert L.ra_kv_read(by(c), 256, 1, 256, 1, 1, 256, 4096, ra.RA_BF16, None) == code
    assert L.ra_attn_paged_workspace_size(by(c), by(p)) == 0
    assert L.ra_attn_paged(by(c), by(p), 256, 4096, 8192, 256, 1 << 30, None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), -1), (dict(Lq=0), -1), (dict(Hq=3), -1), (dict(dtype=ra.RA_E4M3), -1), (dict(scale=0.0), -1),
    (dict(scale=math.nan), -1), (dict(soft_cap=math.nan), -1), (dict(soft_cap=1e-30), -1), (dict(max_pages=0), -1), (dict(page_table=None), -1),
    (dict(kv_len=None), -1), (dict(prefix_pages=1), -1), (dict(prefix_table=256, prefix_len=256), -1),
    (dict(max_pages=1 << 28), -2), (dict(B=1 << 20, Lq=1 << 12), -2),
])
def test_bad_params_are_refused(bad, code):
    import ctypes
    L, c, p = ra.lib(), _c_cache(), _c_params(**bad)
    assert L.ra_attn_paged_workspace_size(ctypes.byref(c), ctypes.byref(p)) == 0
    assert L.ra_attn_paged(ctypes.byref(c), ctypes.byref(p), 256, 4096, 8192, 256, 1 << 30, None) == code


def test_a_call_with_too_much_work_is_refused():
    import ctypes
    L, c, p = ra.lib(), _c_cache(), _c_params(B=1 << 20, max_pages=1 << 14)
    assert L.ra_attn_paged_workspace_size(ctypes.byref(c), ctypes.byref(p)) == 0 and "split the batch" in ra.ra_last_error()
    assert L.ra_attn_paged(ctypes.byref(c), ctypes.byref(p), 256, 1 << 40, 8192, 256, 1 << 30, None) == -2


def test_bad_calls_are_refused():
    import ctypes
    L, c, p = ra.lib(), _c_cache(), _c_params()
    by = ctypes.byref
    n = L.ra_attn_paged_workspace_size(by(c), by(p))
    assert n > 0
    call = lambda q=1 << 20, o=1 << 21, l=1 << 22, w=1 << 23, b=n: L.ra_attn_paged(by(c), by(p), q, o, l, w, b, None)  # noqa: E731
    assert call(q=None) == call(o=None) == call(l=None) == -1
    assert call(q=(1 << 20) + 8) == -1
    assert call(o=(1 << 20) + 16) == -1  # overlaps q
    assert call(w=None) == call(b=n - 1) == call(w=(1 << 23) + 128) == -4
    w = lambda **k: L.ra_kv_write(by(c), k.get("k", 256), k.get("v", 256), k.get("dt", ra.RA_BF16), k.get("B", 1), 1,  # noqa: E731
                                  k.get("ks", 256), k.get("vs", 256), k.get("t", 256), 1, k.get("s", 256), None, None)
    assert w(k=None) == w(s=None) == w(t=None) == w(B=0) == w(dt=ra.RA_E4M3) == w(ks=255) == w(vs=260) == w(k=264) == -1
    assert L.ra_kv_read(by(c), 256, 1, 256, 1, 1, 4096, 4096, ra.RA_BF16, None) == -1  # k and v overlap
    assert L.ra_kv_read(by(c), 256, 1, 256, 1, 1 << 30, 4096, 1 << 50, ra.RA_BF16, None) == -2  # more rows than 2^31
    assert L.ra_kv_write(by(c), 256, 256, ra.RA_BF16, 1, 1 << 30, 256, 256, 256, 1, 256, None, None) == -2


def test_helpers_refuse_what_they_cannot_pass_on():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(TypeError):
        ra.make_kv_cache(t(1, 1, 16, 64, dt=torch.float16), t(1, 1, 16, 64, dt=torch.float16))
    with pytest.raises(ValueError):
        ra.make_kv_cache(t(1, 1, 16, 64), t(1, 1, 16, 128))
    with pytest.raises(ValueError):
        ra.make_kv_cache(t(1, 1, 16, 64, dt=F8), t(1, 1, 16, 64, dt=F8))
    c = ra.new_kv_cache(2, 16, 2, 64, torch.bfloat16, device="cpu")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):  # heads not contiguous
        ra.kv_write(c, t(1, 4, 64, 2).transpose(2, 3), t(1, 4, 2, 64), i(1, 1), i(1))
    with pytest.raises(ValueError):  # batches unevenly spaced
        ra.kv_write(c, t(2, 5, 2, 64)[:, :4], t(2, 4, 2, 64), i(2, 1), i(2))
    with pytest.raises(TypeError):
        ra.kv_write(c, t(1, 4, 2, 64), t(1, 4, 2, 64), i(1, 1).long(), i(1))
    with pytest.raises(ValueError):
        ra.kv_write(c, t(1, 4, 2, 64), t(1, 4, 2, 64), i(1, 1), i(2))
    q = t(1, 1, 4, 64)
    with pytest.raises(ValueError):
        ra.make_paged_params(c, q, i(1, 1), i(1), scale=1.0, prefix_table=i(1))
    with pytest.raises(ValueError):
        ra.make_paged_params(c, t(1, 1, 4, 128), i(1, 1), i(1), scale=1.0)
    with pytest.raises(ra.RaError):
        ra.make_paged_params(c, t(1, 1, 3, 64), i(1, 1), i(1), scale=1.0)
    p = ra.make_paged_params(c, q, i(1, 1), i(1), scale=1.0)
    with pytest.raises(ValueError):
        ra.paged_forward(p, t(1, 1, 2, 64), c)
    with pytest.raises(ValueError):
        ra.paged_forward(p, q, ra.new_kv_cache(3, 16, 2, 64, torch.bfloat16, device="cpu"))
    with pytest.raises(ValueError):
        ra.paged_forward(p, t(1, 1, 64, 4).transpose(2, 3), c)
