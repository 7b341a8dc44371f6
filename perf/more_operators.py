"""What stands between a layer's projections and its attention, and a cache in 4 bits: what one pass computes, on which sizes.

Five operators, one set, in the order in which a model's tokens meet them.  ``rotate`` turns queries and keys by their
positions and takes the gradients back through it; ``norm`` does so behind an RMS norm of each head, in one pass, with the
gradients of the inputs and of the two weights; ``enter`` is serving's form of it: queries come out, keys and values go
into the paged cache on the way.  ``store`` writes tokens into a cache held in 4 bits and gathers the sequences back out
of it; ``attend`` is attention of each sequence's last few tokens over such a cache, with or without a prefix that the
batch shares.  ``run`` computes an operator in its plain form (elementary torch operations in 32 bits, angles in 64), or,
where ``own`` is set, with this package's kernels; ``exact`` is the definition in 64 bits.

Rotation.  Of a head's D values the first ``rot`` are turned in pairs, pair i by the angle position * f_i: values i and
i + rot / 2 (``half``), or 2i and 2i + 1 (interleaved); the result is multiplied by ``amplitude``.  f_i = base^(-2i / rot),
for contexts longer than the trained one divided by a factor: all of them (``linear``), by a larger base (``ntk``), by a
ramp over the number of turns in the trained length (``yarn``, with an amplitude of its own), or between two wavelengths
(``bands``).  The norm is x / sqrt(mean(x^2) + eps) * weight over the D values of a head.

The cache in 4 bits.  Each 32 consecutive values of a row (one token of one kv head) share a power of two, stored as a
byte: value = code * 2^(byte - 127), with the smallest exponent e = byte - 127 >= -110 that brings the largest magnitude
to at most 6, and codes of e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), the even value of a pair in a byte's low half.  A
block with an infinity or a NaN has byte 255 and codes 0, and reads back as NaN.  Sequence b's token at position t is in
page ``page_table[b, t // page size]``.
"""
import math

import torch

own = False

MIN_EXP = -110
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6
TRAINED = 8192  # the length that scaled rotations were trained on


# ---------------------------------------------------------------- cases
def _case(op, **kw):
    c = dict(op=op, B=1, L=1, Hq=32, Hkv=8, D=128, dtype="bf16", rot=128, half=True, base=10000.0, scaling="none", factor=1.0,
             where="start", kv_lo=1, kv_hi=1, ragged=False, cache="e2m1", page=64, prefix=0, causal=True, cap=0.0,
             sinks=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of a batch of 64 with contexts of up to 128K, 16 times the trained length: q and k in place
        # of a bf16 model without norms
        dict(_case("rotate", B=64, kv_lo=1, kv_hi=131072, scaling="yarn", factor=16.0, base=500000.0), name="rotate_step"),
        # training on 32K tokens in zigzag order (the gqa32k shapes): there and back
        dict(_case("rotate", L=32768, where="zigzag", scaling="linear", factor=4.0), name="rotate_long"),
        # a small fp32 model, pairs side by side, half of each head turned
        dict(_case("norm", B=2, L=257, Hq=4, Hkv=2, D=64, dtype="fp32", rot=32, half=False, where="index"),
             name="norm_small"),
        # training on packed documents (the packed16k shapes)
        dict(_case("norm", B=2, L=16384, Hq=16, Hkv=16, where="packed", base=1000000.0), name="norm_packed"),
        # one decoding step into an 8-bit cache, out of a fused projection
        dict(_case("enter", B=64, kv_lo=1, kv_hi=1023, cache="e4m3"), name="enter_step"),
        # prompts of different lengths behind a shared system prompt of 1000 tokens, 16-bit cache
        dict(_case("enter", B=8, L=4096, ragged=True, kv_lo=0, kv_hi=700, cache="bf16", prefix=1000, scaling="bands",
                   factor=8.0, base=500000.0), name="enter_prompt"),
        # a short history of a small fp32 model into 4 bits and back
        dict(_case("store", B=3, L=257, Hq=2, Hkv=2, D=64, page=16, dtype="fp32", kv_lo=0, kv_hi=57), name="store_short"),
        # prompts of different lengths into 4 bits, and the sequences back for dense attention
        dict(_case("store", B=8, L=4096, ragged=True, kv_lo=0, kv_hi=700), name="store_prompt"),
        # one user, a context of a thousand tokens: latency
        dict(_case("attend", B=1, kv_lo=1000, kv_hi=1000), name="attend_one"),
        # a serving batch with ragged contexts
        dict(_case("attend", B=64, kv_lo=17, kv_hi=8192), name="attend_batch"),
        # draft tokens checked against 64K contexts (the long64k heads), a different number for each sequence
        dict(_case("attend", B=2, L=5, Hq=8, Hkv=2, kv_lo=60001, kv_hi=65536, ragged=True, cap=30.0), name="attend_draft64k"),
        # a batch behind an 8K prompt, with sinks
        dict(_case("attend", B=64, prefix=8192, kv_lo=1, kv_hi=512, sinks=True), name="attend_prefix"),
    ]


HEADS = [(32, 8, 128), (16, 16, 128), (32, 1, 128), (8, 2, 128), (6, 3, 128), (4, 2, 64), (2, 2, 64), (8, 1, 64)]
SCALINGS = [("none", 1.0), ("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0), ("bands", 8.0)]
#: No drawn case costs more than the largest listed ones: bytes and operations of one pass.
MOST_BYTES, MOST_FLOPS = {"rotate": 1.3e9, "norm": 1.3e9, "enter": 6.0e8, "store": 4.0e8, "attend": 4.0e8}, 5.0e10


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["rotate", "norm", "enter", "store", "attend", "attend"])
        Hq, Hkv, D = rng.choice(HEADS)
        scaling, factor = rng.choice(SCALINGS)
        c = _case(op, Hq=Hq, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]),
                  rot=16 * rng.randint(1, D // 16), half=rng.random() < 0.6, base=rng.choice([1e4, 5e5, 1e6]),
                  scaling=scaling, factor=factor, page=rng.choice([16, 32, 64, 128]))
        if op in ("rotate", "norm"):
            c.update(B=_log(rng, 1, 64), L=_log(rng, 1, 32768), where=rng.choice(["start", "index", "packed", "zigzag"]))
            c.update(kv_hi=_log(rng, 1, 1 << 20) if c["where"] == "start" else 1)
        elif op in ("enter", "store"):
            c.update(B=_log(rng, 1, 64), L=_log(rng, 1, 4096), kv_lo=0, kv_hi=_log(rng, 1, 4096), ragged=rng.random() < 0.5)
            if op == "enter":
                # (behind a norm a 4-bit code next to a border may fall to either side: the 4-bit cache is in store)
                c.update(cache=rng.choice(["e4m3", "bf16"]), prefix=rng.choice([0, 0, _log(rng, 1, 32768)]))
        else:
            c.update(B=_log(rng, 1, 128), L=rng.choice([1, 1, 1, 2, 3, 5, 8]), causal=rng.random() < 0.8,
                     cap=rng.choice([0.0, 0.0, 30.0, 50.0]), sinks=rng.random() < 0.3, ragged=rng.random() < 0.3)
            c["kv_hi"] = _log(rng, 1, 65536)
            c["kv_lo"] = rng.randint(0, c["kv_hi"])
            if rng.random() < 0.4:
                c.update(prefix=_log(rng, 1, 32768))
        w = work(c)
        # the plain form's dense copies count too, at the longest sequence's length
        dense = 8 * c["B"] * c["Hkv"] * c["D"] * max(c["L"], c["kv_hi"]) if op in ("store", "attend") else 0
        scores = 12 * c["B"] * c["L"] * c["Hq"] * (c["kv_hi"] + c["prefix"]) if op == "attend" else 0
        if w["bytes"] <= MOST_BYTES[op] and w["flops"] <= MOST_FLOPS and dense + scores <= 1.2e10:
            return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly: the lengths of a batch, before they are shuffled."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(c):
    """(cached tokens, new tokens) of the case's sequences, before the shuffles."""
    kv = _spread(c["kv_lo"], c["kv_hi"], c["B"])
    new = _spread((c["L"] + 1) // 2, c["L"], c["B"]) if c["ragged"] else [c["L"]] * c["B"]
    return kv, new


def work(case):
    c = case
    kv, new = _lengths(c)
    D, item = c["D"], 2 if c["dtype"] == "bf16" else 4
    row = {"bf16": 2 * D, "e4m3": D + 1, "e2m1": D // 2 + D // 32}[c["cache"]]  # bytes of one cached row
    tokens = sum(new)
    both = (c["Hq"] + c["Hkv"]) * D * item * tokens  # q and k once
    if c["op"] == "rotate":
        return {"bytes": 4 * both, "flops": 6 * both // item}
    if c["op"] == "norm":
        return {"bytes": 5 * both, "flops": 24 * both // item}  # forward: x, y; backward: x, dy, dx
    if c["op"] == "enter":
        return {"bytes": both + tokens * (c["Hq"] + c["Hkv"]) * D * item + 2 * tokens * c["Hkv"] * row,
                "flops": 7 * both // item}
    if c["op"] == "store":
        end = sum(k + n for k, n in zip(kv, new))
        return {"bytes": 2 * tokens * c["Hkv"] * (D * item + row) + 2 * c["Hkv"] * (end * row + c["B"] * (c["kv_hi"] + c["L"]) * D * item),
                "flops": 0}
    keys = sum(kv) + c["prefix"]
    pairs = sum(n * (t + c["prefix"]) for n, t in zip(new, kv))
    rows = tokens * c["Hq"]
    return {"bytes": 2 * keys * c["Hkv"] * row + rows * (2 * D * item + 4), "flops": 4 * pairs * c["Hq"] * D}


# ---------------------------------------------------------------- rotation
def _frequencies(c):
    """Radians per position of each pair in 64 bits, and what the result is multiplied by."""
    n, base, factor = c["rot"], c["base"], c["factor"]
    if c["scaling"] == "ntk" and n > 2:
        base *= factor ** (n / (n - 2))
    i = torch.arange(n // 2, dtype=torch.float64)
    f = base ** (-2 * i / n)
    amplitude = 1.0
    if c["scaling"] == "linear":
        f = f / factor
    elif c["scaling"] == "yarn":
        # the pair that turns r times in the trained length
        pair = [n * math.log(TRAINED / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (32.0, 1.0)]
        lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), n - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        amplitude = 0.1 * math.log(factor) + 1.0
    elif c["scaling"] == "bands":
        turns = TRAINED * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f / factor * (1 - keep) + f * keep
    return f, amplitude


def _positions(s):
    """(B, L) positions in 64 bits."""
    c = s["case"]
    if s["pos"] is not None:
        return s["pos"].double()
    first = s["kv_len"].double()[:, None] if s["kv_len"] is not None else 0.0
    if c["prefix"]:
        first = first + s["prefix_len"].double()
    return first + torch.arange(c["L"], dtype=torch.float64, device="cuda").expand(c["B"], -1)


def _turn(s, x, back=False):
    """x (B, L, H, D) in 32 bits turned, or a gradient taken back."""
    c, n = s["case"], s["case"]["rot"]
    angle = _positions(s)[..., None, None] * s["freq"]
    cos, sin = torch.cos(angle).float() * s["amplitude"], torch.sin(angle).float() * s["amplitude"]
    if back:
        sin = -sin
    if c["half"]:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., n:]], -1) if n < c["D"] else turned


# ---------------------------------------------------------------- cached rows
def _exponent(x, top, at_most):
    """The smallest e >= MIN_EXP with amax <= top * 2^e, top = at_most * 2^k, 1/2 < at_most < 1; and whether amax is finite."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1
    k = int(math.log2(top / at_most))
    e = torch.where(m <= at_most, e - k, e - k + 1)
    e = torch.where(amax == 0, MIN_EXP, e).clamp(min=MIN_EXP)
    good = torch.isfinite(amax)
    return torch.where(good, e, 0), good


def _quantise(x, cache):
    """fp32 (..., D) -> codes and the scales' bytes of an e4m3 row, or of the 32-value blocks of an e2m1 row."""
    if cache == "e4m3":
        e, good = _exponent(x, 448.0, 0.875)
        y = torch.where(good[..., None], x * torch.exp2(-e.float())[..., None], 0.0)
        return y.to(torch.float8_e4m3fn), torch.where(good, e + 127, 255).to(torch.uint8)
    x = x.unflatten(-1, (-1, 32))
    e, good = _exponent(x, 6.0, 0.75)
    y = torch.where(good[..., None], x * torch.exp2(-e.float())[..., None], 0.0)
    a = y.abs()
    half = torch.round(a * 2)  # codes of values below 2; then steps of 1 and of 2
    code = torch.where(a < 2, half, torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4)).to(torch.uint8)
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.where(good, e + 127, 255).to(torch.uint8)


def _values(codes, exps):
    """The values that rows of a 4-bit cache stand for, in 32 bits."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    m = code & 7
    v = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2.0, (m - 4.0) * 2))
    v = torch.where(code >= 8, -v, v).unflatten(-1, (-1, 32))
    scale = torch.where(exps == 255, float("nan"), torch.exp2(exps.float() - 127))
    return (v * scale[..., None]).flatten(-2)


# ---------------------------------------------------------------- inputs
def _activations(gen, shape):
    """Projections' outputs: a few loud channels, tokens of different size."""
    x = torch.randn(shape, generator=gen, device="cuda")
    gain = torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device="cuda"))
    size = torch.exp(0.25 * torch.randn(shape[:-1], generator=gen, device="cuda"))
    return x.mul_(gain).mul_(size[..., None])


def _packed(c, host):
    """Positions of rows filled with documents of random lengths."""
    pos = torch.zeros((c["B"], c["L"]), dtype=torch.int32)
    for row in pos:
        at = 0
        while at < c["L"]:
            n = int(torch.randint(128, 4097, (1,), generator=host))
            n = min(n, c["L"] - at)
            row[at:at + n] = torch.arange(n, dtype=torch.int32)
            at += n
    return pos


def _zigzag(c):
    """The order of eight shards, each with a chunk of the front and the one opposite it."""
    n = torch.arange(c["L"])
    chunk, k = (n * 16 // c["L"]).clamp(max=15), torch.tensor([x for d in range(8) for x in (d, 15 - d)])
    order = torch.argsort(torch.argsort(k)[chunk], stable=True)
    return order.to(torch.int32).expand(c["B"], -1).contiguous()


def _pool(c, gen, n_pages, filled):
    shape, cache = (n_pages, c["Hkv"], c["page"], c["D"]), c["cache"]
    s = {}
    for n in ("k", "v"):
        x = _activations(gen, shape) if filled else torch.zeros(shape, device="cuda")
        s[n], s[n + "_exp"] = (x.to(torch.bfloat16), None) if cache == "bf16" else _quantise(x, cache)
    return s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    kv, new = (torch.tensor(x)[torch.randperm(c["B"], generator=host)] for x in _lengths(c))
    s = {"case": c, "kv_len": kv.to(torch.int32).cuda(), "new": new.to(torch.int32).cuda() if c["ragged"] else None,
         "pos": None, "prefix_len": torch.tensor([c["prefix"]], dtype=torch.int32, device="cuda") if c["prefix"] else None}
    dt, B, L, Hq, Hkv, D = DTYPES[c["dtype"]], c["B"], c["L"], c["Hq"], c["Hkv"], c["D"]
    if c["op"] in ("enter", "store", "attend"):
        reach = kv if c["op"] == "attend" else kv + new
        need = [-(-int(t) // c["page"]) for t in reach]
        n_prefix = -(-c["prefix"] // c["page"])
        # as many pages for every pairing of old and new lengths
        n_pages = sum(-(-t // c["page"]) for x in _lengths(c)[:1 if c["op"] == "attend" else 2] for t in x) + n_prefix + 3
        order = torch.randperm(n_pages, generator=host).to(torch.int32)
        table = torch.zeros((B, max(1, max(need))), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s["page_table"] = table.cuda()
        s.update(_pool(c, gen, n_pages, c["op"] != "enter"))
    if c["op"] == "attend":
        s["prefix_table"] = order[at:at + n_prefix].cuda() if c["prefix"] else None
        s["q"] = _activations(gen, (B, L, Hq, D)).to(dt)
        s["sinks"] = torch.randn(Hq, generator=gen, device="cuda") if c["sinks"] else None
        # rows behind a sequence's last new token stay as they are
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros((B, Hq, L), device="cuda")
    else:
        # q, k and v as slices of the fused projection's output
        fused = _activations(gen, (B, L, Hq + 2 * Hkv, D)).to(dt)
        s["q"], s["new_k"], s["new_v"] = fused[:, :, :Hq], fused[:, :, Hq:Hq + Hkv], fused[:, :, Hq + Hkv:]
    if c["op"] in ("rotate", "norm", "enter"):
        freq, s["amplitude"] = _frequencies(c)
        s["freq"] = freq.cuda()
        if c["where"] == "index":
            s["kv_len"] = None
        elif c["where"] != "start":
            s["pos"] = (_packed(c, host) if c["where"] == "packed" else _zigzag(c)).cuda()
        if c["op"] != "rotate":
            s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt) for _ in range(2))
        if c["op"] == "enter":
            s["out"] = torch.zeros((B, L, Hq, D), dtype=dt, device="cuda")
        else:
            s["dq"], s["dk"] = (torch.randn((B, L, h, D), generator=gen, device="cuda").to(dt) for h in (Hq, Hkv))
    if own:
        _own_prepare(s)
    return s


def _own_prepare(s):
    import block_sparse_flash_ra_gb300 as ra
    c = s["case"]
    if "page_table" in s:
        codes = (lambda x: x.view(torch.float4_e2m1fn_x2)) if c["cache"] == "e2m1" else (lambda x: x)
        s["pool"] = ra.make_kv_cache(codes(s["k"]), codes(s["v"]), s["k_exp"], s["v_exp"])
    if c["op"] == "attend":
        s["params"] = ra.make_paged_params(
            s["pool"], s["q"], s["page_table"], s["kv_len"], scale=c["D"] ** -0.5, causal=c["causal"], soft_cap=c["cap"],
            q_len=s["new"], sinks=s["sinks"], prefix_table=s["prefix_table"], prefix_len=s["prefix_len"])
    elif c["op"] != "store":
        rope = ra.make_rope(c["rot"], c["base"], interleaved=not c["half"], scaling=None if c["scaling"] == "none" else c["scaling"],
                            factor=c["factor"], trained_length=TRAINED)
        norm = {} if c["op"] == "rotate" else dict(eps=EPS, q_weight=s["wq"], k_weight=s["wk"])
        s["params"] = ra.make_qk_params(s["q"], s["new_k"], rope=rope, pos=s["pos"], start=s["kv_len"] if s["pos"] is None else None,
                                        prefix_len=s["prefix_len"], **norm)


# ---------------------------------------------------------------- plain forms
def _rotate(s):
    dt = s["q"].dtype
    return {"q": _turn(s, s["q"].float()).to(dt), "k": _turn(s, s["new_k"].float()).to(dt),
            "dq": _turn(s, s["dq"].float(), True).to(dt), "dk": _turn(s, s["dk"].float(), True).to(dt)}


def _normed(x, w):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r, w.float()


def _norm(s):
    out, dt = {}, s["q"].dtype
    for n, x, w, dy in (("q", s["q"], s["wq"], s["dq"]), ("k", s["new_k"], s["wk"], s["dk"])):
        z, r, w = _normed(x, w)
        out[n] = _turn(s, z * w).to(dt)
        du = _turn(s, dy.float(), True)
        out["dw" + n] = (du * z).sum((0, 1, 2))
        dz = du * w
        out["d" + n] = (r * (dz - z * (dz * z).mean(-1, keepdim=True))).to(dt)
    return out


def _new_places(s):
    """(kept new tokens, their pages, their places in the pages)"""
    c = s["case"]
    i = torch.arange(c["L"], device="cuda")
    ok = i < s["new"][:, None] if s["new"] is not None else torch.ones((c["B"], c["L"]), dtype=torch.bool, device="cuda")
    pos = (s["kv_len"][:, None] + i)[ok].long()
    page = s["page_table"][torch.nonzero(ok)[:, 0], pos // c["page"]].long()
    return ok, page, pos % c["page"]


def _put(s, k, v):
    ok, page, at = _new_places(s)
    for n, x in (("k", k), ("v", v)):
        if s["case"]["cache"] == "bf16":
            s[n][page, :, at] = x[ok].to(torch.bfloat16)
        else:
            codes, exps = _quantise(x[ok], s["case"]["cache"])
            s[n].view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
            s[n + "_exp"][page, :, at] = exps
    return ok


def _enter(s):
    (zq, _, wq), (zk, _, wk) = _normed(s["q"], s["wq"]), _normed(s["new_k"], s["wk"])
    ok = _put(s, _turn(s, zk * wk), s["new_v"].float())
    s["out"][ok] = _turn(s, zq * wq).to(s["q"].dtype)[ok]
    return _entered(s)


def _entered(s):
    """Queries and the cache; an 8-bit one's scales as the powers of two that their bytes are."""
    exps = {n: s[n].view(torch.float8_e8m0fnu) for n in ("k_exp", "v_exp") if s[n] is not None}
    return {"q": s["out"], "k": s["k"], "v": s["v"], **exps}


def _gather(s, name, table):
    """(sequences, pages) of page numbers -> fp32 (sequences, kv heads, tokens, D)."""
    t = table.long()
    x = _values(s[name][t], s[name + "_exp"][t])
    return x.transpose(1, 2).reshape(t.shape[0], x.shape[2], -1, x.shape[4])


def _store(s):
    c = s["case"]
    _put(s, s["new_k"].float(), s["new_v"].float())
    end, most = s["kv_len"] + (s["new"] if s["new"] is not None else c["L"]), c["kv_hi"] + c["L"]
    out = {}
    for n in ("k", "v"):
        x = _gather(s, n, s["page_table"])[:, :, :most]
        x = torch.where((torch.arange(x.shape[2], device="cuda") < end[:, None])[:, None, :, None], x, 0.0)
        x = torch.nn.functional.pad(x, (0, 0, 0, most - x.shape[2]))
        out[n] = x.transpose(1, 2).to(DTYPES[c["dtype"]]).contiguous()
    return out


def _attend(s):
    c = s["case"]
    B, L, Hq, Hkv, D = c["B"], c["L"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    q = s["q"].float().view(B, L, Hkv, G, D).permute(0, 2, 1, 3, 4)  # B, Hkv, L, G, D
    k, v = _gather(s, "k", s["page_table"]), _gather(s, "v", s["page_table"])
    T = k.shape[2]
    x = (q.reshape(B, Hkv, L * G, D) @ k.transpose(2, 3)).view(B, Hkv, L, G, T)
    i, j = torch.arange(L, device="cuda"), torch.arange(T, device="cuda")
    n = s["new"] if s["new"] is not None else torch.full((B,), L, device="cuda")
    last = s["kv_len"][:, None] - 1 + ((i - n[:, None] + 1) if c["causal"] else torch.zeros_like(i))
    seen = j <= torch.minimum(last, s["kv_len"][:, None] - 1)[..., None]  # B, L, T
    if c["prefix"]:
        pk, pv = (_gather(s, m, s["prefix_table"][None])[0, :, :c["prefix"]] for m in ("k", "v"))
        rows = q.permute(1, 0, 2, 3, 4).reshape(Hkv, B * L * G, D)
        px = (rows @ pk.transpose(1, 2)).view(Hkv, B, L, G, -1).transpose(0, 1)
        x = torch.cat([px, x], -1)
        seen = torch.cat([seen.new_ones(B, L, px.shape[-1]), seen], -1)
    x = x * D ** -0.5
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    x = torch.where(seen[:, None, :, None], x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, Hkv, 1, G, 1)
        top = torch.maximum(top, sink)
    base = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(x - base)
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(sink - base)
    lse = (torch.log(total) + base)[..., 0].permute(0, 1, 3, 2).reshape(B, Hq, L)
    p = p / torch.where(total == 0, 1.0, total)
    o = torch.zeros_like(q)
    if c["prefix"]:
        pp = p[..., :pk.shape[1]].transpose(0, 1).reshape(Hkv, B * L * G, -1)
        o = (pp @ pv).view(Hkv, B, L, G, D).transpose(0, 1)
    v = torch.where((j < s["kv_len"][:, None])[:, None, :, None], v, 0.0)
    o = o + (p[..., x.shape[-1] - T:].reshape(B, Hkv, L * G, T) @ v).view(B, Hkv, L, G, D)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, L, Hq, D).to(s["q"].dtype)
    if s["new"] is not None:
        kept = i < n[:, None]
        o = torch.where(kept[..., None, None], o, s["out"])
        lse = torch.where(kept[:, None], lse, s["lse"])
    return {"out": o, "lse": lse}


def _own(s):
    import block_sparse_flash_ra_gb300 as ra
    c = s["case"]
    if c["op"] in ("rotate", "norm"):
        q, k = ra.qk_forward(s["params"], s["q"], s["new_k"])
        if c["op"] == "rotate":
            dq, dk, _, _ = ra.qk_backward(s["params"], None, None, s["dq"], s["dk"])
            return {"q": q, "k": k, "dq": dq, "dk": dk}
        dq, dk, dwq, dwk = ra.qk_backward(s["params"], s["q"], s["new_k"], s["dq"], s["dk"])
        return {"q": q, "k": k, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if c["op"] == "enter":
        ra.qk_enter(s["params"], s["pool"], s["q"], s["new_k"], s["new_v"], s["page_table"], count=s["new"], out=s["out"])
        return _entered(s)
    if c["op"] == "store":
        ra.kv_write(s["pool"], s["new_k"], s["new_v"], s["page_table"], s["kv_len"], s["new"])
        end = s["kv_len"] + (s["new"] if s["new"] is not None else c["L"])
        k, v = ra.kv_read(s["pool"], s["page_table"], end, c["kv_hi"] + c["L"], DTYPES[c["dtype"]])
        return {"k": k, "v": v}
    out, lse = ra.paged_forward(s["params"], s["q"], s["pool"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"rotate": _rotate, "norm": _norm, "enter": _enter, "store": _store, "attend": _attend}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _phases(c, s):
    """(B, L) complex numbers of each pair: amplitude * e^(i angle)."""
    n = c["rot"]
    base = c["base"] * (c["factor"] ** (n / (n - 2)) if c["scaling"] == "ntk" else 1.0)
    f, amplitude = [], 1.0
    for i in range(n // 2):
        w = base ** (-2.0 * i / n)
        if c["scaling"] == "linear":
            w /= c["factor"]
        elif c["scaling"] == "yarn":
            lo = max(0, math.floor(n * math.log(TRAINED / (64 * math.pi)) / (2 * math.log(base))))
            hi = min(n - 1, math.ceil(n * math.log(TRAINED / (2 * math.pi)) / (2 * math.log(base))))
            share = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            w = w * (1 - share) + w / c["factor"] * share
            amplitude = 1.0 + 0.1 * math.log(c["factor"])
        elif c["scaling"] == "bands":
            length = 2 * math.pi / w
            if length > TRAINED / 1.0:
                w /= c["factor"]
            elif length > TRAINED / 4.0:
                share = (TRAINED / length - 1.0) / 3.0
                w = w * share + w / c["factor"] * (1 - share)
        f.append(w)
    if s["pos"] is not None:
        at = s["pos"].long()
    else:
        at = torch.arange(c["L"], device="cuda").repeat(c["B"], 1) + c["prefix"]
        if s["kv_len"] is not None:
            at = at + s["kv_len"].long().reshape(-1, 1)
    angle = at.to(torch.float64).unsqueeze(-1) * torch.tensor(f, dtype=torch.float64, device="cuda")
    return torch.polar(torch.full_like(angle, amplitude), angle).unsqueeze(2)


def _turn64(c, x, phase):
    n, y = c["rot"], x.clone()
    if c["half"]:
        z = torch.complex(x[..., :n // 2].contiguous(), x[..., n // 2:n].contiguous()) * phase
        y[..., :n // 2], y[..., n // 2:n] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:n:2].contiguous(), x[..., 1:n:2].contiguous()) * phase
        y[..., 0:n:2], y[..., 1:n:2] = z.real, z.imag
    return y


def _table64():
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6] + [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")


def _pow2(e):
    """2^e in 64 bits, of whole numbers."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _value64(s, name, pages, length):
    """Cached rows of the first `length` tokens of a list of pages: (length, kv heads, D) in fp64."""
    codes, exps = s[name][pages.long()].long(), s[name + "_exp"][pages.long()].long()
    v = _table64()[torch.stack([codes % 16, codes // 16], -1)].reshape(codes.shape[:3] + (-1,))
    v = v * _pow2(exps - 127).repeat_interleave(32, -1)
    return v.permute(0, 2, 1, 3).reshape(-1, v.shape[1], v.shape[3])[:length]


def _nearest64(x, cache):
    """fp64 rows as a cache holds them: (codes' values, powers of two for each value)."""
    y = x.reshape(x.shape[:-1] + (-1, x.shape[-1] if cache == "e4m3" else 32))
    m, e = torch.frexp(y.abs().amax(-1, keepdim=True) / (448 if cache == "e4m3" else 6))
    e = torch.where(m > 0.5, e, e - 1).clamp(min=MIN_EXP)  # a power of two itself asks for no more
    y = y / _pow2(e)
    least, bits = (-6, 3) if cache == "e4m3" else (0, 1)
    step = _pow2((torch.frexp(y.abs())[1] - 1).clamp(min=least) - bits)
    return (torch.round(y / step) * step).reshape(x.shape), _pow2(e)[..., 0]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kv = s["kv_len"].tolist() if s["kv_len"] is not None else None
    new = [c["L"]] * c["B"] if s["new"] is None else s["new"].tolist()
    if c["op"] in ("rotate", "norm", "enter"):
        phase, out = _phases(c, s), {}
        for n, x, dy in (("q", s["q"], s.get("dq")), ("k", s["new_k"], s.get("dk"))):
            x = x.double()
            if c["op"] == "rotate":
                out[n], out["d" + n] = _turn64(c, x, phase), _turn64(c, dy.double(), phase.conj())
                continue
            w, size = s["w" + n].double(), torch.sqrt(x.square().sum(-1, keepdim=True) / c["D"] + EPS)
            out[n] = _turn64(c, x / size * w, phase)
            if c["op"] == "norm":
                g = _turn64(c, dy.double(), phase.conj())
                out["dw" + n] = torch.einsum("blhd,blhd->d", g, x / size)
                g *= w
                out["d" + n] = g / size - x * (g * x).sum(-1, keepdim=True) / (c["D"] * size ** 3)
        if c["op"] != "enter":
            return out
        rows, got = {"k": out["k"], "v": s["new_v"].double()}, {"q": torch.zeros_like(out["q"])}
        for n in ("k", "v"):
            pool = torch.zeros(s[n].shape, dtype=torch.float64, device="cuda")
            for b in range(c["B"]):
                got["q"][b, :new[b]] = out["q"][b, :new[b]]
                t = torch.arange(kv[b], kv[b] + new[b], device="cuda")
                x = rows[n][b, :new[b]]
                x = x if c["cache"] == "bf16" else _nearest64(x, c["cache"])[0]
                pool[s["page_table"][b].long()[t // c["page"]], :, t % c["page"]] = x
            got[n] = pool
            if c["cache"] != "bf16":
                got[n + "_exp"] = None
        return got
    if c["op"] == "store":
        out = {}
        for n in ("k", "v"):
            out[n] = torch.zeros((c["B"], c["kv_hi"] + c["L"], c["Hkv"], c["D"]), dtype=torch.float64, device="cuda")
            for b in range(c["B"]):
                out[n][b, :kv[b]] = _value64(s, n, s["page_table"][b], kv[b])
                codes, scale = _nearest64(s["new_" + n][b, :new[b]].double(), "e2m1")
                out[n][b, kv[b]:kv[b] + new[b]] = codes * scale.repeat_interleave(32, -1)
        return out
    G = c["Hq"] // c["Hkv"]
    out, lse = torch.zeros_like(s["q"], dtype=torch.float64), torch.zeros_like(s["lse"], dtype=torch.float64)
    shared = {n: _value64(s, n, s["prefix_table"], c["prefix"]) for n in ("k", "v")} if c["prefix"] else None
    for b in range(c["B"]):
        k, v = (_value64(s, n, s["page_table"][b], kv[b]) for n in ("k", "v"))
        if shared:
            k, v = torch.cat([shared["k"], k]), torch.cat([shared["v"], v])
        q = s["q"][b, :new[b]].double().reshape(new[b], c["Hkv"], G, c["D"])
        x = torch.einsum("ihgd,jhd->higj", q, k) / math.sqrt(c["D"])
        if c["cap"]:
            x = torch.tanh(x / c["cap"]) * c["cap"]
        if c["causal"]:
            i, j = torch.arange(new[b], device="cuda")[:, None], torch.arange(k.shape[0], device="cuda") - c["prefix"]
            x.masked_fill_(((j > kv[b] - new[b] + i) & (j >= 0))[None, :, None], -math.inf)
        if c["sinks"]:
            sink = s["sinks"].double().reshape(c["Hkv"], 1, G, 1).expand(-1, new[b], -1, -1)
            whole = torch.logsumexp(torch.cat([x, sink], -1), -1, keepdim=True)
        else:
            whole = torch.logsumexp(x, -1, keepdim=True) if k.shape[0] else x.new_full(x.shape[:-1] + (1,), -math.inf)
        p = torch.exp(x - torch.where(whole == -math.inf, torch.zeros_like(whole), whole))
        out[b, :new[b]] = torch.einsum("higj,jhd->ihgd", p, v).reshape(new[b], c["Hq"], c["D"])
        lse[b, :, :new[b]] = whole[..., 0].permute(0, 2, 1).reshape(c["Hq"], new[b])
    return {"out": out, "lse": lse}
