"""Serving operators over a paged key/value cache: what one pass of each computes, on which sizes.

Four operators, one set: ``write`` appends new tokens' keys and values to the cache (quantising them where the cache
holds 8-bit values), ``read`` gathers sequences back into dense tensors, ``decode`` is attention of each sequence's last
few tokens over its pages, and ``prefix`` is the same for a batch whose sequences share a long prefix, which is attended
once for all of them.  ``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or,
where ``own`` is set, with this package's kernels; ``exact`` is the definition in 64 bits.

The cache.  ``k`` and ``v`` are (pages, kv heads, page size, D) in bf16 or e4m3.  An e4m3 row (one token of one kv head)
has a power-of-two scale, stored as a byte: value = code * 2^(byte - 127), with the smallest exponent e = byte - 127 that
brings the row's largest magnitude to at most 448, e >= -110; a row with an infinity or a NaN has byte 255 and codes 0
and reads back as NaN.  Sequence b's token at position t is in page ``page_table[b, t // page size]``.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -110
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- cases
def _case(op, **kw):
    c = dict(op=op, B=1, L=1, Hq=32, Hkv=8, D=128, page=64, cache="e4m3", dtype="bf16", kv_lo=1, kv_hi=1, prefix=0,
             causal=True, cap=0.0, sinks=False, ragged=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of a batch of 64: a token each, appended behind contexts of up to 1K
        dict(_case("write", B=64, L=1, kv_lo=1, kv_hi=1023), name="write_step"),
        # prompts of different lengths entering the cache, K and V taken out of a fused projection
        dict(_case("write", B=8, L=4096, ragged=True, kv_lo=0, kv_hi=700), name="write_prompt"),
        # a short history of a small fp32 model read back
        dict(_case("read", B=3, L=257, Hq=2, Hkv=2, D=64, page=16, dtype="fp32", kv_lo=0, kv_hi=257),
             name="read_short"),
        # the history of two 16K sequences gathered for dense attention (the packed16k shapes)
        dict(_case("read", B=2, L=16384, Hq=16, Hkv=16, kv_lo=15001, kv_hi=16384), name="read_history"),
        # one user, a context of a thousand tokens: latency
        dict(_case("decode", B=1, kv_lo=1000, kv_hi=1000), name="decode_one"),
        # a serving batch with ragged contexts
        dict(_case("decode", B=64, kv_lo=17, kv_hi=8192), name="decode_batch"),
        # multi-query heads over 32K with soft cap and sinks (the mqa32k shapes), 16-bit cache
        dict(_case("decode", B=8, Hq=32, Hkv=1, page=128, cache="bf16", kv_lo=30000, kv_hi=32768, cap=50.0,
                   sinks=True), name="decode_mqa32k"),
        # draft tokens checked against 64K contexts (the long64k heads), a different number for each sequence
        dict(_case("decode", B=2, L=5, Hq=8, Hkv=2, kv_lo=60001, kv_hi=65536, ragged=True), name="decode_draft64k"),
        # a few requests behind one system prompt; one of them has no token of its own yet
        dict(_case("prefix", B=4, page=16, prefix=1024, kv_lo=0, kv_hi=128), name="prefix_short"),
        # a batch behind an 8K prompt
        dict(_case("prefix", B=64, prefix=8192, kv_lo=1, kv_hi=512), name="prefix_batch"),
        # one head of K and V per query head, an odd prefix, sinks, 16-bit cache
        dict(_case("prefix", B=16, Hq=16, Hkv=16, page=32, cache="bf16", prefix=4001, kv_lo=1, kv_hi=300, sinks=True),
             name="prefix_mha"),
        # a large batch behind a 32K document
        dict(_case("prefix", B=128, prefix=32768, kv_lo=64, kv_hi=1024), name="prefix_long"),
    ]


HEADS = [(32, 8, 128), (16, 16, 128), (32, 1, 128), (8, 2, 128), (6, 3, 128), (4, 2, 64), (2, 2, 64), (8, 1, 64)]
#: No drawn case costs more than the largest listed ones: bytes and operations of one pass.
MOST_BYTES, MOST_FLOPS = 4.0e8, 5.0e10


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "decode", "prefix"])
        Hq, Hkv, D = rng.choice(HEADS)
        c = _case(op, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]),
                  cache=rng.choice(["e4m3", "e4m3", "bf16"]), dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]))
        if op == "write":
            c.update(B=_log(rng, 1, 64), L=_log(rng, 1, 4096), kv_lo=0, kv_hi=_log(rng, 1, 4096),
                     ragged=rng.random() < 0.5)
        elif op == "read":
            c.update(B=_log(rng, 1, 16), L=_log(rng, 1, 16384))
            c.update(kv_hi=c["L"], kv_lo=rng.randint(0, c["L"]))
        else:
            c.update(B=_log(rng, 1, 128), L=rng.choice([1, 1, 1, 2, 3, 5, 8]), causal=rng.random() < 0.8,
                     cap=rng.choice([0.0, 0.0, 30.0, 50.0]), sinks=rng.random() < 0.3, ragged=rng.random() < 0.3)
            c["kv_hi"] = _log(rng, 1, 65536 if op == "decode" else 2048)
            c["kv_lo"] = rng.randint(0, c["kv_hi"])
            if op == "prefix":
                c.update(prefix=_log(rng, 1, 32768))
        w = work(c)
        # the plain form's dense copies count too, at the longest sequence's length
        dense = 8 * c["B"] * c["Hkv"] * c["D"] * (c["L"] if op == "write" else c["kv_hi"])
        scores = 12 * c["B"] * c["L"] * c["Hq"] * (c["kv_hi"] + c["prefix"]) if op in ("decode", "prefix") else 0
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS and dense + scores <= 1.2e10:
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
    row = c["D"] + 1 if c["cache"] == "e4m3" else 2 * c["D"]  # bytes of one cached row
    item = 2 if c["dtype"] == "bf16" else 4
    dense = c["Hkv"] * c["D"] * item
    if c["op"] == "write":
        return {"bytes": 2 * sum(new) * (dense + c["Hkv"] * row), "flops": 0}
    if c["op"] == "read":
        return {"bytes": 2 * sum(kv) * c["Hkv"] * row + 2 * c["B"] * c["L"] * dense, "flops": 0}
    keys = sum(kv) + c["prefix"]
    pairs = sum(n * (t + c["prefix"]) for n, t in zip(new, kv))
    rows = sum(new) * c["Hq"]
    return {"bytes": 2 * keys * c["Hkv"] * row + rows * (2 * c["D"] * item + 4), "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---------------------------------------------------------------- the cache's 8-bit rows
def _quantise(x):
    """fp32 (..., D) -> e4m3 codes (..., D) and the scales' bytes (...)."""
    x = x.float()
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1, and 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax == 0, MIN_EXP, e).clamp(min=MIN_EXP)
    good = torch.isfinite(amax)
    e = torch.where(good, e, 0)
    y = x * torch.exp2(-e.float())[..., None]
    codes = torch.where(good[..., None], y, 0.0).to(torch.float8_e4m3fn)
    return codes, torch.where(good, e + 127, 255).to(torch.uint8)


def _scale(byte):
    s = (byte.to(torch.int32) << 23).view(torch.float32)
    return torch.where(byte == 255, float("nan"), s)


def _rows(codes, byte):
    """The values that cached rows stand for, in fp32."""
    return codes.float() if byte is None else codes.float() * _scale(byte)[..., None]


# ---------------------------------------------------------------- inputs
def _activations(gen, shape):
    """Keys and values as projections give them: a few loud channels, tokens of different size."""
    x = torch.randn(shape, generator=gen, device="cuda")
    gain = torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device="cuda"))
    size = torch.exp(0.25 * torch.randn(shape[:-1], generator=gen, device="cuda"))
    return x.mul_(gain).mul_(size[..., None])


def _pool(c, gen, n_pages, filled):
    shape = (n_pages, c["Hkv"], c["page"], c["D"])
    s = {}
    for n in ("k", "v"):
        if not filled:
            s[n] = torch.zeros(shape, dtype=torch.uint8 if c["cache"] == "e4m3" else torch.bfloat16, device="cuda")
            s[n] = s[n].view(DTYPES[c["cache"]])
            s[n + "_exp"] = torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") if c["cache"] == "e4m3" else None
        elif c["cache"] == "e4m3":
            s[n], s[n + "_exp"] = _quantise(_activations(gen, shape))
        else:
            s[n], s[n + "_exp"] = _activations(gen, shape).to(torch.bfloat16), None
    return s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    kv, new = (torch.tensor(x)[torch.randperm(c["B"], generator=host)] for x in _lengths(c))
    reach = kv + new if c["op"] == "write" else kv
    need = [-(-int(t) // c["page"]) for t in reach]
    n_prefix = -(-c["prefix"] // c["page"])
    # as many pages for every pairing of old and new lengths
    n_pages = sum(-(-t // c["page"]) for x in _lengths(c)[:2 if c["op"] == "write" else 1] for t in x) + n_prefix + 3
    order = torch.randperm(n_pages, generator=host).to(torch.int32)
    table = torch.zeros((c["B"], max(1, max(need))), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s = {"case": c, "page_table": table.cuda(), "kv_len": kv.to(torch.int32).cuda(),
         "new": new.to(torch.int32).cuda() if c["ragged"] else None}
    s.update(_pool(c, gen, n_pages, c["op"] != "write"))
    dt = DTYPES[c["dtype"]]
    if c["op"] == "write":
        # K and V as slices of the fused projection's output
        fused = _activations(gen, (c["B"], c["L"], c["Hq"] + 2 * c["Hkv"], c["D"])).to(dt)
        s["new_k"], s["new_v"] = fused[:, :, c["Hq"]:c["Hq"] + c["Hkv"]], fused[:, :, c["Hq"] + c["Hkv"]:]
    elif c["op"] in ("decode", "prefix"):
        s["q"] = _activations(gen, (c["B"], c["L"], c["Hq"], c["D"])).to(dt)
        s["sinks"] = torch.randn(c["Hq"], generator=gen, device="cuda") if c["sinks"] else None
        s["prefix_table"] = order[at:at + n_prefix].cuda() if c["prefix"] else None
        s["prefix_len"] = torch.tensor([c["prefix"]], dtype=torch.int32, device="cuda") if c["prefix"] else None
        # rows behind a sequence's last new token stay as they are
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((c["B"], c["Hq"], c["L"]), device="cuda")
    if own:
        import block_sparse_flash_ra_gb300 as ra
        s["pool"] = ra.make_kv_cache(s["k"], s["v"], s["k_exp"], s["v_exp"])
        if c["op"] in ("decode", "prefix"):
            s["params"] = ra.make_paged_params(
                s["pool"], s["q"], s["page_table"], s["kv_len"], scale=c["D"] ** -0.5, causal=c["causal"],
                soft_cap=c["cap"], q_len=s["new"], sinks=s["sinks"], prefix_table=s["prefix_table"],
                prefix_len=s["prefix_len"])
    return s


# ---------------------------------------------------------------- plain forms
def _write(s):
    c, page = s["case"], s["case"]["page"]
    i = torch.arange(c["L"], device="cuda")
    pos = s["kv_len"][:, None] + i
    ok = (i < s["new"][:, None]) if s["new"] is not None else ...
    at = (s["page_table"].long().gather(1, (pos // page).clamp(max=s["page_table"].shape[1] - 1)), (pos % page).long())
    at = (at[0][ok].reshape(-1), at[1][ok].reshape(-1))
    out = {}
    for n in ("k", "v"):
        x = s["new_" + n][ok].reshape(-1, c["Hkv"], c["D"])
        if s["k_exp"] is not None:
            codes, byte = _quantise(x)
            s[n].view(torch.uint8)[at[0], :, at[1]] = codes.view(torch.uint8)
            s[n + "_exp"][at[0], :, at[1]] = byte
            out[n + "_exp"] = s[n + "_exp"]
        else:
            s[n][at[0], :, at[1]] = x.to(torch.bfloat16)
        out[n] = s[n]
    return out


def _gather(s, name, table):
    """(sequences, pages) of page numbers -> fp32 (sequences, kv heads, tokens, D)."""
    t = table.long()
    codes = s[name].view(torch.uint8)[t].view(s[name].dtype) if s["k_exp"] is not None else s[name][t]
    x = _rows(codes, s[name + "_exp"][t] if s["k_exp"] is not None else None)
    return x.transpose(1, 2).reshape(t.shape[0], x.shape[2], -1, x.shape[4])


def _read(s):
    c = s["case"]
    out = {}
    for n in ("k", "v"):
        x = _gather(s, n, s["page_table"])[:, :, :c["L"]]
        live = torch.arange(x.shape[2], device="cuda") < s["kv_len"][:, None]
        x = torch.where(live[:, None, :, None], x, 0.0)
        x = torch.nn.functional.pad(x, (0, 0, 0, c["L"] - x.shape[2]))
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
    j = torch.arange(T, device="cuda")
    i = torch.arange(L, device="cuda")
    n = s["new"] if s["new"] is not None else torch.full((B,), L, device="cuda")
    last = s["kv_len"][:, None] - 1 + ((i - n[:, None] + 1) if c["causal"] else torch.zeros_like(i))
    last = torch.minimum(last, s["kv_len"][:, None] - 1)
    seen = j <= last[..., None]  # B, L, T
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
    if c["op"] == "write":
        ra.kv_write(s["pool"], s["new_k"], s["new_v"], s["page_table"], s["kv_len"], s["new"])
        return {n: s[n] for n in ("k", "v", "k_exp", "v_exp") if s[n] is not None}
    if c["op"] == "read":
        k, v = ra.kv_read(s["pool"], s["page_table"], s["kv_len"], c["L"], DTYPES[c["dtype"]])
        return {"k": k, "v": v}
    out, lse = ra.paged_forward(s["params"], s["q"], s["pool"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"write": _write, "read": _read, "decode": _attend, "prefix": _attend}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _value64(s, name, pages, length):
    """Cached rows of the first `length` tokens of a list of pages: (length, kv heads, D) in fp64."""
    t = pages.long()
    x = s[name][t].double() if s["k_exp"] is None else s[name].view(torch.uint8)[t].view(s[name].dtype).double()
    if s["k_exp"] is not None:
        x = x * torch.pow(2.0, s[name + "_exp"][t].double() - 127)[..., None]
    return x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])[:length]


def _e4m3_64(y):
    """fp64 -> the nearest e4m3 value, ties to even: steps of an eighth of the binade, 2^-9 below 2^-6."""
    step = torch.pow(2.0, torch.floor(torch.log2(y.abs())).clamp(min=-6) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kv = s["kv_len"].tolist()
    new = [c["L"]] * c["B"] if s["new"] is None else s["new"].tolist()
    if c["op"] == "write":
        got = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for n in ("k", "v"):
            for b in range(c["B"]):
                pos = torch.arange(kv[b], kv[b] + new[b], device="cuda")
                x = s["new_" + n][b, :new[b]].double()
                if c["cache"] == "e4m3":
                    e = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 448))
                    x = _e4m3_64(x / torch.pow(2.0, e.clamp(min=MIN_EXP)))
                got[n][s["page_table"][b].long()[pos // c["page"]], :, pos % c["page"]] = x
        if c["cache"] == "e4m3":
            got.update(k_exp=None, v_exp=None)
        return got
    if c["op"] == "read":
        got = {n: torch.zeros((c["B"], c["L"], c["Hkv"], c["D"]), dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for n in ("k", "v"):
            for b in range(c["B"]):
                got[n][b, :kv[b]] = _value64(s, n, s["page_table"][b], kv[b])
        return got
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
