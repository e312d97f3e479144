"""Measured cases of the serving operators around the decode step:

* ``append``: new tokens enter the KV cache (contiguous or paged): keys and queries are
  rotated to their positions, keys and values stored in the cache's type, and the blocks
  that became full get their metadata;
* ``window``: attention over a sliding window and a few first tokens (sinks), for one new
  token per row (a decode step) or several (a chunk of a prompt);
* ``shared``: attention of a batch whose rows share one long prefix, kept once.

``own`` false: elementary torch operations in 32 bits (64 for angles and for values that
are rounded to a cache type); ``own`` true: the calls a serving program makes of
``learned_block_sparse_b200.binding.EtaDecoder``.
"""
import json
import math
import random

import torch

own = False

_KV = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
_BETA = 5.0  # gate temperature


# ------------------------------------------------------------------------- cases

def _case(op, kv, B, Hq, Hkv, d, bs, cap, new, paged, **more):
    c = dict(op=op, kv=kv, B=B, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap=cap, new=new, paged=paged)
    c.update(more)
    return c


def listed():
    return [
        # one decode step of a small batch: the latency of a single append
        dict(_case("append", "bf16", 8, 32, 8, 128, 32, 4096, 1, False, rot=128, pairs="halves"),
             name="append-step-b8"),
        # one decode step of a large continuous batch on an fp8 page pool
        dict(_case("append", "fp8", 256, 32, 8, 128, 32, 1024, 1, True, rot=128, pairs="halves"),
             name="append-step-b256-fp8-paged"),
        # prompt chunks of several requests, one of them decoding and one idle, into pages
        dict(_case("append", "bf16", 8, 32, 8, 128, 32, 4096, 2048, True, rot=128, pairs="halves"),
             name="append-chunk-paged"),
        # a full-precision cache, neighbouring pairs, half of the coordinates rotated
        dict(_case("append", "f32", 3, 16, 16, 64, 16, 2000, 1001, False, rot=32, pairs="neighbours"),
             name="append-prompt-f32-partial"),
        # batch-1 decode of a model with windowed layers
        dict(_case("window", "bf16", 1, 32, 8, 128, 32, 32768, 1, False, window=1024, sinks=4, gate=False, out="f32"),
             name="window-step-b1"),
        # a full decode batch on an fp8 page pool, rows of different lengths
        dict(_case("window", "fp8", 64, 32, 8, 128, 32, 8192, 1, True, window=4096, sinks=64, gate=False, out="bf16"),
             name="window-step-b64-fp8-paged"),
        # full precision with the learned thresholds' gate
        dict(_case("window", "f32", 4, 16, 16, 64, 16, 4000, 1, False, window=1000, sinks=1, gate=True, out="f32"),
             name="window-step-f32-gated"),
        # prompt chunks against caches that already hold tokens
        dict(_case("window", "bf16", 8, 32, 8, 128, 32, 8192, 1024, True, window=4096, sinks=4, gate=False, out="bf16"),
             name="window-chunk-paged"),
        # a few samples of one prompt
        dict(_case("shared", "bf16", 4, 32, 8, 128, 32, 256, 1, False, prefix=2003, gate=False, out="f32"),
             name="shared-step-b4"),
        # a serving batch behind one long system prompt
        dict(_case("shared", "bf16", 64, 32, 8, 128, 32, 1024, 1, True, prefix=32768, gate=False, out="bf16"),
             name="shared-step-b64"),
        # 32/4 heads of 64 with the gate, a prefix of 128K
        dict(_case("shared", "bf16", 32, 32, 4, 64, 64, 512, 1, False, prefix=131072, gate=True, out="bf16"),
             name="shared-step-d64-gated"),
        # several drafted tokens per row checked at once, on an fp8 page pool
        dict(_case("shared", "fp8", 16, 32, 8, 128, 32, 512, 4, True, prefix=8191, gate=False, out="bf16"),
             name="shared-verify-fp8-paged"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "append", "window", "window", "shared", "shared"))
    kv = rng.choice(("bf16", "bf16", "bf16", "fp8", "f32"))
    d = 128 if kv == "fp8" else rng.choice((64, 128, 128))
    Hkv = rng.choice((2, 4, 8, 8, 16)) if kv != "f32" else rng.choice((2, 4, 8))
    G = rng.choice([g for g in (1, 2, 4, 4, 8) if Hkv * g <= 32])
    bs = rng.choice((16, 32, 32, 64, 128))
    paged = rng.random() < 0.5
    few = rng.random() < (0.6 if kv != "f32" else 0.8)  # one token per row
    if op == "append":
        new = 1 if few else _log(rng, 3, 2048)
        B = _log(rng, 1, 256) if few else _log(rng, 1, 8)
        cap = _log(rng, 256, 1024) if few else _log(rng, max(new, 256), 4096)
        more = dict(rot=rng.choice((d, d, d // 2)), pairs=rng.choice(("halves", "halves", "neighbours")))
    else:
        new = 1 if few else _log(rng, 2, 1024 if kv == "bf16" else 64)
        B = _log(rng, 1, 64) if few else _log(rng, 1, 8)
        gate = rng.random() < 0.3
        out = "f32" if kv == "f32" else rng.choice(("bf16", "bf16", "f32"))
        more = dict(gate=gate, out=out)
        if op == "window":
            cap = _log(rng, max(new, 64), 8192)
            more.update(window=_log(rng, 16, 4096), sinks=rng.choice((0, 1, 4, 4, 64, rng.randint(2, 200))))
        else:
            new = min(new, 64)
            cap = _log(rng, max(new, 16), 1024)
            more.update(prefix=_log(rng, 100, 32768 if kv != "f32" else 4096))
    cap = -(-cap // bs) * bs
    return _case(op, kv, B, Hkv * G, Hkv, d, bs, cap, new, paged, **more)


def _rows(case):
    """[(new tokens, cached tokens with them)] of every row: fixed by the case."""
    r = random.Random("rows" + json.dumps([case[k] for k in ("op", "kv", "B", "Hq", "Hkv", "d", "bs", "cap", "new")]))
    rows = []
    for b in range(case["B"]):
        n = case["new"]
        if n > 1 and b > 0:
            n = r.randint(n // 2, n)
        if case["new"] > 1 and b == 2:
            n = 1                      # a row that is decoding
        if case["new"] > 1 and b == 3:
            n = 0                      # a row without new tokens
        old = r.randint(0, case["cap"] - n)
        if case["op"] == "append" and case["new"] == 1 and b % 5 == 0:
            old = max(0, old // case["bs"] * case["bs"] - 1)  # this token fills a block
        if case["op"] == "window" and case["new"] == 1 and b % 4 != 3:
            old = max(old, min(case["cap"] - n, case["window"] + case["sinks"]))
        rows.append((n, max(1, old + n)))
    return rows


# ----------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, Hq, Hkv, d, bs, cap = (case[k] for k in ("B", "Hq", "Hkv", "d", "bs", "cap"))
    kvt = _KV[case["kv"]]
    qt = torch.float32 if case["kv"] == "f32" else torch.bfloat16
    rows = _rows(case)
    T = sum(n for n, _ in rows)

    def normal(*shape, scale=1.0, to=qt):
        return torch.empty(shape, dtype=torch.float32, device=dev).normal_(0.0, scale, generator=g).to(to)

    nb = cap // bs
    prefix = case.get("prefix", 0)
    pb = -(-prefix // bs)  # blocks of the prefix
    s = dict(case=dict(case), T=T, rows=rows)
    offset = normal(Hkv, 1, d, to=torch.float32)  # keys have a mean per coordinate

    def store(*lead):
        k = (normal(*lead, Hkv, bs if case["paged"] else lead_len, d, to=torch.float32) + offset).to(kvt)
        v = normal(*lead, Hkv, bs if case["paged"] else lead_len, d, to=torch.float32).to(kvt)
        return k, v

    lead_len = cap
    if case["paged"]:
        pages = B * nb + pb + 3
        s["K"], s["V"] = store(pages)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        s["table"], s["pages"] = order[: B * nb].view(B, nb).contiguous(), pages
        s["prefix_blocks"] = order[B * nb: B * nb + pb].contiguous()
    else:
        s["K"], s["V"] = store(B)
        s["table"], s["pages"], s["prefix_blocks"] = None, 0, None
        if prefix:
            lead_len = prefix
            s["PK"], s["PV"] = (x.contiguous() for x in store())
    s["lens"] = torch.tensor([n for _, n in rows], dtype=torch.int32, device=dev)
    cu = [0]
    for n, _ in rows:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if case["new"] > 1 else None
    if case["op"] == "append":
        # a fused projection's output: each token's q, k and v side by side
        qkv = normal(T, (Hq + 2 * Hkv) * d)
        s["q"] = qkv[:, : Hq * d].view(T, Hq, d)
        s["k"] = (qkv[:, Hq * d: (Hq + Hkv) * d].view(T, Hkv, d)).add_(offset.view(Hkv, d).to(qt))
        s["v"] = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = (500000.0 ** (-2.0 * i / case["rot"])).float()
        s["mu"] = torch.zeros((B, Hkv, d, nb), dtype=torch.float32, device=dev)
        s["var"] = torch.zeros_like(s["mu"])
        s["maxnorm"] = torch.zeros((B, Hkv, nb), dtype=torch.float32, device=dev)
        s["q_out"] = torch.zeros((T, Hq, d), dtype=qt, device=dev)
    else:
        s["q"] = normal(T, Hq, d, scale=1.5)
        s["tau"] = normal(T, Hq, scale=0.5, to=torch.float32) if case["gate"] else None
        s["out"] = torch.zeros((T, Hq, d), dtype=_KV[case["out"]], device=dev)
    if own:
        from learned_block_sparse_b200 import binding
        dec = binding.EtaDecoder(B, Hq, Hkv, d, bs, cap, kv_dtype=kvt, q_dtype=qt, beta=_BETA)
        s["dec"] = dec
        if case["op"] == "append":
            dec.mu, dec.var, dec.maxnorm = s["mu"], s["var"], s["maxnorm"]
            s["rope"] = binding.Rope(s["inv_freq"], interleaved=case["pairs"] == "neighbours")
        else:
            dec.reserve_queries(T)
        if prefix:
            s["prefix"] = (binding.Prefix(prefix, blocks=s["prefix_blocks"]) if case["paged"]
                           else binding.Prefix(prefix, k=s["PK"], v=s["PV"]))
    return s


# ------------------------------------------------------------- the framework's calls

def _run_own(s):
    c, dec = s["case"], s["dec"]
    pages = dict(block_table=s["table"], num_pages=s["pages"]) if c["paged"] else {}
    if c["op"] == "append":
        q_out = dec.append(s["k"], s["v"], s["K"], s["V"], c["cap"], q=s["q"], rope=s["rope"], seq_lens=s["lens"],
                           cu_new=s["cu"], q_out=s["q_out"], **pages)
        return dict(q=q_out, K=s["K"], V=s["V"], mu=s["mu"], var=s["var"], maxnorm=s["maxnorm"])
    if c["op"] == "window":
        return dec.window(s["q"], s["K"], s["V"], c["cap"], c["window"], sinks=c["sinks"], seq_lens=s["lens"],
                          cu_q=s["cu"], tau=s["tau"], out=s["out"], **pages)
    return dec.shared(s["q"], s["K"], s["V"], c["cap"], s["prefix"], seq_lens=s["lens"], cu_q=s["cu"], tau=s["tau"],
                      out=s["out"], **pages)


# -------------------------------------------------------------------- plain forms

def _to_kv(x, kvt):
    """fp64 values rounded once to the cache's type: to 32 bits with the last bit set
    where anything was cut off, which the second rounding then cannot mistake for a tie."""
    if kvt == torch.float32:
        return x.float()
    f = x.float()
    r = f.double()
    bits = f.view(torch.int32)
    bits = torch.where(r.abs() > x.abs(), bits - 1, bits)
    bits = torch.where(r != x, bits | 1, bits)
    f = bits.view(torch.float32)
    return f.clamp(-448.0, 448.0).to(kvt) if kvt == torch.float8_e4m3fn else f.to(kvt)


def _bytes_of(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _rotate(x, cos, sin, rot, pairs):
    """x [T][H][d] in 64 bits."""
    if pairs == "halves":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    u, w = a * cos - b * sin, b * cos + a * sin
    if pairs == "halves":
        y = torch.cat((u, w), dim=-1)
    else:
        y = torch.stack((u, w), dim=-1).flatten(-2)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _plain_append(s):
    c = s["case"]
    bs, kvt, K, V = c["bs"], _KV[c["kv"]], s["K"], s["V"]
    T, lens = s["T"], s["lens"].long()
    t = torch.arange(T, device=K.device)
    if s["cu"] is None:
        row, start, fresh = t, t, torch.ones_like(lens)
    else:
        cu = s["cu"].long()
        row = torch.searchsorted(cu[1:], t, right=True)
        start, fresh = cu[row], cu[1:] - cu[:-1]
    pos = (lens - fresh)[row] + t - start
    ang = pos[:, None, None].double() * s["inv_freq"].double()
    cos, sin = torch.cos(ang), torch.sin(ang)
    q = _rotate(s["q"].double(), cos, sin, c["rot"], c["pairs"]).to(s["q"].dtype)
    k = _to_kv(_rotate(s["k"].double(), cos, sin, c["rot"], c["pairs"]), kvt)
    v = _to_kv(s["v"].double(), kvt)
    at = (s["table"].long()[row, pos // bs], pos % bs) if c["paged"] else (row, pos)
    for cache, x in ((K, k), (V, v)):
        _bytes_of(cache)[at[0], :, at[1]] = _bytes_of(x)
    # metadata of the blocks that this append filled: at most new // bs + 1 of a row
    nb, most = c["cap"] // bs, c["new"] // bs + 1
    blk = (lens - fresh)[:, None] // bs + torch.arange(most, device=K.device)
    full = blk < (lens // bs)[:, None]
    j = blk.clamp(max=nb - 1)
    b = torch.arange(c["B"], device=K.device)[:, None]
    if c["paged"]:
        keys = _bytes_of(K)[s["table"].long()[b, j]]                        # [B][most][Hkv][bs][d]
    else:
        keys = _bytes_of(K).view(c["B"], c["Hkv"], nb, bs, c["d"])[b, :, j]  # the same
    keys = (keys.view(kvt) if kvt == torch.float8_e4m3fn else keys).float()
    mu = keys.mean(dim=3)
    var = (keys - mu[:, :, :, None]).square().mean(dim=3)
    norm = keys.square().sum(dim=-1).amax(dim=-1).sqrt()
    j = torch.where(full, j, torch.full_like(j, nb))                        # unfilled: a column that is dropped
    for dst, x in ((s["mu"], mu), (s["var"], var), (s["maxnorm"], norm)):
        wide = torch.cat((dst, dst[..., :1]), dim=-1)
        wide.movedim(-1, 1)[b, j] = x
        dst.copy_(wide[..., :nb])
    s["q_out"].copy_(q)
    return dict(q=s["q_out"], K=K, V=V, mu=s["mu"], var=s["var"], maxnorm=s["maxnorm"])


def _gather(s, name, pos):
    """Rows of the cache at pos [B][L], as [B][Hkv][L][d] in 32 bits."""
    c, cache = s["case"], s[name]
    b = torch.arange(c["B"], device=pos.device)[:, None]
    if c["paged"]:
        x = _bytes_of(cache)[s["table"].long()[b, pos // c["bs"]], :, pos % c["bs"]]
    else:
        x = _bytes_of(cache)[b, :, pos]
    x = x.view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else x
    return x.float().transpose(1, 2)


def _padded(s):
    """Queries as [B][n][Hq][d] with their positions [B][n], their thresholds and their places in the batch."""
    c, lens = s["case"], s["lens"].long()
    i = torch.arange(c["new"], device=lens.device)
    if s["cu"] is None:
        start, fresh = torch.arange(c["B"], device=lens.device), torch.ones_like(lens)
    else:
        cu = s["cu"].long()
        start, fresh = cu[:-1], cu[1:] - cu[:-1]
    at = (start[:, None] + i).clamp(max=s["T"] - 1)
    pos = (lens - fresh)[:, None] + i
    tau = None if s["tau"] is None else s["tau"][at]
    return s["q"][at].float(), pos, tau


def _unpadded(s, x):
    """[B][n][Hq][d] back to the packed [T][Hq][d]."""
    if s["cu"] is None:
        return x[:, 0]
    t = torch.arange(s["T"], device=x.device)
    cu = s["cu"].long()
    row = torch.searchsorted(cu[1:], t, right=True)
    return x[row, t - cu[row]]


def _gated(S, tau, exempt):
    if tau is None:
        return S
    g = S / (1.0 + torch.exp(-_BETA * (S - tau)))
    return g if exempt is None else torch.where(exempt, S, g)


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, d, n = c["B"], c["Hq"], c["Hkv"], c["d"], c["new"]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    q, pos, tau = _padded(s)
    lens = s["lens"].long()
    window, sinks = c.get("window", c["cap"]), c.get("sinks", 0)
    # the positions that some query of the row can see: the sinks, then the window's span
    span = min(c["cap"], window + n - 1)
    lo = (lens - span).clamp(min=0)
    key = torch.arange(sinks, device=q.device).clamp(max=c["cap"] - 1).expand(B, sinks)
    key = torch.cat((key, (lo[:, None] + torch.arange(span, device=q.device)).clamp(max=c["cap"] - 1)), dim=1)
    first = torch.arange(sinks + span, device=q.device) < sinks                       # which part an entry is of
    u = torch.arange(sinks + span, device=q.device)
    real = torch.where(first, u, lo[:, None] + u - sinks)                             # before the clamp
    p = pos[:, :, None]
    r = real[:, None, :]
    seen = (r <= p) & torch.where(first, r < sinks, (r > p - window) & (r >= sinks))  # [B][n][L]
    dead = ~seen.any(dim=1)[:, None, :, None]                                         # rows past the last token may hold anything
    k, v = _gather(s, "K", key), _gather(s, "V", key).masked_fill(dead, 0.0)
    qg = q.view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    tg = None if tau is None else tau.view(B, n, Hkv, G).permute(0, 2, 3, 1).reshape(B, Hkv, G * n, 1)
    S = torch.matmul(qg, k.transpose(-1, -2)) * scale
    own_key = (r == p).repeat(1, G, 1)[:, None]
    g = _gated(S, tg, own_key).masked_fill_(~seen.repeat(1, G, 1)[:, None], float("-inf"))
    m = g.amax(dim=-1, keepdim=True)
    if c["op"] == "shared":
        if c["paged"]:
            e = torch.arange(c["prefix"], device=q.device)
            at = (s["prefix_blocks"].long()[e // c["bs"]], e % c["bs"])
            PK, PV = (_bytes_of(s[x])[at[0], :, at[1]].view(s[x].dtype).float().transpose(0, 1) for x in ("K", "V"))
        else:
            PK, PV = s["PK"].float(), s["PV"].float()
        qp = qg.transpose(0, 1).reshape(Hkv, B * G * n, d)
        tp = None if tg is None else tg.transpose(0, 1).reshape(Hkv, B * G * n, 1)
        gp = _gated(torch.matmul(qp, PK.transpose(-1, -2)) * scale, tp, None)
        mp = gp.amax(dim=-1, keepdim=True)
        m = torch.maximum(m, mp.view(Hkv, B, G * n, 1).transpose(0, 1))
        m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
        ep = torch.exp(gp - m.transpose(0, 1).reshape(Hkv, B * G * n, 1))
        num = torch.matmul(ep, PV).view(Hkv, B, G * n, d).transpose(0, 1)
        den = ep.sum(dim=-1, keepdim=True).view(Hkv, B, G * n, 1).transpose(0, 1)
        e = torch.exp(g - m)
        o = (torch.matmul(e, v) + num) / (e.sum(dim=-1, keepdim=True) + den)
    else:
        m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
        e = torch.exp(g - m)
        o = torch.matmul(e, v) / e.sum(dim=-1, keepdim=True)
    o = o.view(B, Hkv, G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, d)
    return _unpadded(s, o).to(_KV[c["out"]])


def run(state):
    if own:
        return _run_own(state)
    if state["case"]["op"] == "append":
        return _plain_append(state)
    return _plain_attend(state)


# --------------------------------------------------------------------------- work

def work(case):
    B, Hq, Hkv, d, bs = (case[k] for k in ("B", "Hq", "Hkv", "d", "bs"))
    kb = {"f32": 4, "bf16": 2, "fp8": 1}[case["kv"]]
    qb = 4 if case["kv"] == "f32" else 2
    rows = _rows(case)
    T = sum(n for n, _ in rows)
    if case["op"] == "append":
        moved = T * d * (2 * Hq * qb + 2 * Hkv * (qb + kb))
        for n, length in rows:
            b0, b1 = (length - n) // bs, length // bs
            if n and b1 > b0:  # full blocks: their earlier keys are read, their metadata written
                moved += Hkv * (((length - n) - b0 * bs) * d * kb + (b1 - b0) * (2 * d + 1) * 4)
        return {"bytes": moved, "flops": T * (Hq + Hkv) * case["rot"] * 3}
    ob = 4 if case["out"] == "f32" else 2
    moved, pairs = T * Hq * d * (qb + ob), 0
    window, sinks = case.get("window", case["cap"]), case.get("sinks", 0)
    for n, length in rows:
        if n == 0:
            continue
        p0 = length - n
        lo = max(0, p0 - window + 1)
        moved += 2 * Hkv * d * kb * (length - lo + min(sinks, lo))
        for p in range(p0, length):
            w = max(0, p - window + 1)
            pairs += p + 1 - w + min(sinks, w)
    if case["op"] == "shared":
        moved += 2 * Hkv * d * kb * case["prefix"]
        pairs += T * case["prefix"]
    return {"bytes": moved, "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------------- 64 bits

def _grid(x, bits, least):
    """x rounded (ties to even) to `bits` significant bits, with 2**least the smallest step."""
    e = torch.frexp(x).exponent.double()
    step = torch.exp2(torch.clamp(e - bits, min=least))
    return torch.round(x / step) * step


def _stored(x, kv):
    if kv == "f32":
        return x.float().double()
    if kv == "bf16":
        return _grid(x, 8, -133)
    return _grid(x, 4, -9).clamp(-448.0, 448.0)


def _exact_append(case, s):
    bs, rot, dev = case["bs"], case["rot"], s["K"].device
    K, V = s["K"].float().double(), s["V"].float().double()
    q_out = s["q"].double().clone()
    mu, var, norm = (s[x].double() for x in ("mu", "var", "maxnorm"))
    f = s["inv_freq"].double()
    t0 = 0
    for b, (n, length) in enumerate(s["rows"]):
        if n == 0:
            continue
        pos = torch.arange(length - n, length, device=dev)
        turn = torch.polar(torch.ones((n, 1, rot // 2), dtype=torch.float64, device=dev),
                           pos[:, None, None].double() * f)
        new = []
        for x in (s["q"], s["k"]):
            x = x[t0: t0 + n].double()
            y = x.clone()
            i = torch.arange(rot // 2, device=dev)
            i, j = (i, i + rot // 2) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
            z = torch.complex(x[..., i], x[..., j]) * turn
            y[..., i], y[..., j] = z.real, z.imag
            new.append(y)
        q_out[t0: t0 + n] = new[0]
        k, v = _stored(new[1], case["kv"]), _stored(s["v"][t0: t0 + n].double(), case["kv"])
        if case["paged"]:
            page = s["table"][b].long()[pos // bs]
            K[page, :, pos % bs], V[page, :, pos % bs] = k, v
        else:
            K[b, :, pos], V[b, :, pos] = k.transpose(0, 1), v.transpose(0, 1)
        for j in range((length - n) // bs, length // bs):
            keys = K[int(s["table"][b, j])] if case["paged"] else K[b, :, j * bs: (j + 1) * bs]
            mu[b, :, :, j] = keys.mean(dim=1)
            var[b, :, :, j] = keys.var(dim=1, correction=0)
            norm[b, :, j] = torch.linalg.vector_norm(keys, dim=-1).amax(dim=-1)
        t0 += n
    return dict(q=q_out, K=K, V=V, mu=mu, var=var, maxnorm=norm)


def _exact_row(case, s, b, length):
    """The row's own K and V, [Hkv][length][d] in 64 bits."""
    out = []
    for x in (s["K"], s["V"]):
        if case["paged"]:
            used = s["table"][b, : -(-length // case["bs"])].long()
            x = _bytes_of(x)[used].view(x.dtype).float().double()       # [blocks][Hkv][bs][d]
            x = x.transpose(0, 1).reshape(case["Hkv"], -1, case["d"])
        else:
            x = x[b].float().double()
        out.append(x[:, :length])
    return out


def _exact_attend(case, s):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    G = Hq // Hkv
    out = torch.zeros((s["T"], Hq, d), dtype=torch.float64, device=s["q"].device)
    prefix = case.get("prefix", 0)
    if prefix and case["paged"]:
        used = s["prefix_blocks"].long()
        pk, pv = (_bytes_of(s[x])[used].view(s[x].dtype).float().double().transpose(0, 1).reshape(Hkv, -1, d)[:, :prefix]
                  for x in ("K", "V"))
    elif prefix:
        pk, pv = s["PK"].float().double(), s["PV"].float().double()
    t0 = 0
    for b, (n, length) in enumerate(s["rows"]):
        if n == 0:
            continue
        k, v = _exact_row(case, s, b, length)
        place = torch.arange(length, device=k.device)
        p = torch.arange(length - n, length, device=k.device)[:, None]
        seen = (place <= p) & ((place < case.get("sinks", 0)) | (place > p - case.get("window", length)))
        for h in range(Hq):
            kh, vh = k[h // G], v[h // G]
            see, mine = seen, place == p
            if prefix:
                kh, vh = torch.cat((pk[h // G], kh)), torch.cat((pv[h // G], vh))
                see = torch.cat((torch.ones((n, prefix), dtype=torch.bool, device=k.device), seen), dim=1)
                mine = torch.cat((torch.zeros((n, prefix), dtype=torch.bool, device=k.device), mine), dim=1)
            S = s["q"][t0: t0 + n, h].double() @ kh.T / math.sqrt(d)
            if s["tau"] is not None:
                S = torch.where(mine, S, S * torch.sigmoid(_BETA * (S - s["tau"][t0: t0 + n, h, None].double())))
            out[t0: t0 + n, h] = torch.softmax(S.masked_fill(~see, -math.inf), dim=-1) @ vh
        t0 += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attend(case, s)
