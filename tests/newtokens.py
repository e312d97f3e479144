"""64-bit references and problem builders for the calls that take new tokens
(append, windowed and shared-prefix attention)."""
from __future__ import annotations

import dataclasses
import math

import torch

from learned_block_sparse_b200 import binding

KV = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
BETA = 5.0


def raw(t):
    """fp8 tensors as bytes (indexing works on every type then)."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def wide(t):
    return t.float().double()


@dataclasses.dataclass
class Case:
    kv: str = "bf16"
    q: str = "bf16"
    Hq: int = 8
    Hkv: int = 2
    d: int = 128
    bs: int = 32
    cap: int = 512
    paged: bool = False
    rows: tuple = ((1, 100),)     # (new tokens, cached tokens with them) per row
    packed: bool = False          # cu given
    seed: int = 0
    pad: int = 0                  # packed tokens past the last row's

    @property
    def B(self):
        return len(self.rows)

    @property
    def T(self):
        return sum(n for n, _ in self.rows) + self.pad if self.packed else self.B


def make(c: Case, prefix: int = 0, device="cuda"):
    """Cache, pages, lengths and offsets of a case; every cache row past a row's last
    token, and every page that no row uses, holds NaN."""
    g = torch.Generator().manual_seed(c.seed + 1000)
    nb, pb = c.cap // c.bs, -(-prefix // c.bs)
    nan = float("nan")

    def normal(*shape, mean=None):
        x = torch.randn(shape, generator=g)
        return x if mean is None else x + mean

    mean = torch.randn((c.Hkv, 1, c.d), generator=g)
    K = normal(c.B, c.Hkv, c.cap, c.d, mean=mean)
    V = normal(c.B, c.Hkv, c.cap, c.d)
    for b, (n, length) in enumerate(c.rows):
        K[b, :, length:], V[b, :, length:] = nan, nan
    PK, PV = normal(c.Hkv, max(prefix, 1), c.d, mean=mean), normal(c.Hkv, max(prefix, 1), c.d)
    p = dict(case=c, prefix_len=prefix, PK=PK.to(KV[c.kv]).to(device), PV=PV.to(KV[c.kv]).to(device))
    p["K_rows"], p["V_rows"] = K.to(KV[c.kv]).to(device), V.to(KV[c.kv]).to(device)
    if c.paged:
        pages = c.B * nb + pb + 2
        order = torch.randperm(pages, generator=g)
        pools = []
        for rows, pre in ((K, PK), (V, PV)):
            pool = torch.full((pages, c.Hkv, c.bs, c.d), nan)
            pool[order[: c.B * nb]] = rows.view(c.B, c.Hkv, nb, c.bs, c.d).transpose(1, 2).reshape(-1, c.Hkv, c.bs, c.d)
            full = torch.full((c.Hkv, pb * c.bs, c.d), nan)
            full[:, :prefix] = pre[:, :prefix]
            pool[order[c.B * nb: c.B * nb + pb]] = full.view(c.Hkv, pb, c.bs, c.d).transpose(0, 1)
            pools.append(pool.to(KV[c.kv]).to(device))
        p["K"], p["V"] = pools
        p["table"] = order[: c.B * nb].view(c.B, nb).to(torch.int32).to(device)
        p["blocks"] = order[c.B * nb: c.B * nb + pb].to(torch.int32).to(device)
        p["page_args"] = dict(block_table=p["table"], num_pages=pages)
        p["prefix"] = binding.Prefix(prefix, blocks=p["blocks"])
    else:
        p["K"], p["V"], p["page_args"], p["table"] = p["K_rows"].clone(), p["V_rows"].clone(), {}, None
        p["prefix"] = binding.Prefix(prefix, k=p["PK"], v=p["PV"])
    p["lens"] = torch.tensor([n for _, n in c.rows], dtype=torch.int32, device=device)
    cu = [0]
    for n, _ in c.rows:
        cu.append(cu[-1] + n)
    p["cu_list"] = cu if c.packed else list(range(c.B + 1))
    p["cu"] = torch.tensor(cu, dtype=torch.int32, device=device) if c.packed else None
    p["q"] = (1.5 * torch.randn((c.T, c.Hq, c.d), generator=g)).to(KV[c.q]).to(device)
    p["tau"] = (0.5 * torch.randn((c.T, c.Hq), generator=g)).to(device)
    return p


def decoder(c: Case, **kw):
    return binding.EtaDecoder(c.B, c.Hq, c.Hkv, c.d, c.bs, c.cap, kv_dtype=KV[c.kv], q_dtype=KV[c.q], beta=BETA,
                              n_splits=4, **kw)


def reference(p, window=None, sinks=0, gated=False, hard=False, prefix=False):
    """(out, tolerance scale) of every live token in 64 bits: out [T][Hq][d], and per
    entry what a relative error of every weight, of every logit's terms, and of every
    addition can move it by (see bound())."""
    c = p["case"]
    G = c.Hq // c.Hkv
    T = p["q"].shape[0]
    dev = p["q"].device
    out = torch.full((T, c.Hq, c.d), float("nan"), dtype=torch.float64, device=dev)
    mass = torch.zeros_like(out)                                            # sum of weight x |v|
    info = torch.zeros((T, c.Hq, 4), dtype=torch.float64, device=dev)       # |q||k| sums, |g|, keys, largest |v|
    P = p["prefix_len"] if prefix else 0
    for b, (n, length) in enumerate(c.rows):
        n = n if c.packed else (1 if length else 0)
        t0 = p["cu_list"][b]
        if n == 0:
            continue
        k, v = wide(p["K_rows"][b][:, :length]), wide(p["V_rows"][b][:, :length])
        place = torch.arange(length, device=dev)
        pos = torch.arange(length - n, length, device=dev)[:, None]
        w = length if window is None else window
        seen = (place <= pos) & ((place < sinks) | (place > pos - w))
        own = place == pos
        if P:
            k = torch.cat((wide(p["PK"][:, :P]), k), dim=1)
            v = torch.cat((wide(p["PV"][:, :P]), v), dim=1)
            seen = torch.cat((torch.ones((n, P), dtype=torch.bool, device=dev), seen), dim=1)
            own = torch.cat((torch.zeros((n, P), dtype=torch.bool, device=dev), own), dim=1)
        qh = wide(p["q"][t0: t0 + n]).transpose(0, 1)                        # [Hq][n][d]
        kh, vh = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        S = qh @ kh.transpose(1, 2) / math.sqrt(c.d)
        g = S
        gain = torch.ones_like(S)
        if gated:
            tau = p["tau"][t0: t0 + n].double().T[:, :, None]
            if hard:
                g = torch.where(own | (S >= tau), S, torch.full_like(S, -math.inf))
            else:
                s = torch.sigmoid(BETA * (S - tau))
                g = torch.where(own, S, S * s)
                gain = 1 + BETA * S.abs() / 4
        e = torch.softmax(torch.where(seen, g, torch.full_like(g, -math.inf)), dim=-1)
        out[t0: t0 + n] = (e @ vh).transpose(0, 1)
        mass[t0: t0 + n] = (e @ vh.abs()).transpose(0, 1)
        terms = qh.abs() @ kh.abs().transpose(1, 2) / math.sqrt(c.d)
        amax = qh.abs().amax(-1, keepdim=True) * kh.abs().sum(-1)[:, None] / math.sqrt(c.d)
        scale = {"fp8": 2.0 ** -21 * amax}.get(c.kv, 0.0 * amax) + c.d * 2.0 ** -22 * terms
        dead = ~seen | ~torch.isfinite(g)
        info[t0: t0 + n, :, 0] = (gain * scale).masked_fill(dead, 0).amax(-1).T
        info[t0: t0 + n, :, 1] = g.abs().masked_fill(dead, 0).amax(-1).T
        info[t0: t0 + n, :, 2] = seen.sum(-1).double()[:, None]
        info[t0: t0 + n, :, 3] = vh.abs().nan_to_num(0.0).amax((-1, -2))
    return out, mass, info


def bound(out, mass, info, out_dtype, floor=0.0):
    """How far a result may be from the 64-bit one. A weight's relative error is the
    error of its logit (d products and additions of 2^-22 each, fp8 queries held to
    2^-21 of their largest; times the gate's slope), plus its own evaluation (2^-22,
    and 2^-23 of the exponent for its rounding), and enters the numerator and the
    denominator: twice. `floor`: what a weight may lose however small it is (of the
    largest weight, which is at most the sum), times the N keys' largest value. Sums over N keys add N 2^-23. Weights that meet values as
    bf16 numbers are off by 2^-8 each (bf16 output), as two bf16 numbers by 2^-16
    (fp32 output). Every error is weighted by sum w |v|. Then the output's rounding."""
    rel = 2 * (info[..., 0] + 2.0 ** -22 + 2.0 ** -23 * info[..., 1]) + 2.0 ** -23 * info[..., 2]
    rel = rel + (2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -16)
    last = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24
    tol = rel[..., None] * mass + floor * info[..., 2, None] * info[..., 3, None]
    return tol + last * (out.abs() + tol)


def live_tokens(c: Case):
    live = torch.zeros(c.T, dtype=torch.bool)
    cu = 0
    for b, (n, length) in enumerate(c.rows):
        if c.packed:
            live[cu: cu + n] = True
            cu += n
        else:
            live[b] = length > 0
    return live


def check(p, got, ref, fill, floor=0.0):
    """Live tokens within the bound, every other output as it was (`fill`)."""
    out, mass, info = ref
    live = live_tokens(p["case"]).to(got.device)
    x = got.float().double()
    assert torch.equal(got[~live], torch.full_like(got[~live], fill))
    err = (x - out).abs()[live]
    tol = bound(out, mass, info, got.dtype, floor)[live]
    assert torch.isfinite(x[live]).all()
    # an output that is exactly zero (one visible key, a zero value) has no room at all
    worst = torch.where(err == 0, torch.zeros_like(err), err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.3g} times the bound"
    return worst
