"""eta_append_kv against its definition in 64 bits: stored keys and values bit for
bit (the rotation rounded once), rotated queries within their rounding, metadata
equal to eta_build_block_meta's bits, and nothing else written."""
import dataclasses

import pytest
import torch

from learned_block_sparse_b200 import binding
from tests.newtokens import KV, Case, decoder, make, raw, wide

pytestmark = pytest.mark.gpu

STEP = (((1, 1), (1, 32), (1, 33), (1, 0), (1, 512), (1, 64)), False)
CHUNK = (((40, 40), (1, 64), (0, 17), (100, 333), (31, 512), (64, 128), (3, 33)), True)


def rounded_once(x, kv):
    """fp64 -> cache type, ties to even, by exact arithmetic on the type's grid."""
    if kv == "f32":
        return x.float()
    bits, least = (8, -133) if kv == "bf16" else (4, -9)
    e = torch.frexp(x).exponent.double()
    step = torch.exp2(torch.clamp(e - bits, min=least))
    y = torch.round(x / step) * step
    if kv == "fp8":
        y = y.clamp(-448.0, 448.0)
    return y.float().to(KV[kv])          # exact: y is on the grid


def rotate(x, pos, inv_freq, interleaved):
    """x [n][H][d] in 64 bits, turned as complex numbers."""
    half = inv_freq.numel()
    i = torch.arange(half, device=x.device)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a = pos[:, None, None].double() * inv_freq.double()
    z = torch.complex(x[..., i], x[..., j]) * torch.polar(torch.ones_like(a), a)
    y = x.clone()
    y[..., i], y[..., j] = z.real, z.imag
    return y


def inputs(c, strided, seed=5):
    g = torch.Generator().manual_seed(seed)
    wide_row = (c.Hq + 2 * c.Hkv) * c.d
    x = torch.randn((c.T, wide_row + (64 if strided else 0)), generator=g).to(KV[c.q]).cuda()
    q = x[:, : c.Hq * c.d].view(c.T, c.Hq, c.d)
    k = x[:, c.Hq * c.d: (c.Hq + c.Hkv) * c.d].view(c.T, c.Hkv, c.d)
    v = x[:, (c.Hq + c.Hkv) * c.d: wide_row].view(c.T, c.Hkv, c.d)
    return (q, k, v) if strided else (q.contiguous(), k.contiguous(), v.contiguous())


def expected_caches(c, p, k, v, inv_freq, interleaved):
    """Row-major caches [B][Hkv][cap][d] after the append."""
    K, V = p["K_rows"].clone(), p["V_rows"].clone()
    for b, (n, length) in enumerate(c.rows):
        n = n if c.packed else min(1, length)
        if n == 0:
            continue
        t0 = p["cu_list"][b]
        pos = torch.arange(length - n, length, device=K.device)
        kk = wide(k[t0: t0 + n])
        kk = kk if inv_freq is None else rotate(kk, pos, inv_freq, interleaved)
        raw(K)[b, :, length - n: length] = raw(rounded_once(kk, c.kv)).transpose(0, 1)
        raw(V)[b, :, length - n: length] = raw(rounded_once(wide(v[t0: t0 + n]), c.kv)).transpose(0, 1)
    return K, V


def rows_of(p, name):
    """A cache or pool as [B][Hkv][cap][d]."""
    c = p["case"]
    if not c.paged:
        return p[name]
    x = raw(p[name])[p["table"].long().view(-1)].view(c.B, -1, c.Hkv, c.bs, c.d).transpose(1, 2)
    return x.reshape(c.B, c.Hkv, c.cap, c.d).view(p[name].dtype)


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


@pytest.mark.parametrize("kv,q,Hq,Hkv,d,bs,paged,rot,interleaved,shape,strided", [
    ("bf16", "bf16", 8, 2, 128, 32, False, 128, False, STEP, True),
    ("bf16", "bf16", 8, 2, 128, 32, True, 128, False, CHUNK, True),
    ("bf16", "bf16", 4, 4, 64, 16, True, 64, True, CHUNK, False),
    ("bf16", "bf16", 8, 1, 64, 64, False, 32, False, CHUNK, True),
    ("bf16", "bf16", 2, 1, 128, 128, True, 96, True, CHUNK, False),
    ("bf16", "f32", 4, 2, 128, 32, False, 64, False, CHUNK, True),
    ("f32", "f32", 4, 4, 64, 16, False, 32, True, CHUNK, True),
    ("f32", "f32", 6, 3, 128, 32, True, 128, False, STEP, False),
    ("f32", "bf16", 4, 2, 64, 64, False, 16, False, CHUNK, False),
    ("fp8", "bf16", 8, 2, 128, 32, True, 128, False, STEP, True),
    ("fp8", "bf16", 24, 3, 128, 64, False, 128, False, CHUNK, True),
    ("bf16", "bf16", 8, 2, 128, 32, False, 0, False, CHUNK, True),
])
def test_append_against_the_definition(kv, q, Hq, Hkv, d, bs, paged, rot, interleaved, shape, strided):
    rows, packed = shape
    c = Case(kv=kv, q=q, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap=512, paged=paged, rows=rows, packed=packed,
             pad=3 if packed else 0, seed=bs + rot)
    p = make(c)
    qn, kn, vn = inputs(c, strided)
    inv = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float().cuda() if rot else None
    dec = decoder(c)
    for t in dec.meta:
        t.fill_(-7.0)
    q_out = torch.full((c.T, Hq, d), -3.0, dtype=KV[q], device="cuda")
    want_K, want_V = expected_caches(c, p, kn, vn, inv, interleaved)
    dec.append(kn, vn, p["K"], p["V"], c.cap, q=qn, rope=None if inv is None else binding.Rope(inv, interleaved),
               seq_lens=p["lens"], cu_new=p["cu"], q_out=q_out, **p["page_args"])
    torch.cuda.synchronize()
    assert dec.device_status() == 0
    # caches: every row, written or not (NaN past the ends), bit for bit
    assert torch.equal(bits(rows_of(p, "K")), bits(want_K))
    assert torch.equal(bits(rows_of(p, "V")), bits(want_V))
    # queries: one rounding, after an fp32 product sum (three roundings of 2^-24)
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[q]
    for b, (n, length) in enumerate(rows):
        n = n if packed else min(1, length)
        t0 = p["cu_list"][b]
        pos = torch.arange(length - n, length, device="cuda")
        x = wide(qn[t0: t0 + n])
        want = x if inv is None else rotate(x, pos, inv, interleaved)
        size = x.abs().amax(-1, keepdim=True)      # both members of a pair are at most this
        tol = half * want.abs() + 8 * 2.0 ** -24 * size
        assert ((wide(q_out[t0: t0 + n]) - want).abs() <= tol).all(), b
        if not packed and n == 0:
            assert (q_out[b] == -3.0).all()
    if packed:
        assert (q_out[c.T - c.pad:] == -3.0).all()
    # metadata of the blocks that became full: the builder's bits; others untouched
    built = decoder(c)
    if paged:
        binding.build_block_meta_paged(built.shape, p["K"], p["table"], p["K"].shape[0], 0, c.cap // bs, *built.meta)
    else:
        built.build_meta(p["K"], 0, c.cap // bs)
    for got, ref in zip(dec.meta, built.meta):
        want = torch.full_like(got, -7.0)
        for b, (n, length) in enumerate(rows):
            n = n if packed else min(1, length)
            for j in range((length - n) // bs, length // bs):
                want[b, ..., j] = ref[b, ..., j]
        assert torch.equal(bits(got), bits(want))


def test_far_positions_keep_their_angles():
    # position 2^20 - 1: an fp32 angle would be off by 0.03 rad
    c = Case(Hq=2, Hkv=1, d=64, bs=32, cap=1 << 20, rows=((1, 1 << 20), (1, (1 << 20) - 1)))
    g = torch.Generator().manual_seed(1)
    K = torch.zeros((2, 1, c.cap, 64), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    k, v = (torch.randn((2, 1, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    dec = decoder(c)
    lens = torch.tensor([n for _, n in c.rows], dtype=torch.int32, device="cuda")
    dec.append(k, v, K, V, c.cap, rope=binding.Rope(inv), seq_lens=lens)
    for b in range(2):
        pos = lens[b: b + 1].long() - 1
        want = rounded_once(rotate(wide(k[b: b + 1]), pos, inv, False), "bf16")
        assert torch.equal(bits(K[b, :, int(pos)]), bits(want[0]))
    assert dec.device_status() == 0


def test_sub_block_metadata_follows_the_envelope():
    c = Case(rows=((70, 70), (33, 129)), packed=True, bs=64, cap=256)
    p = make(c)
    _, k, v = inputs(c, False)
    dec, ref = decoder(c, sub_blocks=4), decoder(c, sub_blocks=4)
    dec.append(k, v, p["K"], p["V"], c.cap, seq_lens=p["lens"], cu_new=p["cu"])
    ref.build_meta(p["K"], 0, 4)
    for got, want in zip(dec.meta, ref.meta):     # 16-token sub-blocks: 70 and 129 tokens fill 4 and 96..128
        assert torch.equal(bits(got[0, ..., :4]), bits(want[0, ..., :4])) and (got[0, ..., 4:] == 0).all()
        assert torch.equal(bits(got[1, ..., 6:8]), bits(want[1, ..., 6:8])) and (got[1, ..., 8:] == 0).all()


@pytest.mark.parametrize("what", ["length", "offsets", "page", "short"])
def test_bad_device_values_are_reported_and_their_rows_skipped(what):
    c = Case(rows=((5, 100), (7, 200), (3, 64)), packed=True, paged=True, seed=9)
    good, bad = make(c), make(c)
    q, k, v = inputs(c, True)
    if what == "length":
        bad["lens"][1] = c.cap + 1
    elif what == "short":
        bad["lens"][1] = 6                        # fewer tokens than the row's new ones
    elif what == "offsets":
        bad["cu"][2] = c.T + 1                    # row 1 ends past the tokens, row 2 runs backwards
    else:
        bad["table"][1, 6] = bad["K"].shape[0]    # tokens 193 .. 199 of row 1 lie there
    dec = decoder(c)
    for p in (good, bad):
        dec.append(k, v, p["K"], p["V"], c.cap, q=q, seq_lens=p["lens"], cu_new=p["cu"], **p["page_args"])
        torch.cuda.synchronize()
        want = binding.ETA_OK if p is good else binding.ETA_ERR_INVALID_ARG
        assert dec.device_status() == want
    if what == "page":
        bad["table"][1, 6] = good["table"][1, 6]
        untouched = rows_of(bad, "K")[1, :, 192:224]
        assert torch.equal(bits(untouched), bits(bad["K_rows"][1, :, 192:224]))
    else:
        assert torch.equal(bits(rows_of(bad, "K")[1]), bits(bad["K_rows"][1]))
    assert torch.equal(bits(rows_of(bad, "K")[0]), bits(rows_of(good, "K")[0]))
    other = bad["K_rows"] if what == "offsets" else rows_of(good, "K")
    assert torch.equal(bits(rows_of(bad, "K")[2]), bits(other[2]))


def test_values_past_the_fp8_range_saturate_and_nan_stays_nan():
    c = Case(kv="fp8", rows=((1, 10),))
    p = make(c)
    k = torch.full((1, 2, 128), 1000.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full((1, 2, 128), -1e30, dtype=torch.bfloat16, device="cuda")
    v[0, 1] = float("nan")
    dec = decoder(c)
    dec.append(k, v, p["K"], p["V"], c.cap, seq_lens=p["lens"])
    assert (p["K"][0, :, 9].float() == 448.0).all() and (p["V"][0, 0, 9].float() == -448.0).all()
    assert torch.isnan(p["V"][0, 1, 9].float()).all()


def test_captured_append_follows_the_lengths():
    """One captured step, replayed while the lengths and inputs change, equals eager steps."""
    c = Case(rows=((1, 30), (1, 61)), cap=128)
    runs = []
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    steps = [inputs(dataclasses.replace(c), True, seed=20 + i) for i in range(6)]
    for captured in (False, True):
        p = make(c)
        dec = decoder(c)
        q, k, v = (x.clone() for x in steps[0])
        q_out = torch.empty_like(q)
        lens = p["lens"].clone()

        def call():
            return dec.append(k, v, p["K"], p["V"], c.cap, q=q, rope=binding.Rope(inv), seq_lens=lens, q_out=q_out)
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call()
        outs = []
        for i, (a, b, d_) in enumerate(steps):
            q.copy_(a), k.copy_(b), v.copy_(d_)
            lens.copy_(p["lens"] + i)
            g.replay() if captured else call()
            outs.append(q_out.clone())
        torch.cuda.synchronize()
        assert dec.device_status() == 0
        runs.append((outs, p["K"], p["V"], dec.mu, dec.var, dec.maxnorm))
    for a, b in zip(runs[0][0], runs[1][0]):
        assert torch.equal(bits(a), bits(b))
    for a, b in zip(runs[0][1:], runs[1][1:]):
        assert torch.equal(bits(a), bits(b))
