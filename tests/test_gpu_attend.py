"""eta_attend_window and eta_attend_shared against softmax attention in 64 bits, over
types, head layouts, lengths from one token on, windows, sinks, gates, pages, padded
and idle rows. Every cache row that no query sees holds NaN (or its page is gone)."""
import pytest
import torch

from learned_block_sparse_b200 import binding
from tests.newtokens import KV, Case, check, decoder, make, reference

pytestmark = pytest.mark.gpu

FILL = -3.0


def hide_unseen(p, window, sinks):
    """NaN in every row token that no query of its row sees; whole unseen pages leave the table."""
    c = p["case"]
    for b, (n, length) in enumerate(c.rows):
        n = n if c.packed else min(1, length)
        lo = max(0, length - n - window + 1)
        a1 = min(sinks, lo)
        for j in range(c.cap // c.bs):
            s0, s1 = j * c.bs, (j + 1) * c.bs
            for s in range(max(s0, a1), min(s1, lo)):
                for name in ("K", "V"):
                    if c.paged:
                        p[name][int(p["table"][b, j]), :, s % c.bs] = float("nan")
                    else:
                        p[name][b, :, s] = float("nan")
            if c.paged and s0 >= a1 and s1 <= lo:
                p["table"][b, j] = -1


def run_window(p, window, sinks=0, gated=False, hard=False, out="bf16", dec=None, hide=True):
    c = p["case"]
    if hide:
        hide_unseen(p, window, sinks)
    dec = dec or decoder(c, gate=binding.GATE_HARD if hard else binding.GATE_SIGMOID)
    o = torch.full((c.T, c.Hq, c.d), FILL, dtype=KV[out], device="cuda")
    dec.window(p["q"], p["K"], p["V"], c.cap, window, sinks=sinks, seq_lens=p["lens"], cu_q=p["cu"],
               tau=p["tau"] if gated else None, out=o, **p["page_args"])
    torch.cuda.synchronize()
    assert dec.device_status() == 0
    return o


def run_shared(p, gated=False, hard=False, out="bf16", dec=None):
    c = p["case"]
    dec = dec or decoder(c, gate=binding.GATE_HARD if hard else binding.GATE_SIGMOID)
    o = torch.full((c.T, c.Hq, c.d), FILL, dtype=KV[out], device="cuda")
    dec.shared(p["q"], p["K"], p["V"], c.cap, p["prefix"], seq_lens=p["lens"], cu_q=p["cu"],
               tau=p["tau"] if gated else None, out=o, **p["page_args"])
    torch.cuda.synchronize()
    assert dec.device_status() == 0
    return o


TYPES = [("bf16", "bf16"), ("fp8", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")]


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("window,sinks,bs,paged,gated", [
    (64, 4, 32, False, False), (100, 0, 16, True, True), (33, 40, 64, True, False), (1, 1, 32, False, True),
    (4096, 0, 128, True, False),
])
def test_window_one_token_per_row(kv, q, window, sinks, bs, paged, gated):
    rows = ((1, 1), (1, 2), (1, 0), (1, 63), (1, 64), (1, 65), (1, 500), (1, 1024), (1, 1000))
    c = Case(kv=kv, q=q, Hq=8, Hkv=2, bs=bs, cap=1024, paged=paged, rows=rows, seed=window)
    for out in ("f32", "bf16"):
        p = make(c)
        check(p, run_window(p, window, sinks, gated, out=out), reference(p, window, sinks, gated), FILL)


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("window,sinks,bs,paged,gated", [
    (64, 4, 32, True, False), (200, 0, 16, False, True), (33, 300, 64, True, False), (1, 0, 32, False, False),
    (4096, 0, 32, True, True),
])
def test_window_chunks(kv, q, window, sinks, bs, paged, gated):
    rows = ((40, 40), (1, 700), (0, 17), (130, 333), (257, 1024), (2, 2), (64, 128))
    c = Case(kv=kv, q=q, Hq=8, Hkv=2, bs=bs, cap=1024, paged=paged, rows=rows, packed=True, pad=5, seed=window)
    for out in ("f32", "bf16"):
        p = make(c)
        check(p, run_window(p, window, sinks, gated, out=out), reference(p, window, sinks, gated), FILL)


@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (3, 3, 128), (8, 1, 64), (8, 1, 128), (16, 8, 64), (12, 3, 128)])
@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_head_layouts(Hq, Hkv, d, kv):
    for packed, rows in ((False, ((1, 5), (1, 300), (1, 77))), (True, ((70, 300), (300, 301), (5, 6)))):
        c = Case(kv=kv, q=kv, Hq=Hq, Hkv=Hkv, d=d, bs=32, cap=320, paged=packed, rows=rows, packed=packed, seed=Hq)
        p = make(c, prefix=150)
        check(p, run_shared(p), reference(p, prefix=True), FILL)
        check(p, run_window(p, 50, 3), reference(p, 50, 3), FILL)   # (hides what it does not see)


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("prefix,bs,paged,gated", [(1, 32, False, False), (127, 16, True, False), (640, 64, True, True),
                                                   (2003, 32, False, True), (0, 32, True, False)])
def test_shared_one_token_per_row(kv, q, prefix, bs, paged, gated):
    rows = ((1, 1), (1, 33), (1, 0), (1, 256), (1, 100))
    c = Case(kv=kv, q=q, Hq=8, Hkv=2, bs=bs, cap=256, paged=paged, rows=rows, seed=prefix)
    for out in ("f32", "bf16"):
        p = make(c, prefix=prefix)
        check(p, run_shared(p, gated, out=out), reference(p, gated=gated, prefix=True), FILL)


@pytest.mark.parametrize("kv,q", TYPES)
@pytest.mark.parametrize("prefix,paged,gated", [(1000, True, False), (129, False, True)])
def test_shared_several_tokens_per_row(kv, q, prefix, paged, gated):
    rows = ((4, 4), (3, 200), (0, 9), (1, 1), (50, 256), (4, 131))
    c = Case(kv=kv, q=q, Hq=8, Hkv=2, bs=32, cap=256, paged=paged, rows=rows, packed=True, pad=2, seed=prefix)
    for out in ("f32", "bf16"):
        p = make(c, prefix=prefix)
        check(p, run_shared(p, gated, out=out), reference(p, gated=gated, prefix=True), FILL)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_hard_gate_leaves_only_the_own_token(kv):
    """A threshold above every logit removes every key but the query's own: its value is the output."""
    rows = ((3, 90), (1, 1), (20, 50))
    c = Case(kv=kv, q="f32" if kv == "f32" else "bf16", rows=rows, packed=True, seed=3)
    p, whole = make(c, prefix=70), make(c, prefix=70)   # the window hides what it does not see
    p["tau"].fill_(1e30), whole["tau"].fill_(1e30)
    for got in (run_window(p, 40, 2, True, True, out="f32"), run_shared(whole, True, True, out="f32")):
        t = 0
        for b, (n, length) in enumerate(rows):
            v = p["V_rows"][b, :, length - n: length].float().transpose(0, 1).repeat_interleave(4, 1)
            assert torch.allclose(got[t: t + n], v, rtol=2.0 ** -15, atol=0.0)
            t += n
    p["tau"].fill_(0.3), whole["tau"].fill_(0.3)
    check(p, run_window(p, 40, 2, True, True, out="f32"), reference(p, 40, 2, True, True), FILL)
    check(whole, run_shared(whole, True, True), reference(whole, gated=True, hard=True, prefix=True), FILL)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_peaked_and_flat_logits(kv):
    """Logits of hundreds (one key holds the mass) and of zero (every key the same)."""
    c = Case(kv=kv, q="f32" if kv == "f32" else "bf16", rows=((1, 400), (60, 256)), packed=True, seed=8)
    for scale in (40.0, 0.0):
        p, whole = make(c, prefix=300), make(c, prefix=300)
        p["q"].mul_(scale), whole["q"].mul_(scale)
        check(p, run_window(p, 128, 4, out="f32"), reference(p, 128, 4), FILL)
        check(whole, run_shared(whole, out="f32"), reference(whole, prefix=True), FILL)


def test_shared_equals_one_long_cache():
    """The prefix form and causal attention over prefix + own tokens in one cache agree."""
    c = Case(rows=((5, 37), (1, 100), (12, 12)), packed=True, seed=4)
    p = make(c, prefix=192)
    got = run_shared(p, out="f32")
    long = Case(rows=tuple((n, 192 + m) for n, m in c.rows), packed=True, seed=4)
    r = make(long)
    for name, pre in (("K", "PK"), ("V", "PV")):
        r[name][:, :, :192] = p[pre]
        for b, (n, m) in enumerate(c.rows):
            r[name][b, :, 192: 192 + m] = p[name][b, :, :m]
    r["q"].copy_(p["q"])
    whole = run_window(r, 512, 0, out="f32", hide=False)
    ref = reference(p, prefix=True)
    check(p, whole, ref, FILL)
    check(p, got, ref, FILL)


def test_uniform_lengths_and_constant_thresholds():
    c = Case(rows=((1, 300),) * 3, seed=6)
    p = make(c)
    dec = decoder(c)
    a = dec.window(p["q"], p["K"], p["V"], 300, 64, sinks=2).clone()
    b = run_window(p, 64, 2, out="f32", dec=dec)
    assert torch.equal(a, b)
    p["tau"][:] = p["tau"][0]
    x = torch.empty_like(a)
    dec.window(p["q"], p["K"], p["V"], 300, 64, tau=p["tau"][0].contiguous(), out=x)
    assert torch.equal(x, run_window(p, 64, 0, True, out="f32", dec=dec))


@pytest.mark.parametrize("what", ["length", "page", "offsets"])
def test_bad_device_values_are_reported(what):
    c = Case(rows=((5, 100), (7, 200), (3, 64)), packed=True, paged=True, seed=9)
    p = make(c, prefix=40)
    dec = decoder(c)
    good = dec.window(p["q"], p["K"], p["V"], c.cap, 50, seq_lens=p["lens"], cu_q=p["cu"],
                      out=torch.full((c.T, c.Hq, c.d), FILL, device="cuda"), **p["page_args"]).clone()
    assert dec.device_status() == 0
    if what == "length":
        p["lens"][1] = 6
    elif what == "offsets":
        p["cu"][2] = c.T + 1                       # row 1 ends past the tokens, row 2 runs backwards
    else:
        p["table"][1, 5] = -1                      # tokens 160 .. 191: row 1 sees 144 .. 199
    for call in ("window", "shared"):
        out = torch.full((c.T, c.Hq, c.d), FILL, device="cuda")
        if call == "window":
            dec.window(p["q"], p["K"], p["V"], c.cap, 50, seq_lens=p["lens"], cu_q=p["cu"], out=out, **p["page_args"])
            assert torch.equal(out[:5], good[:5])
            if what != "offsets":
                assert torch.equal(out[12:], good[12:])
        else:
            dec.shared(p["q"], p["K"], p["V"], c.cap, p["prefix"], seq_lens=p["lens"], cu_q=p["cu"], out=out,
                       **p["page_args"])
        torch.cuda.synchronize()
        assert dec.device_status() == binding.ETA_ERR_INVALID_ARG
        if what == "page":
            assert torch.isfinite(out).all()       # the page's tokens take no part
        else:
            assert (out[5:12] == FILL).all()
            assert (out[12:] == FILL).all() == (what == "offsets")
    if what == "page":
        p["table"][1, 5] = 0                       # and a prefix page outside the pool
        p["blocks"][0] = p["K"].shape[0] + 3
        dec.shared(p["q"], p["K"], p["V"], c.cap, p["prefix"], seq_lens=p["lens"], cu_q=p["cu"],
                   out=torch.empty((c.T, c.Hq, c.d), device="cuda"), **p["page_args"])
        torch.cuda.synchronize()
        assert dec.device_status() == binding.ETA_ERR_INVALID_ARG


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_a_prompt_and_its_decode_steps_together(kv):
    """Append a prompt in chunks, then decode: append -> window / shared / dense, eagerly
    and captured, on another stream, against 64 bits on the cache that append left."""
    c = Case(kv=kv, q="f32" if kv == "f32" else "bf16", Hq=8, Hkv=2, bs=32, cap=256, paged=True,
             rows=((50, 50), (33, 33)), packed=True, seed=12)
    p = make(c, prefix=100)
    dec = decoder(c)
    dec.reserve_queries(c.T)
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    rope = binding.Rope(inv)
    g = torch.Generator().manual_seed(3)

    def fresh(n):
        x = torch.randn((n, (c.Hq + 2 * c.Hkv) * c.d), generator=g).to(KV[c.q]).cuda()
        h = c.Hq * c.d
        return (x[:, :h].view(n, c.Hq, c.d), x[:, h: h + c.Hkv * c.d].view(n, c.Hkv, c.d),
                x[:, h + c.Hkv * c.d:].view(n, c.Hkv, c.d))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        q, k, v = fresh(c.T)
        q_rot = dec.append(k, v, p["K"], p["V"], c.cap, q=q, rope=rope, seq_lens=p["lens"], cu_new=p["cu"],
                           **p["page_args"])
        out = torch.empty((c.T, c.Hq, c.d), device="cuda")
        dec.window(q_rot, p["K"], p["V"], c.cap, 40, sinks=4, seq_lens=p["lens"], cu_q=p["cu"], out=out,
                   **p["page_args"])
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()

    def snapshot(rows, packed, q):
        r = dict(p)
        r["case"] = Case(**{**c.__dict__, "rows": rows, "packed": packed})
        r["q"] = q
        r["cu_list"] = p["cu_list"] if packed else list(range(len(rows) + 1))
        for name in ("K", "V"):
            pool = p[name].view(torch.uint8) if kv == "fp8" else p[name]
            x = pool[p["table"].long().view(-1)].view(c.B, -1, c.Hkv, c.bs, c.d).transpose(1, 2)
            r[name + "_rows"] = x.reshape(c.B, c.Hkv, c.cap, c.d).view(p[name].dtype)
        return r

    r = snapshot(c.rows, True, q_rot)
    check(r, out, reference(r, 40, 4), FILL)

    # decode steps, captured once: append, then both attentions and the dense decode of the framework
    lens = p["lens"].clone()
    q, k, v = (x.clone() for x in fresh(c.B))
    q_out = torch.empty((c.B, c.Hq, c.d), dtype=KV[c.q], device="cuda")
    outs = [torch.empty((c.B, c.Hq, c.d), device="cuda") for _ in range(3)]

    def step():
        dec.append(k, v, p["K"], p["V"], c.cap, q=q, rope=rope, seq_lens=lens, q_out=q_out, **p["page_args"])
        dec.window(q_out, p["K"], p["V"], c.cap, 40, sinks=4, seq_lens=lens, out=outs[0], **p["page_args"])
        dec.shared(q_out, p["K"], p["V"], c.cap, p["prefix"], seq_lens=lens, out=outs[1], **p["page_args"])
        binding.decode_dense_paged(dec.shape, dec.params, q_out, p["K"], p["V"], p["table"],
                                   p["page_args"]["num_pages"], lens, c.cap, None, 0, outs[2], dec.ws)

    lens.add_(1)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for dst, src in zip((q, k, v), fresh(c.B)):
            dst.copy_(src)
        lens.copy_(p["lens"] + 2 + i)
        graph.replay()
        torch.cuda.synchronize()
        assert dec.device_status() == 0
        rows = tuple((1, n + 2 + i) for _, n in c.rows)
        r = snapshot(rows, False, q_out)
        check(r, outs[0], reference(r, 40, 4), FILL)
        check(r, outs[1], reference(r, prefix=True), FILL)
        ref = reference(r)
        check(r, outs[2], ref, FILL)
    # the metadata the steps left is the builder's
    full = [int(n) // c.bs for n in lens.cpu()]
    built = decoder(c)
    binding.build_block_meta_paged(built.shape, p["K"], p["table"], p["page_args"]["num_pages"], 0, c.cap // c.bs,
                                   *built.meta)
    for a, b in zip(dec.meta, built.meta):
        for row, nfull in enumerate(full):
            assert torch.equal(a[row, ..., :nfull], b[row, ..., :nfull])


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_peaked_and_flat_logits_of_single_tokens(kv):
    """As above for one token per row. With fp8 values a weight is two f16 numbers, which
    end at 2^-24 of the largest weight: it may lose half of that."""
    c = Case(kv=kv, q="f32" if kv == "f32" else "bf16", rows=((1, 400), (1, 256), (1, 33)), seed=8)
    for scale in (40.0, 0.0):
        p, whole = make(c, prefix=300), make(c, prefix=300)
        p["q"].mul_(scale), whole["q"].mul_(scale)
        floor = 2.0 ** -25 if kv == "fp8" else 0.0
        check(p, run_window(p, 128, 4, out="f32"), reference(p, 128, 4), FILL, floor)
        check(whole, run_shared(whole, out="f32"), reference(whole, prefix=True), FILL, floor)


@pytest.mark.parametrize("packed", [False, True])
def test_pages_past_32_bit_offsets(packed):
    """A pool of 2.3e9 elements: rows in its last pages give the bits they give in a small one."""
    rows = ((40, 300), (3, 65), (100, 128)) if packed else ((1, 300), (1, 65), (1, 128))
    c = Case(Hq=8, Hkv=8, bs=32, cap=320, paged=True, rows=rows, packed=packed, seed=2)
    p = make(c, prefix=90)
    pages, small = 70000, p["K"].shape[0]
    far = dict(p)
    for name in ("K", "V"):
        far[name] = torch.empty((pages, c.Hkv, c.bs, c.d), dtype=torch.bfloat16, device="cuda")
        far[name][pages - small:] = p[name]
    far["table"] = p["table"] + (pages - small)
    far["blocks"] = p["blocks"] + (pages - small)
    far["page_args"] = dict(block_table=far["table"], num_pages=pages)
    far["prefix"] = binding.Prefix(90, blocks=far["blocks"])
    g = torch.Generator().manual_seed(4)
    new = [torch.randn((c.T, h, c.d), generator=g).to(torch.bfloat16).cuda() for h in (c.Hkv, c.Hkv)]
    got = []
    for r in (p, far):
        dec = decoder(c)
        dec.append(*new, r["K"], r["V"], c.cap, seq_lens=r["lens"], cu_new=r["cu"], **r["page_args"])
        got.append((run_window(r, 50, 4, dec=dec, hide=False), run_shared(r, dec=dec), dec.mu, dec.var, dec.maxnorm,
                    r["K"][pages - small:] if r is far else r["K"], r["V"][pages - small:] if r is far else r["V"]))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                           b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


def test_two_calls_at_once_on_two_streams():
    """Two decoders (workspaces) on two streams give what each gives alone, again and again."""
    cases = [Case(rows=((1, 500), (1, 90), (1, 512)), seed=1), Case(rows=((70, 300), (5, 512)), packed=True, seed=2)]
    ps = [make(c, prefix=200) for c in cases]
    decs = [decoder(c) for c in cases]
    alone = [(run_window(p, 100, 4, dec=d, hide=False), run_shared(p, dec=d)) for p, d in zip(ps, decs)]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.empty_like(alone[i][0]) for _ in range(16)] for i in range(2)]
    torch.cuda.synchronize()
    for k in range(8):
        for i, (p, d, s) in enumerate(zip(ps, decs, streams)):
            c = p["case"]
            with torch.cuda.stream(s):
                d.window(p["q"], p["K"], p["V"], c.cap, 100, sinks=4, seq_lens=p["lens"], cu_q=p["cu"],
                         out=outs[i][2 * k])
                d.shared(p["q"], p["K"], p["V"], c.cap, p["prefix"], seq_lens=p["lens"], cu_q=p["cu"],
                         out=outs[i][2 * k + 1])
    torch.cuda.synchronize()
    for i in range(2):
        assert decs[i].device_status() == 0
        for k in range(8):
            assert torch.equal(outs[i][2 * k], alone[i][0]) and torch.equal(outs[i][2 * k + 1], alone[i][1])


def test_a_captured_chunk_follows_offsets_and_lengths():
    """A captured packed call replayed while the rows' shares of the tokens change, to none and back."""
    c = Case(rows=((30, 200), (34, 90), (0, 10)), packed=True, seed=5)
    p = make(c, prefix=64)
    dec = decoder(c)
    o = [torch.full((c.T, c.Hq, c.d), FILL, device="cuda", dtype=torch.bfloat16) for _ in range(2)]

    def call():
        dec.window(p["q"], p["K"], p["V"], c.cap, 77, sinks=2, seq_lens=p["lens"], cu_q=p["cu"], out=o[0])
        dec.shared(p["q"], p["K"], p["V"], c.cap, p["prefix"], seq_lens=p["lens"], cu_q=p["cu"], out=o[1])

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rows in (((64, 200), (0, 90), (0, 10)), ((0, 200), (1, 90), (10, 10)), ((0, 200), (0, 90), (0, 10)), c.rows):
        r = dict(p)
        r["case"] = Case(**{**c.__dict__, "rows": rows, "pad": c.T - sum(n for n, _ in rows)})
        cu = [0]
        for n, _ in rows:
            cu.append(cu[-1] + n)
        r["cu_list"] = cu
        p["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        for x in o:
            x.fill_(FILL)
        graph.replay()
        torch.cuda.synchronize()
        assert dec.device_status() == 0
        check(r, o[0], reference(r, 77, 2), FILL)
        check(r, o[1], reference(r, prefix=True), FILL)


def test_calls_that_cannot_be_right_are_refused():
    c = Case(rows=((1, 100), (1, 50)), seed=1)
    p = make(c, prefix=40)
    dec = decoder(c)
    K, V, q, lens = p["K"], p["V"], p["q"], p["lens"]
    good = dict(seq_lens=lens)
    dec.window(q, K, V, c.cap, 10, **good)
    one = torch.zeros((2, c.Hkv, c.d), dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: dec.window(q.cpu(), K, V, c.cap, 10), lambda: dec.window(q.float(), K, V, c.cap, 10),
        lambda: dec.window(q, K.cpu(), V.cpu(), c.cap, 10), lambda: dec.window(q, K[:, :, :64], V[:, :, :64], c.cap, 10),
        lambda: dec.window(q, K.transpose(1, 2), V.transpose(1, 2), c.cap, 10),
        lambda: dec.window(q, K, V, c.cap, 10, seq_lens=lens.long()), lambda: dec.window(q, K, V, c.cap, 10, seq_lens=lens[:1]),
        lambda: dec.window(q, K, V, c.cap, 10, cu_q=p["lens"]), lambda: dec.window(q, K, V, c.cap, 0),
        lambda: dec.window(q, K, V, c.cap + 1, 10), lambda: dec.window(q, K, V, c.cap, 10, sinks=-1),
        lambda: dec.window(q, K, V, c.cap, 10, out=torch.empty((2, c.Hq, c.d), dtype=torch.float16, device="cuda")),
        lambda: dec.window(q, K, V, c.cap, 10, out=torch.empty((1, c.Hq, c.d), device="cuda")),
        lambda: dec.window(q, K, V, c.cap, 10, tau=p["tau"].double()), lambda: dec.window(q, K, V, c.cap, 10, tau=p["tau"][0], tau_batch_stride=c.Hq),
        lambda: dec.window(q, K, V, c.cap, 10, block_table=torch.zeros(3, dtype=torch.int32, device="cuda")),
        lambda: dec.shared(q, K, V, c.cap, binding.Prefix(8, blocks=torch.zeros(1, dtype=torch.int32, device="cuda"))),
        lambda: dec.shared(q, K, V, c.cap, binding.Prefix(8, k=p["PK"].cpu(), v=p["PV"].cpu())),
        lambda: dec.shared(q, K, V, c.cap, binding.Prefix(8, k=p["PK"][:1], v=p["PV"][:1])),
        lambda: dec.append(one, one.float(), K, V, c.cap), lambda: dec.append(one[:1], one[:1], K, V, c.cap),
        lambda: dec.append(one.transpose(0, 1), one.transpose(0, 1), K, V, c.cap),
        lambda: dec.append(one, one, K, V, c.cap, q=q[:, :4]), lambda: dec.append(one, one, K, V, c.cap, q_out=q),
        lambda: dec.append(one, one, K, V, c.cap, rope=binding.Rope(torch.zeros(64))),
        lambda: dec.append(one, one, K, V, c.cap, rope=binding.Rope(torch.zeros(65, device="cuda"))),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, binding.EtaError)):
            f()
            print("accepted", i)
    torch.cuda.synchronize()
    assert dec.device_status() == 0


@pytest.mark.parametrize("kv,Hkv,d", [("bf16", 4, 64), ("bf16", 2, 128), ("fp8", 2, 128)])
def test_long_sums_keep_fp32(kv, Hkv, d):
    """Values of one sign behind a long prefix that is not split: an accumulator that
    cuts off each addition would drift with their number (4,096 additions of half a step
    of 2^-23 and more are 2e-4). Counted here: 96 additions of at most 2^-23 between two
    rounded sums (64 of 2^-24), and 2^-22 of each weight for its exponent: 1.6e-5."""
    P, T, Hq = 32768, 12800 // Hkv, 2 * Hkv
    g = torch.Generator(device="cuda").manual_seed(9)

    def normal(*shape):
        return torch.empty(shape, device="cuda").normal_(0, 1, generator=g)

    pk, pv = (0.3 * normal(Hkv, P, d)).to(KV[kv]), (1 + normal(Hkv, P, d).abs()).to(KV[kv])
    k, v = (0.3 * normal(1, Hkv, T, d)).to(KV[kv]), (1 + normal(1, Hkv, T, d).abs()).to(KV[kv])
    q = normal(T, Hq, d).to(torch.bfloat16)
    dec = binding.EtaDecoder(1, Hq, Hkv, d, 32, T, kv_dtype=KV[kv], q_dtype=torch.bfloat16)
    out = torch.empty((T, Hq, d), device="cuda")
    dec.shared(q, k, v, T, binding.Prefix(P, k=pk, v=pv), out=out,
               cu_q=torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert dec.device_status() == 0
    for t in (0, 1, 129, T // 2, T - 1):
        for h in range(Hq):
            keys = torch.cat([pk[h // 2].float(), k[0, h // 2, :t + 1].float()]).double()
            vals = torch.cat([pv[h // 2].float(), v[0, h // 2, :t + 1].float()]).double()
            w = torch.softmax(keys @ q[t, h].double() / d ** 0.5, 0)
            exact = w @ vals
            assert ((out[t, h].double() - exact).abs() / exact).max() < 1.6e-5, (t, h)


def test_a_larger_call_leaves_captured_graphs_valid():
    """A captured call, then a larger one that takes a larger workspace: the graph's own stays."""
    c = Case(rows=((1, 500), (1, 90)), seed=6)
    p = make(c, prefix=300)
    dec = decoder(c)
    out = torch.full((c.T, c.Hq, c.d), FILL, device="cuda")
    dec.shared(p["q"], p["K"], p["V"], c.cap, p["prefix"], seq_lens=p["lens"], out=out)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.shared(p["q"], p["K"], p["V"], c.cap, p["prefix"], seq_lens=p["lens"], out=out)
    ws = dec.attend_ws
    address, size = ws.data_ptr(), ws.numel()
    del ws
    dec.reserve_queries(5000)
    assert dec.attend_ws.data_ptr() != address
    other = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert all(x.data_ptr() + size <= address or x.data_ptr() >= address + size for x in other)
    out.fill_(FILL)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and all(bool((x == 255).all()) for x in other)
    assert dec.device_status() == 0
    check(p, out, reference(p, prefix=True), FILL)
