"""The calls that take new tokens refuse bad arguments on the host, before anything is
launched (no GPU needed), and their ctypes structs match the header."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20        # an aligned address; no call here gets as far as using it
OUT = A + (1 << 24)


def _b():
    from learned_block_sparse_b200 import binding
    return binding


def _shape(**kw):
    d = dict(batch=2, n_q_heads=4, n_kv_heads=2, head_dim=128, block_size=32, capacity=1024, kv_dtype=1, q_dtype=1)
    d.update(kw)
    return _b().Shape(**d)


def _append(shape=None, tokens=None, rope=None, k=A, v=A, pages=None, lens=A, n=1024, meta=None, ws=A, ws_bytes=1 << 20):
    b = _b()
    t = dict(q=A, k=A, v=A, q_out=OUT, q_stride=512, k_stride=256, v_stride=256, cu_new=A, n_new=7)
    t.update(tokens or {})
    r = dict(inv_freq=A, rot_dim=128, interleaved=0)
    r.update(rope or {})
    s, tk, rp = shape or _shape(), b.Tokens(**t), b.RopeArgs(**r)
    pg = ctypes.byref(pages) if pages is not None else None
    return b.lib.eta_append_kv(ctypes.byref(s), ctypes.byref(tk), ctypes.byref(rp), k, v, pg, lens, n,
                               meta or b.Meta(A, A, A), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(tokens=dict(n_new=0)), 0),                                  # nothing to do
    (dict(tokens=dict(n_new=-1)), 1), (dict(tokens=dict(n_new=1 << 31)), 1),
    (dict(tokens=dict(cu_new=None, n_new=3)), 1),                     # one token per row: n_new is the batch
    (dict(tokens=dict(cu_new=A + 2)), 1),
    (dict(tokens=dict(k=None)), 1), (dict(tokens=dict(v=A + 8)), 1), (dict(tokens=dict(q=A + 4)), 1),
    (dict(tokens=dict(q=None)), 1), (dict(tokens=dict(q_out=None)), 1), (dict(tokens=dict(q_out=A + 4)), 1),
    (dict(tokens=dict(k_stride=255)), 1), (dict(tokens=dict(k_stride=260)), 1), (dict(tokens=dict(q_stride=256)), 1),
    (dict(tokens=dict(q_out=A)), 1), (dict(tokens=dict(q_out=A + 7 * 1024 - 16)), 1),  # q_out reaches into q
    (dict(tokens=dict(q_out=A, q=OUT)), 1), (dict(tokens=dict(q_out=A - 16)), 1),      # into k and v; into q from before
    (dict(rope=dict(rot_dim=-16)), 1), (dict(rope=dict(rot_dim=144)), 1), (dict(rope=dict(rot_dim=40)), 1),
    (dict(rope=dict(inv_freq=None)), 1), (dict(rope=dict(inv_freq=A + 2)), 1), (dict(rope=dict(interleaved=2)), 1),
    (dict(k=None), 1), (dict(v=A + 8), 1), (dict(lens=A + 1), 1), (dict(n=0), 1), (dict(n=1025), 1),
    (dict(ws=None), 3), (dict(ws=A + 16), 3), (dict(ws_bytes=100), 3),
])
def test_append_refusals(kw, expect):
    assert _append(**kw) == expect


def test_append_refuses_shapes_and_pages():
    b = _b()
    assert _append(shape=_shape(head_dim=96)) == 2
    assert _append(shape=_shape(kv_dtype=2, q_dtype=0)) == 2
    assert _append(pages=b.Pages(None, 5)) == 1 and _append(pages=b.Pages(A, 0)) == 1
    assert _append(pages=b.Pages(A, 1 << 26)) == 2                    # more pool rows than 32 bits address
    assert _append(meta=b.Meta(A, None, A)) == 1
    assert b.lib.eta_append_kv(None, None, None, A, A, None, None, 1, b.Meta(), A, 1 << 20, None) == 1


def _attend(call="window", shape=None, params=None, queries=None, prefix=None, k=A, v=A, pages=None, lens=A, n=1024,
            window=64, sinks=4, ws=A, ws_bytes=1 << 40):
    b = _b()
    q = dict(q=A, cu_q=A, n_new=7, tau=None, tau_stride=0, out=OUT, out_dtype=1)
    q.update(queries or {})
    s, p, qs = shape or _shape(), params or b.make_params(), b.Queries(**q)
    pg = ctypes.byref(pages) if pages is not None else None
    if call == "window":
        return b.lib.eta_attend_window(ctypes.byref(s), ctypes.byref(p), ctypes.byref(qs), k, v, pg, lens, n, window,
                                       sinks, ws, ws_bytes, None)
    pr = dict(k=A, v=A, blocks=A, capacity=256, n_tokens=200)
    pr.update(prefix or {})
    px = b.PrefixArgs(**pr)
    return b.lib.eta_attend_shared(ctypes.byref(s), ctypes.byref(p), ctypes.byref(qs), ctypes.byref(px), k, v, pg, lens,
                                   n, ws, ws_bytes, None)


COMMON = [
    (dict(queries=dict(n_new=0)), 0),
    (dict(queries=dict(n_new=-1)), 1), (dict(queries=dict(cu_q=None, n_new=3)), 1), (dict(queries=dict(cu_q=A + 1)), 1),
    (dict(queries=dict(q=None)), 1), (dict(queries=dict(q=A + 8)), 1), (dict(queries=dict(out=None)), 1),
    (dict(queries=dict(out=A + 4)), 1), (dict(queries=dict(out_dtype=2)), 1),
    (dict(queries=dict(out=A)), 1), (dict(queries=dict(out=A + 7 * 1024 - 16)), 1),    # out reaches into q
    (dict(queries=dict(out=A - 16)), 1),
    (dict(queries=dict(tau=A, tau_stride=-1)), 1), (dict(queries=dict(tau=A + 2)), 1),
    (dict(queries=dict(n_new=(1 << 31) - 1)), 2),                     # token x head rows past 32 bits
    (dict(k=None), 1), (dict(v=A + 8), 1), (dict(lens=A + 2), 1), (dict(n=0), 1), (dict(n=1025), 1),
    (dict(ws=None), 3), (dict(ws=A + 16), 3), (dict(ws_bytes=33024), 3),
]


@pytest.mark.parametrize("call", ["window", "shared"])
@pytest.mark.parametrize("kw,expect", COMMON)
def test_attend_refusals(call, kw, expect):
    assert _attend(call, **kw) == expect


def test_attend_refuses_windows_prefixes_and_params():
    b = _b()
    assert _attend(window=0) == 1 and _attend(sinks=-1) == 1 and _attend(window=-5) == 1
    for bad in (dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(k=None), dict(v=A + 8), dict(capacity=100)):
        assert _attend("shared", prefix=bad) == 1, bad
    assert _attend("shared", prefix=dict(capacity=1 << 31)) == 2
    pages = b.Pages(A, 64)
    assert _attend("shared", prefix=dict(blocks=None), pages=pages) == 1
    assert _attend("shared", prefix=dict(blocks=A + 2), pages=pages) == 1
    for call in ("window", "shared"):
        assert _attend(call, params=b.make_params(beta=-1.0)) == 1
        assert _attend(call, shape=_shape(block_size=48, capacity=960), n=960) == 2
        assert _attend(call, pages=b.Pages(A, 1 << 26)) == 2
        assert _attend(call, shape=_shape(batch=8192, capacity=64), n=64) == 2     # more (row, kv head) pairs than a call takes


def test_workspace_grows_with_the_queries():
    b = _b()
    for shape in (_shape(), _shape(n_q_heads=16, n_kv_heads=2), _shape(n_q_heads=32, n_kv_heads=32, batch=1)):
        s = ctypes.byref(shape)
        for prefix in (0, 1):
            sizes = [b.lib.eta_attend_workspace_bytes(s, n, prefix) for n in (0, 1, 2, 3, 5, 8, 9, 64, 1000, 5000)]
            assert all(x >= 33024 for x in sizes) and sizes == sorted(sizes)
        assert b.lib.eta_attend_workspace_bytes(s, -1, 0) == 0
    assert b.lib.eta_attend_workspace_bytes(ctypes.byref(_shape(head_dim=96)), 4, 0) == 0


def test_structs_match_the_header(tmp_path):
    b = _b()
    structs = {"eta_rope_t": b.RopeArgs, "eta_tokens_t": b.Tokens, "eta_queries_t": b.Queries,
               "eta_prefix_t": b.PrefixArgs}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "eta.h"', 'int main(void) {']
    for cname, py in structs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "probe.c"
    src.write_text("\n".join(lines + ['  return 0;', '}']))
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in out if x}
    for cname, py in structs.items():
        assert got[(cname, "size")] == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset


def test_python_objects_refuse_what_cannot_be_a_rope_or_a_prefix():
    import torch
    b = _b()
    with pytest.raises(TypeError):
        b.Rope(torch.zeros(4, dtype=torch.float64))
    with pytest.raises(TypeError):
        b.Rope(torch.zeros((2, 2)))
    k = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    for bad in (dict(n_tokens=-1), dict(n_tokens=4, k=k), dict(n_tokens=4), dict(n_tokens=9, k=k, v=k),
                dict(n_tokens=4, k=k, v=k, blocks=torch.zeros(1, dtype=torch.int32)),
                dict(n_tokens=4, k=k, v=k[:1]), dict(n_tokens=4, k=k.transpose(0, 1), v=k.transpose(0, 1))):
        with pytest.raises(ValueError):
            b.Prefix(**bad)
    with pytest.raises(TypeError):
        b.Prefix(4, blocks=torch.zeros(1, dtype=torch.int64))
    assert b.Prefix(0).args.n_tokens == 0
