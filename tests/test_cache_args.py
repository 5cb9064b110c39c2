"""What the rotation, the append to the 8-bit cache and its attention refuse, without a GPU: the C calls
return their errors before any CUDA call, the binding raises before the library is called."""
import ctypes as C
import math
import os
import subprocess

import pytest

from conftest import ROOT

FAKE = 1 << 20


@pytest.fixture(scope="module")
def qz():
    import __graft_entry__
    __graft_entry__.build_library()
    import precision_quantization_gb300 as qz
    qz.lib()
    return qz


def rot(qz, cos=FAKE, sin=FAKE, positions=100, pairs=32, interleaved=0):
    return qz.QzRotaryTable(cos, sin, positions, pairs, interleaved)


def cache(qz, fmt=None, block=16, page=32, kv=2, dim=64, pages=8, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE):
    return qz.QzCache(qz.QZ_INT8 if fmt is None else fmt, block, page, kv, dim, 0, pages, kc, ks, vc, vs)


def batch(qz, n=3, table=FAKE, ld=4, width=4, lengths=FAKE, starts=FAKE):
    return qz.QzBatch(n, table, ld, width, lengths, starts)


def test_layouts_match_header(qz, tmp_path):
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qz.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu %zu %zu %zu %zu\\n", sizeof(qz_rotary_table), offsetof(qz_rotary_table, pairs),'
                   ' sizeof(qz_cache), offsetof(qz_cache, pages), offsetof(qz_cache, v_scales), sizeof(qz_batch),'
                   ' offsetof(qz_batch, table_pages), offsetof(qz_batch, starts)); return 0;}\n')
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    r, c, b = qz.QzRotaryTable, qz.QzCache, qz.QzBatch
    assert got == [C.sizeof(r), r.pairs.offset, C.sizeof(c), c.pages.offset, c.v_scales.offset, C.sizeof(b),
                   b.table_pages.offset, b.starts.offset]


def test_rotary_errors(qz):
    for call in (qz.qz_rotary, qz.qz_rotary_backward):
        f = lambda t=rot(qz), dt=qz.QZ_BF16, x=FAKE, ld=128, hd=64, n=5, h=2, d=64, p=FAKE, y=FAKE, ly=128, hy=64: call(  # noqa: E731
            t, dt, x, ld, hd, n, h, d, p, y, ly, hy)
        assert f(t=None) == f(x=None) == f(y=None) == f(t=rot(qz, cos=None)) == f(t=rot(qz, sin=None)) == qz.QZ_ERR_NULL
        assert f(dt=3) == qz.QZ_ERR_ENUM
        assert f(n=-1) == f(d=62) == f(t=rot(qz, positions=0)) == f(t=rot(qz, positions=-1)) == f(t=rot(qz, pairs=-1)) == qz.QZ_ERR_SHAPE
        assert f(hd=63) == f(ld=127) == f(ly=127) == f(hy=-64) == f(ld=1 << 60) == qz.QZ_ERR_SHAPE  # vectors that overlap, offsets past 64 bits
        assert f(ld=0) == f(hd=0) == qz.QZ_ERR_SHAPE
        assert f(ly=256) == f(hy=320, ly=640) == qz.QZ_ERR_SHAPE  # in place, but elsewhere
        assert f(n=1 << 31) == f(h=1 << 31) == f(h=1 << 26) == f(t=rot(qz, positions=1 << 31)) == qz.QZ_ERR_UNSUPPORTED
        assert f(x=FAKE + 1) == f(y=FAKE + 1) == f(p=FAKE + 2) == f(t=rot(qz, cos=FAKE + 2)) == f(dt=qz.QZ_F32, x=FAKE + 2) == qz.QZ_ERR_ALIGN
        assert f(n=0) == f(h=0) == qz.QZ_OK
        assert f(n=0, x=None, y=None) == qz.QZ_OK
    g = lambda t=FAKE, n=10, p=4, c=FAKE, s=FAKE: qz.qz_rotary_fill(t, n, p, 1.0, c, s)  # noqa: E731
    assert g(t=None) == g(c=None) == g(s=None) == qz.QZ_ERR_NULL
    assert g(n=-1) == g(p=-1) == qz.QZ_ERR_SHAPE and g(n=1 << 31) == qz.QZ_ERR_UNSUPPORTED
    assert g(t=FAKE + 4) == g(c=FAKE + 2) == qz.QZ_ERR_ALIGN and g(n=0) == qz.QZ_OK


CACHES = [(dict(fmt=9), "ENUM"), (dict(fmt=4), "ENUM"), (dict(block=8), "UNSUPPORTED"), (dict(block=48, page=48), "UNSUPPORTED"),
          (dict(page=40), "SHAPE"), (dict(page=0), "SHAPE"), (dict(page=2048), "UNSUPPORTED"), (dict(kv=0), "SHAPE"), (dict(kv=1 << 16), "UNSUPPORTED"),
          (dict(dim=72), "UNSUPPORTED"), (dict(dim=272), "UNSUPPORTED"), (dict(dim=-16), "SHAPE"), (dict(pages=-1), "SHAPE"),
          (dict(pages=1 << 31), "UNSUPPORTED"), (dict(kc=None), "NULL"), (dict(vs=None), "NULL"), (dict(kc=FAKE + 8), "ALIGN"),
          (dict(vc=FAKE + 8), "ALIGN"), (dict(ks=FAKE + 2), "ALIGN")]
BATCHES = [(dict(n=-1), "SHAPE"), (dict(n=1 << 25), "UNSUPPORTED"), (dict(width=-1), "SHAPE"), (dict(ld=3), "SHAPE"), (dict(ld=1 << 62), "SHAPE"),
           (dict(width=1 << 25, ld=1 << 25), "UNSUPPORTED"), (dict(table=None), "NULL"), (dict(lengths=None), "NULL"),
           (dict(table=FAKE + 2), "ALIGN"), (dict(lengths=FAKE + 2), "ALIGN"), (dict(starts=FAKE + 2), "ALIGN"), (dict(starts=None), "SHAPE")]


def test_append_errors(qz):
    f = lambda c=cache(qz), b=batch(qz), dt=qz.QZ_BF16, k=FAKE, lk=128, hk=64, v=FAKE, lv=128, hv=64, n=5, t=rot(qz), q=FAKE, lq=256, hq=64, h=4, o=FAKE, lo=256, ho=64: (  # noqa: E731
        qz.qz_cache_append(c, b, dt, k, lk, hk, v, lv, hv, n, t, q, lq, hq, h, o, lo, ho))
    for bad, err in CACHES:
        assert f(c=cache(qz, **bad)) == getattr(qz, "QZ_ERR_" + err), bad
    for bad, err in BATCHES:
        assert f(b=batch(qz, **bad)) == getattr(qz, "QZ_ERR_" + err), bad
    assert f(c=None) == f(b=None) == f(k=None) == f(v=None) == qz.QZ_ERR_NULL
    assert f(q=None) == f(o=None) == f(t=None) == qz.QZ_ERR_NULL  # queries need both tensors and a table
    assert f(dt=0) == qz.QZ_ERR_ENUM
    assert f(hk=63) == f(lv=127) == f(hq=63) == f(lo=255) == f(n=-1) == f(h=3) == f(t=rot(qz, pairs=33)) == qz.QZ_ERR_SHAPE
    assert f(lo=512) == f(ho=128, lo=512) == qz.QZ_ERR_SHAPE  # in place, but elsewhere
    assert f(n=1 << 31) == f(n=(1 << 30) + 1) == qz.QZ_ERR_UNSUPPORTED
    assert f(k=FAKE + 1) == f(v=FAKE + 1) == f(q=FAKE + 1) == f(o=FAKE + 1) == qz.QZ_ERR_ALIGN
    assert f(n=0) == f(n=0, k=None, v=None) == f(b=batch(qz, n=0)) == qz.QZ_OK


def test_attention_errors(qz):
    need = qz.qz_cache_attention_workspace(cache(qz), 3, 5, 4, 4)
    f = lambda c=cache(qz), b=batch(qz), q=FAKE, lq=256, hq=64, n=5, h=4, s=0.1, w=0, o=FAKE, lo=256, ho=64, l=FAKE, ll=4, ws=FAKE, wb=need: (  # noqa: E731, E741
        qz.qz_cache_attention(c, b, q, lq, hq, n, h, s, w, o, lo, ho, l, ll, ws, wb))
    for bad, err in CACHES:
        assert f(c=cache(qz, **bad)) == getattr(qz, "QZ_ERR_" + err), bad
    for bad, err in BATCHES:
        assert f(b=batch(qz, **bad)) == getattr(qz, "QZ_ERR_" + err), bad
    assert f(c=None) == f(b=None) == f(q=None) == f(o=None) == qz.QZ_ERR_NULL
    assert f(h=3) == f(w=-1) == f(ll=3) == f(hq=63) == f(lo=255) == f(n=-1) == qz.QZ_ERR_SHAPE
    for s in (0.0, -1.0, math.inf, math.nan):
        assert f(s=s) == qz.QZ_ERR_SHAPE
    assert f(q=FAKE + 1) == f(o=FAKE + 1) == f(l=FAKE + 2) == qz.QZ_ERR_ALIGN
    assert f(n=(1 << 30) + 1) == f(n=1 << 30, lq=256) == qz.QZ_ERR_UNSUPPORTED
    assert need == 0 and f(ws=FAKE + 8) == qz.QZ_ERR_ALIGN  # such short sequences take none
    long = batch(qz, ld=4000, width=4000)
    need = qz.qz_cache_attention_workspace(cache(qz), 3, 5, 4, 4000)
    assert need > 0 and f(b=long, ws=None) == f(b=long, wb=need - 1) == qz.QZ_ERR_WORKSPACE
    assert f(n=0) == f(n=0, q=None, o=None, ws=None, wb=0) == f(h=0) == f(b=batch(qz, n=0)) == qz.QZ_OK
    for bad in (dict(fmt=9), dict(block=8)):
        assert qz.qz_cache_attention_workspace(cache(qz, **bad), 3, 5, 4, 4000) == 0
    assert qz.qz_cache_attention_workspace(cache(qz), 0, 0, 4, 4000) == 0


def test_handles_refuse(qz):
    import torch
    u8, f32 = torch.uint8, torch.float32
    good = dict(k_codes=torch.zeros(4, 2, 32, 64, dtype=u8), k_scales=torch.zeros(4, 2, 2), v_codes=torch.zeros(4, 2, 32, 64, dtype=u8),
                v_scales=torch.zeros(4, 2, 2), fmt="e4m3")
    c = qz.KVCache(**good)
    assert (c.pages, c.kv_heads, c.page, c.dim, c.block) == (4, 2, 32, 64, 16)
    for bad in (dict(fmt="mxfp4"), dict(k_codes=torch.zeros(4, 2, 32, 64)), dict(v_codes=torch.zeros(4, 2, 32, 48, dtype=u8)),
                dict(k_scales=torch.zeros(4, 2, 3)), dict(k_scales=torch.zeros(4, 2, 4), v_scales=torch.zeros(4, 2, 4)),
                dict(v_scales=torch.zeros(4, 2, 2, dtype=torch.float64)), dict(k_codes=torch.zeros(2, 4, 32, 64, dtype=u8).transpose(0, 1)),
                dict(k_scales=torch.zeros(4, 2), v_scales=torch.zeros(4, 2))):
        with pytest.raises(ValueError):
            qz.KVCache(**{**good, **bad})
    with pytest.raises(ValueError):
        qz.KVCache.alloc("int8", 4, 2, 40, 64, block=16, device="cpu")
    a = qz.KVCache.alloc("int8", 4, 2, 64, 64, block=16, device="cpu")
    assert a.k_scales.shape == (4, 2, 4) and a.block == 16 and qz.KVCache.alloc("int8", 1, 1, 256, 64, device="cpu").block == 128
    cos = torch.zeros(10, 4)
    for bad in ((cos, torch.zeros(10, 5)), (cos.double(), cos.double()), (cos.T, cos.T), (torch.zeros(0, 4), torch.zeros(0, 4)), (cos[0], cos[0])):
        with pytest.raises(ValueError):
            qz.RotaryTable(*bad)
    t, ints = qz.RotaryTable(cos, cos), lambda *s: torch.zeros(*s, dtype=torch.int32)
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: qz.rotary(x, t), lambda: qz.rotary_backward(x, t), lambda: qz.cache_append(c, x[:, :2], x[:, :2], ints(3, 2), ints(3)),
                 lambda: qz.cache_attention(x, c, ints(3, 2), ints(3)), lambda: qz.cache_attention(x.float(), c, ints(3, 2), ints(3))):
        with pytest.raises(ValueError):  # not on the GPU
            call()
    with pytest.raises(TypeError):
        qz.rotary(x.half(), t)


def test_turns(qz):
    """The scalings of the angles, from their definitions in plain Python."""
    n, base, f = 32, 10000.0, 8.0
    plain = [base ** (-i / n) for i in range(n)]
    close = lambda a, b: all(abs(x - y) <= 1e-12 * abs(y) for x, y in zip(a, b)) and len(a) == len(b)  # noqa: E731
    assert close(qz.rotary_turns(n).tolist(), plain)
    assert close(qz.rotary_turns(n, scaling="linear", factor=f).tolist(), [t / f for t in plain])
    ntk = qz.rotary_turns(n, scaling="ntk", factor=f).tolist()
    assert abs(ntk[0] - 1) < 1e-12 and abs(ntk[-1] - plain[-1] / f) <= 1e-12 * plain[-1]
    parts = qz.rotary_turns(n, scaling="parts", factor=f, original=4096).tolist()
    for i, (t, p) in enumerate(zip(parts, plain)):
        assert p / f * (1 - 1e-12) <= t <= p * (1 + 1e-12)
        if 4096 * p / (2 * math.pi) > 32 * base ** (1 / n):
            assert abs(t - p) <= 1e-12 * p
        if 4096 * p / (2 * math.pi) < base ** (-1 / n):
            assert abs(t - p / f) <= 1e-12 * p
    assert qz.rotary_turns(0).numel() == 0
    for bad in (dict(scaling="x"), dict(scaling="parts", factor=2.0), dict(factor=0.0), dict(base=-1.0)):
        with pytest.raises(ValueError):
            qz.rotary_turns(n, **bad)
