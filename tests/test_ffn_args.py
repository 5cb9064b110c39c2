"""What the products with 4-bit weights and the layer norm refuse, without a GPU: the C calls
return their errors before any CUDA call, the binding raises before the library is called."""
import ctypes as C
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


def weight(qz, fmt=None, rows=64, cols=128, block=None, codes=FAKE, scales=FAKE, ts=FAKE):
    fmt = qz.QZ_NVFP4 if fmt is None else fmt
    return qz.QzWeight(fmt, block or {qz.QZ_MXFP4: 32, qz.QZ_NVFP4: 16}.get(fmt, 128), rows, cols, codes, scales, ts)


def test_weight_layout_matches_header(qz, tmp_path):
    src = tmp_path / "w.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qz.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu %d %d\\n", sizeof(qz_weight), offsetof(qz_weight, rows),'
                   ' offsetof(qz_weight, codes), offsetof(qz_weight, tensor_scale_dev), QZ_ACT_SILU, QZ_ACT_GELU_TANH);'
                   ' return 0;}\n')
    exe = tmp_path / "w"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    w = qz.QzWeight
    assert got == [C.sizeof(w), w.rows.offset, w.codes.offset, w.tensor_scale_dev.offset, qz.QZ_ACT_SILU, qz.QZ_ACT_GELU_TANH]


def test_weight_errors(qz):
    lin = lambda w: qz.qz_linear(w, FAKE, 128, 4, FAKE, 64, qz.QZ_BF16)  # noqa: E731
    assert qz.lib().qz_linear(None, FAKE, 128, 4, FAKE, 64, qz.QZ_BF16, None) == qz.QZ_ERR_NULL
    assert lin(weight(qz, qz.QZ_INT8)) == qz.QZ_ERR_ENUM
    assert lin(weight(qz, 99)) == qz.QZ_ERR_ENUM
    assert lin(weight(qz, qz.QZ_MXFP4, block=16)) == qz.QZ_ERR_UNSUPPORTED
    assert lin(weight(qz, qz.QZ_INT4, block=48)) == qz.QZ_ERR_UNSUPPORTED
    assert lin(weight(qz, qz.QZ_MXFP4, cols=120)) == qz.QZ_ERR_SHAPE
    assert lin(weight(qz, rows=-1)) == qz.QZ_ERR_SHAPE
    assert lin(weight(qz, rows=1 << 31)) == qz.QZ_ERR_UNSUPPORTED
    assert lin(weight(qz, codes=None)) == qz.QZ_ERR_NULL
    assert lin(weight(qz, scales=None)) == qz.QZ_ERR_NULL
    assert lin(weight(qz, qz.QZ_INT4, scales=FAKE + 2)) == qz.QZ_ERR_ALIGN
    assert lin(weight(qz, ts=FAKE + 2)) == qz.QZ_ERR_ALIGN


def test_linear_errors(qz):
    w = weight(qz)
    for call, width, out in ((qz.qz_linear, 128, 64), (qz.qz_linear_backward, 64, 128)):
        ok = (w, FAKE, width, 4, FAKE, out, qz.QZ_F32)
        swap = lambda i, v: call(*ok[:i], v, *ok[i + 1:])  # noqa: E731
        assert swap(1, None) == qz.QZ_ERR_NULL and swap(4, None) == qz.QZ_ERR_NULL
        assert swap(1, FAKE + 1) == qz.QZ_ERR_ALIGN and swap(4, FAKE + 2) == qz.QZ_ERR_ALIGN
        assert swap(2, width - 1) == qz.QZ_ERR_SHAPE and swap(5, out - 1) == qz.QZ_ERR_SHAPE
        assert swap(3, -1) == qz.QZ_ERR_SHAPE and swap(3, 1 << 31) == qz.QZ_ERR_UNSUPPORTED
        assert swap(2, 1 << 62) == qz.QZ_ERR_SHAPE
        assert swap(6, 7) == qz.QZ_ERR_ENUM
        assert swap(3, 0) == qz.QZ_OK  # nothing to do, nothing enqueued


def test_gated_errors(qz):
    g, act = weight(qz), qz.QZ_ACT_SILU
    fwd = lambda up=g, a=act, x=FAKE, ldx=128, t=4, h=FAKE, ldh=64, go=FAKE, uo=FAKE, ldg=64: qz.qz_gated_ffn(  # noqa: E731
        g, up, a, x, ldx, t, h, ldh, go, uo, ldg)
    assert fwd(a=3) == qz.QZ_ERR_ENUM
    assert fwd(up=weight(qz, rows=72)) == qz.QZ_ERR_SHAPE
    assert fwd(up=weight(qz, qz.QZ_MXFP4)) == qz.QZ_ERR_SHAPE
    assert fwd(up=weight(qz, codes=None)) == qz.QZ_ERR_NULL
    assert fwd(go=None) == qz.QZ_ERR_NULL and fwd(uo=None) == qz.QZ_ERR_NULL
    assert fwd(x=None) == qz.QZ_ERR_NULL and fwd(h=None) == qz.QZ_ERR_NULL
    assert fwd(ldx=127) == qz.QZ_ERR_SHAPE and fwd(ldh=63) == qz.QZ_ERR_SHAPE and fwd(ldg=63) == qz.QZ_ERR_SHAPE
    assert fwd(uo=FAKE + 1) == qz.QZ_ERR_ALIGN
    assert fwd(t=0) == qz.QZ_OK
    bwd = lambda up=g, a=act, p=(FAKE,) * 6, ld=(64, 64, 64, 128), t=4: qz.qz_gated_ffn_backward(  # noqa: E731
        g, up, a, p[0], ld[0], p[1], p[2], ld[1], t, p[3], p[4], ld[2], p[5], ld[3])
    for i in range(6):
        p = [FAKE] * 6
        p[i] = None
        assert bwd(p=p) == qz.QZ_ERR_NULL
        p[i] = FAKE + 1
        assert bwd(p=p) == qz.QZ_ERR_ALIGN
    for i in range(4):
        ld = [64, 64, 64, 128]
        ld[i] -= 1
        assert bwd(ld=ld) == qz.QZ_ERR_SHAPE
    assert bwd(a=0) == qz.QZ_ERR_ENUM and bwd(t=0) == qz.QZ_OK and bwd(t=-1) == qz.QZ_ERR_SHAPE


def test_norm_errors(qz):
    f = lambda dt=qz.QZ_BF16, x=FAKE, ldx=64, r=4, c=64, w=None, eps=1e-5, y=FAKE, ldy=64: qz.qz_layer_norm(  # noqa: E731
        dt, x, ldx, r, c, w, None, eps, y, ldy, None, None)
    assert f(dt=9) == qz.QZ_ERR_ENUM
    assert f(x=None) == qz.QZ_ERR_NULL and f(y=None) == qz.QZ_ERR_NULL
    assert f(x=FAKE + 1) == qz.QZ_ERR_ALIGN and f(w=FAKE + 2) == qz.QZ_ERR_ALIGN
    assert f(ldx=63) == qz.QZ_ERR_SHAPE and f(ldy=63) == qz.QZ_ERR_SHAPE and f(r=-1) == qz.QZ_ERR_SHAPE
    assert f(c=0) == qz.QZ_ERR_SHAPE and f(eps=-1.0) == qz.QZ_ERR_SHAPE and f(eps=float("nan")) == qz.QZ_ERR_SHAPE
    assert f(c=1 << 31, ldx=1 << 31, ldy=1 << 31) == qz.QZ_ERR_UNSUPPORTED
    assert f(r=0) == qz.QZ_OK
    need = qz.qz_layer_norm_backward_workspace(4, 64)
    assert need >= 2 * 64 * 4 and qz.qz_layer_norm_backward_workspace(0, 64) == 0
    b = lambda dy=FAKE, x=FAKE, m=FAKE, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, n=need, ld=64: qz.qz_layer_norm_backward(  # noqa: E731
        qz.QZ_F32, dy, 64, x, ld, 4, 64, m, FAKE, None, dx, 64, dw, db, ws, n)
    assert b(dy=None) == b(x=None) == b(m=None) == b(dx=None) == qz.QZ_ERR_NULL
    assert b(dw=None) == b(db=None) == qz.QZ_ERR_NULL  # both or neither
    assert b(ws=None) == b(n=need - 1) == qz.QZ_ERR_WORKSPACE
    assert b(ws=FAKE + 8) == b(dw=FAKE + 2) == b(x=FAKE + 2) == qz.QZ_ERR_ALIGN
    assert b(ld=63) == qz.QZ_ERR_SHAPE


def test_binding_refuses(qz):
    import torch
    q = qz.Quantized(torch.zeros(64, 64, dtype=torch.uint8), torch.zeros(64, 8, dtype=torch.uint8), torch.ones(1),
                     qz.QZ_NVFP4, qz.QZ_GRAN_BLOCK, 0, 64, 128, 16)
    w = qz.Weight(q)
    assert (w.rows, w.cols) == (64, 128)
    import dataclasses
    for bad in (dict(fmt=qz.QZ_INT8), dict(rows=63), dict(scales=torch.zeros(64, 8)), dict(tensor_scale=None),
                dict(codes=torch.zeros(64, 128, dtype=torch.uint8)[:, ::2])):
        with pytest.raises(ValueError):
            qz.Weight(dataclasses.replace(q, **bad))
    for x in (torch.zeros(2, 128, dtype=torch.bfloat16),  # not on the GPU
              torch.zeros(2, 128), torch.zeros(128, dtype=torch.bfloat16), torch.zeros(2, 127, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            qz.linear(x, w)
    with pytest.raises(KeyError):
        qz._activation("relu")
    with pytest.raises(TypeError):
        qz.layer_norm(torch.zeros(2, 8, dtype=torch.float16))
