"""Host-side checks of the transformer-block entry points (no GPU needed, no
kernel launched): every call below is refused, or is a no-op, before the GPU is
touched; the packed structs of the Python binding have the C structs' layout.
"""
from __future__ import annotations

import os
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

tern = pytest.importorskip("ternary_weight_quantized_tern_amd",
                           reason="libternary.so not built")
from ternary_weight_quantized_tern_amd import _block as B  # noqa: E402

lib = tern.library()
A = 1 << 20  # a well-aligned address that is never dereferenced
NULL = None


def test_packed_structs_have_the_c_layout(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text(
        '#include "ternary.h"\n#include <stddef.h>\n#include <stdio.h>\n#include <string.h>\n'
        "static void show(const void* p, size_t n) {\n"
        "  for (size_t i = 0; i < n; ++i) printf(\"%02x\", ((const unsigned char*)p)[i]);\n"
        "  printf(\"\\n\"); }\n"
        "int main(void) {\n"
        "  tern_heads h; memset(&h, 0, sizeof h); h.data = (void*)1; h.batch = 2; h.token = 3;\n"
        "  h.head = 4; show(&h, sizeof h);\n"
        "  tern_rope_axes a; memset(&a, 0, sizeof a); a.count = 3; a.width[0] = 16;\n"
        "  a.width[1] = 24; a.width[2] = 8; a.width[3] = 0; a.theta = 500.0;\n"
        "  a.layout = TERN_ROPE_HALVES; show(&a, sizeof a);\n"
        "  tern_residual_norm_args r; memset(&r, 0, sizeof r); r.m = 1; r.c = 2; r.tokens = 3;\n"
        "  r.r_dtype = TERN_BF16; r.pre = TERN_NORM_RMS; r.post = TERN_NORM_LAYER; r.eps = 0.5f;\n"
        "  r.residual_scale = 0.25f; r.pre_weight = (float*)4; r.post_weight = (float*)5;\n"
        "  r.gate = (float*)6; r.ldgate = 7; r.scale = (float*)8; r.ldscale = 9;\n"
        "  r.shift = (float*)10; r.ldshift = 11; show(&r, sizeof r);\n"
        "  tern_attention_shape s; memset(&s, 0, sizeof s); s.batch = 1; s.queries = 2;\n"
        "  s.keys = 3; s.heads = 4; s.kv_heads = 5; s.width = 6; s.scale = 0.5f;\n"
        "  show(&s, sizeof s);\n"
        '  printf("%d %d %d %d\\n", TERN_ROPE_MAX_AXES, TERN_ROPE_MAX_PAIRS,\n'
        "         TERN_RESIDUAL_NORM_MAX_C, TERN_ATTENTION_MAX_WIDTH);\n"
        "  return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    assert lines[0] == B._heads_struct(1, 2, 3, 4).hex()
    assert lines[1] == B._axes((16, 24, 8), 500.0, "halves").hex()
    assert lines[2] == B._norm_struct(1, 2, 3, 1, 2, 1, 0.5, 0.25, 4, 5, 6, 7, 8, 9, 10, 11).hex()
    assert lines[3] == B._shape_struct(1, 2, 3, 4, 5, 6, 0.5).hex()
    assert lines[4].split() == [str(v) for v in (tern.TERN_ROPE_MAX_AXES, tern.TERN_ROPE_MAX_PAIRS,
                                                 tern.TERN_RESIDUAL_NORM_MAX_C,
                                                 tern.TERN_ATTENTION_MAX_WIDTH)]


def heads(data=A, batch=1024, token=128, head=64):
    return B._heads_struct(data, batch, token, head)


def axes(count=3, width=(16, 24, 24, 0), theta=10000.0, layout=0):
    return struct.pack("@5id2i", count, *width, theta, layout, 0)


def rope(x=heads(), y=heads(), dtype=1, b=1, t=4, h=2, d=64, pos=A, pb=12, pt=3, a=axes()):
    return lib.tern_rope(x, y, dtype, b, t, h, d, pos, pb, pt, a, 0, NULL)


def test_rope_validation():
    assert rope(dtype=5) == tern.TERN_ERR_DTYPE
    assert rope(a=NULL) == tern.TERN_ERR_NULL
    for bad in (axes(count=0), axes(count=5), axes(width=(15, 24, 24, 0)), axes(width=(-2, 24, 24, 0)),
                axes(theta=0.0), axes(theta=float("inf")), axes(theta=float("nan")), axes(layout=2),
                axes(width=(40, 24, 24, 0)), axes(width=(300, 0, 0, 0))):
        assert rope(a=bad) == tern.TERN_ERR_ARG
    for bad in (dict(b=-1), dict(b=65536), dict(t=-1), dict(h=-1), dict(d=0), dict(d=(1 << 20) + 1),
                dict(t=1 << 30, h=4), dict(t=1 << 24, h=2)):
        assert rope(**bad) == tern.TERN_ERR_SHAPE
    assert rope(x=NULL, y=NULL, pos=NULL, t=0) == tern.TERN_OK
    assert rope(x=NULL) == tern.TERN_ERR_NULL
    assert rope(y=heads(data=0)) == tern.TERN_ERR_NULL
    assert rope(pos=NULL) == tern.TERN_ERR_NULL
    assert rope(x=heads(token=-1)) == tern.TERN_ERR_STRIDE
    assert rope(pt=-3) == tern.TERN_ERR_STRIDE
    assert rope(x=heads(data=A + 1)) == tern.TERN_ERR_ALIGN
    assert rope(dtype=0, y=heads(data=A + 2)) == tern.TERN_ERR_ALIGN
    assert rope(pos=A + 2) == tern.TERN_ERR_ALIGN


def norm_args(m=8, c=64, tokens=4, dtype=1, pre=1, post=0, eps=1e-6, alpha=1.0, wpre=0, wpost=0,
              gate=A, ldgate=64, scale=A, ldscale=64, shift=A, ldshift=64):
    return B._norm_struct(m, c, tokens, dtype, pre, post, eps, alpha, wpre, wpost, gate, ldgate,
                          scale, ldscale, shift, ldshift)


def norm(a=norm_args(), r=A, ldr=64, y=A, ldy=64, ro=A, ldro=64, h=A, ldh=64, stats=NULL):
    return lib.tern_residual_norm(a, r, ldr, y, ldy, ro, ldro, h, ldh, stats, NULL)


BAD_NORM = [(dict(dtype=3), tern.TERN_ERR_DTYPE), (dict(pre=3), tern.TERN_ERR_ARG),
            (dict(post=7), tern.TERN_ERR_ARG), (dict(eps=-1.0), tern.TERN_ERR_ARG),
            (dict(eps=float("nan")), tern.TERN_ERR_ARG), (dict(alpha=float("inf")), tern.TERN_ERR_ARG),
            (dict(wpost=A), tern.TERN_ERR_ARG), (dict(m=-1), tern.TERN_ERR_SHAPE),
            (dict(m=1 << 31), tern.TERN_ERR_SHAPE), (dict(c=0), tern.TERN_ERR_SHAPE),
            (dict(c=8193), tern.TERN_ERR_SHAPE), (dict(tokens=0), tern.TERN_ERR_SHAPE),
            (dict(ldgate=63), tern.TERN_ERR_STRIDE), (dict(ldscale=0), tern.TERN_ERR_STRIDE),
            (dict(gate=A + 2), tern.TERN_ERR_ALIGN), (dict(wpre=A + 1), tern.TERN_ERR_ALIGN)]


def test_residual_norm_validation():
    assert norm(a=NULL) == tern.TERN_ERR_NULL
    for bad, status in BAD_NORM:
        assert norm(a=norm_args(**bad)) == status, bad
    assert norm(a=norm_args(pre=0)) == tern.TERN_ERR_ARG        # h without its norm
    assert norm(a=norm_args(m=0), r=NULL, y=NULL, h=NULL) == tern.TERN_OK
    assert norm(r=NULL) == tern.TERN_ERR_NULL
    assert norm(y=NULL, h=NULL) == tern.TERN_ERR_NULL
    assert norm(ro=NULL) == tern.TERN_ERR_NULL
    for bad in (dict(ldr=63), dict(ldy=10), dict(ldro=0), dict(ldh=63)):
        assert norm(**bad) == tern.TERN_ERR_STRIDE
    assert norm(a=norm_args(ldshift=63)) == tern.TERN_ERR_STRIDE
    for bad in (dict(r=A + 1), dict(y=A + 1), dict(h=A + 1), dict(stats=A + 8)):
        assert norm(**bad) == tern.TERN_ERR_ALIGN


def norm_bwd(a=norm_args(), dro=A, lddro=64, dh=A, lddh=64, ro=A, ldro=64, y=A, ldy=64, st=A, dr=A,
             lddr=64, dy=A, lddy=64, dg=A, ds=A, dsh=A, dwpre=NULL, dwpost=NULL, ws=A, wsb=1 << 30):
    return lib.tern_residual_norm_bwd(a, dro, lddro, dh, lddh, ro, ldro, y, ldy, st, dr, lddr, dy,
                                      lddy, dg, ds, dsh, dwpre, dwpost, ws, wsb, NULL)


def test_residual_norm_bwd_validation():
    assert norm_bwd(a=NULL) == tern.TERN_ERR_NULL
    for bad, status in BAD_NORM:
        assert norm_bwd(a=norm_args(**bad)) == status, bad
    assert norm_bwd(dwpost=A) == tern.TERN_ERR_ARG               # no post norm
    assert norm_bwd(dh=NULL) == tern.TERN_ERR_ARG                # dscale without dh
    assert norm_bwd(y=NULL) == tern.TERN_ERR_ARG                 # dgate without y
    need = lib.tern_residual_norm_bwd_workspace(norm_args())
    assert need > 0 and norm_bwd(wsb=need - 1) == tern.TERN_ERR_SHAPE
    assert norm_bwd(dro=NULL, dh=NULL, ds=NULL, dsh=NULL) == tern.TERN_ERR_NULL
    for bad in (dict(ro=NULL), dict(st=NULL), dict(dr=NULL), dict(dy=NULL), dict(ws=NULL)):
        assert norm_bwd(**bad) == tern.TERN_ERR_NULL
    for bad in (dict(lddro=63), dict(lddh=1), dict(ldro=2), dict(ldy=63), dict(lddr=0), dict(lddy=63)):
        assert norm_bwd(**bad) == tern.TERN_ERR_STRIDE
    for bad in (dict(dro=A + 1), dict(dh=A + 1), dict(st=A + 4), dict(ws=A + 8), dict(dg=A + 2)):
        assert norm_bwd(**bad) == tern.TERN_ERR_ALIGN
    assert lib.tern_residual_norm_bwd_workspace(norm_args(m=0)) == 0
    assert lib.tern_residual_norm_bwd_workspace(norm_args(c=9000)) == 0
    # no sums wanted and nothing to sum: an empty call touches nothing
    assert norm_bwd(a=norm_args(m=0), dro=NULL, dh=NULL, y=NULL, dg=NULL, ds=NULL, dsh=NULL, ws=NULL,
                    wsb=0) == tern.TERN_OK


def shape(b=2, s=8, keys=8, h=4, hkv=2, d=64, scale=0.125):
    return B._shape_struct(b, s, keys, h, hkv, d, scale)


def attention(q=heads(), k=heads(), v=heads(), o=heads(), sh=shape(), mask=NULL, ld=0, lse=A, ws=A,
              wsb=1 << 40):
    return lib.tern_attention(q, k, v, o, sh, mask, ld, lse, ws, wsb, NULL)


def attention_bwd(do=heads(), q=heads(), k=heads(), v=heads(), o=heads(), lse=A, dq=heads(),
                  dk=heads(), dv=heads(), sh=shape(), mask=NULL, ld=0, ws=A, wsb=1 << 40):
    return lib.tern_attention_bwd(do, q, k, v, o, lse, dq, dk, dv, sh, mask, ld, ws, wsb, NULL)


@pytest.mark.parametrize("call", [attention, attention_bwd])
def test_attention_validation(call):
    assert call(sh=NULL) == tern.TERN_ERR_NULL
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert call(sh=shape(scale=bad)) == tern.TERN_ERR_ARG
    for bad in (dict(b=-1), dict(s=-1), dict(keys=-1), dict(h=-4), dict(hkv=-1), dict(hkv=3),
                dict(hkv=0), dict(d=0), dict(d=60), dict(d=136), dict(s=1 << 30),
                dict(keys=1 << 36), dict(b=1 << 30, h=4)):
        assert call(sh=shape(**bad)) == tern.TERN_ERR_SHAPE, bad
    assert call(sh=shape(b=0)) == tern.TERN_OK
    assert call(sh=shape(h=0)) == tern.TERN_OK
    assert call(q=NULL) == tern.TERN_ERR_NULL
    assert call(k=heads(data=0)) == tern.TERN_ERR_NULL
    assert call(o=heads(data=0)) == tern.TERN_ERR_NULL
    assert call(mask=A, ld=7) == tern.TERN_ERR_STRIDE
    assert call(v=heads(token=-8)) == tern.TERN_ERR_STRIDE
    assert call(k=heads(token=1 << 22)) == tern.TERN_ERR_STRIDE
    for bad in (dict(q=heads(data=A + 8)), dict(k=heads(head=60)), dict(v=heads(token=12)),
                dict(o=heads(batch=4)), dict(lse=A + 2)):
        assert call(**bad) == tern.TERN_ERR_ALIGN, bad


def test_attention_workspaces():
    ws = lib.tern_attention_workspace
    assert ws(shape(), 0, 0) == 0                               # one part: nothing to join
    long = shape(b=1, s=1, keys=100000)
    need = ws(long, 0, 0)
    assert need > 0 and ws(long, 1, 0) >= need > ws(shape(b=1, s=1, keys=4096), 0, 0)
    assert attention(sh=long, wsb=need - 1) == tern.TERN_ERR_SHAPE
    assert attention(sh=long, ws=NULL, wsb=need) == tern.TERN_ERR_NULL
    assert attention(sh=long, ws=A + 4, wsb=need) == tern.TERN_ERR_ALIGN
    assert ws(shape(), 0, 1) == 0                               # few rows, one part: one kernel
    many = shape(s=40)
    back = ws(many, 0, 1)
    assert back >= 2 * 2 * 4 * 40 * 4                           # two statistics of each row
    assert attention_bwd(sh=many, wsb=back - 1) == tern.TERN_ERR_SHAPE
    assert attention_bwd(sh=many, ws=NULL, wsb=back) == tern.TERN_ERR_NULL
    assert attention_bwd(dk=heads(data=0)) == tern.TERN_ERR_NULL
    assert attention_bwd(lse=NULL) == tern.TERN_ERR_NULL
    for bad in (shape(hkv=3), shape(scale=0.0), NULL):
        assert ws(bad, 0, 0) == 0 and ws(bad, 0, 1) == 0
    assert attention(sh=shape(s=0)) == tern.TERN_OK
    assert attention_bwd(sh=shape(s=0, keys=0)) == tern.TERN_OK
