"""Refusals of the prompt operators that need no GPU: the binding's checks of
what a pointer cannot show, and the library's checks before any CUDA call."""
import ctypes
import os

import pytest
import torch

from test_binding_host import _Spy, _passes, _QUERIES, _refused

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
D = 128
SIZES = {"bitlinear_attention_prefill_workspace_bytes", "bitlinear_adapter_workspace_bytes"}


@pytest.fixture()
def spy(monkeypatch):
    import bit_ternary_weight_b200 as b
    import test_binding_host as host
    monkeypatch.setattr(host, "_QUERIES", _QUERIES | SIZES)
    monkeypatch.setattr(b, "_stream", lambda device: ctypes.c_void_p(0))
    sp = _Spy(b._lib)
    monkeypatch.setattr(b, "_lib", sp)
    return sp


@pytest.fixture()
def bl(spy):
    import bit_ternary_weight_b200 as b
    return b


def _z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def _ws():
    return torch.zeros(1 << 10, dtype=torch.uint8)


def test_heads_struct_matches_the_header(tmp_path):
    import shutil
    import subprocess
    import bit_ternary_weight_b200 as bl
    if not shutil.which("gcc"):
        pytest.skip("no C compiler")
    fields = [f[0] for f in bl.HeadsC._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bitlinear.h"\nint main(void){'
                   'printf("%zu", sizeof(bitlinear_heads));'
                   + "".join(f'printf(" %zu", offsetof(bitlinear_heads, {f}));' for f in fields) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(bl.HeadsC)] + [getattr(bl.HeadsC, f).offset for f in fields]


def test_valid_layouts_reach_the_library(bl, spy):
    T, H, Hkv = 6, 4, 2
    qkv = _z(T, H + 2 * Hkv, D)
    cache = _z(2, Hkv, 32, D)
    pos, table = _z(T, dtype=I32), _z(16, 64, 2, dtype=F32)
    ck, cv = cache[0].transpose(0, 1), cache[1].transpose(0, 1)
    _passes(bl, spy, lambda: bl.qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], pos, table,
                                             q_gain=_z(D), k_gain=_z(D), slots=pos, k_out=ck, v_out=cv))
    _passes(bl, spy, lambda: bl.qk_norm_rope(qkv[:, :H].float(), ck[:T].float(), None, pos, table))
    cu = _z(2, dtype=I32)
    _passes(bl, spy, lambda: bl.attention_prefill(qkv[:, :H], ck, cv, cu, cu, workspace=_ws()))
    _passes(bl, spy, lambda: bl.adapter_add(_z(T, 10), _z(T, 64), _z(3, 8, 64), _z(3, 10, 8), pos, workspace=_ws()))


def test_rope_buffers_are_checked(bl, spy):
    T, H, Hkv = 6, 4, 2
    q, k, v = _z(T, H, D), _z(T, Hkv, D), _z(T, Hkv, D)
    pos, table = _z(T, dtype=I32), _z(16, 64, 2, dtype=F32)

    def refused(status, words, *a, **kw):
        _refused(bl, spy, lambda: bl.qk_norm_rope(*a, **kw), status, words)

    refused(bl.BL_ERR_SHAPE, "k of shape", q, _z(T + 1, Hkv, D), v, pos, table)
    refused(bl.BL_ERR_SHAPE, "q of shape", _z(T, H, 64), k, v, pos, table)
    refused(bl.BL_ERR_SHAPE, "q of shape", _z(T, H * D), k, v, pos, table)
    refused(bl.BL_ERR_SHAPE, "q of shape", _z(T, H, 2 * D)[..., ::2], k, v, pos, table)
    refused(bl.BL_ERR_DTYPE, "mixed", q, k.float(), v, pos, table)
    refused(bl.BL_ERR_DTYPE, "q is float16", q.half(), k.half(), v.half(), pos, table)
    refused(bl.BL_ERR_DTYPE, "positions is int64", q, k, v, pos.long(), table)
    refused(bl.BL_ERR_SHAPE, "positions", q, k, v, pos[:-1], table)
    refused(bl.BL_ERR_SHAPE, "table of shape", q, k, v, pos, table[:, :32])
    refused(bl.BL_ERR_DTYPE, "table is", q, k, v, pos, table.double())
    refused(bl.BL_ERR_SHAPE, "q_gain", q, k, v, pos, table, q_gain=_z(64))
    refused(bl.BL_ERR_DTYPE, "gains of mixed", q, k, v, pos, table, q_gain=_z(D), k_gain=_z(D, dtype=F32))
    refused(bl.BL_ERR_NULL, "slots need", q, k, v, pos, table, slots=pos)
    refused(bl.BL_ERR_NULL, "v_out needs v", q, k, None, pos, table, v_out=v)
    refused(bl.BL_ERR_SHAPE, "rows for", q, k, v, pos, table, k_out=_z(T - 1, Hkv, D), v_out=_z(T - 1, Hkv, D))
    refused(bl.BL_ERR_SHAPE, "v_out of shape", q, k, v, pos, table, slots=pos, k_out=_z(9, Hkv, D),
            v_out=_z(8, Hkv, D))
    refused(bl.BL_ERR_DTYPE, "q_out is float32", q, k, v, pos, table, q_out=_z(T, H, D, dtype=F32))
    refused(bl.BL_ERR_SHAPE, "slots", q, k, v, pos, table, slots=pos[:2], k_out=k, v_out=v)


def test_attention_buffers_are_checked(bl, spy):
    q, k, v, cu = _z(6, 4, D), _z(9, 2, D), _z(9, 2, D), _z(3, dtype=I32)

    def refused(status, words, *a, **kw):
        _refused(bl, spy, lambda: bl.attention_prefill(*a, workspace=_ws(), **kw), status, words)

    refused(bl.BL_ERR_DTYPE, "q is float32", q.float(), k, v, cu)
    refused(bl.BL_ERR_SHAPE, "v of shape", q, k, v[:-1], cu)
    refused(bl.BL_ERR_SHAPE, "query heads", q, _z(9, 3, D), _z(9, 3, D), cu)
    refused(bl.BL_ERR_SHAPE, "out of shape", q, k, v, cu, out=_z(5, 4, D))
    refused(bl.BL_ERR_DTYPE, "cu_q is int64", q, k, v, cu.long())
    refused(bl.BL_ERR_SHAPE, "cu_k of 2", q, k, v, cu, cu[:2])
    refused(bl.BL_ERR_SHAPE, "cu_q", q, k, v, cu[:1])
    refused(bl.BL_ERR_SHAPE, "cu_q", q, k, v, _z(6, dtype=I32)[::2])


def test_adapter_buffers_are_checked(bl, spy):
    T, K, N, r, n = 5, 64, 10, 8, 3
    y, x, down, up, index = _z(T, N), _z(T, K), _z(n, r, K), _z(n, N, r), _z(T, dtype=I32)

    def refused(status, words, *a, **kw):
        _refused(bl, spy, lambda: bl.adapter_add(*a, workspace=_ws(), **kw), status, words)

    refused(bl.BL_ERR_SHAPE, "two dimensions", y[0], x, down, up, index)
    refused(bl.BL_ERR_SHAPE, "up of shape", y, x, down, _z(n, N, r + 8), index)
    refused(bl.BL_ERR_SHAPE, "x of shape", y, x[:-1], down, up, index)
    refused(bl.BL_ERR_DTYPE, "x is float32", y, x.float(), down, up, index)
    refused(bl.BL_ERR_DTYPE, "up is float32", y, x, down, up.float(), index)
    refused(bl.BL_ERR_SHAPE, "down", y, x, _z(n, K, r).transpose(1, 2), up, index)
    refused(bl.BL_ERR_DTYPE, "out and y", y, x, down, up, index, out=y.float())
    refused(bl.BL_ERR_SHAPE, "out of shape", y, x, down, up, index, out=_z(T, N - 1))
    refused(bl.BL_ERR_SHAPE, "index", y, x, down, up, index[:-1])
    refused(bl.BL_ERR_SHAPE, "scale", y, x, down, up, index, scale=_z(n - 1, dtype=F32))
    refused(bl.BL_ERR_DTYPE, "scale is bfloat16", y, x, down, up, index, scale=_z(n))


A = 0x7f0000000000          # a 16-byte aligned address that is never read


def _h(bl, rows=8, row=256, head=128, data=A):
    return bl.HeadsC(data, rows, row, head)


def test_rope_argument_errors_before_any_cuda_call(bl):
    L = bl.lib

    def call(q=None, k=None, v=None, xt=1, H=2, Hkv=2, D=128, pos=A, tab=A, rows=64, qg=None, kg=None, gt=0, eps=1e-5,
             slots=None, qo=None, ko=None, vo=None, flags=0):
        d = _h(bl)
        p = [ctypes.byref(h or d) for h in (q, k, v, qo, ko, vo)]
        return L.bitlinear_qk_norm_rope(*p[:3], xt, H, Hkv, D, pos, tab, rows, qg, kg, gt, eps, slots, *p[3:], flags,
                                        None)

    assert call(pos=None) == bl.BL_ERR_NULL
    assert call(v=_h(bl, data=0)) == bl.BL_ERR_NULL                # values without v, with v_out
    d = ctypes.byref(_h(bl))
    assert L.bitlinear_qk_norm_rope(None, d, None, 1, 2, 2, 128, A, A, 64, None, None, 0, 1e-5, None, d, d, None, 0,
                                    None) == bl.BL_ERR_NULL
    assert call(xt=5) == bl.BL_ERR_DTYPE
    assert call(qg=A, gt=7) == bl.BL_ERR_DTYPE
    for kw in (dict(D=64), dict(H=0), dict(rows=0), dict(flags=1), dict(flags=64), dict(qg=A, eps=-1.0),
               dict(qg=A, eps=float("nan")), dict(q=_h(bl, rows=0)), dict(k=_h(bl, rows=7)), dict(q=_h(bl, row=64)),
               dict(k=_h(bl, head=0)), dict(ko=_h(bl, rows=7), vo=_h(bl, rows=7)), dict(vo=_h(bl, rows=9)),
               dict(qo=_h(bl, row=128)),                           # rows of an output on top of one another
               dict(ko=_h(bl, row=128, head=128 * 7)), dict(q=_h(bl, row=1 << 40))):
        assert call(**kw) == bl.BL_ERR_SHAPE, kw
    for kw in (dict(q=_h(bl, data=A + 8)), dict(q=_h(bl, row=260)), dict(ko=_h(bl, head=132, row=512)), dict(pos=A + 2),
               dict(tab=A + 4), dict(kg=A + 4), dict(slots=A + 1)):
        assert call(**kw) == bl.BL_ERR_ALIGN, kw


def test_attention_argument_errors_before_any_cuda_call(bl):
    L = bl.lib

    def call(q=None, k=None, v=None, cu=A, batch=2, H=2, Hkv=2, D=128, scale=0.1, out=None, ws=A, n=1 << 40, flags=0):
        d = _h(bl)
        p = [ctypes.byref(h or d) for h in (q, k, v, out)]
        return L.bitlinear_attention_prefill(*p[:3], cu, A, batch, H, Hkv, D, scale, p[3], ws, n, flags, None)

    assert call(cu=None) == bl.BL_ERR_NULL
    assert call(out=_h(bl, data=0)) == bl.BL_ERR_NULL
    for kw in (dict(D=64), dict(batch=0), dict(batch=65536), dict(H=3), dict(H=0), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(flags=8), dict(v=_h(bl, rows=9)),
               dict(out=_h(bl, rows=9)), dict(out=_h(bl, row=128)), dict(k=_h(bl, row=0)), dict(q=_h(bl, rows=0)),
               dict(k=_h(bl, rows=1 << 31), v=_h(bl, rows=1 << 31)), dict(H=130, Hkv=2)):
        assert call(**kw) == bl.BL_ERR_SHAPE, kw
    for kw in (dict(q=_h(bl, data=A + 2)), dict(k=_h(bl, row=260)), dict(out=_h(bl, head=130, row=512)), dict(cu=A + 2),
               dict(ws=A + 8)):
        assert call(**kw) == bl.BL_ERR_ALIGN, kw
    # not in place
    for name in "qkv":
        apart = {x: _h(bl, data=A + 4096 * i) for i, x in enumerate(("q", "k", "v", "out"))}
        assert call(**{**apart, "out": apart[name]}) == bl.BL_ERR_SHAPE, name
        assert call(**apart) not in (bl.BL_OK, bl.BL_ERR_NULL, bl.BL_ERR_SHAPE, bl.BL_ERR_ALIGN)   # no such memory
    assert L.bitlinear_attention_prefill_workspace_bytes(3, 2) == 0
    assert L.bitlinear_attention_prefill_workspace_bytes(65, 1) == 0


def test_adapter_argument_errors_before_any_cuda_call(bl):
    L = bl.lib

    def call(y=A, yt=1, ldy=32, x=A, ldx=64, T=4, N=32, K=64, down=A, up=A, n=2, r=8, index=A, scale=None, out=A + 4096,
             ldo=32, ws=A, nb=1 << 40, flags=0):
        return L.bitlinear_adapter_add(y, yt, ldy, x, ldx, T, N, K, down, up, n, r, index, scale, out, ldo, ws, nb,
                                       flags, None)

    for kw in (dict(y=None), dict(x=None), dict(down=None), dict(up=None), dict(index=None), dict(out=None)):
        assert call(**kw) == bl.BL_ERR_NULL, kw
    assert call(yt=4) == bl.BL_ERR_DTYPE
    for kw in (dict(T=0), dict(N=0), dict(K=96), dict(K=0), dict(n=0), dict(n=65537), dict(r=0), dict(r=12),
               dict(r=136), dict(ldy=31), dict(ldo=31), dict(ldx=56), dict(flags=2), dict(out=A, ldo=40)):
        assert call(**kw) == bl.BL_ERR_SHAPE, kw
    for kw in (dict(x=A + 8), dict(ldx=68), dict(down=A + 2), dict(up=A + 8), dict(index=A + 2), dict(out=A + 1),
               dict(yt=0, y=A + 2), dict(scale=A + 2), dict(ws=A + 4)):
        assert call(**kw) == bl.BL_ERR_ALIGN, kw
    assert L.bitlinear_adapter_workspace_bytes(0, 8) == 0
    assert L.bitlinear_adapter_workspace_bytes(4, 12) == 0
