"""The entry points of the layers beside the gated delta rule refuse bad
arguments before any device work (no GPU needed)."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from linear_attn_decode_pace_amd import layers, pace

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK_PTR = 0x10000        # an aligned address; refused calls never read it
EINVAL, EUNSUPPORTED = pace.PACE_EINVAL, pace.PACE_EUNSUPPORTED


@pytest.mark.parametrize("name", ["pace_norm_config", "pace_kv4_config"])
def test_structs_match_header(name, tmp_path):
    struct = getattr(pace, name)
    text = open(os.path.join(ROOT, "include", "pace.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
    names = re.findall(r"\b([a-z0-9_]+);", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
    assert names == [n for n, _ in struct._fields_]
    prog = '#include <stddef.h>\n#include <stdio.h>\n#include "pace.h"\nint main(void) {\n'
    prog += 'printf("%%zu\\n", sizeof(%s));\n' % name
    prog += "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (name, n) for n in names) + "return 0;}\n"
    (tmp_path / "a.c").write_text(prog)
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")],
                   check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(struct)] + [getattr(struct, n).offset for n in names]


def status(fn, *args):
    rc = getattr(pace.LIB, fn)(*args)
    if rc != pace.PACE_OK:
        assert pace.pace_last_error() != ""
    return rc


def norm_call(q=OK_PTR, k=OK_PTR, qw=None, kw=None, pos=None, freq=None, qo=OK_PTR * 2, ko=OK_PTR * 2, **kw2):
    c = dict(tokens=4, heads_q=2, heads_k=1, d=64, in_dtype=pace.PACE_DTYPE_BF16, norm=pace.PACE_NORM_L2, eps=1e-6,
             q_scale=1.0, rot=0, rot_pairs=0, q_stride=128, k_stride=64)
    c.update(kw2)
    cfg = pace.pace_norm_config(**c)
    return status("pace_qk_norm_rope", ctypes.byref(cfg), q, k, qw, kw, pos, freq, qo, ko, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), EINVAL), (dict(heads_q=-1), EINVAL), (dict(heads_k=-2), EINVAL), (dict(d=0), EINVAL),
    (dict(d=1025, q_stride=4096, k_stride=4096), EUNSUPPORTED), (dict(in_dtype=2), EINVAL), (dict(norm=3), EINVAL),
    (dict(eps=-1e-6), EINVAL), (dict(eps=math.nan), EINVAL), (dict(eps=math.inf), EINVAL),
    (dict(q_scale=math.inf), EINVAL), (dict(rot=3, pos=OK_PTR, freq=OK_PTR), EINVAL),
    (dict(rot=66, pos=OK_PTR, freq=OK_PTR), EINVAL), (dict(rot=-2), EINVAL), (dict(rot=2), EINVAL),
    (dict(rot=2, pos=OK_PTR), EINVAL), (dict(rot=2, pos=OK_PTR + 2, freq=OK_PTR), EINVAL), (dict(rot_pairs=2), EINVAL),
    (dict(qw=OK_PTR), EINVAL), (dict(kw=OK_PTR, norm=pace.PACE_NORM_NONE), EINVAL),
    (dict(q=None), EINVAL), (dict(ko=None), EINVAL), (dict(q=OK_PTR + 1), EINVAL), (dict(qo=OK_PTR * 2 + 1), EINVAL),
    (dict(q_stride=127), EINVAL), (dict(k_stride=63), EINVAL), (dict(qo=OK_PTR, q_stride=130), EINVAL),
    (dict(tokens=1 << 40), EUNSUPPORTED),
])
def test_norm_refusals(kw, want):
    assert norm_call(**kw) == want


def test_norm_of_nothing():
    assert norm_call(tokens=0) == pace.PACE_OK
    assert norm_call(heads_q=0, heads_k=0, q=None, k=None, qo=None, ko=None) == pace.PACE_OK
    assert status("pace_qk_norm_rope", None, *[OK_PTR] * 8, None) == EINVAL


def linear_call(B=2, H=2, dk=128, dv=128, T=1, dt=pace.PACE_DTYPE_BF16, q=OK_PTR, k=OK_PTR, v=OK_PTR, decay=OK_PTR,
                lens=None, scale=1.0, si=None, so=OK_PTR, out=OK_PTR, ws=None, n=0):
    return status("pace_linear_attn", B, H, dk, dv, T, dt, q, k, v, decay, lens, scale, si, so, out, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), EINVAL), (dict(H=-1), EINVAL), (dict(dk=96), EUNSUPPORTED), (dict(dv=24), EUNSUPPORTED),
    (dict(dv=272), EUNSUPPORTED), (dict(T=0), EINVAL), (dict(dt=5), EINVAL), (dict(q=None), EINVAL),
    (dict(k=OK_PTR + 8), EINVAL), (dict(v=None), EINVAL), (dict(decay=None), EINVAL), (dict(decay=OK_PTR + 2), EINVAL),
    (dict(lens=OK_PTR + 1), EINVAL), (dict(scale=math.nan), EINVAL), (dict(si=OK_PTR + 4), EINVAL),
    (dict(so=None), EINVAL), (dict(out=None), EINVAL), (dict(out=OK_PTR + 4), EINVAL),
    (dict(B=1 << 14, H=1 << 14, T=1 << 20), EUNSUPPORTED),
])
def test_linear_refusals(kw, want):
    assert linear_call(**kw) == want


def test_linear_workspace():
    n = ctypes.c_uint64()
    args = (1, 16, 128, 128, 16384, pace.PACE_DTYPE_BF16)
    assert status("pace_linear_attn_workspace", *args, None) == EINVAL
    assert status("pace_linear_attn_workspace", 1, 16, 100, 128, 16, 1, ctypes.byref(n)) == EUNSUPPORTED
    assert status("pace_linear_attn_workspace", *args, ctypes.byref(n)) == pace.PACE_OK
    if n.value:
        long = dict(B=1, H=16, T=16384)
        assert linear_call(**long) == EINVAL and "workspace" in pace.pace_last_error()
        assert linear_call(**long, ws=OK_PTR, n=n.value - 1) == EINVAL
        assert linear_call(**long, ws=OK_PTR + 8, n=n.value) == EINVAL
    assert pace.pace_linear_attn_workspace(8, 16, 128, 128, 1, pace.PACE_DTYPE_BF16) == 0


def kv4_config(**kw):
    c = dict(batch=2, heads_q=4, heads_kv=2, d=128, page_tokens=64, n_pages=8, max_pages=4,
             in_dtype=pace.PACE_DTYPE_BF16)
    c.update(kw)
    return pace.pace_kv4_config(**c)


BAD_KV4 = [
    (dict(batch=0), EINVAL), (dict(heads_kv=0), EINVAL), (dict(d=96), EUNSUPPORTED), (dict(page_tokens=16), EUNSUPPORTED),
    (dict(page_tokens=100), EUNSUPPORTED), (dict(page_tokens=2048), EUNSUPPORTED), (dict(n_pages=0), EINVAL),
    (dict(max_pages=0), EINVAL), (dict(in_dtype=9), EINVAL), (dict(max_pages=1 << 26, page_tokens=64), EUNSUPPORTED),
    (dict(batch=1 << 20, heads_kv=1 << 12), EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", BAD_KV4)
def test_cache_config_refusals(kw, want):
    c = ctypes.byref(kv4_config(**{**kw, "heads_q": 2 * kw.get("heads_kv", 2) or 2}))
    n = ctypes.c_uint64()
    T = 64
    assert status("pace_kv4_append", c, OK_PTR, OK_PTR, OK_PTR, None, T, OK_PTR, OK_PTR, None) == want
    assert status("pace_kv4_read", c, OK_PTR, OK_PTR, OK_PTR, None, T, OK_PTR, OK_PTR, None) == want
    assert status("pace_kv4_attention", c, OK_PTR, OK_PTR, OK_PTR, None, T, OK_PTR, 1.0, 0, 0, OK_PTR, OK_PTR,
                  1 << 50, None) == want
    assert status("pace_kv4_attention_workspace", c, T, ctypes.byref(n)) == want


def test_cache_refusals():
    c = ctypes.byref(kv4_config())
    n = ctypes.c_uint64()
    assert status("pace_kv4_pool_bytes", None, ctypes.byref(n)) == EINVAL
    assert status("pace_kv4_pool_bytes", c, None) == EINVAL
    assert status("pace_kv4_pool_bytes", c, ctypes.byref(n)) == pace.PACE_OK
    assert n.value == 8 * 2 * 64 * (128 + 16)
    big = ctypes.byref(kv4_config(n_pages=2 ** 31 - 1, heads_kv=64, page_tokens=1024, d=256))
    assert status("pace_kv4_pool_bytes", big, ctypes.byref(n)) == pace.PACE_OK
    assert n.value == (2 ** 31 - 1) * 64 * 1024 * 288
    a = [c, OK_PTR, OK_PTR, OK_PTR, None, 3, OK_PTR, OK_PTR, None]
    for i, bad in ((0, None), (1, None), (1, OK_PTR + 8), (2, None), (2, OK_PTR + 2), (3, None), (4, OK_PTR + 1),
                   (5, 0), (5, -7), (6, None), (6, OK_PTR + 4), (7, None)):
        assert status("pace_kv4_append", *a[:i], bad, *a[i + 1:]) == EINVAL, i
        if i < 6:
            assert status("pace_kv4_read", *a[:i], bad, *a[i + 1:]) == EINVAL, i
    assert status("pace_kv4_read", *a[:6], OK_PTR + 4, None, None) == EINVAL
    assert status("pace_kv4_read", *a[:6], None, None, None) == pace.PACE_OK
    a = [c, OK_PTR, OK_PTR, OK_PTR, None, 3, OK_PTR, 1.0, 0, 0, OK_PTR, OK_PTR, 1 << 50, None]
    for i, bad in ((0, None), (1, None), (2, None), (3, None), (4, OK_PTR + 1), (5, 0), (5, -1), (6, None),
                   (6, OK_PTR + 8), (7, math.nan), (7, math.inf), (8, -1), (9, -1), (10, None), (10, OK_PTR + 2)):
        assert status("pace_kv4_attention", *a[:i], bad, *a[i + 1:]) == EINVAL, i
    for heads in (0, 3, -2):
        assert status("pace_kv4_attention", ctypes.byref(kv4_config(heads_q=heads)), *a[1:]) == EINVAL
    assert status("pace_kv4_attention_workspace", c, 3, None) == EINVAL
    assert status("pace_kv4_attention_workspace", c, 0, ctypes.byref(n)) == EINVAL
    assert status("pace_kv4_attention_workspace", c, 1, ctypes.byref(n)) == pace.PACE_OK
    if n.value:
        assert status("pace_kv4_attention", *a[:5], 1, *a[6:11], None, 0, None) == EINVAL
        assert "workspace" in pace.pace_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is present")
def test_no_device():
    assert norm_call() == pace.PACE_EDEVICE
    assert linear_call() == pace.PACE_EDEVICE
    c = ctypes.byref(kv4_config())
    assert status("pace_kv4_append", c, OK_PTR, OK_PTR, OK_PTR, None, 3, OK_PTR, OK_PTR, None) == pace.PACE_EDEVICE


def test_host_tensors_are_refused():
    x = torch.zeros((2, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        layers.qk_norm_rope(x, x)
    y = torch.zeros((1, 2, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        layers.linear_attention(y, y, y, torch.zeros(2))
    cache = layers.Kv4Cache(2, 2, 64, 32, device="cpu")
    table = torch.zeros((2, 1), dtype=torch.int32)
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        cache.append(y, y, table, n)
    with pytest.raises(ValueError, match="GPU"):
        cache.read(table, n, 1)
    with pytest.raises(ValueError, match="GPU"):
        cache.attention(y, table, n)
    with pytest.raises(TypeError):
        layers.qk_norm_rope([1.0])
    with pytest.raises(pace.PaceError):
        layers.Kv4Cache(2, 2, 100, 32, device="cpu")
