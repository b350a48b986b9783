"""The 8-bit latent cache on the host (no GPU): the ctypes mirrors, the library's
refusals of bad arguments before anything is launched, the sizes it reports, and the
Python binding's own checks."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import differential_latent_attention_gdla_b200 as gdla
from differential_latent_attention_gdla_b200 import _abi, build
from test_abi import _c_layout

E, U = _abi.GDLA_ERR_INVALID_ARG, _abi.GDLA_ERR_UNSUPPORTED
BASE = 0x10000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        build.build()
    return _abi.load()


@pytest.mark.parametrize("cls,cname", [(_abi.QcacheWriteArgs, "gdla_qcache_write_args"),
                                       (_abi.QcacheReadArgs, "gdla_qcache_read_args"),
                                       (_abi.QcacheDecodeArgs, "gdla_qcache_decode_args")])
def test_ctypes_mirror_matches_c_layout(cls, cname):
    fields = [f[0] for f in cls._fields_]
    assert [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields] == _c_layout(cname, fields)


def pointers(a, names):
    for i, f in enumerate(names):
        setattr(a, f, BASE + i * 0x1000000)
    return a


def good_write():
    a = _abi.QcacheWriteArgs(2, 10, 100, 512, 64, 16, _abi.GDLA_BF16, 0.0, 100)
    pointers(a, ("c_kv", "gamma", "k_rope", "rope_cos", "rope_sin", "start", "lens", "c_cache", "kr_cache", "scales",
                 "workspace"))
    a.workspace_bytes = 256
    return a


def good_read():
    a = _abi.QcacheReadArgs(2, 50, 100, 50, 512, 64, 16, 16, 128, 128, _abi.GDLA_BF16)
    return pointers(a, ("c_cache", "kr_cache", "scales", "lens", "w_ukv", "c_hat_out", "k_rope_out", "kv_out"))


def good_decode():
    a = _abi.QcacheDecodeArgs(4, 1000, 512, 64, 16, 128, 128, 16, 2, 64, _abi.GDLA_MASK_CAUSAL, 0, 0.0,
                              _abi.GDLA_BF16, 1000)
    pointers(a, ("seqlens", "c_cache", "kr_cache", "scales", "q", "w_ukv", "rope_cos", "rope_sin", "lam_logits",
                 "gate_logits", "out", "workspace"))
    a.workspace_bytes = _abi.load().gdla_qcache_decode_workspace_size(ctypes.byref(a))
    return a


def sets(**kw):
    def mut(a):
        for k, v in kw.items():
            if hasattr(a, k):
                setattr(a, k, v)
    return mut


DIMS = [(sets(T_max=0x7FFFFFFF, rope_max_pos=0x7FFFFFFF), U), (sets(B=0), E), (sets(B=65536), E), (sets(T_max=0), E), (sets(scale_block=0), E), (sets(scale_block=3), E),
        (sets(scale_block=256), E), (sets(scale_block=-1), E), (sets(dtype=2), E), (sets(d_c=500), U),
        (sets(d_rope=48), U), (sets(c_cache=0), E), (sets(kr_cache=BASE + 8), E), (sets(scales=BASE + 4), E)]


@pytest.mark.parametrize("mut,want", DIMS + [
    (sets(L=0), E), (sets(L=101), E), (sets(c_kv=0), E), (sets(k_rope=BASE + 2), E), (sets(gamma=BASE + 2), E),
    (sets(rope_cos=0), E), (sets(rope_max_pos=99), E), (sets(start=BASE + 2), E), (sets(lens=BASE + 1), E),
    (sets(workspace=0), E), (sets(workspace=BASE + 16), E), (sets(workspace_bytes=255), E)])
def test_write_rejects_before_launch(lib, mut, want):
    a = good_write()
    mut(a)
    assert lib.gdla_qcache_write(ctypes.byref(a), None) == want
    assert lib.gdla_qcache_write(None, None) == E


@pytest.mark.parametrize("mut,want", DIMS + [
    (sets(L=0), E), (sets(first=-1), E), (sets(L=51), E), (sets(first=0x7FFFFFFF), E), (sets(lens=BASE + 2), E),
    (sets(c_hat_out=0), E), (sets(k_rope_out=BASE + 8), E)])
def test_read_and_expand_reject_before_launch(lib, mut, want):
    for fn in (lib.gdla_qcache_read, lib.gdla_qcache_expand):
        a = good_read()
        mut(a)
        assert fn(ctypes.byref(a), None) == want
        assert fn(None, None) == E


@pytest.mark.parametrize("mut,want", [(sets(n_kv=0), E), (sets(w_ukv=0), E), (sets(kv_out=BASE + 8), E),
                                      (sets(d_nope=64), U), (sets(d_v=96), U)])
def test_expand_rejects_before_launch(lib, mut, want):
    a = good_read()
    mut(a)
    assert lib.gdla_qcache_expand(ctypes.byref(a), None) == want


@pytest.mark.parametrize("mut,want", DIMS + [
    (sets(n_kv=0), E), (sets(g=0), E), (sets(g=9), U), (sets(n_noise=4), U), (sets(d_nope=64), U),
    # the CUDA-core decode (fp32) holds at most 64 heads per block
    (sets(g=4, dtype=_abi.GDLA_FP32), U),
    (sets(mask=7), E), (sets(mask=1, window=0), E), (sets(rope_max_pos=999), E), (sets(seqlens=0), E),
    (sets(q=BASE + 8), E), (sets(out=0), E), (sets(workspace=BASE + 16), E), (sets(workspace_bytes=1024), E)])
def test_decode_rejects_before_launch(lib, mut, want):
    a = good_decode()
    mut(a)
    assert lib.gdla_qcache_decode(ctypes.byref(a), None) == want
    assert lib.gdla_qcache_decode(None, None) == E


def test_sizes(lib):
    assert lib.gdla_qcache_scale_blocks(100, 1) == 100
    assert lib.gdla_qcache_scale_blocks(100, 64) == 2
    assert lib.gdla_qcache_scale_blocks(128, 64) == 2
    assert lib.gdla_qcache_scale_blocks(2147483647, 128) == 16777216
    for T, sb in ((0, 1), (10, 0), (10, 3), (10, 256)):
        assert lib.gdla_qcache_scale_blocks(T, sb) == 0
    # one partial of every share and sequence, and the query images
    a = good_decode()
    n = lib.gdla_qcache_decode_workspace_size(ctypes.byref(a))
    assert n > 4 * 48 * 576 * 2 + 4 * 48 * 512 * 4
    a.workspace_bytes = n - 1
    assert lib.gdla_qcache_decode(ctypes.byref(a), None) == E
    assert lib.gdla_qcache_decode_workspace_size(None) == 0


@pytest.mark.parametrize("n_kv,g", [(1, 1), (16, 2), (16, 4), (16, 5), (3, 8), (48, 1), (49, 1), (512, 8), (65535, 8)])
def test_every_head_has_a_place_in_the_workspace(lib, n_kv, g):
    # images of 48 heads each, enough of them for the heads and no group empty
    a = good_decode()
    a.n_kv = a.n_noise = n_kv
    a.g, a.B, a.T_max = g, 1, 128
    heads = n_kv * (g + 1)
    n = lib.gdla_qcache_decode_workspace_size(ctypes.byref(a))
    assert n >= heads * (2 * 576 + 2 * 512 * 4)
    assert n <= 4096 + (heads + 48 + heads // 24) * (2 * 576 + 260 + 2 * 514 * 4)


def test_no_workspace_for_heads_that_overflow():
    # (in a process of its own: a division by n_kv (g + 1) = 2^32 heads ends it)
    code = """
import ctypes
from differential_latent_attention_gdla_b200 import _abi
for n_kv, g in ((1 << 30, 3), (1 << 29, 7), (65536, 1), (16, 9), (16, 0x7FFFFFFF)):
    for dtype, d_c in ((0, 512), (1, 512), (0, 64)):
        a = _abi.QcacheDecodeArgs(1, 100, d_c, 64, n_kv, 128, 128, n_kv, g, 1)
        a.dtype = dtype
        assert _abi.load().gdla_qcache_decode_workspace_size(ctypes.byref(a)) == 0
"""
    assert subprocess.run([sys.executable, "-c", code], cwd=build.ROOT).returncode == 0


def test_binding_rejects_before_the_library():
    c8, kr8, sc = gdla.qcache_empty(2, 100, d_c=64, d_rope=16, scale_block=16, device="cpu")
    assert c8.shape == (2, 100, 64) and kr8.shape == (2, 100, 16) and sc.shape == (2, 7)
    c = torch.zeros((2, 10, 64))
    k = torch.zeros((2, 10, 16))
    with pytest.raises(ValueError, match="CUDA device tensors"):
        gdla.qcache_write(c8, kr8, sc, c, k, scale_block=16)
    with pytest.raises(ValueError, match="scales"):
        gdla.qcache_write(c8, kr8, sc, c, k, scale_block=8)
    with pytest.raises(ValueError, match="power of two"):
        gdla.qcache_write(c8, kr8, sc, c, k, scale_block=7)
    with pytest.raises(ValueError, match="k_rope"):
        gdla.qcache_write(c8, kr8, sc, c, k[:, :9], scale_block=16)
    with pytest.raises(ValueError, match="k_rope"):
        gdla.qcache_write(c8, kr8, sc, c, k.bfloat16(), scale_block=16)
    with pytest.raises(ValueError, match="rotation"):
        gdla.qcache_write(c8, kr8, sc, c, k, gamma=torch.ones(64), scale_block=16)
    with pytest.raises(ValueError, match="start"):
        gdla.qcache_write(c8, kr8, sc, c, k, start=torch.zeros(2, dtype=torch.int64), scale_block=16)
    with pytest.raises(ValueError, match="8-bit cache"):
        gdla.qcache_read(c8.float(), kr8, sc, length=10, scale_block=16)
    with pytest.raises(ValueError, match="dtype"):
        gdla.qcache_read(c8, kr8, sc, length=10, scale_block=16, dtype=torch.float16)
    with pytest.raises(ValueError, match="T_max"):
        gdla.qcache_read(c8, kr8[:, :99], sc, length=10, scale_block=16)
    with pytest.raises(ValueError, match="w_ukv"):
        gdla.qcache_expand(c8, kr8, sc, torch.zeros((64, 100)), n_kv=4, d_nope=32, d_v=32, length=10, scale_block=16)
    q = torch.zeros((2, 6, 48))
    tab = torch.zeros((100, 8))
    args = dict(w_ukv=torch.zeros((64, 2 * 64)), rope_cos=tab, rope_sin=tab, lam_logits=torch.zeros((2, 4)),
                gate_logits=torch.zeros((2, 4, 32)), seqlens=torch.ones(2, dtype=torch.int32))
    for bad, match in (({"seqlens": torch.ones(2)}, "seqlens"), ({"lam_logits": torch.zeros((2, 3))}, "lam_logits"),
                       ({"gate_logits": torch.zeros((2, 4, 16))}, "gate_logits"), ({"rope_sin": tab[:50]}, "rope_sin"),
                       ({}, "CUDA device tensors")):
        with pytest.raises(ValueError, match=match):
            gdla.qcache_decode(c8, kr8, sc, q, **{**args, **bad}, g=2, scale_block=16)
    with pytest.raises(ValueError, match="noise heads"):
        gdla.qcache_decode(c8, kr8, sc, q, **args, g=4, scale_block=16)


@pytest.mark.parametrize("g,heads", [(0, 6), (-1, 6), (-2, 6), (6, 6), (2, 0)])
def test_binding_rejects_head_counts(g, heads):
    # (g = -1: no division by g + 1 = 0)
    c8, kr8, sc = gdla.qcache_empty(2, 100, d_c=64, d_rope=16, scale_block=16, device="cpu")
    tab = torch.zeros((100, 8))
    with pytest.raises(ValueError, match="noise heads"):
        gdla.qcache_decode(c8, kr8, sc, torch.zeros((2, heads, 48)), torch.zeros((64, 128)), tab, tab, torch.zeros((2, 4)),
                           torch.zeros((2, 4, 32)), torch.ones(2, dtype=torch.int32), g=g, scale_block=16)
