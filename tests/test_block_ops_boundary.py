"""Boundary of the transformer-block operators, without a GPU: struct layouts against the header,
every refusal before any CUDA call, workspace sizes, empty problems."""
import ctypes
import os

import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tile_gather_comm_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned address that is never dereferenced
E = _lib
CLASSES = [(_lib.LinearArgs, "tgc_linear_args"), (_lib.LinearBwdArgs, "tgc_linear_bwd_args"),
           (_lib.BlockNormArgs, "tgc_block_norm_args"), (_lib.BlockNormBwdArgs, "tgc_block_norm_bwd_args")]


@pytest.mark.parametrize("cls,cname", CLASSES)
def test_ctypes_structs_match_the_header(cls, cname, tmp_path):
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    inc = "/usr/local/cuda/include"
    if gcc is None or not os.path.exists(os.path.join(inc, "cuda_runtime_api.h")):
        pytest.skip("gcc or the CUDA headers are not available")
    names = [f[0] for f in cls._fields_]
    body = [f'printf("%zu\\n", sizeof({cname}));']
    body += [f'printf("%zu\\n", offsetof({cname}, {n}));' for n in names]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tgc.h"\nint main(void) {\n' + "\n".join(body)
                   + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), "-I", inc, str(src), "-o", str(exe)],
                   check=True)
    out = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert out[0] == ctypes.sizeof(cls)
    assert out[1:] == [getattr(cls, n).offset for n in names]


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "tgc.h"), encoding="utf-8").read()
    assert f"#define TGC_MAX_GROUPS {_lib.MAX_GROUPS}" in text
    assert f"#define TGC_NORM_MAX_D {_lib.NORM_MAX_D}" in text
    for name, v in _lib.ACTS.items():
        assert f"TGC_ACT_{name.upper()} = {v}" in text
    for name, v in _lib.NORMS.items():
        assert f"TGC_NORM_{name.upper()} = {v}" in text


def _linear(**kw):
    d = dict(x=FAKE, w=FAKE, y=FAKE, M=16, K=64, N=32, dtype=3)
    d.update(kw)
    return _lib.lib().tgc_linear(ctypes.byref(_lib.LinearArgs(**d)))


def _linear_bwd(**kw):
    d = dict(dy=FAKE, x=FAKE, w=FAKE, z=FAKE, dx=FAKE, dw=FAKE, dbias=FAKE, M=16, K=64, N=32, dtype=2, act=2,
             workspace=FAKE, workspace_bytes=1 << 30)
    d.update(kw)
    return _lib.lib().tgc_linear_bwd(ctypes.byref(_lib.LinearBwdArgs(**d)))


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), E.TGC_ERR_INVALID_ARG), (dict(w=None), E.TGC_ERR_INVALID_ARG), (dict(y=None), E.TGC_ERR_INVALID_ARG),
    (dict(M=-1), E.TGC_ERR_INVALID_ARG), (dict(K=0), E.TGC_ERR_INVALID_ARG), (dict(M=1 << 31), E.TGC_ERR_INVALID_ARG),
    (dict(dtype=5), E.TGC_ERR_DTYPE), (dict(dtype=99), E.TGC_ERR_DTYPE), (dict(act=5), E.TGC_ERR_INVALID_ARG),
    (dict(act=-1), E.TGC_ERR_INVALID_ARG), (dict(K=60), E.TGC_ERR_ALIGN), (dict(N=33), E.TGC_ERR_ALIGN),
    (dict(x=FAKE + 2), E.TGC_ERR_ALIGN), (dict(bias=FAKE + 8), E.TGC_ERR_ALIGN), (dict(z=FAKE + 8), E.TGC_ERR_ALIGN),
    (dict(residual=FAKE + 8), E.TGC_ERR_ALIGN), (dict(ldx=63), E.TGC_ERR_INVALID_ARG), (dict(ldy=36), E.TGC_ERR_ALIGN),
    (dict(residual=FAKE, ldres=64), E.TGC_ERR_INVALID_ARG),  # in place with another stride
    (dict(ngroups=2), E.TGC_ERR_INVALID_ARG), (dict(offsets=FAKE), E.TGC_ERR_INVALID_ARG),
    (dict(offsets=FAKE, ngroups=1025), E.TGC_ERR_INVALID_ARG), (dict(offsets=FAKE + 2, ngroups=2), E.TGC_ERR_ALIGN),
    (dict(offsets=FAKE, ngroups=2, w_stride=64 * 8), E.TGC_ERR_INVALID_ARG),
    (dict(offsets=FAKE, ngroups=2, w_stride=64 * 32 + 4), E.TGC_ERR_ALIGN),
    (dict(offsets=FAKE, ngroups=1024, N=1 << 21), E.TGC_ERR_INVALID_ARG),
    (dict(ldx=1 << 39), E.TGC_ERR_INVALID_ARG),
    (dict(M=0), E.TGC_OK), (dict(N=0), E.TGC_OK),
])
def test_linear_refusals(kw, rc):
    assert _linear(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dy=None), E.TGC_ERR_INVALID_ARG), (dict(z=None), E.TGC_ERR_INVALID_ARG), (dict(x=None), E.TGC_ERR_INVALID_ARG),
    (dict(w=None), E.TGC_ERR_INVALID_ARG), (dict(N=0), E.TGC_ERR_INVALID_ARG), (dict(K=0), E.TGC_ERR_INVALID_ARG),
    (dict(dtype=7), E.TGC_ERR_DTYPE), (dict(act=9), E.TGC_ERR_INVALID_ARG), (dict(K=12), E.TGC_ERR_ALIGN),
    (dict(dw=FAKE + 8), E.TGC_ERR_ALIGN), (dict(dx=FAKE + 8), E.TGC_ERR_ALIGN), (dict(dbias=FAKE + 4), E.TGC_ERR_ALIGN),
    (dict(lddy=24), E.TGC_ERR_INVALID_ARG), (dict(ngroups=3), E.TGC_ERR_INVALID_ARG),
    (dict(workspace=None), E.TGC_ERR_WORKSPACE), (dict(workspace_bytes=64), E.TGC_ERR_WORKSPACE),
    (dict(workspace=FAKE + 64), E.TGC_ERR_ALIGN),
])
def test_linear_bwd_refusals(kw, rc):
    assert _linear_bwd(**kw) == rc


def test_linear_bwd_workspace():
    def need(**kw):
        d = dict(dy=FAKE, x=FAKE, w=FAKE, z=FAKE, dx=FAKE, dw=FAKE, dbias=FAKE, M=100, K=64, N=32, dtype=3, act=2)
        d.update(kw)
        return _lib.lib().tgc_linear_bwd_workspace_bytes(ctypes.byref(_lib.LinearBwdArgs(**d)))
    assert need() >= 100 * 32 * 2 + 2 * 32 * 4
    assert need(dbias=None) < need()
    assert need(M=0) == 0 and need(K=5) == 0  # nothing to do; refused
    assert need(M=1000) > need()


def _norm(**kw):
    d = dict(y=FAKE, x=FAKE, r=FAKE, h=FAKE, M=4, D=8, post=1, pre=1, eps=1e-5, dtype=3, res_scale=1, branch_scale=1)
    d.update(kw)
    return _lib.lib().tgc_block_norm(ctypes.byref(_lib.BlockNormArgs(**d)))


def _norm_bwd(**kw):
    d = dict(y=FAKE, r=FAKE, dr=FAKE, dh=FAKE, dx=FAKE, dy=FAKE, dpre_weight=FAKE, M=4, D=8, post=1, pre=1, eps=1e-5,
             dtype=5, res_scale=1, branch_scale=1, workspace=FAKE, workspace_bytes=1 << 30)
    d.update(kw)
    return _lib.lib().tgc_block_norm_bwd(ctypes.byref(_lib.BlockNormBwdArgs(**d)))


@pytest.mark.parametrize("kw,rc", [
    (dict(y=None), E.TGC_ERR_INVALID_ARG), (dict(h=None), E.TGC_ERR_INVALID_ARG), (dict(pre=0), E.TGC_ERR_INVALID_ARG),
    (dict(pre=0, h=None, r=None), E.TGC_ERR_INVALID_ARG), (dict(D=0), E.TGC_ERR_INVALID_ARG),
    (dict(D=16385), E.TGC_ERR_INVALID_ARG), (dict(M=-1), E.TGC_ERR_INVALID_ARG), (dict(dtype=4), E.TGC_ERR_DTYPE),
    (dict(post=3), E.TGC_ERR_INVALID_ARG), (dict(gates=2), E.TGC_ERR_INVALID_ARG),
    (dict(gate=FAKE, gates=3), E.TGC_ERR_INVALID_ARG), (dict(gate=FAKE), E.TGC_ERR_INVALID_ARG),
    (dict(post=0, post_weight=FAKE), E.TGC_ERR_INVALID_ARG), (dict(pre=0, h=None, pre_bias=FAKE), E.TGC_ERR_INVALID_ARG),
    (dict(eps=0.0), E.TGC_ERR_INVALID_ARG), (dict(eps=float("nan")), E.TGC_ERR_INVALID_ARG),
    (dict(y=FAKE + 1), E.TGC_ERR_ALIGN), (dict(pre_weight=FAKE + 1), E.TGC_ERR_ALIGN), (dict(ldx=7), E.TGC_ERR_INVALID_ARG),
    (dict(M=0), E.TGC_OK),
])
def test_block_norm_refusals(kw, rc):
    assert _norm(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(y=None), E.TGC_ERR_INVALID_ARG), (dict(r=None), E.TGC_ERR_INVALID_ARG), (dict(dh=None), E.TGC_ERR_INVALID_ARG),
    (dict(dgate=FAKE), E.TGC_ERR_INVALID_ARG), (dict(gates=2), E.TGC_ERR_INVALID_ARG),
    (dict(post=0, dpost_weight=FAKE), E.TGC_ERR_INVALID_ARG), (dict(pre=0, dh=None), E.TGC_ERR_INVALID_ARG),
    (dict(dtype=0), E.TGC_ERR_DTYPE), (dict(eps=-1.0), E.TGC_ERR_INVALID_ARG), (dict(D=20000), E.TGC_ERR_INVALID_ARG),
    (dict(dx=FAKE + 2), E.TGC_ERR_ALIGN), (dict(lddh=3), E.TGC_ERR_INVALID_ARG),
    (dict(workspace=None), E.TGC_ERR_WORKSPACE), (dict(workspace_bytes=16), E.TGC_ERR_WORKSPACE),
    (dict(workspace=FAKE + 4), E.TGC_ERR_ALIGN),
])
def test_block_norm_bwd_refusals(kw, rc):
    assert _norm_bwd(**kw) == rc


def test_null_arguments():
    L = _lib.lib()
    for f in (L.tgc_linear, L.tgc_linear_bwd, L.tgc_block_norm, L.tgc_block_norm_bwd):
        assert f(None) == E.TGC_ERR_INVALID_ARG
    assert L.tgc_linear_bwd_workspace_bytes(None) == 0 and L.tgc_block_norm_bwd_workspace_bytes(None) == 0


def test_the_binding_refuses_host_tensors():
    x, w, y = torch.zeros(2, 8), torch.zeros(8, 8), torch.zeros(2, 8)
    with pytest.raises(ValueError):
        tgc.tgc_linear(x, w, y)
    with pytest.raises(ValueError):
        tgc.tgc_block_norm(x, y, y)
