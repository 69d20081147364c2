"""Boundary of the attention and cache operators, without a GPU: struct layouts against the header, every
refusal before any CUDA call, frequencies, empty problems."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tile_gather_comm_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned address that is never dereferenced
E = _lib
CLASSES = [(_lib.RopeArgs, "tgc_rope_args"), (_lib.KvAppendArgs, "tgc_kv_append_args"),
           (_lib.PagedAttentionArgs, "tgc_paged_attention_args"), (_lib.KvArgs, "tgc_kv_args")]


@pytest.mark.parametrize("cls,cname", CLASSES)
def test_ctypes_structs_match_the_header(cls, cname, tmp_path):
    gcc = shutil.which("gcc")
    inc = "/usr/local/cuda/include"
    if gcc is None or not os.path.exists(os.path.join(inc, "cuda_runtime_api.h")):
        pytest.skip("gcc or the CUDA headers are not available")
    names = [f[0] for f in cls._fields_]
    body = [f'printf("%zu\\n", sizeof({cname}));']
    body += [f'printf("%zu\\n", offsetof({cname}, {n.rstrip("_")}));' for n in names]
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
    for name in ("ROPE_MAX_D", "ROPE_MAX_HEADS", "ATTENTION_MAX_D", "ATTENTION_MAX_HEADS", "KV_MAX_POOLS"):
        assert f"#define TGC_{name} {getattr(_lib, name)}" in text
    for name, v in _lib.ROPE_LAYOUTS.items():
        assert f"TGC_ROPE_{name.upper()} = {v}" in text
    for name, v in _lib.ROPE_SCALINGS.items():
        assert f"TGC_ROPE_{name.upper()} = {v}" in text


INV, ALIGN, DTYPE, WS, OK = E.TGC_ERR_INVALID_ARG, E.TGC_ERR_ALIGN, E.TGC_ERR_DTYPE, E.TGC_ERR_WORKSPACE, E.TGC_OK


def _rope(back=False, **kw):
    d = dict(q=FAKE, k=FAKE, q_out=2 * FAKE, k_out=2 * FAKE, pos=FAKE, freqs=FAKE, T=4, heads_q=8, heads_k=2, D=64, R=64, dtype=3)
    d.update(kw)
    return (_lib.lib().tgc_rope_bwd if back else _lib.lib().tgc_rope)(ctypes.byref(_lib.RopeArgs(**d)))


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), INV), (dict(q_out=None), INV), (dict(k=None), INV), (dict(k_out=None), INV), (dict(pos=None), INV),
    (dict(freqs=None), INV), (dict(T=-1), INV), (dict(T=1 << 31), INV), (dict(heads_q=0, heads_k=0), INV),
    (dict(heads_q=-1), INV), (dict(heads_q=65536), INV), (dict(D=0), INV), (dict(D=1025), INV), (dict(R=66), INV),
    (dict(R=0), INV), (dict(R=31), INV), (dict(layout=2), INV), (dict(layout=-1), INV), (dict(scale=math.nan), INV),
    (dict(scale=math.inf), INV), (dict(dtype=7), DTYPE), (dict(dtype=4), DTYPE), (dict(q=FAKE + 1), ALIGN),
    (dict(k_out=FAKE + 1), ALIGN), (dict(pos=FAKE + 2), ALIGN), (dict(freqs=FAKE + 4), ALIGN), (dict(q_h=63), INV),
    (dict(q_t=40), INV), (dict(q_t=-64), INV), (dict(q_t=1 << 60), INV), (dict(q_out=FAKE, qo_t=1024), INV),
    (dict(k_out=FAKE, ko_h=128), INV), (dict(T=0), OK), (dict(T=0, pos=None, q=None), OK),
])
def test_rope_refusals(kw, rc, back):
    assert _rope(back, **kw) == rc


def _append(**kw):
    d = dict(k=FAKE, v=FAKE, q=FAKE, q_out=FAKE, k_pages=FAKE, v_pages=FAKE, table=FAKE, pos=FAKE, seqs=FAKE, freqs=FAKE,
             T=4, heads_q=8, heads_k=2, D=64, R=64, num_pages=9, page_size=16, num_seqs=3, max_pages=5, dtype=3)
    d.update(kw)
    return _lib.lib().tgc_kv_append(ctypes.byref(_lib.KvAppendArgs(**d)))


@pytest.mark.parametrize("kw,rc", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(q=None), INV), (dict(q_out=None), INV), (dict(k_pages=None), INV),
    (dict(v_pages=None), INV), (dict(table=None), INV), (dict(pos=None), INV), (dict(seqs=None), INV),  # 4 tokens, 3 sequences
    (dict(freqs=None), INV), (dict(freqs=None, R=0, T=0), OK), (dict(heads_k=0), INV), (dict(heads_k=40000), INV),
    (dict(D=1025, R=64), INV), (dict(R=65), INV), (dict(page_size=0), INV), (dict(num_pages=-1), INV),
    (dict(max_pages=-1), INV), (dict(page_size=1 << 20, max_pages=1 << 11), INV), (dict(num_seqs=1 << 20, max_pages=1 << 11), INV),
    (dict(table_ld=4), INV), (dict(token_s=63), INV), (dict(head_s=63), INV), (dict(page_s=1 << 58), INV),
    (dict(dtype=1), DTYPE), (dict(k_pages=FAKE + 1), ALIGN), (dict(seqs=FAKE + 1), ALIGN), (dict(table=FAKE + 2), ALIGN),
    (dict(v_t=100), INV), (dict(scale=math.nan), INV), (dict(layout=7), INV), (dict(T=0), OK),
])
def test_append_refusals(kw, rc):
    assert _append(**kw) == rc


def _attention(**kw):
    d = dict(q=FAKE, out=2 * FAKE, lse=FAKE, k_pages=FAKE, v_pages=FAKE, table=FAKE, lens=FAKE, num_seqs=3, heads_q=8,
             heads_k=2, D=64, num_pages=9, page_size=16, max_pages=5, dtype=3, workspace=FAKE, workspace_bytes=16)
    d.update(kw)
    return _lib.lib().tgc_paged_attention(ctypes.byref(_lib.PagedAttentionArgs(**d)))


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), INV), (dict(out=None), INV), (dict(lens=None), INV), (dict(table=None), INV), (dict(k_pages=None), INV),
    (dict(v_pages=None), INV), (dict(heads_q=0), INV), (dict(heads_k=0), INV), (dict(heads_k=3), INV), (dict(D=0), INV),
    (dict(D=264), INV), (dict(D=60), ALIGN), (dict(dtype=5), DTYPE), (dict(dtype=99), DTYPE), (dict(num_seqs=-1), INV),
    (dict(window=-1), INV), (dict(softcap=-1.0), INV), (dict(softcap=math.nan), INV), (dict(scale=math.inf), INV),
    (dict(page_size=0), INV), (dict(max_pages=1 << 28), INV), (dict(num_seqs=1 << 28, heads_q=16, max_pages=1), INV),
    (dict(q=FAKE + 8), ALIGN), (dict(v_pages=FAKE + 8), ALIGN), (dict(lse=FAKE + 2), ALIGN), (dict(lens=FAKE + 1), ALIGN),
    (dict(q_h=68), ALIGN), (dict(q_h=56), INV), (dict(token_s=132), ALIGN), (dict(page_s=56), INV),
    (dict(out=FAKE, o_s=1024), INV), (dict(table_ld=3), INV), (dict(num_seqs=0), OK),
])
def test_attention_refusals(kw, rc):
    assert _attention(**kw) == rc


def test_attention_refuses_more_heads_than_its_indices_hold():
    for heads in (65537, 1 << 26):  # times D / 2: past 32 bits
        assert _attention(heads_q=heads, heads_k=1, D=256, num_seqs=1) == INV


def test_attention_wants_a_table_for_an_empty_pool():
    """Lengths lead into the table whether or not its numbers can be pages."""
    assert _attention(num_pages=0, k_pages=None, v_pages=None, table=None) == INV


def _kv(name, **kw):
    pools = (ctypes.c_void_p * 2)(FAKE, 2 * FAKE)
    d = dict(refs=FAKE, table=FAKE, lens=FAKE, num_pages=9, page_size=16, num_seqs=3, max_pages=5, src=FAKE, dst=FAKE,
             add=FAKE, ok=FAKE, used=FAKE, n=2, pools=pools, from_=pools, npools=2, page_bytes=4096, from_pages=9,
             workspace=FAKE, workspace_bytes=1 << 20)
    d.update(kw)
    return getattr(_lib.lib(), "tgc_kv_" + name)(ctypes.byref(_lib.KvArgs(**d)))


BAD = (ctypes.c_void_p * 2)(FAKE, None)
ODD = (ctypes.c_void_p * 2)(FAKE, FAKE + 8)


@pytest.mark.parametrize("name,kw,rc", [
    ("copy", dict(src=None), INV), ("copy", dict(dst=None), INV), ("copy", dict(pools=None), INV), ("copy", dict(from_=None), INV),
    ("copy", dict(pools=BAD), INV), ("copy", dict(from_=ODD), ALIGN), ("copy", dict(page_bytes=24), ALIGN),
    ("copy", dict(page_bytes=0), INV), ("copy", dict(page_bytes=1 << 35), INV), ("copy", dict(npools=257), INV),
    ("copy", dict(npools=-1), INV), ("copy", dict(n=-1), INV), ("copy", dict(n=1 << 31), INV), ("copy", dict(from_pages=-1), INV),
    ("copy", dict(src=FAKE + 2), ALIGN), ("copy", dict(n=0), OK), ("copy", dict(npools=0), OK),
    ("reserve", dict(refs=None), INV), ("reserve", dict(table=None), INV), ("reserve", dict(lens=None), INV),
    ("reserve", dict(dst=None), INV), ("reserve", dict(add=None), INV), ("reserve", dict(page_size=0), INV),
    ("reserve", dict(num_pages=1 << 31), INV), ("reserve", dict(max_pages=1 << 28), INV), ("reserve", dict(table_ld=4), INV),
    ("reserve", dict(workspace=None), WS), ("reserve", dict(workspace_bytes=64), WS), ("reserve", dict(workspace=FAKE + 64), ALIGN),
    ("reserve", dict(ok=FAKE + 1), ALIGN), ("reserve", dict(n=0), OK),
    ("fork", dict(src=None), INV), ("fork", dict(lens=None), INV), ("fork", dict(pools=BAD), INV), ("fork", dict(pools=ODD), ALIGN),
    ("fork", dict(page_bytes=8), ALIGN), ("fork", dict(workspace_bytes=64), WS), ("fork", dict(n=0), OK),
    ("free", dict(dst=None), INV), ("free", dict(lens=None), INV), ("free", dict(refs=None), INV), ("free", dict(lens=FAKE + 1), ALIGN),
    ("free", dict(n=0), OK),
    ("compact", dict(refs=None), INV), ("compact", dict(pools=None), INV), ("compact", dict(used=FAKE + 2), ALIGN),
    ("compact", dict(workspace=None), WS), ("compact", dict(workspace_bytes=128), WS), ("compact", dict(num_pages=0, used=None), OK),
])
def test_cache_refusals(name, kw, rc):
    assert _kv(name, **kw) == rc


def test_null_arguments():
    L = _lib.lib()
    for f in ("rope", "rope_bwd", "kv_append", "paged_attention", "kv_copy", "kv_reserve", "kv_fork", "kv_free", "kv_compact"):
        assert getattr(L, "tgc_" + f)(None) == INV
    assert L.tgc_paged_attention_workspace_bytes(None) == 0 and L.tgc_kv_workspace_bytes(None) == 0


def test_cache_workspace():
    def need(**kw):
        d = dict(num_pages=9, page_size=16, num_seqs=3, max_pages=5, n=2)
        d.update(kw)
        return _lib.lib().tgc_kv_workspace_bytes(ctypes.byref(_lib.KvArgs(**d)))
    assert need() > 0 and need(n=1000) > need() and need(num_pages=100000) > need() and need(page_size=0) == 0


@pytest.mark.parametrize("R", [2, 4, 34, 128])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_frequencies(R, scaling):
    """Against the formulas; pow and its argument round in 64 bits: 2^-53 each on exponents up to ln(5e5) + ln 16 < 16."""
    base, factor, trained = 500000.0, 16.0, 8192.0
    got, scale = tgc.tgc_rope_freqs(R, base, scaling=scaling, factor=factor, trained=trained, device="cpu")
    assert got.dtype == torch.float64 and len(got) == R // 2
    assert scale == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0, rel=1e-15)
    for i, f in enumerate(got.tolist()):
        plain = base ** (-2 * i / R)
        want = plain
        if scaling == "linear":
            want = plain / factor
        if scaling == "ntk" and R > 2:
            want = (base * factor ** (R / (R - 2))) ** (-2 * i / R)
        if scaling == "yarn":
            ramp = min(1.0, max(0.0, (trained * plain / (2 * math.pi) - 1) / 31))
            want = ramp * plain + (1 - ramp) * plain / factor
        assert f == pytest.approx(want, rel=1e-13)
    if scaling == "ntk" and R > 2:  # what the base is chosen for
        assert got[0] == 1 and got[-1] * factor == pytest.approx(base ** (-(R - 2) / R), rel=1e-13)


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=1026), dict(base=1.0),
                                dict(base=math.inf), dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=2.0),
                                dict(scaling="yarn", factor=2.0, trained=4096.0, beta_fast=1.0),
                                dict(scaling="ntk", factor=math.nan)])
def test_frequency_refusals(kw):
    with pytest.raises(tgc.TGCError):
        tgc.tgc_rope_freqs(**{"rotary_dim": 64, "device": "cpu", **kw})


def test_the_binding_refuses_host_tensors():
    x, n = torch.zeros(2, 4, 8), torch.zeros(2, dtype=torch.int32)
    pages, table = torch.zeros(3, 4, 4, 8), torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: tgc.tgc_rope(x, x, n, torch.zeros(4, dtype=torch.float64)),
                 lambda: tgc.tgc_kv_append(x, x, pages, pages, table, n),
                 lambda: tgc.tgc_paged_attention(x, x, pages, pages, table, n),
                 lambda: tgc.tgc_kv_copy([pages], [pages], n, n),
                 lambda: tgc.tgc_kv_reserve(n, table, n, n, n, 4),
                 lambda: tgc.tgc_kv_fork([pages], n, table, n, n, n, 4),
                 lambda: tgc.tgc_kv_free(n, table, n, n), lambda: tgc.tgc_kv_compact([pages], n, table)):
        with pytest.raises(ValueError):
            call()
