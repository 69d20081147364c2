"""The attention and cache operators at the edges of what they accept, without a GPU: refusals before any CUDA call."""
import ctypes

import pytest

import tile_gather_comm_gb300 as tgc
from tile_gather_comm_gb300 import _lib

FAKE = 1 << 20  # an aligned address that is never dereferenced
INV, OK = _lib.TGC_ERR_INVALID_ARG, _lib.TGC_OK


def _attention(name="tgc_paged_attention", **kw):
    d = dict(q=FAKE, out=2 * FAKE, lse=FAKE, k_pages=FAKE, v_pages=FAKE, table=FAKE, lens=FAKE, num_seqs=3, heads_q=8,
             heads_k=2, D=64, num_pages=9, page_size=16, max_pages=5, dtype=3, workspace=FAKE, workspace_bytes=16)
    d.update(kw)
    return getattr(_lib.lib(), name)(ctypes.byref(_lib.PagedAttentionArgs(**d)))


@pytest.mark.parametrize("scale,softcap,rc", [
    (0.0, 3e38, INV), (0.125, 2.4e38, INV), (3e38, 0.0, INV), (-3e38, 0.0, INV),  # times log2(e): past fp32
    (0.0, 1e-40, INV), (8.0, 1e-39, INV), (1e30, 1e-9, INV),                      # scale / softcap past fp32
    (1e-3, 2e37, INV), (-1e-3, 2e37, INV), (1e-40, 1.0, INV),                     # and below its normal numbers
    (0.0, 0.0, OK), (2.35e38, 0.0, OK), (-2.35e38, 0.0, OK), (8.0, 2.3e38, OK), (0.125, 1e37, OK), (0.125, 1e-38, OK),
    (1e-40, 0.0, OK), (-0.5, 30.0, OK)])
def test_scales_and_caps_that_leave_fp32(scale, softcap, rc):
    """num_seqs = 0: what is accepted returns before any CUDA call."""
    assert _attention(scale=scale, softcap=softcap, num_seqs=0) == rc
    if rc == INV:
        assert _attention(scale=scale, softcap=softcap) == INV
        assert _attention("tgc_paged_attention_workspace_bytes", scale=scale, softcap=softcap) == 0


def _kv(name, **kw):
    d = dict(refs=FAKE, table=FAKE, lens=FAKE, num_pages=9, page_size=16, num_seqs=3, max_pages=5, src=FAKE, dst=FAKE,
             add=FAKE, ok=FAKE, used=FAKE, n=0, workspace=FAKE, workspace_bytes=1 << 20)
    d.update(kw)
    return getattr(_lib.lib(), "tgc_kv_" + name)(ctypes.byref(_lib.KvArgs(**d)))


@pytest.mark.parametrize("name,kw,rc", [
    ("fork", {}, OK), ("fork", dict(page_bytes=24), OK), ("fork", dict(page_bytes=-1), OK), ("compact", dict(num_pages=0, used=None), OK),
    ("copy", dict(n=2), OK), ("copy", dict(n=2, page_bytes=8), OK), ("fork", dict(npools=1), INV), ("fork", dict(npools=-1), INV),
    ("copy", dict(n=2, num_pages=-1), INV)])
def test_without_pools_their_fields_are_ignored(name, kw, rc):
    assert _kv(name, **kw) == rc


@pytest.mark.parametrize("name", ["reserve", "fork", "free", "compact"])
@pytest.mark.parametrize("kw", [dict(page_size=0), dict(num_pages=-1), dict(num_seqs=-1), dict(max_pages=-1), dict(table_ld=4)])
def test_every_call_on_a_cache_wants_its_sizes(name, kw):
    assert _kv(name, **kw) == INV


def test_a_base_stretched_past_64_bits_is_refused():
    """R = 4: factor^2 times the base."""
    with pytest.raises(tgc.TGCError):
        tgc.tgc_rope_freqs(4, 10000.0, scaling="ntk", factor=1e153, device="cpu")
    freqs, _ = tgc.tgc_rope_freqs(4, 10000.0, scaling="ntk", factor=1e150, device="cpu")
    assert freqs[0] == 1 and freqs[1] * 1e152 == pytest.approx(1.0, rel=1e-12)
    freqs, _ = tgc.tgc_rope_freqs(2, 10000.0, scaling="ntk", factor=1e300, device="cpu")
    assert freqs.tolist() == [1.0]
