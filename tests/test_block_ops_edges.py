"""The transformer-block operators at the edges of what they accept, without a GPU: index arithmetic for
offsets that decrease, compiled for the host from the kernels' own header; the largest sizes; a binding
that was built for another torch."""
import ctypes
import os
import subprocess

import pytest

from tile_gather_comm_gb300 import _build, _lib

CSRC = _build.CSRC
FAKE = 1 << 20  # an aligned address that is never dereferenced


def _run(tmp_path, body, headers):
    """Compiles a main() around `body` with nvcc and returns the whole numbers it prints."""
    src, exe = tmp_path / "edge.cu", tmp_path / "edge"
    src.write_text("#include <cstdio>\n#include <vector>\n" + "".join(f'#include "{h}"\n' for h in headers) +
                   "using namespace tgc;\nint main() {\n" + body + "\nreturn 0;\n}\n")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-I", CSRC, "-I", _build.INCLUDE, str(src), "-o", str(exe)],
                   check=True)
    return [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]


@pytest.mark.parametrize("M,groups", [(8192, 16), (300, 1024), ((1 << 31) - (1 << 16), 512)])
@pytest.mark.parametrize("offsets", ["e % 2 ? M : 0", "M - e", "e % 3 ? 0x7fffffff : -5", "(int)((long long)M * e / groups)"])
def test_the_bias_sum_stays_inside_its_partials(M, groups, offsets, tmp_path):
    """Groups of 64-row chunks, as many partials as M rows and the groups size: no group's chunks lie past them,
    and offsets that do not decrease lose none."""
    past, lost = _run(tmp_path, f"""
    const int M = {M}, groups = {groups}, kChunk = 64;
    std::vector<int32_t> off(groups + 1);
    for (int e = 0; e <= groups; ++e) off[e] = {offsets};
    const int64_t listed = ((int64_t)M + kChunk - 1) / kChunk + groups;
    int64_t first = 0, past = 0, lost = 0;
    for (int e = 0; e < groups; ++e) {{
        const RowRange g = group_range(off.data(), e, M);
        const int n = (g.end - g.begin + kChunk - 1) / kChunk, k = listed_tiles(first, n, listed);
        past += k < 0 || k > n || (k > 0 && first + k > listed);
        lost += n - k;
        first += n;
    }}
    printf("%lld %lld\\n", (long long)past, (long long)lost);""", ["groups.cuh"])
    assert past == 0
    assert lost >= 0 and (lost == 0 or "groups" not in offsets)


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("M,groups", [(8192, 16), (300, 1024), (65536, 1024), ((1 << 31) - (1 << 16), 1024)])
@pytest.mark.parametrize("offsets", ["e % 2 ? M : 0", "M - e", "(int)((long long)M * e / groups)"])
def test_the_tile_table_ends_where_its_list_does(tile, M, groups, offsets, tmp_path):
    """The products' table of tile rows, 32 groups at a time: places never decrease and never pass the list, and
    are the plain sums where offsets do not decrease."""
    wrong, cut = _run(tmp_path, f"""
    const int M = {M}, groups = {groups}, tile = {tile};
    std::vector<int32_t> off(groups + 1);
    for (int e = 0; e <= groups; ++e) off[e] = {offsets};
    const int listed = M / tile + (groups < M ? groups : M) + 1;
    int64_t sum = 0, wrong = 0, cut = 0;
    int base = 0, last = 0;
    for (int e0 = 0; e0 < groups; e0 += 32) {{
        int upto = 0;
        for (int e = e0; e < e0 + 32 && e < groups; ++e) {{
            const RowRange g = group_range(off.data(), e, M);
            const int at = listed_place(base, upto, listed), n = (g.end - g.begin + tile - 1) / tile;
            wrong += at < last || at > listed || at > sum;
            cut += at < sum;
            last = at;
            upto += n;
            sum += n;
        }}
        base = listed_place(base, upto, listed);
    }}
    wrong += base < last || base > listed;
    printf("%lld %lld\\n", (long long)wrong, (long long)(cut + (base < sum)));""", ["groups.cuh"])
    assert wrong == 0
    assert cut == 0 or "groups" not in offsets


@pytest.mark.parametrize("name", ["M", "K", "N"])
@pytest.mark.parametrize("past", [8, 2048, 4096 - 8])
def test_sizes_a_tile_short_of_32_bits_are_refused(name, past):
    """Between the limit and 2^31 a tile's end leaves 32 bits; 8 is the smallest step of K and N."""
    L, size = _lib.lib(), {"M": 8, "K": 8, "N": 8, name: _lib.MAX_SIZE + past}
    assert f"#define TGC_MAX_SIZE {_lib.MAX_SIZE}\n" in open(os.path.join(_build.INCLUDE, "tgc.h")).read()
    fwd = _lib.LinearArgs(x=FAKE, w=FAKE, y=FAKE, dtype=3, **size)
    assert L.tgc_linear(ctypes.byref(fwd)) == _lib.TGC_ERR_INVALID_ARG
    bwd = dict(dy=FAKE, x=FAKE, w=FAKE, dx=FAKE, dw=FAKE, dbias=FAKE, dtype=3, workspace=FAKE, workspace_bytes=1 << 60)
    assert L.tgc_linear_bwd(ctypes.byref(_lib.LinearBwdArgs(**bwd, **size))) == _lib.TGC_ERR_INVALID_ARG
    query = L.tgc_linear_bwd_workspace_bytes
    assert query(ctypes.byref(_lib.LinearBwdArgs(**bwd, **size))) == 0
    size[name] = _lib.MAX_SIZE  # accepted
    assert query(ctypes.byref(_lib.LinearBwdArgs(**bwd, **size))) >= 4 * size["N"]


@pytest.mark.parametrize("past", [1, 3000, 4095])
def test_norm_rows_a_block_short_of_32_bits_are_refused(past):
    L, M = _lib.lib(), _lib.MAX_SIZE + past
    kw = dict(M=M, D=1, pre=1, eps=1e-5, dtype=3, res_scale=1, branch_scale=1)
    assert L.tgc_block_norm(ctypes.byref(_lib.BlockNormArgs(y=FAKE, h=FAKE, **kw))) == _lib.TGC_ERR_INVALID_ARG
    bwd = _lib.BlockNormBwdArgs(r=FAKE, dh=FAKE, dy=FAKE, workspace=FAKE, workspace_bytes=1 << 60, **kw)
    assert L.tgc_block_norm_bwd(ctypes.byref(bwd)) == _lib.TGC_ERR_INVALID_ARG


@pytest.mark.parametrize("M", [2122219135, 2133429024, 2140000000, _lib.MAX_SIZE])
@pytest.mark.parametrize("D", [1, 8, 64])
def test_the_norm_gradients_deal_out_the_most_rows(M, D):
    """The partial sums go by the number of workers, which a million rows reach as well as any more do."""
    L = _lib.lib()

    def need(rows, **kw):
        a = _lib.BlockNormBwdArgs(r=FAKE, dh=FAKE, dy=FAKE, dpre_weight=FAKE, M=rows, D=D, pre=1, eps=1e-5, dtype=3,
                                  res_scale=1, branch_scale=1, **kw)
        return L.tgc_block_norm_bwd_workspace_bytes(ctypes.byref(a))
    assert 0 < need(M) <= need(1 << 20)
    one = dict(gate=FAKE, gates=1, y=FAKE, dgate=FAKE)
    assert need(M) < need(M, **one) <= need(1 << 20, **one)


@pytest.mark.parametrize("written,current", [(None, False), ("Python 3.12\\ntorch 1.0\\n", False), ("", False), (True, True)])
def test_a_binding_for_another_python_or_torch_is_out_of_date(written, current, tmp_path, monkeypatch):
    _build.build()
    stamp = tmp_path / "ops.stamp"
    if written is not None:
        stamp.write_text(open(_build.OPS_STAMP, encoding="utf-8").read() if written is True else written)
    monkeypatch.setattr(_build, "OPS_STAMP", str(stamp))
    assert _build.up_to_date() is current
