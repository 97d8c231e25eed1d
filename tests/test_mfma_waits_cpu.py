"""No kernel of the language-model operators reads an MFMA's sums before they are written (mfma_waits.py).  Their sources
are compiled to assembly for this; no GPU is needed."""
import subprocess

import pytest

import mfma_waits as waits
from convolution_implicit_gemm_nchw_amd import build

MATRIX_SOURCES = ["matmul_i8.hip", "matmul_f8.hip", "delta_prepare.hip", "delta_fwd.hip", "delta_bwd.hip"]


def test_the_count_itself():
    mfma = "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]"       # 4 passes: 8 states
    read = "v_add_f32_e32 v5, v4, v2"
    assert waits.early_reads([mfma, "s_nop 6", read, "s_endpgm"])[0] == [(read, mfma, 1)]
    assert waits.early_reads([mfma, "s_nop 7", read, "s_endpgm"]) == ([], 1)
    assert waits.early_reads([mfma, "s_nop 7", "v_mov_b32_e32 v7, 0", "s_endpgm"]) == ([], 1)
    # the shorter way counts, over a branch or a loop's end; adding to the same sums does not wait
    skip = [mfma, "s_cbranch_vccnz .L1", "s_nop 7", ".L1:", "ds_write_b128 v9, v[0:3]", "s_endpgm"]
    assert waits.early_reads(skip)[0] == [("ds_write_b128 v9, v[0:3]", mfma, 7)]
    loop = [".L0:", read, "s_nop 7", mfma, "s_cbranch_scc1 .L0", "s_nop 7", read, "s_endpgm"]
    assert waits.early_reads(loop)[0] == [(read, mfma, 7)]
    assert waits.early_reads([mfma, mfma, "s_nop 7", read, "s_endpgm"]) == ([], 2)
    column = "v_mfma_f32_16x16x32_bf16 v[16:19], v[8:11], v[0:3], 0"
    assert waits.early_reads([mfma, column, "s_endpgm"])[0] == [(column, mfma, 8)]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    out = tmp_path_factory.mktemp("assembly")
    paths = dict(build.sources())
    runs = [subprocess.Popen([build._hipcc()] + build.compile_flags() + ["-x", "hip", "--cuda-device-only", "-S", paths[s], "-o",
                                                                         str(out / s)], stderr=subprocess.DEVNULL)
            for s in MATRIX_SOURCES]
    assert [r.wait() for r in runs] == [0] * len(runs)
    return {s: (out / s).read_text() for s in MATRIX_SOURCES}


@pytest.mark.parametrize("source", MATRIX_SOURCES)
def test_sums_are_read_when_they_are_written(assembly, source):
    total = 0
    for name, lines in waits.kernels(assembly[source]):
        early, count = waits.early_reads(lines)
        assert not early, (name, early[:4])
        total += count
    assert total > 0
