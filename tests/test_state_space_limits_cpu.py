"""State-space operators without a GPU: workspace sizes under any limit."""
import ctypes

import pytest

import convolution_implicit_gemm_nchw_amd as mc
import test_state_space_cpu as base

OK = base.OK
SIZE_MAX = (1 << 64) - 1


def sizes(call, limits):
    need, out = ctypes.c_size_t(0), []
    for limit in limits:
        assert call(limit, ctypes.byref(need)) == OK
        assert need.value <= limit
        out.append(need.value)
    return out


@pytest.mark.parametrize("name", ["convolution", "scan", "product"])
def test_workspace_size_under_any_limit(name):
    """Problems that split their sums: no limit gives what a large one gives, a small one less."""
    lib = mc.lib()
    conv, scan = base.conv_args(B=64, L=8192), base.scan_args(B=1, L=8192)
    call = {"convolution": lambda n, p: lib.causal_conv1d_bwd_workspace_size(ctypes.byref(conv), 0, n, p),
            "scan": lambda n, p: lib.selective_scan_fwd_workspace_size(ctypes.byref(scan), 0, n, p),
            "product": lambda n, p: lib.matmul_i8_workspace_size(1, 100, 70, 8192, n, p)}[name]
    none, some, large, huge, top = sizes(call, (0, 1000, 10 ** 9, 1 << 63, SIZE_MAX))
    assert none == 0 and some < large
    assert large == huge == top and large > 0


def test_the_convolutions_need_no_binding_module(tmp_path):
    """A package without _miconv_bind.so imports and serves the convolutions; the operators that need it say so."""
    import os
    import subprocess
    import sys
    package = tmp_path / "convolution_implicit_gemm_nchw_amd"
    package.mkdir()
    here = os.path.dirname(mc.__file__)
    for name in ("__init__.py", "libmiconv.so"):
        os.symlink(os.path.join(here, name), package / name)
    code = """
import torch
import convolution_implicit_gemm_nchw_amd as mc
assert mc.__file__.startswith({0!r})
assert mc.workspace_size(mc.FWD, mc.F32, [2, 8, 16, 16, 8, 3, 3, 1, 1, 1, 1, 16, 16]) >= 0
assert mc.selective_scan_fwd_describe(1, 16, 40, 4)
for _ in range(2):
    try:
        mc.quantize_tokens(torch.zeros(2, 3))
    except ImportError as e:
        assert "_miconv_bind.so" in str(e) and "build.py" in str(e)
    else:
        raise AssertionError("no ImportError")
""".format(str(package))
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr


LARGE = [(8, 4096, 4096, 16), (8, 8192, 8192, 16), (8, 8192, 8192, 64), (1, 8192, 1 << 20, 64), (1 << 20, 16, 3, 64),
         (1, 1 << 30, 1, 64), (4096, 8192, 1, 64), (1, 16, 1 << 22, 64), (16, 1024, 16384, 64, 8)]


@pytest.mark.parametrize("size", LARGE, ids=lambda s: "-".join(map(str, s)))
def test_backward_scan_keeps_to_the_workspace_cap(size):
    need = ctypes.c_size_t(0)
    B, D, L, N, G = (size + (1,))[:5]
    s = mc._Scan(B=B, D=D, L=L, N=N, G=G)
    assert mc.lib().selective_scan_bwd_workspace_size(ctypes.byref(s), 0, ctypes.byref(need)) == OK
    assert 0 < need.value <= mc.MAX_WORKSPACE_BYTES
    assert mc.selective_scan_bwd_workspace(*size, limit=SIZE_MAX) == need.value


@pytest.mark.parametrize("size", LARGE + [(3, 40, 300, 5, 2), (2, 50, 700, 40), (1, 20, 5000, 3), (2, 8, 6000, 20)],
                         ids=lambda s: "-".join(map(str, s)))
def test_backward_scan_under_any_limit(size):
    """The size under a limit is within it, or the least there is; a call given that much uses that much."""
    least = mc.selective_scan_bwd_workspace(*size, limit=0)
    assert least <= 2 * 8 * 128 * 64 * 4                      # a slice of 128 steps of 16 channels at most
    before = 0
    for limit in [0, least - 1, least] + [10 ** k for k in range(4, 10)] + [SIZE_MAX]:
        w = mc.selective_scan_bwd_workspace(*size, limit=limit)
        assert w == least or least < w <= limit
        assert before <= w
        before = w
        assert mc.selective_scan_bwd_workspace(*size, limit=w) == w
        assert mc.selective_scan_bwd_describe(*size, workspace_bytes=w).endswith(f" ws={w}")
    with pytest.raises(ValueError):
        mc.selective_scan_bwd_describe(*size, workspace_bytes=least - 1)
    B, D, L, N, G = (size + (1,))[:5]
    assert base.sbwd(B=B, D=D, L=L, N=N, G=G, ws=base.at(30), wb=least - 1) == base.E_WS
