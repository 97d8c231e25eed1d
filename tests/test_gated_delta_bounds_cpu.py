"""Sizes past what a call can take: refused, with no count that wraps (no GPU needed; addresses are never dereferenced)."""
import ctypes

import convolution_implicit_gemm_nchw_amd as mc
import test_delta_layer_cpu as layer

OK, E_BIG, at = layer.OK, layer.E_BIG, layer.at


def test_saved_states_do_not_wrap():
    need = ctypes.c_size_t(1)

    def size(*a):
        return mc.lib().gated_delta_states_size(*a, ctypes.byref(need))
    assert size(16384, 65536, 256, 512, 1 << 30) == E_BIG      # 2^30 heads x 2^24 chunks x 163840 x 4 bytes, 0 modulo 2^64
    assert size(1 << 30, 1, 1, 1, 1 << 30) == E_BIG
    assert size(4, 32, 128, 128, 8192) == OK and need.value == 4 * 32 * 128 * (128 + 64) * 128 * 4


def step(**kw):
    kw = {**dict(L=1, q=layer.rows(0, 16, 1), k=layer.rows(1, 16, 1), v=layer.rows(2, 24, 1), g=layer.rows(3, 4, 1),
                 beta=layer.rows(4, 4, 1), y=layer.rows(7, 24, 1)), **kw}
    slots = kw.pop("slots")
    return mc.lib().gated_delta_step(ctypes.byref(layer.delta_args(**kw)), 0, at(20), slots, at(22), at(20), None)


def test_pools_of_states_do_not_wrap():
    one = mc._Rows(at(0), 0, 0)
    rows = dict(B=1, Hk=1, Hv=65536, P=256, V=512, q=one, k=mc._Rows(at(1), 0, 0), v=mc._Rows(at(2), 0, 0),
                g=mc._Rows(at(3), 0, 0), beta=mc._Rows(at(4), 0, 0), y=mc._Rows(1 << 60, 1 << 25, 1))
    assert step(slots=1 << 30, **rows) == E_BIG                # 2^63 values


def test_steps_whose_groups_pass_31_bits():
    """A work-group takes 64 value channels of a head and counts in 32 bits with a sign."""
    none = dict(q=mc._Rows(at(0), 0, 0), k=mc._Rows(at(1), 0, 0), v=mc._Rows(at(2), 0, 0), g=mc._Rows(at(3), 0, 0),
                beta=mc._Rows(at(4), 0, 0))
    assert step(slots=1, B=1 << 25, Hk=1, Hv=32, P=1, V=129, y=mc._Rows(1 << 60, 32 * 129, 1), **none) == E_BIG


def test_quantised_blocks_past_31_bits():
    """The same for blocks of 128 channels of all tokens."""
    def quantize(B, L, C, sc):
        return mc.lib().quantize_f8(B, L, C, 1, at(0), 0, 1 if sc != 1 else 0, sc, 1 << 60, 1 << 59, None)
    assert quantize(1 << 25, 1, 128 * 65, 0) == E_BIG
    assert quantize(1 << 21, 1, 131072, 1) == E_BIG


def test_norm_describes_what_it_takes():
    buf, lib = ctypes.create_string_buffer(64), mc.lib()

    def describe(n, dtype=0, backward=1, ws=1 << 20, size=64):
        return lib.layer_norm_describe(None if n is None else ctypes.byref(n), dtype, backward, ws, buf, size)
    n = layer.norm_args()
    assert describe(n) == OK and buf.value == b"algo=norm_tokens threads=64 times=1 parts=20"
    assert describe(n, ws=2 * 8 * 24) == OK and buf.value.endswith(b"parts=2")
    assert describe(n, backward=0) == OK and buf.value == b"algo=norm_tokens threads=64 times=1"
    assert describe(layer.norm_args(major=True), backward=0) == OK and buf.value == b"algo=norm_rows lanes=1 threads=256"
    assert describe(None) == layer.E_NULL and lib.layer_norm_describe(ctypes.byref(n), 0, 0, 0, None, 64) == layer.E_NULL
    assert describe(layer.norm_args(C=0)) == layer.E_DIM and describe(n, dtype=2) == layer.E_DT
    assert describe(n, ws=8 * 24 - 1) == layer.E_WS and buf.value == b""
    assert describe(n, backward=0, size=5) == OK and buf.value == b"algo"
