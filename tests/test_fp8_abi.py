"""The 8-bit operators' and the balance loss's argument checks (no GPU needed:
they come before any device call)."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
GOOD = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_ffn_02_gb300 as m
    return m.binding.raw_lib()


def test_quantize_refusals(lib):
    assert lib.moe_quantize_rows(GOOD, -1, 128, GOOD, GOOD, None) == INVALID
    for K in (0, 64, 100, 200):
        assert lib.moe_quantize_rows(GOOD, 4, K, GOOD, GOOD, None) == INVALID
    assert lib.moe_quantize_rows(GOOD, 4, 16512, GOOD, GOOD, None) == UNSUPPORTED
    assert lib.moe_quantize_rows(None, 4, 128, GOOD, GOOD, None) == INVALID
    assert lib.moe_quantize_rows(ODD, 4, 128, GOOD, GOOD, None) == INVALID
    assert lib.moe_quantize_rows(GOOD, 4, 128, GOOD, None, None) == INVALID
    assert lib.moe_quantize_rows(None, 0, 128, None, None, None) == OK
    assert lib.moe_quantize_weights(GOOD, -1, 128, 128, GOOD, GOOD, None) == INVALID
    assert lib.moe_quantize_weights(GOOD, 1, 130, 128, GOOD, GOOD, None) == INVALID
    assert lib.moe_quantize_weights(GOOD, 1 << 20, 16384, 16384, GOOD, GOOD, None) == INVALID
    assert lib.moe_quantize_weights(None, 0, 128, 128, None, None, None) == OK
    assert b"" == lib.moe_last_error()


def test_product_refusals(lib):
    def call(x=GOOD, xs=GOOD, rows=4, off=GOOD, E=2, N=128, K=128, W=GOOD, Ws=GOOD, y=GOOD, ws=GOOD,
             n=1 << 20):
        return lib.moe_grouped_gemm_fp8(x, xs, rows, off, E, N, K, W, Ws, y, ws, n, None)
    for bad in (dict(rows=-1), dict(E=0), dict(E=1025), dict(N=64), dict(K=0), dict(x=None),
                dict(xs=ODD), dict(off=None), dict(W=ODD), dict(Ws=None), dict(y=ODD)):
        assert call(**bad) == INVALID, bad
    assert call(N=16512) == UNSUPPORTED
    for bad in (dict(ws=None), dict(n=100), dict(ws=ctypes.c_void_p(0x10010))):
        assert call(**bad) == WORKSPACE, bad
    assert call(rows=0, x=None, y=None, ws=None) == OK
    assert lib.moe_grouped_gemm_fp8_workspace_size(-1, 4) == 0
    assert lib.moe_grouped_gemm_fp8_workspace_size(4, 1025) == 0
    assert lib.moe_grouped_gemm_fp8_workspace_size(0, 1) > 0


def test_layer_refusals(lib):
    import routed_expert_ffn_02_gb300 as m
    shape = m.binding.MoeShape(16, 16, 2, 512, 256, 32, 0)
    w = m.binding.MoeFp8Experts(*[0x10000] * 6)
    sp, wp = ctypes.byref(shape), ctypes.byref(w)
    n = lib.moe_fp8_workspace_size(sp)
    assert n >= 32 * (512 * 3 + 256) and lib.moe_expert_ffn_fp8_workspace_size(sp) < n

    def fwd(logits=GOOD, x=GOOD, e=wp, out=GOOD, ws=GOOD, size=n, s=sp):
        return lib.moe_forward_fp8(s, logits, x, e, out, None, None, ws, size, None)
    for bad in (dict(logits=None), dict(x=ODD), dict(e=None), dict(out=None), dict(s=None)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(ws=None) == WORKSPACE and fwd(size=n - 1) == WORKSPACE
    for i in range(6):
        parts = [0x10000] * 6
        parts[i] = 0x10008
        assert fwd(e=ctypes.byref(m.binding.MoeFp8Experts(*parts))) == INVALID
    bad_shape = m.binding.MoeShape(16, 16, 2, 384, 256, 32, 0)
    assert fwd(s=ctypes.byref(bad_shape)) == INVALID
    assert lib.moe_fp8_workspace_size(ctypes.byref(bad_shape)) == 0
    assert lib.moe_expert_ffn_fp8(sp, GOOD, None, GOOD, wp, GOOD, GOOD, n, None) == INVALID
    assert lib.moe_expert_ffn_fp8(sp, GOOD, GOOD, GOOD, wp, GOOD, GOOD, 100, None) == WORKSPACE


def test_balance_refusals(lib):
    def fwd(logits=GOOD, idx=GOOD, T=8, E=4, k=2, seq=None, S=1, loss=GOOD, counts=GOOD, stats=GOOD,
            ws=GOOD, n=1 << 20):
        return lib.moe_balance(logits, idx, T, E, k, seq, S, 1.0, loss, counts, stats, ws, n, None)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=5), dict(k=9, E=100), dict(S=0),
                dict(S=2), dict(logits=None), dict(idx=None), dict(loss=None), dict(counts=None),
                dict(stats=None), dict(stats=ctypes.c_void_p(0x10004))):
        assert fwd(**bad) == INVALID, bad
    assert fwd(ws=None) == WORKSPACE and fwd(n=300) == WORKSPACE
    assert lib.moe_balance_workspace_size(8, 4, 0) == 0

    def bwd(logits=GOOD, stats=GOOD, counts=GOOD, seq=None, T=8, S=1, idx=None, g=None, dg=None, d=GOOD):
        return lib.moe_balance_backward(logits, stats, counts, seq, T, 4, 2, S, 1.0, None, idx, g, dg,
                                        d, None)
    for bad in (dict(logits=None), dict(stats=None), dict(counts=None), dict(d=None), dict(S=3),
                dict(idx=GOOD), dict(idx=GOOD, g=GOOD), dict(dg=GOOD)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(T=0, logits=None, d=None) == OK


def test_host_tensors_without_a_workspace_are_refused():
    """Before a workspace is made beside them and its status word is cleared on
    the device."""
    import torch
    import routed_expert_ffn_02_gb300 as m

    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype)
    f8, u8, i32 = torch.float8_e4m3fn, torch.uint8, torch.int32
    shape = m.Shape(4, 4, 2, 256, 256)
    for call in (
            lambda: m.Workspace(1024, "cpu"),
            lambda: m.moe_grouped_gemm_fp8(z(4, 256, dtype=f8), z(4, 2, dtype=u8), z(3, dtype=i32),
                                           z(2, 256, 256, dtype=f8), z(2, 2, 2, dtype=u8)),
            lambda: m.moe_expert_ffn_fp8(shape, z(4, 256), z(8, dtype=i32), z(5, dtype=i32), None),
            lambda: m.moe_forward_fp8(shape, z(4, 4, dtype=torch.float32), z(4, 256), None),
            lambda: m.moe_balance(z(4, 4, dtype=torch.float32), z(4, 2, dtype=i32)),
            lambda: m.moe_permute(z(4, 2, dtype=i32), 4),
            lambda: m.moe_forward(shape, z(4, 4, dtype=torch.float32), z(4, 256), *[z(4, 256, 256)] * 3)):
        with pytest.raises(AssertionError, match="CUDA"):
            call()
