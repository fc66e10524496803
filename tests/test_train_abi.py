"""Entry points of the experts' training passes and of the product with an
epilogue that need no GPU: their refusals, workspace sizes and no-ops."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
GOOD, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)   # never read: every call is refused
WS, BIG = ctypes.c_void_p(0x100000), 1 << 40


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_expert_ffn_02_gb300 as m
    return m


def saved(moe, fp8=0, x=GOOD, scales=None, **other):
    v = moe.binding.MoeSaved(fp8, x, scales, GOOD, scales, GOOD, scales)
    for n, p in other.items():
        setattr(v, n, p)
    return v


def train(moe, shape=(16, 16, 2, 512, 256), x=GOOD, perm=GOOD, offsets=GOOD, W=GOOD, y=GOOD, kept="bf16", ws=WS,
          n=BIG):
    kept = saved(moe) if kept == "bf16" else kept
    lib = moe.binding.raw_lib()
    c = moe.binding.MoeShape(*shape, 32, 0)
    st = lib.moe_expert_ffn_train(ctypes.byref(c), x, perm, offsets, W, GOOD, GOOD, y,
                                  ctypes.byref(kept) if kept else None, ws, n, None)
    return st, lib.moe_last_error().decode()


def backward(moe, shape=(16, 16, 2, 512, 256), d=GOOD, gates=GOOD, kept="bf16", perm=GOOD, offsets=GOOD, inv=GOOD,
             d_x=GOOD, d_gates=GOOD, dW=(GOOD,) * 3, ws=WS, n=BIG):
    kept = saved(moe) if kept == "bf16" else kept
    lib = moe.binding.raw_lib()
    c = moe.binding.MoeShape(*shape, 32, 0)
    st = lib.moe_expert_ffn_backward(ctypes.byref(c), d, gates, ctypes.byref(kept) if kept else None, perm, offsets,
                                     inv, GOOD, GOOD, GOOD, d_x, d_gates, *dW, ws, n, None)
    return st, lib.moe_last_error().decode()


@pytest.mark.parametrize("change,status,text", [
    (dict(shape=(16, 16, 2, 500, 256)), INVALID, "H"), (dict(shape=(16, 16, 2, 512, 16640)), UNSUPPORTED, "limited"),
    (dict(shape=(-1, 16, 2, 512, 256)), INVALID, "T"), (dict(perm=None), INVALID, "come together"),
    (dict(offsets=None), INVALID, "come together"), (dict(perm=None, offsets=None), INVALID, "dense"),
    (dict(x=None), INVALID, "x is NULL"), (dict(x=ODD), INVALID, "aligned"), (dict(W=ODD), INVALID, "aligned"),
    (dict(y=None), INVALID, "y_sorted"), (dict(kept=None), INVALID, "saved is NULL"), (dict(ws=None), WORKSPACE, "NULL"),
    (dict(n=1000), WORKSPACE, "needs"), (dict(ws=ctypes.c_void_p(0x100010)), WORKSPACE, "aligned"),
])
def test_train_refusals(moe, change, status, text):
    st, said = train(moe, **change)
    assert st == status and text in said, said


@pytest.mark.parametrize("change,text", [
    (dict(gate=None), "gate is NULL"), (dict(up=ODD), "aligned"), (dict(fp8=1, x=None), "x is NULL"),
    (dict(fp8=1), "without scales"), (dict(fp8=1, scales=GOOD, up_scales=None), "without scales")])
def test_saved_refusals(moe, change, text):
    for call in (train, backward):
        st, said = call(moe, kept=saved(moe, **change))
        assert st == INVALID and text in said, said


@pytest.mark.parametrize("change,status,text", [
    (dict(inv=None), INVALID, "come together"), (dict(perm=None), INVALID, "come together"),
    (dict(perm=None, offsets=None, inv=None), INVALID, "dense"),
    (dict(shape=(16, 1, 1, 512, 256), perm=None, offsets=None), INVALID, "come together"),
    (dict(gates=None), INVALID, "d_gates without gates"), (dict(dW=(GOOD, None, GOOD)), INVALID, "dW_up is NULL"),
    (dict(dW=(GOOD, GOOD, ODD)), INVALID, "aligned"), (dict(d=None), INVALID, "d_out is NULL"),
    (dict(d_x=ODD), INVALID, "aligned"), (dict(n=1000), WORKSPACE, "needs"),
])
def test_backward_refusals(moe, change, status, text):
    st, said = backward(moe, **change)
    assert st == status and text in said, said


def test_backward_reads_x_of_either_kind(moe):
    st, said = backward(moe, kept=saved(moe, x=None))
    assert st == INVALID and "x is NULL" in said


@pytest.mark.parametrize("kept", [dict(), dict(fp8=1, scales=GOOD, x_scales=None)])
def test_backward_without_the_weights_gradients_needs_no_x(moe, kept):
    st, said = backward(moe, kept=saved(moe, x=None, **kept), dW=(None,) * 3, ws=None)
    assert st == WORKSPACE and "NULL" in said       # the next thing that is missing
    st, said = backward(moe, kept=saved(moe, x=None, **kept), ws=None)
    assert st == INVALID and "x is NULL" in said
    st, said = backward(moe, kept=saved(moe, x=None, fp8=1, scales=GOOD, gate_scales=None), dW=(None,) * 3, ws=None)
    assert st == INVALID and "without scales" in said


@pytest.mark.parametrize("name", ["perm", "offsets"])
def test_train_refuses_misaligned_lists(moe, name):
    st, said = train(moe, **{name: ctypes.c_void_p(0x10002)}, ws=None)
    assert st == INVALID and f"{name} is not 4-byte aligned" in said


@pytest.mark.parametrize("name", ["perm", "offsets", "inv", "gates", "d_gates"])
def test_backward_refuses_misaligned_lists_and_gates(moe, name):
    st, said = backward(moe, **{name: ctypes.c_void_p(0x10002)}, ws=None)
    assert st == INVALID and "is not 4-byte aligned" in said and name in said


def test_product_refuses_misaligned_offsets(moe):
    lib = moe.binding.raw_lib()
    assert lib.moe_grouped_gemm(GOOD, 5, ctypes.c_void_p(0x10002), 3, 40, 64, GOOD, None, 0, None, GOOD, 0, None, 0, None) == INVALID
    assert "offsets is not 4-byte aligned" in lib.moe_last_error().decode()


def test_nothing_to_do(moe):
    """No token: no buffer is looked at (but the weights' gradients, which would be cleared)."""
    assert train(moe, shape=(0, 16, 2, 512, 256), x=None, y=None, kept=None, ws=None)[0] == 0
    assert backward(moe, shape=(0, 16, 2, 512, 256), d=None, kept=None, ws=None, dW=(None,) * 3)[0] == 0
    lib = moe.binding.raw_lib()
    assert lib.moe_dequantize_rows(None, None, 0, 128, None, None) == 0
    assert lib.moe_grouped_gemm(None, 0, GOOD, 4, 64, 64, None, None, 0, None, None, 0, None, 0, None) == 0


def test_workspace_sizes(moe):
    S = moe.Shape(4096, 64, 4, 1024, 512)
    P = S.P
    assert 2 * P * (1024 + 512) <= moe.expert_ffn_train_workspace_size(S) <= 2 * P * (1024 + 512) + (1 << 20)
    least = 2 * P * (4 * 1024 + 3 * 512) + 4 * P * 512 // 32
    assert least <= moe.expert_ffn_backward_workspace_size(S) <= least + 16 * 64 * 8 * 1024 + (1 << 20)
    with pytest.raises(moe.MoeError):
        moe.expert_ffn_backward_workspace_size(moe.Shape(1, 2, 3, 512, 256))
    assert moe.grouped_gemm_workspace_size(0, 1, 8, 8) >= 256
    for bad in ((-1, 1, 8, 8), (1, 0, 8, 8), (1, 1025, 8, 8), (1, 1, 0, 8), (1, 1, 8, 12), (1, 1, 8, 0), (1, 1, 65537, 8),
                (1, 1, 8, 65544), (2 ** 31 - 1, 1, 8, 8)):
        with pytest.raises(moe.MoeError):
            moe.grouped_gemm_workspace_size(*bad)


@pytest.mark.parametrize("change,status,text", [
    (dict(rows=-1), INVALID, "rows"), (dict(E=0), INVALID, "E"), (dict(E=2, offsets=None), INVALID, "offsets is NULL"),
    (dict(N=0), INVALID, "N"), (dict(K=12), INVALID, "multiple of 8"), (dict(N=65537), UNSUPPORTED, "limited"),
    (dict(act=4), INVALID, "activation"), (dict(act=-1), INVALID, "activation"), (dict(x=None), INVALID, "x is NULL"),
    (dict(W=ODD), INVALID, "aligned"), (dict(y=None), INVALID, "y is NULL"), (dict(ws=None), WORKSPACE, "NULL"),
    (dict(n=16), WORKSPACE, "needs"), (dict(bias=ctypes.c_void_p(0x10002)), INVALID, "bias"),
    (dict(residual=ctypes.c_void_p(0x10001)), INVALID, "residual")])
def test_product_refusals(moe, change, status, text):
    a = dict(x=GOOD, rows=5, offsets=GOOD, E=3, N=40, K=64, W=GOOD, bias=None, act=0, residual=None, y=GOOD, f32=0, ws=WS,
             n=BIG)
    a.update(change)
    lib = moe.binding.raw_lib()
    st = lib.moe_grouped_gemm(*a.values(), None)
    assert st == status and text in lib.moe_last_error().decode(), lib.moe_last_error()


@pytest.mark.parametrize("rows,K,status", [(-1, 128, INVALID), (1, 100, INVALID), (1, 0, INVALID), (1, 16512, UNSUPPORTED)])
def test_dequantize_refusals(moe, rows, K, status):
    assert moe.binding.raw_lib().moe_dequantize_rows(GOOD, GOOD, rows, K, GOOD, None) == status


def test_python_refuses_host_tensors_types_and_kinds(moe):
    S = moe.Shape(4, 1, 1, 256, 256)
    x, W = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(1, 256, 256, dtype=torch.bfloat16)
    with pytest.raises(AssertionError, match="CUDA"):
        moe.moe_expert_ffn_train(S, x, None, None, W, W, W)
    with pytest.raises(AssertionError, match="checkpoint"):
        moe.SavedFfn.empty(S, x, "int8")
    with pytest.raises(AssertionError, match="activation"):
        moe.moe_grouped_gemm(x, W, activation="tanh")
    with pytest.raises(AssertionError, match="out_dtype"):
        moe.moe_grouped_gemm(x, W, out_dtype=torch.float16)
    with pytest.raises(AssertionError, match="CUDA"):
        moe.moe_dequantize_rows(torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8))
