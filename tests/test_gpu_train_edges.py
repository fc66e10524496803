"""GPU: the experts' training passes on route lists that are none: offsets that
start above 0, descend or end short, and positions and slots that do not name
one another.  Recorded in the workspace; what the lists still hold is right and
nothing outside the buffers is written."""
import ctypes

import pytest
import torch

import train_plain as plain
from parity import REL_RMS_TOL
from test_gpu_train import MOE_ERR_BAD_INDEX, Case, moe  # noqa: F401  (moe: the fixture)

pytestmark = pytest.mark.gpu
SIZES = (200, 4, 2, 512, 256)     # 400 sorted rows
OFFSETS = [
    (120, 200, 300, 350, 400),    # start above 0
    (0, 100, 60, 300, 400),       # descend
    (0, 100, 150, 200, 320),      # end short
    (30, 100, 90, 500, 250),      # all three, and past the end
    (-7, 0, 200, 200, 400),
    (400, 400, 400, 400, 400), (2 ** 31 - 1, 0, 0, 0, 0), (0, 0, 0, 0, 0)]
GUARD = 1 << 20


def guarded(moe, nbytes):  # noqa: F811
    """A workspace inside a larger one, and the bytes on its two sides."""
    room = torch.full((nbytes + 2 * GUARD + 256,), 0x5a, dtype=torch.uint8, device="cuda")
    at = GUARD + (-room.data_ptr() - GUARD) % 256
    ws = moe.Workspace.__new__(moe.Workspace)
    ws.tensor = room[at:at + nbytes]
    ws.nbytes, ws.addr = nbytes, ws.tensor.data_ptr()
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert moe.binding.raw_lib().moe_workspace_init(ws.ptr, nbytes, stream) == 0
    return ws, (room[:at], room[at + nbytes:])


def lists_that_are_none(offsets, seed, unmatched):
    """(case, offsets as they count: ascending inside the rows, the slots that
    lost their position).  `unmatched`: some positions name no slot, some slots
    no position, among them the first rows, before the first group."""
    case = Case(*SIZES, seed=seed)
    P = SIZES[0] * SIZES[2]
    case.offsets = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ends = torch.cummax(torch.tensor(offsets).clamp(0, P), 0).values
    lost = torch.zeros(P, dtype=torch.bool, device="cuda")
    if unmatched:
        names = case.perm.long().clone()
        for p, value in ((0, -1), (1, 2 ** 31 - 1), (31, P), (130, -5), (205, P + 7), (399, -1)):
            case.perm[p] = value
            lost[names[p]] = True
        for p, value in ((2, -1), (32, 2 ** 31 - 1), (140, P), (300, -(2 ** 31)), (210, 211)):
            case.inv[names[p]] = value
            lost[names[p]] = True
        case.names = names
    else:
        case.names = case.perm.long()
    return case, ends, lost


def plain_gradients(case, saved, ends, lost):
    """The 64-bit form over the rows that the lists hold; a slot without a
    position counts as one without weight."""
    gates = case.gates.clone()
    gates.view(-1)[lost] = 0
    return plain.backward(case.d_out, gates, case.x, saved.gate, saved.up, case.names.to(torch.int32), ends, SIZES[2], *case.W)


@pytest.mark.parametrize("unmatched", [False, True])
@pytest.mark.parametrize("offsets", OFFSETS, ids=str)
def test_offsets_that_are_no_offsets(moe, offsets, unmatched):  # noqa: F811
    T, E, k, H, I = SIZES
    P = T * k
    good = Case(*SIZES, seed=31)
    case, ends, lost = lists_that_are_none(offsets, 31, unmatched)
    S = moe.Shape(*SIZES)
    # forward: the groups' rows, and no other
    ws, sides = guarded(moe, moe.expert_ffn_train_workspace_size(S))
    y = torch.full((P, H), 7.0, dtype=torch.bfloat16, device="cuda")
    case.forward(moe, ws=ws, y_sorted=y)
    assert ws.status() == MOE_ERR_BAD_INDEX and all((v == 0x5a).all() for v in sides)
    held = torch.zeros(P, dtype=torch.bool, device="cuda")
    held[int(ends[0]):int(ends[-1])] = True
    assert (y[~held] == 7).all()
    named = held & (case.perm == case.names)
    p = plain.forward(case.x, case.names // k, ends, *case.W)["y"]
    assert plain.rel_rms(y[named], p[named]) <= REL_RMS_TOL
    # backward, from what a pass over good lists kept
    _, saved = good.forward(moe)
    ws, sides = guarded(moe, moe.expert_ffn_backward_workspace_size(S))
    dW = tuple(torch.full_like(w, float("nan")) for w in case.W)
    d_x, d_gates, *_ = case.backward(moe, saved, ws=ws, dW=dW)
    assert ws.status() == MOE_ERR_BAD_INDEX and all((v == 0x5a).all() for v in sides)
    want, _, _ = plain_gradients(case, saved, ends, lost)
    for a, n in zip(dW, ("dWg", "dWu", "dWd")):
        assert plain.rel_rms(a, want[n]) <= REL_RMS_TOL, n
    # tokens whose slots all have a position that a group holds
    inside = torch.zeros(P, dtype=torch.bool, device="cuda")
    inside[case.names[held]] = True
    whole = (inside & ~lost).view(T, k).all(1)
    if whole.any():
        assert plain.rel_rms(d_x[whole], want["d_x"][whole]) <= REL_RMS_TOL
        assert plain.rel_rms(d_gates[whole], want["d_gates"][whole]) <= 2e-5


@pytest.mark.parametrize("unmatched", [False, True])
@pytest.mark.parametrize("offsets", OFFSETS, ids=str)
def test_rows_of_no_group_add_nothing(moe, offsets, unmatched):  # noqa: F811
    """Gradients of tokens with slots outside the groups: those slots count as
    zeros, whatever an earlier call left in the workspace."""
    T, k = SIZES[0], SIZES[2]
    _, saved = Case(*SIZES, seed=32).forward(moe)
    case, ends, lost = lists_that_are_none(offsets, 32, unmatched)
    ws, _ = guarded(moe, moe.expert_ffn_backward_workspace_size(moe.Shape(*SIZES)))
    ws.tensor[256:].fill_(0xff)          # NaN, in bf16 and fp32
    d_x, d_gates, *_ = case.backward(moe, saved, ws=ws)
    assert ws.status() == MOE_ERR_BAD_INDEX
    want, _, _ = plain_gradients(case, saved, ends, lost)
    named = ~lost.view(T, k).any(1)
    assert plain.rel_rms(d_x[named], want["d_x"][named]) <= REL_RMS_TOL
    assert plain.rel_rms(d_gates[named], want["d_gates"][named]) <= 2e-5


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
@pytest.mark.parametrize("sizes,dense", [((333, 6, 3, 256, 512), False), ((3, 300, 2, 256, 256), False), ((333, 1, 1, 512, 256), True)],
                         ids=str)
def test_frozen_experts_need_no_x(moe, sizes, dense, checkpoint):  # noqa: F811
    """The gradients of x and of the gates do not depend on x: the same bits from
    a record without it, over whatever the workspace held."""
    case = Case(*sizes, seed=33, dense=dense)
    _, saved = case.forward(moe, checkpoint)
    want = case.backward(moe, saved)
    saved.x = saved.x_scales = None
    ws, sides = guarded(moe, moe.expert_ffn_backward_workspace_size(moe.Shape(*sizes)))
    ws.tensor[256:].fill_(0xff)
    got = case.backward(moe, saved, need_weights=False, ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[2:] == (None,) * 3
    assert ws.status() == 0 and all((v == 0x5a).all() for v in sides)
