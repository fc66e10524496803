"""GPU: the experts' training passes and 8-bit checkpoints against plain 64-bit
forms, and against differences.

Tolerances.  A sum of n terms is off by at most n 2^-23 times the sum of the
terms' magnitudes (see train_plain), a rounding to bf16 by 2^-8 of the value.
Elementwise bounds follow each formula: an output whose terms hold one operand
rounded to bf16 is off by 2^-8 of the sum of its terms' magnitudes, and by 2^-8
of itself for its own rounding; evaluating silu and its slope in fp32 adds less
than 2^-16 of the magnitudes (|g| < 16 here: 2 + 1.2|g| units of 2^-23 from the
fast exponential).  Over whole outputs the relative RMS of r independent
roundings is 1.7e-3 sqrt(r), r <= 3 here: 5e-3, as for the forward layer."""
import pytest
import torch

import fp8_plain
import train_plain as plain
from parity import REL_RMS_TOL

pytestmark = pytest.mark.gpu
MOE_ERR_TIMEOUT, MOE_ERR_BAD_INDEX = 5, 6
SHAPES = [   # T, E, k, H, I
    (64, 16, 2, 512, 256), (1, 1, 1, 256, 256), (7, 5, 3, 256, 512), (300, 3, 2, 512, 256), (333, 24, 4, 768, 512),
    (40, 64, 8, 256, 256), (513, 1, 1, 512, 768), (2, 1024, 8, 256, 256), (1000, 2, 2, 256, 1024)]


@pytest.fixture(scope="module")
def moe():
    import routed_expert_ffn_02_gb300 as m
    return m


class Case:
    def __init__(self, T, E, k, H, I, seed=0, dense=False, gated=True):
        g = torch.Generator(device="cuda")
        g.manual_seed(1000 * seed + T + E)
        randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.sizes, self.dense = (T, E, k, H, I), dense
        self.x = randn(T, H).to(torch.bfloat16)
        self.W = tuple((randn(*s) * s[2] ** -0.5).to(torch.bfloat16) for s in ((E, I, H), (E, I, H), (E, H, I)))
        self.d_out = randn(T, H).to(torch.bfloat16)
        self.perm, self.offsets, self.inv, self.gates = plain.routing(T, E, k, seed, device="cuda")
        if dense:
            self.perm = self.offsets = self.inv = None
            self.gates = torch.rand((T, 1), generator=g, device="cuda")
        if not gated:
            self.gates = None
        self.tokens = self.perm.long() // k if self.perm is not None else torch.arange(T, device="cuda")

    def forward(self, moe, checkpoint="bf16", **kw):
        return moe.moe_expert_ffn_train(moe.Shape(*self.sizes), self.x, self.perm, self.offsets, *self.W,
                                        checkpoint=checkpoint, **kw)

    def backward(self, moe, saved, **kw):
        return moe.moe_expert_ffn_backward(moe.Shape(*self.sizes), self.d_out, saved, self.perm, self.offsets, self.inv,
                                           *self.W, gates=self.gates, **kw)

    def plain_forward(self):
        return plain.forward(self.x, self.tokens, self.offsets, *self.W)

    def plain_backward(self, moe, saved):
        x, g, u = values(moe, saved)
        return plain.backward(self.d_out, self.gates, x, g, u, self.perm, self.offsets, self.sizes[2], *self.W)


def values(moe, saved):
    """x, gate, up of a record, as it stands for them, in 64 bits."""
    if saved.gate_scales is None:
        return saved.x.double(), saved.gate.double(), saved.up.double()
    return tuple(fp8_plain.rows_value(q, s) for q, s in ((saved.x, saved.x_scales), (saved.gate, saved.gate_scales),
                                                          (saved.up, saved.up_scales)))


def within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, bad.sum().item(), bad.nonzero()[0].tolist())


def check_forward(case, y, saved, moe):
    T, E, k, H, I = case.sizes
    p = case.plain_forward()
    sums = {n: (H + 1) * plain.ADD * p[n + "_mag"] for n in "gu"}
    if saved.gate_scales is None:
        assert saved.x is case.x
        for n, got in (("g", saved.gate), ("u", saved.up)):
            within(got, p[n], sums[n] + plain.U * (p[n].abs() + sums[n]), n)
    else:
        q, b = fp8_plain.quantize_rows(case.x)
        assert torch.equal(saved.x.double(), q) and torch.equal(saved.x_scales.long(), b)
        for n, got, scales in (("g", saved.gate, saved.gate_scales), ("u", saved.up, saved.up_scales)):
            code = got.double().abs().reshape(-1, I // 128, 128)
            # the scale is the smallest: the block's largest code is in [224, 448]
            assert ((code.amax(2) >= 224) & (code.amax(2) <= 448)).all()
            value = fp8_plain.rows_value(got, scales)
            # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale below its smallest normal
            step = 2.0 ** -10 * fp8_plain.two_to(scales.long() - 127).repeat_interleave(128, 1)
            within(value, p[n], sums[n] + 2.0 ** -4 * (p[n].abs() + sums[n]) + step, n)
    slack = plain.U + 2.0 ** -16
    gu = p["g"].abs() * p["u_mag"] + 2 * p["g_mag"] * p["u"].abs()          # what errors of g and u do to h
    hs = (H + 1) * plain.ADD * gu
    spread = torch.zeros_like(p["y"])
    for e, r in plain.groups(case.offsets, T * k):
        spread[r] = hs[r] @ case.W[2][e].double().abs().T
    tol = slack * p["y_mag"] + 2 * spread + (I + 1) * plain.ADD * p["y_mag"]
    within(y, p["y"], tol + plain.U * (p["y"].abs() + tol), "y")
    assert plain.rel_rms(y, p["y"]) <= REL_RMS_TOL


def check_backward(case, out, saved, moe):
    T, E, k, H, I = case.sizes
    want, mag, mag_q = case.plain_backward(moe, saved)
    d_x, d_gates, *dW = out
    terms = {"d_x": 2 * I + k, "d_gates": I, "dWg": T * k, "dWu": T * k, "dWd": T * k}
    for n, v in (("d_x", d_x), ("d_gates", d_gates), *zip(("dWg", "dWu", "dWd"), dW)):
        if v is None:
            continue
        roundings = 0 if n == "d_gates" else 1
        tol = (roundings * plain.U * (1 + plain.U) + 2.0 ** -16 + (terms[n] + 1) * plain.ADD) * mag[n]
        tol = tol + (H + 1) * plain.ADD * mag_q[n]           # q's own sum
        if n != "d_gates":
            tol = tol + plain.U * (want[n].abs() + tol)
        within(v, want[n], tol, n)
        # q and its 2^-23 adders: far inside 2e-5 of the norm
        assert plain.rel_rms(v, want[n]) <= (2e-5 if n == "d_gates" else REL_RMS_TOL), n


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
@pytest.mark.parametrize("sizes", SHAPES, ids=str)
def test_forward(moe, sizes, checkpoint):
    case = Case(*sizes)
    ws = moe.Workspace(moe.expert_ffn_train_workspace_size(moe.Shape(*sizes)))
    y, saved = case.forward(moe, checkpoint, ws=ws)
    assert ws.status() == 0
    check_forward(case, y, saved, moe)


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
@pytest.mark.parametrize("sizes", SHAPES, ids=str)
def test_backward(moe, sizes, checkpoint):
    case = Case(*sizes, seed=1)
    _, saved = case.forward(moe, checkpoint)
    ws = moe.Workspace(moe.expert_ffn_backward_workspace_size(moe.Shape(*sizes)))
    out = case.backward(moe, saved, ws=ws)
    assert ws.status() == 0
    check_backward(case, out, saved, moe)


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 15, 16, 17, 32, 33, 255, 257, 700])
@pytest.mark.parametrize("gated", [False, True])
def test_dense_block(moe, T, gated, checkpoint):
    case = Case(T, 1, 1, 512, 256, seed=2, dense=True, gated=gated)
    y, saved = case.forward(moe, checkpoint)
    check_forward(case, y, saved, moe)
    out = case.backward(moe, saved)
    assert (out[1] is not None) == gated
    check_backward(case, out, saved, moe)
