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


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
@pytest.mark.parametrize("sizes", [(4, 8, 2, 256, 256), (600, 8, 2, 256, 256)], ids=str)
def test_experts_without_rows(moe, sizes, checkpoint):
    """Their gradients are zeros, over whatever was there."""
    case = Case(*sizes, seed=3)
    T, E, k, H, I = sizes
    idx = (torch.arange(T * k, device="cuda") % 2 * 3 + 2).view(T, k)     # experts 2 and 5 only
    case.perm = torch.sort(idx.flatten(), stable=True).indices.to(torch.int32)
    counts = torch.bincount(idx.flatten(), minlength=E)
    case.offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    case.inv = torch.empty_like(case.perm)
    case.inv[case.perm.long()] = torch.arange(T * k, device="cuda", dtype=torch.int32)
    case.tokens = case.perm.long() // k
    y, saved = case.forward(moe, checkpoint)
    check_forward(case, y, saved, moe)
    dW = tuple(torch.full_like(w, float("nan")) for w in case.W)
    out = case.backward(moe, saved, dW=dW)
    assert all(a is b for a, b in zip(out[2:], dW))
    check_backward(case, out, saved, moe)
    for e in (0, 1, 3, 4, 6, 7):
        assert all((w[e] == 0).all() for w in dW)


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
@pytest.mark.parametrize("sizes", [(20, 2, 1, 16384, 256), (20, 2, 1, 256, 16384), (300, 2, 2, 256, 16384)], ids=str)
def test_largest_sizes(moe, sizes, checkpoint):
    case = Case(*sizes, seed=26)
    y, saved = case.forward(moe, checkpoint)
    check_forward(case, y, saved, moe)
    check_backward(case, case.backward(moe, saved), saved, moe)


def test_offsets_beyond_32_bits(moe):
    """More than 2^31 values in each kept projection and in the products' results."""
    T, H, I = 140_000, 256, 16384
    case = Case(T, 1, 1, H, I, seed=27, dense=True)
    y, saved = case.forward(moe)
    d_x, d_gates, *_ = case.backward(moe, saved, need_weights=False)
    rows = torch.cat([torch.arange(0, 3), torch.arange(131071, 131074), torch.arange(T - 40, T)]).cuda()
    part = Case(len(rows), 1, 1, H, I, seed=27, dense=True)
    part.W, part.x, part.d_out, part.gates = case.W, case.x[rows], case.d_out[rows], case.gates[rows]
    kept = moe.SavedFfn(part.x, saved.gate[rows], saved.up[rows])
    check_forward(part, y[rows], kept, moe)
    want, _, _ = part.plain_backward(moe, kept)
    assert plain.rel_rms(d_x[rows], want["d_x"]) <= REL_RMS_TOL
    assert plain.rel_rms(d_gates[rows], want["d_gates"]) <= 2e-5


def test_an_expert_twice_for_a_token(moe):
    """Two slots of one token at the same expert: both count."""
    case = Case(50, 4, 2, 256, 256, seed=19)
    idx = torch.stack([torch.arange(50, device="cuda") % 4] * 2, 1).to(torch.int32).contiguous()
    _, case.offsets, case.perm, case.inv = moe.moe_permute(idx, 4)
    case.tokens = case.perm.long() // 2
    y, saved = case.forward(moe)
    check_forward(case, y, saved, moe)
    check_backward(case, case.backward(moe, saved), saved, moe)


def test_two_calls_at_once(moe):
    """Two steps on two streams, each with its own workspaces."""
    cases = [Case(600, 8, 2, 512, 256, seed=20), Case(50, 8, 2, 512, 256, seed=21)]
    want = []
    for c in cases:
        y, saved = c.forward(moe)
        want.append((y, *c.backward(moe, saved)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            y, saved = c.forward(moe, stream=s)
            got.append((y, *c.backward(moe, saved, stream=s)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_calls_that_follow_one_another_on_one_workspace(moe):
    """Kernels may start while the one before finishes: calls of different
    sizes in a row, without a pause, give the bits of calls alone."""
    cases = [Case(700, 1, 1, 512, 256, seed=22, dense=True), Case(33, 1, 1, 512, 256, seed=23, dense=True),
             Case(300, 6, 2, 512, 256, seed=24), Case(40, 6, 2, 512, 256, seed=25)]
    wf = moe.Workspace(max(moe.expert_ffn_train_workspace_size(moe.Shape(*c.sizes)) for c in cases))
    wb = moe.Workspace(max(moe.expert_ffn_backward_workspace_size(moe.Shape(*c.sizes)) for c in cases))
    want = []
    for c in cases:
        y, saved = c.forward(moe, "fp8", ws=wf)
        want.append((y, *(v for v in c.backward(moe, saved, ws=wb))))
        torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for c in cases:
            y, saved = c.forward(moe, "fp8", ws=wf)
            got.append((y, *c.backward(moe, saved, ws=wb)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    assert wf.status() == 0 and wb.status() == 0


def test_no_token(moe):
    case = Case(0, 4, 2, 256, 256)
    y, saved = case.forward(moe)
    assert y.shape == (0, 256) and saved.gate.shape == (0, 256)
    dW = tuple(torch.full_like(w, float("nan")) for w in case.W)
    d_x, d_gates, *_ = case.backward(moe, saved, dW=dW)
    assert d_x.shape == (0, 256) and d_gates.shape == (0, 2)
    assert all((w == 0).all() for w in dW)


@pytest.mark.parametrize("T,dense", [(50, False), (333, False), (333, True)])
def test_only_what_is_needed(moe, T, dense):
    """x alone (frozen experts), the weights alone, neither: the same bits."""
    case = Case(T, 1 if dense else 6, 1 if dense else 3, 256, 512, seed=4, dense=dense)
    _, saved = case.forward(moe)
    whole = case.backward(moe, saved)
    only_x = case.backward(moe, saved, need_weights=False)
    assert torch.equal(only_x[0], whole[0]) and torch.equal(only_x[1], whole[1]) and only_x[2:] == (None,) * 3
    only_w = case.backward(moe, saved, need_x=False)
    assert only_w[0] is None and all(torch.equal(a, b) for a, b in zip(only_w[1:], whole[1:]))
    case.gates = None
    no_gates = case.backward(moe, saved)
    assert no_gates[1] is None
    check_backward(case, no_gates, saved, moe)


def test_repeated_runs_give_the_same_bits(moe):
    case = Case(700, 12, 4, 512, 512, seed=5)
    runs = []
    for _ in range(3):
        y, saved = case.forward(moe, "fp8")
        runs.append((y, saved.gate.view(torch.uint8), saved.up.view(torch.uint8), saved.gate_scales, *case.backward(moe, saved)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_rows_outside_are_left_alone(moe):
    case = Case(100, 1, 1, 256, 256, seed=6, dense=True)
    room = lambda n: torch.full((140, n), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y, g, u, dx = room(256), room(256), room(256), room(256)
    saved = moe.SavedFfn(case.x, g[20:120], u[20:120])
    out, saved = case.forward(moe, y_sorted=y[20:120], saved=saved)
    check_forward(case, out, saved, moe)
    check_backward(case, case.backward(moe, saved, d_x=dx[20:120]), saved, moe)
    for v in (y, g, u, dx):
        assert (v[:20] == 7).all() and (v[120:] == 7).all()


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
def test_values_that_are_not_finite_stay_with_their_rows(moe, checkpoint):
    """NaN and infinities of one token reach its own rows and the gradients of
    its experts' matrices, no other token."""
    case = Case(300, 6, 2, 256, 256, seed=7)
    clean, kept = case.forward(moe, checkpoint)
    grads = case.backward(moe, kept)
    bad = 17
    case.x[bad, 3] = float("inf")
    case.x[bad, 9] = float("nan")
    y, saved = case.forward(moe, checkpoint)
    mine = case.tokens == bad
    assert torch.equal(y[~mine], clean[~mine]) and not torch.isfinite(y[mine]).any()
    values_of = [v[~mine] for v in values(moe, saved)[1:]]
    assert all(torch.equal(a, b[~mine]) for a, b in zip(values_of, values(moe, kept)[1:]))
    d_x, d_gates, *_ = case.backward(moe, saved)
    others = torch.arange(300, device="cuda") != bad
    assert torch.equal(d_x[others], grads[0][others]) and torch.equal(d_gates[others], grads[1][others])
    assert not torch.isfinite(d_x[bad]).any()


def test_infinities_of_an_8bit_block_become_nan_and_leave_its_scale(moe):
    """x finite, a projection that overflows to infinity: NaN there, the block's
    other values as they are."""
    case = Case(40, 1, 1, 256, 256, seed=8, dense=True)
    case.x[5].fill_(1e30)
    case.W[0][0, 7].fill_(3e38)
    _, saved = case.forward(moe, "fp8")
    p = case.plain_forward()
    assert torch.isnan(saved.gate[5, 7].float()) and torch.isfinite(saved.gate[5, 8:].float()).all()
    got = fp8_plain.rows_value(saved.gate, saved.gate_scales)[5, 128:]
    assert ((got - p["g"][5, 128:]).abs() <= 2.0 ** -4 * p["g"][5, 128:].abs() * (1 + 2 ** -10) + 2.0 ** -9 * p["g"][5, 128:].abs().max()).all()
    # the block of the infinity: its scale is that of its finite values
    finite = p["g"][5, :128].clone()
    finite[7] = 0
    want = fp8_plain.scale_bytes(finite.abs().amax())
    assert abs(int(saved.gate_scales[5, 0]) - int(want)) <= 1


@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
@pytest.mark.parametrize("sizes,dense", [((37, 9, 3, 256, 256), False), ((700, 5, 2, 512, 256), False),
                                         ((301, 1, 1, 256, 512), True), ((21, 1, 1, 256, 256), True)], ids=str)
def test_nothing_of_a_workspace_is_read_before_it_is_written(moe, sizes, dense, checkpoint):
    case = Case(*sizes, seed=18, dense=dense)
    wf = moe.Workspace(moe.expert_ffn_train_workspace_size(moe.Shape(*sizes)))
    wb = moe.Workspace(moe.expert_ffn_backward_workspace_size(moe.Shape(*sizes)))
    wf.tensor[256:].fill_(0xff)          # NaN, in bf16 and fp32
    wb.tensor[256:].fill_(0xff)
    y, saved = case.forward(moe, checkpoint, ws=wf)
    check_forward(case, y, saved, moe)
    check_backward(case, case.backward(moe, saved, ws=wb), saved, moe)


@pytest.mark.parametrize("rows,K", [(1, 128), (7, 384), (300, 2048), (5, 16384)])
def test_dequantize_rows(moe, rows, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    q = torch.randint(0, 256, (rows, K), generator=g, device="cuda").to(torch.uint8)
    b = torch.randint(20, 230, (rows, K // 128), generator=g, device="cuda").to(torch.uint8)
    b[0, 0] = 255                                   # stands for NaN
    x = moe.moe_dequantize_rows(q.view(torch.float8_e4m3fn), b)
    want = fp8_plain.rows_value(q.view(torch.float8_e4m3fn), b)
    want[0, :128] = float("nan")
    assert torch.equal(torch.isnan(x), torch.isnan(want))
    assert torch.equal(x.double().nan_to_num(3.0), want.nan_to_num(3.0))


def test_a_checkpoint_and_its_quantised_rows_agree(moe):
    """x's checkpoint is what moe_quantize_rows gives; moe_dequantize_rows reads both."""
    case = Case(77, 4, 2, 512, 256, seed=9)
    _, saved = case.forward(moe, "fp8")
    q, s = moe.moe_quantize_rows(case.x)
    assert torch.equal(q.view(torch.uint8), saved.x.view(torch.uint8)) and torch.equal(s, saved.x_scales)
    assert torch.equal(moe.moe_dequantize_rows(q, s).double(), values(moe, saved)[0])


# ---- gradients against differences --------------------------------------------

def loss(case, x, gates, W):
    """sum d_out . out in 64 bits, out = the layer's sum over slots of gate * y."""
    T, E, k, H, I = case.sizes
    y = plain.forward(x, case.tokens, case.offsets, *W)["y"]
    slot = case.perm.long() if case.perm is not None else torch.arange(T * k, device="cuda")
    w = gates.double().flatten()[slot]
    return (case.d_out.double()[case.tokens] * y * w[:, None]).sum()


@pytest.mark.parametrize("sizes,dense", [((60, 5, 2, 256, 256), False), ((90, 1, 1, 256, 512), True)], ids=str)
def test_gradients_against_differences(moe, sizes, dense):
    """Along each gradient v that the kernel gives, the loss rises by |v|^2 per
    step.  <g, v> differs from |v|^2 by at most |g - v| |v|: the rounding of the
    gradient's operands and of itself (5e-3 of the norm, above) and of the kept
    projections (2^-8 each, through slopes of at most 1.1: 1e-2 in all).  A
    central difference over 2^-10 of the tensor's norm is off by its third
    order, some 2^-20."""
    case = Case(*sizes, seed=10, dense=dense)
    _, saved = case.forward(moe)
    d_x, d_gates, *dW = case.backward(moe, saved)
    at = dict(x=case.x.double(), gates=case.gates.double(), W=[w.double() for w in case.W])
    for name, i, v in (("x", None, d_x), ("gates", None, d_gates), *(("W", i, w) for i, w in enumerate(dW))):
        v = v.double()
        base = at[name] if i is None else at[name][i]
        step = 2.0 ** -10 * base.norm() / v.norm()
        sides = []
        for s in (step, -step):
            moved = {**at, "W": list(at["W"])}
            if i is None:
                moved[name] = base + s * v
            else:
                moved["W"][i] = base + s * v
            sides.append(loss(case, moved["x"], moved["gates"], moved["W"]))
        slope = ((sides[0] - sides[1]) / (2 * step)).item()
        assert abs(slope / v.square().sum().item() - 1) <= 1e-2, (name, i)


# ---- streams, graphs, expired waits -------------------------------------------

def test_another_stream_and_a_graph(moe):
    case = Case(500, 7, 3, 512, 256, seed=11)
    S = moe.Shape(*case.sizes)
    y0, saved0 = case.forward(moe, "fp8")
    want = (y0, *case.backward(moe, saved0))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, saved = case.forward(moe, "fp8", stream=s)
    got = (y, *case.backward(moe, saved, stream=s))
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a step captured once and replayed on other inputs
    wf, wb = moe.Workspace(moe.expert_ffn_train_workspace_size(S)), moe.Workspace(moe.expert_ffn_backward_workspace_size(S))
    y, saved = case.forward(moe, "fp8", ws=wf)
    out = case.backward(moe, saved, ws=wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        case.forward(moe, "fp8", ws=wf, y_sorted=y, saved=saved)
        case.backward(moe, saved, ws=wb, d_x=out[0], d_gates=out[1], dW=out[2:])
    other = Case(500, 7, 3, 512, 256, seed=12)
    for a, b in ((case.x, other.x), (case.d_out, other.d_out), (case.gates, other.gates), (case.perm, other.perm),
                 (case.offsets, other.offsets), (case.inv, other.inv)):
        a.copy_(b)
    case.tokens = other.tokens
    graph.replay()
    torch.cuda.synchronize()
    assert wf.status() == 0 and wb.status() == 0
    check_forward(case, y, saved, moe)
    check_backward(case, out, saved, moe)


def test_a_record_used_twice(moe):
    """saved= of an earlier call is written anew; a bf16 record is of its own x."""
    a, b = Case(90, 4, 2, 256, 256, seed=13), Case(90, 4, 2, 256, 256, seed=14)
    for kind in ("bf16", "fp8"):
        _, room = a.forward(moe, kind)
        y, saved = b.forward(moe, saved=room)
        check_forward(b, y, saved, moe)
        check_backward(b, b.backward(moe, saved), saved, moe)


def test_skipped_routed_index(moe):
    """A routed index outside the experts: recorded, the other tokens' results are right."""
    T, E, k, H, I = 70, 5, 2, 256, 256
    case = Case(T, E, k, H, I, seed=15)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).to(torch.int32)
    idx[8, 1] = 77
    pws = moe.Workspace(moe.permute_workspace_size(T, E, k))
    full = (torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(E + 1, dtype=torch.int32, device="cuda"),
            torch.full((T * k,), -1, dtype=torch.int32, device="cuda"), torch.full((T * k,), -1, dtype=torch.int32, device="cuda"))
    _, case.offsets, case.perm, case.inv = moe.moe_permute(idx, E, ws=pws, out=full)
    assert pws.status() == MOE_ERR_BAD_INDEX
    wf = moe.Workspace(moe.expert_ffn_train_workspace_size(moe.Shape(T, E, k, H, I)))
    wf.tensor[256:].fill_(0xff)
    y, saved = case.forward(moe, ws=wf)
    wb = moe.Workspace(moe.expert_ffn_backward_workspace_size(moe.Shape(T, E, k, H, I)))
    wb.tensor[256:].fill_(0xff)                             # NaN wherever a buffer is read before it is written
    d_x, d_gates, *dW = case.backward(moe, saved, ws=wb)
    assert wf.status() == 0 and wb.status() == 0           # the route lists' call recorded it
    n = T * k - 1                                           # the last position holds no slot
    slot = case.perm[:n].long()
    off = case.offsets.clone()
    off[-1] = n
    p = plain.forward(case.x, slot // k, off, *case.W)
    assert plain.rel_rms(y[:n], p["y"]) <= REL_RMS_TOL
    others = torch.arange(T, device="cuda") != 8
    # the plain form with the skipped slot in the last position and without weight
    perm = torch.cat([slot, torch.tensor([8 * k + 1], device="cuda")]).to(torch.int32)
    gates = case.gates.clone()
    gates[8, 1] = 0
    want, _, _ = plain.backward(case.d_out, gates, case.x, saved.gate, saved.up, perm, case.offsets, k, *case.W)
    assert plain.rel_rms(d_x[others], want["d_x"][others]) <= REL_RMS_TOL
    assert plain.rel_rms(d_gates[others], want["d_gates"][others]) <= 2e-5
    for a, b in zip(dW, (want["dWg"], want["dWu"], want["dWd"])):
        assert plain.rel_rms(a, b) <= REL_RMS_TOL


@pytest.mark.parametrize("sizes,dense", [((64, 16, 2, 512, 256), False), ((1000, 4, 2, 512, 512), False),
                                         ((700, 1, 1, 2048, 512), True)], ids=str)
@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
def test_waits_that_expire_leave_nothing_behind(moe, sizes, dense, checkpoint):
    case = Case(*sizes, seed=16, dense=dense)
    S = moe.Shape(*sizes)
    wf, wb = moe.Workspace(moe.expert_ffn_train_workspace_size(S)), moe.Workspace(moe.expert_ffn_backward_workspace_size(S))
    want, saved = case.forward(moe, checkpoint, ws=wf)
    grads = case.backward(moe, saved, ws=wb)
    outs = []
    for _ in range(6):
        moe.debug_set_wait_limit(1)
        try:
            _, junk = case.forward(moe, checkpoint, ws=wf)
            case.backward(moe, junk, ws=wb)
        finally:
            moe.debug_set_wait_limit(0)
        y, again = case.forward(moe, checkpoint, ws=wf)
        outs.append((y, *case.backward(moe, again, ws=wb)))
    torch.cuda.synchronize()
    assert wf.status(clear=True) == MOE_ERR_TIMEOUT and wb.status(clear=True) == MOE_ERR_TIMEOUT
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, (want, *grads)))


# ---- a training step of the layer -----------------------------------------------

@pytest.mark.parametrize("checkpoint", ["bf16", "fp8"])
def test_a_training_step(moe, checkpoint):
    """Router (product with bias, fp32), route, route lists, experts, combine,
    a shared expert whose output takes the routed one as its residual, balance
    loss; and back to every gradient.  Against the same in 64 bits, with the
    routing and the kept values that the step itself chose."""
    T, E, k, H, I = 700, 12, 3, 512, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(17)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, d_out = randn(T, H).to(torch.bfloat16), randn(T, H).to(torch.bfloat16)
    R, bias = (randn(1, E, H) * H ** -0.5).to(torch.bfloat16), randn(1, E)
    W = tuple((randn(*s) * s[2] ** -0.5).to(torch.bfloat16) for s in ((E, I, H), (E, I, H), (E, H, I)))
    SW = tuple((randn(*s) * s[2] ** -0.5).to(torch.bfloat16) for s in ((1, I, H), (1, I, H), (1, H, I)))
    S, D = moe.Shape(T, E, k, H, I), moe.Shape(T, 1, 1, H, I)
    logits = moe.moe_grouped_gemm(x, R, bias=bias, out_dtype=torch.float32)
    idx, gates = moe.moe_route(logits, k)
    balance, counts, stats = moe.moe_balance(logits, idx, None, 0.01)
    _, offsets, perm, inv = moe.moe_permute(idx, E)
    y, saved = moe.moe_expert_ffn_train(S, x, perm, offsets, *W, checkpoint=checkpoint)
    routed = moe.moe_combine(y, inv, gates, T, k, H)
    shared, saved_d = moe.moe_expert_ffn_train(D, x, None, None, *SW, checkpoint=checkpoint)
    out = moe.moe_grouped_gemm(shared, torch.eye(H, device="cuda", dtype=torch.bfloat16)[None], residual=routed)
    d_x, d_gates, *dW = moe.moe_expert_ffn_backward(S, d_out, saved, perm, offsets, inv, *W, gates=gates)
    d_xs, none, *dSW = moe.moe_expert_ffn_backward(D, d_out, saved_d, None, None, None, *SW)
    d_logits = moe.moe_balance_backward(logits, stats, counts, k, None, 0.01, topk_idx=idx, gates=gates, d_gates=d_gates)
    torch.cuda.synchronize()
    assert none is None
    # forward
    lw, _, mag = plain.product(x, R, None, bias, "none", None)
    assert ((logits.double() - lw).abs() <= (H + 1) * plain.ADD * mag).all()
    tokens = perm.long() // k
    p = plain.forward(x, tokens, offsets, *W)["y"]
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    want.index_add_(0, tokens, p * gates.double().flatten()[perm.long()][:, None])
    ps = plain.forward(x, torch.arange(T, device="cuda"), None, *SW)["y"]
    # roundings: h, y, out of each block, the sum: 4, 1.7e-3 each
    assert plain.rel_rms(out, want + ps) <= REL_RMS_TOL
    # backward
    for got, (r, _, _) in (((d_x, d_gates, *dW), plain.backward(d_out, gates, *values(moe, saved), perm, offsets, k, *W)),
                           ((d_xs, None, *dSW), plain.backward(d_out, None, *values(moe, saved_d), None, None, 1, *SW))):
        for n, v in zip(("d_x", "d_gates", "dWg", "dWu", "dWd"), got):
            if v is not None:
                assert plain.rel_rms(v, r[n]) <= (2e-5 if n == "d_gates" else REL_RMS_TOL), n
    gd, dg = gates.double(), d_gates.double()
    l = logits.double().requires_grad_()
    f = counts.double()[0] * E / (k * T)
    loss_plain = 0.01 * (torch.softmax(l, 1).mean(0) * f).sum()
    loss_plain.backward()
    ref = l.grad.scatter_add(1, idx.long(), gd * (dg - (gd * dg).sum(1, keepdim=True)))
    assert abs(balance.item() - loss_plain.item()) <= 1e-6 * loss_plain.item() + 1e-9
    assert plain.rel_rms(d_logits, ref) <= 1e-5
