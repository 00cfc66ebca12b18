"""SwiGLU with 8-bit checkpoints, forward and backward, against 64-bit plain
forms; codes and scales bit for bit."""
import pytest
import torch

from _train_ref import BF16_HALF, quantize64, restore64, swiglu64, swiglu_backward64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# Sixteen fp32 roundings: exponential, quotient (2 units each), sum and products.
ARITH = 2.0 ** -19
# Quotients 1 / (1 + exp(-g)) under 2^-126 may come out as zero.
TINY = 1e-35


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routed_expert_b200 as m
    return m


def _gate_up(rows, F, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, 2 * F, generator=g) * std).to(BF), g


def _near(got, ref, tol, what):
    off = (got.double().cpu() - ref).abs()
    assert not (off > tol + TINY).any(), "%s: worst %.3e of the tolerance" % (what, float((off / (tol + TINY)).max()))


@pytest.mark.parametrize("rows,F", [(1, 128), (3, 384), (96, 896), (257, 2048), (1030, 128), (2, 16384)])
@pytest.mark.parametrize("weighted", [False, True])
def test_forward(moe, cuda_dev, rows, F, weighted):
    gu, g = _gate_up(rows, F, 1)
    gu[0, :5] = torch.tensor([0.0, -0.0, 100.0, -100.0, 1e-30])
    gu[rows - 1, 128 * (2 * F // 128 - 1):] = 0                      # a block of zeros
    p = torch.rand(rows, generator=g) if weighted else None
    h, codes, scale = moe.moe_swiglu_checkpoint(gu.to(cuda_dev), None if p is None else p.to(cuda_dev))
    assert h.dtype == BF and codes.dtype == torch.uint8 and scale.dtype == F32
    q, s = quantize64(gu)
    assert torch.equal(scale.cpu().double(), s)
    assert torch.equal(codes.cpu().view(torch.float8_e4m3fn).double(), q)
    ref = swiglu64(gu, p)
    _near(h, ref, (BF16_HALF + ARITH) * ref.abs(), "h")
    xq, xs = moe.quantize_fp8_block128(gu.to(cuda_dev))              # the same rule
    assert torch.equal(xq, codes) and torch.equal(xs, scale)


@pytest.mark.parametrize("rows,F", [(1, 128), (3, 384), (96, 896), (257, 2048), (1030, 128), (2, 16384)])
@pytest.mark.parametrize("weighted", [False, True])
def test_backward(moe, cuda_dev, rows, F, weighted):
    gu, g = _gate_up(rows, F, 2)
    dh = torch.randn(rows, F, generator=g).to(BF)
    p = torch.rand(rows, generator=g) if weighted else None
    _, codes, scale = moe.moe_swiglu_checkpoint(gu.to(cuda_dev))
    r = restore64(codes.cpu(), scale.cpu())
    args = (codes, scale, dh.to(cuda_dev), None if p is None else p.to(cuda_dev))
    dgu, h, dp = moe.moe_swiglu_checkpoint_backward(*args)
    rdgu, rh, rdp = swiglu_backward64(r, dh, p)
    _near(h, rh, (BF16_HALF + ARITH) * rh.abs(), "h")
    gate, up = r.chunk(2, 1)
    s = torch.sigmoid(gate)
    q = (torch.ones(rows, 1) if p is None else p[:, None]).double() * dh.double().abs()
    mag = torch.cat([q * up.abs() * (s + (gate * s).abs()), q * (gate * s).abs()], 1)   # before the sum s + a (1 - s)
    _near(dgu, rdgu, BF16_HALF * rdgu.abs() + 2 * ARITH * mag, "dgate_up")
    terms = (dh.double() * gate * s * up).abs().sum(1)
    _near(dp, rdp, terms * (ARITH + F * 2.0 ** -23), "drow_weights")
    again = moe.moe_swiglu_checkpoint_backward(*args)
    assert all(torch.equal(a, b) for a, b in zip(again, (dgu, h, dp)))
    only, no_h, no_dp = moe.moe_swiglu_checkpoint_backward(*args, want_h=False, want_drow_weights=False)
    assert torch.equal(only, dgu) and no_h is None and no_dp is None
    f8 = moe.moe_swiglu_checkpoint_backward(codes.view(torch.float8_e4m3fn), *args[1:])
    assert torch.equal(f8[0], dgu)


def test_backward_against_differences(moe, cuda_dev):
    """The gradients are the slope of the forward: central differences of the
    64-bit forward at the restored activations, in a random direction."""
    rows, F = 5, 256
    gu, g = _gate_up(rows, F, 3)
    dh = torch.randn(rows, F, generator=g).to(BF)
    p = torch.rand(rows, generator=g) + 0.5
    _, codes, scale = moe.moe_swiglu_checkpoint(gu.to(cuda_dev))
    r = restore64(codes.cpu(), scale.cpu())
    dgu, _, dp = moe.moe_swiglu_checkpoint_backward(codes, scale, dh.to(cuda_dev), p.to(cuda_dev))
    v = torch.randn(rows, 2 * F, generator=g, dtype=torch.float64)
    eps = 1e-5
    slope = ((swiglu64(r + eps * v, p) - swiglu64(r - eps * v, p)) * dh.double()).sum() / (2 * eps)
    got = (dgu.double().cpu() * v).sum()
    # each product carries a bf16 rounding; the difference quotient's own error (eps^2) is far below
    tol = (dgu.double().cpu() * v).abs().sum() * (BF16_HALF + 2.0 ** -16)
    assert (got - slope).abs() <= tol
    one = torch.ones(rows, dtype=torch.float64)    # in fp32 1 + eps would itself be off by 1e-3 of eps
    slope_p = ((swiglu64(r, one + eps) - swiglu64(r, one - eps)) * dh.double()).sum(1) / (2 * eps)
    assert (dp.double().cpu() - slope_p).abs().max() <= 1e-5 * (dh.double().abs() * swiglu64(r).abs()).sum(1).max()


@pytest.mark.parametrize("live", [0, 1, 33, 50, 51, -7, 1000])
def test_rows_behind_the_count_stay(moe, cuda_dev, live):
    rows, F = 51, 256
    gu, g = _gate_up(rows, F, 4)
    dh = torch.randn(rows, F, generator=g).to(BF).to(cuda_dev)
    gd = gu.to(cuda_dev)
    n = torch.tensor([3, live], dtype=torch.int32, device=cuda_dev)[1:]
    full = moe.moe_swiglu_checkpoint(gd)
    outs = [torch.full_like(t, 7) for t in full]
    moe.moe_swiglu_checkpoint(gd, n_rows=n, h=outs[0], codes=outs[1], scale=outs[2])
    k = min(max(live, 0), rows)
    for o, f in zip(outs, full):
        assert torch.equal(o[:k], f[:k]) and (o[k:] == 7).all()
    fullb = moe.moe_swiglu_checkpoint_backward(full[1], full[2], dh)
    outs = [torch.full_like(t, 7) for t in fullb]
    moe.moe_swiglu_checkpoint_backward(full[1], full[2], dh, n_rows=n, dgate_up=outs[0], h=outs[1],
                                       drow_weights=outs[2])
    for o, f in zip(outs, fullb):
        assert torch.equal(o[:k], f[:k]) and (o[k:] == 7).all()


def test_values_at_the_ends(moe, cuda_dev):
    """The largest and smallest finite values keep the quantiser's rule; an
    infinity is restored as one and a NaN as one, in its own block alone."""
    F = 256
    gu, _ = _gate_up(3, F, 5)
    gu[0, 3], gu[0, 140] = 3.3895313892515355e38, 9.2e-41           # the largest bf16, a subnormal
    gu[0, 256:384] = 0
    gu[0, 300] = 9.2e-41                                             # alone in its block
    gu[1, 7], gu[1, 300], gu[1, 301] = float("inf"), float("-inf"), 3.3895313892515355e38
    gu[2, 9] = float("nan")
    h, codes, scale = moe.moe_swiglu_checkpoint(gu.to(cuda_dev))
    q, s = quantize64(gu[:1])
    assert torch.equal(scale[:1].cpu().double(), s)
    assert torch.equal(codes[:1].cpu().view(torch.float8_e4m3fn).double(), q)
    back = (codes.cpu().view(torch.float8_e4m3fn).float().view(3, -1, 128) * scale.cpu()[:, :, None]).view(3, -1)
    assert back[1, 7] == float("inf") and back[1, 300] == float("-inf")
    # 1.992 * 2^127 = 255 * 2^120 lies nearest to the code 256, and 256 * 2^120 = 2^128 overflows
    assert back[1, 301] == float("inf")
    assert torch.isnan(back[2, 9]) and torch.isfinite(back[2]).sum() == 2 * F - 1
    clean = torch.ones(2 * F, dtype=torch.bool)
    clean[:128] = clean[256:384] = False
    q1, s1 = quantize64(gu[1:2, clean])
    assert torch.equal(back[1:2, clean].double(), (q1.unflatten(1, (-1, 128)) * s1.unsqueeze(2)).flatten(1))
    dh = torch.ones(3, F, dtype=BF, device=cuda_dev)
    dgu, hb, _ = moe.moe_swiglu_checkpoint_backward(codes, scale, dh)
    assert torch.isfinite(dgu[:1, 128:256]).all() and torch.isfinite(hb[2]).sum() == F - 1
    assert torch.isfinite(h[2]).sum() == F - 1


def test_graph_and_stream(moe, cuda_dev):
    gu, g = _gate_up(40, 384, 6)
    gd = gu.to(cuda_dev)
    dh = torch.randn(40, 384, generator=g).to(BF).to(cuda_dev)

    def call(stream=None):
        h, c, s = moe.moe_swiglu_checkpoint(gd, stream=stream)
        return (h, c, s) + moe.moe_swiglu_checkpoint_backward(c, s, dh, stream=stream)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = call()
    gd.neg_()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(side)
    torch.cuda.synchronize()
    for a, b in zip(caught, other):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(moe, cuda_dev):
    rows, F = 70000, 16384                                   # gate_up: 2.3e9 elements
    last = 64
    gu = torch.zeros(rows, 2 * F, dtype=BF, device=cuda_dev)
    tail, g = _gate_up(last, F, 7)
    gu[-last:] = tail.to(cuda_dev)
    h, codes, scale = moe.moe_swiglu_checkpoint(gu)
    del gu
    q, s = quantize64(tail)
    assert torch.equal(scale[-last:].cpu().double(), s)
    assert torch.equal(codes[-last:].cpu().view(torch.float8_e4m3fn).double(), q)
    ref = swiglu64(tail)
    _near(h[-last:], ref, (BF16_HALF + ARITH) * ref.abs(), "h")
    assert (h[:1000] == 0).all() and (codes[:1000] == 0).all() and (scale[:1000] == 1).all()
    dh = torch.zeros(rows, F, dtype=BF, device=cuda_dev)
    d = torch.randn(last, F, generator=g).to(BF)
    dh[-last:] = d.to(cuda_dev)
    del h
    dgu, hb, dp = moe.moe_swiglu_checkpoint_backward(codes, scale, dh)
    _, rh, _ = swiglu_backward64(restore64(codes[-last:].cpu(), scale[-last:].cpu()), d)
    _near(hb[-last:], rh, (BF16_HALF + ARITH) * rh.abs(), "h")
    assert (dgu[:1000] == 0).all() and (dp[:-last] == 0).all() and (dgu[-last:] != 0).float().mean() > 0.9


@pytest.mark.parametrize("rows,F", [(1300, 128), (1301, 256), (1300, 384), (1300, 896), (2100, 1152), (7300, 896)])
def test_rows_beyond_one_round(moe, cuda_dev, rows, F):
    """Half a warp, one and four on a row, several rows a block: the same formulas."""
    test_forward(moe, cuda_dev, rows, F, True)
    test_backward(moe, cuda_dev, rows, F, True)
