"""Rows to expert order and back: exact copies, and sums whose fp32 order is
fixed and therefore comparable bit for bit."""
import pytest
import torch

from _train_ref import expert_order, restore64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routed_expert_b200 as m
    return m


def _routing(T, K, E, seed, dropped=0.2):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, E, (T, K), generator=g)
    idx[torch.rand(T, K, generator=g) < dropped] = -1
    return idx, g


SIZES = [(1, 1, 8), (1, 8, 128), (5, 16, 1288), (130, 6, 1280), (33, 3, 7168), (700, 2, 24), (2, 2, 65536)]


def _permute_ref(x, inv, n, weights):
    out = torch.full((n, x.shape[1]), 9.0, dtype=BF)
    rw = torch.full((n,), 9.0)
    for t in range(inv.shape[0]):
        for k in range(inv.shape[1]):
            p = int(inv[t, k])
            if 0 <= p < n:
                out[p], rw[p] = x[t], weights[t, k]
    return out, rw


def _unpermute_ref(y, inv, residual):
    T, K = inv.shape
    acc = torch.zeros(T, y.shape[1], dtype=F32)
    for k in range(K):
        for t in range(T):
            p = int(inv[t, k])
            if 0 <= p < y.shape[0]:
                acc[t] += y[p].float()
    if residual is not None:
        acc = acc + residual.float()
    return acc.to(BF)


@pytest.mark.parametrize("T,K,H", SIZES)
def test_permute(moe, cuda_dev, T, K, H):
    idx, g = _routing(T, K, 7, T)
    _, inv = expert_order(idx, 7)
    x = torch.randn(T, H, generator=g).to(BF)
    w = torch.rand(T, K, generator=g)
    n = T * K + 3
    ref, rw = _permute_ref(x, inv, n, w)
    out = torch.full((n, H), 9.0, dtype=BF, device=cuda_dev)
    row = torch.full((n,), 9.0, device=cuda_dev)
    moe.moe_permute_rows(x.to(cuda_dev), inv.to(cuda_dev), w.to(cuda_dev), out=out, row_weights=row)
    assert torch.equal(out.cpu(), ref) and torch.equal(row.cpu(), rw)
    plain = moe.moe_permute_rows(x.to(cuda_dev), inv.to(cuda_dev))
    kept = int((inv >= 0).sum())
    assert plain.shape == (T * K, H) and torch.equal(plain[:kept].cpu(), ref[:kept])


@pytest.mark.parametrize("T,K,H", [(1, 1, 128), (5, 16, 1280), (33, 3, 7168)])
def test_permute_from_codes(moe, cuda_dev, T, K, H):
    idx, g = _routing(T, K, 7, T)
    _, inv = expert_order(idx, 7)
    x = (torch.randn(T, H, generator=g) * torch.logspace(-6, 6, H)).to(BF)
    codes, scale = moe.quantize_fp8_block128(x.to(cuda_dev))
    r = restore64(codes.cpu(), scale.cpu()).to(BF)
    ref, _ = _permute_ref(r, inv, T * K, torch.zeros(T, K))
    kept = int((inv >= 0).sum())
    for c in (codes, codes.view(torch.float8_e4m3fn)):
        out = moe.moe_permute_rows(c, inv.to(cuda_dev), x_scale=scale)
        assert torch.equal(out[:kept].cpu(), ref[:kept])


@pytest.mark.parametrize("T,K,H", SIZES)
@pytest.mark.parametrize("dt", [BF, F32])
def test_unpermute(moe, cuda_dev, T, K, H, dt):
    idx, g = _routing(T, K, 7, T + 1)
    _, inv = expert_order(idx, 7)
    y = torch.randn(T * K, H, generator=g).to(dt)
    y[int((inv >= 0).sum()):] = float("nan")                 # rows of nobody
    res = torch.randn(T, H, generator=g).to(BF)
    drow = torch.randn(T * K, generator=g)
    for r in (None, res):
        out = moe.moe_unpermute_rows(y.to(cuda_dev), inv.to(cuda_dev), None if r is None else r.to(cuda_dev))
        assert torch.equal(out.cpu(), _unpermute_ref(y, inv, r))
    out, dw = moe.moe_unpermute_rows(y.to(cuda_dev), inv.to(cuda_dev), res.to(cuda_dev), drow.to(cuda_dev))
    assert torch.equal(out.cpu(), _unpermute_ref(y, inv, res))
    assert torch.equal(dw.cpu(), torch.where(inv >= 0, drow[inv.clamp_min(0).long()], torch.zeros(T, K)))


def test_positions_outside_are_skipped(moe, cuda_dev):
    """Positions behind the buffers (a capacity smaller than the routing) are
    skipped, like negative ones; a shared row sums into each of its tokens."""
    inv = torch.tensor([[0, 5], [2 ** 31 - 1, 1], [-2 ** 31, 4], [1, 1]], dtype=torch.int32)
    x = torch.randn(4, 64, generator=torch.Generator().manual_seed(0)).to(BF)
    out = torch.full((5, 64), 9.0, dtype=BF, device=cuda_dev)
    moe.moe_permute_rows(x[:3].to(cuda_dev), inv[:3].to(cuda_dev).contiguous(), out=out)
    ref = torch.full((5, 64), 9.0, dtype=BF)
    ref[0], ref[1], ref[4] = x[0], x[1], x[2]
    assert torch.equal(out.cpu(), ref)
    y = torch.randn(5, 64, generator=torch.Generator().manual_seed(1))
    assert torch.equal(moe.moe_unpermute_rows(y.to(cuda_dev), inv.to(cuda_dev)).cpu(), _unpermute_ref(y, inv, None))


def test_empty(moe, cuda_dev):
    inv = torch.full((4, 2), -1, dtype=torch.int32, device=cuda_dev)
    y = torch.empty(0, 64, dtype=BF, device=cuda_dev)
    assert (moe.moe_unpermute_rows(y, inv) == 0).all()
    out, dw = moe.moe_unpermute_rows(y, inv, drow_weights=torch.empty(0, device=cuda_dev))
    assert (out == 0).all() and (dw == 0).all()
    none = torch.empty(0, 2, dtype=torch.int32, device=cuda_dev)
    assert moe.moe_permute_rows(torch.empty(0, 64, dtype=BF, device=cuda_dev), none).shape == (0, 64)
    assert moe.moe_unpermute_rows(torch.ones(3, 64, dtype=BF, device=cuda_dev), none).shape == (0, 64)


def test_offsets_past_32_bits(moe, cuda_dev):
    """More than 2^31 elements on the expert-order side."""
    T, K, H = 9000, 16, 16384
    g = torch.Generator(device=cuda_dev).manual_seed(3)
    inv = torch.randperm(T * K, generator=g, device=cuda_dev).to(torch.int32).view(T, K)
    x = torch.randn(T, H, generator=g, device=cuda_dev).to(BF)
    rows = moe.moe_permute_rows(x, inv)
    for t in (0, 4500, T - 1):
        assert torch.equal(rows[inv[t].long()], x[t].expand(K, H))
    out = moe.moe_unpermute_rows(rows, inv)
    assert torch.equal(out, (x.float() * K).to(BF))         # 16 equal terms: every partial sum is exact in fp32
