"""The operators of a block of experts where their grids go round: several items, rows or tokens behind one another in a CTA or
a warp, and the widths that models have."""
import math

import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
import moe_ref as ref
import test_moe_gemm_gpu as gemm
import test_residual_rmsnorm_gpu as norm

pytestmark = pytest.mark.gpu


def counts_of(n, most, seed):
    """Ragged rows of n experts, some without any, some that fill their last tile."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, most, (n,), generator=g)
    c[::7] = 0
    c[1::9] = (c[1::9] + 127) // 128 * 128
    return c.tolist()


# ------------------------------------------------------------------ products

@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("counts, N, K", [
    (counts_of(40, 700, 1), 2048, 128),          # about 8 items a CTA, a block of K each
    (counts_of(60, 400, 2), 1792, 384),          # 7 (plain) and 9 items, an odd number of blocks
    ([1200, 3, 900, 130, 0, 1027, 2600], 2048, 2048)])   # about 3 items of 16 blocks
def test_many_items_a_cta(counts, N, K, gather):
    gemm.check(gemm.data(counts, 150, N, K, sum(counts), gather=gather, tail=5))


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("counts, N, K", [([300, 0, 128, 77], 4096, 7168), ([260, 513], 512, 14336), ([1] * 8, 2048, 7168),
                                          ([3, 0, 29], 256, 14336), ([0, 128, 5, 256], 14336, 4096)])
def test_the_widths_of_models(counts, N, K, gather):
    gemm.check(gemm.data(counts, 90, N, K, sum(counts) + K, gather=gather))


def test_beyond_32_rows_a_row_has_its_own_bits():
    """More than 32 rows: the order of a row's sums is that of K, whatever rows lie beside it."""
    d = gemm.data([70, 0, 50, 1, 300], 64, 768, 1024, 21)
    Y, H = qz.qz_moe_gemm_fp8(**d), qz.qz_moe_gemm_fp8_swiglu(**d)
    off = d["offsets"].tolist()
    for e, lo, n in ((0, 0, 33), (0, 37, 33), (2, 0, 50), (4, 3, 40), (4, 250, 50)):
        part = dict(d, row_token=d["row_token"][off[e] + lo:off[e] + lo + n].contiguous())
        part["offsets"] = torch.tensor([0 if i <= e else n for i in range(len(off))], dtype=torch.int32, device="cuda")
        at = slice(off[e] + lo, off[e] + lo + n)
        assert torch.equal(qz.qz_moe_gemm_fp8(**part), Y[at])
        assert all(torch.equal(a, b[at]) for a, b in zip(qz.qz_moe_gemm_fp8_swiglu(**part), H))


# ------------------------------------------------------------------ the residual norm

@pytest.mark.parametrize("T, H, k, post", [(5000, 128, 0, False), (20001, 128, 1, False), (2600, 1024, 0, False), (3001, 1024, 1, False),
                                           (400, 16384, 0, False), (317, 16384, 1, False), (1500, 4096, 0, True), (1300, 2048, 4, False)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [True, False])
def test_more_rows_than_the_grid(T, H, k, post, dt, block):
    """k = 1: one gated row a token, in order."""
    d = norm.data(T, H, k, dt, T + H)
    if not post:
        d["gamma_y"] = None
    if k == 1:
        d["token_row"] = None
    if not block:
        d.update(y=None, token_row=None, weights=None, gamma_y=None)
    got = norm.check(d, alpha=0.7, normed=True, fp8=True)
    x = d["x"].clone()
    again = qz.qz_residual_rmsnorm(x, d["gamma"], d["y"], d["token_row"], d["weights"], alpha=0.7, gamma_y=d["gamma_y"], out=x,
                                   normed=True, fp8=True)
    assert again[0] is x and all(torch.equal(a, b) for a, b in zip(got, again))


# ------------------------------------------------------------------ routing

def route_many(logits, k, sigmoid, renorm, scale=1.0, bias=None, groups=1, top_groups=1, group_best=1, n=None):
    """The definition over all tokens at once in 64 bits, for finite logits and biases: sorts that keep the order of the indices."""
    T, E = logits.shape
    n = T if n is None else n
    l = logits.double()
    p = torch.sigmoid(l) if sigmoid else torch.softmax(l, dim=1)
    key = p if bias is None else p + bias.double()
    rank = l if bias is None else key
    if groups > 1:
        best = torch.sort(key.view(T, groups, -1), dim=2, descending=True)[0][:, :, :group_best].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :top_groups]
        keep = torch.zeros((T, groups), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        rank = torch.where(keep.repeat_interleave(E // groups, dim=1), rank, -math.inf)
    ids = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :k]
    w = p.gather(1, ids)
    if renorm:
        w = w / w.sum(dim=1, keepdim=True)
    live = (torch.arange(T, device=l.device) < n)[:, None]
    ids, w = torch.where(live, ids, -1), torch.where(live, w * scale, 0.0)
    flat = torch.where(ids < 0, E, ids).reshape(-1)
    order = torch.sort(flat, stable=True)[1]
    offsets = torch.zeros(E + 1, dtype=torch.long, device=l.device)
    offsets[1:] = torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)
    at = torch.arange(T * k, device=l.device)
    row_token = torch.where(at < offsets[E], order // k, -1)
    token_row = torch.where(flat < E, torch.empty_like(at).scatter_(0, order, at), -1).view(T, k)
    return ids, w, offsets, row_token, token_row


@pytest.mark.parametrize("T, n", [(4864, None), (4865, None), (4865, 4700), (10007, 9001), (16384, None)])
@pytest.mark.parametrize("E, k, G, top, best, biased", [(256, 8, 8, 4, 2, True), (60, 4, 4, 2, 2, False), (128, 8, 1, 1, 1, False),
                                                        (384, 6, 1, 1, 1, True), (512, 16, 16, 5, 1, True)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_more_tokens_than_warps(T, n, E, k, G, top, best, biased, sigmoid):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = torch.randn((T, E), generator=g, device="cuda") * 1.5
    if T % 2:
        logits = logits.bfloat16()
    bias = 0.1 * torch.randn(E, generator=g, device="cuda") if biased else None
    nt = None if n is None else torch.tensor([n], dtype=torch.int32, device="cuda")
    kw = dict(bias=bias, groups=G, top_groups=top, group_best=best)
    renorm = E != 128
    got = qz.qz_moe_route(logits, k, score=qz.SCORE_SIGMOID if sigmoid else qz.SCORE_SOFTMAX, renormalize=renorm, scale=2.5, n_tokens=nt, **kw)
    want = route_many(logits, k, sigmoid, renorm, 2.5, n=n, **kw)
    for i in (0, 2, 3, 4):
        assert torch.equal(got[i].long(), want[i]), ("ids", "", "offsets", "row_token", "token_row")[i]
    w = want[1].cpu().numpy()
    assert bool((abs(got[1].cpu().numpy() - w) <= ref.weight_bound(None, w)).all())
