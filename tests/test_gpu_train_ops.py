"""The operators around the step against plain fp64 forms: the embedding and
its gradient, the head's cross entropy and its gradients, the experts'
products.

Bounds are element by element and follow from the arithmetic, with u the
unit roundoff of a type (2^-24 fp32, 2^-8 bf16, 2^-11 fp16):

  * an fp32 sum of n terms in any order is off by at most
    (n + 1) 2^-24 sum |terms|;
  * a tensor-core sum of K products (exact in fp32) adds at least 8 products
    per rounding or truncation of at most 2^-23 of the sum of magnitudes:
    (K / 8 + 8) 2^-23 sum |a b|;
  * a result rounded once to 16 bits is off by u |result| more (fp16: and
    2^-25, half its smallest subnormal);
  * the logits' gradient is rounded once to 16 bits before its products:
    u |g| per entry, plus what the logits' own error makes of
    exp(z - lse), a factor of 1 + 2 max|dz| + 2^-18 (the fp32 exponential
    and its argument).
"""
import ctypes
import math

import pytest
import torch

import optimizer_muon_step_gb300 as m

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {F32: 2.0 ** -24, BF: 2.0 ** -8, HF: 2.0 ** -11}
TINY = {F32: 0.0, BF: 0.0, HF: 2.0 ** -25}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def strided(t, pad):
    """The same matrix with `pad` more elements (NaN) between its rows."""
    if not pad:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def within(got, want, bound, what):
    assert got.shape == want.shape
    assert torch.isfinite(got.double()).all(), what
    excess = (got.double() - want).abs() - bound
    worst = excess.max().item() if excess.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} past its bound ({(excess > 0).sum().item()} elements)"


def mma_bound(k, magnitude):
    return (k / 8 + 8) * 2.0 ** -23 * magnitude


def rounded(bound, want, dtype):
    return bound + UNIT[dtype] * (want.abs() + bound) + TINY[dtype]


def status_of(ws):
    return m.muon_query_status(ws)


# --------------------------------------------------------------------------
# Embedding
# --------------------------------------------------------------------------

@pytest.mark.parametrize("table_dtype,out_dtype", [(F32, F32), (F32, BF), (F32, HF), (BF, BF), (HF, HF), (BF, F32),
                                                   (HF, BF)])
@pytest.mark.parametrize("vocab,dim,tokens,pad", [(7, 1, 1, 0), (50, 13, 33, 0), (1000, 256, 100, 0), (300, 1001, 513, 3),
                                                  (64, 2048, 5, 8), (5000, 264, 3000, 0)])
def test_lookup_is_one_rounded_product(lib, table_dtype, out_dtype, vocab, dim, tokens, pad):
    g = gen(vocab + dim)
    table = strided(randn(g, (vocab, dim), 0.5, table_dtype), pad)
    ids = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
    ids[0] = vocab - 1
    scale = 3.3
    got = m.muon_embedding_lookup(table, ids, scale=scale, out_dtype=out_dtype)
    want = (table[ids].float() * torch.tensor(scale, dtype=F32, device=DEV)).to(out_dtype)
    assert torch.equal(got, want)
    got32 = m.muon_embedding_lookup(table, ids.int(), scale=scale, out_dtype=out_dtype,
                                    out=strided(torch.empty_like(want), 5))
    assert torch.equal(got32, want)


def test_lookup_padding_outside_ids_and_shapes(lib):
    g = gen(3)
    table = randn(g, (40, 24), 1.0, BF)
    table[7] = float("nan")                       # the padding row is not read
    ids = torch.tensor([[7, 0, 39], [40, -1, 2 ** 40]], device=DEV)
    out = m.muon_embedding_lookup(table, ids, padding_idx=7)
    assert out.shape == (2, 3, 24)
    assert torch.equal(out[0, 1], table[0]) and torch.equal(out[0, 2], table[39])
    assert (out[0, 0] == 0).all() and (out[1] == 0).all()
    assert m.muon_embedding_lookup(table, ids[:0]).shape == (0, 3, 24)


def test_lookup_past_32_bit_offsets(lib):
    table = torch.zeros((300000, 8192), dtype=BF, device=DEV)     # 2.4e9 elements
    table[299999] = 1.5
    out = m.muon_embedding_lookup(table, torch.tensor([299999, 3], device=DEV), scale=2.0)
    assert (out[0] == 3.0).all() and (out[1] == 0).all()


def embed_grad_want(grad, ids, vocab, scale, padding_idx=None):
    live = (ids >= 0) & (ids < vocab)
    if padding_idx is not None:
        live &= ids != padding_idx
    rows, terms = ids[live].long(), grad[live].double() * float(torch.tensor(scale, dtype=F32))
    want = torch.zeros(vocab, grad.shape[1], dtype=torch.float64, device=DEV).index_add_(0, rows, terms)
    mag = torch.zeros_like(want).index_add_(0, rows, terms.abs())
    n = torch.zeros(vocab, dtype=torch.float64, device=DEV).index_add_(0, rows, torch.ones_like(rows, dtype=torch.float64))
    return want, (n[:, None] + 2) * 2.0 ** -24 * mag, n


EMBED_SHAPES = [(1, 1, 1, 0), (50, 13, 33, 0), (7, 264, 1000, 0), (1000, 1001, 513, 3), (1, 40, 700, 0),
                (163840, 64, 129, 0), (3001, 72, 16385, 8), (40000, 32, 40000, 0), (70000, 24, 150001, 0)]


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("vocab,dim,tokens,pad", EMBED_SHAPES)
def test_embedding_grad(lib, dtype, vocab, dim, tokens, pad):
    g = gen(vocab * 7 + dim)
    grad = strided(randn(g, (tokens, dim), 1.0, dtype), pad)
    u = torch.rand(tokens, generator=g, device=DEV)
    ids = ((torch.exp(u * math.log(vocab + 1.0)) - 1.0).long()).clamp_(0, vocab - 1)
    ids = vocab - 1 - ids
    want, bound, _ = embed_grad_want(grad, ids, vocab, 0.7)
    out = torch.full((vocab, dim), float("nan"), device=DEV)
    got = m.muon_embedding_grad(grad, ids, vocab, scale=0.7, out=out)
    assert got is out
    within(got, want, bound, "d_table")
    again = m.muon_embedding_grad(grad, ids.int(), vocab, scale=0.7)
    assert torch.equal(again, got)


def test_embedding_grad_accumulates_and_leaves_other_rows(lib):
    g = gen(5)
    vocab, dim, tokens = 500, 200, 3000
    grad = randn(g, (tokens, dim), 1.0, BF)
    ids = torch.randint(0, 40, (tokens,), generator=g, device=DEV)
    start = torch.randn(vocab, dim, generator=g, device=DEV)
    start[100] = float("nan")                    # a row without tokens
    out = start.clone()
    m.muon_embedding_grad(grad, ids, vocab, out=out, accumulate=True)
    want, bound, n = embed_grad_want(grad, ids, vocab, 1.0)
    assert torch.equal(out[40:].view(torch.int32), start[40:].view(torch.int32))
    total = want[:40] + start[:40].double()
    within(out[:40], total, bound[:40] + 2.0 ** -24 * (total.abs() + bound[:40]), "accumulated")


def test_embedding_grad_padding_outside_ids_and_no_tokens(lib):
    g = gen(6)
    grad = randn(g, (600, 72), 1.0, F32)
    ids = torch.randint(0, 90, (600,), generator=g, device=DEV)
    ids[5], ids[17], ids[300] = -4, 90, 2 ** 33
    grad[ids == 11] = float("nan")               # padded rows' gradients are not read
    grad[5] = grad[17] = grad[300] = float("inf")
    ws = m.allocate_workspace(lib.muon_embedding_grad_workspace(600, 90, 72))
    got = m.muon_embedding_grad(grad, ids, 90, padding_idx=11, workspace=ws)
    want, bound, _ = embed_grad_want(grad, ids, 90, 1.0, 11)
    within(got, want, bound, "d_table")
    assert (got[11] == 0).all()
    assert status_of(ws) == 1                     # ids outside the table were left out
    ids[5] = ids[17] = ids[300] = 11
    m.muon_embedding_grad(grad, ids, 90, padding_idx=11, workspace=ws)
    assert status_of(ws) == 0
    none = m.muon_embedding_grad(grad[:0], ids[:0], 90)
    assert (none == 0).all()
    all_padded = m.muon_embedding_grad(grad, torch.full_like(ids, 11), 90, padding_idx=11)
    assert (all_padded == 0).all()


# --------------------------------------------------------------------------
# Cross entropy
# --------------------------------------------------------------------------

def ce_want(hidden, weight, targets, row_scale, c, ignore):
    h, w = hidden.double(), weight.double()
    c = float(torch.tensor(c, dtype=F32))
    v = w.shape[0]
    z = c * (h @ w.t())
    dz = mma_bound(h.shape[1], abs(c) * (h.abs() @ w.abs().t())) + 2.0 ** -23 * z.abs()
    dz_row = dz.max(dim=1).values
    lse = torch.logsumexp(z, 1)
    live = (targets >= 0) & (targets < v) & (targets != ignore)
    hot = torch.zeros_like(z)
    hot[live.nonzero()[:, 0], targets[live].long()] = 1
    loss = torch.where(live, lse - (z * hot).sum(1), 0.0)
    lse_bound = dz_row + 2.0 ** -20 + 2.0 ** -22 * z.abs().max(dim=1).values
    r = torch.ones_like(lse) if row_scale is None else row_scale.double()
    r = torch.where(live, r, torch.zeros_like(r))
    p = torch.exp(z - lse[:, None])
    g = (p - hot) * r[:, None]
    top = 1.0 if row_scale is None else row_scale.double().abs().max().item()
    u = UNIT[hidden.dtype]
    # p's own error, then the rounding of g relative to the largest |r|
    slack = p * torch.expm1(2 * dz_row + 2.0 ** -18)[:, None] * r.abs()[:, None]
    dg = slack + u * (g.abs() + slack) + TINY[hidden.dtype] * 2.0 ** -15 * top + 2.0 ** -23 * g.abs()
    hl = torch.where(live[:, None], h, torch.zeros_like(h))
    dh = c * (g @ w)
    dw = c * (g.t() @ hl)
    mag_h, mag_w = (g.abs() + dg) @ w.abs(), (g.abs() + dg).t() @ hl.abs()
    bh = abs(c) * (dg @ w.abs() + mma_bound(v, mag_h) + 2.0 ** -21 * mag_h)
    bw = abs(c) * (dg.t() @ hl.abs() + mma_bound(h.shape[0], mag_w) + 2.0 ** -21 * mag_w)
    return dict(loss=loss, lse=lse, loss_bound=2 * lse_bound, lse_bound=lse_bound, dh=dh, dw=dw, bh=bh, bw=bw)


def ce_inputs(seed, n, v, d, dtype, ignored=0.0, lean=8.0):
    g = gen(seed)
    weight = randn(g, (v, d), 0.5 / math.sqrt(d), dtype)
    targets = torch.randint(0, v, (n,), generator=g, device=DEV)
    if n and v:
        targets[-1] = v - 1
    hidden = torch.randn(n, d, generator=g, device=DEV)
    hidden = (hidden + torch.rand(n, 1, generator=g, device=DEV) * lean * 4 * weight[targets].float()).to(dtype)
    if ignored:
        targets[torch.rand(n, generator=g, device=DEV) < ignored] = -100
    return hidden, weight, targets


CE_SHAPES = [(1, 1, 8), (1, 1000, 64), (3, 17, 8), (33, 257, 40), (130, 1000, 200), (129, 511, 13), (300, 3001, 264),
             (257, 50021, 72), (64, 2048, 1031), (600, 640, 520)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,v,d", CE_SHAPES)
def test_cross_entropy_and_gradients(lib, dtype, n, v, d):
    hidden, weight, targets = ce_inputs(n + v, n, v, d, dtype, ignored=0.2 if n > 3 else 0.0)
    scale = torch.rand(n, generator=gen(n), device=DEV) / n
    want = ce_want(hidden, weight, targets, scale, 0.8, -100)
    loss, lse = m.muon_linear_ce(hidden, weight, targets, logit_scale=0.8)
    within(loss, want["loss"], want["loss_bound"], "loss")
    within(lse, want["lse"], want["lse_bound"], "lse")
    assert (loss[targets == -100] == 0).all()
    loss2, lse2, dh, dw = m.muon_linear_ce_grad(hidden, weight, targets.int(), row_scale=scale, logit_scale=0.8)
    within(loss2, want["loss"], want["loss_bound"], "loss with gradients")
    within(lse2, want["lse"], want["lse_bound"], "lse with gradients")
    assert dh.dtype == dw.dtype == dtype
    within(dh, want["dh"], rounded(want["bh"], want["dh"], dtype), "d_hidden")
    within(dw, want["dw"], rounded(want["bw"], want["dw"], dtype), "d_weight")
    again = m.muon_linear_ce_grad(hidden, weight, targets, row_scale=scale, logit_scale=0.8)
    for a, b in zip(again, (loss2, lse2, dh, dw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_cross_entropy_loss_of_many_tokens(lib, dtype):
    hidden, weight, targets = ce_inputs(23, 2100, 700, 40, dtype, ignored=0.2)
    want = ce_want(hidden, weight, targets, None, 1.0, -100)
    loss, lse = m.muon_linear_ce(hidden, weight, targets)
    within(loss, want["loss"], want["loss_bound"], "loss")
    within(lse, want["lse"], want["lse_bound"], "lse")


@pytest.mark.parametrize("n,v,d", [(5, 300, 64), (200, 3000, 520), (40, 900, 1100)])
def test_cross_entropy_small_losses_keep_their_bits(lib, n, v, d):
    """The target's logit leads by 10 and more: losses of 1e-3 and less are sums of
    small terms, not differences of large ones.  A loss is off by a factor of
    1 + 2 dz (the error of two logits) + 2^-18 (exponentials and their
    arguments) + v 2^-24 (the sum) at most, with dz from fp32 and tensor-core
    sums of d products."""
    g = gen(v)
    weight = randn(g, (v, d), 0.5 / math.sqrt(d), BF)
    targets = torch.randint(0, v, (n,), generator=g, device=DEV)
    hidden = (weight[targets].float() * 80).to(BF)
    z = hidden.double() @ weight.double().t()
    zt = z.gather(1, targets[:, None])
    want = torch.log1p(torch.exp(z - zt).sum(1) - 1)
    dz = mma_bound(d, hidden.double().abs() @ weight.double().abs().t()).max(dim=1).values + 2.0 ** -22 * z.abs().max(1).values
    loss, lse = m.muon_linear_ce(hidden, weight, targets)
    assert want.max() < 0.1
    within(loss, want, want * (torch.expm1(2 * dz) + 2.0 ** -18 + v * 2.0 ** -24), "loss")


@pytest.mark.parametrize("n,v,d", [(100, 900, 1400), (200, 1500, 2056), (1100, 100, 72), (1100, 400, 72), (1800, 20000, 2048),
                                   (128, 100000, 7168)])
def test_cross_entropy_long_sums(lib, n, v, d):
    """Sums that are cut into segments: over the width (logits, above 1024),
    over the tokens (an fp32 d_weight, above 1024) and over the vocabulary
    (d_hidden, above 16384 a piece), with up to 128 rows and more."""
    hidden, weight, targets = ce_inputs(n + v + 1, n, v, d, HF, ignored=0.1)
    scale = torch.rand(n, generator=gen(n), device=DEV) / n
    want = ce_want(hidden, weight, targets, scale, 1.0, -100)
    dw = torch.empty(v, d, device=DEV)
    loss, lse, dh, _ = m.muon_linear_ce_grad(hidden, weight, targets, row_scale=scale, d_weight=dw)
    within(loss, want["loss"], want["loss_bound"], "loss")
    within(lse, want["lse"], want["lse_bound"], "lse")
    within(dh, want["dh"], rounded(want["bh"], want["dh"], HF), "d_hidden")
    within(dw, want["dw"], want["bw"], "d_weight")
    # segments keep the truncation of the tensor core's sums at that of their
    # 1024 terms, 2^-23 a MMA of 16 or 64 * 2^-23 of the result at most, and
    # the fp32 additions of 8 segments, exponentials and logarithm below 2^-20
    assert ((lse.double() - want["lse"]).norm() / want["lse"].norm()).item() < 64 * 2.0 ** -23


def test_expert_wgrad_long_sums(lib):
    """fp32 gradients over more than 1024 tokens an expert, few and many rows."""
    for rows in (96, 264):
        x, dy, w, off = expert_case(rows, split(4, 4000, 3), rows, 200, BF)
        expert_check(x, dy, w, off, BF)


@pytest.mark.parametrize("sizes,rows,cols", [([0, 5000, 0], 200, 130), ([1, 9000], 96, 64), ([3000, 0, 64, 4097], 264, 257),
                                             ([20000], 72, 1000)])
def test_expert_wgrad_in_pieces(lib, sizes, rows, cols):
    """Few and small matrices of many tokens: every expert's tokens are cut
    into pieces whose sums are added."""
    g = gen(rows)
    n = sum(sizes)
    off = torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], dtype=torch.int64, device=DEV)
    one = m.load_library().muon_expert_wgrad_workspace(4096, 1024, 4096, 1024, len(sizes), 64, rows, cols)
    assert m.load_library().muon_expert_wgrad_workspace(4096, 1024, 4096, 1024, len(sizes), n, rows, cols) > one
    for dtype in (BF, HF):
        x, dy = randn(g, (n, cols), 1.0, dtype), randn(g, (n, rows), 1.0, dtype)
        start = torch.randn(len(sizes), rows, cols, generator=g, device=DEV)
        want = torch.zeros(len(sizes), rows, cols, dtype=torch.float64, device=DEV)
        mag = torch.zeros_like(want)
        at = 0
        for e, k in enumerate(sizes):
            a, b = dy[at:at + k].double(), x[at:at + k].double()
            want[e], mag[e] = a.t() @ b, a.abs().t() @ b.abs()
            at += k
        bound = mma_bound(max(sizes), mag)
        got = m.muon_expert_wgrad(dy, x, off)
        within(got, want, rounded(bound, want, dtype), "rounded")
        assert torch.equal(got, m.muon_expert_wgrad(dy, x, off))
        within(m.muon_expert_wgrad(dy, x, off, out_dtype=F32), want, bound, "fp32")
        acc = start.clone()
        m.muon_expert_wgrad(dy, x, off, out=acc, accumulate=True)
        total = want + start.double()
        within(acc, total, bound + 2.0 ** -22 * (total.abs() + start.double().abs() + bound), "accumulated")
    for e, k in enumerate(sizes):
        assert k > 0 or (got[e] == 0).all()


def test_expert_wgrad_one_long_sum_of_many(lib):
    """One expert has all of 20000 tokens: its fp32 sums of positive products
    are cut too.  A segment's 1024 terms are 64 tensor-core additions, off by
    at most 2^-23 of the sum each, and the 20 segments are added in fp32."""
    off = torch.tensor([0] * 18 + [20000] * 23, dtype=torch.int32, device=DEV)
    g = gen(5)
    x, dy = (torch.rand(20000, c, generator=g, device=DEV).to(BF) for c in (200, 136))
    got = m.muon_expert_wgrad(dy, x, off, out_dtype=F32)
    want = dy.double().t() @ x.double()
    assert (got[:17] == 0).all() and (got[18:] == 0).all()
    assert ((got[17].double() - want).abs() <= (64 * 2.0 ** -23 + 20 * 2.0 ** -24) * want).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_cross_entropy_in_blocks_of_tokens(lib, dtype):
    """A workspace that holds 256 tokens: the gradient of the weights is summed
    over blocks, into fp32 sums or straight into an fp32 result."""
    n, v, d = 700, 1500, 136
    hidden, weight, targets = ce_inputs(11, n, v, d, dtype, ignored=0.1)
    want = ce_want(hidden, weight, targets, None, 1.0, -100)
    small = m.muon_linear_ce_workspace(hidden, weight, targets, True, budget_bytes=1)
    assert small < m.muon_linear_ce_workspace(hidden, weight, targets, True)
    ws = m.allocate_workspace(small)
    loss, lse, dh, dw = m.muon_linear_ce_grad(hidden, weight, targets, workspace=ws)
    within(loss, want["loss"], want["loss_bound"], "loss")
    within(dh, want["dh"], rounded(want["bh"], want["dh"], dtype), "d_hidden")
    bw = want["bw"] + 2.0 ** -22 * want["dw"].abs()
    within(dw, want["dw"], rounded(bw, want["dw"], dtype), "d_weight")
    dw32 = torch.full((v, d), float("nan"), device=DEV)
    m.muon_linear_ce_grad(hidden, weight, targets, workspace=ws, d_weight=dw32)
    within(dw32, want["dw"], bw, "fp32 d_weight")
    start = torch.randn(v, d, generator=gen(12), device=DEV)
    acc = start.clone()
    m.muon_linear_ce_grad(hidden, weight, targets, workspace=ws, d_weight=acc, accumulate=True)
    total = want["dw"] + start.double()
    within(acc, total, bw + 2.0 ** -22 * (total.abs() + start.double().abs() + bw), "accumulated d_weight")
    tiny = m.allocate_workspace(256)
    with pytest.raises(m.MuonError) as e:
        m.muon_linear_ce_grad(hidden, weight, targets, workspace=tiny)
    assert e.value.status == 4


@pytest.mark.parametrize("d", [768, 776])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_cross_entropy_twice_and_kept(lib, dtype, d):
    """Either side of the width up to which the logits are computed twice:
    blocks of tokens, strided rows, ignored rows that hold NaN, scales."""
    n, v = 700, 1100
    hidden, weight, targets = ce_inputs(d, n, v, d, dtype, ignored=0.1)
    targets[5], targets[600] = v, -3
    out = (targets < 0) | (targets >= v)
    scale = torch.rand(n, generator=gen(d), device=DEV) / n
    want = ce_want(hidden, weight, targets, scale, 1.3, -100)
    small = m.allocate_workspace(m.muon_linear_ce_workspace(hidden, weight, targets, True, budget_bytes=1))
    held = torch.where(out, float("nan"), scale)
    for pads, ws in (((0, 0), None), ((3, 5), None), ((8, 8), small)):
        h = strided(torch.where(out[:, None], float("nan"), hidden.float()).to(dtype), pads[0])
        got = m.muon_linear_ce_grad(h, strided(weight, pads[1]), targets, row_scale=held, logit_scale=1.3, workspace=ws)
        live = ~out
        within(got[0][live], want["loss"][live], want["loss_bound"][live], "loss")
        within(got[1][live], want["lse"][live], want["lse_bound"][live], "lse")
        assert (got[0][out] == 0).all() and (got[2][out] == 0).all()
        within(got[2], want["dh"], rounded(want["bh"], want["dh"], dtype), "d_hidden")
        bw = want["bw"] + 2.0 ** -22 * want["dw"].abs()
        within(got[3], want["dw"], rounded(bw, want["dw"], dtype), "d_weight")


def test_cross_entropy_short_last_block_stays_in_its_workspace(lib):
    """Blocks whose d_hidden is summed in one piece, then one in several."""
    n, v, d = 2048 + 44, 4096, 4864
    hidden, weight, targets = ce_inputs(13, n, v, d, BF)
    of = m.train._ce_struct(hidden[:1024], weight, targets[:1024], 1.0, -100)
    of.d_weight_dtype = 0
    need = m.load_library().muon_linear_ce_workspace(ctypes.addressof(of), 1, 1 << 40)
    ws = m.allocate_workspace(need + (8 << 20))
    ws.fill_(171)
    dw = torch.empty(v, d, device=DEV)
    _, _, dh, _ = m.muon_linear_ce_grad(hidden, weight, targets, d_weight=dw, workspace=ws[:need])
    assert (ws[need:] == 171).all()
    want = ce_want(hidden, weight, targets, None, 1.0, -100)
    within(dh, want["dh"], rounded(want["bh"], want["dh"], BF), "d_hidden")
    within(dw, want["dw"], want["bw"] + 2.0 ** -22 * want["dw"].abs(), "d_weight")


@pytest.mark.parametrize("pads", [(0, 0), (3, 5), (8, 16)])
def test_cross_entropy_strided_rows(lib, pads):
    hidden, weight, targets = ce_inputs(21, 140, 900, 72, BF)
    want = ce_want(hidden, weight, targets, None, 1.0, -100)
    loss, lse, dh, dw = m.muon_linear_ce_grad(strided(hidden, pads[0]), strided(weight, pads[1]), targets)
    within(loss, want["loss"], want["loss_bound"], "loss")
    within(dh, want["dh"], rounded(want["bh"], want["dh"], BF), "d_hidden")
    within(dw, want["dw"], rounded(want["bw"], want["dw"], BF), "d_weight")
    loss3, _ = m.muon_linear_ce(strided(hidden, pads[0]), strided(weight, pads[1]), targets)
    within(loss3, want["loss"], want["loss_bound"], "loss alone")


def test_cross_entropy_ignored_rows_are_not_read_into_the_gradients(lib):
    hidden, weight, targets = ce_inputs(31, 200, 700, 64, BF)
    targets[::3] = -100
    clean = m.muon_linear_ce_grad(hidden, weight, targets)
    dirty = hidden.clone()
    dirty[::3] = float("nan")
    dirty[::6] = float("inf")
    loss, lse, dh, dw = m.muon_linear_ce_grad(dirty, weight, targets)
    assert torch.equal(dw, clean[3]) and torch.equal(dh, clean[2]) and torch.equal(loss, clean[0])
    assert (dh[::3] == 0).all() and (loss[::3] == 0).all()


@pytest.mark.parametrize("d", [64, 1032])
@pytest.mark.parametrize("lo,hi", [(0, 32), (128, 160), (64, 128), (576, 600), (31, 33)])
def test_cross_entropy_nan_columns_reach_the_loss(lib, d, lo, hi):
    """NaN logits of some columns, whole blocks of them among these, are not
    lost on the way to the normaliser."""
    for n in (20, 150):
        hidden, weight, targets = ce_inputs(n, n, 600, d, BF)
        targets[:] = 300
        weight[lo:hi] = float("nan")
        loss, lse = m.muon_linear_ce(hidden, weight, targets)
        assert torch.isnan(loss).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("held", [float("nan"), float("inf"), -1e30])
@pytest.mark.parametrize("n", [90, 300])
def test_cross_entropy_ignored_rows_scale_is_not_read(lib, n, held):
    hidden, weight, targets = ce_inputs(n, n, 500, 72, HF, ignored=0.2)
    targets[1], targets[2] = 500, -7                     # outside: left out as well
    out = (targets < 0) | (targets >= 500)
    scale = torch.rand(n, generator=gen(n), device=DEV) / n
    want = m.muon_linear_ce_grad(hidden, weight, targets, row_scale=torch.where(out, 0.0, scale))
    got = m.muon_linear_ce_grad(hidden, weight, targets, row_scale=torch.where(out, held, scale))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_cross_entropy_all_ignored_and_targets_outside(lib):
    hidden, weight, targets = ce_inputs(41, 70, 300, 64, BF)
    need = m.muon_linear_ce_workspace(hidden, weight, targets, True)
    ws = m.allocate_workspace(need)
    none = torch.full_like(targets, -100)
    loss, lse, dh, dw = m.muon_linear_ce_grad(hidden, weight, none, workspace=ws)
    assert (loss == 0).all() and (dh == 0).all() and (dw == 0).all()
    assert status_of(ws) == 0
    bad = targets.clone()
    bad[3], bad[4], bad[69] = 300, -5, 2 ** 40
    want = ce_want(hidden, weight, bad, None, 1.0, -100)
    loss, lse, dh, dw = m.muon_linear_ce_grad(hidden, weight, bad, workspace=ws)
    assert status_of(ws) == 1
    within(loss, want["loss"], want["loss_bound"], "loss")
    within(dw, want["dw"], rounded(want["bw"], want["dw"], BF), "d_weight")
    assert (dh[[3, 4, 69]] == 0).all()
    m.muon_linear_ce(hidden, weight, bad, workspace=ws)
    assert status_of(ws) == 1
    # an ignore_index inside the vocabulary
    got = m.muon_linear_ce_grad(hidden, weight, targets, ignore_index=int(targets[0]), workspace=ws)
    want = ce_want(hidden, weight, targets, None, 1.0, int(targets[0]))
    within(got[3], want["dw"], rounded(want["bw"], want["dw"], BF), "d_weight")
    # no tokens
    empty = m.muon_linear_ce_grad(hidden[:0], weight, targets[:0])
    assert empty[0].shape == (0,) and (empty[3] == 0).all()
    zero = m.muon_linear_ce_grad(hidden, weight, targets, row_scale=torch.zeros(70, device=DEV))
    assert (zero[2] == 0).all() and (zero[3] == 0).all() and (zero[0] > 0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_cross_entropy_large_logits_and_overflow(lib, dtype):
    """Logits in the hundreds, where exp alone would overflow; and a row whose
    logits are infinite, which must not touch the others."""
    n, v, d = 40, 500, 64
    hidden, weight, targets = ce_inputs(51, n, v, d, dtype)
    want = ce_want(hidden, weight, targets, None, 200.0, -100)
    loss, lse, dh, dw = m.muon_linear_ce_grad(hidden, weight, targets, logit_scale=200.0)
    within(loss, want["loss"], want["loss_bound"], "loss")
    within(lse, want["lse"], want["lse_bound"], "lse")
    within(dh, want["dh"], rounded(want["bh"], want["dh"], dtype), "d_hidden")
    hidden2 = hidden.clone()
    hidden2[7] = float("inf")
    loss2, lse2 = m.muon_linear_ce(hidden2, weight, targets)
    keep = torch.arange(n, device=DEV) != 7
    ref = m.muon_linear_ce(hidden, weight, targets)
    assert torch.equal(loss2[keep], ref[0][keep]) and torch.equal(lse2[keep], ref[1][keep])
    assert not torch.isfinite(lse2[7])


@pytest.mark.parametrize("scale", [-0.7, 0.0, 1e-6])
def test_cross_entropy_other_logit_scales(lib, scale):
    """Negative, zero and tiny logit scales, with an odd vocabulary."""
    hidden, weight, targets = ce_inputs(55, 90, 333, 72, BF, ignored=0.1)
    want = ce_want(hidden, weight, targets, None, scale, -100)
    loss, lse, dh, dw = m.muon_linear_ce_grad(hidden, weight, targets, logit_scale=scale)
    within(loss, want["loss"], want["loss_bound"], "loss")
    within(lse, want["lse"], want["lse_bound"], "lse")
    within(dh, want["dh"], rounded(want["bh"], want["dh"], BF), "d_hidden")
    within(dw, want["dw"], rounded(want["bw"], want["dw"], BF), "d_weight")


def test_cross_entropy_small_gradients_in_fp16(lib):
    """Row scales of 1e-7 would put every fp16 logit gradient below the type's
    subnormals; the rounding is relative to the largest scale instead."""
    hidden, weight, targets = ce_inputs(61, 150, 1200, 72, HF)
    scale = torch.full((150,), 1e-7, device=DEV)
    want = ce_want(hidden, weight, targets, scale, 1.0, -100)
    dw = torch.empty(1200, 72, device=DEV)
    _, _, dh, _ = m.muon_linear_ce_grad(hidden, weight, targets, row_scale=scale, d_weight=dw)
    within(dw, want["dw"], want["bw"], "d_weight")
    within(dh, want["dh"], rounded(want["bh"], want["dh"], HF), "d_hidden")


def test_cross_entropy_gradient_against_differences(lib):
    """Central differences of the op's own loss.  The inputs and the steps are
    multiples of 2^-4, so the moved inputs are exact in bf16; the third
    derivative along a step adds at most |z'|^3 / 6 per counted token."""
    g = gen(71)
    n, v, d = 24, 90, 32
    grid = lambda shape, k: torch.randint(-k, k + 1, shape, generator=g, device=DEV).to(BF) / 16  # noqa: E731
    hidden, weight = grid((n, d), 12), grid((v, d), 6)
    targets = torch.randint(0, v, (n,), generator=g, device=DEV)
    targets[::5] = -100
    scale = torch.rand(n, generator=g, device=DEV)
    want = ce_want(hidden, weight, targets, scale, 1.0, -100)
    _, _, dh, dw = m.muon_linear_ce_grad(hidden, weight, targets, row_scale=scale)
    objective = lambda h, w: (m.muon_linear_ce(h, w, targets)[0].double() * scale.double()).sum().item()  # noqa: E731
    noise = (want["loss_bound"] * scale.double()).sum().item()
    eps = 1 / 16
    for what, grad, bound in (("hidden", dh, rounded(want["bh"], want["dh"], BF)),
                              ("weight", dw, rounded(want["bw"], want["dw"], BF))):
        base = hidden if what == "hidden" else weight
        other = weight if what == "hidden" else hidden
        for k in range(6):
            step = torch.zeros_like(base)
            for _ in range(4):
                i, j = torch.randint(0, base.shape[0], (1,), generator=g, device=DEV), torch.randint(0, d, (1,), generator=g, device=DEV)
                step[i, j] = 1.0 if k % 2 else -1.0
            move = lambda s: (base + s * eps * step).to(BF)  # noqa: E731
            assert torch.equal(move(1).double() - base.double(), eps * step.double())
            f = [objective(move(s), weight) if what == "hidden" else objective(hidden, move(s)) for s in (1, -1)]
            slope = (f[0] - f[1]) / (2 * eps)
            want_slope = (grad.double() * step.double()).sum().item()
            reach = (step.double().abs() @ other.double().abs().t()).abs().amax().item()
            # third derivative of lse along the step <= 8 max|z'|^3, over the rows the step moves
            rows = n if what == "weight" else int((step != 0).any(1).sum())
            limit = noise / eps + rows * 8 * reach ** 3 * eps ** 2 / 6 + (bound * step.double().abs()).sum().item()
            assert abs(slope - want_slope) <= limit, (what, k, slope, want_slope, limit)


# --------------------------------------------------------------------------
# Experts
# --------------------------------------------------------------------------

def split(seed, tokens, experts, empty=()):
    gcpu = torch.Generator().manual_seed(seed)
    w = torch.rand(experts, generator=gcpu) ** 3 + 1e-3
    for e in empty:
        w[e] = 0.0
    sizes = torch.bincount(torch.multinomial(w, tokens, replacement=True, generator=gcpu), minlength=experts)
    return [0, *torch.cumsum(sizes, 0).tolist()]


def expert_case(seed, offsets, rows, cols, dtype, pad=0):
    g = gen(seed)
    n, e = offsets[-1], len(offsets) - 1
    x = strided(randn(g, (n, cols), 1.0, dtype), pad)
    dy = strided(randn(g, (n, rows), 0.5, dtype), pad)
    w = randn(g, (e, rows, cols), 0.1, dtype)
    return x, dy, w, torch.tensor(offsets, dtype=torch.int32, device=DEV)


def expert_check(x, dy, w, off, dtype):
    e, rows, cols = w.shape
    lo = off.tolist()
    y = m.muon_expert_matmul(x, w, off)
    dx = m.muon_expert_matmul(dy, w, off.long(), transpose=True)
    dw = m.muon_expert_wgrad(dy, x, off)
    dw32 = m.muon_expert_wgrad(dy, x, off, out_dtype=F32)
    assert y.dtype == dx.dtype == dw.dtype == dtype and dw32.dtype == F32
    for i in range(e):
        s = slice(lo[i], lo[i + 1])
        xd, gd, wd = x[s].double(), dy[s].double(), w[i].double()
        n = xd.shape[0]
        want = xd @ wd.t()
        within(y[s], want, rounded(mma_bound(cols, xd.abs() @ wd.abs().t()), want, dtype), f"y of expert {i}")
        want = gd @ wd
        within(dx[s], want, rounded(mma_bound(rows, gd.abs() @ wd.abs()), want, dtype), f"dx of expert {i}")
        want = gd.t() @ xd
        bound = mma_bound(n, gd.abs().t() @ xd.abs())
        within(dw32[i], want, bound, f"fp32 dw of expert {i}")
        within(dw[i], want, rounded(bound, want, dtype), f"dw of expert {i}")
        if n == 0:
            assert (dw[i] == 0).all() and (dw32[i] == 0).all()
    return y, dx, dw, dw32


EXPERT_CASES = [([0, 1], 8, 8), ([0, 0, 1, 1], 16, 8), ([0, 5, 5, 12, 40], 13, 21), (split(1, 300, 5), 40, 64),
                (split(2, 1000, 7, empty=(0, 6)), 136, 264), (split(3, 64, 40), 256, 136),
                ([0, 127, 255, 383, 512, 769], 64, 128), ([0, 63, 64, 129, 129, 130], 200, 72),
                (split(4, 2500, 3), 520, 392), ([0, 1300], 1408, 96), (split(5, 700, 130), 24, 40)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case", range(len(EXPERT_CASES)))
def test_expert_products(lib, dtype, case):
    offsets, rows, cols = EXPERT_CASES[case]
    x, dy, w, off = expert_case(case + 1, offsets, rows, cols, dtype)
    first = expert_check(x, dy, w, off, dtype)
    again = expert_check(x, dy, w, off, dtype)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("pad", [1, 8])
def test_expert_products_strided_rows(lib, pad):
    x, dy, w, off = expert_case(77, split(6, 400, 6), 72, 40, BF, pad)
    expert_check(x, dy, w, off, BF)
    out = strided(torch.zeros(400, 72, dtype=BF, device=DEV), pad)
    guard = out.as_strided((400, pad), (72 + pad, 1), 72)
    assert torch.isnan(guard[:-1]).all()
    m.muon_expert_matmul(x, w, off, out=out)
    assert torch.equal(out, m.muon_expert_matmul(x, w, off))
    assert torch.isnan(guard[:-1]).all()


def test_expert_rows_of_no_expert_are_zeros_and_not_summed(lib):
    """Offsets that start late and end early, as with capacity buffers: the
    rows outside hold NaN, give zero rows and enter no sum."""
    x, dy, w, _ = expert_case(81, [0, 500], 136, 72, BF)
    off = [37, 37, 200, 391]
    offt = torch.tensor(off, dtype=torch.int32, device=DEV)
    w = randn(gen(82), (3, 136, 72), 0.1, BF)
    outside = torch.ones(500, dtype=torch.bool, device=DEV)
    outside[37:391] = False
    x[outside] = float("nan")
    dy[outside] = float("inf")
    y, dx, dw, _ = expert_check(x, dy, w, offt, BF)
    assert (y[outside] == 0).all() and (dx[outside] == 0).all()


def test_expert_neighbours_nan_stays_in_its_expert(lib):
    """Ranges end inside tiles: a NaN row of one expert reaches nothing of the
    next one's, forward or backward."""
    x, dy, w, off = expert_case(83, [0, 70, 133, 200, 270], 64, 80, BF)
    clean = expert_check(x, dy, w, off, BF)
    x2, dy2 = x.clone(), dy.clone()
    x2[133:200] = float("nan")
    dy2[133:200] = float("nan")
    keep = torch.ones(270, dtype=torch.bool, device=DEV)
    keep[133:200] = False
    assert torch.equal(m.muon_expert_matmul(x2, w, off)[keep], clean[0][keep])
    assert torch.equal(m.muon_expert_matmul(dy2, w, off, transpose=True)[keep], clean[1][keep])
    dw = m.muon_expert_wgrad(dy2, x2, off)
    assert torch.equal(dw[[0, 1, 3]], clean[2][[0, 1, 3]])
    assert torch.isnan(dw[2]).all()


def test_expert_offsets_outside_are_clipped(lib):
    x, dy, w, _ = expert_case(84, [0, 100], 40, 24, BF)
    w = randn(gen(85), (4, 40, 24), 0.1, BF)
    odd = torch.tensor([-5, 30, 30, 90, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    plain = torch.tensor([0, 30, 30, 90, 100], dtype=torch.int32, device=DEV)
    assert torch.equal(m.muon_expert_matmul(x, w, odd), m.muon_expert_matmul(x, w, plain))
    assert torch.equal(m.muon_expert_wgrad(dy, x, odd), m.muon_expert_wgrad(dy, x, plain))
    backwards = torch.tensor([0, 60, 40, 80, 100], dtype=torch.int32, device=DEV)
    dw = m.muon_expert_wgrad(dy, x, backwards)
    assert (dw[1] == 0).all()
    y = m.muon_expert_matmul(x, w, backwards)
    assert torch.isfinite(y.float()).all()


def test_expert_wgrad_accumulates(lib):
    x, dy, w, off = expert_case(86, split(9, 600, 4, empty=(2,)), 96, 56, BF)
    start = torch.randn(4, 96, 56, generator=gen(87), device=DEV)
    out = start.clone()
    m.muon_expert_wgrad(dy, x, off, out=out, accumulate=True)
    fresh = m.muon_expert_wgrad(dy, x, off, out_dtype=F32)
    assert torch.equal(out, start + fresh)
    assert torch.equal(out[2], start[2])
    odd = torch.randn(4, 13, 7, generator=gen(88), device=DEV)
    o2 = odd.clone()
    m.muon_expert_wgrad(dy[:, :13], x[:, :7], off, out=o2, accumulate=True)
    assert torch.equal(o2, odd + m.muon_expert_wgrad(dy[:, :13], x[:, :7], off, out_dtype=F32))


def test_expert_no_tokens(lib):
    w = randn(gen(90), (3, 16, 8), 0.1, BF)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    x, dy = torch.empty(0, 8, dtype=BF, device=DEV), torch.empty(0, 16, dtype=BF, device=DEV)
    assert m.muon_expert_matmul(x, w, off).shape == (0, 16)
    assert (m.muon_expert_wgrad(dy, x, off) == 0).all()
    acc = torch.ones(3, 16, 8, device=DEV)
    m.muon_expert_wgrad(dy, x, off, out=acc, accumulate=True)
    assert (acc == 1).all()


# --------------------------------------------------------------------------
# Streams, captures, refusals
# --------------------------------------------------------------------------

def test_calls_on_another_stream_are_ordered_with_it(lib):
    """The inputs are made on a side stream behind a long matrix product; the
    calls on that stream must wait for them, and their results for the calls."""
    side = torch.cuda.Stream()
    g = gen(95)
    big = torch.randn(4096, 4096, generator=g, device=DEV)
    hidden, weight, targets = ce_inputs(96, 100, 800, 64, BF)
    x, dy, w, off = expert_case(97, split(7, 300, 4), 64, 64, BF)
    table = randn(g, (500, 64), 1.0, BF)
    ids = torch.randint(0, 500, (200,), generator=g, device=DEV)
    want = (*m.muon_linear_ce_grad(hidden, weight, targets), m.muon_expert_matmul(x, w, off),
            m.muon_expert_wgrad(dy, x, off), m.muon_embedding_lookup(table, ids),
            m.muon_embedding_grad(table[ids], ids, 500))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = big @ big * 1e-3
        late = [t.clone() for t in (hidden, weight, targets, x, dy, w, off, table, ids)]
    h2, w2, t2, x2, dy2, ew2, off2, tab2, ids2 = late
    got = (*m.muon_linear_ce_grad(h2, w2, t2, stream=side), m.muon_expert_matmul(x2, ew2, off2, stream=side),
           m.muon_expert_wgrad(dy2, x2, off2, stream=side.cuda_stream), m.muon_embedding_lookup(tab2, ids2, stream=side))
    with torch.cuda.stream(side):
        rows = tab2[ids2]
    got = (*got, m.muon_embedding_grad(rows, ids2, 500, stream=side))
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_calls_can_be_captured(lib):
    hidden, weight, targets = ce_inputs(98, 100, 800, 64, BF)
    x, dy, w, off = expert_case(99, split(8, 300, 4), 64, 64, BF)
    table = randn(gen(100), (500, 64), 1.0, BF)
    ids = torch.randint(0, 500, (200,), generator=gen(101), device=DEV)

    def step():
        return (*m.muon_linear_ce_grad(hidden, weight, targets), m.muon_expert_matmul(x, w, off),
                m.muon_expert_wgrad(dy, x, off), m.muon_embedding_lookup(table, ids),
                m.muon_embedding_grad(x[:200], ids, 500))

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals(lib):
    hidden, weight, targets = ce_inputs(102, 10, 30, 16, BF)
    x, dy, w, off = expert_case(103, [0, 4, 10], 16, 8, BF)
    ids = torch.zeros(5, dtype=torch.int64, device=DEV)
    table = torch.zeros(9, 16, device=DEV)
    for call in (lambda: m.muon_embedding_lookup(table.cpu(), ids), lambda: m.muon_embedding_lookup(table, ids.float()),
                 lambda: m.muon_embedding_lookup(table.double(), ids),
                 lambda: m.muon_embedding_grad(table[:5], ids.cpu(), 9),
                 lambda: m.muon_linear_ce(hidden.float(), weight.float(), targets),
                 lambda: m.muon_linear_ce(hidden, weight.half(), targets),
                 lambda: m.muon_expert_matmul(x, w.half(), off), lambda: m.muon_expert_matmul(x.cpu(), w, off),
                 lambda: m.muon_expert_wgrad(dy, x.half(), off)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: m.muon_embedding_lookup(table.t(), ids), lambda: m.muon_embedding_lookup(table.expand(1, 9, 16), ids),
                 lambda: m.muon_embedding_grad(table[:4], ids, 9),
                 lambda: m.muon_embedding_grad(table[:5], ids, 9, accumulate=True),
                 lambda: m.muon_embedding_grad(table[:1].expand(5, 16), ids, 9),
                 lambda: m.muon_linear_ce(hidden, weight[:, :8], targets), lambda: m.muon_linear_ce(hidden, weight, targets[:5]),
                 lambda: m.muon_linear_ce_grad(hidden, weight, targets, accumulate=True),
                 lambda: m.muon_expert_matmul(dy, w, off), lambda: m.muon_expert_matmul(x, w, off[:2]),
                 lambda: m.muon_expert_wgrad(dy[:9], x, off), lambda: m.muon_expert_matmul(x, w.transpose(1, 2), off)):
        with pytest.raises(ValueError):
            call()
    for call, code in ((lambda: m.muon_linear_ce(hidden, weight, targets, logit_scale=float("nan")), 1),
                       (lambda: m.muon_embedding_lookup(table, ids, out=table[:5]), 1),     # output over the table
                       (lambda: m.muon_linear_ce_grad(hidden, weight, targets, d_hidden=hidden), 1),
                       (lambda: m.muon_expert_matmul(dy, w, off, transpose=True, out=dy[:, :8]), 1),
                       (lambda: m.muon_embedding_grad(table[:5], ids, 9,
                                                      workspace=torch.empty(300, dtype=torch.uint8, device=DEV)[4:]), 3),
                       (lambda: m.muon_expert_wgrad(dy, x, off, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)), 4)):
        with pytest.raises(m.MuonError) as e:
            call()
        assert e.value.status == code


def test_host_buffers_are_refused(lib):
    """Pinned host memory in one place of an otherwise valid C call."""
    ids = torch.zeros(5, dtype=torch.int64, device=DEV)
    table, out = torch.zeros(9, 16, device=DEV), torch.ones(5, 16, device=DEV)
    pinned = torch.zeros(9, 16).pin_memory()
    st = m._stream(None)
    call = lambda t, o: lib.muon_embedding_lookup(t.data_ptr(), 0, 16, 9, 16, ids.data_ptr(), 1, 5, 1.0, -1,  # noqa: E731
                                                  o.data_ptr(), 0, 16, st)
    assert call(pinned, out) == 1 and call(table, pinned) == 1
    torch.cuda.synchronize()
    assert (out == 1).all()
    assert call(table, out) == 0
    off = torch.tensor([0, 5], dtype=torch.int32).pin_memory()
    x, w = torch.zeros(5, 16, dtype=BF, device=DEV), torch.zeros(1, 16, 16, dtype=BF, device=DEV)
    ws = m.allocate_workspace(4096)
    y = torch.ones(5, 16, dtype=BF, device=DEV)
    assert lib.muon_expert_matmul(x.data_ptr(), 16, w.data_ptr(), off.data_ptr(), 0, 1, 1, 5, 16, 16, 0, y.data_ptr(), 16,
                                  ws.data_ptr(), ws.numel(), st) == 1
    assert (y == 1).all()


# --------------------------------------------------------------------------
# Offsets past 32 bits
# --------------------------------------------------------------------------

def test_expert_weights_past_32_bit_offsets(lib):
    """600 experts of 2048 x 2048 (2.5e9 weights); tokens at both ends."""
    e, d = 600, 2048
    w = torch.zeros(e, d, d, dtype=BF, device=DEV)
    g = gen(111)
    w[0], w[-1] = randn(g, (d, d), 0.05, BF), randn(g, (d, d), 0.05, BF)
    x = randn(g, (40, d), 1.0, BF)
    off = torch.full((e + 1,), 25, dtype=torch.int32, device=DEV)
    off[0], off[-1] = 0, 40
    for tr in (False, True):
        y = m.muon_expert_matmul(x, w, off, transpose=tr)
        for s, i in ((slice(0, 25), 0), (slice(25, 40), e - 1)):
            wd = w[i].double() if tr else w[i].double().t()
            want = x[s].double() @ wd
            within(y[s], want, rounded(mma_bound(d, x[s].double().abs() @ wd.abs()), want, BF), "y")
    dw = m.muon_expert_wgrad(y, x, off, out=w)
    for s, i in ((slice(0, 25), 0), (slice(25, 40), e - 1)):
        want = y[s].double().t() @ x[s].double()
        within(dw[i], want, rounded(mma_bound(25, y[s].double().abs().t() @ x[s].double().abs()), want, BF), "dw")
    assert (dw[1:-1].view(torch.int64) == 0).all()


def test_head_past_32_bit_offsets(lib):
    """300000 x 8192 head weights (2.5e9), targets in its first and last rows."""
    v, d = 300000, 8192
    g = gen(112)
    w = torch.empty(v, d, dtype=BF, device=DEV).normal_(0, 0.01, generator=g)
    h = randn(g, (5, d), 1.0, BF)
    t = torch.tensor([v - 1, 0, 299000, 5, v - 1], device=DEV)
    loss, lse, dh, dw = m.muon_linear_ce_grad(h, w, t)
    z = torch.cat([h.double() @ part.double().t() for part in w.split(20000)], dim=1)
    want = torch.logsumexp(z, 1)
    dz = mma_bound(d, (h.double().abs() @ w[:2000].double().abs().t()).max().item())  # random rows are alike
    assert ((lse.double() - want).abs() <= 2 * dz + 1e-5).all()
    p = torch.exp(z - want[:, None])
    p[torch.arange(5), t] -= 1
    tail = p[:, -1000:].t() @ h.double()
    mag = p[:, -1000:].abs().t() @ h.double().abs()
    within(dw[-1000:], tail, (2.0 ** -8 + 2 * dz) * mag + 2.0 ** -8 * tail.abs() + mma_bound(5, mag), "last rows of d_weight")


def test_embedding_grad_past_32_bit_offsets(lib):
    v, d = 300000, 8192
    grad = torch.ones(3, d, dtype=BF, device=DEV)
    ids = torch.tensor([v - 1, 7, v - 1], device=DEV)
    out = m.muon_embedding_grad(grad, ids, v)
    assert (out[v - 1] == 2).all() and (out[7] == 1).all() and (out[v - 2] == 0).all()
    assert out.sum(dtype=torch.float64).item() == 3 * d
