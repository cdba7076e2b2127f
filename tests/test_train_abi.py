"""Host-side checks of the operators around the step: argument validation and
workspace sizes.  No GPU needed: every refusal here comes before the device
is looked at."""
import ctypes

import pytest

import optimizer_muon_step_gb300 as m
from conftest import cuda_available
from optimizer_muon_step_gb300.train import LinearCe

P = ctypes.c_void_p
OK, INVALID, DTYPE, MISALIGNED, SMALL, NO_DEVICE = 0, 1, 2, 3, 4, 7


@pytest.fixture(scope="module")
def built():
    from optimizer_muon_step_gb300 import build
    build.build()
    return m.load_library()


def lookup(lib, table=4096, dt=1, ld=64, vocab=10, dim=64, ids=1 << 20, idt=1, n=4, scale=1.0, pad=-1, out=1 << 21,
           odt=1, old=64):
    return lib.muon_embedding_lookup(P(table), dt, ld, vocab, dim, P(ids), idt, n, scale, pad, P(out), odt, old, None)


def test_lookup_arguments(built):
    assert lookup(built, n=0) == OK
    for bad in (dict(n=-1), dict(vocab=0), dict(dim=0), dict(ld=63), dict(old=63), dict(table=None), dict(ids=None),
                dict(out=None), dict(vocab=1 << 31)):
        assert lookup(built, **bad) == INVALID, bad
    for bad in (dict(dt=3), dict(odt=-1), dict(idt=2)):
        assert lookup(built, **bad) == DTYPE, bad
    for bad in (dict(table=4097), dict(ids=(1 << 20) + 4), dict(out=(1 << 21) + 1), dict(dt=0, table=4098)):
        assert lookup(built, **bad) == MISALIGNED, bad


def egrad(lib, g=4096, dt=1, ld=64, ids=1 << 20, idt=1, n=4, vocab=10, dim=64, scale=1.0, pad=-1, acc=0, out=1 << 21,
          ws=1 << 22, wsb=1 << 20):
    return lib.muon_embedding_grad(P(g), dt, ld, P(ids), idt, n, vocab, dim, scale, pad, acc, P(out), P(ws), wsb, None)


def test_embedding_grad_arguments(built):
    for bad in (dict(n=-1), dict(vocab=0), dict(dim=0), dict(ld=63), dict(acc=2), dict(g=None), dict(ids=None),
                dict(out=None), dict(ws=None)):
        assert egrad(built, **bad) == INVALID, bad
    for bad in (dict(dt=3), dict(idt=-1)):
        assert egrad(built, **bad) == DTYPE, bad
    for bad in (dict(g=4097), dict(ids=(1 << 20) + 4), dict(out=(1 << 21) + 2), dict(ws=(1 << 22) + 128)):
        assert egrad(built, **bad) == MISALIGNED, bad
    need = built.muon_embedding_grad_workspace(4, 10, 64)
    assert 256 <= need < 1 << 16
    assert egrad(built, wsb=need - 1) == SMALL
    assert built.muon_embedding_grad_workspace(-1, 10, 64) == 0
    assert built.muon_embedding_grad_workspace(1 << 15, 10, 64) > built.muon_embedding_grad_workspace(1 << 14, 10, 64)


def ce(**kw):
    p = LinearCe()
    p.hidden, p.weight, p.targets, p.loss, p.lse = 1 << 12, 1 << 24, 1 << 25, 1 << 26, 1 << 27
    p.tokens, p.vocab, p.dim, p.hidden_ld, p.weight_ld, p.ignore_index = 8, 100, 64, 64, 64, -100
    p.dtype = p.d_weight_dtype = 1
    p.targets_dtype, p.logit_scale = 1, 1.0
    p.row_scale, p.d_hidden, p.d_weight = 1 << 28, 1 << 29, 1 << 30
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_cross_entropy_arguments(built):
    ws = P(1 << 32)
    for call in (built.muon_linear_ce, built.muon_linear_ce_grad):
        assert call(None, ws, 1 << 30, None) == INVALID
        for bad in (dict(tokens=-1), dict(vocab=0), dict(dim=0), dict(hidden_ld=63), dict(weight_ld=63), dict(reserved=1),
                    dict(hidden=None), dict(weight=None), dict(targets=None), dict(loss=None), dict(lse=None),
                    dict(logit_scale=float("inf")), dict(vocab=1 << 30)):
            assert call(ctypes.byref(ce(**bad)), ws, 1 << 30, None) == INVALID, bad
        for bad in (dict(dtype=0), dict(targets_dtype=2)):
            assert call(ctypes.byref(ce(**bad)), ws, 1 << 30, None) == DTYPE, bad
        for bad in (dict(hidden=4097), dict(weight=(1 << 24) + 1), dict(targets=(1 << 25) + 4), dict(lse=(1 << 27) + 2)):
            assert call(ctypes.byref(ce(**bad)), ws, 1 << 30, None) == MISALIGNED, bad
        assert call(ctypes.byref(ce()), P((1 << 32) + 64), 1 << 30, None) == MISALIGNED
        assert call(ctypes.byref(ce()), None, 1 << 30, None) == INVALID
        assert call(ctypes.byref(ce()), ws, 512, None) == SMALL
    grad = built.muon_linear_ce_grad
    assert grad(ctypes.byref(ce(d_weight=None)), ws, 1 << 30, None) == INVALID
    assert grad(ctypes.byref(ce(d_hidden=None)), ws, 1 << 30, None) == INVALID
    assert grad(ctypes.byref(ce(d_weight_dtype=2)), ws, 1 << 30, None) == DTYPE
    assert grad(ctypes.byref(ce(accumulate=1)), ws, 1 << 30, None) == INVALID
    assert grad(ctypes.byref(ce(d_weight=(1 << 30) + 2, d_weight_dtype=0)), ws, 1 << 30, None) == MISALIGNED
    assert built.muon_linear_ce(ctypes.byref(ce(tokens=0)), None, 0, None) == OK


def test_cross_entropy_workspace(built):
    size = lambda p, grad, budget: built.muon_linear_ce_workspace(ctypes.byref(p), grad, budget)  # noqa: E731
    big = ce(tokens=5000, vocab=32003, dim=1000, hidden_ld=1000, weight_ld=1000)
    whole = size(big, 1, 1 << 40)
    assert whole > 4 * 5000 * 32003                       # every token's logits at once
    least = size(big, 1, 0)
    assert 4 * 256 * 32003 < least < whole                 # 256 tokens' logits and the fp32 sums of d_weight
    for budget in (least, least + 1, (least + whole) // 2, whole - 1):
        got = size(big, 1, budget)
        assert least <= got <= budget
    # the loss alone keeps no logits
    assert size(big, 0, 1 << 40) < 64 * 5000 * 1000
    # rows that are not 16 bytes are packed
    assert size(ce(weight_ld=65, dim=65, hidden_ld=72), 0, 1 << 40) > size(ce(), 0, 1 << 40)
    assert size(ce(dim=0), 1, 1 << 40) == 0


@pytest.mark.parametrize("tokens,vocab,dim", [(2000, 32000, 7168), (2048 + 44, 4096, 4864), (5000, 1 << 17, 5120),
                                              (300, 50021, 13), (4096, 163840, 7168)])
def test_cross_entropy_takes_the_workspace_it_asked_for(built, tokens, vocab, dim):
    """Whatever the budget: the size asked for is enough, also when it is the
    budget."""
    p = ce(tokens=tokens, vocab=vocab, dim=dim, hidden_ld=dim, weight_ld=dim, targets=1 << 60, loss=1 << 61, lse=1 << 62,
           weight=1 << 50, d_hidden=1 << 57, d_weight=1 << 58)
    whole = built.muon_linear_ce_workspace(ctypes.byref(p), 1, 1 << 60)
    for i in range(41):
        got = built.muon_linear_ce_workspace(ctypes.byref(p), 1, whole * i // 40)
        assert built.muon_linear_ce_workspace(ctypes.byref(p), 1, got) <= got
        assert built.muon_linear_ce_grad(ctypes.byref(p), P(1 << 40), got, None) != SMALL


def test_cross_entropy_workspace_of_a_short_last_block(built):
    """1024 tokens' d_hidden (4 x 19 tiles, one per pair of CTAs) is summed in
    one piece, 44 tokens' in at least two, which take room of their own: what
    holds 2048 tokens in two such blocks does not hold 44 more in a third."""
    of = dict(vocab=4096, dim=4864, hidden_ld=4864, weight_ld=4864, d_weight_dtype=0)
    size = lambda n, budget: built.muon_linear_ce_workspace(ctypes.byref(ce(tokens=n, **of)), 1, budget)  # noqa: E731
    block = size(1024, 1 << 40)
    assert size(2048, block) == block
    more = next(extra for extra in range(0, 16 << 20, 256) if size(2048 + 44, block + extra) >= block)
    assert more >= 2 * 4 * 44 * 4864


def mm(lib, x=4096, xld=64, w=1 << 20, off=1 << 22, odt=0, dt=1, e=3, n=10, r=32, c=64, tr=0, y=1 << 23, yld=32,
       ws=1 << 24, wsb=1 << 20):
    return lib.muon_expert_matmul(P(x), xld, P(w), P(off), odt, dt, e, n, r, c, tr, P(y), yld, P(ws), wsb, None)


def wg(lib, g=4096, gld=32, x=1 << 20, xld=64, off=1 << 22, odt=0, dt=1, e=3, n=10, r=32, c=64, dw=1 << 23, dwt=1, acc=0,
       ws=1 << 24, wsb=1 << 20):
    return lib.muon_expert_wgrad(P(g), gld, P(x), xld, P(off), odt, dt, e, n, r, c, P(dw), dwt, acc, P(ws), wsb, None)


def test_expert_arguments(built):
    assert mm(built, n=0) == OK
    for bad in (dict(n=-1), dict(e=0), dict(r=0), dict(c=0), dict(xld=63), dict(yld=31), dict(tr=2), dict(x=None),
                dict(w=None), dict(off=None), dict(y=None), dict(ws=None), dict(e=65537), dict(tr=1, xld=31)):
        assert mm(built, **bad) == INVALID, bad
    for bad in (dict(dt=0), dict(odt=2)):
        assert mm(built, **bad) == DTYPE, bad
    for bad in (dict(x=4097), dict(w=(1 << 20) + 1), dict(off=(1 << 22) + 2), dict(y=(1 << 23) + 1), dict(ws=(1 << 24) + 8)):
        assert mm(built, **bad) == MISALIGNED, bad
    assert mm(built, wsb=255) == SMALL
    for bad in (dict(n=-1), dict(e=0), dict(gld=31), dict(xld=63), dict(acc=1), dict(acc=2, dwt=0), dict(g=None),
                dict(x=None), dict(off=None), dict(dw=None), dict(ws=None)):
        assert wg(built, **bad) == INVALID, bad
    for bad in (dict(dt=0), dict(dwt=2), dict(odt=5)):
        assert wg(built, **bad) == DTYPE, bad
    assert wg(built, dw=(1 << 23) + 2, dwt=0) == MISALIGNED
    assert wg(built, wsb=256) == SMALL                     # the experts' tensor maps


@pytest.mark.skipif(cuda_available(), reason="checks the no-device path")
def test_without_device(built):
    assert lookup(built) == NO_DEVICE
    assert egrad(built) == NO_DEVICE
    assert mm(built) == NO_DEVICE and wg(built) == NO_DEVICE
    assert built.muon_linear_ce(ctypes.byref(ce()), P(1 << 32), 1 << 30, None) == NO_DEVICE


def test_binding_declares_every_entry_point(built):
    for name in m.train.EXPORTS:
        assert getattr(built, name).argtypes is not None, name
    assert len(m.KERNEL_KINDS) == 19
    for i, kind in enumerate(m.KERNEL_KINDS):
        assert built.muon_kernel_name(i).decode() == kind
