"""Calls that tensors with a gradient reach: differentiated, or refused."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

from tests.test_gpu_kv8 import cu_of, fill, gen, ints

pytestmark = pytest.mark.gpu


def test_rope_apply_has_a_gradient(tq_lib, cuda):
    r = tq_lib.Rope(64, 32, layout="interleaved")
    x = torch.randn(5, 2, 64, generator=gen(1)).to(cuda).requires_grad_()
    pos = torch.arange(5, device=cuda)
    w = torch.randn(5, 2, 64, generator=gen(2)).to(cuda)
    for transpose in (False, True):
        y = r.apply(x, pos, transpose=transpose)
        g, = torch.autograd.grad((y * w).sum(), x)
        assert torch.equal(g, r.apply(w, pos, transpose=not transpose))
        assert torch.equal(y, r.apply(x.detach(), pos, transpose=transpose))
    with torch.no_grad():
        assert not r.apply(x, pos).requires_grad


def test_rope_refuses_what_has_no_derivative(tq_lib, cuda):
    r = tq_lib.Rope(64)
    pos = torch.arange(5, device=cuda)
    x = torch.randn(5, 2, 64, device=cuda)
    leaf = x.clone().requires_grad_()
    for a, out in ((leaf, torch.empty_like(x)), (x, leaf), (leaf, leaf)):
        with pytest.raises(ValueError):
            r.apply(a, pos, out=out)
    with torch.no_grad():
        r.apply(leaf, pos, out=torch.empty_like(x))
    with fwAD.dual_level():
        dual = fwAD.make_dual(x, torch.ones_like(x))
        with pytest.raises((ValueError, RuntimeError)):
            r.apply(dual, pos)
        with pytest.raises((ValueError, RuntimeError)):
            r(dual, pos)


def test_the_cache_refuses_gradients(tq_lib, cuda):
    c = fill(tq_lib, cuda, "i8", 2, 64, 32, [40])
    x = torch.randn(1, 2, 64, device=cuda)
    q = torch.randn(1, 4, 64, device=cuda).to(torch.bfloat16)
    cu = cu_of([1], cuda)
    before = c.k.clone()
    for k, v in ((x.clone().requires_grad_(), x), (x, x.clone().requires_grad_())):
        with pytest.raises(ValueError):
            c.append(0, k, v, cu, 1)
    assert torch.equal(c.k, before)
    leaf = q.clone().requires_grad_()
    with pytest.raises(ValueError):
        c.attention(0, leaf, cu, 1)
    with pytest.raises(ValueError):
        c.attention(0, q, cu, 1, out=torch.empty_like(q).requires_grad_())
    with pytest.raises(ValueError):
        c.attention(0, q, cu, 1, lse=torch.empty(1, 4, device=cuda).requires_grad_())
    want = c.attention(0, q, cu, 1)
    with torch.no_grad():
        assert torch.equal(c.attention(0, leaf, cu, 1), want)
        c.append(0, x.requires_grad_(), x, cu, 1)
    with fwAD.dual_level():
        with pytest.raises(ValueError):
            c.attention(0, fwAD.make_dual(q, torch.ones_like(q)), cu, 1)
    c.status()


def test_outputs_that_a_graph_holds(tq_lib, cuda):
    """A tensor that is written into counts as changed: a backward pass that needs
    its old values says so."""
    r = tq_lib.Rope(64)
    c = fill(tq_lib, cuda, "i8", 2, 64, 32, [40])
    pos, cu = torch.arange(1, device=cuda), cu_of([1], cuda)
    q = torch.randn(1, 4, 64, device=cuda).to(torch.bfloat16)

    def held(shape, dtype, write):
        t = torch.randn(shape, device=cuda).to(dtype)
        w = torch.ones_like(t).requires_grad_()
        y = (w * t).sum()
        write(t)
        with pytest.raises(RuntimeError):
            y.backward()
    held((1, 4, 64), torch.bfloat16, lambda t: r.apply(t, pos, out=t))
    held((1, 4, 64), torch.bfloat16, lambda t: c.attention(0, q, cu, 1, out=t))
    held((1, 4), torch.float32, lambda t: c.attention(0, q, cu, 1, lse=t))
    with torch.inference_mode():
        t = torch.randn(1, 4, 64, device=cuda)
        r.apply(t, pos, out=t)
    r.apply(t, pos, out=t)  # (a tensor without a version)


def test_outputs_that_overlap(tq_lib, cuda):
    r = tq_lib.Rope(64)
    c = fill(tq_lib, cuda, "i8", 2, 64, 32, [40])
    pos = torch.arange(3, device=cuda)
    x = torch.randn(3, 4, 64, device=cuda)
    line = torch.randn(4 * 4 * 64, device=cuda)
    with pytest.raises(ValueError):  # one row for all tokens
        r.apply(x, pos, out=torch.empty(1, 4, 64, device=cuda).expand(3, 4, 64))
    with pytest.raises(ValueError):  # shifted by a token
        r.apply(line[:768].view(3, 4, 64), pos, out=line[256:].view(3, 4, 64))
    half = line.to(torch.bfloat16)
    with pytest.raises(ValueError):
        c.attention(0, half[:768].view(3, 4, 64), cu_of([3], cuda), 3, out=half[256:].view(3, 4, 64))
    r.apply(x, pos, out=x)
    whole = half[:768].view(3, 4, 64)
    want = c.attention(0, whole, cu_of([3], cuda), 3)  # the same memory: each row after it is read
    assert torch.equal(c.attention(0, whole, cu_of([3], cuda), 3, out=whole), want)
