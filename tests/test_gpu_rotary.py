"""Rotary positions against their definition in 64 bits, with gradients."""

import pytest

import kv_util as ref
from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


def _rotary():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import rotary
    return torch, rotary


def _check(torch, got, x, positions, turns, magnitude, interleaved, inverse=False):
    """Half a step of the type, and 2^-20 of the terms: a sine or cosine is off by the
    rounding of its angle (2^-25 turns, 2 pi of it) and a few units of fp32."""
    want, terms = ref.rotate(x, positions, turns, magnitude, interleaved, inverse)
    half = torch.finfo(x.dtype).eps / 2
    tiny = torch.finfo(x.dtype).smallest_normal * half      # half a subnormal step
    assert got.dtype == x.dtype and got.shape == x.shape and got.is_contiguous()
    bound = half * want.abs() + 2.0 ** -20 * terms + tiny
    n = 2 * turns.numel()
    assert bool(((got.double() - want).abs() <= bound)[..., :n].all())
    assert torch.equal(got[..., n:], x[..., n:])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,hq,hk,d,turned", [(1, 1, 1, 64, 64), (7, 4, 2, 128, 128), (33, 8, 1, 64, 32), (5, 3, 3, 80, 40), (9, 2, 1, 6, 6),
                                              (4, 2, 2, 33, 14), (130, 32, 8, 128, 64), (3, 1, 1, 256, 0), (2050, 5, 2, 96, 96)])
def test_rotate(dtype, interleaved, t, hq, hk, d, turned):
    torch, rotary = _rotary()
    g = torch.Generator(device="cuda").manual_seed(t + d)
    dt = getattr(torch, dtype)
    q, k = (torch.randn((t, h, d), generator=g, device="cuda").to(dt) for h in (hq, hk))
    positions = torch.randint(0, 100000, (t,), generator=g, device="cuda", dtype=torch.int32)
    turns = rotary.turns(turned, device="cuda")[0] if turned else torch.zeros(0, dtype=torch.float64, device="cuda")
    log("rotate %s T=%d heads=%d/%d D=%d of which %d, interleaved=%s" % (dtype, t, hq, hk, d, turned, interleaved))
    q2, k2 = rotary.rotate(q, k, positions, turns, interleaved=interleaved, magnitude=1.25)
    _check(torch, q2, q, positions, turns, 1.25, interleaved)
    _check(torch, k2, k, positions, turns, 1.25, interleaved)
    assert torch.equal(rotary.rotate(q, None, positions, turns, interleaved=interleaved, magnitude=1.25), q2)


def test_far_positions():
    """Positions up to 2^31 - 1, and negative ones: the angle is reduced in 64 bits."""
    torch, rotary = _rotary()
    positions = torch.tensor([0, 1, -1, 2 ** 20, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    q = torch.randn((7, 2, 128), device="cuda")
    turns = rotary.turns(128, device="cuda")[0]
    _check(torch, rotary.rotate(q, None, positions, turns), q, positions, turns, 1.0, False)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("which", ["both", "q", "k", "alone"])
def test_gradients(dtype, interleaved, which):
    torch, rotary = _rotary()
    dt = getattr(torch, dtype)
    q, k = (torch.randn((19, h, 64), device="cuda").to(dt) for h in (4, 2))
    dq, dk = (torch.randn((19, h, 64), device="cuda").to(dt) for h in (4, 2))
    positions = torch.randint(0, 5000, (19,), device="cuda", dtype=torch.int32)
    turns = rotary.turns(48, device="cuda")[0]
    log("gradients %s %s interleaved=%s" % (dtype, which, interleaved))
    q.requires_grad_(which != "k")
    k.requires_grad_(which in ("both", "k"))
    if which == "alone":
        out = rotary.rotate(q, None, positions, turns, interleaved=interleaved, magnitude=0.75)
        grads = {"q": torch.autograd.grad(out, q, dq)[0]}
    else:
        oq, ok = rotary.rotate(q, k, positions, turns, interleaved=interleaved, magnitude=0.75)
        leaves = [x for x in (q, k) if x.requires_grad]
        grads = dict(zip([n for n, x in (("q", q), ("k", k)) if x.requires_grad], torch.autograd.grad((oq, ok), leaves, (dq, dk))))
    for name, d in (("q", dq), ("k", dk)):
        if name in grads:
            _check(torch, grads[name], d, positions, turns, 0.75, interleaved, inverse=True)


def test_gradient_of_one_output():
    """Only one of the outputs is used; expanded and transposed gradients."""
    torch, rotary = _rotary()
    q, k = (torch.randn((6, h, 64), device="cuda", requires_grad=True) for h in (4, 2))
    positions = torch.arange(6, device="cuda", dtype=torch.int32)
    turns = rotary.turns(64, device="cuda")[0]
    oq, ok = rotary.rotate(q, k, positions, turns)
    gq, gk = torch.autograd.grad(ok.sum(), (q, k), allow_unused=True)
    assert gq is None or not bool(gq.any())
    _check(torch, gk, torch.ones_like(ok), positions, turns, 1.0, False, inverse=True)
    oq, ok = rotary.rotate(q, k, positions, turns)
    d = torch.randn((64, 4, 6), device="cuda").permute(2, 1, 0)
    gq, = torch.autograd.grad(oq, q, d)
    _check(torch, gq, d.contiguous(), positions, turns, 1.0, False, inverse=True)


def test_gradient_against_differences():
    torch, rotary = _rotary()
    q = torch.randn((3, 1, 8), device="cuda", requires_grad=True)
    positions = torch.tensor([0, 5, 77], dtype=torch.int32, device="cuda")
    turns = rotary.turns(6, base=50.0, device="cuda")[0]
    d = torch.randn((3, 1, 8), device="cuda")
    g, = torch.autograd.grad(rotary.rotate(q, None, positions, turns, interleaved=True, magnitude=1.5), q, d)
    # linear: a difference over a step of 1 has no error but rounding
    for i in range(q.numel()):
        e = torch.zeros(q.numel(), device="cuda")
        e[i] = 1.0
        e = e.view_as(q)
        with torch.no_grad():
            up, down = (rotary.rotate((q + s * e).detach(), None, positions, turns, interleaved=True, magnitude=1.5) for s in (0.5, -0.5))
        assert abs(float(((up - down) * d).sum()) - float(g.view(-1)[i])) < 1e-4


def test_strides():
    """Heads of a packed projection, head-major tensors, rows that are no multiple of 16 bytes apart."""
    torch, rotary = _rotary()
    positions = torch.arange(40, 51, device="cuda", dtype=torch.int32)
    turns = rotary.turns(64, device="cuda")[0]
    for dt in (torch.bfloat16, torch.float32):
        x = torch.randn((11, 8, 128), device="cuda").to(dt)
        want = rotary.rotate(x[:, :5].contiguous(), x[:, 5:7].contiguous(), positions, turns)
        wide = torch.randn((11, 8, 131), device="cuda").to(dt)
        wide[..., 3:] = x
        for q, k in ((x[:, :5], x[:, 5:7]), (x[:, :5].transpose(0, 1).contiguous().transpose(0, 1), x[:, 5:7]),
                     (wide[:, :5, 3:], wide[:, 5:7, 3:])):
            for a, b in zip(rotary.rotate(q, k, positions, turns), want):
                assert torch.equal(a, b)
        one = x[:1, :1].expand(11, 5, 128)          # the same row for every token and head
        assert torch.equal(rotary.rotate(one, None, positions, turns), rotary.rotate(one.contiguous(), None, positions, turns))


def test_no_tokens():
    torch, rotary = _rotary()
    q = torch.zeros((0, 4, 64), device="cuda")
    positions = torch.zeros(0, dtype=torch.int32, device="cuda")
    a, b = rotary.rotate(q, q, positions, rotary.turns(64, device="cuda")[0])
    assert a.shape == b.shape == (0, 4, 64)


def test_more_than_two_gigabytes():
    """Elements past 2^31, sampled."""
    torch, rotary = _rotary()
    t, h, d = 270000, 64, 128
    log("rotate %d x %d x %d" % (t, h, d))
    q = torch.empty((t, h, d), dtype=torch.bfloat16, device="cuda").normal_()
    positions = torch.arange(t, device="cuda", dtype=torch.int32)
    turns = rotary.turns(d, device="cuda")[0]
    got = rotary.rotate(q, None, positions, turns)
    for at in (0, 131070, 262143, 262144, t - 3):
        rows = slice(at, at + 3)
        _check(torch, got[rows].contiguous(), q[rows], positions[rows], turns, 1.0, False)


def test_refusals():
    torch, rotary = _rotary()
    log("refusals of rotate")
    q, k = torch.zeros((3, 4, 64), device="cuda"), torch.zeros((3, 2, 64), device="cuda")
    p = torch.zeros(3, dtype=torch.int32, device="cuda")
    t = rotary.turns(64, device="cuda")[0]
    for args in ((q.double(), k, p, t), (q[0], k, p, t), (q, k.bfloat16(), p, t), (q, k[:2], p, t), (q, k[..., :32], p, t),
                 (q, k, p.long(), t), (q, k, p[:2], t), (q, k, p, t.float()), (q, k, p, torch.cat((t, t))), (q, k, p.cpu(), t),
                 (q, k.cpu(), p, t), (q.transpose(1, 2), k, p, t), (q, k, p, t[None])):
        with pytest.raises(ValueError):
            rotary.rotate(*args)
    with pytest.raises(TypeError):
        rotary.rotate(q, k, p, t, magnitude="x")
    with pytest.raises(ValueError, match="gradient"):
        rotary.rotate(q, k, p, t.clone().requires_grad_())
    g, = torch.autograd.grad(rotary.rotate(q.requires_grad_(), None, p, t).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        g.sum().backward()
    import torch.autograd.forward_ad as fwad
    with fwad.dual_level():
        dual = fwad.make_dual(k, torch.ones_like(k))
        for args in ((dual, None), (k, dual)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                rotary.rotate(args[0], args[1], p, t)
