"""Second derivatives, which differentiable attention does not have: asking for one raises, under either name."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def names():
    from attention_fa_fwd_03_gb300.autograd import FlashAttention, flash_attention
    return {"flash_attention": lambda *a: flash_attention(*a, causal=True),
            "FlashAttention": lambda q, k, v: FlashAttention.apply(q, k, v, q.shape[-1] ** -0.5, True, 0)[0]}


def inputs(*wanted):
    g = torch.Generator().manual_seed(5)
    x = [torch.randn(1, 4, 130, 64, generator=g).half().cuda() for _ in range(4)]
    return [t.requires_grad_(n in wanted) for n, t in zip("qkv", x)] + [x[3]]


@pytest.mark.parametrize("name", ["flash_attention", "FlashAttention"])
@pytest.mark.parametrize("wanted", ["q", "kv", "qkv"])
def test_second_derivatives_raise(name, wanted):
    """Gradients made with create_graph are the same numbers; what is differentiated through them raises, also where other
    terms of the sum have a derivative, and whether or not the cotangent has one."""
    attend = names()[name]
    q, k, v, do = inputs(*wanted)
    leaves = [t for n, t in zip("qkv", (q, k, v)) if n in wanted]
    plain = torch.autograd.grad(attend(q, k, v), leaves, do)
    for cotangent in (do, do.clone().requires_grad_()):
        grads = torch.autograd.grad(attend(q, k, v), leaves, cotangent, create_graph=True)
        assert all(torch.equal(a, b) and a.requires_grad for a, b in zip(grads, plain))
        penalty = sum((g.float() ** 2).sum() for g in grads) + sum((t.float() ** 2).sum() for t in leaves)
        with pytest.raises(RuntimeError, match="second derivative"):
            penalty.backward()
    for t in leaves:  # (what was added before it raised)
        t.grad = None
    assert not any(g.requires_grad for g in plain)
    attend(q, k, v).backward(do, create_graph=True)
    assert all(torch.equal(t.grad, g) for t, g in zip(leaves, plain))
    for t in leaves:
        t.grad = None  # (a cycle of gradients and their leaves else)
