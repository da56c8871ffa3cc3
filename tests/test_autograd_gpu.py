"""The differentiable wrapper (torch.autograd.Function over the C ABI)
against the oracle, and against direct C-ABI calls bit for bit.

Gradients are taken of the scalar sum(O * dO), so q.grad, k.grad and v.grad
are the VJP the oracle computes for cotangent dO.
"""
import math

import numpy as np
import pytest
import torch

import fa_inputs
import oracle

GRAD_TOL, O_TOL, LSE_TOL = 1e-2, 2e-2, 1e-3


def _wrapper():
    from attention_fa_fwd_03_gb300.autograd import flash_attention
    return flash_attention


def _rel_fro(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def _run(x, w, **kw):
    flash_attention = _wrapper()
    dev = torch.device("cuda")
    q, k, v = (x[n].to(dev).requires_grad_() for n in ("q", "k", "v"))
    do = x["do"].to(dev)
    o, lse = flash_attention(q, k, v, w.scale, w.causal, w.window, return_lse=True, **kw)
    (o.float() * do.float()).sum().backward()
    torch.cuda.synchronize()
    return {"o": o.detach(), "lse": lse, "dq": q.grad, "dk": k.grad, "dv": v.grad}


CASES = [
    ("c1_b1_h2x1_t64_d64_fp16_causal", None),
    (None, fa_inputs.Workload("ag_gqa_window", 1, 4, 2, 300, 300, 128, "bf16", True, 64, seed=41)),
    (None, fa_inputs.Workload("ag_cross", 2, 4, 1, 90, 200, 96, "fp16", False, 0, seed=42)),
    # decode-shaped: split-key forward and dQ, folded dK/dV
    (None, fa_inputs.Workload("ag_short", 2, 8, 2, 4, 600, 128, "bf16", False, 0, seed=45)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("name,w", CASES)
def test_autograd_matches_oracle(name, w):
    w = w or fa_inputs.WORKLOADS[name]
    x = fa_inputs.make_inputs(w)
    got = {n: t.double().cpu().numpy() for n, t in _run(x, w).items()}
    ref = oracle.attn_bwd(*(x[n].double().numpy() for n in ("q", "k", "v", "do")),
                          w.scale, w.causal, w.window)
    assert np.abs(got["o"] - ref["o"]).max() <= O_TOL
    fin = np.isfinite(ref["lse"])
    assert np.array_equal(fin, np.isfinite(got["lse"]))
    assert np.abs(got["lse"][fin] - ref["lse"][fin]).max() <= LSE_TOL
    for n in ("dq", "dk", "dv"):
        assert _rel_fro(got[n], ref[n]) <= GRAD_TOL, n


@pytest.mark.gpu
def test_autograd_equals_direct_abi_calls():
    """Same kernels, same inputs: the wrapper adds no arithmetic of its own."""
    import attention_fa_fwd_03_gb300 as fa
    w = fa_inputs.Workload("ag_direct", 1, 4, 2, 257, 257, 128, "bf16", True, seed=43)
    x = fa_inputs.make_inputs(w)
    got = _run(x, w)
    dev = torch.device("cuda")
    q, k, v, do = (x[n].to(dev) for n in ("q", "k", "v", "do"))
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=dev)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(fa.fa_bwd_workspace_size(*q.shape[:3]), dtype=torch.uint8, device=dev)
    fa.fa_fwd(q, k, v, o, lse, w.scale, w.causal, w.window)
    # the wrapper's cotangent of sum(O * dO) taken in fp32 is dO cast back to O's dtype
    fa.fa_bwd(q, k, v, o, do, lse, dq, dk, dv, w.scale, w.causal, w.window, workspace=ws)
    torch.cuda.synchronize()
    for n, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(got[n], t), n


@pytest.mark.gpu
def test_autograd_default_scale_and_noncontiguous_inputs():
    flash_attention = _wrapper()
    w = fa_inputs.Workload("ag_layout", 1, 2, 1, 130, 130, 64, "fp16", True, seed=44)
    x = fa_inputs.make_inputs(w)
    dev = torch.device("cuda")
    # [B, T, H, D] storage viewed as [B, H, T, D]: not contiguous
    q, k, v = (x[n].transpose(1, 2).contiguous().to(dev).transpose(1, 2) for n in ("q", "k", "v"))
    assert not q.is_contiguous()
    for t in (q, k, v):
        t.requires_grad_()
    o = flash_attention(q, k, v, causal=True)   # scale defaults to 1/sqrt(D)
    o.backward(x["do"].to(dev))
    torch.cuda.synchronize()
    ref = oracle.attn_bwd(*(x[n].double().numpy() for n in ("q", "k", "v", "do")),
                          1.0 / math.sqrt(w.D), True, 0)
    assert np.abs(o.detach().double().cpu().numpy() - ref["o"]).max() <= O_TOL
    for n, t in (("dq", q), ("dk", k), ("dv", v)):
        assert _rel_fro(t.grad.double().cpu().numpy(), ref[n]) <= GRAD_TOL, n


def test_autograd_has_no_cpu_path():
    """CPU tensors are refused (or the missing library is reported), never computed."""
    flash_attention = _wrapper()
    q = torch.zeros(1, 2, 8, 64, dtype=torch.float16, requires_grad=True)
    k = torch.zeros(1, 1, 8, 64, dtype=torch.float16)
    with pytest.raises((ValueError, RuntimeError)):
        flash_attention(q, k, k)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 0), (70, 9)])
def test_function_and_node_give_the_same_bits(window, sinks):
    """flash_attention's compiled node and the Function over the same calls, with gradients of some inputs only."""
    from attention_fa_fwd_03_gb300.autograd import FlashAttention, flash_attention
    w = fa_inputs.Workload("ag_node", 2, 4, 2, 300, 260, 96, "bf16", False, seed=46)
    x = {n: t.cuda() for n, t in fa_inputs.make_inputs(w).items()}
    for wanted in (("q", "k", "v"), ("q",), ("v",)):
        ins = {n: x[n].clone().requires_grad_(n in wanted) for n in ("q", "k", "v")}
        o, lse = flash_attention(*ins.values(), 0.1, True, window, return_lse=True, sinks=sinks)
        of, lf = FlashAttention.apply(*ins.values(), 0.1, True, window, *([sinks] if sinks else []))
        assert torch.equal(o, of) and torch.equal(lse, lf) and not lse.requires_grad and o.requires_grad
        a, b = (torch.autograd.grad(y, [ins[n] for n in wanted], x["do"]) for y in (o, of))
        assert all(torch.equal(i, j) for i, j in zip(a, b))
    with torch.no_grad():
        assert flash_attention(*ins.values(), 0.1, True, window, sinks=sinks).grad_fn is None


@pytest.mark.gpu
def test_node_errors():
    """What the library refuses is an FaError with its status, from the forward and from the graph's thread; saved inputs
    that were written since are found; shapes, types and devices that do not fit are refused."""
    import attention_fa_fwd_03_gb300 as fa
    flash_attention = _wrapper()
    q = torch.randn(1, 4, 40, 64, device="cuda").half().requires_grad_()
    k = torch.randn(1, 2, 50, 64, device="cuda").half().requires_grad_()
    with pytest.raises(fa.FaError) as e:
        flash_attention(q, k, k, window=-1)
    assert e.value.status == 1
    with pytest.raises(fa.FaError):
        flash_attention(q.float(), k.float(), k.float())
    with pytest.raises(fa.FaError):
        flash_attention(q[..., :40], k[..., :40], k[..., :40])
    for a in ((q, k.bfloat16(), k), (q, k, k[:, :, :30]), (q, k[..., :32], k[..., :32]), (q, k.cpu(), k), (q[0], k, k),
              (q, k.expand(2, -1, -1, -1), k.expand(2, -1, -1, -1))):
        with pytest.raises(ValueError):
            flash_attention(*a)
    o = flash_attention(q, k, k)
    odd = torch.empty(o.numel() + 1, dtype=o.dtype, device="cuda")[1:].view(o.shape)  # two bytes off
    with pytest.raises(fa.FaError) as e:
        o.backward(odd)
    assert e.value.status == 4
    o = flash_attention(q, k, k)
    with torch.no_grad():
        k.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        o.backward(torch.ones_like(o))
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_captured_backward_beside_an_eager_graph():
    """A backward captured while an eager graph of the same leaves lives cannot be where the leaves were used on the default
    stream: refused, with the process as it was, and captured once the eager graph is gone."""
    code = """
import torch
from attention_fa_fwd_03_gb300.autograd import flash_attention
q, k, v = (torch.randn(1, 2, 100, 64, device="cuda").half().requires_grad_() for _ in range(3))
do = torch.randn(1, 2, 100, 64, device="cuda").half()
eager = flash_attention(q, k, v, causal=True)
side = torch.cuda.Stream()
torch.cuda.synchronize()
def grads():
    return torch.autograd.grad(flash_attention(q, k, v, causal=True), (q, k, v), do)
for f in (lambda: flash_attention(q, k, v, causal=True).backward(do), grads):
    g = torch.cuda.CUDAGraph()
    try:
        with torch.cuda.graph(g, stream=side):
            f()
        print("captured")
    except RuntimeError as e:
        print("refused" if "eager graph" in str(e) else e)
want = torch.autograd.grad(eager, (q, k, v), do)
del eager
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=side):
    got = grads()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
q.grad = k.grad = v.grad = None
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=side):
    flash_attention(q, k, v, causal=True).backward(do)
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a.grad, b) for a, b in zip((q, k, v), want))
print("done")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["refused", "refused", "done"], (r.stdout, r.stderr[-2000:])
