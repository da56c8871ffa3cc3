"""Weights of dense attention in fp16 beside a dominating key: the tile kernels (more than 8 query rows), the masks they are
built for and the window with visible first keys, where a first key dominates as a rule.

What a weight may lose. It goes to the product with V, times 2^7, as one fp16 number: off by 2^-11 of itself, and where it is
small by half of fp16's smallest number, 2^-25: 2^-32 of the largest weight (the running maximum may be behind the largest
score, never ahead)."""
import math

import pytest
import torch

import attention_fa_fwd_03_gb300 as fa

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("weight", [1.4 * 2.0 ** -24, 0.9 * 2.0 ** -25])
@pytest.mark.parametrize("T,N,causal,window,sinks", [(100, 700, False, 0, 0), (3000, 3000, True, 0, 0), (3000, 3000, True, 400, 1),
                                                     (600, 900, False, 130, 3), (40, 20000, False, 0, 0)])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_small_weights_beside_a_dominating_key(D, T, N, causal, window, sinks, weight):
    """The first key has the largest score and V = 0; the others have a weight far below fp16's normal numbers, V = c, and hold
    all of the row. (In fp16 as it is, 1.4 2^-24 is 2^-24 and 0.9 2^-25 is nothing.)"""
    B, H = 2, 2
    c = 2.0 ** 14
    k = torch.zeros(B, H, N, D, dtype=torch.float16, device="cuda")
    k[:, :, 1:, 0] = -1
    v = torch.full((B, H, N, D), c, dtype=torch.float16, device="cuda")
    v[:, :, 0] = 0
    q = torch.zeros(B, H, T, D, dtype=torch.float16, device="cuda")
    q[..., 0] = 1
    scale = float(torch.tensor(-math.log(weight), dtype=torch.float32))
    w = math.exp(-scale)
    o, lse = torch.full_like(q, float("nan")), torch.full((B, H, T), float("nan"), device="cuda")
    fa.fa_fwd(q, k, v, o, lse, scale, causal, window, sinks=sinks)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    i, j = torch.arange(T)[:, None], torch.arange(N)
    see = torch.ones(T, N, dtype=torch.bool)
    if causal:
        see &= j <= i
    if window:
        see &= ~((i - j >= window) & (j >= sinks))
    first, small = see[:, 0].double(), see[:, 1:].sum(1).double()
    want = c * small * w / (first + small * w)
    h = 2.0 ** -11
    near = 2 * (2 * D + 8) * U * scale + 2.0 ** -20 + 2 * (N + 16) * U
    off = near + 2.0 ** -11 + 2.0 ** -32 / w
    bound = h * want + (1 + h) * off * want + 2.0 ** -25
    rounded = float(torch.tensor(w).half()) / w
    some = want > 2.0 ** -8  # (else fp16's smallest number is more)
    assert (abs(rounded - 1) * want > 5 * bound)[some].all()  # the oracle without headroom does not pass
    assert some.any()
    got = o.double().cpu()
    assert ((got - want[:, None]).abs() <= bound[:, None]).all(), float(((got - want[:, None]).abs() / bound[:, None]).max())
    ln = torch.log(first + small * w)
    assert ((lse.double().cpu() - ln).abs() <= 2.0 ** -20 + 2 * (N + 16) * U + 8 * U * scale).all()
