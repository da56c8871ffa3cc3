"""Weights of attention over a cache of fp16 values beside dominating keys, in every kernel: clusters (short lists) and split
lists of up to 8, 16, 32, 64 and 128 rows per KV head, bf16 beside it.

What a weight may lose. fp16: it goes to the product with V, times 2^7, in two numbers, so it is off by 2^-22 of itself, and
where it is small by half of fp16's smallest number, 2^-25: 2^-32 of the largest weight (the running maximum may be behind the
largest score, never ahead). bf16: two numbers, 2^-17 of itself, and no smallest number within reach."""
import math

import pytest
import torch

import attention_fa_fwd_03_gb300 as fa

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
PAGE = 64


@pytest.mark.parametrize("weight", [1.4 * 2.0 ** -24, 0.9 * 2.0 ** -25])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("n", [500, 30000])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("heads", [4, 12, 20, 40, 100])
@pytest.mark.parametrize("window", [0, 1])
def test_small_weights_beside_dominating_keys(heads, D, n, dt, weight, window):
    """Every 16th key has the largest score and V = 0; the others have a weight far below fp16's normal numbers, V = c, and hold
    all of the row. (In fp16 as it is, 1.4 2^-24 is 2^-24 and 0.9 2^-25 is nothing.) With a window of half the keys and the
    first 16 visible beside it, too."""
    dtype = DT[dt]
    pages = -(-n // PAGE)
    k = torch.zeros(pages, 1, PAGE, D, dtype=dtype)
    k[..., 0] = -1
    k[:, :, ::16, 0] = 0
    c = 2.0 ** 14
    v = torch.full((pages, 1, PAGE, D), c, dtype=dtype)
    v[:, :, ::16] = 0
    q = torch.zeros(1, heads, 1, D, dtype=dtype, device="cuda")
    q[..., 0] = 1
    scale = float(torch.tensor(-math.log(weight), dtype=torch.float32))
    w = math.exp(-scale)
    kv = fa.PagedKV(k.cuda(), v.cuda(), torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                    torch.tensor([n], dtype=torch.int32, device="cuda"))
    o, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
    ws = torch.full((fa.fa_paged_workspace_size(heads, 1, 1, D),), 255, dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(kv, q, o, lse, scale, causal=True, window=window * (n // 2), sinks=16 * window, workspace=ws)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    o, lse = o.double().cpu(), lse.double().cpu()
    j = torch.arange(n)
    see = (n - 1 - j < n // 2) | (j < 16) if window else j >= 0
    big, small = int((see & (j % 16 == 0)).sum()), int((see & (j % 16 > 0)).sum())
    want = c * small * w / (big + small * w)
    h = torch.finfo(dtype).eps / 2
    near = 2 * (2 * D + 8) * U * scale + 2.0 ** -20 + 2 * (n + 16) * U
    off = near + (2.0 ** -22 + 2.0 ** -32 / w if dt == "fp16" else 2.0 ** -17)
    bound = h * want + (1 + h) * off * want + 2.0 ** -25
    if dt == "fp16":
        assert abs(float(torch.tensor(w).half()) / w - 1) * want > 5 * bound  # the oracle without headroom does not pass
    assert (o - want).abs().max() <= bound, (float((o / want - 1).abs().max()), bound / want)
    assert (lse - math.log(big + small * w)).abs().max() <= 2.0 ** -20 + 2 * (n + 16) * U + 8 * U * scale
