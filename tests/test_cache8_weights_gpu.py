"""Weights of attention over the cache held in 8 bits: what they keep of their digits where one key dominates. In every
kernel: clusters (short lists) and split lists of up to 8, 16, 32, 64 and 128 rows per KV head.

What a weight may lose. Relative to its row's running maximum a weight is at most 2^8; it goes to the product with V as one or
two fp16 numbers after it has been multiplied by 2^7 and by its page's part of the largest scale of V so far, at least 1/16.
So it is off by at most 2^-11 of itself (half a step of the first word), and where it is small by half of fp16's smallest
number, 2^-25: 2^-32 of the running maximum's weight over the part, times a value. A running maximum may be behind the
largest score, never ahead, so 2^-32 of the largest weight bounds it."""
import math

import pytest
import torch

import attention_fa_fwd_03_gb300 as fa
import cache8_ref as ref

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
WORD = 2.0 ** -11
U = 2.0 ** -24
PAGE = 64
SIZES = [(heads, D, n) for heads in (4, 12, 20, 40, 100) for D in (64, 96, 128, 256) for n in (500, 30000)]


def run(k, ks, v, vs, q, scale, n, window=0, sinks=0):
    """k, v [pages, 1, PAGE, D] e4m3, one sequence of n keys."""
    kv = fa.PagedKV(k.cuda(), v.cuda(), torch.arange(k.shape[0], dtype=torch.int32, device="cuda")[None],
                    torch.tensor([n], dtype=torch.int32, device="cuda"), k_scales=ks.cuda(), v_scales=vs.cuda())
    q = q.cuda()
    o, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
    ws = torch.full((fa.fa_paged_workspace_size(q.shape[1], 1, 1, q.shape[3]),), 255, dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(kv, q, o, lse, scale, causal=True, window=window, sinks=sinks, workspace=ws)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    return o.double().cpu(), lse.double().cpu()


def near_scores(D, s, n):
    """Relative error of a weight whose score is off as fp32 products and exponents make it, and of the sums."""
    return 2 * (2 * D + 8) * U * s + 2.0 ** -20 + 2 * (n + 16) * U


@pytest.mark.parametrize("weight", [1.4 * 2.0 ** -24, 0.9 * 2.0 ** -25])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("heads,D,n", SIZES)
def test_small_weights_beside_dominating_keys(heads, D, n, dt, weight):
    """Every 16th key has the largest score and V = 0; the others have a weight far below fp16's normal numbers and hold all
    of the row. (In fp16 as it is, 1.4 2^-24 is 2^-24 and 0.9 2^-25 is nothing.) Pages of one scale, of scales within a
    factor of 16, and of scales 2^14 apart; every value is the same number."""
    pages = -(-n // PAGE)
    k = torch.zeros(pages, 1, PAGE, D)
    k[..., 0] = -1
    k[:, :, ::16, 0] = 0
    c = 2.0 ** 14
    q = torch.zeros(1, heads, 1, D, dtype=DT[dt])
    q[..., 0] = 1
    scale = float(torch.tensor(-math.log(weight), dtype=torch.float32))
    w = math.exp(-scale)
    big = -(-n // 16)
    small = n - big
    want = c * small * w / (big + small * w)
    h = torch.finfo(DT[dt]).eps / 2
    for spread, part in ((0, 1), (2, 16), (7, 16)):
        p = torch.arange(pages)
        vs = torch.exp2(13.0 + (p * 5 % (2 * spread + 1) - spread))  # what is held: 2^-6 to 2^8
        v = torch.full((pages, 1, PAGE, D), c) / vs[:, None, None, None]
        v[:, :, ::16] = 0
        assert torch.equal(v.to(ref.E4M3).float(), v)
        o, lse = run(k.to(ref.E4M3), torch.ones(pages, 1), v.to(ref.E4M3), vs[:, None], q, scale, n)
        off = near_scores(D, scale, n) + WORD + part * 2.0 ** -32 / w
        bound = h * want + (1 + h) * off * want + 2.0 ** -25
        if spread == 0:
            as_it_is = float(torch.tensor(w).half()) / w
            assert abs(as_it_is - 1) * want > 5 * bound  # the oracle without headroom does not pass
        assert (o - want).abs().max() <= bound, (spread, float((o / want - 1).abs().max()), bound / want)
        assert (lse - math.log(big + small * w)).abs().max() <= 2.0 ** -20 + 2 * (n + 16) * U + 8 * U * scale


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("heads,D,n", SIZES)
def test_first_token_dominates(heads, D, n, dt):
    """The first key's score is 16 above scores N(0, 1) and its value next to nothing, pages of V of different sizes: in the
    window with visible first keys and without one, against the definition."""
    g = torch.Generator().manual_seed(heads + D + n)
    pages = -(-n // PAGE)
    q = torch.randn(1, heads, 1, D, generator=g) / math.sqrt(D)
    q[..., 0] = 8
    k = torch.randn(pages, 1, PAGE, D, generator=g)
    k[..., 0] = 0
    k[0, 0, 0] = 0
    k[0, 0, 0, 0] = 2
    v = (torch.randn(pages, 1, PAGE, D, generator=g) + 1) * torch.exp2(torch.randint(-2, 3, (pages, 1, 1, 1), generator=g).float())
    v[0, 0, 0] = 2.0 ** -8
    (k, ks), (v, vs) = ref.hold(k), ref.hold(v)
    q, scale = q.to(DT[dt]), 1.0
    kd, vd = (ref.held_value(*x).reshape(-1, D)[:n] for x in ((k, ks), (v, vs)))
    h = torch.finfo(DT[dt]).eps / 2
    for window, sinks in ((0, 0), (n // 2, 1)):
        o, lse = run(k, ks, v, vs, q, scale, n, window, sinks)
        j = torch.arange(n)
        see = (n - 1 - j < window) | (j < sinks) if window else j >= 0
        kk, vv, x = kd[see], vd[see], q[0, :, 0].double()
        s = scale * (x @ kk.T)
        lz = torch.logsumexp(s, -1)
        p = torch.exp(s - lz[:, None])
        want = p @ vv
        ds = ((2 * D + 8) * U * scale * (x.abs() @ kk.abs().T)).amax(-1)
        if dt == "bf16":  # rows in fp16 under a power of two: elements below 2^-28 of the largest
            ds = ds + 2.0 ** -39 * scale * x.abs().amax(-1) * kk.abs().sum(-1).amax()
        sums = 2 * (len(kk) + 16) * U
        rel = WORD + 2 * (2 * ds + 2.0 ** -21 + sums)
        lost = len(kk) * 2.0 ** -32 * p.amax(-1) * 448 * float(vs.max())
        bound = (1 + h) * (rel[:, None] * (p @ vv.abs()) + lost[:, None]) + h * want.abs() + 2.0 ** -25
        assert ((o[0, :, 0] - want).abs() <= bound).all(), float(((o[0, :, 0] - want).abs() / bound).max())
        assert ((lse[0, :, 0] - lz).abs() <= ds + 2.0 ** -21 + sums + 8 * U * (lz.abs() + s.abs().amax(-1))).all()


WORDS = {"fp16": 2.0 ** -22, "bf16": 2.0 ** -11}  # of a weight, what the words it goes to its product in leave out


def weights_that_round_alike(dtype):
    """A score x whose weight exp(x) beside weights of 1 is as far from fp16's numbers as can be; x a number of the type."""
    xs = torch.linspace(-0.45 * 2.0 ** -10, -0.05 * 2.0 ** -10, 4000).to(dtype).unique()
    w = xs.double().exp()
    i = (w.half().double() - w).abs().argmax()
    return float(xs[i]), float(w[i]), float(w[i].half())


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("heads,D,n", SIZES)
def test_values_that_cancel(heads, D, n, dt):
    """Every other key has the weight w < 1 and V = -1, the others 1 and V = 1: O = (1 - w) / (1 + w), next to nothing, and
    all weights w round alike. For fp16 outputs the second word is what O is made of; for bf16 outputs there is one word, and O
    is off by its half step of the weights' sum of |V| and no more.

    Bound. The exponential is off by 2^-21 w and the score's by (2 D + 8) u |x| w. Partial sums of O are at most 64 of one sign
    beyond what cancels, n (1 - w) / 2 in all (with one word n 2^-12 / 2 more), so n additions of 2 u each leave 2 u (64 + that)
    n over a sum of weights of n (1 + w) / 2; joins a few u."""
    x, w, rounded = weights_that_round_alike(DT[dt])
    pages = -(-n // PAGE)
    k = torch.zeros(pages, 1, PAGE, D)
    v = torch.ones(pages, 1, PAGE, D)
    k[:, :, 1::2, 0] = 1
    v[:, :, 1::2] = -1
    q = torch.zeros(1, heads, 1, D, dtype=DT[dt])
    q[..., 0] = x
    ones, ws = (n + 1) // 2, n // 2
    want = (ones - ws * w) / (ones + ws * w)
    h = torch.finfo(DT[dt]).eps / 2
    o, lse = run(k.to(ref.E4M3), torch.ones(pages, 1), v.to(ref.E4M3), torch.ones(pages, 1), q, 1.0, n)
    bound = (h * abs(want) + WORDS[dt] + 2.0 ** -32 + 2.0 ** -20 + (2 * D + 8) * U * abs(x) + 4 * U * (64 + n * (1 - w + 2.0 ** -11) / 2)
             + 16 * U + 2.0 ** -25)
    if dt == "fp16":
        one_word = (ones - ws * rounded) / (ones + ws * w)
        assert abs(one_word - want) > 5 * bound  # the oracle with one word does not pass
    assert (o - want).abs().max() <= bound, (float((o - want).abs().max()), bound)
    assert (lse - math.log(ones + ws * w)).abs().max() <= 2.0 ** -20 + 2 * (n + 16) * U
