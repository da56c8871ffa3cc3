"""The paged cache held in 8 bits, on the GPU, against its definitions in 64 bits (cache8_ref.py, where the error bounds are
derived): appending under growing scales, attention over what is held, and both together as a serving loop does."""
import math

import pytest
import torch

import attention_fa_fwd_03_gb300 as fa
import cache8_ref as ref
import paged_ref

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
NAN, INF = float("nan"), float("inf")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def make_table(g, B, max_pages, spare=3):
    n = B * max_pages + spare
    return torch.randperm(n, generator=g)[: B * max_pages].view(B, max_pages).to(torch.int32), n


def held_pool(g, P, Hkv, page, D, spread=2.0):
    """Random pages of different sizes and their scales."""
    return ref.hold(randn(g, P, Hkv, page, D) * torch.exp2(spread * randn(g, P, Hkv, 1, 1)))


def handle(k, v, ks, vs, table, lens):
    return fa.PagedKV(k.cuda(), v.cuda(), table.cuda(), lens.cuda(), k_scales=ks.cuda(), v_scales=vs.cuda())


def attend(kv, q, scale, causal=True, window=0, sinks=0, new_lens=None, sel=None, sel_lens=None, stream=None):
    q = q.cuda()
    o, lse = torch.full_like(q, NAN), torch.full(q.shape[:3], NAN, device="cuda")
    ws = torch.full((fa.fa_paged_workspace_size(q.shape[1], kv.Hkv, q.shape[2], kv.D),), 255, dtype=torch.uint8, device="cuda")
    d = [None if t is None else t.cuda() for t in (new_lens, sel, sel_lens)]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    fa.fa_paged_fwd(kv, q, o, lse, scale, causal=causal, window=window, sinks=sinks, new_lens=d[0], sel=d[1], sel_lens=d[2],
                    workspace=ws, stream=stream)
    return o, lse


def check(o, lse, want, what=""):
    ro, rl, bo, bl = want
    most = torch.finfo(o.dtype).max * (1 + torch.finfo(o.dtype).eps / 4)  # from here on a number is rounded to infinity
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(lse == -math.inf, rl == -math.inf), f"{what}: rows without keys"
    bad = ~((o - ro).abs() <= bo) & ~((o.abs() == math.inf) & (o.sign() == ro.sign()) & (ro.abs() + bo >= most))
    assert not bad.any(), f"{what}: O off by {((o - ro).abs() / bo.clamp(min=1e-300))[bad].max():.3g} bounds at {bad.nonzero()[0].tolist()}"
    fin = rl > -math.inf
    bad = ~((lse - rl).abs()[fin] <= bl[fin])
    assert not bad.any(), f"{what}: LSE off by {(lse - rl).abs()[fin].max():.3g}"


def clear():
    torch.cuda.synchronize()
    return fa.fa_device_status() == 0


def bits(x):
    return x.view(torch.uint8)


# ------------------------------------------------------------------ append
def append_ref(pools, scales, table, lens, new, T, k, v, cos, sin, rot, inter):
    """The pools and scales after the call: exact bytes of rows from before, and for new rows x and the bound of |held s - x|."""
    page = pools[0].shape[2]
    out = []
    for name, x, pool, sc in (("k", k, pools[0], scales[0]), ("v", v, pools[1], scales[1])):
        held, sc = pool.clone(), sc.double().clone()
        want, err = torch.full(pool.shape, NAN, dtype=torch.float64), torch.zeros(pool.shape, dtype=torch.float64)
        fresh_rows = torch.zeros(pool.shape[0], page, dtype=torch.bool)
        border = torch.zeros(sc.shape, dtype=torch.bool)
        for b, (first, m) in enumerate(paged_ref.positions(lens, new, T)):
            by_page = {}
            for t in range(m):
                by_page.setdefault((first + t) // page, []).append(t)
            for pg, ts in by_page.items():
                i = int(table[b, pg])
                if i < 0:
                    continue
                rows = []
                for t in ts:
                    y, e = x[b, :, t].double(), torch.zeros_like(x[b, :, t], dtype=torch.float64)
                    if name == "k" and rot:
                        y, e = paged_ref.rotate(y, cos[first + t].double(), sin[first + t].double(), rot, inter)
                    rows.append((t, y, e))
                for hd in range(pool.shape[1]):
                    most = max(float(torch.where(y[hd].isfinite(), y[hd].abs(), 0.0).max()) for _, y, _ in rows)
                    s = ref.scale_for(most)
                    # where a rotation in fp32 may see another power of two than 64 bits (without one it is exact)
                    most_of = [max(float(torch.where(y[hd].isfinite(), y[hd].abs() + sign * e[hd], 0.0).max()) for _, y, e in rows)
                               for sign in (1, -1)]
                    border[i, hd] = ref.scale_for(most_of[0]) != ref.scale_for(max(most_of[1], 0.0))
                    slot = (first + ts[0]) % page
                    if slot > 0:
                        s = max(s, float(sc[i, hd]))
                        if s > sc[i, hd]:
                            held[i, hd, :slot] = ref.round8(pool[i, hd, :slot].double() * (sc[i, hd] / s))
                    sc[i, hd] = s
                    for t, y, e in rows:
                        r = (first + t) % page
                        want[i, hd, r] = y[hd]
                        err[i, hd, r] = e[hd] + torch.maximum(2.0 ** -4 * (y[hd].abs() + e[hd]), torch.tensor(2.0 ** -10 * s))
                for t in ts:
                    fresh_rows[i, (first + t) % page] = True
        out.append((held, sc, want, err, fresh_rows, border))
    return out


def check_append(kv, want, what=""):
    for name, (held, sc, x, err, rows, border) in zip("kv", want):
        got, gs = getattr(kv, name).cpu(), getattr(kv, f"{name}_scales").cpu().double()
        assert not border.any(), f"{what}: the test's inputs lie at a border"
        assert torch.equal(gs, sc), f"{what}: scales of {name}"
        new = rows[:, None, :].expand(got.shape[:3])
        assert torch.equal(bits(got)[~new], bits(held)[~new]), f"{what}: rows of {name} that are not new"
        y, x, err = ref.held_value(got, gs)[new], x[new], err[new]
        assert torch.equal(y.isnan(), ~x.isfinite()), f"{what}: {name} NaN"
        ok = x.isfinite()
        assert ((y - x).abs()[ok] <= err[ok]).all(), f"{what}: {name} off by {((y - x).abs() / err)[ok].max():.3g} bounds"


APPEND = [  # B, Hq, Hkv, D, page, T, start lengths, new lengths (None: T), rot, interleaved, dtype, with q
    (1, 4, 2, 64, 16, 1, [0], None, 64, False, "fp16", True),
    (2, 4, 1, 128, 64, 1, [63, 64], None, 128, False, "bf16", True),
    (3, 6, 2, 96, 16, 5, [0, 14, 31], [5, 0, 3], 96, False, "fp16", True),
    (2, 4, 4, 96, 32, 8, [1, 29], None, 32, True, "bf16", True),
    (3, 3, 3, 96, 32, 70, [0, 5, 31], [70, 1, 69], 48, True, "bf16", True),
    (2, 16, 2, 256, 128, 200, [100, 0], [200, 131], 256, True, "fp16", True),
    (2, 1, 1, 256, 256, 33, [250, 223], None, 128, False, "bf16", True),
    (2, 8, 8, 128, 16, 64, [1, 16], None, 0, False, "bf16", False),
    (5, 5, 5, 64, 32, 129, [0, 1, 31, 32, 33], [129, 128, 0, 1, 97], 32, True, "fp16", True),
    (1, 40, 8, 128, 64, 300, [37], None, 128, False, "bf16", True),
    (2, 2, 2, 256, 16, 3, [15, 255], None, 256, False, "fp16", False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"B{c[0]}h{c[1]}x{c[2]}d{c[3]}p{c[4]}T{c[5]}{c[10]}")
@pytest.mark.parametrize("fused", [False, True])
def test_append_matches_the_definition(case, fused):
    B, Hq, Hkv, D, page, T, start, new, rot, inter, dt, with_q = case
    dtype = DT[dt]
    g = gen(B * 1000 + T)
    n = new or [T] * B
    lens = [s + m for s, m in zip(start, n)]
    mp = -(-max(max(lens), 1) // page)
    table, P = make_table(g, B, mp)
    (k_pool, ks), (v_pool, vs) = held_pool(g, P, Hkv, page, D), held_pool(g, P, Hkv, page, D)
    size = torch.exp2(3 * randn(g, B, T, 1, 1))  # tokens of different sizes: some raise the scale, some do not
    if fused:
        qkv = (randn(g, B, T, Hq + 2 * Hkv, D) * size).to(dtype).cuda()
        q, k, v = (t.transpose(1, 2) for t in qkv.split([Hq, Hkv, Hkv], 2))
    else:
        q, k, v = ((randn(g, B, h, T, D) * size.transpose(1, 2)).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    ang = torch.arange(max(max(lens), 1))[:, None] * 100.0 ** (-torch.arange(rot // 2) / max(rot // 2, 1))
    cos, sin = ang.cos().float(), ang.sin().float()
    kv = handle(k_pool, v_pool, ks, vs, table, i32(lens))
    q_out = torch.full((B, Hq, T, D), NAN, dtype=dtype, device="cuda")
    fa.fa_kv_append(kv, k, v, cos=cos.cuda() if rot else None, sin=sin.cuda() if rot else None, interleaved=inter,
                    q=q if with_q else None, q_out=q_out if with_q else None, new_lens=None if new is None else i32(new).cuda())
    assert clear()
    check_append(kv, append_ref((k_pool, v_pool), (ks, vs), table, lens, new, T, k.cpu(), v.cpu(), cos, sin, rot, inter))
    if with_q:
        got, q = q_out.cpu(), q.cpu()
        h, tiny = paged_ref.half_step(dtype), paged_ref.smallest(dtype)
        for b, (first, m) in enumerate(paged_ref.positions(lens, new, T)):
            for t in range(m):
                x, err = (paged_ref.rotate(q[b, :, t].double(), cos[first + t].double(), sin[first + t].double(), rot, inter)
                          if rot else (q[b, :, t].double(), 0.0))
                assert ((got[b, :, t].double() - x).abs() <= h * x.abs() + err + tiny).all(), (b, t)
            assert (got[b, :, m:] == 0).all()


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_append_of_values_that_are_not_ordinary(T, dt):
    """Zeros alone, the largest and smallest numbers of the type, infinities and NaN, beside a page of old rows."""
    dtype, Hkv, D, page = DT[dt], 7, 64, 64
    g = gen(T)
    table, P = make_table(g, 1, 1)
    (k_pool, ks), (v_pool, vs) = held_pool(g, P, Hkv, page, D), held_pool(g, P, Hkv, page, D)
    ks[:], vs[:] = 2.0 ** -126, 2.0 ** -126  # as after zeros
    x = randn(g, 1, Hkv, T, D, dtype=dtype)
    x[:, 1] = 0
    x[:, 2] = torch.finfo(dtype).max
    x[:, 3] = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    x[:, 4, 0, 3], x[:, 4, 0, 5], x[:, 4, T - 1, 60] = INF, -INF, NAN
    x[:, 5] = NAN
    x[:, 6] = -INF
    lens = [20 + T]
    for values in (k_pool, v_pool):  # rows of every kind before it, NaN too
        bits(values)[int(table[0, 0]), :, :20] = torch.arange(20 * D, dtype=torch.int64).remainder(256).to(torch.uint8).view(20, D)
    kv = handle(k_pool, v_pool, ks, vs, table, i32(lens))
    fa.fa_kv_append(kv, x.cuda(), x.flip(1).cuda())
    assert clear()
    want = append_ref((k_pool, v_pool), (ks, vs), table, lens, None, T, x, x.flip(1), None, None, 0, False)
    for name, (held, sc, y, err, rows, border) in zip("kv", want):
        got, gs = getattr(kv, name).cpu(), getattr(kv, f"{name}_scales").cpu().double()
        assert torch.equal(gs, sc)
        old = ~rows[:, None, :].expand(got.shape[:3])
        assert torch.equal(got.double()[old].nan_to_num(1000.0), held.double()[old].nan_to_num(1000.0))  # any NaN is one
        y, z, err = y[~old], ref.held_value(got, gs)[~old], err[~old]
        assert torch.equal(z.isnan(), ~y.isfinite())
        assert ((z - y).abs() <= err)[y.isfinite()].all()


def test_append_keeps_values_while_the_scale_grows():
    """Token by token, each larger than the last: what is held of a row stays the same number until it falls below the
    scale's normal numbers; and a page that is begun anew forgets the old scale."""
    g = gen(3)
    Hkv, D, page, n = 2, 128, 32, 32
    table, P = make_table(g, 1, 2)
    zero = torch.zeros(P, Hkv, page, D).to(ref.E4M3)
    kv = handle(zero, zero.clone(), torch.full((P, Hkv), 2.0 ** 100), torch.full((P, Hkv), 2.0 ** 100), table, i32([0]))
    k = randn(g, 1, Hkv, n, D, dtype=torch.bfloat16) * torch.exp2(torch.arange(n) / 4.0).to(torch.bfloat16)[:, None]
    k, v = k.cuda(), (-k).cuda()
    page_of = int(table[0, 0])
    before = None
    for t in range(n):
        kv.kv_lens += 1
        fa.fa_kv_append(kv, k[:, :, t:t + 1], v[:, :, t:t + 1])
        now, s = kv.k[page_of].cpu().double() * kv.k_scales[page_of].cpu().double()[:, None, None], kv.k_scales[page_of].cpu().double()
        if before is not None:
            big = before.abs() >= 2.0 ** -6 * s[:, None, None]
            assert torch.equal(now[:, :t][big], before[big])
            assert ((now[:, :t] - before).abs() <= 2.0 ** -10 * s[:, None, None])[~big].all()
        before = now[:, : t + 1].clone()
    assert clear()
    assert torch.equal(kv.v[page_of].cpu().double(), -kv.k[page_of].cpu().double())
    s1 = kv.k_scales[page_of].cpu().clone()
    kv.kv_lens.fill_(1)  # the sequence begins anew
    fa.fa_kv_append(kv, k[:, :, :1], v[:, :, :1])
    assert clear()
    assert (kv.k_scales[page_of].cpu() < s1).all()


def test_append_meets_bad_pages_and_lengths():
    g = gen(8)
    B, Hkv, D, page, mp = 4, 2, 64, 16, 3
    table, P = make_table(g, B, mp)
    (k_pool, ks), (v_pool, vs) = held_pool(g, P, Hkv, page, D), held_pool(g, P, Hkv, page, D)
    k, v = (randn(g, B, Hkv, 20, D, dtype=torch.float16) for _ in range(2))
    bad = table.clone()
    bad[1, 0] = -1
    bad[2, 1] = P
    lens = [20, 20, 40, 60]  # 60: beyond the three pages, taken as 48
    kv = handle(k_pool, v_pool, ks, vs, bad, i32(lens))
    fa.fa_kv_append(kv, k.cuda(), v.cuda())
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 4
    ok = table.clone()
    ok[1, 0], ok[2, 1] = -1, -1
    check_append(kv, append_ref((k_pool, v_pool), (ks, vs), ok, [20, 20, 40, 48], None, 20, k, v, None, None, 0, False))


# ------------------------------------------------------------------ attend
ATTEND = [  # B, Hq, Hkv, D, page, T, max length, ragged, causal, window, sinks, dtype
    (1, 1, 1, 64, 16, 1, 1, False, True, 0, 0, "fp16"),
    (2, 8, 2, 128, 64, 1, 1000, False, True, 0, 0, "bf16"),
    (3, 6, 2, 96, 16, 1, 333, True, True, 0, 0, "fp16"),
    (2, 4, 2, 256, 32, 1, 700, True, True, 0, 0, "bf16"),
    (5, 21, 3, 64, 32, 5, 500, True, True, 0, 0, "fp16"),
    (2, 16, 1, 128, 128, 1, 3000, True, True, 0, 0, "bf16"),
    (2, 16, 1, 128, 16, 4, 900, True, True, 100, 7, "bf16"),
    (2, 24, 1, 256, 64, 2, 600, True, False, 0, 0, "fp16"),
    (2, 16, 1, 96, 256, 8, 1500, True, True, 300, 70, "fp16"),
    (3, 7, 7, 128, 64, 3, 400, True, False, 50, 0, "bf16"),
    (1, 8, 8, 128, 64, 1, 20000, False, True, 0, 0, "bf16"),
    (1, 4, 2, 64, 16, 1, 9000, False, True, 5000, 3, "fp16"),
    (1, 16, 8, 256, 128, 1, 9000, False, True, 0, 0, "fp16"),
    (1, 8, 4, 96, 32, 8, 9000, False, True, 6000, 130, "bf16"),
    (1, 48, 2, 128, 64, 2, 12000, False, True, 0, 0, "fp16"),
    (1, 64, 1, 64, 16, 8, 9000, False, True, 7000, 64, "bf16"),
    (1, 20, 1, 256, 64, 4, 9000, False, True, 0, 0, "bf16"),
    (40, 4, 2, 128, 16, 2, 300, True, True, 40, 17, "bf16"),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"B{c[0]}h{c[1]}x{c[2]}d{c[3]}p{c[4]}T{c[5]}L{c[6]}w{c[9]}s{c[10]}{c[11]}")
def test_attend_matches_the_definition(case):
    B, Hq, Hkv, D, page, T, L, ragged, causal, window, sinks, dt = case
    g = gen(B * 77 + L + D)
    lens = [max(1, int(L * (b + 1) / B)) for b in range(B)] if ragged else [L] * B
    new = [min(n, b % (T + 1)) for b, n in enumerate(lens)] if ragged else None
    if ragged and B > 2:
        lens[1] = 0
        new[1] = 0
    mp = -(-L // page)
    table, P = make_table(g, B, mp)
    (k_pool, ks), (v_pool, vs) = held_pool(g, P, Hkv, page, D, 1.0), held_pool(g, P, Hkv, page, D)
    kd, vd = ref.held_value(k_pool, ks), ref.held_value(v_pool, vs)
    for b in range(B):  # slots that hold no key: NaN
        if lens[b] % page:
            i = int(table[b, lens[b] // page])
            bits(k_pool)[i, :, lens[b] % page:] = 127
            bits(v_pool)[i, :, lens[b] % page:] = 255
    kv = handle(k_pool, v_pool, ks, vs, table, i32(lens))
    q = randn(g, B, Hq, T, D, dtype=DT[dt])
    o, lse = attend(kv, q, 0.5 / math.sqrt(D), causal, window, sinks, None if new is None else i32(new))
    assert clear()
    want = ref.attend(q, kd, vd, table, lens, 0.5 / math.sqrt(D), causal, window, sinks, new, held=True)
    check(o, lse, want)
    again = attend(kv, q, 0.5 / math.sqrt(D), causal, window, sinks, None if new is None else i32(new))
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("rep,T", [(8, 1), (4, 4), (16, 2), (9, 5), (8, 8), (16, 8)])
def test_attend_over_long_lists_of_all_sizes(rep, T, D, dt):
    """Every kernel of a long list: rows up to 8, 16, 32, 64 and 128, pages whose scales are far apart."""
    g = gen(rep * T + D)
    Hkv, page, L = 2, 32, 20011
    table, P = make_table(g, 1, -(-L // page))
    (k_pool, ks), (v_pool, vs) = held_pool(g, P, Hkv, page, D, 1.0), held_pool(g, P, Hkv, page, D, 10.0)
    kd, vd = ref.held_value(k_pool, ks), ref.held_value(v_pool, vs)
    kv = handle(k_pool, v_pool, ks, vs, table, i32([L]))
    q = randn(g, 1, rep * Hkv, T, D, dtype=DT[dt])
    got = attend(kv, q, 0.5 / math.sqrt(D))
    assert clear()
    check(*got, ref.attend(q, kd, vd, table, [L], 0.5 / math.sqrt(D), True, 0, 0, held=True))


@pytest.mark.parametrize("rep,T,D", [(1, 1, 64), (4, 3, 64), (8, 5, 64), (3, 1, 256)])
def test_attend_over_more_sequences_than_a_window_holds(rep, T, D):
    """Lists of more items than a CTA keeps lengths of, empty sequences and padding among them."""
    g = gen(rep + T)
    B, Hkv, page, L = 300, 1, 16, 1200
    lens = [0 if b % 7 == 3 else 1 + (b * 401) % L for b in range(B)]
    new = [min(n, b % (T + 1)) for b, n in enumerate(lens)]
    table, P = make_table(g, B, -(-L // page))
    k, ks = held_pool(g, 100, Hkv, page, D, 1.0)
    v, vs = held_pool(g, 100, Hkv, page, D)
    at = torch.arange(P) % 100  # (the pool's pages repeat a hundred)
    k_pool, v_pool = (bits(t)[at].view(ref.E4M3) for t in (k, v))
    kv = handle(k_pool, v_pool, ks[at], vs[at], table, i32(lens))
    q = randn(g, B, rep, T, D, dtype=torch.bfloat16)
    got = attend(kv, q, 0.1, new_lens=i32(new))
    assert clear()
    kd, vd = ref.held_value(k_pool, ks[at]), ref.held_value(v_pool, vs[at])
    check(*got, ref.attend(q, kd, vd, table, lens, 0.1, True, 0, 0, new, held=True))


@pytest.mark.parametrize("B,rep,T,L", [(75, 7, 5, 3000), (36, 8, 8, 2990), (18, 16, 8, 3000), (70, 10, 2, 4000)])
@pytest.mark.parametrize("D,dt", [(64, "fp16"), (128, "bf16"), (96, "bf16")])
def test_attend_in_clusters_of_many_tiles(B, rep, T, L, D, dt):
    """So many units that all SMs have one, of more tiles than the other kernels' clusters take."""
    g = gen(B + D)
    Hkv, page = 2, 64
    lens = [L - 13 * b for b in range(B)]
    table, P = make_table(g, B, -(-L // page))
    k, ks = held_pool(g, 64, Hkv, page, D, 1.0)
    v, vs = held_pool(g, 64, Hkv, page, D)
    at = torch.arange(P) % 64
    k_pool, v_pool = (bits(t)[at].view(ref.E4M3) for t in (k, v))
    q = randn(g, B, rep * Hkv, T, D, dtype=DT[dt])
    got = attend(handle(k_pool, v_pool, ks[at], vs[at], table, i32(lens)), q, 0.5 / math.sqrt(D))
    assert clear()
    some = list(range(0, B, 9))  # sequences that are compared
    kd, vd = ref.held_value(k, ks), ref.held_value(v, vs)
    want = ref.attend(q[some], kd, vd, table[some] % 64, [lens[b] for b in some], 0.5 / math.sqrt(D), True, 0, 0, held=True)
    check(got[0][some], got[1][some], want)
    assert got[0].isfinite().all() and got[1].isfinite().all()


def test_pool_beyond_32_bits():
    """Appending to and attending over pages that lie behind 2^32 bytes of the pools: the bytes and bits of a small pool."""
    g = gen(33)
    B, Hq, Hkv, D, page, T = 2, 8, 2, 128, 64, 70
    lens = [150, 3 * page]
    small, P = make_table(g, B, 3, spare=2)
    far = 2 ** 32 // (Hkv * page * D)
    runs = []
    for base in (0, far):
        k, v = (torch.zeros(base + P, Hkv, page, D, dtype=torch.uint8, device="cuda").view(ref.E4M3) for _ in range(2))
        ks, vs = (torch.full((base + P, Hkv), 2.0 ** -126, device="cuda") for _ in range(2))
        g.manual_seed(5)
        kv = fa.PagedKV(k, v, (small + base).cuda(), i32([n - T for n in lens]).cuda(), k_scales=ks, v_scales=vs)
        for new in ([n - T for n in lens], [T, T], [1, 1]):  # many tokens, many on top of a begun page, one
            if new[0] == T:
                kv.kv_lens += T
            t = max(new)
            x = [randn(g, B, h, t, D, dtype=torch.bfloat16).cuda() for h in (Hkv, Hkv, Hq)]
            out = torch.empty_like(x[2])
            fa.fa_kv_append(kv, x[0], x[1], q=x[2], q_out=out, new_lens=i32(new).cuda())
        o = [attend(kv, out, 0.1)]
        assert clear()
        runs.append([t[base:].clone() for t in (bits(k), bits(v), ks, vs)] + [t for pair in o for t in pair])
        del k, v, kv
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    assert runs[0][4].isfinite().all()


@pytest.mark.parametrize("D,page,window", [(64, 16, 0), (128, 64, 90), (256, 32, 0), (96, 128, 0)])
def test_attend_over_selected_pages(D, page, window):
    g = gen(D)
    B, Hq, Hkv, L = 3, 8, 2, 900
    lens, mp = [900, 17, 450], -(-L // page)
    table, P = make_table(g, B, mp)
    (k_pool, ks), (v_pool, vs) = held_pool(g, P, Hkv, page, D, 1.0), held_pool(g, P, Hkv, page, D)
    n_sel = 5
    sel, count = torch.full((B, Hkv, n_sel), -1, dtype=torch.int32), torch.zeros(B, Hkv, dtype=torch.int32)
    for b in range(B):
        pages = -(-lens[b] // page)
        for h in range(Hkv):
            pick = torch.randperm(pages, generator=g)[:n_sel]
            sel[b, h, : len(pick)] = pick.to(torch.int32)
            count[b, h] = len(pick)
    kv = handle(k_pool, v_pool, ks, vs, table, i32(lens))
    q = randn(g, B, Hq, 1, D, dtype=torch.bfloat16)
    o, lse = attend(kv, q, 0.1, True, window, 3, None, sel, count)
    assert clear()
    check(o, lse, ref.attend(q, ref.held_value(k_pool, ks), ref.held_value(v_pool, vs), table, lens, 0.1, True, window, 3, None,
                             sel, count, held=True))


@pytest.mark.parametrize("rep,T,L,window", [(4, 1, 200, 60), (3, 4, 200, 60), (16, 2, 200, 60), (8, 8, 200, 60), (4, 2, 9500, 9000),
                                            (16, 2, 9500, 9000), (8, 8, 9500, 9000), (32, 4, 9500, 9000)])
def test_attend_with_values_that_are_no_numbers(rep, T, L, window):
    """NaN in keys and values that some rows see and others do not reaches only those that see it; pages whose scales are
    2^60 apart; queries of every size, zeros among them."""
    g = gen(rep * 10 + T)
    B, Hkv, D, page = 2, 2, 128, 16
    table, P = make_table(g, B, -(-L // page))
    (k_pool, ks), (v_pool, vs) = held_pool(g, P, Hkv, page, D, 1.0), held_pool(g, P, Hkv, page, D, 20.0)
    lens = [L, L - 5]
    q = randn(g, B, rep * Hkv, T, D, dtype=torch.bfloat16)
    q[:, 0] = 0
    q[:, 1] = (q[:, 1].float() * 2.0 ** -90).to(torch.bfloat16)
    # the key of the first new token is NaN in V for one head; the last token's K is NaN in the other
    for b, n in enumerate(lens):
        first, last = n - T, n - 1
        v_pool.view(torch.uint8)[int(table[b, first // page]), 0, first % page, 5] = 127
        k_pool.view(torch.uint8)[int(table[b, last // page]), 1, last % page, 9] = 255
    kv = handle(k_pool, v_pool, ks, vs, table, i32(lens))
    o, lse = attend(kv, q, 0.1, True, window, 4)
    assert clear()
    kd, vd = ref.held_value(k_pool, ks), ref.held_value(v_pool, vs)
    ro, rl, bo, bl = ref.attend(q, kd.nan_to_num(0.0), vd.nan_to_num(0.0), table, lens, 0.1, True, window, 4, held=True)
    o, lse = o.double().cpu(), lse.double().cpu()
    nan_o = torch.zeros(o.shape, dtype=torch.bool)
    nan_o[:, :rep, :, 5] = True        # every token sees the first one's value
    nan_o[:, rep:, T - 1] = True       # only the last token sees its own key
    assert torch.equal(o.isnan(), nan_o)
    assert torch.equal(lse.isnan(), nan_o.all(-1))
    assert ((o - ro).abs() <= bo)[~nan_o].all() and ((lse - rl).abs() <= bl)[~lse.isnan()].all()


def test_attend_meets_bad_pages():
    g = gen(4)
    B, Hkv, D, page, L = 3, 2, 64, 32, 300
    table, P = make_table(g, B, -(-L // page))
    (k_pool, ks), (v_pool, vs) = held_pool(g, P, Hkv, page, D, 1.0), held_pool(g, P, Hkv, page, D)
    bad = table.clone()
    bad[0, 3], bad[1, :] = -7, P + 100
    kv = handle(k_pool, v_pool, ks, vs, bad, i32([L, L, L]))
    q = randn(g, B, 4, 1, D, dtype=torch.float16)
    o, lse = attend(kv, q, 0.1)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 4
    check(o, lse, ref.attend(q, ref.held_value(k_pool, ks), ref.held_value(v_pool, vs), bad, [L] * B, 0.1, True, 0, 0, held=True))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dt,D,window,sinks", [("bf16", 128, 0, 0), ("fp16", 96, 70, 5)])
def test_serving_loop(dt, D, window, sinks):
    """A prompt, then tokens one by one with page assignment, appending and attention on a side stream, and the same steps
    replayed as a captured graph: the graph gives the eager loop's outputs bit for bit, and they are near the attention over
    the values before rounding, within what e4m3 makes of them."""
    dtype, B, Hq, Hkv, page, mp, steps = DT[dt], 3, 6, 2, 16, 12, 40
    g = gen(11)
    P = B * mp
    prompt = [33, 1, 16]
    xs = [randn(g, B, Hq + 2 * Hkv, max(prompt), D, dtype=dtype).cuda()]
    xs += [randn(g, B, Hq + 2 * Hkv, 1, D, dtype=dtype).cuda() for _ in range(steps)]
    ang = torch.arange(mp * page)[:, None] * 100.0 ** (-torch.arange(D // 2) / (D // 2))
    cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()

    def fresh():
        s = {"table": torch.full((B, mp), -1, dtype=torch.int32), "lens": torch.zeros(B, dtype=torch.int32),
             "held": torch.zeros(B, 3, dtype=torch.int32), "free": torch.arange(P, dtype=torch.int32), "count": i32([P, 0]),
             "x": torch.zeros(B, Hq + 2 * Hkv, 1, D, dtype=dtype), "q": torch.zeros(B, Hq, 1, D, dtype=dtype),
             "o": torch.zeros(B, Hq, 1, D, dtype=dtype), "lse": torch.zeros(B, Hq, 1),
             "ws": torch.zeros(fa.fa_paged_workspace_size(Hq, Hkv, 1, D), dtype=torch.uint8)}
        s = {n: t.cuda() for n, t in s.items()}
        zero = torch.zeros(P, Hkv, page, D, device="cuda").to(ref.E4M3)
        s["kv"] = fa.PagedKV(zero, zero.clone(), s["table"], s["lens"], k_scales=torch.zeros(P, Hkv, device="cuda"),
                             v_scales=torch.zeros(P, Hkv, device="cuda"))
        return s

    def split(x):
        return x.split([Hq, Hkv, Hkv], 1)

    def first(s):
        new = i32(prompt).cuda()
        s["lens"] += new
        T = max(prompt)
        fa.fa_page_assign(s["table"], s["lens"], s["held"], s["free"], s["count"], page, T, new_lens=new, window=window, sinks=sinks)
        q, k, v = split(xs[0])
        fa.fa_kv_append(s["kv"], k, v, cos=cos, sin=sin, new_lens=new)

    def step(s):
        s["lens"] += 1
        fa.fa_page_assign(s["table"], s["lens"], s["held"], s["free"], s["count"], page, 1, window=window, sinks=sinks)
        q, k, v = split(s["x"])
        fa.fa_kv_append(s["kv"], k, v, cos=cos, sin=sin, q=q, q_out=s["q"])
        fa.fa_paged_fwd(s["kv"], s["q"], s["o"], s["lse"], 0.2, causal=True, window=window, sinks=sinks, workspace=s["ws"])

    outs = {}
    side = torch.cuda.Stream()
    for how in ("eager", "graph"):
        s = fresh()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            first(s)
            outs[how] = []
            if how == "graph":
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step(s)
            for i in range(steps):
                s["x"].copy_(xs[1 + i])
                graph.replay() if how == "graph" else step(s)
                outs[how].append((s["o"].clone(), s["lse"].clone()))
        assert clear()
        assert int(s["count"][1]) == 0
    for a, b in zip(*outs.values()):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # against attention over the values before rounding: a key is off by 2^-4 of itself at most, so scores by
    # 2^-4 scale sum |q k| (and as much again for the page's smallest values) and O by that factor and 2^-4 max|v|
    keys, vals = [], []
    for b in range(B):
        x = torch.cat([xs[0][b, :, : prompt[b]]] + [y[b] for y in xs[1:]], 1).double().cpu()
        pos = torch.arange(x.shape[1])
        rot = torch.stack([paged_ref.rotate(x[Hq:Hq + Hkv, p], cos[p].double().cpu(), sin[p].double().cpu(), D, False)[0] for p in pos], 1)
        keys.append(rot)
        vals.append(x[Hq + Hkv:])
    last = steps - 1
    for b in range(B):
        n = prompt[b] + steps
        p = n - 1
        q = paged_ref.rotate(xs[-1][b, :Hq, 0].double().cpu(), cos[p].double().cpu(), sin[p].double().cpu(), D, False)[0]
        see = torch.arange(n) >= 0
        if window:
            see = (p - torch.arange(n) < window) | (torch.arange(n) < sinks)
        for h in range(Hq):
            kk, vv = keys[b][h // (Hq // Hkv)][see], vals[b][h // (Hq // Hkv)][see]
            w = torch.softmax(0.2 * (kk @ q[h]), 0)
            ds = 2 * 0.2 * 2.0 ** -4 * (kk.abs() @ q[h].abs()).max()
            bound = (torch.expm1(2 * ds) + 2.0 ** -4 + 2.0 ** -7) * (w @ vv.abs()) + 2.0 ** -8 * vv.abs().max()
            assert ((outs["eager"][last][0][b, h, 0].double().cpu() - w @ vv).abs() <= bound).all()


def test_on_another_stream_and_beside_another_call():
    """Two calls at once on two streams, each with its own workspace, give what each gives alone."""
    g = gen(21)
    B, Hq, Hkv, D, page, L = 4, 8, 2, 128, 64, 5000
    table, P = make_table(g, B, -(-L // page))
    (k_pool, ks), (v_pool, vs) = held_pool(g, P, Hkv, page, D, 1.0), held_pool(g, P, Hkv, page, D)
    kv = handle(k_pool, v_pool, ks, vs, table, i32([L, 40, 3000, 1]))
    qs = [randn(g, B, Hq, t, D, dtype=torch.bfloat16).cuda() for t in (1, 5)]
    alone = [attend(kv, q, 0.1) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(3):
        both = [attend(kv, q, 0.1, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert clear()


def test_waits_give_up():
    """With a bound of a few cycles the loads' waits give up, the call ends and says so, and the next one is right."""
    g = gen(6)
    B, Hq, Hkv, D, page, L = 1, 8, 2, 128, 64, 130000
    table, P = make_table(g, B, -(-L // page))
    k, ks = held_pool(g, 64, Hkv, page, D, 1.0)
    k, ks = k.cuda().view(torch.uint8).repeat(P // 64 + 1, 1, 1, 1)[:P].view(ref.E4M3), ks.cuda().repeat(P // 64 + 1, 1)[:P].contiguous()
    kv = handle(k, k, ks, ks, table, i32([L]))
    q = randn(g, B, Hq, 1, D, dtype=torch.bfloat16)
    want = attend(kv, q, 0.1)
    assert clear()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(1)  # the keys have to come from memory
    fa.fa_set_wait_limit_cycles(8)
    try:
        attend(kv, q, 0.1)
        torch.cuda.synchronize()
    finally:
        fa.fa_set_wait_limit_cycles(0)
    assert fa.fa_device_status() & 1 and flush.numel()
    got = attend(kv, q, 0.1)
    assert clear()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
