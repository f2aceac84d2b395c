"""The paged key/value cache on the GPU against the definition in float64.

Tolerances. u = finfo(T).eps / 2 is one rounding to the output type, e = 2^-24 one fp32
rounding. A rotated element x c - y s takes at most three fp32 roundings and one to T:
|error| <= u |ref| + 4 e (|x c| + |y s|). An attention output sum_t p_t v_t / sum_t p_t with
scores of absolute error d has |error| <= u |ref| + max_t |v_t| (2 d + 2^-16 + (n + 64) 2 e):
d = S hd 2 e for S = max_t scale sum_d |q_d k_td| (an fp32 sum of hd exact or once rounded
products), n additions each in the numerator and the denominator, 2^-16 for weights held as
a pair of bf16 (their sum is off by at most 2^-8 2^-8 of the weight; 0 for fp32 caches).
|error of lse| <= d + (n + 64) 2 e + 4 e |ref|.
"""
import math

import numpy as np
import pytest
import torch

import train_step_b200 as tsb

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def pool(pages, page, nkv, hd, dtype, layout, g):
    """A cache tensor, logical [page, token, head, element], in one of four storage orders."""
    if layout == "tokens":
        return torch.randn(pages, page, nkv, hd, generator=g).to(dtype).cuda()
    if layout == "heads":
        return torch.randn(pages, nkv, page, hd, generator=g).to(dtype).cuda().transpose(1, 2)
    if layout == "heads first":  # every head's pages together
        return torch.randn(nkv, pages, page, hd, generator=g).to(dtype).cuda().permute(1, 2, 0, 3)
    # "padded": rows and heads with gaps, neither keys nor values next to each other
    big = torch.randn(pages, page + 1, nkv + 1, hd + 16, generator=g).to(dtype).cuda()
    return big[:, :page, 1:, 8:8 + hd]


def tables(lens, page, spare, rng, n_seqs=None):
    per = [-(-n // page) for n in lens]
    ids = rng.permutation(sum(per) + spare).astype(np.int32)
    table = np.full((len(lens), max(1, max(per))), 0x7FFFFFFF, np.int32)  # unused entries: never followed
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, sum(per) + spare


def visible(n, window, sinks):
    return [t for t in range(n) if window == 0 or t >= n - window or t < sinks]


def reference(kc, vc, table, q, lens, scale, window=0, sinks=0):
    """(out, lse, bound of out, bound of lse) in float64; caches as CPU float64 tensors."""
    B, NH, hd = q.shape
    page, nkv = kc.shape[1], kc.shape[2]
    out = torch.zeros(B, NH, hd, dtype=torch.float64)
    lse = torch.full((B, NH), -math.inf, dtype=torch.float64)
    tol = torch.zeros(B, NH, hd, dtype=torch.float64)
    tol_lse = torch.zeros(B, NH, dtype=torch.float64)
    for b in range(B):
        see = visible(int(lens[b]), window, sinks)
        if not see:
            continue
        t = torch.tensor(see)
        pg = torch.from_numpy(table[b].astype(np.int64))[t // page]
        k, v = kc[pg, t % page], vc[pg, t % page]  # [n, nkv, hd]
        n = len(see)
        for h in range(NH):
            hk = h // (NH // nkv)
            qh = q[b, h].double()
            z = (k[:, hk] @ qh) * scale
            lse[b, h] = torch.logsumexp(z, 0)
            out[b, h] = torch.softmax(z, 0) @ v[:, hk]
            S = float((k[:, hk].abs() @ qh.abs()).max()) * scale
            d = S * hd * 2 * E
            tol[b, h] = v[:, hk].abs().amax(0) * (2 * d + 2.0 ** -16 + (n + 64) * 2 * E)
            tol_lse[b, h] = d + (n + 64) * 2 * E + 4 * E * abs(float(lse[b, h]))
    return out, lse, tol, tol_lse


def check(out, lse, ref, dtype):
    o, l, tol, tol_lse = ref
    err = (out.double().cpu() - o).abs()
    bound = unit(dtype) * o.abs() + tol
    assert torch.isfinite(out.float()).all()
    assert (err <= bound).all(), float((err - bound).max())
    if lse is not None:
        empty = l == -math.inf
        got = lse.double().cpu()
        assert (got[empty] == -math.inf).all()
        assert ((got - l).abs()[~empty] <= tol_lse[~empty]).all()


def attention_case(lens, NH, nkv, hd, page, dtype, layout, window=0, sinks=0, scale=None, seed=0, q_scale=1.5,
                   poison=True):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    table, pages = tables(lens, page, 2, rng)
    kc, vc = pool(pages, page, nkv, hd, dtype, layout, g), pool(pages, page, nkv, hd, dtype, layout, g)
    q = (q_scale * torch.randn(len(lens), NH, hd, generator=g)).to(dtype).cuda()
    scale = hd ** -0.5 if scale is None else scale
    ref = reference(kc.double().cpu(), vc.double().cpu(), table, q.double().cpu(), lens, scale, window, sinks)
    if poison:
        # everything no query may see holds NaN or infinity: slots behind the last token,
        # tokens outside the window, pages of nobody
        seen = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for t in visible(n, window, sinks):
                seen[table[b, t // page], t % page] = True
        hidden = ~seen.cuda()
        kc[hidden] = math.nan
        vc[hidden] = math.inf
        vc[~hidden] += 0  # (touches nothing else)
    kv = tsb.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    out = torch.full_like(q, math.nan)
    lse = torch.full((len(lens), NH), math.nan, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    tsb.paged_attention(kv, q, ln, out, scale=scale, window=window, sinks=sinks, lse=lse)
    kv.check()
    check(out, lse, ref, dtype)
    return kv, q, ln, out, lse, ref


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
BOTH = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("hd", [32, 64, 96, 128])
@pytest.mark.parametrize("NH,nkv", [(1, 1), (12, 12), (6, 2), (7, 1), (16, 2), (9, 1), (16, 1), (40, 2)])
def test_attention_head_layouts(dtype, hd, NH, nkv):
    attention_case([1, 37, 0, 150], NH, nkv, hd, 16, dtype, "heads", seed=hd + NH)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("page", [1, 2, 8, 32, 128, 1024])
@pytest.mark.parametrize("layout", ["tokens", "heads", "heads first", "padded"])
def test_attention_pages_and_strides(dtype, page, layout):
    attention_case([129, 1, 64, 300], 4, 2, 64, page, dtype, layout, seed=page)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, 1000])
def test_attention_lengths(dtype, n):
    attention_case([n], 3, 1, 64, 16, dtype, "heads", seed=n)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 4), (17, 17), (64, 1), (100, 250), (1000, 7),
                                          (400, 0), (401, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_attention_window_and_sinks(dtype, window, sinks):
    attention_case([1, 5, 0, 16, 17, 123, 400], 4, 2, 64, 16, dtype, "heads", window, sinks, seed=window % 97)


@pytest.mark.parametrize("dtype,hd,NH,nkv", [(torch.bfloat16, 128, 8, 1), (torch.bfloat16, 64, 12, 12),
                                             (torch.float32, 64, 4, 2)])
def test_attention_long_and_ragged(dtype, hd, NH, nkv):
    # one sequence spread over many workers beside many that are not split
    attention_case([20000] + [1 + 7 * i for i in range(40)], NH, nkv, hd, 32, dtype, "heads", seed=5)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("NH,nkv,hd,page,n", [(1, 1, 64, 16, 20000), (12, 12, 64, 16, 1024), (8, 1, 128, 64, 131071),
                                              (16, 2, 64, 8, 9999), (6, 3, 32, 32, 30001), (5, 1, 96, 16, 7777)])
def test_attention_counts_every_key_once(dtype, NH, nkv, hd, page, n):
    """Equal scores (queries of zero): every weight is 1/n, the sum of exponentials is n, and an
    output is the mean of a value that is 1 at some keys and 0 at the others. A tile of 16 keys
    that is lost or counted twice moves the logarithm by 16/n. Weights are one power of two, sums
    of them exact up to 2^24 of them, so the logarithm is off by its own roundings, 4 e (|log n| +
    1) at most, and a mean c/n by those of the reciprocal and the product, 2 e, and one to T."""
    assert n < 2 ** 24 and 16 / n > 64 * E * (math.log(n) + 1)
    kc = torch.randn(-(-n // page) + 2, page, nkv, hd, device="cuda").to(dtype)
    vc = torch.zeros_like(kc)
    ids = torch.randperm(kc.shape[0], generator=torch.Generator().manual_seed(n))[:-(-n // page)].int()
    t = torch.arange(n)
    # element e: the keys of the tiles e, e + hd, e + 2 hd ...
    flat = torch.zeros(ids.numel() * page, hd)
    flat[t, (t // 16) % hd] = 1
    vc[ids.long().cuda()] = flat.view(-1, page, 1, hd).to(dtype).cuda()
    kv = tsb.PagedKV(kc, vc, ids[None].cuda())
    q = torch.zeros(1, NH, hd, dtype=dtype, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, NH, device="cuda")
    ws = kv.attention_workspace(NH)
    for length in (n, n - 1, n - 15, n - 16, n - 17, n // 2 + 1):
        tsb.paged_attention(kv, q, torch.tensor([length], dtype=torch.int32, device="cuda"), out, lse=lse, ws=ws)
        count = torch.bincount((t[:length] // 16) % hd, minlength=hd).double()
        assert ((lse.double().cpu() - math.log(length)).abs() <= 4 * E * (math.log(length) + 1)).all()
        want = count / length
        assert ((out.double().cpu() - want).abs() <= (unit(dtype) + 2 * E) * want).all()
    kv.check()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("hd,NH,nkv,page", [(32, 6, 2, 16), (64, 16, 1, 8), (64, 40, 2, 16), (96, 9, 1, 64),
                                            (96, 5, 1, 4), (128, 16, 2, 32), (128, 12, 1, 16), (128, 3, 3, 2)])
def test_attention_of_items_spread_over_blocks(dtype, hd, NH, nkv, page):
    # items too large for one block, next to empty and small ones; several orders of the lengths
    lens = [1500, 1, 40, 0, 2100]
    for k in range(2):
        attention_case(lens[k:] + lens[:k], NH, nkv, hd, page, dtype, "heads", seed=hd + page + k)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("window,sinks", [(1200, 0), (1200, 20), (1111, 1000), (3, 2500)])
def test_attention_through_large_windows(dtype, window, sinks):
    attention_case([5000, 1100, 77, 3001], 4, 2, 64, 16, dtype, "heads", window, sinks, seed=window)


@pytest.mark.parametrize("layout", ["heads", "tokens", "padded"])
@pytest.mark.parametrize("NH,nkv,page", [(2, 2, 16), (3, 3, 32), (5, 5, 16), (12, 3, 64), (56, 7, 16), (6, 3, 8)])
def test_attention_of_pairs_of_small_heads(NH, nkv, page, layout):
    # an odd head alone in its pair: split over warps and blocks, in windows, beside padding rows
    # that nothing may write
    for lens, window, sinks in (([1, 37, 0, 150, 16], 0, 0), ([2500, 1, 40, 0, 1800], 0, 0), ([900, 5, 0, 333], 200, 9)):
        kv, q, ln, out, lse, ref = attention_case(lens, NH, nkv, 32, page, torch.bfloat16, layout, window, sinks,
                                                  seed=NH + page)
        wide = torch.full((len(lens), NH + 16, 32), 7.0, dtype=torch.bfloat16, device="cuda")
        tsb.paged_attention(kv, q, ln, wide[:, :NH], window=window, sinks=sinks)
        assert torch.equal(wide[:, :NH], out) and (wide[:, NH:] == 7).all()


def test_attention_more_sequences_than_workers():
    attention_case([(i * 13) % 40 for i in range(700)], 5, 5, 32, 8, torch.bfloat16, "heads", seed=8)


@pytest.mark.parametrize("dtype", BOTH)
def test_attention_of_empty_sequences_only(dtype):
    attention_case([0, 0, 0], 4, 2, 64, 16, dtype, "heads")


@pytest.mark.parametrize("dtype", BOTH)
def test_calls_on_no_sequences(dtype):
    kc, vc = (torch.zeros(4, 16, 2, 64, dtype=dtype, device="cuda") for _ in range(2))
    kv = tsb.PagedKV(kc, vc, torch.zeros(0, 3, dtype=torch.int32, device="cuda"))
    q, n = torch.zeros(0, 4, 64, dtype=dtype, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    tsb.paged_attention(kv, q, n, torch.empty_like(q), lse=torch.empty(0, 4, device="cuda"))
    tsb.paged_kv_append(kv, q[:, :2], q[:, 2:], n, q=q, q_out=q)
    kv.check()


@pytest.mark.parametrize("dtype", BOTH)
def test_attention_of_extreme_scores(dtype):
    # one key dominates by hundreds of units; large negative scores; a scale of its own
    attention_case([300, 77], 4, 2, 64, 16, dtype, "heads", scale=1.0, q_scale=20.0, seed=3)
    attention_case([300, 77], 4, 2, 64, 16, dtype, "heads", scale=1e-6, q_scale=1.0, seed=4)


def test_attention_of_increasing_scores():
    # every later key scores higher, so the running maximum moves at each step
    hd, n = 64, 900
    q = torch.zeros(1, 1, hd)
    q[0, 0, 0] = 1.0
    kc = torch.zeros(n, 1, 1, hd)
    kc[:, 0, 0, 0] = torch.arange(n) / 8.0
    g = torch.Generator().manual_seed(1)
    vc = torch.randn(n, 1, 1, hd, generator=g)
    for dtype in BOTH:
        k, v, qq = kc.to(dtype).cuda(), vc.to(dtype).cuda(), q.to(dtype).cuda()
        table = np.arange(n, dtype=np.int32)[None]
        for order in (table, table[:, ::-1].copy()):
            kv = tsb.PagedKV(k, v, torch.from_numpy(order).cuda())
            out, lse = torch.empty_like(qq), torch.empty(1, 1, device="cuda")
            tsb.paged_attention(kv, qq, torch.tensor([n], dtype=torch.int32).cuda(), out, scale=1.0, lse=lse)
            check(out, lse, reference(k.double().cpu(), v.double().cpu(), order, qq.double().cpu(), [n], 1.0), dtype)


@pytest.mark.parametrize("dtype", BOTH)
def test_attention_with_infinite_and_lowest_values_in_view(dtype):
    # a visible key at the type's lowest value scores far below the rest: weight exactly 0
    kv, q, ln, out, lse, ref = attention_case([40], 2, 1, 64, 16, dtype, "heads", seed=2, poison=False)
    t = 7
    pg, sl = int(kv.page_table[0, t // 16]), t % 16
    q.abs_()
    kv.k_cache[pg, sl] = torch.finfo(dtype).min / 256
    tsb.paged_attention(kv, q, ln, out, lse=lse)
    keep = reference(kv.k_cache.double().cpu(), kv.v_cache.double().cpu(), kv.page_table.cpu().numpy(),
                     q.double().cpu(), [40], 64 ** -0.5)
    # the bound's score error comes from the keys that carry weight
    small = kv.k_cache.double().cpu().clone()
    small[pg, sl] = 0
    tol = reference(small, kv.v_cache.double().cpu(), kv.page_table.cpu().numpy(), q.double().cpu(), [40], 64 ** -0.5)
    check(out, lse, (keep[0], keep[1], tol[2], tol[3]), dtype)
    kv.k_cache[pg, sl] = -math.inf
    again = torch.empty_like(out)
    tsb.paged_attention(kv, q, ln, again, lse=lse)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", BOTH)
def test_attention_row_strides_and_optional_outputs(dtype):
    kv, q, ln, out, lse, ref = attention_case([33, 0, 80], 4, 2, 64, 16, dtype, "heads", seed=6)
    wide = torch.full((3, 11, 64), 7.0, dtype=dtype, device="cuda")
    wide[:, 3:7] = q
    got = torch.full((3, 9, 64), 7.0, dtype=dtype, device="cuda")
    tsb.paged_attention(kv, wide[:, 3:7], ln, got[:, 2:6])  # no lse, workspace of the call
    assert torch.equal(got[:, 2:6], out)
    assert (got[:, :2] == 7).all() and (got[:, 6:] == 7).all()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("n", [10, 5000])  # within one worker, and spread over many
def test_attention_passes_on_nan(dtype, n):
    kv, q, ln, out, lse, ref = attention_case([n, 33], 4, 2, 64, 16, dtype, "heads", seed=31, poison=False)
    q[0, 1] = math.nan  # one query: its row alone
    got, l2 = torch.empty_like(out), torch.empty_like(lse)
    tsb.paged_attention(kv, q, ln, got, lse=l2)
    assert torch.isnan(got[0, 1]).all() and torch.isnan(l2[0, 1])
    keep = torch.ones(2, 4, dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(got[keep], out[keep]) and torch.equal(l2[keep], lse[keep])
    q[0, 1] = 0
    pg = int(kv.page_table[0, (n - 1) // 16])
    kv.v_cache[pg, (n - 1) % 16, 1, 5] = math.nan  # one element of a value: that element of its heads
    tsb.paged_attention(kv, q, ln, got)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 2:, 5] = True
    assert torch.equal(torch.isnan(got), bad)
    kv.k_cache[pg, (n - 1) % 16, 1, 5] = math.nan  # a key: all of its heads
    tsb.paged_attention(kv, q, ln, got, lse=l2)
    bad[0, 2:] = True
    assert torch.equal(torch.isnan(got), bad) and torch.isnan(l2[0, 2:]).all() and not torch.isnan(l2[0, :2]).any()


INFINITE = [(12, 12, 64, 16), (8, 2, 64, 16), (16, 2, 64, 16), (9, 1, 128, 16), (40, 2, 96, 64), (6, 3, 32, 16), (4, 2, 64, 8)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("n", [10, 5000])  # within one worker, and spread over many
@pytest.mark.parametrize("NH,nkv,hd,page", INFINITE)
def test_attention_of_infinite_values_in_view(dtype, n, NH, nkv, hd, page):
    # softmax weights are positive: an infinite value is the output of its element, two of both
    # signs have no sum, and everything else is as without them
    kv, q, ln, out, lse, _ = attention_case([n, 33], NH, nkv, hd, page, dtype, "heads", seed=61, poison=False)
    table = kv.page_table.cpu()
    z = [torch.stack([kv.k_cache[int(table[0, t // page]), t % page, h] for t in range(min(n, 48))]).double().cpu()
         @ q[0, h * (NH // nkv)].double().cpu() for h in range(nkv)]

    def value(t, h):
        return kv.v_cache[int(table[0, t // page]), t % page, h]

    want = out.clone()
    for h in range(nkv):
        heads = slice(h * (NH // nkv), (h + 1) * (NH // nkv))
        # of the tokens at the front, the one that scores highest (its weight can be exactly a
        # power of two) and the lowest; and the last of all
        for t, e, x in ((int(z[h].argmax()), 3, math.inf), (int(z[h].argmin()), 4, -math.inf), (n - 1, 11, math.inf),
                        (0, 17, math.inf), (1, 17, math.inf), (2, 30, math.inf), (n - 1, 30, -math.inf)):
            value(t, h)[e] = x
            want[0, heads, e] = math.nan if e == 30 and x < 0 else x
    got, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    tsb.paged_attention(kv, q, ln, got, lse=l2)
    kv.check()
    assert torch.equal(l2, lse)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("lens", [[10, 1, 33], [5000, 77], [20000, 1]])
@pytest.mark.parametrize("NH,nkv,hd,page", [(12, 12, 64, 16), (16, 2, 64, 16), (6, 3, 32, 16), (8, 2, 128, 32), (4, 2, 96, 8)])
def test_attention_of_values_near_the_largest(dtype, lens, NH, nkv, hd, page):
    # the output is between the smallest and the largest visible value, so it is finite where the
    # values are: bf16 at the type's largest (its rounding errors leave fp32 256 steps of room),
    # fp32 at half of it
    top = torch.finfo(dtype).max / (1 if dtype == torch.bfloat16 else 2)
    kv, q, ln, out, lse, _ = attention_case(lens, NH, nkv, hd, page, dtype, "heads", seed=71, poison=False)
    kv.v_cache.clamp_(-1, 1).mul_(top)
    kv.v_cache[..., 0] = top
    kv.v_cache[..., 1] = -top
    args = (kv.v_cache.double().cpu(), kv.page_table.cpu().numpy(), q.double().cpu(), lens)
    ref = reference(kv.k_cache.double().cpu(), *args, hd ** -0.5)
    tsb.paged_attention(kv, q, ln, out, lse=lse)
    check(out, lse, ref, dtype)
    # scores that rise by 4 with every token and so leave every older maximum behind
    for b, n in enumerate(lens):
        for t in range(min(n, 200)):
            kv.k_cache[int(kv.page_table[b, t // page]), t % page] = 0
            kv.k_cache[int(kv.page_table[b, t // page]), t % page, :, 0] = 4.0 * t
    q.zero_()
    q[..., 0] = 1
    args = (kv.v_cache.double().cpu(), kv.page_table.cpu().numpy(), q.double().cpu(), lens)
    ref = reference(kv.k_cache.double().cpu(), *args, 1.0)
    tsb.paged_attention(kv, q, ln, out, scale=1.0, lse=lse)
    check(out, lse, ref, dtype)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("page", [8, 16, 64])
def test_attention_over_an_expanded_cache(dtype, page):
    # one stored head shown as four (head stride 0)
    g = torch.Generator().manual_seed(17)
    rng = np.random.default_rng(17)
    lens = [100, 1, 37]
    table, pages = tables(lens, page, 1, rng)
    kc, vc = (pool(pages, page, 1, 64, dtype, "tokens", g).expand(-1, -1, 4, -1) for _ in range(2))
    q = torch.randn(3, 8, 64, generator=g).to(dtype).cuda()
    kv = tsb.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    tsb.paged_attention(kv, q, torch.tensor(lens, dtype=torch.int32).cuda(), out, lse=lse)
    kv.check()
    check(out, lse, reference(kc.double().cpu(), vc.double().cpu(), table, q.double().cpu(), lens, 0.125), dtype)


def test_attention_of_the_most_sequences():
    attention_case([(i * 29) % 23 for i in range(4096)], 2, 1, 32, 16, torch.bfloat16, "heads", seed=41)


def test_attention_offsets_beyond_32_bits():
    # two pages more than 2^32 bytes and 2^31 elements apart, in caches of 4.5 GB
    page, nkv, hd = 16, 1, 64
    pages = 2 ** 31 // (page * hd) + 8
    kc = torch.zeros(pages, page, nkv, hd, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros(pages, page, nkv, hd, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(2)
    table = np.array([[pages - 1, 0, pages - 3]], np.int32)
    k, v = torch.randn(40, 1, hd, generator=g).bfloat16().cuda(), torch.randn(40, 1, hd, generator=g).bfloat16().cuda()
    kv = tsb.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    pos = torch.arange(40, dtype=torch.int32).cuda()
    tsb.paged_kv_append(kv, k, v, pos, torch.zeros(40, dtype=torch.int32).cuda())
    assert torch.equal(kc[pages - 1].flatten(), k[:16].flatten()) and torch.equal(vc[pages - 3, :8].flatten(), v[32:].flatten())
    q = torch.randn(1, 2, hd, generator=g).bfloat16().cuda()
    out = torch.empty_like(q)
    tsb.paged_attention(kv, q, torch.tensor([40], dtype=torch.int32).cuda(), out)
    near = np.array([[0, 1, 2]], np.int32)
    kk, vv = torch.zeros(3 * 16, 1, hd).double(), torch.zeros(3 * 16, 1, hd).double()
    kk[:40], vv[:40] = k.double().cpu(), v.double().cpu()
    check(out, None, reference(kk.view(3, 16, 1, hd), vv.view(3, 16, 1, hd), near, q.double().cpu(), [40], 0.125),
          torch.bfloat16)
    kv.check()


def test_attention_reports_bad_pages_and_lengths():
    kv, q, ln, out, lse, ref = attention_case([40, 64], 4, 2, 64, 16, torch.bfloat16, "heads", seed=9, poison=False)
    good = kv.page_table.clone()
    for bad in (-1, kv.k_cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        kv.page_table[0, 1] = bad
        tsb.paged_attention(kv, q, ln, out)
        with pytest.raises(tsb.Gpt2Error) as e:
            kv.check()
        assert e.value.code == -9
        kv.check()  # cleared
        # the other sequence is as it was, and the bad page's keys are left out
        keep = [t for t in range(40) if t // 16 != 1]
        z = torch.zeros_like(ref[0])
        kc, vc = kv.k_cache.double().cpu(), kv.v_cache.double().cpu()
        for h in range(4):
            pg = good.cpu()[0].long()[torch.tensor(keep) // 16]
            k, v = kc[pg, torch.tensor(keep) % 16, h // 2], vc[pg, torch.tensor(keep) % 16, h // 2]
            z[0, h] = torch.softmax(k @ q[0, h].double().cpu() * 0.125, 0) @ v
        z[1] = ref[0][1]
        check(out, None, (z, None, ref[2], None), torch.bfloat16)
    kv.page_table.copy_(good)
    whole = kv.page_table.shape[1] * 16
    for n in (-1, -2 ** 31, whole + 1, 2 ** 31 - 1):
        ln[0] = n
        tsb.paged_attention(kv, q, ln, out, lse=lse)
        with pytest.raises(tsb.Gpt2Error):
            kv.check()
        check(out[1:], lse[1:], tuple(r[1:] for r in ref), torch.bfloat16)
        if n < 0:
            assert (out[0] == 0).all() and (lse[0] == -math.inf).all()


@pytest.mark.parametrize("dtype", BOTH)
def test_attention_is_deterministic_on_a_used_workspace(dtype):
    kv, q, ln, out, lse, _ = attention_case([3000, 10, 700], 8, 2, 64, 16, dtype, "heads", seed=12)
    ws = kv.attention_workspace(8)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        again, l2 = torch.full_like(out, math.nan), torch.empty_like(lse)
        tsb.paged_attention(kv, q, ln, again, lse=l2, ws=ws)
        assert torch.equal(again, out) and torch.equal(l2, lse)
    short = torch.tensor([1, 10, 2], dtype=torch.int32).cuda()
    tsb.paged_attention(kv, q, short, again, ws=ws)  # other lengths in between leave no trace
    tsb.paged_attention(kv, q, ln, again, ws=ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("NH,nkv", [(40, 2), (20, 1), (17, 1), (11, 1), (5, 5), (3, 3)])
@pytest.mark.parametrize("hd", [32, 64, 128])
def test_attention_does_not_depend_on_what_ran_before(dtype, NH, nkv, hd):
    # groups that are no multiple of a query tile: rows of the tile that do not exist
    lens = [3000, 10, 700, 1, 64, 129, 333, 1500]
    kv, q, ln, out, lse, _ = attention_case(lens, NH, nkv, hd, 16, dtype, "heads", seed=81)
    most = torch.full_like(ln, 3000 - 3000 % 16)
    other = tsb.PagedKV(*(torch.randn(200, 16, 1, hd, device="cuda").to(dtype) for _ in range(2)),
                        torch.arange(200, dtype=torch.int32, device="cuda").repeat(len(lens), 1))
    for x in (0.0, 30.0, -30.0, 1e4, math.nan):
        # large queries of every row of the tile in all of the SMs' shared memory
        big = (torch.randn(len(lens), 32, hd, device="cuda") * x).to(dtype)
        tsb.paged_attention(other, big, most, torch.empty_like(big))
        got, l2 = torch.empty_like(out), torch.empty_like(lse)
        tsb.paged_attention(kv, q, ln, got, lse=l2)
        assert torch.equal(l2, lse) and torch.equal(got, out)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def rotated(x, cs, rot, pairs):
    """float64 rotation of x [n, heads, hd] by table rows cs [n, rot], and the bound's scale."""
    x = x.double().cpu()
    out, mag = x.clone(), torch.zeros_like(x)
    if rot:
        i = torch.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        c, s = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., a] * s).abs() + (x[..., b] * c).abs()
    return out, mag


def near(got, want, mag, dtype):
    err = (got.double().cpu() - want).abs()
    assert (err <= unit(dtype) * want.abs() * (mag > 0) + 4 * E * mag).all()


def append_case(rows, seqs, ctx, NH, nkv, hd, rot, pairs, page, dtype, layout, seed=0, with_q=True, in_place=False,
                pad=0, far=0):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    table, pages = tables([ctx] * seqs, page, 3, rng)
    kc, vc = pool(pages, page, nkv, hd, dtype, layout, g), pool(pages, page, nkv, hd, dtype, layout, g)
    slots = rng.permutation(seqs * ctx)[:rows]
    seq, pos = (slots // ctx).astype(np.int32), (slots % ctx).astype(np.int32)
    live = np.ones(rows + pad, bool)
    live[rng.permutation(rows + pad)[:pad]] = False
    full_seq, full_pos = np.full(rows + pad, 10 ** 6, np.int32), np.full(rows + pad, -1, np.int32)
    full_seq[live], full_pos[live] = seq, pos
    full_pos[~live] = -1 - rng.integers(0, 2 ** 31 - 1, pad)
    qkv = torch.randn(rows + pad, (NH + 2 * nkv) * hd, generator=g).to(dtype).cuda()
    qkv[torch.from_numpy(~live).cuda()] = math.nan
    q, k, v = (t.unflatten(1, (-1, hd)) for t in qkv.split([NH * hd, nkv * hd, nkv * hd], 1))
    cs = tsb.rotation_table(ctx + far, rot) if rot else None
    before = [t.clone() for t in (kc, vc)]
    q_in = q.clone()
    q_out = q if in_place else torch.full((rows + pad, NH, hd), 5.0, dtype=dtype, device="cuda")
    kv = tsb.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    tsb.paged_kv_append(kv, k, v, torch.from_numpy(full_pos).cuda(), torch.from_numpy(full_seq).cuda(),
                        q=q if with_q else None, q_out=q_out if with_q else None, cos_sin=cs, interleaved=pairs)
    kv.check()
    pg, sl = torch.from_numpy(table[seq, pos // page].astype(np.int64)), torch.from_numpy((pos % page).astype(np.int64))
    rowsl = torch.from_numpy(np.flatnonzero(live))
    csr = cs.double().cpu()[torch.from_numpy(pos.astype(np.int64))] if rot else None
    want, mag = rotated(k.cpu()[rowsl], csr, rot, pairs)
    got = kc.cpu()[pg, sl]
    near(got, want, mag, dtype)
    assert torch.equal(vc.cpu()[pg, sl], v.cpu()[rowsl])
    # everything else is as it was
    rest = torch.ones(pages, page, dtype=torch.bool)
    rest[pg, sl] = False
    for t, old in ((kc, before[0]), (vc, before[1])):
        assert torch.equal(t.cpu()[rest], old.cpu()[rest])
    if with_q:
        want, mag = rotated(q_in.cpu()[rowsl], csr, rot, pairs)
        near(q_out.cpu()[rowsl], want, mag, dtype)
        if pad:
            dead = torch.from_numpy(np.flatnonzero(~live))
            assert torch.isnan(q_out.cpu()[dead]).all() if in_place else (q_out.cpu()[dead] == 5).all()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("hd", [32, 64, 96, 128])
@pytest.mark.parametrize("pairs", [False, True])
def test_append_rotations(dtype, hd, pairs):
    for rot in range(0, hd + 1, 16):
        append_case(37, 5, 33, 6, 2, hd, rot, pairs, 8, dtype, "heads", seed=rot, pad=rot // 16)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("layout", ["tokens", "heads", "heads first", "padded"])
@pytest.mark.parametrize("page", [1, 4, 64])
def test_append_layouts(dtype, layout, page):
    append_case(50, 3, 70, 4, 4, 64, 32, False, page, dtype, layout, seed=page, pad=2)


@pytest.mark.parametrize("rows,seqs,ctx,NH,nkv", [(1, 1, 1, 1, 1), (2, 7, 9, 3, 1), (1000, 2, 700, 2, 1),
                                                  (5000, 8, 800, 2, 2), (64, 64, 5, 128, 8), (3, 2, 40, 25, 25)])
@pytest.mark.parametrize("dtype", BOTH)
def test_append_sizes(dtype, rows, seqs, ctx, NH, nkv):
    append_case(rows, seqs, ctx, NH, nkv, 64, 64, False, 16, dtype, "heads", seed=rows, pad=rows % 3)
    append_case(rows, seqs, ctx, NH, nkv, 64, 0, False, 16, dtype, "heads", seed=rows, with_q=False)


@pytest.mark.parametrize("pairs", [False, True])
def test_append_rotates_queries_in_place(pairs):
    append_case(90, 4, 50, 12, 12, 64, 48, pairs, 16, torch.bfloat16, "heads", in_place=True, pad=3)


def test_append_without_sequence_indices():
    g = torch.Generator().manual_seed(0)
    kc, vc = (torch.zeros(8, 4, 2, 32, device="cuda") for _ in range(2))
    kv = tsb.PagedKV(kc, vc, torch.arange(8, dtype=torch.int32).view(4, 2).cuda())
    k, v = torch.randn(3, 2, 32, generator=g).cuda(), torch.randn(3, 2, 32, generator=g).cuda()
    tsb.paged_kv_append(kv, k, v, torch.tensor([6, -1, 1], dtype=torch.int32).cuda())
    kv.check()
    assert torch.equal(kc[1, 2], k[0]) and torch.equal(vc[4, 1], v[2])
    assert int((kc != 0).any(-1).any(-1).sum()) == 2
    tsb.paged_kv_append(kv, k[:0], v[:0], torch.empty(0, dtype=torch.int32, device="cuda"))


def test_append_reports_rows_outside_the_cache():
    def fresh():
        kc, vc = (torch.zeros(8, 4, 2, 32, device="cuda") for _ in range(2))
        return tsb.PagedKV(kc, vc, torch.arange(8, dtype=torch.int32).view(4, 2).cuda())
    k = torch.ones(2, 2, 32, device="cuda")
    q_out = torch.full((2, 4, 32), 5.0, device="cuda")
    q = torch.ones(2, 4, 32, device="cuda")
    cs = tsb.rotation_table(6, 32)
    for pos, seq, entry in ((8, 0, None), (2 ** 31 - 1, 0, None), (6, 0, None), (0, 4, None), (0, -1, None),
                            (0, 0, 8), (0, 0, -1), (0, 2 ** 31 - 1, None)):
        kv = fresh()
        if entry is not None:
            kv.page_table[0, 0] = entry
        q_out.fill_(5.0)
        tsb.paged_kv_append(kv, k, k, torch.tensor([pos, 3], dtype=torch.int32).cuda(),
                            torch.tensor([seq, 1], dtype=torch.int32).cuda(), q=q, q_out=q_out, cos_sin=cs)
        with pytest.raises(tsb.Gpt2Error) as e:
            kv.check()
        assert e.value.code == -9
        kv.check()
        assert (kv.v_cache[2, 3] == 1).all() and int((kv.v_cache != 0).any(-1).any(-1).sum()) == 1
        assert (q_out[0] == 5).all() and (q_out[1] != 5).all()


def test_bindings_refuse():
    kc, vc = (torch.zeros(8, 4, 2, 32, device="cuda") for _ in range(2))
    table = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    kv = tsb.PagedKV(kc, vc, table)
    with pytest.raises(ValueError):
        tsb.PagedKV(kc, vc.bfloat16(), table)
    with pytest.raises(ValueError):
        tsb.PagedKV(kc, vc[:, :, :1], table)
    with pytest.raises(ValueError):
        tsb.PagedKV(kc, vc, table.long())
    with pytest.raises(ValueError):
        tsb.PagedKV(kc, vc, table.cpu())
    with pytest.raises(ValueError):
        tsb.PagedKV(kc.transpose(2, 3), vc.transpose(2, 3), table)
    q, n = torch.zeros(3, 4, 32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    for bad in (dict(q=q.bfloat16()), dict(q=q[:2]), dict(q=q[..., :16]), dict(q=q[0]), dict(out=out[:, :2]),
                dict(seq_lens=n.long()), dict(seq_lens=n[:2]), dict(seq_lens=n.cpu()),
                dict(lse=torch.zeros(3, 5, device="cuda")), dict(q=torch.zeros(3, 4, 64, device="cuda")[..., ::2]),
                dict(ws=torch.zeros(1 << 26, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            tsb.paged_attention(kv, **{**dict(q=q, seq_lens=n, out=out), **bad})
    for bad in (dict(window=-1), dict(window=2 ** 32 + 5), dict(sinks=-1), dict(sinks=2 ** 31)):
        with pytest.raises(ValueError):
            tsb.paged_attention(kv, q, n, out, **bad)
    with pytest.raises(ValueError):  # an explicit stream needs its own workspace
        tsb.paged_attention(kv, q, n, out, stream=torch.cuda.current_stream().cuda_stream)
    with pytest.raises(tsb.Gpt2Error):
        tsb.paged_attention(kv, q, n, out, ws=torch.zeros(4, device="cuda")[:0])
    with pytest.raises(tsb.Gpt2Error):
        tsb.paged_attention(kv, torch.zeros(3, 3, 32, device="cuda"), n, torch.zeros(3, 3, 32, device="cuda"))
    k = torch.zeros(3, 2, 32, device="cuda")
    for bad in (dict(v=k[:2]), dict(k=k[:, :1]), dict(positions=n.long()), dict(seqs=n[:1]), dict(q=q),
                dict(q=q, q_out=out[:2]), dict(cos_sin=torch.zeros(9, 32, device="cuda").double()),
                dict(cos_sin=torch.zeros(9, 64, device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            tsb.paged_kv_append(kv, **{**dict(k=k, v=k, positions=n), **bad})


# ---------------------------------------------------------------------------
# together, as a program that serves requests uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,window,sinks", [(torch.bfloat16, 0, 0), (torch.float32, 0, 0), (torch.bfloat16, 9, 2)])
def test_prompts_then_tokens_equal_causal_attention(dtype, window, sinks):
    """Ragged prompts appended at once, then tokens one by one: each step's output is the row of
    causal attention over the whole sequence, and (without a window) the row that the training
    attention computes."""
    NH, hd, page, prompts, steps = 4, 64, 8, [5, 1, 30], 12
    C = NH * hd
    T = [p + steps for p in prompts]
    g = torch.Generator().manual_seed(4)
    qkv = [torch.randn(t, 3 * C, generator=g).to(dtype).cuda() for t in T]
    rng = np.random.default_rng(0)
    table, pages = tables(T, page, 0, rng)
    kc, vc = pool(pages, page, NH, hd, dtype, "heads", g), pool(pages, page, NH, hd, dtype, "heads", g)
    kv = tsb.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    ws = kv.attention_workspace(NH)
    rows = torch.cat([x[:p] for x, p in zip(qkv, prompts)])
    k, v = rows[:, C:2 * C].unflatten(1, (NH, hd)), rows[:, 2 * C:].unflatten(1, (NH, hd))
    pos = torch.cat([torch.arange(p) for p in prompts]).int().cuda()
    seq = torch.cat([torch.full((p,), b) for b, p in enumerate(prompts)]).int().cuda()
    tsb.paged_kv_append(kv, k, v, pos, seq)
    got = [[] for _ in prompts]
    for s in range(steps):
        x = torch.stack([qkv[b][prompts[b] + s] for b in range(3)]).view(3, 3, NH, hd)
        at = torch.tensor([p + s for p in prompts], dtype=torch.int32).cuda()
        tsb.paged_kv_append(kv, x[:, 1], x[:, 2], at)
        out = torch.empty(3, NH, hd, dtype=dtype, device="cuda")
        tsb.paged_attention(kv, x[:, 0], at + 1, out, window=window, sinks=sinks, ws=ws)
        for b in range(3):
            got[b].append(out[b])
    kv.check()
    for b in range(3):
        x = qkv[b].double().cpu().view(T[b], 3, NH, hd)
        flat = np.arange(T[b], dtype=np.int32)[None]
        for s in range(steps):
            n = prompts[b] + s + 1
            ref = reference(x[:, 1].unsqueeze(1), x[:, 2].unsqueeze(1), flat, x[n - 1:n, 0], [n], 0.125, window, sinks)
            check(got[b][s][None], None, ref, dtype)
        if window == 0:
            whole, lse = torch.zeros(T[b], C, dtype=dtype, device="cuda"), torch.zeros(1, NH, T[b], device="cuda")
            tsb.attention_fwd(qkv[b], whole, lse, 1, T[b], NH, hd)
            a, w = torch.stack(got[b]).double(), whole[prompts[b]:].view(steps, NH, hd).double()
            # two bf16 results, the training kernel's with bf16 weights: the bar of its own tests
            assert float((a - w).norm() / w.norm()) <= (2e-2 if dtype == torch.bfloat16 else 1e-5)


@pytest.mark.parametrize("dtype", BOTH)
def test_captured_step_replays_with_new_lengths(dtype):
    NH, nkv, hd, page, B = 8, 2, 64, 16, 3
    g = torch.Generator().manual_seed(7)
    table = torch.arange(B * 64, dtype=torch.int32).view(B, 64).cuda()
    kc, vc = (torch.randn(B * 64, page, nkv, hd, generator=g).to(dtype).cuda() for _ in range(2))
    kv = tsb.PagedKV(kc, vc, table)
    q, k, v = (torch.randn(B, n, hd, generator=g).to(dtype).cuda() for n in (NH, nkv, nkv))
    pos, lens = torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros(B, dtype=torch.int32).cuda()
    out, out2, qr = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    cs = tsb.rotation_table(1024, hd)
    ws, ws2 = kv.attention_workspace(NH), kv.attention_workspace(NH)

    def step(o, w):
        tsb.paged_kv_append(kv, k, v, pos, q=q, q_out=qr, cos_sin=cs)
        tsb.paged_attention(kv, qr, lens, o, ws=w)

    pos.fill_(5), lens.fill_(6)
    step(out, ws)  # sets kernel attributes
    torch.cuda.synchronize()
    graphs = []
    for o, w in ((out, ws), (out2, ws2)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(o, w)
        graphs.append(gr)
    for n in ([1, 300, 1024], [0, 0, 7], [900, 901, 902], [64, 1, 128]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        pos.copy_(lens - 1)
        for gr in graphs:
            gr.replay()
        want = torch.empty_like(q)
        tsb.paged_attention(kv, qr, lens, want)
        assert torch.equal(out, want) and torch.equal(out2, want)
    kv.check()


def test_captured_behind_copies_and_other_streams():
    # the calls start early behind other kernels; here copies, fills and a joined stream precede
    kv, q, ln, out, lse, _ = attention_case([3000, 10, 700], 8, 2, 64, 16, torch.bfloat16, "heads", seed=23)
    ws, got, n, qq = kv.attention_workspace(8), torch.empty_like(out), torch.zeros_like(ln), torch.zeros_like(q)
    k, v = torch.randn(2, 3, 2, 64).bfloat16().cuda().unbind(0)
    pos = torch.empty_like(ln)
    side = torch.cuda.Stream()
    before = kv.k_cache.clone(), kv.v_cache.clone()
    torch.cuda.synchronize()

    def body():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            qq.copy_(q)
        n.copy_(ln)
        got.zero_()
        torch.sub(ln, 1, out=pos)
        torch.cuda.current_stream().wait_stream(side)
        tsb.paged_kv_append(kv, k, v, pos)
        tsb.paged_attention(kv, qq, n, got, ws=ws)
        kv.k_cache.copy_(before[0])  # as it was, for the next run
        kv.v_cache.copy_(before[1])

    body()
    torch.cuda.synchronize()
    want = got.clone()
    assert not torch.equal(want, out)  # the appended tokens count
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        body()
    for _ in range(20):
        for t in (qq, n, pos, got):
            t.zero_()
        gr.replay()
        assert torch.equal(got, want)
    for _ in range(20):
        body()
        assert torch.equal(got, want)
    kv.check()


def test_captured_calls_share_a_workspace_in_turn():
    kv, q, ln, out, lse, _ = attention_case([3000, 10, 700], 8, 2, 64, 16, torch.bfloat16, "heads", seed=22)
    ws = kv.attention_workspace(8)
    # the second reads past the third sequence's tokens, into NaN and bad pages: the same each time
    lens = [ln] + [torch.tensor(n, dtype=torch.int32).cuda() for n in ([77, 0, 2999], [500, 3, 650])]
    want = [out] + [torch.empty_like(out) for _ in lens[1:]]
    for n, o in zip(lens[1:], want[1:]):
        tsb.paged_attention(kv, q, n, o)
    assert torch.isfinite(want[2].float()).all()
    outs, graphs = [torch.empty_like(out) for _ in lens], []
    for o, n in zip(outs, lens):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            tsb.paged_attention(kv, q, n, o, ws=ws)
            tsb.paged_attention(kv, q, n, o, ws=ws)
        graphs.append(gr)
    for fill in (None, 85, 255):
        if fill is not None:
            ws.fill_(fill)
        for which in (0, 0, 1, 2, 0, 2, 2, 1, 1, 0):
            outs[which].zero_()
            graphs[which].replay()
            assert torch.equal(outs[which].view(torch.int16), want[which].view(torch.int16))


def test_calls_on_other_streams():
    kv, q, ln, out, lse, ref = attention_case([3000, 10, 700], 8, 2, 64, 16, torch.bfloat16, "heads", seed=21)
    streams = [torch.cuda.Stream() for _ in range(3)]
    work = [kv.attention_workspace(8) for _ in streams]
    outs = [torch.full_like(out, math.nan) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, w, o in zip(streams, work, outs):
            tsb.paged_attention(kv, q, ln, o, ws=w, stream=s.cuda_stream)
    with torch.cuda.stream(streams[0]):
        own = torch.empty_like(out)
        tsb.paged_attention(kv, q, ln, own)
    torch.cuda.synchronize()
    for o in outs + [own]:
        assert torch.equal(o, out)


def small_cache():
    kc, vc = (torch.zeros(8, 4, 2, 32, device="cuda") for _ in range(2))
    return tsb.PagedKV(kc, vc, torch.arange(8, dtype=torch.int32).view(4, 2).cuda())


def raises_page_range(kv, stream=None):
    try:
        kv.check(stream)
    except tsb.Gpt2Error as e:
        assert e.code == -9
        return True
    return False


def test_no_report_is_lost_between_streams():
    # a call on one stream meets a bad position while the word is read and cleared on another:
    # that check or the next one reports it
    kv = small_cache()
    k = torch.ones(1, 2, 32, device="cuda")
    pos = torch.tensor([8], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kv.check()
    for i in range(3000):
        with torch.cuda.stream(side):
            torch.cuda._sleep(97 * (i % 300))  # up to some 15 us
            tsb.paged_kv_append(kv, k, k, pos)
        first = raises_page_range(kv)
        side.synchronize()
        assert raises_page_range(kv) or first, i


def test_a_wait_that_gave_up_is_reported_before_a_bad_page():
    # the word as the header describes it: 1 for something outside the cache, 2 for a wait that
    # gave up (after which the results are void, whatever else was met)
    kv = small_cache()
    for word, code in ((1, -9), (2, -8), (3, -8)):
        kv.status.fill_(word)
        with pytest.raises(tsb.Gpt2Error) as e:
            kv.check()
        assert e.value.code == code
        kv.check()
    k = torch.ones(1, 2, 32, device="cuda")
    kv.status.fill_(2)
    tsb.paged_kv_append(kv, k, k, torch.tensor([8], dtype=torch.int32, device="cuda"))
    with pytest.raises(tsb.Gpt2Error) as e:
        kv.check()
    assert e.value.code == -8


def test_a_cache_is_ready_for_every_stream():
    # the status word is set up behind other work on the constructor's stream; a call on another
    # stream does not wait for that, and its report must last
    k = torch.ones(1, 2, 32, device="cuda")
    pos = torch.tensor([8], dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(8, 4, 2, 32, device="cuda") for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    kv = tsb.PagedKV(kc, vc, table)
    tsb.paged_kv_append(kv, k, k, pos, stream=side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert raises_page_range(kv)


def test_append_into_rows_between_others():
    # queries, keys, values and the rotated queries side by side in one tensor's rows
    g = torch.Generator().manual_seed(91)
    for dtype in BOTH:
        kc, vc = (torch.zeros(8, 4, 2, 32, dtype=dtype, device="cuda") for _ in range(2))
        kv = tsb.PagedKV(kc, vc, torch.arange(8, dtype=torch.int32).view(4, 2).cuda())
        rows = torch.randn(4, 12, 32, generator=g).to(dtype).cuda()
        pos = torch.tensor([6, 0, -1, 3], dtype=torch.int32, device="cuda")
        cs, was = tsb.rotation_table(8, 32), rows.clone()
        own = torch.full((4, 4, 32), 3.0, dtype=dtype, device="cuda")
        tsb.paged_kv_append(kv, rows[:, 4:6], rows[:, 6:8], pos, q=rows[:, :4], q_out=own, cos_sin=cs)
        tsb.paged_kv_append(kv, rows[:, 4:6], rows[:, 6:8], pos, q=rows[:, :4], q_out=rows[:, 8:], cos_sin=cs)
        kv.check()
        live = pos >= 0
        assert torch.equal(rows[:, :8], was[:, :8]) and torch.equal(rows[live][:, 8:], own[live])
        assert torch.equal(rows[2, 8:], was[2, 8:])
        for bad in (rows[:, 1:5], rows[:, 7:11]):
            with pytest.raises(tsb.Gpt2Error):
                tsb.paged_kv_append(kv, rows[:, 4:6], rows[:, 6:8], pos, q=rows[:, :4], q_out=bad, cos_sin=cs)
