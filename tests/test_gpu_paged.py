"""GPU parity of the paged serving operators (page plan, e4m3 cache write, prompt
attention, decode attention over the cache) with the float64 paged oracle.

Integers, codes and scales are equal. Attention: with u = 2^-8 (a bf16 rounding
is off by at most half a step, eps / 2, relative), every output is

    |err| <= u |o| + (u + 2 d + n 2^-24) a,      |err lse| <= d + n 2^-24 + 2^-23 |lse|

with a = the softmax average of |v| (from the oracle), n the keys of the row: u |o|
rounds the output, u a the probabilities, n 2^-24 the fp32 sums, and d bounds the
error of a score and its exponential: 128 + 2 roundings to fp32 of sums of at most
s = scale * sum |q||k| (from the oracle), and 2^-20 for exp2 and its argument.
"""

import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from oracle.cslc_oracle import e4m3_decode
from tests.helpers import f64

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32
SCALE = 1 / math.sqrt(128)
U = 2.0 ** -8


@pytest.fixture(scope="module")
def C(cuda_device):
    from compressed_sparse_long_compress_b200 import cslc
    return cslc


def i32(x):
    return torch.tensor(np.asarray(x), dtype=I32, device="cuda")


def randn(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def check_attention(got, lse, ref, n, what=""):
    o, l, a, s = ref
    rows = ~np.isnan(l)
    got, lse, o, l, a, s = f64(got)[rows], f64(lse)[rows], o[rows], l[rows], a[rows], s[rows]
    d = s * 130 * 2.0 ** -24 + 2.0 ** -20
    tol = U * np.abs(o) + (U + 2 * d + n * 2.0 ** -24)[..., None] * a
    bad = ~(np.abs(got - o) <= tol + 1e-30)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outputs, worst {np.nanmax(np.abs(got - o) - tol):.3e} beyond"
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(lse), empty), what
    e = np.abs(lse[~empty] - l[~empty])
    tl = (d + n * 2.0 ** -24)[~empty] + 2.0 ** -23 * np.abs(l[~empty])
    assert (e <= tl).all(), f"{what}: lse off by {e.max():.3e}, allowed {tl[e.argmax()]:.3e}"


def check_peaked(got, lse, ref, what):
    """Rows whose weight is on one key or on equal ones: the roundings of P and of the output are left, and of the
    lse six to fp32 of numbers of its size (scale, log2(e), their product, the score, the sum, ln(2)), less than 2^-21
    of it, and what log2 of a few equal ones adds."""
    o, l, a, _ = ref
    got, lse = f64(got), f64(lse)
    err, tol = np.abs(got - o), U * np.abs(o) + (U + 2.0 ** -16) * a
    assert (err <= tol).all(), f"{what}: {(~(err <= tol)).any(-1).sum()} of {l.size} rows, lse off by {np.abs(lse - l).max():.3e}"
    tl = 2.0 ** -21 * np.abs(l) + 2.0 ** -16
    assert (np.abs(lse - l) <= tl).all(), f"{what}: lse off by {np.abs(lse - l).max():.3e}"


# ---------------------------------------------------------------- page plan

def run_plan(C, old, new, free, table, page, n_pages, max_tokens):
    got = i32(table)
    slots, cu, n, st = C.page_plan(i32(old), i32(new), i32(free), got, page, n_pages, max_tokens=max_tokens)
    ref = PO.page_plan(old, new, free, table, page, n_pages, max_tokens)
    for g, r, name in zip((got, slots, cu, n, st), ref, ("table", "slots", "cu", "seq_len", "status")):
        assert np.array_equal(g.cpu().numpy(), r), name
    return got, slots, cu, n, st


def plan_case(seed, B, max_old, max_new, page, extra=3, width=None):
    r = np.random.RandomState(seed)
    old, new = r.randint(0, max_old + 1, B), r.randint(0, max_new + 1, B)
    p0, p1 = -(-old // page), -(-(old + new) // page)
    n_pages = int(p1.sum()) + extra
    pool = r.permutation(n_pages)
    width = int(p1.max()) + 1 if width is None else width
    table = np.full((B, width), -7)
    at = 0
    for b in range(B):
        m = min(p0[b], width)
        table[b, :m] = pool[at:at + m]
        at += m
    return old, new, pool[at:], table, n_pages


@pytest.mark.parametrize("B,max_old,max_new,page", [(1, 0, 1, 16), (1, 100, 700, 64), (7, 50, 1, 128), (64, 300, 40, 32),
                                                    (513, 90, 33, 16), (1500, 20, 2, 64)])
def test_plan(C, B, max_old, max_new, page):
    old, new, free, table, n_pages = plan_case(B + page, B, max_old, max_new, page)
    run_plan(C, old, new, free, table, page, n_pages, int(new.sum()) + 9)


def test_plan_runs_short_of_pages(C):
    old, new, free, table, n_pages = plan_case(5, 40, 60, 70, 16)
    need = int(PO.page_plan(old, new, free, table, 16, n_pages, 1)[4][0])
    for k in (0, 1, need // 2, need - 1):
        run_plan(C, old, new, free[:k], table, 16, n_pages, int(new.sum()))


def test_plan_bad_pages_short_tables_and_few_slots(C):
    old, new, free, table, n_pages = plan_case(6, 40, 60, 70, 16)
    bad = free.copy()
    bad[::3] = -1
    bad[1::5] = n_pages + 4
    run_plan(C, old, new, bad, table, 16, n_pages, int(new.sum()))
    held = table.copy()
    held[::2] = -1                                             # partly full pages that do not exist
    run_plan(C, old, new, free, held, 16, n_pages, int(new.sum()))
    run_plan(C, old, new, free, table[:, :3].copy(), 16, n_pages, int(new.sum()))
    run_plan(C, old, new, free, table, 16, n_pages, int(new.sum()) // 3)
    run_plan(C, old, new, free, table, 16, n_pages, 0)
    neg = old.copy()
    neg[:5] = -9
    neg_new = new.copy()
    neg_new[3:9] = -2
    run_plan(C, neg, neg_new, free, np.abs(table), 16, n_pages, int(new.sum()))


def test_plan_most_sequences_and_none(C):
    old, new, free, table, n_pages = plan_case(8, 8192, 30, 3, 16)
    run_plan(C, old, new, free, table, 16, n_pages, int(new.sum()) + 1)
    e = np.zeros(0, dtype=np.int32)
    run_plan(C, e, e, [1, 2], np.zeros((0, 3)), 16, 4, 5)


def test_plan_large_lengths(C):
    big = 2 ** 31 - 1
    table = np.full((3, 2), -1)
    run = C.page_plan(i32([big, 0, 5]), i32([0, 3, 0]), i32([4, 5]), i32(table), 64, 8, max_tokens=4)
    assert run[0].tolist() == [256, 257, 258, -1] and run[3].tolist() == [1, 0]
    assert run[1].tolist() == [0, 0, 3, 3] and run[2].tolist() == [big, 3, 5]


def test_plan_counts_more_lost_tokens_than_32_bits_hold(C):
    table = i32(np.full((4, 2), -1))
    for n, lost in (([2 ** 30] * 4, 2 ** 31 - 1), ([2 ** 30, 2 ** 30, 0, 0], 2 ** 31 - 1), ([2 ** 30, 2 ** 30 - 1, 0, 0], 2 ** 31 - 1),
                    ([2 ** 30, 5, 0, 0], 2 ** 30 + 5)):
        slots, cu, total, st = C.page_plan(i32([0] * 4), i32(n), i32([]), table.clone(), 16, 8, max_tokens=3)
        assert st.tolist()[1] == lost and slots.tolist() == [-1] * 3
        assert cu.tolist() == [min(sum(n[:i]), 2 ** 31 - 1) for i in range(5)] and total.tolist() == n


# -------------------------------------------------------------- cache write

def empty_cache(n_pages, Hkv, P, fill=0):
    c = torch.full((n_pages, Hkv, P, 128), fill, dtype=torch.uint8, device="cuda")
    return c, torch.full((n_pages, Hkv), 2.0 ** -5, device="cuda")


def run_write(C, k, v, slots, kc, vc, ks, vs):
    ref = [PO.page_write(f64(x), slots.cpu().numpy(), c.cpu().numpy(), f64(s)) for x, c, s in ((k, kc, ks), (v, vc, vs))]
    C.page_write_e4m3(k, v, slots, kc, vc, ks, vs)
    for (codes, scale), c, s, name in zip(ref, (kc, vc), (ks, vs), "kv"):
        assert np.array_equal(f64(s), scale), name
        assert np.array_equal(c.cpu().numpy(), codes), name


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,lens", [(1, [1]), (3, [5, 130, 1, 64]), (8, [1] * 33), (2, [127, 128, 129, 300])])
def test_write_ragged(C, P, Hkv, lens):
    r = np.random.RandomState(P + Hkv)
    old = r.randint(0, 2 * P, len(lens))
    p0, p1 = -(-old // P), -(-(old + lens) // P)
    n_pages = int(p1.sum()) + 2
    pool = r.permutation(n_pages)
    table, at = np.full((len(lens), int(p1.max())), -1), 0
    for b in range(len(lens)):
        table[b, :p0[b]] = pool[at:at + p0[b]]
        at += p0[b]
    _, slots, _, _, _ = run_plan(C, old, lens, pool[at:], table, P, n_pages, sum(lens) + 3)
    kc, ks = empty_cache(n_pages, Hkv, P, 0x31)
    vc, vs = empty_cache(n_pages, Hkv, P, 0xC5)
    kv = randn((slots.numel(), 2, Hkv, 128), 40 + P)             # one fused projection: rows lie apart
    for step in range(3):                                        # the same slots again, smaller and larger values
        x = kv * [1.0, 0.01, 300.0][step]
        run_write(C, x[:, 0], x[:, 1], slots, kc, vc, ks, vs)


def test_write_extremes(C):
    P, Hkv = 16, 2
    kc, ks = empty_cache(8, Hkv, P)
    vc, vs = empty_cache(8, Hkv, P)
    k, v = randn((40, Hkv, 128), 1), randn((40, Hkv, 128), 2)
    k[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 5.0])
    k[1:16, 1] = 0.0                                             # zeros but for one value
    k[17:21] = math.nan                                          # a run of NaN only: no finite value
    k[22:30] *= 1e30                                             # above the largest scale
    v[:16] *= 1e-30                                              # below the smallest
    v[16:21] = math.inf
    v[21:40] = torch.finfo(BF16).max
    slots = i32(list(range(16, 32)) + [0, 1, 2, 3, 4] + list(range(40, 48)) + [-1, 8 * 16, 2 ** 31 - 1, -2 ** 31] +
                list(range(64, 71)))
    run_write(C, k, v, slots, kc, vc, ks, vs)
    run_write(C, v, k, slots, kc, vc, ks, vs)


def test_write_moves_every_code_to_every_scale(C):
    """Codes before the run, all 256 of them, to scales 2^1 .. 2^14 larger."""
    P, shifts = 16, list(range(1, 15)) + [40, 60]
    n = len(shifts)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(8).view(1, 1, 16, 128)
    kc = codes.expand(n, 1, 16, 128).contiguous()
    vc, (_, vs) = kc.clone(), empty_cache(n, 1, P)
    ks = torch.full((n, 1), 2.0 ** -20, device="cuda")
    k = torch.zeros(n, 1, 128, dtype=BF16, device="cuda")
    k[:, 0, 5] = torch.tensor([448.0 * 2.0 ** (s - 20) for s in shifts], dtype=BF16)
    run_write(C, k, k, i32([i * P + 15 for i in range(n)]), kc, vc, ks, vs)


def test_write_nothing(C):
    kc, ks = empty_cache(3, 2, 16)
    k = randn((4, 2, 128), 3)
    run_write(C, k, k, i32([-1] * 4), kc, kc.clone(), ks, ks.clone())
    C.page_write_e4m3(k[:0], k[:0], i32([]), kc, kc, ks, ks)


# --------------------------------------------------------- prompt attention

def run_prompt(C, nq, nk, H, Hkv, window=0, seed=0, scale=SCALE, lead=0, tail=0, edit=None, rows=None):
    """Packed sequences, `lead` and `tail` rows of no sequence; q, k, v are views of one fused projection."""
    Tq, Tk = sum(nq) + lead + tail, sum(nk) + lead + tail
    T = max(Tq, Tk)
    qkv = randn((T, H + 2 * Hkv, 128), 100 + seed)
    q, k, v = qkv[:Tq, :H], qkv[:Tk, H:H + Hkv], qkv[:Tk, H + Hkv:]
    if edit:
        edit(q, k, v)
    cu_q, cu_k = np.concatenate([[0], np.cumsum(nq)]) + lead, np.concatenate([[0], np.cumsum(nk)]) + lead
    out = torch.full((Tq, H, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((Tq, H), 9.0, device="cuda")
    C.prompt_attn(q, k, v, i32(cu_q), i32(cu_k), scale, window, out=out, lse=lse)
    C.sync_status()
    ref = PO.prompt_attention(f64(q), f64(k), f64(v), cu_q, cu_k, scale, window, rows=rows)
    if rows is None:
        none = np.isnan(ref[1][:, 0]) & (np.arange(Tq) >= 0)
        none[lead:Tq - tail if tail else Tq] = False
        assert (f64(out)[none] == 7).all() and (f64(lse)[none] == 9).all()
    check_attention(out, lse, ref, max(nk + [1]), f"nq {nq} nk {nk} H {H}/{Hkv} window {window}")
    return out, lse


@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 2), (3, 1), (8, 2), (16, 2), (10, 2), (7, 1), (12, 1), (48, 8), (64, 8)])
def test_prompt_heads(C, H, Hkv):
    run_prompt(C, [1, 67, 33], [1, 67, 40], H, Hkv, seed=H)


@pytest.mark.parametrize("H,Hkv", [(33, 1), (96, 1), (128, 1), (128, 128)])
def test_prompt_extreme_heads(C, H, Hkv):
    run_prompt(C, [9, 14], [9, 30], H, Hkv, seed=H)


@pytest.mark.parametrize("nq,nk", [([1], [1]), ([1], [129]), ([2], [1000]), ([127], [127]), ([128], [128]), ([129], [129]),
                                   ([255, 1, 257], [255, 1, 257]), ([300], [600]), ([64, 0, 5, 0], [64, 0, 5, 70]),
                                   ([5, 9, 40], [0, 3, 40])])
def test_prompt_lengths(C, nq, nk):
    run_prompt(C, nq, nk, 4, 2, seed=len(nq) + nq[0])


@pytest.mark.parametrize("window", [1, 2, 63, 64, 127, 128, 129, 200, 100000])
def test_prompt_window(C, window):
    run_prompt(C, [290, 40], [290, 170], 8, 2, window=window, seed=window % 97)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 129])
def test_prompt_largest_window(C, window):
    """The difference of a query without a key and the window stays within 32 bits."""
    run_prompt(C, [200, 70, 300, 4], [73, 0, 299, 4], 8, 2, window=window, seed=11)
    run_prompt(C, [150] * 90, [1, 0, 150] * 30, 4, 2, window=window, seed=12)


def test_prompt_rows_of_no_sequence(C):
    run_prompt(C, [40, 3], [40, 60], 8, 2, lead=5, tail=21, seed=3)
    run_prompt(C, [0, 0], [4, 0], 4, 4, tail=130, seed=4)


def test_prompt_many_short_sequences(C):
    r = np.random.RandomState(2)
    nq = r.randint(0, 4, 600).tolist()
    run_prompt(C, nq, [n + int(e) for n, e in zip(nq, r.randint(0, 3, 600))], 4, 1, seed=9)


@pytest.mark.parametrize("grow", [3.0, 40.0])
def test_prompt_scores_that_grow(C, grow):
    """Later keys score far higher (the running reference has to move) or lower."""
    def edit(q, k, v):
        d = torch.linspace(-1, 1, k.shape[0], device="cuda")[:, None, None]
        k.copy_((k + grow * d * torch.sign(k[:1])).to(BF16))
    run_prompt(C, [400], [400], 4, 2, seed=1, edit=edit)
    run_prompt(C, [200, 150], [400, 150], 4, 2, seed=2, edit=lambda q, k, v: (edit(q, k, v), q.mul_(4)), window=90)


def test_prompt_what_is_not_seen_has_no_influence(C):
    """NaN and infinities in keys and values that a row does not see: after the
    causal edge, before the window, in other sequences and behind the last."""
    nq, H, Hkv, w = [150, 90], 8, 2, 40
    clean = {}

    def edit(q, k, v):
        clean.update(q=q.clone(), k=k.clone(), v=v.clone())
        for x, at in ((k, 100), (v, 100), (k, 3), (v, 3), (v, 149)):
            x[at, 0, ::7] = math.nan
            x[at, 1, 1::5] = math.inf
            x[at, 1, 2::5] = -math.inf
        k[240:], v[240:] = math.nan, math.nan

    T = 240 + 30
    qkv = randn((T, H + 2 * Hkv, 128), 55)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    edit(q, k, v)
    cu = np.array([0, 150, 240])
    for window in (0, w):
        out, lse = C.prompt_attn(q, k, v, i32(cu), i32(cu), SCALE, window, lse=True)
        C.sync_status()
        ref = PO.prompt_attention(f64(clean["q"]), f64(clean["k"]), f64(clean["v"]), cu, cu, SCALE, window)
        i = np.arange(240)
        lo = np.maximum(np.where(i < 150, 0, 150), i - (window - 1 if window else 10 ** 6))
        sees = lambda at: (lo <= at) & (at <= i)  # noqa: E731
        touched = sees(100) | sees(3) | sees(149)
        for x in ref:
            x[:240][touched] = np.nan
        assert (~touched).sum() > 90
        check_attention(out, lse, ref, 150, f"window {window}")
        got = f64(out)[:240]
        assert np.isnan(got[sees(100)][:, :, ::7]).any(axis=2).all()       # rows that do see them


def test_prompt_nan_value_of_no_weight_that_is_seen(C):
    """A NaN that a row sees stays NaN where its probability is 0 in fp32, in whole tiles and in those that are masked in part."""
    T = 200
    q, k, v = (torch.zeros(T, 1, 128, dtype=BF16, device="cuda") for _ in range(3))
    q[:, 0, 0], k[:, 0, 0] = 1.0, 1.0
    v[:] = 1.0
    for at in (3, 70, 130):
        k[at, 0, 0] = -1000.0
        v[at, 0, at % 7] = math.nan
    out, lse = C.prompt_attn(q, k, v, i32([0, T]), i32([0, T]), 1.0, lse=True)
    C.sync_status()
    o, sees = f64(out)[:, 0], np.zeros((T, 128), dtype=bool)
    for at in (3, 70, 130):
        sees[at:, at % 7] = True
    assert np.array_equal(np.isnan(o), sees) and np.isfinite(f64(lse)).all()


def test_prompt_infinite_value_is_infinite_where_it_is_seen(C):
    q, k, v = randn((200, 2, 128), 1), randn((200, 1, 128), 2), randn((200, 1, 128), 3)
    v[130, 0, 5], v[131, 0, 9] = math.inf, -math.inf
    cu = i32([0, 200])
    out, _ = C.prompt_attn(q, k, v, cu, cu, SCALE)
    o = f64(out)
    assert np.isfinite(o[:130]).all() and np.isposinf(o[130:, :, 5]).all() and np.isneginf(o[131:, :, 9]).all()
    o[130:, :, 5], o[131:, :, 9] = 0, 0
    assert np.isfinite(o).all()


def test_prompt_masked_by_the_lowest_value(C):
    """Keys whose scores are the lowest finite values next to plain ones, and alone."""
    q, k, v = randn((64, 2, 128), 4), randn((64, 1, 128), 5), randn((64, 1, 128), 6)
    q[:, :, 0], k[:, :, 0] = 1.0, 0.0
    k[::2, :, 0] = torch.finfo(BF16).min
    cu = i32([0, 64])
    out, lse = C.prompt_attn(q, k, v, cu, cu, 1.0, lse=True)
    C.sync_status()
    o, l, a, s = PO.prompt_attention(f64(q), f64(k), f64(v), [0, 64], [0, 64], 1.0)
    got = f64(out)
    assert np.isfinite(got).all() and np.isfinite(f64(lse)).all()
    # row 0 sees only such a key; the later ones ignore them: their scores' products are small
    assert np.abs(got[0] - f64(v)[0]).max() <= U * np.abs(f64(v)[0]).max()
    plain = PO.prompt_attention(f64(q)[1:], f64(k)[1::2], f64(v)[1::2], [0, 63], [0, 32], 1.0)[0]
    for t in (1, 2, 3, 40, 63):
        j = np.arange(1, t + 1, 2)
        ref = PO.attend_rows(f64(q)[t], f64(k)[j, 0], f64(v)[j, 0], 1.0)
        assert (np.abs(got[t] - ref[0]) <= U * np.abs(ref[0]) + (U + 2.0 ** -14) * ref[2]).all()
    assert plain.shape == (63, 2, 128)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("top", [20, 23, 24, 26, 28, 33, 60, 95, 110])
def test_prompt_large_finite_scores(C, top, sign):
    """Scores of up to about 2^top whose products are exact, with ties in different tiles: the largest one or the
    equal largest ones have all the weight, whatever the rounding of a score times log2(e) is."""
    r = np.random.RandomState(top)
    T, H, Hkv = 400, 4, 2
    q, k = torch.zeros(T, H, 128, dtype=BF16, device="cuda"), torch.zeros(T, Hkv, 128, dtype=BF16, device="cuda")
    v = randn((T, Hkv, 128), top)
    a = (top + 3) // 2
    q[:, :, 0] = torch.tensor(sign * 2.0 ** a * (1 + r.randint(0, 128, (T, H)) / 128), dtype=BF16)
    k[:, :, 0] = torch.tensor(2.0 ** (top + 2 - a - r.randint(0, 3, (T, Hkv))) * (1 + r.randint(0, 8, (T, Hkv)) / 8), dtype=BF16)
    cu = [0, 270, 400]
    for window in (0, 90):
        out, lse = C.prompt_attn(q, k, v, i32(cu), i32(cu), 0.125, window, lse=True)
        C.sync_status()
        check_peaked(out, lse, PO.prompt_attention(f64(q), f64(k), f64(v), cu, cu, 0.125, window), f"2^{top}, window {window}")


@pytest.mark.parametrize("top", [26, 33, 36, 60, 95])
def test_prompt_large_finite_scores_alike_in_a_tile(C, top):
    """As above with one query for all rows of a sequence, so that no other row has a warp compute its scores anew."""
    r = np.random.RandomState(top)
    B, n, H = 40, 64, 2
    q, k = torch.zeros(B * n, H, 128, dtype=BF16, device="cuda"), torch.zeros(B * n, 1, 128, dtype=BF16, device="cuda")
    v = randn((B * n, 1, 128), top)
    a = (top + 3) // 2
    head = np.where(np.arange(B) % 2, -1.0, 1.0) * 2.0 ** a * (1 + r.randint(0, 128, B) / 128)
    q[:, :, 0] = torch.tensor(np.repeat(head, n)[:, None], dtype=BF16)
    k[:, 0, 0] = torch.tensor(2.0 ** (top + 2 - a) * (1 + r.randint(0, 8, B * n) / 8), dtype=BF16)
    cu = list(range(0, B * n + 1, n))
    out, lse = C.prompt_attn(q, k, v, i32(cu), i32(cu), 0.125, lse=True)
    C.sync_status()
    check_peaked(out, lse, PO.prompt_attention(f64(q), f64(k), f64(v), cu, cu, 0.125), f"2^{top}")


def test_prompt_long_rows_sampled(C):
    rows = {0, 1, 500, 4000, 5200, 5201, 5202, 9000, 9300, 9301}
    run_prompt(C, [5201, 4101], [5201, 4101], 8, 1, seed=77, rows=rows)


# --------------------------------------------------------- decode attention

def make_cache(n_pages, Hkv, P, seed, spread=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (n_pages, Hkv, P, 128)
    codes = [(torch.randn(shape, device="cuda", generator=g) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
             .view(torch.uint8) for _ in range(2)]
    scales = [torch.ldexp(torch.ones(n_pages, Hkv, device="cuda"),
                          torch.randint(-8 - spread, -5, (n_pages, Hkv), device="cuda", generator=g)) for _ in range(2)]
    return codes + scales


def run_decode(C, lens, H, Hkv, P, window=0, seed=0, q_std=1.0, spread=3, cache=None, bad=(), width=None):
    r = np.random.RandomState(seed + 7 * H + P)
    pages = [-(-max(n, 0) // P) for n in lens]
    n_pages = sum(pages) + 3
    cache = make_cache(n_pages, Hkv, P, seed + 200, spread) if cache is None else cache
    pool = r.permutation(n_pages)
    width = max(pages + [1]) + 1 if width is None else width
    table, at = np.full((len(lens), width), n_pages + 99), 0
    for b, m in enumerate(pages):
        table[b, :min(m, width)] = pool[at:at + min(m, width)]
        at += m
    for b, j, p in bad:
        table[b, j] = p
    q = randn((len(lens), H + 2, 128), seed, q_std)[:, :H]
    out, lse = C.page_decode_attn(q, *cache, i32(table), i32(lens), SCALE, window, lse=True)
    C.sync_status()
    kc, vc, ks, vs = (x.cpu().numpy() for x in cache)
    ref = PO.page_decode_attention(f64(q), kc, vc, ks.astype(np.float64), vs.astype(np.float64), table, lens, SCALE, window)
    check_attention(out, lse, ref, max(lens), f"lens {lens} H {H}/{Hkv} P {P} window {window}")
    return out, lse


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", [[1], [0], [17, 0, 1, 300], [127, 128, 129, 255, 256, 257], [1500]])
def test_decode_lengths(C, P, lens):
    run_decode(C, lens, 8, 2, P, seed=len(lens))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (5, 1), (8, 1), (9, 1), (16, 1), (12, 2), (17, 1), (64, 8), (32, 1),
                                   (40, 1), (128, 2), (128, 1), (128, 128)])
def test_decode_heads(C, H, Hkv):
    run_decode(C, [70, 5, 333], H, Hkv, 64, seed=H)


@pytest.mark.parametrize("window", [1, 15, 64, 100, 129, 5000])
@pytest.mark.parametrize("P", [16, 128])
def test_decode_window(C, window, P):
    run_decode(C, [3, 200, 777, 130], 8, 2, P, window=window, seed=window)


@pytest.mark.parametrize("B,H,Hkv,P,window", [(36, 8, 4, 64, 0), (36, 8, 4, 16, 130), (37, 16, 8, 32, 1), (38, 16, 8, 32, 700),
                                              (33, 64, 4, 128, 1153), (33, 64, 4, 128, 1154), (3, 40, 1, 64, 300),
                                              (296, 3, 1, 16, 0), (297, 3, 1, 16, 0)])
def test_decode_short_units(C, B, H, Hkv, P, window):
    """Around the sizes where a unit is one CTA's: lengths of 0, 1, the table's and around the window's."""
    r = np.random.RandomState(B + window)
    most = 1200 if window == 0 and B < 100 else 3000 if window else 300
    lens = r.randint(0, most + 1, B)
    lens[:3] = [0, most, 1]
    if window and B > 8:
        lens[3:7] = [window - 1, window, window + 1, window + 127]
    run_decode(C, [int(n) for n in lens], H, Hkv, P, window=window, seed=B)


def test_decode_many_sequences(C):
    r = np.random.RandomState(4)
    run_decode(C, r.randint(0, 90, 400).tolist(), 4, 1, 16, seed=2)


def test_decode_long_context(C):
    run_decode(C, [20001, 3, 9000], 4, 2, 64, seed=5)


@pytest.mark.parametrize("q_std", [0.0, 0.01, 8.0, 60.0])
def test_decode_flat_and_peaked(C, q_std):
    run_decode(C, [900, 40], 8, 2, 32, seed=6, q_std=q_std)


@pytest.mark.parametrize("wide", [2.0 ** 12, 2.0 ** 16])
def test_decode_query_with_a_wide_channel(C, wide):
    """Components of q from 2^-13 of the row's largest on are exact, the others off by at most 2^-21 of it: seen
    where the keys are 0 in the wide channel."""
    n, P = 500, 64
    cache = make_cache(8, 2, P, 31)
    cache[0][..., 0] = 0
    q = randn((1, 8, 128), 32)
    q = torch.sign(q) * (1 + q.abs().clamp(max=0.99)).to(BF16)
    q[..., 0] = wide
    table = np.arange(8)[None]
    out, lse = C.page_decode_attn(q, *cache, i32(table), i32([n]), SCALE, lse=True)
    C.sync_status()
    kc, vc, ks, vs = (x.cpu().numpy() for x in cache)
    ref = list(PO.page_decode_attention(f64(q), kc, vc, ks.astype(float), vs.astype(float), table, [n], SCALE))
    if wide > 2.0 ** 13:                                       # as if the sum of |q||k| were larger by that error
        most = np.abs(e4m3_decode(kc) * ks[..., None, None].astype(float)).sum(-1).max()
        ref[3] = ref[3] + SCALE * 2.0 ** -21 * wide * most / (130 * 2.0 ** -24)
    check_attention(out, lse, tuple(ref), n)


@pytest.mark.parametrize("H,P", [(8, 16), (8, 64), (16, 64)])
@pytest.mark.parametrize("top", [24, 26, 27, 28, 29, 33, 60, 95])
def test_decode_large_finite_scores(C, top, H, P):
    """Base-2 scores around +-2^top (from 2^27 on 8 is no whole step of fp32's): equal largest ones share all the weight."""
    r = np.random.RandomState(top + H)
    lens = [700, 40, 1, 3000] * 3
    pages = [-(-n // P) for n in lens]
    kc, vc, ks, vs = make_cache(sum(pages), 1, P, top)
    vs[:] = 2.0 ** -7
    ks[:] = 2.0 ** -7
    levels = torch.tensor([1, 1.125, 1.25, 1.5, 2], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    kc[:, 0, :, 0] = levels[torch.tensor(r.randint(0, 5, (sum(pages), P)), device="cuda")]
    table, at = np.zeros((len(lens), max(pages)), dtype=np.int64), 0
    for b, m in enumerate(pages):
        table[b, :m] = at + r.permutation(m)
        at += m
    q = torch.zeros(len(lens), H, 128, dtype=BF16, device="cuda")
    sign = np.where(np.arange(H) % 2, -1.0, 1.0)
    q[:, :, 0] = torch.tensor(sign * 2.0 ** (top + 7 + 2) * (1 + r.randint(0, 128, (len(lens), H)) / 128), dtype=BF16)
    out, lse = C.page_decode_attn(q, kc, vc, ks, vs, i32(table), i32(lens), 0.125, lse=True)
    C.sync_status()
    ref = PO.page_decode_attention(f64(q), kc.cpu().numpy(), vc.cpu().numpy(), f64(ks), f64(vs), table, lens, 0.125)
    check_peaked(out, lse, ref, f"2^{top}")


def test_decode_scales_far_apart(C):
    """Pages whose scales differ by up to 2^30: neither values nor weights get lost."""
    run_decode(C, [700, 129], 8, 2, 16, seed=8, spread=30)


def test_scales_are_read_as_their_power_of_two(C):
    """Of a scale that is no power of two the largest one below it counts, for keys and for values, read and written."""
    cache, q = make_cache(9, 2, 16, 3), randn((2, 8, 128), 4)
    table, n = i32([[0, 3, 5, 7], [1, 2, 4, 8]]), i32([60, 33])
    want = C.page_decode_attn(q, *cache, table, n, SCALE, lse=True)
    for x in (1.25, 1.9999):
        for i in (2, 3):
            odd = list(cache)
            odd[i] = cache[i] * x
            got = C.page_decode_attn(q, *odd, table, n, SCALE, lse=True)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (i, x)
    kv, slots = randn((3, 2, 128), 5) * 100, i32([16 + 13, 16 + 14, 16 + 15])
    plain = [x.clone() for x in cache]
    C.page_write_e4m3(kv, kv, slots, *plain)
    odd = [x.clone() for x in cache]
    odd[2], odd[3] = cache[2] * 1.25, cache[3] * 1.9999
    C.page_write_e4m3(kv, kv, slots, *odd)
    C.sync_status()
    assert torch.equal(plain[0], odd[0]) and torch.equal(plain[1], odd[1])
    assert torch.equal(plain[2][1], odd[2][1]) and torch.equal(plain[3][1], odd[3][1])
    # out of the range: held to it, in all three
    far = [x.clone() for x in cache]
    for x, e in ((0.0, -40), (2.0 ** -41, -40), (2.0 ** 100, 60)):
        far[2][:], far[3][:] = x, x
        held = [far[0], far[1], torch.full_like(far[2], 2.0 ** e), torch.full_like(far[3], 2.0 ** e)]
        for a, b in zip(C.page_decode_attn(q, *far, table, n, SCALE, lse=True), C.page_decode_attn(q, *held, table, n, SCALE, lse=True)):
            assert torch.equal(a, b), x
        w = [[y.clone() for y in c] for c in (far, held)]
        for c in w:
            C.page_write_e4m3(kv, kv, slots, *c)
        assert all(torch.equal(a, b) for a, b in zip(w[0][:2], w[1][:2])) and torch.equal(w[0][2][1], w[1][2][1]), x
    C.sync_status()


def test_decode_pages_that_do_not_exist(C):
    run_decode(C, [100, 200, 50], 8, 2, 16, seed=9, bad=[(0, 2, -1), (1, 0, 10 ** 6), (1, 11, -2 ** 31), (2, 0, -1), (2, 1, -1),
                                                         (2, 2, -1), (2, 3, 2 ** 31 - 1)])
    run_decode(C, [1000, 40], 8, 2, 16, seed=10, width=5)               # longer than its table
    run_decode(C, [-5, 40], 8, 2, 16, seed=11)


def test_decode_stale_pages_have_no_influence(C):
    """NaN codes behind a sequence's end, before its window and in pages of nobody."""
    P, lens = 64, [70, 129, 64, 1]
    cache = make_cache(12, 2, P, 77)
    table = np.array([[3, 0, 11], [5, 6, 2], [1, 11, 11], [8, 11, 11]])
    q = randn((4, 8, 128), 5)
    for window in (0, 40):
        kc, vc, ks, vs = (x.clone() for x in cache)
        ref = PO.page_decode_attention(f64(q), kc.cpu().numpy(), vc.cpu().numpy(), f64(ks), f64(vs), table, lens, SCALE, window)
        for b, n in enumerate(lens):
            lo = max(0, n - window) if window else 0
            for x in list(range(0, lo)) + list(range(n, 3 * P)):
                p = table[b, x // P]
                if p != 11:
                    kc[p, :, x % P], vc[p, :, x % P] = 0x7F, 0xFF
        for p in (4, 7, 9, 10, 11):
            kc[p], vc[p] = 0x7F, 0x7F
            ks[p], vs[p] = math.nan, math.inf
        out, lse = C.page_decode_attn(q, kc, vc, ks, vs, i32(table), i32(lens), SCALE, window, lse=True)
        C.sync_status()
        check_attention(out, lse, ref, 129, f"window {window}")


def test_decode_nan_code_that_is_seen(C):
    cache = make_cache(4, 1, 64, 3)
    cache[1][2, 0, 10, 5] = 0x7F
    out, _ = C.page_decode_attn(randn((2, 4, 128), 1), *cache, i32([[2, 1], [3, 1]]), i32([100, 100]), SCALE)
    o = f64(out)
    assert np.isnan(o[0, :, 5]).all() and np.isfinite(np.delete(o[0], 5, axis=1)).all() and np.isfinite(o[1]).all()


# --------------------------------------------------------------- a run of them

def test_serving_run(C):
    """Prompts of different lengths are planned, written and attended to, then
    decoded for 40 steps; one step is captured and replayed. Every output equals
    the oracle's on the cache's own content, and the cache equals the oracle's."""
    P, H, Hkv, B, n_pages, width = 16, 8, 2, 3, 40, 12
    lens = [37, 1, 90]
    cache = [torch.zeros(n_pages, Hkv, P, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.zeros(n_pages, Hkv, device="cuda") for _ in range(2)]
    table = i32(np.full((B, width), -1))
    free = i32(np.random.RandomState(1).permutation(n_pages))
    T = sum(lens)
    q, k, v = randn((T, H, 128), 1), randn((T, Hkv, 128), 2), randn((T, Hkv, 128), 3)
    slots, cu, n, st = C.page_plan(i32([0] * B), i32(lens), free, table, P, n_pages, max_tokens=T)
    C.page_write_e4m3(k, v, slots, *cache)
    out, lse = C.prompt_attn(q, k, v, cu, cu, SCALE, lse=True)
    check_attention(out, lse, PO.prompt_attention(f64(q), f64(k), f64(v), cu.tolist(), cu.tolist(), SCALE), max(lens))
    used = st.tolist()[0]
    assert st.tolist()[1] == 0 and n.tolist() == lens

    def np_cache():
        return [x.cpu().numpy().astype(x.cpu().numpy().dtype if x.dtype == torch.uint8 else np.float64) for x in cache]

    one = i32([1] * B)
    free_now = torch.zeros(B, dtype=I32, device="cuda")
    held = n.clone()
    q1, k1, v1 = randn((B, H, 128), 4), randn((B, Hkv, 128), 5), randn((B, Hkv, 128), 6)
    bufs = dict(slots=torch.empty(B, dtype=I32, device="cuda"), cu=torch.empty(B + 1, dtype=I32, device="cuda"),
                seq_len=torch.empty(B, dtype=I32, device="cuda"), status=torch.empty(2, dtype=I32, device="cuda"))
    o1, l1 = torch.empty_like(q1), torch.empty(B, H, device="cuda")
    ws = torch.empty(max(16, C.page_decode_workspace_bytes(B, H, Hkv)), dtype=torch.uint8, device="cuda")

    def step():
        C.page_plan(held, one, free_now, table, P, n_pages, **bufs)
        C.page_write_e4m3(k1, v1, bufs["slots"], *cache)
        C.page_decode_attn(q1, *cache, table, bufs["seq_len"], SCALE, out=o1, lse=l1, ws=ws)

    graph = None
    for i in range(40):
        free_now.copy_(free[used:used + B])
        q1.copy_(randn((B, H, 128), 100 + i))
        k1.copy_(randn((B, Hkv, 128), 200 + i) * (1 + i // 8))
        v1.copy_(randn((B, Hkv, 128), 300 + i) * (1 + i // 8))
        before = np_cache()
        if i < 3:
            step()
        else:
            if graph is None:
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        after, sl = np_cache(), bufs["slots"].cpu().numpy()
        for x, c in ((k1, 0), (v1, 1)):
            codes, scale = PO.page_write(f64(x), sl, before[c], before[2 + c])
            assert np.array_equal(codes, after[c]) and np.array_equal(scale, after[2 + c]), i
        ref = PO.page_decode_attention(f64(q1), after[0], after[1], after[2], after[3], table.cpu().numpy(),
                                       bufs["seq_len"].tolist(), SCALE)
        check_attention(o1, l1, ref, 200, f"step {i}")
        assert bufs["status"].tolist()[1] == 0
        used += bufs["status"].tolist()[0]
        held.copy_(bufs["seq_len"])
    C.sync_status()


@pytest.mark.parametrize("nd,prompts", [(5, [40, 1, 133]), (0, [17]), (3, [])])
@pytest.mark.parametrize("window", [0, 30])
def test_step_of_running_requests_and_prompts(C, nd, prompts, window):
    """One plan and one write for requests of both kinds, running ones first; then each kind's attention into its
    rows of one output."""
    P, H, Hkv = 16, 8, 2
    old = [3, 16, 77, 31, 1][:nd] + [0] * len(prompts)
    new = [1] * nd + prompts
    B, n_pages = len(new), 40
    pages = [-(-n // P) for n in old]
    pool = np.random.RandomState(nd).permutation(n_pages)
    table, at = np.full((B, 12), -1), 0
    for b, m in enumerate(pages):
        table[b, :m] = pool[at:at + m]
        at += m
    cache = make_cache(n_pages, Hkv, P, nd + 1)
    T = sum(new)
    q, k, v = randn((T, H, 128), 1), randn((T, Hkv, 128), 2), randn((T, Hkv, 128), 3)
    table = i32(table)
    slots, cu, seq_len, status = C.page_plan(i32(old), i32(new), i32(pool[at:]), table, page=P, n_pages=n_pages, max_tokens=T)
    C.page_write_e4m3(k, v, slots, *cache)
    out, lse = torch.empty_like(q), torch.empty(T, H, device="cuda")
    C.page_decode_attn(q[:nd], *cache, table[:nd], seq_len[:nd], SCALE, window, out=out[:nd], lse=lse[:nd])
    C.prompt_attn(q, k, v, cu[nd:], cu[nd:], SCALE, window, out=out, lse=lse)
    C.sync_status()
    assert status.tolist()[1] == 0
    c = cu.tolist()[nd:]
    ref = [x.copy() for x in PO.prompt_attention(f64(q), f64(k), f64(v), c, c, SCALE, window)]
    kc, vc, ks, vs = (x.cpu().numpy() for x in cache)
    dec = PO.page_decode_attention(f64(q)[:nd], kc, vc, ks.astype(float), vs.astype(float), table.cpu().numpy()[:nd],
                                   seq_len.tolist()[:nd], SCALE, window)
    for x, y in zip(ref, dec):
        x[:nd] = y
    assert not np.isnan(ref[1]).any()
    check_attention(out, lse, tuple(ref), 200)


def test_calls_on_other_streams_and_repeated(C):
    """Two streams at once, each call twice: the same bits."""
    T, H, Hkv = 700, 8, 2
    q, k, v = randn((T, H, 128), 1), randn((T, Hkv, 128), 2), randn((T, Hkv, 128), 3)
    cu = i32([0, 123, 700])
    cache = make_cache(60, Hkv, 64, 4)
    table, n = i32(np.random.RandomState(1).randint(0, 60, (9, 30))), i32([1900, 5, 0, 64, 65, 700, 1, 1920, 333])
    want = C.prompt_attn(q, k, v, cu, cu, SCALE, lse=True), C.page_decode_attn(q[:9], *cache, table, n, SCALE, lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(6):
        for s in streams:
            got.append((C.prompt_attn(q, k, v, cu, cu, SCALE, lse=True, stream=s),
                        C.page_decode_attn(q[:9], *cache, table, n, SCALE, lse=True, stream=s)))
    torch.cuda.synchronize()
    C.sync_status()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------- calls that the above do not make

def test_prompt_captured_with_its_schedule(C):
    """More items than SMs (a schedule in the workspace), captured and replayed with
    other lengths and rows."""
    B, H, Hkv, T = 40, 16, 4, 2600
    q, k, v = randn((T, H, 128), 1), randn((T, Hkv, 128), 2), randn((T, Hkv, 128), 3)
    cu, out, lse = i32(np.zeros(B + 1)), torch.zeros(T, H, 128, dtype=BF16, device="cuda"), torch.zeros(T, H, device="cuda")
    ws = torch.empty(C.prompt_attn_workspace_bytes(B, T, H, Hkv), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        C.prompt_attn(q, k, v, cu, cu, SCALE, 70, out=out, lse=lse, ws=ws)
    r = np.random.RandomState(3)
    for i in range(3):
        n = r.multinomial(T - 100 * i, np.ones(B) / B)
        c = np.concatenate([[0], np.cumsum(n)])
        cu.copy_(i32(c))
        for x in (q, k, v):
            x.copy_(randn(x.shape, 50 + i))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        C.sync_status()
        rows = set(r.randint(0, c[-1], 60).tolist())
        check_attention(out, lse, PO.prompt_attention(f64(q), f64(k), f64(v), c, c, SCALE, 70, rows=rows), 200, f"replay {i}")
        assert (f64(out)[c[-1]:] == 7).all()


def test_prompt_two_graphs_and_an_eager_call_at_once(C):
    """Each with a workspace of its own, on three streams."""
    T, H, Hkv = 1500, 16, 4
    cu = i32([0, 700, 1500])
    x = [[randn((T, n, 128), 10 * g + i) for i, n in enumerate((H, Hkv, Hkv))] for g in range(3)]
    want = [C.prompt_attn(*y, cu, cu, SCALE, lse=True) for y in x]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for g in range(2):
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            outs.append(C.prompt_attn(*x[g], cu, cu, SCALE, lse=True))
        graphs.append((graph, side))
    for _ in range(4):
        for graph, side in graphs:
            with torch.cuda.stream(side):
                graph.replay()
        got = C.prompt_attn(*x[2], cu, cu, SCALE, lse=True)
        torch.cuda.synchronize()
        for a, b in zip(outs + [got], want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    C.sync_status()


def test_prompt_many_empty_sequences_few_tokens(C):
    """8192 sequences, 60 of them with tokens; and lengths beyond the tensors, which are cut."""
    r = np.random.RandomState(5)
    n = np.zeros(8192, dtype=np.int64)
    n[r.choice(8192, 60, replace=False)] = 1
    c = np.concatenate([[0], np.cumsum(n)])
    q, k, v = randn((60, 4, 128), 1), randn((60, 2, 128), 2), randn((60, 2, 128), 3)
    out, lse = C.prompt_attn(q, k, v, i32(c), i32(c), SCALE, lse=True)
    C.sync_status()
    check_attention(out, lse, PO.prompt_attention(f64(q), f64(k), f64(v), c, c, SCALE), 1)
    out, lse = C.prompt_attn(q, k, v, i32([-5, 30, 999]), i32([-7, 30, 2 ** 31 - 1]), SCALE, lse=True)
    C.sync_status()
    check_attention(out, lse, PO.prompt_attention(f64(q), f64(k), f64(v), [0, 30, 60], [0, 30, 60], SCALE), 30)


def test_prompt_without_keys(C):
    q, k = randn((70, 4, 128), 1), randn((0, 2, 128), 2)
    out, lse = C.prompt_attn(q, k, k, i32([0, 30, 70]), i32([0, 0, 0]), SCALE, lse=True)
    C.sync_status()
    assert (f64(out) == 0).all() and np.isneginf(f64(lse)).all()


def test_prompt_all_values_not_finite(C):
    q, k, v = randn((300, 4, 128), 1), randn((300, 2, 128), 2), randn((300, 2, 128), 3)
    v[:] = math.nan
    out, lse = C.prompt_attn(q, k, v, i32([0, 300]), i32([0, 300]), SCALE, lse=True)
    C.sync_status()
    assert np.isnan(f64(out)).all() and np.isfinite(f64(lse)).all()
    k[::3] = math.nan
    out, lse = C.prompt_attn(q, k, v, i32([0, 300]), i32([0, 300]), SCALE, lse=True)
    C.sync_status()
    assert np.isnan(f64(out)).all() and np.isnan(f64(lse)).all()
    q[5] = math.inf
    C.prompt_attn(q, k.zero_(), v.fill_(1), i32([0, 300]), i32([0, 300]), SCALE)
    C.sync_status()


def test_decode_query_not_finite(C):
    """A head of q that is not finite has no finite output, the others are untouched."""
    cache = make_cache(30, 2, 64, 4)
    q = randn((3, 8, 128), 9)
    table, n = i32(np.random.RandomState(1).randint(0, 30, (3, 9))), i32([500, 64, 1])
    want, _ = C.page_decode_attn(q, *cache, table, n, SCALE)
    q2 = q.clone()
    q2[0, 3, 7], q2[2, 0, 0] = math.inf, math.nan
    got, lse = C.page_decode_attn(q2, *cache, table, n, SCALE, lse=True)
    C.sync_status()
    a, b = f64(got), f64(want)
    assert np.isnan(a[0, 3]).all() and np.isnan(a[2, 0]).all() and np.isnan(f64(lse)[0, 3])
    a[0, 3], a[2, 0] = b[0, 3], b[2, 0]
    assert np.array_equal(a, b)


def test_decode_small_and_large_queries(C):
    """Rows of q from the type's smallest to 1e30 (the parts of q are relative to the row)."""
    for std in (1e-38, 1e-30, 1e6):
        run_decode(C, [300, 77], 8, 2, 64, seed=3, q_std=std)


def test_decode_empty_cache_and_no_table(C):
    cache = [x[:0].contiguous() for x in make_cache(1, 2, 16, 1)]
    q = randn((3, 4, 128), 1)
    for table in (i32(np.zeros((3, 4))), i32(np.zeros((3, 0)))):
        out, lse = C.page_decode_attn(q, *cache, table, i32([50, 0, 3]), SCALE, lse=True)
        C.sync_status()
        assert (f64(out) == 0).all() and np.isneginf(f64(lse)).all()


def test_decode_shared_pages(C):
    """A common prefix: sequences that hold the same pages."""
    P = 32
    cache = make_cache(20, 2, P, 6)
    r = np.random.RandomState(2)
    table = np.concatenate([np.tile(r.permutation(8), (5, 1)), 8 + r.randint(0, 12, (5, 4))], axis=1)
    lens = [300, 256, 257, 384, 100]
    q = randn((5, 6, 128), 2)
    out, lse = C.page_decode_attn(q, *cache, i32(table), i32(lens), SCALE, lse=True)
    C.sync_status()
    kc, vc, ks, vs = (x.cpu().numpy() for x in cache)
    ref = PO.page_decode_attention(f64(q), kc, vc, ks.astype(float), vs.astype(float), table, lens, SCALE)
    check_attention(out, lse, ref, 384)


def test_write_rows_far_apart(C):
    """Keys and values that are views with a row stride of their own, and misaligned ones refused."""
    kc, ks = empty_cache(6, 2, 16)
    vc, vs = empty_cache(6, 2, 16)
    big = randn((50, 9, 128), 4)
    run_write(C, big[:, 1:3], big[:, 6:8], i32(range(20, 70)), kc, vc, ks, vs)
    bad = randn((50, 9 * 128 + 4), 4)[:, 4:4 + 256].unflatten(1, (2, 128))
    with pytest.raises(C.CslcError, match="multiple of 8"):
        C.page_write_e4m3(bad, bad, i32(range(20, 70)), kc, vc, ks, vs)
    with pytest.raises(ValueError, match="dense within a row"):
        C.page_write_e4m3(big[:, 1:5:2], big[:, 1:3], i32(range(20, 70)), kc, vc, ks, vs)


@pytest.mark.parametrize("P,Hkv", [(128, 8), (16, 5)])
def test_cache_beyond_32_bits(C, P, Hkv):
    """Pages whose codes lie more than 2^32 bytes into the cache: written, and read by the decode attention."""
    n_pages = (2 ** 32 + 2 ** 30) // (Hkv * P * 128)
    first, last = [0, 5, 2], [n_pages - 1, n_pages - 70, n_pages * 7 // 8, n_pages // 2 + 1]
    pages = last + first                                       # the sequence's pages, in order
    kc, vc = (torch.empty((n_pages, Hkv, P, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((n_pages, Hkv), device="cuda") for _ in range(2))
    at = i32(pages).long()
    for c in (kc, vc):
        c[at] = 0x7F
    for c in (ks, vs):
        c[at] = 2.0 ** -9
    n = len(pages) * P - 5
    k, v = randn((n, Hkv, 128), 21), randn((n, Hkv, 128), 22)
    small = [c[at].cpu().numpy() for c in (kc, vc)]
    C.page_write_e4m3(k, v, i32([pages[x // P] * P + x % P for x in range(n)]), kc, vc, ks, vs)
    C.sync_status()
    near = []
    for x, c, sc, (cache, scale) in ((k, small[0], ks, (kc, ks)), (v, small[1], vs, (vc, vs))):
        codes, ref = PO.page_write(f64(x), np.arange(n), c, np.full((len(pages), Hkv), 2.0 ** -9))
        assert np.array_equal(cache[at].cpu().numpy(), codes) and np.array_equal(f64(scale[at]), ref)
        near.append((codes, ref))
    lens = [n, 2 * P + 3]
    q = randn((2, 2 * Hkv, 128), 23)
    out, lse = C.page_decode_attn(q, kc, vc, ks, vs, i32([pages, pages]), i32(lens), SCALE, lse=True)
    C.sync_status()
    table = np.tile(np.arange(len(pages)), (2, 1))
    check_attention(out, lse, PO.page_decode_attention(f64(q), near[0][0], near[1][0], near[0][1], near[1][1], table, lens, SCALE),
                    n, "far pages")


def test_prompt_rows_beyond_32_bits(C):
    """Rows of q, k and v that lie up to 5 GB apart."""
    T, H, Hkv = 600, 4, 2
    big = torch.empty((T, 2 ** 22), dtype=BF16, device="cuda")
    q, k, v = (big[:, c * 2 ** 20:c * 2 ** 20 + h * 128].unflatten(1, (h, 128)) for c, h in ((0, H), (1, Hkv), (3, Hkv)))
    for i, x in enumerate((q, k, v)):
        x.copy_(randn(x.shape, 30 + i))
    cu = [0, 170, T]
    out, lse = C.prompt_attn(q, k, v, i32(cu), i32(cu), SCALE, lse=True)
    C.sync_status()
    check_attention(out, lse, PO.prompt_attention(f64(q), f64(k), f64(v), cu, cu, SCALE), 430, "far rows")


def test_binding_refusals_on_the_device(C):
    q, k = randn((4, 8, 128), 1), randn((4, 2, 128), 2)
    cu = i32([0, 4])
    with pytest.raises(ValueError, match="expected"):
        C.prompt_attn(q, k, k[:3], cu, cu, SCALE)
    with pytest.raises(C.CslcError, match="scale"):
        C.prompt_attn(q, k, k, cu, cu, 0.0)
    with pytest.raises(C.CslcError, match="scale"):
        C.prompt_attn(q, k, k, cu, cu, math.nan)
    with pytest.raises(TypeError, match="int32"):
        C.prompt_attn(q, k, k, cu.long(), cu, SCALE)
    cache = make_cache(3, 2, 16, 1)
    with pytest.raises(C.CslcError, match="multiple of H_kv"):
        C.page_decode_attn(q[:, :7], *cache, i32(np.zeros((4, 2))), i32([1] * 4), SCALE)
    with pytest.raises(C.CslcError, match="page size"):
        C.page_decode_attn(q, *[x[:, :, :8].contiguous() if x.dim() == 4 else x for x in cache], i32(np.zeros((4, 2))),
                           i32([1] * 4), SCALE)
    with pytest.raises(ValueError, match="max_tokens"):
        C.page_plan(cu, cu, cu, i32(np.zeros((2, 2))), 16, 4)


def test_plans_one_after_another_from_what_is_left(C):
    """The caller takes status[0] pages off the front of its list, whatever their number; other lists as slices, too."""
    page, n_pages, lists = 16, 40, i32([9] + [20, 0, 5, 3, 9] + [7])
    pool = np.random.RandomState(3).permutation(n_pages)
    free, at = i32(pool), 0
    for new, taken in (([3, 16, 0, 13, 0], 1), ([13, 0, 12, 0, 0], 2), ([29, 0, 12, 0, 0], 3), ([1, 1, 1, 1, 1], 1), ([30] * 5, 10)):
        old = lists[1:6]
        table = np.full((5, 9), -1)
        for b, m in enumerate((2, 0, 1, 1, 1)):
            table[b, :m] = 30 + b
        got = C.page_plan(old, i32([0] + new)[1:], free[at:], i32(table), page, n_pages, max_tokens=200)
        ref = PO.page_plan(old.tolist(), new, pool[at:], table, page, n_pages, 200)
        for g, r in zip(got, ref[1:]):
            assert np.array_equal(g.cpu().numpy(), r)
        assert int(got[3][0]) == taken
        at += taken


def test_lists_that_are_slices(C):
    q, k, v = randn((90, 4, 128), 1), randn((90, 2, 128), 2), randn((90, 2, 128), 3)
    cu = i32([0, 3, 4, 50, 90])
    for i in (1, 2, 3):
        out, lse = torch.full_like(q, 7.0), torch.full((90, 4), 9.0, device="cuda")
        C.prompt_attn(q, k, v, cu[i:], cu[i:], SCALE, out=out, lse=lse)
        C.sync_status()
        c = cu.tolist()[i:]
        check_attention(out, lse, PO.prompt_attention(f64(q), f64(k), f64(v), c, c, SCALE), 50)
        assert (f64(out)[:c[0]] == 7).all() and (f64(lse)[:c[0]] == 9).all()
    kc, ks = empty_cache(6, 2, 16)
    vc, vs = empty_cache(6, 2, 16)
    slots = i32(range(17, 17 + 70))
    run_write(C, k[:61], v[:61], slots[3:64], kc, vc, ks, vs)
