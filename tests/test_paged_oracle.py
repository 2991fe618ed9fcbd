"""Pins of the paged oracle (CPU only) and refusals of the paged entry points
(every call below fails validation, or has nothing to do, before any CUDA work)."""

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from oracle.cslc_oracle import e4m3_decode
from compressed_sparse_long_compress_b200 import cslc


def test_scale_exponent_is_the_smallest_that_holds():
    for amax in [0.0, 2.0 ** -45, 1e-12, 0.4375, 0.44, 1.0, 448.0, 450.0, 3.5, 3.5156, 1e20, 1e30]:
        e = PO.scale_exponent(amax)
        assert -40 <= e <= 60
        assert amax <= 448 * 2.0 ** e or e == 60
        assert e == -40 or amax > 448 * 2.0 ** (e - 1)


def test_encode_is_torchs_cast_and_saturates():
    x = torch.randn(4096, generator=torch.Generator().manual_seed(3)) * 100
    x = x.clamp(-448, 448)
    assert np.array_equal(PO.encode(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    got = e4m3_decode(PO.encode(np.array([np.inf, -np.inf, 500.0, -1e9, np.nan])))
    assert np.array_equal(got[:4], [448, -448, 448, -448]) and np.isnan(got[4])


def test_plan_by_hand():
    # page 16: request 0 holds 20 tokens (2 pages) and gets 13 (1 more page), request 1 is new with 5, request 2 idle
    table = np.array([[7, 3, -1, 9], [-1, -1, -1, -1], [5, -1, -1, -1]])
    t, slots, cu, n, st = PO.page_plan([20, 0, 16], [13, 5, 0], [11, 2], table, 16, 20, 20)
    assert t.tolist() == [[7, 3, 11, 9], [2, -1, -1, -1], [5, -1, -1, -1]]
    assert slots.tolist() == [3 * 16 + x for x in range(4, 16)] + [11 * 16] + [32, 33, 34, 35, 36] + [-1, -1]
    assert cu.tolist() == [0, 13, 18, 18] and n.tolist() == [33, 5, 16] and st.tolist() == [2, 0]
    # one page too few: the last request's tokens have none
    t, slots, _, _, st = PO.page_plan([20, 0, 16], [13, 5, 0], [11], table, 16, 20, 18)
    assert t[1, 0] == -1 and slots[13:].tolist() == [-1] * 5 and st.tolist() == [2, 5]


def test_write_by_hand():
    cache, scale = np.zeros((2, 1, 16, 128), dtype=np.uint8), np.ones((2, 1))
    x = np.zeros((3, 1, 128))
    x[:, 0, 0] = [1.0, 3.5, 7.0]
    c, s = PO.page_write(x[:1], [16], cache, scale)           # page 1 is new: 1 <= 448 * 2^-8
    assert s[1, 0] == 2.0 ** -8 and s[0, 0] == 1 and e4m3_decode(c[1, 0, 0, 0]) == 256
    c, s = PO.page_write(x[1:], [17, 18], c, s)               # 7 needs 2^-6: the first code moves
    assert s[1, 0] == 2.0 ** -6 and e4m3_decode(c[1, 0, :3, 0]).tolist() == [64, 224, 448]
    c2, s2 = PO.page_write(x[:1], [19], c, s)                 # a smaller token keeps the scale
    assert s2[1, 0] == 2.0 ** -6 and np.array_equal(c2[1, 0, :3], c[1, 0, :3])
    c3, s3 = PO.page_write(x, [-1, 32, -5], c, s)             # no slot, or none of the cache
    assert np.array_equal(c3, c) and np.array_equal(s3, s)


@pytest.mark.parametrize("window", [0, 1, 5])
def test_prompt_attention_is_masked_sdpa(window):
    g = torch.Generator().manual_seed(11)
    H, Hkv, nq, nk = 4, 2, 6, 9
    q, k, v = (torch.randn(n, h, 16, generator=g, dtype=torch.float64) for n, h in ((nq, H), (nk, Hkv), (nk, Hkv)))
    o, lse, _, _ = PO.prompt_attention(q.numpy(), k.numpy(), v.numpy(), [0, nq], [0, nk], 0.25, window)
    i, j = torch.arange(nq)[:, None] + nk - nq, torch.arange(nk)
    seen = (j <= i) & ((j > i - window) if window else torch.ones(1, dtype=torch.bool))
    kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    ref = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk.transpose(0, 1), vv.transpose(0, 1),
                                                           attn_mask=seen, scale=0.25).transpose(0, 1)
    a = torch.einsum("ihd,jhd->ihj", q, kk) * 0.25
    ref_lse = a.masked_fill(~seen[:, None], -math.inf).logsumexp(-1)
    assert np.abs(o - ref.numpy()).max() < 1e-13 and np.abs(lse - ref_lse.numpy()).max() < 1e-13


def test_more_queries_than_keys_leaves_rows_empty():
    q, k = np.ones((5, 1, 16)), np.ones((2, 1, 16))
    o, lse, _, _ = PO.prompt_attention(q, k, k, [0, 5], [0, 2], 1.0)
    assert np.array_equal(o[:3], np.zeros((3, 1, 16))) and np.isneginf(lse[:3]).all() and np.allclose(o[3:], 1)


def test_decode_equals_the_last_prompt_row():
    r = np.random.RandomState(5)
    k, v = PO.encode(r.randn(3, 2, 16, 128) * 50), PO.encode(r.randn(3, 2, 16, 128) * 50)
    ks, vs = 2.0 ** r.randint(-8, -4, (3, 2)), 2.0 ** r.randint(-8, -4, (3, 2))
    table, n = np.array([[2, 0, 1]]), 37
    q = r.randn(1, 4, 128)
    flat = lambda c, s: (e4m3_decode(c) * s[..., None, None])[table[0]].transpose(0, 2, 1, 3).reshape(48, 2, 128)[:n]  # noqa: E731
    for w in (0, 9):
        o, lse, _, _ = PO.page_decode_attention(q, k, v, ks, vs, table, [n], 0.1, w)
        full = np.concatenate([np.zeros((n - 1, 4, 128)), q])
        o2, lse2, _, _ = PO.prompt_attention(full, flat(k, ks), flat(v, vs), [0, n], [0, n], 0.1, w, rows={n - 1})
        assert np.allclose(o, o2[n - 1]) and np.allclose(lse, lse2[n - 1])


# ------------------------------------------------------------------ refusals

P0 = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)


def _err(st):
    return st, cslc.LIB.cslc_last_error().decode()


def _plan(**kw):
    a = dict(old=P0, new=P0, B=2, free=P0, n_free=4, page=16, n_pages=10, max_pages=4, max_tokens=8, table=P0, slots=P0,
             cu=P0, seq=P0, status=P0)
    a.update(kw)
    return _err(cslc.LIB.cslc_page_plan(*a.values(), None))


def test_plan_refusals():
    for bad, status in ((dict(B=-1), 2), (dict(n_free=-1), 2), (dict(max_pages=-1), 2), (dict(max_tokens=-1), 2),
                        (dict(n_pages=-1), 2), (dict(page=8), 4), (dict(page=48), 4), (dict(page=256), 4),
                        (dict(B=8193), 4), (dict(n_pages=1 << 27), 4), (dict(old=None), 1), (dict(table=None), 1),
                        (dict(free=None), 1), (dict(slots=None), 1), (dict(cu=None), 1), (dict(status=None), 1),
                        (dict(seq=ODD), 3), (dict(slots=ODD), 3)):
        st, msg = _plan(**bad)
        assert st == status and "cslc_page_plan" in msg, (bad, st, msg)


def _write(**kw):
    a = dict(k=P0, v=P0, slots=P0, T=8, Hkv=2, D=128, page=64, n_pages=10, ks=256, vs=256, kc=P0, vc=P0, ksc=P0, vsc=P0)
    a.update(kw)
    return _err(cslc.LIB.cslc_page_write_e4m3(*a.values(), None))


def test_write_refusals():
    for bad, status in ((dict(T=-1), 2), (dict(D=64), 4), (dict(Hkv=0), 4), (dict(Hkv=129, ks=1 << 16, vs=1 << 16), 4),
                        (dict(page=100), 4), (dict(n_pages=-2), 2), (dict(n_pages=1 << 25), 4), (dict(ks=255), 4),
                        (dict(vs=260), 4), (dict(vs=128), 4), (dict(ks=-256), 4), (dict(k=None), 1), (dict(v=ODD), 3),
                        (dict(kc=ODD), 3), (dict(vsc=None), 1)):
        st, msg = _write(**bad)
        assert st == status and "cslc_page_write_e4m3" in msg, (bad, st, msg)
    assert _write(T=0, k=None)[0] == 0 and _write(n_pages=0, kc=None)[0] == 0


def _prompt(**kw):
    a = dict(q=P0, k=P0, v=P0, cq=P0, ck=P0, B=2, Tq=8, Tk=8, H=8, Hkv=2, D=128, qs=1024, ks=256, vs=256, window=0,
             scale=0.1, out=P0, lse=None, ws=P0, nws=1 << 30)
    a.update(kw)
    return _err(cslc.LIB.cslc_prompt_attn(*a.values(), None))


def test_prompt_refusals():
    for bad, status in ((dict(B=-1), 2), (dict(Tq=-1), 2), (dict(Tk=-1), 2), (dict(window=-1), 2), (dict(B=8193), 4),
                        (dict(D=64), 4), (dict(H=9), 4), (dict(H=0), 4), (dict(H=256, qs=1 << 16), 4), (dict(qs=1020), 4),
                        (dict(qs=512), 4), (dict(ks=64), 4), (dict(vs=1 << 36), 4), (dict(Tq=1 << 28), 4), (dict(q=None), 1),
                        (dict(k=None), 1), (dict(cq=None), 1), (dict(out=ODD), 3), (dict(lse=ODD), 3), (dict(ws=ODD), 3)):
        st, msg = _prompt(**bad)
        assert st == status and "cslc_prompt_attn" in msg, (bad, st, msg)
    assert _prompt(B=0, q=None)[0] == 0 and _prompt(Tq=0, q=None)[0] == 0
    if cslc.prompt_attn_workspace_bytes(2, 8, 8, 2):
        assert _prompt(ws=None, nws=0)[0] == 5 and _prompt(nws=1)[0] == 5
    assert cslc.prompt_attn_workspace_bytes(0, 8, 8, 2) == 0


def _decode(**kw):
    a = dict(q=P0, kc=P0, vc=P0, ks=P0, vs=P0, table=P0, n=P0, B=2, H=8, Hkv=2, D=128, page=64, n_pages=10, max_pages=4,
             qs=1024, window=0, scale=0.1, out=P0, lse=None, ws=P0, nws=1 << 30)
    a.update(kw)
    return _err(cslc.LIB.cslc_page_decode_attn(*a.values(), None))


def test_decode_refusals():
    for bad, status in ((dict(B=-1), 2), (dict(max_pages=-1), 2), (dict(window=-1), 2), (dict(B=8193), 4), (dict(D=64), 4),
                        (dict(H=9), 4), (dict(Hkv=0), 4), (dict(page=24), 4), (dict(n_pages=-1), 2),
                        (dict(n_pages=1 << 25), 4), (dict(qs=8), 4), (dict(q=None), 1), (dict(kc=None), 1),
                        (dict(vs=None), 1), (dict(table=None), 1), (dict(n=ODD), 3), (dict(out=None), 1), (dict(lse=ODD), 3),
                        (dict(ws=ODD), 3)):
        st, msg = _decode(**bad)
        assert st == status and "cslc_page_decode_attn" in msg, (bad, st, msg)
    assert _decode(B=0, q=None)[0] == 0
    if cslc.page_decode_workspace_bytes(2, 8, 2):
        assert _decode(ws=None, nws=0)[0] == 5 and _decode(nws=1)[0] == 5


def test_results_over_inputs_are_refused():
    at0, n = 1 << 30, 1 << 20                                  # n: bytes between pointers that do not overlap
    far = dict(zip(("old", "new", "free", "table", "slots", "cu", "len", "status"), (at0 + i * n for i in range(8))))
    for res, size in (("table", 12), ("slots", 40), ("cu", 3), ("len", 2), ("status", 2)):
        for inp, count in (("old", 2), ("new", 2), ("free", 4)):
            for at in (far[inp], far[inp] - (size * 4 - 1) // 16 * 16):
                a = dict(far, **{res: at})
                st, msg = _err(cslc.LIB.cslc_page_plan(a["old"], a["new"], 2, a["free"], count, 16, 9, 6, 40, a["table"],
                                                       a["slots"], a["cu"], a["len"], a["status"], None))
                assert st == 4 and "overlaps" in msg, (res, inp)
    for out in (at0, at0 + 7 * 2048, at0 + n + 16, at0 + 2 * n - 16):
        a = dict(q=at0, k=at0 + n, v=at0 + 2 * n, out=out)
        st, msg = _prompt(**a)
        assert st == 4 and "overlaps" in msg, out
    for out in (at0, at0 + 1024 * 2, at0 - 16):
        st, msg = _decode(q=at0, out=out)
        assert st == 4 and "overlaps" in msg


def test_scales_beyond_fp32_are_refused():
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert _prompt(scale=scale, out=1 << 30)[0] == 4
        assert _decode(scale=scale, out=1 << 30)[0] == 4


def test_workspace_of_head_counts_that_are_refused():
    """The binding asks for the size before the call checks its arguments."""
    for H, Hkv in ((256, 1), (129, 1), (1 << 20, 1), (0, 1), (8, 0), (8, 3), (-8, 1), (8, -1)):
        assert cslc.prompt_attn_workspace_bytes(1, 10, H, Hkv) == 0, (H, Hkv)
        assert cslc.page_decode_workspace_bytes(1, H, Hkv) == 0, (H, Hkv)


def test_binding_refuses_what_it_cannot_pass_on():
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        cslc.prompt_attn(q, q[:, :2], q[:, :2], cu, cu, 0.1)
    with pytest.raises(TypeError, match="bfloat16"):
        cslc.prompt_attn(q.float(), q[:, :2], q[:, :2], cu, cu, 0.1)


def test_lanes_of_a_warp_leave_together():
    """In the prompt kernel a wait gives up by each lane's own clock. Warps that go on to collective instructions
    (elections, shuffles) take one decision for all lanes; the producer is a single lane."""
    text = open(os.path.join(os.path.dirname(cslc.__file__), "csrc", "prompt_attn_sm100.cu")).read()
    text = text[text.index("prompt_attn_sm100_kernel("):text.index("size_t prompt_attn_workspace_bytes")]
    text = re.sub(r"//[^\n]*", "", text)
    at = [text.index(x) for x in ("if (warp == PA_PROD_WARP)", "else if (warp >= PA_MMA_WARP)", "const int row = tid & 127")]
    producer, issue, softmax = text[at[0]:at[1]], text[at[1]:at[2]], text[at[2]:]
    assert producer.index("if (lane == 0) {") < producer.index("pa_wait(") and text.count("pa_wait(") == producer.count("pa_wait(")
    voted = re.findall(r"(\S+ )(?:mbar_wait|pa_wait_slow)\(", softmax)
    assert voted and set(voted) <= {"__all_sync(0xffffffffu, ", "return ", "0xffffffffu, "} and "return mbar" not in softmax
    # the issuing warps: what a lane's wait says stays its own, and no collective is reached by some lanes only
    assert len(re.findall(r"mbar_wait\(", issue)) == 1 and "ok = ok && mbar_wait(" in issue
    leave = re.findall(r"[^\n]*\b(?:break|return);", issue)
    assert leave and all("!__all_sync(0xffffffffu, ok)" in x or "!t.there" in x for x in leave), leave
    elected = re.findall(r"if \(elect_one\(\)\) \{.*?\n +__syncwarp\(\);", issue, re.S)
    assert len(elected) == 2
    for block in elected:
        assert not re.search(r"uni\(|__shfl|__all|__any|elect_one", block[len("if (elect_one())"):])
        issue = issue.replace(block, "")
    assert re.findall(r"\bwait\(&bars\.(\w+)", issue) == ["item_full", "q_full"]


def test_lists_may_be_slices():
    """4-byte alignment of what is only read element by element (shown by the next check's refusal), 16 of the rest."""
    four, two = 0x1004, 0x1002
    for name in ("old", "new", "free"):
        st, msg = _plan(**{name: two})
        assert st == 3 and "4-byte" in msg, name
        st, msg = _plan(**{name: four, "cu": four})               # the result is not aligned
        assert st == 3 and "cu is not 16-byte" in msg, name
        at = {"old": 1 << 30, "new": 1 << 31, "free": 1 << 32, "table": 5 << 30, "slots": 6 << 30, "seq": 7 << 30, "cu": 8 << 30}
        st, msg = _plan(**{**at, name: at[name] + 4, "status": at[name]})
        assert st == 4 and "overlaps" in msg, name
    assert _write(slots=two)[0] == 3 and "4-byte" in _write(slots=two)[1]
    st, msg = _write(slots=four, kc=ODD)
    assert st == 3 and "k_cache" in msg
    for name in ("cq", "ck"):
        assert _prompt(**{name: two})[0] == 3
        st, msg = _prompt(**{name: four}, q=1 << 30, out=1 << 30)
        assert st == 4 and "overlaps" in msg, name
