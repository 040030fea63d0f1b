"""What the calls on a cache in pages and TokenScorer refuse, and how the kernels reach a page (no GPU: refused before anything is
enqueued, or read from the source)."""
import ctypes
import glob
import os
import re

import pytest
import torch

from tests import paged_oracle as P
from tests.test_target_waits_cpu import CSRC, part, source

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
E4M3 = torch.float8_e4m3fn
FAKE = 0x100000  # never dereferenced: a call is refused before any launch


@pytest.fixture(scope="module")
def T():
    from draft_head_gb300 import build
    build.build()
    from draft_head_gb300 import target
    return target


def pools(dtype=E4M3, pages=5, hkv=2, page=16, D=64):
    k = torch.zeros(pages, hkv, page, D).to(dtype)
    scale = [torch.zeros(pages, hkv, page, dtype=U8) for _ in "kv"] if dtype == E4M3 else [None, None]
    return k, k.clone(), *scale


def table(batch=3, places=2):
    return torch.zeros(batch, places, dtype=I32)


def layer(T, dtype=E4M3, page_table=None, n_q_heads=4, max_tokens=12, max_q=4, max_ctx=16, **kw):
    k, v, ks, vs = pools(dtype)
    return T.PagedAttention(k, v, table() if page_table is None else page_table, n_q_heads, max_tokens, max_q, max_ctx, k_scale=ks,
                            v_scale=vs, **kw)


def test_the_plain_form_knows_the_type():
    """The codes' values by their fields are torch's, but for the two that are NaN there; its rounding is the search's."""
    c = torch.arange(256, dtype=U8)
    want = c.view(E4M3).double()
    got = P.code_values()
    fine = ~torch.isnan(want)
    assert torch.equal(got[fine], want[fine]) and got[127] == 480 and got[255] == -480 and int((~fine).sum()) == 2
    x = torch.randn(64, 32, generator=torch.Generator().manual_seed(1)) * torch.logspace(-3, 3, 64)[:, None]
    codes, scale = P.quantise(x)
    y = (x.double() / torch.pow(2.0, scale.double() - 127)[:, None]).float().to(E4M3)
    assert torch.equal(codes.view(E4M3).double(), y.double())
    most = x.abs().amax(1).double() / torch.pow(2.0, scale.double() - 127)
    assert bool((most <= 448).all()) and bool((most > 224).all())


def test_pools_that_are_refused(T):
    k, v, ks, vs = pools()
    ok = dict(k_scale=ks, v_scale=vs)
    make = lambda k=k, v=v, t=table(), **kw: T.PagedAttention(k, v, t, 4, 12, 4, 16, **{**ok, **kw})  # noqa: E731
    make()
    make(k_scale=ks.view(torch.float8_e8m0fnu))
    for bad in (dict(k=k[:4]), dict(k=k.to(BF)), dict(k=k[0], v=v[0]), dict(k=k[..., ::2], v=v[..., ::2]), dict(v=v.transpose(1, 2))):
        with pytest.raises(ValueError, match="k and v"):
            make(**bad)
    with pytest.raises(ValueError, match="page type"):
        make(k=k.to(torch.float16), v=v.to(torch.float16))
    for bad in (None, ks[:4], ks.float(), ks.transpose(1, 2), ks[..., ::2], torch.zeros(5, 2, 32, dtype=U8)[..., ::2]):
        with pytest.raises(ValueError, match="v_scale"):
            make(v_scale=bad)
    with pytest.raises(ValueError, match="k_scale"):
        T.PagedAttention(k.to(BF), v.to(BF), table(), 4, 12, 4, 16, k_scale=ks)
    for bad in (table().long(), table()[0], table(3, 4)[:, ::2], torch.zeros(3, 0, dtype=I32)):
        with pytest.raises(ValueError, match="page_table"):
            make(t=bad)


@pytest.mark.parametrize("page,D,dtype,hq", [(8, 64, E4M3, 4), (24, 64, E4M3, 4), (8192, 64, E4M3, 4), (16, 72, E4M3, 4), (16, 72, BF, 3),
                                             (16, 272, BF, 4), (16, 4, F32, 4)])
def test_sizes_that_are_not_supported(T, page, D, dtype, hq):
    k, v, ks, vs = pools(dtype, page=page, D=D)
    with pytest.raises(ValueError, match="not supported"):
        T.PagedAttention(k, v, table(), hq, 12, 4, 16, k_scale=ks, v_scale=vs)


@pytest.mark.parametrize("dtype", [E4M3, BF, F32])
def test_weights_of_a_norm(T, dtype):
    row = BF if dtype == E4M3 else dtype
    layer(T, dtype, q_weight=torch.ones(64, dtype=row), k_weight=torch.ones(64, dtype=row), rope=torch.ones(30, 64))
    for name in ("q_weight", "k_weight"):
        with pytest.raises(ValueError, match="weight"):
            layer(T, dtype, norm=False, **{name: torch.ones(64, dtype=row)})
        with pytest.raises(ValueError, match=name):
            layer(T, dtype, **{name: torch.ones(64, dtype=F32 if row == BF else BF)})


def ints(*x, dtype=I32):
    return torch.tensor(x, dtype=dtype)


CTX, START, POS = ints(1, 2, 3), ints(0, 4, 8, 12), torch.arange(12, dtype=I32)
BAD_ROWS = [dict(ctx_len=ints(1, 2, 3, dtype=torch.int64)), dict(ctx_len=ints(1, 2)), dict(q_start=ints(0, 4, 8)), dict(q_start=START.float()),
            dict(positions=POS[:11]), dict(positions=POS.long())]


@pytest.mark.parametrize("i", range(len(BAD_ROWS)))
def test_lengths_and_positions_that_are_refused(T, i):
    p = layer(T)
    a = {**dict(ctx_len=CTX, q_start=START, positions=POS), **BAD_ROWS[i]}
    with pytest.raises(ValueError, match=next(iter(BAD_ROWS[i]))):
        p.append(torch.zeros(12, 8 * 64, dtype=BF), **a)
    with pytest.raises(ValueError, match=next(iter(BAD_ROWS[i]))):
        p.attend(torch.zeros(12, 4, 64, dtype=BF), **a)


def test_rows_that_are_refused(T):
    p = layer(T)
    for bad in (torch.zeros(12, 8 * 64), torch.zeros(12, 8 * 64).to(E4M3), torch.zeros(13, 8 * 64, dtype=BF), torch.zeros(12, 7 * 64, dtype=BF)):
        with pytest.raises(ValueError):
            p.append(bad, CTX, q_start=START)
    for bad in (torch.zeros(12, 4, 64), torch.zeros(12, 4, 32, dtype=BF), torch.zeros(13, 4, 64, dtype=BF), torch.zeros(4, 12, 64, dtype=BF).transpose(0, 1)):
        with pytest.raises(ValueError):
            p.attend(bad, CTX, q_start=START)
    for mask in (torch.ones(3, 4, 5, dtype=U8), torch.ones(2, 4, 4, dtype=U8), torch.ones(3, 4, 4)):
        with pytest.raises(ValueError, match="mask"):
            p.attend(torch.zeros(12, 4, 64, dtype=BF), CTX, q_start=START, mask=mask)


def test_reads_that_are_refused(T):
    p = layer(T)
    k = torch.zeros(3, 2, 20, 64, dtype=BF)
    for bad in (k.float(), k[:2], k[:, :1], k[..., :32]):
        with pytest.raises(ValueError):
            p.read(bad, bad.clone(), CTX)
    with pytest.raises(ValueError, match="k and v"):
        p.read(k, k[:, :, :10].clone(), CTX)
    for bad in (CTX.long(), CTX[:2], ints(1, 1).repeat(3)[::2]):
        with pytest.raises(ValueError, match="count"):
            p.read(k, k.clone(), bad)
        with pytest.raises(ValueError, match="first"):
            p.read(k, k.clone(), CTX, first=bad)


def test_scores_that_are_refused(T):
    with pytest.raises(ValueError, match="top_n"):
        T.TokenScorer(3, 100, F32, 33, device="cpu")
    with pytest.raises(ValueError, match="top_n"):
        T.TokenScorer(3, 100, F32, -1, device="cpu")
    s = T.TokenScorer(3, 100, F32, 4, device="cpu")
    for bad in (torch.zeros(4, 100), torch.zeros(3, 99), torch.zeros(3, 100, dtype=BF), torch.zeros(3, 200)[:, ::2], torch.zeros(1, 3, 100)):
        with pytest.raises(ValueError, match="logits"):
            s.score(bad)
    x = torch.zeros(3, 100)
    for bad in (CTX.long(), CTX[:2], CTX.float(), ints(1, 1).repeat(3)[::2]):
        with pytest.raises(ValueError, match="tokens"):
            s.score(x, bad)
    for bad in (torch.ones(2), torch.ones(3, dtype=BF), CTX, torch.ones(6)[::2]):
        with pytest.raises(ValueError, match="temperature"):
            s.score(x, CTX, bad)


def paged(B, **kw):
    a = dict(dtype=B.E4M3, batch=3, n_kv_heads=2, head_dim=64, n_pages=9, page_size=16, max_pages=4, k=FAKE, v=FAKE, page_stride=2048,
             head_stride=1024, slot_stride=64, k_scale=FAKE, v_scale=FAKE, page_table=FAKE, table_stride=4)
    a.update(kw)
    return B.domino_paged_cache(*(a[f[0]] for f in B.domino_paged_cache._fields_))


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
BAD_CACHES = [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(batch=-1), INVALID), (dict(n_kv_heads=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(n_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(max_pages=0), INVALID), (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(page_stride=-16), INVALID), (dict(head_stride=1032), INVALID), (dict(slot_stride=72), INVALID), (dict(k_scale=None), INVALID),
    (dict(v_scale=None), INVALID), (dict(page_table=None), INVALID), (dict(page_table=FAKE + 2), INVALID), (dict(table_stride=3), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=8192), UNSUPPORTED), (dict(head_dim=72), UNSUPPORTED),
    (dict(head_dim=272), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(dtype=1, slot_stride=68), INVALID)]


@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_the_library_refuses_caches(T, i):
    B = T.B
    change, status = BAD_CACHES[i]
    c, block = paged(B, **change), B.block(3, 1, 10, FAKE)
    ref, rows = ctypes.byref(c), ctypes.byref(block)
    assert B.lib.domino_paged_attention_workspace_bytes(ref, rows, 4) == 0
    assert B.lib.domino_paged_attention(ref, rows, 4, FAKE, 1.0, 0, None, 0, 0, FAKE, None, FAKE, 1 << 30, None) == status
    assert B.lib.domino_paged_append(ref, rows, 4, FAKE, 256, FAKE, 128, FAKE, 128, 1, None, None, 1e-6, None, 0, 0, 0, FAKE, FAKE, 256,
                                     None) == status
    out = B.domino_kv_cache(1, 3, 2, 64, 40, FAKE, FAKE, 40 * 128, 40 * 64, 64)
    assert B.lib.domino_paged_read(ref, None, FAKE, 40, ctypes.byref(out), FAKE, 256, None) == status


def test_the_library_refuses_arguments(T):
    B, lib = T.B, T.B.lib
    c = paged(B)
    ref = ctypes.byref(c)
    rows = ctypes.byref(B.block(3, 1, 10, FAKE))
    need = lib.domino_paged_attention_workspace_bytes(ref, rows, 4)
    assert need > 256

    def attend(block=rows, hq=4, q=FAKE, scale=1.0, mode=0, mask=None, window=0, sinks=0, out=FAKE, ws=FAKE, size=need - 1):
        return lib.domino_paged_attention(ref, block, hq, q, scale, mode, mask, window, sinks, out, None, ws, size, None)

    assert attend() == WORKSPACE and attend(ws=None) == WORKSPACE and attend(ws=FAKE + 64, size=1 << 30) == WORKSPACE
    for bad in (dict(block=None), dict(hq=3), dict(hq=0), dict(q=None), dict(q=FAKE + 4), dict(scale=-1.0), dict(scale=float("nan")), dict(mode=3),
                dict(mode=2), dict(window=-1), dict(sinks=-1), dict(out=None), dict(block=ctypes.byref(B.block(3, 1, 10, None))),
                dict(block=ctypes.byref(B.block(4, 1, 10, FAKE))), dict(block=ctypes.byref(B.block(2, 1, 10, FAKE)))):
        assert attend(**bad) == INVALID, bad
    assert attend(block=ctypes.byref(B.block(0, 0, 10, FAKE))) == 0  # no rows: nothing to do

    def append(norm=1, qw=None, kw=None, eps=1e-6, rope=FAKE, rot=64, stride=256, k=FAKE, ws=FAKE, size=255):
        return lib.domino_paged_append(ref, rows, 4, FAKE, stride, k, 128, FAKE, 128, norm, qw, kw, eps, rope, 50, rot, 0, FAKE, ws, size, None)

    assert append() == WORKSPACE
    for bad in (dict(norm=0, qw=FAKE), dict(norm=0, kw=FAKE), dict(eps=-1.0), dict(eps=float("inf")), dict(rope=None), dict(rot=66), dict(rot=3),
                dict(stride=250), dict(k=None), dict(qw=FAKE + 4)):
        assert append(**bad) == INVALID, bad

    def read(dtype=1, batch=3, heads=2, dim=64, cap=40, count=FAKE, most=40, size=255):
        out = B.domino_kv_cache(dtype, batch, heads, dim, cap, FAKE, FAKE, 40 * 128, 40 * 64, 64)
        return lib.domino_paged_read(ref, None, count, most, ctypes.byref(out), FAKE, size, None)

    assert read() == WORKSPACE and read(most=0) == 0
    for bad in (dict(dtype=0), dict(dtype=2), dict(batch=2), dict(heads=1), dict(dim=32), dict(most=41), dict(most=-1), dict(count=None)):
        assert read(**bad) == INVALID, bad
    assert lib.domino_paged_read(ref, None, FAKE, 40, None, FAKE, 256, None) == INVALID

    def score(dtype=0, logits=FAKE, stride=100, n=3, V=100, top=4, ws=FAKE, size=255):
        return lib.domino_token_logprobs(dtype, logits, stride, n, V, FAKE, FAKE, top, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ws, size, None)

    assert score() == WORKSPACE and score(ws=None) == WORKSPACE and score(n=0) == 0
    for bad in (dict(dtype=2), dict(logits=None), dict(logits=FAKE + 2), dict(dtype=1, logits=FAKE + 1), dict(stride=99), dict(n=-1), dict(V=0), dict(top=-1)):
        assert score(**bad) == INVALID, bad
    assert score(top=33) == UNSUPPORTED


def test_pages_are_reached_through_the_check_alone():
    """A page's number is read from the table in one place, which answers -1 for one that is not there."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        found += [(os.path.basename(path), m) for m in re.findall(r"\b\w*\.table\b(?!_)", source(os.path.basename(path)))]
    assert found == [("pages.cuh", "p.table")]
    check = part(source("pages.cuh"), "int page_of(const PagesArgs& p, int b, int s) {", "}")
    assert "(unsigned)page < (unsigned)p.n_pages ? page : -1" in check


def test_waits_over_pages_follow_the_rules():
    """Whole warps leave a wait with one answer; boxes in flight land on every way out; who converts codes waits on every use of a
    buffer, in order, and is told when no more come."""
    text = source("attention_tc.cu")
    convert = part(text, "if (C::kCodes && warp >= 12) {", "} else if (CACHE != kWhole && warp == 0) {")
    bring = part(text, "} else if (CACHE != kWhole && warp == 0) {", "} else if (warp == 0 && lane == 0) {")
    for role in (convert, bring):
        assert "warp_wait(" in role and not re.search(r"(!|=|&&|\breturn)\s*mbar_wait\(", role)
    assert "if (note & kNoteEnd) break;" in convert and "++from == in_slots" in convert and "++to == slots" in convert
    after = bring[bring.index("walk.next("):]
    assert after.index("kNoteEnd") < after.index("mbar_land(&full[") and "mbar_land(&full[j % in_slots]" in after
    ring = part(source("attention_rows.cu"), "if (kCodes) {\n    asm volatile(", "}")
    assert "cp.async.wait_all" in ring  # before the ring's memory becomes the warps' sums
