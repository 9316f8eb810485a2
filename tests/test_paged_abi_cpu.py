"""Refusals of the paged-cache and 4-bit entry points, without a GPU: every
bad argument is returned as an error before any launch, and the binding checks
what the C interface cannot see."""
import ctypes

import pytest
import torch

import __graft_entry__ as entry
import long_context_hybrid_kv_b200 as L
import paged_ref as P
import numpy as np


@pytest.fixture(scope="module", autouse=True)
def built():
    entry.build()


A = 1 << 20   # an aligned address that nothing follows: the checks come first
MIS = A + 2


def cfg(**kw):
    c = dict(n_heads=64, head_dim=512, rope_dim=64, window=128, idx_heads=64, idx_dim=128, topk=512, ratio=4,
             sm_scale=512 ** -0.5, rope_base=10000.0, rms_eps=1e-6)
    c.update(kw)
    return L.LayerCfg(*c.values())


def kv(**kw):
    c = dict(pages=A, table=A, table_stride=8, format=0, n_pages=100, page_size=64, max_pages=8)
    c.update(kw)
    return L.PagedKv(*c.values())


BAD_KV = [dict(pages=None), dict(pages=MIS), dict(table=None), dict(table=A + 1), dict(table_stride=7), dict(format=2), dict(format=-1),
          dict(n_pages=-1), dict(page_size=0), dict(max_pages=-1), dict(page_size=1 << 28), dict(n_pages=1 << 30)]
BAD_CFG = [dict(n_heads=0), dict(n_heads=129), dict(head_dim=1024), dict(head_dim=12), dict(rope_dim=3), dict(ratio=0), dict(window=-1),
           dict(sm_scale=0.0)]


def attend(c=None, k=None, **kw):
    c, k = c or cfg(), k or kv()
    a = dict(B=2, pos=A, q=A, g=A, drop=None, idx=None, win=A, cap=128, wbs=128 * 512, sink=A, out=A, w=None, w_len=0, ws_=0,
             ws=A, nb=1 << 40)
    a.update(kw)
    return L.lib().ds4a_paged_attend(c, k, a["B"], a["pos"], a["q"], a["g"], a["drop"], a["idx"], a["win"], a["cap"], a["wbs"],
                                     a["sink"], a["out"], a["w"], a["w_len"], a["ws_"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("bad", BAD_KV)
def test_bad_caches(bad):
    k = kv(**bad)
    assert attend(k=k) == L.DS4A_EINVAL
    assert evict(k=k) == L.DS4A_EINVAL
    assert append(k=k) == L.DS4A_EINVAL
    assert L.ds4a_paged_attend_workspace(cfg(), k, 2) == 0


@pytest.mark.parametrize("bad", BAD_CFG)
def test_bad_layers(bad):
    assert attend(c=cfg(**bad)) == L.DS4A_EINVAL
    assert evict(c=cfg(**bad)) == L.DS4A_EINVAL
    assert append(c=cfg(**bad)) == L.DS4A_EINVAL


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(B=65536), dict(pos=None), dict(q=None), dict(g=None), dict(sink=None), dict(out=None), dict(win=None),
    dict(cap=127), dict(wbs=128 * 512 - 8), dict(wbs=128 * 512 + 4), dict(q=MIS), dict(out=MIS), dict(win=MIS), dict(idx=MIS),
    dict(drop=MIS), dict(w=MIS, w_len=8, ws_=8), dict(w=A, w_len=-1), dict(w=A, w_len=9, ws_=8), dict(ws=MIS),
])
def test_attend_refuses(bad):
    assert attend(**bad) == L.DS4A_EINVAL


def test_attend_other_refusals():
    assert attend(w=A, w_len=8, ws_=8, idx=A) == L.DS4A_EUNSUPPORTED
    assert attend(ws=None) == L.DS4A_ENOSPACE
    need = L.ds4a_paged_attend_workspace(cfg(), kv(), 2)
    assert need > 0 and attend(nb=need - 1) == L.DS4A_ENOSPACE
    assert attend(c=cfg(topk=0), idx=A) == L.DS4A_EINVAL
    assert attend(c=cfg(topk=5000), idx=A) == L.DS4A_EINVAL
    assert attend(B=0) == L.DS4A_OK
    # an FP8 row holds whole 32-value blocks
    assert attend(c=cfg(head_dim=488), k=kv(format=L.DS4A_MX_KV_FP8)) == L.DS4A_EUNSUPPORTED
    assert L.ds4a_paged_attend_workspace(cfg(), kv(), 0) == 0
    # more tiles than the schedule counts
    far = kv(max_pages=1 << 24, table_stride=1 << 24)
    assert L.ds4a_paged_attend_workspace(cfg(), far, 4) > 0 and L.ds4a_paged_attend_workspace(cfg(), far, 65535) == 0
    assert attend(k=far, B=65535) == L.DS4A_EINVAL
    assert L.ds4a_paged_attend_workspace(cfg(), kv(), 2, weights=True) > need


def evict(c=None, k=None, **kw):
    c, k = c or cfg(), k or kv()
    a = dict(B=2, pos=A, w=A, w_s=512, budget=100, recent=10, n=512, acc=A, entry=A, stride=512, drop=A, ws=A, nb=1 << 40)
    a.update(kw)
    return L.lib().ds4a_paged_evict(c, k, a["B"], a["pos"], a["w"], a["w_s"], a["budget"], a["recent"], a["n"], a["acc"], a["entry"],
                                    a["stride"], a["drop"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(B=65536), dict(pos=None), dict(acc=None), dict(entry=None), dict(drop=None), dict(w_s=511), dict(stride=511),
    dict(budget=0), dict(budget=513), dict(recent=-1), dict(recent=101), dict(n=0), dict(n=513), dict(acc=MIS), dict(entry=MIS),
    dict(w=MIS), dict(drop=MIS), dict(ws=MIS),
])
def test_evict_refuses(bad):
    assert evict(**bad) == L.DS4A_EINVAL


def test_evict_other_refusals():
    assert evict(B=0) == L.DS4A_OK
    need = L.ds4a_paged_evict_workspace(kv(), 2)
    assert need > 0 and evict(nb=need - 1) == L.DS4A_ENOSPACE and evict(ws=None) == L.DS4A_ENOSPACE
    assert L.ds4a_paged_evict_workspace(kv(), 0) == 0


def append(c=None, k=None, **kw):
    c, k = c or cfg(), k or kv()
    a = dict(B=2, pos=A, drop=None, ca=A, cb=None, za=A, zb=None, ba=A, bb=None, g=A, st=A)
    a.update(kw)
    return L.lib().ds4a_paged_append(c, k, a["B"], a["pos"], a["drop"], a["ca"], a["cb"], a["za"], a["zb"], a["ba"], a["bb"], a["g"],
                                     a["st"], None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(pos=None), dict(ca=None), dict(za=None), dict(ba=None), dict(st=None), dict(cb=A), dict(zb=A), dict(drop=MIS),
    dict(ca=MIS), dict(st=MIS),
])
def test_append_refuses(bad):
    assert append(**bad) == L.DS4A_EINVAL


def test_append_refuses_fp8_rows_without_a_norm():
    # (their RoPE dims are bf16, which an entry without norm and rotation does not have)
    k = kv(format=L.DS4A_MX_KV_FP8)
    assert append(k=k, g=None) == L.DS4A_EUNSUPPORTED
    assert append(k=k, g=None, cb=A, zb=A, bb=A) == L.DS4A_EUNSUPPORTED
    assert append(k=k, g=None, B=0, c=cfg(rope_dim=0)) == L.DS4A_OK


@pytest.mark.parametrize("norm", [False, True])
def test_binding_checks_the_rows_that_append_writes(norm):
    table = torch.zeros((2, 2), dtype=torch.int32)
    x = torch.zeros((2, 512), dtype=torch.bfloat16)
    state = torch.zeros(L.ds4a_compress_state_bytes(cfg(), 2, 512, False), dtype=torch.uint8)
    g = torch.ones(512) if norm else None
    pos, bias = torch.zeros(2, dtype=torch.int32), torch.zeros((4, 512))
    for pages, fmt in ((torch.zeros((4, 16, 256), dtype=torch.bfloat16), 0), (torch.zeros((4, 16, 528), dtype=torch.uint8), 1)):
        with pytest.raises(ValueError, match="rows must have"):
            L.ds4a_paged_append(cfg(), L.paged_kv(pages, table, 16, fmt=fmt), pos, x, x, bias, state, norm_g=g, stream=0)


def test_append_empty():
    assert append(B=0) == L.DS4A_OK


def test_mxfp4_refusals():
    lib = L.lib()
    q = lambda n=4, k=256, i=A, s=256, c=A, sc=A: lib.ds4a_quantize_mxfp4(n, k, i, s, c, sc, None)  # noqa: E731
    for bad in (dict(n=-1), dict(k=0), dict(k=96), dict(i=None), dict(c=None), dict(sc=None), dict(i=MIS), dict(c=MIS),
                dict(sc=MIS), dict(s=255), dict(s=260)):
        assert q(**bad) == L.DS4A_EINVAL, bad
    assert q(n=0) == L.DS4A_OK
    assert L.ds4a_mxfp4_scale_bytes(1, 128) == 512 and L.ds4a_mxfp4_scale_bytes(129, 256) == 2048
    assert L.ds4a_mxfp4_scale_bytes(0, 128) == 0 and L.ds4a_mxfp4_scale_bytes(4, 100) == 0
    oc = L.OprojCfg(64, 512, 8, 1024, 4096)
    need = L.ds4a_out_proj_mxfp4_workspace(oc, 4)
    assert need > 0

    def call(c=oc, M=4, o=A, wa=A, sa=A, wb=A, sb=A, y=A, ws=A, nb=need):
        return lib.ds4a_out_proj_mxfp4(c, M, o, wa, sa, wb, sb, y, ws, nb, None)

    for bad in (dict(M=-1), dict(o=None), dict(wa=None), dict(sa=None), dict(wb=None), dict(sb=None), dict(y=None), dict(o=MIS),
                dict(sa=MIS), dict(y=MIS), dict(ws=MIS), dict(c=L.OprojCfg(64, 512, 7, 1024, 4096))):
        assert call(**bad) == L.DS4A_EINVAL, bad
    assert call(nb=need - 1) == L.DS4A_ENOSPACE and call(ws=None) == L.DS4A_ENOSPACE
    assert call(M=0) == L.DS4A_OK
    for c in (L.OprojCfg(64, 512, 8, 1000, 4096), L.OprojCfg(64, 512, 8, 1024, 4000), L.OprojCfg(6, 64, 2, 256, 256)):
        assert call(c=c) == L.DS4A_EUNSUPPORTED
        assert L.ds4a_out_proj_mxfp4_workspace(c, 4) == 0


def test_binding_checks():
    pages = torch.zeros((4, 16, 512), dtype=torch.bfloat16)
    table = torch.zeros((2, 2), dtype=torch.int32)
    k = L.paged_kv(pages, table, 16)
    assert (k.n_pages, k.page_size, k.max_pages, k.table_stride, k.format) == (4, 16, 2, 2, 0)
    wide = torch.zeros((2, 9), dtype=torch.int32)
    assert L.paged_kv(pages, wide[:, :3], 16).table_stride == 9
    with pytest.raises(TypeError):
        L.paged_kv(pages.float(), table, 16)
    with pytest.raises(TypeError):
        L.paged_kv(pages, table.long(), 16)
    with pytest.raises(ValueError):
        L.paged_kv(pages, table.t(), 16)
    with pytest.raises(ValueError):
        L.paged_kv(pages, table, 8)
    with pytest.raises(ValueError):
        L.paged_kv(pages, table, 16, fmt=L.DS4A_MX_KV_FP8)
    acc = torch.zeros((2, 32))
    entry = torch.zeros((2, 32), dtype=torch.int32)
    i2 = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        L.ds4a_paged_evict(cfg(), k, i2, 4, 0, acc, entry[:, :31], i2, ws, stream=0)
    with pytest.raises(TypeError):
        L.ds4a_paged_evict(cfg(), k, i2, 4, 0, acc.double(), entry, i2, ws, stream=0)
    with pytest.raises(ValueError):
        L.ds4a_paged_evict(cfg(), k, i2, 4, 0, acc, entry, i2, ws, weights=torch.zeros((2, 31), dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError):
        L.ds4a_paged_evict(cfg(), k, i2.long(), 4, 0, acc, entry, i2, ws, stream=0)
    with pytest.raises(ValueError):
        L.ds4a_quantize_mxfp4(torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros(4 * 127, dtype=torch.uint8), ws, stream=0)


def test_plain_forms_of_the_scale_order():
    s = np.arange(130 * 8, dtype=np.int64).reshape(130, 8).astype(np.uint8)
    t = P.tile_scales(s)
    assert t.size == L.ds4a_mxfp4_scale_bytes(130, 256)
    assert np.array_equal(P.untile_scales(t, 130, 256), s)
    assert t[(32 * 0 + 5) * 16 + 1 * 4 + 2] == s[37, 2]
