"""Append into paged caches at their edges: no pages at all."""
import numpy as np
import pytest
import torch

import long_context_hybrid_kv_b200 as L
from gen import host
from gpu_util import bf, f32, i32
from test_paged_gpu import SEED, layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("overlap", [False, True])
@pytest.mark.parametrize("m", [1, 4, 128])
def test_append_without_pages_is_recorded(m, overlap, fp8):
    """An empty table has no address: nothing is stored, the rows enter the state."""
    cfg = layer(m=m)
    B = 3
    rb = L.ds4a_kv_fp8_row_bytes(512, 64) if fp8 else 512
    pages = torch.full((2, 4, rb), 9, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    kv = L.paged_kv(pages, torch.zeros((B, 0), dtype=torch.int32, device="cuda"), 4, fmt=L.DS4A_MX_KV_FP8 if fp8 else 0)
    assert kv.table is None and kv.max_pages == 0
    state = torch.zeros(L.ds4a_compress_state_bytes(cfg, B, 512, overlap), dtype=torch.uint8, device="cuda")
    x = bf(host.normal_bf16(SEED, "none", (B, 512)))
    bias = f32(np.zeros((m, 512)))
    more = dict(cb=x, zb=x, bias_b=bias) if overlap else {}
    L.ds4a_paged_append(cfg, kv, i32([m - 1] * B), x, x, bias, state, norm_g=f32(np.ones(512)), **more)
    rc, bits = L.ds4a_check()
    assert rc == L.DS4A_EDEVICE and bits == 1
    assert (pages == 9).all() and (state != 0).any()


def test_attend_without_pages_reads_the_window():
    cfg = layer(W=4, m=4)
    B = 2
    pages = torch.full((2, 4, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    kv = L.paged_kv(pages, torch.zeros((B, 0), dtype=torch.int32, device="cuda"), 4)
    q, win = bf(host.normal_bf16(SEED, "nq", (B, 64, 512))), torch.ones((B, 4, 512), dtype=torch.bfloat16, device="cuda")
    win[..., 448:] = 0  # (nothing to rotate)
    out = torch.zeros_like(q)
    ws = torch.empty(L.ds4a_paged_attend_workspace(cfg, kv, B), dtype=torch.uint8, device="cuda")
    L.ds4a_paged_attend(cfg, kv, i32([2, 900]), q, f32(np.ones(512)), win, 4, f32(np.full(64, -1e4)), out, ws)
    assert L.ds4a_check()[0] == L.DS4A_OK
    assert (out[..., :448] == 1).all() and (out[..., 448:] == 0).all()


@pytest.mark.parametrize("overlap", [False, True])
def test_append_at_the_last_position_of_32_bits(overlap):
    """Entry 2^24 - 1 of ratio 128: into pages by its slot, and into a pool that has it, or just not."""
    m, D, last = 128, 8, 2 ** 24 - 1
    cfg = layer(H=1, D=D, R=2, m=m)
    pool = torch.full((1, last + 1, D), 9.0, dtype=torch.bfloat16, device="cuda")
    pages = torch.full((2, 3, D), 9.0, dtype=torch.bfloat16, device="cuda")
    table = i32([[1]])
    kv = L.paged_kv(pages, table, 3)
    nb = L.ds4a_compress_state_bytes(cfg, 1, D, overlap)
    fill = bf(host.normal_bf16(SEED, "last.st", (nb // 2,)))
    x = {k: bf(host.normal_bf16(SEED, "last." + k, (1, D))) for k in ("ca", "za", "cb", "zb")}
    bias, g = f32(host.normal_f32(SEED, "last.b", (m, D))), f32(np.ones(D))
    more = dict(norm_g=g, **(dict(cb=x["cb"], zb=x["zb"], bias_b=bias) if overlap else {}))
    pos = i32([2 ** 31 - 1])
    L.ds4a_paged_append(cfg, kv, pos, x["ca"], x["za"], bias, fill.clone(), drop=i32([last - 2]), **more)
    L.ds4a_compress_append(cfg, pos, x["ca"], x["za"], bias, fill.clone(), pool, **more)
    assert L.ds4a_check() == (L.DS4A_OK, 0)
    got = pages[1, 2].clone()
    assert (got != 9.0).any() and torch.equal(got, pool[0, last]) and (pool[0, :last] == 9.0).all()
    assert (pages[0] == 9.0).all() and (pages[1, :2] == 9.0).all()
    pool[0, last] = 9.0
    L.ds4a_compress_append(cfg, pos, x["ca"], x["za"], bias, fill.clone(), pool[:, :last], **more)
    assert L.ds4a_check() == (L.DS4A_EDEVICE, 1)
    assert (pool == 9.0).all()
