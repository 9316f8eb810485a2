"""Eviction at its edges: more entries in use than the call has slots for,
large batches of large caches."""
import numpy as np
import pytest
import torch

import long_context_hybrid_kv_b200 as L
import paged_ref as P
from gpu_util import bf, bits, f32, i32
from oracle import ds4a_oracle as O
from test_paged_schedule_gpu import bf_bits, evict_many

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,n_slots,budget", [(3, 64, 20), (3, 900, 895), (3, 9000, 4000), (3, 40000, 10000), (2, 262150, 262000)])
@pytest.mark.parametrize("weights", [False, True])
def test_more_entries_than_slots_is_recorded(B, n_slots, budget, weights):
    """One block, a cluster, and the form for more slots than a cluster holds:
    the sequence stays as it is, the others are cut; with enough slots it is cut too."""
    D, m, page, extra = 8, 4, 50, 60
    per = -(-(n_slots + extra) // page)
    cfg = L.LayerCfg(2, D, 0, 0, 64, 128, 16, m, D ** -0.5, 10000.0, 1e-6)
    rng = np.random.default_rng(n_slots)
    table = rng.permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
    pages = rng.integers(0, 60000, (B * per + 1, page, D)).astype(np.uint16)
    d_pages, d_table = bf(pages), i32(table)
    kv = L.paged_kv(d_pages, d_table, page)
    drop = np.full(B, 5, np.int32)
    lens = [n_slots, n_slots + 1, n_slots - 1][:B]  # the second has one too many
    pos = np.asarray([(n + 5) * m + 1 for n in lens], np.int32)
    wide = n_slots + extra
    acc, entry = rng.random((B, wide)).astype(np.float32), np.full((B, wide), -1, np.int32)
    w = bf_bits(rng.random((B, wide)))
    d_acc, d_entry, d_drop, d_w = f32(acc), i32(entry), i32(drop), bf(w) if weights else None
    ws = torch.empty(L.ds4a_paged_evict_workspace(kv, B), dtype=torch.uint8, device="cuda")

    def call(n):
        L.ds4a_paged_evict(cfg, kv, i32(pos), budget, 3, d_acc[:, :n], d_entry[:, :n], d_drop, ws,
                           weights=d_w[:, :n] if weights else None)
        return L.ds4a_check()

    def follow(b, n):
        x = O.widen(w[b][:n]) if weights else None
        acc[b, :n], entry[b, :n], drop[b], moves = P.evict(x, acc[b, :n], entry[b, :n], int(drop[b]), lens[b], lens[b] + 5, budget, 3)
        if moves:
            fr, to = np.asarray(moves).T
            pages[table[b][to // page], to % page] = pages[table[b][fr // page], fr % page]

    def agree():
        assert np.array_equal(d_drop.cpu().numpy(), drop)
        assert np.array_equal(d_entry.cpu().numpy(), entry)
        assert np.array_equal(d_acc.cpu().numpy(), acc)
        assert np.array_equal(bits(d_pages), pages)

    assert call(n_slots) == (L.DS4A_EDEVICE, 1)
    for b in range(B):
        if b != 1:
            follow(b, n_slots)
    agree()
    # the others have `budget` entries now and stay as they are but for their weights
    assert call(wide) == (L.DS4A_OK, 0)
    for b in range(B):
        if b != 1:
            lens[b] = budget
        follow(b, wide)
    agree()
    assert drop[1] == 5 + n_slots + 1 - budget


def test_batch_that_leaves_no_room_for_clusters():
    # more slots than one block holds: the form that selects from memory
    evict_many("no clusters", 75, 33000, 16000, 7, D=8)
