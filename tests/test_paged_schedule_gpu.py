"""Every way in which decode attention over the paged cache spreads a batch
over the GPU, against the plain 64-bit form: pieces of cut items, short items
that share blocks, the row of all tiles cut into ranges; with head groups,
FP8 rows, items of many pieces, and the refusals of the binding that need a
device."""
import numpy as np
import pytest
import torch

import long_context_hybrid_kv_b200 as L
import paged_ref as P
from gpu_util import bf, bits, check_ok, f32, i32
from oracle import ds4a_oracle as O
from test_paged_gpu import Case

pytestmark = pytest.mark.gpu


def bf_bits(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


def spread(name, lens, weights=True, **kw):
    c = Case(name, lens, kw.pop("page", 64), m=16, **kw)
    w = torch.full((c.B, max(lens) + 1), 7.0, dtype=torch.bfloat16, device="cuda") if weights else None
    c.run(weights=w)
    check_ok()
    c.check(weights=w)
    first = c.out.clone()
    c.out.fill_(7.0)
    c.run(weights=w)  # the same bits from a workspace of other leftovers
    check_ok()
    assert torch.equal(first, c.out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [8, 72])
def test_pieces_next_to_shared_blocks(H, fp8):
    # long items cut into pieces, short ones that share blocks, none at all
    spread(f"pieces{H}{fp8}", [9000, 3, 0, 700, 64, 1, 130, 65, 2500, 40, 256, 129], H=H, fp8=fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_equal_items_as_a_row_of_tiles(fp8):
    # 100 items of 24 tiles: one a block would leave a third of the blocks idle
    spread(f"row{fp8}", [1400] * 100, H=8, fp8=fp8, weights=not fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_more_items_than_blocks_as_a_row_of_tiles(fp8):
    # 152 items of 20 tiles on 148 blocks; some short ones whose ends move
    spread(f"many{fp8}", [1150] * 100 + [70, 1, 0, 200] * 10 + [1150] * 52, H=5, fp8=fp8, weights=not fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_more_items_than_blocks_share_them(fp8):
    lens = [int(v) for v in np.random.default_rng(3).integers(0, 300, 290)]
    spread(f"share{fp8}", lens, H=6, fp8=fp8, page=16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,most", [(2500, 4), (900, 260)])
def test_many_segments_a_block(B, most, fp8):
    # 6 to 17 whole items one after the other in every block
    lens = [int(v) for v in np.random.default_rng(B).integers(0, most, B)]
    c = Case(f"segs{B}{fp8}", lens, 16, m=16, H=2, W=4, fp8=fp8, spare=0)
    c.run()
    check_ok()
    got = c.out.double().cpu().numpy()
    for b in list(range(0, B, 13)) + [B - 1]:
        out, _, bound, _ = c.ref(b)
        assert (np.abs(got[b] - out) <= bound).all(), b


def test_more_sequences_than_the_schedule_keeps():
    # lengths behind the first 36864 are computed where they are needed
    B = 37000
    rng = np.random.default_rng(8)
    cfg = L.LayerCfg(1, 512, 64, 2, 64, 128, 512, 16, 512 ** -0.5, 10000.0, 1e-6)
    pages = rng.standard_normal((64, 4, 512)).astype(np.float32)
    table = rng.integers(0, 64, (B, 1)).astype(np.int32)  # attention may share pages
    n = rng.integers(0, 5, B)
    pos = (n * 16 + rng.integers(0, 15, B)).astype(np.int32)
    q, win = rng.standard_normal((B, 1, 512)).astype(np.float32), rng.standard_normal((B, 2, 512)).astype(np.float32)
    bfc = lambda x: torch.from_numpy(x).bfloat16().cuda()  # noqa: E731
    d_pages, d_table, d_q, d_win = bfc(pages), i32(table), bfc(q), bfc(win)
    kv = L.paged_kv(d_pages, d_table, 4)
    out = torch.full((B, 1, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(L.ds4a_paged_attend_workspace(cfg, kv, B), dtype=torch.uint8, device="cuda")
    L.ds4a_paged_attend(cfg, kv, i32(pos), d_q, torch.ones(512, device="cuda"), d_win, 2, torch.zeros(1, device="cuda"), out, ws)
    check_ok()
    got = out.double().cpu().numpy()
    dp, dq, dw = (t.double().cpu().numpy() for t in (d_pages, d_q, d_win))
    for b in list(range(0, B, 501)) + [36863, 36864, 36865, B - 1]:
        p = int(pos[b])
        near = np.arange(max(0, p - 1), p + 1) % 2
        rows = np.concatenate([dp[table[b, 0]][:n[b]], dw[b][near]])
        ref, _, bound, _ = P.attend(dq[b], np.ones(512), rows, int(n[b]), np.zeros(1), p, 512 ** -0.5, 64, 10000.0, 1e-6)
        assert (np.abs(got[b] - ref) <= bound).all(), b


def test_more_items_than_blocks_by_head_groups():
    # 80 sequences x 2 groups of heads
    lens = [int(v) for v in np.random.default_rng(4).integers(0, 500, 80)]
    spread("groups", lens, H=70, page=16)


def test_many_pieces_of_two_head_groups():
    # each group's item is cut into more pieces than one warp joins at once
    spread("long groups", [4000], H=100)


def test_without_a_window_empty_sequences_between_cut_ones():
    spread("nowin", [0, 3000, 0, 0, 1, 2000, 0], H=8, W=0)


def test_selected_slots_of_many_sequences():
    lens = [int(v) for v in np.random.default_rng(5).integers(0, 700, 170)]
    c = Case("selmany", lens, 16, m=16, H=4)
    k = 300
    cfg = L.LayerCfg(4, 512, 64, 128, 64, 128, k, 16, 512 ** -0.5, 10000.0, 1e-6)
    c.cfg = cfg
    idx = np.full((c.B, k), -1, np.int32)
    slots = []
    rng = np.random.default_rng(6)
    for b, n in enumerate(lens):
        take = np.sort(rng.choice(n, min(n, k), replace=False)) if n else np.zeros(0, np.int64)
        idx[b, :len(take)] = take
        slots.append(take)
    c.run(idx=i32(idx))
    check_ok()
    c.check(slots=slots)


def test_generic_shape_of_many_sequences():
    lens = [int(v) for v in np.random.default_rng(7).integers(0, 120, 320)]
    spread("generic", lens, H=3, D=64, R=16, W=8, page=7)


def evict_many(name, B, cap, budget, recent, D=32, page=40):
    """A batch of caches of unequal lengths, weights with ties, small rows."""
    rng = np.random.default_rng(sum(map(ord, name)))
    m, per = 4, -(-cap // page)
    cfg = L.LayerCfg(2, D, 0, 0, 64, 128, 16, m, D ** -0.5, 10000.0, 1e-6)
    table = rng.permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
    pages = rng.integers(0, 60000, (B * per + 1, page, D)).astype(np.uint16)
    lens = [cap, budget + 1, budget] + [int(v) for v in rng.integers(budget // 2, cap + 1, max(0, B - 3))]
    lens = lens[:B]
    acc = (rng.integers(0, 64, (B, cap)) / 8).astype(np.float32)  # many ties
    acc[0] = rng.random(cap)
    entry, drop = np.full((B, cap), -1, np.int32), np.zeros(B, np.int32)
    w = bf_bits(rng.random((B, cap)))
    pos = np.asarray([n * m + 1 for n in lens], np.int32)
    d_pages, d_w, d_table = bf(pages), bf(w), i32(table)
    kv = L.paged_kv(d_pages, d_table, page)
    d_acc, d_entry, d_drop = f32(acc), i32(entry), i32(drop)
    ws = torch.full((L.ds4a_paged_evict_workspace(kv, B),), 0xFF, dtype=torch.uint8, device="cuda")
    L.ds4a_paged_evict(cfg, kv, i32(pos), budget, recent, d_acc, d_entry, d_drop, ws, weights=d_w)
    check_ok()
    for b, n in enumerate(lens):
        acc[b], entry[b], drop[b], moves = P.evict(O.widen(w[b]), acc[b], entry[b], 0, n, n, budget, recent)
        if len(moves):
            fr, to = np.asarray(moves).T
            pages[table[b][to // page], to % page] = pages[table[b][fr // page], fr % page]
    assert np.array_equal(d_drop.cpu().numpy(), drop)
    assert np.array_equal(d_entry.cpu().numpy(), entry)
    assert np.array_equal(d_acc.cpu().numpy(), acc)
    assert np.array_equal(bits(d_pages), pages)


# a cluster of 1 to 8 blocks a sequence, 1 to 32 slots a thread
@pytest.mark.parametrize("B,cap", [(3, 1024), (3, 1025), (3, 4096), (1, 4097), (3, 8193), (2, 16385), (1, 40000), (2, 100000),
                                   (1, 200001), (40, 9000), (38, 30000), (75, 1030), (80, 5000), (80, 9000), (76, 20000)])
def test_evict_every_size_of_cache(B, cap):
    evict_many(f"size{B}.{cap}", B, cap, cap // 2, 7)
    evict_many(f"few{B}.{cap}", B, cap, cap - 3, cap // 3)


def test_evict_more_slots_than_a_cluster_holds():
    evict_many("huge", 1, 262150, 262000, 100)
    evict_many("half", 1, 300000, 150000, 100)


def test_binding_refuses_other_devices_and_sizes():
    c = Case("refuse", [40, 100], 16, m=16, H=8)
    ws = c.workspace()

    def call(**kw):
        a = dict(kv=c.kv, q_pos=c.d_pos, q=c.d_q, g=c.d_g, win=c.d_win, sink=c.d_sink, out=c.out, ws=ws)
        a.update(kw)
        L.ds4a_paged_attend(c.cfg, a["kv"], a["q_pos"], a["q"], a["g"], a["win"], c.win_cap, a["sink"], a["out"], a["ws"],
                            drop=a.get("drop"), idx=a.get("idx"), weights=a.get("weights"))

    call()
    for bad in (dict(q_pos=c.d_pos.cpu()), dict(q=c.d_q.cpu()), dict(g=c.d_g.cpu()), dict(win=c.d_win.cpu()),
                dict(sink=c.d_sink.cpu()), dict(out=c.out.cpu()), dict(ws=ws.cpu()), dict(drop=c.d_pos.cpu()),
                dict(kv=L.paged_kv(c.pages.cpu(), c.d_table.cpu(), 16)), dict(kv=L.paged_kv(c.pages, c.d_table[:1], 16)),
                dict(kv=L.paged_kv(c.pages[..., :256].contiguous(), c.d_table, 16)),
                dict(q=c.d_q[:, :7].contiguous()), dict(out=c.out[:, :7].contiguous()), dict(g=c.d_g[:511]),
                dict(sink=c.d_sink[:7]), dict(win=c.d_win[:, :100]), dict(win=c.d_win[:1]),
                dict(q_pos=c.d_pos.long()), dict(idx=c.d_table[:, :2].contiguous()),
                dict(weights=torch.zeros((1, 200), dtype=torch.bfloat16, device="cuda")),
                dict(weights=torch.zeros((2, 200), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError):
        L.paged_kv(c.pages, c.d_table.cpu(), 16)
    B, n = 2, 128
    acc, entry = torch.zeros((B, n), device="cuda"), torch.full((B, n), -1, dtype=torch.int32, device="cuda")
    drop = torch.zeros(B, dtype=torch.int32, device="cuda")
    ews = torch.zeros(L.ds4a_paged_evict_workspace(c.kv, B), dtype=torch.uint8, device="cuda")
    for bad in (dict(acc=acc.cpu()), dict(entry=entry.cpu()), dict(drop=drop.cpu()), dict(q_pos=c.d_pos.cpu()),
                dict(ws=ews.cpu()), dict(drop=drop[:1])):
        a = dict(q_pos=c.d_pos, acc=acc, entry=entry, drop=drop, ws=ews)
        a.update(bad)
        with pytest.raises(ValueError):
            L.ds4a_paged_evict(c.cfg, c.kv, a["q_pos"], 64, 8, a["acc"], a["entry"], a["drop"], a["ws"])
    o = torch.zeros((2, 8, 512), dtype=torch.bfloat16, device="cuda")
    oc = L.OprojCfg(8, 512, 8, 128, 256)
    u = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda")  # noqa: E731
    args = [o, u(8 * 128 * 512 // 2), u(8 * 128 * 512 // 32), u(256 * 1024 // 2), u(256 * 1024 // 32),
            torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda"), u(L.ds4a_out_proj_mxfp4_workspace(oc, 2))]
    for i in range(7):
        with pytest.raises(ValueError):
            L.ds4a_out_proj_mxfp4(oc, *[t.cpu() if j == i else t for j, t in enumerate(args)])
    check_ok()
