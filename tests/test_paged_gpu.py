"""The paged cache on the GPU (ds4a_paged_attend, ds4a_paged_append,
ds4a_paged_evict) against plain 64-bit forms.  Attention is held to a bound
counted from its bf16 roundings (paged_ref.attend) and to max-abs-relative
1e-2 per sequence; eviction exactly."""
import math

import numpy as np
import pytest
import torch

import long_context_hybrid_kv_b200 as L
import paged_ref as P
from gen import host
from gpu_util import bf, bits, check_ok, f32, f64, i32
from oracle import compare as C
from oracle import ds4a_oracle as O

pytestmark = pytest.mark.gpu
SEED = 2718
BASE, EPS = 10000.0, 1e-6
POISON = 0x7FC0  # bf16 NaN: rows that no key may read


def layer(H=64, D=512, R=64, W=128, m=128, k=512):
    return L.LayerCfg(H, D, R, W, 64, 128, k, m, D ** -0.5, BASE, EPS)


class Case:
    """A batch of sequences of the given lengths over a paged cache whose
    unused rows hold NaN."""

    def __init__(self, name, lens, page, H=64, D=512, R=64, W=128, m=128, fp8=False, spare=2, drop=None, pos=None,
                 win_cap=None):
        self.cfg, self.fp8, self.page = layer(H, D, R, W, m), fp8, page
        self.H, self.D, self.R, self.W, self.m = H, D, R, W, m
        B = len(lens)
        self.lens, self.B = lens, B
        per = max(1, -(-max(lens + [1]) // page)) + spare
        rng = np.random.default_rng(sum(map(ord, name)))
        n_pages = B * per + 3
        self.table = rng.permutation(n_pages)[:B * per].reshape(B, per).astype(np.int32)
        full = np.full((n_pages, page, D), POISON, np.uint16)
        for b, n in enumerate(lens):
            if n:
                s = np.arange(n)
                full[self.table[b][s // page], s % page] = host.normal_bf16(SEED, f"{name}.kv{b}", (n, D))
        self.drop = None if drop is None else np.asarray(drop, np.int32)
        gone = np.zeros(B, np.int64) if drop is None else np.asarray(drop, np.int64)
        if pos is None:
            pos = [(int(g) + n) * m + int(rng.integers(0, max(1, m - 1))) for n, g in zip(lens, gone)]
        self.pos = np.asarray(pos, np.int32)
        self.win_cap = win_cap or max(1, W)
        self.q = host.normal_bf16(SEED, f"{name}.q", (B, H, D))
        self.g = (1 + 0.1 * host.normal_f32(SEED, f"{name}.g", (D,))).astype(np.float32)
        self.win = host.normal_bf16(SEED, f"{name}.win", (B, self.win_cap, D))
        self.sink = host.normal_f32(SEED, f"{name}.sink", (H,)).astype(np.float32)
        if fp8:
            clean = np.where(full == POISON, np.uint16(0), full)
            q8 = O.quantize_kv_fp8(clean.reshape(-1, D), D, R).reshape(n_pages, page, -1)
            q8[(full == POISON).all(-1)] = 0xFF  # NaN codes and scales
            self.pages_np, self.pages = q8, torch.from_numpy(q8).cuda()
        else:
            self.pages_np, self.pages = full, bf(full)
        self.d_table, self.d_pos = i32(self.table), i32(self.pos)
        self.d_drop = None if drop is None else i32(self.drop)
        self.kv = L.paged_kv(self.pages, self.d_table, page, fmt=L.DS4A_MX_KV_FP8 if fp8 else 0)
        self.d_q, self.d_g, self.d_sink, self.d_win = bf(self.q), f32(self.g), f32(self.sink), bf(self.win)
        self.out = torch.full((B, H, D), 7.0, dtype=torch.bfloat16, device="cuda")

    def run(self, idx=None, weights=None, ws=None, stream=None):
        if ws is None:
            ws = self.workspace(idx is not None, weights is not None)
        L.ds4a_paged_attend(self.cfg, self.kv, self.d_pos, self.d_q, self.d_g, self.d_win if self.W else None,
                            self.win_cap, self.d_sink, self.out, ws, drop=self.d_drop, idx=idx, weights=weights,
                            stream=stream)

    def workspace(self, sparse=False, weights=False):
        n = L.ds4a_paged_attend_workspace(self.cfg, self.kv, self.B, sparse, weights)
        assert n > 0
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def ref(self, b, slots=None):
        p = int(self.pos[b])
        slots = np.arange(self.lens[b]) if slots is None else np.asarray(slots, np.int64)
        rows = [P.cache_rows(self.pages_np, self.table[b], slots, self.page, self.D, self.R, self.fp8)] if len(slots) else []
        if self.W:
            near = np.arange(max(0, p - self.W + 1), p + 1) % self.win_cap
            rows.append(O.widen(self.win[b][near]))
        rows = np.concatenate(rows) if rows else np.zeros((0, self.D))
        return P.attend(O.widen(self.q[b]), self.g.astype(np.float64), rows, len(slots), self.sink.astype(np.float64), p,
                        self.D ** -0.5, self.R, BASE, EPS)

    def check(self, slots=None, weights=None):
        got = f64(self.out)
        for b in range(self.B):
            out, w, b_out, b_w = self.ref(b, None if slots is None else slots[b])
            off = np.abs(got[b] - out)
            assert (off <= b_out).all(), f"sequence {b} (n {self.lens[b]}): {np.max(off - b_out):.3g} over the bound"
            assert C.max_abs_rel(got[b], out) < C.OUT_TOL
            if weights is not None:
                gw = f64(weights)[b]
                n = self.lens[b]
                assert (np.abs(gw[:n] - w) <= b_w).all(), f"weights of sequence {b}"
                assert (gw[n:] == 7.0).all(), "slots behind the last entry were written"


SHAPES = [dict(), dict(H=16), dict(H=128), dict(H=3), dict(R=0), dict(D=96, R=32, H=5, W=7), dict(D=8, R=2, H=2, W=4),
          dict(D=128, R=64, H=9, W=0)]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("page", [1, 16, 100])
def test_attend_lengths(shape, page):
    # nothing, one entry, around tile and page borders, several tiles
    lens = [0, 1, 31, 32, 33, 95, 96, 97, 100, 128, 129, 300]
    c = Case(f"len{shape}.{page}", lens, page, m=16, **SHAPES[shape])
    w = torch.full((c.B, 301), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(weights=w)
    check_ok()
    c.check(weights=w)


@pytest.mark.parametrize("fp8", [False, True])
def test_attend_one_long_sequence(fp8):
    c = Case("long", [5000], 64, fp8=fp8)
    w = torch.full((1, 5000), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(weights=w)
    check_ok()
    c.check(weights=w)


@pytest.mark.parametrize("H", [64, 20])
def test_attend_fp8_ragged(H):
    c = Case("fp8r", [700, 0, 1, 97, 1300, 64], 48, H=H, fp8=True)
    w = torch.full((c.B, 1300), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(weights=w)
    check_ok()
    c.check(weights=w)


def test_attend_fp8_small_shape():
    c = Case("fp8s", [40, 3], 7, H=4, D=96, R=32, W=5, m=4, fp8=True)
    c.run()
    check_ok()
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_attend_selected(fp8):
    # a packed row, one with fewer entries than k, one without any, and -1 among them
    lens = [2000, 300, 0, 700]
    c = Case("sel", lens, 48, m=4, fp8=fp8)
    rng = np.random.default_rng(5)
    idx = np.full((4, 512), -1, np.int32)
    sel = [np.sort(rng.choice(2000, 512, replace=False)), np.arange(300), np.zeros(0, int), np.sort(rng.choice(700, 90, replace=False))]
    for b, s in enumerate(sel):
        idx[b, :len(s)] = s
    idx[3, 10] = -1
    sel[3] = np.delete(sel[3], 10)
    c.run(idx=i32(idx))
    check_ok()
    c.check(slots=sel)


def test_attend_many_sequences():
    # more sequences than a warp and than blocks: the schedule's sums
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 40, 333)]
    c = Case("many", lens, 16, H=64, W=3, m=8)
    c.run()
    check_ok()
    c.check()


def test_attend_after_eviction_and_long_positions():
    # positions near 2^20 with most entries evicted; a ring longer than the window
    c = Case("drop", [50, 7], 16, drop=[8000, 8100], win_cap=200)
    c.run()
    check_ok()
    c.check()


def test_attend_largest_position_and_far_pages():
    # the last position that 32 bits hold; rows behind 2^31 bytes of pages
    D, page = 512, 1024
    n_pages = 2100
    pages = torch.zeros((n_pages, page, D), dtype=torch.bfloat16, device="cuda")
    row = host.normal_bf16(SEED, "far", (2, D))
    pages[n_pages - 1, 5:7] = bf(row)
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    cfg = layer(W=1, m=128)
    pos = 2 ** 31 - 1
    drop = (pos + 1) // 128 - 7
    win = host.normal_bf16(SEED, "farw", (1, 1, D))
    q = host.normal_bf16(SEED, "farq", (1, 64, D))
    out = torch.zeros((1, 64, D), dtype=torch.bfloat16, device="cuda")
    kv = L.paged_kv(pages, table, page)
    ws = torch.empty(L.ds4a_paged_attend_workspace(cfg, kv, 1), dtype=torch.uint8, device="cuda")
    sink = np.zeros(64, np.float32)
    L.ds4a_paged_attend(cfg, kv, i32([pos]), bf(q), f32(np.ones(D)), bf(win), 1, f32(sink), out, ws, drop=i32([drop]))
    check_ok()
    rows = np.concatenate([np.zeros((5, D)), O.widen(row), O.widen(win[0])])
    ref, _, bound, _ = P.attend(O.widen(q[0]), np.ones(D), rows, 7, sink.astype(np.float64), pos, D ** -0.5, 64, BASE, EPS)
    assert (np.abs(f64(out)[0] - ref) <= bound).all()


def test_attend_no_keys_and_bad_position():
    c = Case("none", [0, 3, 5], 16, W=0, m=4)
    c.d_pos[2] = -1
    c.run()
    rc, b = L.ds4a_check()
    assert rc == L.DS4A_EDEVICE and b == 2
    got = f64(c.out)
    assert (got[0] == 0).all(), "no keys: nothing but the sink"
    assert (got[2] == 7.0).all(), "a bad position's output is left as it was"
    out, _, bound, _ = c.ref(1)
    assert (np.abs(got[1] - out) <= bound).all()


def test_attend_bad_pages_and_indices_are_skipped():
    c = Case("bad", [40, 40], 16, m=4)
    c.d_table[0, 1] = 1 << 30  # slots 16..31 of sequence 0
    c.d_table[1, 0] = -1       # slots 0..15 of sequence 1
    c.run()
    rc, b = L.ds4a_check()
    assert rc == L.DS4A_EDEVICE and b == 1
    c.check(slots=[np.r_[0:16, 32:40], np.r_[16:40]])
    c = Case("bad2", [40], 16, m=4)
    idx = np.full((1, 512), -1, np.int32)
    idx[0, :5] = [3, 8, 40, 1 << 30, -7]
    c.run(idx=i32(idx))
    rc, b = L.ds4a_check()
    assert rc == L.DS4A_EDEVICE and b == 1
    c.check(slots=[np.array([3, 8])])


def test_attend_large_logits_and_sinks():
    # one head dominated by its sink, rows of widely different size
    c = Case("big", [200], 16)
    pg = c.pages_np.copy()
    s = np.arange(200)
    rows = O.widen(pg[c.table[0][s // 16], s % 16]) * np.where(s % 50 == 7, 30.0, 1.0)[:, None]
    pg[c.table[0][s // 16], s % 16] = O.store_bf16(rows)
    c.pages_np = pg
    c.pages.copy_(bf(pg))
    c.sink[0], c.sink[1] = 80.0, -80.0
    c.d_sink.copy_(f32(c.sink))
    c.run()
    check_ok()
    out, _, bound, _ = c.ref(0)
    assert (np.abs(f64(c.out)[0] - out) <= bound).all()


def test_attend_table_rows_apart_and_weights_rows_apart():
    c = Case("apart", [60, 90], 16, m=4)
    wide = torch.full((2, 40), -5, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.d_table
    c.kv = L.paged_kv(c.pages, wide[:, :c.table.shape[1]], 16)
    buf = torch.full((2, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(weights=buf[:, :100])
    check_ok()
    c.check(weights=buf)


def test_attend_weights_shorter_than_the_cache():
    c = Case("short", [60], 16, m=4)
    w = torch.full((1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(weights=w[:, :50])
    rc, b = L.ds4a_check()
    assert rc == L.DS4A_EDEVICE and b == 1
    assert (f64(w)[0, 50:] == 7.0).all() and (f64(w)[0, :50] != 7.0).all()


def test_attend_same_bits_streams_and_graph():
    """Twice the same bits; two calls at once on two streams with a workspace
    each; a captured call that serves later positions."""
    a, c = Case("sa", [900, 20], 32, m=16), Case("sb", [33, 1500], 64, m=16)
    a.run(), c.run()
    check_ok()
    first = bits(a.out).copy(), bits(c.out).copy()
    a.check(), c.check()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wc = a.workspace(), c.workspace()
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(ws=wa, stream=s1)
        c.run(ws=wc, stream=s2)
    torch.cuda.synchronize()
    assert np.array_equal(bits(a.out), first[0]) and np.array_equal(bits(c.out), first[1])
    long = Case("sg", [700, 400], 32, m=16)
    ws = long.workspace()
    graph = torch.cuda.CUDAGraph()
    final = long.pos.copy()
    with torch.cuda.graph(graph):
        long.run(ws=ws)
    for lens in ([3, 0], [250, 399], [700, 400]):
        long.lens = lens
        long.pos = np.asarray([n * 16 + 3 for n in lens], np.int32) if lens != [700, 400] else final
        long.d_pos.copy_(i32(long.pos))
        graph.replay()
        torch.cuda.synchronize()
        check_ok()
        long.check()


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def _evict_case(name, lens, n_slots, budget, recent, page, m=4, acc=None, entry=None, drop=None, weights=True, fp8=False,
                steps=1):
    B = len(lens)
    rng = np.random.default_rng(sum(map(ord, name)))
    D = 512
    cfg = layer(m=m)
    per = -(-n_slots // page)
    n_pages = B * per + 2
    table = rng.permutation(n_pages)[:B * per].reshape(B, per).astype(np.int32)
    width = 592 if fp8 else D
    pages = rng.integers(0, 60000, (n_pages, page, width)).astype(np.uint16)
    d_pages = torch.from_numpy((pages & 255).astype(np.uint8)).cuda() if fp8 else bf(pages)
    if fp8:
        pages = pages & 255
    drop = np.zeros(B, np.int32) if drop is None else np.asarray(drop, np.int32)
    acc = (rng.random((B, n_slots)) * 5).astype(np.float32) if acc is None else np.broadcast_to(acc, (B, n_slots)).astype(np.float32).copy()
    entry = np.full((B, n_slots), -1, np.int32) if entry is None else entry
    w_bits = host.normal_bf16(SEED, name + ".w", (B, n_slots)) & 0x7FFF
    pos = np.asarray([(int(d) + n) * m + 1 for d, n in zip(drop, lens)], np.int32)
    kv_table = i32(table)
    kv = L.paged_kv(d_pages, kv_table, page, fmt=L.DS4A_MX_KV_FP8 if fp8 else 0)
    d_acc, d_entry, d_drop = f32(acc), i32(entry), i32(drop)
    ws = torch.full((L.ds4a_paged_evict_workspace(kv, B),), 0xFF, dtype=torch.uint8, device="cuda")
    d_w = bf(w_bits) if weights else None
    for _ in range(steps):
        L.ds4a_paged_evict(cfg, kv, i32(pos), budget, recent, d_acc, d_entry, d_drop, ws, weights=d_w)
        check_ok()
        for b, n in enumerate(lens):
            closed = (int(pos[b]) + 1) // m
            used = max(0, min(closed - int(drop[b]), n_slots))
            acc[b], entry[b], drop[b], moves = P.evict(O.widen(w_bits[b]) if weights else None, acc[b], entry[b],
                                                       int(drop[b]), used, closed, budget, recent)
            before = pages.copy()
            for fr, to in moves:
                pages[table[b][to // page], to % page] = before[table[b][fr // page], fr % page]
        got = d_pages.cpu().numpy().astype(np.uint16) if fp8 else bits(d_pages)
        assert np.array_equal(d_drop.cpu().numpy(), drop)
        assert np.array_equal(d_entry.cpu().numpy(), entry)
        assert np.array_equal(d_acc.cpu().numpy(), acc, equal_nan=True)
        assert np.array_equal(got, pages)
        pos = pos + 5 * m  # five more entries close before the next step


@pytest.mark.parametrize("page", [1, 16, 100])
@pytest.mark.parametrize("recent", [0, 3, 20])
def test_evict_lengths(page, recent):
    _evict_case(f"el{page}.{recent}", [0, 1, 19, 20, 21, 22, 39, 40, 64], 64, 20, recent, page)


def test_evict_long_and_fp8():
    _evict_case("elong", [5000, 4097, 4095], 5003, 4096, 100, 64)
    _evict_case("elong8", [3000, 1500], 3000, 1400, 1400, 48, fp8=True)


def test_evict_very_long():
    # more keys than shared memory would hold
    _evict_case("evl", [70000, 66000], 70000, 65000, 1000, 256)


def test_evict_ties_and_special_values():
    _evict_case("tie", [50, 33], 50, 17, 0, 16, acc=np.float32(1.0), weights=False)
    odd = np.ones(50, np.float32)
    odd[[3, 40]] = np.nan
    odd[[5, 41]] = np.inf
    odd[[7, 8]] = -np.inf
    odd[[9, 42]] = -0.0
    odd[[10, 43]] = 0.0
    odd[[11, 44]] = -1e-42
    for budget in (1, 4, 44, 45, 46, 47, 49):
        _evict_case(f"odd{budget}", [50], 50, budget, 0, 16, acc=odd, weights=False)


def test_evict_steps_keep_numbers():
    # entries keep their numbers over several evictions, and protect by them
    _evict_case("steps", [30, 22, 9], 40, 20, 6, 16, steps=6)


def test_evict_whole_cache_replaced():
    # every old entry goes: all of the kept ones move
    acc = np.concatenate([np.zeros(40), np.full(40, 9.0)]).astype(np.float32)
    _evict_case("swap", [80, 80], 80, 40, 40, 16, acc=acc)


def test_evict_bad_position_and_captured():
    B, n, page, D = 2, 40, 16, 512
    cfg = layer(m=4)
    pages = bf(host.normal_bf16(SEED, "ecap", (8, page, D)))
    table = i32(np.arange(6).reshape(2, 3))
    kv = L.paged_kv(pages, table, page)
    acc = f32(np.random.default_rng(1).random((B, n)))
    start = acc.clone(), pages.clone()
    entry = torch.full((B, n), -1, dtype=torch.int32, device="cuda")
    drop, pos = i32([0, 0]), i32([-1, 160])
    ws = torch.empty(L.ds4a_paged_evict_workspace(kv, B), dtype=torch.uint8, device="cuda")
    L.ds4a_paged_evict(cfg, kv, pos, 30, 4, acc, entry, drop, ws)
    rc, b = L.ds4a_check()
    assert rc == L.DS4A_EDEVICE and b == 2
    assert drop.tolist() == [0, 10] and torch.equal(acc[0], start[0][0]) and (entry[0] == -1).all()
    done = acc.clone(), entry.clone(), pages.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.ds4a_paged_evict(cfg, kv, pos, 30, 4, acc, entry, drop, ws)
    acc.copy_(start[0]), pages.copy_(start[1]), entry.fill_(-1), drop.zero_(), pos.copy_(i32([3, 160]))
    graph.replay()
    torch.cuda.synchronize()
    check_ok()
    assert drop.tolist() == [0, 10] and torch.equal(acc[1], done[0][1]) and torch.equal(entry[1], done[1][1])
    assert torch.equal(pages, done[2])


# ---------------------------------------------------------------------------
# append, and the operators one after another
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fp8,overlap,D,R", [(False, False, 512, 64), (True, False, 512, 64), (False, True, 512, 64),
                                             (True, True, 512, 64), (False, False, 96, 32), (False, True, 96, 32)])
def test_append_matches_contiguous(fp8, overlap, D, R):
    """Token by token into pages, beside the contiguous call: the same rows."""
    m, B, T, page = 4, 3, 23, 3
    cfg = layer(D=D, R=R, m=m)
    n_cap = T // m + 1
    rb = L.ds4a_kv_fp8_row_bytes(D, R) if fp8 else D
    drop = [0, 2, 0]
    per = 3
    n_pages = B * per + 1
    table = np.random.default_rng(2).permutation(n_pages)[:B * per].reshape(B, per).astype(np.int32)
    d_table, d_drop = i32(table), i32(drop)
    dt = torch.uint8 if fp8 else torch.bfloat16
    pages = torch.full((n_pages, page, rb), 99, dtype=dt, device="cuda")
    pool = torch.zeros((B, n_cap, rb), dtype=dt, device="cuda")
    kv = L.paged_kv(pages, d_table, page, fmt=L.DS4A_MX_KV_FP8 if fp8 else 0)
    nb = L.ds4a_compress_state_bytes(cfg, B, D, overlap)
    st1 = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    st2 = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    mk = lambda n, sh: host.normal_bf16(SEED, f"app{fp8}{overlap}{D}.{n}", sh)  # noqa: E731
    X = {k: bf(mk(k, (T, B, D))) for k in ("ca", "za", "cb", "zb")}
    ba, bb = f32(0.5 * host.normal_f32(SEED, "app.ba", (m, D))), f32(0.5 * host.normal_f32(SEED, "app.bb", (m, D)))
    g = f32(1 + 0.1 * host.normal_f32(SEED, "app.g", (D,)))
    for t in range(T):
        pos = i32([t] * B)
        more = dict(cb=X["cb"][t], zb=X["zb"][t], bias_b=bb) if overlap else {}
        if fp8:
            L.ds4a_compress_append_mx(cfg, pos, X["ca"][t], X["za"][t], ba, st1, L.DS4A_MX_KV_FP8, pool, norm_g=g, **more)
        else:
            L.ds4a_compress_append(cfg, pos, X["ca"][t], X["za"][t], ba, st1, pool, norm_g=g, **more)
        L.ds4a_paged_append(cfg, kv, pos, X["ca"][t], X["za"][t], ba, st2, drop=d_drop, norm_g=g, **more)
    # sequence 1's first two entries have no slot (evicted before they came): recorded
    rc, bts = L.ds4a_check()
    assert rc == L.DS4A_EDEVICE and bts == 1
    got, want = pages.cpu(), pool.cpu()
    for b in range(B):
        for i in range(T // m):
            s = i - drop[b]
            if s >= 0:
                assert torch.equal(got[table[b][s // page], s % page], want[b, i]), (b, i)
    assert torch.equal(st1, st2)
    used = {(int(table[b][(i - drop[b]) // page]), (i - drop[b]) % page) for b in range(B) for i in range(drop[b], T // m)}
    for p in range(n_pages):
        for r in range(page):
            if (p, r) not in used:
                assert (got[p, r] == 99).all(), "a row that no entry owns was written"


def test_append_past_the_table_is_recorded():
    cfg = layer(m=1)
    pages = torch.zeros((2, 2, 512), dtype=torch.bfloat16, device="cuda")
    table = i32([[1]])
    kv = L.paged_kv(pages, table, 2)
    state = torch.zeros(L.ds4a_compress_state_bytes(cfg, 1, 512, False), dtype=torch.uint8, device="cuda")
    x = bf(host.normal_bf16(SEED, "past", (1, 512)))
    for p, want in ((0, L.DS4A_OK), (1, L.DS4A_OK), (2, L.DS4A_EDEVICE)):
        L.ds4a_paged_append(cfg, kv, i32([p]), x, x, f32(np.zeros((1, 512))), state)
        assert L.ds4a_check()[0] == want
    assert (pages[0] == 0).all() and (pages[1] != 0).any(-1).all()


def test_decode_with_a_bounded_cache():
    """A dense layer decodes with a cache of 12 entries: append, attend with
    weights, evict, project.  Each step is checked on the state it begins
    with; the entries by their numbers, whose rows never change."""
    B, m, page, budget, recent, slots = 3, 4, 5, 12, 4, 15
    c = Case("loop", [0] * B, page, m=m, spare=2)
    D, H = 512, 64
    cfg = c.cfg
    oc = L.OprojCfg(H, D, 8, 256, 512)
    k1, n1 = 8 * D, 8 * 256
    wts = {}
    for name, (n, k) in dict(a=(n1, k1), b=(512, n1)).items():
        src = bf(host.normal_bf16(SEED, "loop.w" + name, (n, k), 1 / math.sqrt(k)))
        codes = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
        sc = torch.empty(L.ds4a_mxfp4_scale_bytes(n, k), dtype=torch.uint8, device="cuda")
        L.ds4a_quantize_mxfp4(src, codes, sc)
        wts[name] = codes, sc
    state = torch.zeros(L.ds4a_compress_state_bytes(cfg, B, D, False), dtype=torch.uint8, device="cuda")
    acc = torch.zeros((B, slots), dtype=torch.float32, device="cuda")
    entry = torch.full((B, slots), -1, dtype=torch.int32, device="cuda")
    drop = torch.zeros(B, dtype=torch.int32, device="cuda")
    w = torch.zeros((B, slots), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((B, 512), dtype=torch.bfloat16, device="cuda")
    c.d_drop = drop
    T = 90
    ca, za = host.normal_bf16(SEED, "loop.ca", (B, T, D)), host.normal_bf16(SEED, "loop.za", (B, T, D))
    ba = (0.5 * host.normal_f32(SEED, "loop.ba", (m, D))).astype(np.float32)
    g = (1 + 0.1 * host.normal_f32(SEED, "loop.g", (D,))).astype(np.float32)
    d_ca, d_za, d_ba, d_g = bf(ca), bf(za), f32(ba), f32(g)
    want = O.store_bf16(O.compress_batch(m, 0, T // m, 0, ca, za, ba.astype(np.float64), norm_g=g.astype(np.float64), rope_dim=64))
    ws = c.workspace(weights=True)
    ews = torch.empty(L.ds4a_paged_evict_workspace(c.kv, B), dtype=torch.uint8, device="cuda")
    ows = torch.empty(L.ds4a_out_proj_mxfp4_workspace(oc, B), dtype=torch.uint8, device="cuda")
    n_acc, n_entry, n_drop = np.zeros((B, slots), np.float32), np.full((B, slots), -1, np.int32), np.zeros(B, np.int64)
    evicted = 0
    for t in range(T):
        c.pos[:] = t
        c.d_pos.copy_(i32(c.pos))
        L.ds4a_paged_append(cfg, c.kv, c.d_pos, d_ca[:, t].contiguous(), d_za[:, t].contiguous(), d_ba, state, drop=drop, norm_g=d_g)
        c.run(weights=w, ws=ws)
        L.ds4a_paged_evict(cfg, c.kv, c.d_pos, budget, recent, acc, entry, drop, ews, weights=w)
        L.ds4a_out_proj_mxfp4(oc, c.out, *wts["a"], *wts["b"], y, ows)
        check_ok()
        closed = (t + 1) // m
        gw = f64(w)
        for b in range(B):
            n = closed - int(n_drop[b])
            if t % 13 == 5 or t > T - 4:
                num = np.where(n_entry[b, :n] < 0, np.arange(n) + n_drop[b], n_entry[b, :n])
                near = np.arange(max(0, t - 127), t + 1) % 128
                rows = np.concatenate([O.widen(want[b][num]), O.widen(c.win[b][near])])
                out, wr, b_out, b_w = P.attend(O.widen(c.q[b]), c.g.astype(np.float64), rows, n, c.sink.astype(np.float64), t,
                                               D ** -0.5, 64, BASE, EPS, key_off=2 * P.U16)
                # (key_off: an entry near a tie may round to the neighbour of the oracle's)
                assert (np.abs(f64(c.out)[b] - out) <= b_out).all(), (t, b)
                assert (np.abs(gw[b, :n] - wr) <= b_w).all(), (t, b)
            a, e, d, moves = P.evict(gw[b].astype(np.float32), n_acc[b], n_entry[b], int(n_drop[b]), n, closed, budget, recent)
            n_acc[b], n_entry[b], n_drop[b] = a, e, d
            evicted += closed > budget and (t + 1) % m == 0
        assert np.array_equal(drop.cpu().numpy(), n_drop)
        assert np.array_equal(entry.cpu().numpy(), n_entry)
        assert np.array_equal(acc.cpu().numpy(), n_acc)
    assert evicted > 20
    assert torch.isfinite(y.float()).all()
