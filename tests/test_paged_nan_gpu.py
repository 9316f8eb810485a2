"""NaN and infinity in what decode attention over the paged cache reads: they
must show in exactly the outputs that they reach, however a batch is spread
over the GPU."""
import numpy as np
import pytest
import torch

import long_context_hybrid_kv_b200 as L
from gpu_util import bf, check_ok, f32
from test_paged_gpu import Case

pytestmark = pytest.mark.gpu

NAN, INF = 0x7FC0, 0x7F80  # bf16

# finished in one block; cut into pieces of a block each (of few and of many
# segments); the row of all tiles cut into ranges; whole items that share blocks
SPREADS = {"whole": [100, 30], "pieces": [5000, 300], "few pieces": [700] * 40, "ranges": [400] * 152,
           "shared": [120] * 300}
KINDS = {"bf16": dict(H=5), "fp8": dict(H=5, fp8=True), "two groups": dict(H=70),
         "generic": dict(H=3, D=64, R=16, W=8)}


def twice(name, lens, change, **kw):
    """The outputs before and after change(case, sequence): (out, weights) each."""
    c = Case(name, lens, 64, m=16, spare=0, **kw)
    w = torch.full((c.B, max(lens)), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = c.workspace(weights=True)
    got = []
    for i in range(2):
        if i:
            change(c)
        c.out.fill_(7.0), w.fill_(7.0)
        c.run(weights=w, ws=ws)
        check_ok()
        got.append((c.out.clone(), w.clone()))
    return c, got[0], got[1]


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def reached(c, first, then, b, heads):
    """Sequence b's outputs of `heads` and its slots' weights are NaN, all else has the same bits."""
    hit = torch.zeros((c.B, c.H), dtype=torch.bool, device="cuda")
    hit[b, heads] = True
    assert torch.isnan(then[0][hit]).all(), "outputs that are not NaN"
    assert same(first[0][~hit], then[0][~hit]), "other outputs changed"
    assert torch.isfinite(first[0]).all()
    slots = torch.zeros((c.B, then[1].shape[1]), dtype=torch.bool, device="cuda")
    slots[b, :c.lens[b]] = True
    assert torch.isnan(then[1][slots]).all(), "weights that are not NaN"
    assert same(first[1][~slots], then[1][~slots]), "other weights changed"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spread", SPREADS)
def test_nan_in_a_query(kind, spread):
    nan_query(kind, spread, NAN)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spread", ["whole", "pieces"])
def test_infinity_in_a_query(kind, spread):
    # (its root mean square is infinite: infinity times 0)
    nan_query(kind, spread, INF)


def nan_query(kind, spread, value):
    lens = SPREADS[spread]
    b, h = len(lens) // 2 - 1, KINDS[kind]["H"] - 1

    def change(c):
        c.d_q.view(torch.int16)[b, h, 6] = value

    c, first, then = twice(f"nq{kind}{spread}", lens, change, **KINDS[kind])
    reached(c, first, then, b, [h])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("all_rows", [False, True])
def test_nan_in_rows_in_use(kind, spread, all_rows):
    """One row of a sequence, or all of its cache's (pieces then hold nothing else)."""
    lens = SPREADS[spread]
    b = len(lens) // 2 - 1

    def change(c):
        n = c.lens[b]
        s = torch.arange(n, device="cuda") if all_rows else torch.tensor([n // 3], device="cuda")
        at = c.d_table[b].long()[s // 64], s % 64
        if c.fp8:
            c.pages[at[0], at[1], 3] = 0x7F  # the code of NaN
        else:
            c.pages.view(torch.int16)[at[0], at[1], 3] = NAN

    c, first, then = twice(f"nr{kind}{spread}{all_rows}", lens, change, **KINDS[kind])
    reached(c, first, then, b, list(range(c.H)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spread", SPREADS)
def test_nan_in_a_sink(kind, spread):
    h = KINDS[kind]["H"] - 2

    def change(c):
        c.d_sink[h] = float("nan")

    c, first, then = twice(f"ns{kind}{spread}", SPREADS[spread], change, **KINDS[kind])
    assert torch.isnan(then[0][:, h]).all()
    keep = [i for i in range(c.H) if i != h]
    assert same(first[0][:, keep], then[0][:, keep])
    for b, n in enumerate(c.lens):
        assert torch.isnan(then[1][b, :n]).all() and same(first[1][b, n:], then[1][b, n:])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens", [[40], [3000]])
def test_sinks_of_minus_infinity(kind, lens):
    """No sink at all; then no key either (every page is bad): zeros, no NaN."""
    c = Case(f"mi{kind}", lens, 64, m=16, spare=0, **{**KINDS[kind], "W": 0})
    c.sink[:] = -np.inf
    c.d_sink.copy_(f32(c.sink))
    w = torch.full((c.B, max(lens) + 1), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(weights=w)
    check_ok()
    c.check(weights=w)
    c.d_table.fill_(-1)
    c.run(weights=w)
    rc, bits = L.ds4a_check()
    assert rc == L.DS4A_EDEVICE and bits == 1
    assert (c.out == 0).all() and (w[:, :lens[0]] == 0).all() and (w[:, lens[0]:] == 7.0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spread", ["whole", "pieces", "ranges"])
@pytest.mark.parametrize("which", ["one", "front"])
@pytest.mark.filterwarnings("ignore:invalid value")
def test_infinity_in_rows_in_use(kind, spread, which):
    """Logits of plus and of minus infinity: NaN where the plain form has it (the
    weights are those of the heads that are there)."""
    lens = SPREADS[spread]
    b = len(lens) // 2 - 1

    def change(c):
        n, d = c.lens[b], c.D - c.R + 4  # (a dim that FP8 rows hold in bf16)
        s = dict(one=np.array([n // 3]), front=np.arange(n // 2))[which]
        at = c.table[b][s // 64], s % 64
        if c.fp8:
            c.pages_np[at[0], at[1], c.D - c.R + 8] = INF & 255
            c.pages_np[at[0], at[1], c.D - c.R + 9] = INF >> 8
            c.pages.copy_(torch.from_numpy(c.pages_np))
        else:
            c.pages_np[at[0], at[1], d] = INF
            c.pages.copy_(bf(c.pages_np))

    c, first, then = twice(f"ir{kind}{spread}{which}", lens, change, **KINDS[kind])
    out, w, _, _ = c.ref(b)
    nan = np.isnan(out)
    assert nan.any()
    assert np.array_equal(torch.isnan(then[0][b]).cpu().numpy(), nan)
    assert np.array_equal(torch.isnan(then[1][b, :lens[b]]).cpu().numpy(), np.isnan(w))
    keep = [i for i in range(c.B) if i != b]
    assert same(first[0][keep], then[0][keep]) and same(first[1][keep], then[1][keep])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.filterwarnings("ignore:invalid value")
def test_infinity_in_all_rows_of_a_piece(kind):
    """The first piece of a cut sequence, one tile: logits of minus infinity
    give it no weight, but 0 times infinity is NaN."""
    c = Case(f"ip{kind}", [5000], 64, m=16, spare=0, **KINDS[kind])
    s, d = np.arange(32 if kind == "generic" else 64), c.D - c.R + 4
    at = c.table[0][s // 64], s % 64
    if c.fp8:
        c.pages_np[at[0], at[1], c.D - c.R + 8] = INF & 255
        c.pages_np[at[0], at[1], c.D - c.R + 9] = INF >> 8
        c.pages.copy_(torch.from_numpy(c.pages_np))
    else:
        c.pages_np[at[0], at[1], d] = INF
        c.pages.copy_(bf(c.pages_np))
    c.q[0, 1] = c.q[0, 0] ^ 0x8000  # heads of either sign
    c.d_q.copy_(bf(c.q))
    c.run()
    check_ok()
    out, _, _, _ = c.ref(0)
    nan = np.isnan(out)
    assert nan.any() and not nan.all()
    assert np.array_equal(torch.isnan(c.out[0]).cpu().numpy(), nan)
