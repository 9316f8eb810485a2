"""Measured cases of the serving operators of a decode step: attention of one
new token per sequence over a paged K=V cache, eviction from that cache by
accumulated attention weight, and the grouped output projection in
microscaled 4-bit floating point.

`run` computes each operator in its plain form (elementary torch operations in
32 bits) or, with `own` set, calls the library's entry points.  A case is a
dict of plain values; `prepare` makes its inputs on the GPU from the seed.

The cache: pages of `page` rows of 512 (bf16, or FP8 codes with bf16 RoPE dims
in 592-byte rows), a table of physical pages for each sequence, and a window
ring of the last 128 raw rows.  A sequence at position p has closed
(p + 1) // ratio compressed entries; `drop` of them have been evicted, the
others lie in the slots 0, 1, ... of its pages.
"""
import math

import torch

own = False

D, R, WINDOW, BASE, EPS = 512, 64, 128, 10000.0, 1e-6
ROW8 = 592  # FP8 row: 448 codes, 64 bf16, 14 scale bytes, 2 zero bytes
DEV = "cuda" if torch.cuda.is_available() else "cpu"

ATTEND, EVICT, PROJ = "attend", "evict", "proj"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _attend(name, B, n, page, ratio=128, ragged=False, fp8=False, sparse=0, weights=False, heads=64):
    c = dict(op=ATTEND, B=B, n=n, page=page, ratio=ratio, ragged=ragged, fp8=fp8, sparse=sparse, weights=weights,
             heads=heads)
    return dict(c, name=name) if name else c


def _evict(name, B, budget, extra, page, recent, fp8=False, ratio=4):
    c = dict(op=EVICT, B=B, budget=budget, extra=extra, page=page, recent=recent, fp8=fp8, ratio=ratio)
    return dict(c, name=name) if name else c


def _proj(name, M, heads=64, dim=512, groups=8, rank=1024, hidden=4096):
    c = dict(op=PROJ, M=M, heads=heads, dim=dim, groups=groups, rank=rank, hidden=hidden)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user at an 8k context, HCA layer: 64 entries and the window; latency is all
        _attend("attend_b1_ctx8k", 1, 64, 16),
        # one user at a 1M context, HCA layer: one long sequence split over the GPU
        _attend("attend_b1_ctx1m", 1, 8192, 64),
        # a decode batch at a 128k context, HCA layer
        _attend("attend_b32_ctx128k", 32, 1024, 64),
        # the CSA layer of a decode batch: 512 selected entries scattered over the pages
        _attend("attend_csa_b24", 24, 16000, 48, ratio=4, sparse=512),
        # sequences of very different lengths in one batch, FP8 rows
        _attend("attend_fp8_ragged_b61", 61, 8000, 100, ragged=True, fp8=True),
        # a large batch at a 1M context with the attention weights that the eviction reads
        _attend("attend_weights_b48_ctx1m", 48, 8192, 128, weights=True),
        # steady state of a bounded cache: one entry came, one goes
        _evict("evict_one_b32", 32, 1023, 1, 64, 32, ratio=128),
        # after a chunk of a prompt: thousands of entries go at once; FP8 rows
        _evict("evict_chunk_fp8_b8", 8, 4096, 3500, 100, 256, fp8=True),
        # a large batch whose caches are halved
        _evict("evict_half_b32", 32, 16384, 16384, 256, 1024),
        # one token through the projection: the weights stream past
        _proj("proj_m1", 1),
        # a decode batch with an odd number of rows
        _proj("proj_m77", 77),
        # a 16k-token prompt
        _proj("proj_m16k", 16384),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice([ATTEND, ATTEND, EVICT, PROJ])
    if op == ATTEND:
        sparse = rng.random() < 0.3
        n = _log(rng, 1, 32768 if sparse else 8192)
        B = _log(rng, 1, 48)
        weights = not sparse and rng.random() < 0.4
        return _attend(None, B, n, rng.choice([16, 32, 48, 64, 100, 128, 256]), ratio=4 if sparse else 128,
                       ragged=rng.random() < 0.5, fp8=rng.random() < 0.35, sparse=512 if sparse else 0,
                       weights=weights, heads=rng.choice([64, 64, 64, 32, 16]))
    if op == EVICT:
        budget = _log(rng, 8, 16384)
        return _evict(None, _log(rng, 1, 32), budget, _log(rng, 1, budget), rng.choice([16, 48, 64, 100, 256]),
                      rng.randint(0, budget // 4), fp8=rng.random() < 0.4)
    M = _log(rng, 1, 16384)
    if rng.random() < 0.25:
        return _proj(None, M, 16, 128, 4, 256, 1024)
    return _proj(None, M)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _lengths(c):
    """Entries of each sequence: all n, or spread from 0 to n (by the case alone)."""
    if not c["ragged"]:
        return [c["n"]] * c["B"]
    return [c["n"] if b == 0 else int(c["n"] * ((b * 0.6180339887) % 1.0) ** 2) for b in range(c["B"])]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _big_normal(g, rows, width):
    out = torch.empty((rows, width), dtype=torch.bfloat16, device=DEV)
    for r0 in range(0, rows, 1 << 18):
        r1 = min(rows, r0 + (1 << 18))
        out[r0:r1] = _normal(g, (r1 - r0, width))
    return out


def _scale_exp(amax, largest_frac, largest_exp):
    """Smallest s with amax <= largest * 2^s, largest = frac * 2^exp."""
    f, e = torch.frexp(amax)
    s = e - largest_exp + (f > largest_frac).to(e.dtype)
    return torch.where(amax > 0, s, torch.full_like(s, -127)).clamp(-127, 127)


def _pow2(s, dtype=torch.float32):
    return torch.ldexp(torch.ones(s.shape, dtype=dtype, device=s.device), s.to(torch.int32))


def _fp8_rows(rows):
    """bf16 rows [n, 512] -> uint8 [n, 592]."""
    n = rows.shape[0]
    out = torch.zeros((n, ROW8), dtype=torch.uint8, device=rows.device)
    for r0 in range(0, n, 1 << 18):
        x = rows[r0:r0 + (1 << 18)]
        blk = x[:, :D - R].float().reshape(-1, (D - R) // 32, 32)
        s = _scale_exp(blk.abs().amax(-1), 0.875, 9)
        q = (blk * _pow2(-s).unsqueeze(-1)).to(torch.float8_e4m3fn)
        o = out[r0:r0 + (1 << 18)]
        o[:, :D - R] = q.reshape(-1, D - R).view(torch.uint8)
        o[:, D - R:D + R] = x[:, D - R:].contiguous().view(torch.uint8)
        o[:, D + R:D + R + (D - R) // 32] = (s + 127).to(torch.uint8)
    return out


def _cache(g, lens, cap, page, fp8):
    """Pages in a random physical order, and the table; pages of slots that
    no sequence fills are there too."""
    B, per = len(lens), -(-cap // page)
    n_pages = B * per + 3
    rows = _big_normal(g, n_pages * page, D)
    pages = _fp8_rows(rows) if fp8 else rows
    order = torch.randperm(n_pages, generator=g, device=DEV)[:B * per]
    return pages.view(n_pages, page, -1), order.view(B, per).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == ATTEND:
        return _prepare_attend(case, g)
    if case["op"] == EVICT:
        return _prepare_evict(case, g)
    return _prepare_proj(case, g)


def _prepare_attend(c, g):
    lens, B, H = _lengths(c), c["B"], c["heads"]
    pages, table = _cache(g, lens, max(1, c["n"]), c["page"], c["fp8"])
    n = torch.tensor(lens, dtype=torch.int64, device=DEV)
    # the new token lies somewhere in the block after the last closed entry
    pos = n * c["ratio"] + torch.randint(0, c["ratio"] - 1, (B,), generator=g, device=DEV)
    st = dict(case=c, pages=pages, table=table, n_max=max(1, c["n"]), pos=pos.to(torch.int32),
              q=_normal(g, (B, H, D)), g=1 + 0.1 * _normal(g, (D,), torch.float32), sink=_normal(g, (H,), torch.float32),
              win=_normal(g, (B, WINDOW, D)), out=torch.zeros((B, H, D), dtype=torch.bfloat16, device=DEV))
    if c["sparse"]:
        k = c["sparse"]
        key = torch.rand((B, st["n_max"]), generator=g, device=DEV)
        key = torch.where(torch.arange(st["n_max"], device=DEV) < n[:, None], key, torch.full_like(key, 2.0))
        sel = key.argsort(dim=1)[:, :k]
        ok = torch.arange(sel.shape[1], device=DEV) < n[:, None]
        sel = torch.where(ok, sel, torch.full_like(sel, 1 << 30)).sort(dim=1).values
        idx = torch.full((B, k), -1, dtype=torch.int32, device=DEV)
        idx[:, :sel.shape[1]] = torch.where(sel < (1 << 30), sel, torch.full_like(sel, -1)).to(torch.int32)
        st["idx"] = idx
    if c["weights"]:
        st["weights"] = torch.zeros((B, st["n_max"]), dtype=torch.bfloat16, device=DEV)
    return st


def _prepare_evict(c, g):
    B, cap = c["B"], c["budget"] + c["extra"]
    pages, table = _cache(g, [cap] * B, cap, c["page"], c["fp8"])
    # weights fall off as those of a softmax do: most entries get little
    acc = torch.exp(2 * torch.randn((B, cap), generator=g, device=DEV)) * (64.0 / cap)
    w = (torch.exp(2 * torch.randn((B, cap), generator=g, device=DEV)) * (8.0 / cap)).to(torch.bfloat16)
    entry = torch.full((B, cap), -1, dtype=torch.int32, device=DEV)
    acc[:, c["budget"]:] = 0
    # `extra` entries close before each call: this is the position before the first
    pos = torch.full((B,), c["budget"] * c["ratio"] - 1, dtype=torch.int32, device=DEV)
    return dict(case=c, pages=pages, table=table, acc=acc, w=w, entry=entry, pos=pos,
                drop=torch.zeros((B,), dtype=torch.int32, device=DEV))


def _tile_scales(s):
    """Scale bytes [rows, K/32] -> the product's order: blocks of 128 rows x 4
    scales, 512 bytes each (row r at (r % 32) * 16 + (r / 32) * 4), blocks of
    one row range side by side along K."""
    rows, kb = s.shape
    pad = -rows % 128
    if pad:
        s = torch.cat([s, s.new_zeros((pad, kb))])
    return s.view(-1, 4, 32, kb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(t, rows, kb):
    return t.view(-1, kb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, kb)[:rows]


def _round_e2m1(x):
    """To the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, ties to the even code; |x| <= 6."""
    a = x.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(x.dtype)
    return torch.round(x / step) * step


def _mx4(x):
    """x [..., K] -> (values on the E2M1 grid, exponents [..., K/32])."""
    blk = x.reshape(*x.shape[:-1], -1, 32)
    s = _scale_exp(blk.abs().amax(-1), 0.75, 3)
    return _round_e2m1(blk * _pow2(-s, x.dtype).unsqueeze(-1)), s


def _mx4_value(x):
    q, s = _mx4(x)
    return (q * _pow2(s, x.dtype).unsqueeze(-1)).reshape(x.shape)


def _mx4_pack(x):
    q, s = _mx4(x)
    a = (q.abs() * 2).to(torch.int64)
    code = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], device=x.device)[a] | ((q < 0).to(torch.int64) << 3)
    code = code.reshape(x.shape)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), (s + 127).to(torch.uint8)


def _mx4_unpack(codes, scales):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6.0], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(codes.shape[0], -1, 32)
    return (grid[c.to(torch.int64)] * _pow2(scales.to(torch.int32) - 127).unsqueeze(-1)).reshape(codes.shape[0], -1)


def _prepare_proj(c, g):
    k1, n1 = c["heads"] // c["groups"] * c["dim"], c["groups"] * c["rank"]
    wa, sa = _mx4_pack(_normal(g, (n1, k1), torch.float32) / math.sqrt(k1))
    wb, sb = _mx4_pack(_normal(g, (c["hidden"], n1), torch.float32) / math.sqrt(n1))
    return dict(case=c, wa=wa, sa=_tile_scales(sa), wb=wb, sb=_tile_scales(sb),
                o=_big_normal(g, c["M"], c["heads"] * c["dim"]).view(c["M"], c["heads"], c["dim"]),
                y=torch.zeros((c["M"], c["hidden"]), dtype=torch.bfloat16, device=DEV))


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == ATTEND:
        return _own_attend(state) if own else _plain_attend(state)
    if op == EVICT:
        state["pos"].add_(state["case"]["extra"] * state["case"]["ratio"])  # entries close
        return _own_evict(state) if own else _plain_evict(state)
    return _own_proj(state) if own else _plain_proj(state)


def _own_cfg(L, heads, ratio):
    return L.LayerCfg(heads, D, R, WINDOW, 64, 128, 512, ratio, D ** -0.5, BASE, EPS)


def _own_attend(st):
    import long_context_hybrid_kv_b200 as L
    c = st["case"]
    if "cfg" not in st:
        st["cfg"] = _own_cfg(L, c["heads"], c["ratio"])
        st["kv"] = L.paged_kv(st["pages"], st["table"], c["page"], fmt=L.DS4A_MX_KV_FP8 if c["fp8"] else 0)
        st["ws"] = torch.empty(L.ds4a_paged_attend_workspace(st["cfg"], st["kv"], c["B"], bool(c["sparse"]),
                                                             c["weights"]), dtype=torch.uint8, device=DEV)
    L.ds4a_paged_attend(st["cfg"], st["kv"], st["pos"], st["q"], st["g"], st["win"], WINDOW, st["sink"], st["out"],
                        st["ws"], idx=st.get("idx"), weights=st.get("weights"))
    return {k: st[k] for k in ("out", "weights") if k in st}


def _own_evict(st):
    import long_context_hybrid_kv_b200 as L
    c = st["case"]
    if "cfg" not in st:
        st["cfg"] = _own_cfg(L, 64, c["ratio"])
        st["kv"] = L.paged_kv(st["pages"], st["table"], c["page"], fmt=L.DS4A_MX_KV_FP8 if c["fp8"] else 0)
        st["ws"] = torch.empty(L.ds4a_paged_evict_workspace(st["kv"], c["B"]), dtype=torch.uint8, device=DEV)
    L.ds4a_paged_evict(st["cfg"], st["kv"], st["pos"], c["budget"], c["recent"], st["acc"], st["entry"], st["drop"],
                       st["ws"], weights=st["w"])
    return {k: st[k] for k in ("pages", "acc", "entry", "drop")}


def _own_proj(st):
    import long_context_hybrid_kv_b200 as L
    c = st["case"]
    if "cfg" not in st:
        st["cfg"] = L.OprojCfg(c["heads"], c["dim"], c["groups"], c["rank"], c["hidden"])
        st["ws"] = torch.empty(L.ds4a_out_proj_mxfp4_workspace(st["cfg"], c["M"]), dtype=torch.uint8, device=DEV)
    L.ds4a_out_proj_mxfp4(st["cfg"], st["o"], st["wa"], st["sa"], st["wb"], st["sb"], st["y"], st["ws"])
    return st["y"]


def _row_values(rows, fp8):
    if not fp8:
        return rows.float()
    q = rows[..., :D - R].contiguous().view(torch.float8_e4m3fn).float().reshape(*rows.shape[:-1], (D - R) // 32, 32)
    s = rows[..., D + R:D + R + (D - R) // 32].to(torch.int32) - 127
    low = (q * _pow2(s).unsqueeze(-1)).reshape(*rows.shape[:-1], D - R)
    return torch.cat([low, rows[..., D - R:D + R].contiguous().view(torch.bfloat16).float()], dim=-1)


def _turns(pos, sign):
    """cos and sin of the RoPE angles of positions [B], in 64 bits, as 32."""
    theta = BASE ** (-2.0 * torch.arange(R // 2, dtype=torch.float64, device=pos.device) / R)
    a = sign * pos.double()[:, None] * theta
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, pos, sign):
    co, si = _turns(pos, sign)
    a, b = x[..., D - R::2], x[..., D - R + 1::2]
    turned = torch.stack([a * co - b * si, a * si + b * co], dim=-1).flatten(-2)
    return torch.cat([x[..., :D - R], turned], dim=-1)


def _plain_attend(st):
    c = st["case"]
    pos, page, dev = st["pos"].long(), c["page"], st["pos"].device
    n = torch.div(pos + 1, c["ratio"], rounding_mode="floor").clamp(max=st["n_max"])
    if c["sparse"]:
        slot = st["idx"].long().clamp(min=0)
        live = st["idx"] >= 0
    else:
        slot = torch.arange(st["n_max"], device=dev).expand(c["B"], -1)
        live = slot < n[:, None]
    phys = st["table"].long().gather(1, torch.div(slot, page, rounding_mode="floor")) * page + slot % page
    rows = _row_values(st["pages"].view(-1, st["pages"].shape[-1])[phys], c["fp8"])
    wpos = pos[:, None] - (WINDOW - 1) + torch.arange(WINDOW, device=dev)
    wrow = st["win"].gather(1, (wpos % WINDOW)[..., None].expand(-1, -1, D)).float()
    keys = torch.cat([rows, wrow], dim=1)
    live = torch.cat([live, wpos >= 0], dim=1)
    q = st["q"].float()
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * st["g"]
    q = _rotate(q, pos, 1.0)
    z = torch.matmul(q, keys.transpose(1, 2)) * D ** -0.5
    z = z.masked_fill(~live[:, None], -math.inf)
    top = torch.maximum(z.amax(-1), st["sink"]).unsqueeze(-1)
    e = torch.exp(z - top)
    p = e / (e.sum(-1, keepdim=True) + torch.exp(st["sink"][:, None] - top))
    o = torch.matmul(p, keys)
    st["out"].copy_(_rotate(o, pos, -1.0))
    if not c["weights"]:
        return {"out": st["out"]}
    w = p[:, :, :st["n_max"]].sum(1)
    st["weights"].copy_(torch.where(live[:, :st["n_max"]], w, st["weights"].float()))
    return {"out": st["out"], "weights": st["weights"]}


def _plain_evict(st):
    c = st["case"]
    acc, entry, drop, budget, page = st["acc"], st["entry"], st["drop"], c["budget"], c["page"]
    cap, dev = acc.shape[1], acc.device
    closed = torch.div(st["pos"].long() + 1, c["ratio"], rounding_mode="floor")
    n = (closed - drop).clamp(0, cap)[:, None]
    slot = torch.arange(cap, device=dev).expand(c["B"], -1)
    there = slot < n
    total = torch.where(there, acc + st["w"].float(), acc)
    ident = torch.where(entry < 0, slot + drop[:, None], entry.long())
    newest = closed[:, None] - 1
    key = torch.where(ident > newest - c["recent"], torch.full_like(total, math.inf), total)
    key = torch.where(there, key, torch.full_like(total, -math.inf))
    order = key.sort(dim=1, descending=True, stable=True).indices
    keep = torch.zeros_like(there).scatter_(1, order[:, :budget], True)
    full = n > budget
    keep = torch.where(full, keep, there)
    hole = full & there & ~keep & (slot < budget)
    mover = full & keep & (slot >= budget)
    moves = min(budget, cap - budget)
    dst = (~hole).to(torch.int8).sort(dim=1, stable=True).indices[:, :moves]
    src = (~mover).to(torch.int8).sort(dim=1, stable=True).indices[:, :moves]
    used = slot[:, :moves] < hole.sum(1, keepdim=True)
    src = torch.where(used, src, dst)
    flat = st["pages"].view(-1, st["pages"].shape[-1])
    where_is = lambda s: st["table"].long().gather(1, torch.div(s, page, rounding_mode="floor")) * page + s % page  # noqa: E731
    flat[where_is(dst).reshape(-1)] = flat[where_is(src).reshape(-1)]
    total = total.scatter(1, dst, total.gather(1, src))
    ident = ident.scatter(1, dst, ident.gather(1, src))
    behind = full & (slot >= budget)
    acc.copy_(torch.where(behind, torch.zeros_like(total), total))
    entry.copy_(torch.where(full, torch.where(behind, -1, torch.where(there, ident, entry.long())), entry.long()))
    drop.add_((n[:, 0] - budget).clamp(min=0).to(torch.int32))
    return {k: st[k] for k in ("pages", "acc", "entry", "drop")}


def _plain_proj(st):
    c = st["case"]
    M, G, k1, n1 = c["M"], c["groups"], c["heads"] // c["groups"] * c["dim"], c["groups"] * c["rank"]
    wa = _mx4_unpack(st["wa"], _untile_scales(st["sa"], n1, k1 // 32)).view(G, c["rank"], k1)
    wb = _mx4_unpack(st["wb"], _untile_scales(st["sb"], c["hidden"], n1 // 32))
    x = _mx4_value(st["o"].reshape(M, -1).float()).view(M, G, k1)
    mid = torch.matmul(x.transpose(0, 1), wa.transpose(1, 2)).transpose(0, 1).reshape(M, n1)
    st["y"].copy_(torch.matmul(_mx4_value(mid), wb.t()))
    return st["y"]


# --------------------------------------------------------------------------
# what one pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == ATTEND:
        lens = _lengths(c)
        row = ROW8 if c["fp8"] else 2 * D
        pool = sum(min(n, c["sparse"]) if c["sparse"] else n for n in lens)
        near = sum(min(WINDOW, n * c["ratio"] + 1) for n in lens)
        H = c["heads"]
        b = pool * row + near * 2 * D + c["B"] * 2 * H * D * 2 + c["B"] * 4 + H * 4 + D * 4
        b += c["B"] * c["sparse"] * 4 + (pool * 2 if c["weights"] else 0)
        b += sum(-(-n // c["page"]) for n in lens) * 4
        return {"bytes": b, "flops": 4.0 * H * D * (pool + near)}
    if c["op"] == EVICT:
        cap = c["budget"] + c["extra"]
        # entries of equal chances: extra of cap go, as many of the kept ones move
        loose = max(1, cap - c["recent"])
        inside = c["budget"] if c["extra"] >= c["recent"] else c["budget"] + c["extra"] - c["recent"]
        moves = c["extra"] * inside / loose
        row = ROW8 if c["fp8"] else 2 * D
        return {"bytes": c["B"] * (cap * (2 + 4 + 4 + 4 + 4) + moves * 2 * row), "flops": c["B"] * cap}
    k = c["heads"] * c["dim"]
    n1 = c["groups"] * c["rank"]
    k1 = k // c["groups"]
    b = c["M"] * (2 * k + 2 * c["hidden"]) + (n1 * k1 + c["hidden"] * n1) * (0.5 + 1 / 32)
    return {"bytes": b, "flops": 2.0 * c["M"] * (n1 * k1 + c["hidden"] * n1)}


# --------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == ATTEND:
        return _exact_attend(case, st)
    if case["op"] == EVICT:
        return _exact_evict(case, st)
    return _exact_proj(case, st)


def _exact_row8(b):
    """FP8 rows [n, 592] from their bits: sign, four exponent bits (bias 7), three of the fraction."""
    code = b[:, :D - R].long()
    e, f = (code >> 3) & 15, (code & 7).double()
    mag = torch.where(e > 0, (8 + f) * torch.exp2((e - 10).double()), f * 2.0 ** -9)
    low = torch.where(code > 127, -mag, mag)
    scale = torch.exp2((b[:, D + R:D + R + (D - R) // 32].long() - 127).double())
    halves = b[:, D - R:D + R].long().view(-1, R, 2)
    high = (halves[..., 0] | (halves[..., 1] << 8)).to(torch.int32) << 16
    return torch.cat([low * scale.repeat_interleave(32, dim=1), high.view(torch.float32).double()], dim=1)


def _exact_mx4(x):
    """The MX form of x [n, K] by its thresholds: the smallest power of two
    that keeps a block's largest value within 6, and the E2M1 code as the
    number of midpoints passed (a midpoint itself goes to the even code)."""
    blk = x.reshape(x.shape[0], -1, 32)
    top = blk.abs().amax(-1, keepdim=True)
    s = torch.ceil(torch.log2(top.clamp(min=1e-30) / 6))
    s = torch.where(top <= 6 * torch.exp2(s - 1), s - 1, s)
    s = torch.where(top > 6 * torch.exp2(s), s + 1, s)
    a = blk.abs() / torch.exp2(s)
    code = torch.zeros_like(a)
    for i, mid in enumerate([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]):
        code += (a > mid) if i % 2 == 0 else (a >= mid)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=x.dtype, device=x.device)
    return (torch.sign(blk) * grid[code.long()] * torch.exp2(s)).reshape(x.shape)


def _exact_weight(codes, tiles, n, k):
    """FP4 weight [n, k] from its bytes and its scales in the product's order."""
    r, kb = torch.arange(n, device=DEV)[:, None], torch.arange(k // 32, device=DEV)
    at = ((r // 128) * (k // 128) + kb // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + kb % 4
    nib = torch.stack([codes % 16, codes // 16], dim=-1).reshape(n, k).long()
    e, f = (nib // 2) % 4, (nib % 2).double()
    mag = torch.where(e > 0, (2 + f) * torch.exp2((e - 2).double()), f / 2)
    return torch.where(nib > 7, -mag, mag) * torch.exp2(tiles[at].double() - 127).repeat_interleave(32, dim=1)


def _exact_attend(c, st):
    H, f64 = c["heads"], torch.float64
    out = torch.zeros((c["B"], H, D), dtype=f64, device=DEV)
    weights = torch.zeros((c["B"], st["n_max"]), dtype=f64, device=DEV)
    ladder = torch.tensor([BASE ** (-2.0 * j / R) for j in range(R // 2)], dtype=f64, device=DEV)
    for b, p in enumerate(st["pos"].tolist()):
        n = min((p + 1) // c["ratio"], st["n_max"])
        slots = torch.arange(n, device=DEV)
        if c["sparse"]:
            slots = st["idx"][b][st["idx"][b] >= 0].long()
        at = st["pages"][st["table"][b].long()[slots // c["page"]], slots % c["page"]]
        ring = torch.tensor([t % WINDOW for t in range(max(0, p - WINDOW + 1), p + 1)], device=DEV)
        rows = torch.cat([_exact_row8(at) if c["fp8"] else at.to(f64), st["win"][b][ring].to(f64)])
        phase = torch.polar(torch.ones_like(ladder), ladder * p)
        q = st["q"][b].to(f64)
        q = q / (q.pow(2).sum(1, keepdim=True) / D + EPS).sqrt() * st["g"].to(f64)
        q[:, D - R:] = torch.view_as_real(torch.view_as_complex(q[:, D - R:].reshape(H, -1, 2).contiguous()) * phase).reshape(H, R)
        score = torch.cat([q @ rows.T / math.sqrt(D), st["sink"].to(f64)[:, None]], dim=1)
        prob = torch.softmax(score, dim=1)[:, :-1]
        o = prob @ rows
        o[:, D - R:] = torch.view_as_real(torch.view_as_complex(o[:, D - R:].reshape(H, -1, 2).contiguous()) * phase.conj()).reshape(H, R)
        out[b] = o
        if c["weights"]:
            weights[b, :n] = prob[:, :n].sum(0)
    return {"out": out, "weights": weights} if c["weights"] else {"out": out}


def _exact_evict(c, st):
    # the pages are copies of whole rows and the other outputs whole numbers:
    # only the accumulated weights are computed
    budget = c["budget"]
    acc = st["acc"].double()
    for b, p in enumerate((st["pos"] + c["extra"] * c["ratio"]).tolist()):
        n = (p + 1) // c["ratio"]
        a = (acc[b, :n] + st["w"][b, :n].double()).float().cpu().numpy()
        old = [s for s in range(n) if s <= n - 1 - c["recent"]]
        gone = sorted(old, key=lambda s: (a[s], -s))[:n - budget]
        lost = set(gone)
        holes = [s for s in range(budget) if s in lost]
        movers = [s for s in range(budget, n) if s not in lost]
        row = acc[b].clone()
        row[:n] += st["w"][b, :n].double()
        if holes:
            row[torch.tensor(holes, device=DEV)] = row[torch.tensor(movers, device=DEV)]
        row[budget:] = 0
        acc[b] = row
    return {"pages": None, "acc": acc, "entry": None, "drop": None}


def _exact_proj(c, st):
    f64 = torch.float64
    M, k1, n1 = c["M"], c["heads"] // c["groups"] * c["dim"], c["groups"] * c["rank"]
    wa, wb = _exact_weight(st["wa"], st["sa"], n1, k1), _exact_weight(st["wb"], st["sb"], c["hidden"], n1)
    y = torch.empty((M, c["hidden"]), dtype=f64, device=DEV)
    for m0 in range(0, M, 2048):
        x = st["o"][m0:m0 + 2048].reshape(-1, c["groups"], k1).to(f64)
        mid = [_exact_mx4(_exact_mx4(x[:, j]) @ wa[j * c["rank"]:(j + 1) * c["rank"]].T) for j in range(c["groups"])]
        y[m0:m0 + 2048] = torch.cat(mid, dim=1) @ wb.T
    return y
