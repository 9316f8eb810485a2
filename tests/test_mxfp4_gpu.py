"""MXFP4 quantisation and the output projection on it, against the oracle's
MX rounding and 64-bit products."""
import math

import numpy as np
import pytest
import torch

import long_context_hybrid_kv_b200 as L
import paged_ref as P
from gen import host
from gpu_util import bf, bits, check_ok, f64
from oracle import ds4a_oracle as O

pytestmark = pytest.mark.gpu
SEED = 4242


def _quantize(rows):
    n, k = rows.shape
    codes = torch.full((n, k // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((L.ds4a_mxfp4_scale_bytes(n, k),), 0xAA, dtype=torch.uint8, device="cuda")
    L.ds4a_quantize_mxfp4(rows, codes, scales)
    check_ok()
    return codes, scales


def _value(codes, scales, n, k):
    return O.dequantize_idx_fp4(codes, P.untile_scales(scales, n, k))


@pytest.mark.parametrize("n,k", [(1, 128), (3, 256), (127, 128), (128, 512), (129, 384), (300, 4096)])
def test_quantize_bit_exact(n, k):
    x = host.normal_f32(SEED, f"q{n}.{k}", (n, k)).astype(np.float64)
    x *= np.repeat(np.exp2(8 * host.normal_f32(SEED, f"qm{n}.{k}", (n, k // 32)).astype(np.float64)), 32, axis=1)
    x[0, :32] = 0.0
    x[0, 32:64] = np.tile([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25], 4)  # ties
    b = O.store_bf16(x)
    codes, scales = _quantize(bf(b))
    want_c, want_s = O.quantize_idx_fp4(b)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(scales.cpu().numpy(), P.tile_scales(want_s))


def test_quantize_rows_apart():
    x = bf(host.normal_bf16(SEED, "apart", (130, 512)))
    codes, scales = _quantize(x[:, :256])
    c2, s2 = _quantize(x[:, :256].contiguous())
    assert torch.equal(codes, c2) and torch.equal(scales, s2)


SHAPES = {"small": (16, 128, 4, 256, 1024), "one_group": (4, 64, 1, 256, 256), "odd": (24, 96, 3, 512, 768),
          "flash": (64, 512, 8, 1024, 4096)}


def _project(name, shape, M):
    H, D, g, r, hidden = shape
    k1, n1 = H // g * D, g * r
    o = host.normal_bf16(SEED, f"{name}.o", (M, H, D))
    wa = _quantize(bf(host.normal_bf16(SEED, f"{name}.wa", (n1, k1), 1 / math.sqrt(k1))))
    wb = _quantize(bf(host.normal_bf16(SEED, f"{name}.wb", (hidden, n1), 1 / math.sqrt(n1))))
    cfg = L.OprojCfg(H, D, g, r, hidden)
    y = torch.full((M, hidden), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((L.ds4a_out_proj_mxfp4_workspace(cfg, M),), 0xFF, dtype=torch.uint8, device="cuda")
    args = (cfg, bf(o), *wa, *wb, y, ws)
    L.ds4a_out_proj_mxfp4(*args)
    check_ok()
    return o, wa, wb, y, args


def _reference(o, wa, wb, shape, rows):
    """y in 64 bits, and its bound: every intermediate value whose float32 sum
    (off by at most K 2^-24 of its terms' sizes) may round to another code is
    allowed a step of its block, the product K 2^-24 of its terms, the result
    half a bf16 step."""
    H, D, g, r, hidden = shape
    k1, n1 = H // g * D, g * r
    A = _value(wa[0].cpu().numpy(), wa[1].cpu().numpy(), n1, k1).reshape(g, r, k1)
    Bm = _value(wb[0].cpu().numpy(), wb[1].cpu().numpy(), hidden, n1)
    x = O.widen(o[rows]).reshape(len(rows) * g, k1)
    c, s = O.mx_quantize(x, "e2m1")
    xq = O.mx_dequantize(c, s, "e2m1").reshape(len(rows), g, k1)
    mid = np.concatenate([xq[:, j] @ A[j].T for j in range(g)], axis=1)
    err = np.concatenate([np.abs(xq[:, j]) @ np.abs(A[j]).T for j in range(g)], axis=1) * k1 * 2.0 ** -24

    def value(v):
        cc, ss = O.mx_quantize(v, "e2m1")
        return O.mx_dequantize(cc, ss, "e2m1")

    blocks = lambda v: v.reshape(len(rows), -1, 32)  # noqa: E731
    mq, lo, hi = value(mid), value(mid - err), value(mid + err)
    # a block whose largest value may pass a power of two may take the next scale: any of its values may move by its step
    top, te = np.abs(blocks(mid)).max(-1), np.abs(blocks(err)).max(-1)
    jump = np.ceil(np.log2(np.maximum(top - te, 1e-30) / 6)) != np.ceil(np.log2(np.maximum(top + te, 1e-30) / 6))
    step = np.maximum(np.abs(hi - mq), np.abs(mq - lo))
    step = np.where(np.repeat(jump, 32, axis=1), np.repeat(2 * top / 6, 32, axis=1), step)
    ref = mq @ Bm.T
    bound = step @ np.abs(Bm).T + (np.abs(mq) @ np.abs(Bm).T) * n1 * 2.0 ** -24
    return ref, bound + P.U16 * (np.abs(ref) + bound) + 1e-30


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 127, 128, 129, 300])
@pytest.mark.parametrize("name", ["small", "one_group", "odd"])
def test_project(name, M):
    o, wa, wb, y, _ = _project(name, SHAPES[name], M)
    ref, bound = _reference(o, wa, wb, SHAPES[name], np.arange(M))
    off = np.abs(f64(y) - ref)
    assert (off <= bound).all(), f"{np.max(off / bound):.3g} of the bound at {np.argwhere(off > bound)[:3].tolist()}"


@pytest.mark.parametrize("M", [1, 8, 77, 515, 4096 + 77])
def test_project_flash(M):
    o, wa, wb, y, _ = _project("flash", SHAPES["flash"], M)
    rows = np.unique(np.r_[0, M // 2, M - 1, np.random.default_rng(M).integers(0, M, 5)])
    ref, bound = _reference(o, wa, wb, SHAPES["flash"], rows)
    off = np.abs(f64(y)[rows] - ref)
    assert (off <= bound).all(), f"{np.max(off / bound):.3g} of the bound"


def test_project_same_bits_and_own_rows():
    """Twice the same bits; a row's result does not depend on the rows beside
    it, a NaN in one row stays there."""
    shape = SHAPES["flash"]
    o, wa, wb, y, args = _project("rows", shape, 40)
    first = bits(y).copy()
    L.ds4a_out_proj_mxfp4(*args)
    check_ok()
    assert np.array_equal(bits(y), first)
    o2 = o.copy()
    o2[7, 3, 5] = 0x7FC0
    args = (args[0], bf(o2)) + args[2:]
    L.ds4a_out_proj_mxfp4(*args)
    check_ok()
    keep = np.arange(40) != 7
    assert np.array_equal(bits(y)[keep], first[keep])


def test_project_zero_rows_and_streams():
    shape = SHAPES["small"]
    H, D, g, r, hidden = shape
    o, wa, wb, y, args = _project("st", shape, 33)
    first = bits(y).copy()
    zero = torch.zeros((5, H, D), dtype=torch.bfloat16, device="cuda")
    y0 = torch.full((5, hidden), 7.0, dtype=torch.bfloat16, device="cuda")
    L.ds4a_out_proj_mxfp4(args[0], zero, *wa, *wb, y0, args[-1])
    check_ok()
    assert (f64(y0) == 0).all()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws2 = torch.empty_like(args[-1])
    y2 = torch.empty_like(y)
    torch.cuda.synchronize()
    for _ in range(10):
        L.ds4a_out_proj_mxfp4(*args, stream=s1)
        L.ds4a_out_proj_mxfp4(*args[:-2], y2, ws2, stream=s2)
    torch.cuda.synchronize()
    assert np.array_equal(bits(y), first) and np.array_equal(bits(y2), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.ds4a_out_proj_mxfp4(*args)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(y), first)
