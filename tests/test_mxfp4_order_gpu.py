"""Weights that are quantised right before they are used, on one stream and
without a wait of the host between: the projection reads them early, so it must
not start before they are written."""
import math

import pytest
import torch

import long_context_hybrid_kv_b200 as L
from gen import host
from gpu_util import bf, check_ok

pytestmark = pytest.mark.gpu
SEED = 77

SHAPES = {"small": (16, 128, 4, 256, 1024), "flash": (64, 512, 8, 1024, 4096)}


@pytest.mark.parametrize("M", [1, 77, 128, 129, 1500])
@pytest.mark.parametrize("name", SHAPES)
def test_quantised_weights_are_there(name, M):
    H, D, g, r, hidden = SHAPES[name]
    k1, n1 = H // g * D, g * r
    cfg = L.OprojCfg(H, D, g, r, hidden)
    o = bf(host.normal_bf16(SEED, f"{name}.o", (M, H, D)))
    src = [bf(host.normal_bf16(SEED, f"{name}.{n}{k}", (n, k), 1 / math.sqrt(k))) for n, k in ((n1, k1), (hidden, n1))]
    mats = [(torch.empty((n, k // 2), dtype=torch.uint8, device="cuda"),
             torch.empty(L.ds4a_mxfp4_scale_bytes(n, k), dtype=torch.uint8, device="cuda")) for n, k in ((n1, k1), (hidden, n1))]
    ws = torch.empty(L.ds4a_out_proj_mxfp4_workspace(cfg, M), dtype=torch.uint8, device="cuda")
    y = torch.empty((M, hidden), dtype=torch.bfloat16, device="cuda")

    def quantise():
        for x, m in zip(src, mats):
            L.ds4a_quantize_mxfp4(x, *m)

    def project():
        L.ds4a_out_proj_mxfp4(cfg, o, *mats[0], *mats[1], y, ws)

    def spoil():  # codes and scales of other weights
        for codes, scales in mats:
            codes.fill_(0x77), scales.fill_(127)
        y.fill_(7.0)

    spoil(), torch.cuda.synchronize()
    quantise(), torch.cuda.synchronize()
    project()
    check_ok()
    want = y.clone()
    for _ in range(10):
        spoil(), torch.cuda.synchronize()
        quantise(), project()
        check_ok()
        assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        quantise(), project()
    for _ in range(10):
        spoil(), torch.cuda.synchronize()
        graph.replay()
        check_ok()
        assert torch.equal(y, want)
    # a captured run of several, and the same matrices anew behind a projection that reads them
    with torch.cuda.graph(graph2 := torch.cuda.CUDAGraph()):
        for _ in range(4):
            quantise(), project()
    spoil(), torch.cuda.synchronize()
    graph2.replay()
    check_ok()
    assert torch.equal(y, want)
