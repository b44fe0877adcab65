"""The operators beside one another: the int8-row layer spread over ranks, and the few-token launch on one
stream beside int8 products on others."""
import pytest
import torch

import inputgen
import sparse_expert_ffn_router_b200 as colibri
from sparse_expert_ffn_router_b200.expert_parallel import ExpertParallelMoE
from tests import gpu_harness as H
from tests import test_int_products as P
from tests.test_gpu_decode import BF16, F32, Case

I8A8 = colibri.COLIBRI_I8A8


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,k,f", [(1, 128, 4, 2, 192), (90, 256, 8, 3, 320), (700, 512, 16, 2, 256)])
def test_int8_rows_in_the_expert_parallel_layer(T, d, E, k, f):
    """One rank's layer against the oracle, and the same values as the plain int8-row layer up to the
    rounding of its expert outputs (both round each row of Yp to bf16 before the weighted sum)."""
    wl = inputgen.custom(f"ep88_{T}", T=T, d=d, E=E, k=k, f=f, act=inputgen.BF16, wdt=inputgen.I8)
    p = inputgen.make_problem(wl, seed=T)
    t = H.to_device(p)
    ep = ExpertParallelMoE(d, f, E, k, BF16, I8A8, max_tokens=T)
    assert ep.expert_stride == p.expert_stride
    plain = colibri.MoELayer(d, f, E, k, 0, BF16, I8A8, max_tokens=T)
    y, ref = (torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for _ in range(2):
        ep.forward(t["x"], t["router_w"], t["router_b"], t["expert_w"], y, t["expert_scales"])
    plain.forward(t["x"], t["router_w"], t["router_b"], t["expert_w"], ref, t["expert_scales"])
    torch.cuda.synchronize()
    ep.local.sync_status()
    plain.sync_status()
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    plain.routing(topk_idx=idx, topk_w=w)
    torch.cuda.synchronize()
    oracle_y = H.oracle.combine(p.x, idx.cpu(), w.cpu(), p.expert_w, p.expert_stride, f, p.expert_scales, None, 0, list(range(T)))
    H.check_y(p, y.float().cpu(), oracle_y, tol=5e-2)
    far = (y.float() - ref.float()).abs().max().item()
    assert far <= 2e-2 * ref.float().abs().max().item()
    ep.close()


@pytest.mark.gpu
def test_decode_beside_int8_products():
    """The few-token launch needs every SM, the products hold some: whatever order they run in, each gives the
    bits that it gives alone, with calls of both kinds queued at once and as replayed graphs."""
    c = Case(9, 1024, 704, 12, 3, 128, BF16, bias=True)
    small = Case(2, 256, 128, 4, 2, 0, F32)
    probs = [P._problem(8, 4096, 1024, 31), P._problem(100, 1000, 512, 32), P._problem(1500, 2100, 256, 33)]
    alone = [c.decode().clone(), small.decode().clone()] + [P._run_gemm(*p, F32) for p in probs]
    dev = [[v.cuda() for v in p] for p in probs]
    ys = [torch.zeros_like(alone[0]), torch.zeros_like(alone[1])] + [torch.zeros(p[0].shape[0], p[2].shape[0], device="cuda") for p in probs]
    streams = [torch.cuda.Stream() for _ in ys]
    torch.cuda.synchronize()

    def call(i, stream):
        if i < 2:
            (c, small)[i].decode(ys[i], stream)
        else:
            q, s, w, t = dev[i - 2]
            colibri.colibri_int_gemm(q, q.shape[1], s, w, q.shape[1], t, q.shape[0], w.shape[0], q.shape[1], ys[i], w.shape[0], F32, stream)

    def same():
        torch.cuda.synchronize()
        c.layer.sync_status()
        small.layer.sync_status()
        colibri.colibri_int_check()
        for y, ref in zip(ys, alone):
            assert torch.equal(y.cpu(), ref.cpu())
            y.zero_()
        torch.cuda.synchronize()

    for r in range(30):
        for i in range(len(ys)):
            call((i + r) % len(ys), streams[(i + r) % len(ys)])
    same()
    graphs = []
    for i in range(len(ys)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, torch.cuda.current_stream())
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    same()
