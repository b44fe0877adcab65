"""The MoE layer with int8 weights and int8 activations (weight_dtype COLIBRI_I8A8).

Two references: the CPU oracle on the same int8 weights with exact activations, within the
quantised-weight tolerance (5e-2 of the largest output); and the layer's own steps called one by one
(each checked against 64-bit arithmetic elsewhere), which must give the same bits.
"""
import pytest
import torch

import inputgen
import sparse_expert_ffn_router_b200 as colibri
from tests import gpu_harness as H

BF16, I8A8 = colibri.COLIBRI_BF16, colibri.COLIBRI_I8A8


def _desc(**kw):
    base = dict(d_model=256, d_ff=512, num_experts=8, top_k=2, act_dtype=BF16, weight_dtype=I8A8, max_tokens=64)
    base.update(kw)
    return base


@pytest.mark.parametrize("code,kw", [
    (-3, dict(act_dtype=colibri.COLIBRI_F32)), (-3, dict(shared_d_ff=64)), (-1, dict(weight_scale_mode=1)),
    (-3, dict(d_ff=131072)), (-1, dict(weight_dtype=5)), (-1, dict(act_dtype=I8A8)),
])
def test_init_refuses(code, kw):
    with pytest.raises(colibri.ColibriError) as ei:
        colibri.colibri_init(**_desc(**kw))
    assert ei.value.status == code and colibri.colibri_last_error()


def _layer(wl, flags=0, max_tokens=None):
    return colibri.MoELayer(wl.d, wl.f, wl.E, wl.k, 0, BF16, I8A8, max_tokens=max_tokens or max(wl.T, 1), router_flags=flags)


def _wl(T, d, E, k, f, bias=None):
    return inputgen.custom(f"i8a8_{T}_{d}_{E}_{k}_{f}", T=T, d=d, E=E, k=k, f=f, act=inputgen.BF16, wdt=inputgen.I8, bias=bias)


def _by_parts(t, wl, stride):
    """Router and grouping, rows, gate/up, H rows, down, weighted sum, each by its own entry point."""
    T, d, f, E, k, R = wl.T, wl.d, wl.f, wl.E, wl.k, wl.T * wl.k
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, src, dst, counts, off = (torch.empty(n, **i32) for n in ((T, k), R, (T, k), E, E + 1))
    w = torch.empty(T, k, device="cuda")
    xp = torch.empty(R, d, dtype=torch.bfloat16, device="cuda")
    colibri.colibri_route_noalloc(t["x"], BF16, T, d, t["router_w"], t["router_b"], E, k, idx, w, counts, off, src, dst, xp)
    q, s = torch.empty(R, d, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    h = torch.empty(R, f, dtype=torch.bfloat16, device="cuda")
    hq, hs = torch.empty(R, f, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    yp, y = torch.empty(R, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    ew, sc, per = t["expert_w"], t["expert_scales"], 2 * f + d
    colibri.colibri_quantize_rows(xp, BF16, R, d, d, q, d, s)
    colibri.colibri_int_swiglu_experts(q, d, s, R, off, E, ew, stride, sc, per, f, d, h, f, BF16)
    colibri.colibri_quantize_rows(h, BF16, R, f, f, hq, f, hs)
    colibri.colibri_int_gemm_experts(hq, f, hs, R, off, E, ew.data_ptr() + 2 * f * d, stride, sc.data_ptr() + 8 * f, per,
                                     d, f, yp, d, BF16)
    colibri.colibri_combine(yp, BF16, dst, w, T, k, d, y)
    colibri.colibri_int_check()
    return y.float().cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,k,f,bias", [
    (1, 64, 4, 1, 64, None), (3, 128, 4, 2, 256, None), (64, 256, 8, 2, 512, None), (65, 192, 16, 4, 320, None),
    (300, 256, 8, 8, 192, None), (700, 128, 5, 2, 640, ((0, 6.0), (4, -40.0))), (1000, 512, 128, 4, 128, None),
    (40, 64, 1, 1, 1088, None), (257, 320, 2, 2, 64, None),
])
def test_layer(T, d, E, k, f, bias):
    wl = _wl(T, d, E, k, f, bias)
    p = inputgen.make_problem(wl, seed=T + E)
    layer = _layer(wl)
    t = H.to_device(p)
    H.parity(p, layer=layer, dev_inputs=t)
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    layer.forward(t["x"], t["router_w"], t["router_b"], t["expert_w"], y, t["expert_scales"])
    layer.sync_status()
    parts = _by_parts(t, wl, layer.expert_stride)
    if T > 64:  # smaller batches route through another kernel, whose logits may round differently
        assert torch.equal(y.float().cpu(), parts)
    else:
        scale = parts.abs().max()
        assert (y.float().cpu() - parts).abs().max() <= 2e-2 * scale


@pytest.mark.gpu
def test_layer_graph_streams_host_and_routed():
    wl = _wl(150, 256, 6, 3, 384)
    p = inputgen.make_problem(wl, seed=2)
    t = H.to_device(p)
    layer = _layer(wl, max_tokens=200)
    y = torch.empty(wl.T, wl.d, dtype=torch.bfloat16, device="cuda")
    call = lambda x, y, st: layer.forward(x, t["router_w"], None, t["expert_w"], y, t["expert_scales"], stream=st, T=wl.T)  # noqa: E731
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # the context's first forward is a captured one
        call(t["x"], y, torch.cuda.current_stream())
    g.replay()
    torch.cuda.synchronize()
    first = y.clone()
    st = torch.cuda.Stream()
    for _ in range(4):
        y.zero_()
        torch.cuda.synchronize()
        call(t["x"], y, st)
        st.synchronize()
        assert torch.equal(y, first)
    hx, hy = p.x.pin_memory(), torch.zeros_like(p.x).pin_memory()
    for _ in range(3):
        call(hx, hy, st)
    st.synchronize()
    assert torch.equal(hy, first.cpu())
    idx, w = torch.empty(wl.T, wl.k, dtype=torch.int32, device="cuda"), torch.empty(wl.T, wl.k, device="cuda")
    layer.routing(topk_idx=idx, topk_w=w)
    y.zero_()
    layer.forward_routed(t["x"], idx, w, t["expert_w"], y, t["expert_scales"])
    torch.cuda.synchronize()
    layer.sync_status()
    assert torch.equal(y, first)
    with pytest.raises(colibri.ColibriError) as ei:
        layer.forward(t["x"], t["router_w"], None, t["expert_w"], y)  # scales missing
    assert ei.value.status == -1
    with pytest.raises(colibri.ColibriError) as ei:
        layer.decode(t["x"][:2], t["router_w"], None, t["expert_w"], y)
    assert ei.value.status == -3
    y.fill_(7.0)
    layer.forward(t["x"], t["router_w"], None, t["expert_w"], y, t["expert_scales"], T=0)
    torch.cuda.synchronize()
    assert (y == 7.0).all()


@pytest.mark.gpu
def test_layer_stage_events():
    wl = _wl(2048, 1024, 8, 2, 2048)
    p = inputgen.make_problem(wl, seed=1)
    t = H.to_device(p)
    layer = _layer(wl)
    y = torch.empty(wl.T, wl.d, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    colibri.colibri_profile_begin(layer.ctx, 4)
    for _ in range(4):
        layer.forward(t["x"], t["router_w"], None, t["expert_w"], y, t["expert_scales"], stream=st)
    ms, n = colibri.colibri_profile_end(layer.ctx)
    assert n == 4 and all(v > 0 for v in ms.values())


@pytest.mark.gpu
def test_layer_overlapped_launches(monkeypatch):
    # programmatic dependent launch only starts a kernel's set-up early: the same bits, as plain launches
    # and as a replayed graph
    wl = _wl(260, 256, 6, 2, 448)
    p = inputgen.make_problem(wl, seed=5)
    t = H.to_device(p)
    outs = []
    for pdl in ("0", "1"):
        monkeypatch.setenv("COLIBRI_PDL", pdl)
        layer = _layer(wl)
        s = torch.cuda.Stream()
        for stream in (None, s, s):
            y = torch.full((wl.T, wl.d), 5.0, dtype=torch.bfloat16, device="cuda")
            torch.cuda.synchronize()
            layer.forward(t["x"], t["router_w"], None, t["expert_w"], y, t["expert_scales"], stream=stream)
            torch.cuda.synchronize()
            outs.append(y)
        layer.sync_status()
        layer.close()
    for y in outs[1:]:
        assert torch.equal(y, outs[0])
