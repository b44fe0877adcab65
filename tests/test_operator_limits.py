"""The int8 products, the int8-row layer and the few-token launch at the largest sizes that the header allows
(one dimension at a time, so that the data stays small)."""
import pytest
import torch

import inputgen
import sparse_expert_ffn_router_b200 as colibri
from tests import gpu_harness as H
from tests import test_gpu_int8_layer as L
from tests import test_int_products as P
from tests.test_gpu_decode import BF16, F32, Case

U = P.U


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1 << 24, 1, 16), (1, 1 << 20, 16), (17, 1 << 20, 32), (300, 1 << 20, 16), ((1 << 24) - 3, 5, 16)])
def test_largest_dense_products(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(N + K)
    q, w = (torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8) for s in ((M, K), (N, K)))
    s, t = torch.rand(M, generator=g, device="cuda") + 0.5, torch.rand(N, generator=g, device="cuda") / 127 + 2.0 ** -10
    y = torch.full((M + 1, N), P.SENTINEL, device="cuda")
    colibri.colibri_int_gemm(q, K, s, w, K, t, M, N, K, y, N, F32, torch.cuda.current_stream())
    colibri.colibri_int_check(torch.cuda.current_stream())
    assert (y[M] == P.SENTINEL).all()
    for a in range(0, M, 1 << 20):  # in pieces: the 64-bit reference is 8 bytes a value
        b = min(M, a + (1 << 20))
        for c in range(0, N, 1 << 16):
            d = min(N, c + (1 << 16))
            ref = P._ref_product(q[a:b], s[a:b], w[c:d], t[c:d])
            assert ((y[a:b, c:d].double() - ref).abs() <= 4 * U * (1 + 1e-6) * ref.abs() + 1e-37).all(), (a, c)


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True])
def test_a_row_in_each_of_256_experts_and_a_million_rows(swiglu):
    g = torch.Generator(device="cuda").manual_seed(3)
    E, N, K, R = 256, 16, 32, 1 << 20
    cols = 2 * N if swiglu else N
    counts = torch.ones(E, dtype=torch.int64)
    counts[200] = R - (E - 1)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
    q, w = (torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8) for s in ((R, K), (E, cols, K)))
    s, t = torch.rand(R, generator=g, device="cuda") + 0.5, torch.rand(E, cols, generator=g, device="cuda") / 3e4
    y = torch.empty(R, N, device="cuda")
    call = colibri.colibri_int_swiglu_experts if swiglu else colibri.colibri_int_gemm_experts
    call(q, K, s, R, off, E, w, cols * K, t, cols, N, K, y, N, F32, torch.cuda.current_stream())
    colibri.colibri_int_check(torch.cuda.current_stream())
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), counts.cuda())
    acc = torch.empty(R, cols, dtype=torch.float64, device="cuda")
    for a in range(0, R, 1 << 17):
        b = a + (1 << 17)
        acc[a:b] = torch.einsum("rk,rck->rc", q[a:b].double(), w[e[a:b]].double()) * s[a:b, None].double() * t[e[a:b]].double()
    ref, rel = acc, torch.full_like(acc, 4 * U)
    if swiglu:
        gt, up = acc[:, :N], acc[:, N:]
        ref, rel = gt / (1 + torch.exp(-gt)) * up, (24 + 8 * gt.abs()) * U
    assert ((y.double() - ref).abs() <= rel * (1 + 1e-6) * ref.abs() + 1e-37).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 70])
def test_int8_row_layer_of_the_widest_ffn(T):
    # Against the layer's own steps, each checked against 64 bits elsewhere.  (Not against exact activations: H
    # has one scale per row, max |h| / 127, and the largest of 131008 values stands far above the rest, so the
    # rounding of the rest, up to half a scale each, is a tenth of the output.)
    wl = L._wl(T, 64, 2, 2, 131008)
    p = inputgen.make_problem(wl, seed=1)
    layer = L._layer(wl)
    t = H.to_device(p)
    y = torch.empty(T, 64, dtype=torch.bfloat16, device="cuda")
    layer.forward(t["x"], t["router_w"], t["router_b"], t["expert_w"], y, t["expert_scales"])
    layer.sync_status()
    parts = L._by_parts(t, wl, layer.expert_stride)
    assert torch.equal(y.float().cpu(), parts) if T > 64 else (y.float().cpu() - parts).abs().max() <= 2e-2 * parts.abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,d,f,E,k,fs", [(16, 65536, 64, 2, 2, 64), (1, 65536, 64, 3, 1, 0), (3, 64, 262144, 2, 1, 262144), (16, 64, 262144, 1, 1, 0)])
def test_decode_of_the_widest_layers(T, d, f, E, k, fs, dt):
    c = Case(T, d, f, E, k, fs, dt)
    c.check(c.decode())


@pytest.mark.gpu
@pytest.mark.parametrize("pdl", ["0", "1"])
def test_decode_and_forward_in_turn_with_overlapped_launches(pdl, monkeypatch):
    # forward's launches may overlap one another, never the few-token launch, whose barriers and workspace it shares
    monkeypatch.setenv("COLIBRI_PDL", pdl)
    c = Case(14, 512, 320, 6, 2, 64, BF16, bias=True)
    y, f = c.decode().clone(), torch.empty(14, 512, dtype=torch.bfloat16, device="cuda")
    fwd = lambda out, st: c.layer.forward(c.x, c.rw, c.rb, c.ew, out, shared_w=c.sw, stream=st)  # noqa: E731
    fwd(f, None)
    torch.cuda.synchronize()
    c.check(y)
    for st in (torch.cuda.current_stream(), torch.cuda.Stream()):
        ys, fs = torch.zeros_like(y), torch.zeros_like(f)
        torch.cuda.synchronize()
        for _ in range(10):
            c.decode(ys, st)
            fwd(fs, st)
            c.decode(ys, st)
        st.synchronize()
        c.layer.sync_status(st)
        assert torch.equal(ys, y) and torch.equal(fs, f)
