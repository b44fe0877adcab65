"""colibri_moe_decode, the whole layer for a few tokens in one launch, against 64-bit arithmetic.

The tolerance of every output value is a bound formed beside the reference, with u = 2^-24 and half a
step r of the activation type (2^-8 for bf16, u for fp32, where H and y are fp32 anyway):

* a dot product of n terms is off by at most n u times the sum of the terms' magnitudes, in any order
  (bf16 products are exact in fp32; an fp32 product rounds once), plus one addition per partial sum.
  Sums are cut into runs of 16 or 32 terms and more, so besides the runs' own additions there are at most
  n / 16 of them that are not zero, which the runs leave room for, and 32 where warps meet: (n + 32) u;
* h = silu(g) * v: |silu'| <= 1.1, and the exponential, quotient and product are good to (24 + 8 |g|) u;
  h is kept as fp32, or as two bf16: what the first leaves is at most r |h|, and of that the second
  leaves r again, r^2 |h| = 2^-16 |h| in all;
* the weight of a chosen expert: its logit and the largest are each off by at most el, which enters the
  softmax with at most 4 el, and exponential, sum and quotient add less than 32 u (raw weights: el);
* the weighted sum over k experts and the shared one adds (k + 2) u of the magnitudes, and y is rounded
  once, r |y|.
"""
import pytest
import torch

import sparse_expert_ffn_router_b200 as colibri

F32, BF16 = colibri.COLIBRI_F32, colibri.COLIBRI_BF16
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
U = 2.0 ** -24
HALF = {F32: U, BF16: torch.finfo(torch.bfloat16).eps / 2}
HALF_H = {F32: U, BF16: HALF[BF16] ** 2}


def test_decode_refuses_a_null_context():
    assert colibri.load().colibri_moe_decode(None, None, 0, None, None, None, None, None, None) == -1


class Case:
    def __init__(self, T, d, f, E, k, fs=0, dt=BF16, bias=False, flags=0, seed=0, max_tokens=None, x_std=1.0):
        self.T, self.d, self.f, self.E, self.k, self.fs, self.dt, self.flags = T, d, f, E, k, fs, dt, flags
        g = torch.Generator(device="cuda").manual_seed(seed * 1009 + T * 31 + d + f + E)
        n = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda").mul_(std).to(TORCH[dt])  # noqa: E731
        self.x = n(T, d, std=x_std)
        self.rw = n(E, d, std=d ** -0.5)
        self.rb = torch.randn(E, generator=g, device="cuda") if bias else None
        self.layer = colibri.MoELayer(d, f, E, k, fs, dt, dt, max_tokens=max_tokens or max(T, 1), router_flags=flags)
        self.ew = torch.full((E, self.layer.expert_stride), float("nan"), dtype=TORCH[dt], device="cuda")
        self.ew[:, : 2 * f * d] = n(E, 2 * f * d, std=d ** -0.5)
        self.ew[:, 2 * f * d: 3 * f * d] = n(E, d * f, std=f ** -0.5)
        self.sw = torch.cat([n(2 * fs * d, std=d ** -0.5), n(d * fs, std=fs ** -0.5)]) if fs else None

    def decode(self, y=None, stream=None, x=None):
        y = torch.full((self.T, self.d), 7.0, dtype=TORCH[self.dt], device="cuda") if y is None else y
        self.layer.decode(self.x if x is None else x, self.rw, self.rb, self.ew, y, shared_w=self.sw, stream=stream, T=self.T)
        return y

    def routing(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        r = dict(topk_idx=torch.empty(self.T, self.k, **i32), topk_w=torch.empty(self.T, self.k, device="cuda"),
                 counts=torch.empty(self.E, **i32), offsets=torch.empty(self.E + 1, **i32),
                 src_row=torch.empty(self.T * self.k, **i32), dst_row=torch.empty(self.T, self.k, **i32))
        self.layer.routing(**r)
        return r

    def _ffn(self, w, width, x):
        """FFN of rows x in 64 bits and the bound on its error."""
        w = w.double()
        d, half = self.d, HALF_H[self.dt]
        w1, w3, w2 = w[: width * d].view(width, d), w[width * d: 2 * width * d].view(width, d), w[2 * width * d: 3 * width * d].view(d, width)
        g, v, xa = x @ w1.T, x @ w3.T, x.abs()
        eg, ev = (d + 32) * U * (xa @ w1.abs().T), (d + 32) * U * (xa @ w3.abs().T)
        sg = g / (1 + torch.exp(-g))
        h = sg * v
        eh = 1.1 * eg * v.abs() + sg.abs() * ev + 1.1 * eg * ev + h.abs() * ((24 + 8 * g.abs()) * U + half * 1.01)
        return h @ w2.T, (eh + (width + 32) * U * (h.abs() + eh)) @ w2.abs().T

    def check(self, y):
        self.layer.sync_status()
        r = self.routing()
        torch.cuda.synchronize()
        x = self.x.double()
        logits = x @ self.rw.double().T
        el = (self.d + 32) * U * (x.abs() @ self.rw.double().abs().T)
        if self.rb is not None:
            logits = logits + self.rb.double()
            el = el + 2 * U * logits.abs()
        if self.flags & colibri.COLIBRI_ROUTER_CLAMP:
            logits = logits.clamp(-50, 50)
        idx = r["topk_idx"].long()
        assert ((idx >= 0) & (idx < self.E)).all()
        # the choice: distinct experts, in falling order, none left out that is clearly larger
        chosen = torch.zeros_like(logits).scatter_(1, idx, 1.0)
        assert (chosen.sum(1) == self.k).all()
        lc, slack = logits.gather(1, idx), 2 * el.amax(1, keepdim=True)
        assert (lc[:, 1:] <= lc[:, :-1] + slack).all()
        assert (logits.masked_fill(chosen > 0, -float("inf")) <= lc[:, -1:] + slack).all()
        if self.flags & colibri.COLIBRI_ROUTER_RAW_WEIGHTS:
            p, ep = lc, el.amax(1, keepdim=True).expand_as(lc)
        else:
            p = torch.softmax(lc, 1)
            ep = p * (4 * el.amax(1, keepdim=True) + 32 * U)
        assert ((r["topk_w"].double() - p).abs() <= ep).all()
        counts = chosen.sum(0).int()
        assert torch.equal(r["counts"], counts)
        off = torch.cat([torch.zeros(1, device="cuda"), counts.cumsum(0)]).int()
        assert torch.equal(r["offsets"], off)
        src = chosen.T.nonzero()[:, 1].int()  # ascending token within an expert
        assert torch.equal(r["src_row"], src)
        dst = (off[:-1][idx] + (torch.cumsum(chosen, 0) - chosen).gather(1, idx)).int()
        assert torch.equal(r["dst_row"], dst)

        ref = torch.zeros(self.T, self.d, dtype=torch.float64, device="cuda")
        err, mag = torch.zeros_like(ref), torch.zeros_like(ref)
        for e in torch.unique(idx).tolist():
            t, j = (idx == e).nonzero(as_tuple=True)
            o, eo = self._ffn(self.ew[e], self.f, x[t])
            pe, epe = p[t, j][:, None], ep[t, j][:, None]
            ref[t] += pe * o
            mag[t] += pe.abs() * o.abs()
            err[t] += (pe.abs() + epe) * eo + epe * o.abs()
        if self.fs:
            o, eo = self._ffn(self.sw, self.fs, x)
            ref += o
            mag += o.abs()
            err += eo
        err += (self.k + 2) * U * (mag + err)
        err += HALF[self.dt] * (ref.abs() + err)
        bad = ~((y.double() - ref).abs() <= err + 1e-37)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"
        return err


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,d,f,E,k,fs", [
    (1, 64, 64, 1, 1, 0), (1, 64, 64, 1, 1, 64), (2, 64, 128, 3, 3, 0), (3, 256, 512, 8, 2, 0), (16, 128, 64, 2, 1, 192),
    (1, 2048, 768, 128, 4, 1536), (7, 192, 320, 256, 8, 64), (8, 1024, 704, 16, 8, 0), (9, 576, 1088, 2, 2, 128),
    (15, 320, 2048, 5, 5, 0), (16, 64, 64, 256, 8, 0), (16, 4096, 192, 6, 2, 0), (5, 8192, 64, 3, 2, 64), (12, 4992, 128, 4, 1, 0),
    (4, 64, 14336, 2, 2, 0), (1, 4096, 1536, 8, 2, 0), (2, 192, 6208, 20, 8, 320), (16, 1280, 448, 30, 5, 64),
    (3, 1344, 320, 9, 3, 0), (16, 1152, 64, 3, 1, 0), (10, 2048, 192, 40, 3, 64), (2, 2368, 832, 7, 2, 0), (16, 2432, 64, 4, 2, 0), (16, 512, 512, 1, 1, 512), (6, 16384, 64, 2, 1, 0),
])
def test_decode(T, d, f, E, k, fs, dt):
    c = Case(T, d, f, E, k, fs, dt, bias=E > 4)
    c.check(c.decode())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T", range(1, 17))
def test_decode_every_token_count(T, dt):
    # a context for 40 tokens; expert 0 is chosen by every token, so its rows fill one and two column blocks
    c = Case(T, 128, 192, 6, 2, 64, dt, max_tokens=40)
    c.rb = torch.tensor([9.0, 0, 0, 0, 0, 0], device="cuda")
    c.check(c.decode())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("flags", [1, 2, 3])
def test_decode_router_variants(flags, dt):
    c = Case(6, 256, 128, 12, 3, 0, dt, bias=True, flags=flags, x_std=40.0 if flags == 2 else 1.0)
    if flags & 1:  # several logits beyond the clamp tie there and go to the lower index
        c.rb = torch.tensor([0, 70.0, 0, 90.0, 0, 80.0, 0, 0, -90.0, 0, 0, 0], device="cuda")
    y = c.decode()
    c.check(y)
    if flags & 1:
        assert c.routing()["topk_idx"].tolist() == [[1, 3, 5]] * 6


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_decode_ties_go_to_the_lower_index(dt):
    c = Case(3, 128, 64, 40, 4, 0, dt)
    c.rw.zero_()
    y = c.decode()
    c.check(y)
    assert c.routing()["topk_idx"].tolist() == [[0, 1, 2, 3]] * 3


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_decode_values_that_are_not_finite_stay_in_their_token(dt):
    c = Case(4, 256, 128, 4, 2, 0, dt)
    clean = c.decode().clone()
    err = c.check(clean)
    c.x[1, 3] = float("nan")
    c.x[2, 7] = float("inf")
    y = c.decode()
    torch.cuda.synchronize()
    c.layer.sync_status()
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    # The other tokens: where a warp's run of a sum ends depends on which experts the batch touches, and
    # tokens 1 and 2 may now choose others, so the sums may be grouped differently; both results are
    # within `err` of the same exact value, so they are within twice that of each other.
    for t in (0, 3):
        assert ((y[t].double() - clean[t].double()).abs() <= 2 * err[t]).all()


@pytest.mark.gpu
def test_decode_refusals_and_empty():
    c = Case(20, 128, 64, 4, 2)
    y = torch.full((20, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (c.layer.ctx, c.x, 16, c.rw, None, c.ew, None, y)

    def refused(code, **kw):
        names = ["ctx", "x", "T", "router_w", "router_b", "expert_w", "shared_w", "y"]
        a = dict(zip(names, args), **kw)
        with pytest.raises(colibri.ColibriError) as ei:
            colibri.colibri_moe_decode(*a.values())
        assert ei.value.status == code and colibri.colibri_last_error(c.layer.ctx)

    refused(-1, T=17)
    refused(-1, T=-1)
    refused(-1, x=None)
    refused(-1, router_w=None)
    refused(-1, expert_w=None)
    refused(-1, y=None)
    refused(-1, shared_w=c.ew)            # no shared expert in this layer
    refused(-1, expert_w=c.ew.cpu())      # weights in host memory
    refused(-2, x=c.x.data_ptr() + 2)
    colibri.colibri_moe_decode(*(args[:2] + (0,) + args[3:]))
    torch.cuda.synchronize()
    assert (y == 7.0).all()
    small = Case(2, 128, 64, 4, 2)
    with pytest.raises(colibri.ColibriError) as ei:   # above the context's max_tokens
        colibri.colibri_moe_decode(small.layer.ctx, c.x, 3, c.rw, None, c.ew, None, y)
    assert ei.value.status == -1
    for wdt in (colibri.COLIBRI_I8, colibri.COLIBRI_I4):
        q = colibri.MoELayer(128, 128, 4, 2, 0, BF16, wdt, max_tokens=4)
        with pytest.raises(colibri.ColibriError) as ei:
            colibri.colibri_moe_decode(q.ctx, c.x, 1, c.rw, None, c.ew, None, y)
        assert ei.value.status == -3


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_decode_beside_forward_streams_graphs_and_host_buffers(dt):
    """One context, both entry points in turn; repeated calls, another stream (replayed graphs), a caller's
    graph, and host x and y all give the same bits."""
    c = Case(11, 384, 640, 10, 3, 128, dt, bias=True, max_tokens=11)
    first = c.decode()
    c.check(first)
    fwd = torch.empty_like(first)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(first)
    torch.cuda.synchronize()
    for _ in range(5):
        c.layer.forward(c.x, c.rw, c.rb, c.ew, fwd, shared_w=c.sw, stream=st)
        c.decode(y, st)
    st.synchronize()
    assert torch.equal(y, first)
    # the two entry points agree to a few roundings of H and of the experts' outputs
    far = (fwd.double() - first.double()).abs().max().item()
    assert far <= (2e-2 if dt == BF16 else 1e-4) * first.double().abs().max().item()
    g = torch.cuda.CUDAGraph()
    y.zero_()
    with torch.cuda.graph(g):
        c.decode(y, torch.cuda.current_stream())
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first)
    hx, hy = c.x.cpu().pin_memory(), torch.zeros_like(first, device="cpu").pin_memory()
    for _ in range(3):
        hy.zero_()
        c.decode(hy, st, x=hx)
        st.synchronize()
        assert torch.equal(hy, first.cpu())
    # in place: x is read before the first value of y is written
    xs = c.x.clone()
    c.decode(xs, x=xs)
    torch.cuda.synchronize()
    assert torch.equal(xs, first)


@pytest.mark.gpu
def test_decode_two_contexts_on_two_streams():
    a, b = Case(5, 512, 384, 9, 2, 64, BF16), Case(16, 256, 256, 7, 3, 0, F32, seed=3)
    ra, rb = a.decode().clone(), b.decode().clone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    ya, yb = torch.zeros_like(ra), torch.zeros_like(rb)
    for _ in range(30):
        a.decode(ya, sa)
        b.decode(yb, sb)
    torch.cuda.synchronize()
    a.layer.sync_status()
    b.layer.sync_status()
    assert torch.equal(ya, ra) and torch.equal(yb, rb)


@pytest.mark.gpu
def test_decode_stage_events_count_the_launch():
    c = Case(4, 1024, 1024, 8, 2)
    st = torch.cuda.Stream()
    y = torch.empty_like(c.x)
    torch.cuda.synchronize()
    c.decode(y, st)
    colibri.colibri_profile_begin(c.layer.ctx, 8)
    for _ in range(4):
        c.decode(y, st)
    ms, n = colibri.colibri_profile_end(c.layer.ctx)
    assert n == 4 and ms["expert_gateup"] > 0
    assert ms["expert_gateup"] > sum(v for k, v in ms.items() if k != "expert_gateup")


@pytest.mark.gpu
def test_decode_experts_past_32_bits():
    # the last experts start more than 2^31 elements into the weight buffer
    c = Case(2, 4096, 14336, 14, 2)
    assert 13 * c.layer.expert_stride > 1 << 31
    c.rb = torch.zeros(14, device="cuda")
    c.rb[12:] = 30.0
    c.check(c.decode())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_decode_weights_that_are_not_finite_stay_with_their_tokens(dt):
    # an expert whose weights are broken touches only the tokens that chose it
    c = Case(6, 128, 192, 4, 1, 0, dt)
    c.x.zero_()
    c.x[:3, 0], c.x[3:, 1] = 1.0, 1.0
    c.x[:, 2:] = 0.25
    c.rw.zero_()
    c.rw[1, 0], c.rw[2, 1] = 9.0, 9.0            # tokens 0-2 take expert 1, tokens 3-5 expert 2
    clean = c.decode().clone()
    f, d = c.f, c.d
    c.ew[2, 5] = float("inf")
    c.ew[2, 2 * f * d: 3 * f * d] = float("nan")
    c.ew[0] = c.ew[3] = float("nan")             # experts that nobody takes
    y = c.decode()
    torch.cuda.synchronize()
    assert c.routing()["topk_idx"].flatten().tolist() == [1, 1, 1, 2, 2, 2]
    assert torch.equal(y[:3], clean[:3]) and torch.isnan(y[3:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_decode_infinite_activations_stay_infinite(dt):
    # h overflows in one expert: its products are infinities of their weights' signs, as h alone would give
    c = Case(2, 64, 64, 2, 1, 0, dt)
    c.x.fill_(1.0)
    c.rw.zero_()
    c.ew.zero_()
    f, d = c.f, c.d
    w = c.ew[0]
    w[0:d], w[f * d: f * d + d] = 2.0 ** 60, 2.0 ** 62       # g = 2^66, u = 2^68: h[0] = 2^134 overflows
    w[2 * f * d: 3 * f * d].view(d, f)[:, 0] = torch.where(torch.arange(d, device="cuda") % 2 == 0, 1.0, -1.0).to(w.dtype)
    y = c.decode()
    torch.cuda.synchronize()
    assert (y[:, 0::2] == float("inf")).all() and (y[:, 1::2] == -float("inf")).all()
