"""int8 products whose two scales multiply to something that fp32 cannot hold, though the result can.

y = s t acc: with s and t from 2^-149 to the largest float, s t alone may be subnormal (bits are lost) or
infinite (a sum of zero becomes NaN).  The scaling rounds at most four times (the conversion of the sum,
the product of the scales, the product with it, or once from 64 bits), each u = 2^-24 of itself, and a
result that is itself subnormal by at most half of fp32's smallest step: 4 u |y| + 2^-149 in all;
SwiGLU by (24 + 8 |g|) u |h| as for ordinary scales, and since g, u and silu(g) are fp32 values by definition
(the header's "the two products in fp32"), each of them that is subnormal is off by half a smallest step,
2^-150, more: 2^-150 on g moves silu(g) by at most 1.1 * 2^-150 (the largest slope of silu), on silu(g) by 2^-150,
both times |u|; 2^-150 on u counts |silu(g)| times.  So (2.1 |u| + |silu(g)|) 2^-150 is added.
"""
import pytest
import torch

from tests import test_int_products as P

U, F32, BF16 = P.U, P.F32, P.BF16
TINY = 2.0 ** -149
# pairs (row scale, column scale), as powers of two; their products run from 2^-149 to beyond 2^128
ROWS = (-149, -126, -100, -70, -64, -63, -10, 0, 63, 64, 90, 120, 127)
COLS = (-149, -90, -64, -63, -41, -20, 0, 30, 63, 64, 100, 127)


def _scales(n, exps, g):
    """n scales 1.x * 2^e over the exponents in turn, one of them zero"""
    s = torch.ldexp(1 + torch.rand(n, generator=g, dtype=torch.float64), torch.tensor([exps[i % len(exps)] for i in range(n)]))
    s = s.clamp(max=torch.finfo(torch.float32).max).float()
    s[n // 2] = 0.0
    return s


def _data(shape, g):
    v = P._ints(g, *shape, lo=100, hi=128)  # sums near their largest, so that small products of scales still show
    v[..., -1, :] = 0                        # and sums that are zero
    return v


def _close(got, ref, rel, out, more=0.0):
    top = torch.finfo(P.TORCH[out]).max
    got, sure = got.double(), ref.abs() <= top * (1 - 2.0 ** -6)
    over = ref.abs() > top * (1 + 2.0 ** -6)
    assert torch.equal(got[over], torch.sign(ref[over]) * float("inf"))
    tol = ref.abs() * (rel + P.HALF[out]) * (1 + 1e-6) + (TINY if out == F32 else 2.0 ** -133) + more
    bad = sure & ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values off, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [(1, 40, 4096), (7, 300, 2064), (16, 129, 512), (40, 200, 1040), (300, 260, 512),
                                   (20, 19000, 400), (64, 19456, 128), (300, 8192, 144), (16, 100001, 336)])
def test_products_of_extreme_scales(M, N, K, out):
    # the sizes of the 16-row stream, the split tiles, the pair tiles and their swapped tails
    g = torch.Generator().manual_seed(M * 3 + N)
    q, w, s, t = _data((M, K), g), _data((N, K), g), _scales(M, ROWS, g), _scales(N, COLS, g)
    if M == 1:
        q, s = P._ints(g, 1, K, lo=100, hi=128), torch.tensor([1.3 * 2.0 ** -80])
    _close(P._run_gemm(q, s, w, t, out), P._ref_product(q, s, w, t), 4 * U, out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("N", [64, 77, 5008])
@pytest.mark.parametrize("counts", [(3, 0, 9), (40, 1, 150), (300, 10, 257)])
def test_expert_products_of_extreme_scales(counts, N, out):
    c = P._experts_case(counts, N, 272, 5, False)
    g = torch.Generator().manual_seed(N)
    c.update(q=_data((c["R"], 272), g), w=_data(tuple(c["w"].shape), g), s=_scales(c["R"], ROWS, g),
             t=_scales(c["E"] * N, COLS, g).view(c["E"], N))
    ref, _, own = P._ref_experts(c)
    assert own.all()
    _close(P._run_experts(c, out), ref, 4 * U, out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("N", [64, 77, 5008])
@pytest.mark.parametrize("counts", [(3, 0, 9), (40, 1, 150), (300, 10, 257)])
def test_swiglu_of_extreme_scales(counts, N, out):
    # gates of 2^-120 to 2^3 beside ups of any size
    c = P._experts_case(counts, N, 272, 6, True)
    g = torch.Generator().manual_seed(N + 1)
    R, E = c["R"], c["E"]
    c.update(q=_data((R, 272), g), w=_data(tuple(c["w"].shape), g), s=_scales(R, (-60, -75, -64, -90), g))
    gate, up = _scales(E * N, (-80, -40, 40, -85), g).view(E, N), _scales(E * N, (60, 20, 70, -70), g).view(E, N)
    c["t"] = torch.cat([gate, up], 1)
    ref, gabs, own = P._ref_experts(c)
    assert own.all() and float(gabs.max()) < 60
    ups = dict(c, swiglu=False, w=c["w"][:, N:], t=up)
    u = P._ref_experts(ups)[0].abs()
    silu = torch.where(u > 0, ref.abs() / u, torch.zeros_like(u))
    _close(P._run_experts(c, out), ref, (24 + 8 * gabs.double()) * U, out, (2.1 * u + silu) * 2.0 ** -150 * 1.01)
