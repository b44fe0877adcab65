"""int8 rows and products (colibri_quantize_rows, colibri_int_gemm, colibri_int_gemm_experts,
colibri_int_swiglu_experts) against plain 64-bit arithmetic.

Tolerances, with u = 2^-24 (half a step of fp32): the int32 sum is exact, its conversion to fp32, the
product of the two scales and the product with it round once each, so a product is off by at most
(1 + u)^3 - 1 < 4 u of itself.  silu(g) * u multiplies g's relative error by at most 1 + |g| (the
derivative of silu), the library's exponential is good to (2 + 1.173 |g|) 2^-23 and enters with a
factor below 1, and the sum, quotient and product round once each: in all below (24 + 8 |g|) u.  A result
in bf16 is off by half a step of bf16, 2^-8 of itself, more.
"""
import pytest
import torch

import sparse_expert_ffn_router_b200 as colibri

F32, BF16 = colibri.COLIBRI_F32, colibri.COLIBRI_BF16
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
U = 2.0 ** -24
HALF = {F32: 0.0, BF16: torch.finfo(torch.bfloat16).eps / 2}
SENTINEL = 7.0


# ------------------------------------------------------------------ refusals (no GPU needed)

def _quant(**kw):
    a = dict(x=16, act_dtype=BF16, rows=4, cols=64, ldx=64, q=16, ldq=64, scale=16)
    a.update(kw)
    return colibri.colibri_quantize_rows(*a.values())


def _gemm(**kw):
    a = dict(A=16, lda=64, a_scale=16, W=16, ldw=64, w_scale=16, M=4, N=8, K=64, y=16, ldy=8, out_dtype=BF16)
    a.update(kw)
    return colibri.colibri_int_gemm(*a.values())


def _experts(call, **kw):
    a = dict(A=16, lda=64, a_scale=16, rows=4, offsets=16, num_experts=2, W=16, w_stride=2 * 8 * 64, w_scale=16,
             s_stride=16, N=8, K=64, y=16, ldy=8, out_dtype=BF16)
    a.update(kw)
    return call(*a.values())


def _refused(code, fn, **kw):
    with pytest.raises(colibri.ColibriError) as ei:
        fn(**kw)
    assert ei.value.status == code, str(ei.value)
    assert colibri.colibri_last_error()


INVALID, ALIGN, UNSUP = -1, -2, -3


@pytest.mark.parametrize("code,kw", [
    (UNSUP, dict(act_dtype=colibri.COLIBRI_I8)), (INVALID, dict(rows=-1)), (INVALID, dict(cols=0)),
    (INVALID, dict(cols=72, ldx=80, ldq=80)), (INVALID, dict(cols=131072, ldx=131072, ldq=131072)),
    (INVALID, dict(ldx=48)), (INVALID, dict(ldq=48)), (ALIGN, dict(ldx=68)), (ALIGN, dict(ldq=72)),
    (INVALID, dict(x=None)), (INVALID, dict(q=None)), (INVALID, dict(scale=None)),
    (ALIGN, dict(x=8)), (ALIGN, dict(scale=20)), (INVALID, dict(ldx=1 << 31)), (INVALID, dict(rows=(1 << 24) + 1)),
])
def test_quantize_rows_refuses(code, kw):
    _refused(code, _quant, **kw)


@pytest.mark.parametrize("code,kw", [
    (UNSUP, dict(out_dtype=colibri.COLIBRI_I8)), (INVALID, dict(M=-1)), (INVALID, dict(N=0)),
    (INVALID, dict(K=8)), (INVALID, dict(K=40)), (INVALID, dict(K=131072, lda=131072, ldw=131072)),
    (INVALID, dict(lda=48)), (INVALID, dict(ldw=48)), (INVALID, dict(ldy=7)), (ALIGN, dict(lda=72)),
    (ALIGN, dict(ldw=72)), (INVALID, dict(A=None)), (INVALID, dict(a_scale=None)), (INVALID, dict(W=None)),
    (INVALID, dict(w_scale=None)), (INVALID, dict(y=None)), (ALIGN, dict(A=24)), (ALIGN, dict(y=2)),
    (INVALID, dict(N=(1 << 20) + 1, ldy=1 << 21)),
])
def test_int_gemm_refuses(code, kw):
    _refused(code, _gemm, **kw)


@pytest.mark.parametrize("call", ["colibri_int_gemm_experts", "colibri_int_swiglu_experts"])
@pytest.mark.parametrize("code,kw", [
    (UNSUP, dict(out_dtype=5)), (INVALID, dict(rows=-1)), (INVALID, dict(num_experts=0)),
    (INVALID, dict(num_experts=257)), (INVALID, dict(N=0)), (INVALID, dict(K=24)), (INVALID, dict(lda=48)),
    (ALIGN, dict(lda=72)), (INVALID, dict(w_stride=8 * 64 - 16)), (ALIGN, dict(w_stride=16 * 64 + 8)),
    (INVALID, dict(s_stride=7)), (INVALID, dict(ldy=4)), (INVALID, dict(offsets=None)), (ALIGN, dict(offsets=4)),
    (INVALID, dict(A=None)), (INVALID, dict(y=None)), (INVALID, dict(w_stride=(1 << 38) + 16)),
])
def test_expert_products_refuse(call, code, kw):
    _refused(code, lambda **k: _experts(getattr(colibri, call), **k), **kw)


def test_swiglu_needs_both_matrices_in_a_stride():
    _refused(INVALID, lambda **k: _experts(colibri.colibri_int_swiglu_experts, **k), w_stride=2 * 8 * 64 - 16)
    _refused(INVALID, lambda **k: _experts(colibri.colibri_int_swiglu_experts, **k), s_stride=15)


def test_no_rows_launch_nothing():
    # zero rows are fine with any buffers, also where there is no device
    _quant(rows=0, x=None, q=None, scale=None)
    _gemm(M=0, A=None, y=None)
    for call in (colibri.colibri_int_gemm_experts, colibri.colibri_int_swiglu_experts):
        _experts(call, rows=0, offsets=None)


@pytest.mark.gpu
def test_host_buffers_are_refused():
    host = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    s = torch.zeros(4, device="cuda")
    _refused(INVALID, _quant, x=host, q=q, scale=s)
    _refused(INVALID, _gemm, A=q, a_scale=s, W=q, w_scale=host, N=4, y=s, M=1, ldy=4, out_dtype=F32)


# ------------------------------------------------------------------ rows

def _ref_quantize(x):
    """Scale and integers in 64 bits; rows that are all zero, tiny or not finite by their rule."""
    xd = x.double()
    top = xd.abs().amax(1)
    s = (top / 127.0).float()
    bad = ~torch.isfinite(xd).all(1)
    flat = (s < 2.0 ** -126) & ~bad
    s[flat] = 1.0
    q = torch.round(xd / s.double()[:, None])
    q[flat | bad] = 0
    s[bad] = float("nan")
    return q.to(torch.int8), s


def _quantize(x, ldx=None, ldq=None, cols=None, act=None):
    rows, cols = x.shape
    ldx, ldq = ldx or cols, ldq or cols
    xb = torch.full((rows, ldx), SENTINEL, dtype=x.dtype, device="cuda")
    xb[:, :cols] = x
    q = torch.full((rows + 1, ldq), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), SENTINEL, device="cuda")
    colibri.colibri_quantize_rows(xb, F32 if x.dtype == torch.float32 else BF16, rows, cols, ldx, q, ldq, s,
                                  torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert (q[:, cols:] == 77).all() and (q[rows:] == 77).all() and s[rows].item() == SENTINEL
    return q[:rows, :cols].cpu(), s[:rows].cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,ldx,ldq", [
    (1, 16, 0, 0), (3, 64, 72, 80), (9, 2048, 0, 0), (7, 2064, 0, 0), (5, 4096, 4104, 4112), (2, 16384, 0, 0),
    (3, 16400, 0, 0), (2, 131056, 0, 0), (20000, 48, 0, 0),
])
def test_quantize_rows(dt, rows, cols, ldx, ldq):
    g = torch.Generator().manual_seed(rows * 131 + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))).to(dt)
    q, s = _quantize(x, ldx, ldq)
    rq, rs = _ref_quantize(x)
    assert torch.equal(s, rs)
    assert torch.equal(q, rq)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_quantize_rows_special_rows(dt):
    cols = 96
    x = torch.zeros(12, cols, dtype=torch.float32)
    x[1] = torch.arange(cols) % 128 - 47.0  # with a 127 below: every value is an integer multiple of the scale
    x[1, 0] = 127.0
    x[2] = torch.arange(cols) + 0.5          # halves, to even
    x[2, 0] = -127.0
    x[3, 5] = float("nan")
    x[4, 6] = float("inf")
    x[5, 7] = float("-inf")
    x[6] = 1e-40                             # below 127 * 2^-126
    x[7, 3] = 127 * 2.0 ** -126              # the smallest scale
    x[7, 4] = 64 * 2.0 ** -126
    x[8] = torch.finfo(dt).max
    x[9] = -torch.finfo(dt).max
    x[9, 1] = 1.0
    x[10, 95] = 3.0                          # only the last value
    x = x.to(dt)
    q, s = _quantize(x)
    rq, rs = _ref_quantize(x)
    assert torch.equal(torch.isnan(s), torch.isnan(rs))
    assert torch.equal(s.nan_to_num(0.0), rs.nan_to_num(0.0))
    assert torch.equal(q, rq)
    assert s[0] == 1.0 and (q[0] == 0).all() and torch.isnan(s[3:6]).all() and (q[3:6] == 0).all()


@pytest.mark.gpu
def test_quantize_rows_near_ties():
    # fp32 values one ulp to either side of (n + 1/2) s, and on it where it is representable
    g = torch.Generator().manual_seed(5)
    rows, cols = 64, 127 * 8
    top = torch.exp(4 * torch.randn(rows, 1, generator=g))
    s = (top.double() / 127).float()
    n = torch.arange(cols) % 127
    x = ((n + 0.5).double() * s.double()).float()
    step = torch.randint(-2, 3, (rows, cols), generator=g)
    for k in (1, 2):
        x = torch.where(step >= k, torch.nextafter(x, torch.tensor(float("inf"))), x)
        x = torch.where(step <= -k, torch.nextafter(x, torch.tensor(0.0)), x)
    x = x * (1 - 2 * torch.randint(0, 2, (rows, cols), generator=g))
    x = torch.minimum(torch.maximum(x, -top), top)
    x[:, 0:1] = top
    pad = torch.zeros(rows, 8)
    x = torch.cat([x, pad], 1)[:, : (cols + 15) // 16 * 16]
    q, sg = _quantize(x)
    rq, rs = _ref_quantize(x)
    assert torch.equal(sg, rs) and torch.equal(q, rq)


# ------------------------------------------------------------------ products

def _ints(g, *shape, lo=-127, hi=128):
    return torch.randint(lo, hi, shape, generator=g, dtype=torch.int32).to(torch.int8)


def _check(got, ref, rel, out):
    got, ref = got.double(), ref.double()
    tol = ref.abs() * (rel + HALF[out]) * (1 + 1e-6) + 1e-37
    bad = (got - ref).abs() > tol
    assert torch.isfinite(got).all()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values off, first at {bad.nonzero()[0].tolist()}"


def _ref_product(q, s, w, t):
    return (q.double() @ w.double().T) * s.double()[:, None] * t.double()[None, :]


def _padded(v, ld, rows_more=0, fill=0):
    out = torch.full((v.shape[0] + rows_more, ld), fill, dtype=v.dtype, device="cuda")
    out[: v.shape[0], : v.shape[1]] = v.cuda()
    return out


def _run_gemm(q, s, w, t, out, lda=None, ldw=None, ldy=None, stream=None):
    M, K = q.shape
    N = w.shape[0]
    lda, ldw, ldy = lda or K, ldw or K, ldy or N
    y = torch.full((M + 2, ldy), SENTINEL, dtype=TORCH[out], device="cuda")
    qa, wa = _padded(q, lda, fill=99), _padded(w, ldw, fill=99)
    sd, td = s.cuda(), t.cuda()
    stream = stream or torch.cuda.current_stream()
    stream.wait_stream(torch.cuda.current_stream())
    colibri.colibri_int_gemm(qa, lda, sd, wa, ldw, td, M, N, K, y, ldy, out, stream)
    torch.cuda.synchronize()
    assert (y[:, N:] == SENTINEL).all() and (y[M:] == SENTINEL).all()
    return y[:M, :N].cpu()


def _problem(M, N, K, seed, lo=-127, hi=128):
    g = torch.Generator().manual_seed(seed)
    s = torch.exp(torch.randn(M, generator=g)) / 50
    t = (0.5 + torch.rand(N, generator=g)) / 127
    return _ints(g, M, K, lo=lo, hi=hi), s, _ints(g, N, K, lo=lo, hi=hi), t


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 4096, 4096), (1, 77, 1040), (2, 130, 48), (5, 129, 512), (8, 256, 2064), (9, 64, 128), (16, 1000, 4096),
    (17, 100, 144), (31, 333, 272), (33, 2048, 1024), (64, 96, 4112), (100, 4096, 1360), (127, 511, 256), (128, 256, 512),
    (129, 257, 80), (200, 1536, 4096), (255, 72, 640), (256, 512, 128), (257, 1025, 192), (513, 300, 384), (1000, 2000, 1008),
    (2049, 520, 272), (300, 8192, 320),
])
def test_int_gemm(M, N, K, out):
    q, s, w, t = _problem(M, N, K, M * 7919 + N * 31 + K)
    _check(_run_gemm(q, s, w, t, out), _ref_product(q, s, w, t), 4 * U, out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K,lda,ldw,ldy", [
    (3, 50, 64, 80, 96, 51), (12, 130, 1040, 1056, 2064, 131), (40, 77, 256, 272, 256, 80), (150, 264, 128, 144, 160, 267),
    (600, 515, 512, 528, 544, 520), (300, 512, 256, 256, 256, 513),
])
def test_int_gemm_strides(M, N, K, lda, ldw, ldy, out):
    q, s, w, t = _problem(M, N, K, 17 + M)
    _check(_run_gemm(q, s, w, t, out, lda, ldw, ldy), _ref_product(q, s, w, t), 4 * U, out)


def _tiles(rows, groups, N, cols):
    """Upper bound on the 128 x `cols` tiles of a product: more than there are SMs run as 256 x 256 pair tiles."""
    return (rows // 128 + groups) * -(-N // cols)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [
    (17, 19500, 16), (20, 19000, 400), (32, 19201, 144), (33, 20001, 272), (64, 19456, 128), (100, 19208, 80), (128, 19600, 64),
    (129, 9700, 144), (256, 9601, 208), (257, 9001, 144), (300, 8192, 1040), (513, 5000, 272), (1500, 2100, 80), (4100, 1040, 640),
])
def test_int_gemm_pair_tiles(M, N, K, out):
    assert -(-M // 128) * -(-N // 128) > torch.cuda.get_device_properties(0).multi_processor_count
    q, s, w, t = _problem(M, N, K, M * 7919 + N * 31 + K)
    _check(_run_gemm(q, s, w, t, out, ldy=N + 3 if M % 2 else N), _ref_product(q, s, w, t), 4 * U, out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [
    (17, 1, 16), (17, 128, 5120), (18, 129, 5136), (24, 300, 5104), (25, 257, 5264), (31, 2049, 144), (32, 10000, 272),
    (32, 1030, 8208), (33, 1030, 8208), (33, 129, 5120),
])
def test_int_gemm_few_rows(M, N, K, out):
    # 17 to 33 rows, where the kind of tile depends on K
    q, s, w, t = _problem(M, N, K, M * 131 + N + K)
    _check(_run_gemm(q, s, w, t, out, ldy=N + 3), _ref_product(q, s, w, t), 4 * U, out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [
    (1, 40001, 48), (16, 80003, 16), (5, 39000, 528), (1, 9472, 4432), (8, 9500, 4416), (8, 9500, 4400), (9, 14337, 2352),
    (9, 14337, 2336), (16, 100001, 336),
])
def test_int_gemm_many_columns(M, N, K, out):
    # at most 16 rows, where the kernel depends on the weights' shape; many groups of columns per block
    q, s, w, t = _problem(M, N, K, M * 131 + N + K)
    _check(_run_gemm(q, s, w, t, out, ldy=N + 1), _ref_product(q, s, w, t), 4 * U, out)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 16, 20, 130, 300])
def test_int_gemm_largest_sums(M):
    # every product at its largest: K * 2^14 just below 2^31
    K = 131056
    q, w = torch.full((M, K), -128, dtype=torch.int8), torch.full((5, K), -128, dtype=torch.int8)
    w[1] = 127
    w[2, ::2] = 127
    s, t = torch.full((M,), 2.0 ** -20), torch.full((5,), 2.0 ** -3)
    _check(_run_gemm(q, s, w, t, F32), _ref_product(q, s, w, t), 4 * U, F32)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (40, 64, 64), (300, 300, 64)])
def test_nan_scale_stays_in_its_row(M, N, K):
    q, s, w, t = _problem(M, N, K, 3)
    s[M // 2] = float("nan")
    y = _run_gemm(q, s, w, t, F32)
    assert torch.isnan(y[M // 2]).all()
    keep = torch.arange(M) != M // 2
    _check(y[keep], _ref_product(q, s, w, t)[keep], 4 * U, F32)


def _experts_case(counts, N, K, seed, swiglu, before=0, after=0):
    g = torch.Generator().manual_seed(seed)
    E, R = len(counts), before + sum(counts) + after
    cols = 2 * N if swiglu else N
    off = torch.tensor([0] + list(counts)).cumsum(0).to(torch.int32) + before
    return dict(q=_ints(g, R, K), s=torch.exp(torch.randn(R, generator=g) / 2) / 60, w=_ints(g, E, cols, K),
                t=(0.5 + torch.rand(E, cols, generator=g)) / (127 * K ** 0.5), off=off, E=E, R=R, N=N, K=K, swiglu=swiglu)


def _ref_experts(c, off=None):
    """(reference rows, |g| of each value or 0, rows that some expert owns)"""
    off = c["off"] if off is None else off
    y, gabs, own = torch.zeros(c["R"], c["N"], dtype=torch.float64), torch.zeros(c["R"], c["N"]), torch.zeros(c["R"], dtype=bool)
    for e in range(c["E"]):
        a, b = int(off[e]), int(off[e + 1])
        v = _ref_product(c["q"][a:b], c["s"][a:b], c["w"][e], c["t"][e])
        own[a:b] = True
        if c["swiglu"]:
            gt, up = v[:, : c["N"]], v[:, c["N"]:]
            gabs[a:b] = gt.abs().float()
            v = gt / (1 + torch.exp(-gt)) * up
        y[a:b] = v
    return y, gabs, own


def _run_experts(c, out, w_more=0, s_more=0, lda=None, ldy=None, off=None):
    E, R, N, K = c["E"], c["R"], c["N"], c["K"]
    cols = c["w"].shape[1]
    lda, ldy, w_stride, s_stride = lda or K, ldy or N, cols * K + w_more, cols + s_more
    w = torch.full((E, w_stride), 99, dtype=torch.int8, device="cuda")
    w[:, : cols * K] = c["w"].reshape(E, -1).cuda()
    t = torch.full((E, s_stride), float("nan"), device="cuda")
    t[:, :cols] = c["t"].cuda()
    y = torch.full((R + 1, ldy), SENTINEL, dtype=TORCH[out], device="cuda")
    offd = (c["off"] if off is None else off).cuda()
    call = colibri.colibri_int_swiglu_experts if c["swiglu"] else colibri.colibri_int_gemm_experts
    q, s = _padded(c["q"], lda, fill=99), c["s"].cuda()
    call(q, lda, s, R, offd, E, w, w_stride, t, s_stride, N, K, y, ldy, out, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert (y[:, N:] == SENTINEL).all() and (y[R:] == SENTINEL).all()
    return y[:R, :N].cpu()


def _check_experts(c, y, out, off=None):
    ref, gabs, own = _ref_experts(c, off)
    assert (y[~own] == SENTINEL).all()
    rel = (24 + 8 * gabs.double()) * U if c["swiglu"] else 4 * U
    _check(y[own], ref[own], rel[own] if c["swiglu"] else rel, out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,K", [
    ((1,), 16, 16), ((0, 1, 0), 40, 48), ((3, 0, 5, 8, 0, 2), 128, 256), ((16, 9, 33), 100, 272), ((64, 1, 63, 65), 192, 128),
    ((130, 0, 255, 1), 264, 512), ((256, 257, 128, 129), 300, 192), ((700, 3, 0, 20), 256, 1024), ((1,) * 256, 64, 64),
    ((0,) * 5, 64, 64), ((17,) * 40, 96, 128), ((40, 300, 90), 520, 1040), ((5, 2000), 72, 144),
])
def test_expert_products(counts, N, K, swiglu, out):
    c = _experts_case(counts, N, K, len(counts) * 101 + N + K, swiglu)
    _check_experts(c, _run_experts(c, out), out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,K", [
    ((3, 0, 5, 8, 0, 2), 4096, 256), ((16, 9, 33), 6400, 144), ((64, 1, 63, 65), 5008, 128), ((130, 0, 255, 1), 5000, 512),
    ((256, 257, 128, 129), 2600, 192), ((700, 3, 0, 20), 2216, 256), ((40, 300, 90), 4005, 208), ((5, 2000), 1300, 144),
    ((33,) * 20, 1000, 64), ((1, 0, 290, 31, 32, 600), 2056, 272), ((0, 0, 0, 4), 5008, 16),
])
def test_expert_products_pair_tiles(counts, N, K, swiglu, out):
    assert _tiles(sum(counts), len(counts), N, 128) > torch.cuda.get_device_properties(0).multi_processor_count
    c = _experts_case(counts, N, K, len(counts) * 7 + N + K, swiglu)
    _check_experts(c, _run_experts(c, out, ldy=N + 5 if K % 32 else None), out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N", [77, 80, 1000, 1008])
@pytest.mark.parametrize("counts,K", [((1, 0, 16, 15), 5120), ((1, 0, 16, 15), 5136), ((32,), 5200), ((2, 30, 1), 5136), ((0, 1), 144)])
def test_expert_products_few_rows(counts, K, N, swiglu, out):
    c = _experts_case(counts, N, K, len(counts) * 13 + N + K, swiglu)
    _check_experts(c, _run_experts(c, out, ldy=N + 5), out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N", [77, 4077])
@pytest.mark.parametrize("counts", [(3, 0, 9), (40, 0, 150), (300, 10, 500)])
def test_expert_products_strides_and_rows_outside(counts, N, swiglu, out):
    # gaps between experts, padded rows, and rows before the first and behind the last group
    c = _experts_case(counts, N, 144, 9, swiglu, before=5, after=70)
    _check_experts(c, _run_experts(c, out, w_more=48, s_more=5, lda=160, ldy=N + 4), out)


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N", [64, 6400])
@pytest.mark.parametrize("scale", [1, 40])
def test_expert_products_bad_offsets(swiglu, N, scale):
    # entries out of range or falling: each counts as the largest so far, within [0, rows]
    c = _experts_case((scale * 5, scale * 7, scale * 4), N, 128, 4, swiglu)
    bad = torch.tensor([-9, scale * 6, scale * 2, 10 ** 9], dtype=torch.int32)
    seen = torch.cummax(bad.clamp(0, c["R"]), 0).values
    _check_experts(c, _run_experts(c, F32, off=bad), F32, off=seen)


@pytest.mark.gpu
def test_two_streams_and_graph():
    """Calls that overlap on two streams, and replays of a captured pair, give what a lone call gives."""
    a, b = _problem(700, 900, 512, 1), _problem(5, 700, 1024, 2)
    ca = _experts_case((100, 0, 300, 7), 256, 256, 6, True)
    alone = [_run_gemm(*a, BF16), _run_gemm(*b, BF16), _run_experts(ca, BF16)]
    dev = [[v.cuda() for v in p] for p in (a, b)]
    e = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in ca.items()}
    ys = [torch.empty(700, 900, dtype=torch.bfloat16, device="cuda"), torch.empty(5, 700, dtype=torch.bfloat16, device="cuda"),
          torch.empty(407, 256, dtype=torch.bfloat16, device="cuda")]
    torch.cuda.synchronize()

    def call(i, stream):
        if i < 2:
            q, s, w, t = dev[i]
            colibri.colibri_int_gemm(q, q.shape[1], s, w, q.shape[1], t, q.shape[0], w.shape[0], q.shape[1], ys[i],
                                     w.shape[0], BF16, stream)
        else:
            colibri.colibri_int_swiglu_experts(e["q"], 256, e["s"], 407, e["off"], 4, e["w"], 512 * 256, e["t"], 512, 256,
                                               256, ys[2], 256, BF16, stream)

    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        for i in range(3):
            call(i, streams[i])
    torch.cuda.synchronize()
    for y, ref in zip(ys, alone):
        assert torch.equal(y.cpu(), ref)
    graphs = []
    for i in range(3):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, torch.cuda.current_stream())
        graphs.append(g)
    for y in ys:
        y.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for y, ref in zip(ys, alone):
        assert torch.equal(y.cpu(), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("act", [F32, BF16])
@pytest.mark.parametrize("T,d,f,E", [(1, 64, 128, 3), (50, 128, 192, 4), (600, 256, 320, 4)])
def test_expert_ffn_from_the_parts(T, d, f, E, act):
    """Scatter, quantise, gate/up, quantise, down, combine: the parts chained as a user would."""
    k = 2
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, d, generator=g).to(TORCH[act])
    rw = (torch.randn(E, d, generator=g) / d ** 0.5).to(TORCH[act])
    w13, w2 = _ints(g, E, 2 * f, d), _ints(g, E, d, f)
    t13, t2 = (0.5 + torch.rand(E, 2 * f, generator=g)) / (127 * d ** 0.5), (0.5 + torch.rand(E, d, generator=g)) / (127 * f ** 0.5)
    R = T * k
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, src, dst = torch.empty(T, k, **i32), torch.empty(R, **i32), torch.empty(T, k, **i32)
    counts, off = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    wt = torch.empty(T, k, device="cuda")
    xp = torch.empty(R, d, dtype=TORCH[act], device="cuda")
    dev = [v.cuda() for v in (x, rw, w13, w2, t13, t2)]
    colibri.colibri_route_noalloc(dev[0], act, T, d, dev[1], None, E, k, idx, wt, counts, off, src, dst, xp)
    colibri.colibri_route_noalloc_check()
    q, s = torch.empty(R, d, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    h, hq, hs = torch.empty(R, f, device="cuda"), torch.empty(R, f, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    yp, y = torch.empty(R, d, dtype=TORCH[act], device="cuda"), torch.empty(T, d, dtype=TORCH[act], device="cuda")
    colibri.colibri_quantize_rows(xp, act, R, d, d, q, d, s)
    colibri.colibri_int_swiglu_experts(q, d, s, R, off, E, dev[2], 2 * f * d, dev[4], 2 * f, f, d, h, f, F32)
    colibri.colibri_quantize_rows(h, F32, R, f, f, hq, f, hs)
    colibri.colibri_int_gemm_experts(hq, f, hs, R, off, E, dev[3], d * f, dev[5], d, d, f, yp, d, act)
    colibri.colibri_combine(yp, act, dst, wt, T, k, d, y)
    torch.cuda.synchronize()
    # the same steps in 64 bits, on the integers of each step (they are checked bit for bit above)
    rq, rs = _ref_quantize(xp.cpu())
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)
    c = dict(q=rq, s=rs, w=w13, t=t13, off=off.cpu(), E=E, R=R, N=f, K=d, swiglu=True)
    _check_experts(c, h.cpu(), F32)
    rhq, rhs = _ref_quantize(h.cpu())
    assert torch.equal(hq.cpu(), rhq) and torch.equal(hs.cpu(), rhs)
    c = dict(q=rhq, s=rhs, w=w2, t=t2, off=off.cpu(), E=E, R=R, N=d, K=f, swiglu=False)
    _check_experts(c, yp.cpu(), act)
    # k products and sums of at most sum |w Yp|, each rounded once, then the output's rounding
    terms = wt.cpu().double()[:, :, None] * yp.cpu().double()[dst.cpu().long()]
    bound = terms.abs().sum(1) * 2 * k * U + terms.sum(1).abs() * HALF[act] * 1.001
    assert ((y.cpu().double() - terms.sum(1)).abs() <= bound + 1e-37).all()


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts", [(1, 2), (150, 40)])
def test_offsets_past_32_bits(counts, swiglu):
    """Rows, experts and output rows that lie more than 2^31 bytes (and elements) apart."""
    c = _experts_case(counts, 48, 64, 3, swiglu)
    R, N, K, cols = c["R"], 48, 64, c["w"].shape[1]
    far = (1 << 31) // (R - 1) // 16 * 16 + 16       # the last row starts past 2^31 elements
    w_stride = (1 << 31) + 16
    a = torch.empty(far * (R - 1) + K, dtype=torch.int8, device="cuda")
    rows = torch.arange(R, device="cuda")[:, None] * far
    a[rows + torch.arange(K, device="cuda")] = c["q"].cuda()
    w = torch.empty(w_stride + cols * K, dtype=torch.int8, device="cuda")
    for e in range(2):
        w[e * w_stride: e * w_stride + cols * K] = c["w"][e].reshape(-1).cuda()
    y = torch.empty(far * (R - 1) + N, dtype=torch.bfloat16, device="cuda")
    s, t, off = c["s"].cuda(), c["t"].cuda(), c["off"].cuda()
    call = colibri.colibri_int_swiglu_experts if swiglu else colibri.colibri_int_gemm_experts
    call(a, far, s, R, off, 2, w, w_stride, t, cols, N, K, y, far, BF16, torch.cuda.current_stream())
    colibri.colibri_int_check(torch.cuda.current_stream())
    _check_experts(c, y[rows + torch.arange(N, device="cuda")].cpu(), BF16)
    if not swiglu:
        q, sq, wt = c["q"], c["s"], c["w"][1]
        y.zero_()
        colibri.colibri_int_gemm(a, far, s, w.data_ptr() + w_stride, K, t[1], R, N, K, y, far, BF16,
                                 torch.cuda.current_stream())
        torch.cuda.synchronize()
        _check(y[rows + torch.arange(N, device="cuda")].cpu(), _ref_product(q, sq, wt, c["t"][1]), 4 * U, BF16)
    xq, xs = torch.empty(far * (R - 1) + K, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    x = torch.empty(far * (R - 1) + K, dtype=torch.bfloat16, device="cuda")
    xv = torch.randn(R, K, device="cuda").bfloat16()
    x[rows + torch.arange(K, device="cuda")] = xv
    colibri.colibri_quantize_rows(x, BF16, R, K, far, xq, far, xs)
    torch.cuda.synchronize()
    rq, rs = _ref_quantize(xv.cpu())
    assert torch.equal(xq[rows + torch.arange(K, device="cuda")].cpu(), rq) and torch.equal(xs.cpu(), rs)


@pytest.mark.gpu
def test_check_reports_nothing_after_good_calls():
    q, s, w, t = _problem(300, 300, 256, 8)
    _run_gemm(q, s, w, t, F32)
    colibri.colibri_int_check()
    colibri.colibri_int_check(torch.cuda.Stream())


@pytest.mark.gpu
def test_two_host_threads():
    """Context-free calls from two host threads, each with its own stream and its own last error."""
    import threading

    probs = [_problem(90, 700, 512, 21), _problem(9, 333, 1024, 22)]
    alone = [_run_gemm(*p, F32) for p in probs]
    dev = [[v.cuda() for v in p] for p in probs]
    torch.cuda.synchronize()
    out, errors = [None, None], []

    def work(i):
        try:
            q, s, w, t = dev[i]
            st = torch.cuda.Stream()
            y = torch.empty(q.shape[0], w.shape[0], device="cuda")
            st.wait_stream(torch.cuda.default_stream())
            for _ in range(50):
                colibri.colibri_int_gemm(q, q.shape[1], s, w, q.shape[1], t, q.shape[0], w.shape[0], q.shape[1], y, w.shape[0], F32, st)
                _refused(INVALID, _gemm, K=8 + 16 * i, lda=64)
                assert f"K={8 + 16 * i}" in colibri.colibri_last_error()
            st.synchronize()
            out[i] = y.cpu()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    for y, ref in zip(out, alone):
        assert torch.equal(y, ref)
