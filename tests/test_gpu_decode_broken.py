"""colibri_moe_decode with values that are not finite in the router or the weights: what colibri_moe_forward
makes of them holds here too (the ordinary tolerances are in test_gpu_decode.py)."""
import pytest
import torch

import sparse_expert_ffn_router_b200 as colibri
from tests.test_gpu_decode import BF16, F32, Case

NAN, INF = float("nan"), float("inf")
NEG_NAN = torch.tensor([-4194304], dtype=torch.int32).view(torch.float32)  # 0xffc00000


def _both(c):
    """Outputs and chosen experts of decode and of forward."""
    y = c.decode()
    a = c.routing()
    f = torch.empty_like(y)
    c.layer.forward(c.x, c.rw, c.rb, c.ew, f, shared_w=c.sw, T=c.T)
    b = c.routing()
    torch.cuda.synchronize()
    c.layer.sync_status()
    return y, f, a, b


def _near(a, b, dt):
    far = (a.double() - b.double()).abs().max().item()
    assert far <= (2e-2 if dt == BF16 else 1e-4) * b.double().abs().max().item()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("flags", [0, colibri.COLIBRI_ROUTER_CLAMP, colibri.COLIBRI_ROUTER_RAW_WEIGHTS])
@pytest.mark.parametrize("level", [-20.0, 0.0, 20.0])
@pytest.mark.parametrize("T,E,k", [(6, 5, 2), (16, 40, 4), (3, 256, 8)])
def test_a_nan_logit_is_not_chosen(T, E, k, level, flags, dt):
    c = Case(T, 128, 192, E, k, 64, dt, bias=True, flags=flags)
    c.rb += level  # whatever number a NaN were taken for, it would be chosen at some level
    c.rb[1] = -1e30  # never chosen (with the clamp: at -50)
    clean = c.decode().clone()
    want = c.routing()["topk_idx"]
    assert not (want == 1).any()
    for broken in (NAN, NEG_NAN.item()):
        c.rb[1] = broken
        y, f, a, b = _both(c)
        assert torch.equal(a["topk_idx"], want) and torch.equal(b["topk_idx"], want)
        assert torch.equal(y, clean)
        _near(y, f, dt)
    c.rb[1] = 0.0
    c.rw[1] = NAN
    y, f, a, b = _both(c)
    assert torch.equal(a["topk_idx"], want) and torch.equal(b["topk_idx"], want)
    assert torch.equal(y, clean)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
def test_fewer_numbers_than_choices(dt):
    # one logit is a number: it has all of the weight; none: the token is NaN, as from forward
    c = Case(4, 128, 64, 4, 2, 0, dt)
    c.rb = torch.tensor([NAN, NAN, 0.5, NAN], device="cuda")
    y, f, a, b = _both(c)
    assert (a["topk_idx"][:, 0] == 2).all() and (b["topk_idx"][:, 0] == 2).all()
    assert torch.equal(a["topk_w"], torch.tensor([[1.0, 0.0]] * 4, device="cuda")) and torch.equal(b["topk_w"], a["topk_w"])
    assert len(set(a["topk_idx"][0].tolist())) == 2
    _near(y, f, dt)
    c.rb = torch.tensor([-INF, NAN, -INF, 1.0], device="cuda")  # -inf goes before NaN
    y, f, a, b = _both(c)
    assert a["topk_idx"].tolist() == [[3, 0]] * 4 and b["topk_idx"].tolist() == [[3, 0]] * 4
    _near(y, f, dt)
    c.rb = torch.full((4,), NAN, device="cuda")
    y, f, a, b = _both(c)
    assert torch.isnan(y).all() and torch.isnan(f).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,d,f,fs", [(2, 64, 64, 0), (12, 256, 320, 64), (16, 4096, 192, 0)])
def test_infinite_down_weights(T, d, f, fs, dt):
    """One infinite value in W2: the output it belongs to is an infinity of its and h's sign in every token,
    as the product with h itself gives, and the other outputs stay as they were."""
    c = Case(T, d, f, 3, 2, fs, dt)
    c.rb = torch.tensor([9.0, 0.0, 0.0], device="cuda")  # every token chooses expert 0
    clean = c.decode().clone()
    x = c.x.double()
    w1, w3 = (c.ew[0, i * f * d: (i + 1) * f * d].view(f, d).double() for i in (0, 1))
    g = x @ w1.T
    h = g * torch.sigmoid(g) * (x @ w3.T)
    col = int(h.abs().amin(0).argmax())          # h of this column is clear of zero in every token
    assert float(h[:, col].abs().min()) > 1e-4
    w2 = c.ew[0, 2 * f * d: 3 * f * d].view(d, f)
    rows = [0, 5, d - 1]
    for i, o in enumerate(rows):
        w2[o, col] = INF if i % 2 == 0 else -INF
    y, fwd, _, _ = _both(c)
    for i, o in enumerate(rows):
        want = torch.sign(h[:, col]) * (INF if i % 2 == 0 else -INF)
        assert torch.equal(y[:, o].double(), want) and torch.equal(fwd[:, o].double(), want)
    keep = [o for o in range(d) if o not in rows]
    assert torch.equal(y[:, keep], clean[:, keep])


@pytest.mark.gpu
def test_infinite_down_weights_beside_a_short_h():
    # h is a bf16 number as it is, or just above or below one: nothing, or something of either sign, is left of it
    c = Case(3, 64, 64, 1, 1, 0, BF16)
    f, d = c.f, c.d
    c.x.zero_()
    c.x[:, 0] = torch.tensor([1.0, 1.0, 1.0])
    c.ew.zero_()
    c.ew[0, 0] = 64.0                                          # g = 64, silu(g) = 64
    c.ew[0, f * d] = 1.0                                       # u = 1 (+ small parts of x[1], x[2])
    c.ew[0, f * d + 1] = 2.0 ** -10
    c.ew[0, f * d + 2] = -2.0 ** -10
    c.x[1, 1] = 1.0
    c.x[2, 2] = 1.0
    c.ew[0, 2 * f * d: 3 * f * d].view(d, f)[:, 0] = INF       # h = 64, 64 (1 + 2^-10), 64 (1 - 2^-10)
    y = c.decode()
    torch.cuda.synchronize()
    assert (y == INF).all()
