"""Cases of the operators around the MoE layer that serve it at few tokens and in 8-bit integers.

Three operators:

* ``linear``   rows of activations rounded to int8 with one scale per row, then their product with
               int8 weights that carry one scale per output channel:
               ``y[m][n] = s_m t_n sum_k q[m][k] w[n][k]``.
* ``experts``  the same product for rows grouped by expert: the gate and up projections with
               ``h = silu(g) * u`` (``swiglu``), and the down projection (plain).
* ``layer``    a whole MoE layer (router, top-k, SwiGLU experts, weighted sum, shared expert) for
               at most 16 tokens.

``own`` false computes them in plain torch operations; ``own`` true calls the library.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token through a square projection of a 4096-wide model: a latency-bound call
        {"name": "linear 1 token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "act": "bf16", "out": "bf16"},
        # a small decode batch through a wide projection: a stream over the weights
        {"name": "linear 13 tokens", "op": "linear", "M": 13, "N": 14336, "K": 4096, "act": "bf16", "out": "bf16"},
        # a medium batch, odd sizes, fp32 in and out: a small model's projection in fp32
        {"name": "linear ragged f32", "op": "linear", "M": 150, "N": 4999, "K": 1360, "act": "f32", "out": "f32"},
        # prefill of 4096 tokens through the widest projection
        {"name": "linear prefill", "op": "linear", "M": 4096, "N": 14336, "K": 4096, "act": "bf16", "out": "bf16"},
        # gate and up projections of 32 decoded tokens, top-2 of 8 experts: a stream over the weights
        {"name": "experts decode", "op": "experts", "swiglu": True, "R": 64, "E": 8, "N": 14336, "K": 4096,
         "skew": 0.0, "empty": 0, "out": "bf16"},
        # gate and up projections of a prefill of 4096 tokens, top-2 of 8 experts
        {"name": "experts prefill", "op": "experts", "swiglu": True, "R": 8192, "E": 8, "N": 14336, "K": 4096,
         "skew": 0.0, "empty": 0, "out": "bf16"},
        # down projection of a fine-grained layer: 8192 tokens, top-4 of 128 small experts
        {"name": "experts fine down", "op": "experts", "swiglu": False, "R": 32768, "E": 128, "N": 2048, "K": 768,
         "skew": 0.0, "empty": 0, "out": "bf16"},
        # down projection under skewed routing: two experts take nearly all rows, four take none
        {"name": "experts skewed down", "op": "experts", "swiglu": False, "R": 4096, "E": 16, "N": 4096, "K": 8192,
         "skew": 0.98, "empty": 4, "out": "bf16"},
        # three tokens through a tiny fp32 layer: launches and barriers only
        {"name": "layer tiny f32", "op": "layer", "T": 3, "d": 256, "f": 512, "E": 8, "k": 2, "fs": 0,
         "bias": False, "dt": "f32"},
        # one token through a layer with 8 large experts: a stream over two experts' weights
        {"name": "layer 1 token", "op": "layer", "T": 1, "d": 4096, "f": 14336, "E": 8, "k": 2, "fs": 0,
         "bias": False, "dt": "bf16"},
        # eight tokens through 128 small experts, top-4, with a shared expert
        {"name": "layer fine shared", "op": "layer", "T": 8, "d": 2048, "f": 768, "E": 128, "k": 4, "fs": 1536,
         "bias": True, "dt": "bf16"},
        # sixteen tokens through 8 large experts: nearly every expert is touched
        {"name": "layer 16 tokens", "op": "layer", "T": 16, "d": 4096, "f": 14336, "E": 8, "k": 2, "fs": 0,
         "bias": False, "dt": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "experts", "layer"])
    if op == "linear":
        M, N, K = _log(rng, 1, 8192), _log(rng, 64, 14336), 16 * _log(rng, 4, 512)
        while M * N * K > 4096 * 14336 * 4096:
            M = max(1, M // 2)
        act = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "M": M, "N": N, "K": K, "act": act, "out": act}
    if op == "experts":
        swiglu = rng.random() < 0.5
        E = _log(rng, 2, 128)
        R, N, K = _log(rng, 1, 32768), 16 * _log(rng, 8, 896), 64 * _log(rng, 2, 128)
        while E * N * K * (2 if swiglu else 1) > 8 * 2 * 14336 * 4096 and E > 2:
            E = max(2, E // 2)
        while R * N * K * (2 if swiglu else 1) > 8192 * 2 * 14336 * 4096 / 4:
            R = max(1, R // 2)
        skew = rng.choice([0.0, 0.0, round(rng.uniform(0.3, 0.9), 2)])
        return {"op": op, "swiglu": swiglu, "R": R, "E": E, "N": N, "K": K, "skew": skew,
                "empty": rng.randint(0, max(0, E - 3)) if rng.random() < 0.3 else 0,
                "out": rng.choice(["bf16", "bf16", "f32"])}
    T, E, dt = rng.randint(1, 16), _log(rng, 2, 128), rng.choice(["bf16", "bf16", "bf16", "f32"])
    d, f, k = 64 * _log(rng, 2, 64), 64 * _log(rng, 1, 224), rng.randint(1, min(8, E))
    while (E * d * f > 8 * 4096 * 14336 or T * k * d * f > 16 * 4096 * 14336) and f > 64:
        f = max(64, f // 128 * 64)
    fs = 64 * _log(rng, 1, 32) if rng.random() < 0.4 else 0
    return {"op": op, "T": T, "d": d, "f": f, "E": E, "k": k, "fs": fs, "bias": rng.random() < 0.3, "dt": dt}


def _counts(case, seed):
    """Rows of each expert, from the seed: uniform draws, `skew` of them on experts 0 and 1, the last `empty`
    experts without any."""
    E, R = case["E"], case["R"]
    live = E - case["empty"]
    p = np.full(E, 0.0)
    p[:live] = 1.0 / live
    if case["skew"]:
        two = min(2, live)
        p[:live] = (1.0 - case["skew"]) / live
        p[:two] += case["skew"] / two
    return np.random.RandomState(seed % (1 << 31)).multinomial(R, p / p.sum())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dt=torch.float32):
        return torch.empty(*shape, dtype=dt, device="cuda").normal_(0.0, std, generator=g)

    def ints(*shape):
        return torch.empty(*shape, dtype=torch.int8, device="cuda").random_(-127, 128, generator=g)

    def scales(n, fan_in):
        return torch.empty(n, device="cuda").uniform_(0.5, 1.5, generator=g) / (127.0 * math.sqrt(fan_in))

    s = dict(case)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        # token rows differ in size, and a few channels stand out, as a model's activations do
        x = normal(M, K) * torch.exp(normal(M, 1, std=0.5))
        x[:, :: max(1, K // 7)] *= 8.0
        s.update(x=x.to(DT[case["act"]]), w=ints(N, K), ws=scales(N, K),
                 q=torch.empty(M, K, dtype=torch.int8, device="cuda"), xs=torch.empty(M, device="cuda"),
                 y=torch.empty(M, N, dtype=DT[case["out"]], device="cuda"))
    elif case["op"] == "experts":
        R, E, N, K = case["R"], case["E"], case["N"], case["K"]
        cols = 2 * N if case["swiglu"] else N
        counts = _counts(case, seed)
        s.update(q=ints(R, K), qs=torch.exp(normal(R, std=0.5)) * (3.0 / 127.0), w=ints(E, cols, K),
                 ws=scales(E * cols, K).view(E, cols),
                 offsets=torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda"),
                 most=int(counts.max()),  # known to a program that plans its batch
                 y=torch.empty(R, N, dtype=DT[case["out"]], device="cuda"))
    else:
        T, d, f, E, fs, dt = case["T"], case["d"], case["f"], case["E"], case["fs"], DT[case["dt"]]
        stride = -(-3 * d * f // 128) * 128  # elements between experts: 128-byte aligned starts

        def ffn(buf, d, f):
            buf[: 2 * f * d].normal_(0.0, 1.0 / math.sqrt(d), generator=g)
            buf[2 * f * d: 3 * f * d].normal_(0.0, 1.0 / math.sqrt(f), generator=g)

        ew = torch.zeros(E, stride, dtype=dt, device="cuda")
        for e in range(E):
            ffn(ew[e], d, f)
        sw = None
        if fs:
            sw = torch.empty(3 * d * fs, dtype=dt, device="cuda")
            ffn(sw, d, fs)
        s.update(x=normal(T, d, dt=dt), rw=normal(E, d, std=1.0 / math.sqrt(d), dt=dt),
                 rb=normal(E, std=0.5) if case["bias"] else None, ew=ew, sw=sw,
                 y=torch.empty(T, d, dtype=dt, device="cuda"))
        if own:
            import sparse_expert_ffn_router_b200 as colibri

            code = {"f32": colibri.COLIBRI_F32, "bf16": colibri.COLIBRI_BF16}[case["dt"]]
            s["layer"] = colibri.MoELayer(d, f, E, case["k"], fs, code, code, max_tokens=T)
    return s


def _run_own(s):
    import sparse_expert_ffn_router_b200 as colibri

    code = {"f32": colibri.COLIBRI_F32, "bf16": colibri.COLIBRI_BF16}
    stream = torch.cuda.current_stream()
    if s["op"] == "linear":
        M, N, K = s["M"], s["N"], s["K"]
        colibri.colibri_quantize_rows(s["x"], code[s["act"]], M, K, K, s["q"], K, s["xs"], stream)
        colibri.colibri_int_gemm(s["q"], K, s["xs"], s["w"], K, s["ws"], M, N, K, s["y"], N, code[s["out"]], stream)
        return {"y": s["y"], "scale": s["xs"]}
    if s["op"] == "experts":
        R, E, N, K = s["R"], s["E"], s["N"], s["K"]
        call = colibri.colibri_int_swiglu_experts if s["swiglu"] else colibri.colibri_int_gemm_experts
        cols = 2 * N if s["swiglu"] else N
        call(s["q"], K, s["qs"], R, s["offsets"], E, s["w"], cols * K, s["ws"], cols, N, K, s["y"], N,
             code[s["out"]], stream)
        return {"y": s["y"]}
    s["layer"].decode(s["x"], s["rw"], s["rb"], s["ew"], s["y"], shared_w=s["sw"], stream=stream)
    return {"y": s["y"]}


def _swiglu(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def run(state):
    if own:
        return _run_own(state)
    s = state
    if s["op"] == "linear":
        x = s["x"].float()
        top = x.abs().amax(1)
        # tensors on both sides: a division by a Python number is a product with its reciprocal
        scale = top / torch.full_like(top, 127.0)
        scale = torch.where(scale < 2.0 ** -126, torch.ones_like(scale), scale)
        # in 64 bits: a quotient next to a half goes to the same side everywhere
        q = torch.round(x.double() / scale.double()[:, None]).float()
        y = (q @ s["w"].float().T) * (scale[:, None] * s["ws"][None, :])
        return {"y": y.to(s["y"].dtype), "scale": scale}
    if s["op"] == "experts":
        R, E, N, K = s["R"], s["E"], s["N"], s["K"]
        row = torch.arange(R, device="cuda")
        e = torch.searchsorted(s["offsets"][1:].contiguous(), row, right=True)
        at = row - s["offsets"].long()[e]
        a = torch.zeros(E, s["most"], K, device="cuda")
        a[e, at] = s["q"].float()
        p = torch.bmm(a, s["w"].float().transpose(1, 2)) * s["ws"][:, None, :]
        p = p[e, at] * s["qs"][:, None]
        if s["swiglu"]:
            p = _swiglu(p[:, :N], p[:, N:])
        return {"y": p.to(s["y"].dtype)}
    T, d, f, k, fs = s["T"], s["d"], s["f"], s["k"], s["fs"]
    x = s["x"].float()
    # in 64 bits: the choice between two experts with nearly the same logit
    logits = s["x"].double() @ s["rw"].double().T
    if s["rb"] is not None:
        logits = logits + s["rb"].double()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = idx[:, :k].reshape(-1)
    p = torch.exp(top[:, :k] - top[:, :1])
    p = (p / p.sum(1, keepdim=True)).float()
    xr = x.repeat_interleave(k, 0)[:, :, None]
    w13 = s["ew"][:, : 2 * f * d].index_select(0, idx).view(T * k, 2 * f, d)
    gu = torch.bmm(w13.float(), xr)[:, :, 0]
    h = _swiglu(gu[:, :f], gu[:, f:])
    w2 = s["ew"][:, 2 * f * d: 3 * f * d].index_select(0, idx).view(T * k, d, f)
    o = torch.bmm(w2.float(), h[:, :, None])[:, :, 0].view(T, k, d)
    y = (o * p[:, :, None]).sum(1)
    if fs:
        w = s["sw"].float()
        gu = x @ w[: 2 * fs * d].view(2 * fs, d).T
        y = y + _swiglu(gu[:, :fs], gu[:, fs:]) @ w[2 * fs * d:].view(d, fs).T
    return {"y": y.to(s["y"].dtype)}


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * size[case["act"]] + N * K + 4 * N + 4 * M + M * N * size[case["out"]],
                "flops": 2.0 * M * N * K}
    if case["op"] == "experts":
        R, E, N, K = case["R"], case["E"], case["N"], case["K"]
        cols = 2 * N if case["swiglu"] else N
        live = E - case["empty"]
        hit = 0.0  # experts that are expected to have rows: an expert without any is not read
        for e in range(live):
            p = (1.0 - case["skew"]) / live + (case["skew"] / min(2, live) if e < 2 else 0.0)
            hit += 1.0 - (1.0 - min(1.0, p)) ** R
        return {"bytes": R * (K + 4) + hit * cols * (K + 4) + 4 * (E + 1) + R * N * size[case["out"]],
                "flops": 2.0 * R * cols * K}
    T, d, f, E, k, fs, b = case["T"], case["d"], case["f"], case["E"], case["k"], case["fs"], size[case["dt"]]
    hit = E * (1.0 - (1.0 - k / E) ** T)  # experts that T tokens are expected to touch
    return {"bytes": b * (hit * 3 * d * f + 3 * d * fs + E * d + 2 * T * d),
            "flops": 2.0 * T * (k * 3 * d * f + 3 * d * fs + E * d)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x = s["x"].double()
        scale = (x.abs().max(1).values / 127.0).float()  # held in 32 bits by definition
        scale[scale < 2.0 ** -126] = 1.0
        q = (x / scale.double().unsqueeze(1)).round()
        acc = torch.matmul(q, s["w"].double().t())
        return {"y": acc * scale.double().unsqueeze(1) * s["ws"].double(), "scale": scale.double()}
    if case["op"] == "experts":
        N = case["N"]
        y = torch.zeros(case["R"], N, dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        for e in range(case["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            v = torch.matmul(s["q"][a:b].double(), s["w"][e].double().t())
            v = v * s["qs"][a:b].double().unsqueeze(1) * s["ws"][e].double()
            y[a:b] = v[:, :N] * torch.sigmoid(v[:, :N]) * v[:, N:] if case["swiglu"] else v
        return {"y": y}
    T, d, f, E, k, fs = case["T"], case["d"], case["f"], case["E"], case["k"], case["fs"]
    x = s["x"].double()

    def ffn(buf, width, v):
        w1, w3, w2 = (buf[i * width * d: (i + 1) * width * d].double() for i in range(3))
        g = torch.mv(w1.view(width, d), v)
        h = g * torch.sigmoid(g) * torch.mv(w3.view(width, d), v)
        return torch.mv(w2.view(d, width), h)

    logits = torch.matmul(x, s["rw"].double().t())
    if s["rb"] is not None:
        logits += s["rb"].double()
    y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for t, row in enumerate(logits.cpu().tolist()):
        chosen = sorted(range(E), key=lambda e: (-row[e], e))[:k]
        p = [math.exp(row[e] - row[chosen[0]]) for e in chosen]
        for e, v in zip(chosen, p):
            y[t] += v / sum(p) * ffn(s["ew"][e], f, x[t])
        if fs:
            y[t] += ffn(s["sw"], fs, x[t])
    return {"y": y}
