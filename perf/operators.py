"""The FP8 (E4M3, one scale per 128) linear layer's operators as measured calls: the
RMS norm that writes 8-bit activations, the activation and weight quantizers, the
block-scaled matrix product and the one grouped by expert.

Values are q * s with q in E4M3 and s in fp32: activations have one scale per row
and 128 columns ([M, ceil(K/128)]), weights one per 128 x 128 block
([ceil(N/128), ceil(K/128)]); the last block of a row or column may be short.
"""
import math
import random

import torch

own = False

F8, BF16, F32, F64 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.float64
BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
EPS = 1e-6


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token between two decode layers: launch latency
        {"name": "norm decode", "op": "norm", "M": 1, "K": 5120, "residual": True, "y": False},
        # a mixed batch whose norm feeds FP8 and BF16 consumers; the last block of a row is short
        {"name": "norm mixed odd K", "op": "norm", "M": 333, "K": 2064, "residual": True, "y": True},
        # a long prompt
        {"name": "norm prefill", "op": "norm", "M": 8192, "K": 5120, "residual": True, "y": False},
        # the MLP's gated activation in a small decode batch
        {"name": "gated quantize decode", "op": "quantize", "M": 8, "K": 17408, "gated": True},
        # attention output of a long prompt, ahead of its projection
        {"name": "quantize prefill", "op": "quantize", "M": 4096, "K": 5120, "gated": False},
        # a layer's weights, once at load
        {"name": "quantize weights", "op": "weights", "N": 17408, "K": 5120},
        # one token through the up projection: the weight stream
        {"name": "product decode", "op": "product", "M": 1, "N": 17408, "K": 5120},
        # an odd decode batch through the down projection: few weight rows, long K
        {"name": "product batch down", "op": "product", "M": 47, "N": 5120, "K": 17408},
        # a long prompt through the up projection: the tensor pipe
        {"name": "product prefill", "op": "product", "M": 4096, "N": 17408, "K": 5120},
        # eight tokens with eight experts each: most experts have no row or one
        {"name": "experts decode", "op": "experts", "T": 64, "E": 128, "N": 1536, "K": 2048, "tail": 0},
        # odd sizes, experts without rows, and rows behind the last expert
        {"name": "experts ragged", "op": "experts", "T": 1501, "E": 17, "N": 1001, "K": 2064, "tail": 37},
        # a long prompt's tokens, eight experts each
        {"name": "experts prefill", "op": "experts", "T": 32768, "E": 128, "N": 1536, "K": 2048, "tail": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "weights", "product", "product", "experts", "experts"])
    if op == "norm":
        K = 16 * _log(rng, 8, 1024)
        M = min(_log(rng, 1, 16384), 8192 * 5120 // K)
        return {"op": op, "M": M, "K": K, "residual": rng.random() < 0.7, "y": rng.random() < 0.3}
    if op == "quantize":
        K, gated = 16 * _log(rng, 8, 1088), rng.random() < 0.5
        M = min(_log(rng, 1, 16384), 4096 * 5120 // ((2 if gated else 1) * K))
        return {"op": op, "M": M, "K": K, "gated": gated}
    if op == "weights":
        K = 16 * _log(rng, 8, 1088)
        return {"op": op, "N": min(_log(rng, 64, 50176), 17408 * 5120 // K), "K": K}
    if op == "product":
        K, N = 16 * _log(rng, 8, 1088), _log(rng, 100, 17408)
        M = min(_log(rng, 1, 8192), 4096 * 17408 * 5120 // (N * K))
        return {"op": op, "M": M, "N": N, "K": K}
    E, K, N = _log(rng, 2, 160), 16 * _log(rng, 16, 256), _log(rng, 100, 4096)
    while E * N * K > 128 * 1536 * 2048:
        E = E // 2 + 1
        N = N // 2 + 50
    T = min(_log(rng, 1, 32768), 32768 * 1536 * 2048 // (N * K))
    return {"op": op, "T": T, "E": E, "N": N, "K": K, "tail": rng.choice([0, 0, rng.randrange(1, 300)])}


def _rows_of_experts(case):
    """Rows of each expert: a skewed routing that the sizes alone fix (the seed only
    says which expert gets which count)."""
    E, T = case["E"], case["T"]
    r = random.Random(E * 1000003 + T)
    weights = [1.0 / math.sqrt(1 + i) for i in range(E)]
    counts = [0] * E
    for e in r.choices(range(E), weights, k=T):
        counts[e] += 1
    return counts


def work(case):
    op = case["op"]
    if op == "norm":
        M, K = case["M"], case["K"]
        read = M * K * 2 * (2 if case["residual"] else 1) + K * 2
        wrote = M * K * (1 + (2 if case["residual"] else 0) + (2 if case["y"] else 0)) + M * _ceil(K, BLOCK) * 4
        return {"bytes": read + wrote, "flops": 6 * M * K}
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (4 if case["gated"] else 2) + M * K + M * _ceil(K, BLOCK) * 4,
                "flops": (8 if case["gated"] else 3) * M * K}
    if op == "weights":
        N, K = case["N"], case["K"]
        return {"bytes": 3 * N * K + _ceil(N, BLOCK) * _ceil(K, BLOCK) * 4, "flops": 3 * N * K}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        kb = _ceil(K, BLOCK)
        return {"bytes": M * K + M * kb * 4 + N * K + _ceil(N, BLOCK) * kb * 4 + M * N * 2, "flops": 2 * M * N * K}
    T, N, K = case["T"], case["N"], case["K"]
    kb, active = _ceil(K, BLOCK), sum(c > 0 for c in _rows_of_experts(case))
    return {"bytes": T * K + T * kb * 4 + active * (N * K + _ceil(N, BLOCK) * kb * 4) + T * N * 2 + 4 * case["E"] + 4,
            "flops": 2 * T * N * K}


# ----------------------------------------------------------------- the inputs

def _activations(M, K, gen):
    """Unit-scale activations with a few strong channels, as a residual stream has them."""
    x = torch.randn((M, K), generator=gen, device="cuda", dtype=F32)
    channel = torch.exp(0.5 * torch.randn((K,), generator=gen, device="cuda", dtype=F32))
    strong = torch.rand((K,), generator=gen, device="cuda") < 0.004
    return (x * torch.where(strong, 20.0 * channel, channel)).to(BF16)


def _layer_weights(N, K, gen):
    w = 0.02 * torch.randn((N, K), generator=gen, device="cuda", dtype=F32)
    return (w * (0.5 + 1.5 * torch.rand((N, 1), generator=gen, device="cuda"))).to(BF16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    st = dict(case)
    new = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op in ("norm", "quantize"):
        M, K = case["M"], case["K"]
        kb = _ceil(K, BLOCK)
        st["q"], st["s"] = new((M, K), F8), new((M, kb), F32)
        if op == "norm":
            st["x"] = _activations(M, K, gen)
            st["weight"] = (1.0 + 0.2 * torch.randn((K,), generator=gen, device="cuda", dtype=F32)).to(BF16)
            st["r"] = _activations(M, K, gen) if case["residual"] else None
            st["h"] = new((M, K), BF16) if case["residual"] else None
            st["out"] = new((M, K), BF16) if case["y"] else None
        else:
            st["x"] = _activations(M, K * (2 if case["gated"] else 1), gen)
        return st
    if op == "weights":
        N, K = case["N"], case["K"]
        st["x"] = _layer_weights(N, K, gen)
        st["q"], st["s"] = new((N, K), F8), new((_ceil(N, BLOCK), _ceil(K, BLOCK)), F32)
        return st
    N, K = case["N"], case["K"]
    if op == "product":
        st["x"], st["sx"] = _quantize_rows(_activations(case["M"], K, gen).to(F32))
        st["w"], st["sw"] = _quantize_blocks(_layer_weights(N, K, gen).to(F32))
        st["out"] = new((case["M"], N), BF16)
        return st
    E, T = case["E"], case["T"]
    st["x"], st["sx"] = _quantize_rows(_activations(T + case["tail"], K, gen).to(F32))
    w = new((E, N, K), F8)
    sw = new((E, _ceil(N, BLOCK), _ceil(K, BLOCK)), F32)
    for e in range(E):
        w[e], sw[e] = _quantize_blocks(_layer_weights(N, K, gen).to(F32))
    st["w"], st["sw"] = w, sw
    counts = _rows_of_experts(case)
    random.Random(int(seed)).shuffle(counts)
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    st["most"] = max(counts)
    st["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    st["out"] = new((T + case["tail"], N), BF16)
    return st


# ------------------------------------------------------------- the plain form

def _spread(s, K):
    """One value per column from one per 128 columns."""
    return s.repeat_interleave(BLOCK, dim=-1)[..., :K]


def _quantize_rows(v):
    """fp32 v [M, K] -> E4M3 q [M, K] and fp32 s [M, ceil(K/128)]."""
    M, K = v.shape
    kb = _ceil(K, BLOCK)
    a = torch.nn.functional.pad(v.abs(), (0, kb * BLOCK - K)).reshape(M, kb, BLOCK).amax(-1)
    s = torch.clamp(a / E4M3_MAX, min=SCALE_MIN)
    q = torch.clamp(v * _spread(1.0 / s, K), -E4M3_MAX, E4M3_MAX).to(F8)
    return q, s


def _quantize_blocks(w):
    """fp32 w [N, K] -> E4M3 q [N, K] and fp32 s [ceil(N/128), ceil(K/128)]."""
    N, K = w.shape
    nb, kb = _ceil(N, BLOCK), _ceil(K, BLOCK)
    a = torch.nn.functional.pad(w.abs(), (0, kb * BLOCK - K, 0, nb * BLOCK - N))
    s = torch.clamp(a.reshape(nb, BLOCK, kb, BLOCK).amax((1, 3)) / E4M3_MAX, min=SCALE_MIN)
    r = _spread((1.0 / s).repeat_interleave(BLOCK, dim=0)[:N], K)
    return torch.clamp(w * r, -E4M3_MAX, E4M3_MAX).to(F8), s


def _weights_f32(w, sw):
    N, K = w.shape[-2:]
    return w.to(F32) * _spread(sw.repeat_interleave(BLOCK, dim=-2)[..., :N, :], K)


def _plain(st):
    op = st["op"]
    if op == "norm":
        h = st["x"].to(F32)
        got = {}
        if st["residual"]:
            got["h"] = (h + st["r"].to(F32)).to(BF16)
            h = got["h"].to(F32)
        v = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["weight"].to(F32)
        got["q"], got["s"] = _quantize_rows(v)
        if st["y"]:
            got["y"] = v.to(BF16)
        return got
    if op == "quantize":
        v = st["x"].to(F32)
        if st["gated"]:
            gate, up = v[:, :st["K"]], v[:, st["K"]:]
            v = gate / (1.0 + torch.exp(-gate)) * up
        q, s = _quantize_rows(v)
        return {"q": q, "s": s}
    if op == "weights":
        q, s = _quantize_blocks(st["x"].to(F32))
        return {"q": q, "s": s}
    x = st["x"].to(F32) * _spread(st["sx"], st["K"])
    w = _weights_f32(st["w"], st["sw"])
    if op == "product":
        return {"y": (x @ w.T).to(BF16)}
    # rows padded to the largest expert, one product per expert, and back
    E, T, most = st["E"], st["T"], st["most"]
    off = st["offsets"].to(torch.int64)
    row = torch.arange(T, device="cuda")
    e = torch.searchsorted(off[1:], row, right=True)
    at = e * most + row - off[e]
    padded = torch.zeros((E * most, st["K"]), dtype=F32, device="cuda")
    padded[at] = x[:T]
    y = torch.bmm(padded.reshape(E, most, -1), w.transpose(1, 2)).reshape(E * most, -1)[at]
    out = torch.zeros_like(st["out"])
    out[:T] = y.to(BF16)
    return {"y": out}


# ------------------------------------------------------- the framework's calls

def _own(st):
    import gemm_decode_nvfp4_b200 as nv
    op = st["op"]
    if op == "norm":
        nv.fp8_rmsnorm(st["x"], st["weight"], EPS, residual=st["r"], residual_out=st["h"], y=st["out"], q=st["q"],
                       s=st["s"])
        got = {"q": st["q"], "s": st["s"]}
        if st["residual"]:
            got["h"] = st["h"]
        if st["y"]:
            got["y"] = st["out"]
        return got
    if op == "quantize":
        nv.fp8_quantize(st["x"], st["q"], st["s"], gated=st["gated"])
        return {"q": st["q"], "s": st["s"]}
    if op == "weights":
        nv.fp8_quantize_weights(st["x"], st["q"], st["s"])
        return {"q": st["q"], "s": st["s"]}
    if op == "product":
        nv.fp8_gemm(st["x"], st["sx"], st["w"], st["sw"], st["out"], static_weights=True)
        return {"y": st["out"]}
    nv.fp8_gemm_grouped(st["x"], st["sx"], st["w"], st["sw"], st["offsets"], st["out"], static_weights=True)
    return {"y": st["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------- the definition, in 64 bits

def _e4m3_grid(v):
    """v rounded to the nearest E4M3 value (ties to even, saturating), in 64 bits."""
    v = v.clamp(-448.0, 448.0)
    _, e = torch.frexp(v)                       # |v| = m 2^e with m in [1/2, 1)
    step = torch.exp2(torch.clamp(e.to(F64) - 4.0, min=-9.0))
    return torch.round(v / step) * step


def _exact_scales(v, rows):
    """q and s of v in 64 bits, one scale per `rows` rows and 128 columns."""
    R, K = v.shape
    rb, kb = _ceil(R, rows), _ceil(K, 128)
    big = torch.zeros((rb * rows, kb * 128), dtype=F64, device=v.device)
    big[:R, :K] = v
    tiles = big.view(rb, rows, kb, 128)
    s = (tiles.abs().amax(dim=3).amax(dim=1) / 448.0).clamp(min=2.0 ** -126)
    q = _e4m3_grid(tiles / s[:, None, :, None]).view(rb * rows, kb * 128)[:R, :K]
    return q.contiguous(), s


def _exact_values(q, s, rows):
    """q * s in 64 bits."""
    r = torch.arange(q.shape[0], device=q.device) // rows
    k = torch.arange(q.shape[1], device=q.device) // 128
    return q.to(F32).to(F64) * s.to(F64)[r[:, None], k[None, :]]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h, got = st["x"].to(F64), {}
        if case["residual"]:
            got["h"] = (h + st["r"].to(F64)).to(BF16).to(F64)   # the sum is defined as its BF16 value
            h = got["h"]
        v = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["K"] + EPS) * st["weight"].to(F64)
        got["q"], got["s"] = _exact_scales(v, 1)
        if case["y"]:
            got["y"] = v
        return got
    if op == "quantize":
        v = st["x"].to(F64)
        if case["gated"]:
            v = v[:, :case["K"]] * torch.sigmoid(v[:, :case["K"]]) * v[:, case["K"]:]
        q, s = _exact_scales(v, 1)
        return {"q": q, "s": s}
    if op == "weights":
        q, s = _exact_scales(st["x"].to(F64), 128)
        return {"q": q, "s": s}
    x = _exact_values(st["x"], st["sx"], 1)
    if op == "product":
        return {"y": torch.matmul(x, _exact_values(st["w"], st["sw"], 128).T)}
    y = torch.zeros(tuple(st["out"].shape), dtype=F64, device="cuda")
    ends = st["offsets"].tolist()
    for e in range(case["E"]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            y[a:b] = torch.matmul(x[a:b], _exact_values(st["w"][e], st["sw"][e], 128).T)
    return {"y": y}
