"""Cases of the 8-bit (W8A8) operators: their inputs, their plain form in elementary torch operations, and their
definition in 64 bits.

The operators, with kQ = 127 and kMin = 2^-100:

* ``rmsnorm``: h = round(x + residual) to x's type (the residual stream that goes on), n = h / sqrt(mean(h^2) + eps)
  * gamma, then each row in 8 bits: scale = max(max|n|, kMin) / kQ, code = rint(n / scale) within +-kQ;
* ``quantize``: each row of x in 8 bits the same way; with K > 0 stages the row first goes through K stages of
  disjoint-pair Givens rotations and a division by the channel scales;
* ``pack``: weight rows in 8 bits, in 64-bit arithmetic; with K > 0 stages folded: rotated the same way and
  multiplied by the channel scales;
* ``linear``: y[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k], codes and scales as above;
* ``gated``: y = silu(g) u with g and u two such products (gate rows, then up rows).

What is held in 8 bits is returned as the values it stands for, in the type of the row it came from.
"""
import math

import numpy as np
import torch

own = False

KQ = 127.0
KMIN = 2.0 ** -100
EPS = 1e-6
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step between two layers of an 8B-class model
        {"name": "rmsnorm 1x4096 f16", "op": "rmsnorm", "M": 1, "D": 4096, "type": "f16"},
        # a prefill of 4096 tokens of the same model
        {"name": "rmsnorm 4096x4096 bf16", "op": "rmsnorm", "M": 4096, "D": 4096, "type": "bf16"},
        # the down projection's input in a decode batch of 64
        {"name": "quantize 64x14336 f16", "op": "quantize", "M": 64, "D": 14336, "K": 0, "type": "f16"},
        # the attention projections' input of a 1.5B-class model in a decode batch, with its transform
        {"name": "quantize 16x1536 K8 f16", "op": "quantize", "M": 16, "D": 1536, "K": 8, "type": "f16"},
        # a projection's input in an 8B-class prefill, with its transform
        {"name": "quantize 4096x4096 K8 f16", "op": "quantize", "M": 4096, "D": 4096, "K": 8, "type": "f16"},
        # build time: the k projection of a 1.5B-class model, and a square projection of an 8B-class one
        {"name": "pack 256x1536 K8", "op": "pack", "N": 256, "D": 1536, "K": 8, "type": "f16"},
        {"name": "pack 4096x4096 K8", "op": "pack", "N": 4096, "D": 4096, "K": 8, "type": "f16"},
        # a single token through a square projection: latency, the weights read once
        {"name": "linear 1x4096->4096 f16", "op": "linear", "M": 1, "D": 4096, "N": 4096, "type": "f16"},
        # a decode batch through the down projection
        {"name": "linear 64x14336->4096 f16", "op": "linear", "M": 64, "D": 14336, "N": 4096, "type": "f16"},
        # a ragged prompt through a down projection with one column more than its tiles hold
        {"name": "linear 1021x8960->1537 f32", "op": "linear", "M": 1021, "D": 8960, "N": 1537, "type": "f32"},
        # a small decode batch through gate and up of a 1.5B-class model
        {"name": "gated 5x1536->8960 f16", "op": "gated", "M": 5, "D": 1536, "N": 8960, "type": "f16"},
        # an 8B-class prefill of 4096 tokens through gate and up: the largest product
        {"name": "gated 4096x4096->14336 bf16", "op": "gated", "M": 4096, "D": 4096, "N": 14336, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rmsnorm", "quantize", "quantize", "pack", "linear", "linear", "linear", "gated", "gated"])
    # channels: every multiple of 128 that the library takes
    D = 128 * _log(rng, 1, 128)
    case = {"op": op, "D": D, "type": rng.choice(["f16", "bf16"])}
    if op == "rmsnorm":
        case["M"] = _log(rng, 1, min(8192, (1 << 24) // D))
    elif op == "quantize":
        case["K"] = rng.choice([0, 2, 8, 8])
        case["M"] = _log(rng, 1, min(8192, (1 << 24) // D))
    elif op == "pack":
        case["K"] = rng.choice([0, 2, 8, 8])
        case["N"] = _log(rng, 1, min(16384, (1 << 24) // D))
    elif op == "linear":
        case["M"] = _log(rng, 1, 4096)
        case["N"] = _log(rng, 16, 32768)
        case["type"] = rng.choice(["f16", "bf16", "f32"])
        while case["M"] * case["N"] * D > 4096 * 4096 * 14336 or case["N"] * D > 1 << 28:
            case["N"] = max(1, case["N"] // 2)
    else:
        case["M"] = _log(rng, 1, 4096)
        case["N"] = _log(rng, 16, 16384)
        while case["M"] * case["N"] * D > 4096 * 4096 * 14336 or case["N"] * D > 1 << 27:
            case["N"] = max(1, case["N"] // 2)
    return case


def _rows(g, M, D, spread, dtype):
    """Activations: normal, with 1 channel in 200 ten times as large in every row."""
    x = torch.randn(M, D, generator=g, device="cuda")
    out = torch.rand(D, generator=g, device="cuda") < 0.005
    return (x * torch.where(out, 10.0 * spread, spread)).to(dtype)


def _transform(seed, D, K):
    """A learned transform's host arrays: stages of channel pairs, their angles, and the channel scales."""
    r = np.random.default_rng([seed, D, K])
    pairs = np.stack([r.permutation(D).reshape(D // 2, 2) for _ in range(K)]).astype(np.int32)
    theta = r.uniform(-math.pi, math.pi, (K, D // 2)).astype(np.float32)
    scale = np.exp(r.normal(0.0, 0.3, D)).astype(np.float32)
    return pairs, theta, scale


def _inputs(case, seed):
    """The tensors both sides start from, by the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, D, dtype = case["op"], case["D"], TYPES[case["type"]]
    if op == "rmsnorm":
        gamma = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype)
        return {"x": _rows(g, case["M"], D, 0.5, dtype), "residual": _rows(g, case["M"], D, 1.0, dtype), "gamma": gamma}
    if op in ("quantize", "pack"):
        t = _transform(seed, D, case["K"]) if case["K"] else None
        if op == "quantize":
            return {"x": _rows(g, case["M"], D, 1.0, dtype), "transform": t}
        return {"x": _rows(g, case["N"], D, 0.02, dtype), "transform": t}
    M, N = case["M"], case["N"] * (2 if op == "gated" else 1)

    def codes(rows):
        return (torch.randn(rows, D, generator=g, device="cuda") * 32.0).round_().clamp_(-KQ, KQ).to(torch.int8)

    xq, wq = codes(M), codes(N)
    xs = 0.02 + 0.04 * torch.rand(M, generator=g, device="cuda")
    ws = (0.5 + torch.rand(N, generator=g, device="cuda")) / (32.0 * math.sqrt(D))
    return {"xq": xq, "xs": xs, "wq": wq, "ws": ws}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    t = s.pop("transform", None)
    s["rot"] = None
    if t is not None:
        pairs, theta, scale = t
        if own:
            import rotated_linear_amd as rl

            s["rot"] = rl.paro_rotation_prepare(pairs, theta, scale)
        else:
            # the angles' cosines and sines in 64 bits, rounded once; 1 / scale rounded once
            at = torch.from_numpy(pairs.astype(np.int64)).cuda()
            cs = np.stack([np.cos(theta.astype(np.float64)), np.sin(theta.astype(np.float64))]).astype(np.float32)
            inv = (1.0 / scale.astype(np.float64)).astype(np.float32)
            s["rot"] = (at, torch.from_numpy(cs).cuda(), torch.from_numpy(inv).cuda(), torch.from_numpy(scale).cuda())
    return s


def _stages(v, rot):
    """The K rotation stages on rows v, in v's type: each pair (i, j) becomes (c i + s j, c j - s i)."""
    at, cs = rot[0], rot[1].to(v.dtype)
    for k in range(at.shape[0]):  # each stage needs the last one's result
        i, j = at[k, :, 0], at[k, :, 1]
        a, b = v[:, i], v[:, j]
        c, s = cs[0, k], cs[1, k]
        v = torch.empty_like(v)
        v[:, i] = c * a + s * b
        v[:, j] = c * b - s * a
    return v


def _eight(n, dtype):
    """Rows n in 8 bits: the values that the codes stand for, in `dtype`, and the scales."""
    top = n.abs().amax(1, keepdim=True).clamp(min=KMIN)
    scale = top / KQ
    code = torch.round(n * (KQ / top)).clamp(-KQ, KQ)
    return (code * scale).to(dtype), scale[:, 0]


def run(s):
    case = s["case"]
    op, dtype = case["op"], TYPES[case["type"]]
    if own:
        import rotated_linear_amd as rl

        if op == "rmsnorm":
            q, sc, h = rl.paro_rmsnorm_q8(s["x"], s["gamma"], EPS, residual=s["residual"])
            return rl.paro_dequantize_q8(q, sc, dtype), sc, h
        if op == "quantize":
            q, sc = rl.paro_quantize_q8(s["x"], s["rot"])
            return rl.paro_dequantize_q8(q, sc, dtype), sc
        if op == "pack":
            q, sc = rl.paro_pack_weights_q8(s["x"], s["rot"])
            return rl.paro_dequantize_q8(q, sc, dtype), sc
        if op == "linear":
            return rl.paro_w8a8_linear(s["xq"], s["xs"], s["wq"], s["ws"], dtype)
        return rl.paro_w8a8_gated_linear(s["xq"], s["xs"], s["wq"], s["ws"], dtype)
    if op == "rmsnorm":
        h = (s["x"].float() + s["residual"].float()).to(dtype)
        v = h.float()
        n = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["gamma"].float()
        return (*_eight(n, dtype), h)
    if op == "quantize":
        v = s["x"].float()
        if s["rot"] is not None:
            v = _stages(v, s["rot"]) * s["rot"][2]
        return _eight(v, dtype)
    if op == "pack":  # in 64 bits: a weight next to a rounding border decides a code that is kept
        v = s["x"].double()
        if s["rot"] is not None:
            v = _stages(v, s["rot"]) * s["rot"][3].double()
        values, scale = _eight(v, dtype)
        return values, scale.float()
    y = (s["xq"].float() @ s["wq"].float().T) * s["xs"][:, None] * s["ws"]
    if op == "gated":
        gate, up = y[:, : case["N"]], y[:, case["N"] :]
        y = gate * torch.sigmoid(gate) * up
    return y.to(dtype)


def work(case):
    op, D, e = case["op"], case["D"], TYPES[case["type"]].itemsize
    if op == "rmsnorm":  # x and residual in, the stream and the 8-bit values (as values) out
        M = case["M"]
        return {"bytes": 4 * e * M * D + e * D + 4 * M, "flops": 8 * M * D}
    if op in ("quantize", "pack"):  # rows in, values out, the transform's pairs, angles and scales
        M, K = case["M" if op == "quantize" else "N"], case["K"]
        return {"bytes": 2 * e * M * D + 4 * M + 4 * K * D + (4 * D if K else 0), "flops": (3 * K + 4) * M * D}
    M, N = case["M"], case["N"]
    rows = 2 * N if op == "gated" else N
    return {"bytes": M * D + rows * D + 4 * (M + rows) + e * M * N, "flops": 2 * M * rows * D}


def exact(case, seed):
    s = _inputs(case, seed)
    op, dtype = case["op"], TYPES[case["type"]]

    def whole(n):  # every row over its own step: the nearest whole number of steps
        step = n.abs().max(dim=1).values.clamp_min(KMIN) / KQ
        return torch.round(n / step[:, None]) * step[:, None], step

    if op == "rmsnorm":
        h = (s["x"].double() + s["residual"].double()).to(dtype)  # the stream's own type is part of the definition
        d = h.double()
        n = d / torch.sqrt(d.square().sum(1, keepdim=True) / case["D"] + EPS) * s["gamma"].double()
        return (*whole(n), d)
    if op in ("quantize", "pack"):
        v = s["x"].double()
        if s["transform"] is not None:
            pairs, theta, scale = s["transform"]
            # each angle's cosine and sine and 1 / scale are parameters in 32 bits
            for pair, t in zip(pairs, theta):
                p = torch.from_numpy(pair.astype(np.int64)).cuda()
                c = torch.from_numpy(np.cos(t.astype(np.float64)).astype(np.float32)).cuda().double()
                r = torch.from_numpy(np.sin(t.astype(np.float64)).astype(np.float32)).cuda().double()
                old = v[:, p.reshape(-1)].reshape(v.shape[0], -1, 2)
                new = torch.stack([c * old[..., 0] + r * old[..., 1], c * old[..., 1] - r * old[..., 0]], -1)
                v = torch.empty_like(v).index_copy_(1, p.reshape(-1), new.reshape(v.shape[0], -1))
            by = scale.astype(np.float64) if op == "pack" else (1.0 / scale.astype(np.float64)).astype(np.float32).astype(np.float64)
            v = v * torch.from_numpy(by).cuda()
        return whole(v)
    acc = torch.matmul(s["xq"].double(), s["wq"].double().t())
    y = acc * torch.outer(s["xs"].double(), s["ws"].double())
    if op == "gated":
        gate, up = y.split(case["N"], dim=1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y
