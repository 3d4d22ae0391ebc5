"""Cases of the operators around the products of a served decoder block: their inputs, their plain form in elementary
torch operations, and their definition in 64 bits.

* ``linear``: the 8-bit (W8A8) product with its epilogue,
  y[m][n] = act(xs[m] ws[n] sum_k xq[m][k] wq[n][k] + bias[n]) + residual[m][n];
  act is one of none, relu, relu2 (the square of relu), silu, gelu (with erf) and gelu_tanh.
* ``norm``: the norms after one block and before the next, with the gate and the residual scale between them,
  p = x / sqrt(mean(x^2) + eps) * post_gamma   (p = x without a norm after the block),
  h = round(residual_scale residual + gate p) to x's type, the residual stream that goes on,
  n = h / sqrt(mean(h^2) + eps) * gamma, in x's type or each row in 8 bits
  (scale = max(max|n|, 2^-100) / 127, code = rint(n / scale)).
* ``moe``: a mixture-of-experts layer on INT4 weights (groups of 128 channels, float16 scale and zero) for a few tokens:
  the top_k experts of each token by its router logits (ties to the lower index), weights the softmax or the sigmoid
  of the logits, made to sum to 1 or as they are, and
  y[m] = sum_e weight[m][e] down_e(silu(gate_e x[m]) * up_e x[m]),
  where the rows of x, and those between the two products, go through K stages of channel-pair rotations and a
  division by channel scales first, if the weights were packed for that. Or the experts alone, with ids and weights
  given; an id of -1 takes no expert.

What is held in 8 bits is returned as the values it stands for, in the type of the row it came from.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
GROUP = 128
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"]


def _lin(M, D, N, act, bias, residual, type):
    name = f"linear {M}x{D}->{N} {act}{' bias' if bias else ''}{' residual' if residual else ''} {type}"
    return {"name": name, "op": "linear", "M": M, "D": D, "N": N, "act": act, "bias": bias, "residual": residual, "type": type}


def _norm(M, D, post, gates, alpha, q8, type):
    name = f"norm {M}x{D}{' post' if post else ''} gates{gates}{' q8' if q8 else ''} {type}"
    return {"name": name, "op": "norm", "M": M, "D": D, "post": post, "gates": gates, "alpha": alpha, "q8": q8, "type": type}


def _moe(M, D, F, E, top_k, K, routed=True, scoring="softmax", renormalize=True):
    name = f"moe {M}x{D} {top_k} of {E} F{F} K{K}{'' if routed else ' ids given'}"
    return {"name": name, "op": "moe", "M": M, "D": D, "F": F, "E": E, "top_k": top_k, "K": K, "routed": routed,
            "scoring": scoring, "renormalize": renormalize, "type": "f16"}


def listed():
    return [
        # one token through the k projection of a 1.5B-class model, which has a bias: latency
        _lin(1, 1536, 256, "none", True, False, "f16"),
        # a decode batch through the first product of an ungated feed-forward block
        _lin(64, 4096, 14336, "gelu", True, False, "bf16"),
        # a ragged prompt through a layer with one column more than its tiles hold, everything in the epilogue
        _lin(1021, 1536, 1537, "relu2", True, True, "f32"),
        # an 8B-class prefill of 4096 tokens through the down projection, added to the stream: the largest
        _lin(4096, 14336, 4096, "none", False, True, "bf16"),
        # one token between two blocks with norms on both sides
        _norm(1, 4096, True, 0, 1.0, True, "f16"),
        # a ragged prompt between two blocks without a norm after them, one gate for all rows and a scaled stream
        _norm(1021, 8960, False, 1, 0.7, False, "f16"),
        # a prefill of 8 sequences of 512 tokens, a gate for each sequence
        _norm(4096, 4096, True, 8, 1.0, True, "bf16"),
        # one token through many small experts: latency, the experts that it takes are read once
        _moe(1, 2048, 1024, 64, 8, 0),
        # a few tokens through few experts of 8B-class width
        _moe(4, 4096, 14336, 8, 2, 0),
        # a small batch, an odd number of experts, weights packed for rotated rows
        _moe(13, 1536, 1408, 60, 4, 8, scoring="sigmoid"),
        # a decode batch that reaches nearly every expert
        _moe(64, 4096, 1408, 64, 8, 0),
        # the share of one GPU of a larger layer: the ids come from elsewhere, most tokens miss some of the experts
        _moe(32, 4096, 2048, 16, 4, 0, routed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "norm", "moe"])
    if op == "linear":
        # channels: every multiple of 128 that the library takes
        D = 128 * _log(rng, 1, 128)
        M, N = _log(rng, 1, 4096), _log(rng, 16, 32768)
        while M * N * D > 4096 * 4096 * 14336 or N * D > 1 << 27:
            N = max(1, N // 2)
        bias, residual = rng.choice([(True, False), (False, True), (True, True)])
        c = _lin(M, D, N, rng.choice(ACTS), bias, residual, rng.choice(["f16", "bf16", "f32"]))
    elif op == "norm":
        D = 128 * _log(rng, 1, 128)
        M = _log(rng, 1, min(8192, (1 << 24) // D))
        gates = rng.choice([0, 1, M, rng.choice([g for g in range(1, M + 1) if M % g == 0])])
        c = _norm(M, D, rng.random() < 0.7, gates, rng.choice([1.0, 0.25, 0.7]), rng.random() < 0.5, rng.choice(["f16", "bf16"]))
    else:
        D, F = 128 * _log(rng, 2, 64), 128 * _log(rng, 1, 112)
        E = _log(rng, 2, 128)
        while E > 2 and E * F * D > 64 * 1408 * 4096:
            E = max(2, E // 2)
        top_k = rng.randint(1, min(8, E))
        c = _moe(_log(rng, 1, 64), D, F, E, top_k, rng.choice([0, 0, 2, 8]), rng.random() < 0.7,
                 rng.choice(["softmax", "sigmoid"]), rng.random() < 0.7)
    del c["name"]
    return c


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


def _experts(g, E, N, D):
    """Packed INT4 weights of E experts, rows normal with a spread of 1 / sqrt(D): the bytes (blocks of 16 rows, each
    block group by group, the lower channel of a pair in the lower 4 bits), scales and zeros."""
    qw = torch.empty(E, N // 16, D // GROUP, 16, 64, dtype=torch.uint8, device="cuda")
    for e in range(E):
        code = (torch.randn(N // 16, D // GROUP, 16, 64, 2, generator=g, device="cuda") * 2.6 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
        qw[e] = code[..., 0] | (code[..., 1] << 4)
    sc = ((0.7 + 0.6 * torch.rand(E, N, D // GROUP, generator=g, device="cuda")) / (2.6 * math.sqrt(D))).half()
    z = torch.randint(6, 10, (E, N, D // GROUP), generator=g, device="cuda").half()
    return qw.view(E, N, D // 2), sc, z


def _inputs(case, seed):
    """The tensors both sides start from, by the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, M, D, dtype = case["op"], case["M"], case["D"], TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "norm":
        s = {"x": _rows(g, M, D, 0.5, dtype), "residual": _rows(g, M, D, 1.0, dtype), "gamma": (1.0 + 0.2 * normal(D)).to(dtype)}
        s["post_gamma"] = (0.5 + 0.1 * normal(D)).to(dtype) if case["post"] else None
        s["gate"] = (0.5 * normal(case["gates"], D)).to(dtype) if case["gates"] else None
        return s
    if op == "linear":
        N = case["N"]

        def codes(rows):
            return (normal(rows, D) * 32.0).round_().clamp_(-127, 127).to(torch.int8)

        s = {"xq": codes(M), "wq": codes(N), "xs": 0.02 + 0.04 * torch.rand(M, generator=g, device="cuda")}
        s["ws"] = (0.5 + torch.rand(N, generator=g, device="cuda")) / (32.0 * math.sqrt(D))
        s["bias"] = (0.5 * normal(N)).to(dtype) if case["bias"] else None
        s["residual"] = _rows(g, M, N, 1.0, dtype) if case["residual"] else None
        return s
    E, F, k = case["E"], case["F"], case["top_k"]
    s = {"x": (normal(M, D)).to(dtype), "gate_up": _experts(g, E, 2 * F, D), "down": _experts(g, E, D, F)}
    if case["routed"]:
        s["router"] = (normal(E, D) * (1.5 / math.sqrt(D))).to(dtype)
    else:
        s["ids"] = torch.rand(M, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
        s["ids"][torch.rand(M, k, generator=g, device="cuda") < 0.4] = -1
        s["weights"] = torch.rand(M, k, generator=g, device="cuda")
    s["transforms"] = (_transform(seed, D, case["K"]), _transform(seed + 1, F, case["K"])) if case["K"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    t = s.pop("transforms", None)
    s["rot_x"] = s["rot_a"] = None
    if t is not None:
        made = []
        for pairs, theta, scale in t:
            if own:
                import rotated_linear_amd as rl

                made.append(rl.paro_rotation_prepare(pairs, theta, scale))
            else:
                # the angles' cosines and sines in 64 bits, rounded once; 1 / scale rounded once
                cs = np.stack([np.cos(theta.astype(np.float64)), np.sin(theta.astype(np.float64))]).astype(np.float32)
                inv = (1.0 / scale.astype(np.float64)).astype(np.float32)
                made.append((torch.from_numpy(pairs.astype(np.int64)).cuda(), torch.from_numpy(cs).cuda(), torch.from_numpy(inv).cuda()))
        s["rot_x"], s["rot_a"] = made
    return s


def _rotate(v, rot):
    """The K rotation stages on float32 rows v, each pair (i, j) to (c i + s j, c j - s i), then 1 / scale."""
    if rot is None:
        return v
    at, cs, inv = rot
    for k in range(at.shape[0]):  # each stage needs the last one's result
        i, j = at[k, :, 0], at[k, :, 1]
        a, b = v[:, i], v[:, j]
        c, s = cs[0, k], cs[1, k]
        v = torch.empty_like(v)
        v[:, i] = c * a + s * b
        v[:, j] = c * b - s * a
    return v * inv


def _unpack(packed, e):
    """The weights of expert e (a tensor of one number) in float32, row by row."""
    qw, sc, z = (t.index_select(0, e)[0] for t in packed)
    N, half = qw.shape
    q = qw.view(N // 16, half // 64, 16, 64).transpose(1, 2).reshape(N, half)
    q = torch.stack([q & 15, q >> 4], -1).view(N, half // 64, GROUP)
    return ((q.float() - z.float()[..., None]) * sc.float()[..., None]).view(N, 2 * half)


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "relu2":
        return v.clamp(min=0) ** 2
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        # 0.5 (1 + tanh z) is sigmoid(2 z)
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def _moe_plain(s):
    case, dtype = s["case"], TYPES[s["case"]["type"]]
    M, E, F, k = case["M"], case["E"], case["F"], case["top_k"]
    if case["routed"]:
        # logits in 64 bits: two close ones decide which expert a token takes
        logits = s["x"].double() @ s["router"].double().T
        top, ids = logits.sort(dim=1, descending=True, stable=True)
        top, ids = top[:, :k], ids[:, :k]
        if case["scoring"] == "softmax":
            weights = torch.exp(top - top[:, :1]) / torch.exp(logits - top[:, :1]).sum(1, keepdim=True)
        else:
            weights = torch.sigmoid(top)
        if case["renormalize"]:
            weights = weights / weights.sum(1, keepdim=True)
        weights, ids = weights.float(), ids.to(torch.int32)
    else:
        ids, weights = s["ids"], s["weights"]
    x = _rotate(s["x"].float(), s["rot_x"])
    y = torch.zeros(M, case["D"], device="cuda")

    def block(e, rows):
        g = rows @ _unpack(s["gate_up"], e).T
        return _rotate(g[:, :F] * torch.sigmoid(g[:, :F]) * g[:, F:], s["rot_a"]) @ _unpack(s["down"], e).T

    if M * k < E:  # the experts that the tokens name, one by one; else every expert, for the tokens that name it
        for m in range(M):
            for j in range(k):
                e = ids[m, j : j + 1]
                y[m] += torch.where(e >= 0, weights[m, j] * block(e.clamp(min=0), x[m : m + 1])[0], 0.0)
    else:
        for e in torch.arange(E, dtype=torch.int32, device="cuda").split(1):
            takes = ids == e
            w = torch.where(takes, weights, 0.0).sum(1, keepdim=True)
            y += torch.where(takes.any(1, keepdim=True), w * block(e, x), 0.0)
    y = y.to(dtype)
    return (y, ids, weights) if case["routed"] else (y,)


def run(s):
    case = s["case"]
    op, dtype = case["op"], TYPES[case["type"]]
    if own:
        import rotated_linear_amd as rl

        if op == "linear":
            return rl.paro_w8a8_linear_epilogue(s["xq"], s["xs"], s["wq"], s["ws"], bias=s["bias"], activation=case["act"],
                                                residual=s["residual"], out_dtype=dtype)
        if op == "norm":
            call = rl.paro_block_norm_q8 if case["q8"] else rl.paro_block_norm
            out = call(s["x"], s["residual"], s["gamma"], EPS, post_gamma=s["post_gamma"], gate=s["gate"], residual_scale=case["alpha"])
            return (rl.paro_dequantize_q8(out[0], out[1], dtype), *out[1:]) if case["q8"] else out
        if case["routed"]:
            return rl.paro_moe_layer_w4a16(s["x"], s["router"], case["top_k"], s["gate_up"], s["down"], rot_x=s["rot_x"],
                                           rot_a=s["rot_a"], scoring=case["scoring"], renormalize=case["renormalize"])
        return (rl.paro_moe_w4a16(s["x"], s["ids"], s["weights"], s["gate_up"], s["down"], rot_x=s["rot_x"], rot_a=s["rot_a"]),)
    if op == "linear":
        v = (s["xq"].float() @ s["wq"].float().T) * s["xs"][:, None] * s["ws"]
        if s["bias"] is not None:
            v = v + s["bias"].float()
        v = _act(v, case["act"])
        if s["residual"] is not None:
            v = v + s["residual"].float()
        return v.to(dtype)
    if op == "norm":
        p = s["x"].float()
        if s["post_gamma"] is not None:
            p = p * torch.rsqrt((p * p).mean(1, keepdim=True) + EPS) * s["post_gamma"].float()
        if s["gate"] is not None:
            p = p * s["gate"].float().repeat_interleave(case["M"] // case["gates"], 0)
        h = (case["alpha"] * s["residual"].float() + p).to(dtype)
        v = h.float()
        n = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["gamma"].float()
        if not case["q8"]:
            return n.to(dtype), h
        top = n.abs().amax(1, keepdim=True).clamp(min=2.0 ** -100)
        scale = top / 127.0
        return (torch.round(n * (127.0 / top)).clamp(-127, 127) * scale).to(dtype), scale[:, 0], h
    return _moe_plain(s)


def work(case):
    op, M, D, e = case["op"], case["M"], case["D"], TYPES[case["type"]].itemsize
    if op == "linear":
        N = case["N"]
        out = M * N * e * (2 if case["residual"] else 1) + (N * e if case["bias"] else 0)
        return {"bytes": M * D + N * D + 4 * (M + N) + out, "flops": 2 * M * N * D}
    if op == "norm":  # x and residual in, the stream and the rows (as values) out, the gains and the gates
        return {"bytes": 4 * e * M * D + e * D * (2 if case["post"] else 1) + e * D * case["gates"] + (4 * M if case["q8"] else 0),
                "flops": 16 * M * D}
    # the weights of the experts that a batch reaches, on average, with their scales and zeros; rows in and out
    E, F, K = case["E"], case["F"], case["K"]
    k = case["top_k"] * (1.0 if case["routed"] else 0.6)
    reached = E * (1.0 - (1.0 - k / E) ** M)
    bytes_ = reached * 3 * F * D * (0.5 + 4 / GROUP) + 4 * M * D + 4 * K * (D + F) + (2 * E * D if case["routed"] else 0)
    return {"bytes": int(bytes_), "flops": int(2 * M * k * 3 * F * D + (2 * M * E * D if case["routed"] else 0))}


def _moe_exact(case, s):
    M, F, E, k = case["M"], case["F"], case["E"], case["top_k"]
    dev = s["x"].device

    def turned(v, t):  # the transform's parameters are those of 32 bits
        if t is None:
            return v
        for pair, angle in zip(t[0], t[1]):
            p = torch.from_numpy(pair.astype(np.int64).reshape(-1)).to(dev)
            c = torch.from_numpy(np.cos(angle.astype(np.float64)).astype(np.float32)).to(dev).double()
            r = torch.from_numpy(np.sin(angle.astype(np.float64)).astype(np.float32)).to(dev).double()
            old = v.index_select(1, p).reshape(v.shape[0], -1, 2)
            new = torch.stack([c * old[..., 0] + r * old[..., 1], c * old[..., 1] - r * old[..., 0]], -1)
            v = torch.empty_like(v).index_copy_(1, p, new.reshape(v.shape[0], -1))
        return v * torch.from_numpy((1.0 / t[2].astype(np.float64)).astype(np.float32)).to(dev).double()

    def expert(packed, e):  # byte b of a block's group g: row b // 64 of its 16, channels 128 g + 2 (b % 64) and the next
        blocks = packed[0][e].reshape(-1, packed[0].shape[2] // 64, 16, 64)
        w = torch.empty(blocks.shape[0], 16, blocks.shape[1], GROUP, dtype=torch.float64, device=dev)
        for parity in (0, 1):
            w[..., parity::2] = torch.bitwise_and(torch.bitwise_right_shift(blocks, 4 * parity), 15).permute(0, 2, 1, 3).double()
        w = w.reshape(-1, blocks.shape[1], GROUP)
        return torch.mul(w - packed[2][e].double().unsqueeze(2), packed[1][e].double().unsqueeze(2)).flatten(1)

    tx, ta = s["transforms"] if s["transforms"] is not None else (None, None)
    share = torch.zeros(M, E, dtype=torch.float64, device=dev)
    ids = weights = None
    if case["routed"]:
        logits = torch.einsum("md,ed->me", s["x"].double(), s["router"].double())
        rows = logits.cpu().numpy()
        ids = torch.from_numpy(np.argsort(-rows, axis=1, kind="stable")[:, :k].astype(np.int32)).to(dev)
        score = torch.softmax(logits, 1) if case["scoring"] == "softmax" else 1.0 / (1.0 + torch.exp(-logits))
        weights = score.gather(1, ids.long())
        if case["renormalize"]:
            weights = weights / weights.sum(dim=1).unsqueeze(1)
        share.scatter_(1, ids.long(), weights)
    else:
        for m, (row, w) in enumerate(zip(s["ids"].tolist(), s["weights"].double().tolist())):
            for i, v in zip(row, w):
                if 0 <= i < E:
                    share[m, i] += v
    x = turned(s["x"].double(), tx)
    y = torch.zeros(M, case["D"], dtype=torch.float64, device=dev)
    for e in range(E):
        at = torch.nonzero(share[:, e]).flatten()
        if at.numel():
            gate, up = torch.matmul(x[at], expert(s["gate_up"], e).t()).split(F, dim=1)
            a = turned(gate / (1.0 + torch.exp(-gate)) * up, ta)
            y[at] += share[at, e].unsqueeze(1) * torch.matmul(a, expert(s["down"], e).t())
    return (y, ids, weights) if case["routed"] else (y,)


def exact(case, seed):
    s = _inputs(case, seed)
    op, dtype = case["op"], TYPES[case["type"]]
    if op == "moe":
        return _moe_exact(case, s)
    if op == "linear":
        y = torch.matmul(s["xq"].double(), s["wq"].double().t()) * torch.outer(s["xs"].double(), s["ws"].double())
        if s["bias"] is not None:
            y += s["bias"].double()
        kind = case["act"]
        if kind in ("relu", "relu2"):
            y = torch.where(y > 0, y if kind == "relu" else y.square(), torch.zeros_like(y))
        elif kind == "silu":
            y = y / (1.0 + torch.exp(-y))
        elif kind == "gelu":
            y = y * torch.erfc(-y / math.sqrt(2.0)) / 2.0
        elif kind == "gelu_tanh":  # (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)), without its cancellation below 0
            z = math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)
            y = y / (1.0 + torch.exp(-2.0 * z))
        return y if s["residual"] is None else y + s["residual"].double()
    p = s["x"].double()
    if case["post"]:
        p = p / torch.sqrt(p.square().sum(1, keepdim=True) / case["D"] + EPS) * s["post_gamma"].double()
    if case["gates"]:
        p = (p.reshape(case["gates"], -1, case["D"]) * s["gate"].double().unsqueeze(1)).reshape(p.shape)
    h = (p + case["alpha"] * s["residual"].double()).to(dtype).double()  # the stream's own type is part of the definition
    n = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["D"] + EPS) * s["gamma"].double()
    if not case["q8"]:
        return n, h
    step = n.abs().max(dim=1).values.clamp_min(2.0 ** -100) / 127.0
    return torch.round(n / step[:, None]) * step[:, None], step, h
