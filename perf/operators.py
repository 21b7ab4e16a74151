"""Measured cases of two operators that stand around the attention of a layer.

linear   The projection product in 8-bit floating point.  The weight is held as
         E4M3 codes with one power-of-two scale for each 128 x 128 block, each
         token's row is quantised in the call to E4M3 with one power-of-two
         scale for each 128 of its values, and the sums are held in fp32:
             y[t][o] = sum_b 2^(ex[t][b] + ew[o/128][b]) sum_(c in b) X[t][c] W[o][c]
         A weight with groups is block diagonal: the rows of a group read its
         own k / groups columns.  The outputs are an fp32 part (what the
         compressor and the index read) and a BF16 part (queries, latents).
norm     The RMS norm of every query head and key head, and the rotation of its
         last `rope` dims at the token's position, in one pass:
             y = x / sqrt(mean(x^2) + eps) * weight, pairs (2i, 2i+1) rotated by
             position * base^(-2i / rope)

Sizes are those of this repository's workloads (hidden 256 with 8 heads x 64;
hidden 4096 with 64 heads x 512; hidden 7168 with 128 heads x 512, query latent
1024, 16 output groups of 1024), and what lies between them.
"""
import math

import torch

own = False

EPS, BASE = 1e-6, 10000.0
MOST_PRODUCTS = 2048 * 73728 * 1024       # multiply-adds of the largest listed product
MOST_VALUES = 4096 * 128 * 512            # values of the largest listed norm
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    def linear(name, tokens, n_f32, n_bf16, k, groups=1):
        return {"name": name, "op": "linear", "tokens": tokens, "n_f32": n_f32, "n_bf16": n_bf16, "k": k, "groups": groups}

    def norm(name, tokens, heads, kv_heads, dim, rope, q_type, k_type, rotate_k, fused, far):
        return {"name": name, "op": "norm", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rope": rope,
                "q_type": q_type, "k_type": k_type, "rotate_k": rotate_k, "fused": fused, "far": far}

    return [
        # one token of the tiny layer: c, z, c_I, z_I and w, then the latent; latency is all there is
        linear("linear tiny 1 token", 1, 196, 64, 256),
        # a decode step of 4 requests: hidden state to c, z, c_I, z_I, w (fp32) and the query latent (BF16)
        linear("linear input 4 tokens", 4, 1344, 1024, 7168),
        # the same step: query latent to 128 heads x 512 and the index heads 64 x 128, a stream of the weight
        linear("linear queries 4 tokens", 4, 8192, 65536, 1024),
        # the same step: the attention's output, 16 groups of 8 heads, to 1024 per group
        linear("linear grouped 4 tokens", 4, 0, 16384, 65536, 16),
        # a ragged batch of 37 requests: grouped output to the model's width
        linear("linear output 37 tokens", 37, 7168, 0, 16384),
        # a prefill chunk, 128 tokens of each of 4 requests, hidden 4096 to the compressor's inputs and the latent
        linear("linear input 512 tokens", 512, 1344, 1024, 4096),
        # a long prefill: 2048 tokens from the latent to every query head, where the tensor cores bound it
        linear("linear queries 2048 tokens", 2048, 8192, 65536, 1024),
        # one token of the tiny fp32 layer: its query heads and its KV candidate (the append rotates that later)
        norm("norm tiny 1 token", 1, 8, 1, 64, 16, "fp32", "fp32", False, False, 1024),
        # a decode step of 4 requests near 1M tokens: query heads in BF16, the KV candidate in fp32
        norm("norm decode 4 tokens", 4, 128, 1, 512, 64, "bf16", "fp32", False, False, 1 << 20),
        # 130 tokens whose queries and keys come from one fused product and are both rotated; heads of 96
        norm("norm fused 130 tokens", 130, 24, 3, 96, 32, "bf16", "bf16", True, True, 131072),
        # a long prefill's queries and KV candidates: one read and one write of half a gigabyte
        norm("norm prefill 4096 tokens", 4096, 128, 1, 512, 64, "bf16", "fp32", False, False, 1 << 20),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    if rng.random() < 0.6:
        tokens, k = spread(1, 4096), 8 * spread(8, 2048)
        groups = rng.choice((1, 1, 1, 2, 4, 16))
        if groups > 1:
            kg, rows = 8 * spread(4, 512), 128 * spread(1, 8)
            k, n = kg * groups, rows * groups
        else:
            kg, n = k, spread(33, 73728)
        n = max(groups * 128 if groups > 1 else 33, min(n, MOST_PRODUCTS // kg))
        tokens = max(1, min(tokens, MOST_PRODUCTS // (n * kg)))
        part = rng.choice((0, n, n // 2, n // 3))
        return {"op": "linear", "tokens": tokens, "n_f32": part, "n_bf16": n - part, "k": k, "groups": groups}
    dim = 8 * rng.randint(4, 64)
    rope = 2 * rng.randint(0, min(dim, 128) // 2)
    heads, kv_heads = spread(1, 128), rng.randint(0, 8)
    tokens = max(1, min(spread(1, 8192), MOST_VALUES // ((heads + kv_heads) * dim)))
    q_type = rng.choice(("bf16", "bf16", "fp32"))
    fused = kv_heads > 0 and rng.random() < 0.4
    if q_type == "fp32":
        tokens = max(1, tokens // 2)
    return {"op": "norm", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rope": rope, "q_type": q_type,
            "k_type": q_type if fused else rng.choice(("bf16", "fp32")), "rotate_k": rng.random() < 0.5, "fused": fused,
            "far": spread(128, 1 << 20)}


def _blocks(v, groups):
    """[rows, groups * kg] -> [rows, groups, blocks of a group, 128], the last block of a group filled up with zeros."""
    v = v.reshape(v.shape[0], groups, -1)
    v = torch.nn.functional.pad(v, (0, -v.shape[2] % 128))
    return v.reshape(v.shape[0], groups, -1, 128)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e (0 for an empty block), within E8M0's range."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875)
    return torch.where(amax > 0, e, 0).clamp(-127, 127)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    t = case["tokens"]
    if case["op"] == "linear":
        k, groups, n = case["k"], case["groups"], case["n_f32"] + case["n_bf16"]
        kg = k // groups
        # hidden states have a few channels far larger than the others
        loud = 1 + 20 * (torch.rand(k, generator=g, device="cuda") < 0.01)
        x = (normal(t, k) * loud).to(torch.bfloat16)
        w = normal(n, kg) / math.sqrt(kg)
        wb = torch.nn.functional.pad(_blocks(w, 1)[:, 0], (0, 0, 0, 0, 0, -n % 128))
        wb = wb.reshape(-1, 128, wb.shape[1], 128)
        e = _exponent(wb.abs().amax((1, 3)))                      # [row blocks, column blocks]
        codes = (wb * torch.exp2(-e.float())[:, None, :, None]).reshape(-1, wb.shape[2] * 128)[:n, :kg]
        state = {"case": case, "x": x, "codes": codes.to(torch.float8_e4m3fn).contiguous(), "scales": (e + 127).to(torch.uint8).contiguous(),
                 "outs": [torch.empty((t, r), dtype=d, device="cuda") for r, d in ((case["n_f32"], torch.float32), (case["n_bf16"], torch.bfloat16)) if r]}
        if own:
            from compressed_sparse_long_hca_b200.api import LinearFP8
            state["linear"] = LinearFP8(state["codes"], state["scales"], groups=groups)
        return state
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    qt, kt = TYPES[case["q_type"]], TYPES[case["k_type"]]
    if case["fused"]:
        both = (normal(t, h + hk, d) * 2).to(qt)
        q, key = both[:, :h], both[:, h:]
    else:
        q, key = (normal(t, h, d) * 2).to(qt), (normal(t, hk, d) * 2).to(kt) if hk else None
    state = {"case": case, "q": q, "k": key,
             "q_weight": 1 + 0.1 * normal(d), "k_weight": 1 + 0.1 * normal(d),
             "positions": torch.randint(0, case["far"], (t,), generator=g, device="cuda"),
             "q_out": torch.empty((t, h, d), dtype=qt, device="cuda"), "k_out": torch.empty((t, hk, d), dtype=kt, device="cuda") if hk else None}
    if own:
        from compressed_sparse_long_hca_b200.api import HeadNorm
        state["norm"] = HeadNorm(d, case["rope"], q_weight=state["q_weight"], k_weight=state["k_weight"], eps=EPS, rope_base=BASE,
                                 rotate_k=case["rotate_k"])
    return state


def _linear(s):
    case, x = s["case"], s["x"]
    groups, t, kg = case["groups"], case["tokens"], case["k"] // case["groups"]
    xb = _blocks(x.float(), groups)
    e = _exponent(xb.abs().amax(-1))[..., None]
    xq = torch.ldexp(torch.ldexp(xb, -e).to(torch.float8_e4m3fn).float(), e)
    xq = xq.reshape(t, groups, -1)[:, :, :kg]
    n = s["codes"].shape[0]
    scale = torch.exp2(s["scales"].float() - 127).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :kg]
    w = (s["codes"].float() * scale).reshape(groups, n // groups, kg)
    y = torch.bmm(xq.transpose(0, 1), w.transpose(1, 2)).transpose(0, 1).reshape(t, n)
    parts = y.split([case["n_f32"], case["n_bf16"]], dim=1)
    return [p.contiguous() if d else p.to(torch.bfloat16) for p, d in zip(parts, (True, False)) if p.shape[1]]


def _norm(x, weight, turn):
    v = x.float()
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * weight
    if turn is not None:
        c, s = turn
        r = 2 * c.shape[-1]
        a, b = v[..., -r::2], v[..., v.shape[-1] - r + 1::2]
        v = torch.cat([v[..., :-r], torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)], -1)
    return v.to(x.dtype)


def run(state):
    case = state["case"]
    if case["op"] == "linear":
        if own:
            return state["linear"](state["x"], state["outs"])
        return _linear(state)
    if own:
        state["norm"](state["positions"], state["q"], state["q_out"], state["k"], state["k_out"])
        return [state["q_out"], state["k_out"]] if case["kv_heads"] else [state["q_out"]]
    turn = None
    if case["rope"]:
        theta = BASE ** (-2.0 * torch.arange(case["rope"] // 2, device="cuda", dtype=torch.float64) / case["rope"])
        angle = state["positions"].double()[:, None, None] * theta
        turn = torch.cos(angle).float(), torch.sin(angle).float()
    outs = [_norm(state["q"], state["q_weight"], turn)]
    if case["kv_heads"]:
        outs.append(_norm(state["k"], state["k_weight"], turn if case["rotate_k"] else None))
    return outs


def work(case):
    t = case["tokens"]
    if case["op"] == "linear":
        n, kg = case["n_f32"] + case["n_bf16"], case["k"] // case["groups"]
        scales = -(-n // 128) * -(-kg // 128)
        return {"bytes": n * kg + scales + 2 * t * case["k"] + t * (4 * case["n_f32"] + 2 * case["n_bf16"]), "flops": 2 * t * n * kg}
    size = {"bf16": 2, "fp32": 4}
    q, k = t * case["heads"] * case["dim"], t * case["kv_heads"] * case["dim"]
    return {"bytes": 2 * (q * size[case["q_type"]] + k * size[case["k_type"]]) + 8 * t + 8 * case["dim"], "flops": 4 * (q + k)}


def exact(case, seed):
    s = prepare(case, seed)
    t = case["tokens"]
    if case["op"] == "linear":
        groups, kg = case["groups"], case["k"] // case["groups"]
        # the value of every E4M3 code, from its bits: sign, 4 exponent bits (bias 7), 3 mantissa bits
        bits = torch.arange(256, device="cuda")
        ex, man = (bits >> 3) & 15, (bits & 7).double()
        value = torch.where(ex > 0, (8 + man) * torch.exp2((ex - 10).double()), man * 2.0 ** -9)
        value = torch.where(bits >= 128, -value, value)
        xs = s["x"].double().split(kg, dim=1)
        ws = s["codes"].view(torch.uint8).split(s["codes"].shape[0] // groups)
        y, row = [], 0
        for xg, wg in zip(xs, ws):
            total = torch.zeros((t, wg.shape[0]), dtype=torch.float64, device="cuda")
            which = torch.arange(row, row + wg.shape[0], device="cuda") // 128
            for b, c0 in enumerate(range(0, kg, 128)):
                xb = xg[:, c0: c0 + 128]
                top = xb.abs().amax(1, keepdim=True)
                e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp_min(1e-300) / 448) - 1e-9), torch.zeros_like(top)).clamp(-127, 127)
                v = xb / torch.exp2(e)
                step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)) + 1e-12) - 3)
                v = torch.round(v / step) * step * torch.exp2(e)
                total.addmm_(v, (value[wg[:, c0: c0 + 128].long()] * torch.exp2(s["scales"][which, b].double() - 127)[:, None]).T)
            y.append(total)
            row += wg.shape[0]
        y = torch.cat(y, 1)
        return [p.contiguous() for p in (y[:, :case["n_f32"]], y[:, case["n_f32"]:]) if p.shape[1]]

    def one(x, weight, rotate):
        v = x.double()
        v = weight.double() * v / (v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt()
        r = case["rope"] if rotate else 0
        if r:
            i = torch.arange(0, r, 2, device="cuda", dtype=torch.float64)
            z = torch.view_as_complex(v[..., v.shape[-1] - r:].reshape(*v.shape[:-1], r // 2, 2).contiguous())
            angle = s["positions"].double()[:, None] * torch.exp(-i / r * math.log(BASE))
            z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
            v[..., v.shape[-1] - r:] = torch.view_as_real(z).flatten(-2)
        return v

    out = [one(s["q"], s["q_weight"], True)]
    return out + [one(s["k"], s["k_weight"], case["rotate_k"])] if case["kv_heads"] else out
