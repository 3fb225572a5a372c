"""Measured cases of the FP8 block-scaled operators and of routing to experts.

Three operators of a served language model:

``linear``   y = x W^T with W held as E4M3 codes and one fp32 scale for each block of 128 x 128, and x
             (bf16) quantised on the way in to E4M3 codes with one fp32 scale for each 128 channels of a
             token.  Scale s = a / 448 (fp32 division, a = the block's largest magnitude; a = 0 gives s = 0
             and zero codes), code = the E4M3 value nearest to the fp32 quotient x / s.
``route``    the experts of each token from its router logits: p = softmax or sigmoid of the logits, chosen
             by p + bias (by the logit itself where there is no bias and no sum over a group), within the
             best groups where the experts are grouped (a group counts the sum of its `group_top` best
             scores), ties to the lower index, in 64 bits; the weights are p at the chosen experts, divided
             by their sum + 1e-20 where `renorm`, times `scale`.  An expert whose logit is -inf is never
             chosen: where none is left the index is -1 and the weight 0.
``experts``  the chosen experts' products: h = silu(x G_e^T) * (x U_e^T), y = sum over the token's experts of
             weight * (h D_e^T), every product as in ``linear`` (h quantised like x, straight from fp32).
             Index -1 adds nothing.
"""
import math

import torch

own = False

B = 128


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through a square projection: pure latency and weight streaming
        {"name": "linear_token", "op": "linear", "M": 1, "K": 8192, "N": 8192},
        # a handful of decoded sequences, nothing a multiple of the block
        {"name": "linear_ragged", "op": "linear", "M": 77, "K": 1000, "N": 1048},
        # Llama-3-8B fused QKV, a prompt of 2048 tokens
        {"name": "linear_qkv", "op": "linear", "M": 2048, "K": 4096, "N": 6144},
        # Llama-3-70B fused gate+up, 8192 tokens
        {"name": "linear_gateup", "op": "linear", "M": 8192, "K": 8192, "N": 57344},
        # one decoded token, softmax over 64 experts
        {"name": "route_token", "op": "route", "T": 1, "E": 64, "k": 8, "scoring": "softmax", "bias": False,
         "groups": 1, "keep": 1, "group_top": 1, "renorm": True, "scale": 1.0, "bf16": False},
        # a prompt, bf16 logits, softmax shares kept as they are
        {"name": "route_softmax", "op": "route", "T": 8192, "E": 128, "k": 8, "scoring": "softmax", "bias": False,
         "groups": 1, "keep": 1, "group_top": 1, "renorm": False, "scale": 1.0, "bf16": True},
        # a prompt, sigmoid scores, a balancing bias, 4 of 8 groups
        {"name": "route_groups", "op": "route", "T": 4093, "E": 256, "k": 8, "scoring": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "group_top": 2, "renorm": True, "scale": 2.5, "bf16": False},
        # one decoded token through 8 of 64 experts
        {"name": "experts_token", "op": "experts", "T": 1, "pad": 0, "E": 64, "k": 8, "H": 4096, "I": 1024},
        # a decode batch whose last 7 rows are padding
        {"name": "experts_batch", "op": "experts", "T": 96, "pad": 7, "E": 64, "k": 8, "H": 4096, "I": 1024},
        # few rows, sizes that are not multiples of the block
        {"name": "experts_ragged", "op": "experts", "T": 333, "pad": 0, "E": 12, "k": 3, "H": 1032, "I": 360},
        # a prompt over many small experts
        {"name": "experts_prompt", "op": "experts", "T": 4096, "pad": 0, "E": 64, "k": 8, "H": 4096, "I": 1024},
        # a prompt over a few experts of Llama-3-8B's MLP sizes
        {"name": "experts_large", "op": "experts", "T": 4096, "pad": 0, "E": 8, "k": 2, "H": 4096, "I": 14336},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["linear", "route", "experts"])
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 256, 8192, 8), "N": _log(rng, 256, 57344, 8)}
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log(rng, 2, 512 // groups)
        keep = rng.randint(1, groups)
        return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(8, E // groups * keep)),
                "scoring": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "keep": keep, "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "bf16": rng.random() < 0.3}
    E = _log(rng, 4, 96)
    T = _log(rng, 1, 4096)
    return {"op": op, "T": T, "pad": rng.choice([0, T // 5]), "E": E, "k": rng.randint(1, min(8, E)),
            "H": _log(rng, 256, 4096, 8), "I": _log(rng, 128, 2048, 8)}


# ------------------------------------------------------------------ inputs
def _up(v, m):
    return (v + m - 1) // m * m


def _block_weights(G, N, K, gen):
    """G weight matrices N x K ~ N(0, 1/K) as a checkpoint holds them: codes [G, N, K up to a multiple of 128], zero
    behind K, and scales [G, N/128, K up to a multiple of 512 / 128], zero behind the last block."""
    Kp, Np, ls = _up(K, B), _up(N, B), _up(K, 4 * B) // B
    codes = torch.zeros(G, N, Kp, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.zeros(G, Np // B, ls, dtype=torch.float32, device="cuda")
    for g in range(G):
        w = torch.zeros(Np, Kp, device="cuda")
        w[:N, :K] = torch.randn(N, K, device="cuda", generator=gen).mul_(K ** -0.5).bfloat16().float()
        w = w.view(Np // B, B, Kp // B, B)
        s = w.abs().amax((1, 3)) / 448.0
        q = w.div_(torch.where(s > 0, s, 1.0)[:, None, :, None])
        codes[g] = q.view(Np, Kp)[:N].to(torch.float8_e4m3fn)
        scales[g, :, :Kp // B] = s
    return codes, scales


def _activations(T, K, gen):
    """Normalised activations with a few channels that are large for every token."""
    x = torch.randn(T, K, device="cuda", generator=gen)
    loud = torch.randperm(K, device="cuda", generator=gen)[:max(1, K // 64)]
    x[:, loud] *= 30.0
    return x.bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    st = {"case": case}
    if case["op"] == "linear":
        st["w"], st["s"] = (t[0] for t in _block_weights(1, case["N"], case["K"], gen))
        st["x"] = _activations(case["M"], case["K"], gen)
    elif case["op"] == "route":
        T, E = case["T"], case["E"]
        logits = 1.5 * torch.randn(T, E, device="cuda", generator=gen) + torch.randn(E, device="cuda", generator=gen)
        st["logits"] = logits.bfloat16() if case["bf16"] else logits
        st["bias"] = 0.1 * torch.randn(E, device="cuda", generator=gen) if case["bias"] else None
    else:
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        w, s = _block_weights(2 * E, I, H, gen)
        st["w13"], st["s13"] = w.view(E, 2, I, -1), s.view(E, 2, *s.shape[1:])
        st["w2"], st["s2"] = _block_weights(E, H, I, gen)
        st["x"] = _activations(T, H, gen)
        # some experts are asked for more often than others
        logits = torch.randn(T, E, device="cuda", generator=gen) + 0.5 * torch.randn(E, device="cuda", generator=gen)
        top = logits.topk(k, dim=1)
        st["ids"], st["weights"] = top.indices.int(), torch.softmax(top.values, 1)
        st["ids"][T - case["pad"]:] = -1
    return st


# ------------------------------------------------------------------ plain form
def _rounded(x):
    """x (fp32) as its block codes stand for it: E4M3 values times their block's scale."""
    K = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -K % B)).unflatten(-1, (-1, B))
    a = b.abs().amax(-1, keepdim=True)
    s = a / torch.full_like(a, 448.0)  # (a Python number as divisor would be a product with its reciprocal)
    q = (b / torch.where(s > 0, s, 1.0)).to(torch.float8_e4m3fn).float()
    return (q * s).flatten(-2)[..., :K]


def _dense(codes, scales, K):
    """The weights (..., N, K) that codes and scales stand for, in fp32."""
    N, kb = codes.shape[-2], codes.shape[-1] // B
    w = codes.float().unflatten(-1, (kb, B))
    w *= scales[..., :kb].repeat_interleave(B, -2)[..., :N, :].unsqueeze(-1)
    return w.flatten(-2)[..., :K]


def _plain_linear(x, w, s):
    return (_rounded(x.float()) @ _dense(w, s, x.shape[1]).T).bfloat16()


def _plain_route(c, logits, bias):
    E, k = c["E"], c["k"]
    l = logits.double()
    p = torch.softmax(l, 1) if c["scoring"] == "softmax" else torch.sigmoid(l)
    score = p + bias.double() if bias is not None else p if c["groups"] > 1 and c["group_top"] > 1 else l
    if c["groups"] > 1:
        g = score.view(-1, c["groups"], E // c["groups"])
        best = g.sort(dim=-1, descending=True).values[..., :c["group_top"]].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        open_ = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        score = g.masked_fill(~open_.unsqueeze(-1), -math.inf).flatten(1)
    ids = score.sort(dim=1, descending=True, stable=True).indices[:, :k]
    weights = p.gather(1, ids)
    if c["renorm"]:
        weights = weights / (weights.sum(1, keepdim=True) + 1e-20)
    return {"ids": ids.int(), "weights": (weights * c["scale"]).float()}


def _plain_mlp(x, w13, s13, w2, s2):
    """Rows x (G, R, H) through G experts' weights."""
    x = _rounded(x)
    g = x @ _dense(w13[:, 0], s13[:, 0], x.shape[-1]).mT
    u = x @ _dense(w13[:, 1], s13[:, 1], x.shape[-1]).mT
    h = _rounded(g * torch.sigmoid(g) * u)
    return h @ _dense(w2, s2, h.shape[-1]).mT


def _plain_experts(x, ids, weights, w13, s13, w2, s2):
    (T, k), E = ids.shape, w2.shape[0]
    slot = ids.flatten().long()
    share = torch.where(slot >= 0, weights.flatten(), 0.0)
    rows = x.float().repeat_interleave(k, 0)
    if T * k <= E:  # fewer rows than experts: each row with its own copy of its expert's weights
        e = slot.clamp_min(0)
        z = _plain_mlp(rows[:, None], w13[e], s13[e], w2[e], s2[e])[:, 0]
    else:           # the experts' rows side by side, each expert with room for the fullest one's
        e, order = torch.where(slot >= 0, slot, E).sort(stable=True)
        count = torch.bincount(e, minlength=E + 1)
        room = max(1, int(count[:E].max()))
        at = e * room + torch.arange(T * k, device=e.device) - (count.cumsum(0) - count)[e]
        order, at = order[e < E], at[e < E]
        full = x.new_zeros(E * room, x.shape[1], dtype=torch.float32)
        full[at] = rows[order]
        out = _plain_mlp(full.view(E, room, -1), w13, s13, w2, s2).flatten(0, 1)
        z = torch.zeros_like(rows)
        z[order] = out[at]
    return (z * share[:, None]).view(T, k, -1).sum(1).bfloat16()


def run(state):
    c = state["case"]
    if own:
        import mixed_precision_gemm_b200 as sq
        if c["op"] == "linear":
            return sq.linear_fp8b(state["x"], sq.PreparedFP8B(c["N"], c["K"], state["w"].view(torch.uint8), state["s"]))
        if c["op"] == "route":
            ids, weights = sq.route(state["logits"], c["k"], bias=state["bias"], scoring=c["scoring"],
                                    groups=c["groups"], keep_groups=c["keep"], group_top=c["group_top"],
                                    renormalize=c["renorm"], scale=c["scale"])
            return {"ids": ids, "weights": weights}
        gate_up = sq.PreparedFP8B(c["I"], c["H"], state["w13"].view(torch.uint8), state["s13"])
        down = sq.PreparedFP8B(c["H"], c["I"], state["w2"].view(torch.uint8), state["s2"])
        return sq.experts_fp8b(state["x"], state["ids"], state["weights"], gate_up, down)
    if c["op"] == "linear":
        return _plain_linear(state["x"], state["w"], state["s"])
    if c["op"] == "route":
        return _plain_route(c, state["logits"], state["bias"])
    return _plain_experts(state["x"], state["ids"], state["weights"], state["w13"], state["s13"], state["w2"], state["s2"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    def weights(n, k):
        return n * k + 4 * math.ceil(n / B) * math.ceil(k / B)
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + weights(N, K) + 2 * M * N, "flops": 2 * M * N * K}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (2 if case["bf16"] else 4) + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    rows = (T - case["pad"]) * k
    used = E * (1 - (1 - 1 / E) ** rows)  # experts that even shares would reach
    return {"bytes": int(used * (2 * weights(I, H) + weights(H, I))) + 4 * T * H + 8 * T * k, "flops": 6 * rows * H * I}


# ------------------------------------------------------------------ the definition in 64 bits
def _codes64(x):
    """Values that the block codes of x (float64 [R, K]) stand for; scale and quotient are rounded to fp32 as defined."""
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], B):
        part = x[:, lo:lo + B]
        s = (part.abs().max(1, keepdim=True).values / 448).float().double()
        q = (part / s.masked_fill(s == 0, 1)).float()
        # nearest E4M3 value: steps of 2^(e-3), no finer than 2^-9
        step = torch.ldexp(torch.ones_like(q), torch.frexp(q).exponent.clamp_min(-5) - 4)
        out[:, lo:lo + B] = ((q / step).round() * step).clamp(-448, 448).double() * s
    return out


def _weight64(codes, scales, K):
    w = codes[:, :K].double()
    for i in range(scales.shape[0]):
        w[i * B:(i + 1) * B] *= scales[i].double().repeat_interleave(B)[:K]
    return w


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        return _codes64(st["x"].double()) @ _weight64(st["w"], st["s"], case["K"]).T
    if case["op"] == "route":
        l = st["logits"].double()
        if case["scoring"] == "sigmoid":
            p = 1 / (1 + torch.exp(-l))
        else:
            p = torch.exp(l - l.max(1, keepdim=True).values)
            p = p / p.sum(1, keepdim=True)
        rank = p if st["bias"] is None else p + st["bias"].double()
        G, per = case["groups"], case["E"] // case["groups"]
        worth = torch.stack([rank[:, g * per:(g + 1) * per].topk(min(case["group_top"], per), 1).values.sum(1) for g in range(G)], 1)
        if G > 1:  # (no bias and one best score a group: p rises with the logit, and equal logits tie alike)
            left_out = torch.argsort(-worth, dim=1, stable=True)[:, case["keep"]:]
            gone = torch.zeros_like(worth).scatter_(1, left_out, 1.0) > 0
            rank = rank.masked_fill(gone.repeat_interleave(per, 1), -math.inf)
        w = p.gather(1, torch.argsort(-rank, dim=1, stable=True)[:, :case["k"]])
        return {"ids": None, "weights": w * case["scale"] / (w.sum(1, keepdim=True) + 1e-20 if case["renorm"] else 1)}
    T, E, H = case["T"], case["E"], case["H"]
    x, y = _codes64(st["x"].double()), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (st["ids"] == e).nonzero(as_tuple=True)
        if len(t):
            a = x[t] @ _weight64(st["w13"][e, 0], st["s13"][e, 0], H).T
            b = x[t] @ _weight64(st["w13"][e, 1], st["s13"][e, 1], H).T
            h = _codes64(a / (1 + torch.exp(-a)) * b)
            y.index_add_(0, t, (h @ _weight64(st["w2"][e], st["s2"][e], case["I"]).T) * st["weights"][t, j].double()[:, None])
    return y
