"""Plain statements of the block-scaled FP8 layer, of routing and of the experts' MLPs for the tests: torch on
the inputs' device, sums in 64 bits, nothing of the library."""
from __future__ import annotations

import torch

B = 128


def up(v: int, m: int) -> int:
    return -(-v // m) * m


def encode(q: torch.Tensor) -> torch.Tensor:
    """E4M3 bytes nearest to the fp32 values q (|q| <= 448 (1 + 2^-23)), ties to even."""
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def decode(codes: torch.Tensor) -> torch.Tensor:
    return codes.view(torch.float8_e4m3fn).double()


def scale_of(amax: torch.Tensor) -> torch.Tensor:
    """fl(a / 448): through 64 bits, whose quotient of two fp32 values rounds to fp32 as the exact one does
    (torch multiplies by a reciprocal where the divisor is a Python number)."""
    return (amax.double() / 448.0).float()


def quant_rows(x: torch.Tensor):
    """(codes u8 [M, k_pad], scales f32 [M, s_ld]) of x [M, K] (any float type; decisions in fp32)."""
    M, K = x.shape
    kp, ld = up(K, B), up(K, 4 * B) // B
    f = torch.zeros(M, kp, dtype=torch.float32, device=x.device)
    f[:, :K] = x.float()
    b = f.view(M, kp // B, B)
    s = scale_of(b.abs().amax(2))
    q = b / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(2)
    scales = torch.zeros(M, ld, dtype=torch.float32, device=x.device)
    scales[:, :kp // B] = s
    codes = encode(q).view(M, kp)
    codes = torch.where((s > 0).repeat_interleave(B, 1), codes, torch.zeros_like(codes))
    return codes, scales


def quant_weights(w: torch.Tensor):
    """(codes u8 [N, k_pad], scales f32 [ceil(N / 128), s_ld]) of w [N, K]."""
    N, K = w.shape
    kp, np_, ld = up(K, B), up(N, B), up(K, 4 * B) // B
    f = torch.zeros(np_, kp, dtype=torch.float32, device=w.device)
    f[:N, :K] = w.float()
    b = f.view(np_ // B, B, kp // B, B)
    s = scale_of(b.abs().amax((1, 3)))
    q = b / torch.where(s > 0, s, torch.ones_like(s))[:, None, :, None]
    codes = encode(q)
    codes = torch.where((s > 0)[:, None, :, None], codes, torch.zeros_like(codes)).view(np_, kp)[:N].contiguous()
    scales = torch.zeros(np_ // B, ld, dtype=torch.float32, device=w.device)
    scales[:, :kp // B] = s
    return codes, scales


def rows64(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    kp = codes.shape[1]
    return decode(codes) * scales[:, :kp // B].double().repeat_interleave(B, 1)


def weights64(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    N, kp = codes.shape
    s = scales[:, :kp // B].double().repeat_interleave(B, 1).repeat_interleave(B, 0)[:N]
    return decode(codes) * s


def product(xc, xs, wc, ws):
    """(sum, sum of magnitudes) in 64 bits of the coded operands' products, [M, N] each."""
    x, w = rows64(xc, xs), weights64(wc, ws)
    return x @ w.T, x.abs() @ w.abs().T


def route(logits, k, bias=None, scoring="softmax", groups=1, keep_groups=1, group_top=1, renormalize=True, scale=1.0):
    """(ids, weights64) by loops over one token's experts, in 64 bits."""
    T, E = logits.shape
    l = logits.double().cpu()
    l = torch.where(torch.isnan(l), torch.full_like(l, -float("inf")), l).clamp(max=3.4028234663852886e38)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    weights = torch.zeros(T, k, dtype=torch.float64)
    b = None if bias is None else bias.double().cpu()
    per = E // groups
    by_logit = bias is None and (groups == 1 or group_top == 1)
    for t in range(T):
        alive = [e for e in range(E) if l[t, e] != -float("inf")]
        if not alive:
            continue
        p = torch.zeros(E, dtype=torch.float64)
        if scoring == "softmax":
            ex = torch.exp(l[t] - l[t].max())
            p = ex / ex.sum()
        else:
            p = 1 / (1 + torch.exp(-l[t]))
        score = l[t] if by_logit else p if b is None else p + b
        score = score.tolist()
        if groups > 1:
            worth = []
            for g in range(groups):
                best = sorted((score[e] for e in alive if e // per == g), reverse=True)[:group_top]
                if best:
                    worth.append((-sum(best), g))
            open_ = {g for _, g in sorted(worth)[:keep_groups]}
            alive = [e for e in alive if e // per in open_]
        chosen = sorted(alive, key=lambda e: (-score[e], e))[:k]
        w = p[chosen]
        if renormalize:
            w = w / (w.sum() + 1e-20)
        ids[t, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        weights[t, :len(chosen)] = w * scale
    return ids, weights


def dispatch(ids, E):
    """(offsets, pos) by a loop over the pairs."""
    flat = ids.cpu().flatten().tolist()
    count = [0] * E
    for e in flat:
        if 0 <= e < E:
            count[e] += 1
    offsets = [0]
    for c in count:
        offsets.append(offsets[-1] + c)
    nxt, pos = offsets[:-1].copy(), []
    for e in flat:
        if 0 <= e < E:
            pos.append(nxt[e])
            nxt[e] += 1
        else:
            pos.append(-1)
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(pos, dtype=torch.int32).view(ids.shape)
