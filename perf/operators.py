"""The FP8 (e4m3) linear layer and its mixture of experts: the operators that are timed.

  quantize  activations in groups of 128 along a row, weights in blocks of 128 x 128
  gemm      Y = X W of such operands, one scale per group and block
  route     scores, top-k experts and their weights; the slots sorted by expert
  experts   each expert's product over its slots, the rows gathered from the tokens
  combine   the weighted sum of each token's slots

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, or
64 next to a border), or through the library when ``own`` is true.  A case is a dict of plain
values; ``listed`` gives the fixed ones and ``draw`` one more of the same ranges.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token's activations before a layer: latency alone
        {"name": "quantize token", "op": "quantize", "what": "act", "M": 1, "K": 4096, "dtype": "bf16"},
        # a prefill batch in front of the widest down projection
        {"name": "quantize prefill", "op": "quantize", "what": "act", "M": 8192, "K": 28672, "dtype": "bf16"},
        # a layer's weight, offline (and again after each update of a served model)
        {"name": "quantize weight", "op": "quantize", "what": "weight", "E": 1, "K": 4096, "N": 12288, "dtype": "f32"},
        # one token through a layer: the weight is read once
        {"name": "gemm token", "op": "gemm", "M": 1, "K": 4096, "N": 12288, "dtype": "bf16"},
        # a short ragged batch, sizes that no tile divides, fp16 out
        {"name": "gemm ragged", "op": "gemm", "M": 333, "K": 11008, "N": 4144, "dtype": "f16"},
        # prefill of a wide layer: the tensor cores' bound
        {"name": "gemm prefill", "op": "gemm", "M": 8192, "K": 8192, "N": 28672, "dtype": "bf16"},
        # a decode batch over a few experts, softmax scores
        {"name": "route decode", "op": "route", "M": 16, "E": 64, "topk": 8, "score": "softmax", "bias": False,
         "n_group": 1, "topk_group": 1, "group_top": 1, "renorm": True, "padded": 0, "dtype": "f32"},
        # a padded prefill batch, sigmoid scores with a balance bias and limited groups
        {"name": "route prefill", "op": "route", "M": 16384, "E": 256, "topk": 8, "score": "sigmoid", "bias": True,
         "n_group": 8, "topk_group": 4, "group_top": 2, "renorm": True, "padded": 100, "dtype": "bf16"},
        # a decode batch: few rows per expert, the weights of the chosen experts are read once
        {"name": "experts decode", "op": "experts", "M": 8, "E": 32, "topk": 4, "K": 4096, "N": 4096, "dtype": "bf16"},
        # prefill: hundreds of rows per expert, unevenly spread
        {"name": "experts prefill", "op": "experts", "M": 4096, "E": 32, "topk": 4, "K": 4096, "N": 4096,
         "dtype": "bf16"},
        # a decode batch's outputs
        {"name": "combine decode", "op": "combine", "M": 16, "topk": 8, "N": 4096, "padded": 0, "dtype": "bf16"},
        # a padded prefill batch's outputs
        {"name": "combine prefill", "op": "combine", "M": 16384, "topk": 8, "N": 4096, "padded": 100,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "route", "experts", "experts", "combine"])
    if op == "quantize" and rng.random() < 0.6:
        return {"op": op, "what": "act", "M": _log(rng, 1, 8192), "K": _log(rng, 256, 28672, 16),
                "dtype": rng.choice(["bf16", "f16"])}
    if op == "quantize":
        return {"op": op, "what": "weight", "E": _log(rng, 1, 4), "K": _log(rng, 256, 8192, 16),
                "N": _log(rng, 256, 12288, 16), "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "gemm":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 256, 8192, 16), "N": _log(rng, 256, 28672, 16),
                "dtype": rng.choice(["bf16", "f16"])}
    if op == "route":
        n_group = rng.choice([1, 1, 4, 8])
        E = n_group * _log(rng, 4, 256 // n_group)
        kept = rng.randint(max(1, n_group // 2), n_group)
        M = _log(rng, 1, 16384)
        return {"op": op, "M": M, "E": E, "topk": rng.randint(1, min(8, E // n_group * kept)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "n_group": n_group,
                "topk_group": kept, "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.7,
                "padded": rng.randint(0, M // 8), "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "experts":
        E = _log(rng, 2, 64)
        return {"op": op, "M": _log(rng, 1, 4096), "E": E, "topk": rng.randint(1, min(4, E)),
                "K": _log(rng, 256, 4096, 16), "N": _log(rng, 256, 4096, 16), "dtype": rng.choice(["bf16", "f16"])}
    M = _log(rng, 1, 16384)
    return {"op": op, "M": M, "topk": rng.randint(1, 8), "N": _log(rng, 256, 8192, 8),
            "padded": rng.randint(0, M // 8), "dtype": rng.choice(["bf16", "f16"])}


# --------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _activations(M, K, g):
    """Unit normal with eight channels fifty times as large, as activations have them."""
    x = torch.randn(M, K, generator=g, device=DEV)
    x[:, torch.randint(0, K, (8,), generator=g, device=DEV)] *= 50.0
    return x


def _routing(M, E, k, g):
    """k distinct experts for each token, some of them liked more than others."""
    like = torch.randn(E, generator=g, device=DEV) * 0.5
    return (torch.randn(M, E, generator=g, device=DEV) + like).topk(k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "quantize" and case["what"] == "act":
        s["X"] = _activations(case["M"], case["K"], g).to(TYPES[case["dtype"]])
    elif op == "quantize":
        s["W"] = (torch.randn(case["E"], case["K"], case["N"], generator=g, device=DEV) * 0.02).to(
            TYPES[case["dtype"]])
    elif op == "gemm":
        s["Xq"], s["xs"] = _quantize_act(_activations(case["M"], case["K"], g))
        w = torch.randn(1, case["K"], case["N"], generator=g, device=DEV) * 0.02
        s["Wq"], s["ws"] = (t[0] for t in _quantize_weight(w))
    elif op == "route":
        x = torch.randn(case["M"], case["E"], generator=g, device=DEV) * 2.0
        if case["padded"]:
            x[case["M"] - case["padded"]:] = -math.inf   # padding goes to no expert
        s["logits"] = x.to(TYPES[case["dtype"]])
        s["bias"] = torch.randn(case["E"], generator=g, device=DEV) * 0.1 if case["bias"] else None
    elif op == "experts":
        M, E, k = case["M"], case["E"], case["topk"]
        s["Xq"], s["xs"] = _quantize_act(_activations(M, case["K"], g))
        w = [_quantize_weight(torch.randn(1, case["K"], case["N"], generator=g, device=DEV) * 0.02) for _ in range(E)]
        s["Wq"], s["ws"] = (torch.cat(t) for t in zip(*w))
        s["offsets"], s["slot_token"], _ = _slots(_routing(M, E, k, g), E)
        s["rows"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())   # the fullest expert's, for the plain form
    else:
        M, k = case["M"], case["topk"]
        idx = _routing(M, 64, k, g)
        idx[M - case["padded"]:] = -1
        _, _, s["token_slot"] = _slots(idx, 64)
        s["D"] = torch.randn(M * k, case["N"], generator=g, device=DEV).to(TYPES[case["dtype"]])
        w = torch.rand(M, k, generator=g, device=DEV) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
    return s


# ---------------------------------------------------------------------------- plain forms
def _scale(a):
    return a / torch.full_like(a, F8_MAX)   # by a tensor: by a number, torch multiplies with its rounded reciprocal


def _quantize_act(x):
    """Per row and group of 128: scale = max|x| / 448, codes = e4m3(x / scale)."""
    x = x.float()
    M, K = x.shape
    G = -(-K // 128)
    p = torch.nn.functional.pad(x, (0, G * 128 - K)).view(M, G, 128)
    s = _scale(p.abs().amax(2))
    c = torch.where(s[..., None] > 0, p / s[..., None], 0.0)
    return c.view(M, G * 128)[:, :K].contiguous().to(F8), s


def _quantize_weight(w):
    """Per expert and block of 128 x 128: scale = max|w| / 448, codes = e4m3(w / scale)."""
    w = w.float()
    E, K, N = w.shape
    a, b = -(-K // 128), -(-N // 128)
    p = torch.nn.functional.pad(w, (0, b * 128 - N, 0, a * 128 - K)).view(E, a, 128, b, 128)
    s = _scale(p.abs().amax((2, 4)))
    t = s[:, :, None, :, None]
    c = torch.where(t > 0, p / t, 0.0)
    return c.reshape(E, a * 128, b * 128)[:, :K, :N].contiguous().to(F8), s


def _weight_values(Wq, ws):
    K, N = Wq.shape[-2:]
    return Wq.float() * ws.repeat_interleave(128, -2)[..., :K, :].repeat_interleave(128, -1)[..., :N]


def _act_values(Xq, xs):
    return Xq.float() * xs.repeat_interleave(128, 1)[:, :Xq.shape[1]]


def _route(c, logits, bias):
    """In 64 bits: which of two nearly equal experts comes first is a matter of the last bits."""
    x = logits.double()
    there = x > -math.inf
    score = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.where(there, torch.softmax(x, 1), 0.0)
    key = score if bias is None else score + bias.double()
    key = torch.where(there, key, -math.inf)
    M, E = key.shape
    if c["n_group"] > 1:
        size = E // c["n_group"]
        top = key.view(M, c["n_group"], size).sort(2, descending=True).values[..., :min(c["group_top"], size)].sum(2)
        best = top.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        kept = torch.zeros(M, c["n_group"], dtype=torch.bool, device=key.device).scatter(1, best, True)
        key = torch.where(kept.repeat_interleave(size, 1), key, -math.inf)
    order = key.sort(dim=1, descending=True, stable=True)
    idx, key = order.indices[:, :c["topk"]], order.values[:, :c["topk"]]
    chosen = key > -math.inf
    w = torch.where(chosen, score.gather(1, idx), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(chosen, idx, -1).to(torch.int32), w.float()


def _slots(idx, E):
    """The choices sorted by expert, then by token: where each expert's begin, each slot's token, each choice's slot."""
    M, k = idx.shape
    flat = idx.reshape(-1).long()
    flat = torch.where(flat < 0, E, flat)
    order = flat.sort(dim=0, stable=True)
    offsets = torch.searchsorted(order.values, torch.arange(E + 1, device=idx.device)).to(torch.int32)
    slot_token = torch.where(order.values < E, order.indices // k, -1).to(torch.int32)
    slot = torch.empty_like(flat).scatter_(0, order.indices, torch.arange(M * k, device=idx.device))
    token_slot = torch.where(flat < E, slot, -1).to(torch.int32).view(M, k)
    return offsets, slot_token, token_slot


def _experts(s):
    E, K, N = s["Wq"].shape
    offsets, token = s["offsets"].long(), s["slot_token"].long()
    slot = torch.arange(token.numel(), device=token.device)
    e = torch.searchsorted(offsets[1:], slot, right=True)
    row = slot - offsets[e]
    x = _act_values(s["Xq"], s["xs"])
    padded = torch.zeros(E, s["rows"], K, device=x.device).index_put_((e, row), x[token])
    return torch.bmm(padded, _weight_values(s["Wq"], s["ws"]))[e, row]


def _combine(s):
    slot = s["token_slot"].long()
    d = s["D"].float()[slot.clamp(min=0)]
    return (d * torch.where(slot >= 0, s["weights"], 0.0)[..., None]).sum(1)


def run(s):
    c = s["case"]
    op, t = c["op"], TYPES[c["dtype"]]
    if own:
        import bit_quantized_gemm_group_b200 as q
        if op == "quantize" and c["what"] == "act":
            X = s["X"]
            Xq = torch.empty(X.shape, dtype=F8, device=X.device)
            xs = torch.empty(X.shape[0], -(-X.shape[1] // 128), dtype=torch.float32, device=X.device)
            q.qg_quantize_act_fp8(X, Xq, xs)
            return Xq, xs
        if op == "quantize":
            W = s["W"]
            E, K, N = W.shape
            Wq = torch.empty(W.shape, dtype=F8, device=W.device)
            ws = torch.empty(E, -(-K // 128), -(-N // 128), dtype=torch.float32, device=W.device)
            q.qg_quantize_weight_fp8(W, Wq, ws)
            return Wq, ws
        if op == "gemm":
            Y = torch.empty(s["Xq"].shape[0], s["Wq"].shape[1], dtype=t, device=s["Xq"].device)
            q.qg_gemm_fp8(s["Xq"], s["xs"], s["Wq"], s["ws"], Y)
            return Y
        if op == "route":
            M, E = s["logits"].shape
            idx = torch.empty(M, c["topk"], dtype=torch.int32, device=s["logits"].device)
            weights = torch.empty(M, c["topk"], dtype=torch.float32, device=idx.device)
            q.qg_route_topk(s["logits"], s["bias"], idx, weights, score=c["score"], n_group=c["n_group"],
                            topk_group=c["topk_group"], group_top=c["group_top"], renorm=c["renorm"])
            offsets = torch.empty(E + 1, dtype=torch.int32, device=idx.device)
            slot_token = torch.empty(M * c["topk"], dtype=torch.int32, device=idx.device)
            token_slot = torch.empty_like(idx)
            q.qg_expert_slots(idx, offsets, slot_token, token_slot)
            return idx, weights, offsets, slot_token, token_slot
        if op == "experts":
            Y = torch.empty(s["slot_token"].shape[0], s["Wq"].shape[2], dtype=t, device=s["Xq"].device)
            q.qg_gemm_fp8_experts(s["Xq"], s["xs"], s["slot_token"], s["offsets"], s["Wq"], s["ws"], Y)
            return Y
        Y = torch.empty(s["token_slot"].shape[0], s["D"].shape[1], dtype=t, device=s["D"].device)
        q.qg_combine_experts(s["D"], s["token_slot"], s["weights"], Y)
        return Y
    if op == "quantize":
        return _quantize_act(s["X"]) if c["what"] == "act" else _quantize_weight(s["W"])
    if op == "gemm":
        return (_act_values(s["Xq"], s["xs"]) @ _weight_values(s["Wq"], s["ws"])).to(t)
    if op == "route":
        idx, weights = _route(c, s["logits"], s["bias"])
        return (idx, weights, *_slots(idx, c["E"]))
    return (_experts(s) if op == "experts" else _combine(s)).to(t)


# ------------------------------------------------------------------------- work and exact
def _size(c):
    return torch.empty(0, dtype=TYPES[c["dtype"]]).element_size()


def work(c):
    op = c["op"]
    if op == "quantize" and c["what"] == "act":
        n, s = c["M"] * c["K"], c["M"] * -(-c["K"] // 128)
        return {"bytes": n * (_size(c) + 1) + 4 * s, "flops": 2 * n}
    if op == "quantize":
        n, s = c["E"] * c["K"] * c["N"], c["E"] * -(-c["K"] // 128) * -(-c["N"] // 128)
        return {"bytes": n * (_size(c) + 1) + 4 * s, "flops": 2 * n}
    if op == "gemm":
        M, K, N = c["M"], c["K"], c["N"]
        G = -(-K // 128)
        return {"bytes": M * K + 4 * M * G + K * N + 4 * G * -(-N // 128) + 2 * M * N, "flops": 2 * M * K * N}
    if op == "route":
        n = c["M"] * c["topk"]
        return {"bytes": c["M"] * c["E"] * _size(c) + 4 * c["E"] * c["bias"] + 16 * n + 4 * c["E"] + 4,
                "flops": 4 * c["M"] * c["E"]}
    if op == "experts":
        M, E, K, N, S = c["M"], c["E"], c["K"], c["N"], c["M"] * c["topk"]
        G = -(-K // 128)
        hit = E * (1 - (1 - c["topk"] / E) ** M)   # experts that some token chose, were the choices even
        return {"bytes": M * K + 4 * M * G + hit * (K * N + 4 * G * -(-N // 128)) + 4 * (S + E + 1) + 2 * S * N,
                "flops": 2 * S * K * N}
    M, k, N = c["M"], c["topk"], c["N"]
    return {"bytes": ((M - c["padded"]) * k + M) * N * _size(c) + 8 * M * k, "flops": 2 * M * k * N}


def _e4m3(v):
    """v to four significant bits (three below 2^-6), ties to even, as a 64-bit number."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.clamp(torch.round(v / step) * step, -F8_MAX, F8_MAX)


def _spread(v, dim, n):
    at = torch.div(torch.arange(n, device=v.device), 128, rounding_mode="floor")
    return v.double().index_select(dim, at)


def _exact_quantize(v, cut):
    """Group by group (activations: v is [M, K]) or block row by block row ([E, K, N]).  By definition the scale and
    the quotient are what 32 bits hold of them."""
    codes, scales = torch.empty_like(v, dtype=F8), []
    for k in range(0, v.shape[1], 128):
        part = v[:, k:k + 128].double()
        if cut:
            a = torch.stack([part[..., n:n + 128].abs().amax((1, 2)) for n in range(0, v.shape[2], 128)], 1)
            s = (a / F8_MAX).float()
            wide = _spread(s, 1, v.shape[2])[:, None, :]
        else:
            s = (part.abs().amax(1) / F8_MAX).float()
            wide = s.double()[:, None]
        codes[:, k:k + 128] = _e4m3(torch.where(wide > 0, part / wide, 0.0).float().double()).to(F8)
        scales.append(s)
    return codes, torch.stack(scales, 1)


def _exact_product(Xq, xs, Wq, ws):
    K, N = Wq.shape
    w = Wq.double() * _spread(_spread(ws, 0, K), 1, N)
    return torch.cat([(Xq[m:m + 4096].double() * _spread(xs[m:m + 4096], 1, K)) @ w
                      for m in range(0, max(1, Xq.shape[0]), 4096)])


def _first_largest(v, among=None):
    """The index of the last dimension's largest value, the lowest one if several (of those in `among`)."""
    top = v == v.amax(-1, keepdim=True)
    top = top if among is None else top & among
    n = v.shape[-1]
    return torch.where(top, torch.arange(n, device=v.device), n).amin(-1, keepdim=True)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        act = case["what"] == "act"
        return _exact_quantize(s["X"] if act else s["W"], not act)
    if op == "gemm":
        return _exact_product(s["Xq"], s["xs"], s["Wq"], s["ws"])
    if op == "route":
        x = s["logits"].double()
        if case["score"] == "sigmoid":
            p = 1.0 / (1.0 + torch.exp(-x))
        else:
            p = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        key = (p if s["bias"] is None else p + s["bias"].double()).masked_fill(x == -math.inf, -math.inf)
        if case["n_group"] > 1:
            size = case["E"] // case["n_group"]
            high, rest = 0.0, key.unflatten(1, (case["n_group"], size))
            for _ in range(min(case["group_top"], size)):
                at = _first_largest(rest)
                high = high + rest.gather(2, at)[..., 0]
                rest = rest.scatter(2, at, -math.inf)
            out = torch.ones_like(high, dtype=torch.bool)
            for _ in range(case["topk_group"]):
                out.scatter_(1, _first_largest(high.masked_fill(~out, -math.inf), out), False)
            key = key.masked_fill(out.repeat_interleave(size, 1), -math.inf)
        w = []
        for _ in range(case["topk"]):
            at = _first_largest(key)
            w.append(torch.where(key.gather(1, at) > -math.inf, p.gather(1, at), 0.0))
            key = key.scatter(1, at, -math.inf)
        w = torch.cat(w, 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        return None, w, None, None, None
    if op == "experts":
        at = s["offsets"].tolist()
        return torch.cat([_exact_product(s["Xq"][t], s["xs"][t], s["Wq"][e], s["ws"][e]) for e in range(case["E"])
                          if (t := s["slot_token"][at[e]:at[e + 1]].long()).numel()])
    out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEV)
    for j in range(case["topk"]):
        slot = s["token_slot"][:, j].long()
        have = slot >= 0
        out[have] += s["weights"][have, j].double()[:, None] * s["D"][slot[have]].double()
    return out
