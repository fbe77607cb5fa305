"""What is measured of the operators that stand around this library's products in a language model: 4-bit weights for
single tokens, the norm before a product, the router before the products by expert, and the rows' way there and back.

Each case is one pass as a serving or training step makes it.  With ``own`` false, ``run`` computes the operator in its
plain form (elementary torch operations in 32 bits, in 64 where a value lies next to a border); with ``own`` true it
makes the library's calls.

Operators (T tokens, each with k of E experts; slot (t, j) is token t's choice j; 4-bit numbers are e2m1, 8-bit e4m3):

  gemv_fp4      y[m,n]   = sum_k x[m,k] W[n,k] 2^(s[n,k/32] - 127)
  quantize_fp4  s = the least with amax <= 6 * 2^(s - 127) in each block of 32 of a row, q = e2m1(x / 2^(s - 127))
  rmsnorm       h = x + residual in 16 bits, y = h / sqrt(mean(h^2) + eps) * weight; y in 16 bits, or in e4m3 with a
                scale max(amax / 448, 2^-80) for each block of 128 of a row
  rmsnorm_grad  dx = r (w dy) - h r^3 mean(w dy h) + dh and dweight[c] = sum_t dy h r, with r = 1 / sqrt(mean(h^2) + eps)
  route         the k largest score + bias of each token (ties to the lowest index) within its best groups of experts,
                their scores made to add up to a scale; then the slots sorted by expert: where each expert's rows
                begin, and the row of each slot
  route_grad    the gradient of such weights with respect to the logits
  gather        Xs[row(t,j)] = X[t]                               (numbers of 8 bits and their scales, or of 16 bits)
  combine       Y[t] = sum_j weight(t,j) D[row(t,j)]
  combine_grad  dD[row(t,j)] = weight(t,j) dY[t], dweight(t,j) = sum_c dY[t,c] D[row(t,j),c]
"""
import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BLOCK = 128
_EPS = 1e-6
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # One token through a down projection held in 4 bits (the shape of this library's GEMV benchmark).
        {"name": "fp4 one token", "op": "gemv_fp4", "type": "bf16", "M": 1, "N": 4096, "K": 14336},
        # A decode batch of an odd size against a projection of odd sizes.
        {"name": "fp4 decode batch", "op": "gemv_fp4", "type": "f16", "M": 27, "N": 8195, "K": 4128},
        # A weight matrix of odd height, brought to 4 bits when it is loaded.
        {"name": "fp4 weights", "op": "quantize_fp4", "type": "bf16", "N": 4095, "K": 14336},
        # The norm of a single token before an 8-bit product: latency counts.
        {"name": "norm one token", "op": "rmsnorm", "type": "bf16", "T": 1, "C": 4096, "residual": True, "out": 8},
        # The same for a prompt's worth of tokens.
        {"name": "norm prompt", "op": "rmsnorm", "type": "f16", "T": 8192, "C": 4096, "residual": True, "out": 8},
        # The norm's gradients in a training step, with the gradient that comes along the residual.
        {"name": "norm gradient", "op": "rmsnorm_grad", "type": "bf16", "T": 8191, "C": 2048, "residual": True},
        # Four tokens' choice of 8 among 64 experts, before a grouped product.
        {"name": "route decode", "op": "route", "type": "f32", "T": 4, "E": 64, "k": 8, "groups": 1, "top_groups": 1,
         "score": "softmax", "norm": True, "bias": False},
        # Prompts over 256 experts in 8 groups, sigmoid scores with a bias for balance.
        {"name": "route prompt", "op": "route", "type": "bf16", "T": 16384, "E": 256, "k": 8, "groups": 8, "top_groups": 4,
         "score": "sigmoid", "norm": True, "bias": True},
        # The router's gradient in a training step; scores are not made to add up.
        {"name": "route gradient", "op": "route_grad", "type": "bf16", "T": 8200, "E": 128, "k": 6, "score": "softmax",
         "norm": False},
        # A prompt's 8-bit rows on their way to the experts, a few of whose choices go to another card.
        {"name": "gather prompt", "op": "gather", "type": "fp8", "T": 4100, "k": 8, "K": 4096, "drop": 0.05},
        # A decode batch's rows on their way back.
        {"name": "combine decode", "op": "combine", "type": "bf16", "T": 27, "k": 8, "K": 2048, "drop": 0.0},
        # The gradients of a prompt's way back.
        {"name": "combine gradient", "op": "combine_grad", "type": "bf16", "T": 4096, "k": 8, "K": 2048, "drop": 0.0},
    ]


def _log(rng, low, high, multiple=1):
    """A size of low .. high, spread over its logarithm, and a multiple of `multiple`."""
    v = int(round(low * (high / low) ** rng.random()))
    return max(multiple, v // multiple * multiple)


def draw(rng):
    op = rng.choice(("gemv_fp4", "gemv_fp4", "quantize_fp4", "rmsnorm", "rmsnorm", "rmsnorm_grad", "route", "route",
                     "route_grad", "gather", "combine", "combine_grad"))
    case = {"op": op, "type": rng.choice(("f16", "bf16"))}
    if op == "gemv_fp4":
        while True:
            M, N, K = _log(rng, 1, 64), _log(rng, 16, 32768), _log(rng, 32, 16384, 32)
            if 1 << 18 <= N * K <= 1 << 27:
                return {**case, "M": M, "N": N, "K": K}
    if op == "quantize_fp4":
        return {**case, "N": _log(rng, 1, 4000), "K": _log(rng, 32, 14336, 32)}
    if op in ("rmsnorm", "rmsnorm_grad"):
        while True:
            T, C = _log(rng, 1, 16384), _log(rng, 16, 16384, 16)
            if T * C <= 1 << 24:
                case = {**case, "T": T, "C": C, "residual": rng.random() < 0.7}
                return case if op == "rmsnorm_grad" else {**case, "out": rng.choice((8, 8, 16))}
    if op in ("route", "route_grad"):
        T, groups = _log(rng, 1, 16384), rng.choice((1, 1, 2, 4, 8, 16))
        E = groups * max(2, _log(rng, 8, 256) // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, top_groups * (E // groups)))
        case = {**case, "type": rng.choice(("f16", "bf16", "f32")), "T": T, "E": E, "k": k,
                "score": rng.choice(("softmax", "sigmoid")), "norm": rng.random() < 0.7}
        if op == "route_grad":
            return case
        return {**case, "groups": groups, "top_groups": top_groups, "bias": rng.random() < 0.5}
    while True:
        T, k, K = _log(rng, 1, 8192), rng.randint(1, 8), _log(rng, 16, 8192, 16)
        if T * k * K <= 1 << 26:
            kind = rng.choice(("f16", "bf16", "fp8")) if op == "gather" else case["type"]
            return {**case, "type": kind, "T": T, "k": k, "K": K, "drop": rng.choice((0.0, 0.0, 0.1))}


# ---- inputs -----------------------------------------------------------------
def _pow2(e, dtype):
    """2^e for whole e, exactly (`dtype` has to hold it): the exponent's field of a number of 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64).to(dtype)


def _quantise_fp4(w):
    """(two e2m1 numbers a byte, scale bytes) of w [N, K] in 32 bits."""
    N, K = w.shape
    b = w.reshape(N, K // 32, 32)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1; amax <= 6 * 2^(e - 3) where m <= 3/4
    e = torch.where(amax > 0, e - 3 + (m > 0.75).int(), torch.full_like(e, -127)).clamp(min=-127)
    v = b.double() * _pow2(-e, torch.float64)[..., None]
    a = v.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i, middle in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):  # in the middle the even number is taken
        code += (a >= middle) if i % 2 else (a > middle)
    code = (code + 8 * torch.signbit(b)).to(torch.uint8).reshape(N, K // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _slots(case, g):
    """The row of each slot as a sort by random experts gives it: pos [T, k] int32, -1 for a choice that goes elsewhere."""
    T, k = case["T"], case["k"]
    order = torch.rand(T * k, device="cuda", generator=g)
    away = torch.rand(T * k, device="cuda", generator=g) < case["drop"]
    pos = torch.empty(T * k, dtype=torch.int32, device="cuda")
    pos[(order + away * 2).argsort()] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    pos[away] = -1
    return pos.reshape(T, k)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=g) * scale

    def activations(rows, cols):  # a few columns carry much larger values, as a model's hidden states do
        x = normal(rows, cols)
        x[:, torch.randint(cols, (max(1, cols // 200),), device="cuda", generator=g)] *= 12
        return x

    op = case["op"]
    t = _TYPES.get(case["type"])
    if op == "gemv_fp4":
        M, N, K = case["M"], case["N"], case["K"]
        W, sW = _quantise_fp4(normal(N, K, scale=K**-0.5))
        return {**case, "x": activations(M, K).to(t), "W": W, "sW": sW, "y": torch.empty(M, N, dtype=t, device="cuda"),
                "e2m1": torch.tensor(_E2M1, device="cuda")}
    if op == "quantize_fp4":
        N, K = case["N"], case["K"]
        return {**case, "w": normal(N, K, scale=K**-0.5).to(t), "q": torch.empty(N, K // 2, dtype=torch.uint8, device="cuda"),
                "s": torch.empty(N, K // 32, dtype=torch.uint8, device="cuda")}
    if op in ("rmsnorm", "rmsnorm_grad"):
        T, C = case["T"], case["C"]
        state = {**case, "weight": (1 + normal(C, scale=0.1)).to(t)}
        if op == "rmsnorm":
            state["x"] = activations(T, C).to(t)
            state["r"] = activations(T, C).to(t) if case["residual"] else None
            state["h"] = torch.empty(T, C, dtype=t, device="cuda") if case["residual"] else None
            if case["out"] == 8:
                state["q"] = torch.empty(T, C, dtype=torch.float8_e4m3fn, device="cuda")
                state["scale"] = torch.empty(T, -(-C // _BLOCK), device="cuda")
            else:
                state["y"] = torch.empty(T, C, dtype=t, device="cuda")
            return state
        h = activations(T, C).to(t)
        state.update(h=h, rstd=(h.double().square().mean(1) + _EPS).rsqrt().float(), dy=normal(T, C, scale=0.1).to(t),
                     dh=normal(T, C, scale=0.1).to(t) if case["residual"] else None,
                     dx=torch.empty(T, C, dtype=t, device="cuda"), dweight=torch.empty(C, device="cuda"))
        if own:
            import gemv_tile_pipelined_amd as gt

            state["workspace"] = gt.alloc_rmsnorm_grad_workspace(h)
        return state
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        logits = (normal(T, E, scale=1.5) + normal(E, scale=0.5)).to(t)
        state = {**case, "logits": logits}
        if op == "route":
            state["b"] = normal(E, scale=0.05) if case["bias"] else None
            state["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            state["pos"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            state["weights"] = torch.empty(T, k, device="cuda")
            state["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            if own:
                import gemv_tile_pipelined_amd as gt

                state["workspace"] = gt.alloc_route_sort_workspace(T, E, k, logits.device)
        else:
            state["ids"] = logits.float().argsort(dim=1, descending=True, stable=True)[:, :k].to(torch.int32).contiguous()
            state["dweights"] = normal(T, k)
            state["dlogits"] = torch.empty_like(logits)
        return state
    T, k, K = case["T"], case["k"], case["K"]
    state = {**case, "pos": _slots(case, g)}
    if op == "gather":
        x = activations(T, K)
        if case["type"] == "fp8":
            kb = -(-K // _BLOCK)
            state["x"] = (x * 20).clamp(-448, 448).to(torch.float8_e4m3fn)
            state["s"] = torch.rand(T, kb, device="cuda", generator=g) + 0.01
            state["out"] = torch.full((T * k, K), 0.5, device="cuda").to(torch.float8_e4m3fn)
            state["out_s"] = torch.full((T * k, kb), 0.5, device="cuda")
        else:
            state["x"] = x.to(t)
            state["out"] = torch.full((T * k, K), 0.5, dtype=t, device="cuda")
        return state
    w = torch.rand(T, k, device="cuda", generator=g) + 0.05
    state["weights"] = w / w.sum(1, keepdim=True)
    state["D"] = activations(T * k, K).to(t)
    if op == "combine":
        state["Y"] = torch.empty(T, K, dtype=t, device="cuda")
    else:
        state["dY"] = normal(T, K, scale=0.1).to(t)
        state["dD"] = torch.full((T * k, K), 0.5, dtype=t, device="cuda")
        state["dweights"] = torch.empty(T, k, device="cuda")
    return state


# ---- one pass ---------------------------------------------------------------
def run(state):
    return _kernels(state) if own else _plain(state)


def _kernels(s):
    import gemv_tile_pipelined_amd as gt

    op, t = s["op"], s["type"]

    def call(name):
        return getattr(gt, f"{name}_{t}")

    if op == "gemv_fp4":
        return call("gemv_fp4")(s["x"], s["W"], s["sW"], s["y"])
    if op == "quantize_fp4":
        return call("quantize_fp4")(s["w"], s["q"], s["s"])
    if op == "rmsnorm":
        if s["out"] == 8:
            q, scale, h = call("rmsnorm_fp8")(s["x"], s["weight"], s["r"], _EPS, h=s["h"], q=s["q"], scale=s["scale"])
            return (q, scale, h) if s["residual"] else (q, scale)
        y, h = call("rmsnorm")(s["x"], s["weight"], s["r"], _EPS, h=s["h"], y=s["y"])
        return (y, h) if s["residual"] else y
    if op == "rmsnorm_grad":
        return call("rmsnorm_grad")(s["dy"], s["h"], s["weight"], s["rstd"], s["dh"], s["dx"], s["dweight"],
                                    workspace=s["workspace"])
    if op == "route":
        ids, weights = call("route_topk")(s["logits"], s["k"], s["b"], groups=s["groups"], top_groups=s["top_groups"],
                                          group_best=2 if s["bias"] else 1, score=s["score"], norm=s["norm"], scale=2.5,
                                          ids=s["ids"], weights=s["weights"])
        offsets, pos = gt.route_sort(ids, s["E"], s["offsets"], s["pos"], workspace=s["workspace"])
        return ids, weights, offsets, pos
    if op == "route_grad":
        return call("route_topk_grad")(s["logits"], s["ids"], s["dweights"], score=s["score"], norm=s["norm"], scale=2.5,
                                       dlogits=s["dlogits"])
    if op == "gather":
        if t == "fp8":
            return gt.route_gather_fp8(s["x"], s["s"], s["pos"], s["out"], s["out_s"])
        return call("route_gather")(s["x"], s["pos"], s["out"])
    if op == "combine":
        return call("route_combine")(s["D"], s["pos"], s["weights"], s["Y"])
    return call("route_combine_grad")(s["dY"], s["D"], s["pos"], s["weights"], s["dD"], s["dweights"])


def _widen_fp4(W, sW, table):
    """The values that two e2m1 numbers a byte and their scales stand for."""
    N, half = W.shape
    v = torch.stack([table[(W & 15).int()], table[(W >> 4).int()]], -1).reshape(N, half // 16, 32)
    return (v * _pow2(sW.int() - 127, table.dtype)[..., None]).reshape(N, 2 * half)


def _to_e4m3(y):
    """(numbers, scales) of y [T, C] in 64 bits, a scale for each block of 128 of a row."""
    T, C = y.shape
    b = torch.nn.functional.pad(y, (0, -C % _BLOCK)).reshape(T, -1, _BLOCK)
    scale = (b.abs().amax(-1) / 448).float().clamp(min=2.0**-80)
    v = b / scale.double()[..., None]
    e = torch.frexp(v)[1].clamp(min=-5)  # |v| < 2^e, and e4m3 numbers below that are 2^(e-4) apart
    step = _pow2(e - 4, torch.float64)
    q = (torch.round(v / step) * step).clamp(-448, 448)
    return q.reshape(T, -1)[:, :C].float().contiguous().to(torch.float8_e4m3fn), scale


def _plain(s):
    op, t = s["op"], _TYPES.get(s["type"])
    if op == "gemv_fp4":
        return (s["x"].float() @ _widen_fp4(s["W"], s["sW"], s["e2m1"]).t()).to(t)
    if op == "quantize_fp4":
        return _quantise_fp4(s["w"].float())
    if op == "rmsnorm":
        h = s["x"]
        if s["residual"]:
            h = (s["x"].float() + s["r"].float()).to(t)
        if s["out"] == 8:  # in 64: a value can lie next to the border between two 8-bit numbers
            v = h.double()
            q, scale = _to_e4m3(v * (v.square().mean(1, keepdim=True) + _EPS).rsqrt() * s["weight"].double())
            return (q, scale, h) if s["residual"] else (q, scale)
        v = h.float()
        y = (v * (v.square().mean(1, keepdim=True) + _EPS).rsqrt() * s["weight"].float()).to(t)
        return (y, h) if s["residual"] else y
    if op == "rmsnorm_grad":
        h, r, dy = s["h"].float(), s["rstd"][:, None], s["dy"].float()
        n = h * r
        wdy = dy * s["weight"].float()
        dx = r * (wdy - n * (wdy * n).mean(1, keepdim=True))
        if s["residual"]:
            dx = dx + s["dh"].float()
        return dx.to(t), (dy * n).sum(0, dtype=torch.float64).float()
    if op == "route":
        return _plain_route(s)
    if op == "route_grad":
        l, ids, g = s["logits"].float(), s["ids"].long(), s["dweights"] * 2.5
        if s["score"] == "softmax":
            p = torch.softmax(l, 1) if not s["norm"] else None
            if s["norm"]:
                w = torch.softmax(l.gather(1, ids), 1)
                return torch.zeros_like(l).scatter(1, ids, w * (g - (g * w).sum(1, keepdim=True))).to(t)
            full = torch.zeros_like(l).scatter(1, ids, g)
            return (p * (full - (full * p).sum(1, keepdim=True))).to(t)
        c = torch.sigmoid(l.gather(1, ids))
        if s["norm"]:
            total = c.sum(1, keepdim=True)
            g = (g - (g * c).sum(1, keepdim=True) / total) / total
        return torch.zeros_like(l).scatter(1, ids, g * c * torch.sigmoid(-l.gather(1, ids))).to(t)
    pos, T, k = s["pos"], s["T"], s["k"]
    here = pos >= 0
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)[here]
    rows = pos[here].long()
    if op == "gather":
        if s["type"] == "fp8":
            s["out"].view(torch.uint8)[rows] = s["x"].view(torch.uint8)[token]
            s["out_s"][rows] = s["s"][token]
            return s["out"], s["out_s"]
        s["out"][rows] = s["x"][token]
        return s["out"]
    w = s["weights"] * here
    at = pos.clamp(min=0).long()
    if op == "combine":
        y = torch.zeros(T, s["K"], device="cuda")
        for j in range(k):
            y += w[:, j, None] * s["D"][at[:, j]].float()
        return y.to(t)
    dY = s["dY"].float()
    dw = torch.stack([(dY * s["D"][at[:, j]].float()).sum(1) for j in range(k)], 1) * here
    s["dD"][rows] = (dY[token] * w[here][:, None]).to(t)
    return s["dD"], dw


def _plain_route(s):
    l, k, E, T = s["logits"].double(), s["k"], s["E"], s["T"]  # in 64: two choices can lie next to each other
    score = torch.softmax(l, 1) if s["score"] == "softmax" else torch.sigmoid(l)
    choice = score + s["b"].double() if s["bias"] else l  # without a bias scores are ordered as logits are
    if s["groups"] > 1:
        best = choice.reshape(T, s["groups"], -1).sort(-1, descending=True)[0]
        best = best[..., :2].sum(-1) if s["bias"] else best[..., 0]
        kept = best.argsort(dim=1, descending=True, stable=True)[:, : s["top_groups"]]
        mask = torch.zeros(T, s["groups"], dtype=torch.bool, device="cuda").scatter(1, kept, True)
        choice = choice.masked_fill(~mask.repeat_interleave(E // s["groups"], 1), float("-inf"))
    ids = choice.argsort(dim=1, descending=True, stable=True)[:, :k]
    w = score.gather(1, ids)
    if s["norm"]:
        w = w / w.sum(1, keepdim=True)
    flat = ids.reshape(-1)
    pos = torch.empty(T * k, dtype=torch.int32, device="cuda")
    pos[flat.argsort(stable=True)] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    offsets = torch.searchsorted(flat.sort()[0], torch.arange(E + 1, device="cuda"))
    return ids.int(), (w * 2.5).float(), offsets.int(), pos.reshape(T, k)


# ---- the work of a pass -------------------------------------------------------
def work(case):
    op = case["op"]
    size = {"f32": 4, "fp8": 1}.get(case["type"], 2)
    if op == "gemv_fp4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K // 2 + N * K // 32 + 2 * M * (K + N), "flops": 2 * M * N * K}
    if op == "quantize_fp4":
        n = case["N"] * case["K"]
        return {"bytes": 2 * n + n // 2 + n // 32, "flops": 2 * n}
    if op in ("rmsnorm", "rmsnorm_grad"):
        T, C, r = case["T"], case["C"], case["residual"]
        if op == "rmsnorm_grad":
            return {"bytes": T * C * 2 * (3 + r) + 4 * T + 6 * C, "flops": 10 * T * C}
        out = C + 4 * -(-C // _BLOCK) if case["out"] == 8 else 2 * C
        return {"bytes": T * (2 * C * (1 + 2 * r) + out) + 2 * C, "flops": 6 * T * C}
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        if op == "route":
            return {"bytes": T * E * size + 12 * T * k + 4 * (E + 1) + 4 * E * case["bias"], "flops": 8 * T * E}
        return {"bytes": 2 * T * E * size + 8 * T * k, "flops": 8 * T * E}
    T, k, K = case["T"], case["k"], case["K"]
    rows = T * k * (1 - case["drop"])
    if op == "gather":
        row = K * size + (4 * -(-K // _BLOCK) if case["type"] == "fp8" else 0)
        return {"bytes": int(row * (T + rows) + 4 * T * k), "flops": 0}
    if op == "combine":
        return {"bytes": int(K * size * (T + rows) + 8 * T * k), "flops": int(2 * rows * K)}
    return {"bytes": int(K * size * (T + 2 * rows) + 12 * T * k), "flops": int(3 * rows * K)}


# ---- the definition in 64 bits ------------------------------------------------
def _numbers(fraction_bits, lowest, bias_top):
    """Every non-negative number of a format with subnormals, up to (2 - 2^-fraction_bits) 2^bias_top."""
    steps = 1 << fraction_bits
    low = [m * 2.0 ** (lowest - fraction_bits) for m in range(steps)]
    high = [(steps + m) * 2.0 ** (e - fraction_bits) for e in range(lowest, bias_top + 1) for m in range(steps)]
    return torch.tensor(low + high, dtype=torch.float64, device="cuda")


def _nearest(v, table):
    """Index of the number nearest to v >= 0, the even one of two equally near; beyond the table its largest."""
    middle = (table[1:] + table[:-1]) / 2
    at = torch.searchsorted(middle, v.contiguous())
    tie = (at < middle.numel()) & (v == middle[at.clamp(max=middle.numel() - 1)]) & (at % 2 == 1)
    return at + tie.long()


def _exact_norm(s):
    h = s["x"].double()
    if s["residual"]:
        h = (h + s["r"].double()).to(_TYPES[s["type"]]).double()  # both are 16-bit numbers: the sum in 64 bits is exact
    y = h / ((h * h).sum(1, keepdim=True) / s["C"] + _EPS).sqrt() * s["weight"].double()
    if s["out"] == 16:
        return (y, h) if s["residual"] else y
    table = _numbers(3, -6, 8)[:-1]
    q, scales = torch.empty_like(y), torch.empty(s["T"], -(-s["C"] // _BLOCK), dtype=torch.float64, device="cuda")
    for j in range(scales.shape[1]):
        cut = slice(j * _BLOCK, (j + 1) * _BLOCK)
        scales[:, j] = (y[:, cut].abs().amax(1) / 448).clamp(min=2.0**-80)
        q[:, cut] = torch.copysign(table[_nearest(y[:, cut].abs() / scales[:, j, None].float().double(), table)], y[:, cut])
    return (q, scales, h) if s["residual"] else (q, scales)


def _exact_route(s):
    T, E, k, size = s["T"], s["E"], s["k"], s["E"] // s["groups"]
    l = s["logits"].double()
    if s["score"] == "softmax":
        p = (l - l.amax(1, keepdim=True)).exp()
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + (-l).exp())
    left = p + s["b"].double() if s["bias"] else l.clone()
    index = torch.arange(E, device="cuda")
    low = torch.finfo(torch.float64).min

    def best(v):  # the largest of each row and the lowest index that has it
        top = v.amax(-1, keepdim=True)
        return top[..., 0], torch.where(v == top, index[: v.shape[-1]], E).amin(-1)

    if s["groups"] > 1:
        g = left.reshape(T, s["groups"], size).clone()
        first, at = best(g)
        if s["bias"]:
            first = first + best(g.scatter(2, at[..., None], low))[0]
        kept = torch.zeros(T, s["groups"], dtype=torch.bool, device="cuda")
        for _ in range(s["top_groups"]):
            at = best(first)[1]
            kept.scatter_(1, at[:, None], True)
            first = first.scatter(1, at[:, None], low)
        left = torch.where(kept[:, index // size], left, low)
    ids = torch.empty(T, k, dtype=torch.int64, device="cuda")
    for j in range(k):
        ids[:, j] = best(left)[1]
        left = left.scatter(1, ids[:, j, None], low)
    w = p.gather(1, ids)
    w = 2.5 * (w / w.sum(1, keepdim=True) if s["norm"] else w)
    count = torch.bincount(ids.reshape(-1), minlength=E)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    key = ids.reshape(-1) * (T * k) + torch.arange(T * k, device="cuda")  # by expert, then by slot
    pos = torch.empty_like(key)
    pos[key.sort()[1]] = torch.arange(T * k, device="cuda")
    return ids.int(), w, offsets.int(), pos.reshape(T, k).int()


def _exact_route_grad(s):
    l, ids = s["logits"].double(), s["ids"].long()
    g = 2.5 * s["dweights"].double()
    if s["score"] == "softmax":
        p = (l - l.amax(1, keepdim=True)).exp()
        p = p / p.sum(1, keepdim=True)
        slope = None
    else:
        p = 1 / (1 + (-l).exp())
        slope = p / (1 + l.exp())
    c = p.gather(1, ids)
    if s["norm"]:  # w_j = c_j / sum c
        total = c.sum(1, keepdim=True)
        g = g / total - (g * c).sum(1, keepdim=True) / total**2
    full = torch.zeros_like(l).scatter(1, ids, g)  # with respect to every score
    if slope is not None:
        return full * slope
    return p * (full - (full * p).sum(1, keepdim=True))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemv_fp4":
        out = torch.empty(s["M"], s["N"], dtype=torch.float64, device="cuda")
        magnitude = _numbers(1, 0, 2)
        x = s["x"].double()
        for low in range(0, s["N"], 4096):
            cut = slice(low, low + 4096)
            code = torch.stack([s["W"][cut] % 16, s["W"][cut] // 16], -1).reshape(-1, s["K"]).long()
            v = magnitude[code % 8] * (1 - 2 * (code // 8)).double()
            v = v * _pow2(s["sW"][cut].long() - 127, torch.float64).repeat_interleave(32, 1)
            out[:, cut] = x @ v.t().contiguous()
        return out
    if op == "quantize_fp4":
        N, K = case["N"], case["K"]
        w = s["w"].double().reshape(N, K // 32, 32)
        e = torch.full((N, K // 32), -127, dtype=torch.int64, device="cuda")
        top = w.abs().amax(-1)
        for step in (128, 64, 32, 16, 8, 4, 2, 1):  # the least e from -127 with top <= 6 * 2^e
            e = torch.where(6 * _pow2(e + step - 1, torch.float64) < top, e + step, e)
        code = _nearest(w.abs() / _pow2(e, torch.float64)[..., None], _numbers(1, 0, 2)) + 8 * torch.signbit(w).long()
        code = code.reshape(N, K // 2, 2)
        return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), (e + 127).to(torch.uint8)
    if op == "rmsnorm":
        return _exact_norm(s)
    if op == "rmsnorm_grad":
        h, w, dy, r = s["h"].double(), s["weight"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        dot = (w * dy * h).sum(1, keepdim=True) / case["C"]
        dx = r * w * dy - r**3 * h * dot
        return dx + s["dh"].double() if case["residual"] else dx, (dy * h * r).sum(0)
    if op == "route":
        return _exact_route(s)
    if op == "route_grad":
        return _exact_route_grad(s)
    pos, T, k = s["pos"].long(), case["T"], case["k"]
    if op == "gather":
        out = s["out"].float().double()
        scale = s["out_s"].double() if case["type"] == "fp8" else None
        for j in range(k):
            t = (pos[:, j] >= 0).nonzero()[:, 0]
            out[pos[t, j]] = s["x"].float().double()[t]
            if scale is not None:
                scale[pos[t, j]] = s["s"].double()[t]
        return out if scale is None else (out, scale)
    D, w = s["D"].double(), s["weights"].double()
    if op == "combine":
        padded = torch.cat([D, D.new_zeros(1, case["K"])])  # row -1 is zeros
        return sum(w[:, j, None] * padded[pos[:, j]] for j in range(k))
    dY = s["dY"].double()
    dD, dw = s["dD"].double(), torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = (pos[:, j] >= 0).nonzero()[:, 0]
        dD[pos[t, j]] = dY[t] * w[t, j, None]
        dw[t, j] = (dY[t] * D[pos[t, j]]).sum(1)
    return dD, dw
