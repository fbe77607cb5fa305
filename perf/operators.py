"""What is measured of the block-scaled 8-bit and the expert-grouped matrix products.

Each case is one call of an operator of this library on inputs as a language model's serving or training step has
them.  With ``own`` false, ``run`` computes the operator in its plain form (elementary torch operations in 32 bits, in
64 where a value lies next to a rounding border); with ``own`` true it makes the library's call.

Operators (T rows sorted by expert, expert e owning rows offsets[e] .. offsets[e+1]; 8-bit values are e4m3):

  fp8          D[m,n]   = sum_k (sA[m,k/128] A[m,k]) (sB[n/r,k/128] B[n,k]),  r = 128 or 1
  grouped      D[t,n]   = sum_k X[t,k] W[e(t),n,k]
  dgrad        dX[t,k]  = sum_n dY[t,n] W[e(t),n,k]
  wgrad        dW[e,n,k] = sum over the rows t of e of dY[t,n] X[t,k]
  grouped_fp8  D[t,n]   = sum_k (sX[t,k/128] X[t,k]) (sW[e(t),n/128,k/128] W[e(t),n,k])
  quant_rows   scale = max(amax / 448, 2^-80) of each row's blocks of 128 columns, q = e4m3(x / scale)
  quant_tiles  the same of 128 x 128 tiles of each matrix
"""
import numpy as np
import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
_BLOCK = 128


def listed():
    return [
        # One token through a down projection held in 8 bits (the shape of this library's GEMV benchmark).
        {"name": "fp8 one token", "op": "fp8", "type": "bf16", "M": 1, "N": 4096, "K": 14336, "b_rows": 128},
        # A decode batch of an odd size against a square projection.
        {"name": "fp8 decode batch", "op": "fp8", "type": "f16", "M": 27, "N": 8192, "K": 4096, "b_rows": 128},
        # A prompt's worth of tokens (the benchmark's GEMM shape).
        {"name": "fp8 prefill", "op": "fp8", "type": "bf16", "M": 4096, "N": 4096, "K": 4096, "b_rows": 128},
        # A weight's gradient of an 8-bit training step: both sides scaled by rows, ragged sizes.
        {"name": "fp8 ragged rows", "op": "fp8", "type": "f16", "M": 4000, "N": 4035, "K": 4112, "b_rows": 1},
        # Four tokens, each sent to eight of 64 experts.
        {"name": "grouped decode", "op": "grouped", "type": "bf16", "T": 32, "pad": 0, "E": 64, "N": 2048, "K": 2048,
         "skew": 0.0},
        # A prompt over 16 experts of uneven load, in a buffer with spare rows at its end.
        {"name": "grouped prefill", "op": "grouped", "type": "f16", "T": 8200, "pad": 137, "E": 16, "N": 4096,
         "K": 2048, "skew": 0.5},
        # The two gradients of such a layer in a training step.
        {"name": "grouped dgrad", "op": "dgrad", "type": "bf16", "T": 8192, "pad": 0, "E": 16, "N": 4096, "K": 2048,
         "skew": 0.5},
        {"name": "grouped wgrad", "op": "wgrad", "type": "bf16", "T": 8192, "pad": 5, "E": 16, "N": 4096, "K": 2048,
         "skew": 0.5},
        # One token's eight experts of 64, weights held in 8 bits.
        {"name": "grouped fp8 one token", "op": "grouped_fp8", "type": "bf16", "T": 8, "pad": 0, "E": 64, "N": 4096,
         "K": 2048, "skew": 0.0},
        # Many prompts at once through 32 experts held in 8 bits.
        {"name": "grouped fp8 prefill", "op": "grouped_fp8", "type": "bf16", "T": 16384, "pad": 0, "E": 32, "N": 4096,
         "K": 4096, "skew": 0.5},
        # Activations of a prompt, quantised before a product.
        {"name": "quantise rows", "op": "quant_rows", "type": "bf16", "M": 8192, "K": 4096},
        # A weight matrix of odd height, quantised when it is loaded or after a step.
        {"name": "quantise tiles", "op": "quant_tiles", "type": "f16", "E": 1, "N": 4095, "K": 14336},
    ]


def _log(rng, low, high, multiple=1):
    """A size of low .. high, spread over its logarithm, and a multiple of `multiple`."""
    v = int(round(low * (high / low) ** rng.random()))
    return max(multiple, v // multiple * multiple)


def draw(rng):
    op = rng.choice(("fp8", "grouped", "dgrad", "wgrad", "grouped_fp8", "quant_rows", "quant_tiles"))
    case = {"op": op, "type": rng.choice(("f16", "bf16"))}
    if op == "fp8":
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 1, 16384), _log(rng, 16, 16384, 16)
            if 1 << 16 <= M * N * K <= 1 << 37:
                return {**case, "M": M, "N": N, "K": K, "b_rows": rng.choice((128, 128, 1))}
    if op == "quant_rows":
        return {**case, "M": _log(rng, 1, 8192), "K": _log(rng, 16, 8192, 16)}
    if op == "quant_tiles":
        return {**case, "E": _log(rng, 1, 8), "N": _log(rng, 1, 4096), "K": _log(rng, 16, 8192, 16)}
    step_n = 8 if op in ("dgrad", "wgrad") else 1
    step_k = 16 if op == "grouped_fp8" else 8
    while True:
        T, E = _log(rng, 1, 16384), _log(rng, 1, 128)
        N, K = _log(rng, 16, 8192, step_n), _log(rng, 16, 8192, step_k)
        pad = min(T - 1, rng.choice((0, 0, 1, 37)))
        if E * N * K <= 1 << 29 and (T + 8 * E) * N * K <= 1 << 36:
            return {**case, "T": T, "pad": pad, "E": E, "N": N, "K": K, "skew": rng.choice((0.0, 0.5, 1.0))}


# ---- inputs -----------------------------------------------------------------
def _sizes(case, seed=None):
    """Rows of each expert: the same numbers for every seed, dealt out to the experts by the seed."""
    r = np.random.RandomState((case["E"] * 1000003 + case["T"]) % (1 << 31))
    p = np.exp(case["skew"] * r.standard_normal(case["E"]))
    sizes = r.multinomial(case["T"] - case["pad"], p / p.sum())
    if seed is not None:
        np.random.RandomState(seed % (1 << 31)).shuffle(sizes)
    return sizes


def _quantise(x, rows):
    """(e4m3 values, scales) of the blocks of `rows` x 128 of x [..., R, C] in 32 bits."""
    *lead, R, C = x.shape
    pr, pc = -R % rows, -C % _BLOCK
    y = torch.nn.functional.pad(x, (0, pc, 0, pr)) if pr or pc else x
    y = y.reshape(*lead, (R + pr) // rows, rows, (C + pc) // _BLOCK, _BLOCK)
    scale = y.abs().amax((-3, -1)) / 448
    q = y / scale.clamp(min=2.0**-80)[..., :, None, :, None]
    q = q.reshape(*lead, R + pr, C + pc)[..., :R, :C]
    return q.contiguous().to(torch.float8_e4m3fn), scale.clamp(min=2.0**-80)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=g) * scale

    def activations(rows, cols):  # a few columns carry much larger values, as a model's hidden states do
        x = normal(rows, cols)
        x[:, torch.randint(cols, (max(1, cols // 200),), device="cuda", generator=g)] *= 12
        return x

    op, t = case["op"], _TYPES[case["type"]]
    if op == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        A, sA = _quantise(activations(M, K), 1)
        B, sB = _quantise(normal(N, K, scale=K**-0.5), case["b_rows"])
        return {**case, "A": A, "sA": sA, "B": B, "sB": sB, "D": torch.empty(M, N, dtype=t, device="cuda")}
    if op == "quant_rows":
        x = activations(case["M"], case["K"]).to(t)
        return {**case, "x": x, "q": torch.empty_like(x, dtype=torch.float8_e4m3fn),
                "scale": torch.empty(case["M"], -(-case["K"] // _BLOCK), device="cuda")}
    if op == "quant_tiles":
        E, N, K = case["E"], case["N"], case["K"]
        x = normal(E, N, K, scale=K**-0.5).to(t)
        return {**case, "x": x, "q": torch.empty_like(x, dtype=torch.float8_e4m3fn),
                "scale": torch.empty(E, -(-N // _BLOCK), -(-K // _BLOCK), device="cuda")}
    T, E, N, K = case["T"], case["E"], case["N"], case["K"]
    sizes = _sizes(case, seed)
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    state = {**case, "offsets": offsets, "rows": int(sizes.sum()), "most": int(sizes.max())}
    if op != "wgrad":
        W = normal(E, N, K, scale=K**-0.5)
        if op == "grouped_fp8":
            state["W"], state["sW"] = _quantise(W, _BLOCK)
        else:
            state["W"] = W.to(t)
        del W
    if op == "grouped_fp8":
        state["X"], state["sX"] = _quantise(activations(T, K), 1)
    elif op != "dgrad":
        state["X"] = activations(T, K).to(t)
    if op in ("dgrad", "wgrad"):
        state["dY"] = normal(T, N, scale=0.1).to(t)
    shape = (E, N, K) if op == "wgrad" else (T, K) if op == "dgrad" else (T, N)
    state["D"] = torch.full(shape, 0.5, dtype=t, device="cuda")  # rows behind the last expert keep this
    return state


# ---- one pass ---------------------------------------------------------------
def run(state):
    return _kernels(state) if own else _plain(state)


def _kernels(s):
    import gemv_tile_pipelined_amd as gt

    op, t = s["op"], s["type"]
    if op == "fp8":
        call = gt.gemm_fp8_f16 if t == "f16" else gt.gemm_fp8_bf16
        return call(s["A"], s["sA"], s["B"], s["sB"], s["D"])
    if op == "grouped":
        call = gt.gemm_grouped_f16 if t == "f16" else gt.gemm_grouped_bf16
        return call(s["X"], s["W"], s["offsets"], s["D"])
    if op == "dgrad":
        call = gt.gemm_grouped_dgrad_f16 if t == "f16" else gt.gemm_grouped_dgrad_bf16
        return call(s["dY"], s["W"], s["offsets"], s["D"])
    if op == "wgrad":
        call = gt.gemm_grouped_wgrad_f16 if t == "f16" else gt.gemm_grouped_wgrad_bf16
        return call(s["dY"], s["X"], s["offsets"], s["D"])
    if op == "grouped_fp8":
        call = gt.gemm_grouped_fp8_f16 if t == "f16" else gt.gemm_grouped_fp8_bf16
        return call(s["X"], s["sX"], s["W"], s["sW"], s["offsets"], s["D"])
    if op == "quant_rows":
        call = gt.quantize_fp8_rows_f16 if t == "f16" else gt.quantize_fp8_rows_bf16
    else:
        call = gt.quantize_fp8_tiles_f16 if t == "f16" else gt.quantize_fp8_tiles_bf16
    return call(s["x"], s["q"], s["scale"])


def _widen(q, scale, rows):
    """The values that e4m3 numbers and their scales stand for, in 32 bits."""
    R, C = q.shape[-2:]
    if rows > 1:
        scale = scale.repeat_interleave(rows, -2)[..., :R, :]
    return q.float() * scale.repeat_interleave(_BLOCK, -1)[..., :C]


def _buckets(s, x):
    """x [T, C] as [E, most rows of an expert, C] in 32 bits, zeros behind each expert's rows, and the row and expert
    numbers that take a result back."""
    at = torch.arange(s["rows"], device="cuda")
    expert = torch.searchsorted(s["offsets"][1:], at, right=True)
    slot = at - s["offsets"][expert]
    b = torch.zeros(s["E"], max(1, s["most"]), x.shape[1], device="cuda")
    b[expert, slot] = x[: s["rows"]].float()
    return b, expert, slot


def _plain(s):
    op, t = s["op"], _TYPES[s["type"]]
    if op == "fp8":
        return (_widen(s["A"], s["sA"], 1) @ _widen(s["B"], s["sB"], s["b_rows"]).t()).to(t)
    if op in ("grouped", "grouped_fp8"):
        x, w = (s["X"], s["W"].float()) if op == "grouped" else (_widen(s["X"], s["sX"], 1), _widen(s["W"], s["sW"], _BLOCK))
        b, expert, slot = _buckets(s, x)
        out = torch.bmm(b, w.transpose(1, 2).contiguous())
    elif op == "dgrad":
        b, expert, slot = _buckets(s, s["dY"])
        out = torch.bmm(b, s["W"].float())
    elif op == "wgrad":
        b, expert, slot = _buckets(s, s["dY"])
        return torch.bmm(b.transpose(1, 2).contiguous(), _buckets(s, s["X"])[0]).to(t)
    else:
        return _plain_quantise(s["x"], 1 if op == "quant_rows" else _BLOCK)
    s["D"][: s["rows"]] = out[expert, slot].to(t)
    return s["D"]


def _plain_quantise(x, rows):
    *lead, R, C = x.shape
    pr, pc = -R % rows, -C % _BLOCK
    y = torch.nn.functional.pad(x.float(), (0, pc, 0, pr))
    y = y.reshape(*lead, (R + pr) // rows, rows, (C + pc) // _BLOCK, _BLOCK)
    scale = (y.abs().amax((-3, -1)).double() / 448).float().clamp(min=2.0**-80)  # in 64: the nearest 32-bit number
    # A quotient can lie closer to the middle between two e4m3 numbers than 32 bits show.
    v = y.double() / scale.double()[..., :, None, :, None]
    e = torch.frexp(v)[1].clamp(min=-5)  # |v| < 2^e, and e4m3 numbers below that are 2^(e-4) apart
    step = torch.bitwise_left_shift(torch.ones_like(e), e + 5).double() / 512
    q = (torch.round(v / step) * step).reshape(*lead, R + pr, C + pc)[..., :R, :C]
    return q.to(torch.float32).contiguous().to(torch.float8_e4m3fn), scale


# ---- the work of a pass -------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // _BLOCK)
        scales = 4 * kb * (M + -(-N // case["b_rows"]))
        return {"bytes": M * K + N * K + scales + 2 * M * N, "flops": 2 * M * N * K}
    if op in ("quant_rows", "quant_tiles"):
        n = case.get("E", 1) * case.get("N", case.get("M", 0)) * case["K"]
        per = _BLOCK if op == "quant_rows" else _BLOCK * _BLOCK
        return {"bytes": 3 * n + 4 * (n // per), "flops": 2 * n}
    N, K, rows = case["N"], case["K"], case["T"] - case["pad"]
    used = int((_sizes(case) > 0).sum())
    flops = 2 * rows * N * K
    if op == "wgrad":
        return {"bytes": 2 * (rows * (N + K) + case["E"] * N * K), "flops": flops}
    if op == "grouped_fp8":
        kb = -(-K // _BLOCK)
        scales = 4 * kb * (rows + used * -(-N // _BLOCK))
        return {"bytes": rows * K + used * N * K + scales + 2 * rows * N, "flops": flops}
    return {"bytes": 2 * (rows * (N + K) + used * N * K), "flops": flops}


# ---- the definition in 64 bits ------------------------------------------------
def _e4m3_numbers():
    """Every non-negative e4m3 number in order: m 2^-9 below 2^-6, then (8 + m) 2^(e-3), up to 448."""
    values = [m * 2.0**-9 for m in range(8)]
    values += [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)]
    return torch.tensor(values[:-1], dtype=torch.float64, device="cuda")


def _exact_quantise(x, rows):
    """Block by block: the scale as a 32-bit number, then the nearest e4m3 number, the even one of two equally near."""
    R, C = x.shape
    table = _e4m3_numbers()
    middle = (table[1:] + table[:-1]) / 2
    q = torch.empty(R, C, dtype=torch.float64, device="cuda")
    scales = torch.empty(-(-R // rows), -(-C // _BLOCK), dtype=torch.float64, device="cuda")
    for j in range(scales.shape[1]):
        block = x[:, j * _BLOCK : (j + 1) * _BLOCK].double()
        top = block.abs().amax(1)
        top = torch.stack([part.max() for part in top.split(rows)]) if rows > 1 else top
        scale = (top / 448).float().double().clamp(min=2.0**-80)
        scales[:, j] = scale
        v = block.abs() / scale.repeat_interleave(rows)[:R, None]
        at = torch.searchsorted(middle, v.contiguous())  # middle[at-1] < v <= middle[at]
        tie = (at < middle.numel()) & (v == middle[at.clamp(max=middle.numel() - 1)]) & (at % 2 == 1)
        q[:, j * _BLOCK : (j + 1) * _BLOCK] = torch.copysign(table[at + tie.long()], block)
    return q, scales


def _block_product(a, sa, b, sb, b_rows):
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device="cuda")
    for j in range(sa.shape[1]):
        cut = slice(j * _BLOCK, (j + 1) * _BLOCK)
        right = sb[torch.arange(b.shape[0], device="cuda") // b_rows, j].double()
        out += (a[:, cut].double() @ b[:, cut].double().t().contiguous()) * sa[:, j, None].double() * right
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fp8":
        return _block_product(s["A"], s["sA"], s["B"], s["sB"], case["b_rows"])
    if op == "quant_rows":
        return _exact_quantise(s["x"], 1)
    if op == "quant_tiles":
        parts = [_exact_quantise(x, _BLOCK) for x in s["x"]]
        return torch.stack([q for q, _ in parts]), torch.stack([c for _, c in parts])
    out = s["D"].double()
    cuts = s["offsets"].tolist()
    for e, (low, high) in enumerate(zip(cuts[:-1], cuts[1:])):
        if op == "wgrad":
            out[e] = s["dY"][low:high].double().t().contiguous() @ s["X"][low:high].double()
        elif low == high:
            continue
        elif op == "dgrad":
            out[low:high] = s["dY"][low:high].double() @ s["W"][e].double()
        elif op == "grouped":
            out[low:high] = s["X"][low:high].double() @ s["W"][e].double().t().contiguous()
        else:
            out[low:high] = _block_product(s["X"][low:high], s["sX"][low:high], s["W"][e], s["sW"][e], _BLOCK)
    return out
