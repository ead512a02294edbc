"""What is measured of the operators of a training step around its linears:
layer norm with its output packed (mx.layernorm_fwd) and its backward pass
(mx.layernorm_bwd), the cross entropy of a vocabulary projection whose logits
are never kept (mx.head_loss) and its gradient (mx.head_loss_bwd), and the
AdamW step over many tensors with states in 32 or 8 bits (mx.adamw).

Definitions.  A packed operand is [rows] x K codes (E2M1, E2M3 or E4M3) with
one power of two per 32 consecutive elements of K, in the library's
K-group-major layout.  Q packs along the inner dimension of the product that
follows, for E2M3 after a 32-point Hadamard rotation.

  norm           h = (x - mean) rstd,  y = h gamma + beta; the row operand
                 packs y rounded to bf16.
  norm backward  g = dy gamma,  dx = rstd (g - mean(g) - h mean(g h)) + residual,
                 dgamma, dbeta = sums over the tokens of dy h, dy.
  loss           l = X W^T,  lse = log sum exp l,  loss = lse - l[label]; 0
                 where the label is no class.
  gradient       G = dloss (exp(l - lse) - [class = label]), 0 where the label
                 is no class;  dX = Q(G) W,  dW = Q(G^T) Q(X^T)^T.
  update         m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
                 p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps).
                 States in 8 bits hold m and sqrt(v) in E4M3, one scale a
                 block of 32; a value between two codes becomes the one
                 further from zero where its share of the step, in 2^-16,
                 is above 16 random bits (low half of the element's word for m,
                 high half for sqrt(v)).  Words: Philox4x32-10, counter
                 (i / 4, 0, tensor, step) and the key from the seed, word i % 4.

With `own` false everything is computed by elementary torch operations in 32
bits; with `own` true by the library's calls on the same data."""
import math
import random

import torch

own = False

E2M1, E2M3, E4M3 = 1, 2, 3
BITS = {E2M1: 4, E2M3: 6, E4M3: 8}
FORMATS = {"mxfp4": E2M1, "mxfp6": E2M3, "mxfp8": E4M3}
EPS = 1e-5
PIECE = 16384  # classes whose gradient is in memory at a time
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP, SEED = 3e-4, 0.9, 0.999, 1e-8, 0.1, 37, 0x5EED0001
SCALE = 0.75  # what gradient clipping multiplies every gradient with


def listed():
    return [
        # the norm in front of a served MXFP8 linear, one token: latency is all that counts
        norm("norm token mxfp8", 1, 4096, "bf16", True),
        # a short ragged prompt, residual stream and weights in binary32, nothing packed
        norm("norm odd", 333, 2080, "f32", False),
        # a training step's tokens, one short of whole tiles, packed for an MXFP8 linear
        norm("norm large mxfp8", 8191, 8192, "bf16", True),
        # a small ragged batch's backward pass, width off every power of two
        norm_bwd("norm backward odd", 1003, 776, "f32", False),
        # the backward pass of a training step, the residual stream's gradient added
        norm_bwd("norm backward large", 8191, 4096, "bf16", True),
        # the score of one served token: the projection's weights are read once
        head("loss", "loss token mxfp4", 1, 32000, 4096, "mxfp4"),
        # a ragged evaluation batch, classes in no multiple of anything
        head("loss", "loss odd mxfp6", 333, 50257, 800, "mxfp6"),
        # the loss of a training step's tokens
        head("loss", "loss large mxfp6", 8192, 128000, 2048, "mxfp6"),
        # fine-tuning on a ragged batch: two pieces of the vocabulary, the last one odd
        head("gradient", "gradient odd mxfp4", 1003, 32003, 2080, "mxfp4"),
        # the gradient of a training step: four pieces
        head("gradient", "gradient large mxfp8", 8192, 65536, 4096, "mxfp8"),
        # a step over norms' and biases' many small tensors
        update("update small", 148, 1, 12288, 32, "f32", False),
        # a step over the matrices of a few layers: bf16 gradients, states in 8 bits, bf16 weights for the packers
        update("update large 8-bit", 9, 1 << 20, 1 << 26, 8, "bf16", True),
    ]


def norm(name, M, C, dtype, packed):
    return {"name": name, "op": "norm", "M": M, "C": C, "dtype": dtype, "packed": packed}


def norm_bwd(name, M, C, dtype, residual):
    return {"name": name, "op": "norm backward", "M": M, "C": C, "dtype": dtype, "residual": residual}


def head(op, name, M, V, K, fmt):
    return {"name": name, "op": op, "M": M, "V": V, "K": K, "fmt": fmt}


def update(name, count, least, most, bits, grad, copy):
    return {"name": name, "op": "update", "count": count, "least": least, "most": most, "bits": bits, "grad": grad,
            "copy": copy}


def draw(rng):
    """One more case: sizes spread over their logarithm, tokens, classes and tensor lengths of any number."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm backward", "loss", "gradient", "update"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "norm":
        packed = rng.random() < 0.6
        C = 32 * log(2, 512) if packed else 8 * log(8, 2048)
        return {"op": op, "M": min(log(1, 16384), 8191 * 8192 // C), "C": C, "dtype": dtype, "packed": packed}
    if op == "norm backward":
        C = 8 * log(8, 2048)
        return {"op": op, "M": min(log(1, 16384), 8191 * 4096 // C), "C": C, "dtype": dtype,
                "residual": rng.random() < 0.5}
    if op in ("loss", "gradient"):
        M, V, K = log(1, 8192), log(128, 131072), 32 * log(2, 256)
        return {"op": op, "M": max(1, min(M, 8192 * 65536 * 4096 // (V * K))), "V": V, "K": K,
                "fmt": rng.choice(sorted(FORMATS))}
    count, most = log(1, 200), log(1024, 1 << 26)
    while count * most > 1 << 28:
        count = max(1, count // 2)
    return {"op": op, "count": count, "least": rng.choice([1, min(most, 777)]), "most": most,
            "bits": rng.choice([8, 32]), "grad": dtype, "copy": rng.random() < 0.5}


def lengths(case):
    """The tensors' lengths: spread over their logarithm, the first the longest (the case alone says them)."""
    r = random.Random("%d %d %d" % (case["count"], case["least"], case["most"]))
    lo, hi = math.log(case["least"]), math.log(case["most"])
    return [case["most"]] + [int(round(math.exp(r.uniform(lo, hi)))) for _ in range(case["count"] - 1)]


def work(case):
    def packed(rows, k, fmt):
        return rows * k * (BITS[fmt] / 8 + 1 / 32)

    if case["op"] in ("norm", "norm backward"):
        M, C = case["M"], case["C"]
        size = 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "norm":
            b = 2 * size * M * C + 2 * size * C + 8 * M + (packed(M, C, E4M3) if case["packed"] else 0)
            return {"bytes": b, "flops": 8 * M * C}
        b = (4 if case["residual"] else 3) * size * M * C + size * C + 8 * M + 8 * C
        return {"bytes": b, "flops": 14 * M * C}
    if case["op"] == "update":
        n = sum(lengths(case))
        b = 8 + (2 if case["grad"] == "bf16" else 4) + (16 if case["bits"] == 32 else 4 * 33 / 32) + (2 if case["copy"] else 0)
        return {"bytes": n * b, "flops": 20 * n}
    M, V, K, fmt = case["M"], case["V"], case["K"], FORMATS[case["fmt"]]
    b = packed(M, K, fmt) + packed(V, K, fmt) + 16 * M
    if case["op"] == "loss":
        return {"bytes": b, "flops": 2 * M * V * K}
    b += packed(K, V, fmt) + packed(K, M, fmt) + 2 * M * K + 2 * V * K
    return {"bytes": b, "flops": 6 * M * V * K}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm backward"):
        M, C = case["M"], case["C"]
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a residual stream: channels of unlike size and offset
        x = normal(M, C) * torch.exp(normal(1, C, std=0.5)) + 0.3 + normal(1, C, std=0.5)
        s["x"], s["gamma"], s["beta"] = x.to(t), (1 + normal(C, std=0.1)).to(t), normal(C, std=0.1).to(t)
        s["mean"], s["rstd"] = empty(M), empty(M)
        if op == "norm":
            s["y"] = empty(M, C, dtype=t)
            s["row"] = empty_operand(M, C, E4M3) if case["packed"] else None
            return s
        xd = s["x"].double()
        mean = xd.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = ((xd - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        s["dy"] = normal(M, C, std=0.01).to(t)
        s["residual"] = normal(M, C, std=0.01).to(t) if case["residual"] else None
        s["dx"], s["dgamma"], s["dbeta"] = empty(M, C, dtype=t), empty(C), empty(C)
        s["partials"] = empty(256, 2, C)
        return s
    if op == "update":
        return prepare_update(s, case, normal)
    M, V, K, fmt = case["M"], case["V"], case["K"], FORMATS[case["fmt"]]
    s["rotation"] = rotation(torch.float32)
    s["table"] = torch.tensor(code_values(fmt), device="cuda")
    rotate = s["rotation"] if fmt == E2M3 else None
    w = normal(V, K, std=0.02)
    labels = torch.randint(0, V, (M,), generator=g, device="cuda")
    # hidden states of a model that has learnt something: some lean towards their label's row
    lean = 8 * torch.rand(M, 1, generator=g, device="cuda") * (torch.rand(M, 1, generator=g, device="cuda") < 0.5)
    x = normal(M, K) + lean * torch.nn.functional.normalize(w[labels], dim=1)
    # the prompt's tokens have no label
    s["labels"] = torch.where(torch.rand(M, generator=g, device="cuda") < 0.125, torch.full_like(labels, -100), labels)
    s["A"], s["B"] = pack(x, fmt, rotate), pack(w, fmt, rotate)
    s["loss"], s["lse"] = empty(M), empty(M)
    s["work"] = empty((V + 127) // 128 * 2 * M + M)
    if op == "loss":
        return s
    s["Wc"], s["Xc"] = pack(pad_rows(w).t(), fmt, rotate), pack(pad_rows(x).t(), fmt, rotate)
    l = unpacked(s["A"], K, fmt, s["table"]) @ unpacked(s["B"], K, fmt, s["table"]).t()
    s["lse"] = torch.logsumexp(l.double(), 1).float()
    n = (s["labels"] >= 0).sum().clamp(min=1)
    s["dloss"] = (0.5 + torch.rand(M, generator=g, device="cuda")) / n  # the tokens' weights in the mean
    s["dX"], s["dW"] = empty(M, K, dtype=torch.bfloat16), empty(V, K, dtype=torch.bfloat16)
    piece = min(PIECE, (V + 127) // 128 * 128)
    s["Gr"], s["Gc"] = empty_operand(M, piece, fmt), empty_operand(piece, M, fmt)
    s["sums"] = empty(M, K) if V > piece else None
    return s


def prepare_update(s, case, normal):
    """Tensors one after the other in flat buffers, each at a multiple of 128 elements, and the library's table of them."""
    sizes = lengths(case)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += (n + 127) // 128 * 128
    used = torch.zeros(total, dtype=torch.bool, device="cuda")
    for at, n in zip(starts, sizes):
        used[at:at + n] = True
    scale = torch.exp(normal(total // 128, 1, std=1.0)).expand(total // 128, 128).reshape(total)  # rows of unlike gradients
    s["sizes"], s["starts"], s["used"] = sizes, starts, used
    s["p"] = normal(total, std=0.02) * used
    s["g"] = (normal(total, std=1e-3) * scale * used).to(torch.bfloat16 if case["grad"] == "bf16" else torch.float32)
    m, u = normal(total, std=3e-4) * scale * used, normal(total, std=1e-3).abs() * scale * used
    s["copy"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
    s["scale"] = torch.full((1,), SCALE, device="cuda")
    if case["bits"] == 8:
        s["m"], s["v"] = pack(m[None], E4M3, None), pack(u[None], E4M3, None)
    else:
        s["m"], s["v"] = m, u * u
    if own:
        from microscaling_block_scaled_mx_amd import mx

        def state(t, at, n):
            if case["bits"] == 32:
                return t[at:at + n]
            groups = (n + 127) // 128
            return t[0][at // 128:at // 128 + groups], t[1][at // 128:at // 128 + groups]

        s["items"] = mx.adamw_items([
            {"p": s["p"][at:at + n], "g": s["g"][at:at + n], "m": state(s["m"], at, n), "v": state(s["v"], at, n),
             "copy": s["copy"][at:at + n] if case["copy"] else None} for at, n in zip(starts, sizes)])
    return s


def empty_operand(rows, K, fmt):
    groups = (K + 127) // 128
    return (torch.empty(groups, rows, 16 * BITS[fmt], dtype=torch.uint8, device="cuda"),
            torch.empty(groups, rows, 4, dtype=torch.uint8, device="cuda"))


def code_values(fmt):
    """The value of every code of a format (sign, exponent, mantissa; bias 1, 1 and 7)."""
    e_bits, m_bits, bias = {E2M1: (2, 1, 1), E2M3: (2, 3, 1), E4M3: (4, 3, 7)}[fmt]
    out = []
    for c in range(1 << (1 + e_bits + m_bits)):
        m, e = c & ((1 << m_bits) - 1), (c >> m_bits) & ((1 << e_bits) - 1)
        v = (m / 2 ** m_bits if e == 0 else 1 + m / 2 ** m_bits) * 2.0 ** (max(e, 1) - bias)
        out.append(-v if c >> (e_bits + m_bits) else v)
    if fmt == E4M3:
        out[0x7F] = out[0xFF] = math.nan
    return out


def rotation(dtype):
    """The 32-point Hadamard matrix (Sylvester order), normalised."""
    i = torch.arange(32, device="cuda")
    bits = i[:, None] & i[None, :]
    odd = (bits ^ (bits >> 1) ^ (bits >> 2) ^ (bits >> 3) ^ (bits >> 4)) & 1
    return (1.0 - 2.0 * odd.to(dtype)) / math.sqrt(32.0)


def quantise(x, fmt, rotate):
    """x [rows][K] float32 -> element values v / 2^X on the format's grid and the exponents X, per block of 32."""
    b = x.reshape(x.shape[0], -1, 32)
    if rotate is not None:
        b = b @ rotate
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1
    if fmt == E4M3:
        X = e - 9 + (m > 0.875).to(e.dtype)  # smallest X with 448 2^X >= amax
    else:
        X = e - 3  # floor(log2 amax) - 2
    X = torch.where(amax == 0, torch.full_like(X, -127), X.clamp(-127, 127))
    v = torch.ldexp(b, -X[..., None])
    if fmt == E4M3:
        q = v.to(torch.float8_e4m3fn).float()
    else:
        a = v.abs()
        fine = 2.0 if fmt == E2M1 else 8.0  # codes per unit below 2
        step = torch.where(a < 2, fine, torch.where(a < 4, fine / 2, fine / 4))
        q = ((a * step).round() / step).clamp(max=6.0 if fmt == E2M1 else 7.5).copysign(v)
    return q, X


def values(x, fmt, rotate):
    """What x [rows][K] stands for after packing (in the rotated basis where there is one), float32."""
    q, X = quantise(x, fmt, rotate)
    return torch.ldexp(q, X[..., None]).reshape(x.shape)


def pack(x, fmt, rotate):
    """x [rows][K] -> (codes, scales) of the packed layout."""
    q, X = quantise(x, fmt, rotate)
    return layout(q, X, x.shape[0], x.shape[1], fmt)


def layout(q, X, rows, K, fmt):
    bits = BITS[fmt]
    groups = (K + 127) // 128
    if fmt == E4M3:
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8).reshape(rows, K)
    else:
        a = q.abs()
        fine = 2 if fmt == E2M1 else 8
        mag = torch.where(a < 2, a * fine, torch.where(a < 4, a * fine / 2 + fine, a * fine / 4 + 2 * fine))
        codes = (mag.to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << (bits - 1))).reshape(rows, K)
    codes = torch.nn.functional.pad(codes, (0, groups * 128 - K)).reshape(rows, groups, 4, 32)
    scales = torch.nn.functional.pad((X + 127).to(torch.uint8), (0, groups * 4 - K // 32)).reshape(rows, groups, 4)
    if fmt == E2M1:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    elif fmt == E2M3:
        c = codes.reshape(rows, groups, 4, 8, 4).int()
        word = c[..., 0] | (c[..., 1] << 6) | (c[..., 2] << 12) | (c[..., 3] << 18)
        stream = torch.stack((word & 255, (word >> 8) & 255, word >> 16), -1).to(torch.uint8).reshape(rows, groups, 4, 24)
        tails = torch.gather(stream[..., 16:], 2, tail_order(rows, groups, q.device))
        codes = torch.cat((stream[..., :16].reshape(rows, groups, 64), tails.reshape(rows, groups, 32)), -1)
    codes = codes.reshape(rows, groups, 16 * bits)
    return codes.transpose(0, 1).contiguous(), scales.transpose(0, 1).contiguous()


def tail_order(rows, groups, device):
    """E2M3: which block's last 8 bytes stand at each of a row's four places (pairs swapped where bit 4 of the row is set)."""
    swap = (torch.arange(rows, device=device) >> 4) & 1
    at = torch.arange(4, device=device)[None, :] ^ swap[:, None]
    return at[:, None, :, None].expand(rows, groups, 4, 8)


def pad_rows(x):
    return torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % 32))


def eight_bits(codes, scales):
    """An E4M3 operand as the values it is made of: its elements' and its blocks' scales."""
    return {"elements": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


# ------------------------------------------------------------------ the plain forms
def unpacked(operand, K, fmt, table):
    """(codes, scales) -> the values [rows][K] that they stand for, float32."""
    codes, scales = operand[0].transpose(0, 1), operand[1].transpose(0, 1)
    rows, groups = codes.shape[:2]
    if fmt == E4M3:
        q = codes.contiguous().view(torch.float8_e4m3fn).float()
    elif fmt == E2M1:
        q = table[torch.stack((codes & 15, codes >> 4), -1).int()]
    else:
        tails = torch.gather(codes[..., 64:].reshape(rows, groups, 4, 8), 2, tail_order(rows, groups, codes.device))
        t = torch.cat((codes[..., :64].reshape(rows, groups, 4, 16), tails), -1).reshape(rows, groups, 4, 8, 3).int()
        word = t[..., 0] | (t[..., 1] << 8) | (t[..., 2] << 16)
        q = table[torch.stack((word & 63, (word >> 6) & 63, (word >> 12) & 63, word >> 18), -1)]
    v = torch.ldexp(q.reshape(rows, groups * 4, 32), scales.reshape(rows, groups * 4, 1).int() - 127)
    return v.reshape(rows, groups * 128)[:, :K]


def random_words(n, tensor, device):
    """Words 0 .. n - 1 of Philox4x32-10 at counter (i / 4, 0, tensor, STEP), key SEED."""
    low = 0xFFFFFFFF
    c0 = torch.arange((n + 3) // 4, device=device)
    c1, c2, c3 = torch.zeros_like(c0), torch.full_like(c0, tensor), torch.full_like(c0, STEP)
    k0, k1 = SEED & low, SEED >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64 bits; the upper half survives the sign
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), -1).reshape(-1)[:n]


def rounded(x, draw16):
    """x [n] to E4M3 under its blocks' scales, rounded by 16 random bits: element values and exponents."""
    b = x.reshape(-1, 32)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)
    X = e - 9 + (m > 0.875).to(e.dtype)
    X = torch.where(amax == 0, torch.full_like(X, -127), X.clamp(-127, 127))[:, None]
    a = torch.ldexp(b.abs(), -X)
    _, e = torch.frexp(a)
    ulp = (e - 1).clamp(min=-6) - 3
    steps = torch.ldexp(a, -ulp)
    low = steps.floor()
    up = draw16.reshape(-1, 32) < ((steps - low) * 65536).floor()
    return torch.ldexp(low + up, ulp).copysign(b), X


def plain_update(s):
    case = s["case"]
    eight = case["bits"] == 8
    f1, f2 = 1 - BETA1 ** STEP, 1 - BETA2 ** STEP
    g = s["g"].float() * SCALE
    p = s["p"]
    if eight:
        m = (s["m"][0].view(torch.float8_e4m3fn).float().reshape(-1, 32)
             * torch.ldexp(torch.ones_like(s["m"][1], dtype=torch.float32), s["m"][1].int() - 127).reshape(-1, 1)).reshape(-1)
        u = (s["v"][0].view(torch.float8_e4m3fn).float().reshape(-1, 32)
             * torch.ldexp(torch.ones_like(s["v"][1], dtype=torch.float32), s["v"][1].int() - 127).reshape(-1, 1)).reshape(-1)
        v = u * u
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    root = v.sqrt()
    p = p * (1 - LR * DECAY) - (LR / f1) * (m / (root / math.sqrt(f2) + ADAM_EPS))
    s["p"].copy_(p)
    if case["copy"]:
        s["copy"].copy_(p)
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return
    words = torch.cat([random_words((n + 127) // 128 * 128, i, p.device) for i, n in enumerate(s["sizes"])])
    for x, half, state in ((m, words & 0xFFFF, s["m"]), (root, words >> 16, s["v"])):
        q, X = rounded(x, half)
        state[0].copy_(q.to(torch.float8_e4m3fn).view(torch.uint8).reshape(state[0].shape))
        state[1].copy_((X + 127).to(torch.uint8).reshape(state[1].shape))


def update_outputs(s):
    out = {"p": s["p"], "copy": s["copy"]}
    if s["case"]["bits"] == 8:
        return {**out, "m": eight_bits(*s["m"]), "v": eight_bits(*s["v"])}
    return {**out, "m": s["m"], "v": s["v"]}


def plain(s):
    case = s["case"]
    op = case["op"]
    if op == "update":
        plain_update(s)
        return update_outputs(s)
    if op in ("norm", "norm backward"):
        x, gamma = s["x"].float(), s["gamma"].float()
        if op == "norm":
            mean = x.mean(1, keepdim=True)
            rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
            y = ((x - mean) * rstd) * gamma + s["beta"].float()
            out = {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
            if case["packed"]:
                out["row"] = eight_bits(*pack(y.bfloat16().float(), E4M3, None))
            return out
        mean, rstd, dy = s["mean"][:, None], s["rstd"][:, None], s["dy"].float()
        h, g = (x - mean) * rstd, dy * gamma
        dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        if case["residual"]:
            dx = dx + s["residual"].float()
        return dx.to(s["x"].dtype), (dy * h).sum(0), dy.sum(0)
    V, K, fmt = case["V"], case["K"], FORMATS[case["fmt"]]
    table = s["table"]
    l = unpacked(s["A"], K, fmt, table) @ unpacked(s["B"], K, fmt, table).t()
    labels = s["labels"]
    valid = (labels >= 0) & (labels < V)
    at = torch.where(valid, labels, torch.zeros_like(labels))[:, None]
    if op == "loss":
        top = l.amax(1, keepdim=True)
        lse = torch.log(torch.exp(l - top).sum(1)) + top[:, 0]
        return torch.where(valid, lse - l.gather(1, at)[:, 0], torch.zeros_like(lse)), lse
    rotate = s["rotation"] if fmt == E2M3 else None
    d = torch.exp(l - s["lse"][:, None])
    d = d.scatter_add(1, at, -torch.ones_like(s["lse"])[:, None])
    d = d * torch.where(valid, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    dr = torch.nn.functional.pad(d, (0, -V % 32))
    dX = values(dr, fmt, rotate) @ unpacked(s["Wc"], dr.shape[1], fmt, table).t()
    dp = pad_rows(d)
    dW = values(dp.t(), fmt, rotate) @ unpacked(s["Xc"], dp.shape[0], fmt, table).t()
    return dX.bfloat16(), dW.bfloat16()


def run(s):
    return framework(s) if own else plain(s)


# ------------------------------------------------------------------ the library's calls
def framework(s):
    from microscaling_block_scaled_mx_amd import mx

    case = s["case"]
    op = case["op"]
    if op == "norm":
        mx.layernorm_fwd(s["x"], s["y"], gamma=s["gamma"], beta=s["beta"], eps=EPS, mean=s["mean"], rstd=s["rstd"],
                         row=s["row"], fmt=mx.E4M3, scale_mode=mx.RCEIL)
        out = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        if case["packed"]:
            out["row"] = eight_bits(*s["row"])
        return out
    if op == "norm backward":
        mx.layernorm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], gamma=s["gamma"], residual=s["residual"],
                         dgamma=s["dgamma"], dbeta=s["dbeta"], partials=s["partials"])
        return s["dx"], s["dgamma"], s["dbeta"]
    if op == "update":
        mx.adamw(s["items"], lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY, step=STEP, seed=SEED,
                 grad_scale=s["scale"])
        return update_outputs(s)
    M, V, K, fmt = case["M"], case["V"], case["K"], FORMATS[case["fmt"]]
    if op == "loss":
        mx.head_loss(s["A"], s["B"], M, V, K, fmt, s["labels"], s["loss"], s["lse"], s["work"])
        return s["loss"], s["lse"]
    mx.head_loss_bwd(s["A"], s["B"], s["Wc"], s["Xc"], M, V, K, fmt, mx.RCEIL if fmt == E4M3 else mx.FLOOR, s["labels"],
                     s["lse"], s["dloss"], dX=s["dX"], dW=s["dW"], Gr=s["Gr"], Gc=s["Gc"], piece=PIECE, sums=s["sums"],
                     hadamard=fmt == E2M3)
    return s["dX"], s["dW"]


# ------------------------------------------------------------------ the definition in 64 bits
def stands_for(operand, K, fmt):
    """The values of a packed operand from the bits of its codes, float64."""
    codes, scales = operand[0].permute(1, 0, 2), operand[1].permute(1, 0, 2)
    rows, groups, nbytes = codes.shape
    byte = codes.reshape(rows, groups, nbytes).int()
    k = torch.arange(128, device=byte.device)
    blk, e = k // 32, k % 32
    if fmt == E2M3:
        # element e of a block begins at bit 6 e of the block's 24 bytes: bytes 0-15 at 16 blk, bytes 16-23 at 64 + 8 (blk ^ swap)
        swap = ((torch.arange(rows, device=byte.device) >> 4) & 1)[:, None]

        def at(j):
            return torch.where(j < 16, 16 * blk + j, 64 + 8 * (blk ^ swap) + j - 16)

        first = (6 * e) // 8
        lo = torch.gather(byte, 2, at(first).expand(rows, 128)[:, None, :].expand(rows, groups, 128))
        hi = torch.gather(byte, 2, at((first + 1).clamp(max=23)).expand(rows, 128)[:, None, :].expand(rows, groups, 128))
        c = ((lo | (hi << 8)) >> ((6 * e) % 8)) & 63
    elif fmt == E2M1:
        c = (byte[..., k // 2] >> (4 * (k % 2))) & 15
    else:
        c = byte
    m_bits, e_bits, bias = {E2M1: (1, 2, 1), E2M3: (3, 2, 1), E4M3: (3, 4, 7)}[fmt]
    man, ex = (c & (2 ** m_bits - 1)).double() / 2 ** m_bits, (c >> m_bits) & (2 ** e_bits - 1)
    v = torch.where(ex == 0, man, man + 1) * torch.exp2((ex.clamp(min=1) - bias).double())
    v = torch.where((c >> (m_bits + e_bits)) == 1, -v, v)
    v = v.reshape(rows, groups, 4, 32) * torch.exp2(scales.double() - 127)[..., None]
    return v.reshape(rows, groups * 128)[:, :K]


def nearest(v, m_bits, least, top):
    """v rounded to m_bits after the leading one (spacing fixed below 2^least), ties to even, at most top."""
    ex = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** least))).clamp(min=least)
    ulp = torch.exp2(ex - m_bits)
    return (torch.round(v / ulp) * ulp).clamp(-top, top)


def block_exponents(b, fmt):
    """X of blocks b [..., 32], float64 [..., 1]."""
    amax = b.abs().amax(-1, keepdim=True)
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    E = torch.floor(torch.log2(safe))
    E = E + (safe >= torch.exp2(E + 1)) - (safe < torch.exp2(E)).double()
    X = torch.where(448 * torch.exp2(E - 8) >= safe, E - 8, E - 7) if fmt == E4M3 else E - 2
    return torch.where(amax > 0, X.clamp(-127, 127), torch.full_like(X, -127))


def quantised(x, fmt, rotate):
    """x [rows][K] float64 -> the values of its packed form, float64."""
    b = x.reshape(x.shape[0], -1, 32)
    if rotate:
        b = b @ rotation(torch.float64)
    m_bits, least, top = {E2M1: (1, 0, 6.0), E2M3: (3, 0, 7.5), E4M3: (3, -6, 448.0)}[fmt]
    scale = torch.exp2(block_exponents(b, fmt))
    return (nearest(b / scale, m_bits, least, top) * scale).reshape(x.shape)


def grouped(v, rows, width):
    """[rows][groups * width] -> [groups][rows][width]."""
    return v.reshape(rows, -1, width).transpose(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "update":
        return exact_update(s)
    if op in ("norm", "norm backward"):
        M, C = case["M"], case["C"]
        x, gamma = s["x"].double(), s["gamma"].double()
        if op == "norm":
            var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
            h = (x - mean) / torch.sqrt(var + EPS)
            y = torch.addcmul(s["beta"].double(), h, gamma)
            out = {"y": y, "mean": mean[:, 0], "rstd": (var + EPS).pow(-0.5)[:, 0]}
            if case["packed"]:
                pad = -C % 128
                b = torch.nn.functional.pad(nearest(y, 7, -126, math.inf), (0, pad)).reshape(M, -1, 32)
                scale = torch.exp2(block_exponents(b, E4M3))
                out["row"] = {"elements": grouped(nearest(b / scale, 3, -6, 448.0).reshape(M, -1), M, 128),
                              "scales": grouped(scale.reshape(M, -1), M, 4)}
            return out
        mean, rstd, dy = s["mean"].double()[:, None], s["rstd"].double()[:, None], s["dy"].double()
        h = (x - mean) * rstd
        g = dy * gamma
        dx = (g - (g.sum(1, keepdim=True) + h * (g * h).sum(1, keepdim=True)) / C) * rstd
        if case["residual"]:
            dx += s["residual"].double()
        return dx, (dy * h).sum(0), dy.sum(0)
    M, V, K, fmt = case["M"], case["V"], case["K"], FORMATS[case["fmt"]]
    l = stands_for(s["A"], K, fmt) @ stands_for(s["B"], K, fmt).t()
    labels = s["labels"]
    counts = (labels >= 0).double()
    if op == "loss":
        lse = torch.logsumexp(l, 1)
        return (lse - l[torch.arange(M, device="cuda"), labels.clamp(min=0)]) * counts, lse
    rotate = fmt == E2M3
    l.sub_(s["lse"].double()[:, None]).exp_()
    l[torch.arange(M, device="cuda"), labels.clamp(min=0)] -= 1
    l.mul_((s["dloss"].double() * counts)[:, None])
    Vp = (V + 31) // 32 * 32
    dX = quantised(torch.nn.functional.pad(l, (0, Vp - V)), fmt, rotate) @ stands_for(s["Wc"], Vp, fmt).t()
    l = pad_rows(l)
    return dX, quantised(l.t().contiguous(), fmt, rotate) @ stands_for(s["Xc"], l.shape[0], fmt).t()


def exact_update(s):
    case = s["case"]
    g = s["g"].double() * SCALE
    if case["bits"] == 8:
        total = g.numel()
        m, v = stands_for(s["m"], total, E4M3)[0], stands_for(s["v"], total, E4M3)[0].square()
    else:
        m, v = s["m"].double(), s["v"].double()
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g * g - v)
    p = s["p"].double()
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** STEP)) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + ADAM_EPS)
    out = {"p": p, "copy": p if case["copy"] else None}
    if case["bits"] == 32:
        return {**out, "m": m, "v": v}
    # the words once more, by halves of 16 bits so that no product leaves 53
    words = torch.cat([exact_words((n + 127) // 128 * 128, i) for i, n in enumerate(s["sizes"])])
    return {**out, "m": exact_rounded(m, words % 65536, s["m"]), "v": exact_rounded(v.sqrt(), words // 65536, s["v"])}


def exact_words(n, tensor):
    c = [torch.arange(n // 4, device="cuda"), 0, tensor, STEP]
    key = [SEED % 2 ** 32, SEED // 2 ** 32]

    def product(a, x):
        lo, hi = a % 65536 * x, a // 65536 * x  # below 2^48 each
        low = lo + hi % 65536 * 65536
        return hi // 65536 + low // 2 ** 32, low % 2 ** 32

    for i in range(10):
        (h0, l0), (h1, l1) = product(0xD2511F53, c[0]), product(0xCD9E8D57, c[2])
        k0, k1 = (key[0] + i * 0x9E3779B9) % 2 ** 32, (key[1] + i * 0xBB67AE85) % 2 ** 32
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
    full = torch.zeros(n // 4, dtype=torch.int64, device="cuda")
    return torch.stack([full + x for x in c], 1).reshape(n)


def exact_rounded(x, draw16, like):
    """Elements and scales of x rounded to E4M3 by 16 random bits, float64, laid out as `like`."""
    b = x.reshape(-1, 32)
    scale = torch.exp2(block_exponents(b, E4M3))
    a = b.abs() / scale
    ulp = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    share = torch.floor(a / ulp % 1 * 65536)
    q = (torch.floor(a / ulp) + (draw16.reshape(-1, 32) < share)) * ulp * torch.sign(b)
    return {"elements": q.reshape(like[0].shape), "scales": scale.reshape(like[1].shape)}
