"""The linear operators (mx_gemm_act, mx_checkpoint_save / _load,
mx_quantize_saved, mx_linear_bwd_saved) against plain implementations in 64
bits, and their refusals.

Tolerances.  A rounding is off by at most half a step: bf16 2^-8, E4M3 2^-4
relative.  A GEMM's sums follow the library's bar for scaled matrix-core
accumulation, 2e-3 of the largest result (parity_checks.REL), except where
every partial sum is exact in binary32: there outputs must be equal.  The
activations take the hardware's exp2 and reciprocal (1 ulp each): z is formed
with 3 roundings, so s carries a relative error of at most (3 |z| + 4) 2^-24,
and x s as much plus one rounding; |z| <= 24 is allowed for (past that s is 1
or the value is below 1e-9 of x): 2^-24 (3*24 + 6) < 2^-17."""
import ctypes

import numpy as np
import pytest
import torch

from microscaling_block_scaled_mx_amd import mx
from packed_layout import blocked, tiled, unblocked, untiled
from parity_checks import REL

gpu = pytest.mark.gpu
FMTS = [(mx.E2M1, mx.FLOOR, False), (mx.E2M3, mx.FLOOR, True), (mx.E4M3, mx.RCEIL, False)]
ACTS = [mx.ACT_NONE, mx.ACT_GELU_TANH, mx.ACT_SILU]
ACT_REL = 2.0 ** -17
K0, K1 = np.sqrt(2 / np.pi), 0.044715


# ---------------------------------------------------------------- plain forms, 64 bits
def sigmoid(z):
    return 1 / (1 + np.exp(-np.clip(z, -700, 700)))


def act64(p, act):
    if act == mx.ACT_GELU_TANH:
        return p * sigmoid(2 * K0 * (p + K1 * p ** 3))
    return p * sigmoid(p) if act == mx.ACT_SILU else p.copy()


def slope64(p, act):
    if act == mx.ACT_GELU_TANH:
        s = sigmoid(2 * K0 * (p + K1 * p ** 3))
        return s + p * s * (1 - s) * 2 * K0 * (1 + 3 * K1 * p * p)
    if act == mx.ACT_SILU:
        s = sigmoid(p)
        return s + p * s * (1 - s)
    return np.ones_like(p)


def code_values(fmt):
    e_bits, m_bits, bias = {mx.E2M1: (2, 1, 1), mx.E2M3: (2, 3, 1), mx.E4M3: (4, 3, 7)}[fmt]
    c = np.arange(1 << (1 + e_bits + m_bits))
    m, e = c & ((1 << m_bits) - 1), (c >> m_bits) & ((1 << e_bits) - 1)
    v = np.where(e == 0, m / 2.0 ** m_bits, 1 + m / 2.0 ** m_bits) * 2.0 ** (np.maximum(e, 1) - bias)
    v = np.where(c >> (e_bits + m_bits), -v, v)
    if fmt == mx.E4M3:
        v[[0x7F, 0xFF]] = np.nan
    return v


def codes_of(plain, K, fmt):
    """Element codes [rows][K] of plain packed bytes [rows][K*bits/8]."""
    bits = np.unpackbits(plain, axis=1, bitorder="little")[:, :K * mx.BITS[fmt]]
    bits = bits.reshape(plain.shape[0], K, mx.BITS[fmt]).astype(np.int64)
    return (bits << np.arange(mx.BITS[fmt])).sum(-1)


def decode(p, rows, K, fmt):
    """Values [rows][K] of a packed operand (device tensors), float64; K a multiple of 32."""
    codes = untiled(p[0].cpu().numpy(), K, mx.BITS[fmt])
    scales = unblocked(p[1].cpu().numpy(), K // 32).astype(np.float64)
    v = code_values(fmt)[codes_of(codes, K, fmt)].reshape(rows, K // 32, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        out = v * np.where(scales == 255, np.nan, 2.0 ** (scales - 127))[..., None]
    return out.reshape(rows, K)


def quantised64(x, fmt, mode, had):
    """The values [rows][K] float64 that packing stands for, and its exponents (no NaN, no clamping range)."""
    b = x.reshape(x.shape[0], -1, 32)
    if had:
        i = np.arange(32)
        odd = np.array([[bin(a & c).count("1") & 1 for c in i] for a in i])
        b = b @ ((1 - 2.0 * odd) / np.sqrt(32))
    amax = np.abs(b).max(-1)
    m, e = np.frexp(amax)
    X = (e - 9 + (m > 0.875)) if mode == mx.RCEIL else e - 1 - {mx.E2M1: 2, mx.E2M3: 2, mx.E4M3: 8}[fmt]
    X = np.where(amax == 0, -127, np.clip(X, -127, 127))
    mb, least, top = {mx.E2M1: (1, 0, 6.0), mx.E2M3: (3, 0, 7.5), mx.E4M3: (3, -6, 448.0)}[fmt]
    v = np.ldexp(b, -X[..., None])
    _, ev = np.frexp(np.abs(v))
    ulp = 2.0 ** (np.maximum(ev - 1, least) - mb)
    q = np.clip(np.rint(v / ulp) * ulp, -top, top)
    return np.ldexp(q, X[..., None]).reshape(x.shape), X


def bf16_round(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


def dev_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().cuda()


def f64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def operand(rng, rows, K, fmt, mode, had, std=1.0):
    """A packed operand of random values and what it stands for."""
    x = torch.from_numpy(rng.standard_normal((rows, K)).astype(np.float32) * np.float32(std)).bfloat16().cuda()
    p = mx.alloc_packed(rows, K, fmt)
    mx.quantize_saved(rows, K, fmt, mode, had, x=x, row=p)
    return p, decode(p, rows, K, fmt)


def exact_operand(rng, rows, K, fmt):
    """Small integers under one scale of 1: every sum of products is exact in binary32 (K * 16 < 2^24)."""
    v = rng.integers(-4, 5, (rows, K)).astype(np.float64)
    values = code_values(fmt)
    table = {float(x): c for c, x in reversed(list(enumerate(values))) if np.isfinite(x)}
    codes = np.vectorize(lambda x: table[float(x)])(v)
    bits = ((codes[..., None] >> np.arange(mx.BITS[fmt])) & 1).astype(np.uint8).reshape(rows, -1)
    plain = np.packbits(bits, axis=1, bitorder="little")
    scales = np.full((rows, K // 32), 127, np.uint8)
    return (torch.from_numpy(tiled(plain, mx.BITS[fmt])).cuda(), torch.from_numpy(blocked(scales)).cuda()), v


@pytest.fixture(scope="module", autouse=True)
def need_device(request):
    if torch.cuda.is_available():
        assert mx.device_supported(0)


# ---------------------------------------------------------------- refusals (no GPU call)
P = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(16)]
NULL, SHAPE, ALIGN, FORMAT, OVERFLOW, DEVICE = 1, 2, 3, 4, 6, 7
NONE = mx.Packed(None, None)


def pk(i):
    return mx.Packed(P[i], P[i + 1])


def gemm_args(**kw):
    a = dict(M=5, N=64, K=96, fmt=mx.E2M3, act=0, A=pk(0), B=pk(2), bias=P[4], residual=P[5], C=P[6], ldr=64, ldc=64,
             bias_dtype=0, c_dtype=0, saved=pk(7))
    a.update(kw)
    return mx.GemmActArgs(*[a[f] for f, _ in mx.GemmActArgs._fields_])


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=0), FORMAT), (dict(fmt=4), FORMAT), (dict(act=3), FORMAT), (dict(act=-1), FORMAT),
    (dict(c_dtype=2), FORMAT), (dict(bias_dtype=-1), FORMAT),
    (dict(M=-1), SHAPE), (dict(N=48), SHAPE), (dict(K=100), SHAPE), (dict(N=-32), SHAPE), (dict(K=-32), SHAPE),
    (dict(ldc=56), SHAPE), (dict(ldc=68), SHAPE), (dict(ldr=32), SHAPE), (dict(ldr=65), SHAPE),
    (dict(residual=P[6], ldr=72), SHAPE),
    (dict(A=NONE), NULL), (dict(B=mx.Packed(P[2], None)), NULL), (dict(C=None), NULL), (dict(C=None, residual=None, saved=NONE), NULL),
    (dict(saved=mx.Packed(P[7], None)), NULL), (dict(saved=mx.Packed(None, P[7])), NULL),
    (dict(C=ctypes.c_void_p(0x1008)), ALIGN), (dict(bias=ctypes.c_void_p(0x1002)), ALIGN),
    (dict(saved=mx.Packed(ctypes.c_void_p(0x1001), P[1])), ALIGN),
    (dict(M=1 << 31), OVERFLOW), (dict(M=1 << 25, K=4096), OVERFLOW), (dict(N=1 << 25, K=4096, ldc=1 << 25, ldr=1 << 25), OVERFLOW),
    (dict(M=1 << 50), OVERFLOW), (dict(ldc=1 << 60), OVERFLOW), (dict(ldr=1 << 60), OVERFLOW), (dict(M=1 << 20, N=1 << 20, K=32, ldc=1 << 20, ldr=1 << 20), OVERFLOW),
])
def test_gemm_act_refusals(kw, want):
    assert mx.lib().mx_gemm_act(ctypes.byref(gemm_args(**kw)), None) == want


def test_gemm_act_empty_products_need_no_pointers():
    want = 0 if torch.cuda.is_available() else DEVICE
    for kw in (dict(M=0), dict(N=0, ldc=0, ldr=0)):
        a = gemm_args(A=NONE, B=NONE, C=None, residual=None, saved=NONE, bias=None, **kw)
        assert mx.lib().mx_gemm_act(ctypes.byref(a), None) == want
    assert mx.lib().mx_gemm_act(None, None) == NULL


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), FORMAT), (dict(R=-1), SHAPE), (dict(C=40), SHAPE), (dict(ld=32), SHAPE), (dict(ld=68), SHAPE),
    (dict(x=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(x=ctypes.c_void_p(0x1004)), ALIGN),
    (dict(scales=ctypes.c_void_p(0x1004)), ALIGN), (dict(R=1 << 41), OVERFLOW),
    (dict(R=1 << 39), OVERFLOW),
])
def test_checkpoint_refusals(kw, want):
    a = dict(x=P[0], dtype=0, R=3, C=64, ld=64, codes=P[1], scales=P[2])
    a.update(kw)
    L = mx.lib()
    assert L.mx_checkpoint_save(a["x"], a["dtype"], a["R"], a["C"], a["ld"], a["codes"], a["scales"], None) == want
    assert L.mx_checkpoint_load(a["codes"], a["scales"], a["R"], a["C"], a["x"], a["dtype"], a["ld"], None) == want


def saved_args(**kw):
    a = dict(R=5, C=64, fmt=mx.E2M3, scale_mode=0, hadamard=1, act=1, x=P[0], ldx=64, saved=pk(1), row=pk(3), col=pk(5),
             colsum_partials=P[7], colsum=P[8])
    a.update(kw)
    return mx.QuantizeSavedArgs(*[a[f] for f, _ in mx.QuantizeSavedArgs._fields_])


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=9), FORMAT), (dict(scale_mode=1), FORMAT), (dict(fmt=mx.E2M1), FORMAT), (dict(act=3), FORMAT),
    (dict(act=0), FORMAT),                      # x with no activation takes no checkpoint
    (dict(saved=NONE), NULL), (dict(x=None, act=0, saved=NONE), NULL), (dict(saved=mx.Packed(P[1], None)), NULL),
    (dict(row=mx.Packed(None, P[1])), NULL), (dict(col=mx.Packed(P[1], None)), NULL),
    (dict(row=NONE, col=NONE, colsum_partials=None, colsum=None), NULL), (dict(colsum_partials=None), NULL),
    (dict(R=-1), SHAPE), (dict(C=65), SHAPE), (dict(ldx=32), SHAPE), (dict(ldx=100), SHAPE),
    (dict(x=ctypes.c_void_p(0x1002)), ALIGN), (dict(colsum=ctypes.c_void_p(0x1004)), ALIGN), (dict(R=1 << 41), OVERFLOW),
])
def test_quantize_saved_refusals(kw, want):
    assert mx.lib().mx_quantize_saved(ctypes.byref(saved_args(**kw)), None) == want


def bwd_args(**kw):
    a = dict(M=5, N=64, K=96, fmt=mx.E4M3, scale_mode=1, hadamard=0, act=1, x_act=0, accumulate=0, dY=P[0], lddy=64,
             saved_pre=pk(1), saved_x=pk(3), Wc=pk(5), dX=P[7], lddx=96, dW=P[8], lddw=96, dw_dtype=1, reserved=0,
             db=P[9], db_partials=P[10], dPr=pk(11), dPc=pk(12), Xc=pk(13))
    a.update(kw)
    return mx.LinearBwdArgs(*[a[f] for f, _ in mx.LinearBwdArgs._fields_])


@pytest.mark.parametrize("kw,want", [
    (dict(accumulate=2), FORMAT), (dict(act=5), FORMAT), (dict(x_act=-1), FORMAT), (dict(act=0), FORMAT),
    (dict(dw_dtype=3), FORMAT), (dict(hadamard=1), FORMAT),
    (dict(M=-2), SHAPE), (dict(N=33), SHAPE), (dict(K=31), SHAPE), (dict(lddy=32), SHAPE), (dict(lddx=64), SHAPE),
    (dict(lddw=97), SHAPE),
    (dict(dY=None), NULL), (dict(saved_pre=NONE), NULL), (dict(saved_x=NONE), NULL), (dict(Wc=NONE), NULL),
    (dict(dPr=NONE), NULL), (dict(dPc=NONE), NULL), (dict(Xc=NONE), NULL), (dict(db_partials=None), NULL),
    (dict(dX=None, dW=None, db=None), NULL),
    (dict(dW=ctypes.c_void_p(0x1008)), ALIGN), (dict(dY=ctypes.c_void_p(0x1008)), ALIGN),
    (dict(M=1 << 30), OVERFLOW),
])
def test_linear_bwd_refusals(kw, want):
    assert mx.lib().mx_linear_bwd_saved(ctypes.byref(bwd_args(**kw)), None) == want


def test_binding_refuses_what_the_kernels_would_misread():
    x = torch.zeros(4, 64)
    p = (torch.zeros(1, 4, 128, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8))
    with pytest.raises(mx.MXError, match="not on a GPU"):
        mx.checkpoint_save(x, p)
    with pytest.raises(mx.MXError, match="neither float32 nor bf16"):
        mx.checkpoint_save(x.half(), p)
    with pytest.raises(mx.MXError, match="dense rows"):
        mx.checkpoint_save(torch.zeros(64, 4).t(), p)
    with pytest.raises(mx.MXError, match="does not hold"):
        mx.quantize_saved(5, 64, mx.E4M3, mx.RCEIL, x=x.bfloat16(), row=p)


# ---------------------------------------------------------------- checkpoints
def special_rows(rng, R, C):
    x = rng.standard_normal((R, C)).astype(np.float32) * np.exp2(rng.integers(-20, 20, (R, 1))).astype(np.float32)
    t = torch.from_numpy(x).bfloat16()
    u = t.view(torch.int16)
    u[0, 0:32] = 0
    if R > 1:
        u[1, 3] = 0x7FC0                                   # NaN
        u[1 % R, 40 % C] = -128                            # -Inf (0xff80)
    if R > 2:
        u[2, :32] = torch.arange(32, dtype=torch.int16)    # zero and subnormals
        u[2, 32 % C] = 0x7F7F                              # the largest finite
        u[2, 1] = -32768                                   # -0
    return t


@gpu
@pytest.mark.parametrize("R,C", [(1, 32), (1, 4096), (3, 96), (17, 160), (64, 128), (65, 2080), (200, 1024)])
def test_checkpoint_save_is_the_mxfp8_rowwise_pack(orc, R, C):
    rng = np.random.default_rng(R * 1000 + C)
    t = special_rows(rng, R, C)
    p = mx.alloc_packed(R, C, mx.E4M3)
    for b in p:
        b.fill_(0xA5)
    mx.checkpoint_save(t.cuda(), p)
    pad = torch.zeros((R + 31) // 32 * 32, C, dtype=torch.bfloat16)
    pad[:R] = t
    want = orc.quantize(pad.view(torch.int16).numpy().view(np.uint16), pad.shape[0], C, mx.E4M3, mx.RCEIL)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(p[0].cpu().numpy(), tiled(want["row_codes"][:R], 8))
    np.testing.assert_array_equal(p[1].cpu().numpy(), blocked(want["row_scales"][:R]))
    # and back: the value of every code, bf16 and binary32
    ref = decode(p, R, C, mx.E4M3)
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.empty(R, C, dtype=dtype, device="cuda")
        mx.checkpoint_load(p, y)
        got = f64(y)
        want_y = torch.from_numpy(ref).to(dtype).double().numpy()
        np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
        np.testing.assert_array_equal(got[~np.isnan(ref)], want_y[~np.isnan(ref)])


@gpu
@pytest.mark.parametrize("R,C", [(1, 64), (7, 224), (130, 512)])
def test_checkpoint_of_binary32(R, C):
    rng = np.random.default_rng(R + C)
    x = (rng.standard_normal((R, C)) * np.exp2(rng.integers(-30, 30, (R, 1)))).astype(np.float32)
    x[0, :32] = 448 * np.float32(2.0 ** -5) * np.linspace(0, 1, 32, dtype=np.float32)  # the block's top on the grid's top
    p = mx.alloc_packed(R, C, mx.E4M3)
    mx.checkpoint_save(torch.from_numpy(x).cuda(), p)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(decode(p, R, C, mx.E4M3), quantised64(x.astype(np.float64), mx.E4M3, mx.RCEIL, False)[0])


@gpu
def test_checkpoint_of_a_column_slice_leaves_its_neighbours():
    rng = np.random.default_rng(5)
    wide = torch.from_numpy(rng.standard_normal((37, 320)).astype(np.float32)).bfloat16().cuda()
    x = wide[:, 64:64 + 160]
    p, q = mx.alloc_packed(37, 160, mx.E4M3), mx.alloc_packed(37, 160, mx.E4M3)
    mx.checkpoint_save(x, p)
    mx.checkpoint_save(x.contiguous(), q)
    torch.cuda.synchronize()
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
    out = torch.full((37, 320), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.checkpoint_load(p, out[:, 64:64 + 160])
    y = torch.empty(37, 160, dtype=torch.bfloat16, device="cuda")
    mx.checkpoint_load(p, y)
    torch.cuda.synchronize()
    assert torch.equal(out[:, 64:224], y)
    assert (out[:, :64] == 7).all() and (out[:, 224:] == 7).all()


# ---------------------------------------------------------------- GEMM
SIZES = [(1, 32, 32), (1, 2080, 160), (5, 96, 128), (16, 64, 2048), (17, 64, 96), (32, 160, 384), (33, 32, 1056),
         (3, 8224, 160), (29, 8224, 416), (64, 288, 256), (65, 64, 32), (100, 352, 800), (130, 2080, 416), (257, 4096, 96),
         (200, 4128, 640), (300, 8224, 64), (2039, 8160, 96), (4100, 4128, 160), (4090, 8160, 64)]


@gpu
@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E2M3, mx.E4M3])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm_act_exact_products(M, N, K, fmt):
    """Integers: bias, residual and sums are exact, so C is, and its checkpoint is the checkpoint of C."""
    rng = np.random.default_rng(M * 7 + N + K + fmt)
    A, a = exact_operand(rng, M, K, fmt)
    B, b = exact_operand(rng, N, K, fmt)
    bias = rng.integers(-8, 9, N).astype(np.float32)
    res = torch.from_numpy(rng.integers(-100, 101, (M, N)).astype(np.float32)).cuda()
    pre = torch.from_numpy(a).cuda() @ torch.from_numpy(b).cuda().t() + torch.from_numpy(bias).cuda().double()
    for dtype in (torch.float32, torch.bfloat16):
        ld = N + 24
        wide = torch.full((M, ld), 3.0, dtype=dtype, device="cuda")
        saved = mx.alloc_packed(M, N, mx.E4M3)
        for s in saved:
            s.fill_(0x5A)
        r = res.to(dtype)
        mx.gemm_act(A, B, M, N, K, fmt, wide[:, :N], bias=torch.from_numpy(bias).to(dtype).cuda(), residual=r, saved=saved)
        torch.cuda.synchronize()
        assert torch.equal(wide[:, :N].double(), (pre + r.double()).to(dtype).double())
        assert (wide[:, N:] == 3).all()
        want = mx.alloc_packed(M, N, mx.E4M3)
        mx.checkpoint_save(pre.float(), want)
        torch.cuda.synchronize()
        assert torch.equal(saved[0], want[0]) and torch.equal(saved[1], want[1])
        # the checkpoint alone, and the product alone
        only = mx.alloc_packed(M, N, mx.E4M3)
        mx.gemm_act(A, B, M, N, K, fmt, bias=torch.from_numpy(bias).cuda(), saved=only)
        c = torch.empty(M, N, dtype=dtype, device="cuda")
        mx.gemm_act(A, B, M, N, K, fmt, c)
        torch.cuda.synchronize()
        assert torch.equal(only[0], want[0]) and torch.equal(only[1], want[1])
        assert torch.equal(c.double(), (pre - torch.from_numpy(bias).cuda().double()).to(dtype).double())


@gpu
@pytest.mark.parametrize("fmt,mode,had", FMTS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 96, 4096), (24, 256, 512), (77, 160, 224), (1500, 4096, 320)])
def test_gemm_act_against_64_bits(M, N, K, act, fmt, mode, had):
    rng = np.random.default_rng(M + N + K + act)
    A, a = operand(rng, M, K, fmt, mode, had)
    B, b = operand(rng, N, K, fmt, mode, had, std=2.0 / np.sqrt(K))
    bias = dev_bf16(rng.standard_normal(N))
    res = dev_bf16(rng.standard_normal((M, N)))
    pre = a @ b.T + f64(bias)
    want = act64(pre, act) + f64(res)
    c = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    saved = mx.alloc_packed(M, N, mx.E4M3)
    mx.gemm_act(A, B, M, N, K, fmt, c, act=act, bias=bias, residual=res, saved=saved)
    # |act'| <= 1.13; the sum's error, the activation's, then one rounding to bf16
    sums = REL * np.abs(a @ b.T).max()
    err = 1.13 * sums + ACT_REL * np.abs(pre) + 2.0 ** -8 * (np.abs(want) + sums)
    assert (np.abs(f64(c) - want) <= err).all()
    # the checkpoint: half an E4M3 step of each value (or of the least step under the block's scale)
    q = decode(saved, M, N, mx.E4M3)
    top = np.abs(pre).reshape(M, -1, 32).max(-1, keepdims=True).repeat(32, -1).reshape(M, N)
    assert (np.abs(q - pre) <= sums + 2.0 ** -4 * (np.abs(pre) + sums) + 2.0 ** -17 * top).all()
    # without an output the checkpoint is the same
    only = mx.alloc_packed(M, N, mx.E4M3)
    mx.gemm_act(A, B, M, N, K, fmt, act=act, bias=bias, saved=only)
    torch.cuda.synchronize()
    assert torch.equal(only[0], saved[0]) and torch.equal(only[1], saved[1])


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_activation_values_over_their_range(act):
    """K = 0: C = act(bias) in binary32, so the epilogue's activation is seen alone, in both kernels."""
    N = 4096
    x = np.concatenate([np.linspace(-30, 30, N - 8), [0.0, -0.0, 1e-30, -1e-30, 1e4, -1e4, 3e38, -3e38]]).astype(np.float32)
    for M in (1, 600 * 16):
        c = torch.empty(M, N, device="cuda")
        mx.gemm_act(None, None, M, N, 0, mx.E4M3, c, act=act, bias=torch.from_numpy(x).cuda())
        got = f64(c[0]), f64(c[-1])
        want = act64(x.astype(np.float64), act)
        for g in got:
            assert (np.abs(g - want) <= ACT_REL * np.abs(want) + 2.0 ** -24 * np.abs(x) * (np.abs(x) < 1e4) + 1e-37).all()


@gpu
def test_gemm_act_zero_lengths_and_nan_blocks():
    c = torch.full((3, 64), 9.0, device="cuda")
    mx.gemm_act(None, None, 3, 64, 0, mx.E2M1, c)                       # an empty sum
    torch.cuda.synchronize()
    assert (c == 0).all()
    mx.gemm_act(None, None, 0, 64, 32, mx.E2M1, c[:0])                  # no rows
    rng = np.random.default_rng(3)
    for M in (20, 1100):
        x = rng.standard_normal((M, 256)).astype(np.float32)
        x[M // 2, 70] = np.nan
        A, B = mx.alloc_packed(M, 256, mx.E4M3), mx.alloc_packed(8192, 256, mx.E4M3)
        mx.checkpoint_save(torch.from_numpy(x).cuda(), A)
        mx.checkpoint_save(torch.from_numpy(rng.standard_normal((8192, 256)).astype(np.float32)).cuda(), B)
        c = torch.empty(M, 8192, device="cuda")
        saved = mx.alloc_packed(M, 8192, mx.E4M3)
        mx.gemm_act(A, B, M, 8192, 256, mx.E4M3, c, act=mx.ACT_GELU_TANH, saved=saved)
        back = torch.empty(M, 8192, device="cuda")
        mx.checkpoint_load(saved, back)
        torch.cuda.synchronize()
        bad = torch.arange(M, device="cuda") == M // 2
        for t in (c, back):
            assert torch.isnan(t[bad]).all() and torch.isfinite(t[~bad]).all()


@gpu
@pytest.mark.parametrize("M,N,K", [(40, 96, 128), (700, 8192, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm_act_accumulates_into_its_output(M, N, K, dtype):
    rng = np.random.default_rng(M)
    A, a = exact_operand(rng, M, K, mx.E2M1)
    B, b = exact_operand(rng, N, K, mx.E2M1)
    old = torch.from_numpy(rng.integers(-50, 50, (M, N)).astype(np.float32)).to(dtype).cuda()
    c = old.clone()
    mx.gemm_act(A, B, M, N, K, mx.E2M1, c, residual=c)
    torch.cuda.synchronize()
    want = torch.from_numpy(a @ b.T).cuda() + old.double()
    assert torch.equal(c.double(), want.to(dtype).double())


# ---------------------------------------------------------------- packs from checkpoints
@gpu
@pytest.mark.parametrize("fmt,mode,had", FMTS + [(mx.E2M3, mx.FLOOR, False), (mx.E4M3, mx.FLOOR, False)])
@pytest.mark.parametrize("R,C", [(1, 32), (31, 96), (33, 160), (128, 128), (129, 320), (300, 2080)])
def test_packs_without_activation_are_the_packers(orc, R, C, fmt, mode, had):
    """bf16 rows, and a checkpoint's values, packed as mx_quantize packs the same rows followed by zeros."""
    rng = np.random.default_rng(R + C + fmt)
    t = special_rows(rng, R, C)
    ck = mx.alloc_packed(R, C, mx.E4M3)
    mx.checkpoint_save(t.cuda(), ck)
    back = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    mx.checkpoint_load(ck, back)
    Rp = (R + 31) // 32 * 32
    for src, kw in ((t, dict(x=t.cuda())), (back.cpu(), dict(saved=ck))):
        pad = torch.zeros(Rp, C, dtype=torch.bfloat16)
        pad[:R] = src
        want = orc.quantize(pad.view(torch.int16).numpy().view(np.uint16), Rp, C, fmt, mode, had, col=True)
        row, col = mx.alloc_packed(R, C, fmt), mx.alloc_packed(C, Rp, fmt)
        for b in row + col:
            b.fill_(0x77)
        mx.quantize_saved(R, C, fmt, mode, had, row=row, col=col, **kw)
        torch.cuda.synchronize()
        bits = mx.BITS[fmt]
        np.testing.assert_array_equal(row[0].cpu().numpy(), tiled(want["row_codes"], bits)[:, :R])
        np.testing.assert_array_equal(row[1].cpu().numpy(), blocked(want["row_scales"])[:, :R])
        np.testing.assert_array_equal(col[0].cpu().numpy(), tiled(want["col_codes"], bits))
        np.testing.assert_array_equal(col[1].cpu().numpy(), blocked(want["col_scales"]))


@gpu
@pytest.mark.parametrize("act,grad", [(a, g) for a in ACTS for g in (False, True) if a or not g])  # (x alone: above)
@pytest.mark.parametrize("R,C", [(1, 64), (45, 96), (100, 96), (260, 352)])
def test_packs_with_activation_against_64_bits(R, C, grad, act):
    rng = np.random.default_rng(R * 3 + C + act)
    ck = mx.alloc_packed(R, C, mx.E4M3)
    mx.checkpoint_save(dev_bf16(rng.standard_normal((R, C)) * 3), ck)
    s = decode(ck, R, C, mx.E4M3)
    x = dev_bf16(rng.standard_normal((R, C))) if grad else None
    v = f64(x) * slope64(s, act) if grad else act64(s, act)
    Rp = (R + 31) // 32 * 32
    row, col = mx.alloc_packed(R, C, mx.E4M3), mx.alloc_packed(C, Rp, mx.E4M3)
    part = torch.empty((R + 127) // 128, C, device="cuda")
    total = torch.empty(C, device="cuda")
    mx.quantize_saved(R, C, mx.E4M3, mx.RCEIL, act=act, x=x, saved=ck, row=row, col=col, colsum_partials=part, colsum=total)
    # the slope is s + x z' s (1 - s): each factor to ACT_REL, |x z' s (1 - s)| <= 1.13
    dv = ACT_REL * (1.2 * np.abs(f64(x)) * 2 if grad else np.abs(v)) + 2.0 ** -24 * np.abs(v)
    vp = np.zeros((Rp, C))
    vp[:R] = v
    dvp = np.zeros((Rp, C))
    dvp[:R] = dv
    for p, ref, e in ((row, v, dv), (col, vp.T, dvp.T)):
        n, k = ref.shape
        got = decode(p, n, k, mx.E4M3)
        top = np.abs(ref).reshape(n, -1, 32).max(-1, keepdims=True).repeat(32, -1).reshape(n, k)
        half = 2.0 ** -8 * np.abs(ref) + e  # before the packing
        assert (np.abs(got - ref) <= half + 2.0 ** -4 * (np.abs(ref) + half) + 2.0 ** -17 * top).all()
    # sums of binary32 values in R / 16 + 6 steps at most per element
    bound = dv.sum(0) + 2.0 ** -24 * (R / 128 + 16) * np.abs(v).sum(0)
    assert (np.abs(f64(total) - v.sum(0)) <= bound).all()
    np.testing.assert_array_equal(f64(part).astype(np.float32)[0], f64(total).astype(np.float32)) if R <= 128 else None


@gpu
@pytest.mark.parametrize("act", [mx.ACT_GELU_TANH, mx.ACT_SILU])
def test_slope_is_the_difference_quotient_of_the_forward(act):
    """One row, gradient 1: its column sum is act'(s) in binary32, against central differences of the GEMM's activation."""
    C = 2048
    ck = mx.alloc_packed(1, C, mx.E4M3)
    mx.checkpoint_save(torch.linspace(-6, 6, C, device="cuda").reshape(1, C), ck)
    s = decode(ck, 1, C, mx.E4M3)[0]
    part, slope = torch.empty(1, C, device="cuda"), torch.empty(C, device="cuda")
    mx.quantize_saved(1, C, mx.E4M3, mx.RCEIL, act=act, x=torch.ones(1, C, dtype=torch.bfloat16, device="cuda"), saved=ck,
                      colsum_partials=part, colsum=slope)
    h = 2.0 ** -6

    def forward(x):
        c = torch.empty(1, C, device="cuda")
        mx.gemm_act(None, None, 1, C, 0, mx.E4M3, c, act=act, bias=torch.from_numpy(x.astype(np.float32)).cuda())
        return f64(c)[0]

    quotient = (forward(s + h) - forward(s - h)) / (2 * h)
    # |act'''| < 2: h^2 / 6 * 2; values to ACT_REL * 6.02 each over 2 h
    assert np.abs(f64(slope) - quotient).max() <= h * h / 3 + ACT_REL * 6.1 / h + ACT_REL * 4


@gpu
def test_no_rows_give_zero_sums_and_touch_nothing():
    C = 96
    total = torch.full((C,), 5.0, device="cuda")
    mx.quantize_saved(0, C, mx.E4M3, mx.RCEIL, x=torch.empty(0, C, dtype=torch.bfloat16, device="cuda"),
                      colsum_partials=torch.empty(0, C, device="cuda"), colsum=total)
    dW = torch.full((64, C), 5.0, device="cuda")
    db = torch.full((64,), 5.0, device="cuda")
    empty = lambda rows, k: mx.alloc_packed(rows, k, mx.E4M3)
    kw = dict(fmt=mx.E4M3, scale_mode=mx.RCEIL, dPr=empty(0, 64), dPc=empty(64, 0), Xc=empty(C, 0),
              db_partials=torch.empty(0, 64, device="cuda"))
    y = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    mx.linear_bwd_saved(0, 64, C, y, empty(0, C), empty(C, 64), dW=dW, db=db, accumulate=True, **kw)
    torch.cuda.synchronize()
    assert (total == 0).all() and (dW == 5).all() and (db == 0).all()
    mx.linear_bwd_saved(0, 64, C, y, empty(0, C), empty(C, 64), dW=dW, db=db, **kw)
    torch.cuda.synchronize()
    assert (dW == 0).all()


# ---------------------------------------------------------------- backward
def bwd_work(M, N, K, fmt):
    Mp = (M + 31) // 32 * 32
    return dict(dPr=mx.alloc_packed(M, N, fmt), dPc=mx.alloc_packed(N, Mp, fmt), Xc=mx.alloc_packed(K, Mp, fmt),
                db_partials=torch.empty((M + 127) // 128, N, device="cuda"))


@gpu
@pytest.mark.parametrize("fmt,mode,had", FMTS)
@pytest.mark.parametrize("act,x_act", [(mx.ACT_NONE, mx.ACT_GELU_TANH), (mx.ACT_GELU_TANH, mx.ACT_NONE),
                                       (mx.ACT_SILU, mx.ACT_SILU)])
@pytest.mark.parametrize("M,N,K", [(1, 64, 96), (50, 96, 160), (333, 256, 416), (200, 768, 2048), (700, 2080, 1024), (300, 320, 1024),
                                   (700, 704, 1024), (20, 32, 8224)])
def test_linear_bwd_against_64_bits(M, N, K, act, x_act, fmt, mode, had):
    rng = np.random.default_rng(M + N + K + fmt + act)
    dY = dev_bf16(rng.standard_normal((M, N)))
    cx, cp = mx.alloc_packed(M, K, mx.E4M3), mx.alloc_packed(M, N, mx.E4M3)
    mx.checkpoint_save(dev_bf16(rng.standard_normal((M, K))), cx)
    mx.checkpoint_save(dev_bf16(rng.standard_normal((M, N))), cp)
    Wc, wc = operand(rng, K, N, fmt, mode, had, std=0.1)
    dX, dW = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), torch.empty(N, K, device="cuda")
    db = torch.empty(N, device="cuda")
    work = bwd_work(M, N, K, fmt)
    kw = dict(fmt=fmt, scale_mode=mode, hadamard=had, act=act, saved_pre=cp if act else None, x_act=x_act)
    mx.linear_bwd_saved(M, N, K, dY, cx, Wc, dX=dX, dW=dW, db=db, **kw, **work)
    G = f64(dY) * slope64(decode(cp, M, N, mx.E4M3), act)
    X = act64(decode(cx, M, K, mx.E4M3), x_act)
    Mp = (M + 31) // 32 * 32
    assert np.abs(f64(db) - G.sum(0)).max() <= ACT_REL * 2.4 * np.abs(f64(dY)).sum(0).max() + 2.0 ** -20 * np.abs(G).sum(0).max()

    # the products of what was packed ...
    g, gc, xc = decode(work["dPr"], M, N, fmt), decode(work["dPc"], N, Mp, fmt), decode(work["Xc"], K, Mp, fmt)
    for got, want in ((dX, g @ wc.T), (dW, gc @ xc.T)):
        e = REL * np.abs(want).max() + (2.0 ** -8 * np.abs(want) if got.dtype == torch.bfloat16 else 0)
        assert (np.abs(f64(got) - want) <= e).all()
    # ... and what was packed is G and X, up to values on an edge of a rounding (flips of one step)
    pad = lambda a: np.concatenate([a, np.zeros((Mp - M, a.shape[1]))])
    for got, v in ((g, bf16_round(G)), (gc, bf16_round(pad(G)).T), (xc, bf16_round(pad(X)).T)):
        want = quantised64(np.ascontiguousarray(v), fmt, mode, had)[0]
        assert (np.abs(got - want) > 2.0 ** -12 * np.abs(want).max()).mean() <= 2e-3
        assert np.abs(got - want).max() <= np.abs(want).max() / 2

    # the same through its parts: packs and db bit for bit, products up to the order of the sums
    same = lambda x, y: np.abs(f64(x) - f64(y)).max() <= REL * np.abs(f64(y)).max() + 2.0 ** -8 * np.abs(f64(y)).max() * (
        x.dtype == torch.bfloat16)
    parts, dX2, dW2, db2 = bwd_work(M, N, K, fmt), torch.empty_like(dX), torch.empty_like(dW), torch.empty_like(db)
    q = dict(fmt=fmt, scale_mode=mode, hadamard=had)
    mx.quantize_saved(M, N, act=act, x=dY, saved=cp if act else None, row=parts["dPr"], col=parts["dPc"],
                      colsum_partials=parts["db_partials"], colsum=db2, **q)
    mx.quantize_saved(M, K, act=x_act, saved=cx, col=parts["Xc"], **q)
    mx.gemm_act(parts["dPr"], Wc, M, K, N, fmt, dX2)
    mx.gemm_act(parts["dPc"], parts["Xc"], N, K, Mp, fmt, dW2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for k in ("dPr", "dPc", "Xc") for x, y in zip(work[k], parts[k]))
    assert torch.equal(db, db2) and same(dX, dX2) and same(dW, dW2)

    # one output at a time gives the same, accumulation adds
    only = torch.empty_like(dX)
    mx.linear_bwd_saved(M, N, K, dY, None, Wc, dX=only, dPr=work["dPr"], **kw)
    sums = torch.empty_like(db)
    mx.linear_bwd_saved(M, N, K, dY, None, None, db=sums, db_partials=work["db_partials"], **kw)
    acc = torch.ones_like(dW)
    mx.linear_bwd_saved(M, N, K, dY, cx, None, dW=acc, dPc=work["dPc"], Xc=work["Xc"], accumulate=True, **kw)
    torch.cuda.synchronize()
    assert torch.equal(sums, db) and same(only, dX) and same(acc - 1, dW)


@gpu
@pytest.mark.parametrize("fmt,mode,had", FMTS)
def test_linear_bwd_of_large_tiles_is_its_parts(fmt, mode, had):
    """Both products of 256 x 256 tiles, column sums beside them: one launch, bit for bit the separate calls."""
    M, N, K = 2040, 2048, 8192
    rng = np.random.default_rng(fmt)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().cuda()
    dY, cx, cp = t(M, N), mx.alloc_packed(M, K, mx.E4M3), mx.alloc_packed(M, N, mx.E4M3)
    mx.checkpoint_save(t(M, K), cx)
    mx.checkpoint_save(t(M, N), cp)
    Wc = mx.alloc_packed(K, N, fmt)
    mx.quantize_saved(K, N, fmt, mode, had, x=t(K, N), row=Wc)
    outs = [[torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")]
            for _ in range(2)]
    (dX, dW, db), (dX2, dW2, db2) = outs
    w, v = bwd_work(M, N, K, fmt), bwd_work(M, N, K, fmt)
    q = dict(fmt=fmt, scale_mode=mode, hadamard=had)
    mx.linear_bwd_saved(M, N, K, dY, cx, Wc, act=mx.ACT_SILU, saved_pre=cp, dX=dX, dW=dW, db=db, **q, **w)
    mx.quantize_saved(M, N, act=mx.ACT_SILU, x=dY, saved=cp, row=v["dPr"], col=v["dPc"], colsum_partials=v["db_partials"],
                      colsum=db2, **q)
    mx.quantize_saved(M, K, saved=cx, col=v["Xc"], **q)
    mx.gemm_act(v["dPr"], Wc, M, K, N, fmt, dX2)
    mx.gemm_act(v["dPc"], v["Xc"], N, K, 2048, fmt, dW2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*outs))


@gpu
@pytest.mark.parametrize("M", [1, 77, 640])
def test_mlp_step_from_checkpoints(M):
    """An MLP as it is trained: up projection (GELU, checkpoint) -> down projection + residual stream, then its
    backward pass from two checkpoints, against the unquantised MLP's values and gradients in 64 bits."""
    D, F, fmt, mode = 256, 512, mx.E4M3, mx.RCEIL
    rng = np.random.default_rng(M)
    t = lambda *s, std=1.0: dev_bf16(rng.standard_normal(s) * std)
    X, W1, W2, b1, dY = t(M, D), t(F, D, std=0.06), t(D, F, std=0.04), t(F, std=0.1), t(M, D)
    rows = lambda x: (lambda p: (mx.quantize_saved(x.shape[0], x.shape[1], fmt, mode, x=x, row=p), p)[1])(
        mx.alloc_packed(x.shape[0], x.shape[1], fmt))
    sx, W1r, W2r = rows(X), rows(W1), rows(W2)
    W1c, W2c = rows(W1.t().contiguous()), rows(W2.t().contiguous())
    sh, ar = mx.alloc_packed(M, F, fmt), mx.alloc_packed(M, F, fmt)
    Y = torch.empty_like(X)
    mx.gemm_act(sx, W1r, M, F, D, fmt, bias=b1, saved=sh)                 # the pre-activation in 8 bits only
    mx.quantize_saved(M, F, fmt, mode, act=mx.ACT_GELU_TANH, saved=sh, row=ar)
    mx.gemm_act(ar, W2r, M, D, F, fmt, Y, residual=X)
    dA, dW2 = torch.empty(M, F, dtype=torch.bfloat16, device="cuda"), torch.empty(D, F, device="cuda")
    mx.linear_bwd_saved(M, D, F, dY, sh, W2c, fmt, mode, x_act=mx.ACT_GELU_TANH, dX=dA, dW=dW2, **bwd_work(M, D, F, fmt))
    dX, dW1, db1 = torch.empty_like(X), torch.empty(F, D, device="cuda"), torch.empty(F, device="cuda")
    mx.linear_bwd_saved(M, F, D, dA, sx, W1c, fmt, mode, act=mx.ACT_GELU_TANH, saved_pre=sh, dX=dX, dW=dW1, db=db1,
                        **bwd_work(M, F, D, fmt))
    x, w1, w2, dy = f64(X), f64(W1), f64(W2), f64(dY)
    h = x @ w1.T + f64(b1)
    a = act64(h, mx.ACT_GELU_TANH)
    da = dy @ w2
    dh = da * slope64(h, mx.ACT_GELU_TANH)
    # each MXFP8 factor is within 2^-4 of itself (RMS about 2^-4 / sqrt(3) * 0.7 = 2.5%): products of two factors and
    # one checkpoint between them stay within 5 such errors in the 2-norm, 13%
    for name, got, want in (("Y - X", f64(Y) - x, a @ w2.T), ("dW2", f64(dW2), dy.T @ a), ("dX", f64(dX), dh @ w1),
                            ("dW1", f64(dW1), dh.T @ x), ("db1", f64(db1), dh.sum(0))):
        assert np.linalg.norm(got - want) <= 0.13 * np.linalg.norm(want), name


@gpu
def test_captured_steps_replay_and_other_streams():
    """A captured forward and backward replays to the eager results, beside eager work; a step on another stream too."""
    M, N, K, fmt, mode = 150, 160, 256, mx.E2M3, mx.FLOOR
    rng = np.random.default_rng(8)
    X, W, dY, b = dev_bf16(rng.standard_normal((M, K))), dev_bf16(rng.standard_normal((N, K)) * 0.1), dev_bf16(
        rng.standard_normal((M, N))), dev_bf16(rng.standard_normal(N))
    Wr, Wc = mx.alloc_packed(N, K, fmt), mx.alloc_packed(K, N, fmt)
    mx.quantize_saved(N, K, fmt, mode, True, x=W, row=Wr, col=Wc)
    torch.cuda.synchronize()

    def buffers():
        return dict(A=mx.alloc_packed(M, K, fmt), sx=mx.alloc_packed(M, K, mx.E4M3), sp=mx.alloc_packed(M, N, mx.E4M3),
                    C=torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), dX=torch.empty(M, K, dtype=torch.bfloat16, device="cuda"),
                    dW=torch.empty(N, K, device="cuda"), db=torch.empty(N, device="cuda"), work=bwd_work(M, N, K, fmt))

    def step(s):
        mx.quantize_saved(M, K, fmt, mode, True, x=X, row=s["A"])
        mx.checkpoint_save(X, s["sx"])
        mx.gemm_act(s["A"], Wr, M, N, K, fmt, s["C"], act=mx.ACT_GELU_TANH, bias=b, saved=s["sp"])
        mx.linear_bwd_saved(M, N, K, dY, s["sx"], Wc, fmt, mode, True, act=mx.ACT_GELU_TANH, saved_pre=s["sp"], dX=s["dX"],
                            dW=s["dW"], db=s["db"], **s["work"])

    def outs(s):
        return [s["C"], s["sp"][0], s["sp"][1], s["dX"], s["dW"], s["db"]]

    eager, captured, other = buffers(), buffers(), buffers()
    step(eager)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(other)
    step(captured)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs(eager), outs(other)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(captured)
    for _ in range(3):
        for o in outs(captured):
            o.zero_()
        step(eager)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs(eager), outs(captured)))


@gpu
def test_two_streams_at_once_do_not_disturb_each_other():
    """Two backward passes with buffers of their own, issued alternately on two streams."""
    M, N, K, fmt, mode = 333, 416, 800, mx.E4M3, mx.RCEIL
    rng = np.random.default_rng(4)
    t = lambda *s: dev_bf16(rng.standard_normal(s))
    Wc = mx.alloc_packed(K, N, fmt)
    mx.quantize_saved(K, N, fmt, mode, x=t(K, N), row=Wc)
    sides = []
    for _ in range(2):
        dY, X, cx, cp = t(M, N), t(M, K), mx.alloc_packed(M, K, mx.E4M3), mx.alloc_packed(M, N, mx.E4M3)
        mx.checkpoint_save(X, cx)
        mx.checkpoint_save(t(M, N), cp)
        out = dict(dX=torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), dW=torch.empty(N, K, device="cuda"),
                   db=torch.empty(N, device="cuda"))
        sides.append((dY, cx, cp, out, bwd_work(M, N, K, fmt), torch.cuda.Stream()))

    def step(dY, cx, cp, out, work, stream):
        mx.linear_bwd_saved(M, N, K, dY, cx, Wc, fmt, mode, act=mx.ACT_GELU_TANH, saved_pre=cp, stream=stream, **out, **work)

    want = []
    for s in sides:
        torch.cuda.synchronize()
        step(*s)
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in s[3].items()})
    for _ in range(5):
        for s in sides:
            for v in s[3].values():
                v.zero_()
        torch.cuda.synchronize()
        for s in sides:
            step(*s)
        torch.cuda.synchronize()
        assert all(torch.equal(s[3][k], w[k]) for s, w in zip(sides, want) for k in w)


@gpu
def test_checkpoint_offsets_past_32_bits():
    """A checkpoint of more than 2^31 values (4.3 GB of bf16): first and last rows survive the round trip."""
    R, C = (1 << 31) // 4096 + 65, 4096
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(1)
    edge = dev_bf16(rng.standard_normal((64, C)))
    x[:64] = edge
    x[-64:] = edge
    p = mx.alloc_packed(R, C, mx.E4M3)
    mx.checkpoint_save(x, p)
    x.fill_(1.0)
    mx.checkpoint_load(p, x)
    small = mx.alloc_packed(64, C, mx.E4M3)
    want = torch.empty_like(edge)
    mx.checkpoint_save(edge, small)
    mx.checkpoint_load(small, want)
    torch.cuda.synchronize()
    assert torch.equal(x[:64], want) and torch.equal(x[-64:], want) and not x[64:-64].any()


@gpu
@pytest.mark.parametrize("fmt,mode,had", FMTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(4096, 2048, 16384), (2100, 1952, 16352), (520, 4096, 2080)])
def test_accumulating_backward_with_every_output_is_its_parts(M, N, K, dtype, fmt, mode, had):
    """dX, dW added into its main_grad, and db in one call, against the separate calls.  The first two sizes give the
    MXFP4 weight gradient 256 x 128 tiles and the longer sums.  Where the products share a launch of unlike variants
    the sums' order may differ, so those agree to REL; packs and db are bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(M + N + K + fmt)
    t = lambda *s: torch.randn(s, generator=g, device="cuda")
    dY, cx, cp = t(M, N).bfloat16(), mx.alloc_packed(M, K, mx.E4M3), mx.alloc_packed(M, N, mx.E4M3)
    mx.checkpoint_save(t(M, K), cx)
    mx.checkpoint_save(t(M, N), cp)
    Wc = mx.alloc_packed(K, N, fmt)
    q = dict(fmt=fmt, scale_mode=mode, hadamard=had)
    mx.quantize_saved(K, N, x=t(K, N).bfloat16(), row=Wc, **q)
    old = (t(N, K) * 8).to(dtype)
    dX, dW, db = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), old.clone(), torch.empty(N, device="cuda")
    w, v = bwd_work(M, N, K, fmt), bwd_work(M, N, K, fmt)
    mx.linear_bwd_saved(M, N, K, dY, cx, Wc, act=mx.ACT_GELU_TANH, saved_pre=cp, dX=dX, dW=dW, db=db, accumulate=True, **q, **w)
    dX2, dW2, db2 = torch.empty_like(dX), old.clone(), torch.empty_like(db)
    mx.quantize_saved(M, N, act=mx.ACT_GELU_TANH, x=dY, saved=cp, row=v["dPr"], col=v["dPc"], colsum_partials=v["db_partials"],
                      colsum=db2, **q)
    mx.quantize_saved(M, K, saved=cx, col=v["Xc"], **q)
    mx.gemm_act(v["dPr"], Wc, M, K, N, fmt, dX2)
    mx.gemm_act(v["dPc"], v["Xc"], N, K, (M + 31) // 32 * 32, fmt, dW2, residual=dW2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for k in ("dPr", "dPc", "Xc") for x, y in zip(w[k], v[k]))
    assert torch.equal(db, db2)
    for got, want, grad in ((dX, dX2, dX2.double()), (dW, dW2, dW2.double() - old.double())):
        step = 2.0 ** -7 if got.dtype == torch.bfloat16 else 2.0 ** -23  # two roundings, half a step each
        assert ((got.double() - want.double()).abs() <= REL * grad.abs().max() + step * want.double().abs()).all()
    assert not torch.equal(dW, old)


@gpu
@pytest.mark.parametrize("fmt,mode,had", FMTS)
@pytest.mark.parametrize("M,N", [(8192, 8192), (4096, 12288), (1500, 4096), (30, 96)])
def test_empty_sums_at_every_tile_size(M, N, fmt, mode, had):
    """K = 0 is act(bias) + residual, and a backward pass without tokens zeroes dW (N = 0: dX), whatever variant serves it."""
    c = torch.full((M, N), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.gemm_act(None, None, M, N, 0, fmt, c)
    torch.cuda.synchronize()
    assert not c.any()
    bias = torch.arange(N, device="cuda").float() % 64 - 32
    for residual in (None, c):
        c.fill_(3.0)
        saved = mx.alloc_packed(M, N, mx.E4M3)
        mx.gemm_act(None, None, M, N, 0, fmt, c, bias=bias, residual=residual, saved=saved)
        torch.cuda.synchronize()
        want = bias + (0 if residual is None else 3)  # small integers: exact
        assert torch.equal(c.float(), want.expand(M, N))
        mx.checkpoint_load(saved, c)
        ref = mx.alloc_packed(1, N, mx.E4M3)
        mx.checkpoint_save(bias.reshape(1, N), ref)
        row = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
        mx.checkpoint_load(ref, row)
        torch.cuda.synchronize()
        assert torch.equal(c, row.expand(M, N))
    O = (M + 31) // 32 * 32  # (an output width)
    dW, db = torch.full((O, N), 5.0, device="cuda"), torch.full((O,), 5.0, device="cuda")
    e = lambda rows, k, f=fmt: mx.alloc_packed(rows, k, f)
    y = torch.empty(0, O, dtype=torch.bfloat16, device="cuda")
    kw = dict(fmt=fmt, scale_mode=mode, hadamard=had)
    for accumulate in (True, False):
        db.fill_(5.0)
        mx.linear_bwd_saved(0, O, N, y, e(0, N, mx.E4M3), e(N, O), dX=torch.empty(0, N, dtype=torch.bfloat16, device="cuda"), dW=dW,
                            db=db, dPr=e(0, O), dPc=e(O, 0), Xc=e(N, 0), db_partials=torch.empty(0, O, device="cuda"),
                            accumulate=accumulate, **kw)
        torch.cuda.synchronize()
        assert (dW == (5 if accumulate else 0)).all() and not db.any()
    dX = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
    mx.linear_bwd_saved(M, 0, N, torch.empty(M, 0, dtype=torch.bfloat16, device="cuda"), None, None, dX=dX, dPr=None, **kw)
    torch.cuda.synchronize()
    assert not dX.any()


@gpu
@pytest.mark.parametrize("fmt,mode,had", FMTS)
def test_every_size_and_choice_of_outputs_reaches_a_kernel(fmt, mode, had):
    """Sizes over the whole range, every epilogue and every choice of outputs: each call is served.  (Zero operands, so
    that the outputs have to be bias, residual or zero.)"""
    rng = np.random.default_rng(fmt)
    big = 8192 * 8192
    room = {k: torch.zeros(big * b, dtype=torch.uint8, device="cuda") for k, b in
            dict(a=1, as_=1, b=1, bs=1, x=1, xs=1, p=1, ps=1, c=1, cs=1, r=1, rs=1).items()}
    out, add, g2 = (torch.zeros(big, dtype=torch.float32, device="cuda") for _ in range(3))
    bf = torch.zeros(2, big, dtype=torch.bfloat16, device="cuda")

    def operand_of(name, rows, k, f):
        n, b = (k + 127) // 128 * rows * 4, mx.BITS[f] * 4
        return room[name][:n * b], room[name + ("s" if name != "a" else "s_")][:n]

    size = lambda top: int(round(np.exp(rng.uniform(0, np.log(top)))))
    for _ in range(120):
        M, N, K = size(8192), 32 * size(256), 32 * size(256)
        if rng.random() < 0.15:
            K = 0
        act, flags = int(rng.integers(3)), rng.random(4) < 0.5
        f32 = bool(flags[0])
        store = out if f32 else bf[0]
        c = store[:M * N].fill_(9.0).reshape(M, N)
        res = (add if f32 else bf[1])[:M * N].reshape(M, N) if flags[1] else None
        mx.gemm_act(operand_of("a", M, K, fmt), operand_of("b", N, K, fmt), M, N, K, fmt, c, act=act, residual=res,
                    saved=operand_of("x", M, N, mx.E4M3) if flags[2] else None)
        assert not c.any(), (M, N, K, act, flags)
        room["x"][:((N + 127) // 128) * M * 128].zero_()
        room["xs"][:((N + 127) // 128) * M * 4].zero_()

        want = rng.random(3) < 0.7
        if not want.any():
            want[:] = True
        N, K = max(32, N), max(32, K)
        Mp = (M + 31) // 32 * 32
        acc = bool(rng.random() < 0.5)
        dW = (g2 if f32 else bf[1])[:N * K].fill_(1.0).reshape(N, K)
        dX = bf[0][:M * K].fill_(9.0).reshape(M, K)
        db, part = torch.full((N,), 9.0, device="cuda"), out[:(M + 127) // 128 * N].reshape(-1, N)
        dY = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        mx.linear_bwd_saved(M, N, K, dY, operand_of("x", M, K, mx.E4M3), operand_of("b", K, N, fmt), fmt, mode, had, act=act,
                            saved_pre=operand_of("a", M, N, mx.E4M3) if act else None, dX=dX if want[0] else None,
                            dW=dW if want[1] else None, db=db if want[2] else None, db_partials=part,
                            dPr=operand_of("p", M, N, fmt), dPc=operand_of("c", N, Mp, fmt), Xc=operand_of("r", K, Mp, fmt),
                            accumulate=acc)
        case = (M, N, K, act, f32, want, acc)
        assert (dX == (0 if want[0] else 9)).all() and (db == (0 if want[2] else 9)).all(), case
        assert (dW == (1 if acc or not want[1] else 0)).all(), case
        bf[1].zero_()
        room["a"].zero_(), room["as_"].zero_()


@gpu
def test_a_nan_scale_is_nan_whatever_the_codes():
    """Operands packed elsewhere may hold any codes under the scale byte 0xff: zeros, numbers of either sign, NaN codes."""
    R, C = 40, 128
    codes = torch.arange(R * C, dtype=torch.int64, device="cuda").remainder(256).to(torch.uint8).reshape(1, R, C)
    scales = torch.full((1, R, 4), 127, dtype=torch.uint8, device="cuda")
    scales[0, 5:33, 2] = 255
    bad = torch.zeros(R, C, dtype=torch.bool, device="cuda")
    bad[5:33, 64:96] = True
    bad |= (codes[0] & 0x7F) == 0x7F
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.empty(R, C, dtype=dtype, device="cuda")
        mx.checkpoint_load((codes, scales), y)
        torch.cuda.synchronize()
        assert torch.equal(y.isnan(), bad) and not y.isinf().any()
    ones = torch.ones(R, C, dtype=torch.bfloat16, device="cuda")
    for act in ACTS:
        for x in (None, ones) if act else (None,):
            row, total = mx.alloc_packed(R, C, mx.E4M3), torch.empty(C, device="cuda")
            part = torch.empty(1, C, device="cuda")
            mx.quantize_saved(R, C, mx.E4M3, mx.RCEIL, act=act, x=x, saved=(codes, scales), row=row, colsum_partials=part,
                              colsum=total)
            torch.cuda.synchronize()
            assert torch.equal(total.isnan(), bad.any(0)) and not total.isinf().any()
            assert torch.equal(row[1][0] == 255, bad.reshape(R, 4, 32).any(-1))


@gpu
def test_checkpoint_error_bound_at_its_edges():
    """Half an E4M3 step: 2^-4 of a value, and below the format's normal range 2^-10 of the scale 2^X, with the block's
    largest value in (224, 448] 2^X: 2^-10 / 224 < 2^-17 of it, or 2^-137 at the least scale 2^-127."""
    rng = np.random.default_rng(2)
    R, C = 64, 256
    x = rng.standard_normal((R, C // 32, 32)) * 2.0 ** rng.integers(-12, 1, (R, C // 32, 32))
    x /= np.abs(x).max(-1, keepdims=True)
    x[..., 0] = 1                                                     # the block's largest
    x[::2, :, 1:8] = 2.0 ** -10 / 225 * np.linspace(0.9, 0.9999, 7)   # just under half the least step
    top = rng.choice([225.0, 224.125, 448.0, 300.0, 2.0 ** 100, 2.0 ** -100, 225 * 2.0 ** -127, 2.0 ** -121, 2.0 ** -130], (R, C // 32, 1))
    x = (x * top).reshape(R, C).astype(np.float32)
    p, y = mx.alloc_packed(R, C, mx.E4M3), torch.empty(R, C, device="cuda")
    mx.checkpoint_save(torch.from_numpy(x).cuda(), p)
    mx.checkpoint_load(p, y)
    v, err = np.abs(x.astype(np.float64)), np.abs(f64(y) - x.astype(np.float64))
    largest = v.reshape(R, -1, 32).max(-1, keepdims=True).repeat(32, -1).reshape(R, C)
    bound = np.where(largest < 2.0 ** -119, 2.0 ** -137, 2.0 ** -10 / 224 * largest)
    assert (err <= np.maximum(2.0 ** -4 * v, bound)).all()
    assert (2.0 ** -10 / 224 * largest < 2.0 ** -17 * largest).all()
    assert (err[::2][largest[::2] == 225] > 2.0 ** -18 * 225).any()   # no smaller power of two would do


@gpu
@pytest.mark.parametrize("act", [mx.ACT_GELU_TANH, mx.ACT_SILU])
def test_activation_and_slope_error_bounds(act):
    """The header's bounds, z to +-120: act to (4 |z| + 6) 2^-24 of itself or 2^-126 |x|, act' to 2^-17.

    act: x^2 and the constants (GELU: A + B x^2 to 2.6 u, u = 2^-24; SiLU: 0.7 u), two products at most: 3.6 u of z, then
    exp2 2 u, 1 + e u, the reciprocal 2 u, x s u.  Where 1 + e is past 2^126 its reciprocal may be flushed to 0: 2^-126 |x|.
    act': s + x z' s (1 - s); s next to 1 is off by 2 u at most and x z' <= 33 there, elsewhere the product is smaller."""
    top = 11.2 if act == mx.ACT_GELU_TANH else 120.0
    x = np.linspace(-top, top, 8192).astype(np.float32)
    x64 = x.astype(np.float64)
    z = 2 * K0 * (x64 + K1 * x64 ** 3) if act == mx.ACT_GELU_TANH else x64
    want = act64(x64, act)
    for M in (1, 9600):  # the few-rows kernel and the tiles
        c = torch.empty(M, 8192, device="cuda")
        mx.gemm_act(None, None, M, 8192, 0, mx.E2M3, c, act=act, bias=torch.from_numpy(x).cuda())
        assert (np.abs(f64(c[-1]) - want) <= (4 * np.abs(z) + 6) * 2.0 ** -24 * np.abs(want) + 2.0 ** -126 * np.abs(x64)).all()
    ck = mx.alloc_packed(1, 8192, mx.E4M3)
    t = np.exp2(np.linspace(-10, np.log2(top), 8192)) * np.where(np.arange(8192) % 2, -1, 1)  # both signs, by magnitude
    mx.checkpoint_save(torch.from_numpy(t.astype(np.float32).reshape(1, -1)).cuda(), ck)
    s = decode(ck, 1, 8192, mx.E4M3)[0]
    part, slope = torch.empty(1, 8192, device="cuda"), torch.empty(8192, device="cuda")
    mx.quantize_saved(1, 8192, mx.E4M3, mx.RCEIL, act=act, x=torch.ones(1, 8192, dtype=torch.bfloat16, device="cuda"), saved=ck,
                      colsum_partials=part, colsum=slope)
    assert np.abs(f64(slope) - slope64(s, act)).max() <= 2.0 ** -17


def test_sizes_past_the_thread_limit_of_a_launch_are_refused():
    """2^32 threads: 2^24 workgroups of 256 (checkpoints, 64 x 128 values each), 2^23 of 512 (packs, 128 x 128)."""
    L = mx.lib()
    for R, C in ((1 << 30, 128), ((1 << 22) * 64 - 63, 512), (64, 1 << 31)):
        assert L.mx_checkpoint_save(P[0], 0, R, C, C, P[1], P[2], None) == OVERFLOW
        assert L.mx_checkpoint_load(P[1], P[2], R, C, P[0], 0, C, None) == OVERFLOW
    for R, C in ((1 << 30, 128), ((1 << 21) * 128 - 127, 512), (128, 1 << 30)):
        for x in (None, P[0]):
            a = saved_args(R=R, C=C, x=x, ldx=C)
            assert L.mx_quantize_saved(ctypes.byref(a), None) == OVERFLOW
    if not torch.cuda.is_available():  # one tile less passes the checks of the arguments
        assert L.mx_checkpoint_save(P[0], 0, (1 << 30) - 64, 128, 128, P[1], P[2], None) == DEVICE
        assert L.mx_quantize_saved(ctypes.byref(saved_args(R=(1 << 30) - 128, C=128, ldx=128)), None) == DEVICE


@gpu
@pytest.mark.parametrize("fmt,mode,had", FMTS)
def test_captured_accumulating_backward(fmt, mode, had):
    """Every replay adds the gradient once more, as every eager call does; products in a launch each (MXFP4) or in one."""
    M, N, K = 2100, 1952, 16352
    g = torch.Generator(device="cuda").manual_seed(fmt)
    t = lambda *s: torch.randn(s, generator=g, device="cuda")
    dY, cx, cp, Wc = t(M, N).bfloat16(), mx.alloc_packed(M, K, mx.E4M3), mx.alloc_packed(M, N, mx.E4M3), mx.alloc_packed(K, N, fmt)
    mx.checkpoint_save(t(M, K), cx)
    mx.checkpoint_save(t(M, N), cp)
    q = dict(fmt=fmt, scale_mode=mode, hadamard=had)
    mx.quantize_saved(K, N, x=t(K, N).bfloat16(), row=Wc, **q)
    sides = [(dict(dX=torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), dW=torch.zeros(N, K, device="cuda"),
                   db=torch.empty(N, device="cuda")), bwd_work(M, N, K, fmt)) for _ in range(2)]

    def step(out, work):
        mx.linear_bwd_saved(M, N, K, dY, cx, Wc, act=mx.ACT_SILU, saved_pre=cp, accumulate=True, **q, **out, **work)

    step(*sides[0])  # eager first, so that nothing is loaded during the capture
    sides[0][0]["dW"].zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*sides[1])
    sides[1][0]["dW"].zero_()
    for _ in range(3):
        for out, _ in sides:
            out["dX"].zero_(), out["db"].zero_()
        step(*sides[0])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(sides[0][0][k], sides[1][0][k]) for k in ("dX", "dW", "db"))
        assert sides[0][0]["dW"].any()
