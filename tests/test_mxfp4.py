"""Microscaled 4-bit (MXFP4) quantisation and product against their
definitions in binary64, at the sizes and values where they can go wrong, and
their refusals.

Tolerances.  Quantisation and dequantisation are exact: codes, scales and
values are compared for equality.  The product of E2M1 codes is exact in FP32;
a K = 64 step adds one 64-element sum to the FP32 accumulator, so with
chopping instead of rounding in every addition the error is below
(K / 64 + 2) * 2^-22 * sum_k |a w|; a bf16 output lies between the bf16
roundings of the two ends of that interval (rounding is monotone).  Where every product and sum is a small multiple of 1/4 the FP32
sum is exact and the comparison is for equality."""
import ctypes

import numpy as np
import pytest
import torch

import w4a16_int4_mixture_moe_gb300 as chord

DEV = "cuda:0"
MAG = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float64)
gpu = pytest.mark.gpu


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    chord.build()
    chord.load()
    chord.chord_get_device_error()


# ------------------------------------------------------ the definition, in 64 bits

def ref_quantise(v):
    """float64 [..., K] -> (codes uint8 [..., K], b uint8 [..., K / 32])."""
    v = np.asarray(v, np.float64)
    blk = v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32))
    bad = ~np.isfinite(blk).all(axis=-1)
    a = np.where(bad[..., None], 0.0, np.abs(blk))
    top = a.max(axis=-1)
    _, ex = np.frexp(top)                        # top = m * 2^ex, m in [1/2, 1)
    e = np.clip(np.where(top > 0, ex - 1 - 2, -127), -127, 127)
    y = np.ldexp(a, -e[..., None])
    dist = np.abs(y[..., None] - MAG)
    best = dist.min(axis=-1, keepdims=True)
    tie = dist == best                           # one code, or two neighbours: take the even one
    even = np.array([1, 0, 1, 0, 1, 0, 1, 0], bool)
    code = np.where((tie & even).any(axis=-1), np.argmax(tie & even, axis=-1), np.argmax(tie, axis=-1))
    code = code.astype(np.uint8) | (np.signbit(blk).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    b = np.where(bad, 255, e + 127).astype(np.uint8)
    return code.reshape(v.shape), b


def ref_values(code, b):
    v = MAG[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(b == 255, np.nan, np.ldexp(1.0, b.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def unpack(packed, G, N, K):
    """Codes and scales of a packed matrix, from the written-out layout."""
    raw = packed.cpu().numpy()
    rt, kb = -(-N // 128), -(-K // 256)
    assert raw.size == 256 + G * rt * kb * 17408
    tiles = raw[256:].reshape(G, rt, kb, 17408)
    codes = np.zeros((G, N, K), np.uint8)
    b = np.zeros((G, N, K // 32), np.uint8)
    for r in range(N):
        for j in range(K // 32):
            t = tiles[:, r // 128, j // 8]
            q, jj = r % 128, j % 8
            o = q * 128 + 16 * (jj ^ (q % 8))
            by = t[:, o:o + 16]
            codes[:, r, 32 * j:32 * j + 32:2] = by & 15
            codes[:, r, 32 * j + 1:32 * j + 32:2] = by >> 4
            b[:, r, j] = t[:, 16384 + 512 * (jj // 4) + 16 * (q % 32) + 4 * (q // 32) + jj % 4]
    return codes, b


def quantise(src):
    G, N, K = src.shape
    packed = torch.full((chord.chord_mxfp4_bytes(G, N, K),), 0xA5, dtype=torch.uint8, device=DEV)
    chord.chord_mxfp4_quantize(src, packed)
    return packed


def values_of(packed, G, N, K, dtype=torch.float32):
    out = torch.empty((G, N, K), dtype=dtype, device=DEV)
    chord.chord_mxfp4_dequantize(packed, out)
    return out


# ------------------------------------------------------------- CPU: sizes, refusals

def test_sizes():
    assert chord.chord_mxfp4_bytes(1, 1, 32) == 256 + 17408
    assert chord.chord_mxfp4_bytes(3, 129, 288) == 256 + 3 * 2 * 2 * 17408
    assert chord.chord_mxfp4_bytes(0, 5, 32) == chord.chord_mxfp4_bytes(2, 0, 32) == 256
    for bad in [(1, 1, 0), (1, 1, 33), (-1, 1, 32), (1, -1, 32)]:
        assert chord.chord_mxfp4_bytes(*bad) == 0
    assert chord.chord_mxfp4_rows_bytes(96, 32, 64) == chord.chord_mxfp4_bytes(3, 32, 64) + 512
    assert chord.chord_mxfp4_rows_bytes(95, 32, 64) == 0


def test_sizes_past_64_bits_are_refused():
    """A byte count that does not fit is no size (2^30 groups of 2^31 x 2^31 once
    gave 256), and every call that checks against it refuses the shape."""
    big = 2 ** 31 - 32
    assert chord.chord_mxfp4_bytes(2 ** 30, 2 ** 31 - 1, big) == 0
    assert chord.chord_mxfp4_bytes(2 ** 31 - 1, 2 ** 31 - 1, big) == 0
    assert chord.chord_mxfp4_rows_bytes(2 ** 31 - 2, 2, big) == 0
    assert chord.chord_mxfp4_bytes(1, 2 ** 31 - 1, big) == 256 + 2 ** 24 * 2 ** 23 * 17408      # 2^61: the largest group
    p = ctypes.c_void_p(1 << 20)
    lib = chord.load()
    assert lib.chord_mxfp4_quantize(p, 0, big, 0, 2 ** 30, 2 ** 31 - 1, big, p, 256, None) == 2
    assert lib.chord_mxfp4_dequantize(p, 256, 2 ** 30, 2 ** 31 - 1, big, p, 0, None) == 2
    for wrong in (0, 256):
        assert lib.chord_mxfp4_quantize_rows(p, 0, 4, big, 1, big, p, p, 2 ** 31 - 2, 2, 4, p, wrong, None) == 3
        assert lib.chord_mxfp4_moe_gemm(p, chord.chord_mxfp4_rows_bytes(64, 32, big), p, wrong, 2 ** 30, big, big, p, p, p,
                                        64, 32, 8, p, 0, None, None) == 3


@pytest.mark.parametrize("T,topk,E_local,E_global", [(-1, 8, 8, 8), (-2 ** 31, 1, 1, 1), (5, -3, 0, 0), (2 ** 31 - 1, 2 ** 31 - 1, 1, 1),
                                                     (64, 8, 48, 0), (64, 8, 48, -5)])
def test_select_block_m_is_valid_for_any_arguments(T, topk, E_local, E_global):
    bm = chord.chord_mxfp4_select_block_m(T, topk, E_local, E_global)
    assert bm % 16 == 0 and 16 <= bm <= 208


def test_select_block_m():
    for T, topk, E in [(1, 1, 8), (1, 8, 384), (64, 8, 48), (1024, 8, 48), (4096, 8, 48), (100000, 8, 8), (0, 8, 8)]:
        bm = chord.chord_mxfp4_select_block_m(T, topk, E, E)
        assert bm % 16 == 0 and 16 <= bm <= 208
        tok = T * topk / E
        if tok + 2 * tok ** .5 + 1 <= 208:
            assert bm >= min(tok + 3 * tok ** .5 + 1, 208)


def test_refusals():
    lib = chord.load() if not chord._lib else chord._lib
    vp = ctypes.c_void_p
    p = vp(1 << 20)
    n = chord.chord_mxfp4_bytes
    q = lib.chord_mxfp4_quantize
    assert q(p, 0, 64, 0, 1, 4, 48, p, 10 ** 6, None) == 2                       # K % 32
    assert q(p, 2, 64, 0, 1, 4, 64, p, n(1, 4, 64), None) == 1                   # dtype
    assert q(p, 0, 64, 0, 1, 4, 64, p, n(1, 4, 64) + 1, None) == 3               # size
    assert q(p, 0, 63, 0, 1, 4, 64, p, n(1, 4, 64), None) == 1                   # rows overlap
    assert q(None, 0, 64, 0, 1, 4, 64, p, n(1, 4, 64), None) == 1
    assert q(p, 0, 64, 0, 1, 4, 64, vp((1 << 20) + 8), n(1, 4, 64), None) == 1   # alignment
    assert q(vp((1 << 20) + 1), 0, 64, 0, 1, 4, 64, p, n(1, 4, 64), None) == 1
    assert q(p, 0, 64, 0, -1, 4, 64, p, n(1, 4, 64), None) == 1
    d = lib.chord_mxfp4_dequantize
    assert d(p, n(1, 4, 64), 1, 4, 64, None, 0, None) == 1
    assert d(p, 5, 1, 4, 64, p, 0, None) == 3
    assert d(p, n(1, 4, 64), 1, 4, 64, p, 7, None) == 1
    r = lib.chord_mxfp4_quantize_rows
    nb = chord.chord_mxfp4_rows_bytes(64, 32, 64)
    assert r(p, 0, 4, 64, 0, 64, p, p, 64, 32, 8, p, nb, None) == 1              # divisor
    assert r(p, 0, 4, 64, 2, 40, p, p, 64, 32, 8, p, nb, None) == 2              # K
    assert r(p, 0, 4, 64, 2, 64, p, p, 65, 32, 8, p, nb, None) == 1              # capacity % block_m
    assert r(p, 0, 4, 64, 2, 64, None, p, 64, 32, 8, p, nb, None) == 1
    assert r(p, 0, 4, 64, 2, 64, p, p, 64, 32, 8, p, nb - 16, None) == 3
    g = lib.chord_mxfp4_moe_gemm
    wb = n(2, 100, 64)
    ok = [p, nb, p, wb, 2, 100, 64, p, p, p, 64, 32, 8, p, 0, None, None]
    for at, v, st in [(11, 40, 2), (11, 224, 2), (6, 48, 2), (1, nb + 16, 3), (3, wb - 16, 3), (14, 3, 1), (4, 0, 1),
                      (13, vp((1 << 20) + 4), 1), (0, None, 1), (7, None, 1), (9, None, 1), (10, 63, 1)]:
        a = list(ok)
        a[at] = v
        assert g(*a) == st, (at, v)
    dg = lib.chord_mxfp4_gemm
    assert dg(p, n(1, 8, 64), 8, p, n(1, 100, 64), 100, 48, p, 0, None, None) == 2
    assert dg(p, n(1, 129, 64), 8, p, n(1, 100, 64), 100, 64, p, 0, None, None) == 3
    assert dg(p, n(1, 8, 64), -1, p, n(1, 100, 64), 100, 64, p, 0, None, None) == 1
    assert dg(p, n(1, 8, 64), 8, p, n(1, 100, 64), 100, 64, None, 0, None, None) == 1


def test_reference_quantiser_on_hand_worked_values():
    v = np.zeros((1, 32))
    v[0, :8] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5]     # scale 1, every tie to the even code
    c, b = ref_quantise(v)
    assert b[0, 0] == 127 and c[0, :8].tolist() == [7, 0, 2, 2, 4, 4, 6, 6]
    c, b = ref_quantise(-1.99 * v)                        # 11.94: scale 2, codes of the unscaled ratios
    assert b[0, 0] == 128 and c[0, 0] == 15
    assert ref_quantise(np.zeros((1, 32)))[1][0, 0] == 0
    assert ref_quantise(np.full((1, 32), 2.0 ** -140))[1][0, 0] == 0


# --------------------------------------------------------------- GPU: quantisation

def nasty(rng, G, N, K, dtype):
    v = rng.standard_normal((G, N, K)) * np.exp2(rng.integers(-30, 30, (G, N, 1)))
    v[:, 0, :32] = 0.0
    if N > 1:
        v[:, 1, :32] = np.tile([6, -.25, .75, 1.25, -1.75, 2.5, 3.5, 5], 4) * 2.0 ** 9    # ties
        v[:, 1, 0] = 7.0 * 2.0 ** 9                                                        # saturates
    if N > 2:
        v[:, 2, :32] = 2.0 ** -130 * np.arange(32)            # subnormal in both types
    if N > 3:
        v[:, 3, 3] = np.inf
        v[:, 3, K - 1] = np.nan
    if N > 4:
        v[:, 4, :32] = 3.3e38
        v[:, 4, 1] = -0.0
    return torch.from_numpy(v).to(dtype)


@gpu
@pytest.mark.parametrize("G,N,K", [(1, 1, 32), (1, 5, 96), (2, 33, 256), (3, 129, 288), (1, 200, 544), (5, 7, 1056)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_quantise_bit_exact(G, N, K, dtype, pad):
    need_gpu()
    rng = np.random.default_rng(G * 1000 + N + K + pad)
    src = nasty(rng, G, N, K, dtype)
    full = torch.full((G, N, K + pad), 1e30, dtype=dtype, device=DEV)
    full[:, :, :K] = src.to(DEV)
    packed = quantise(full[:, :, :K])
    codes, b = ref_quantise(src.double().numpy())
    gc, gb = unpack(packed, G, N, K)
    np.testing.assert_array_equal(gb, b)
    live = np.repeat(b != 255, 32, axis=-1)
    np.testing.assert_array_equal(gc[live], codes[live])
    want = ref_values(codes, b)
    np.testing.assert_array_equal(values_of(packed, G, N, K).double().cpu().numpy(), want.astype(np.float32))
    got16 = values_of(packed, G, N, K, torch.bfloat16).cpu()
    np.testing.assert_array_equal(got16.double().numpy(),
                                  torch.from_numpy(want).float().to(torch.bfloat16).double().numpy())
    # the padding of the last tiles: zero codes, scale 1
    raw = packed.cpu().numpy()[256:].reshape(G, -(-N // 128), -(-K // 256), 17408)
    if N % 128:
        r = N % 128
        o = r * 128
        assert (raw[:, -1, :, o:16384] == 0).all()
    assert chord.chord_get_device_error() == 0


@gpu
@pytest.mark.parametrize("G,N,K", [(1, 1, 32), (2, 33, 256), (3, 129, 288), (1, 200, 544), (2, 128, 1056)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padding_of_the_last_tiles(G, N, K, dtype):
    """Every byte that belongs to no row or no group: zero codes and the scale 1, which the
    products and the layer rely on (a NaN scale there would make NaN of zero codes)."""
    need_gpu()
    rng = np.random.default_rng(N + K)
    packed = quantise(nasty(rng, G, N, K, dtype).to(DEV))
    raw = packed.cpu().numpy()[256:].reshape(G, -(-N // 128), -(-K // 256), 17408)
    for r in range(raw.shape[1] * 128):
        for j in range(raw.shape[2] * 8):
            if r < N and 32 * j < K:
                continue
            t, q, jj = raw[:, r // 128, j // 8], r % 128, j % 8
            o = q * 128 + 16 * (jj ^ (q % 8))
            assert (t[:, o:o + 16] == 0).all()
            assert (t[:, 16384 + 512 * (jj // 4) + 16 * (q % 32) + 4 * (q // 32) + jj % 4] == 127).all()


@gpu
@pytest.mark.parametrize("div", [1, 2])
def test_padding_columns_of_routed_rows(div):
    """The same for the columns past K of rows quantised in routed order."""
    need_gpu()
    T, K, bm, E = 20, 288, 16, 3
    g = torch.Generator().manual_seed(div)
    ids = torch.rand(T, E, generator=g).argsort(dim=1)[:, :div].to(torch.int32).contiguous()
    s, _, n = align(ids.to(DEV), E, bm)
    xq = torch.full((chord.chord_mxfp4_rows_bytes(s.numel(), bm, K),), 0xFF, dtype=torch.uint8, device=DEV)
    chord.chord_mxfp4_quantize_rows(torch.randn(T, K, generator=g).to(DEV), div, s, n, bm, T * div, xq)
    G = s.numel() // bm
    raw = xq.cpu().numpy()[256:chord.chord_mxfp4_bytes(G, bm, K)].reshape(G, 2, 17408)
    pos = s[:int(n)].cpu().numpy()
    for i in np.nonzero(pos < T * div)[0]:
        t, q = raw[i // bm, 1], i % bm
        for jj in range(1, 8):
            o = q * 128 + 16 * (jj ^ (q % 8))
            assert (t[o:o + 16] == 0).all()
            assert t[16384 + 512 * (jj // 4) + 16 * (q % 32) + 4 * (q // 32) + jj % 4] == 127


@gpu
def test_matrices_past_32_bits():
    """More than 2^31 values in a matrix and in its dequantised form, more than 2^31 results of
    a product: the last rows are as right as the first."""
    need_gpu()
    one = torch.randn(1, 4100, 7200, device=DEV, dtype=torch.bfloat16)
    G = 75
    assert G * one.numel() > 2 ** 31
    packed = quantise(one.expand(G, 4100, 7200))
    alone = quantise(one)[256:]
    assert torch.equal(packed[256:].view(G, -1), alone.expand(G, -1))
    out = torch.empty((G, 4100, 7200), dtype=torch.bfloat16, device=DEV)
    chord.chord_mxfp4_dequantize(packed, out)
    want = values_of(quantise(one), 1, 4100, 7200, torch.bfloat16)[0]
    for i in (0, 36, 73, G - 1):
        assert torch.equal(out[i], want)
    del out, packed
    M, N, K = 70000, 32000, 64
    assert M * N > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(3)
    vals = torch.tensor([0., 1, -1, 2, -2, 3, -3, 4, 6, -6, .5, 1.5], device=DEV)
    a, w = (vals[torch.randint(0, 12, (1, n, K), generator=g, device=DEV)] for n in (M, N))
    a[:, :, ::32] = 4.0
    w[:, :, 31::32] = -4.0
    C = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    chord.chord_mxfp4_gemm(quantise(a), M, quantise(w), N, K, C)
    for lo in (0, 34000, 67100, M - 500):
        assert torch.equal(C[lo:lo + 500], (a[0, lo:lo + 500].double() @ w[0].double().T).to(torch.bfloat16))
    assert chord.chord_get_device_error() == 0


@gpu
def test_quantise_strided_groups_and_broadcast():
    need_gpu()
    big = torch.randn(4, 6, 40, 64, device=DEV)
    src = big[:, 2]                                   # matrix stride larger than a matrix
    p = quantise(src)
    c, b = ref_quantise(src.double().cpu().numpy())
    gc, gb = unpack(p, 4, 40, 64)
    np.testing.assert_array_equal(gc, c)
    np.testing.assert_array_equal(gb, b)
    one = torch.randn(1, 40, 64, device=DEV, dtype=torch.bfloat16)
    np.testing.assert_array_equal(values_of(quantise(one.expand(3, 40, 64)), 3, 40, 64).cpu().numpy(),
                                  values_of(quantise(one), 1, 40, 64).expand(3, 40, 64).cpu().numpy())
    with pytest.raises(chord.ChordError):
        chord.chord_mxfp4_quantize(one.transpose(1, 2), p)


@gpu
def test_empty_matrices():
    need_gpu()
    for G, N in ((0, 5), (2, 0)):
        p = quantise(torch.empty(G, N, 64, device=DEV))
        assert values_of(p, G, N, 64).numel() == 0
    w = quantise(torch.randn(1, 40, 64, device=DEV))
    C = torch.empty(0, 40, device=DEV)
    chord.chord_mxfp4_gemm(quantise(torch.empty(1, 0, 64, device=DEV)), 0, w, 40, 64, C)
    assert chord.chord_get_device_error() == 0


@gpu
def test_header_mismatch_is_reported():
    need_gpu()
    p = quantise(torch.randn(1, 256, 64, device=DEV))
    out = torch.full((1, 128, 320), 7.0, device=DEV)          # the same bytes, another shape
    chord.chord_mxfp4_dequantize(p, out)
    assert chord.chord_get_device_error() == 3 and (out == 7).all()
    a = quantise(torch.randn(1, 16, 320, device=DEV))
    C = torch.full((16, 128), 7.0, device=DEV)
    with pytest.raises(chord.ChordError) as ei:
        chord.chord_mxfp4_gemm(a, 16, p, 128, 320, C, opts=chord.ChordOpts(validate=1))
    assert ei.value.status == 6 and (C == 7).all()


# -------------------------------------------------------------------- GPU: product

def bound(av, wv, K):
    return (K / 64 + 2) * 2.0 ** -22 * (np.abs(av) @ np.abs(wv).T)


def check(got, ref, tol, what=""):
    """got (bf16 or float32 tensor) within tol of ref before its last rounding."""
    lo, hi = (torch.from_numpy(v).to(got.dtype).double().numpy() for v in (ref - tol, ref + tol))
    got = got.double().cpu().numpy()
    ok = (lo <= got) & (got <= hi)
    assert ok.all(), f"{what}: {np.argwhere(~ok)[:4].tolist()} got {got[~ok][:4]} ref {ref[~ok][:4]}"


SHAPES = [(1, 1, 32), (1, 128, 256), (3, 17, 64), (16, 200, 288), (31, 129, 96), (64, 256, 512), (65, 1003, 2080),
          (128, 130, 1024), (191, 257, 352), (193, 384, 256), (300, 129, 800), (448, 100, 1536)]


@gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dense_product(M, N, K, dtype):
    need_gpu()
    g = torch.Generator().manual_seed(M * 7 + N + K)
    a = (torch.randn(1, M, K, generator=g) * torch.exp2(torch.randint(-6, 6, (1, M, 1), generator=g).float())).to(DEV)
    w = (torch.randn(1, N, K, generator=g) * 0.05).to(torch.bfloat16).to(DEV)
    aq, wq = quantise(a), quantise(w)
    C = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
    chord.chord_mxfp4_gemm(aq, M, wq, N, K, C)
    av = ref_values(*ref_quantise(a[0].double().cpu().numpy()))
    wv = ref_values(*ref_quantise(w[0].double().cpu().numpy()))
    ref = av @ wv.T
    check(C, ref, bound(av, wv, K))
    assert chord.chord_get_device_error() == 0


@gpu
@pytest.mark.parametrize("M,N,K", [(5, 300, 7168), (130, 140, 2048), (224, 128, 288)])
def test_dense_product_exact_regime(M, N, K):
    """Small integers with scale 1: every sum is exact, so equality; each row
    and column is different, so a misplaced row, column or group shows."""
    need_gpu()
    g = torch.Generator().manual_seed(K)
    vals = torch.tensor([0., 1, -1, 2, -2, 3, -3, 4, 6, -6, .5, 1.5])
    a, w = (vals[torch.randint(0, 12, (1, n, K), generator=g)] for n in (M, N))
    a[:, :, ::32] = 4.0
    w[:, :, 31::32] = -4.0          # the largest of each group is 4 or 6: scale 1
    sa = 2.0 ** torch.randint(-3, 4, (1, M, K // 32, 1), generator=g).float()
    sw = 2.0 ** torch.randint(-2, 3, (1, N, K // 32, 1), generator=g).float()
    for xa, xw in ((a, w), ((a.view(1, M, -1, 32) * sa).view(1, M, K), w),
                   (a, (w.view(1, N, -1, 32) * sw).view(1, N, K))):
        C = torch.empty((M, N), device=DEV)
        chord.chord_mxfp4_gemm(quantise(xa.to(DEV)), M, quantise(xw.to(DEV)), N, K, C)
        np.testing.assert_array_equal(C.double().cpu().numpy(), (xa[0].double() @ xw[0].double().T).numpy())


@gpu
@pytest.mark.parametrize("M,N,K", [(840, 4900, 4640), (64, 20500, 2080)])
def test_dense_product_many_items(M, N, K):
    """More blocks of C than resident CTAs or pairs of CTAs, and more K stages than
    any ring holds, in the exact regime (sums below 36 * K < 2^24)."""
    need_gpu()
    g = torch.Generator(device=DEV).manual_seed(M)
    vals = torch.tensor([0., 1, -1, 2, -2, 3, -3, 4, 6, -6, .5, 1.5], device=DEV)
    a, w = (vals[torch.randint(0, 12, (1, n, K), generator=g, device=DEV)] for n in (M, N))
    a[:, :, ::32] = 4.0
    w[:, :, 31::32] = -4.0
    C = torch.empty((M, N), device=DEV)
    aq, wq = quantise(a), quantise(w)
    for _ in range(2):
        C.fill_(float("nan"))
        chord.chord_mxfp4_gemm(aq, M, wq, N, K, C)
        assert torch.equal(C.double(), a[0].double() @ w[0].double().T)
    assert chord.chord_get_device_error() == 0


@gpu
@pytest.mark.parametrize("M,N,K", [(96, 200, 256), (97, 640, 2304), (208, 1100, 7200), (1000, 3000, 1312), (2500, 388, 4640)])
def test_pairs_of_ctas_repeat_bit_for_bit(M, N, K):
    """Blocks that run in pairs of CTAs (dense blocks of 128 or 192 rows, an odd or even
    number of 128-row tiles of N, odd and even numbers of K stages up to more than any
    ring holds): exact in every one of many calls, other work between them."""
    need_gpu()
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    vals = torch.tensor([0., 1, -1, 2, -2, 3, -3, 4, 6, -6, .5, 1.5], device=DEV)
    a, w = (vals[torch.randint(0, 12, (1, n, K), generator=g, device=DEV)] for n in (M, N))
    a[:, :, ::32] = 4.0
    w[:, :, 31::32] = -4.0
    aq, wq = quantise(a), quantise(w)
    want = (a[0].double() @ w[0].double().T).float()
    C = torch.empty((M, N), device=DEV)
    noise = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    for i in range(30):
        C.fill_(float("nan"))
        if i % 3 == 0:
            noise.fill_(i)                       # the operands leave part of L2
        chord.chord_mxfp4_gemm(aq, M, wq, N, K, C)
        assert torch.equal(C, want), i
    assert chord.chord_get_device_error() == 0


@gpu
@pytest.mark.parametrize("bm", [96, 112, 160, 208])
@pytest.mark.parametrize("N,K", [(384, 544), (640, 2080), (1000, 4096)])
def test_grouped_pairs_of_ctas(bm, N, K):
    """Grouped blocks that run in pairs: full, ragged and nearly empty blocks of one
    call, exact regime."""
    need_gpu()
    g = torch.Generator().manual_seed(bm + N + K)
    vals = torch.tensor([0., 1, -1, 2, -2, 3, -3, 4, 6, -6, .5, 1.5])
    E, counts = 9, [bm, 1, 0, 2 * bm + 17, bm - 8, 16, bm + 1, 129, 64]
    flat = torch.tensor([e for e, c in enumerate(counts) for _ in range(c)], dtype=torch.int32)
    flat = flat[torch.randperm(flat.numel(), generator=g)]
    T = flat.numel()
    x, w = vals[torch.randint(0, 12, (T, K), generator=g)], vals[torch.randint(0, 12, (E, N, K), generator=g)]
    x[:, ::32] = 4.0
    w[:, :, 31::32] = -4.0
    s, e, n = align(flat.view(T, 1).to(DEV), E, bm)
    xq = torch.full((chord.chord_mxfp4_rows_bytes(s.numel(), bm, K),), 0xFF, dtype=torch.uint8, device=DEV)
    wq = quantise(w.to(DEV))
    xd, wd, fd = x.to(DEV).double(), w.to(DEV).double(), flat.to(DEV)
    want = torch.empty((T, N), dtype=torch.float64, device=DEV)
    for ex in range(E):
        want[fd == ex] = xd[fd == ex] @ wd[ex].T
    for _ in range(5):
        chord.chord_mxfp4_quantize_rows(x.to(DEV), 1, s, n, bm, T, xq)
        C = torch.full((T, N), float("nan"), device=DEV)
        chord.chord_mxfp4_moe_gemm(xq, wq, E, N, K, s, e, n, bm, T, C)
        assert torch.equal(C.double(), want)
    assert chord.chord_get_device_error() == 0


@gpu
def test_dense_product_extreme_scales():
    """Scales far from 1 on both sides: powers of two that cancel, and NaN
    scales that stay in their row and column."""
    need_gpu()
    g = torch.Generator().manual_seed(5)
    a, w = torch.randn(1, 40, 256, generator=g), torch.randn(1, 150, 256, generator=g)
    aq, wq = quantise((a * 2.0 ** 60).to(DEV)), quantise((w * 2.0 ** -60).to(DEV))
    C = torch.empty((40, 150), device=DEV)
    chord.chord_mxfp4_gemm(aq, 40, wq, 150, 256, C)
    av, wv = (ref_values(*ref_quantise(t[0].double().numpy())) for t in (a, w))
    check(C, av @ wv.T, bound(av, wv, 256))
    a[0, 7, 100] = float("nan")
    w[0, 33, 255] = float("inf")
    chord.chord_mxfp4_gemm(quantise(a.to(DEV)), 40, quantise(w.to(DEV)), 150, 256, C)
    nan = torch.isnan(C).cpu().numpy()
    want = np.zeros((40, 150), bool)
    want[7, :] = True
    want[:, 33] = True
    np.testing.assert_array_equal(nan, want)


def align(ids, E, bm):
    T, topk = ids.shape
    cap = chord.chord_align_capacity(T, topk, E, bm)
    s = torch.empty(cap, dtype=torch.int32, device=DEV)
    e = torch.empty(cap // bm, dtype=torch.int32, device=DEV)
    n = torch.empty(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(chord.chord_align_workspace_bytes(T, topk, E), dtype=torch.uint8, device=DEV)
    chord.chord_moe_align(ids, E, bm, s, e, n, ws)
    return s, e, n


@gpu
@pytest.mark.parametrize("T,E,topk,N,K,bm,div", [
    (1, 4, 1, 128, 256, 32, 1), (3, 8, 2, 200, 96, 32, 2), (40, 3, 2, 129, 288, 64, 1), (50, 2, 1, 256, 512, 96, 1),
    (200, 2, 2, 130, 320, 128, 2), (150, 1, 1, 140, 64, 160, 1), (300, 4, 2, 260, 1056, 192, 2),
    (250, 1, 1, 128, 256, 208, 1), (500, 3, 2, 384, 800, 208, 2), (30, 3, 2, 150, 544, 16, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped_product(T, E, topk, N, K, bm, div, dtype):
    need_gpu()
    g = torch.Generator().manual_seed(T + N + K)
    keys = torch.rand(T, max(E, topk), generator=g)
    ids = keys.argsort(dim=1)[:, :topk].to(torch.int32)
    ids[torch.rand(T, topk, generator=g) < 0.15] = -1            # other GPUs' experts
    if T > 2:
        ids[1] = -1
    P = T * topk
    x = torch.randn(P // div, K, generator=g).to(torch.bfloat16)
    w = torch.randn(E, N, K, generator=g) * 0.1
    s, e, n = align(ids.to(DEV), E, bm)
    xq = torch.full((chord.chord_mxfp4_rows_bytes(s.numel(), bm, K),), 0xFF, dtype=torch.uint8, device=DEV)
    chord.chord_mxfp4_quantize_rows(x.to(DEV), div, s, n, bm, P, xq)
    C = torch.full((P, N), 77.0, dtype=dtype, device=DEV)
    chord.chord_mxfp4_moe_gemm(xq, quantise(w.to(DEV)), E, N, K, s, e, n, bm, P, C)
    assert chord.chord_get_device_error() == 0
    got = C.double().cpu().numpy()
    xv = ref_values(*ref_quantise(x.double().numpy()))
    flat = ids.view(-1).numpy()
    assert (got[flat < 0] == 77).all()                            # no block names them
    for ex in range(E):
        rows = np.nonzero(flat == ex)[0]
        wv = ref_values(*ref_quantise(w[ex].double().numpy()))
        av = xv[rows // div]
        ref = av @ wv.T
        check(C[torch.from_numpy(rows).to(DEV)], ref, bound(av, wv, K), f"expert {ex}")


@gpu
@pytest.mark.parametrize("topk", [3, 17, 40])
def test_quantised_rows_of_shared_tokens(topk):
    """Rows shared by many pairs, some without a position; and routing arrays
    that name a few pairs of many.  Every routed position holds its row."""
    need_gpu()
    T, E, K, bm = 9, 50, 352, 16
    g = torch.Generator().manual_seed(topk)
    x = torch.randn(T, K, generator=g)
    c, b = ref_quantise(x.double().numpy())
    ids = torch.rand(T, E, generator=g).argsort(dim=1)[:, :topk].to(torch.int32)
    ids[torch.rand(T, topk, generator=g) < 0.3] = -1
    s, e, n = align(ids.to(DEV), E, bm)
    few = torch.full((32,), T * topk, dtype=torch.int32, device=DEV)       # 32 positions, up to 360 pairs
    few[:5] = torch.tensor([0, topk, 2 * topk + 1, 4 * topk, T * topk - 1], dtype=torch.int32)
    few[16] = 3 * topk + 2
    for order, cnt in ((s, n), (few, torch.tensor([32], dtype=torch.int32, device=DEV))):
        xq = torch.full((chord.chord_mxfp4_rows_bytes(order.numel(), bm, K),), 0x11, dtype=torch.uint8, device=DEV)
        chord.chord_mxfp4_quantize_rows(x.to(DEV), topk, order, cnt, bm, T * topk, xq)
        assert chord.chord_get_device_error() == 0
        G = order.numel() // bm
        gc, gb = unpack(xq[:chord.chord_mxfp4_bytes(G, bm, K)], G, bm, K)
        pos = order[:int(cnt)].cpu().numpy()
        at = np.nonzero(pos < T * topk)[0]
        assert at.size
        np.testing.assert_array_equal(gc.reshape(-1, K)[at], c[pos[at] // topk])
        np.testing.assert_array_equal(gb.reshape(-1, K // 32)[at], b[pos[at] // topk])


@gpu
def test_grouped_product_reports_bad_routing():
    need_gpu()
    E, N, K, bm, P = 2, 128, 256, 32, 8
    ids = torch.tensor([[0], [1], [0], [1], [0], [1], [0], [0]], dtype=torch.int32, device=DEV)
    s, e, n = align(ids, E, bm)
    x = torch.randn(P, K, device=DEV)
    xq = torch.zeros(chord.chord_mxfp4_rows_bytes(s.numel(), bm, K), dtype=torch.uint8, device=DEV)
    wq = quantise(torch.randn(E, N, K, device=DEV))
    chord.chord_mxfp4_quantize_rows(x, 1, s, n, bm, P, xq)
    good = torch.zeros(P, N, device=DEV)
    chord.chord_mxfp4_moe_gemm(xq, wq, E, N, K, s, e, n, bm, P, good)
    assert chord.chord_get_device_error() == 0
    for arr, at, v, code in ((e, 0, 9, 1), (s, 1, -3, 2), (s, 1, 900, 2), (n, 0, 33, 6), (n, 0, 32 * 100, 6)):
        keep = arr[at].clone()
        arr[at] = v
        C = torch.zeros(P, N, device=DEV)
        chord.chord_mxfp4_moe_gemm(xq, wq, E, N, K, s, e, n, bm, P, C)
        assert chord.chord_get_device_error() == code, (v, code)
        arr[at] = keep
        same = (C == good).all(dim=1)
        assert (same | (C == 0).all(dim=1)).all()


@gpu
@pytest.mark.parametrize("div", [1, 2])
@pytest.mark.parametrize("bad", [None, -3, 900])
def test_rows_that_ids_do_not_have_are_reported(div, bad):
    """A pair whose row lies past A (fewer rows than pairs / divisor), and ids that are no
    pair: CHORD_DEV_BAD_ROW, as the INT4 product reports them; the other rows are right."""
    need_gpu()
    T, K, bm, E = 8, 96, 16, 2
    ids = torch.tensor([[t % E, (t + 1) % E][:div] for t in range(T)], dtype=torch.int32, device=DEV)
    P = T * div
    s, e, n = align(ids, E, bm)
    x = torch.randn(T, K, device=DEV)
    have = T
    if bad is None:
        have = T - 3
    else:
        s[0] = bad
    xq = torch.zeros(chord.chord_mxfp4_rows_bytes(s.numel(), bm, K), dtype=torch.uint8, device=DEV)
    chord.chord_mxfp4_quantize_rows(x[:have], div, s, n, bm, P, xq)
    assert chord.chord_get_device_error() == 2
    G = s.numel() // bm
    gc, gb = unpack(xq[:chord.chord_mxfp4_bytes(G, bm, K)], G, bm, K)
    c, b = ref_quantise(x.double().cpu().numpy())
    pos = s[:int(n)].cpu().numpy()
    at = np.nonzero((pos >= 0) & (pos < have * div))[0]
    np.testing.assert_array_equal(gc.reshape(-1, K)[at], c[pos[at] // div])
    np.testing.assert_array_equal(gb.reshape(-1, K // 32)[at], b[pos[at] // div])
    chord.chord_mxfp4_quantize_rows(x, div, align(ids, E, bm)[0], n, bm, P, xq)
    assert chord.chord_get_device_error() == 0


@gpu
def test_product_on_its_own_stream_and_in_a_graph():
    need_gpu()
    a, w = torch.randn(1, 70, 512, device=DEV), torch.randn(1, 300, 512, device=DEV)
    want = torch.empty(70, 300, device=DEV)
    chord.chord_mxfp4_gemm(quantise(a), 70, quantise(w), 300, 512, want)
    aq = torch.empty(chord.chord_mxfp4_bytes(1, 70, 512), dtype=torch.uint8, device=DEV)
    wq, C = quantise(w), torch.zeros(70, 300, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    chord.chord_mxfp4_quantize(a, aq, stream=st)
    chord.chord_mxfp4_gemm(aq, 70, wq, 300, 512, C, stream=st)
    st.synchronize()
    assert torch.equal(C, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chord.chord_mxfp4_quantize(a, aq)
        chord.chord_mxfp4_gemm(aq, 70, wq, 300, 512, C)
    a.mul_(2.0)                       # a power of two: the result doubles exactly
    for _ in range(2):
        C.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, 2.0 * want)
