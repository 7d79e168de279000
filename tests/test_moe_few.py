"""The mixture-of-experts layer for a few tokens against its formula in
binary64, and its refusals.

Tolerance, derived element by element.  The weights are bf16 numbers and x is
bf16, so products are exact in FP32; with chopping in every addition of a K = 16
step the gate and up sums are off by at most c(H) * sum |x w|, c(K) = (K / 16 +
40) * 2^-22 (40: partial sums joined at the end).  SiLU's slope is below 1.1
and its own FP32 evaluation is good to 2^-18; h is carried with at least 16
significant bits (2^-16).  The down sum adds c(I topk) * sum |w2 h|.  The bf16 output
lies between the bf16 roundings of the two ends of that interval."""
import ctypes

import numpy as np
import pytest
import torch

import w4a16_int4_mixture_moe_gb300 as chord

DEV = "cuda:0"
gpu = pytest.mark.gpu
MAG = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    chord.build()
    chord.load()
    chord.chord_get_device_error()


def make_weights(fmt, E, N, K, g, wide=False, scales=None):
    """(values float64 [E, N, K], pack(layout) -> device blob); scales: INT4 scales to use"""
    codes = torch.randint(0, 16, (E, N, K), generator=g, dtype=torch.uint8)
    if fmt == "int4":
        s = (torch.randn((E, N, K // 32), generator=g).abs() * 0.02 + 1e-3)
        if wide:     # scales outside the one-FMA dequantisation's range
            s[:, ::3] *= 64.0
            s[:, 1::5] = -s[:, 1::5]
        s = (s if scales is None else scales).to(torch.bfloat16)
        v = ((codes.double() - 8) * s.double().repeat_interleave(32, -1)).float().to(torch.bfloat16).double()

        def pack(layout=chord.LAYOUT_TCGEN05):
            blob = torch.empty(chord.chord_packed_weight_bytes(E, N, K, layout), dtype=torch.uint8, device=DEV)
            chord.chord_pack_weights(codes.to(DEV), s.to(DEV), blob, layout=layout)
            return blob
    else:
        lo, hi = (60, 190) if wide else (118, 123)
        b = torch.randint(lo, hi, (E, N, K // 32), generator=g)
        if wide:     # large and tiny groups side by side, every one representable
            b = 120 + (b - 120) // 8
        v = MAG[(codes & 7).long()] * (1.0 - 2.0 * (codes >> 3).double())
        v = v * torch.exp2(b.double() - 127).repeat_interleave(32, -1)

        def pack(layout=None):
            blob = torch.empty(chord.chord_mxfp4_bytes(E, N, K), dtype=torch.uint8, device=DEV)
            chord.chord_mxfp4_quantize(v.float().to(DEV), blob)
            return blob
    return v, pack


def reference(x, ids, w, v13, v2):
    """Output in binary64 and the element-wise bound described above."""
    T, H = x.shape
    E, _, I = v2.shape
    out = torch.zeros((T, H), dtype=torch.float64)
    tol = torch.zeros((T, H), dtype=torch.float64)

    def c(k):
        return (k / 16 + 40) * 2.0 ** -22

    mag = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            if not 0 <= e < E:
                continue
            xt = x[t].double()
            gu, s = v13[e] @ xt, v13[e].abs() @ xt.abs() * c(H)
            g, u, eg, eu = gu[:I], gu[I:], s[:I], s[I:]
            silu = g * torch.sigmoid(g)
            wt = float(w[t, k])
            h = wt * silu * u
            eh = abs(wt) * (1.1 * eg * (u.abs() + eu) + silu.abs() * eu) + h.abs() * (2.0 ** -16 + 2.0 ** -18)
            out[t] += v2[e] @ h
            tol[t] += v2[e].abs() @ eh
            mag[t] += v2[e].abs() @ (h.abs() + eh)
    tol += mag * c(I * ids.shape[1])
    return out, tol


def run(x, ids, w, E, I, b13, b2, fmt, **kw):
    T, H = x.shape
    ws = torch.full((chord.chord_moe_few_workspace_bytes(T, ids.shape[1], E, H, I),), 0xFF, dtype=torch.uint8,
                    device=DEV)                         # NaN bit patterns: nothing may be read before it is written
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    chord.chord_moe_layer_few(x.to(DEV), ids.to(DEV), w.to(DEV), E, I, b13, b2, ws, out,
                              weights=chord.WEIGHTS_INT4 if fmt == "int4" else chord.WEIGHTS_MXFP4, **kw)
    return out


def check(out, ref, tol):
    lo, hi = ((ref + s * tol).to(torch.bfloat16).double() for s in (-1, 1))
    got = out.double().cpu()
    bad = ~((lo <= got) & (got <= hi))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}: got {got[bad][:4]} ref {ref[bad][:4]} tol {tol[bad][:4]}"


def routing(T, E, topk, g, Eg=None):
    Eg = Eg or E
    ids = torch.rand(T, Eg, generator=g).argsort(dim=1)[:, :topk].to(torch.int32)
    ids[ids >= E] = -1
    w = torch.softmax(torch.randn(T, topk, generator=g), dim=1)
    return ids, w


CASES = [  # T, E, Eg, topk, H, I
    (1, 1, 1, 1, 128, 64), (1, 8, 8, 2, 256, 128), (1, 4, 4, 4, 7168, 64), (2, 3, 6, 3, 384, 192),
    (5, 16, 16, 4, 640, 320), (8, 4, 4, 2, 256, 2048), (9, 8, 8, 8, 512, 64), (16, 8, 8, 2, 256, 128),
    (17, 2, 2, 1, 1152, 128), (24, 40, 80, 6, 256, 64), (32, 5, 5, 5, 2176, 192), (32, 64, 64, 8, 128, 64)]


@gpu
@pytest.mark.parametrize("T,E,Eg,topk,H,I", CASES)
@pytest.mark.parametrize("fmt,layout", [("int4", 2), ("int4", 3), ("mxfp4", 4)])
def test_against_formula(T, E, Eg, topk, H, I, fmt, layout):
    need_gpu()
    g = torch.Generator().manual_seed(T * 31 + E + H + I)
    v13, p13 = make_weights(fmt, E, 2 * I, H, g)
    v2, p2 = make_weights(fmt, E, H, I, g)
    ids, w = routing(T, E, topk, g, Eg)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    b13, b2 = p13(layout), p2()
    out = run(x, ids, w, E, I, b13, b2, fmt)
    assert chord.chord_get_device_error() == 0
    ref, tol = reference(x, ids, w, v13, v2)
    check(out, ref, tol)
    again = run(x, ids, w, E, I, b13, b2, fmt)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@gpu
@pytest.mark.parametrize("H,I", [(32, 32), (96, 32), (288, 96), (800, 160), (1056, 352)])
@pytest.mark.parametrize("T", [1, 7, 20])
def test_mxfp4_odd_sizes(T, H, I):
    need_gpu()
    g = torch.Generator().manual_seed(H + I + T)
    E, topk = 5, 3
    v13, p13 = make_weights("mxfp4", E, 2 * I, H, g)
    v2, p2 = make_weights("mxfp4", E, H, I, g)
    ids, w = routing(T, E, topk, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    out = run(x, ids, w, E, I, p13(), p2(), "mxfp4")
    check(out, *reference(x, ids, w, v13, v2))
    assert chord.chord_get_device_error() == 0


@gpu
@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_wide_scales(fmt):
    need_gpu()
    g = torch.Generator().manual_seed(11)
    T, E, topk, H, I = 6, 4, 2, 256, 128
    v13, p13 = make_weights(fmt, E, 2 * I, H, g, wide=True)
    v2, p2 = make_weights(fmt, E, H, I, g, wide=True)
    ids, w = routing(T, E, topk, g)
    x = (torch.randn(T, H, generator=g) * 0.05).to(torch.bfloat16)
    check(run(x, ids, w, E, I, p13(), p2(), fmt), *reference(x, ids, w, v13, v2))


@gpu
@pytest.mark.parametrize("lo,hi", [(-126, -116), (-119, -117), (-8, -2)])
def test_int4_scales_at_the_ends_of_the_normal_range(lo, hi):
    """Scales from the smallest normal number on, and up to 1/2, one per group
    at random: every weight is exact, so the bound is the usual one."""
    need_gpu()
    g = torch.Generator().manual_seed(-lo)
    T, E, topk, H, I = 5, 3, 2, 384, 192
    def scales(N, K):
        return torch.exp2(torch.randint(lo, hi + 1, (E, N, K // 32), generator=g).double()) * (
            1 + torch.randint(0, 128, (E, N, K // 32), generator=g).double() / 128)
    v13, p13 = make_weights("int4", E, 2 * I, H, g, scales=scales(2 * I, H).clamp(max=0.498))
    v2, p2 = make_weights("int4", E, H, I, g, scales=scales(H, I).clamp(max=0.498))
    ids, w = routing(T, E, topk, g)
    x = (torch.randn(T, H, generator=g) * 2.0 ** -(hi + 5)).to(torch.bfloat16)
    for layout in (2, 3):
        check(run(x, ids, w, E, I, p13(layout), p2(), "int4"), *reference(x, ids, w, v13, v2))


@gpu
@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_routing_edges(fmt):
    """Tokens without a local expert, one expert with every token, an expert
    named twice by a token, NaN weights of skipped choices, ids out of range."""
    need_gpu()
    g = torch.Generator().manual_seed(3)
    T, E, topk, H, I = 32, 6, 3, 256, 64
    v13, p13 = make_weights(fmt, E, 2 * I, H, g)
    v2, p2 = make_weights(fmt, E, H, I, g)
    b13, b2 = p13(), p2()
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    w = torch.softmax(torch.randn(T, topk, generator=g), dim=1)
    ids = torch.full((T, topk), -1, dtype=torch.int32)
    out = run(x, ids, torch.full_like(w, float("nan")), E, I, b13, b2, fmt)
    assert (out.view(torch.int16) == 0).all()                      # +0 everywhere
    ids[:, 1] = 4                                                  # one expert, all tokens
    wn = w.clone()
    wn[:, 0] = float("nan")
    wn[:, 2] = float("inf")
    check(run(x, ids, wn, E, I, b13, b2, fmt), *reference(x, ids, w, v13, v2))
    ids[:, 2] = 4                                                  # named twice
    ids[5] = -1
    ids[7, 0] = 0
    check(run(x, ids, w, E, I, b13, b2, fmt), *reference(x, ids, w, v13, v2))
    assert chord.chord_get_device_error() == 0
    ids[9, 0] = E                                                  # skipped, reported when validating
    ids[10, 0] = -7
    ref = reference(x, ids, w, v13, v2)
    check(run(x, ids, w, E, I, b13, b2, fmt), *ref)
    assert chord.chord_get_device_error() == 0
    with pytest.raises(chord.ChordError) as ei:
        run(x, ids, w, E, I, b13, b2, fmt, opts=chord.ChordOpts(validate=1))
    assert ei.value.status == 6


@gpu
def test_infinite_activation_stays_in_its_token():
    need_gpu()
    g = torch.Generator().manual_seed(8)
    T, E, topk, H, I = 4, 3, 2, 256, 128
    _, p13 = make_weights("int4", E, 2 * I, H, g)
    _, p2 = make_weights("int4", E, H, I, g)
    b13, b2 = p13(), p2()
    ids, w = routing(T, E, topk, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    clean = run(x, ids, w, E, I, b13, b2, "int4")
    x[2, 17] = float("nan")
    got = run(x, ids, w, E, I, b13, b2, "int4")
    assert torch.isnan(got[2]).all()
    keep = [0, 1, 3]
    assert torch.equal(got[keep], clean[keep])


@gpu
def test_agrees_with_the_layer():
    """chord_moe_layer rounds the gate_up result and SiLU * up to bf16; the
    two differ by that propagation only (a few bf16 steps of the output's
    scale)."""
    need_gpu()
    g = torch.Generator().manual_seed(21)
    T, E, topk, H, I = 16, 8, 2, 512, 256
    _, p13 = make_weights("int4", E, 2 * I, H, g)
    _, p2 = make_weights("int4", E, H, I, g)
    b13, b2 = p13(), p2()
    ids, w = routing(T, E, topk, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    few = run(x, ids, w, E, I, b13, b2, "int4").double()
    ws = torch.empty(chord.chord_layer_workspace_bytes(T, topk, E, H, I, 8), dtype=torch.uint8, device=DEV)
    out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    chord.chord_moe_layer(x.to(DEV), ids.to(DEV), w.to(DEV), E, E, I, b13, b2, ws, out, block_m=8)
    scale = few.abs().mean()
    assert ((few - out.double()).abs() <= 2.0 ** -6 * (few.abs() + scale)).all()


@gpu
def test_stream_and_graph_replay():
    need_gpu()
    g = torch.Generator().manual_seed(2)
    T, E, topk, H, I = 3, 8, 2, 384, 128
    v13, p13 = make_weights("int4", E, 2 * I, H, g)
    v2, p2 = make_weights("int4", E, H, I, g)
    b13, b2 = p13(3), p2()
    ids, w = routing(T, E, topk, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    xd, idd, wd = x.to(DEV), ids.to(DEV), w.to(DEV)
    ws = torch.empty(chord.chord_moe_few_workspace_bytes(T, topk, E, H, I), dtype=torch.uint8, device=DEV)
    out = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    chord.chord_moe_layer_few(xd, idd, wd, E, I, b13, b2, ws, out, stream=st)
    st.synchronize()
    check(out, *reference(x, ids, w, v13, v2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):            # back to back on one workspace
            chord.chord_moe_layer_few(xd, idd, wd, E, I, b13, b2, ws, out)
    ids2, w2 = routing(T, E, topk, torch.Generator().manual_seed(77))
    idd.copy_(ids2)
    wd.copy_(w2)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(out, *reference(x, ids2, w2, v13, v2))


@gpu
def test_wrong_blob_is_reported_and_nothing_written():
    need_gpu()
    g = torch.Generator().manual_seed(4)
    T, E, topk, H, I = 2, 4, 2, 256, 128
    _, p13 = make_weights("int4", E, 2 * I, H, g)
    _, p2 = make_weights("int4", E, H, I, g)
    ids, w = routing(T, E, topk, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    out = run(x, ids, w, E, I, p13(), p2(3), "int4")      # w2 packed as a gate_up weight
    assert chord.chord_get_device_error() == 3
    assert torch.isnan(out).all()


@gpu
def test_refused_blob_leaves_the_stream_order_intact():
    """Work behind a call whose blob is refused comes after both of its kernels:
    the workspace keeps what is written there next, and the next call on it is right."""
    need_gpu()
    g = torch.Generator().manual_seed(6)
    T, E, topk, H, I = 16, 4, 2, 4096, 128
    v13, p13 = make_weights("int4", E, 2 * I, H, g)
    v2, p2 = make_weights("int4", E, H, I, g)
    ids, w = routing(T, E, topk, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    b13, b2, bad = p13(), p2(), p2(3)
    xd, idd, wd = x.to(DEV), ids.to(DEV), w.to(DEV)
    ws = torch.empty(chord.chord_moe_few_workspace_bytes(T, topk, E, H, I), dtype=torch.uint8, device=DEV)
    out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    for _ in range(20):
        chord.chord_moe_layer_few(xd, idd, wd, E, I, b13, bad, ws, out)
        ws.fill_(0xAB)
        assert (ws == 0xAB).all()
        chord.chord_moe_layer_few(xd, idd, wd, E, I, b13, bad, ws, out)
        chord.chord_moe_layer_few(xd, idd, wd, E, I, b13, b2, ws, out)
    assert chord.chord_get_device_error() == 3
    check(out, *reference(x, ids, w, v13, v2))


def test_refusals():
    lib = chord.load()
    vp = ctypes.c_void_p
    p = vp(1 << 20)
    T, topk, E, H, I = 4, 2, 8, 256, 128
    n13, n2 = chord.chord_packed_weight_bytes(E, 2 * I, H), chord.chord_packed_weight_bytes(E, H, I)
    ws = chord.chord_moe_few_workspace_bytes(T, topk, E, H, I)
    assert ws >= T * topk * I * 4
    assert chord.chord_moe_few_workspace_bytes(0, 0, E, H, I) == 0
    ok = [p, p, p, T, topk, E, H, I, 0, p, n13, p, n2, p, ws, p, None, None]
    for at, v, st in [(3, -1, 1), (3, 33, 2), (4, 0, 1), (4, 33, 2), (5, 0, 1), (5, 1025, 2), (6, 192, 2), (7, 96, 2),
                      (8, 2, 1), (8, 1, 3), (10, n13 + 1, 3), (12, n2 - 1, 3), (14, ws - 1, 4), (0, None, 1),
                      (1, None, 1), (2, None, 1), (9, None, 1), (11, None, 1), (13, None, 1), (15, None, 1),
                      (0, vp((1 << 20) + 2), 1), (9, vp((1 << 20) + 8), 1), (13, vp((1 << 20) + 8), 1)]:
        a = list(ok)
        a[at] = v
        assert lib.chord_moe_layer_few(*a) == st, (at, v)
    a = list(ok)
    a[6], a[7], a[8] = 48, 32, 1
    assert lib.chord_moe_layer_few(*a) == 2
