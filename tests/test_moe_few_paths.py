"""The launch plans of the layer for a few tokens that large models take, at sizes
whose formula is still quick: many experts a thread in the routing prologue, more
items than CTAs (with and without clusters), rings of two stages, list slices joined by
the last CTA; and scales, infinities and NaN where they can spread.  The bound is the
one derived in test_moe_few.

The sizes are chosen by the launch arithmetic for 152 SMs: an item is 64 columns of I
of up to eight tokens of one expert; at most 608 CTAs share the items."""
import pytest
import torch

import w4a16_int4_mixture_moe_gb300 as chord
from test_moe_few import DEV, check, make_weights, need_gpu, routing, run

gpu = pytest.mark.gpu


def reference(x, ids, w, v13, v2):
    """test_moe_few's output and bound in binary64, an expert's tokens at a time."""
    T, H = x.shape
    E, _, I = v2.shape
    topk = ids.shape[1]
    x, ids, w = x.to(DEV).double(), ids.to(DEV), w.to(DEV).double()
    out, tol, mag = (torch.zeros((T, H), dtype=torch.float64, device=DEV) for _ in range(3))

    def c(k):
        return (k / 16 + 40) * 2.0 ** -22

    for e in range(E):
        t = (ids == e).any(dim=1).nonzero().view(-1)
        if t.numel() == 0:
            continue
        a13, a2 = v13[e].to(DEV), v2[e].to(DEV)
        for k in range(topk):                        # a choice at a time, as the bound adds them
            s = t[ids[t, k] == e]
            if s.numel() == 0:
                continue
            gu, b = x[s] @ a13.T, (x[s].abs() @ a13.abs().T) * c(H)
            g, u, eg, eu = gu[:, :I], gu[:, I:], b[:, :I], b[:, I:]
            silu, wt = g * torch.sigmoid(g), w[s, k].unsqueeze(1)
            h = wt * silu * u
            eh = wt.abs() * (1.1 * eg * (u.abs() + eu) + silu.abs() * eu) + h.abs() * (2.0 ** -16 + 2.0 ** -18)
            out[s] += h @ a2.T
            tol[s] += eh @ a2.abs().T
            mag[s] += (h.abs() + eh) @ a2.abs().T
    tol += mag * c(I * topk)
    return out.cpu(), tol.cpu()


def formula(fmt, layout, T, E, topk, H, I, ids, w, seed, times=2, x=None):
    g = torch.Generator().manual_seed(seed)
    v13, p13 = make_weights(fmt, E, 2 * I, H, g)
    v2, p2 = make_weights(fmt, E, H, I, g)
    if x is None:
        x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    b13, b2 = p13(layout), p2()
    first = run(x, ids, w, E, I, b13, b2, fmt)
    assert chord.chord_get_device_error() == 0
    check(first, *reference(x, ids, w, v13, v2))
    for _ in range(times):
        assert torch.equal(run(x, ids, w, E, I, b13, b2, fmt).view(torch.int16), first.view(torch.int16))


@gpu
@pytest.mark.parametrize("fmt,layout", [("int4", 2), ("int4", 3), ("mxfp4", 4)])
@pytest.mark.parametrize("T,E,topk,H,I", [
    (16, 384, 8, 256, 128),      # three experts a thread; one-wave plan
    (1, 384, 8, 1152, 64),       # clusters of gate_up CTAs over few experts of many
    (5, 700, 6, 384, 64),
    (32, 1024, 32, 128, 64),     # the largest routing: 20 KB of tables, rings of two stages
    (8, 1024, 32, 256, 64)])
def test_many_experts(T, E, topk, H, I, fmt, layout):
    need_gpu()
    ids, w = routing(T, E, topk, torch.Generator().manual_seed(T + E))
    formula(fmt, layout, T, E, topk, H, I, ids, w, T * E)


@gpu
@pytest.mark.parametrize("fmt,layout", [("int4", 2), ("int4", 3), ("mxfp4", 4)])
@pytest.mark.parametrize("E,topk,H,I", [
    (16, 16, 640, 2560),         # 64 passes of 40 items on 608 CTAs: four items and five for some
    (8, 8, 1152, 2496)])         # 32 passes of 39: two or three; nine stages a pass
def test_more_items_than_ctas(E, topk, H, I, fmt, layout):
    """Ring positions carried from item to item, with more K stages than the ring has slots."""
    need_gpu()
    T = 32
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:topk] for t in range(T)]).to(torch.int32)
    w = torch.softmax(torch.randn(T, topk, generator=torch.Generator().manual_seed(E)), dim=1)
    formula(fmt, layout, T, E, topk, H, I, ids, w, H + I, times=3)


@gpu
@pytest.mark.parametrize("fmt,layout,H", [("int4", 2, 768), ("int4", 3, 896), ("mxfp4", 4, 1536)])
def test_clusters_that_take_a_second_item(fmt, layout, H):
    """32 tokens on 32 different experts: half as many again as an even routing hits, so
    clusters of two come round to a second item and its other join buffer."""
    need_gpu()
    T = E = 32
    ids = torch.randperm(E, generator=torch.Generator().manual_seed(9)).to(torch.int32).view(T, 1)
    w = torch.rand(T, 1, generator=torch.Generator().manual_seed(10))
    formula(fmt, layout, T, E, 1, H, 896, ids, w, H, times=5)


@gpu
@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 16, 24])
@pytest.mark.parametrize("H,I", [(256, 128), (640, 320)])
def test_lists_joined_by_the_last_cta(T, H, I, fmt):
    """Pass lists long enough for slices that are no cluster: sums through the workspace."""
    need_gpu()
    E, topk = 64, 16
    ids, w = routing(T, E, topk, torch.Generator().manual_seed(T))
    formula(fmt, 2 if fmt == "int4" else 4, T, E, topk, H, I, ids, w, T + H, times=5)


@gpu
@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
@pytest.mark.parametrize("T,H,I", [(1, 65664, 64), (9, 65664, 64), (2, 128, 16384), (1, 128, 64)])
def test_long_hidden_and_inner_sizes(T, H, I, fmt):
    """More output tiles than CTAs (a list is then one slice), and lists of one expert only."""
    need_gpu()
    ids, w = torch.zeros((T, 1), dtype=torch.int32), torch.rand(T, 1, generator=torch.Generator().manual_seed(T))
    formula(fmt, 2 if fmt == "int4" else 4, T, 1, 1, H, I, ids, w, H + I)


def mx_matrix(E, N, K, g, lo, hi):
    """MXFP4 values with scale exponents b - 127 for b in [lo, hi], one per group at random."""
    mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    codes = torch.randint(0, 16, (E, N, K), generator=g)
    codes[..., ::32] = 6                              # the largest is 4 or 6: the quantiser keeps b
    b = torch.randint(lo, hi + 1, (E, N, K // 32), generator=g)
    v = mag[codes & 7] * (1.0 - 2.0 * (codes >> 3).double())
    return v * torch.exp2(b.double() - 127).repeat_interleave(32, -1)


def mx_blob(v):
    blob = torch.empty(chord.chord_mxfp4_bytes(*v.shape), dtype=torch.uint8, device=DEV)
    chord.chord_mxfp4_quantize(v.float().to(DEV), blob)
    return blob


@gpu
@pytest.mark.parametrize("T", [1, 6, 12, 32])
@pytest.mark.parametrize("b13,b2,xe", [((112, 160), (112, 130), -25), ((118, 122), (112, 200), 0), ((112, 252), (112, 140), -120),
                                       ((127, 130), (126, 131), -4), ((1, 130), (0, 129), 0), ((125, 129), (200, 252), -40)])
def test_mxfp4_scales_of_every_size(T, b13, b2, xe):
    """Scales above 2 (which take two multiplications) beside smaller ones, up to the largest
    that the quantiser gives and down to the smallest there is."""
    need_gpu()
    g = torch.Generator().manual_seed(T + b13[1] + b2[1])
    E, topk, H, I = 4, 2, 544, 160
    v13, v2 = mx_matrix(E, 2 * I, H, g, *b13), mx_matrix(E, H, I, g, *b2)
    ids, w = routing(T, E, topk, g)
    x = (torch.randn(T, H, generator=g) * 2.0 ** xe).to(torch.bfloat16)
    out = run(x, ids, w, E, I, mx_blob(v13), mx_blob(v2), "mxfp4")
    ref, tol = reference(x, ids, w, v13, v2)
    assert torch.isfinite(ref.to(torch.bfloat16)).all()
    check(out, ref, tol)
    assert chord.chord_get_device_error() == 0


@gpu
@pytest.mark.parametrize("T", [5, 20])
def test_mxfp4_nan_blocks_stay_in_their_expert_and_row(T):
    """A block with the NaN scale in W13 makes every output of its expert's tokens NaN, one
    in W2 one output of them; nothing else changes by a bit."""
    need_gpu()
    g = torch.Generator().manual_seed(T)
    E, topk, H, I = 6, 2, 544, 160
    v13, v2 = mx_matrix(E, 2 * I, H, g, 118, 122), mx_matrix(E, H, I, g, 118, 122)
    ids, w = routing(T, E, topk, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    clean = run(x, ids, w, E, I, mx_blob(v13), mx_blob(v2), "mxfp4").cpu()
    ex = int(ids[0, 0])
    has = (ids == ex).any(dim=1)
    assert not has.all()
    for row, col in ((7, 100), (I + 159, 543), (I - 1, 0)):
        bad = v13.clone()
        bad[ex, row, col] = float("nan")
        got = run(x, ids, w, E, I, mx_blob(bad), mx_blob(v2), "mxfp4").cpu()
        assert torch.isnan(got[has]).all()
        assert torch.equal(got[~has].view(torch.int16), clean[~has].view(torch.int16))
    bad = v2.clone()
    bad[ex, 300, 33] = float("inf")                    # the quantiser gives its block the NaN scale
    got = run(x, ids, w, E, I, mx_blob(v13), mx_blob(bad), "mxfp4").cpu()
    hit = torch.zeros((T, H), dtype=torch.bool)
    hit[has, 300] = True
    assert torch.equal(torch.isnan(got), hit)
    assert torch.equal(got[~hit].view(torch.int16), clean[~hit].view(torch.int16))


@gpu
@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T", [4, 11, 30])
def test_infinity_in_an_activation_stays_in_its_token(T, value, fmt):
    need_gpu()
    g = torch.Generator().manual_seed(T)
    E, topk, H, I = 3, 2, 256, 128
    _, p13 = make_weights(fmt, E, 2 * I, H, g)
    _, p2 = make_weights(fmt, E, H, I, g)
    b13, b2 = p13(), p2()
    ids, w = routing(T, E, topk, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    clean = run(x, ids, w, E, I, b13, b2, fmt)
    x[2, 17] = value
    got = run(x, ids, w, E, I, b13, b2, fmt)
    assert torch.isnan(got[2]).all()                  # weights of 0 and both signs in that column
    keep = [t for t in range(T) if t != 2]
    assert torch.equal(got[keep].view(torch.int16), clean[keep].view(torch.int16))


U0, U1 = 16760391 + 64, 16760391      # 24 bits each; 32 U rounded to two bf16 parts is off by 1024 either way


@gpu
@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 32])
def test_activation_is_kept_in_fp32(T, fmt):
    """h_0 = 32 U0 and h_1 = 32 U1 (g = 32, whose SiLU is 32 to within 2^-22, and up sums that are
    integers of 24 bits), and output rows that are s (h_0 - h_1): the sum cancels all but the
    last bits.  Every partial sum is a multiple of 32 s below 2^29 s, so exact; an FP32 product
    rounds each h to 2^-24 of 2^29, and the common error of SiLU scales the result."""
    need_gpu()
    H, I, base, digits, s = (128, 64, 8, 8, 0.25) if fmt == "int4" else (128, 64, 4, 12, 1.0)
    v13, v2 = torch.zeros(1, 2 * I, H, dtype=torch.float64), torch.zeros(1, H, I, dtype=torch.float64)
    x = torch.zeros(T, H, dtype=torch.float64)
    for k in range(digits):
        x[:, k] = base ** k / s
        for i, u in enumerate((U0, U1)):
            v13[0, I + i, k] = s * (u // base ** k % base)
    x[:, 20] = 32 / s
    v13[0, :2, 20] = s
    v2[0, :, 0], v2[0, :, 1] = s, -s
    assert torch.equal(x, x.to(torch.bfloat16).double())
    if fmt == "int4":
        blobs = []
        for v in (v13, v2):
            scale = torch.full((1, v.shape[1], v.shape[2] // 32), s, dtype=torch.bfloat16)
            blob = torch.empty(chord.chord_packed_weight_bytes(1, v.shape[1], v.shape[2]), dtype=torch.uint8, device=DEV)
            chord.chord_pack_weights((v / s + 8).to(torch.uint8).to(DEV), scale.to(DEV), blob)
            blobs.append(blob)
    else:
        blobs = [mx_blob(v13), mx_blob(v2)]
    ids, w = torch.zeros((T, 1), dtype=torch.int32), torch.ones(T, 1)
    out = run(x.to(torch.bfloat16), ids, w, 1, I, *blobs, fmt)
    ref = torch.full((T, H), 32 * s * (U0 - U1), dtype=torch.float64)
    check(out, ref, ref * 2.0 ** -22 + 2 * s * 2.0 ** 29 * 2.0 ** -24)


@gpu
@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_few_results_differ_from_the_exact_sum_rounded(fmt):
    """A relative error r in front of the last rounding changes r / 2^-7.5 of the results (the mean
    step of bf16).  Chopping additions leave out half a unit of FP32 at most, of a partial
    sum that is half of the final one on average: chains of 32 instructions (gate and up, 1024
    columns in two sums) and of 48 (down), (2 * 32 + 48) / 2 * 2^-24 = 3.3e-6, 0.6 of 1000
    results; a single chain of 7168 columns 3 of 1000."""
    need_gpu()
    T, E, topk, H, I = 16, 4, 4, 7168, 1984
    g = torch.Generator().manual_seed(77)
    v13, p13 = make_weights(fmt, E, 2 * I, H, g)
    v2, p2 = make_weights(fmt, E, H, I, g)
    ids, w = routing(T, E, topk, g)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    out = run(x, ids, w, E, I, p13(), p2(), fmt)
    ref, tol = reference(x, ids, w, v13, v2)
    check(out, ref, tol)
    assert (out.cpu() != ref.to(torch.bfloat16)).double().mean() <= 1e-3
