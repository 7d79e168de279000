"""Router: logits against sums in binary64, the choice of experts against its
definition in binary64, weights within derived bounds, refusals.

Logits.  Products of bf16 numbers are exact in FP32.  An addition in a matrix
instruction may chop, an error of at most 2^-22 of the magnitudes added; chains of them are kept
to 64 and at most 64 sums are joined afterwards, so |error| <= 128 * 2^-22 * sum |x w|.  Small
integers have no error at all, in any order.

Weights.  Relative error of exp(a) in FP32: 2 units of the result (the documented bound of the
function) and |a| times the half unit that a = l - c was rounded by; a sum of E of them adds a
half unit for each of its E / 32 + 5 additions, the product and quotient one each.  With u = 2^-24:
(2 |a|max + 8 + E / 32 + 16) u, next to the smallest normal number."""
import math

import pytest
import torch

import w4a16_int4_mixture_moe_gb300 as chord

DEV = "cuda:0"
gpu = pytest.mark.gpu
U = 2.0 ** -24
NINF = float("-inf")
SOFTMAX, SIGMOID = chord.SCORE_SOFTMAX, chord.SCORE_SIGMOID


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    chord.build()
    chord.load()
    chord.chord_get_device_error()


def gen(seed):
    return torch.Generator().manual_seed(seed)


# -------------------------------------------------------------------- logits

SHAPES = [(1, 1, 8), (1, 384, 7168), (2, 7, 24), (3, 384, 512), (7, 16, 72), (8, 64, 64), (15, 17, 136), (16, 8, 1000), (17, 161, 264),
          (31, 33, 2088), (32, 384, 1024), (33, 129, 320), (48, 384, 7168), (64, 256, 96), (65, 100, 4104), (127, 385, 520),
          (128, 128, 128), (129, 512, 640), (200, 1024, 1032), (257, 3, 88), (300, 384, 1024), (513, 60, 2048), (1003, 161, 2088),
          (1024, 384, 1024), (1500, 256, 1536), (2048, 1024, 256), (2100, 48, 72), (2500, 513, 264), (4100, 384, 448)]


def run_logits(x, W):
    out = torch.full((x.shape[0], W.shape[-2]), float("nan"), device=DEV)
    chord.chord_router_logits(x, W, out)
    assert chord.chord_get_device_error() == 0
    return out


@gpu
@pytest.mark.parametrize("T,E,H", SHAPES)
def test_logits_of_integers_are_exact(T, E, H):
    need_gpu()
    g = gen(T * 1000003 + E * 1009 + H)
    x = torch.randint(-3, 4, (T, H), generator=g)
    W = torch.randint(-3, 4, (E, H), generator=g)
    ref = (x.double() @ W.double().t()).float()
    assert ref.abs().max() < 2 ** 24
    got = run_logits(x.to(torch.bfloat16).to(DEV), W.to(torch.bfloat16).to(DEV)).cpu()
    assert torch.equal(got, ref)
    # three parts: integers of up to 24 bits, 1 in 2^8 of each part's range
    big = torch.randint(-2 ** 23, 2 ** 23, (E, H), generator=g).float() * 2.0 ** -8
    x1 = torch.zeros((T, H))
    x1[torch.arange(T), torch.randint(0, H, (T,), generator=g)] = 1.0
    parts = torch.empty((3, E, H), dtype=torch.bfloat16, device=DEV)
    chord.chord_router_split_weights(big.to(DEV), parts)
    got = run_logits(x1.to(torch.bfloat16).to(DEV), parts).cpu()
    assert torch.equal(got, x1 @ big.t())


@gpu
@pytest.mark.parametrize("T,E,H", SHAPES)
@pytest.mark.parametrize("parts", [1, 3])
def test_logits_against_binary64(T, E, H, parts):
    need_gpu()
    g = gen(T + 7 * E + 13 * H)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    W = torch.randn((E, H), generator=g) * H ** -0.5
    x[:, ::5] *= 50
    if parts == 1:
        Wd = W.to(torch.bfloat16).to(DEV)
        W = Wd.cpu().float()
    else:
        Wd = torch.empty((3, E, H), dtype=torch.bfloat16, device=DEV)
        chord.chord_router_split_weights(W.to(DEV), Wd)
        assert torch.equal(Wd.cpu().double().sum(0).float(), W)
    got = run_logits(x.to(DEV), Wd).cpu().double()
    ref = x.double() @ W.double().t()
    mag = x.double().abs() @ W.double().abs().t()
    assert ((got - ref).abs() <= 128 * 2.0 ** -22 * mag * (1.02 if parts == 3 else 1.0)).all()


@gpu
def test_logits_of_strided_rows_and_special_values():
    need_gpu()
    g = gen(5)
    for T in (3, 70, 1300):
        big = torch.randint(-3, 4, (T, 400), generator=g).to(torch.bfloat16).to(DEV)
        W = torch.randint(-3, 4, (40, 264), generator=g).to(torch.bfloat16).to(DEV)
        x = big[:, 8:272]
        assert torch.equal(run_logits(x, W), (x.double() @ W.double().t()).float())
        # an infinity or NaN reaches its own row's logits only
        big[1, 100], big[2, 200] = float("inf"), float("nan")
        W[:] = W.abs() + 1
        got = run_logits(x, W)
        assert (got[1] == float("inf")).all() and got[2].isnan().all()
        rest = [t for t in range(T) if t not in (1, 2)]
        assert torch.equal(got[rest], (x[rest].double() @ W.double().t()).float())


@gpu
def test_split_weights():
    need_gpu()
    g = gen(9)
    w = torch.randn((5, 333), generator=g) * torch.exp2(torch.randint(-90, 90, (5, 333), generator=g).float())
    w[0, :8] = torch.tensor([0.0, -0.0, 3.4028234e38, -3.4028234e38, 1.0, 2.0 ** -100, float("inf"), float("nan")])
    parts = torch.empty((3, 5, 333), dtype=torch.bfloat16, device=DEV)
    chord.chord_router_split_weights(w.to(DEV), parts)
    p = parts.cpu().double()
    assert p[0, 0, 6] == float("inf") and p[0, 0, 7].isnan() and (p[1:, 0, 6:8] == 0).all()
    keep = torch.ones_like(w, dtype=torch.bool)
    keep[0, 6:8] = False
    assert torch.equal(p.sum(0)[keep], w.double()[keep])


@gpu
@pytest.mark.parametrize("T,E,H", [(1, 384, 7168), (40, 161, 2088), (600, 256, 1024), (2100, 384, 1024)])
def test_logits_repeat_bit_for_bit_and_in_a_graph(T, E, H):
    need_gpu()
    g = gen(T)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).to(DEV)
    W = torch.randn((3, E, H), generator=g).to(torch.bfloat16).to(DEV)
    ref = run_logits(x, W).clone()
    for _ in range(5):
        assert torch.equal(run_logits(x, W), ref)
    out = torch.zeros((T, E), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chord.chord_router_logits(x, W, out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chord.chord_router_logits(x, W, out)
    for sign in (-1.0, 1.0):
        x.mul_(-1)
        out.zero_()
        graph.replay()
        assert torch.equal(out, sign * ref)


@gpu
def test_logits_of_no_rows():
    need_gpu()
    out = torch.empty((0, 5), device=DEV)
    chord.chord_router_logits(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV),
                              torch.zeros((5, 64), dtype=torch.bfloat16, device=DEV), out)


# --------------------------------------------------------------------- route

def reference(l, topk, score, bias=None, groups=1, topk_groups=1, group_best=1, renormalize=True, scale=1.0, first=0, E_local=None):
    """The definition, one token at a time, in binary64 (Python floats)."""
    T, E = l.shape
    E_local = E - first if E_local is None else E_local
    l = l.double().clamp(max=3.4028234663852886e38)
    open_ = l > NINF
    if score == SIGMOID:
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = torch.where(open_, l, torch.full_like(l, NINF)).max(dim=1, keepdim=True).values
        e = torch.where(open_, torch.exp(l - torch.where(m > NINF, m, torch.zeros_like(m))), torch.zeros_like(l))
        s = e / e.sum(dim=1, keepdim=True).clamp(min=1e-300)
    avail = open_ if bias is None else open_ & (bias.double() > NINF)
    z = s if bias is None else s + bias.double()
    ids, w = torch.full((T, topk), -1, dtype=torch.int64), torch.zeros((T, topk), dtype=torch.float64)
    size = E // groups
    for t in range(T):
        rank = l[t].tolist() if bias is None else z[t].tolist()
        gsc = l[t].tolist() if bias is None and group_best == 1 else z[t].tolist()
        ok = avail[t].tolist()
        if groups > 1:
            val = []
            for g in range(groups):
                best = sorted((gsc[i] for i in range(g * size, (g + 1) * size) if ok[i]), reverse=True)[:group_best]
                if best:
                    val.append((-sum(best), g))
            allowed = {g for _, g in sorted(val)[:topk_groups]}
            ok = [o and i // size in allowed for i, o in enumerate(ok)]
        chosen = [i for _, i in sorted((-rank[i], i) for i in range(E) if ok[i])][:topk]
        if not chosen:
            continue
        if renormalize and score == SOFTMAX:
            e = torch.exp(l[t, chosen] - l[t, chosen].max())
            wt = e / e.sum()
        elif renormalize:
            # log of the sigmoid, so that far negative logits keep their ratio
            ls = torch.where(l[t, chosen] < -30, l[t, chosen], -torch.log1p(torch.exp(-l[t, chosen].clamp(min=-30))))
            e = torch.exp(ls - ls.max())
            wt = e / e.sum()
        else:
            wt = s[t, chosen]
        for k, i in enumerate(chosen):
            ids[t, k] = i - first if first <= i < first + E_local else -1
            w[t, k] = float(wt[k]) * scale
    return ids.to(torch.int32), w


def run_route(l, topk, bias=None, **kw):
    T = l.shape[0]
    ids = torch.full((T, topk), -77, dtype=torch.int32, device=DEV)
    w = torch.full((T, topk), float("nan"), device=DEV)
    chord.chord_moe_route(l, ids, w, bias=bias, **kw)
    return ids.cpu(), w.cpu()


def check(l, topk, bias=None, **kw):
    """Ids equal the definition's, weights are within the bound."""
    ids, w = run_route(l.to(DEV) if not l.is_cuda else l, topk, None if bias is None else bias.to(DEV), **kw)
    lc = l.cpu().float()
    rid, rw = reference(lc, topk, kw.pop("score", SOFTMAX), bias, **kw)
    assert torch.equal(ids, rid), (ids[(ids != rid).any(1)][:3], rid[(ids != rid).any(1)][:3])
    f = lc[lc.abs() < 1e30]
    span = min(float(f.max() - f.min()), 110.0) if f.numel() else 0.0   # exp of less than -110 is 0 in FP32
    tol = (2 * span + 8 + l.shape[1] / 32 + 16) * U * rw.abs() + 2.0 ** -126 * abs(kw.get("scale", 1.0))
    assert ((w.double() - rw).abs() <= tol).all(), ((w.double() - rw).abs() / tol).max()
    return ids, w


CASES = [(1, 384, 8, 1, 1), (1, 1, 1, 1, 1), (2, 8, 2, 1, 1), (33, 61, 6, 1, 1), (100, 384, 8, 1, 1), (64, 256, 8, 8, 4), (40, 1024, 32, 1, 1),
         (40, 1024, 32, 32, 1), (50, 60, 5, 3, 2), (30, 31, 31, 1, 1), (30, 96, 32, 3, 1), (77, 512, 1, 4, 4), (20, 66, 16, 33 - 11, 6),
         (20, 64, 2, 32, 1), (300, 128, 4, 2, 1), (9, 33, 32, 1, 1), (25, 160, 6, 8, 3), (25, 500, 20, 5, 2)]


@gpu
@pytest.mark.parametrize("T,E,topk,groups,topk_groups", CASES)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(T, E, topk, groups, topk_groups, score, with_bias, dtype):
    need_gpu()
    g = gen(T * 31 + E + topk + groups * 7 + score + 2 * with_bias)
    l = (torch.randn((T, E), generator=g) * 2).to(dtype)
    bias = torch.randn(E, generator=g) * 0.1 if with_bias else None
    for best in (1, 2):
        for renorm in (True, False):
            check(l, topk, bias, score=score, groups=groups, topk_groups=topk_groups, group_best=best, renormalize=renorm,
                  scale=2.5 if renorm else 1.0, first=E // 3, E_local=max(1, E // 2))


@gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lower_index(score, with_bias):
    need_gpu()
    g = gen(3)
    for E, topk, groups, tg in ((384, 8, 1, 1), (64, 32, 1, 1), (256, 8, 8, 4), (40, 7, 5, 2), (1024, 32, 1, 1)):
        bias = torch.randint(-1, 2, (E,), generator=g) * 0.25 if with_bias else None
        for values in (1, 2, 5):
            l = torch.randint(0, values, (50, E), generator=g).float()
            l[7] = -3.3895313892515355e38       # the lowest bf16 number, everywhere
            l[8] = 50.0                         # scores of 1 in FP32
            l[9] = torch.where(torch.arange(E) % 3 == 0, 60.0, 70.0)
            for best in (1, 2):
                check(l, topk, bias, score=score, groups=groups, topk_groups=tg, group_best=best)
                check(l.to(torch.bfloat16), topk, bias, score=score, groups=groups, topk_groups=tg, group_best=best, renormalize=False)


@gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_values_that_fp32_cannot_tell_apart(score):
    """Experts whose scores plus biases differ by far less than an FP32 rounding, in every position
    of the choice and between groups: the order is that of binary64."""
    need_gpu()
    g = gen(11)
    T, E = 64, 128
    l = torch.randn((T, E), generator=g)
    s = torch.sigmoid(l.double()) if score == SIGMOID else torch.softmax(l.double(), dim=1)
    # every row has its own bias that makes all values nearly equal: one call per row
    for t in range(0, T, 4):
        bias = (0.75 - s[t]).float()
        for groups, tg, best in ((1, 1, 1), (8, 3, 2), (4, 2, 1)):
            check(l[t:t + 1].clone(), 12, bias, score=score, groups=groups, topk_groups=tg, group_best=best)
    # neighbours in the last place of the logit, without a bias and with a common one
    l = torch.full((T, E), 1.25) + torch.randint(0, 4, (T, E), generator=g) * 2.0 ** -23
    check(l, 9, None, score=score)
    check(l, 9, torch.full((E,), 0.5), score=score)
    check(l, 9, torch.full((E,), -1000.0), score=score)


@gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("E,topk", [(384, 8), (384, 31), (384, 32), (512, 16), (1024, 30), (33, 32), (40, 32)])
@pytest.mark.parametrize("same", [2, 3, 8, 40])
def test_near_ties_in_clusters(score, E, topk, same):
    """Clusters of `same` experts whose values agree to an FP32 rounding, well apart from one another, in any places of
    the choice and across its end."""
    need_gpu()
    g = gen(E + topk * 5 + same)
    for scale in (1.0, 0.01):
        l = torch.randn((1, E), generator=g)
        s = torch.sigmoid(l.double()) if score == SIGMOID else torch.softmax(l.double(), dim=1)
        target = torch.empty(E, dtype=torch.float64)
        target[torch.randperm(E, generator=g)] = (torch.arange(E) // same).double() * scale
        bias = (target - s[0]).float()
        check(l, topk, bias, score=score)
        check(l.repeat(5, 1), topk, bias, score=score, renormalize=False)


@gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 3)])
def test_masked_experts_and_empty_rows(score, with_bias, groups, topk_groups):
    need_gpu()
    g = gen(21)
    T, E, topk = 60, 64, 8
    nan = float("nan")
    l = torch.randn((T, E), generator=g) * 3
    bias = torch.randn(E, generator=g) * 0.1 if with_bias else None
    l[0] = NINF
    l[1] = nan
    l[2] = NINF
    l[2, 5] = 1.0
    l[3, :60] = NINF
    l[4, ::2] = nan
    l[5] = float("inf")
    l[6, 10:14] = float("inf")
    l[7, :] = -3.4028234e38
    l[8, 3] = 3.4028234e38
    l[9] = -200.0
    l[9, 7] = -150.0
    l[10] = -3.4028234e38
    l[10, 1] = NINF
    l[11, 8:16] = NINF                       # one whole group
    l[12, :] = NINF
    l[12, 0::8] = torch.randn(8, generator=g)    # one expert a group
    l[20:40][torch.rand((20, E), generator=g) < 0.9] = NINF
    if with_bias:
        bias[[1, 9, 33]] = NINF
        bias[40] = nan
        bias[50] = float("inf")
        bias[51] = 1e30
    for best in (1, 2):
        for renorm in (True, False):
            ids, w = check(l, topk, bias, score=score, groups=groups, topk_groups=topk_groups, group_best=best, renormalize=renorm)
            assert (ids[:2] == -1).all() and (w[:2] == 0).all()
            assert not w.isnan().any()
            check(l.to(torch.bfloat16), topk, bias, score=score, groups=groups, topk_groups=topk_groups, group_best=best,
                  renormalize=renorm, first=8, E_local=8)


@gpu
def test_strides_and_many_rows():
    need_gpu()
    g = gen(8)
    for dtype in (torch.float32, torch.bfloat16):
        for E, off in ((61, 3), (64, 1), (384, 0), (383, 5)):
            big = torch.randn((211, E + 10), generator=g).to(dtype).to(DEV)
            check(big[:, off:off + E], 5, None, score=SOFTMAX)
            check(big[::3, off:off + E], 5, torch.randn(E, generator=g) * 0.1, score=SIGMOID)
    # rows behind one another past 2^31 elements: the last of them
    stride = 2 ** 30 + 64
    big = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device=DEV)
    rows = big.as_strided((3, 64), (stride, 1))
    rows.copy_(torch.randn((3, 64), generator=g))
    check(rows, 4, None, score=SIGMOID)


@gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T", [7295, 7296, 12345])
def test_many_tokens(T, score, with_bias):
    """More tokens than the GPU has warps for: two at a time, an odd one left over; ties, close values, empty
    rows and rows with many candidates next to one another."""
    need_gpu()
    g = gen(T + score)
    E, topk = 40, 5
    l = torch.randn((T, E), generator=g) * 2
    l[::7] = l[::7].to(torch.bfloat16).float()
    l[5::50] = torch.randint(0, 3, l[5::50].shape, generator=g).float()
    l[9::100] = 1.5
    l[13::100] = NINF
    l[14::100, 3:] = NINF
    l[15::200] = torch.full((E,), 1.25) + torch.randint(0, 4, l[15::200].shape, generator=g) * 2.0 ** -23
    bias = torch.randn(E, generator=g) * 0.1 if with_bias else None
    if with_bias:
        bias[:8] = 0.0
    check(l, topk, bias, score=score)
    check(l.to(torch.bfloat16), topk, bias, score=score, groups=8, topk_groups=3, group_best=2, renormalize=False)


@gpu
def test_route_in_a_graph_and_on_another_stream():
    need_gpu()
    g = gen(4)
    l = torch.randn((500, 384), generator=g).to(DEV)
    ids, w = torch.empty((500, 8), dtype=torch.int32, device=DEV), torch.empty((500, 8), device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chord.chord_moe_route(l, ids, w)
    for _ in range(2):
        l.copy_(torch.randn((500, 384), generator=g))
        graph.replay()
        ri, rw = run_route(l, 8)
        assert torch.equal(ids.cpu(), ri) and torch.equal(w.cpu(), rw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = torch.empty_like(ids), torch.empty_like(w)
    chord.chord_moe_route(l, a, b, stream=side)
    side.synchronize()
    assert torch.equal(a, ids) and torch.equal(b, w)
    chord.chord_moe_route(l[:0], ids[:0], w[:0])


@gpu
def test_router_to_align():
    """Logits, choice and align, as a layer uses them: the choice's ids are the align's pairs."""
    need_gpu()
    g = gen(12)
    T, E, H, topk, first, local = 300, 64, 512, 6, 16, 32
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).to(DEV)
    W = (torch.randn((E, H), generator=g) * H ** -0.5).to(torch.bfloat16).to(DEV)
    logits = run_logits(x, W)
    ids = torch.empty((T, topk), dtype=torch.int32, device=DEV)
    w = torch.empty((T, topk), device=DEV)
    chord.chord_moe_route(logits, ids, w, score=SIGMOID, bias=torch.zeros(E, device=DEV), scale=2.5, first=first, E_local=local)
    rid, _ = reference(logits.cpu(), topk, SIGMOID, torch.zeros(E), scale=2.5, first=first, E_local=local)
    assert torch.equal(ids.cpu(), rid)
    bm = 16
    cap = chord.chord_align_capacity(T, topk, local, bm)
    order = torch.empty(cap, dtype=torch.int32, device=DEV)
    blocks = torch.empty(cap // bm, dtype=torch.int32, device=DEV)
    count = torch.empty(1, dtype=torch.int32, device=DEV)
    chord.chord_moe_align(ids, local, bm, order, blocks, count,
                          torch.empty(chord.chord_align_workspace_bytes(T, topk, local), dtype=torch.uint8, device=DEV))
    flat, order, blocks = rid.reshape(-1), order.cpu(), blocks.cpu()
    pairs = order[order < T * topk]
    assert torch.equal(torch.sort(pairs).values, torch.nonzero(flat >= 0).reshape(-1).int())
    at = torch.nonzero(order < T * topk).reshape(-1)
    assert torch.equal(flat[pairs.long()], blocks[torch.div(at, bm, rounding_mode="floor")])
    assert math.isclose(float(w.sum(1).mean()), 2.5, rel_tol=1e-5)


@gpu
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_groups_of_biases_whose_sum_leaves_fp32(score, renorm):
    """Experts switched off by the lowest (or raised by the largest) number: the sum of a group's two best is beyond FP32 and
    still a number, above a group without an available expert and in order with the other groups' sums."""
    need_gpu()
    g = gen(31)
    low = -3.4028234663852886e38
    for size, groups in ((8, 4), (16, 8), (2, 32), (5, 3)):
        E = size * groups
        l = torch.randn((6, E), generator=g)
        l[3] = 1.0
        l[4, ::2] = NINF
        for tg in (1, 2):
            topk = min(4, tg * size)
            for kind in range(5):
                b = torch.full((groups, size), low)
                if kind == 0:                       # only the second group has anybody
                    b[:] = NINF
                    b[1] = low
                elif kind == 1:                     # sums of -2, -1.5 (the last group) and -1.75 of the largest number
                    b[-1, ::2] = low * 0.5
                    b[groups // 2, 1::2] = low * 0.75
                elif kind == 2:                     # one expert of the first group against two of the last
                    b[0, 1:] = NINF
                elif kind == 3:                     # the same above zero
                    b[:] = -low
                    b[0] = -low * 0.75
                    b[1] = NINF
                else:                               # the first two groups have nobody, the others one expert or several
                    b[:2] = NINF
                    b[2, :-1] = NINF if groups > 3 else low
                check(l, topk, b.reshape(-1), score=score, groups=groups, topk_groups=tg, group_best=2, renormalize=renorm)
                check(l.to(torch.bfloat16), topk, b.reshape(-1), score=score, groups=groups, topk_groups=tg, group_best=1, renormalize=renorm)


def split(W):
    parts = torch.empty((3, *W.shape), dtype=torch.bfloat16, device=DEV)
    chord.chord_router_split_weights(W.to(DEV), parts)
    return parts


@gpu
def test_split_weights_of_few_bits():
    """Every number from 2^-110 on ends in three parts that are not 0, of its sign, whose sum it is: however few bits it has."""
    need_gpu()
    g = gen(14)
    n = 4000
    for bits in (1, 2, 7, 8, 9, 15, 16, 17, 24):
        m = torch.randint(2 ** (bits - 1), 2 ** bits, (n,), generator=g).double()
        e = torch.randint(-110, 127, (n,), generator=g).double()
        e[:4] = torch.tensor([-110.0, -110.0, 127.0, 0.0], dtype=torch.float64)
        w = (m * torch.exp2(e - (bits - 1)) * (torch.randint(0, 2, (n,), generator=g) * 2 - 1)).float()
        assert w.abs().min() >= 2.0 ** -110 and w.abs().max() < float("inf")
        p = split(w).cpu().double()
        assert torch.equal(p.sum(0), w.double())
        assert (p * w.double().sign() > 0).all()
    assert (split(torch.tensor([0.0, -0.0])) == 0).all()


@gpu
@pytest.mark.parametrize("T,E", [(1, 40), (3, 40), (70, 40), (3000, 40), (1300, 161)])
def test_infinite_activations_with_fp32_weights(T, E):
    """The logit is the infinity or NaN of the sum, as with bf16 weights, in every kernel; other rows are untouched."""
    need_gpu()
    g = gen(T + E)
    H = 264
    x = torch.randint(-3, 4, (T, H), generator=g).to(torch.bfloat16)
    W = torch.randint(-3, 4, (E, H), generator=g).float()           # 0 among them: infinity times 0 is NaN
    W[1::2] += 0.375
    W[3 % E], W[4] = W[3 % E] * (1 + 2.0 ** -22), W[4] * (1 + 2.0 ** -12)
    inf = float("inf")
    for k, t in enumerate((0, 1, 65, 130, 200, 255, 257, T - 1)):
        if 0 <= t < T:
            x[t, 3 + 31 * k] = inf if k % 2 else -inf
    if T > 2:
        x[2, 7], x[2, 9] = inf, -inf
    ref = x.double() @ W.double().t()
    got = run_logits(x.to(DEV), split(W)).cpu().double()
    bad = ~ref.isfinite()
    assert bad.any(1).sum() >= min(T, 2) and torch.equal(got[bad].isnan(), ref[bad].isnan())
    both = bad & ~ref.isnan()
    assert both.any() and torch.equal(got[both], ref[both])
    mag = x.double().abs() @ W.double().abs().t()
    assert ((got - ref).abs()[~bad] <= 128 * 2.0 ** -22 * 1.02 * mag[~bad]).all()


#        T, E, H of the pairs of CTAs: groups of 32, 160, 192, 224 and 256 experts, fewer experts than a box has rows, a ring
#        that wraps, a last pair of CTAs with tokens for one of the two only and for a part of one
WIDE = [(8192, 3, 136), (5888, 7, 264), (3000, 40, 392), (8192, 384, 264), (16384, 160, 264), (16290, 187, 136), (16384, 200, 136),
        (16290, 224, 520), (16384, 256, 264), (16221, 250, 648), (19456, 1024, 136)]


@gpu
@pytest.mark.parametrize("T,E,H", WIDE)
@pytest.mark.parametrize("parts", [1, 3])
def test_logits_of_many_tokens(T, E, H, parts):
    """Strided rows: integers exactly, real numbers within the bound, infinities and NaN in their own rows only."""
    need_gpu()
    g = torch.Generator(device=DEV).manual_seed(T + E + H)
    big = torch.randint(-3, 4, (T, H + 136), generator=g, device=DEV).to(torch.bfloat16)
    x = big[:, 8:8 + H]
    W = torch.randint(-3, 4, (E, H), generator=g, device=DEV).float()
    Wd = W.to(torch.bfloat16) if parts == 1 else split(W)
    ref = x.double() @ W.double().t()
    assert torch.equal(run_logits(x, Wd), ref.float())
    rows = [0, 127, 128, 200, 255, 256, T - 1]       # of both CTAs of a pair
    inf, nan = float("inf"), float("nan")
    big[rows, 20] = torch.tensor([inf, nan, nan, inf, -inf, nan, inf], dtype=torch.bfloat16, device=DEV)
    pos = W.abs() + 1
    got = run_logits(x, pos.to(torch.bfloat16) if parts == 1 else split(pos))
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[rows] = False
    assert torch.equal(got[keep], (x[keep].double() @ pos.double().t()).float())
    assert (got[[0, 200, T - 1]] == inf).all() and (got[255] == -inf).all() and got[[127, 128, 256]].isnan().all()
    big.copy_(torch.randn(big.shape, generator=g, device=DEV))
    W = torch.randn((E, H), generator=g, device=DEV) * H ** -0.5
    W = W.to(torch.bfloat16).float() if parts == 1 else W
    got = run_logits(x, W.to(torch.bfloat16) if parts == 1 else split(W)).double()
    mag = x.double().abs() @ W.double().abs().t()
    assert ((got - x.double() @ W.double().t()).abs() <= 128 * 2.0 ** -22 * mag * (1.02 if parts == 3 else 1.0)).all()
