"""Low-rank adapters beside a shared projection against the formula in
binary64, and with the calls that they stand beside.

Bound, element by element.  Products are exact in FP32 (v is carried in three bf16 parts of eight bits
each, or as it is).  An addition in a matrix instruction may chop, an error of at most 2^-22 of the
magnitudes added; chains of them are kept to 64, at most 80 partial sums are joined afterwards, so
|v error| <= 144 * 2^-22 * sum |A x|, and the sum over the rank (chains of at most 24 instructions)
adds 32 * 2^-22 of its own magnitudes; the scale and the base's addition round once each.  So
  |y - exact| <= scale * 180 * 2^-22 * sum_j |B| sum_k |A x| + 2^-23 (|base| + |delta|)
and a bf16 y lies between the bf16 roundings of that interval's ends.  Small integers have no error
at all before the last rounding."""
import pytest
import torch

import w4a16_int4_mixture_moe_gb300 as chord

DEV = "cuda:0"
gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    chord.build()
    chord.load()
    chord.chord_get_device_error()


def make(T, topk, S, E, rank, parts, K, N, div, out, seed, dense=False, integer=False, none=0.2, foreign=0.2):
    g = torch.Generator().manual_seed(seed)
    P = T * topk

    def values(*shape, std=1.0, hi=2):
        if integer:
            return torch.randint(-hi, hi + 1, shape, generator=g).float()
        return torch.randn(shape, generator=g) * std

    c = {"div": div, "topk": topk, "S": S, "E": E, "rank": rank, "parts": parts, "N": N, "K": K}
    a = torch.randint(0, S, (T,), generator=g, dtype=torch.int32)
    a[torch.rand(T, generator=g) < none] = -1
    c["a"] = a
    lead = (S,) if dense else (S, E)
    c["ids"] = None
    if not dense:
        ids = torch.randint(0, E, (T, topk), generator=g, dtype=torch.int32)
        ids[torch.rand((T, topk), generator=g) < foreign] = -1
        c["ids"] = ids
    c["x"] = values(-(-P // div), K).to(BF)
    c["A"] = values(*lead, parts * rank, K, std=K ** -0.5, hi=1).to(BF)
    c["B"] = values(*lead, N, rank, std=0.5 * rank ** -0.5, hi=1).to(BF)
    c["scale"] = torch.randint(1, 4, (S,), generator=g).float() if integer else torch.rand(S, generator=g) + 0.5
    c["base"] = values(P, N, hi=100).to(out)
    return c


def reference(c):
    """(y, error bound, rows that are written) in binary64."""
    S, E, rank, parts, N, K, topk = (c[n] for n in ("S", "E", "rank", "parts", "N", "K", "topk"))
    A, B = c["A"].double().reshape(S, E, parts, rank, K), c["B"].double().reshape(S, E, parts, N // parts, rank)
    P = c["base"].shape[0]
    y, tol = c["base"].double().clone(), torch.zeros(c["base"].shape, dtype=torch.float64)
    pair = torch.arange(P)
    e = torch.zeros(P, dtype=torch.long) if c["ids"] is None else c["ids"].reshape(-1).long()
    written = (e >= 0) & (e < E)
    a = c["a"].long()[pair // topk]
    for s in range(S):
        for i in range(E):
            rows = pair[(a == s) & (e == i)]
            if not rows.numel():
                continue
            x = c["x"][rows // c["div"]].double()
            scale = float(c["scale"][s]) if c["scale"] is not None else 1.0
            d = torch.cat([x @ A[s, i, p].t() @ B[s, i, p].t() for p in range(parts)], 1) * scale
            mag = torch.cat([x.abs() @ A[s, i, p].abs().t() @ B[s, i, p].abs().t() for p in range(parts)], 1) * abs(scale)
            tol[rows] = 180 * 2.0 ** -22 * mag + 2.0 ** -23 * (y[rows].abs() + d.abs())
            y[rows] += d
    return y, tol, written


def on_gpu(c):
    return {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in c.items()}


def workspace(c, T):
    n = chord.chord_adapter_workspace_bytes(T, c["topk"], c["S"], c["E"], c["rank"], c["parts"])
    assert n > 0
    return torch.empty(n, dtype=torch.uint8, device=DEV).random_(0, 256)


def add(d, y, base=None, ws=None, **kw):
    chord.chord_adapter_add(d["x"], d["div"], d["a"], d["ids"], d["A"], d["B"], d["scale"], d["base"] if base is None else base, y,
                            workspace(d, d["a"].numel()) if ws is None else ws, **kw)
    return y


def check(c, exact=False):
    d = on_gpu(c)
    ref, tol, written = reference(c)
    sentinel = 12345.0
    y = add(d, torch.full_like(d["base"], sentinel))
    assert chord.chord_get_device_error() == 0
    got = y.cpu()
    assert (got[~written] == torch.tensor(sentinel).to(got.dtype)).all()
    got, want, tol = got[written], ref[written], tol[written]
    if exact:
        assert torch.equal(got, want.to(F32).to(got.dtype) if got.dtype == BF else want.to(F32))
    elif got.dtype == F32:
        assert ((got.double() - want).abs() <= tol).all()
    else:
        lo, hi = (want - tol).float().to(BF).double(), (want + tol).float().to(BF).double()
        assert ((got.double() >= lo) & (got.double() <= hi)).all()
    # in place: the same bits where an adapter adds, every other row untouched
    b = d["base"].clone()
    add(d, b, base=b)
    assert torch.equal(b.cpu()[written], got) and torch.equal(b.cpu()[~written], c["base"][~written])
    return y


#        T, topk, S, E, rank, parts, K, N, div, dense
SHAPES = [(1, 1, 1, 1, 8, 1, 8, 8, 1, True), (1, 1, 8, 1, 16, 1, 7168, 4096, 1, True), (2, 1, 3, 1, 24, 2, 72, 48, 1, True),
          (5, 1, 2, 1, 64, 1, 1000, 1032, 1, True), (16, 1, 16, 1, 32, 1, 264, 264, 1, True), (33, 1, 4, 1, 128, 3, 96, 72, 1, True),
          (100, 1, 1, 1, 16, 1, 512, 520, 1, True), (257, 1, 5, 1, 8, 4, 136, 160, 1, True), (700, 1, 3, 1, 40, 1, 320, 136, 1, True),
          (1, 8, 2, 8, 16, 2, 256, 256, 8, False), (3, 4, 4, 16, 16, 1, 128, 256, 1, False), (32, 8, 16, 8, 16, 2, 512, 512, 8, False),
          (40, 2, 3, 300, 8, 1, 64, 64, 2, False), (64, 6, 40, 64, 24, 2, 88, 112, 1, False), (300, 8, 4, 12, 16, 1, 256, 384, 1, False),
          (513, 4, 2, 3, 64, 2, 200, 176, 4, False), (2000, 2, 1, 2, 72, 1, 72, 88, 2, False), (1500, 8, 3, 10, 32, 2, 64, 64, 8, False)]


@gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_integers_are_exact(shape, out):
    need_gpu()
    T, topk, S, E, rank, parts, K, N, div, dense = shape
    check(make(T, topk, S, E, rank, parts, K, N, div, out, seed=hash(shape) % 1000, dense=dense, integer=True), exact=True)


@gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_binary64(shape, out):
    need_gpu()
    T, topk, S, E, rank, parts, K, N, div, dense = shape
    check(make(T, topk, S, E, rank, parts, K, N, div, out, seed=1 + hash(shape) % 1000, dense=dense))


@gpu
@pytest.mark.parametrize("T", [1, 3, 40, 1000, 9000])
def test_one_adapter_no_adapter_and_all_different(T):
    need_gpu()
    for S, none in ((1, 0.0), (1, 1.0), (64, 0.0), (64, 0.5)):
        c = make(T, 1, S, 1, 16, 1, 64, 64, 1, BF, seed=T + S, dense=True, integer=True, none=none)
        if S == 64:
            c["a"] = torch.where(c["a"] >= 0, (torch.arange(T) % S).to(torch.int32), c["a"])
        check(c, exact=True)


#        T, topk, S, E, rank, parts, K, N, div, dense: more pairs than one cluster plans, ranks and parts of every kernel
LARGE = [(20000, 1, 3, 1, 16, 1, 64, 40, 1, True), (5000, 4, 2, 7, 8, 2, 40, 48, 4, False), (400, 1, 9, 1, 128, 4, 136, 416, 1, True),
         (300, 2, 2, 3, 104, 1, 520, 264, 2, False), (300, 1, 2, 1, 48, 2, 328, 336, 1, True), (260, 1, 200, 1, 24, 1, 72, 136, 1, True),
         (257, 1, 1, 1, 8, 1, 8, 8, 1, True), (1000, 3, 4, 5, 16, 4, 96, 1056, 3, False)]


@gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("shape", LARGE)
def test_many_pairs(shape, out):
    need_gpu()
    T, topk, S, E, rank, parts, K, N, div, dense = shape
    check(make(T, topk, S, E, rank, parts, K, N, div, out, seed=7 + T, dense=dense, integer=True), exact=True)
    check(make(T, topk, S, E, rank, parts, K, N, div, out, seed=8 + T, dense=dense))


#        the same: long K, so that clusters of four, of two and none share an item, with one slice and with several
LONG = [(300, 1, 1, 1, 16, 1, 7176, 64, 1, True), (700, 1, 4, 1, 64, 1, 4104, 40, 1, True), (4096, 1, 8, 1, 128, 1, 1288, 72, 1, True),
        (3000, 1, 8, 1, 64, 1, 1032, 48, 1, True), (1024, 8, 4, 48, 16, 1, 1000, 64, 1, False), (512, 8, 2, 200, 8, 2, 776, 64, 8, False),
        (300, 1, 300, 1, 32, 1, 2056, 48, 1, True), (600, 1, 2, 1, 24, 2, 264, 48, 1, True), (257, 1, 2, 1, 96, 4, 3080, 64, 1, True)]


@gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("shape", LONG)
def test_many_pairs_of_long_rows(shape, out):
    need_gpu()
    T, topk, S, E, rank, parts, K, N, div, dense = shape
    check(make(T, topk, S, E, rank, parts, K, N, div, out, seed=9 + T, dense=dense, integer=True), exact=True)
    check(make(T, topk, S, E, rank, parts, K, N, div, out, seed=10 + T, dense=dense))
    check(make(T, topk, S, E, rank, parts, K, N, div, out, seed=11 + T, dense=dense, none=0.9))


@gpu
def test_every_pair_elsewhere():
    need_gpu()
    c = make(20, 4, 3, 5, 16, 1, 64, 64, 1, F32, seed=2, integer=True, foreign=1.0)
    y = torch.full((80, 64), 7.0, device=DEV)
    add(on_gpu(c), y)
    assert (y == 7).all()


@gpu
def test_ids_that_are_none_repeat_or_are_invalid():
    need_gpu()
    c = make(50, 4, 3, 5, 16, 1, 64, 64, 1, F32, seed=3, integer=True)
    c["ids"][3] = 2                     # one expert four times
    c["ids"][4] = torch.tensor([-5, 5, 1000, -2 ** 31], dtype=torch.int32)
    check(c, exact=True)
    bad = on_gpu(c)
    bad["a"][7], bad["a"][9], bad["a"][11] = 3, -2, 2 ** 31 - 1
    c["a"][7] = c["a"][9] = c["a"][11] = -1
    ref, _, written = reference(c)
    y = add(bad, torch.zeros_like(bad["base"]))
    assert chord.chord_get_device_error() == 7
    assert torch.equal(y.cpu()[written], ref[written].float())
    with pytest.raises(chord.ChordError) as ei:
        add(bad, y, opts=chord.ChordOpts(validate=1))
    assert ei.value.status == 6
    assert chord.chord_get_device_error() == 0


@gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("T", [4, 300])
def test_strides_and_column_ranges(T, out):
    """Rows of a wider buffer, and an adapter of one half of the columns in place."""
    need_gpu()
    c = make(T, 2, 3, 4, 16, 1, 96, 128, 1, out, seed=T, integer=True)
    d = on_gpu(c)
    ref, _, written = reference(c)
    wide = torch.full((2 * T, 400), 3.0, dtype=out, device=DEV)
    wide[:, 128:256] = d["base"]
    xw = torch.zeros((2 * T, 200), dtype=BF, device=DEV)
    xw[:, 16:112] = d["x"]
    d["x"] = xw[:, 16:112]
    view = wide[:, 128:256]
    add(d, view, base=view)
    want = ref.float().to(out)
    want[~written] = c["base"][~written]
    assert torch.equal(view.cpu(), want)
    assert (wide[:, :128] == 3).all() and (wide[:, 256:] == 3).all()
    y = torch.zeros((2 * T, 136), dtype=out, device=DEV)
    d["base"] = torch.cat([torch.zeros_like(d["base"]), d["base"]], 1)[:, 128:]
    add(d, y[:, 8:])
    assert torch.equal(y.cpu()[written][:, 8:], want[written]) and (y[:, :8] == 0).all()


@gpu
def test_no_scale_special_values_and_rows_alone():
    need_gpu()
    for T in (6, 200):
        c = make(T, 1, 2, 1, 16, 1, 64, 64, 1, F32, seed=8, dense=True, integer=True, none=0.0)
        c["scale"] = None
        check(c, exact=True)
        # an infinity or NaN of one row reaches that row only
        ref, _, _ = reference(c)
        c["x"][1, 3] = float("inf")
        c["x"][2, 5] = float("nan")
        c["A"] = c["A"].abs() + 1
        c["B"] = c["B"].abs() + 1
        ref, _, _ = reference(c)
        got = add(on_gpu(c), torch.zeros((T, 64), device=DEV)).cpu()
        assert (got[1] == float("inf")).all() and got[2].isnan().all()
        rest = [t for t in range(T) if t not in (1, 2)]
        assert torch.equal(got[rest], ref[rest].float())


@gpu
@pytest.mark.parametrize("T,topk,S,E", [(8, 1, 4, 1), (32, 8, 16, 8), (2000, 4, 4, 6)])
def test_repeats_bit_for_bit_on_streams_and_in_graphs(T, topk, S, E):
    need_gpu()
    c = make(T, topk, S, E, 16, 2, 512, 256, topk, F32, seed=T, dense=E == 1)
    d = on_gpu(c)
    ref = add(d, torch.zeros_like(d["base"])).clone()
    for _ in range(5):
        assert torch.equal(add(d, torch.zeros_like(d["base"])), ref)
    side = [torch.cuda.Stream() for _ in range(2)]
    ys, wss = [torch.zeros_like(ref) for _ in side], [workspace(c, T) for _ in side]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for s, y, ws in zip(side, ys, wss):
            add(d, y, ws=ws, stream=s)
    for s, y in zip(side, ys):
        s.synchronize()
        assert torch.equal(y, ref)
    # two graphs that share a workspace, replayed one after the other with other inputs
    ws, x0 = workspace(c, T), d["x"].clone()
    y1, y2 = torch.zeros_like(ref), torch.zeros_like(ref)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        add(d, y1, ws=ws)
    with torch.cuda.graph(g2):
        add(d, y2, ws=ws)
        add(d, y2, base=y2, ws=ws)
    for k in range(3):
        d["x"].copy_(torch.randn(x0.shape, generator=torch.Generator().manual_seed(k)))
        g1.replay()
        g2.replay()
        want = add(d, torch.zeros_like(ref))
        assert torch.equal(y1, want)
        twice = add(d, want.clone(), base=want.clone())
        assert torch.equal(y2, twice)
    d["x"].copy_(x0)
    g1.replay()
    assert torch.equal(y1, ref)


@gpu
def test_large_offsets():
    """Rows of y past 2^31 elements and an adapter past 2^31 elements of A."""
    need_gpu()
    T, K, N, rank = 300, 4096, 64, 16
    c = make(T, 1, 2, 1, rank, 1, K, N, 1, BF, seed=1, dense=True, integer=True)
    d = on_gpu(c)
    ref, _, _ = reference(c)
    stride = (2 ** 31 // 256 + 4096) // 8 * 8
    big = torch.empty(T * stride, dtype=BF, device=DEV)
    y = big.as_strided((T, N), (stride, 1))
    y.copy_(d["base"])
    add(d, y, base=y)
    assert torch.equal(y.cpu(), ref.float().to(BF))
    del big, y
    S = 2 ** 31 // (rank * K * 256) + 2          # adapters of 256 experts
    A = torch.zeros((S, 256, rank, K), dtype=BF, device=DEV)
    B = torch.zeros((S, 256, N, rank), dtype=BF, device=DEV)
    assert A.numel() > 2 ** 31
    A[S - 1, 255], B[S - 1, 255] = d["A"][1], d["B"][1]
    a = torch.full((T,), S - 1, dtype=torch.int32, device=DEV)
    ids = torch.full((T, 1), 255, dtype=torch.int32, device=DEV)
    ws = torch.empty(chord.chord_adapter_workspace_bytes(T, 1, S, 256, rank, 1), dtype=torch.uint8, device=DEV)
    y = torch.zeros((T, N), dtype=BF, device=DEV)
    chord.chord_adapter_add(d["x"], 1, a, ids, A, B, None, d["base"], y, ws)
    c["a"][:] = 1
    c["scale"] = None
    ref, _, _ = reference(c)
    assert torch.equal(y.cpu(), ref.float().to(BF))


@gpu
def test_layer_from_router_to_combine_with_adapters():
    """Logits, choice, align, gate_up with adapters, SiLU*up, down with adapters, combine: each stage against
    binary64 on the GPU's own previous stage."""
    need_gpu()
    g = torch.Generator().manual_seed(77)
    T, E, topk, H, I, S, rank = 70, 8, 2, 256, 128, 3, 16
    x = torch.randn((T, H), generator=g).to(BF).to(DEV)
    Wg = (torch.randn((E, H), generator=g) * H ** -0.5).to(BF).to(DEV)
    logits = torch.empty((T, E), device=DEV)
    chord.chord_router_logits(x, Wg, logits)
    ids = torch.empty((T, topk), dtype=torch.int32, device=DEV)
    w = torch.empty((T, topk), device=DEV)
    chord.chord_moe_route(logits, ids, w)
    sm = torch.softmax(logits.double(), 1).topk(topk, 1)
    assert torch.equal(ids.long(), sm.indices)
    want = sm.values / sm.values.sum(1, keepdim=True)
    assert ((w.double() - want).abs() <= 100 * 2.0 ** -24 * want).all()

    def pack(N, K):
        codes = torch.randint(0, 16, (E, N, K), generator=g, dtype=torch.uint8).to(DEV)
        scales = (torch.rand((E, N, K // 32), generator=g) * 0.02 + 1e-3).to(BF).to(DEV)
        blob = torch.empty(chord.chord_packed_weight_bytes(E, N, K), dtype=torch.uint8, device=DEV)
        chord.chord_pack_weights(codes, scales, blob)
        return blob

    p13, p2 = pack(2 * I, H), pack(H, I)
    P = T * topk
    bm = chord.chord_select_block_m(T, topk, E, E, 2 * I, H)
    cap = chord.chord_align_capacity(T, topk, E, bm)
    order = torch.empty(cap, dtype=torch.int32, device=DEV)
    blocks = torch.empty(cap // bm, dtype=torch.int32, device=DEV)
    count = torch.empty(1, dtype=torch.int32, device=DEV)
    chord.chord_moe_align(ids, E, bm, order, blocks, count,
                          torch.empty(chord.chord_align_workspace_bytes(T, topk, E), dtype=torch.uint8, device=DEV))
    a = torch.randint(-1, S, (T,), generator=g, dtype=torch.int32)

    def adapters(rows, parts, K, N, div, xin, base):
        c = {"div": div, "topk": topk, "S": S, "E": E, "rank": rank, "parts": parts, "N": N, "K": K, "a": a, "ids": ids.cpu(),
             "x": xin.cpu(), "base": base.cpu(), "scale": torch.rand(S, generator=g) + 0.5,
             "A": (torch.randn((S, E, parts * rank, K), generator=g) * K ** -0.5).to(BF),
             "B": (torch.randn((S, E, N, rank), generator=g) * rank ** -0.5).to(BF)}
        return c, check(c)

    C1 = torch.empty((P, 2 * I), dtype=BF, device=DEV)
    chord.chord_w4a16_moe_gemm(x, topk, p13, E, 2 * I, H, order, blocks, count, bm, P, C1)
    _, C1 = adapters(P, 2, H, 2 * I, topk, x, C1)
    h = torch.empty((P, I), dtype=BF, device=DEV)
    chord.chord_silu_mul(C1, ids, E, h)
    gate, up = C1.double()[:, :I], C1.double()[:, I:]
    hd = gate * torch.sigmoid(gate) * up
    assert ((h.double() - hd).abs() <= (2.0 ** -8 + 2.0 ** -18) * hd.abs() + 1e-30).all()
    C2 = torch.empty((P, H), device=DEV)
    chord.chord_w4a16_moe_gemm(h, 1, p2, E, H, I, order, blocks, count, bm, P, C2, opts=chord.ChordOpts(out_dtype=chord.DTYPE_F32))
    _, C2 = adapters(P, 1, I, H, 1, h, C2)
    out = torch.empty((T, H), dtype=BF, device=DEV)
    chord.chord_moe_combine(C2, ids, w, E, out)
    assert chord.chord_get_device_error() == 0
    ref = (C2.double().reshape(T, topk, H) * w.double().unsqueeze(2)).sum(1)
    mag = (C2.double().reshape(T, topk, H) * w.double().unsqueeze(2)).abs().sum(1)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -21 * mag).all()


@gpu
@pytest.mark.parametrize("T", [20, 200, 6000])
def test_invalid_ids_of_tokens_whose_pairs_are_elsewhere(T):
    """An adapter id out of range is reported wherever the token's experts live (one launch, one plan, three kernels' plan)."""
    need_gpu()
    c = make(T, 4, 3, 5, 16, 1, 64, 64, 1, F32, seed=T, integer=True, foreign=0.3)
    c["ids"][7] = -1
    ref, _, written = reference(c)
    for value in (3, -2, 2 ** 31 - 1, -2 ** 31):
        d = on_gpu(c)
        d["a"][7] = value
        y = add(d, torch.zeros_like(d["base"]))
        assert chord.chord_get_device_error() == 7
        assert torch.equal(y.cpu()[written], ref[written].float()) and (y.cpu()[~written] == 0).all()


@gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("T", [4, 300])
def test_column_ranges_of_one_buffer(T, out):
    """x, base and y side by side in the rows of one buffer: none overlaps another."""
    need_gpu()
    c = make(T, 2, 3, 4, 16, 1, 96, 128, 1, out, seed=T + 1, integer=True)
    d = on_gpu(c)
    ref, _, written = reference(c)
    row = torch.full((2 * T, 128 + 128 + (96 if out == BF else 48) + 16), 3.0, dtype=out, device=DEV)
    for y0, b0 in ((0, 128), (128, 0)):
        base, y = row[:, b0:b0 + 128], row[:, y0:y0 + 128]
        base.copy_(d["base"])
        y.fill_(5.0)
        x = row.view(BF)[:, 256 * (1 if out == BF else 2):][:, :96]
        x.copy_(c["x"].to(DEV))
        d["x"] = x
        add(d, y, base=base)
        assert torch.equal(y.cpu()[written], ref.float().to(out)[written]) and (y.cpu()[~written] == 5).all()
        assert torch.equal(base.cpu(), c["base"]) and torch.equal(x.cpu(), c["x"]) and (row[:, -16:] == 3).all()
