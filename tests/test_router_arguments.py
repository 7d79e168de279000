"""What the router and adapter calls refuse, before anything is launched: the
binding's checks of tensors, and the library's of sizes and pointers."""
import ctypes

import pytest
import torch

import w4a16_int4_mixture_moe_gb300 as chord
from test_four_bit_arguments import BF, F32, I32, dev, every_other, refused


@pytest.fixture(scope="module", autouse=True)
def lib():
    chord.build()
    return chord.load()


def status(call, args, at, bad):
    a = list(args)
    a[at] = bad
    return call(*a)


def test_logits_tensors():
    args = [dev(4, 64), dev(8, 64), dev(4, 8, dtype=F32)]
    for at, bad, name in ((0, dev(4, 64, dtype=F32), "x"), (0, dev(64), "x"), (0, dev(64, 4).t(), "x"), (0, torch.zeros(4, 64, dtype=BF), "x"),
                          (0, every_other(dev(4, 64)), "x"), (1, dev(8, 72), "W"), (1, dev(64), "W"), (1, dev(1, 3, 8, 64), "W"),
                          (1, dev(8, 64, dtype=F32), "W"), (1, every_other(dev(8, 64)), "W"), (2, dev(4, 8), "logits"),
                          (2, dev(3, 8, dtype=F32), "logits"), (2, dev(4, 16, dtype=F32)[:, :8], "logits")):
        refused(chord.chord_router_logits, args, at, bad, name)
    s = [dev(8, 64, dtype=F32), dev(3, 8, 64)]
    for at, bad, name in ((0, dev(8, 64), "W"), (0, dev(64, 8, dtype=F32).t(), "W"), (1, dev(2, 8, 64), "parts"), (1, dev(3, 8, 64, dtype=F32), "parts"),
                          (1, torch.zeros(3, 8, 64, dtype=BF), "parts")):
        refused(chord.chord_router_split_weights, s, at, bad, name)


def test_route_tensors():
    args = [dev(4, 16, dtype=F32), dev(4, 2, dtype=I32), dev(4, 2, dtype=F32)]
    for at, bad, name in ((0, dev(4, 16, dtype=torch.float16), "logits"), (0, dev(16), "logits"), (0, dev(16, 4).t(), "logits"),
                          (0, torch.zeros(4, 16), "logits"), (1, dev(4, 2, dtype=torch.int64), "topk_ids"), (1, dev(3, 2, dtype=I32), "topk_ids"),
                          (1, every_other(dev(4, 2, dtype=I32)), "topk_ids"), (2, dev(4, 3, dtype=F32), "topk_w"), (2, dev(4, 2), "topk_w")):
        refused(chord.chord_moe_route, args, at, bad, name)
    for bad in (dev(16), dev(15, dtype=F32), torch.zeros(16), every_other(dev(16, dtype=F32))):
        with pytest.raises(chord.ChordError) as ei:
            chord.chord_moe_route(*args, bias=bad)
        assert ": bias must be" in str(ei.value)


def adapter_args():
    # x, div, adapter_ids, topk_ids, A, B, scale, base, y, workspace
    return [dev(6, 64), 1, dev(3, dtype=I32), dev(3, 2, dtype=I32), dev(4, 5, 16, 64), dev(4, 5, 32, 16), dev(4, dtype=F32), dev(6, 32), dev(6, 32),
            dev(chord.chord_adapter_workspace_bytes(3, 2, 4, 5, 16, 1), dtype=torch.uint8)]


def test_adapter_tensors():
    args = adapter_args()
    for at, bad, name in ((0, dev(6, 64, dtype=F32), "x"), (0, dev(64, 6).t(), "x"), (2, dev(3, dtype=torch.int64), "adapter_ids"),
                          (3, dev(3, 2, dtype=torch.int64), "topk_ids"), (4, dev(4, 5, 24, 64), "A"), (4, dev(4, 5, 16, 72), "A"),
                          (4, dev(4, 16, 64), "A"), (4, dev(3, 5, 16, 64), "A"), (4, dev(4, 5, 16, 64, dtype=F32), "A"),
                          (5, dev(4, 5, 40, 16), "B"), (5, dev(4, 32, 16), "B"), (6, dev(3, dtype=F32), "scale"), (6, dev(4), "scale"),
                          (7, dev(6, 40), "base"), (7, dev(6, 32, dtype=torch.float16), "base"), (8, dev(6, 32, dtype=F32), "y"),
                          (8, dev(5, 32), "y"), (8, dev(32, 6).t(), "y"), (9, every_other(dev(4096, dtype=torch.uint8)), "workspace")):
        refused(chord.chord_adapter_add, args, at, bad, name)
    with pytest.raises(chord.ChordError):
        chord.chord_adapter_add(*args[:3], None, *args[4:])      # experts' adapters without their ids


def test_adapter_tensors_of_other_dimensions():
    args = adapter_args()
    for at, bad, name in ((0, dev(64), "x"), (3, dev(6, dtype=torch.int32), "topk_ids"), (3, dev(dtype=torch.int32), "topk_ids"),
                          (3, dev(1, 3, 2, dtype=torch.int32), "topk_ids"), (4, dev(64), "A"), (5, dev(16), "B"), (7, dev(32), "base"),
                          (7, dev(1, 6, 32), "base"), (8, dev(32), "y"), (8, dev(), "y")):
        refused(chord.chord_adapter_add, args, at, bad, name)


def test_workspace_bytes():
    f = chord.chord_adapter_workspace_bytes
    assert f(1, 1, 1, 1, 8, 1) > 0 and f(0, 1, 1, 1, 8, 1) > 0
    prev = 0
    for T in (1, 10, 100, 1000, 10000, 100000):
        assert f(T, 8, 4, 48, 16, 2) >= prev
        prev = f(T, 8, 4, 48, 16, 2)
    for bad in ((-1, 1, 1, 1, 8, 1), (1, 0, 1, 1, 8, 1), (1, 1, 0, 1, 8, 1), (1, 1, 1, 0, 8, 1), (1, 1, 1, 1, 0, 1), (1, 1, 1, 1, 8, 0),
                (1, 1, 1, 1, 136, 1), (1, 1, 1, 1, 8, 5), (2 ** 31, 1, 1, 1, 8, 1), (2 ** 30, 2, 1, 1, 8, 1), (1, 1, 65537, 1, 8, 1),
                (1, 1, 2, 65536, 8, 1)):
        assert f(*bad) == 0, bad


P = 0x10000   # an aligned address that nothing reads: every call below is refused first


def test_logits_sizes(lib):
    #       x  stride T  W  parts E  H   logits opts stream
    args = [P, 64, 4, P, 1, 8, 64, P, None, None]
    call = lib.chord_router_logits
    for at, bad, st in ((0, None, 1), (0, P + 8, 1), (1, 56, 1), (1, 68, 2), (2, -1, 1), (3, None, 1), (3, P + 2, 1), (4, 2, 2), (4, 0, 2),
                        (5, 0, 1), (5, 1025, 2), (6, 0, 1), (6, -8, 1), (7, None, 1), (7, P + 2, 1)):
        assert status(call, args, at, bad) == st, (at, bad)
    assert call(P, 68, 4, P, 1, 8, 68, P, None, None) == 2
    assert call(None, 64, 0, P, 1, 8, 64, None, None, None) == 0       # no rows
    split = lib.chord_router_split_weights
    assert split(P, -1, P, None) == 1 and split(None, 8, P, None) == 1 and split(P, 8, None, None) == 1
    assert split(P + 1, 8, P, None) == 1 and split(P, 8, P + 1, None) == 1 and split(P, 2 ** 62, P, None) == 2
    assert split(None, 0, None, None) == 0


def test_route_sizes(lib):
    call = lib.chord_moe_route

    def how(**kw):
        h = dict(score=0, groups=1, topk_groups=1, group_best=1, renormalize=1, scale=1.0, first=0, E_local=16)
        h.update(kw)
        return ctypes.byref(chord.ChordRoute(**h))

    #       logits dtype stride T E bias topk how ids w stream
    args = [P, 1, 16, 4, 16, None, 2, how(), P, P, None]
    for at, bad, st in ((0, None, 1), (0, P + 2, 1), (1, 2, 1), (2, 15, 1), (3, -1, 1), (4, 0, 1), (4, 1025, 1), (6, 0, 1), (6, 17, 1), (7, None, 1),
                        (8, None, 1), (9, None, 1),
                        (7, how(score=2), 1), (7, how(groups=0), 1), (7, how(groups=3), 1), (7, how(topk_groups=2), 1), (7, how(topk_groups=0), 1),
                        (7, how(group_best=0), 1), (7, how(group_best=3), 1), (7, how(first=-1), 1), (7, how(first=1), 1), (7, how(E_local=0), 1),
                        (7, how(E_local=17), 1), (7, how(first=2 ** 31 - 1, E_local=2 ** 31 - 1), 1), (7, how(groups=16, topk_groups=1), 1)):
        assert status(call, args, at, bad) == st, (at, bad)
    assert call(P, 1, 2048, 4, 2048, None, 2, how(E_local=2048), P, P, None) == 2
    assert call(P, 1, 64, 4, 64, None, 33, how(E_local=64), P, P, None) == 2
    assert call(P, 1, 64, 4, 64, None, 2, how(E_local=64, groups=64, topk_groups=64), P, P, None) == 2
    assert call(P, 1, 64, 2 ** 30, 64, None, 2, how(E_local=64), P, P, None) == 2
    assert call(P + 1, 0, 16, 4, 16, None, 2, how(), P, P, None) == 1
    assert call(None, 1, 0, 0, 16, None, 2, how(), None, None, None) == 0


def test_adapter_sizes(lib):
    call = lib.chord_adapter_add
    names = ("x x_rows x_stride div adapter_ids topk_ids T topk adapters E A B scale rank parts N K base base_stride y y_stride dtype ws ws_bytes "
             "opts stream").split()
    far = [P * (k + 1) for k in range(16)]
    args = [far[0], 6, 64, 1, far[1], far[2], 3, 2, 4, 5, far[3], far[4], None, 16, 1, 32, 64, far[5], 32, far[6], 32, 0, far[7],
            chord.chord_adapter_workspace_bytes(3, 2, 4, 5, 16, 1), None, None]
    at = {n: i for i, n in enumerate(names)}
    assert len(args) == len(names)
    for n, bad, st in (("x", None, 1), ("x", far[0] + 8, 1), ("x_rows", 5, 1), ("x_rows", -1, 1), ("x_stride", 56, 1), ("x_stride", 68, 2), ("div", 0, 1),
                       ("adapter_ids", None, 1), ("topk_ids", None, 1), ("T", -1, 1), ("T", 2 ** 31 - 1, 2), ("topk", 0, 1), ("adapters", 0, 1),
                       ("adapters", 13108, 2), ("E", 0, 1), ("A", None, 1), ("A", far[3] + 2, 1), ("B", None, 1), ("B", far[4] + 4, 1), ("rank", 0, 1),
                       ("rank", 12, 2), ("rank", 136, 2), ("parts", 0, 1), ("parts", 5, 2), ("parts", 3, 2), ("N", 0, 1), ("N", 36, 2), ("K", 0, 1),
                       ("K", 60, 2), ("base", None, 1), ("base", far[5] + 8, 1), ("base_stride", 24, 1), ("base_stride", 36, 2), ("y", None, 1),
                       ("y", far[6] + 8, 1), ("y_stride", 24, 1), ("y_stride", 36, 2), ("dtype", 2, 1), ("ws", None, 1), ("ws", far[7] + 8, 1),
                       ("ws_bytes", args[at["ws_bytes"]] - 1, 4),
                       ("y", far[5] + 64, 1), ("y", far[0], 1), ("y", far[0] + 16, 1)):      # y over base, over x
        assert status(call, args, at[n], bad) == st, (n, bad)
    a = list(args)
    a[at["y"]], a[at["y_stride"]] = a[at["base"]], 40         # in place with another stride
    assert call(*a) == 1
    a = list(args)
    a[at["T"]] = 0
    assert call(*a) == 0


def test_workspace_never_shrinks_with_more_tokens():
    """Scratch for the largest batch is enough for every smaller one."""
    f = chord.chord_adapter_workspace_bytes
    for topk, S, E, rank, parts in ((8, 4, 48, 16, 2), (1, 8, 1, 64, 1), (3, 200, 1, 8, 1), (2, 1, 300, 128, 4)):
        # every number of tokens up to 3000, and both sides of every step of 16384 / pairs
        counts = {*range(3000), *(p // topk + d for k in range(1, 17) for p in (16384 // k, 32768 * k) for d in (-1, 0, 1, 2))}
        prev = 0
        for T in sorted(counts):
            now = f(T, topk, S, E, rank, parts)
            assert now >= prev, (T, topk)
            prev = now


def test_overlap_is_of_rows_not_of_their_range(lib):
    """y and base, or y and x, may be column ranges of one buffer; not with a byte in common.  The scratch is too small in
    every call, which is found after the overlap: nothing is launched."""
    n = chord.chord_adapter_workspace_bytes(3, 2, 4, 5, 16, 1)

    def call(x, xs, base, bs, y, ys, dtype=0):
        return lib.chord_adapter_add(x, 6, xs, 1, P * 9, P * 10, 3, 2, 4, 5, P * 11, P * 12, None, 16, 1, 32, 64, base, bs, y, ys, dtype, P * 13, n - 1,
                                     None, None)

    far = P * 20
    # 6 rows of x are 64 bf16, of base and y 32 bf16; a buffer of 128 bf16 a row
    for y, st in ((P + 64, 4), (P + 128, 4), (P + 192, 4), (P + 48, 1), (P + 16, 1), (P - 16, 1), (P - 64, 4), (P + 256 * 6, 4), (P + 256 * 3 + 64, 4),
                  (P + 256 * 3 + 48, 1), (P + 256 * 5 - 16, 1), (P + 256 * 5 + 64, 4), (P - 256 * 2 + 128, 4), (P - 256 * 2 + 208, 1)):
        assert call(far, 64, P, 128, y, 128) == st, y - P
    for y, st in ((P, 1), (P + 64, 1), (P + 128, 4), (P + 192, 4), (P + 208, 1), (P - 64, 4), (P - 48, 1), (P + 256 * 2 + 112, 1), (P + 256 * 2 + 128, 4)):
        assert call(P, 128, far, 32, y, 128) == st, y - P
    # another row distance: the ranges decide; FP32 rows in the buffer of bf16 ones
    assert call(far, 64, P, 128, P + 64, 136) == 1 and call(far, 64, P, 128, P + 256 * 6, 136) == 4
    assert call(P, 128, far, 32, P + 128, 64, dtype=1) == 4 and call(P, 128, far, 32, P + 112, 64, dtype=1) == 1
    # rows of base that lie closer than y's are wide
    assert call(far, 64, P, 32, P + 32, 32) == 1 and call(far, 64, P, 32, P, 32) == 4


def test_route_outputs_without_dimensions():
    args = [dev(4, 16, dtype=F32), dev(4, 2, dtype=I32), dev(4, 2, dtype=F32)]
    refused(chord.chord_moe_route, args, 1, dev(dtype=I32), "topk_ids")
    refused(chord.chord_moe_route, args, 2, dev(dtype=F32), "topk_w")
