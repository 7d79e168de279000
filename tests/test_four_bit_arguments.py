"""The binding refuses tensors that the library would misread: other types (int64
ids, as topk returns them), other shapes, strided tensors, host memory.  The
library sees addresses only, so nothing below it can notice."""
import pytest
import torch

import w4a16_int4_mixture_moe_gb300 as chord

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Dev(torch.Tensor):
    """A host tensor that says it is in device memory: what is left to find is what is wrong with it."""

    @property
    def is_cuda(self):
        return True


def dev(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(Dev)


def refused(call, args, at, bad, name):
    a = list(args)
    a[at] = bad
    with pytest.raises(chord.ChordError) as ei:
        call(*a)
    assert ei.value.status == 1 and f": {name} must be" in str(ei.value)


class FakeStream:
    cuda_stream = 77


def test_current_stream_without_torch_internals(monkeypatch):
    """The stream handle comes from torch's public call where its internal ones are
    missing, take other arguments or disagree; a given stream is used as it is."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: FakeStream)
    for raw, device in ((None, None), (lambda: 5, lambda: 0), (lambda d: 5, lambda: 0), (lambda d: 77, lambda: 0)):
        monkeypatch.setattr(chord, "_current_stream", None)
        for name, f in (("_cuda_getCurrentRawStream", raw), ("_cuda_getDevice", device)):
            if f is None:
                monkeypatch.delattr(torch._C, name, raising=False)
            else:
                monkeypatch.setattr(torch._C, name, f, raising=False)
        assert chord._s(None) == 77 and chord._s(None) == 77
    assert chord._s(FakeStream) == 77 and chord._s(0) == 0 and chord._s(9) == 9


def every_other(t):
    """The same shape, two elements apart."""
    return t.repeat_interleave(2, dim=-1)[..., ::2]


def test_layer():
    T, topk, E, H, I = 4, 2, 8, 256, 128
    args = [dev(T, H), dev(T, topk, dtype=I32), dev(T, topk, dtype=F32), E, I,
            dev(chord.chord_packed_weight_bytes(E, 2 * I, H), dtype=torch.uint8),
            dev(chord.chord_packed_weight_bytes(E, H, I), dtype=torch.uint8),
            dev(chord.chord_moe_few_workspace_bytes(T, topk, E, H, I), dtype=torch.uint8), dev(T, H)]
    for at, name in ((0, "x"), (1, "topk_ids"), (2, "topk_w"), (5, "packed_w13"), (6, "packed_w2"), (7, "workspace"),
                     (8, "out")):
        refused(chord.chord_moe_layer_few, args, at, every_other(args[at]), name)
        refused(chord.chord_moe_layer_few, args, at, torch.zeros_like(args[at].as_subclass(torch.Tensor)), name)
    for at, bad, name in ((0, dev(T, H, dtype=F32), "x"), (0, dev(T, H, dtype=torch.float16), "x"),
                          (1, dev(T, topk, dtype=torch.int64), "topk_ids"), (2, dev(T, topk), "topk_w"),
                          (2, dev(T, topk, dtype=torch.float64), "topk_w"), (2, dev(T, topk + 1, dtype=F32), "topk_w"),
                          (1, dev(T - 1, topk, dtype=I32), "topk_ids"), (8, dev(T, H, dtype=F32), "out"),
                          (8, dev(T - 1, H), "out"), (8, dev(T, H + 8), "out"),
                          (0, dev(H, T).t(), "x")):
        refused(chord.chord_moe_layer_few, args, at, bad, name)


def test_quantise_and_dequantise():
    blob = dev(chord.chord_mxfp4_bytes(2, 8, 64), dtype=torch.uint8)
    q = [dev(2, 8, 64), blob]
    refused(chord.chord_mxfp4_quantize, q, 0, dev(8, 64), "src")
    refused(chord.chord_mxfp4_quantize, q, 0, dev(2, 64, 8).transpose(1, 2), "src")
    refused(chord.chord_mxfp4_quantize, q, 0, torch.zeros(2, 8, 64), "src")
    refused(chord.chord_mxfp4_quantize, q, 1, every_other(blob), "packed")
    d = [blob, dev(2, 8, 64)]
    refused(chord.chord_mxfp4_dequantize, d, 1, dev(2, 8, 72)[:, :, :64], "out")
    refused(chord.chord_mxfp4_dequantize, d, 1, dev(8, 2, 64).transpose(0, 1), "out")
    refused(chord.chord_mxfp4_dequantize, d, 0, every_other(blob), "packed")
    for call, args in ((chord.chord_mxfp4_quantize, q), (chord.chord_mxfp4_dequantize, list(reversed(d)))):
        with pytest.raises(chord.ChordError):
            call(*([dev(2, 8, 64, dtype=torch.float16), blob] if call is chord.chord_mxfp4_quantize
                   else [blob, dev(2, 8, 64, dtype=torch.float16)]))
    bm, cap, K = 32, 64, 64
    r = [dev(8, K), 2, dev(cap, dtype=I32), dev(1, dtype=I32), bm, 16,
         dev(chord.chord_mxfp4_rows_bytes(cap, bm, K), dtype=torch.uint8)]
    for at, bad, name in ((0, dev(K, 8).t(), "A"), (0, dev(1, 8, K), "A"), (2, dev(cap, dtype=torch.int64), "sorted_ids"),
                          (2, every_other(dev(cap, dtype=I32)), "sorted_ids"),
                          (3, dev(1, dtype=torch.int64), "num_tokens_padded"), (3, dev(0, dtype=I32), "num_tokens_padded")):
        refused(chord.chord_mxfp4_quantize_rows, r, at, bad, name)


@pytest.mark.parametrize("shape", [(8, 40), (9, 40), (4, 2, 40), (1, 8, 40)])
def test_dense_tensors_of_other_leading_dimensions_pass(shape):
    t = dev(*shape, dtype=F32)
    assert chord._dense("call", "C", t, None, 8, 40) == t.data_ptr()
    assert chord._dense("call", "C", t, F32, 8, 40) == t.data_ptr()


def test_products():
    E, N, K, bm, cap, P = 2, 40, 64, 32, 64, 8
    xq = dev(chord.chord_mxfp4_rows_bytes(cap, bm, K), dtype=torch.uint8)
    wq = dev(chord.chord_mxfp4_bytes(E, N, K), dtype=torch.uint8)
    g = [xq, wq, E, N, K, dev(cap, dtype=I32), dev(cap // bm, dtype=I32), dev(1, dtype=I32), bm, P, dev(P, N)]
    for at, bad, name in ((5, dev(cap, dtype=torch.int64), "sorted_ids"), (6, dev(cap // bm, dtype=torch.int64), "expert_ids"),
                          (6, dev(cap // bm - 1, dtype=I32), "expert_ids"), (7, dev(1, dtype=F32), "num_tokens_padded"),
                          (10, dev(P - 1, N), "C"), (10, dev(P, N + 8)[:, :N], "C"), (10, dev(N, P).t(), "C"),
                          (0, every_other(xq), "Aq"), (1, every_other(wq), "packed"), (10, torch.zeros(P, N), "C")):
        refused(chord.chord_mxfp4_moe_gemm, g, at, bad, name)
    d = [dev(chord.chord_mxfp4_bytes(1, P, K), dtype=torch.uint8), P, dev(chord.chord_mxfp4_bytes(1, N, K), dtype=torch.uint8),
         N, K, dev(P, N, dtype=F32)]
    for bad in (dev(P, N + 1), dev(P - 1, N), dev(N, P).t(), every_other(dev(P, N))):
        refused(chord.chord_mxfp4_gemm, d, 5, bad, "C")
    with pytest.raises(chord.ChordError):
        chord.chord_mxfp4_gemm(*d[:5], dev(P, N, dtype=I32))
