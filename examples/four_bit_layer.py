"""A mixture-of-experts layer with 4-bit experts, from bf16 weights to tokens.

    python examples/four_bit_layer.py [--tokens 512] [--experts 16] [--hidden 1024] [--inter 512]

1. load time: the bf16 expert weights are quantised to MXFP4 (chord_mxfp4_quantize);
2. prefill: a chunk of tokens goes through the microscaled products, the routed
   activation rows quantised on the way in;
3. decode: a few tokens go through the two-kernel layer, bf16 activations times
   the same packed weights.

Prints how far each path is from the bf16 layer: what 4-bit weights cost, and
what 4-bit activations add in prefill.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a16_int4_mixture_moe_gb300 as chord

DEV = "cuda:0"


def empty(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device=DEV)


class FourBitLayer:
    """Expert weights w13 [E, 2I, H] (gate rows, then up rows) and w2 [E, H, I], packed once."""

    def __init__(self, w13, w2):
        self.E, I2, self.H = w13.shape
        self.I = I2 // 2
        self.w13 = empty(chord.chord_mxfp4_bytes(self.E, I2, self.H))
        self.w2 = empty(chord.chord_mxfp4_bytes(self.E, self.H, self.I))
        chord.chord_mxfp4_quantize(w13, self.w13)
        chord.chord_mxfp4_quantize(w2, self.w2)

    def _product(self, x, div, weights, N, K, route, bm, P, dtype):
        """Rows of x (one per token or per pair), quantised in routed order, times each expert's weights."""
        ids, experts, count = route
        xq = empty(chord.chord_mxfp4_rows_bytes(ids.numel(), bm, K))
        C = empty(P, N, dtype=dtype)
        chord.chord_mxfp4_quantize_rows(x, div, ids, count, bm, P, xq)
        chord.chord_mxfp4_moe_gemm(xq, weights, self.E, N, K, ids, experts, count, bm, P, C)
        return C

    def prefill(self, x, topk_ids, topk_w):
        T, topk = topk_ids.shape
        P = T * topk
        bm = chord.chord_mxfp4_select_block_m(T, topk, self.E, self.E)
        cap = chord.chord_align_capacity(T, topk, self.E, bm)
        route = (empty(cap, dtype=torch.int32), empty(cap // bm, dtype=torch.int32), empty(1, dtype=torch.int32))
        chord.chord_moe_align(topk_ids, self.E, bm, *route, empty(chord.chord_align_workspace_bytes(T, topk, self.E)))
        C1 = self._product(x, topk, self.w13, 2 * self.I, self.H, route, bm, P, torch.bfloat16)
        h = empty(P, self.I, dtype=torch.bfloat16)
        chord.chord_silu_mul(C1, topk_ids, self.E, h)
        C2 = self._product(h, 1, self.w2, self.H, self.I, route, bm, P, torch.float32)
        out = empty(T, self.H, dtype=torch.bfloat16)
        chord.chord_moe_combine(C2, topk_ids, topk_w, self.E, out)
        return out

    def decode(self, x, topk_ids, topk_w):
        T, topk = topk_ids.shape
        ws = empty(chord.chord_moe_few_workspace_bytes(T, topk, self.E, self.H, self.I))
        out = empty(T, self.H, dtype=torch.bfloat16)
        chord.chord_moe_layer_few(x, topk_ids, topk_w, self.E, self.I, self.w13, self.w2, ws, out,
                                  weights=chord.WEIGHTS_MXFP4)
        return out

    def values(self):
        """The weights the packed matrices stand for."""
        v13, v2 = empty(self.E, 2 * self.I, self.H, dtype=torch.float32), empty(self.E, self.H, self.I, dtype=torch.float32)
        chord.chord_mxfp4_dequantize(self.w13, v13)
        chord.chord_mxfp4_dequantize(self.w2, v2)
        return v13, v2


def reference(x, topk_ids, topk_w, w13, w2):
    """The layer's formula in fp32."""
    out = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    I = w2.shape[2]
    for e in range(w13.shape[0]):
        t, k = (topk_ids == e).nonzero(as_tuple=True)
        if t.numel():
            c1 = x[t].float() @ w13[e].float().t()
            h = torch.nn.functional.silu(c1[:, :I]) * c1[:, I:]
            out.index_add_(0, t, (h @ w2[e].float().t()) * topk_w[t, k].unsqueeze(1))
    return out


def relative(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inter", type=int, default=512)
    a = ap.parse_args(argv)
    chord.build()
    g = torch.Generator(device=DEV).manual_seed(1)
    w13 = (torch.randn(a.experts, 2 * a.inter, a.hidden, generator=g, device=DEV) * a.hidden ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(a.experts, a.hidden, a.inter, generator=g, device=DEV) * a.inter ** -0.5).to(torch.bfloat16)
    x = torch.randn(a.tokens, a.hidden, generator=g, device=DEV).to(torch.bfloat16)
    logits = torch.randn(a.tokens, a.experts, generator=g, device=DEV)
    w, ids = torch.softmax(logits, dim=1).topk(a.topk, dim=1)
    ids, w = ids.to(torch.int32).contiguous(), (w / w.sum(dim=1, keepdim=True)).contiguous()
    layer = FourBitLayer(w13, w2)
    few = min(a.tokens, chord.FEW_MAX_TOKENS)
    out = {"prefill": layer.prefill(x, ids, w),
           "decode": layer.decode(x[:few].contiguous(), ids[:few].contiguous(), w[:few].contiguous())}
    code = chord.chord_get_device_error()
    if code:
        raise RuntimeError(f"device error word {code}")
    full = reference(x, ids, w, w13, w2)
    same = reference(x, ids, w, *layer.values())
    result = {"weights": relative(same, full), "decode": relative(out["decode"], same[:few]),
              "prefill": relative(out["prefill"], same)}
    print(f"4-bit weights against bf16 weights        {result['weights']:.4f}")
    print(f"decode  ({few} tokens) against those weights  {result['decode']:.4f}")
    print(f"prefill ({a.tokens} tokens) against those weights {result['prefill']:.4f}  (activations in 4 bits)")
    return result


if __name__ == "__main__":
    main()
