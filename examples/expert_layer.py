"""An expert layer from router logits to combined hidden states, for one token,
a small decode batch and a prefill chunk, with its times.

    python examples/expert_layer.py [--hidden 2048 --inner 1024 --experts 128 --topk 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_ep_layout_02_gb300 as ep  # noqa: E402


def fp8_weights(E, N, K, dev):
    """Random weights of variance 1 / K as e4m3 codes with a scale per 128 x 128 block."""
    w = torch.randn(E, N // 128, 128, K // 128, 128, device=dev) * K ** -0.5
    scale = w.abs().amax(dim=(2, 4)) / 448.0
    q = (w / scale[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(E, N, K)
    return q, scale


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--topk", type=int, default=8)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    torch.manual_seed(0)
    layer = ep.ExpertLayer(*fp8_weights(a.experts, 2 * a.inner, a.hidden, dev),
                           *fp8_weights(a.experts, a.hidden, a.inner, dev), a.topk)
    gate = torch.randn(a.hidden, a.experts, device=dev, dtype=torch.bfloat16) * a.hidden ** -0.5
    for tokens in (1, 32, 4096):
        x = torch.randn(tokens, a.hidden, device=dev).to(torch.bfloat16)
        out = layer(x, x @ gate)
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            out = layer(x, x @ gate)
        stop.record()
        if ep.status_read(layer.status):
            raise RuntimeError("device status %d" % ep.status_read(layer.status))
        print("%5d tokens: %8.1f us per layer, |out| %.3f" % (
            tokens, start.elapsed_time(stop) * 1e3 / 20, out.float().abs().mean().item()))


if __name__ == "__main__":
    main()
