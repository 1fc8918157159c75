"""A feed-forward block in 8-bit floating point, dense and by expert, on one GPU.

    h = x + residual;  y = down(silu(gate(norm(h))) * up(norm(h)))

Four calls: the norm with the residual's addition ends in quantised rows, the first
product gives the gate's and the up projection's columns side by side, the gated
activation reads the two halves and ends in quantised rows, the second product gives y.
Tokens of requests with a low-rank adapter get its part added to the first product's
columns, read from the same quantised rows.
By expert, the first product gathers each token's row for every expert it chose, and the
rows stay in the experts' order.  With a router's scores, its choice and order are one
call ahead of the products, and the weighted sum back in the tokens' order one behind.

    python examples/fp8_feed_forward.py [--tokens 4096] [--hidden 4096] [--ffn 8192]
                                        [--experts 16] [--top 2]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w4a16_dequant_gemm_amd import fp8, lora, route, rowquant  # noqa: E402


def quantise_weights(w):
    """[..., N, K] float weights -> E4M3 codes and a scale per block of 128 x 128."""
    *lead, N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    padded = torch.nn.functional.pad(w.float(), (0, kb * 128 - K, 0, nb * 128 - N))
    tiles = padded.view(*lead, nb, 128, kb, 128)
    s = tiles.abs().amax((-3, -1)).clamp(min=2.0 ** -110) / 448.0
    q = (tiles / s[..., :, None, :, None]).view(*lead, nb * 128, kb * 128)[..., :N, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), s


class FeedForward:
    """Dense: gate_up [2F][H], down [H][F].  By expert: the same with a leading [E]."""

    def __init__(self, norm_weight, gate_up, down, eps=1e-6):
        self.norm_weight, self.eps = norm_weight, eps
        self.ffn = down.shape[-1]
        self.gate_up = fp8.fp8_repack(*quantise_weights(gate_up))
        self.down = fp8.fp8_repack(*quantise_weights(down))

    def _activation(self, both):
        return rowquant.swiglu_quantize_rows(both[:, :self.ffn], both[:, self.ffn:])

    def dense(self, x, residual, adapters=None):
        """adapters: (a [L][R][H], b [L][2F][R], ids int32 [T], scale [L])."""
        q, s, h = rowquant.rmsnorm_quantize_rows(x, self.norm_weight, residual=residual,
                                                 eps=self.eps)
        both = fp8.fp8_gemm(q, s, self.gate_up)
        if adapters is not None:
            a, b, ids, scale = adapters
            lora.lora_add(both, q, a, b, ids, scale=scale, xs=s, out=both)
        q, s = self._activation(both)
        return fp8.fp8_gemm(q, s, self.down), h

    def experts(self, x, residual, chosen, weight):
        """chosen, weight [T][top]: each token's experts and how much of each it takes."""
        top = chosen.shape[1]
        order = torch.argsort(chosen.reshape(-1), stable=True)
        offsets = torch.zeros(self.down.E + 1, dtype=torch.int32, device=x.device)
        offsets[1:] = torch.bincount(chosen.reshape(-1), minlength=self.down.E).cumsum(0)
        rows = (order // top).to(torch.int32)
        q, s, h = rowquant.rmsnorm_quantize_rows(x, self.norm_weight, residual=residual,
                                                 eps=self.eps)
        q, s = self._activation(fp8.fp8_grouped_gemm(q, s, self.gate_up, offsets, rows=rows))
        y = fp8.fp8_grouped_gemm(q, s, self.down, offsets)
        back = torch.empty_like(y)
        back[order] = y
        return (back.view(*chosen.shape, -1).float() * weight[..., None]).sum(1).to(x.dtype), h

    def routed(self, x, residual, logits, top):
        """logits [T][E]: the router's scores; each token takes its top experts, weighted by
        the softmax over them."""
        r = route.route_tokens(logits, top)
        q, s, h = rowquant.rmsnorm_quantize_rows(x, self.norm_weight, residual=residual,
                                                 eps=self.eps)
        q, s = self._activation(fp8.fp8_grouped_gemm(q, s, self.gate_up, r.offsets, rows=r.rows))
        y = fp8.fp8_grouped_gemm(q, s, self.down, r.offsets)
        return route.combine_rows(y, r.weights, r.places), h


def reference(x, residual, norm_weight, gate_up, down, eps=1e-6):
    """The block in fp32 with unquantised weights."""
    h = x.float() + residual.float()
    v = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * norm_weight.float()
    g, u = (v @ gate_up.float().t()).chunk(2, dim=1)
    return (torch.nn.functional.silu(g) * u) @ down.float().t()


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("hidden", 4096), ("ffn", 8192), ("experts", 16),
                        ("top", 2)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    torch.manual_seed(0)
    d, dt = "cuda", torch.bfloat16
    x, r = (torch.randn(a.tokens, a.hidden, device=d, dtype=dt) for _ in range(2))
    wn = torch.ones(a.hidden, device=d, dtype=dt)
    gu = torch.randn(a.experts, 2 * a.ffn, a.hidden, device=d, dtype=dt) * a.hidden ** -0.5
    dn = torch.randn(a.experts, a.hidden, a.ffn, device=d, dtype=dt) * a.ffn ** -0.5

    one = FeedForward(wn, gu[0], dn[0])
    many = FeedForward(wn, gu, dn)
    logits = torch.randn(a.tokens, a.experts, device=d)
    weight, chosen = logits.softmax(1).topk(a.top, dim=1)
    weight = weight / weight.sum(1, keepdim=True)
    n = min(a.tokens, 64)
    y, _ = one.dense(x, r)
    want = reference(x[:n], r[:n], wn, gu[0], dn[0])
    err = ((y[:n].float() - want).norm() / want.norm()).item()
    ye, _ = many.experts(x, r, chosen, weight)
    yr, _ = many.routed(x, r, logits, a.top)
    wante = torch.stack([sum(weight[t, i] * reference(x[t:t + 1], r[t:t + 1], wn, gu[e], dn[e])[0]
                             for i, e in enumerate(chosen[t].tolist())) for t in range(min(n, 8))])
    erre, errr = (((z[:len(wante)].float() - wante).norm() / wante.norm()).item() for z in (ye, yr))
    # four adapters of rank 16, each for runs of tokens; every fifth run has none
    la = torch.randn(4, 16, a.hidden, device=d, dtype=dt) * a.hidden ** -0.5
    lb = torch.randn(4, 2 * a.ffn, 16, device=d, dtype=dt) * 0.25 * a.hidden ** -0.5
    ids = (torch.arange(a.tokens, device=d) // 16 % 5 - 1).to(torch.int32)
    adapters = (la, lb, ids, torch.ones(4, device=d))
    ya, _ = one.dense(x, r, adapters)
    wanta = torch.cat([reference(x[t:t + 1], r[t:t + 1], wn,
                                 gu[0] if i < 0 else gu[0].float() + lb[i].float() @ la[i].float(),
                                 dn[0]) for t, i in enumerate(ids[:n].tolist())])
    erra = ((ya[:n].float() - wanta).norm() / wanta.norm()).item()

    def us(f, reps=20):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(reps):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / reps * 1e6

    print(f"dense   {a.tokens} tokens {a.hidden} -> {a.ffn}: {us(lambda: one.dense(x, r)):.1f} us, "
          f"off by {err:.4f} of the fp32 block with unquantised weights")
    print(f"experts {a.tokens} tokens, {a.top} of {a.experts}: "
          f"{us(lambda: many.experts(x, r, chosen, weight)):.1f} us, off by {erre:.4f}; with the "
          f"router {us(lambda: many.routed(x, r, logits, a.top)):.1f} us, off by {errr:.4f}")
    print(f"dense with adapters of 4 requests: {us(lambda: one.dense(x, r, adapters)):.1f} us, "
          f"off by {erra:.4f}")
    # 8-bit rows and weights: 4 significant bits each, about 2.6% per operand in the norm
    assert max(err, erre, errr, erra) < 0.08


if __name__ == "__main__":
    main()
