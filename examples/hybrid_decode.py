"""Serves a small random-weight hybrid stack: Gated DeltaNet, decayed linear attention and
softmax attention over a paged 4-bit key/value cache, one after the other.

    python examples/hybrid_decode.py [--prompts 4] [--length 2000] [--tokens 64]

Packed prompts of different lengths go through ``prefill``; then every ``step`` feeds one
token per sequence, replayed as one CUDA graph.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_11_gb300 as gdn  # noqa: E402

D = 128                          # head size of every mixer
DELTA, LINEAR, ATTENTION = "delta", "linear", "attention"


def rms_norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class HybridStack:
    """Token mixers ``kinds`` with residuals around them; Hk key and Hv value heads (for
    attention: Hv query heads over Hk key/value heads).  Holds the states of up to
    ``sequences`` sequences of up to ``max_len`` tokens."""

    def __init__(self, kinds, hidden=512, vocab=1000, Hk=2, Hv=8, sequences=4, max_len=4096,
                 page=32, seed=0, device="cuda"):
        self.kinds, self.Hk, self.Hv, self.N, self.max_len = kinds, Hk, Hv, sequences, max_len
        gen = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen) * rows ** -0.5).bfloat16().to(device)

        self.embed = weight(hidden, vocab).t().contiguous() * hidden ** 0.5
        self.out = weight(hidden, vocab)
        self.qkv_width = (2 * Hk + Hv) * D
        extra = {DELTA: 2 * Hv, LINEAR: 0, ATTENTION: 0}
        self.w_in = [weight(hidden, self.qkv_width + extra[x]) for x in kinds]
        self.w_out = [weight(Hv * D, hidden) for _ in kinds]
        self.conv = weight(4, self.qkv_width).t().contiguous()
        self.decay = -torch.exp2(-torch.linspace(3, 9, Hv, device=device))      # LINEAR's, per head
        angle = torch.arange(max_len)[:, None] * 10000.0 ** (-torch.arange(0, D, 2) / D)
        self.cos, self.sin = angle.cos().to(device), angle.sin().to(device)
        # per layer: recurrent states, or the cache; one table of pages serves every cache
        self.state = [None if x == ATTENTION else
                      torch.zeros(sequences, Hv, D, D, device=device) for x in kinds]
        self.conv_state = [torch.zeros(sequences, 3, self.qkv_width, dtype=torch.bfloat16,
                                       device=device) if x == DELTA else None for x in kinds]
        width = -(-max_len // page)
        self.cache = [gdn.gdn_kv_cache(sequences * width, page, Hk, D, device)
                      if x == ATTENTION else None for x in kinds]
        pages = torch.randperm(sequences * width, generator=gen)
        self.table = pages.int().view(sequences, width).to(device)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)

    def _split(self, qkv):
        q, k, v = qkv.split([self.Hk * D, self.Hk * D, self.Hv * D], dim=-1)
        return q.unflatten(-1, (-1, D)), k.unflatten(-1, (-1, D)), v.unflatten(-1, (-1, D))

    def _split_attention(self, qkv):        # Hv query heads, Hk heads each of keys and values
        q, k, v = qkv.split([self.Hv * D, self.Hk * D, self.Hk * D], dim=-1)
        return q.unflatten(-1, (-1, D)), k.unflatten(-1, (-1, D)), v.unflatten(-1, (-1, D))

    def _gates(self, h):
        a, b = h[:, self.qkv_width:].float().chunk(2, dim=-1)
        return -torch.nn.functional.softplus(a), torch.sigmoid(b)

    def _attend(self, i, qkv, **new):
        q, k, v = self._split_attention(qkv)
        q = gdn.gdn_kv_append(k, v, self.cache[i], self.table, self.lens, cos=self.cos,
                              sin=self.sin, q=q, **new)
        return gdn.gdn_kv_attention(q, self.cache[i], self.table, self.lens, **new)

    def prefill(self, tokens, cu):
        """Logits [N, vocab] after packed prompts; ``cu`` int32 offsets, on the host."""
        cu_dev = cu.to(tokens.device)
        self.lens.copy_(cu[1:] - cu[:-1])
        new = dict(cu_seqlens=cu_dev, cu_seqlens_host=cu)
        x = self.embed[tokens]
        for i, kind in enumerate(self.kinds):
            h = rms_norm(x) @ self.w_in[i]
            qkv = h[:, :self.qkv_width]
            if kind == DELTA:
                g, beta = self._gates(h)
                o, _, _ = gdn.gdn_layer_prefill(
                    qkv.contiguous(), self.conv, None, g, beta, cu_dev, self.Hk, self.Hv, D, D,
                    cu_seqlens_host=cu, conv_state_out=self.conv_state[i],
                    final_state=self.state[i])
            elif kind == LINEAR:
                q, k, v = self._split(qkv)
                o, _ = gdn.gdn_linear_prefill(q, k, v, self.decay, scale=1 / D,
                                              final_state=self.state[i], **new)
            else:
                o = self._attend(i, qkv, **new)
            x = x + o.flatten(1) @ self.w_out[i]
        return rms_norm(x[cu_dev[1:].long() - 1]) @ self.out

    def step(self, tokens):
        """Logits [N, vocab] after one more token per sequence."""
        self.lens += 1
        x = self.embed[tokens]
        for i, kind in enumerate(self.kinds):
            h = rms_norm(x) @ self.w_in[i]
            qkv = h[:, :self.qkv_width]
            if kind == DELTA:
                g, beta = self._gates(h)
                o = gdn.gdn_layer_decode(qkv.contiguous(), self.conv, None, g, beta,
                                         self.conv_state[i], self.state[i], self.Hk, self.Hv,
                                         D, D)
            elif kind == LINEAR:
                q, k, v = self._split(qkv)
                o = gdn.gdn_linear_decode(q, k, v, self.decay, self.state[i], scale=1 / D)
            else:
                o = self._attend(i, qkv)
            x = x + o.flatten(1) @ self.w_out[i]
        return rms_norm(x) @ self.out


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompts", type=int, default=4)
    ap.add_argument("--length", type=int, default=2000, help="of the longest prompt")
    ap.add_argument("--tokens", type=int, default=64, help="to answer with, per prompt")
    a = ap.parse_args()
    kinds = (DELTA, LINEAR, DELTA, ATTENTION)
    net = HybridStack(kinds, sequences=a.prompts, max_len=a.length + a.tokens + 4)
    lens = [max(1, a.length * (i + 1) // a.prompts) for i in range(a.prompts)]
    cu = torch.tensor([0] + lens).cumsum(0).int()
    prompt = torch.randint(0, 1000, (int(cu[-1]),), generator=torch.Generator().manual_seed(1))
    prompt = prompt.cuda()
    net.prefill(prompt, cu).argmax(-1)              # the first call loads the kernels
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    token = net.prefill(prompt, cu).argmax(-1)
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    answer = [token.clone()]

    # warm up on a side stream, capture, and put the states back as the prompts left them
    saved = [None if s is None else s.clone() for s in net.state + net.conv_state]
    lens_dev, side = net.lens.clone(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        net.step(token)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token.copy_(net.step(token).argmax(-1))
    for s, old in zip(net.state + net.conv_state, saved):
        if s is not None:
            s.copy_(old)
    net.lens.copy_(lens_dev)

    torch.cuda.synchronize()
    t2 = time.perf_counter()
    for _ in range(a.tokens - 1):
        graph.replay()
        answer.append(token.clone())
    torch.cuda.synchronize()
    t3 = time.perf_counter()
    print("prompts: %d tokens in %.2f ms" % (int(cu[-1]), 1e3 * (t1 - t0)))
    if a.tokens > 1:
        print("answers: %d x %d tokens, %.3f ms a step"
              % (a.prompts, a.tokens, 1e3 * (t3 - t2) / (a.tokens - 1)))
    print("first answer:", " ".join(str(int(t[0])) for t in answer[:16]))


if __name__ == "__main__":
    main()
