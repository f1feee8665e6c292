"""One decoder block's expert half on MX4 weights, step by step through the
library: the norm before the block with the MX4 codes of its result, the
router on that result, the expert layer on those codes, and the norm, gate and
residual add behind it fused with the next block's norm.

    n0 = rms(x) pre_w                              coli_moe_block_norm  (n0, codes)
    idx, w = route(n0)                             coli_moe_route
    y = experts(MX4(n0), idx, w)                   coli_mx4_forward
    x' = x + res_scale gate rms(y) post_w,
    n1 = rms(x') next_w                            coli_moe_block_norm  (x', n1, codes)

A stack of blocks needs the first norm once: every block leaves the next one's
input behind.  ``capture`` records a whole stack as a CUDA graph.

    python -m quantized_expert_ffn_sigmoid_gb300.mx4_block      # runs a small stack and times it
"""
from __future__ import annotations

from dataclasses import dataclass

import quantized_expert_ffn_sigmoid_gb300 as cm


@dataclass
class Block:
    """Weights of one block (tensors on the GPU; see include/coli_moe.h for the layouts)."""
    cfg: "cm.Cfg"
    experts: object         # [n_experts, record bytes] uint8 and its scales
    expert_scales: object
    shared: object          # None without shared experts
    shared_scales: object
    router_w: object        # [n_experts, hidden] float32
    corr_bias: object       # [n_experts] float32
    post_w: object          # [hidden] float32: norm behind the block
    next_w: object          # [hidden] float32: norm before the next block
    gate: object = None     # [hidden] or [positions, hidden] of the stream's type
    res_scale: float = 1.0

    def weights(self):
        return cm.make_mx4_weights(self.experts, self.expert_scales, self.shared, self.shared_scales)


class Stack:
    """Blocks run one after the other on the residual stream ``x`` [positions, hidden] (float32,
    bfloat16 or float16), in place.  All buffers are allocated here, once.  The layers are whole:
    shards of an expert-parallel layer are refused, since nothing here sums their parts."""

    def __init__(self, blocks, pre_w, positions: int, dtype, eps: float = 1e-6):
        import torch
        self.blocks, self.pre_w, self.eps = list(blocks), pre_w, eps
        cfg = self.blocks[0].cfg
        if any(b.cfg.ep_size > 1 for b in self.blocks):
            raise ValueError("whole layers, no expert-parallel shards: a shard's y is a part of the sum that the norm behind it needs")
        dev, H, T, k = pre_w.device, cfg.hidden, positions, cfg.top_k
        sizes = [cm.coli_mx4_workspace_size(b.cfg, T) for b in self.blocks]   # 0: outside the layer's limits
        if 0 in sizes or any(b.cfg.hidden != H or b.cfg.top_k != k for b in self.blocks):
            raise ValueError("blocks of one hidden size and top_k, within the layer's limits")
        self.x = torch.empty(T, H, dtype=dtype, device=dev)
        self.norm = torch.empty(T, H, device=dev)                       # the router reads float32
        self.codes = torch.empty(T, H // 2, dtype=torch.uint8, device=dev)
        self.scales = torch.empty(T, H // 32, dtype=torch.uint8, device=dev)
        self.y = torch.empty(T, H, dtype=dtype, device=dev)
        # an allocation each: the library wants its arrays 16-byte aligned, which slices of T * k words need not be
        self.idx = [torch.empty(T, k, dtype=torch.int32, device=dev) for _ in self.blocks]
        self.w = [torch.empty(T, k, device=dev) for _ in self.blocks]
        self.ws = torch.empty(max(sizes), dtype=torch.uint8, device=dev)
        cm.coli_moe_workspace_init(self.ws)
        self._weights = [b.weights() for b in self.blocks]

    def step(self):
        """All blocks on the stream ``self.x``; leaves the normed stream in ``self.norm``."""
        cm.coli_moe_block_norm(self.x, pre_w=self.pre_w, eps=self.eps, n_out=self.norm, codes=self.codes, scales=self.scales)
        for b, weights, idx, w in zip(self.blocks, self._weights, self.idx, self.w):
            cm.coli_moe_route(b.cfg, self.norm, b.router_w, b.corr_bias, idx, w, self.ws)
            cm.coli_mx4_forward(b.cfg, weights, self.codes, idx, w, self.y, self.ws, x_scales=self.scales)
            cm.coli_moe_block_norm(self.x, self.y, post_w=b.post_w, gate=b.gate, res_scale=b.res_scale, pre_w=b.next_w, eps=self.eps,
                                   x_out=self.x, n_out=self.norm, codes=self.codes, scales=self.scales)

    def capture(self):
        """The step as a CUDA graph on the same buffers (``replay()`` runs it); the stream is left as it is."""
        import torch
        x = self.x.clone()
        self.step()                                                     # first launches set kernel attributes
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            self.step()
        self.x.copy_(x)
        return g


def random_block(cfg, seed: int, dtype) -> Block:
    """A block of random normal weights, quantised on the GPU by the library."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H = cfg.hidden

    def records(n, inter):
        codes = torch.empty(n, 3 * inter * H // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(n, 3 * inter * H // 32, dtype=torch.uint8, device="cuda")
        for e in range(n):
            for at, rows, k in ((0, 2 * inter, H), (2 * inter * H, H, inter)):
                m = torch.randn(rows, k, generator=gen, device="cuda") * k ** -0.5
                cm.coli_mx4_quantize(m, codes[e, at // 2:(at + m.numel()) // 2].view(rows, k // 2),
                                     scales[e, at // 32:(at + m.numel()) // 32].view(rows, k // 32))
        return codes, scales

    shared = records(cfg.n_shared, cfg.shared_inter) if cfg.n_shared else (None, None)
    near_one = lambda: 1.0 + 0.1 * torch.randn(H, generator=gen, device="cuda")  # noqa: E731
    return Block(cfg, *records(cfg.n_experts, cfg.inter), *shared,
                 torch.randn(cfg.n_experts, H, generator=gen, device="cuda") * 0.02,
                 torch.zeros(cfg.n_experts, device="cuda"), near_one(), near_one(),
                 torch.rand(H, generator=gen, device="cuda").to(dtype), 0.5)


def main():
    import torch
    cfg = cm.Cfg(hidden=2048, n_experts=64, n_groups=8, topk_group=4, top_k=8, inter=1024, n_shared=1, shared_inter=1024, weight_bits=4,
                 routed_scaling_factor=2.5)
    blocks = [random_block(cfg, 10 + i, torch.bfloat16) for i in range(4)]
    for T in (1, 32, 512):
        s = Stack(blocks, torch.ones(cfg.hidden, device="cuda"), T, torch.bfloat16)
        s.x.copy_(torch.randn(T, cfg.hidden, device="cuda"))
        g = s.capture()
        for _ in range(3):
            g.replay()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            g.replay()
        b.record()
        torch.cuda.synchronize()
        print(f"{T:4d} positions: {a.elapsed_time(b) / 20 / len(blocks) * 1e3:8.1f} us a block, status {cm.coli_moe_status(s.ws)}")


if __name__ == "__main__":
    main()
