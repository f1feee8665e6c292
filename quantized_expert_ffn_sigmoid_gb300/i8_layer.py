"""The routed expert layer on the library's int8 expert records (codes and one
scale per output row) for activations quantised per token, step by step
through the library:

    idx, w = select(x)                              coli_moe_select
    offsets, rows, slots = group(idx)               coli_moe_group
    xq = codes(x)                                   coli_i8_quantize
    gu[p] = [Wg; Wu] xq[rows[p]]                    coli_i8_product
    hq = codes(silu(g) u)                           coli_i8_quantize (SwiGLU)
    o = Wd hq                                       coli_i8_product
    y[t] = sum_j w[t, j] o[slots[t, j]] + shared    coli_moe_combine

The shared experts run as groups of all positions and enter y with weight 1.
``capture`` records the step as a CUDA graph.

    python -m quantized_expert_ffn_sigmoid_gb300.i8_layer      # runs a layer and times it
"""
from __future__ import annotations

import quantized_expert_ffn_sigmoid_gb300 as cm


def matrices(experts, scales, inter: int, hidden: int):
    """Gate and up of all records [E, 2 inter, hidden] with their scales [E, 2 inter], and down [E, hidden, inter]
    with its scales [E, hidden]: views of the records, nothing is copied."""
    n, cut = experts.shape[0], 2 * inter * hidden
    if experts.shape != (n, 3 * inter * hidden) or scales.shape != (n, 2 * inter + hidden):
        raise ValueError(f"int8 records of {inter} x {hidden}: codes [E, {3 * inter * hidden}] and scales [E, {2 * inter + hidden}], "
                         f"not {tuple(experts.shape)} and {tuple(scales.shape)}")
    return (experts[:, :cut].view(n, 2 * inter, hidden), scales[:, :2 * inter]), (experts[:, cut:].view(n, hidden, inter), scales[:, 2 * inter:])


class Layer:
    """One layer for ``positions`` positions per step; all buffers are allocated here, once.

    experts [E, 3 inter hidden] int8 and expert_scales [E, 2 inter + hidden] float32 (with ``ep_size`` > 1 those of
    shard ``ep_rank``: experts e = ep_rank mod ep_size), router_w [experts of all shards, hidden] float32.  The
    selection's arguments are those of coli_moe_select.  A shard's y is its part of the sum over the shards; the
    shared experts (records of ``shared_inter``, or ``inter``) belong to shard 0.  ``dtype`` is the type of y and of
    the values between the products."""

    def __init__(self, experts, expert_scales, router_w, inter: int, positions: int, dtype, top_k: int, bias=None, shared=None, shared_scales=None,
                 score=cm.SCORE_SOFTMAX, n_groups=1, topk_group=1, group_score=cm.GROUP_TOP2, renorm=True, scaling=1.0, ep_rank=0, ep_size=0,
                 shared_inter=None):
        import torch
        dev, (E, H), T, k = router_w.device, router_w.shape, positions, top_k
        si = inter if shared_inter is None else shared_inter
        if inter % 16 or si % 16 or H % 16:
            raise ValueError("hidden, inter and shared_inter must be multiples of 16: rows of codes begin on 16-byte boundaries")
        if T < 1:
            raise ValueError("at least one position")
        local = E if ep_size <= 1 else (E - ep_rank + ep_size - 1) // ep_size
        if experts.shape[0] != local:
            raise ValueError(f"records of {local} experts, not {experts.shape[0]}")
        self.gate_up, self.down = matrices(experts, expert_scales, inter, H)
        self.router_w, self.bias, self.experts, self.ep = router_w, bias, E, (ep_rank, ep_size)
        self.choice = dict(score=score, n_groups=n_groups, topk_group=topk_group, group_score=group_score, renorm=renorm, scaling=scaling)
        ns = shared.shape[0] if shared is not None and ep_rank == 0 else 0
        P, most = T * k, T * max(k, ns)

        def new(*shape, of=torch.float32):
            return torch.zeros(*shape, dtype=of, device=dev)   # (rows of skipped slots are quantised too: they hold no garbage)

        self.x = new(T, H)                                     # float32, as the router reads it
        self.idx, self.w, self.slots = new(T, k, of=torch.int32), new(T, k), new(T, k, of=torch.int32)
        self.offsets, self.rows = new(local + 1, of=torch.int32), new(P, of=torch.int32)
        self.xq, self.xs = new(T, H, of=torch.int8), new(T)
        self.gu, self.hq, self.hs, self.o = new(P, 2 * inter, of=dtype), new(P, inter, of=torch.int8), new(P), new(P, H, of=dtype)
        self.y = new(T, H, of=dtype)
        self.ws_select = cm.new_select_workspace(T, H, E, dev)
        self.ws_group = cm.new_group_workspace(T, k, E, dev)
        self.ws = cm.new_i8_product_workspace(most, max(H, inter, si if ns else 0), dev)
        self.shared = None
        if ns:
            self.shared = matrices(shared[:ns], shared_scales, si, H)
            position = torch.arange(T, dtype=torch.int32, device=dev)
            self.s_rows, self.s_offsets = position.repeat(ns), torch.arange(ns + 1, dtype=torch.int32, device=dev) * T
            self.s_slots = (position[:, None] + torch.arange(ns, dtype=torch.int32, device=dev) * T).contiguous()
            self.s_w = torch.ones(T, ns, device=dev)
            self.s_gu, self.s_hq, self.s_hs, self.s_o = (new(ns * T, 2 * si, of=dtype), new(ns * T, si, of=torch.int8), new(ns * T),
                                                        new(ns * T, H, of=dtype))

    def step(self):
        """The layer on ``self.x`` into ``self.y`` (also idx and w, and everything between)."""
        rank, size = self.ep
        cm.coli_moe_select(self.x, self.idx, self.w, router_w=self.router_w, bias=self.bias, ws=self.ws_select, **self.choice)
        cm.coli_moe_group(self.idx, self.offsets, self.rows, self.slots, self.ws_group, n_experts=self.experts, ep_rank=rank, ep_size=size)
        cm.coli_i8_quantize(self.x, self.xq, self.xs)
        if self.shared is not None:
            (w, s), (wd, sd) = self.shared
            cm.coli_i8_product(self.xq, self.xs, w, s, self.s_gu, self.ws, offsets=self.s_offsets, rows=self.s_rows)
            cm.coli_i8_quantize(self.s_gu, self.s_hq, self.s_hs, swiglu=True)
            cm.coli_i8_product(self.s_hq, self.s_hs, wd, sd, self.s_o, self.ws, offsets=self.s_offsets)
            cm.coli_moe_combine(self.s_o, self.s_slots, self.s_w, self.y)
        (w, s), (wd, sd) = self.gate_up, self.down
        cm.coli_i8_product(self.xq, self.xs, w, s, self.gu, self.ws, offsets=self.offsets, rows=self.rows)
        cm.coli_i8_quantize(self.gu, self.hq, self.hs, swiglu=True)
        cm.coli_i8_product(self.hq, self.hs, wd, sd, self.o, self.ws, offsets=self.offsets)
        cm.coli_moe_combine(self.o, self.slots, self.w, self.y, add=self.y if self.shared is not None else None)
        return self.y

    def status(self) -> int:
        """The status bits of all workspaces (synchronises, and clears them)."""
        return cm.coli_moe_status(self.ws_select) | cm.coli_moe_status(self.ws_group) | cm.coli_moe_status(self.ws)

    def capture(self):
        """The step as a CUDA graph on the same buffers (``replay()`` runs it)."""
        import torch
        self.step()                                            # first launches set kernel attributes
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            self.step()
        return g


def random_records(n: int, inter: int, hidden: int, gen):
    """Records of random normal weights, quantised per row by the library: codes [n, 3 inter hidden], scales [n, 2 inter + hidden]."""
    import torch
    codes = torch.empty(n, 3 * inter * hidden, dtype=torch.int8, device="cuda")
    scales = torch.empty(n, 2 * inter + hidden, device="cuda")
    for e in range(n):
        for at, first, rows, k in ((0, 0, 2 * inter, hidden), (2 * inter * hidden, 2 * inter, hidden, inter)):
            m = torch.randn(rows, k, generator=gen, device="cuda") * k ** -0.5
            s = torch.empty(rows, device="cuda")
            cm.coli_i8_quantize(m, codes[e, at:at + m.numel()].view(rows, k), s)
            scales[e, first:first + rows] = s
    return codes, scales


def main():
    import torch
    E, H, inter, k = 64, 2048, 1024, 8
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes, scales = random_records(E, inter, H, gen)
    shared, shared_scales = random_records(1, inter, H, gen)
    router = torch.randn(E, H, generator=gen, device="cuda") * H ** -0.5
    for T in (1, 32, 2048):
        layer = Layer(codes, scales, router, inter, T, torch.bfloat16, k, shared=shared, shared_scales=shared_scales, n_groups=8, topk_group=4, scaling=2.5)
        layer.x.copy_(torch.randn(T, H, generator=gen, device="cuda"))
        g = layer.capture()
        for _ in range(3):
            g.replay()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            g.replay()
        b.record()
        torch.cuda.synchronize()
        print(f"{T:4d} positions: {a.elapsed_time(b) / 20 * 1e3:8.1f} us a layer, status {layer.status()}")


if __name__ == "__main__":
    main()
