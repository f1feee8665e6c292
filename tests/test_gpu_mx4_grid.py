"""The MX4 expert layer starts as many CTAs as can work at once.

A CTA claims items from a counter in the workspace until a claim lies past the
last item, so after a call the counter is the number of items plus the number
of CTAs.  Fewer CTAs than the larger pass has items, with SMs left, is a call
that runs on a part of the GPU; results do not depend on it."""
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402

CLAIM_AT = 8704 + 256   # behind the workspace's header and the tables' own (256-byte slots)


def items_and_ctas(T, hidden, inter, experts, top_k, n_shared=0, shared_inter=0, skip=0.0):
    cfg = cm.Cfg.of(types.SimpleNamespace(hidden=hidden, n_experts=experts, n_groups=1, topk_group=1, top_k=top_k, inter=inter, n_shared=n_shared,
                                          shared_inter=shared_inter, weight_bits=4, routed_scaling_factor=1.0))
    g = torch.Generator("cuda").manual_seed(T + hidden)

    def records(n, i):
        return (torch.randint(0, 256, (n, 3 * i * hidden // 2), generator=g, device="cuda", dtype=torch.uint8),
                torch.full((n, 3 * i * hidden // 32), 118, device="cuda", dtype=torch.uint8))

    rec = (*records(experts, inter), *(records(n_shared, shared_inter) if n_shared else ()))
    w = cm.make_mx4_weights(*rec)
    idx = torch.rand(T, experts, generator=g, device="cuda").topk(top_k, -1)[1].int()
    idx[torch.rand(T, top_k, generator=g, device="cuda") < skip] = -1
    x, y = torch.randn(T, hidden, generator=g, device="cuda"), torch.empty(T, hidden, device="cuda")
    ws = cm.new_mx4_workspace(cfg, T)
    cm.coli_mx4_forward(cfg, w, x, idx, torch.rand(T, top_k, generator=g, device="cuda"), y, ws)
    assert cm.coli_moe_status(ws) == 0 and torch.isfinite(y).all()
    tile = next(n for n in (16, 32, 64, 128) if n >= min(T, 128))
    ids = idx.cpu().numpy().ravel()
    tiles = int((-(-np.bincount(ids[ids >= 0], minlength=experts) // tile)).sum())
    shared_tiles = n_shared * -(-T // tile)
    gate_up = tiles * (inter // 64) + shared_tiles * (shared_inter // 64)
    down = (tiles + shared_tiles) * (hidden // 128)
    claims = int(ws[CLAIM_AT:CLAIM_AT + 4].view(torch.int32))
    return gate_up, down, claims - gate_up - down


@pytest.mark.parametrize("kw", [
    dict(T=1, hidden=256, inter=1664, experts=8, top_k=4, n_shared=1, shared_inter=1664),   # many gate/up items an entry
    dict(T=1, hidden=1024, inter=4096, experts=8, top_k=2),
    dict(T=1, hidden=256, inter=128, experts=8, top_k=1, n_shared=1, shared_inter=4096),    # most of them the shared expert's
    dict(T=700, hidden=256, inter=2048, experts=8, top_k=2),                                # many tiles of positions an entry
    dict(T=700, hidden=256, inter=128, experts=4, top_k=4, n_shared=1, shared_inter=128),
    dict(T=700, hidden=512, inter=2048, experts=8, top_k=2, n_shared=1, shared_inter=256),
    dict(T=130, hidden=128, inter=1024, experts=2, top_k=1, skip=0.5),
    dict(T=40, hidden=2048, inter=256, experts=64, top_k=8),                                # more items than SMs in either pass
    dict(T=1, hidden=512, inter=256, experts=16, top_k=2, n_shared=1, shared_inter=256),    # fewer in both
])
def test_no_sm_is_left_without_work(kw):
    gate_up, down, ctas = items_and_ctas(**kw)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert min(sms, max(gate_up, down)) <= ctas <= sms, (gate_up, down, ctas)
