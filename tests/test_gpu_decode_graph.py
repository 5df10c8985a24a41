"""decode_paged and decode_paged_window captured once and replayed on new queries
and lengths, for each way the split results are joined: each replay gives that
step's output, and eager calls between the replays theirs."""

import pytest
import torch

from exact_softmax_attention_causal_b200 import decode_paged, decode_paged_window, decode_workspace_bytes
from test_gpu_prefill_varlen import BF16, I32, Batch

pytestmark = pytest.mark.gpu


def _replay(ctx, Hq, Hkv, d, bs, steps, call, mask):
    """Tolerances: those of the ragged attention's tests; the same masks."""
    b = Batch([1] * len(ctx), ctx, Hq, Hkv, d, bs, 41)
    q, kc, vc, bt, _, sl = b.args()
    status = torch.zeros(1, dtype=I32, device="cuda")
    max_len = b.max_len
    call(q, kc, vc, bt, sl, max_len, status)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = call(q, kc, vc, bt, sl, max_len, status)
    g = torch.Generator().manual_seed(6)
    for step in range(steps):
        if step:
            b.ctx = [max(1, c - 37 * step) for c in ctx]
            b.q = torch.randn(b.q.shape, generator=g).to(BF16)
            q.copy_(b.q)
            sl.copy_(torch.tensor(b.ctx, dtype=I32))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        eager = call(q, kc, vc, bt, sl, max_len, status)
        t = [torch.arange(c) for c in b.ctx]
        b.k, b.v = ([pool[b.table[s].long()[t[s] // bs], t[s] % bs] for s in range(len(b.ctx))] for pool in (b.k_cache, b.v_cache))
        b.check(*got, **mask)
        b.check(*eager, **mask)
    assert int(status.item()) == 0


# joined in the launch; by the second kernel; work handed out at run time; 32 heads a CTA
@pytest.mark.parametrize("ctx,Hq,Hkv,d", [([700, 40, 1500, 900], 8, 2, 128), ([30000], 8, 2, 128), ([5000, 3000], 4, 1, 64),
                                          ([2000] * 40, 32, 8, 64), ([4000, 100], 32, 1, 128), ([300], 4, 4, 64)])
def test_decode(ctx, Hq, Hkv, d):
    _replay(ctx, Hq, Hkv, d, 16, 3,
            lambda q, kc, vc, bt, sl, m, st: decode_paged(q, kc, vc, bt, sl, m, status=st), dict(mask="causal"))


@pytest.mark.parametrize("window,n_sink", [(130, 4), (1500, 0)])
def test_decode_window(window, n_sink):
    _replay([2000, 90, 3000], 8, 2, 64, 32, 3,
            lambda q, kc, vc, bt, sl, m, st: decode_paged_window(q, kc, vc, bt, sl, m, window=window, n_sink=n_sink, status=st),
            dict(mask="window", window=window, n_sink=n_sink))


def test_two_graphs_and_an_eager_call_share_a_workspace_in_turn():
    Hq, Hkv, d = 8, 2, 64
    b = Batch([1] * 3, [900, 2500, 1200], Hq, Hkv, d, 16, 42)
    q, kc, vc, bt, _, sl = b.args()
    ws = torch.full((decode_workspace_bytes(3, Hq, Hkv, d, b.max_len, 16),), 0xA5, dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = decode_paged(q, kc, vc, bt, sl, b.max_len, workspace=ws)
        graphs.append((graph, *out))
    for _ in range(3):
        for graph, o, lse in graphs:
            o.fill_(9.0), lse.fill_(9.0)
            graph.replay()
            torch.cuda.synchronize()
            b.check(o, lse)
            b.check(*decode_paged(q, kc, vc, bt, sl, b.max_len, workspace=ws))
