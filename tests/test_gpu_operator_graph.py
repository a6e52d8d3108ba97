"""The training operators in a captured graph and on a side stream: every replay, with other inputs
and with eager work between the replays, gives what the eager calls give, bit for bit (no sum
depends on the order of atomics)."""
import pytest
import torch

import bit_block_scaled_quant_amd as nv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def inputs(M, F, K, V, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    tok = torch.randint(-1, V, (M,), generator=g, device=DEV, dtype=torch.int32)
    idx = torch.randint(-1, V, (M, 9), generator=g, device=DEV, dtype=torch.int32)
    return dict(x=x, tok=tok, idx=idx, top=torch.randn(M, 9, generator=g, device=DEV),
                dh=torch.randn(M, F, generator=g, device=DEV).bfloat16(),
                logits=torch.randn(M, V, generator=g, device=DEV).bfloat16())


def step(s, w, V):
    q, qt = nv.quantize_cast_transpose(s["x"], rht_t=True, rht_seed=3)
    h = nv.gated_ffn(q, w, nv.GELU)
    dx, dw = nv.gated_ffn_backward(s["dh"], q, qt, w, nv.GELU, rht_t=True, rht_seed=3)
    amax = torch.empty(1, device=DEV)
    plain = nv.gated_ffn_grad(s["dh"], q, w, nv.SILU, amax=amax)
    loss, lse, grad = nv.distill_topk_loss_and_grad(s["logits"], s["idx"], s["top"])
    again = nv.distill_topk_grad(s["logits"], s["idx"], s["top"], lse)
    table = nv.embed_grad(s["tok"], dx, V, scale=2.0)
    return h, dx, dw, plain, amax, loss, lse, grad, again, table, nv.embed(s["tok"], table)


@pytest.mark.parametrize("M,F,K,V", [(48, 120, 192, 700), (512, 256, 512, 1031), (9008, 64, 128, 50)])
def test_graph_replays_match_eager(M, F, K, V):
    w = nv.quantize_2d(torch.randn(2 * F, K, device=DEV).bfloat16())
    buffers = inputs(M, F, K, V, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(buffers, w, V)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(buffers, w, V)
    for seed in range(1, 5):
        new = inputs(M, F, K, V, seed)
        want = step(new, w, V)
        for k, v in new.items():
            buffers[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert torch.equal(got, ref)


def test_side_streams():
    """Each stream's calls wait for that stream's producers and for nothing else."""
    w = nv.quantize_2d(torch.randn(2 * 256, 512, device=DEV).bfloat16())
    sets = [inputs(512, 256, 512, 1031, s) for s in (11, 12)]
    want = [step(s, w, 1031) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for s, stream in zip(sets, streams):
        with torch.cuda.stream(stream):
            filler = torch.randn(2048, 2048, device=DEV)
            for _ in range(10):
                filler = filler @ filler * 1e-3
            moved = {k: v.clone() for k, v in s.items()}  # written behind the products
            got.append(step(moved, w, 1031))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
