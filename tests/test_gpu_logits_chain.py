"""The operators together, as a decode step uses them: a router's 4-bit product,
the choice of experts, their balance, the experts' FFN, the output head's 4-bit
product and the draw of a token; eager, on a side stream, and from a graph."""
import numpy as np
import pytest
import torch

import guard

from lfsr_seeded_moe_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nslm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lfsr_seeded_moe_b200 import nslm as n
    return n


def _q4(N, K, G, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randint(-2**31, 2**31, (N, K // 8), generator=g, device="cuda", dtype=torch.int32)
    s = (0.01 * torch.exp(0.2 * torch.randn(N, K // G, generator=g, device="cuda"))).bfloat16()
    b = (-7.5 * s.float()).bfloat16()
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    n = ((q.unsqueeze(-1) >> shift) & 15).double().reshape(N, K)
    return (q, s, b), n * s.double().repeat_interleave(G, 1) + b.double().repeat_interleave(G, 1)


def test_decode_step(nslm):
    T, E, hidden, inter, k, V = 4, 32, 256, 128, 4, 5003
    (rq, rs, rb), rw = _q4(E, hidden, 64, 1)
    (hq, hs, hb), hw = _q4(V, hidden, 32, 2)
    router, head = nslm.q4_matrix(rq, rs, rb, 64), nslm.q4_matrix(hq, hs, hb, 32)
    L = synth.moe_layer(0, E, hidden, inter, 4, device="cuda", config=960)
    x = guard.buffer((T, hidden), torch.bfloat16)
    h = guard.buffer((T, hidden), torch.bfloat16)
    rl = guard.buffer((T, E), torch.float32, fill=float("nan"))
    ids = guard.buffer((T, k), torch.int32)
    w = guard.buffer((T, k), torch.float32)
    counts = guard.buffer(E + 1, torch.int32)
    loss = guard.buffer(1, torch.float32)
    dl = guard.buffer((T, E), torch.float32)
    wsb = nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_FFN, T, E, hidden, inter, k)
    ws = guard.buffer(wsb, torch.uint8)
    y = guard.buffer((T, hidden), torch.float32)
    logits = guard.buffer((T, V), torch.float32, fill=float("nan"))
    u = torch.tensor([0.1, 0.5, 0.9, 0.3], device="cuda")
    top_p = torch.full((T,), 0.9, device="cuda")
    params = nslm.sample_params(None, None, top_p, None)
    token = guard.buffer(T, torch.int32)
    prob = guard.buffer(T, torch.float32)

    def step():
        nslm.nslm_q4_gemv(router, x, T, rl, nslm.NSLM_GEMV_FIELDS_READY)
        nslm.nslm_moe_route_topk(rl, T, E, k, ids, w)
        nslm.nslm_moe_balance(rl, ids, None, T, E, k, 1.0, counts, None, None, loss)
        nslm.nslm_moe_balance_grad(rl, counts, None, T, E, k, 1.0, None, dl)
        nslm.nslm_moe_seed_ffn(L.gate, L.up, L.down, E, x, ids, w, T, k, y, ws, wsb)
        h.copy_(y / y.square().mean(1, keepdim=True).sqrt())
        nslm.nslm_q4_gemv(head, h, T, logits, nslm.NSLM_GEMV_FIELDS_READY)
        nslm.nslm_sample(logits, nslm.NSLM_TYPE_F32, T, V, V, params, u, token, prob)

    def check():
        # each step against 64 bits, from what the step before it left
        want = x.double() @ rw.t()
        assert float((rl.double() - want).norm()) <= 2e-6 * float(want.norm())
        assert torch.equal(ids.long(), torch.sort(rl, dim=1, descending=True, stable=True).indices[:, :k])
        assert torch.equal(counts[:E].long(), torch.bincount(ids.reshape(-1).long(), minlength=E)) and int(counts[E]) == T
        z = rl.double().requires_grad_(True)
        ref = E * (torch.softmax(z, 1).mean(0) * counts[:E].double() / (k * T)).sum()
        (d,) = torch.autograd.grad(ref, z)
        assert abs(float(loss) - float(ref.detach())) <= 97 * 2.0 ** -24 * float(ref.detach())
        p = torch.softmax(rl.double(), 1)
        f = counts[:E].double() / (k * T)
        size = E / T * p * (f + (p * f).sum(1, keepdim=True))
        assert bool(((dl.double() - d).abs() <= 2 * 96 * 2.0 ** -24 * size).all())
        want = h.double() @ hw.t()
        assert float((logits.double() - want).norm()) <= 2e-6 * float(want.norm())
        l = logits.double().cpu().numpy()
        for t in range(T):
            e = np.exp(l[t] - l[t].max())
            order = np.argsort(-l[t], kind="stable")
            c = np.cumsum(e[order])
            n = int(np.count_nonzero(c < float(top_p[t]) * c[-1])) + 1
            keep = np.sort(order[:n])
            c = np.cumsum(e[keep])
            i = keep[int(np.count_nonzero(c <= float(u[t]) * c[-1]))]
            assert int(token[t]) == i
            assert abs(float(prob[t]) - e[i] / c[-1]) <= (2.0 ** -24 + 2.0 ** -29) * e[i] / c[-1]

    x.copy_(synth.activations((960, 1), T, hidden))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for tag in (2, 3):
        x.copy_(synth.activations((960, tag), T, hidden))
        g.replay()
        torch.cuda.synchronize()
        check()


def test_counts_group_rows_for_the_grouped_product(nslm):
    # offsets from the balance call are what the grouped product reads
    T, E, k, K, rows = 40, 6, 2, 128, 64
    W = synth.seed_matrix(rows, K, 4, (961,), E, device="cuda")
    z = synth.router_logits((961,), T, E).cuda()
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    nslm.nslm_moe_route_topk(z, T, E, k, ids, w)
    counts = guard.buffer(E + 1, torch.int32)
    offsets = guard.buffer(E + 1, torch.int32)
    loss = guard.buffer(1, torch.float32)
    nslm.nslm_moe_balance(z, ids, None, T, E, k, 1.0, counts, offsets, None, loss)
    x = synth.activations((961,), T, K).cuda()
    order = torch.sort(ids.reshape(-1), dim=0, stable=True).indices
    xs = x[order // k].contiguous()
    wsb = nslm.nslm_workspace_bytes(nslm.NSLM_OP_GROUPED_GEMM, T * k, E, K, rows, 1)
    ws = guard.buffer(wsb, torch.uint8)
    y = guard.buffer((T * k, rows), torch.float32, fill=float("nan"))
    nslm.nslm_seed_grouped_gemm(W, E, xs, offsets, T * k, y, ws, wsb)
    dense = guard.buffer((E * rows, K), torch.float32)
    nslm.nslm_debug_decompress(W, dense)
    picked = dense.double().reshape(E, rows, K)[ids.reshape(-1)[order].long()]
    want = torch.einsum("trk,tk->tr", picked, xs.double())
    # the grouped product rounds weights to bf16: 8 significant bits, steps of
    # 2^-7 at 1, so half a step is finfo(bfloat16).eps / 2 = 2^-8 of a weight
    size = torch.einsum("trk,tk->tr", picked.abs(), xs.double().abs())
    assert bool(((y.double() - want).abs() <= (2.0 ** -8 + K * 2.0 ** -23) * size).all())
