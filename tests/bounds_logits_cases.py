"""Small cases of the 4-bit GEMV, the balance loss and sampling on the
bounds-check build of the library.

Started by tests/test_gpu_bounds_logits.py in a subprocess with
NSLM_LIB_VARIANT=boundscheck.  Prints one JSON line: whether each case's result
is right, and the bounds status after each operator's (0: no index left its
buffer, in global or in shared memory).
"""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

from lfsr_seeded_moe_b200 import nslm  # noqa: E402

DEV = "cuda"


def q4(res, gen):
    # integers and scales of 1 and 2: every sum is exact
    for N, K, G, M, affine in [(1, 32, 32, 1, True), (17, 96, 32, 2, True), (33, 1408, 128, 5, False), (100, 1408, 64, 8, True),
                               (257, 2048, 32, 3, True), (40000, 512, 32, 1, True), (40001, 512, 64, 4, True),
                               (38000, 1024, 128, 3, False), (2500, 8192, 32, 8, True), (700, 65536, 32, 1, True),
                               (33, 65536, 128, 1, False), (120, 32768, 64, 2, True), (60, 8160, 32, 7, True)]:
        q = torch.randint(-2**31, 2**31, (N, K // 8), generator=gen, device=DEV, dtype=torch.int32)
        scales = torch.randint(1, 3, (N, K // G), generator=gen, device=DEV).bfloat16()
        biases = torch.randint(-15, 16, (N, K // G), generator=gen, device=DEV).bfloat16() if affine else None
        x = torch.randint(-1, 2, (M, K), generator=gen, device=DEV).bfloat16()
        y = torch.full((M, N), float("nan"), device=DEV)
        nslm.nslm_q4_gemv(nslm.q4_matrix(q, scales, biases, G), x, M, y, N & 1)
        right = True
        for i in range(0, N, 8192):
            n = ((q[i:i + 8192].unsqueeze(-1) >> torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)) & 15).double()
            n = n.reshape(n.shape[0], K)
            s = scales[i:i + 8192].double().repeat_interleave(G, 1)
            w = s * n + biases[i:i + 8192].double().repeat_interleave(G, 1) if affine else s * (n - 8)
            right = right and torch.equal(y[:, i:i + 8192].double(), x.double() @ w.t())
        res[f"q4_{N}x{K}_G{G}_M{M}_{int(affine)}"] = right
    res["status_q4"] = nslm.nslm_debug_bounds_status()


def balance(res, gen):
    for T, E, k in [(0, 8, 2), (1, 1, 1), (7, 100, 8), (65, 33, 4), (1024, 1023, 3), (1024, 100, 8), (1025, 4, 1),
                    (3000, 257, 6), (2500, 1024, 8), (20000, 64, 4), (950000, 8, 2)]:
        z = torch.randn(max(T, 1), E, generator=gen, device=DEV)[:T]
        ids = torch.randint(0, E, (max(T, 1), k), generator=gen, device=DEV, dtype=torch.int32)[:T]
        need = nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_BALANCE, T, E, 0, 0, k)
        ws = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
        counts, offsets = (torch.full((E + 1,), -1, dtype=torch.int32, device=DEV) for _ in range(2))
        mean, loss, d = torch.empty(E, device=DEV), torch.empty(1, device=DEV), torch.empty(T, E, device=DEV)
        nslm.nslm_moe_balance(z, ids, None, T, E, k, 1.0, counts, offsets, mean, loss, ws, need)
        nslm.nslm_moe_balance_grad(z, counts, None, T, E, k, 1.0, None, d)
        p = torch.softmax(z.double(), 1)
        c = torch.bincount(ids.reshape(-1).long(), minlength=E)
        f = c.double() / (k * max(1, T))
        want = p.sum(0) / max(1, T)
        dwant = E / max(1, T) * p * (f - (p * f).sum(1, keepdim=True))
        size = E / max(1, T) * p * (f + (p * f).sum(1, keepdim=True))
        # wide bounds: their own tests hold the rounding, these the indices
        res[f"balance_{T}x{E}_k{k}"] = bool(
            torch.equal(counts[:E].long(), c) and int(counts[E]) == T and int(offsets[E]) == T * k
            and ((mean - want).abs() <= 1e-4 * want).all() and ((d - dwant).abs() <= 1e-4 * size + 1e-30).all()
            and abs(float(loss) - E * float((f * want).sum())) <= 1e-4 * (float(loss) + 1e-30))
    res["status_balance"] = nslm.nslm_debug_bounds_status()


def _token(l, u, k, p):
    """Each row's token in 64 bits."""
    order = torch.sort(l.double(), dim=1, descending=True, stable=True)
    w = torch.exp(order.values - order.values[:, :1])
    keep = torch.ones_like(w, dtype=torch.bool)
    keep[:, k or w.shape[1]:] = False
    m = torch.where(keep, w, 0.0)
    keep &= torch.cumsum(m, 1) - m < float(torch.tensor(p)) * m.sum(1, keepdim=True)
    kept = torch.zeros_like(w).scatter_(1, order.indices, torch.where(keep, w, 0.0))
    c = torch.cumsum(kept, 1)
    return (c <= u.double().unsqueeze(1) * c[:, -1:]).sum(1).to(torch.int32)


def sample(res, gen):
    for B, V, pad in [(1, 1, 0), (3, 2, 1), (5, 100, 0), (7, 1000, 3), (2, 4097, 0), (2, 32003, 5), (1, 262144, 0),
                      (300, 33, 0), (310, 3001, 0), (100, 60001, 3)]:
        for kind, make in (("wide", lambda z: 3 * z), ("even", lambda z: 0.1 * z), ("equal", lambda z: 0 * z),
                           ("tiny", lambda z: z * 2.0 ** -60 * 2.0 ** -70)):
            for dtype in (torch.float32, torch.bfloat16):
                whole = torch.zeros(B, V + pad, device=DEV, dtype=dtype)
                l = whole[:, :V]
                l.copy_(make(torch.randn(B, V, generator=gen, device=DEV)))
                u = torch.rand(B, generator=gen, device=DEV)
                right = True
                for k, p in ((0, 1.0), (1, 1.0), (50, 1.0), (500, 0.9), (0, 0.9), (5000, 0.99)):
                    if k >= V:
                        continue
                    token, prob = torch.full((B,), -7, dtype=torch.int32, device=DEV), torch.empty(B, device=DEV)
                    ks, ps = torch.full((B,), k, dtype=torch.int32, device=DEV), torch.full((B,), p, device=DEV)
                    nslm.nslm_sample(whole, nslm.NSLM_TYPE_BF16 if dtype == torch.bfloat16 else nslm.NSLM_TYPE_F32, B, V,
                                     V + pad, nslm.sample_params(None, ks, ps, None), u, token, prob)
                    right = right and torch.equal(token, _token(l, u, k, p))
                res[f"sample_{B}x{V}_{kind}_{str(dtype)[6:]}"] = right
    res["status_sample"] = nslm.nslm_debug_bounds_status()


def main():
    assert nslm.LIB_PATH.endswith(os.path.join("boundscheck", "libnslm.so")), nslm.LIB_PATH
    gen = torch.Generator(DEV).manual_seed(17)
    res = {"status_start": nslm.nslm_debug_bounds_status()}
    q4(res, gen)
    balance(res, gen)
    sample(res, gen)
    print(json.dumps(res))


if __name__ == "__main__":
    main()
