"""The operators around the router and the output head, as measured cases.

Four operators work on logits or make them:

* q4_gemv: y = W x for M = 1..8 vectors, W in 4 bits with a scale (and an
  offset) for each group of 32, 64 or 128 weights along K;
* balance: the load-balance loss of a router, with the experts' counts;
* balance_grad: that loss's gradient with respect to the router's logits;
* sample: one token a row from logits, with temperature, top-k, top-p and
  min-p, at given random numbers.

``own`` False computes them from elementary torch operations, True calls the
framework.  The outputs are the same in both.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a router or another small projection of one decoded token: launch and latency
        dict(name="q4 512x1024 g64 m1", op="q4_gemv", N=512, K=1024, group=64, M=1, affine=True),
        # an expert-sized projection of one token, the finest groups
        dict(name="q4 2048x4096 g32 m1", op="q4_gemv", N=2048, K=4096, group=32, M=1, affine=True),
        # a small decode batch on a ragged K (11 groups of 128), scales only
        dict(name="q4 2048x1408 g128 m5", op="q4_gemv", N=2048, K=1408, group=128, M=5, affine=False),
        # an output head with an odd vocabulary, one token
        dict(name="q4 50257x2048 g64 m1", op="q4_gemv", N=50257, K=2048, group=64, M=1, affine=True),
        # the largest output head, a full decode batch
        dict(name="q4 131072x4096 g64 m8", op="q4_gemv", N=131072, K=4096, group=64, M=8, affine=True),
        # one routed layer's decode or prompt batch: 64 tokens, 100 experts, top 8
        dict(name="balance 64x100", op="balance", T=64, E=100, k=8, padded=0.0),
        # a training step's tokens of one layer, a padded batch
        dict(name="balance 65536x128", op="balance", T=65536, E=128, k=8, padded=0.1),
        # the gradient of a prompt-sized batch
        dict(name="balance_grad 512x100", op="balance_grad", T=512, E=100, k=8, padded=0.0),
        # the gradient of a training step's tokens
        dict(name="balance_grad 65536x128", op="balance_grad", T=65536, E=128, k=8, padded=0.1),
        # one token of one request, a small odd vocabulary, the usual filters
        dict(name="sample 1x32003 k50 p0.9", op="sample", B=1, V=32003, bits=32, top_k=50, top_p=0.9, min_p=0.0),
        # a serving batch whose requests set top-p and min-p only, 16-bit logits
        dict(name="sample 16x50257 p0.95", op="sample", B=16, V=50257, bits=16, top_k=0, top_p=0.95, min_p=0.02),
        # a large batch sampled from the whole distribution
        dict(name="sample 64x131072", op="sample", B=64, V=131072, bits=32, top_k=0, top_p=1.0, min_p=0.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["q4_gemv", "q4_gemv", "balance", "balance_grad", "sample", "sample"])
    if op == "q4_gemv":
        group = rng.choice([32, 64, 128])
        K = group * _log_int(rng, 1, 8192 // group)
        N = _log_int(rng, 16, 131072)
        N = max(1, min(N, 131072 * 4096 // K))
        return dict(op=op, N=N, K=K, group=group, M=rng.randint(1, 8), affine=rng.random() < 0.7)
    if op == "sample":
        V = _log_int(rng, 64, 262144)
        B = max(1, min(_log_int(rng, 1, 64), 64 * 131072 // V))
        return dict(op=op, B=B, V=V, bits=rng.choice([16, 32]), top_k=rng.choice([0, 0, _log_int(rng, 1, 1000)]),
                    top_p=rng.choice([1.0, round(rng.uniform(0.5, 0.99), 3)]),
                    min_p=rng.choice([0.0, round(rng.uniform(0.01, 0.2), 3)]))
    E = _log_int(rng, 4, 512)
    T = max(1, min(_log_int(rng, 1, 65536), 65536 * 128 // E))
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), padded=rng.choice([0.0, 0.25]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "q4_gemv":
        N, K, G, M = case["N"], case["K"], case["group"], case["M"]
        # quantised weights lie thicker in the middle of a group's range: each
        # nibble is the mean of two uniform ones
        a, b = (torch.randint(-2**31, 2**31, (N, K // 8), generator=g, device=DEV, dtype=torch.int32) for _ in range(2))
        s["q"] = (a & b) + ((((a ^ b) & -0x11111112) >> 1) & 0x77777777)
        del a, b
        scales = 0.004 * torch.exp(0.3 * torch.randn(N, K // G, generator=g, device=DEV))
        s["scales"] = scales.bfloat16()
        s["biases"] = (-7.5 * scales * (1 + 0.1 * torch.randn(N, K // G, generator=g, device=DEV))).bfloat16() if case["affine"] else None
        s["x"] = torch.randn(M, K, generator=g, device=DEV).bfloat16()
        s["y"] = torch.empty(M, N, device=DEV)
        return s
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        # a bulk of unlikely tokens, some tens of likely ones, and a padded end
        # of the vocabulary that is never to be drawn
        logits = 2.0 * torch.randn(B, V, generator=g, device=DEV)
        n = min(V, 40)
        at = torch.randint(0, V, (B, n), generator=g, device=DEV)
        logits.scatter_add_(1, at, 4 + 6 * torch.rand(B, n, generator=g, device=DEV))
        logits[:, V - V // 200:] = -math.inf
        s["logits"] = logits.bfloat16() if case["bits"] == 16 else logits
        s["temperature"] = 0.6 + 0.6 * torch.rand(B, generator=g, device=DEV)
        if B > 8:  # a request that asks for the most likely token
            s["temperature"][3] = 0.0
        s["top_k"] = torch.full((B,), case["top_k"], dtype=torch.int32, device=DEV) if case["top_k"] else None
        s["top_p"] = torch.full((B,), case["top_p"], device=DEV) if case["top_p"] < 1 else None
        s["min_p"] = torch.full((B,), case["min_p"], device=DEV) if case["min_p"] > 0 else None
        s["u"] = torch.rand(B, generator=g, device=DEV)
        s["token"] = torch.empty(B, dtype=torch.int32, device=DEV)
        s["prob"] = torch.empty(B, device=DEV)
        return s
    T, E, k = case["T"], case["E"], case["k"]
    s["logits"] = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    s["ids"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32).contiguous()
    s["mask"] = None
    if case["padded"]:  # the batch's end is padding: what stands there is not to be looked at
        s["mask"] = (torch.arange(T, device=DEV) < T - int(T * case["padded"])).to(torch.uint8)
        s["logits"][T - int(T * case["padded"]):] = math.nan
    s["coef"] = 0.01
    s["counts"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    if case["op"] == "balance":
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        s["mean_p"] = torch.empty(E, device=DEV)
        s["loss"] = torch.empty(1, device=DEV)
    else:
        s["counts"] = _plain_counts(s)
        s["dloss"] = 0.5 + torch.rand(1, generator=g, device=DEV)
        s["dlogits"] = torch.empty(T, E, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_q4(s):
    N, K, G = s["N"], s["K"], s["group"]
    q = (s["q"].unsqueeze(-1) >> torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)) & 15
    w = q.view(N, K // G, G).float()
    scales = s["scales"].float().unsqueeze(-1)
    w = w * scales + s["biases"].float().unsqueeze(-1) if s["biases"] is not None else (w - 8) * scales
    return torch.matmul(s["x"].float(), w.view(N, K).t())


def _valid(s):
    T = s["T"]
    return torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] != 0


def _plain_counts(s):
    """The experts' counts over the tokens that count, then the number of these."""
    E, ids, valid = s["E"], s["ids"].long(), _valid(s)
    fine = valid.unsqueeze(1) & (ids >= 0) & (ids < E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    counts.index_add_(0, torch.where(fine, ids, 0).reshape(-1), fine.reshape(-1).long())
    counts[E] = valid.sum()
    return counts.to(torch.int32)


def _plain_probs(s):
    z = torch.where(_valid(s).unsqueeze(1), s["logits"], 0.0)
    e = torch.exp(z - z.amax(1, keepdim=True))
    return torch.where(_valid(s).unsqueeze(1), e / e.sum(1, keepdim=True), 0.0)


def _plain_balance(s):
    E, k = s["E"], s["k"]
    counts = _plain_counts(s)
    n = counts[E].clamp(min=1).float()
    mean_p = _plain_probs(s).sum(0) / n
    loss = s["coef"] * E * (counts[:E].float() / (k * n) * mean_p).sum()
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts[:E], 0).to(torch.int32)])
    return dict(counts=counts, offsets=offsets, mean_p=mean_p, loss=loss.reshape(1))


def _plain_balance_grad(s):
    E, k = s["E"], s["k"]
    p, counts = _plain_probs(s), s["counts"]
    n = counts[E].clamp(min=1).float()
    f = counts[:E].float() / (k * n)
    f = f - f.mean()  # a softmax's gradient does not see a constant
    return s["dloss"] * s["coef"] * E / n * p * (f - (p * f).sum(1, keepdim=True))


def _plain_sample(s):
    # in 64 bits: which token comes out depends on sums next to a border
    B, V = s["B"], s["V"]
    logits = s["logits"].double()
    order_l, order = torch.sort(logits, dim=1, descending=True, stable=True)
    top = order_l[:, :1]
    greedy = s["temperature"] <= 0
    t = torch.where(greedy, 1.0, s["temperature"].double()).unsqueeze(1)
    w = torch.exp((order_l - top) / t)
    keep = torch.ones(B, V, dtype=torch.bool, device=DEV)
    if s["top_k"] is not None:
        keep &= torch.arange(V, device=DEV) < s["top_k"].unsqueeze(1)
    if s["top_p"] is not None:
        wk = torch.where(keep, w, 0.0)
        before = torch.cumsum(wk, 1) - wk
        keep &= before < s["top_p"].double().unsqueeze(1) * wk.sum(1, keepdim=True)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double().unsqueeze(1)
    keep[:, 0] = True
    keep &= ~greedy.unsqueeze(1) | (torch.arange(V, device=DEV) == 0)
    weight = torch.zeros(B, V, dtype=torch.float64, device=DEV).scatter_(1, order, torch.where(keep, w, 0.0))
    c = torch.cumsum(weight, 1)
    total = c[:, -1:]
    token = (c <= s["u"].double().unsqueeze(1) * total).sum(1, keepdim=True).clamp(max=V - 1)
    prob = weight.gather(1, token) / total
    return dict(token=token[:, 0].to(torch.int32), prob=prob[:, 0].float())


# ------------------------------------------------------------------ the framework's calls

def _own_q4(s):
    from lfsr_seeded_moe_b200 import nslm
    if "W" not in s:
        s["W"] = nslm.q4_matrix(s["q"], s["scales"], s["biases"], s["group"])
    nslm.nslm_q4_gemv(s["W"], s["x"], s["M"], s["y"], nslm.NSLM_GEMV_FIELDS_READY)
    return s["y"]


def _own_balance(s):
    from lfsr_seeded_moe_b200 import nslm
    if "ws" not in s:
        s["ws_bytes"] = nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_BALANCE, s["T"], s["E"], 0, 0, s["k"])
        s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device=DEV)
    nslm.nslm_moe_balance(s["logits"], s["ids"], s["mask"], s["T"], s["E"], s["k"], s["coef"], s["counts"], s["offsets"],
                          s["mean_p"], s["loss"], s["ws"], s["ws_bytes"])
    return {n: s[n] for n in ("counts", "offsets", "mean_p", "loss")}


def _own_balance_grad(s):
    from lfsr_seeded_moe_b200 import nslm
    nslm.nslm_moe_balance_grad(s["logits"], s["counts"], s["mask"], s["T"], s["E"], s["k"], s["coef"], s["dloss"], s["dlogits"])
    return s["dlogits"]


def _own_sample(s):
    from lfsr_seeded_moe_b200 import nslm
    if "params" not in s:
        s["params"] = nslm.sample_params(s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    kind = nslm.NSLM_TYPE_BF16 if s["bits"] == 16 else nslm.NSLM_TYPE_F32
    nslm.nslm_sample(s["logits"], kind, s["B"], s["V"], s["V"], s["params"], s["u"], s["token"], s["prob"])
    return dict(token=s["token"], prob=s["prob"])


def run(state):
    op = state["op"]
    if own:
        return {"q4_gemv": _own_q4, "balance": _own_balance, "balance_grad": _own_balance_grad, "sample": _own_sample}[op](state)
    return {"q4_gemv": _plain_q4, "balance": _plain_balance, "balance_grad": _plain_balance_grad, "sample": _plain_sample}[op](state)


def work(case):
    if case["op"] == "q4_gemv":
        N, K, G, M = case["N"], case["K"], case["group"], case["M"]
        return dict(bytes=N * K // 2 + N * (K // G) * (4 if case["affine"] else 2) + 2 * M * K + 4 * M * N, flops=2 * M * N * K)
    if case["op"] == "sample":
        return dict(bytes=case["B"] * case["V"] * case["bits"] // 8, flops=4 * case["B"] * case["V"])
    T, E, k = case["T"], case["E"], case["k"]
    live = T - int(T * case["padded"])
    masked = T if case["padded"] else 0
    if case["op"] == "balance":
        return dict(bytes=4 * live * (E + k) + masked + 12 * E, flops=5 * live * E)
    return dict(bytes=4 * live * E + 4 * T * E + masked + 4 * E, flops=7 * live * E)


# ------------------------------------------------------------------ in 64 bits

def _exact_q4(s):
    N, K, G, M = s["N"], s["K"], s["group"], s["M"]
    y = torch.empty(M, N, dtype=torch.float64, device=DEV)
    x = s["x"].double()
    step = max(1, (1 << 26) // K)
    for r in range(0, N, step):
        b = s["q"][r:r + step].contiguous().view(torch.uint8)
        w = torch.stack([b & 15, b >> 4], -1).reshape(b.shape[0], K).double()
        scale = s["scales"][r:r + step].double().repeat_interleave(G, 1)
        shift = s["biases"][r:r + step].double().repeat_interleave(G, 1) if s["biases"] is not None else -8.0 * scale
        y[:, r:r + step] = x @ torch.addcmul(shift, w, scale).t()
    return y


def _exact_balance(s, grad):
    E, k, T = s["E"], s["k"], s["T"]
    rows = torch.arange(T, device=DEV) if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
    n = max(1, rows.numel())
    z = s["logits"][rows].double().requires_grad_(True)
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    picked = s["ids"][rows].reshape(-1).long()
    counts = torch.bincount(picked[(picked >= 0) & (picked < E)], minlength=E)
    mean_p = p.sum(0) / n
    loss = s["coef"] * E * torch.dot(counts.double(), mean_p) / (k * n)
    if not grad:
        ends = torch.cumsum(counts, 0)
        return dict(counts=torch.cat([counts, counts.new_tensor([rows.numel()])]).to(torch.int32),
                    offsets=torch.cat([ends.new_zeros(1), ends]).to(torch.int32), mean_p=mean_p.detach(), loss=loss.detach().reshape(1))
    d = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    if rows.numel():
        d[rows] = torch.autograd.grad(loss * s["dloss"].double()[0], z)[0]
    return d


def _exact_sample(s):
    B, V = s["B"], s["V"]
    host = lambda t: None if t is None else t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    logits, u, temp = host(s["logits"]), host(s["u"]), host(s["temperature"])
    top_p, min_p = host(s["top_p"]), host(s["min_p"])
    top_k = None if s["top_k"] is None else s["top_k"].cpu().numpy()
    token, prob = np.zeros(B, np.int32), np.zeros(B, np.float64)
    for b in range(B):
        if temp[b] <= 0:
            token[b], prob[b] = int(np.argmax(logits[b])), 1.0
            continue
        p = np.exp((logits[b] - logits[b].max()) / temp[b])
        rank = np.lexsort((np.arange(V), -logits[b]))
        n = V if top_k is None else min(V, int(top_k[b]))
        if top_p is not None:
            sums = np.cumsum(p[rank[:n]])
            n = min(n, int(np.searchsorted(sums, top_p[b] * sums[-1])) + 1)
        if min_p is not None:
            n = max(1, min(n, int(np.count_nonzero(p >= min_p[b]))))
        kept = np.sort(rank[:n])
        sums = np.cumsum(p[kept])
        i = kept[min(n - 1, int(np.searchsorted(sums, u[b] * sums[-1], side="right")))]
        token[b], prob[b] = i, p[i] / sums[-1]
    return dict(token=token, prob=prob)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "q4_gemv":
        return _exact_q4(s)
    if case["op"] == "sample":
        return _exact_sample(s)
    return _exact_balance(s, case["op"] == "balance_grad")
