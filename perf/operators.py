"""The operators of the routing's training step, as cases to measure: the load-balance loss with its
gradient, 8-bit activation checkpoints, the routing's slot gradients from 8-bit expert outputs, and
the router's linear backward (its weight gradient from an 8-bit x, its input gradient).

listed() and draw() give the cases, prepare() a case's inputs on the GPU, run() one pass (the plain
form in elementary torch operations, or the package's call where `own` is set), work() the bytes and
operations that the pass cannot do without, and exact() the result in 64 bits.

The layer shapes are the ones of the synthetic layers: (D, E, K) = (4096, 8, 2), (2048, 64, 6),
(2048, 60, 4), (1536, 212, 16) and the tiny float32 layer (256, 8, 2).
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 32          # columns that share one power-of-two scale
K_MIN = -120        # smallest scale exponent kept


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # the loss of a 64-token micro-batch of the Mixtral-like layer: two tiny launches
        dict(name="balance 64x8", op="balance", T=64, E=8, K=2, dtype="f32", seqs=0, pad=0.0),
        # sequence-wise loss of a packed 16384-token batch (60 experts), padded tokens left out
        dict(name="balance 16384x60 packed", op="balance", T=16384, E=60, K=4, dtype="bf16",
             seqs=24, pad=0.1),
        # the full logit gradient of the fine-grained layer: balance term plus the slots' terms
        dict(name="balance grad 8192x212 slots", op="balance_grad", T=8192, E=212, K=16,
             dtype="f32", seqs=0, pad=0.0, slots=True),
        # the balance term alone, sequence-wise, odd token count (64 experts)
        dict(name="balance grad 1237x64 packed", op="balance_grad", T=1237, E=64, K=6,
             dtype="bf16", seqs=7, pad=0.05, slots=False),
        # expert outputs of a 4096-token Mixtral-like batch (two slots each), saved and read back
        dict(name="checkpoint 8192x4096 f16", op="checkpoint", N=8192, D=4096, dtype="f16",
             stride=0),
        # a short batch of float32 rows, odd width, cut out of a wider tensor
        dict(name="checkpoint 323x1413 f32", op="checkpoint", N=323, D=1413, dtype="f32",
             stride=27),
        # slot gradients of the fine-grained layer, the largest batch
        dict(name="route grad 8192x16x1536", op="route_grad", T=8192, K=16, D=1536, dtype="f32",
             seg=0),
        # slot gradients of a small Mixtral-like micro-batch
        dict(name="route grad 33x2x4096", op="route_grad", T=33, K=2, D=4096, dtype="bf16",
             seg=0),
        # dW of both routers of the fine-grained layer (2 x 212 logit columns)
        dict(name="weight grad 8192x1536x424", op="weight_grad", T=8192, D=1536, C=424,
             dtype="f32"),
        # dW of a DeepSeek-like router from bf16 logit gradients, ragged token count
        dict(name="weight grad 1003x2048x128", op="weight_grad", T=1003, D=2048, C=128,
             dtype="bf16"),
        # dx of both DeepSeek-like routers at prefill length
        dict(name="input grad 8192x2048x128", op="input_grad", T=8192, D=2048, C=128,
             dtype="f32", wdtype="bf16"),
        # dx of the tiny float32 layer
        dict(name="input grad 64x256x16", op="input_grad", T=64, D=256, C=16, dtype="f32",
             wdtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance_grad", "checkpoint", "route_grad", "weight_grad",
                     "input_grad"])
    if op in ("balance", "balance_grad"):
        E = _log(rng, 2, 256)
        K = rng.randint(1, min(32, E))
        T = min(_log(rng, 1, 65536), 4_000_000 // E)
        c = dict(op=op, T=T, E=E, K=K, dtype=rng.choice(["f32", "bf16"]),
                 seqs=rng.choice([0, _log(rng, 1, 64)]), pad=rng.choice([0.0, 0.1, 0.5]))
        if op == "balance_grad":
            c["slots"] = rng.random() < 0.5
        return c
    if op == "checkpoint":
        D = rng.choice([_log(rng, 8, 8192), 32 * rng.randint(1, 256)])
        N = min(_log(rng, 1, 131072), 32_000_000 // D)
        return dict(op=op, N=N, D=D, dtype=rng.choice(["f32", "bf16", "f16"]),
                    stride=rng.choice([0, 0, 8, 27]))
    if op == "route_grad":
        D = rng.choice([_log(rng, 32, 8192), 64 * rng.randint(1, 128)])
        K = _log(rng, 1, 32)
        T = min(_log(rng, 1, 16384), 150_000_000 // (K * D))
        return dict(op=op, T=T, K=K, D=D, dtype=rng.choice(["f32", "bf16"]),
                    seg=rng.choice([0, 0, 16]))
    D = rng.choice([_log(rng, 32, 8192), 64 * rng.randint(1, 128)])
    C = _log(rng, 2, 512)
    T = min(_log(rng, 1, 32768), 5_000_000_000 // (C * D), 24_000_000 // D)
    c = dict(op=op, T=T, D=D, C=C, dtype=rng.choice(["f32", "bf16"]))
    if op == "input_grad":
        c["wdtype"] = rng.choice(["f32", "bf16"])
    return c


# ------------------------------------------------------------------------------------ inputs
def _pow2(k):
    """2^k in float32 for integer k in [-126, 127], exactly: the exponent field of its bits."""
    return ((k.int() + 127) << 23).view(torch.float32)


def _encode(x):
    """(q int8 [N][D rounded up to 32], scale uint8 [N][D/32]): per block of 32 columns the
    smallest k >= -120 with max|x| <= 127 * 2^k, q = x * 2^-k rounded to nearest even."""
    N, D = x.shape
    nb = (D + BLOCK - 1) // BLOCK
    x = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - D)).view(N, nb, BLOCK)
    m, e = torch.frexp(x.abs().amax(2))            # a = m 2^e with m in [0.5, 1)
    k = torch.where(m <= 127 / 128, e - 7, e - 6).clamp(min=K_MIN)
    q = torch.round(x * _pow2(-k)[:, :, None]).clamp(-127, 127)
    return q.to(torch.int8).view(N, nb * BLOCK), (k + 127).to(torch.uint8)


def _decode(q, scale, D):
    N, nb = scale.shape
    v = q.view(N, nb, BLOCK).float() * _pow2(scale.int() - 127)[:, :, None]
    return v.view(N, nb * BLOCK)[:, :D]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    op = case["op"]
    s = dict(op=op)
    if op in ("balance", "balance_grad"):
        T, E, K = case["T"], case["E"], case["K"]
        # router logits with a popularity bias, so that some experts are chosen more often
        logits = (randn(T, E) + 0.5 * randn(1, E)).to(_DT[case["dtype"]])
        s.update(E=E, K=K, logits=logits, valid=None, cu=None,
                 topk=torch.topk(logits.float(), K, dim=1).indices.to(torch.int32))
        if case["pad"]:
            s["valid"] = (rand(T) >= case["pad"]).to(torch.uint8)
        if case["seqs"]:
            # packed sequences of different lengths (some empty), the last few rows unused
            end = T - T // 50
            cuts = torch.sort((rand(case["seqs"] - 1) * (end + 1)).to(torch.int32)).values
            ends = torch.tensor([0, end], dtype=torch.int32, device="cuda")
            s["cu"] = torch.cat([ends[:1], cuts, ends[1:]])
        if op == "balance_grad":
            s["scale"] = 0.01
            s["fwd"] = _balance(s)
            s["dgl"] = s["dml"] = None
            if case["slots"]:
                s["dgl"], s["dml"] = 1e-4 * randn(T, K), 1e-4 * randn(T, K)
    elif op == "checkpoint":
        N, D = case["N"], case["D"]
        x = randn(N, D + case["stride"]) * torch.exp(randn(N, 1))
        s.update(x=x.to(_DT[case["dtype"]])[:, :D])
    elif op == "route_grad":
        T, K, D, S = case["T"], case["K"], case["D"], max(1, case["seg"])
        q, scale = _encode(randn(T * K, D))
        lead = torch.arange(T, device="cuda") // S * S   # a segment's tokens share a decision
        gate = torch.softmax(randn(T, K), 1)[lead].contiguous()
        mlogit = randn(T, K)[lead].contiguous()
        s.update(q=q, qscale=scale, D=D, gate=gate, mlogit=mlogit, seg=case["seg"], reg=0.1,
                 dy=(randn(T, D) / D ** 0.5).to(_DT[case["dtype"]]))
    elif op == "weight_grad":
        T, D, C = case["T"], case["D"], case["C"]
        q, scale = _encode(randn(T, D))
        s.update(q=q, qscale=scale, D=D, g=(1e-3 * randn(T, C)).to(_DT[case["dtype"]]))
    else:
        T, D, C = case["T"], case["D"], case["C"]
        s.update(g=(1e-3 * randn(T, C)).to(_DT[case["dtype"]]),
                 w=(randn(D, C) / D ** 0.5).to(_DT[case["wdtype"]]))
    return s


# ------------------------------------------------------------------------------------ plain forms
def _groups(s):
    """One-hot membership [G][T] of the valid tokens in the loss's groups, and each token's group
    (G for a row behind the last sequence)."""
    T = s["logits"].shape[0]
    t = torch.arange(T, device="cuda")
    if s["cu"] is None:
        g, G = torch.zeros_like(t), 1
    else:
        g, G = torch.searchsorted(s["cu"][1:].long().contiguous(), t, right=True), len(s["cu"]) - 1
    member = g[None, :] == torch.arange(G, device="cuda")[:, None]
    if s["valid"] is not None:
        member = member & (s["valid"] != 0)[None, :]
    return member, g


def _softmax(logits):
    x = logits.float()
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _balance(s):
    E, K = s["E"], s["K"]
    member, g = _groups(s)
    G = member.shape[0]
    n = member.sum(1)
    inside = member.any(0)
    place = torch.where(inside, g, G)[:, None] * E + s["topk"].long()
    counts = torch.zeros((G + 1) * E, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, place.view(-1), torch.ones_like(place.view(-1), dtype=torch.int32))
    counts = counts.view(G + 1, E)[:G]
    nf = n.clamp(min=1).float()[:, None]
    prob = (member.float() @ _softmax(s["logits"])) / nf
    f = counts.float() * E / (K * nf)
    loss = (f * prob).sum() / (n > 0).sum().clamp(min=1)
    return dict(loss=loss, counts=counts, prob=prob, tokens=n.to(torch.int32))


def _balance_grad(s):
    E, K = s["E"], s["K"]
    member, g = _groups(s)
    n, counts = s["fwd"]["tokens"], s["fwd"]["counts"]
    nf = n.clamp(min=1).float()[:, None]
    f = counts.float() * E / (K * nf)
    coef = s["scale"] / ((n > 0).sum().clamp(min=1) * nf)
    inside, g = member.any(0), g.clamp(max=len(n) - 1)
    p, f = _softmax(s["logits"]), f[g]
    d = torch.where(inside[:, None], coef[g] * p * (f - (f * p).sum(1, keepdim=True)), 0.0)
    if s["dgl"] is None:
        return d
    ids = s["topk"].long()
    d = d.scatter_add(1, ids, s["dgl"])
    return torch.cat([d, torch.zeros_like(d).scatter_add(1, ids, s["dml"])], 1)


def _route_grad(s):
    T, K = s["gate"].shape
    S = max(1, s["seg"])
    y = _decode(s["q"], s["qscale"], s["D"]).view(T, K, s["D"])
    dghat = torch.matmul(y, s["dy"].float()[:, :, None])[:, :, 0]
    Tr = (T + S - 1) // S
    run = torch.nn.functional.pad(dghat, (0, 0, 0, Tr * S - T)).view(Tr, S, K).sum(1)
    length = (T - torch.arange(Tr, device="cuda") * S).clamp(max=S)[:, None]
    gate, l = s["gate"][::S], s["mlogit"][::S]
    sig = 1 / (1 + torch.exp(-l))
    dgl, dml = torch.zeros_like(dghat), torch.zeros_like(dghat)
    dml[::S] = (run * gate + length * (s["reg"] / (T * K))) * sig * (1 - sig)
    dg = torch.where(l >= 0, run, 0.0)
    dgl[::S] = gate * (dg - (gate * dg).sum(1, keepdim=True))
    return dict(dghat=dghat, d_gate_logit=dgl, d_mask_logit=dml)


def run(s):
    op = s["op"]
    if own:
        import dynamic_expert_routing_b200 as beam
        if op == "balance":
            return beam.balance_loss(s["logits"], s["topk"], valid=s["valid"], cu_seqlens=s["cu"])
        if op == "balance_grad":
            return beam.balance_loss_backward(s["logits"], s["topk"], s["fwd"], scale=s["scale"],
                                              valid=s["valid"], cu_seqlens=s["cu"],
                                              d_gate_logit=s["dgl"], d_mask_logit=s["dml"])
        if op == "checkpoint":
            return beam.checkpoint_load(beam.checkpoint_save(s["x"]), s["x"].dtype)
        ckpt = dict(q=s.get("q"), scale=s.get("qscale"), d=s.get("D"))
        if op == "route_grad":
            return beam.checkpoint_route_grad(ckpt, s["gate"], s["mlogit"], s["dy"],
                                              reg_scale=s["reg"], segment_len=s["seg"])
        if op == "weight_grad":
            return beam.router_weight_grad(ckpt, s["g"])
        return beam.router_input_grad(s["g"], s["w"])
    if op == "balance":
        return _balance(s)
    if op == "balance_grad":
        return _balance_grad(s)
    if op == "checkpoint":
        return _decode(*_encode(s["x"]), s["x"].shape[1]).to(s["x"].dtype)
    if op == "route_grad":
        return _route_grad(s)
    if op == "weight_grad":
        return _decode(s["q"], s["qscale"], s["D"]).t() @ s["g"].float()
    return s["g"].float() @ s["w"].float().t()


# ------------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    es = _SIZE[case["dtype"]]
    if op in ("balance", "balance_grad"):
        T, E, K, G = case["T"], case["E"], case["K"], max(1, case["seqs"])
        head = T * (1 if case["pad"] else 0) + 4 * case["seqs"]
        if op == "balance":
            return dict(bytes=T * E * es + 4 * T * K + head + 8 * G * E + 4 * G + 4,
                        flops=4 * T * E)
        out = 2 if case["slots"] else 1
        return dict(bytes=T * E * es + head + 4 * G * E + (12 * T * K if case["slots"] else 0) +
                    4 * T * E * out, flops=8 * T * E)
    if op == "checkpoint":
        n = case["N"] * case["D"]
        return dict(bytes=2 * n * es, flops=4 * n)
    if op == "route_grad":
        T, K, D = case["T"], case["K"], case["D"]
        return dict(bytes=T * K * (D + D // BLOCK) + T * D * es + 20 * T * K,
                    flops=2 * T * K * D)
    T, D, C = case["T"], case["D"], case["C"]
    if op == "weight_grad":
        return dict(bytes=T * (D + D // BLOCK) + T * C * es + 4 * D * C, flops=2 * T * D * C)
    return dict(bytes=T * C * es + D * C * _SIZE[case["wdtype"]] + 4 * T * D,
                flops=2 * T * D * C)


# ------------------------------------------------------------------------------------ 64 bits
def _step64(k):
    """2^k in float64 for integer k, exactly."""
    return torch.bitwise_left_shift(k.long() + 1023, 52).view(torch.float64)


def _values64(s):
    """The checkpoint's values in float64."""
    rep = _step64(s["qscale"].int() - 127).repeat_interleave(BLOCK, 1)
    return (s["q"].double() * rep)[:, :s["D"]]


def _member64(s):
    T = s["logits"].shape[0]
    cu = [0, T] if s["cu"] is None else s["cu"].tolist()
    inside = torch.zeros(len(cu) - 1, T, dtype=torch.float64, device="cuda")
    for g in range(len(cu) - 1):
        inside[g, cu[g]:cu[g + 1]] = 1
    return inside if s["valid"] is None else inside * (s["valid"] != 0).double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("balance", "balance_grad"):
        E, K, T = case["E"], case["K"], case["T"]
        inside = _member64(s)
        n = inside.sum(1)
        p = torch.softmax(s["logits"].double(), 1)
        chosen = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        chosen.scatter_add_(1, s["topk"].long(), torch.ones_like(s["topk"], dtype=torch.float64))
        counts = inside @ chosen
        per = torch.where(n > 0, 1 / n.clamp(min=1), 0.0)[:, None]
        f, prob = counts * per * (E / K), (inside @ p) * per
        active = max(1, int((n > 0).sum()))
        if op == "balance":
            return dict(loss=(f * prob).sum() / active, counts=counts.round().int(), prob=prob,
                        tokens=n.round().int())
        w = (inside * per * (s["scale"] / active)).sum(0)[:, None]
        ft = inside.t() @ f
        d = w * p * (ft - (ft * p).sum(1, keepdim=True))
        if s["dgl"] is None:
            return d
        d = torch.cat([d, torch.zeros_like(d)], 1)
        d.scatter_add_(1, s["topk"].long(), s["dgl"].double())
        d.scatter_add_(1, s["topk"].long() + E, s["dml"].double())
        return d
    if op == "checkpoint":
        x = s["x"].double()
        N, D = x.shape
        wide = torch.zeros(N, -(-D // BLOCK) * BLOCK, dtype=torch.float64, device="cuda")
        wide[:, :D] = x
        a = wide.view(N, -1, BLOCK).abs().amax(2)
        k = torch.ceil(torch.log2(a / 127)).clamp(min=K_MIN, max=127)
        k = torch.where(a > 127 * _step64(k), k + 1, k)
        k = torch.where((a <= 127 * _step64(k - 1)) & (k > K_MIN), k - 1, k)
        step = _step64(k).repeat_interleave(BLOCK, 1)
        return (torch.round(wide / step) * step)[:, :D].contiguous()
    if op == "route_grad":
        T, K, S = case["T"], case["K"], max(1, case["seg"])
        y, dy = _values64(s), s["dy"].double()
        dghat = torch.stack([(y[k::K] * dy).sum(1) for k in range(K)], 1)
        lead = torch.arange(T, device="cuda") // S
        run = torch.zeros(int(lead[-1]) + 1, K, dtype=torch.float64, device="cuda")
        run.index_add_(0, lead, dghat)
        size = torch.bincount(lead).double()[:, None]
        g, l = s["gate"][::S].double(), s["mlogit"][::S].double()
        dg = run * (l >= 0)
        dgl, dml = torch.zeros_like(dghat), torch.zeros_like(dghat)
        dgl[::S] = g * (dg - (g * dg).sum(1, keepdim=True))
        dml[::S] = (run * g + size * s["reg"] / (T * K)) * torch.sigmoid(l) * torch.sigmoid(-l)
        return dict(dghat=dghat, d_gate_logit=dgl, d_mask_logit=dml)
    if op == "weight_grad":
        return torch.einsum("td,tc->dc", _values64(s), s["g"].double())
    return torch.einsum("tc,dc->td", s["g"].double(), s["w"].double())
