"""Cases of the operators around the norm: layer norm, the embedding and its
gradient, and the linear cross entropy (the projection onto the vocabulary and
the softmax loss), forward and backward.

``run`` computes a case in its plain form (torch operations in fp32, rounded once
at the end) or, where ``own`` is true, through this package's entry points.
``exact`` gives the same outputs from the definitions in fp64.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_EB = {"bf16": 2, "f16": 2, "f32": 4}
_EPS = 1e-5


def listed():
    ln, em, xe = "layer_norm", "embedding", "linear_xent"
    return [
        # a latency-bound step: the smallest batch of a head-sized norm, both directions
        dict(name="layer_norm step 64x128 f32", op=ln, grad=True, rows=64, width=128, dtype="f32",
             bias=True),
        # one layer's norm over a prompt batch, no gradient kept
        dict(name="layer_norm fwd 16384x2048 bf16", op=ln, grad=False, rows=16384, width=2048,
             dtype="bf16", bias=True),
        # a training step's norm at a wide hidden size
        dict(name="layer_norm step 16384x5120 bf16", op=ln, grad=True, rows=16384, width=5120,
             dtype="bf16", bias=True),
        # an odd batch of a ragged width, no bias
        dict(name="layer_norm step 8191x1032 f16", op=ln, grad=True, rows=8191, width=1032,
             dtype="f16", bias=False),
        # decoding: one new token of each of a few sequences
        dict(name="embedding fwd 24 tokens bf16", op=em, grad=False, tokens=24, vocab=151936,
             width=2048, dtype="bf16", zipf=1.0, add=False),
        # a packed prompt batch
        dict(name="embedding fwd 32768 tokens bf16", op=em, grad=False, tokens=32768,
             vocab=151936, width=2048, dtype="bf16", zipf=1.0, add=False),
        # the dense gradient of a training batch, words distributed as in text
        dict(name="embedding bwd 32768 tokens bf16", op=em, grad=True, tokens=32768,
             vocab=151936, width=2048, dtype="bf16", zipf=1.0, add=False),
        # a tied table: added to the gradient that the head left there; ragged sizes
        dict(name="embedding bwd 4999 tokens f32 add", op=em, grad=True, tokens=4999,
             vocab=50021, width=1032, dtype="f32", zipf=1.0, add=True),
        # scoring the last token of a few sequences
        dict(name="linear_xent fwd 7x2048 V151936 bf16", op=xe, grad=False, rows=7, width=2048,
             vocab=151936, dtype="bf16", softcap=0.0, ignored=0.0),
        # log-probabilities of a rollout batch, with the soft cap
        dict(name="linear_xent fwd 4096x2048 V151936 cap bf16", op=xe, grad=False, rows=4096,
             width=2048, vocab=151936, dtype="bf16", softcap=30.0, ignored=0.0),
        # a training step; a quarter of the tokens is prompt and carries no loss
        dict(name="linear_xent step 4096x2048 V151936 bf16", op=xe, grad=True, rows=4096,
             width=2048, vocab=151936, dtype="bf16", softcap=0.0, ignored=0.25),
        # a small step with ragged sizes
        dict(name="linear_xent step 509x1032 V32771 f16", op=xe, grad=True, rows=509, width=1032,
             vocab=32771, dtype="f16", softcap=0.0, ignored=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer_norm", "embedding", "linear_xent"])
    if op == "layer_norm":
        width = 8 * _log_int(rng, 8, 1024)
        rows = _log_int(rng, 1, max(2, min(100_000, 16384 * 5120 // width)))
        return dict(op=op, grad=rng.random() < 0.6, rows=rows, width=width,
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), bias=rng.random() < 0.7)
    if op == "embedding":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        width = 8 * _log_int(rng, 8, 640)
        vocab = _log_int(rng, 100, min(200_000, 150_000_000 // width))
        tokens = _log_int(rng, 1, min(65_536, 80_000_000 // width))
        return dict(op=op, grad=rng.random() < 0.6, tokens=tokens, vocab=vocab, width=width,
                    dtype=dtype, zipf=rng.choice([0.0, 1.0, 1.0, 2.0]), add=rng.random() < 0.4)
    width = 8 * _log_int(rng, 16, 512)
    vocab = _log_int(rng, 500, min(160_000, 300_000_000 // width))
    rows = _log_int(rng, 1, max(2, min(4096, 1_200_000_000_000 // (width * vocab))))
    return dict(op=op, grad=rng.random() < 0.5, rows=rows, width=width, vocab=vocab,
                dtype=rng.choice(["bf16", "bf16", "f16"]), softcap=rng.choice([0.0, 0.0, 30.0]),
                ignored=rng.choice([0.0, 0.0, 0.25, 0.6]))


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    dt = _DT[case["dtype"]]
    s = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    H = case["width"]
    if case["op"] == "layer_norm":
        R = case["rows"]
        x = normal(R, H).add_(0.5 * normal(R, 1))      # rows with a mean of their own
        x[:, : max(1, H // 100)] *= 8.0                # and a few strong channels
        s["x"] = x.to(dt)
        s["w"] = 1.0 + 0.1 * normal(H)
        s["b"] = 0.1 * normal(H) if case["bias"] else None
        if case["grad"]:
            s["dy"] = normal(R, H).to(dt)
    elif case["op"] == "embedding":
        N, V = case["tokens"], case["vocab"]
        u = torch.rand(N, generator=g, device=dev, dtype=torch.float64)
        if case["zipf"] == 0.0:
            r = u * V
        elif case["zipf"] == 1.0:                      # rank r with a weight of 1 / r
            r = torch.exp(u * math.log(V + 1.0)) - 1.0
        else:                                          # 1 / r^2: a few ids take most tokens
            r = 1.0 / (1.0 - u * (V / (V + 1.0))) - 1.0
        rank = r.to(torch.int64).clamp_(0, V - 1)
        perm = torch.randperm(V, generator=g, device=dev)
        s["ids"] = perm[rank].contiguous()
        s["scale"] = math.sqrt(H)
        if case["grad"]:
            s["dy"] = normal(N, H).to(dt)
            if case["add"]:
                s["old"] = (0.1 * normal(V, H)).to(dt)
        else:
            s["table"] = (normal(V, H) / math.sqrt(H)).to(dt)
    else:
        R, V = case["rows"], case["vocab"]
        w = (normal(V, H) * (2.0 / math.sqrt(H))).to(dt)
        t = torch.randint(0, V, (R,), generator=g, device=dev)
        # targets from hardly to almost certainly predicted
        a = 8.0 * torch.rand(R, 1, generator=g, device=dev)
        x = normal(R, H) + a * torch.nn.functional.normalize(w[t].float(), dim=1)
        if case["ignored"] > 0:
            gone = torch.rand(R, generator=g, device=dev) < case["ignored"]
            t = torch.where(gone, torch.full_like(t, -100), t)
        s.update(x=x.to(dt), w=w, target=t)
        if case["grad"]:
            s["dnll"] = (0.5 + torch.rand(R, generator=g, device=dev)) / R * 1024.0
    return s


# ---- plain forms ---------------------------------------------------------------


def _layer_norm(s):
    x, w = s["x"].float(), s["w"]
    H = x.shape[1]
    mean = x.sum(1, keepdim=True) / H
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).sum(1, keepdim=True) / H + _EPS)
    xh = c * rstd
    y = xh * w
    if s["b"] is not None:
        y = y + s["b"]
    out = {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["grad"]:
        dy = s["dy"].float()
        gd = dy * w
        dx = rstd * (gd - gd.sum(1, keepdim=True) / H - xh * ((gd * xh).sum(1, keepdim=True) / H))
        out["dx"] = dx.to(s["x"].dtype)
        out["dw"] = (dy * xh).sum(0)
        if s["b"] is not None:
            out["db"] = dy.sum(0)
    return out


def _embedding(s):
    if not s["grad"]:
        return {"y": (s["table"][s["ids"]].float() * s["scale"]).to(s["table"].dtype)}
    dy = s["dy"]
    total = torch.zeros(s["vocab"], s["width"], device=dy.device)
    total.index_add_(0, s["ids"], dy.float())
    total *= s["scale"]
    if s["add"]:
        total += s["old"].float()
    return {"dtable": total.to(dy.dtype)}


def _linear_xent(s):
    x, w, t, cap = s["x"].float(), s["w"].float(), s["target"], s["softcap"]
    kept = t >= 0
    at = t.clamp(min=0)[:, None]
    z = x @ w.T
    if cap > 0:
        z = cap * torch.tanh(z / cap)
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    nll = torch.where(kept, (lse - z.gather(1, at))[:, 0], 0.0)
    out = {"nll": nll, "lse": lse[:, 0]}
    if s["grad"]:
        d = torch.exp(z - lse)
        d.scatter_add_(1, at, torch.full_like(lse, -1.0))
        d *= torch.where(kept, s["dnll"], 0.0)[:, None]
        if cap > 0:
            d *= 1.0 - (z / cap) ** 2
        out["dx"] = (d @ w).to(s["x"].dtype)
        out["dw"] = (d.T @ x).to(s["w"].dtype)
    return out


# ---- this package's calls --------------------------------------------------------


def _own_layer_norm(s):
    from rollout_parity_b200 import ops

    y, mean, rstd = ops.layernorm_fwd(s["x"], s["w"], s["b"], _EPS)
    out = {"y": y, "mean": mean, "rstd": rstd}
    if s["grad"]:
        dx, dw, db = ops.layernorm_bwd(s["x"], s["w"], s["dy"], mean, rstd,
                                       want_db=s["b"] is not None)
        out["dx"], out["dw"] = dx, dw
        if db is not None:
            out["db"] = db
    return out


def _own_embedding(s):
    from rollout_parity_b200 import ops

    if not s["grad"]:
        return {"y": ops.embed_fwd(s["ids"], s["table"], s["scale"])}
    if s["add"]:   # into a copy, so that the case can be run again
        return {"dtable": ops.embed_bwd(s["ids"], s["dy"], s["vocab"], s["scale"],
                                        dtable=s["old"].clone(), accumulate=True)}
    return {"dtable": ops.embed_bwd(s["ids"], s["dy"], s["vocab"], s["scale"])}


def _own_linear_xent(s):
    from rollout_parity_b200 import ops

    nll, lse = ops.linear_xent_fwd(s["x"], s["w"], s["target"], s["softcap"])
    out = {"nll": nll, "lse": lse}
    if s["grad"]:
        out["dx"], out["dw"] = ops.linear_xent_bwd(s["x"], s["w"], s["target"], lse, s["dnll"],
                                                   s["softcap"])
    return out


def run(state):
    if own:
        return {"layer_norm": _own_layer_norm, "embedding": _own_embedding,
                "linear_xent": _own_linear_xent}[state["op"]](state)
    return {"layer_norm": _layer_norm, "embedding": _embedding,
            "linear_xent": _linear_xent}[state["op"]](state)


def work(case):
    H, e = case["width"], _EB[case["dtype"]]
    if case["op"] == "layer_norm":
        R, n = case["rows"], case["rows"] * case["width"]
        vec = (2 if case["bias"] else 1) * H * 4
        if case["grad"]:   # x and dy read, y and dx written, the statistics, the weights' gradients
            return {"bytes": 4 * n * e + 8 * R + 2 * vec, "flops": 20 * n}
        return {"bytes": 2 * n * e + 8 * R + vec, "flops": 8 * n}
    if case["op"] == "embedding":
        N, V = case["tokens"], case["vocab"]
        if not case["grad"]:
            return {"bytes": 2 * N * H * e + 8 * N, "flops": N * H}
        return {"bytes": (N + (2 if case["add"] else 1) * V) * H * e + 8 * N, "flops": 2 * N * H}
    R, V = case["rows"], case["vocab"]
    kept = R * (1.0 - case["ignored"])
    b = (R * H + V * H) * e + 16 * R
    f = 2.0 * R * V * H
    if case["grad"]:
        b += (R * H + V * H) * e + 4 * R
        f += 4.0 * kept * V * H
    return {"bytes": b, "flops": f}


# ---- the definitions in 64 bits ----------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer_norm":
        x = s["x"].double().requires_grad_(True)
        w = s["w"].double().requires_grad_(True)
        b = None if s["b"] is None else s["b"].double().requires_grad_(True)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + _EPS)
        y = torch.nn.functional.layer_norm(x, (case["width"],), w, b, _EPS)
        out = {"y": y.detach(), "mean": mean.detach(), "rstd": rstd.detach()}
        if case["grad"]:
            got = torch.autograd.grad(y, [x, w] + ([b] if b is not None else []), s["dy"].double())
            out.update(zip(("dx", "dw", "db"), got))
        return out
    if case["op"] == "embedding":
        if not case["grad"]:
            return {"y": s["scale"] * torch.nn.functional.embedding(s["ids"], s["table"]).double()}
        # sorted tokens: differences of a running sum over blocks of columns
        ids, order = torch.sort(s["ids"], stable=True)
        total = s["old"].double() if case["add"] else \
            torch.zeros(case["vocab"], case["width"], device="cuda", dtype=torch.float64)
        u, n = torch.unique_consecutive(ids, return_counts=True)
        end = torch.cumsum(n, 0)
        for c in range(0, case["width"], 256):
            run_sum = torch.cumsum(s["dy"][order, c:c + 256].double(), 0)
            run_sum = torch.cat([torch.zeros_like(run_sum[:1]), run_sum])
            total[u, c:c + 256] += s["scale"] * (run_sum[end] - run_sum[end - n])
        return {"dtable": total}
    x, w, t, cap = s["x"].double(), s["w"].double(), s["target"], case["softcap"]
    nll, lse, dx = [], [], []
    dw = torch.zeros_like(w) if case["grad"] else None
    for i in range(0, case["rows"], 512):   # blocks of rows: the gradient by autograd
        xi = x[i:i + 512].requires_grad_(case["grad"])
        wi = w.detach().requires_grad_(case["grad"])
        z = xi @ wi.T
        z = z if cap == 0 else cap * torch.tanh(z / cap)
        n = torch.nn.functional.cross_entropy(z, t[i:i + 512], reduction="none")
        lse.append(torch.logsumexp(z.detach(), 1))
        nll.append(n.detach())
        if case["grad"]:
            gx, gw = torch.autograd.grad(n, [xi, wi], s["dnll"][i:i + 512].double())
            dx.append(gx)
            dw += gw
        del z, n
    out = {"nll": torch.cat(nll), "lse": torch.cat(lse)}
    if case["grad"]:
        out.update(dx=torch.cat(dx), dw=dw)
    return out
