"""Cases that measure the training and adapter operators of the MoE layer.

Four operators:

* ``balance``: the load-balance loss of a routing decision with its per-expert
  counts, over one batch or over the sequences packed into it;
* ``gate_backward``: the gradient of the router's logits, from the gradient of
  the gate weights and that of the balance loss;
* ``lora``: a shared projection with the low-rank adapters of many requests
  beside it;
* ``lora_backward``: the gradients of that projection's input and of every
  adapter.

``run`` computes them in plain torch operations, or through the framework's
entry points where ``own`` is true.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the loss of a small fp32 layer's step: nothing but latency
        dict(name="balance_small", op="balance", T=256, E=8, k=2, S=1, masked=False),
        # a training step's batch of packed sequences, fine-grained experts,
        # with padding inside the sequences and rows behind the last one
        dict(name="balance_sequences", op="balance", T=32749, E=256, k=8, S=16, masked=True),
        # the Mixtral-shape layer's step, renormalised gates
        dict(name="gate_backward_mixtral", op="gate_backward", T=4096, E=8, k=2, S=1,
             masked=False, renorm=True),
        # the DeepSeek-shape layer's step over packed sequences
        dict(name="gate_backward_sequences", op="gate_backward", T=16381, E=256, k=8, S=8,
             masked=True, renorm=False),
        # one request's next token
        dict(name="lora_token", op="lora", T=1, K=4096, N=4096, r=16, n=8, dt="bf16",
             out="bf16", rows="requests"),
        # a decode batch of 128 requests on 64 adapters, up to the Mixtral d_ff
        dict(name="lora_decode", op="lora", T=128, K=4096, N=14336, r=16, n=64, dt="bf16",
             out="bf16", rows="mixed"),
        # prompts of 16 requests in one batch
        dict(name="lora_prompts", op="lora", T=4096, K=4096, N=4096, r=16, n=16, dt="bf16",
             out="bf16", rows="requests"),
        # an odd number of rows, higher rank, the DeepSeek expert widths
        dict(name="lora_odd", op="lora", T=1331, K=7168, N=2048, r=64, n=7, dt="bf16",
             out="bf16", rows="requests"),
        # an adapted router: few outputs, fp32 logits
        dict(name="lora_router", op="lora", T=4096, K=7168, N=256, r=8, n=4, dt="bf16",
             out="f32", rows="requests"),
        # the small fp32 layer's width
        dict(name="lora_f32", op="lora", T=256, K=128, N=256, r=8, n=4, dt="f32", out="f32",
             rows="mixed"),
        # a fine-tuning step of eight adapters at once
        dict(name="lora_backward_step", op="lora_backward", T=4096, K=4096, N=4096, r=16, n=8,
             dt="bf16", rows="requests"),
        # few rows spread over many adapters, odd sizes
        dict(name="lora_backward_odd", op="lora_backward", T=777, K=7168, N=2048, r=32, n=33,
             dt="bf16", rows="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["balance", "gate_backward", "lora", "lora", "lora_backward"])
    if op in ("balance", "gate_backward"):
        E = rng.choice([_log(rng, 2, 512), 8, 64, 256])
        T = _log(rng, 1, max(1, (1 << 23) // max(E, 64)))
        c = dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 10)), S=min(T, _log(rng, 1, 64)),
                 masked=rng.random() < 0.5)
        if op == "gate_backward":
            c["renorm"] = rng.random() < 0.5
        return c
    dt = "f32" if rng.random() < 0.2 else "bf16"
    K = 8 * _log(rng, 8, 1024)
    N = _log(rng, 4, 14336) if op == "lora" else 8 * _log(rng, 1, 1024)
    room = (1 << 36) if dt == "bf16" else (1 << 30)
    T = _log(rng, 1, max(1, min(8192, room // (K * N))))
    c = dict(op=op, T=T, K=K, N=N, r=8 * _log(rng, 1, 16), n=_log(rng, 1, 64), dt=dt,
             rows=rng.choice(["requests", "mixed"]))
    if op == "lora":
        c["out"] = "f32" if dt == "f32" else rng.choice(["bf16", "bf16", "f32"])
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _routing(c, g):
    """Router logits of normalised activations with a skewed expert
    popularity, the selection they give, and the batch's sequences."""
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    logits = 1.28 * torch.randn((T, E), generator=g, device=DEV)
    logits -= 0.4 * torch.log1p(torch.randperm(E, generator=g, device=DEV).float())
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    s = dict(c, logits=logits, idx=idx, offsets=None, mask=None)
    if S > 1 or c["masked"]:
        # S packed sequences of random lengths; masked batches also leave some
        # rows behind the last sequence
        end = T - T // 64 if c["masked"] else T
        cut = torch.randint(0, end + 1, (S - 1,), generator=g, device=DEV).sort().values
        s["offsets"] = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), end)]).to(torch.int32)
    if c["masked"]:
        s["mask"] = torch.rand((T,), generator=g, device=DEV) < 0.9
        # padding rows hold whatever the computation before left there
        logits.masked_fill_(~s["mask"][:, None], float("nan"))
    return s


def _adapter_rows(c, g):
    T, n = c["T"], c["n"]
    if c["rows"] == "mixed":  # each row its own request; some without an adapter
        a = torch.randint(-1, n, (T,), generator=g, device=DEV)
    else:  # the rows of a request follow each other
        cut = torch.randint(0, T + 1, (n - 1,), generator=g, device=DEV)
        run = (torch.arange(T, device=DEV)[:, None] >= cut[None, :]).sum(1)
        a = (torch.randperm(n + 1, generator=g, device=DEV) - 1)[run]
    return a.to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["op"] in ("balance", "gate_backward"):
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        s = _routing(c, g)
        s["alpha"] = 0.01
        i32 = torch.int32
        if c["op"] == "balance":
            s["counts"] = torch.empty((S, E), dtype=i32, device=DEV)
            s["probs"] = torch.empty((S, E), device=DEV)
            s["tokens"] = torch.empty((S + 1,), dtype=i32, device=DEV)
            s["loss"] = torch.empty((1,), device=DEV)
        else:
            # gradients of a loss that is a mean over the tokens
            s["d_topk_w"] = torch.randn((T, k), generator=g, device=DEV) / T
            s["d_loss"] = 0.5 + torch.rand((1,), generator=g, device=DEV)
            s["counts"], _, s["tokens"], _ = _balance(s)  # what the forward pass left
            s["d_logits"] = torch.empty((T, E), device=DEV)
        return s
    T, K, N, r, n = c["T"], c["K"], c["N"], c["r"], c["n"]
    dt = TYPES[c["dt"]]
    f32 = torch.float32

    def normal(shape, std, dtype=dt):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(c, adapter=_adapter_rows(c, g),
             scale=0.5 + 1.5 * torch.rand((n,), generator=g, device=DEV),
             A=normal((n, r, K), K ** -0.5), B=normal((n, r, N), 0.5 * r ** -0.5),
             x=normal((T, K), 1.0), v=torch.empty((T, r), dtype=f32, device=DEV))
    if c["op"] == "lora":
        s["W"] = normal((N, K), K ** -0.5)
        s["y"] = torch.empty((T, N), dtype=TYPES[c["out"]], device=DEV)
    else:
        s["W_t"] = normal((K, N), K ** -0.5)
        s["dy"] = normal((T, N), 1e-3)
        s["v"].copy_(_shrink(s, s["x"].float(), s["A"].float()))  # what the forward pass left
        s["u"] = torch.empty((T, r), dtype=f32, device=DEV)
        s["dx"] = torch.empty((T, K), dtype=dt, device=DEV)
        s["dA"] = torch.empty((n, r, K), dtype=f32, device=DEV)
        s["dB"] = torch.empty((n, r, N), dtype=f32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _member(s):
    """[T][S] 0/1: the sequence that a token counts for (none for padding)."""
    T, S = s["T"], s["S"]
    t = torch.arange(T, device=DEV)[:, None]
    off = s["offsets"] if s["offsets"] is not None else torch.tensor([0, T], device=DEV)
    m = (t >= off[None, :S]) & (t < off[None, 1:])
    if s["mask"] is not None:
        m = m & s["mask"][:, None]
    return m


def _softmax(logits, valid):
    z = torch.where(valid[:, None], logits, torch.zeros_like(logits))
    e = torch.exp(z - z.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _balance(s):
    E = s["E"]
    m = _member(s)
    p = _softmax(s["logits"], m.any(1))
    hot = m.float()
    picked = (s["idx"][:, :, None] == torch.arange(E, device=DEV)).sum(1).float()
    tokens = m.sum(0)
    counts = hot.t() @ picked
    per = tokens.float()[:, None].clamp_min(1.0)
    probs = (hot.t() @ p) / per
    each = E * (counts / (per * s["k"]) * probs).sum(1)
    some = (tokens > 0).sum()
    loss = s["alpha"] * each.sum() / some.clamp_min(1).float()
    return (counts.to(torch.int32), probs, torch.cat([tokens, some[None]]).to(torch.int32),
            loss[None])


def _gate_backward(s):
    E, k = s["E"], s["k"]
    m = _member(s)
    valid = m.any(1)
    p = _softmax(s["logits"], valid)
    pick = s["idx"][:, :, None] == torch.arange(E, device=DEV)
    dw = s["d_topk_w"]
    if s["renorm"]:
        w = torch.where(pick, p[:, None, :], torch.zeros_like(p)[:, None, :]).sum(2)
        w = w / w.sum(1, keepdim=True)
        part = w * (dw - (dw * w).sum(1, keepdim=True))
        grad = (pick.float() * part[:, :, None]).sum(1)
    else:
        up = (pick.float() * dw[:, :, None]).sum(1)
        grad = p * (up - (up * p).sum(1, keepdim=True))
    tokens = s["tokens"][:-1].float().clamp_min(1.0)
    some = s["tokens"][-1].float().clamp_min(1.0)
    load = s["counts"].float() / (tokens[:, None] * k)
    coef = s["d_loss"] * s["alpha"] * E / (some * tokens)
    F = m.float() @ (coef[:, None] * load)
    grad = grad + p * (F - (F * p).sum(1, keepdim=True))
    return torch.where(valid[:, None], grad, torch.zeros_like(grad))


def _hot(s):
    return (s["adapter"][:, None] == torch.arange(s["n"], device=DEV)).float()


def _shrink(s, x, A):
    """[T][r]: every row's product with its own adapter's factor, scaled."""
    n, r = s["n"], s["r"]
    every = (x @ A.reshape(n * r, -1).t()).reshape(-1, n, r)
    return (every * (_hot(s) * s["scale"])[:, :, None]).sum(1)


def _spread(s, v):
    """[T][n r]: a row's low-rank vector at its adapter's place, else zero."""
    return (_hot(s)[:, :, None] * v[:, None, :]).reshape(s["T"], -1)


def _lora(s):
    x = s["x"].float()
    v = _shrink(s, x, s["A"].float())
    y = x @ s["W"].float().t() + _spread(s, v) @ s["B"].float().reshape(s["n"] * s["r"], -1)
    return y.to(TYPES[s["out"]]), v


def _lora_backward(s):
    n, r = s["n"], s["r"]
    dy, x, A, B = s["dy"].float(), s["x"].float(), s["A"].float(), s["B"].float()
    u = _shrink(s, dy, B)
    spread = _spread(s, u)
    dx = dy @ s["W_t"].float().t() + spread @ A.reshape(n * r, -1)
    dA = (spread.t() @ x).reshape(n, r, -1)
    dB = (_spread(s, s["v"]).t() @ dy).reshape(n, r, -1)
    return dx.to(TYPES[s["dt"]]), dA, dB


def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"balance": _balance, "gate_backward": _gate_backward, "lora": _lora,
                "lora_backward": _lora_backward}[op](s)
    from grouped_gemm_router_amd import api
    if "ws" not in s:  # a program keeps the workspace of its sizes
        if op == "balance":
            size = api.moe_balance_loss_workspace_size(s["T"], s["E"], s["S"])
        elif op == "lora":
            size = api.moe_lora_linear_workspace_size(s["T"], s["N"], s["K"], s["r"], s["n"],
                                                      s["x"].dtype)
        elif op == "lora_backward":
            size = api.moe_lora_backward_workspace_size(s["T"], s["N"], s["K"], s["r"], s["n"],
                                                        s["x"].dtype)
        else:
            size = 0
        s["ws"] = torch.empty((max(size, 16),), dtype=torch.uint8, device=DEV)
    if op == "balance":
        api.moe_balance_loss(s["logits"], s["idx"], s["counts"], s["probs"], s["tokens"],
                             s["loss"], alpha=s["alpha"], seq_offsets=s["offsets"],
                             token_mask=s["mask"], ws=s["ws"])
        return s["counts"], s["probs"], s["tokens"], s["loss"]
    if op == "gate_backward":
        api.moe_route_backward(s["logits"], s["idx"], s["d_logits"], d_topk_w=s["d_topk_w"],
                               flags=api.MOE_ROUTE_RENORM if s["renorm"] else 0,
                               counts=s["counts"], tokens=s["tokens"], alpha=s["alpha"],
                               d_loss=s["d_loss"], seq_offsets=s["offsets"],
                               token_mask=s["mask"])
        return s["d_logits"]
    if op == "lora":
        api.moe_lora_linear(s["x"], s["A"], s["B"], s["scale"], s["adapter"], s["y"], s["v"],
                            W=s["W"], ws=s["ws"])
        return s["y"], s["v"]
    api.moe_lora_linear_backward(s["dy"], s["x"], s["A"], s["B"], s["scale"], s["adapter"],
                                 s["v"], s["u"], W_t=s["W_t"], dx=s["dx"], dA=s["dA"],
                                 dB=s["dB"], ws=s["ws"])
    return s["dx"], s["dA"], s["dB"]


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its value in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] in ("balance", "gate_backward"):
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        if c["op"] == "balance":
            return {"bytes": 4 * T * E + 4 * T * k + 8 * S * E + 4 * S + 8, "flops": 5 * T * E}
        return {"bytes": 8 * T * E + 8 * T * k + 4 * S * E, "flops": 10 * T * E}
    T, K, N, r = c["T"], c["K"], c["N"], c["r"]
    es = 2 if c["dt"] == "bf16" else 4
    n = min(c["n"], T)  # adapters that a row can ask for
    factors = n * r * (K + N)
    if c["op"] == "lora":
        ys = 2 if c["out"] == "bf16" else 4
        return {"bytes": es * (T * K + N * K + factors) + ys * T * N + 4 * T * r + 8 * T,
                "flops": 2 * T * N * K + 2 * T * r * (K + N)}
    return {"bytes": es * (2 * T * K + T * N + N * K + factors) + 4 * T * r + 8 * T
            + 4 * c["n"] * r * (K + N),
            "flops": 2 * T * N * K + 4 * T * r * (K + N)}


def _exact_routing(s):
    T, E, k, S = s["T"], s["E"], s["k"], s["S"]
    off = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    keep = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
    l64 = s["logits"].double()
    parts = []
    for b, e in zip(off[:-1], off[1:]):
        rows = b + torch.nonzero(keep[b:e]).flatten()
        l = l64[rows]
        p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
        cnt = torch.bincount(s["idx"][rows].flatten().long(), minlength=E)
        parts.append((rows, p, cnt))
    return parts


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "balance":
        parts = _exact_routing(s)
        S, E, k = s["S"], s["E"], s["k"]
        probs = torch.zeros((S, E), dtype=f64, device=DEV)
        loss = torch.zeros((), dtype=f64, device=DEV)
        some = sum(len(rows) > 0 for rows, _, _ in parts)
        for i, (rows, p, cnt) in enumerate(parts):
            if len(rows):
                probs[i] = p.mean(0)
                loss += s["alpha"] * E * (cnt.double() / (len(rows) * k) * probs[i]).sum() / some
        counts = torch.stack([c for _, _, c in parts]).to(torch.int32)
        tokens = torch.tensor([len(rows) for rows, _, _ in parts] + [some], dtype=torch.int32)
        return counts, probs, tokens.to(DEV), loss[None]
    if s["op"] == "gate_backward":
        parts = _exact_routing(s)
        E, k = s["E"], s["k"]
        out = torch.zeros((s["T"], E), dtype=f64, device=DEV)
        some = sum(len(rows) > 0 for rows, _, _ in parts)
        for rows, p, cnt in parts:
            if not len(rows):
                continue
            # d(loss)/dp, then through the softmax's Jacobian p_i (1[i=j] - p_j)
            idx, dw = s["idx"][rows].long(), s["d_topk_w"][rows].double()
            dp = torch.zeros_like(p)
            if s["renorm"]:
                sel = p.gather(1, idx)
                tot = sel.sum(1, keepdim=True)
                dsel = dw / tot - (dw * sel).sum(1, keepdim=True) / tot ** 2
                dp.scatter_add_(1, idx, dsel)
            else:
                dp.scatter_add_(1, idx, dw)
            n_s = len(rows)
            dp += s["d_loss"].double() * s["alpha"] * E * (cnt.double() / (n_s * k)) / (some * n_s)
            out[rows] = p * dp - p * (p * dp).sum(1, keepdim=True)
        return out
    T, n, r = s["T"], s["n"], s["r"]
    x = s["x"].double()
    if s["op"] == "lora":
        y = torch.matmul(x, s["W"].double().t())
        v = torch.zeros((T, r), dtype=f64, device=DEV)
        for a in range(n):
            rows = torch.nonzero(s["adapter"] == a).flatten()
            if len(rows):
                va = torch.matmul(x[rows], s["A"][a].double().t()) * s["scale"][a].double()
                v[rows] = va
                y[rows] += torch.matmul(va, s["B"][a].double())
        return y, v
    dy = s["dy"].double()
    dx = torch.matmul(dy, s["W_t"].double().t())
    dA = torch.zeros(s["dA"].shape, dtype=f64, device=DEV)
    dB = torch.zeros(s["dB"].shape, dtype=f64, device=DEV)
    for a in range(n):
        rows = torch.nonzero(s["adapter"] == a).flatten()
        if len(rows):
            ua = torch.matmul(dy[rows], s["B"][a].double().t()) * s["scale"][a].double()
            dx[rows] += torch.matmul(ua, s["A"][a].double())
            dA[a] = torch.matmul(ua.t(), x[rows])
            dB[a] = torch.matmul(s["v"][rows].double().t(), dy[rows])
    return dx, dA, dB
