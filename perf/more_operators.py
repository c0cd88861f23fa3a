"""Cases that measure the backward pass of the expert layer and what ends a
training step.

Five operators, in the order in which a step runs them:

* ``combine_backward``: gradients of the gather and gate-weighted sum, for the
  expert outputs and the gate weights;
* ``dgrad``: the gradient of a grouped product's input, of one product, of the
  gate and up products together, or with SwiGLU's gradient behind it;
* ``wgrad``: the gradient of a grouped product's weights;
* ``permute_backward``: the gradient of the scatter into expert order;
* ``clip``: the global norm of many gradients, and their clipping.

``run`` computes them in plain torch operations, or through the framework's
entry points where ``own`` is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the small fp32 layer: nothing but latency
        dict(name="combine_backward_small", op="combine_backward", T=256, d=128, E=8, k=2,
             shared=0, dt="f32", rows="f32", capped=False),
        # the DeepSeek-shape layer's step
        dict(name="combine_backward_deepseek", op="combine_backward", T=4096, d=7168, E=256, k=8,
             shared=1, dt="bf16", rows="f32", capped=False),
        # the Mixtral-shape layer's step
        dict(name="permute_backward_mixtral", op="permute_backward", T=4096, d=4096, E=8, k=2,
             shared=0, dt="bf16", rows="f32", capped=False, addend=True),
        # an odd batch through capped experts: dropped entries, unused rows
        dict(name="permute_backward_capped", op="permute_backward", T=3001, d=2056, E=60, k=6,
             shared=2, dt="f32", rows="bf16", capped=True, addend=False),
        # the Mixtral-shape down projection and SwiGLU behind it
        dict(name="dgrad_swiglu_mixtral", op="dgrad", form="swiglu", rows=8192, G=8, N=4096,
             K=14336, dt="bf16", out="bf16", spare=0),
        # gate and up of fine-grained experts into one gradient, skewed and ragged
        dict(name="dgrad_pair_fine", op="dgrad", form="pair", rows=24571, G=64, N=2048, K=7168,
             dt="bf16", out="f32", spare=300),
        # the small fp32 layer's down projection
        dict(name="dgrad_f32", op="dgrad", form="one", rows=512, G=8, N=128, K=256, dt="f32",
             out="f32", spare=0),
        # the Mixtral-shape gate projection's weights
        dict(name="wgrad_mixtral", op="wgrad", rows=8192, G=8, N=14336, K=4096, dt="bf16",
             out="bf16", spare=0),
        # fine-grained experts of odd widths, gradients kept in fp32
        dict(name="wgrad_fine", op="wgrad", rows=24571, G=64, N=1416, K=2056, dt="bf16",
             out="f32", spare=300),
        # the small fp32 layer
        dict(name="wgrad_f32", op="wgrad", rows=512, G=8, N=256, K=128, dt="f32", out="f32",
             spare=0),
        # the factors of eight adapters in 48 layers, over the limit
        dict(name="clip_adapters", op="clip", kind="adapters", n=96, most=8 * 16 * 4096,
             dt="f32", over=True),
        # the Mixtral-shape layer's weights, under the limit: nothing to scale
        dict(name="clip_experts", op="clip", kind="experts", n=3, most=8 * 14336 * 4096,
             dt="bf16", over=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["combine_backward", "permute_backward", "dgrad", "dgrad", "wgrad", "wgrad",
                     "clip"])
    if op in ("combine_backward", "permute_backward"):
        E = _log(rng, 2, 256)
        k, shared = rng.randint(1, min(E, 10)), rng.choice([0, 0, 1, 2])
        d = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, max(1, min(8192, (1 << 28) // ((k + shared) * d))))
        c = dict(op=op, T=T, d=d, E=E, k=k, shared=shared, dt=rng.choice(["bf16", "bf16", "f32"]),
                 rows=rng.choice(["bf16", "f32"]), capped=rng.random() < 0.3)
        if op == "permute_backward":
            c["addend"] = rng.random() < 0.5
        return c
    if op == "clip":
        n = _log(rng, 1, 200)
        return dict(op=op, kind="ragged", n=n, most=_log(rng, 8, (1 << 28) // n),
                    dt=rng.choice(["f32", "bf16", "mixed"]), over=rng.random() < 0.7)
    dt = "f32" if rng.random() < 0.2 else "bf16"
    N, K = 8 * _log(rng, 4, 1024), 8 * _log(rng, 4, 1024)
    G = _log(rng, 1, max(1, min(256, (1 << 28) // (N * K))))
    room = (1 << 38) if dt == "bf16" else (1 << 32)
    c = dict(op=op, rows=_log(rng, 1, max(1, min(32768, room // (N * K)))), G=G, N=N, K=K, dt=dt,
             out="f32" if dt == "f32" else rng.choice(["bf16", "f32"]),
             spare=0)
    c["spare"] = rng.choice([0, 0, c["rows"] // 8])
    if op == "dgrad":
        c["form"] = rng.choice(["one", "pair", "swiglu"])
        if c["form"] == "swiglu":
            c["out"] = dt
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _sorted_rows(c, g):
    """flat_to_row [T k + shared T] of a routing with a skewed expert
    popularity: entries sorted by expert, those over an expert's capacity
    dropped (-1), then the shared experts' rows."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn((T, E), generator=g, device=DEV)
    logits -= 0.4 * torch.log1p(torch.randperm(E, generator=g, device=DEV).float())
    e = torch.topk(logits, k, dim=1).indices.reshape(-1)
    order = torch.argsort(e, stable=True)
    n = torch.bincount(e, minlength=E)
    rank = torch.arange(T * k, device=DEV) - (n.cumsum(0) - n)[e[order]]
    keep = rank < (-(-T * k // E) if c["capped"] else T)
    at = torch.where(keep, keep.cumsum(0) - 1, torch.full_like(rank, -1))
    row = torch.empty_like(at)
    row[order] = at
    shared = keep.sum() + torch.arange(c["shared"] * T, device=DEV)
    return torch.cat([row, shared]).to(torch.int32)


def _groups(c, g):
    """offsets [G+1] of groups of uneven sizes, some of them empty; the last
    `spare` rows belong to none."""
    G, rows = c["G"], max(0, c["rows"] - c["spare"])
    share = torch.exp(0.5 * torch.randn((G,), generator=g, device=DEV))
    if G > 2:
        share *= torch.rand((G,), generator=g, device=DEV) > 0.05
    share = share.double().clamp_min(1e-9).cumsum(0)
    cut = (share / share[-1] * rows).round().to(torch.int32)
    return torch.cat([cut.new_zeros(1), cut])


def _sizes(c):
    if c["kind"] == "adapters":
        return [c["most"]] * c["n"]
    if c["kind"] == "experts":
        return [c["most"]] * c["n"]
    r = random.Random(c["n"] * 1000003 + c["most"])
    return [_log(r, 1, c["most"]) for _ in range(c["n"])]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(shape, std, dtype):
        return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)

    if c["op"] == "clip":
        # gradients as views of one buffer for each type, one behind the other
        s = dict(c)
        sizes = _sizes(c)
        kinds = [c["dt"] if c["dt"] != "mixed" else ("f32", "bf16")[i % 2]
                 for i in range(len(sizes))]
        for t in ("f32", "bf16"):
            total = sum(n for n, k in zip(sizes, kinds) if k == t)
            s[t] = normal((total,), 1e-3, TYPES[t])
            s["clipped_" + t] = torch.empty_like(s[t]) if c["over"] else s[t]
        s["grads"], s["clipped"], at = [], [], {"f32": 0, "bf16": 0}
        for n, k in zip(sizes, kinds):
            s["grads"].append(s[k][at[k]:at[k] + n])
            s["clipped"].append(s["clipped_" + k][at[k]:at[k] + n])
            at[k] += n
        expected = 1e-3 * math.sqrt(sum(sizes))
        s["max_norm"] = expected / 3 if c["over"] else expected * 3 + 1e-2
        s["norm"] = torch.empty((1,), device=DEV)
        return s
    if c["op"] in ("combine_backward", "permute_backward"):
        T, d, k = c["T"], c["d"], c["k"]
        dt, rows = TYPES[c["dt"]], TYPES[c["rows"]]
        R = T * k + c["shared"] * T
        s = dict(c, R=R, flat_to_row=_sorted_rows(c, g))
        if c["op"] == "combine_backward":
            s["d_out"] = normal((T, d), 1e-3, dt)
            s["Y"] = normal((R, d), 1.0, rows)
            s["topk_w"] = torch.softmax(torch.randn((T, k), generator=g, device=DEV), 1)
            s["dY"] = torch.zeros((R, d), dtype=dt, device=DEV)
            s["d_topk_w"] = torch.empty((T, k), device=DEV)
        else:
            s["dx_perm"] = normal((R, d), 1e-3, rows)
            s["sum"] = normal((T, d), 1e-3, dt) if c["addend"] else None
            s["dx"] = torch.empty((T, d), dtype=dt, device=DEV)
        return s
    rows, G, N, K = c["rows"], c["G"], c["N"], c["K"]
    dt, out = TYPES[c["dt"]], TYPES[c["out"]]
    s = dict(c, offsets=_groups(c, g), dC=normal((rows, N), 1e-3, dt))
    s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
    if c["op"] == "wgrad":
        s["A"] = normal((rows, K), 1.0, dt)
        s["dB"] = torch.empty((G, N, K), dtype=out, device=DEV)
        return s
    s["B"] = normal((G, N, K), K ** -0.5, dt)
    s["dA"] = torch.zeros((rows, K), dtype=out, device=DEV)
    if c["form"] == "pair":
        s["dC2"] = normal((rows, N), 1e-3, dt)
        s["B2"] = normal((G, N, K), K ** -0.5, dt)
    if c["form"] == "swiglu":
        s["gate"], s["up"] = normal((rows, K), 1.0, dt), normal((rows, K), 1.0, dt)
        s["d_up"], s["h"] = torch.zeros_like(s["dA"]), torch.zeros_like(s["dA"])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _combine_backward(s):
    T, k, d, R = s["T"], s["k"], s["d"], s["R"]
    row = s["flat_to_row"][:T * k].long().reshape(T, k)
    at = torch.where(row >= 0, row, torch.full_like(row, R))  # one row more, for dropped entries
    grad = s["d_out"].float()
    dY = grad.new_zeros((R + 1, d))
    dY[at.reshape(-1)] = (s["topk_w"][:, :, None] * grad[:, None, :]).reshape(-1, d)
    shared = s["flat_to_row"][T * k:].long()
    dY[shared] = grad.repeat(s["shared"], 1)
    dw = (s["Y"].float()[row.clamp_min(0)] * grad[:, None, :]).sum(2)
    return dY[:R].to(s["dY"].dtype), torch.where(row >= 0, dw, torch.zeros_like(dw))


def _permute_backward(s):
    T, k, d = s["T"], s["k"], s["d"]
    row = s["flat_to_row"][:T * k].long().reshape(T, k)
    part = s["dx_perm"].float()[row.clamp_min(0)]
    dx = torch.where((row >= 0)[:, :, None], part, torch.zeros_like(part)).sum(1)
    if s["shared"]:
        shared = s["flat_to_row"][T * k:].long()
        dx = dx + s["dx_perm"].float()[shared].reshape(s["shared"], T, d).sum(0)
    if s["sum"] is not None:
        dx = dx + s["sum"].float()
    return dx.to(s["dx"].dtype)


def _places(s):
    """Group and place within it of every row; rows of no group get group G."""
    off = s["offsets"].long()
    r = torch.arange(s["rows"], device=DEV)
    grp = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return grp, (r - off[grp]).remainder(s["most"])


def _padded(s, x):
    """[G][most rows][columns] in fp32, zeros behind a group's rows."""
    grp, at = _places(s)
    p = x.new_zeros((s["G"] + 1, s["most"], x.shape[1]), dtype=torch.float32)
    p[grp, at] = x.float()
    return p[:s["G"]]


def _dgrad(s):
    grp, at = _places(s)
    live = (grp < s["G"])[:, None]
    dA = torch.matmul(_padded(s, s["dC"]), s["B"].float())
    if s["form"] == "pair":
        dA = dA + torch.matmul(_padded(s, s["dC2"]), s["B2"].float())
    dA = dA[grp.clamp_max(s["G"] - 1), at]
    dA = torch.where(live, dA, torch.zeros_like(dA))
    out = s["dA"].dtype
    if s["form"] != "swiglu":
        return dA.to(out)
    z, u = s["gate"].float(), s["up"].float()
    sig = 1 / (1 + torch.exp(-z))
    h = torch.where(live, z * sig * u, torch.zeros_like(dA))
    return (dA * u * sig * (1 + z * (1 - sig))).to(out), (dA * z * sig).to(out), h.to(out)


def _wgrad(s):
    dB = torch.matmul(_padded(s, s["dC"]).transpose(1, 2), _padded(s, s["A"]))
    return dB.to(s["dB"].dtype)


def _clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    scale = (s["max_norm"] / (norm + 1e-6)).clamp_max(1.0)
    [out.copy_(g.float() * scale) for g, out in zip(s["grads"], s["clipped"])]
    return norm[None], s["clipped_f32"], s["clipped_bf16"]


def _workspace(s, size):
    if "ws" not in s:  # a program keeps the workspace of its sizes
        s["ws"] = torch.empty((max(size, 16),), dtype=torch.uint8, device=DEV)
    return s["ws"]


def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"combine_backward": _combine_backward, "permute_backward": _permute_backward,
                "dgrad": _dgrad, "wgrad": _wgrad, "clip": _clip}[op](s)
    from grouped_gemm_router_amd import api
    if op == "combine_backward":
        api.moe_combine_backward(s["d_out"], s["Y"], s["flat_to_row"], s["topk_w"], s["dY"],
                                 s["d_topk_w"], n_shared=s["shared"])
        return s["dY"], s["d_topk_w"]
    if op == "permute_backward":
        api.moe_permute_backward(s["dx_perm"], s["flat_to_row"], s["dx"], s["k"],
                                 n_shared=s["shared"], addend=s["sum"])
        return s["dx"]
    if op == "dgrad":
        if "ws" not in s:
            _workspace(s, api.moe_grouped_gemm_dgrad_workspace_size(
                s["G"], s["rows"], s["N"], s["K"], s["dC"].dtype))
        if s["form"] == "swiglu":
            api.moe_grouped_gemm_dgrad_swiglu(s["dC"], s["B"], s["gate"], s["up"], s["dA"],
                                              s["d_up"], s["offsets"], h=s["h"], ws=s["ws"])
            return s["dA"], s["d_up"], s["h"]
        pair = s["form"] == "pair"
        api.moe_grouped_gemm_dgrad(s["dC"], s["B"], s["dA"], s["offsets"],
                                   dC2=s["dC2"] if pair else None, B2=s["B2"] if pair else None,
                                   ws=s["ws"])
        return s["dA"]
    if op == "wgrad":
        if "ws" not in s:
            _workspace(s, api.moe_grouped_gemm_wgrad_workspace_size(
                s["G"], s["rows"], s["N"], s["K"], s["dC"].dtype))
        api.moe_grouped_gemm_wgrad(s["dC"], s["A"], s["dB"], s["offsets"], ws=s["ws"])
        return s["dB"]
    if "ws" not in s:
        _workspace(s, api.moe_grad_norm_workspace_size(len(s["grads"])))
    api.moe_grad_norm(s["grads"], s["norm"], ws=s["ws"])
    api.moe_grad_clip(s["grads"], s["norm"], s["max_norm"], out=s["clipped"])
    return s["norm"], s["clipped_f32"], s["clipped_bf16"]


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its value in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "clip":
        sizes = _sizes(c)
        per = {"bf16": 2, "f32": 4, "mixed": 3}[c["dt"]]
        # over the limit, every gradient is read once and written once
        return {"bytes": per * sum(sizes) * (2 if c["over"] else 1) + 4, "flops": 3 * sum(sizes)}
    if c["op"] in ("combine_backward", "permute_backward"):
        T, d, k, ns = c["T"], c["d"], c["k"], c["shared"]
        es, rs, R = size[c["dt"]], size[c["rows"]], T * (k + ns)
        if c["op"] == "combine_backward":
            return {"bytes": es * T * d + rs * T * k * d + es * R * d + 4 * R + 8 * T * k,
                    "flops": 3 * T * k * d}
        return {"bytes": rs * R * d + es * T * d * (2 if c["addend"] else 1) + 4 * R,
                "flops": R * d}
    rows, G, N, K = max(0, c["rows"] - c["spare"]), c["G"], c["N"], c["K"]
    es, os = size[c["dt"]], size[c["out"]]
    flops = 2 * rows * N * K
    if c["op"] == "wgrad":
        return {"bytes": es * rows * (N + K) + os * G * N * K, "flops": flops}
    G = min(G, max(rows, 1))
    if c["form"] == "pair":
        return {"bytes": 2 * es * (rows * N + G * N * K) + os * rows * K, "flops": 2 * flops}
    if c["form"] == "swiglu":
        return {"bytes": es * (rows * N + G * N * K + 2 * rows * K) + 3 * os * rows * K,
                "flops": flops + 12 * rows * K}
    return {"bytes": es * (rows * N + G * N * K) + os * rows * K, "flops": flops}


def _d64(x):
    return x.to(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "clip":
        both = torch.cat([s["f32"].new_zeros(1, dtype=f64)] + [
            torch.linalg.vector_norm(s[t], dtype=f64)[None] for t in ("f32", "bf16")
            if s[t].numel()])
        norm = torch.linalg.vector_norm(both)
        scale = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        return norm[None], _d64(s["f32"]).mul_(scale), _d64(s["bf16"]).mul_(scale)
    if s["op"] == "combine_backward":
        T, k, d = s["T"], s["k"], s["d"]
        dY = torch.zeros((s["R"], d), dtype=f64, device=DEV)
        dw = torch.zeros((T, k), dtype=f64, device=DEV)
        grad = _d64(s["d_out"])
        for j in range(k):
            row = s["flat_to_row"][j:T * k:k].long()
            t = torch.nonzero(row >= 0).flatten()
            dY[row[t]] = grad[t] * _d64(s["topk_w"][t, j])[:, None]
            dw[t, j] = (_d64(s["Y"][row[t]]) * grad[t]).sum(1)
        for j in range(s["shared"]):
            dY[s["flat_to_row"][T * (k + j):T * (k + j + 1)].long()] = grad
        return dY, dw
    if s["op"] == "permute_backward":
        T, k, d = s["T"], s["k"], s["d"]
        dx = torch.zeros((T, d), dtype=f64, device=DEV)
        for j in range(k + s["shared"]):
            row = (s["flat_to_row"][j:T * k:k] if j < k
                   else s["flat_to_row"][T * j:T * (j + 1)]).long()
            t = torch.nonzero(row >= 0).flatten()
            dx[t] += _d64(s["dx_perm"][row[t]])
        return dx if s["sum"] is None else dx + _d64(s["sum"])
    off = s["offsets"].tolist()
    if s["op"] == "wgrad":
        dB = torch.zeros((s["G"], s["N"], s["K"]), dtype=f64, device=DEV)
        for i, (a, b) in enumerate(zip(off[:-1], off[1:])):
            dB[i] = torch.mm(_d64(s["dC"][a:b]).t(), _d64(s["A"][a:b]))
        return dB
    dA = torch.zeros((s["rows"], s["K"]), dtype=f64, device=DEV)
    for i, (a, b) in enumerate(zip(off[:-1], off[1:])):
        dA[a:b] = torch.mm(_d64(s["dC"][a:b]), _d64(s["B"][i]))
        if s["form"] == "pair":
            dA[a:b] += torch.mm(_d64(s["dC2"][a:b]), _d64(s["B2"][i]))
    if s["form"] != "swiglu":
        return dA
    z, u = _d64(s["gate"]), _d64(s["up"])
    silu = torch.nn.functional.silu(z)
    # the derivative through the quotient z / (1 + e^-z)
    e = torch.exp(-z)
    slope = (1 + e + z * e) / (1 + e) ** 2
    h = silu * u
    h[off[-1]:] = 0
    return dA * u * slope, dA * silu, h
