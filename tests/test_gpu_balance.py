"""GPU parity of moe_balance_loss and moe_route_backward against 64-bit
references, and the two together with the layer.

Tolerances from the fp32 arithmetic (u = 2^-24).  A softmax term errs by at
most (E + 60) u relative: the argument l - max (rounded once, its error times
the argument's size, at most 20 here, goes into the exponential), the
exponential (2 ulp), a normaliser summed over at most E positive terms, one
division.  probs adds one rounding per addition of positive terms: at most
128 + 16 tokens and waves inside a block, the blocks, and a division.  The loss
sums E S more positive terms.  counts and tokens are exact.
A gradient p (g - sum g p) errs by at most 3 (E + 60) u of p (|g| + sum |g| p):
the factor p, and the sum, each within (E + 60) u, and the roundings of g.
"""
import pytest
import torch

from grouped_gemm_router_amd import synth
from gpu_util import DEV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ALPHA = 0.02


def api():
    from grouped_gemm_router_amd import api as a
    return a


def make(T, E, k, seed, S=1, masked=False, behind=0, drop=False):
    """logits [T][E], idx [T][k], offsets (or None), mask (or None) on the CPU."""
    g = torch.Generator().manual_seed(seed)
    lg = 1.5 * torch.randn((T, E), generator=g)
    idx = torch.topk(lg, k, dim=1).indices.to(torch.int32).contiguous()
    if drop:  # entries outside [0, E) are dropped
        bad = torch.rand((T, k), generator=g) < 0.2
        idx = torch.where(bad, torch.randint(-3, 0, (T, k), generator=g, dtype=torch.int32), idx)
        idx[0, 0] = E
    off = mask = None
    if S > 1 or behind:
        cut = torch.randint(0, T - behind + 1, (S - 1,), generator=g).sort().values
        off = torch.cat([torch.zeros(1), cut, torch.tensor([T - behind])]).to(torch.int32)
    if masked:
        mask = torch.rand((T,), generator=g) < 0.8
        lg[~mask] = float("nan")
        if behind:
            lg[T - behind:] = float("inf")
    return lg, idx, off, mask


def members(T, off, mask):
    off = [0, T] if off is None else off.tolist()
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask
    return [b + torch.nonzero(keep[b:e]).flatten() for b, e in zip(off[:-1], off[1:])]


def softmax64(l):
    l = l.double()
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    z = e.sum(1, keepdim=True)
    return e / torch.where(z > 0, z, torch.ones_like(z))


def reference(lg, idx, off, mask, k):
    T, E = lg.shape
    parts = members(T, off, mask)
    some = sum(len(r) > 0 for r in parts)
    counts = torch.zeros((len(parts), E), dtype=torch.int64)
    probs = torch.zeros((len(parts), E), dtype=torch.float64)
    loss = 0.0
    for s, rows in enumerate(parts):
        if not len(rows):
            continue
        i = idx[rows].flatten().long()
        counts[s] = torch.bincount(i[(i >= 0) & (i < E)], minlength=E)
        probs[s] = softmax64(lg[rows]).mean(0)
        loss += E * float((counts[s].double() / (len(rows) * k) * probs[s]).sum())
    tokens = [len(r) for r in parts] + [some]
    return counts, probs, tokens, ALPHA * loss / max(some, 1)


def dev(t):
    return None if t is None else t.to(DEV)


def buffers(T, E, S):
    return (torch.full((S, E), -7, dtype=torch.int32, device=DEV),
            torch.full((S, E), float("nan"), device=DEV),
            torch.full((S + 1,), -7, dtype=torch.int32, device=DEV),
            torch.full((1,), float("nan"), device=DEV))


def run_loss(lg, idx, off, mask):
    T, E = lg.shape
    S = 1 if off is None else off.numel() - 1
    out = buffers(T, E, S)
    api().moe_balance_loss(dev(lg), dev(idx), *out, alpha=ALPHA, seq_offsets=dev(off),
                           token_mask=dev(mask))
    torch.cuda.synchronize()
    return [t.cpu() for t in out]


def check_loss(lg, idx, off, mask):
    T, E = lg.shape
    k = idx.shape[1]
    counts, probs, tokens, loss = run_loss(lg, idx, off, mask)
    rc, rp, rt, rl = reference(lg, idx, off, mask, k)
    assert torch.equal(counts.long(), rc)
    assert tokens.tolist() == rt
    tol = (E + 60 + 200 + T // 16) * U
    assert ((probs.double() - rp).abs() <= tol * rp + 1e-37).all()
    assert abs(float(loss) - rl) <= (tol + (E + len(rt) + 8) * U) * abs(rl) + 1e-37
    return counts, probs, tokens, loss


SHAPES = [  # every lane count and values-per-lane variant, odd and even E
    (1, 1, 1), (1, 8, 2), (2, 2, 1), (15, 3, 2), (16, 4, 4), (17, 8, 2), (256, 8, 2),
    (300, 12, 3), (513, 16, 4), (100, 31, 5), (129, 32, 8), (200, 60, 6), (65, 63, 4),
    (1000, 64, 6), (333, 100, 8), (70, 130, 7), (2049, 256, 8), (40, 255, 32), (90, 384, 10),
    (64, 500, 16), (33, 513, 3), (50, 1000, 32), (20, 1021, 9), (48, 1024, 32), (9001, 128, 4)]


@pytest.mark.parametrize("T,E,k", SHAPES)
def test_loss_of_one_sequence(T, E, k):
    print("balance loss", T, E, k, flush=True)
    check_loss(*make(T, E, k, T * 7 + E))


@pytest.mark.parametrize("T,E,k,S,masked,behind", [
    (1, 8, 2, 1, True, 0), (50, 8, 2, 50, False, 0), (777, 64, 6, 5, True, 13),
    (4096, 8, 2, 64, True, 100), (300, 256, 8, 300, True, 7), (5000, 17, 3, 9, False, 1),
    (20011, 256, 8, 16, True, 300), (64, 1024, 4, 3, True, 0), (40000, 9, 2, 1000, False, 0)])
def test_loss_of_sequences_and_padding(T, E, k, S, masked, behind):
    print("balance sequences", T, E, k, S, masked, behind, flush=True)
    lg, idx, off, mask = make(T, E, k, T + E + S, S=S, masked=masked, behind=behind)
    check_loss(lg, idx, off, mask)
    if S > 2:  # empty sequences at the ends and in the middle
        off = off.clone()
        off[1] = 0
        off[-2] = off[-1]
        check_loss(lg, idx, off, mask)


def test_loss_where_nothing_takes_part():
    lg, idx, _, _ = make(40, 8, 2, 3)
    mask = torch.zeros(40, dtype=torch.bool)
    lg[:] = float("nan")
    counts, probs, tokens, loss = check_loss(lg, idx, torch.tensor([0, 10, 40], dtype=torch.int32),
                                             mask)
    assert float(loss) == 0 and counts.sum() == 0 and probs.sum() == 0
    # every token behind the only, empty sequence
    counts, probs, tokens, loss = check_loss(lg, idx, torch.zeros(2, dtype=torch.int32), None)
    assert float(loss) == 0 and tokens.tolist() == [0, 0]


def test_empty_batch():
    for off in (None, torch.zeros(4, dtype=torch.int32)):
        lg, idx = torch.zeros((0, 8)), torch.zeros((0, 2), dtype=torch.int32)
        counts, probs, tokens, loss = run_loss(lg, idx, off, None)
        assert not counts.any() and not probs.any() and not tokens.any() and float(loss) == 0
        run_backward(lg, idx, torch.zeros((0, 2)), None, off, None, False, None, None)


def test_loss_of_dropped_entries_and_closed_experts():
    lg, idx, off, mask = make(700, 24, 4, 11, S=3, drop=True)
    lg[:, 5] = float("-inf")     # an expert of probability 0
    lg[17] = float("-inf")       # a row with no expert at all
    check_loss(lg, idx, off, mask)
    lg[:, :20] = -3e38           # masks of nearly the type's lowest value
    check_loss(lg, idx, off, mask)


def test_loss_matches_router_stats():
    a = api()
    T, E, k = 1000, 64, 6
    lg, idx, _, _ = make(T, E, k, 5)
    l, i = lg.to(DEV), idx.to(DEV)
    w = torch.empty((T, k), device=DEV)
    ps = torch.empty((a.prob_sum_blocks(T), E), device=DEV)
    sel = torch.empty_like(i)
    a.moe_route(None, None, sel, w, logits=l, flags=a.MOE_ROUTE_FROM_LOGITS, prob_sums=ps)
    counts, probs, tokens, loss = buffers(T, E, 1)
    a.moe_balance_loss(l, sel, counts, probs, tokens, loss, alpha=ALPHA)
    f, P, s = torch.empty(E, device=DEV), torch.empty(E, device=DEV), torch.empty(3, device=DEV)
    a.moe_router_stats(ps, counts.view(E), T, k, ALPHA, f, P, s)
    tol = 2 * (E + 260 + T // 16) * U
    assert (P - probs[0]).abs().max() <= tol * P.abs().max()
    assert abs(float(s[0] - loss)) <= (tol + 2 * E * U) * float(loss)


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def objective(l, idx, dw, dl, off, mask, renorm, counts, tokens):
    """sum dw . topk_w + dl . loss in 64 bits, f constant; l requires grad or not."""
    T, E = l.shape
    k = idx.shape[1]
    out = l.new_zeros(())
    for s, rows in enumerate(members(T, off, mask)):
        if not len(rows):
            continue
        p = torch.softmax(l[rows], 1)
        if dw is not None:
            ok = (idx[rows] >= 0) & (idx[rows] < E)
            at = torch.where(ok, idx[rows], torch.zeros_like(idx[rows])).long()
            w = torch.where(ok, p.gather(1, at), torch.zeros((), dtype=p.dtype))
            if renorm:
                z = w.sum(1, keepdim=True)
                w = w / torch.where(z > 0, z, torch.ones_like(z))
            out = out + (dw[rows].double() * w).sum()
        if counts is not None:
            f = counts[s].double() / (len(rows) * k)
            out = out + dl * ALPHA * E / tokens[-1] * (f * p.mean(0)).sum()
    return out


def run_backward(lg, idx, dw, dl, off, mask, renorm, counts, tokens):
    a = api()
    out = torch.full(lg.shape, float("nan"), device=DEV)
    a.moe_route_backward(dev(lg), dev(idx), out, d_topk_w=dev(dw),
                         flags=a.MOE_ROUTE_RENORM if renorm else 0, counts=dev(counts),
                         tokens=dev(tokens), alpha=ALPHA,
                         d_loss=None if dl is None else torch.tensor([dl], device=DEV),
                         seq_offsets=dev(off), token_mask=dev(mask))
    torch.cuda.synchronize()
    return out.cpu()


def check_backward(lg, idx, off, mask, renorm, gate=True, balance=True, seed=0):
    T, E = lg.shape
    k = idx.shape[1]
    g = torch.Generator().manual_seed(seed)
    dw = torch.randn((T, k), generator=g) / T if gate else None
    dl = 1.7 if balance else None
    counts = tokens = None
    if balance:
        c, _, t, _ = reference(lg, idx, off, mask, k)
        counts, tokens = c.to(torch.int32), torch.tensor(t, dtype=torch.int32)
    if dw is not None and mask is not None:
        dw[~mask] = float("nan")
    got = run_backward(lg, idx, dw, dl, off, mask, renorm, counts, tokens).double()
    parts = members(T, off, mask)
    on = torch.zeros(T, dtype=torch.bool)
    for rows in parts:
        on[rows] = True
    assert (got[~on] == 0).all()  # padding rows are written as zero
    l = torch.where(on[:, None], lg, torch.zeros_like(lg)).double().requires_grad_(True)
    objective(l, idx, dw, dl if balance else 0, off, mask, renorm, counts, tokens).backward()
    ref = l.grad
    # the bound: p (|g| + sum |g| p) for each term
    bound = torch.zeros((T, E), dtype=torch.float64)
    for s, rows in enumerate(parts):
        if not len(rows):
            continue
        p = torch.softmax(l.detach()[rows], 1)
        if gate:
            hot = torch.zeros((len(rows), E), dtype=torch.float64)
            ok = (idx[rows] >= 0) & (idx[rows] < E)
            at = torch.where(ok, idx[rows], torch.zeros_like(idx[rows])).long()
            hot.scatter_add_(1, at, torch.where(ok, dw[rows].double().abs(),
                                                torch.zeros((), dtype=torch.float64)))
            if renorm:
                sel = torch.zeros((len(rows), E), dtype=torch.float64).scatter_add_(
                    1, at, ok.double())
                q = p * (sel > 0)
                q = q / q.sum(1, keepdim=True).clamp_min(1e-300)
                bound[rows] += q * (hot + sel * (hot * q).sum(1, keepdim=True))
            else:
                bound[rows] += p * (hot + (hot * p).sum(1, keepdim=True))
        if balance:
            b = dl * ALPHA * E / max(int(tokens[-1]), 1) / len(rows) * (
                counts[s].double() / (len(rows) * k))
            bound[rows] += p * (b + (b * p).sum(1, keepdim=True))
    # The reference's own rounding: an expert that is not selected has a
    # renormalised gradient of exactly 0 in the formula, where the 64-bit
    # autograd cancels k terms of at most max |dw| (each within 2^-53 of
    # itself, and once more when they are summed).
    own = k * 2.0 ** -52 * float(dw[on].abs().max()) if gate and renorm and on.any() else 0.0
    assert ((got - ref).abs() <= 3 * (E + 60) * U * bound + own + 1e-40).all(), float(
        ((got - ref).abs() / (bound + own + 1e-40)).max() / U)
    return got


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gradient_of_one_sequence(T, E, k, renorm):
    print("route backward", T, E, k, renorm, flush=True)
    check_backward(*make(T, E, k, T * 5 + E), renorm)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k,S,masked,behind", [
    (1, 8, 2, 1, True, 0), (50, 8, 2, 50, False, 0), (777, 64, 6, 5, True, 13),
    (4096, 8, 2, 64, True, 100), (300, 256, 8, 300, True, 7), (5000, 17, 3, 9, False, 1),
    (64, 1024, 4, 3, True, 0)])
def test_gradient_of_sequences_and_padding(T, E, k, S, masked, behind, renorm):
    print("route backward sequences", T, E, k, S, masked, behind, renorm, flush=True)
    check_backward(*make(T, E, k, T + S, S=S, masked=masked, behind=behind), renorm)


@pytest.mark.parametrize("gate,balance,renorm", [(True, False, False), (True, False, True),
                                                 (False, True, False)])
def test_gradient_of_either_term(gate, balance, renorm):
    check_backward(*make(513, 40, 4, 2, S=4, masked=True, behind=9), renorm, gate, balance)


def test_gradient_of_dropped_and_repeated_entries():
    lg, idx, off, mask = make(400, 24, 4, 8, S=2, drop=True)
    for renorm in (False, True):
        check_backward(lg, idx, off, mask, renorm)
        twice = idx.clone()
        twice[:, 1] = twice[:, 2]  # the same expert twice in a token
        if not renorm:  # (the reference's renormalised form counts it twice as well)
            check_backward(lg, twice, off, mask, renorm)
    none = torch.full_like(idx, -1)  # a token with no expert: no gate gradient
    check_backward(lg, none, off, mask, True)


def test_gradient_against_differences():
    """Directional derivatives of the 64-bit objective: the central
    difference's truncation error is e^2 / 6 of a third derivative whose size
    the objective's own terms bound (softmax derivatives are at most a few
    units); e = 1e-3 leaves 1e-6 of sum |terms|, the fp32 gradient 1e-5."""
    for renorm in (False, True):
        lg, idx, off, mask = make(200, 20, 4, 6, S=3, masked=True, behind=5)
        got = check_backward(lg, idx, off, mask, renorm, seed=4)
        g = torch.Generator().manual_seed(4)
        dw = torch.randn((200, 4), generator=g) / 200
        c, _, t, _ = reference(lg, idx, off, mask, 4)
        l = torch.nan_to_num(lg.double(), nan=0.0, posinf=0.0)
        d = torch.randn((200, 20), generator=g, dtype=torch.float64)
        e = 1e-3
        f = lambda z: float(objective(z, idx, dw, 1.7, off, mask, renorm, c, torch.tensor(t)))  # noqa: E731
        slope = (f(l + e * d) - f(l - e * d)) / (2 * e)
        assert abs(slope - float((got * d).sum())) <= 1e-5 * float((got * d).abs().sum())


# ---------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------

def test_deterministic_other_stream_and_graph():
    """Twice the same bits; a side stream; a captured step replayed four
    times on new inputs with eager work in between."""
    a = api()
    T, E, k, S = 3000, 64, 6, 7
    sets = []
    for seed in range(5):
        lg, idx, off, mask = make(T, E, k, seed, S=S, masked=True, behind=40)
        sets.append((lg.to(DEV), idx.to(DEV), off.to(DEV), mask.to(DEV),
                     torch.randn((T, k), generator=torch.Generator().manual_seed(seed)).to(DEV)))
    st = [t.clone() for t in sets[0]]
    out = buffers(T, E, S)
    dlg = torch.empty((T, E), device=DEV)
    ws = torch.empty(a.moe_balance_loss_workspace_size(T, E, S), dtype=torch.uint8, device=DEV)

    def step(b, o, d, w):
        a.moe_balance_loss(b[0], b[1], *o, alpha=ALPHA, seq_offsets=b[2], token_mask=b[3], ws=w)
        a.moe_route_backward(b[0], b[1], d, d_topk_w=b[4], counts=o[0], tokens=o[2], alpha=ALPHA,
                             seq_offsets=b[2], token_mask=b[3])

    def eager(b):
        o, d, w = buffers(T, E, S), torch.empty((T, E), device=DEV), torch.empty_like(ws)
        step(b, o, d, w)
        torch.cuda.synchronize()
        return list(o) + [d]

    want = [eager(b) for b in sets]
    for x, y in zip(want[0], eager(sets[0])):
        assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(st, out, dlg, ws)
    side.synchronize()
    for x, y in zip(want[0], list(out) + [dlg]):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(st, out, dlg, ws)
    for i in (1, 2, 3, 4):
        for d, s in zip(st, sets[i]):
            d.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want[i], list(out) + [dlg]):
            assert torch.equal(x, y)
        eager(sets[0])


@pytest.mark.parametrize("renorm", [False, True])
def test_layer_balance_loss_and_route_backward(renorm):
    """The layer's own routing: loss, counts equal to the permutation's, and
    the logits' gradient against the 64-bit objective of its logits."""
    from grouped_gemm_router_amd.layer import MoELayer
    cfg = synth.scaled(synth.CONFIGS["deepseek_bf16"], name="small", T=300, d=256, dff=128, E=24,
                       k=4)
    wg, wu, wd = synth.gen_experts(cfg, DEV)
    layer = MoELayer(synth.gen_router(cfg, DEV), wg, wu, wd, cfg.k, n_shared=cfg.n_shared,
                     renorm=renorm)
    layer(synth.gen_x(cfg, DEV))
    bal = layer.balance_loss(alpha=ALPHA)
    assert torch.equal(bal["counts"][0], layer.counts)
    lg, idx = layer.logits.cpu(), layer.topk_idx.cpu()
    c, p, t, loss = reference(lg, idx, None, None, cfg.k)
    assert abs(float(bal["loss"]) - loss) <= (2 * cfg.E + 400) * U * loss
    dw = torch.randn((cfg.T, cfg.k), generator=torch.Generator().manual_seed(1))
    got = layer.route_backward(dw.to(DEV), balance=bal, alpha=ALPHA).cpu().double()
    l = lg.double().requires_grad_(True)
    objective(l, idx, dw, 1.0, None, None, renorm, c, torch.tensor(t)).backward()
    # every term is at most p (|g| + sum |g| p) <= 2 max |g|
    tol = 3 * (cfg.E + 60) * U * (2 * cfg.k * float(dw.abs().max()) + 2 * ALPHA * cfg.E / cfg.T)
    assert float((got - l.grad).abs().max()) <= tol


@pytest.mark.parametrize("E", [8, 100, 256])
def test_many_empty_sequences(E):
    """60000 sequences of which four have tokens: long runs of empty ones
    before, between and behind them."""
    T, S, k = 300, 60000, 4
    lg, idx, _, _ = make(T, E, k, E)
    off = torch.zeros(S + 1, dtype=torch.int32)
    for at, end in ((777, 1), (778, 130), (41000, 131), (59990, 290)):
        off[at + 1:] = end
    check_loss(lg, idx, off, None)
    check_backward(lg, idx, off, None, True)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(40, 8, 2), (70, 60, 6), (33, 256, 8), (50, 31, 5)])
def test_gradient_of_closed_experts(T, E, k, renorm):
    """Experts whose logit is -inf have probability and gradient 0, selected
    or not."""
    lg, idx, _, _ = make(T, E, k, 3 * T + E)
    lg[:, 1] = lg[::3, E - 1] = float("-inf")
    idx[::2, k - 1] = 1
    got = check_backward(lg, idx, None, None, renorm)
    assert (got[:, 1] == 0).all() and (got[::3, E - 1] == 0).all()
