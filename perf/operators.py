"""What the model-side operators are measured on: the embedding of tokens and
its gradient, the routing of tokens to experts and its gradient, and the gated
feed-forward block of the experts with its gradients.

Each case names one pass through one operator with its sizes.  The ranks are
the logical ranks of the library: rank r's buffers are row r of every tensor.
`run` computes a pass in elementary torch operations, or with `own` set
through the calls of the library; `exact` gives the same values in 64 bits.

Sizes come from this repository's own MoE workload (8 ranks, 4096 tokens,
top-8 of 64 experts) and its textbook napkin (width 2048), or are generic.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the lookup of one decoding step: 4 new tokens a rank, latency counts
        dict(name="lookup decode bf16", op="lookup", ranks=8, tokens=4, vocab=32000, width=2048, dtype="bf16"),
        # the lookup of one training step: a micro-batch of 4096 tokens a rank
        dict(name="lookup train f32", op="lookup", ranks=8, tokens=4096, vocab=32000, width=2048, dtype="f32"),
        # each rank's own gradient, a small model of odd sizes whose rows are not 16-byte aligned
        dict(name="lookup-grad odd f32", op="lookup_grad", ranks=3, tokens=1023, vocab=10007, width=515, dtype="f32"),
        # the table's gradient of a data-parallel step, summed over the ranks onto every rank
        dict(name="lookup-grad-sum train bf16", op="lookup_grad_sum", ranks=8, tokens=4096, vocab=32000, width=2048,
             dtype="bf16"),
        # routing of one decoding step
        dict(name="route decode f32", op="route", ranks=8, tokens=4, experts=64, topk=8, normalize=True, dtype="f32"),
        # routing of one training step of the MoE workload
        dict(name="route train bf16", op="route", ranks=8, tokens=4096, experts=64, topk=8, normalize=True,
             dtype="bf16"),
        # its gradient, weights taken from the softmax over all experts
        dict(name="route-grad train f32", op="route_grad", ranks=8, tokens=4096, experts=64, topk=8, normalize=False,
             dtype="f32"),
        # the experts of one decoding step: few rows an expert, the weights' bytes count
        dict(name="ffn decode bf16", op="ffn", ranks=8, tokens=4, experts=64, topk=8, width=2048, hidden=1024,
             factor=0, act="silu", dtype="bf16"),
        # the experts of one training step, keeping the pre-activations for the gradient
        dict(name="ffn train bf16", op="ffn", ranks=8, tokens=4096, experts=16, topk=2, width=2048, hidden=2048,
             factor=5, act="silu", dtype="bf16"),
        # a small float32 model of odd sizes, whose rows are not 16-byte aligned
        dict(name="ffn odd f32", op="ffn", ranks=2, tokens=333, experts=6, topk=2, width=515, hidden=331, factor=6,
             act="gelu", dtype="f32"),
        # the gradients of that training step
        dict(name="ffn-grad train bf16", op="ffn_grad", ranks=8, tokens=4096, experts=16, topk=2, width=2048,
             hidden=2048, factor=5, act="silu", dtype="bf16"),
        # the gradients of a float32 step with ragged rows
        dict(name="ffn-grad f32", op="ffn_grad", ranks=4, tokens=509, experts=8, topk=2, width=1024, hidden=1100,
             factor=5, act="gelu", dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi):
    """A row width: a multiple of 8 (16-byte rows in both types) three times in four, any number otherwise."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["lookup", "lookup_grad", "lookup_grad_sum", "route", "route_grad", "ffn", "ffn", "ffn_grad",
                     "ffn_grad"])
    c = dict(op=op, ranks=rng.choice([1, 2, 3, 4, 5, 8]), tokens=_log(rng, 1, 4096), dtype=rng.choice(["f32", "bf16"]))
    if op.startswith("lookup"):
        c.update(vocab=_log(rng, 50, 32000), width=_wide(rng, 16, 2048))
        return c
    per = _log(rng, 1, 16)
    while per * c["ranks"] > 64:
        per -= 1
    c["experts"] = max(per * c["ranks"], 1)
    c["topk"] = rng.randint(1, min(8, c["experts"]))
    if op.startswith("route"):
        c["normalize"] = rng.random() < 0.5
        return c
    # the products: at most 2 of the experts for each token, and a float32 pass of at most a sixteenth of the work
    c["topk"] = min(c["topk"], 2)
    c["factor"] = rng.choice([0, 4, 5, 6, 8])
    if c["factor"] == 0:
        c["tokens"] = min(c["tokens"], 512)
    c["act"] = rng.choice(["silu", "gelu"])
    big = 2048 if c["dtype"] == "bf16" else 768
    c.update(width=_wide(rng, 32, big), hidden=_wide(rng, 32, big))
    return c


# ------------------------------------------------------------------ what a pass cannot do without

def _shares(tokens, experts, topk):
    """Rows one source rank routes to the experts, most loaded first: shares of
    (e + 1)^-0.4, at most `tokens` each, tokens * topk in all."""
    w = np.arange(1, experts + 1, dtype=np.float64) ** -0.4
    left, out = tokens * topk, np.zeros(experts, dtype=np.int64)
    for e in range(experts):
        out[e] = min(tokens, left, int(math.ceil(left * w[e] / w[e:].sum())))
        left -= out[e]
    e = 0
    while left > 0:
        add = min(left, tokens - int(out[e]))
        out[e] += add
        left -= add
        e += 1
    return out


def _capacity(c):
    """Rows of one (source, expert) block: factor / 4 times the even share, or
    room for every row where nothing may be dropped (factor 0)."""
    if c["factor"] == 0:
        return max(c["tokens"], 1)
    return -(-c["tokens"] * c["topk"] * c["factor"] // (4 * c["experts"]))


def work(c):
    n, t, s = c["ranks"], c["tokens"], SIZE[c["dtype"]]
    if c["op"] == "lookup":
        rows = n * t * c["width"]
        return {"bytes": 2 * rows * s + 4 * n * t, "flops": rows}
    if c["op"] in ("lookup_grad", "lookup_grad_sum"):
        rows = n * t * c["width"]
        return {"bytes": rows * s + 4 * n * t + n * c["vocab"] * c["width"] * s, "flops": rows}
    if c["op"] == "route":
        e, k = c["experts"], c["topk"]
        return {"bytes": n * t * (e * s + 12 * k) + 4 * n * e, "flops": n * t * e * (3 + k)}
    if c["op"] == "route_grad":
        e, k = c["experts"], c["topk"]
        return {"bytes": n * t * (2 * e * s + 8 * k), "flops": n * t * e * 6}
    kept = np.minimum(_shares(t, c["experts"], c["topk"]), _capacity(c))
    rows, live = n * int(kept.sum()), int((kept > 0).sum())
    w, h, e = c["width"], c["hidden"], c["experts"]
    if c["op"] == "ffn":
        return {"bytes": s * (rows * (2 * w + 2 * h) + live * 3 * w * h), "flops": 6 * rows * w * h}
    return {"bytes": s * (rows * (3 * w + 2 * h) + (live + e) * 3 * w * h), "flops": 12 * rows * w * h}


# ------------------------------------------------------------------ inputs

def _randn(g, shape, dtype, sigma):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(sigma).to(TORCH[dtype])


def _plan(c, seed):
    """The exchange's plan: the counts of every (source, expert), the same
    experts popular on every source, and each expert's kept rows (their
    positions in its rank's buffer)."""
    n, e = c["ranks"], c["experts"]
    perm = np.random.default_rng([seed, 7]).permutation(e)
    share = _shares(c["tokens"], e, c["topk"])[np.argsort(perm)]
    cap, per = _capacity(c), e // n
    counts = [[int(v) for v in share] for _ in range(n)]
    rows = []
    for x in range(e):
        kept = min(counts[0][x], cap)
        at = (np.arange(n)[:, None] * per + x % per) * cap + np.arange(kept)[None, :]
        rows.append(torch.from_numpy(at.reshape(-1)).to(DEV))
    return counts, cap, rows


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)
    n, t, dt = c["ranks"], c["tokens"], c["dtype"]
    st = {"c": c}
    if own:
        from ring_allreduce_reduction_02_amd import ccgpu
        st["cc"] = ccgpu
    if c["op"].startswith("lookup"):
        v, w = c["vocab"], c["width"]
        # words by 1 / rank, as in text, and one position in 32 without a token (-1)
        u = torch.rand((n, t), generator=g, device=DEV, dtype=torch.float64)
        ids = torch.exp(u * math.log(v + 1.0)).to(torch.int32).sub_(1).clamp_(0, v - 1)
        ids[torch.rand((n, t), generator=g, device=DEV) < 1 / 32] = -1
        st["ids"] = ids
        if c["op"] == "lookup":
            st["table"] = _randn(g, (n, v * w), dt, 0.02)
            st["out"] = torch.empty((n, t * w), dtype=TORCH[dt], device=DEV)
            st["scale"] = math.sqrt(w)
        else:
            st["grad"] = _randn(g, (n, t * w), dt, 1e-2)
            st["dtable"] = torch.empty((n, v * w), dtype=TORCH[dt], device=DEV)
            st["scale"] = math.sqrt(w)
            if own:
                st["ws"] = st["cc"].make_embedding_grad_workspace(n, v, t, w, dt)
        return st
    e, k = c["experts"], c["topk"]
    if c["op"].startswith("route"):
        lg = torch.randn((n, t, e), generator=g, device=DEV) + torch.randn((1, 1, e), generator=g, device=DEV)
        lg[torch.rand((n, t, e), generator=g, device=DEV) < 1 / 64] = -math.inf      # experts a token may not use
        lg[torch.rand((n, t), generator=g, device=DEV) < 1 / 32] = -math.inf         # padding tokens
        st["logits"] = lg.to(TORCH[dt]).view(n, t * e)
        st["experts"] = torch.empty((n, t * k), dtype=torch.int32, device=DEV)
        if c["op"] == "route":
            st["weights"] = torch.empty((n, t * k), dtype=torch.float32, device=DEV)
            st["order"] = torch.empty((n, t * k), dtype=torch.int32, device=DEV)
            st["counts"] = torch.empty((n, e), dtype=torch.int32, device=DEV)
            if own:
                st["ws"] = st["cc"].make_moe_route_workspace(n, t, e, k)
        else:
            st["experts"].copy_(_route_plain(st)[0])
            st["dweights"] = torch.randn((n, t * k), generator=g, device=DEV)
            st["dlogits"] = torch.empty((n, t * e), dtype=TORCH[dt], device=DEV)
        return st
    w, h = c["width"], c["hidden"]
    per = e // n
    counts, cap, rows = _plan(c, seed)
    st.update(counts=counts, cap=cap, rows=rows)
    keep = torch.zeros((n, e * cap, 1), dtype=torch.bool, device=DEV)
    for x in range(e):
        keep[x // per, rows[x]] = True

    def side(width, sigma):                          # an expert-side buffer: zero rows behind the kept ones
        b = _randn(g, (n, e * cap, width), dt, sigma)
        b.masked_fill_(~keep, 0)
        return b.view(n, -1)
    st["x"] = side(w, 1.0)
    st["w_in"] = _randn(g, (n, per * 2 * h * w), dt, 1 / math.sqrt(w))
    st["w_out"] = _randn(g, (n, per * w * h), dt, 1 / math.sqrt(h))
    st["pre"] = torch.zeros((n, e * cap * 2 * h), dtype=TORCH[dt], device=DEV)
    if c["op"] == "ffn":
        st["y"] = torch.zeros((n, e * cap * w), dtype=TORCH[dt], device=DEV)
    else:
        st["dy"] = side(w, 1e-2)
        pre, xs, wi = st["pre"].view(n, e * cap, 2 * h), st["x"].view(n, e * cap, w), st["w_in"].view(e, 2 * h, w)
        for x in range(e):
            if len(rows[x]):
                pre[x // per, rows[x]] = (xs[x // per, rows[x]].float() @ wi[x].float().t()).to(TORCH[dt])
        st["dx"] = torch.zeros((n, e * cap * w), dtype=TORCH[dt], device=DEV)
        st["dw_in"] = torch.empty_like(st["w_in"])
        st["dw_out"] = torch.empty_like(st["w_out"])
    if own:
        st["ws"] = st["cc"].make_moe_ffn_workspace(counts, cap, w, h, dt, grad=c["op"] == "ffn_grad")
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return (_run_own if own else _PLAIN[st["c"]["op"]])(st)


def _run_own(st):
    c, cc = st["c"], st["cc"]
    op = c["op"]
    if op == "lookup":
        cc.embedding(st["table"], st["ids"], st["out"], c["width"], scale=st["scale"])
        return st["out"]
    if op == "lookup_grad":
        cc.embedding_grad(st["grad"], st["ids"], st["dtable"], c["width"], scale=st["scale"], workspace=st["ws"])
        return st["dtable"]
    if op == "lookup_grad_sum":
        cc.all_reduce_embedding_grad(st["grad"], st["ids"], st["dtable"], c["width"], scale=st["scale"],
                                     workspace=st["ws"])
        return st["dtable"]
    if op == "route":
        cc.moe_route(st["logits"], st["experts"], st["weights"], st["order"], st["counts"], c["topk"],
                     normalize=c["normalize"], workspace=st["ws"])
        return st["experts"], st["weights"], st["order"], st["counts"]
    if op == "route_grad":
        cc.moe_route_grad(st["logits"], st["experts"], st["dweights"], st["dlogits"], c["topk"],
                          normalize=c["normalize"])
        return st["dlogits"]
    if op == "ffn":
        cc.moe_ffn(st["x"], st["w_in"], st["w_out"], st["y"], st["counts"], st["cap"], c["width"], pre=st["pre"],
                   act=c["act"], workspace=st["ws"])
        return st["y"], st["pre"]
    cc.moe_ffn_grad(st["x"], st["w_in"], st["w_out"], st["pre"], st["dy"], st["dx"], st["dw_in"], st["dw_out"],
                    st["counts"], st["cap"], c["width"], act=c["act"], workspace=st["ws"])
    return st["dx"], st["dw_in"], st["dw_out"]


# ------------------------------------------------------------------ the plain forms

def _lookup_plain(st):
    c = st["c"]
    n, t, w, v = c["ranks"], c["tokens"], c["width"], c["vocab"]
    ids = st["ids"].long()
    r = torch.arange(n, device=ids.device)[:, None]
    rows = st["table"].view(n, v, w)[r, ids.clamp(min=0)].float() * st["scale"]
    return torch.where((ids >= 0)[:, :, None], rows, 0.0).to(TORCH[c["dtype"]]).view(n, t * w)


def _lookup_grad_plain(st):
    c = st["c"]
    n, t, w, v = c["ranks"], c["tokens"], c["width"], c["vocab"]
    ids = st["ids"].long()
    into = torch.where(ids >= 0, torch.arange(n, device=ids.device)[:, None] * v + ids, n * v).view(-1)
    d = torch.zeros((n * v + 1, w), dtype=torch.float32, device=ids.device)
    d.index_add_(0, into, st["grad"].view(n * t, w).float())
    return (d[:-1] * st["scale"]).to(TORCH[c["dtype"]]).view(n, v * w)


def _lookup_grad_sum_plain(st):
    c = st["c"]
    n, t, w, v = c["ranks"], c["tokens"], c["width"], c["vocab"]
    ids = st["ids"].long().view(-1)
    d = torch.zeros((v + 1, w), dtype=torch.float32, device=ids.device)
    d.index_add_(0, torch.where(ids >= 0, ids, v), st["grad"].view(n * t, w).float())
    return (d[:-1] * st["scale"]).to(TORCH[c["dtype"]]).view(1, v * w).repeat(n, 1)


def _masked_softmax(x, dim):
    top = x.amax(dim, keepdim=True)
    ex = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    s = ex.sum(dim, keepdim=True)
    return torch.where(s > 0, ex / s, 0.0)


def _route_plain(st):
    c = st["c"]
    n, t, e, k = c["ranks"], c["tokens"], c["experts"], c["topk"]
    x = st["logits"].view(n, t, e).float()
    val, idx = torch.sort(x, dim=-1, descending=True, stable=True)
    val, idx = val[..., :k], idx[..., :k]
    live = val > -math.inf
    p = _masked_softmax(val, -1) if c["normalize"] else torch.gather(_masked_softmax(x, -1), -1, idx)
    experts = torch.where(live, idx, -1).view(n, t * k)
    key = torch.where(experts >= 0, experts, e)
    order = torch.sort(key, dim=-1, stable=True)[1]
    counts = (experts[:, :, None] == torch.arange(e, device=x.device)).sum(1)
    rows = (experts >= 0).sum(1, keepdim=True)
    order = torch.where(torch.arange(t * k, device=x.device) < rows, order, -1)
    return experts.int(), torch.where(live, p, 0.0).view(n, t * k), order.int(), counts.int()


def _route_grad_plain(st):
    c = st["c"]
    n, t, e, k = c["ranks"], c["tokens"], c["experts"], c["topk"]
    x = st["logits"].view(n, t, e).float()
    idx = st["experts"].view(n, t, k).long()
    live = idx >= 0
    at = idx.clamp(min=0)
    dw = torch.where(live, st["dweights"].view(n, t, k), 0.0)
    if c["normalize"]:
        p = _masked_softmax(torch.where(live, torch.gather(x, -1, at), -math.inf), -1)
        d = torch.zeros_like(x)
        d.scatter_add_(-1, at, p * (dw - (p * dw).sum(-1, keepdim=True)))
    else:
        p = _masked_softmax(x, -1)
        up = torch.zeros_like(x)
        up.scatter_add_(-1, at, dw)
        d = p * (up - (p * up).sum(-1, keepdim=True))
    return d.to(TORCH[c["dtype"]]).view(n, t * e)


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _dact(g, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _ffn_plain(st, as_type=torch.float32):
    c = st["c"]
    n, e, w, h = c["ranks"], c["experts"], c["width"], c["hidden"]
    per, cap = e // n, st["cap"]
    out = TORCH[c["dtype"]] if as_type == torch.float32 else as_type
    x = st["x"].view(n, e * cap, w)
    y = torch.zeros((n, e * cap, w), dtype=out, device=x.device)
    pre = torch.zeros((n, e * cap, 2 * h), dtype=out, device=x.device)
    wi, wo = st["w_in"].view(e, 2 * h, w), st["w_out"].view(e, w, h)
    for i in range(e):
        j, rows = i // per, st["rows"][i]
        if not len(rows):
            continue
        gu = x[j, rows].to(as_type) @ wi[i].to(as_type).t()
        pre[j, rows] = gu.to(out)
        y[j, rows] = ((_act(gu[:, :h], c["act"]) * gu[:, h:]) @ wo[i].to(as_type).t()).to(out)
    return y.view(n, -1), pre.view(n, -1)


def _ffn_grad_plain(st):
    c = st["c"]
    n, e, w, h = c["ranks"], c["experts"], c["width"], c["hidden"]
    per, cap = e // n, st["cap"]
    x, dy, pre = (st[k].view(n, e * cap, -1) for k in ("x", "dy", "pre"))
    wi, wo = st["w_in"].view(e, 2 * h, w), st["w_out"].view(e, w, h)
    dx = torch.zeros_like(x)
    dwi, dwo = torch.zeros_like(wi), torch.zeros_like(wo)
    for i in range(e):
        j, rows = i // per, st["rows"][i]
        if not len(rows):
            continue
        xe, de, gu = x[j, rows].float(), dy[j, rows].float(), pre[j, rows].float()
        g, u = gu[:, :h], gu[:, h:]
        a = _act(g, c["act"])
        dh = de @ wo[i].float()
        dgu = torch.cat([dh * u * _dact(g, c["act"]), dh * a], 1)
        dwo[i] = (de.t() @ (a * u)).to(wo.dtype)
        dwi[i] = (dgu.t() @ xe).to(wi.dtype)
        dx[j, rows] = (dgu @ wi[i].float()).to(x.dtype)
    return dx.view(n, -1), dwi.view(n, -1), dwo.view(n, -1)


_PLAIN = {"lookup": _lookup_plain, "lookup_grad": _lookup_grad_plain, "lookup_grad_sum": _lookup_grad_sum_plain,
          "route": _route_plain, "route_grad": _route_grad_plain, "ffn": _ffn_plain, "ffn_grad": _ffn_grad_plain}


# ------------------------------------------------------------------ the definitions in 64 bits

def _softmax64(z):
    """Row softmax of a float64 array; a row of -inf gives zeros."""
    m = np.max(z, axis=-1, keepdims=True)
    ex = np.exp(z - np.where(np.isneginf(m), 0.0, m))
    s = np.sum(ex, axis=-1, keepdims=True)
    return np.divide(ex, s, out=np.zeros_like(ex), where=s > 0)


def _exact_lookup(st, c):
    n, t, w, v = c["ranks"], c["tokens"], c["width"], c["vocab"]
    out = torch.zeros((n, t, w), dtype=torch.float64, device=DEV)
    for r in range(n):
        ids = st["ids"][r].long()
        at = (ids >= 0).nonzero().view(-1)
        out[r, at] = torch.index_select(st["table"][r].view(v, w), 0, ids[at]).double() * st["scale"]
    return out.view(n, t * w)


def _exact_lookup_grad(st, c, summed):
    n, t, w, v = c["ranks"], c["tokens"], c["width"], c["vocab"]
    out = torch.zeros((n, v, w), dtype=torch.float64, device=DEV)
    for r in range(n):
        ids = st["ids"][r].long()
        at = (ids >= 0).nonzero().view(-1)
        out[0 if summed else r].index_add_(0, ids[at], st["grad"][r].view(t, w)[at].double())
    if summed:
        out[1:] = out[0]
    return out.mul_(st["scale"]).view(n, v * w)


def _exact_route(st, c):
    n, t, e, k = c["ranks"], c["tokens"], c["experts"], c["topk"]
    z = st["logits"].double().cpu().numpy().reshape(n * t, e)
    pick = np.argsort(-z, axis=-1, kind="stable")[:, :k]
    top = np.take_along_axis(z, pick, -1)
    dead = np.isneginf(top)
    wt = _softmax64(top) if c["normalize"] else np.take_along_axis(_softmax64(z), pick, -1)
    pick = np.where(dead, -1, pick).reshape(n, t * k)
    order, counts = np.full((n, t * k), -1, np.int32), np.zeros((n, e), np.int32)
    for r in range(n):
        at = np.flatnonzero(pick[r] >= 0)
        order[r, :len(at)] = at[np.argsort(pick[r, at], kind="stable")]
        counts[r] = np.bincount(pick[r, at], minlength=e)
    dev = [torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
           for a in (pick.astype(np.int32), np.where(dead, 0.0, wt).reshape(n, t * k), order, counts)]
    return tuple(dev)


def _exact_route_grad(st, c):
    n, t, e, k = c["ranks"], c["tokens"], c["experts"], c["topk"]
    z = st["logits"].double().cpu().numpy().reshape(n * t, e)
    pick = st["experts"].cpu().numpy().reshape(n * t, k)
    dw = st["dweights"].double().cpu().numpy().reshape(n * t, k)
    chosen, up = np.zeros((n * t, e), bool), np.zeros((n * t, e))
    row, slot = np.nonzero(pick >= 0)
    chosen[row, pick[row, slot]] = True
    up[row, pick[row, slot]] = dw[row, slot]
    p = _softmax64(np.where(chosen, z, -np.inf)) if c["normalize"] else _softmax64(z)
    d = p * (up - np.sum(p * up, axis=-1, keepdims=True))
    return torch.from_numpy(d.reshape(n, t * e)).to(DEV)


def _gate64(g, act):
    """The activation and its derivative at g, in float64."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
    return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def _exact_ffn(st, c):
    n, e, w, h, cap = c["ranks"], c["experts"], c["width"], c["hidden"], st["cap"]
    y = torch.zeros((n, e * cap, w), dtype=torch.float64, device=DEV)
    pre = torch.zeros((n, e * cap, 2 * h), dtype=torch.float64, device=DEV)
    for i in range(e):
        j, rows = i * n // e, st["rows"][i]
        if len(rows) == 0:
            continue
        xe = st["x"][j].view(e * cap, w).index_select(0, rows).double()
        gate, up = st["w_in"].view(e, 2, h, w)[i].double()
        g, u = torch.mm(xe, gate.t()), torch.mm(xe, up.t())
        pre[j, rows, :h], pre[j, rows, h:] = g, u
        y[j, rows] = torch.mm(_gate64(g, c["act"])[0] * u, st["w_out"].view(e, w, h)[i].double().t())
    return y.view(n, -1), pre.view(n, -1)


def _exact_ffn_grad(st, c):
    n, e, w, h, cap = c["ranks"], c["experts"], c["width"], c["hidden"], st["cap"]
    dx = torch.zeros((n, e * cap, w), dtype=torch.float64, device=DEV)
    dwi = torch.zeros((e, 2, h, w), dtype=torch.float64, device=DEV)
    dwo = torch.zeros((e, w, h), dtype=torch.float64, device=DEV)
    for i in range(e):
        j, rows = i * n // e, st["rows"][i]
        if len(rows) == 0:
            continue
        xe, de, gu = (st[k][j].view(e * cap, -1).index_select(0, rows).double() for k in ("x", "dy", "pre"))
        gate, up = st["w_in"].view(e, 2, h, w)[i].double()
        a, da = _gate64(gu[:, :h], c["act"])
        u = gu[:, h:]
        dh = torch.mm(de, st["w_out"].view(e, w, h)[i].double())
        dg, du = dh * u * da, dh * a
        dwo[i] = torch.mm(de.t(), a * u)
        dwi[i, 0], dwi[i, 1] = torch.mm(dg.t(), xe), torch.mm(du.t(), xe)
        dx[j, rows] = torch.mm(dg, gate) + torch.mm(du, up)
    return dx.view(n, -1), dwi.view(n, -1), dwo.view(n, -1)


def exact(c, seed):
    st = prepare(c, seed)
    op = c["op"]
    if op == "lookup":
        return _exact_lookup(st, c)
    if op in ("lookup_grad", "lookup_grad_sum"):
        return _exact_lookup_grad(st, c, op == "lookup_grad_sum")
    if op == "route":
        return _exact_route(st, c)
    if op == "route_grad":
        return _exact_route_grad(st, c)
    return _exact_ffn(st, c) if op == "ffn" else _exact_ffn_grad(st, c)
