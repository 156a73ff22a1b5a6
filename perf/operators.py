"""Operators of a mixture of gated feed-forward experts and of 8-bit products:
what they compute, in plain torch, and the calls a user makes for the same.

  route   router logits -> top-k experts and weights of each token, tokens per
          expert, the balance loss, the expert-ordered list of the
          assignments; its gradient
  linear  activations quantised for each token, times 8-bit weights with a
          scale for each output channel
  gate    the same product as the gate projection, ReLU, packed into TwELL
  ffn     the gated feed-forward block on 8-bit weights, of one expert or of
          the experts that a route chose

8-bit rows: scale = max|row| / 127, q = rint(row * (127 / max|row|)), each of
these operations in 32 bits (round to nearest even); the products of the
integers and their sums are exact.  The ffn's hidden units are quantised in
groups of 128 per token; they are the 32-bit products ReLU(g) * u of
g = (sum * token scale) * channel scale and u alike, so that the integers are
part of the definition.
"""
import torch

own = False  # True: run() calls the framework's operators

GROUP = 128      # hidden units that share one activation scale in the ffn
TINY = 2.0 ** -100  # rows (groups) whose largest magnitude is below: taken as zeros

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one new token through the router of a many-expert layer: latency
        dict(name="route_token", op="route", n=1, e=64, k=8, dtype=F32, renorm=True, masked=False, train=False),
        # a prompt batch with padding tokens
        dict(name="route_prompt", op="route", n=8192, e=64, k=2, dtype=BF16, renorm=False, masked=True, train=False),
        # the training step's token count, few experts
        dict(name="route_train", op="route", n=8192, e=8, k=2, dtype=F32, renorm=True, masked=False, train=True),
        # a ragged training batch with padding, many experts
        dict(name="route_train_wide", op="route", n=16381, e=256, k=8, dtype=BF16, renorm=False, masked=True, train=True),
        # one token through a 1B projection
        dict(name="linear_token", op="linear", n=1, d=2048, m=8192, dtype=BF16),
        # nothing divides anything; 32-bit activations
        dict(name="linear_ragged", op="linear", n=777, d=1001, m=4099, dtype=F32),
        # the 2B shape, all tokens
        dict(name="linear_2b", op="linear", n=16384, d=2560, m=10240, dtype=BF16),
        # the gate projection of 64 decoded tokens and of the 1B forward
        dict(name="gate_decode", op="gate", n=64, d=2048, f=8192, tile=128, cap=128),
        dict(name="gate_1b", op="gate", n=8192, d=2048, f=8192, tile=128, cap=32),
        # a few decoded tokens over small experts; 32-bit activations
        dict(name="ffn_decode", op="ffn", n=4, d=1024, f=1024, e=32, k=4, dtype=F32),
        # the block without experts, the 1B shape
        dict(name="ffn_dense_1b", op="ffn", n=8192, d=2048, f=8192, e=1, k=1, dtype=BF16),
        # a prompt batch over experts, uneven loads
        dict(name="ffn_experts", op="ffn", n=8000, d=2048, f=2048, e=16, k=2, dtype=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "linear", "gate", "ffn"])
    if op == "route":
        e = _log(rng, 2, 256)
        return dict(op=op, n=_log(rng, 1, 16384), e=e, k=rng.randint(1, min(8, e)), dtype=rng.choice([BF16, F32]),
                    renorm=rng.random() < 0.5, masked=rng.random() < 0.5, train=rng.random() < 0.5)
    if op == "linear":
        return dict(op=op, n=_log(rng, 1, 16384), d=_log(rng, 64, 2560), m=_log(rng, 64, 10240),
                    dtype=rng.choice([BF16, F32]))
    if op == "gate":
        tile = rng.choice([32, 64, 128])
        return dict(op=op, n=_log(rng, 1, 8192), d=_log(rng, 128, 2560), f=128 * rng.randint(4, 64), tile=tile,
                    cap=rng.choice([tile // 4, tile // 2, tile]))
    e = rng.choice([1, 2, 5, 8, 16, 32])
    return dict(op=op, n=_log(rng, 1, 8192), d=8 * _log(rng, 16, 256), f=8 * _log(rng, 16, 256 if e > 1 else 1024),
                e=e, k=rng.randint(1, min(4, e)) if e > 1 else 1, dtype=rng.choice([BF16, F32]))


# ------------------------------------------------------------------ inputs


def _gen(case, seed):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, n, d, dtype, mean=0.0):
    """Activations: normal features, an uneven scale for each token."""
    x = _randn(g, n, d) + mean
    return (x * torch.exp(0.5 * _randn(g, n, 1))).to(dtype)


def _weights(g, rows, cols, std, mean=0.0):
    """8-bit weight rows (zero-padded to a multiple of 16 bytes) and scales,
    as a checkpoint of such a model holds them."""
    w = _randn(g, rows, cols) * std + mean
    amax = w.abs().amax(1)
    q = torch.round(w * (127.0 / amax)[:, None]).to(torch.int8)
    return torch.nn.functional.pad(q, (0, -cols % 16)), amax / 127.0


def _logits(g, n, e, dtype):
    """Some experts are liked better than others."""
    return (_randn(g, n, e) + 0.5 * _randn(g, 1, e)).to(dtype)


def prepare(case, seed):
    g = _gen(case, seed)
    op = case["op"]
    s = dict(case=case)
    if op == "route":
        n, e, k = case["n"], case["e"], case["k"]
        s["logits"] = _logits(g, n, e, DT[case["dtype"]])
        # padding tokens: not routed, whatever their logits hold
        s["mask"] = (torch.rand(n, generator=g, device="cuda") < 0.9).to(torch.uint8) if case["masked"] else None
        if case["train"]:
            s["dloss"] = torch.full((1,), 0.01, device="cuda")
            s["dw"] = _randn(g, n, k) / n
    elif op == "linear":
        s["x"] = _tokens(g, case["n"], case["d"], DT[case["dtype"]])
        s["wq"], s["sw"] = _weights(g, case["m"], case["d"], case["d"] ** -0.5)
    elif op == "gate":
        n, d, f, tile, cap = case["n"], case["d"], case["f"], case["tile"], case["cap"]
        # weights leaning against a common direction of the tokens: about 1% of the gates are open
        s["x"] = _tokens(g, n, d, torch.bfloat16, 0.5)
        s["wq"], s["sw"] = _weights(g, f, d, d ** -0.5, -5.2 / d)
        # the pack's buffers: slots past a tile's count are left as they were
        s["count"] = torch.zeros(n, f // tile, dtype=torch.uint8, device="cuda")
        s["idx"] = torch.zeros(n, f // tile, cap, dtype=torch.uint8, device="cuda")
        s["val"] = torch.zeros(n, f // tile, cap, dtype=torch.bfloat16, device="cuda")
    else:
        n, d, f, e, k = (case[key] for key in "ndfek")
        s["x"] = _tokens(g, n, d, DT[case["dtype"]])
        s["wg"], s["sg"] = _weights(g, e * f, d, d ** -0.5)
        s["wu"], s["su"] = _weights(g, e * f, d, d ** -0.5)
        s["wd"], s["sd"] = _weights(g, e * d, f, f ** -0.5)
        if e > 1:
            # the route that the layer's router gave for these tokens
            ids = torch.sort(_logits(g, n, e, torch.float32), dim=1, descending=True, stable=True)[1][:, :k]
            w = torch.rand(n, k, generator=g, device="cuda") + 0.1
            s["ids"], s["w"] = ids.to(torch.int32).contiguous(), (w / w.sum(1, keepdim=True)).contiguous()
            s["counts"], s["offsets"], s["pos"], s["order"] = _order(ids, e)
    return s


# ------------------------------------------------------------ plain forms


def _quant(x):
    """Rows of x (last dimension) as integers (in floats) and their scales."""
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    amax = torch.where(amax < TINY, 0.0, amax)
    top = torch.full_like(amax, 127.0)
    inv = torch.where(amax > 0, top / amax, 0.0)
    return torch.round(x * inv), amax / top


def _order(ids, e):
    """Tokens per expert, their prefix sums, and the assignments in expert
    order (token order within an expert): pos[n][j] is the place of token n's
    j-th assignment, order[] its inverse; -1 where there is none."""
    flat = ids.reshape(-1).long()
    there = flat >= 0
    key = torch.where(there, flat, e)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts[:e], 0)])
    order = torch.sort(key, stable=True)[1]
    pos = torch.empty_like(order).scatter_(0, order, torch.arange(len(order), device=ids.device))
    pos = torch.where(there, pos, -1).reshape(ids.shape)
    order = torch.where(torch.arange(len(order), device=ids.device) < offsets[e], order, -1)
    return (t.to(torch.int32).contiguous() for t in (counts[:e], offsets, pos, order))


def _route(logits, mask, k, renorm):
    n, e = logits.shape
    l = logits.float()
    live = torch.ones(n, dtype=torch.bool, device=l.device) if mask is None else mask != 0
    l = torch.where(live[:, None], l, -torch.inf)
    top = l.amax(1, keepdim=True)
    live = (top > -torch.inf).squeeze(1)
    p = torch.exp(l - torch.where(live[:, None], top, 0.0))
    p = torch.where(live[:, None], p / p.sum(1, keepdim=True), 0.0)
    v, ids = torch.sort(l, dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k]
    there = v > -torch.inf
    w = p.gather(1, ids)
    if renorm:
        ex = torch.exp(v - torch.where(live[:, None], top, 0.0))
        w = ex / ex.sum(1, keepdim=True)
    w = torch.where(there, w, 0.0)
    ids = torch.where(there, ids, -1)
    counts, offsets, pos, order = _order(ids, e)
    n_live = live.sum()
    f = counts.double() / counts.sum().clamp(min=1)  # sums over all tokens: in 64 bits
    mean = p.double().sum(0) / n_live.clamp(min=1)
    loss = (e * (f * mean).sum()).float().reshape(1)
    out = dict(ids=ids.to(torch.int32), w=w, counts=counts, offsets=offsets, pos=pos, order=order, loss=loss)
    return out, p, f, n_live


def _route_bwd(out, p, f, n_live, k, renorm, dloss, dw, dtype):
    n, e = p.shape
    there = out["ids"] >= 0
    at = out["ids"].long().clamp(min=0)
    dw = torch.where(there, dw, 0.0)
    dp = (dloss * e * f / n_live.clamp(min=1)).float().expand(n, e)
    if not renorm:
        dp = dp + torch.zeros_like(p).scatter_add_(1, at, dw)
    dl = p * (dp - (p * dp).sum(1, keepdim=True))
    if renorm:
        w = out["w"]
        dl = dl + torch.zeros_like(p).scatter_add_(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    return dl.to(dtype)


def _product(xq, wq):
    # 64 bits: sums of products of integers pass 2^24, and a gate that is next to zero or a
    # hidden unit next to a rounding border must not move
    return torch.matmul(xq.double(), wq.double().transpose(-1, -2)).float()


def _linear(x, wq, sw):
    q, sx = _quant(x)
    return (_product(q, wq[:, :x.shape[1]]) * sx * sw).to(x.dtype)


def _gate(x, wq, sw, tile, cap):
    n, f = x.shape[0], wq.shape[0]
    q, sx = _quant(x)
    gate = (_product(q, wq[:, :x.shape[1]]) * sx * sw).view(n, f // tile, tile)
    on = gate > 0
    col = torch.arange(tile, device=x.device).expand_as(gate)
    col = torch.sort(torch.where(on, col, tile).to(torch.uint8), dim=2)[0][..., :cap].long()
    stored = col < tile
    col = torch.where(stored, col, 0)
    val = torch.where(stored, gate.gather(2, col), 0.0).to(torch.bfloat16)
    return dict(count=on.sum(2).to(torch.uint8), idx=col.to(torch.uint8), val=val)


def _ffn(s):
    x, case = s["x"], s["case"]
    n, d, f, e, k = (case[key] for key in "ndfek")
    q, sx = _quant(x)
    wg, wu, wd = s["wg"].view(e, f, -1), s["wu"].view(e, f, -1), s["wd"].view(e, d, -1)
    sg, su, sd = s["sg"].view(e, 1, f), s["su"].view(e, 1, f), s["sd"].view(e, 1, d)
    if e > 1:
        # the assignments in expert order, padded to the longest list of an expert that has any
        used = torch.nonzero(s["counts"])[:, 0]
        wg, wu, wd, sg, su, sd = (t[used] for t in (wg, wu, wd, sg, su, sd))
        lens, first = s["counts"][used].long(), s["offsets"][used].long()
        slot = torch.arange(int(lens.max()), device=x.device)
        at = torch.where(slot < lens[:, None], first[:, None] + slot, 0)
        token = s["order"].long()[at] // k
        q, sx = q[token], sx[token]
    else:
        q, sx = q[None], sx[None]
    gate = _product(q, wg[..., :d]) * sx * sg
    up = _product(q, wu[..., :d]) * sx * su
    h = torch.clamp(gate, min=0) * up
    h = torch.nn.functional.pad(h, (0, -f % GROUP)).unflatten(2, (-1, GROUP))
    hq, sh = _quant(h)
    w = torch.nn.functional.pad(wd[..., :f], (0, -f % GROUP)).unflatten(2, (-1, GROUP))
    z = torch.matmul((hq * sh).flatten(2).double(), w.flatten(2).double().transpose(1, 2))
    z = z * sd
    if e == 1:
        return z[0].to(x.dtype)
    flat = torch.zeros(n * k, d, dtype=torch.float64, device=x.device)
    rows = s["order"].long()[at][slot < lens[:, None]]
    flat[rows] = z[slot < lens[:, None]]
    return (flat.view(n, k, d) * s["w"][..., None]).sum(1).to(x.dtype)


# -------------------------------------------------------------------- run


def _kept(s, key, make):
    """A buffer that a program keeps from call to call."""
    if key not in s:
        s[key] = make()
    return s[key]


def _run_own(s):
    import activation_sparse_gated_epilogue_b200 as sge

    case = s["case"]
    op = case["op"]
    dev = torch.device("cuda", torch.cuda.current_device())
    if op == "route":
        n, e, k = case["n"], case["e"], case["k"]
        out = _kept(s, "route", lambda: sge.MoeRoute.empty(n, e, k, dev))
        ws = _kept(s, "ws", lambda: sge.moe_route_workspace(n, e, k, dev))
        r = sge.moe_route_fwd(s["logits"], k, renorm=case["renorm"], mask=s["mask"], out=out, workspace=ws)
        got = dict(ids=r.ids, w=r.w, counts=r.counts, offsets=r.offsets, pos=r.pos, order=r.order, loss=r.loss)
        if case["train"]:
            got["dlogits"] = sge.moe_route_bwd(s["logits"], r, dloss=s["dloss"], dw=s["dw"], mask=s["mask"])
        return got
    if op == "linear":
        x = s["x"]
        q = sge.int8_quant_rows(x)
        return sge.int8_linear(q, sge.Int8Rows(s["wq"], s["sw"], case["d"]), x.dtype)
    if op == "gate":
        q = sge.int8_quant_rows(s["x"])
        tw = sge.TwELL(s["count"], s["idx"], s["val"], case["tile"], case["cap"])
        sge.twell_gate_pack_int8(q, sge.Int8Rows(s["wq"], s["sw"], case["d"]), case["tile"], case["cap"], out=tw)
        return dict(count=tw.count, idx=tw.idx, val=tw.val)
    n, d, f, e, k = (case[key] for key in "ndfek")
    wg, wu = sge.Int8Rows(s["wg"], s["sg"], d), sge.Int8Rows(s["wu"], s["su"], d)
    wd_t = sge.Int8Rows(s["wd"], s["sd"], f)
    ws = _kept(s, "ws", lambda: sge.int8_ffn_workspace(n, d, f, e, k, s["x"].dtype, dev))
    if e == 1:
        return sge.int8_ffn_fwd(s["x"], wg, wu, wd_t, workspace=ws)
    return sge.moe_int8_ffn_fwd(s["x"], wg, wu, wd_t, s["w"], s["offsets"], s["pos"], workspace=ws)


def run(state):
    if own:
        return _run_own(state)
    s, case = state, state["case"]
    op = case["op"]
    if op == "route":
        out, p, f, n_live = _route(s["logits"], s["mask"], case["k"], case["renorm"])
        if case["train"]:
            out["dlogits"] = _route_bwd(out, p, f, n_live, case["k"], case["renorm"], s["dloss"], s["dw"],
                                        s["logits"].dtype)
        return out
    if op == "linear":
        return _linear(s["x"], s["wq"], s["sw"])
    if op == "gate":
        return _gate(s["x"], s["wq"], s["sw"], case["tile"], case["cap"])
    return _ffn(s)


# ------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "route":
        n, e, k = case["n"], case["e"], case["k"]
        lb = 2 if case["dtype"] == BF16 else 4
        b = n * e * lb + (n if case["masked"] else 0) + n * k * 16 + (2 * e + 1) * 4 + 4
        fl = n * e * 8
        if case["train"]:
            b += n * e * lb + n * k * 4  # the gradient out, dw in
            fl += n * e * 8
        return dict(bytes=b, flops=fl)
    if op == "linear":
        n, d, m = case["n"], case["d"], case["m"]
        xb = 2 if case["dtype"] == BF16 else 4
        return dict(bytes=n * d * xb + m * d + 4 * m + n * m * xb, flops=2 * n * d * m)
    if op == "gate":
        n, d, f = case["n"], case["d"], case["f"]
        nt = f // case["tile"]
        stored = 0.01 * n * f  # about: what the tokens leave open
        return dict(bytes=n * d * 2 + f * d + 4 * f + n * nt + 3 * stored, flops=2 * n * d * f)
    n, d, f, e, k = (case[key] for key in "ndfek")
    xb = 2 if case["dtype"] == BF16 else 4
    used = e * (1 - (1 - k / e) ** n) if e > k else e  # experts that get a token, on average
    b = 2 * n * d * xb + used * (3 * d * f + 4 * (2 * f + d)) + (n * k * 8 + 4 * (e + 1) if e > 1 else 0)
    return dict(bytes=b, flops=6 * n * k * d * f)


# ------------------------------------------------------------------ exact


def _ints(x):
    """The 8-bit integers of rows of x: defined by these 32-bit operations."""
    a = x.float().abs().max(-1, keepdim=True).values
    q = (x.float() * (torch.tensor(127.0, device=x.device) / a)).round()
    zero = a < TINY
    return torch.where(zero, 0.0, q).double(), torch.where(zero, 0.0, a).double() / 127


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        l = s["logits"].double()
        if s["mask"] is not None:
            l = l.masked_fill((s["mask"] == 0)[:, None], float("nan"))
        live = ~torch.isnan(l[:, 0])
        rows = l[live].requires_grad_()
        n, e, k = len(rows), case["e"], case["k"]
        chosen = torch.argsort(-rows.detach(), dim=1, stable=True)[:, :k]
        lp = torch.log_softmax(rows, 1)
        w = lp.gather(1, chosen)
        w = torch.softmax(w, 1) if case["renorm"] else w.exp()
        hits = torch.nn.functional.one_hot(chosen, e).sum((0, 1)).double()
        loss = e * torch.dot(hits / max(1, n * k), lp.exp().sum(0) / max(1, n))
        full = torch.zeros(case["n"], k, dtype=torch.float64, device=l.device)
        full[live] = w.detach()
        got = dict(ids=None, w=full, counts=None, offsets=None, pos=None, order=None, loss=loss.detach().reshape(1))
        if case["train"]:
            (loss * s["dloss"].double().item() + (w * s["dw"].double()[live]).sum()).backward()
            dl = torch.zeros_like(l)
            dl[live] = rows.grad
            got["dlogits"] = dl
        return got
    q, sx = _ints(s["x"])
    if op in ("linear", "gate"):
        y = sx * (q @ (s["wq"][:, :case["d"]].double() * s["sw"].double()[:, None]).T)
        if op == "linear":
            return y
        tile, cap = case["tile"], case["cap"]
        y = y.clamp(min=0).view(len(y), -1, tile)
        place = torch.cumsum(y > 0, 2) - 1
        keep = (y > 0) & (place < cap)
        a, b, c = torch.nonzero(keep, as_tuple=True)
        val = torch.zeros(y.shape[0], y.shape[1], cap, dtype=torch.float64, device=y.device)
        val[a, b, place[a, b, c]] = y[a, b, c]
        return dict(count=None, idx=None, val=val)
    n, d, f, e, k = (case[key] for key in "ndfek")
    y = torch.zeros(n, d, dtype=torch.float64, device=q.device)
    for i in range(e):
        if e > 1:
            tok, j = torch.nonzero(s["ids"] == i, as_tuple=True)
            share = s["w"].double()[tok, j][:, None]
        else:
            tok, share = torch.arange(n, device=q.device), 1.0
        deq = lambda key, rows, cols: (s[key].view(e, rows, -1)[i, :, :cols].double()  # noqa: E731
                                       * s["s" + key[1]].double().view(e, rows, 1)[i])
        a, at = q[tok], sx[tok].float()
        g, u = (((a @ s[key].view(e, f, -1)[i, :, :d].double().T).float() * at) * s["s" + key[1]].view(e, f)[i]
                for key in ("wg", "wu"))
        h = torch.where(g > 0, g * u, 0.0)
        out, wd = 0.0, deq("wd", d, f)
        for c in range(0, f, GROUP):
            hq, sh = _ints(h[:, c:c + GROUP])
            out = out + (hq * sh) @ wd[:, c:c + GROUP].T
        y.index_add_(0, tok, out * share)
    return y
