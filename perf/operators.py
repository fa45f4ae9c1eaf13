"""The gated delta rule and the layer norm as measured workloads.

A case names an operator ("delta" or "norm"), a direction and sizes.  ``run``
computes it in plain torch operations, or, with ``own`` set, through the
package's entry points ``delta_fwd`` / ``delta_bwd`` and ``layer_norm_fwd`` /
``layer_norm_bwd``.  ``exact`` is the definition in 64 bits.
"""
import functools
import math

import torch

own = False

CHUNK = 64      # tokens per chunk of the plain chunked form
EPS = 1e-5


def _delta(name, sequences, tokens, Hk, Hv, dk, dv, dtype, state=True, ragged=False, train=False):
    c = {"op": "delta", "sequences": sequences, "tokens": tokens, "Hk": Hk, "Hv": Hv, "dk": dk,
         "dv": dv, "dtype": dtype, "state": state, "ragged": ragged, "train": train}
    return c if name is None else dict(c, name=name)


def _norm(name, outer, D, inner, dtype, train=False):
    c = {"op": "norm", "outer": outer, "D": D, "inner": inner, "dtype": dtype, "train": train}
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # one user's next token in a small layer: launch latency
        _delta("decode_one", 1, 1, 4, 4, 64, 64, "bfloat16"),
        # the next token of 128 users at once: the states' traffic
        _delta("decode_batch", 128, 128, 8, 16, 128, 128, "bfloat16"),
        # one long prompt: the chunks of a sequence follow one another
        _delta("prompt_long", 1, 16384, 8, 16, 128, 128, "bfloat16"),
        # prompts of mixed lengths in one packed batch, empty and one-token ones among them
        _delta("prompts_ragged", 13, 5003, 4, 8, 64, 128, "bfloat16", ragged=True),
        # single precision with odd head sizes
        _delta("prompt_single", 2, 1554, 3, 3, 40, 72, "float32", state=False),
        # a training step of a layer: forward, then all gradients
        _delta("train", 4, 16384, 16, 16, 128, 128, "bfloat16", state=False, train=True),
        # a small training step in single precision, grouped heads, carried state
        _delta("train_single", 3, 1500, 2, 4, 64, 64, "float32", train=True),
        # the pre-norm of a decode step
        _norm("norm_decode", 16, 1024, 1, "bfloat16"),
        # the pre-norm of a long prompt
        _norm("norm_tokens", 16384, 4096, 1, "bfloat16"),
        # its gradients in training
        _norm("norm_train", 16384, 2048, 1, "bfloat16", train=True),
        # gradients at an odd width in single precision
        _norm("norm_train_odd", 3001, 1001, 1, "float32", train=True),
        # gradients over the channels of [batch, H, L] (the "mid" workload's sizes)
        _norm("norm_train_channels", 32, 256, 1024, "float32", train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.5:
        dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
        train = rng.random() < 0.4
        dk, dv = rng.choice([32, 64, 128, 128, 80]), rng.choice([32, 64, 128, 128, 56, 256])
        Hk = _log(rng, 1, 16)
        Hv = Hk * rng.choice([1, 1, 2])
        # as many tokens as the largest listed case of the kind affords
        top = (1 << 30) if dtype == "bfloat16" else (1 << 27)
        most = max(64, min(16384, top // (4 if train else 1) // (Hv * dk * dv)))
        if rng.random() < 0.3:                       # decode
            S = _log(rng, 1, min(160, most))
            return _delta(None, S, S, Hk, Hv, dk, dv, dtype)
        S = _log(rng, 1, 12)
        tokens = _log(rng, S, most)
        ragged = rng.random() < 0.5
        if not ragged:
            tokens = max(1, tokens // S) * S
        return _delta(None, S, tokens, Hk, Hv, dk, dv, dtype, state=rng.random() < 0.5,
                      ragged=ragged, train=train)
    train = rng.random() < 0.5
    dtype = rng.choice(["bfloat16", "float32", "float16"])
    if rng.random() < 0.3:
        outer, D, inner = _log(rng, 1, 32), _log(rng, 8, 512), _log(rng, 16, 1024)
    else:
        outer, D, inner = _log(rng, 1, 16384), _log(rng, 16, 8192), 1
        outer = max(1, min(outer, (1 << 26) // D // (2 if train else 1)))
    return _norm(None, outer, D, inner, dtype, train)


def _type(case):
    return getattr(torch, case["dtype"])


def _lengths(case, seed):
    """Sequence lengths of a packed batch: an empty one, a one-token one, the rest uneven."""
    S, tokens = case["sequences"], case["tokens"]
    if not case["ragged"]:
        return [tokens // S] * S
    gen = torch.Generator().manual_seed(seed * 7919 + 17)
    w = torch.rand(S, generator=gen, dtype=torch.float64) + 0.05
    n = (w / w.sum() * tokens).floor().to(torch.int64)
    if S >= 3:
        n[S // 2] = 0
        n[1] = 1
    n[0] += tokens - n.sum()
    return [int(x) for x in n]


def prepare(case, seed):
    dev, dt = "cuda", _type(case)
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    if case["op"] == "norm":
        o, D, i = case["outer"], case["D"], case["inner"]
        shape = (o, D) if i == 1 else (o, D, i)
        st = {"case": case, "axis": 1,
              "x": (0.3 + rnd(*shape) * (1.0 + rnd(o, *[1] * (len(shape) - 1)).abs())).to(dt),
              "gamma": 1.0 + 0.1 * rnd(D), "beta": 0.1 * rnd(D)}
        if case["train"]:
            # what the forward pass left: each normalized vector's mean and 1 / deviation
            x = st["x"].double()
            m = x.mean(1, keepdim=True)
            r = 1.0 / torch.sqrt((x - m).square().mean(1, keepdim=True) + EPS)
            st["mean"] = m.squeeze(1).float().contiguous()
            st["rstd"] = r.squeeze(1).float().contiguous()
            st["dy"] = rnd(*shape).to(dt)
        return st
    S, tokens, Hk, Hv, dk, dv = (case[k] for k in ("sequences", "tokens", "Hk", "Hv", "dk", "dv"))
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1)  # noqa: E731
    lengths = _lengths(case, seed)
    st = {"case": case, "longest": max(lengths), "scale": dk ** -0.5,
          "q": unit(rnd(tokens, Hk, dk)).to(dt), "k": unit(rnd(tokens, Hk, dk)).to(dt),
          "v": rnd(tokens, Hv, dv).to(dt),
          # log decays of heads with short and long memories; a write strength in (0, 1)
          "g": -torch.nn.functional.softplus(rnd(tokens, Hv) - 2.0)
               * torch.exp(0.7 * rnd(Hv)),
          "beta": torch.sigmoid(rnd(tokens, Hv)), "state": None, "offsets": None}
    if case["ragged"]:
        st["offsets"] = torch.tensor([0] + lengths, device=dev).cumsum(0).to(torch.int32)
    if case["state"]:
        st["state"] = rnd(S, Hv, dk, dv) * 0.2
    if case["train"]:
        st["do"] = rnd(tokens, Hv, dv).to(dt)
        st["dstate"] = rnd(S, Hv, dk, dv) * 0.2 if case["state"] else None
    return st


# ---------------------------------------------------------------- plain forms


def _norm_plain(st):
    x, gamma = st["x"].float(), st["gamma"]
    D = x.shape[1]
    wide = (1, D) + (1,) * (x.dim() - 2)
    g = gamma.view(wide)
    if not st["case"]["train"]:
        m = x.mean(1, keepdim=True)
        r = torch.rsqrt((x - m).square().mean(1, keepdim=True) + EPS)
        y = (x - m) * r * g + st["beta"].view(wide)
        return {"y": y.to(st["x"].dtype), "mean": m.squeeze(1), "rstd": r.squeeze(1)}
    m, r, dy = st["mean"].unsqueeze(1), st["rstd"].unsqueeze(1), st["dy"].float()
    xh = (x - m) * r
    w = dy * g
    dx = r * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    over = [0] + list(range(2, x.dim()))
    return {"dx": dx.to(st["x"].dtype), "dgamma": (dy * xh).sum(over), "dbeta": dy.sum(over)}


def _delta_plain(st, q, k, v, g, beta, state):
    """o and the last states by chunks of at most CHUNK tokens, all in 32 bits."""
    case = st["case"]
    S, Hk, Hv = case["sequences"], case["Hk"], case["Hv"]
    dev, dv = q.device, case["dv"]
    longest = st["longest"]
    C = max(1, min(CHUNK, longest))
    nc = max(1, -(-longest // C))
    # packed rows to [S, nc * C] with zeros behind each sequence's end
    t = torch.arange(nc * C, device=dev)
    if st["offsets"] is None:
        first = torch.arange(S, device=dev) * longest
        count = torch.full((S,), longest, device=dev)
    else:
        first, count = st["offsets"][:-1].long(), st["offsets"].diff().long()
    keep = t < count[:, None]
    at = torch.where(keep, first[:, None] + t, torch.zeros_like(t))
    rows = lambda x: (x.float()[at] * keep.view(*keep.shape, *[1] * (x.dim() - 1))  # noqa: E731
                      ).unflatten(1, (nc, C)).movedim(3, 1)
    heads = lambda x: rows(x).repeat_interleave(Hv // Hk, 1)  # noqa: E731
    Q, K, V = heads(q), heads(k), rows(v)              # [S, Hv, nc, C, d]
    w, G = rows(beta), rows(g).double().cumsum(-1)
    low = torch.ones(C, C, device=dev, dtype=torch.bool).tril()
    gam = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).float()
    e, d = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    Kt = K.transpose(-1, -2).contiguous()
    H = ((K @ Kt) * gam).tril(-1) * w[..., None, :]
    P = (Q @ Kt) * gam * st["scale"]
    # (I + H)^-1 by doubling diagonal blocks: [A 0; B D]^-1 = [A^-1 0; -D^-1 B A^-1 D^-1]
    X, i, b = torch.eye(C, device=dev), torch.arange(C, device=dev), 1
    while b < C:
        below = (i[:, None] // b % 2 == 1) & (i[None, :] // b == i[:, None] // b - 1)
        X, b = X - X @ (H * below) @ X, 2 * b
    XV, XK = X @ V, X @ (e * K)
    w, Qe, last = w[..., None], Q * e * st["scale"], e[..., -1:, :]
    s = torch.zeros(S, Hv, case["dk"], dv, device=dev) if state is None else state
    out = []
    for c in range(nc):
        U = w[:, :, c] * (XV[:, :, c] - XK[:, :, c] @ s)
        out.append(Qe[:, :, c] @ s + P[:, :, c] @ U)
        s = last[:, :, c] * s + Kt[:, :, c] @ (d[:, :, c] * U)
    o = torch.stack(out, 2).movedim(1, 3).flatten(1, 2)  # [S, nc * C, Hv, dv]
    back = torch.zeros(q.shape[0], Hv, dv, device=dev)
    return back.index_put((at[keep],), o[keep]), s


def _delta_plain_run(st):
    names = ("q", "k", "v", "g", "beta")
    if not st["case"]["train"]:
        o, s = _delta_plain(st, *(st[n] for n in names), st["state"])
        return {"o": o.to(st["v"].dtype), "state": s}
    leaves = [st[n].float().requires_grad_() for n in names]
    if st["state"] is not None:
        leaves.append(st["state"].detach().requires_grad_())
    o, s = _delta_plain(st, *leaves[:5], leaves[5] if len(leaves) > 5 else None)
    outs, grads = [o], [st["do"].float()]
    if st["dstate"] is not None:
        outs, grads = [o, s], [grads[0], st["dstate"]]
    got = torch.autograd.grad(outs, leaves, grads)
    r = {"o": o.detach().to(st["v"].dtype), "state": s.detach()}
    for n, x in zip(names + ("state",), got):
        r["d" + n] = x.to(st[n].dtype)
    return r


# ------------------------------------------------------ the package's own calls


@functools.lru_cache(maxsize=1)
def _plan(S, tokens, Hk, Hv, dk, dv, dtype, train):
    """The layer's plan, its workspace and, in training, the buffer that the
    forward pass fills for the backward pass."""
    import structured_state_space_dplr_amd as s4
    p = s4.DeltaPlan(S, tokens, Hk, Hv, dk, dv, getattr(torch, dtype), training=train)
    return p, p.workspace(), p.saved() if train else None


def _delta_own(st):
    import structured_state_space_dplr_amd as s4
    c = st["case"]
    p, ws, saved = _plan(c["sequences"], c["tokens"], c["Hk"], c["Hv"], c["dk"], c["dv"],
                         c["dtype"], c["train"])
    q, k, v, g, beta = st["q"], st["k"], st["v"], st["g"], st["beta"]
    o = torch.empty_like(v)
    new = torch.empty(c["sequences"], c["Hv"], c["dk"], c["dv"], device=v.device)
    s4.delta_fwd(p, q, k, v, g, beta, st["state"], o, new, ws, saved=saved, scale=st["scale"],
                 offsets=st["offsets"])
    if not c["train"]:
        return {"o": o, "state": new}
    dq, dk, dv, dg, db = (torch.empty_like(x) for x in (q, k, v, g, beta))
    ds = None if st["state"] is None else torch.empty_like(new)
    s4.delta_bwd(p, q, k, v, g, beta, saved, st["do"], st["dstate"], dq, dk, dv, dg, db, ds, ws,
                 scale=st["scale"], offsets=st["offsets"])
    r = {"o": o, "state": new, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": db}
    return r if ds is None else dict(r, dstate=ds)


def _norm_own(st):
    import structured_state_space_dplr_amd as s4
    x, gamma = st["x"], st["gamma"]
    if not st["case"]["train"]:
        y = torch.empty_like(x)
        stat = (x.shape[0],) + x.shape[2:]
        mean, rstd = torch.empty(stat, device=x.device), torch.empty(stat, device=x.device)
        s4.layer_norm_fwd(x, gamma, st["beta"], y, mean, rstd, eps=EPS, axis=1)
        return {"y": y, "mean": mean, "rstd": rstd}
    ws = torch.empty(s4.layer_norm_workspace_bytes(x, axis=1), dtype=torch.uint8, device=x.device)
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    s4.layer_norm_bwd(x, gamma, st["mean"], st["rstd"], st["dy"], dx, dgamma, dbeta, ws, axis=1)
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def run(state):
    if state["case"]["op"] == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    return _delta_own(state) if own else _delta_plain_run(state)


# ------------------------------------------------------------------- accounting


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "norm":
        n, vec = case["outer"] * case["D"] * case["inner"], case["outer"] * case["inner"]
        if case["train"]:
            return {"bytes": 3 * n * size + 8 * vec + 12 * case["D"], "flops": 14 * n}
        return {"bytes": 2 * n * size + 8 * vec + 8 * case["D"], "flops": 8 * n}
    S, T, Hk, Hv, dk, dv = (case[k] for k in ("sequences", "tokens", "Hk", "Hv", "dk", "dv"))
    qk, vo, gb, st = 2 * T * Hk * dk * size, T * Hv * dv * size, 8 * T * Hv, 4 * S * Hv * dk * dv
    states = st * (2 if case["state"] else 1)
    # the recurrence token by token: decay, prediction, update and read of dk x dv values
    flops = 7 * T * Hv * dk * dv
    if not case["train"]:
        return {"bytes": qk + 2 * vo + gb + states, "flops": flops}
    # forward: q, k, v, o; backward: do read, dq, dk, dv written
    return {"bytes": 2 * qk + 4 * vo + 2 * gb + states * (2 if case["state"] else 1),
            "flops": 3 * flops}


# ------------------------------------------------------------ the definition, 64 bits


def _norm_exact(st):
    x, dims = st["x"].double(), None
    x = x.movedim(1, -1)
    gamma, beta = st["gamma"].double(), st["beta"].double()
    if not st["case"]["train"]:
        var, m = torch.var_mean(x, -1, correction=0, keepdim=True)
        r = (var + EPS) ** -0.5
        return {"y": ((x - m) * r * gamma + beta).movedim(-1, 1), "mean": m[..., 0], "rstd": r[..., 0]}
    m, r = st["mean"].double()[..., None], st["rstd"].double()[..., None]
    dy = st["dy"].double().movedim(1, -1)
    n = (x - m) * r
    a = (dy * gamma).sum(-1, keepdim=True)
    b = (dy * gamma * n).sum(-1, keepdim=True)
    dx = (dy * gamma - (a + n * b) / x.shape[-1]) * r
    dims = tuple(range(x.dim() - 1))
    return {"dx": dx.movedim(-1, 1), "dgamma": (dy * n).sum(dims), "dbeta": dy.sum(dims)}


def _delta_exact(st, seed):
    """The recurrence token by token, and its reverse from states kept every SPAN tokens."""
    case, SPAN = st["case"], 64
    S, T, Hk, Hv, dk, dv = (case[x] for x in ("sequences", "tokens", "Hk", "Hv", "dk", "dv"))
    dev, scale = st["q"].device, st["scale"]
    lengths = _lengths(case, seed)
    starts = [sum(lengths[:i]) for i in range(S)]
    longest = max(lengths)
    heads = torch.arange(Hv, device=dev) // (Hv // Hk)
    # time-major copies: [longest, S, ...]; a finished sequence sees g = 0, beta = 0, q = k = v = 0
    def major(x):
        z = torch.zeros((longest, S) + tuple(x.shape[1:]), dtype=torch.float64, device=dev)
        for s in range(S):
            z[:lengths[s], s] = x[starts[s]:starts[s] + lengths[s]].double()
        return z
    q, k = major(st["q"])[:, :, heads], major(st["k"])[:, :, heads]
    v, a, beta = major(st["v"]), major(st["g"]).exp(), major(st["beta"])
    s = torch.zeros(S, Hv, dk, dv, dtype=torch.float64, device=dev)
    if st["state"] is not None:
        s = st["state"].double().clone()

    def step(s, t):
        s = s * a[t][..., None, None]
        n = v[t] - (s * k[t][..., None]).sum(2)
        return s, n, torch.addcmul(s, k[t][..., None], (beta[t][..., None] * n)[:, :, None])

    o, kept = torch.zeros_like(v), {}
    for t in range(longest):
        if case["train"] and t % SPAN == 0:
            kept[t] = s
        _, _, s = step(s, t)
        o[t] = (s * q[t][..., None]).sum(2) * scale

    def packed(z):
        return torch.cat([z[:lengths[i], i] for i in range(S)], 0)

    r = {"o": packed(o), "state": s}
    if not case["train"]:
        return r
    do = major(st["do"])
    dq, dkey, dval = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(a), torch.zeros_like(beta)
    ds = torch.zeros_like(s) if st["dstate"] is None else st["dstate"].double().clone()
    for t0 in sorted(kept, reverse=True):
        line, s = [], kept[t0]
        for t in range(t0, min(t0 + SPAN, longest)):
            faded, n, s = step(s, t)
            line.append((faded, n, s))
        for t in range(min(t0 + SPAN, longest) - 1, t0 - 1, -1):
            faded, n, after = line[t - t0]
            dq[t] = (after * do[t][:, :, None]).sum(3) * scale
            ds = torch.addcmul(ds, q[t][..., None], do[t][:, :, None], value=scale)
            du = (ds * k[t][..., None]).sum(2)
            dn = du * beta[t][..., None]
            db[t] = (du * n).sum(-1)
            dval[t] = dn
            dkey[t] = (ds * (beta[t][..., None] * n)[:, :, None]).sum(3) - (faded * dn[:, :, None]).sum(3)
            ds = torch.addcmul(ds, k[t][..., None], dn[:, :, None], value=-1)
            dg[t] = (ds * faded).sum((2, 3))
            ds = ds * a[t][..., None, None]
    shared = lambda z: packed(z).unflatten(1, (Hk, Hv // Hk)).sum(2)  # noqa: E731
    r.update(dq=shared(dq), dk=shared(dkey), dv=packed(dval), dg=packed(dg), dbeta=packed(db))
    return r if st["state"] is None else dict(r, dstate=ds)


def exact(case, seed):
    st = prepare(case, seed)
    return _norm_exact(st) if case["op"] == "norm" else _delta_exact(st, seed)
