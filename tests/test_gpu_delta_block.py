"""GPU test of the layer norm and the gated delta rule together, as a block uses
them: x + Wo . delta(q, k, v of Wi . norm(x)), its training step against
reverse-mode gradients in 64 bits, and the serving of the same block (a prompt,
then tokens one by one) against the block over the whole sequence.

The projections are plain products in fp32.  Tolerances: every value passes at most
ten products of at most 256 terms, whose fp32 rounding errors add up as the square
root of their number (2^-24 sqrt(256) = 2^-20 of the largest value each); ten of
those, with a factor 4 for the largest of many values, are 2.5e-5 * 2 = 4e-5 of the
largest value of an output."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TOL = 4e-5
S, T, D, H, K, V = 2, 150, 96, 3, 32, 40      # sequences, tokens, width, heads, sizes


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


def parameters(seed, dtype, device):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    w = {"gamma": 1 + 0.1 * rnd(D), "beta": 0.1 * rnd(D),
         "Wi": rnd(D, H * (2 * K + V)) * D ** -0.5, "Wg": rnd(D, 2 * H) * D ** -0.5,
         "Wo": rnd(H * V, D) * (H * V) ** -0.5}
    x, dy = rnd(S * T, D), rnd(S * T, D)
    return {n: t.to(device=device, dtype=dtype) for n, t in {**w, "x": x, "dy": dy}.items()}


def split(z):
    q, k, v = z.split([H * K, H * K, H * V], -1)
    return q.unflatten(-1, (H, K)), k.unflatten(-1, (H, K)), v.unflatten(-1, (H, V))


def unit(t):
    return t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()


def gates(a):
    g, b = a.split(H, -1)
    return -torch.nn.functional.softplus(g - 1), torch.sigmoid(b)


def block_reference(w):
    """The block in 64 bits, token by token."""
    x = w["x"]
    m = x.mean(-1, keepdim=True)
    n = (x - m) * ((x - m).square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w["gamma"] + w["beta"]
    q, k, v = split(n @ w["Wi"])
    q, k = unit(q), unit(k)
    g, beta = gates(n @ w["Wg"])
    rows = []
    for s in range(S):
        st = torch.zeros(H, K, V, dtype=x.dtype)
        for t in range(s * T, s * T + T):
            st = st * g[t].exp()[:, None, None]
            e = v[t] - (st * k[t][:, :, None]).sum(1)
            st = st + k[t][:, :, None] * (beta[t][:, None] * e)[:, None, :]
            rows.append(K ** -0.5 * (st * q[t][:, :, None]).sum(1))
    return x + torch.stack(rows).flatten(1) @ w["Wo"]


def close(got, ref, name):
    err = float((got.double().cpu() - ref).abs().max() / ref.abs().max())
    assert err <= TOL, (name, err)


def test_training_step(s4):
    ref = {n: t.requires_grad_(n != "dy") for n, t in parameters(1, torch.float64, "cpu").items()}
    y = block_reference(ref)
    names = ["x", "gamma", "beta", "Wi", "Wg", "Wo"]
    want = dict(zip(names, torch.autograd.grad((y * ref["dy"]).sum(), [ref[n] for n in names])))

    w = parameters(1, torch.float32, "cuda")
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    plan = s4.DeltaPlan(S, S * T, H, H, K, V, torch.float32, training=True)
    ws, saved = plan.workspace(), plan.saved()
    # forward
    x, n, mean, rstd = w["x"], f(S * T, D), f(S * T), f(S * T)
    s4.layer_norm_fwd(x, w["gamma"], w["beta"], n, mean, rstd)
    z = (n @ w["Wi"]).requires_grad_()
    a = (n @ w["Wg"]).requires_grad_()
    zq, zk, zv = split(z)
    q, k = unit(zq), unit(zk)
    g, beta = gates(a)
    qd, kd, vd = q.detach().contiguous(), k.detach().contiguous(), zv.detach()   # v: a column range
    gd, bd = g.detach().contiguous(), beta.detach().contiguous()
    o = f(S * T, H, V)
    s4.delta_fwd(plan, qd, kd, vd, gd, bd, None, o, None, ws, saved=saved)
    out = x + o.flatten(1) @ w["Wo"]
    close(out, y.detach(), "out")
    # backward
    dy, got = w["dy"], {}
    got["Wo"] = o.flatten(1).t() @ dy
    do = (dy @ w["Wo"].t()).view(S * T, H, V)
    dq, dk, dv, dg, db = f(S * T, H, K), f(S * T, H, K), f(S * T, H, V), f(S * T, H), f(S * T, H)
    s4.delta_bwd(plan, qd, kd, vd, gd, bd, saved, do, None, dq, dk, dv, dg, db, None, ws)
    dz, da = torch.autograd.grad([q, k, zv, g, beta], [z, a], [dq, dk, dv, dg, db])
    got["Wi"], got["Wg"] = n.t() @ dz, n.t() @ da
    dn = dz @ w["Wi"].t() + da @ w["Wg"].t()
    dx, got["gamma"], got["beta"] = f(S * T, D), f(D), f(D)
    nws = torch.empty(s4.layer_norm_workspace_bytes(x), dtype=torch.uint8, device="cuda")
    s4.layer_norm_bwd(x, w["gamma"], mean, rstd, dn, dx, got["gamma"], got["beta"], nws)
    got["x"] = dx + dy
    for name in names:
        close(got[name], want[name], "d" + name)


def test_prompt_then_tokens(s4):
    ref = parameters(2, torch.float64, "cpu")
    y = block_reference(ref).view(S, T, D)
    w = parameters(2, torch.float32, "cuda")
    x = w["x"].view(S, T, D)
    state = torch.zeros(S, H, K, V, device="cuda")
    at = 0
    for n in (100, 1, 1, 1, 47):
        xs = x[:, at:at + n].reshape(S * n, D).contiguous()
        norm = torch.empty_like(xs)
        s4.layer_norm_fwd(xs, w["gamma"], w["beta"], norm)
        q, k, v = split(norm @ w["Wi"])
        g, beta = gates(norm @ w["Wg"])
        o = torch.empty(S * n, H, V, device="cuda")
        plan = s4.DeltaPlan(S, S * n, H, H, K, V, torch.float32)
        s4.delta_fwd(plan, unit(q), unit(k), v, g, beta, state, o, state, plan.workspace())
        out = (xs + o.flatten(1) @ w["Wo"]).view(S, n, D)
        close(out, y[:, at:at + n], f"tokens {at} ..")
        at += n
    assert at == T
