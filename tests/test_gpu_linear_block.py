"""GPU test of the root-mean-square norm with 8-bit output, the 8-bit product and linear attention
together, as a block uses them: h = x + r, q, k, v of the projection of norm(h), out = h +
Wo . attention(q, k, v).  Its training step (operands in 8 bits in every product, gradients too)
against the same formulas in 64 bits on the very operands in 8 bits, and the serving of the same
block (a prompt, then tokens one by one) against the block over the whole sequence.

Tolerances.  The reference takes the 8-bit operands that the block made, so what is left are the
roundings to bf16 between the operators and fp32 sums: each bf16 tensor is off by 2^-8 of
its values, and no value passes more than eight of them, products adding up independent errors
as the square root of their number: 8 * 2^-8 of a result's largest value would be a bound with a
wide margin; 4 * 2^-8 of the largest value is asked.  Serving rounds the same values at the same places but
for the order of sums: a value of 8 bits next to a border may go to either side (a step of 2^-3 of
it), of 256 in a product, so the same limit holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, E4M3, E8M0 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu
TOL = 4 * 2.0 ** -8
S, T, D, H, K = 2, 200, 256, 2, 64          # sequences, tokens, width, heads, size of a head


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


def groups(n):
    return -(-n // 128)


def eight(rows, cols, square=False):
    return (torch.empty(rows, cols, dtype=E4M3, device="cuda"),
            torch.empty(groups(rows) if square else rows, groups(cols), dtype=E8M0, device="cuda"))


def values(q, s):
    s = s.double().repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.double() * s.repeat_interleave(1 if s.shape[0] == q.shape[0] else 128, 0)[:q.shape[0]]


def parameters(seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return {n: t.cuda() for n, t in {
        "x": rnd(S * T, D).to(BF), "r": (2 * rnd(S * T, D)).to(BF), "gamma": 1 + 0.1 * rnd(D),
        "Wi": (rnd(3 * H * K, D) * D ** -0.5).to(BF), "Wo": (rnd(D, H * K) * (H * K) ** -0.5).to(BF),
        "g": -torch.nn.functional.softplus(rnd(S * T, H) - 2), "dout": rnd(S * T, D).to(BF)}.items()}


class Block:
    """The block over the package's operators; ``rows`` tokens in ``sequences`` sequences."""

    def __init__(self, s4, w, sequences, rows, training=False):
        self.s4, self.w, self.rows, self.training = s4, w, rows, training
        self.plan = s4.LinearAttentionPlan(sequences, rows, H, H, K, K, BF, training=training)
        self.wi, self.wit = eight(3 * H * K, D, True), eight(D, 3 * H * K, True)
        self.wo, self.wot = eight(D, H * K, True), eight(H * K, D, True)
        s4.quantize_fp8(w["Wi"], *self.wi, *self.wit)
        s4.quantize_fp8(w["Wo"], *self.wo, *self.wot)

    def heads(self, z):
        return [z[:, i * H * K:(i + 1) * H * K].unflatten(1, (H, K)) for i in range(3)]

    def forward(self, x, r, g, state=None):
        s4, n, new = self.s4, self.rows, lambda *s: torch.empty(*s, dtype=BF, device="cuda")
        self.h, self.y, self.rstd = new(n, D), new(n, D), torch.empty(n, device="cuda")
        self.q8 = eight(n, D)
        s4.rms_norm_fwd(x, r, self.w["gamma"], self.h, self.y, self.rstd, *self.q8)
        self.z, self.o, out = new(n, 3 * H * K), new(n, H, K), new(n, D)
        s4.matmul_fp8(*self.q8, *self.wi, self.z)
        self.saved = self.plan.saved() if self.training else None
        s4.linear_attention_fwd(self.plan, *self.heads(self.z), g, state, self.o, state, self.plan.workspace(),
                                saved=self.saved)
        self.o8 = eight(n, H * K)
        s4.quantize_fp8(self.o.flatten(1), *self.o8)
        s4.matmul_fp8(*self.o8, *self.wo, out)
        return out + self.h

    def backward(self, g, dout):
        s4, n = self.s4, self.rows
        new = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.d8, self.d8t, ot = eight(n, D), eight(D, n), eight(H * K, n)
        s4.quantize_fp8(dout, *self.d8, *self.d8t)
        s4.quantize_fp8(self.o.flatten(1), None, None, *ot)
        self.do, dWo = new(n, H * K), f32(D, H * K)
        s4.matmul_fp8(*self.d8, *self.wot, self.do)
        s4.matmul_fp8(*self.d8t, *ot, dWo)
        dq, dk, dv, dg = new(n, H, K), new(n, H, K), new(n, H, K), f32(n, H)
        s4.linear_attention_bwd(self.plan, *self.heads(self.z), g, self.saved, self.do.unflatten(1, (H, K)), None,
                                dq, dk, dv, dg, None, self.plan.workspace())
        self.dz = torch.cat([t.flatten(1) for t in (dq, dk, dv)], 1)
        self.z8, self.z8t, yt = eight(n, 3 * H * K), eight(3 * H * K, n), eight(D, n)
        s4.quantize_fp8(self.dz, *self.z8, *self.z8t)
        s4.quantize_fp8(self.y, None, None, *yt)
        self.dy, dWi = new(n, D), f32(3 * H * K, D)
        s4.matmul_fp8(*self.z8, *self.wit, self.dy)
        s4.matmul_fp8(*self.z8t, *yt, dWi)
        dx, dgamma = new(n, D), f32(D)
        ws = torch.empty(s4.rms_norm_workspace_bytes(self.h), dtype=torch.uint8, device="cuda")
        s4.rms_norm_bwd(self.h, self.w["gamma"], self.rstd, self.dy, dout, dx, dgamma, ws)
        self.ot, self.yt = ot, yt
        return {"dx": dx, "dgamma": dgamma, "dWi": dWi, "dWo": dWo, "dg": dg}


def attention(q, k, v, g):
    """Linear attention by its definition over pairs, [T, H, K] in 64 bits."""
    G = g.cumsum(0)
    n = q.shape[0]
    low = torch.ones(n, n, device=q.device, dtype=torch.bool).tril()
    decay = torch.exp((G[:, None] - G[None]).masked_fill(~low[..., None], float("-inf")))
    p = (q[:, None] * k[None]).sum(-1) * decay * K ** -0.5
    return (p[..., None] * v[None]).sum(1)


def near(got, want, what):
    off = float((got.double() - want).abs().max() / want.abs().max())
    assert off <= TOL, f"{what}: {off:.1e}"


def test_training_step(s4):
    w = parameters(1)
    b = Block(s4, w, S, S * T, training=True)
    out = b.forward(w["x"], w["r"], w["g"])
    got = b.backward(w["g"], w["dout"])
    torch.cuda.synchronize()
    # 64 bits, from operator to operator; every product on the operands in 8 bits that the block took
    h = (w["x"].double() + w["r"].double()).to(BF).double()
    rstd = (h.square().mean(1, keepdim=True) + 1e-5) ** -0.5
    gamma = w["gamma"].double()
    y = h * rstd * gamma
    z = (values(*b.q8) @ values(*b.wi).T).requires_grad_()
    g = w["g"].double().requires_grad_()
    q, k, v = (t.unflatten(1, (H, K)) for t in z.split(H * K, 1))
    o = torch.cat([attention(*(t[i * T:(i + 1) * T] for t in (q, k, v, g))) for i in range(S)])
    near(b.z, z.detach(), "z")
    near(b.o, o.detach(), "o")
    near(out, h + values(*b.o8) @ values(*b.wo).T, "out")
    do = values(*b.d8) @ values(*b.wot).T
    near(b.do, do, "do")
    near(got["dWo"], values(*b.d8t) @ values(*b.ot).T, "dWo")
    dz, dg = torch.autograd.grad(o.flatten(1), (z, g), do)
    near(b.dz, dz, "dz")
    near(got["dg"], dg, "dg")
    near(got["dWi"], values(*b.z8t) @ values(*b.yt).T, "dWi")
    dy = values(*b.z8) @ values(*b.wit).T
    near(b.dy, dy, "dy")
    xh = h * rstd
    t = dy * gamma
    near(got["dx"], w["dout"].double() + rstd * (t - xh * (t * xh).mean(1, keepdim=True)), "dx")
    near(got["dgamma"], (dy * xh).sum(0), "dgamma")
    # the operands in 8 bits stand for what went into them: half a step, 2^-4, of each value or of the
    # least one under its scale
    for (q8, s8), what in ((b.q8, y), (b.wi, w["Wi"]), (b.wit, w["Wi"].T), (b.d8, w["dout"]), (b.z8, b.dz),
                           (b.z8t, b.dz.T), (b.ot, b.o.flatten(1).T)):
        what = what.double()
        assert bool(((values(q8, s8) - what).abs() <= 2.0 ** -4 * 1.001 * what.abs() + 2.0 ** -17 * what.abs().max()).all())


def test_prompt_then_tokens(s4):
    w = parameters(2)
    whole = Block(s4, w, S, S * T).forward(w["x"], w["r"], w["g"]).unflatten(0, (S, T))
    x, r, g = (w[n].unflatten(0, (S, T)) for n in ("x", "r", "g"))
    state, n = torch.zeros(S, H, K, K, device="cuda"), T - 6
    cut = lambda t, a, b: t[:, a:b].flatten(0, 1).contiguous()  # noqa: E731
    prompt = Block(s4, w, S, S * n).forward(*(cut(t, 0, n) for t in (x, r, g)), state)
    near(prompt.unflatten(0, (S, n)), whole[:, :n].double(), "prompt")
    step = Block(s4, w, S, S)
    for t in range(n, T):
        near(step.forward(*(cut(z, t, t + 1) for z in (x, r, g)), state), whole[:, t].double(), f"token {t}")
