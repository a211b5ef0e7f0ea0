"""Cases of the operators around a transformer's feed-forward block, with a plain form of each.

The operators, on matrices whose rows are tokens:

* ``epilogue``: y = act(a b + bias) + residual, one matrix product with what follows it
  (and z = a b + bias where the backward pass keeps it);
* ``epilogue_backward``: from dy, z, a and b, with dz = dy act'(z): da = dz b^T, db = a^T dz,
  dbias = the column sums of dz;
* ``gated``: h = act(x wg) * (x wu) (and the two products where the backward pass keeps them);
* ``gated_backward``: from dh and the kept g = x wg, u = x wu, with dg = dh u act'(g) and
  du = dh act(g): dx = dg wg^T + du wu^T, dwg = x^T dg, dwu = x^T du;
* ``norm``: y = (x - mean) rstd w + b over each row, with mean and rstd where they are kept;
* ``norm_backward``: dx, dw and db from dy, x, w and the kept mean and rstd.

Weights are stored as [outputs, inputs], as models keep them, and passed as the transposed
view. ``own`` chooses between the plain form (torch operations in 32 bits, rounded once at
the end) and the library's operators.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # one token of a generation step: the projection back onto the residual stream
        dict(name="epilogue_token", op="epilogue", dtype="bf16", tokens=1, k=4096, n=4096,
             act="none", bias=True, residual=True, keep=False),
        # odd sizes in 32 bits at full precision, as a small model's tests run
        dict(name="epilogue_odd_f32", op="epilogue", dtype="f32", tokens=1023, k=1000, n=1025,
             act="gelu", bias=True, residual=False, keep=True),
        # a long prompt or a training batch through the down projection
        dict(name="epilogue_batch", op="epilogue", dtype="bf16", tokens=8192, k=8192, n=2048,
             act="none", bias=True, residual=True, keep=False),
        # training: gradients of a hidden layer with its activation
        dict(name="epilogue_backward", op="epilogue_backward", dtype="bf16", tokens=4096, k=1024,
             n=4096, act="gelu_tanh", bias=True),
        # one token of a generation step through the gated half of the block
        dict(name="gated_token", op="gated", dtype="bf16", tokens=1, k=4096, n=8192, act="silu",
             keep=False),
        # a server's batch of single tokens
        dict(name="gated_decode_batch", op="gated", dtype="f16", tokens=64, k=2048, n=8192,
             act="silu", keep=False),
        # a training batch, keeping what the backward pass needs
        dict(name="gated_train", op="gated", dtype="bf16", tokens=8192, k=2048, n=8192,
             act="silu", keep=True),
        # its backward pass
        dict(name="gated_backward", op="gated_backward", dtype="bf16", tokens=8192, k=2048,
             n=8192, act="silu"),
        # one token's row
        dict(name="norm_token", op="norm", dtype="bf16", params="bf16", tokens=1, n=4096,
             keep=False),
        # a training batch's rows, keeping the statistics
        dict(name="norm_train", op="norm", dtype="bf16", params="f32", tokens=16384, n=4096,
             keep=True),
        # its backward pass
        dict(name="norm_backward", op="norm_backward", dtype="bf16", params="f32", tokens=16384,
             n=4096),
        # an odd width in 32 bits
        dict(name="norm_backward_odd_f32", op="norm_backward", dtype="f32", params="f32",
             tokens=1023, n=1025),
    ]


# The largest listed case's cost, which no drawn case passes.
MAX_FLOPS = 8.0 * 8192 * 2048 * 8192
MAX_BYTES = 6.0 * 16384 * 4096


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def width(rng, lo, hi):
    """A row width: mostly what models use (multiples of 64 or 8), some of any size."""
    n = log_uniform(rng, lo, hi)
    step = rng.choice((64, 64, 8, 8, 1))
    return max(step, n // step * step)


def draw(rng):
    while True:
        op = rng.choice(("epilogue", "epilogue_backward", "gated", "gated_backward", "norm",
                         "norm_backward"))
        case = dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
        if op.startswith("norm"):
            case.update(tokens=log_uniform(rng, 1, 16384), n=width(rng, 16, 16384))
            case["params"] = rng.choice(("f32", case["dtype"]))
            if op == "norm":
                case["keep"] = rng.random() < 0.5
        else:
            # generation steps and small batches as often as prompts and training batches
            lo = 64 if "backward" in op else 1
            case.update(tokens=log_uniform(rng, lo, 8192), k=width(rng, 64, 8192),
                        n=width(rng, 64, 8192))
            if op.startswith("gated"):
                case["act"] = rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"))
            else:
                case["act"] = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
                case["bias"] = rng.random() < 0.75
            if op == "epilogue":
                case["residual"] = rng.random() < 0.5
            if op in ("epilogue", "gated"):
                case["keep"] = case["tokens"] >= 64 and rng.random() < 0.5
        w = work(case)
        # matrix products in 32 bits cost several times those in 16 bits
        times = 3 if case["dtype"] == "f32" else 1
        if w["flops"] * times <= MAX_FLOPS and (not op.startswith("norm") or w["bytes"] <= MAX_BYTES):
            return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    t = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    op, m, n = case["op"], case["tokens"], case["n"]
    s = dict(case)
    if op.startswith("norm"):
        p = TYPES[case["params"]]
        # residual streams sit off centre and have a few columns far larger than the others
        x = torch.randn(m, n, generator=gen, device="cuda") + 0.25
        x[:, ::97] *= 8.0
        s["x"] = x.to(t)
        s["w"] = 1.0 + normal(n, scale=0.1, dtype=torch.float32)
        s["w"] = s["w"].to(p)
        s["b"] = normal(n, scale=0.1, dtype=p)
        if op == "norm_backward":
            xf = s["x"].float()
            mean = xf.mean(1)
            s["mean"] = mean
            s["rstd"] = ((xf - mean[:, None]).square().mean(1) + EPS).rsqrt()
            s["dy"] = normal(m, n, scale=0.5)
        return s
    k = case["k"]
    s["x"] = normal(m, k)
    if op.startswith("gated"):
        s["wg"] = normal(n, k, scale=1.0 / math.sqrt(k)).t()
        s["wu"] = normal(n, k, scale=1.0 / math.sqrt(k)).t()
        if op == "gated_backward":
            s["g"] = normal(m, n)
            s["u"] = normal(m, n)
            s["dh"] = normal(m, n, scale=0.5)
        return s
    s["w"] = normal(n, k, scale=1.0 / math.sqrt(k)).t()
    if op == "epilogue":
        s["bias_values"] = normal(n, scale=0.5) if case["bias"] else None
        s["residual_rows"] = normal(m, n) if case["residual"] else None
    else:
        s["dy"] = normal(m, n, scale=0.5)
        s["z"] = normal(m, n) if case["act"] != "none" else None
    return s


def sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z * sigmoid(z) if name == "silu" else sigmoid(z)


def act_slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        density = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * density
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * z * z)
    s = sigmoid(z)
    return s * (1.0 + z * (1.0 - s)) if name == "silu" else s * (1.0 - s)


def plain(s):
    op, t = s["op"], TYPES[s["dtype"]]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
        y = (d * rstd * s["w"].float() + s["b"].float()).to(t)
        return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0]) if s["keep"] else dict(y=y)
    if op == "norm_backward":
        p = TYPES[s["params"]]
        dy = s["dy"].float()
        r = s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * r
        v = dy * s["w"].float()
        dx = r * (v - v.mean(1, keepdim=True) - xhat * (v * xhat).mean(1, keepdim=True))
        return dict(dx=dx.to(t), dw=(dy * xhat).sum(0).to(p), db=dy.sum(0).to(p))
    x = s["x"].float()
    if op == "gated":
        g, u = x @ s["wg"].float(), x @ s["wu"].float()
        h = (act(g, s["act"]) * u).to(t)
        return dict(h=h, g=g.to(t), u=u.to(t)) if s["keep"] else dict(h=h)
    if op == "gated_backward":
        g, u, dh = s["g"].float(), s["u"].float(), s["dh"].float()
        dg, du = dh * u * act_slope(g, s["act"]), dh * act(g, s["act"])
        dx = dg @ s["wg"].float().t() + du @ s["wu"].float().t()
        return dict(dx=dx.to(t), dwg=(x.t() @ dg).to(t), dwu=(x.t() @ du).to(t))
    w = s["w"].float()
    if op == "epilogue":
        z = x @ w
        if s["bias_values"] is not None:
            z = z + s["bias_values"].float()
        y = act(z, s["act"])
        if s["residual_rows"] is not None:
            y = y + s["residual_rows"].float()
        return dict(y=y.to(t), z=z.to(t)) if s["keep"] else dict(y=y.to(t))
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * act_slope(s["z"].float(), s["act"])
    out = dict(da=(dz @ w.t()).to(t), dw=(x.t() @ dz).to(t))
    if s["bias"]:
        out["dbias"] = dz.sum(0).to(t)
    return out


def kernels(s):
    import dense_tiled_gemm_05_gb300 as lib
    op = s["op"]
    if op == "norm":
        if s["keep"]:
            y, mean, rstd = lib.layer_norm(s["x"], s["w"], s["b"], eps=EPS, save=True)
            return dict(y=y, mean=mean, rstd=rstd)
        return dict(y=lib.layer_norm(s["x"], s["w"], s["b"], eps=EPS))
    if op == "norm_backward":
        dx, dw, db = lib.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"])
        return dict(dx=dx, dw=dw, db=db)
    if op == "gated":
        if s["keep"]:
            h, g, u = lib.gated(s["x"], s["wg"], s["wu"], activation=s["act"], save=True)
            return dict(h=h, g=g, u=u)
        return dict(h=lib.gated(s["x"], s["wg"], s["wu"], activation=s["act"]))
    if op == "gated_backward":
        dx, dwg, dwu = lib.gated_backward(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"],
                                          activation=s["act"])
        return dict(dx=dx, dwg=dwg, dwu=dwu)
    if op == "epilogue":
        r = lib.matmul_epilogue(s["x"], s["w"], bias=s["bias_values"], activation=s["act"],
                                residual=s["residual_rows"], save=s["keep"])
        return dict(y=r[0], z=r[1]) if s["keep"] else dict(y=r)
    da, dw, dbias = lib.matmul_epilogue_backward(s["dy"], s["x"], s["w"], pre=s["z"],
                                                 activation=s["act"],
                                                 need=(True, True, s["bias"]))
    out = dict(da=da, dw=dw)
    if s["bias"]:
        out["dbias"] = dbias
    return out


def run(state):
    return kernels(state) if own else plain(state)


def work(case):
    op, m, n, e = case["op"], case["tokens"], case["n"], BYTES[case["dtype"]]
    if op.startswith("norm"):
        p = BYTES[case["params"]]
        if op == "norm":
            return dict(bytes=2 * m * n * e + 2 * n * p + (8 * m if case["keep"] else 0),
                        flops=8 * m * n)
        return dict(bytes=3 * m * n * e + 3 * n * p + 8 * m, flops=14 * m * n)
    k = case["k"]
    if op == "gated":
        return dict(bytes=(m * k + 2 * n * k + (3 if case["keep"] else 1) * m * n) * e,
                    flops=4 * m * n * k + 8 * m * n)
    if op == "gated_backward":
        # reads dh, g, u, x and both weights, writes dx and both weights' gradients
        return dict(bytes=(3 * m * n + 2 * m * k + 4 * n * k) * e,
                    flops=8 * m * n * k + 12 * m * n)
    if op == "epilogue":
        rows = 1 + (1 if case["residual"] else 0) + (1 if case["keep"] else 0)
        return dict(bytes=(m * k + n * k + rows * m * n + (n if case["bias"] else 0)) * e,
                    flops=2 * m * n * k + 4 * m * n)
    rows = 2 if case["act"] != "none" else 1
    return dict(bytes=(rows * m * n + 2 * m * k + 2 * n * k + (n if case["bias"] else 0)) * e,
                flops=4 * m * n * k + 6 * m * n)


def exact(case, seed):
    """The definitions, term by term in 64 bits."""
    s = {key: v.double() if isinstance(v, torch.Tensor) else v
         for key, v in prepare(case, seed).items()}
    op, n = s["op"], s["n"]

    def phi(z, name):
        return {"none": lambda: z,
                "relu": lambda: z.clamp(min=0),
                "gelu": lambda: z * torch.special.ndtr(z),
                "gelu_tanh": lambda: z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi)
                                                        * (z + 0.044715 * z ** 3))),
                "silu": lambda: z / (1 + torch.exp(-z)),
                "sigmoid": lambda: 1 / (1 + torch.exp(-z))}[name]()

    def slope(z, name):
        # by automatic differentiation of the definition (0 at relu's corner)
        if name == "relu":
            return (z > 0).double()
        with torch.enable_grad():
            z = z.detach().clone().requires_grad_(True)
            return torch.autograd.grad(phi(z, name).sum(), z)[0]

    if op == "norm":
        mean = s["x"].sum(1) / n
        var = torch.einsum("ij,ij->i", s["x"] - mean[:, None], s["x"] - mean[:, None]) / n
        rstd = 1 / torch.sqrt(var + EPS)
        out = dict(y=torch.addcmul(s["b"], (s["x"] - mean[:, None]) * rstd[:, None], s["w"]))
        return dict(out, mean=mean, rstd=rstd) if s["keep"] else out
    if op == "norm_backward":
        xhat = (s["x"] - s["mean"][:, None]) * s["rstd"][:, None]
        v = s["dy"] * s["w"]
        along = torch.einsum("ij,ij->i", v, xhat) / n
        dx = s["rstd"][:, None] * (v - (v.sum(1) / n)[:, None] - along[:, None] * xhat)
        return dict(dx=dx, dw=torch.einsum("ij,ij->j", s["dy"], xhat), db=s["dy"].sum(0))
    if op == "gated":
        g, u = torch.mm(s["x"], s["wg"]), torch.mm(s["x"], s["wu"])
        out = dict(h=phi(g, s["act"]) * u)
        return dict(out, g=g, u=u) if s["keep"] else out
    if op == "gated_backward":
        dg = s["dh"] * s["u"] * slope(s["g"], s["act"])
        du = s["dh"] * phi(s["g"], s["act"])
        return dict(dx=torch.mm(dg, s["wg"].t()) + torch.mm(du, s["wu"].t()),
                    dwg=torch.mm(s["x"].t(), dg), dwu=torch.mm(s["x"].t(), du))
    if op == "epilogue":
        z = torch.mm(s["x"], s["w"])
        z = z if s["bias_values"] is None else z + s["bias_values"]
        y = phi(z, s["act"])
        y = y if s["residual_rows"] is None else y + s["residual_rows"]
        return dict(y=y, z=z) if s["keep"] else dict(y=y)
    dz = s["dy"] if s["z"] is None else s["dy"] * slope(s["z"], s["act"])
    out = dict(da=torch.mm(dz, s["w"].t()), dw=torch.mm(s["x"].t(), dz))
    return dict(out, dbias=dz.sum(0)) if s["bias"] else out
