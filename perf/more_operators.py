"""Cases of the operators of a feed-forward block with experts, with a plain form of each.

``tokens`` tokens choose ``k`` of ``experts`` experts each; the rows = tokens * k (token, expert)
pairs are sorted by expert, go through their experts' products and come back, weighted:

* ``dispatch``: from the tokens' expert ids (-1: none, the padding of a batch) each pair's
  position in the order by expert and the experts' first rows, and the tokens' vectors copied to
  those rows;
* ``dispatch_backward``: dx[t] = the sum of the gradients of token t's rows;
* ``combine``: y[t] = sum_j w[t, j] rows[position[t, j]] + residual[t];
* ``combine_backward``: drows[position[t, j]] = w[t, j] dy[t], dw[t, j] = dy[t] . rows[position[t, j]];
* ``product``: y[r] = x[r] W[e] for the rows r of each expert e;
* ``product_backward``: dx[r] = dy[r] W[e]^T, dW[e] = the sum of x[r]^T dy[r] over e's rows;
* ``gated``: h[r] = act(x[r] Wg[e]) * (x[r] Wu[e]) (and the two products where they are kept);
* ``gated_backward``: its gradients from dh and the kept products;
* ``dropout``: y = residual + x * mask / (1 - p), the mask from Philox4x32-10 (Salmon, Moraes,
  Dror and Shaw, 2011) at each element's place, in 16-bit numbers;
* ``dropout_backward``: dx = dy * mask / (1 - p), the mask made again.

Weights are stored as [experts, outputs, inputs] and passed as the transposed view. ``own``
chooses between the plain form (torch operations in 32 bits, rounded once at the end) and the
library's operators.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token of a generation step, sent to its experts
        dict(name="dispatch_token", op="dispatch", dtype="bf16", tokens=1, k=4, experts=32, n=2048,
             padded=False),
        # a training batch sent to its experts; the last sequences are shorter than the batch
        dict(name="dispatch_train", op="dispatch", dtype="bf16", tokens=16384, k=4, experts=64,
             n=2048, padded=True),
        # a training batch back from its experts, onto the residual stream
        dict(name="combine_train", op="combine", dtype="bf16", weights="f32", tokens=16384, k=4,
             experts=64, n=2048, padded=True, residual=True),
        # odd sizes in 32 bits, as a small model's tests run
        dict(name="combine_backward_odd_f32", op="combine_backward", dtype="f32", weights="f32",
             tokens=1023, k=3, experts=17, n=1025),
        # a server's batch of single tokens through the experts' down projections
        dict(name="product_decode_batch", op="product", dtype="f16", tokens=64, k=4, experts=32,
             inputs=4096, n=2048),
        # a training batch through the experts' down projections
        dict(name="product_train", op="product", dtype="bf16", tokens=8192, k=2, experts=16,
             inputs=4096, n=2048),
        # its backward pass, with more and smaller experts
        dict(name="product_backward", op="product_backward", dtype="bf16", tokens=8192, k=2,
             experts=64, inputs=1024, n=2048),
        # one token of a generation step through the gated half of its experts
        dict(name="gated_token", op="gated", dtype="bf16", tokens=1, k=4, experts=32, inputs=2048,
             n=4096, act="silu", keep=False),
        # a training batch, keeping what the backward pass needs
        dict(name="gated_train", op="gated", dtype="bf16", tokens=8192, k=2, experts=16,
             inputs=2048, n=4096, act="silu", keep=True),
        # its backward pass
        dict(name="gated_backward", op="gated_backward", dtype="bf16", tokens=8192, k=2,
             experts=16, inputs=2048, n=4096, act="silu"),
        # a training batch's block output, dropped and added to the residual stream
        dict(name="dropout_train", op="dropout", dtype="bf16", tokens=16384, n=4096, p=0.1,
             residual=True),
        # the backward pass of an odd width in 32 bits
        dict(name="dropout_backward_odd_f32", op="dropout_backward", dtype="f32", tokens=1023,
             n=1025, p=0.5),
    ]


# The largest listed case's cost, which no drawn case passes.
MAX_FLOPS = 8.0 * 8192 * 2 * 2048 * 4096
MAX_BYTES = 2.0 * 16384 * 5 * 2048
MAX_WEIGHTS = 2 * 32 * 2048 * 4096


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def width(rng, lo, hi):
    """A row width: mostly what models use (multiples of 64 or 8), some of any size."""
    n = log_uniform(rng, lo, hi)
    step = rng.choice((64, 64, 8, 8, 1))
    return max(step, n // step * step)


def draw(rng):
    while True:
        op = rng.choice(("dispatch", "dispatch_backward", "combine", "combine_backward", "product",
                         "product_backward", "gated", "gated_backward", "dropout",
                         "dropout_backward"))
        case = dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16")))
        if op.startswith("dropout"):
            case["dtype"] = rng.choice(("bf16", "f16", "f32"))
            case.update(tokens=log_uniform(rng, 1, 16384), n=width(rng, 16, 16384),
                        p=rng.choice((0.05, 0.1, 0.2, 0.5)))
            if op == "dropout":
                case["residual"] = rng.random() < 0.5
            if work(case)["bytes"] <= MAX_BYTES:
                return case
            continue
        case.update(experts=log_uniform(rng, 2, 256), k=rng.choice((1, 2, 2, 3, 4, 6, 8)))
        case["k"] = min(case["k"], case["experts"])
        if op.startswith(("dispatch", "combine")):
            case["dtype"] = rng.choice(("bf16", "f16", "f32"))
            case.update(tokens=log_uniform(rng, 1, 16384), n=width(rng, 16, 8192))
            if op in ("dispatch", "combine"):
                case["padded"] = rng.random() < 0.3
            if op.startswith("combine"):
                case["weights"] = rng.choice(("f32", case["dtype"]))
            if op == "combine":
                case["residual"] = rng.random() < 0.5
            if work(case)["bytes"] <= MAX_BYTES:
                return case
            continue
        # generation steps and small batches as often as prompts and training batches
        case.update(tokens=log_uniform(rng, 64 if "backward" in op else 1, 16384),
                    inputs=width(rng, 64, 8192), n=width(rng, 64, 8192))
        if op.startswith("gated"):
            case["act"] = rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"))
        if op == "gated":
            case["keep"] = case["tokens"] >= 64 and rng.random() < 0.5
        w = work(case)
        if (w["flops"] <= MAX_FLOPS and w["bytes"] <= 16 * MAX_BYTES
                and case["experts"] * case["inputs"] * case["n"] <= MAX_WEIGHTS):
            return case


def choices(case, gen):
    """The tokens' experts, as a router gives them: distinct for a token, some experts more in
    demand than others; -1 for the padding at a batch's end."""
    t, e = case["tokens"], case["experts"]
    demand = 0.5 * torch.randn(e, generator=gen, device="cuda")
    ids = (torch.randn(t, e, generator=gen, device="cuda") + demand).topk(case["k"], 1).indices
    if case.get("padded"):
        ids[t - t // 8:] = -1
    return ids


def order(ids, experts):
    """Each entry's position in the stable order by expert, and the experts' first rows."""
    flat = ids.reshape(-1)
    chosen = (torch.arange(experts, device=flat.device)[:, None] == flat).to(torch.int32)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = chosen.sum(1).cumsum(0)
    before = chosen.cumsum(1, dtype=torch.int32) - chosen
    position = ((before + offsets[:-1, None].to(torch.int32)) * chosen).sum(0)
    position = torch.where(chosen.sum(0) > 0, position, torch.full_like(position, -1))
    return position.view(ids.shape).to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    t = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    op, m, n = case["op"], case["tokens"], case["n"]
    s = dict(case)
    if op.startswith("dropout"):
        s["x"] = normal(m, n)
        s["residual_rows"] = normal(m, n) if case.get("residual") else None
        # a run's seed and the number of this call in it, on the GPU so that a graph can advance it
        s["key"] = torch.randint(0, 2 ** 62, (2,), generator=gen, device="cuda")
        return s
    s["ids"] = choices(case, gen)
    s["position"], s["offsets"] = order(s["ids"], case["experts"])
    rows = m * case["k"]
    if op == "dispatch":
        s["x"] = normal(m, n)
        # rows behind the last expert's stay as they are in the caller's buffer
        s["rows"] = torch.zeros(rows, n, dtype=t, device="cuda") if case["padded"] else None
    elif op == "dispatch_backward":
        s["drows"] = normal(rows, n, scale=0.5)
    elif op in ("combine", "combine_backward"):
        s["rows"] = normal(rows, n)
        w = torch.randn(m, case["k"], generator=gen, device="cuda").exp()
        s["w"] = (w / w.sum(1, keepdim=True)).to(TYPES[case["weights"]])
        if op == "combine":
            s["residual_rows"] = normal(m, n) if case["residual"] else None
        else:
            s["dy"] = normal(m, n, scale=0.5)
    else:
        k, e = case["inputs"], case["experts"]
        s["x"] = normal(rows, k)
        scale = 1.0 / math.sqrt(k)
        if op.startswith("product"):
            s["w"] = normal(e, n, k, scale=scale).transpose(1, 2)
            if op == "product_backward":
                s["dy"] = normal(rows, n, scale=0.5)
        else:
            s["wg"] = normal(e, n, k, scale=scale).transpose(1, 2)
            s["wu"] = normal(e, n, k, scale=scale).transpose(1, 2)
            if op == "gated_backward":
                s["g"], s["u"] = normal(rows, n), normal(rows, n)
                s["dh"] = normal(rows, n, scale=0.5)
    return s


# ------------------------------------------------------------------------------ plain form


def sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z * sigmoid(z) if name == "silu" else sigmoid(z)


def act_slope(z, name):
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


def by_expert(x, w, offsets, transposed=False):
    """x[r] @ w[e] in 32 bits for the rows of each expert, whose numbers differ: one product each."""
    bounds = offsets.tolist()
    y = torch.empty(x.shape[0], w.shape[1] if transposed else w.shape[2], device=x.device)
    for e in range(w.shape[0]):
        a, b = bounds[e], bounds[e + 1]
        if a < b:
            we = w[e].float()
            y[a:b] = x[a:b].float() @ (we.t() if transposed else we)
    return y


def weight_gradient(x, dy, offsets, t):
    """x^T dy over the rows of each expert, as a view of [experts, outputs, inputs]."""
    bounds = offsets.tolist()
    e = len(bounds) - 1
    dw = torch.zeros(e, dy.shape[1], x.shape[1], dtype=t, device=x.device)
    for i in range(e):
        a, b = bounds[i], bounds[i + 1]
        if a < b:
            dw[i] = (dy[a:b].float().t() @ x[a:b].float()).to(t)
    return dw.transpose(1, 2)


def philox_words(key, rows, blocks):
    """Four 32-bit words (in 64-bit integers) at the counters (block, row, offset)."""
    low = 0xFFFFFFFF
    c0 = torch.arange(blocks, device=key.device)[None, :].expand(rows, blocks)
    c1 = torch.arange(rows, device=key.device)[:, None].expand(rows, blocks)
    c2, c3 = (key[1] & low).expand(rows, blocks), ((key[1] >> 32) & low).expand(rows, blocks)
    k0, k1 = key[0] & low, (key[0] >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def dropout_scale(s, rows, n):
    """The factor of each element: 0, or 1 over the probability to be kept."""
    blocks = -(-n // 8)
    words = torch.stack(philox_words(s["key"], rows, blocks), 2)
    numbers = torch.stack((words & 0xFFFF, words >> 16), 3).reshape(rows, blocks * 8)[:, :n]
    q = int(s["p"] * 65536 + 0.5)
    return (numbers >= q).to(torch.float32) * (65536.0 / (65536 - q))


def plain(s):
    op, t = s["op"], TYPES[s["dtype"]]
    if op.startswith("dropout"):
        x = s["x"].float()
        y = x * dropout_scale(s, *x.shape)
        if s["residual_rows"] is not None:
            y = y + s["residual_rows"].float()
        return dict(y=y.to(t))
    if op == "dispatch":
        position, offsets = order(s["ids"], s["experts"])
        rows = s["rows"]
        if rows is None:
            rows = torch.empty(position.numel(), s["n"], dtype=t, device=position.device)
        flat = position.reshape(-1).long()
        token = torch.arange(flat.numel(), device=flat.device) // s["k"]
        sent = flat >= 0
        rows[flat[sent]] = s["x"][token[sent]]
        return dict(position=position, offsets=offsets, rows=rows)
    if op == "dispatch_backward":
        return dict(dx=s["drows"][s["position"].long()].float().sum(1).to(t))
    if op == "combine":
        position = s["position"].long()
        w = torch.where(position >= 0, s["w"].float(), torch.zeros_like(position, dtype=torch.float32))
        y = (s["rows"][position.clamp(min=0)].float() * w[:, :, None]).sum(1)
        if s["residual_rows"] is not None:
            y = y + s["residual_rows"].float()
        return dict(y=y.to(t))
    if op == "combine_backward":
        position = s["position"].long()
        dy, w = s["dy"].float(), s["w"].float()
        drows = torch.empty_like(s["rows"])
        drows[position] = (w[:, :, None] * dy[:, None, :]).to(t)
        dw = (s["rows"][position].float() * dy[:, None, :]).sum(2)
        return dict(drows=drows, dw=dw.to(s["w"].dtype))
    if op == "product":
        return dict(y=by_expert(s["x"], s["w"], s["offsets"]).to(t))
    if op == "product_backward":
        return dict(dx=by_expert(s["dy"], s["w"], s["offsets"], True).to(t),
                    dw=weight_gradient(s["x"], s["dy"], s["offsets"], t))
    if op == "gated":
        g = by_expert(s["x"], s["wg"], s["offsets"])
        u = by_expert(s["x"], s["wu"], s["offsets"])
        h = (act(g, s["act"]) * u).to(t)
        return dict(h=h, g=g.to(t), u=u.to(t)) if s["keep"] else dict(h=h)
    g, u, dh = s["g"].float(), s["u"].float(), s["dh"].float()
    dg, du = dh * u * act_slope(g, s["act"]), dh * act(g, s["act"])
    dx = by_expert(dg, s["wg"], s["offsets"], True) + by_expert(du, s["wu"], s["offsets"], True)
    return dict(dx=dx.to(t), dwg=weight_gradient(s["x"], dg, s["offsets"], t),
                dwu=weight_gradient(s["x"], du, s["offsets"], t))


# ---------------------------------------------------------------------------- the library's


def kernels(s):
    import dense_tiled_gemm_05_gb300 as lib
    op = s["op"]
    if op == "dropout":
        return dict(y=lib.dropout(s["x"], s["p"], s["key"], residual=s["residual_rows"]))
    if op == "dropout_backward":
        return dict(y=lib.dropout_backward(s["x"], s["p"], s["key"]))
    if op == "dispatch":
        position, offsets = lib.expert_sort(s["ids"], s["experts"])
        rows = lib.expert_gather(s["x"], position, out=s["rows"])
        return dict(position=position, offsets=offsets, rows=rows)
    if op == "dispatch_backward":
        return dict(dx=lib.expert_gather_backward(s["drows"], s["position"]))
    if op == "combine":
        return dict(y=lib.expert_combine(s["rows"], s["position"], s["w"],
                                         residual=s["residual_rows"]))
    if op == "combine_backward":
        drows, dw = lib.expert_combine_backward(s["dy"], s["rows"], s["position"], s["w"])
        return dict(drows=drows, dw=dw)
    if op == "product":
        return dict(y=lib.expert_matmul(s["x"], s["w"], s["offsets"]))
    if op == "product_backward":
        dx, dw = lib.expert_matmul_backward(s["dy"], s["x"], s["w"], s["offsets"])
        return dict(dx=dx, dw=dw)
    if op == "gated":
        r = lib.expert_gated(s["x"], s["wg"], s["wu"], s["offsets"], activation=s["act"],
                             save=s["keep"])
        return dict(h=r[0], g=r[1], u=r[2]) if s["keep"] else dict(h=r)
    dx, dwg, dwu = lib.expert_gated_backward(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"],
                                             s["offsets"], activation=s["act"])
    return dict(dx=dx, dwg=dwg, dwu=dwu)


def run(state):
    return kernels(state) if own else plain(state)


def work(case):
    op, m, n, b = case["op"], case["tokens"], case["n"], BYTES[case["dtype"]]
    if op.startswith("dropout"):
        return dict(bytes=(3 if case.get("residual") else 2) * m * n * b, flops=10 * m * n)
    e, rows = case["experts"], m * case["k"]
    sent = rows - m // 8 * case["k"] if case.get("padded") else rows
    if op == "dispatch":
        return dict(bytes=(sent // case["k"] + sent) * n * b + 12 * rows + 4 * e, flops=0)
    if op == "dispatch_backward":
        return dict(bytes=(m + rows) * n * b + 4 * rows, flops=rows * n)
    if op == "combine":
        lines = m + sent + (m if case["residual"] else 0)
        return dict(bytes=lines * n * b + rows * (4 + BYTES[case["weights"]]), flops=2 * sent * n)
    if op == "combine_backward":
        return dict(bytes=(m + 2 * rows) * n * b + rows * (4 + 2 * BYTES[case["weights"]]),
                    flops=3 * rows * n)
    k = case["inputs"]
    # experts with rows: at most one a row; of few rows, as many as even choices would meet
    used = e * (1.0 - (1.0 - case["k"] / e) ** m)
    weights = int(used * k * n)
    if op == "product":
        return dict(bytes=(rows * (k + n) + weights) * b, flops=2 * rows * k * n)
    if op == "product_backward":
        return dict(bytes=(rows * (2 * k + n) + weights + e * k * n) * b, flops=4 * rows * k * n)
    if op == "gated":
        return dict(bytes=(rows * (k + (3 if case["keep"] else 1) * n) + 2 * weights) * b,
                    flops=4 * rows * k * n + 8 * rows * n)
    return dict(bytes=(rows * (2 * k + 3 * n) + 2 * weights + 2 * e * k * n) * b,
                flops=8 * rows * k * n + 12 * rows * n)


# ----------------------------------------------------------------------- the definitions


def exact(case, seed):
    """The definitions, term by term in 64 bits."""
    prepared = prepare(case, seed)
    s = {key: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for key, v in prepared.items()}
    op = case["op"]
    if op.startswith("dropout"):
        rows, n = s["x"].shape
        seed_, offset = (int(v) for v in s["key"].cpu())
        y = s["x"] * torch.from_numpy(_mask_by_numpy(rows, n, case["p"], seed_, offset)).cuda()
        return dict(y=y if s["residual_rows"] is None else y + s["residual_rows"])

    # the pairs in their order: (expert, token and choice)
    ids = s["ids"].reshape(-1).cpu().numpy()
    pairs = np.nonzero((ids >= 0) & (ids < case["experts"]))[0]
    pairs = pairs[np.argsort(ids[pairs], kind="stable")]
    expert_of_row = torch.from_numpy(ids[pairs]).cuda()
    token_of_row = torch.from_numpy(pairs // case["k"]).cuda()
    choice_of_row = torch.from_numpy(pairs % case["k"]).cuda()
    live = len(pairs)
    if op == "dispatch":
        position = np.full(ids.shape, -1, dtype=np.int32)
        position[pairs] = np.arange(live)
        offsets = np.searchsorted(ids[pairs], np.arange(case["experts"] + 1)).astype(np.int32)
        rows = torch.zeros(ids.size, case["n"], dtype=torch.float64, device="cuda")
        rows[:live] = s["x"][token_of_row]
        return dict(position=torch.from_numpy(position.reshape(case["tokens"], case["k"])),
                    offsets=torch.from_numpy(offsets), rows=rows)
    if op == "dispatch_backward":
        dx = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
        return dict(dx=dx.index_add_(0, token_of_row, s["drows"]))
    if op == "combine":
        y = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
        if s["residual_rows"] is not None:
            y += s["residual_rows"]
        weighted = s["rows"][:live] * s["w"][token_of_row, choice_of_row][:, None]
        return dict(y=y.index_add_(0, token_of_row, weighted))
    if op == "combine_backward":
        dy = s["dy"][token_of_row]
        dw = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device="cuda")
        dw[token_of_row, choice_of_row] = torch.einsum("rn,rn->r", dy, s["rows"])
        return dict(drows=dy * s["w"][token_of_row, choice_of_row][:, None], dw=dw)

    def phi(z, name):
        return {"relu": lambda: z.clamp(min=0),
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

    def each(x, w):
        y = torch.zeros(x.shape[0], w.shape[2], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            mine = torch.nonzero(expert_of_row == e)[:, 0]
            y[mine] = torch.einsum("rk,kn->rn", x[mine], w[e])
        return y

    def outer(x, dy):
        dw = [torch.einsum("rk,rn->kn", x[expert_of_row == e], dy[expert_of_row == e])
              for e in range(case["experts"])]
        return torch.stack(dw)

    if op == "product":
        return dict(y=each(s["x"], s["w"]))
    if op == "product_backward":
        return dict(dx=each(s["dy"], s["w"].transpose(1, 2)), dw=outer(s["x"], s["dy"]))
    if op == "gated":
        g, u = each(s["x"], s["wg"]), each(s["x"], s["wu"])
        out = dict(h=phi(g, case["act"]) * u)
        return dict(out, g=g, u=u) if case["keep"] else out
    dg = s["dh"] * s["u"] * slope(s["g"], case["act"])
    du = s["dh"] * phi(s["g"], case["act"])
    return dict(dx=each(dg, s["wg"].transpose(1, 2)) + each(du, s["wu"].transpose(1, 2)),
                dwg=outer(s["x"], dg), dwu=outer(s["x"], du))


def _mask_by_numpy(rows, n, p, seed, offset):
    """The mask's factors from unsigned 64-bit integers, block by block of eight elements."""
    u64, low = np.uint64, np.uint64(0xFFFFFFFF)
    block, row = np.meshgrid(np.arange(-(-n // 8), dtype=u64), np.arange(rows, dtype=u64))
    x = [block, row, np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)]
    for i in range(10):
        key0 = u64((seed + i * 0x9E3779B9) & 0xFFFFFFFF)
        key1 = u64(((seed >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)
        first, second = x[0] * u64(0xD2511F53), x[2] * u64(0xCD9E8D57)
        x = [(second >> u64(32)) ^ x[1] ^ key0, second & low,
             (first >> u64(32)) ^ x[3] ^ key1, first & low]
    halves = np.empty((rows, block.shape[1], 4, 2), dtype=np.int64)
    for i in range(4):
        halves[:, :, i, 0] = x[i] & u64(0xFFFF)
        halves[:, :, i, 1] = x[i] >> u64(16)
    q = int(math.floor(p * 65536 + 0.5))
    return (halves.reshape(rows, -1)[:, :n] >= q) * (65536.0 / (65536 - q))
