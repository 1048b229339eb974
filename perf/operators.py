"""Cases of the dense and expert layers for timing and comparison.

Three operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and through the framework's entry points:

  forward   Z = X W^T + b, Y = act(Z) + R            layers.DenseLinear.forward
  backward  dZ = dY * act'(Z), dX = dZ W,
            dW = dZ^T X, db = sum over rows of dZ     layers.DenseLinear.backward
  moe       a mixture-of-experts layer for a few tokens: router, top-k and
            the gated experts                         layers.MoeLayer.forward

`own` chooses which of the two `run` computes.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SQRT1_2 = math.sqrt(0.5)
TANH_C = math.sqrt(2.0 / math.pi)


# ---- the cases ----

def dense(op, name, N, d_in, d_out, dtype="bf16", act="none", bias=True, residual=False,
          save_z=False):
    c = dict(op=op, N=N, d_in=d_in, d_out=d_out, dtype=dtype, act=act, bias=bias)
    if op == "forward":
        c.update(residual=residual, save_z=save_z)
    return dict(c, name=name) if name else c


def moe(name, N, d_model, d_ff, experts, top_k, dtype="bf16", renorm=True, residual=False):
    c = dict(op="moe", N=N, d_model=d_model, d_ff=d_ff, experts=experts, top_k=top_k, dtype=dtype,
             renorm=renorm, residual=residual)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the fp32 configuration of the synthetic set, one call's latency
        dense("forward", "fwd_tiny_f32", 64, 256, 256, "f32", "gelu", residual=True),
        # ViT-L/16 fc1 over 32 images of 201 tokens, its GELU in the epilogue
        dense("forward", "fwd_vit_fc1", 6432, 1024, 4096, act="gelu"),
        # ViT-L/16 fc2 over 64 images, the block's residual in the epilogue
        dense("forward", "fwd_vit_block_fc2", 12864, 4096, 1024, residual=True),
        # a decoding step of the Llama-shaped up-projection
        dense("forward", "fwd_llama_up_1", 1, 4096, 14336, act="silu", bias=False),
        # one short ragged sequence through the Whisper-shaped fc1, pre-activations kept for training
        dense("forward", "fwd_whisper_201", 201, 1280, 5120, act="gelu_tanh", save_z=True),
        # training steps of ViT-L/16 fc1 and of Whisper-large fc1 (8 clips of 1500 frames)
        dense("backward", "bwd_vit_fc1", 6432, 1024, 4096, act="gelu"),
        dense("backward", "bwd_whisper_fc1", 12000, 1280, 5120, act="gelu"),
        # odd sizes in fp32
        dense("backward", "bwd_odd_f32", 77, 250, 190, "f32", "relu"),
        # a decoding step of one sequence: two of eight Llama-shaped experts
        moe("moe_llama_1", 1, 4096, 14336, 8, 2),
        # a decoding step of 64 sequences over many small experts
        moe("moe_wide_64", 64, 2048, 1024, 128, 8),
        # odd sizes, softmax weights as they are, the block's residual
        moe("moe_odd_13", 13, 1000, 488, 17, 3, renorm=False, residual=True),
        # fp32, one call's latency
        moe("moe_small_f32", 3, 256, 512, 8, 2, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _flops(c):
    if c["op"] == "moe":
        return 6.0 * c["N"] * c["top_k"] * c["d_model"] * c["d_ff"]
    return (4.0 if c["op"] == "backward" else 2.0) * c["N"] * c["d_in"] * c["d_out"]


def _expert_values(c):
    """Weight values of the experts that the tokens can reach."""
    reached = min(c["experts"], c["N"] * c["top_k"])
    return reached * 3.0 * c["d_model"] * c["d_ff"]


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "moe", "moe"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    q = 8 if dtype == "bf16" else 1  # bf16 rows are whole 16-byte pieces
    size = lambda lo, hi: max(q, _log(rng, lo, hi) // q * q)  # noqa: E731
    while True:
        if op == "moe":
            experts = _log(rng, 4, 128)
            c = moe("", _log(rng, 1, 64), size(128, 4096), size(64, 14336), experts,
                    rng.randint(1, min(8, experts)), dtype, rng.random() < 0.5, rng.random() < 0.5)
            total = experts * 3.0 * c["d_model"] * c["d_ff"]
            if total <= (1.0e9 if dtype == "bf16" else 1.0e8):
                return c
            continue
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        big = dtype == "bf16"
        c = dense(op, "", _log(rng, 1, 12864 if big else 2048), size(64, 5120 if big else 2048),
                  size(64, 14336 if big else 2048), dtype, act, rng.random() < 0.7,
                  rng.random() < 0.5, rng.random() < 0.3)
        if _flops(c) <= (3.0e11 if big else 1.0e10):
            return c


# ---- inputs ----

def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _acts(g, n, d, dtype):
    """Activations: normal rows under log-normal channel scales."""
    return (torch.randn(n, d, generator=g, device="cuda")
            * torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    N = case["N"]
    if case["op"] == "moe":
        d, f, E = case["d_model"], case["d_ff"], case["experts"]
        s["X"] = _acts(g, N, d, dt)
        s["Wr"] = _normal(g, E, d, scale=d ** -0.5, dtype=dt)
        s["Wgu"] = torch.empty(E, 2 * f, d, device="cuda", dtype=dt)
        s["Wd"] = torch.empty(E, d, f, device="cuda", dtype=dt)
        for W, fan in ((s["Wgu"], d), (s["Wd"], f)):
            for e in range(E):
                W[e] = _normal(g, W.shape[1], W.shape[2], scale=fan ** -0.5, dtype=dt)
        s["R"] = _normal(g, N, d, dtype=dt) if case["residual"] else None
        if own:
            from rank_structured_matmul_b200 import layers
            s["layer"] = layers.MoeLayer(d, f, E, case["top_k"], case["dtype"],
                                         renorm=case["renorm"])
        return s
    d_in, d_out = case["d_in"], case["d_out"]
    s["X"] = _acts(g, N, d_in, dt)
    s["W"] = _normal(g, d_out, d_in, scale=d_in ** -0.5, dtype=dt)
    s["b"] = _normal(g, d_out, scale=0.1, dtype=dt) if case["bias"] else None
    if case["op"] == "forward":
        s["R"] = _normal(g, N, d_out, dtype=dt) if case["residual"] else None
    else:
        # the pre-activations that the forward kept, in its type
        z = s["X"].float() @ s["W"].float().t()
        s["Z"] = (z + s["b"].float() if case["bias"] else z).to(dt)
        s["dY"] = _normal(g, N, d_out, dtype=dt)
    if own:
        from rank_structured_matmul_b200 import layers
        s["layer"] = layers.DenseLinear(d_in, d_out, case["dtype"])
    return s


# ---- the operators ----

def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * SQRT1_2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(TANH_C * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * SQRT1_2)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(TANH_C * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * TANH_C * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _forward(s, c, dt):
    z = s["X"].float() @ s["W"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return (y.to(dt), z.to(dt)) if c["save_z"] else (y.to(dt),)


def _backward(s, c, dt):
    dZ = s["dY"].float() * _act_grad(s["Z"].float(), c["act"])
    out = [(dZ @ s["W"].float()).to(dt), (dZ.t() @ s["X"].float()).to(dt)]
    return out + [dZ.sum(0).to(dt)] if c["bias"] else out


def _moe(s, c, dt):
    N, K, f = c["N"], c["top_k"], c["d_ff"]
    x = s["X"].float()
    # the logits in 64 bits: experts next to the border of the top k must not change places
    logits = s["X"].double() @ s["Wr"].double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = order.indices[:, :K]
    p = torch.exp(order.values - order.values[:, :1]).float()
    w = p[:, :K] / (p[:, :K] if c["renorm"] else p).sum(1, keepdim=True)
    if N * K <= c["experts"]:  # only the chosen experts' weights
        e = ids.reshape(-1)
        rows = x.repeat_interleave(K, dim=0).unsqueeze(2)
        gu = (s["Wgu"][e].float() @ rows).squeeze(2)
        h = (_act(gu[:, :f], "silu") * gu[:, f:]).unsqueeze(2)
        y = (s["Wd"][e].float() @ h).reshape(N, K, -1)
        y = (y * w.unsqueeze(2)).sum(1)
    else:  # every expert on every token, weighted by zero where it is not chosen
        full = torch.zeros(N, c["experts"], device=x.device).scatter_(1, ids, w)
        gu = torch.matmul(x, s["Wgu"].float().transpose(1, 2))  # E x N x 2f
        h = _act(gu[..., :f], "silu") * gu[..., f:]
        y = torch.matmul(h, s["Wd"].float().transpose(1, 2))
        y = (y * full.t().unsqueeze(2)).sum(0)
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.to(dt), ids.to(torch.int32), w


def run(state):
    c = state["case"]
    if own:
        layer = state["layer"]
        if c["op"] == "moe":
            return layer.forward(state["X"], state["Wr"], state["Wgu"], state["Wd"],
                                 residual=state["R"])
        if c["op"] == "forward":
            out = layer.forward(state["X"], state["W"], bias=state["b"], residual=state["R"],
                                act=c["act"], save_z=c["save_z"])
            return out if c["save_z"] else (out,)
        dX, dW, db = layer.backward(state["dY"], state["X"], state["W"], Z=state["Z"],
                                    act=c["act"], need_dbias=c["bias"])
        return [dX, dW, db] if c["bias"] else [dX, dW]
    dt = DTYPES[c["dtype"]]
    return {"forward": _forward, "backward": _backward, "moe": _moe}[c["op"]](state, c, dt)


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    N = case["N"]
    if case["op"] == "moe":
        d, E, K = case["d_model"], case["experts"], case["top_k"]
        vals = N * d * (3 if case["residual"] else 2) + E * d + _expert_values(case)
        return {"bytes": vals * es + N * K * 8.0, "flops": _flops(case) + 2.0 * N * E * d}
    d_in, d_out = case["d_in"], case["d_out"]
    if case["op"] == "forward":
        vals = N * d_in + d_in * d_out + d_out * case["bias"] \
            + N * d_out * (1 + case["residual"] + case["save_z"])
    else:  # dY, X, W and (with an activation) Z in; dX, dW and db out
        vals = N * d_out * (1 + (case["act"] != "none")) + 2 * (N * d_in + d_in * d_out) \
            + d_out * case["bias"]
    return {"bytes": float(vals * es), "flops": _flops(case)}


# ---- the definition in 64 bits ----

def _phi(z):
    """The normal distribution function."""
    return 0.5 * torch.special.erfc(-z * SQRT1_2)


def _sigmoid64(z):
    return torch.where(z >= 0, 1 / (1 + torch.exp(-z.abs())),
                       torch.exp(-z.abs()) / (1 + torch.exp(-z.abs())))


def _act64(z, act):
    if act == "gelu_tanh":  # (1 + tanh u) / 2 is the logistic function of 2 u
        return z * _sigmoid64(2 * TANH_C * (z + 0.044715 * z ** 3))
    return {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, torch.zeros_like(z)),
            "gelu": lambda: z * _phi(z), "silu": lambda: z * _sigmoid64(z)}[act]()


def exact(case, seed):
    s = prepare(case, seed)
    X = s["X"].double()
    if case["op"] == "moe":
        f, K = case["d_ff"], case["top_k"]
        p = torch.softmax(torch.einsum("nd,ed->ne", X, s["Wr"].double()), dim=1)
        y = torch.zeros_like(X) if s["R"] is None else s["R"].double()
        left, ids, picked = p.clone(), [], []
        for _ in range(K):  # the largest left, the lowest index among equals
            top = left.max(1, keepdim=True).values
            i = (left == top).to(torch.uint8).argmax(1)
            ids.append(i)
            picked.append(p.gather(1, i[:, None])[:, 0])
            left.scatter_(1, i[:, None], -1.0)
        ids, w = torch.stack(ids, 1), torch.stack(picked, 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        for e in ids.unique().tolist():
            n, slot = (ids == e).nonzero(as_tuple=True)
            gu = X[n] @ s["Wgu"][e].double().t()
            h = _act64(gu[:, :f], "silu") * gu[:, f:]
            y.index_add_(0, n, w[n, slot][:, None] * (h @ s["Wd"][e].double().t()))
        return y, None, w
    W = s["W"].double()
    if case["op"] == "forward":
        z = torch.einsum("ni,oi->no", X, W)
        if s["b"] is not None:
            z += s["b"].double()
        y = _act64(z, case["act"])
        if s["R"] is not None:
            y = y + s["R"].double()
        return (y, z) if case["save_z"] else (y,)
    z = s["Z"].double().requires_grad_(True)
    with torch.enable_grad():
        dZ, = torch.autograd.grad(_act64(z, case["act"]), z, s["dY"].double())
    out = [torch.einsum("no,oi->ni", dZ, W), torch.einsum("no,ni->oi", dZ, X)]
    return out + [dZ.sum(0)] if case["bias"] else out
