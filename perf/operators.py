"""The dense operators beside the routed layer: the matrix product with bias,
activation and residual, and the gated feed-forward block, each with its
backward pass.

A case's sizes: T rows, `inner` features in, `outer` features out (linear) or
the FFN width (ffn).  Weights are bf16; x, residual and y are bf16 or fp32.
"""
import math

import torch

own = False

DEV = "cuda"
MAX_T, MAX_INNER, MAX_OUTER = 8192, 4096, 11008


def listed():
    """Decode windows, prefill chunks and training steps, from one row to 8192."""
    return [
        # a bf16 shared expert of the decode model, one token: its output is added to the routed layer's fp32 y
        dict(name="ffn_decode_1", op="ffn", T=1, inner=2048, outer=768, act="silu", x="bf16", y="fp32", residual=True, save=False),
        # a dense first layer in a 16-row window, bf16 throughout
        dict(name="ffn_window_16", op="ffn", T=16, inner=2048, outer=5632, act="silu", x="bf16", y="bf16", residual=True, save=False),
        # the shared expert of the large-expert-count layer over a 2048-token prefill chunk, added to the fp32 y
        dict(name="ffn_prefill_2048", op="ffn", T=2048, inner=2048, outer=512, act="silu", x="bf16", y="fp32", residual=True, save=False),
        # a training step's forward pass of a large dense block, gate and up kept for the backward pass
        dict(name="ffn_train_8192", op="ffn", T=8192, inner=4096, outer=11008, act="silu", x="bf16", y="bf16", residual=True, save=True),
        # fine-tuning a shared expert on a ragged batch of 1003 tokens
        dict(name="ffn_bwd_ragged_1003", op="ffn_bwd", T=1003, inner=2048, outer=768, act="silu"),
        # the backward pass of the large dense block
        dict(name="ffn_bwd_8192", op="ffn_bwd", T=8192, inner=4096, outer=11008, act="silu"),
        # a projection of one token with its residual, the latency of a decode step
        dict(name="linear_decode_1", op="linear", T=1, inner=2048, outer=2048, act="none", x="bf16", y="bf16", bias=True, residual=True, save=False),
        # odd sizes with fp32 activations, a small window of the kind the tiny layer runs
        dict(name="linear_fp32_37", op="linear", T=37, inner=1000, outer=520, act="gelu", x="fp32", y="fp32", bias=True, residual=False, save=False),
        # a prefill chunk through a projection with bias and activation
        dict(name="linear_prefill_2048", op="linear", T=2048, inner=2048, outer=4096, act="gelu_tanh", x="bf16", y="bf16", bias=True, residual=False, save=True),
        # a large projection added to an fp32 residual stream
        dict(name="linear_large_8192", op="linear", T=8192, inner=4096, outer=8192, act="none", x="bf16", y="fp32", bias=True, residual=True, save=False),
        # the backward pass of a projection with activation on a ragged batch
        dict(name="linear_bwd_ragged_777", op="linear_bwd", T=777, inner=1032, outer=2048, act="gelu_tanh", bias=True, dw="bf16"),
        # the backward pass of the large projection, weight gradients kept in fp32
        dict(name="linear_bwd_8192", op="linear_bwd", T=8192, inner=4096, outer=4096, act="none", bias=True, dw="fp32"),
    ]


def _log_int(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    """Rows from 1 to 8192, widths from 64 to 11008 in multiples of 8, each activation and type."""
    op = rng.choice(["ffn", "ffn_bwd", "linear", "linear_bwd"])
    case = dict(op=op, T=_log_int(rng, 1, MAX_T), inner=_log_int(rng, 64, MAX_INNER, 8),
                outer=_log_int(rng, 64, MAX_OUTER, 8))
    case["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu"] + (["none", "none"] if op.startswith("linear") else []))
    if op in ("ffn", "linear"):
        case["x"] = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        case["y"] = rng.choice(["bf16", "fp32"]) if case["x"] == "bf16" else "fp32"
        case["residual"] = rng.random() < 0.5
        case["save"] = rng.random() < 0.3
    if op.startswith("linear"):
        case["bias"] = rng.random() < 0.5
    if op == "linear_bwd":
        case["dw"] = rng.choice(["bf16", "fp32"]) if case["act"] == "none" else "bf16"
    return case


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    T, K, N, op = case["T"], case["inner"], case["outer"], case["op"]
    s = {"case": case}
    if op in ("ffn", "linear"):
        s["x"] = normal(T, K, dtype=_TYPES[case["x"]])
        ydt = _TYPES[case["y"]]
        width = K if op == "ffn" else N
        s["residual"] = normal(T, width, dtype=ydt) if case["residual"] else None
        s["y"] = torch.empty((T, width), dtype=ydt, device=DEV)
    else:
        s["x"] = normal(T, K)
        s["dy"] = normal(T, K if op == "ffn_bwd" else N, std=0.01)
        s["dx"] = torch.empty((T, K), dtype=torch.bfloat16, device=DEV)
    if op.startswith("ffn"):
        s["gate"], s["up"], s["down"] = normal(N, K, std=0.02), normal(N, K, std=0.02), normal(K, N, std=0.02)
        if op == "ffn_bwd":
            # what the forward pass keeps: gate and up projections, [T][2F]
            s["gu"] = torch.cat([s["x"].float() @ s["gate"].float().T, s["x"].float() @ s["up"].float().T], 1).to(torch.bfloat16)
            s["dgate"], s["dup"], s["ddown"] = (torch.empty_like(s[k]) for k in ("gate", "up", "down"))
        else:
            s["gu"] = torch.empty((T, 2 * N), dtype=torch.bfloat16, device=DEV) if case["save"] else None
    else:
        s["w"] = normal(N, K, std=0.02)
        s["bias"] = normal(N, std=0.1) if case["bias"] else None
        if op == "linear_bwd":
            s["z"] = normal(T, N) if case["act"] != "none" else None
            s["dw"] = torch.empty((N, K), dtype=_TYPES[case["dw"]], device=DEV)
            s["dbias"] = torch.empty((N,), dtype=_TYPES[case["dw"]], device=DEV) if case["bias"] else None
        else:
            s["z"] = torch.empty((T, N), dtype=torch.bfloat16, device=DEV) if case["save"] else None
    return s


# ---------------------------------------------------------------------------
# The plain forms: fp32 throughout, one rounding at the end
# ---------------------------------------------------------------------------
_C = math.sqrt(2.0 / math.pi)


def _act(name, z):
    if name == "none":
        return z
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(_C * (z + 0.044715 * z * z * z)))


def _act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    t = torch.tanh(_C * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * z * z)


def _plain(s):
    case = s["case"]
    op, act = case["op"], case["act"]
    x = s["x"].float()
    if op == "linear":
        z = x @ s["w"].float().T
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(act, z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"y": y.to(s["y"].dtype)}
        if s["z"] is not None:
            out["z"] = z.to(torch.bfloat16)
        return out
    if op == "ffn":
        g, u = x @ s["gate"].float().T, x @ s["up"].float().T
        y = (_act(act, g) * u) @ s["down"].float().T
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"y": y.to(s["y"].dtype)}
        if s["gu"] is not None:
            out["gu"] = torch.cat([g, u], 1).to(torch.bfloat16)
        return out
    dy = s["dy"].float()
    if op == "linear_bwd":
        dz = dy if act == "none" else dy * _act_grad(act, s["z"].float())
        out = {"dx": (dz @ s["w"].float()).to(torch.bfloat16), "dw": (dz.T @ x).to(s["dw"].dtype)}
        if s["dbias"] is not None:
            out["dbias"] = dz.sum(0).to(s["dbias"].dtype)
        return out
    F = case["outer"]
    g, u = s["gu"][:, :F].float(), s["gu"][:, F:].float()
    a = _act(act, g)
    dh = dy @ s["down"].float()
    dg, du = dh * u * _act_grad(act, g), dh * a
    return {"dx": (dg @ s["gate"].float() + du @ s["up"].float()).to(torch.bfloat16),
            "dgate": (dg.T @ x).to(torch.bfloat16), "dup": (du.T @ x).to(torch.bfloat16),
            "ddown": (dy.T @ (a * u)).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    from quantized_routed_expert_amd import moe

    case = s["case"]
    op = case["op"]
    if "ws" not in s:  # kept by the program next to its weights: workspace, weight description, activation code
        T, K, N = case["T"], case["inner"], case["outer"]
        s["act"] = {"none": moe.ACT_NONE, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU, "gelu_tanh": moe.ACT_GELU_TANH,
                    "relu": moe.ACT_RELU}[case["act"]]
        if op.startswith("ffn"):
            s["ws"] = moe.gated_ffn_workspace(T, K, N, device=s["x"].device)
            s["ffn"] = moe.dense_ffn(s["gate"], s["up"], s["down"], s["act"])
        else:
            s["ws"] = moe.linear_workspace(T, K, N, device=s["x"].device)
    if op == "linear":
        out = {"y": moe.linear(s["x"], s["w"], s["ws"], bias=s["bias"], act=s["act"], residual=s["residual"], z=s["z"], y=s["y"])}
        if s["z"] is not None:
            out["z"] = s["z"]
        return out
    if op == "ffn":
        out = {"y": moe.gated_ffn(s["x"], s["ffn"], s["ws"], residual=s["residual"], gu=s["gu"], y=s["y"])}
        if s["gu"] is not None:
            out["gu"] = s["gu"]
        return out
    if op == "linear_bwd":
        moe.linear_backward(s["dy"], s["x"], s["w"], s["ws"], z=s["z"], act=s["act"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"])
        out = {"dx": s["dx"], "dw": s["dw"]}
        if s["dbias"] is not None:
            out["dbias"] = s["dbias"]
        return out
    moe.gated_ffn_backward(s["dy"], s["x"], s["gu"], s["ffn"], s["ws"], dx=s["dx"], dgate=s["dgate"], dup=s["dup"],
                           ddown=s["ddown"])
    return {"dx": s["dx"], "dgate": s["dgate"], "dup": s["dup"], "ddown": s["ddown"]}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """Every input read once and every output written once; two operations per product term."""
    T, K, N, op = case["T"], case["inner"], case["outer"], case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "linear":
        b = T * K * size[case["x"]] + 2 * N * K + T * N * size[case["y"]] * (2 if case["residual"] else 1)
        return {"bytes": b + 2 * N * case["bias"] + 2 * T * N * case["save"], "flops": 2 * T * K * N}
    if op == "ffn":
        b = T * K * size[case["x"]] + 6 * N * K + T * K * size[case["y"]] * (2 if case["residual"] else 1)
        return {"bytes": b + 4 * T * N * case["save"], "flops": 6 * T * K * N}
    if op == "linear_bwd":
        b = 2 * T * N + 4 * T * K + 2 * N * K + N * K * size[case["dw"]] + N * size[case["dw"]] * case["bias"]
        return {"bytes": b + (2 * T * N if case["act"] != "none" else 0), "flops": 4 * T * K * N}
    return {"bytes": 6 * T * K + 4 * T * N + 12 * N * K, "flops": 12 * T * K * N}


# ---------------------------------------------------------------------------
# The definition in 64 bits: torch's own activations, gradients by
# differentiating the forward definition
# ---------------------------------------------------------------------------
def _definition(name):
    F = torch.nn.functional
    return {"none": lambda z: z, "silu": F.silu, "relu": F.relu, "gelu": F.gelu,
            "gelu_tanh": lambda z: F.gelu(z, approximate="tanh")}[name]


def exact(case, seed):
    s = prepare(case, seed)
    act, op = _definition(case["act"]), case["op"]
    d = {k: v.double() for k, v in s.items() if k in ("x", "w", "bias", "gate", "up", "down", "residual", "dy", "z", "gu") and v is not None}
    lin = torch.nn.functional.linear
    if op == "linear":
        z = lin(d["x"], d["w"], d.get("bias"))
        out = {"y": act(z) + d["residual"] if "residual" in d else act(z)}
        if case["save"]:
            out["z"] = z
        return out
    if op == "ffn":
        g, u = lin(d["x"], d["gate"]), lin(d["x"], d["up"])
        y = lin(act(g) * u, d["down"])
        out = {"y": y + d["residual"] if "residual" in d else y}
        if case["save"]:
            out["gu"] = torch.cat([g, u], 1)
        return out
    leaves = [d[k].requires_grad_() for k in (("x", "w") if op == "linear_bwd" else ("x", "gate", "up", "down"))]

    def kept(value, at):  # the forward pass's kept (rounded) value, with the gradient of the product
        return value + (at - value).detach()

    if op == "linear_bwd":
        if case["bias"]:
            leaves.append(torch.zeros_like(d["bias"]).requires_grad_())
        z = lin(d["x"], d["w"], leaves[2] if case["bias"] else None)
        y = act(kept(z, d["z"]) if "z" in d else z)
        grads = torch.autograd.grad(y, leaves, d["dy"])
        return dict(zip(("dx", "dw", "dbias"), grads))
    N = case["outer"]
    g, u = kept(lin(d["x"], d["gate"]), d["gu"][:, :N]), kept(lin(d["x"], d["up"]), d["gu"][:, N:])
    grads = torch.autograd.grad(lin(act(g) * u, d["down"]), leaves, d["dy"])
    return dict(zip(("dx", "dgate", "dup", "ddown"), grads))
