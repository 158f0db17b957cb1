"""The operators over decoded weights, in plain form and as the library calls them.

Three operators are here.  ``linear``: y = s * (x W^T) + alpha_a * (x A_a^T) B_a^T, a
projection by decoded E4M3 weights with the low-rank adapters of many requests
beside it.  ``backward``: its gradients for the input and for every adapter,
the weights being frozen.  ``clip``: the global L2 norm of many gradient
tensors, and the tensors scaled by min(1, max_norm / (norm + 1e-6)).

Requests are runs of rows: request i is rows offsets[i]..offsets[i+1]-1 and
uses adapter ids[i], or none where ids[i] is -1.  Rows from offsets[-1] on
belong to no request and take the shared projection alone.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _linear(name, rows, n, k, rank, adapters, requests, kind, dtype, per_row, op="linear"):
    return {"name": name, "op": op, "rows": rows, "n": n, "k": k, "rank": rank, "adapters": adapters,
            "requests": requests, "kind": kind, "dtype": dtype, "scale_per_row": per_row}


def _clip(name, tensors, kind, rank, layers, total, dtype, max_norm):
    return {"name": name, "op": "clip", "tensors": tensors, "kind": kind, "rank": rank, "layers": layers,
            "total": total, "dtype": dtype, "max_norm": max_norm}


def listed():
    return [
        # one user's next token through a Llama-3-8B k projection: latency alone
        _linear("decode 1, 1024x4096 r16", 1, 1024, 4096, 16, 1, 1, "decode", "bf16", False),
        # a serving batch of single tokens, each request with its own adapter, some without, padded to a batch size
        _linear("decode 32, 4096x4096 r16", 32, 4096, 4096, 16, 24, 29, "decode", "bf16", False),
        # a large batch of single tokens at the widest projection of the Llama-3-70B set
        _linear("decode 200, 28672x8192 r64", 200, 28672, 8192, 64, 12, 200, "decode", "fp16", True),
        # prompts of a few requests, of odd lengths, through a down projection
        _linear("prompts 1777, 4096x14336 r32", 1777, 4096, 14336, 32, 6, 9, "prompts", "bf16", True),
        # long prompts through an up projection: bound by the product
        _linear("prompts 8192, 14336x4096 r16", 8192, 14336, 4096, 16, 4, 5, "prompts", "fp16", False),
        # sizes and rows that no vector load fits (the codec takes tensors of any shape)
        _linear("odd 333, 1001x1999 r12", 333, 1001, 1999, 12, 5, 7, "prompts", "bf16", True),
        # a small fine-tuning step
        _linear("train 256, 1024x4096 r8", 256, 1024, 4096, 8, 1, 1, "prompts", "bf16", False, "backward"),
        # several adapters trained side by side on sequences of their own
        _linear("train 4096, 4096x4096 r16", 4096, 4096, 4096, 16, 4, 8, "prompts", "bf16", False, "backward"),
        # a full batch at a 70B square projection with a large rank
        _linear("train 8192, 8192x8192 r64", 8192, 8192, 8192, 64, 2, 6, "prompts", "fp16", True, "backward"),
        # the adapters of one 8B layer
        _clip("clip 14 tensors, 8B layer", 14, "8b", 16, 1, 0, "bf16", 1.0),
        # the adapters of a whole 8B model
        _clip("clip 448 tensors, 8B", 448, "8b", 16, 32, 0, "bf16", 0.3),
        # the adapters of a 70B model with gradients kept in 32 bits
        _clip("clip 1120 tensors, 70B", 1120, "70b", 16, 80, 0, "fp32", 1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "clip"])
    if op == "clip":
        return {"op": "clip", "tensors": _log_int(rng, 1, 1200), "kind": "ragged", "rank": 0, "layers": 0,
                "total": _log_int(rng, 2_000, 150_000_000), "dtype": rng.choice(["bf16", "fp16", "fp32", "mixed"]),
                "max_norm": rng.choice([0.1, 1.0, 1e6])}
    while True:
        n, k = _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
        if rng.random() < 0.75:
            n, k = -(-n // 16) * 16, -(-k // 16) * 16
        kind = rng.choice(["decode", "prompts"]) if op == "linear" else "prompts"
        rows = _log_int(rng, 1, 256) if kind == "decode" else _log_int(rng, 2, 8192)
        if rows * n * k <= 2.5e11:
            break
    requests = rows - rng.randint(0, rows // 8) if kind == "decode" else rng.randint(1, min(12, rows))
    rank = rng.choice([4, 8, 16, 16, 32, 64, 128, rng.randint(1, 128)])
    most = max(1, min(requests, 2048 // rank, 48))
    return {"op": op, "rows": rows, "n": n, "k": k, "rank": rank, "adapters": rng.randint(1, most),
            "requests": requests, "kind": kind, "dtype": rng.choice(["bf16", "fp16"]),
            "scale_per_row": rng.random() < 0.5}


# ---- inputs ---------------------------------------------------------------

#: (out, in) of the projections of one layer
_SHAPES = {"8b": [(4096, 4096), (1024, 4096), (1024, 4096), (4096, 4096), (14336, 4096), (14336, 4096), (4096, 14336)],
           "70b": [(8192, 8192), (1024, 8192), (1024, 8192), (8192, 8192), (28672, 8192), (28672, 8192), (8192, 28672)]}


def _request_layout(case):
    """offsets (requests + 1) and adapter ids, on the host: a function of the case."""
    r = np.random.default_rng(case["rows"] * 1009 + case["requests"])
    rows, requests = case["rows"], case["requests"]
    if case["kind"] == "decode":
        offsets = np.arange(requests + 1)
    else:
        # odd lengths, empty requests among them where there is more than one; all rows used
        cuts = np.sort(r.integers(0, rows + 1, size=requests - 1))
        offsets = np.concatenate([[0], cuts, [rows]])
    ids = r.integers(0, case["adapters"], size=requests)
    if requests > 3:
        ids[r.integers(0, requests, size=max(1, requests // 10))] = -1
    return offsets.astype(np.int32), ids.astype(np.int32)


def _clip_sizes(case):
    if case["kind"] == "ragged":
        r = np.random.default_rng(case["tensors"] * 7919 + case["total"])
        part = r.dirichlet(np.full(case["tensors"], 0.5))
        sizes = [int(p * case["total"]) for p in part]  # some are empty
        kinds = [case["dtype"]] * len(sizes)
        if case["dtype"] == "mixed":
            kinds = [("bf16", "fp32", "fp16")[i] for i in r.integers(0, 3, size=len(sizes))]
        return sizes, kinds
    sizes = []
    for _ in range(case["layers"]):
        for n, k in _SHAPES[case["kind"]]:
            sizes += [case["rank"] * k, n * case["rank"]]
    return sizes, [case["dtype"]] * len(sizes)


def _prepare_clip(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    sizes, kinds = _clip_sizes(case)
    flat, out, views, outs = {}, {}, [], []
    ragged = case["kind"] == "ragged"
    for kind in sorted(set(kinds)):
        mine = [s for s, q in zip(sizes, kinds) if q == kind]
        # a ragged set lies packed in one buffer, as flattened gradients do; the others start at 256-byte bounds
        at, starts = 0, []
        for s in mine:
            starts.append(at)
            at += s if ragged else -(-s // 128) * 128
        flat[kind] = (torch.randn(max(at, 1), generator=g, device="cuda") * 3e-4).to(DTYPES[kind])
        out[kind] = torch.zeros(max(at, 1), device="cuda", dtype=DTYPES[kind])
        views.append([flat[kind][a:a + s] for a, s in zip(starts, mine)])
        outs.append([out[kind][a:a + s] for a, s in zip(starts, mine)])
    views, outs = sum(views, []), sum(outs, [])
    state = {"case": case, "grads": views, "outs": outs, "flat": flat, "flat_out": out,
             "norm": torch.zeros(1, device="cuda", dtype=torch.float32)}
    if own:
        import lossless_fp8_weight_b200 as L
        state["status"] = torch.zeros(1, device="cuda", dtype=torch.int32)
        state["set"] = L.GradSet(views, outs)
    return state


def prepare(case, seed):
    if case["op"] == "clip":
        return _prepare_clip(case, seed)
    g = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    rows, n, k, rank, adapters = (case[q] for q in ("rows", "n", "k", "rank", "adapters"))
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # the weight as a checkpoint quantised to E4M3 holds it: bytes, and a scale that undoes the stretch to +-448
    w = normal(n, k)
    most = w.abs().amax(dim=1) if case["scale_per_row"] else w.abs().amax().reshape(1)
    w = (w * (448.0 / most).unsqueeze(1)).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = (most / 448.0) * (1.0 / math.sqrt(k))
    offsets, ids = _request_layout(case)
    state = {
        "case": case, "w": w, "scale": scale,
        "x": (normal(rows, k) * torch.exp(0.5 * normal(k))).to(dtype),  # channels of unequal size, as activations have
        "a": (normal(adapters, rank, k) / math.sqrt(k)).to(dtype),
        "b": (normal(adapters, n, rank) * 0.3).to(dtype),
        "alpha": 0.5 + torch.rand(adapters, generator=g, device="cuda"),
        "offsets": torch.from_numpy(offsets).cuda(), "ids": torch.from_numpy(ids).cuda(),
        "last": int(offsets[-1]),
    }
    if case["op"] == "backward":
        state["dy"] = (normal(rows, n) * 0.01).to(dtype)
        # x A_a^T as the forward pass left it
        hot = _hot(state)
        u = state["x"].float() @ state["a"].float().reshape(adapters * rank, k).T
        state["u"] = (u.reshape(rows, adapters, rank) * hot.unsqueeze(2)).sum(dim=1)
        state["dx"] = torch.empty(rows, k, device="cuda", dtype=dtype)
        state["da"] = torch.empty_like(state["a"])
        state["db"] = torch.empty_like(state["b"])
    else:
        state["y"] = torch.empty(rows, n, device="cuda", dtype=dtype)
    if own:
        import lossless_fp8_weight_b200 as L
        state["status"] = torch.zeros(1, device="cuda", dtype=torch.int32)
        state["linear"] = L.Linear(state["w"], scale=state["scale"], dtype=dtype,
                                   adapters=L.Adapters(state["a"], state["b"], state["alpha"]))
        state["requests"] = L.Requests(state["offsets"], state["ids"])
        state["workspace"] = torch.empty(max(16, state["linear"].workspace_size(rows)), device="cuda",
                                         dtype=torch.uint8)
    return state


# ---- one pass -------------------------------------------------------------

def _hot(s):
    """(rows, adapters) with 1 where the row's request uses the adapter."""
    rows = torch.arange(s["case"]["rows"], device="cuda")
    request = torch.searchsorted(s["offsets"].long(), rows, right=True) - 1
    inside = request < s["ids"].numel()
    ids = torch.where(inside, s["ids"][request.clamp(max=s["ids"].numel() - 1)].long(), -1)
    return (ids.unsqueeze(1) == torch.arange(s["case"]["adapters"], device="cuda")).float()


def _plain_linear(s):
    c = s["case"]
    x = s["x"].float()
    w = s["w"].view(torch.float8_e4m3fn).float() * s["scale"].unsqueeze(1)
    a = s["a"].float().reshape(c["adapters"] * c["rank"], c["k"])
    b = s["b"].float().permute(1, 0, 2).reshape(c["n"], c["adapters"] * c["rank"])
    u = (x @ a.T).reshape(c["rows"], c["adapters"], c["rank"]) * (_hot(s) * s["alpha"]).unsqueeze(2)
    y = x @ w.T + u.reshape(c["rows"], -1) @ b.T
    return y.to(s["x"].dtype)


def _plain_backward(s):
    c = s["case"]
    x, dy = s["x"].float(), s["dy"].float()
    w = s["w"].view(torch.float8_e4m3fn).float() * s["scale"].unsqueeze(1)
    a = s["a"].float().reshape(c["adapters"] * c["rank"], c["k"])
    b = s["b"].float().permute(1, 0, 2).reshape(c["n"], c["adapters"] * c["rank"])
    hot = (_hot(s) * s["alpha"]).unsqueeze(2)
    v = ((dy @ b).reshape(c["rows"], c["adapters"], c["rank"]) * hot).reshape(c["rows"], -1)
    u = (s["u"].unsqueeze(1) * hot).reshape(c["rows"], -1)
    dx = dy @ w + v @ a
    da = (v.T @ x).reshape(c["adapters"], c["rank"], c["k"])
    db = (dy.T @ u).reshape(c["n"], c["adapters"], c["rank"]).permute(1, 0, 2).contiguous()
    dtype = s["x"].dtype
    return {"dx": dx.to(dtype), "da": da.to(dtype), "db": db.to(dtype)}


def _plain_clip(s):
    total = torch.stack([f.double().square().sum() for f in s["flat"].values()]).sum()
    norm = total.sqrt()
    factor = (s["case"]["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float().reshape(1), **{k: (f.float() * factor).to(f.dtype) for k, f in s["flat"].items()}}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"linear": _plain_linear, "backward": _plain_backward, "clip": _plain_clip}[op](state)
    if op == "clip":
        state["set"].clip(state["case"]["max_norm"], state["norm"], status=state["status"])
        return {"norm": state["norm"], **state["flat_out"]}
    if op == "linear":
        state["linear"].forward(state["x"], state["y"], requests=state["requests"], workspace=state["workspace"],
                                status=state["status"])
        return state["y"]
    state["linear"].backward(state["x"], state["dy"], state["u"], dx=state["dx"], da=state["da"], db=state["db"],
                             requests=state["requests"], workspace=state["workspace"], status=state["status"])
    return {"dx": state["dx"], "da": state["da"], "db": state["db"]}


# ---- the definition in 64 bits --------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float((v.double() ** 2).sum()) for v in s["grads"]))
        factor = min(1.0, case["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
                **{k: f.double() * factor for k, f in s["flat"].items()}}
    wide = {q: s[q].double() for q in ("x", "a", "b", "scale", "alpha")}
    w = s["w"].view(torch.float8_e4m3fn).double()
    at, ids = s["offsets"].tolist(), s["ids"].tolist()
    runs = [(lo, hi, i) for lo, hi, i in zip(at, at[1:], ids) if hi > lo and i >= 0]
    if case["op"] == "linear":
        y = (wide["x"] @ w.T) * wide["scale"]
        for lo, hi, i in runs:
            y[lo:hi] += wide["alpha"][i] * ((wide["x"][lo:hi] @ wide["a"][i].T) @ wide["b"][i].T)
        return y
    dy, u = s["dy"].double(), s["u"].double()
    dx = (dy * wide["scale"]) @ w
    da, db = torch.zeros_like(wide["a"]), torch.zeros_like(wide["b"])
    for lo, hi, i in runs:
        v = wide["alpha"][i] * (dy[lo:hi] @ wide["b"][i])
        dx[lo:hi] += v @ wide["a"][i]
        da[i] += v.T @ wide["x"][lo:hi]
        db[i] += wide["alpha"][i] * (dy[lo:hi].T @ u[lo:hi])
    return {"dx": dx, "da": da, "db": db}


def work(case):
    """Each input read once, each output written once; products at two operations a term."""
    if case["op"] == "clip":
        sizes, kinds = _clip_sizes(case)
        size = {"bf16": 2, "fp16": 2, "fp32": 4}
        return {"bytes": 2 * sum(s * size[q] for s, q in zip(sizes, kinds)) + 4, "flops": 3 * sum(sizes)}
    rows, n, k, rank = (case[q] for q in ("rows", "n", "k", "rank"))
    offsets, ids = _request_layout(case)
    lengths = np.diff(offsets)
    used = len({int(i) for i, ln in zip(ids, lengths) if i >= 0 and ln > 0})
    adapted = int(lengths[ids >= 0].sum())
    scale = 4 * (n if case["scale_per_row"] else 1)
    index = 4 * (2 * len(ids) + 1) + 4 * used
    factors = 2 * used * rank * (n + k)
    if case["op"] == "linear":
        return {"bytes": n * k + scale + index + 2 * rows * (n + k) + factors,
                "flops": 2 * rows * n * k + 2 * adapted * rank * (n + k)}
    return {"bytes": n * k + scale + index + 2 * rows * (n + 2 * k) + factors + 4 * adapted * rank
            + 2 * case["adapters"] * rank * (n + k),
            "flops": 2 * rows * n * k + 4 * adapted * rank * (n + k)}
