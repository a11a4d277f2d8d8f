"""Cases of the token-order and adapter operators, for measuring and comparing them.

Six operators that surround the experts of a mixture-of-experts layer:

* ``dispatch``: tokens sorted by expert.  ids [T, k] name the picked experts (-1: no pick).  The valid
  picks p = t*k + j, ordered by (expert, p), become rows: offsets [E+1] bounds each expert's rows,
  pos[t, j] is the row of a pick (-1), src[row] its pick and expert[row] its expert (-1 behind the
  last row), rows[pos[t, j]] = x[t].  Rows behind the last stay as they were.
* ``dispatch_backward``: d_x[t] = sum_j d_rows[pos[t, j]].
* ``combine``: out[t] = base[t] + sum_j gate[t, j] rows[pos[t, j]] over the valid picks.
* ``combine_backward``: d_rows[pos[t, j]] = gate[t, j] d_out[t], d_gate[t, j] = <d_out[t], rows[pos[t, j]]>
  (0 for no pick).
* ``adapters``: out[i] = base[i] + scale[e] B_e (A_e x[i]) with e = adapter[i] (-1: no adapter),
  A [n, r, inner], B [n, outer, r].
* ``adapters_backward``: with u = scale[e] B_e^T d_out[i] and v = A_e x[i]: d_x[i] = dx_base[i] + A_e^T u,
  d_A[e] = sum_i u x[i]^T, d_B[e] = scale[e] sum_i d_out[i] v^T (both fp32).

``own`` chooses between the plain form in torch and the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
TOKEN_OPS = ("dispatch", "dispatch_backward", "combine", "combine_backward")


def listed():
    def tokens(name, op, T, k, E, H, dtype, base=False, drop=0.0):
        return dict(name=name, op=op, T=T, k=k, E=E, H=H, dtype=dtype, base=base, drop=drop)

    def adapters(name, op, T, n, r, inner, outer, dtype, wtype, order):
        return dict(name=name, op=op, T=T, n=n, r=r, inner=inner, outer=outer, dtype=dtype, wtype=wtype, order=order)

    return [
        # one decoded token of the Qwen3-30B-A3B shape: the latency of a call
        tokens("dispatch one token", "dispatch", 1, 8, 128, 2048, "f32"),
        # a long prompt (four of 2048 tokens packed) before the experts' products
        tokens("dispatch 8192", "dispatch", 8192, 8, 128, 2048, "bf16"),
        # odd sizes: rows that no 16-byte load fits, picks dropped by a capacity limit
        tokens("dispatch back odd", "dispatch_backward", 777, 6, 60, 1001, "f16", drop=0.05),
        # a training micro-batch with fp32 activations, as the layer itself has them
        tokens("dispatch back 4096", "dispatch_backward", 4096, 8, 128, 2048, "f32"),
        # four requests decoded together, the residual added
        tokens("combine four tokens", "combine", 4, 8, 128, 2048, "f32", base=True),
        # two packed prompts, some picks dropped
        tokens("combine 4096", "combine", 4096, 8, 128, 2048, "bf16", base=True, drop=0.06),
        # a small model's training step with few picks a token
        tokens("combine back ragged", "combine_backward", 333, 3, 16, 770, "bf16", drop=0.1),
        # the large training micro-batch
        tokens("combine back 8192", "combine_backward", 8192, 8, 128, 2048, "bf16"),
        # 32 requests decoded together (the layer's largest decode call), each with its adapter, on fp32 activations
        adapters("adapters decode 32", "adapters", 32, 64, 16, 2048, 2048, "f32", "bf16", "mixed"),
        # the packed prompts of several requests
        adapters("adapters 8192", "adapters", 8192, 8, 16, 2048, 2048, "bf16", "bf16", "runs"),
        # a short fine-tuning step in fp32 on a projection of another width
        adapters("adapters back 300", "adapters_backward", 300, 3, 8, 768, 2048, "f32", "f32", "runs"),
        # a large fine-tuning micro-batch
        adapters("adapters back 16384", "adapters_backward", 16384, 4, 32, 2048, 2048, "bf16", "bf16", "runs"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(TOKEN_OPS + ("adapters", "adapters_backward"))
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op in TOKEN_OPS:
        E = _spread(rng, 4, 512)
        k = rng.randint(1, min(10, E))
        H = _spread(rng, 64, 6144)
        if rng.random() < 0.7:
            H = max(64, H // 32 * 32)
        most = max(1, (8192 * 8 * 2048 * 2 // SIZE[dtype] // (k * H)) * 7 // 10)
        T = _spread(rng, 1, min(32768, most))
        return dict(op=op, T=T, k=k, E=E, H=H, dtype=dtype, base=rng.random() < 0.5,
                    drop=rng.choice([0.0, 0.0, 0.03, 0.3]))
    r = rng.choice([4, 8, 8, 16, 16, 32, 64, 12, 5])
    n = _spread(rng, 1, 48)
    inner, outer = _spread(rng, 128, 6144), _spread(rng, 128, 6144)
    if rng.random() < 0.8:
        inner, outer = max(128, inner // 64 * 64), max(128, outer // 64 * 64)
    most = 16384 * 4096 * 2 * 7 // 10 // SIZE[dtype] // (inner + outer)
    T = _spread(rng, 1, max(1, min(16384, most, (1 << 25) // (n * r))))
    wtype = rng.choice(["f16", "bf16", "f32"]) if dtype == "f32" else dtype
    # a short call mixes its requests' rows; in a long one each request's rows follow each other
    return dict(op=op, T=T, n=n, r=r, inner=inner, outer=outer, dtype=dtype, wtype=wtype,
                order="mixed" if T <= 128 else "runs")


# ------------------------------------------------------------------------------------------ inputs

def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _order(ids, E):
    """The order of the valid picks: offsets, pos, src, expert (stable in the pick's number)."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    sorted_key, src = torch.sort(key, stable=True)
    rank = torch.empty_like(src)
    rank[src] = torch.arange(T * k, device=ids.device)
    offsets = torch.searchsorted(sorted_key, torch.arange(E + 1, device=ids.device))
    valid = sorted_key < E
    pos = torch.where(flat < 0, -1, rank).reshape(T, k)
    return (offsets.int(), pos.int(), torch.where(valid, src, -1).int(), torch.where(valid, sorted_key, -1).int())


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] in TOKEN_OPS:
        T, k, E, H = c["T"], c["k"], c["E"], c["H"]
        # a router's logits: some experts are picked far more often than others
        logits = torch.randn((T, E), generator=g, device="cuda") + torch.randn((1, E), generator=g, device="cuda")
        top, ids = torch.topk(torch.softmax(logits, -1), k, dim=-1)
        if c["drop"]:
            ids = torch.where(torch.rand((T, k), generator=g, device="cuda") < c["drop"], -1, ids)
        s["ids"], s["gate"] = ids.int().contiguous(), top.float().contiguous()
        i32 = dict(dtype=torch.int32, device="cuda")
        if c["op"] == "dispatch":
            s["x"] = _normal(g, (T, H), dtype)
            s["rows"] = torch.zeros((T * k, H), dtype=dtype, device="cuda")
            s["offsets"], s["pos"] = torch.zeros(E + 1, **i32), torch.zeros((T, k), **i32)
            s["src"], s["expert"] = torch.zeros(T * k, **i32), torch.zeros(T * k, **i32)
            return s
        s["pos"] = _order(s["ids"], E)[1]
        if c["op"] == "dispatch_backward":
            s["d_rows"] = _normal(g, (T * k, H), dtype)
            s["d_x"] = torch.zeros((T, H), dtype=dtype, device="cuda")
        else:
            s["rows"] = _normal(g, (T * k, H), dtype)
            if c["op"] == "combine":
                s["base"] = _normal(g, (T, H), dtype) if c["base"] else None
                s["out"] = torch.zeros((T, H), dtype=dtype, device="cuda")
            else:
                s["d_out"] = _normal(g, (T, H), dtype)
                s["d_rows"] = torch.zeros((T * k, H), dtype=dtype, device="cuda")
                s["d_gate"] = torch.zeros((T, k), dtype=torch.float32, device="cuda")
        return s
    T, n, r, inner, outer = c["T"], c["n"], c["r"], c["inner"], c["outer"]
    wtype = DTYPES[c["wtype"]]
    at = torch.randint(0, n + 1, (T,), generator=g, device="cuda") if c["order"] == "mixed" else None
    if at is None:
        # n+1 runs of uneven lengths, one of them of rows without an adapter
        cuts = torch.sort(torch.randint(0, T + 1, (n,), generator=g, device="cuda"))[0]
        at = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
    s["adapter"] = torch.where(at == n, -1, at).int().contiguous()
    s["a"] = _normal(g, (n, r, inner), wtype, inner ** -0.5)
    s["b"] = _normal(g, (n, outer, r), wtype, r ** -0.5)
    s["scale"] = 0.25 + torch.rand(n, generator=g, device="cuda")
    s["x"] = _normal(g, (T, inner), dtype)
    if c["op"] == "adapters":
        s["base"] = _normal(g, (T, outer), dtype)
        s["out"] = torch.zeros((T, outer), dtype=dtype, device="cuda")
    else:
        s["d_out"] = _normal(g, (T, outer), dtype)
        s["dx_base"] = _normal(g, (T, inner), dtype)
        s["d_x"] = torch.zeros((T, inner), dtype=dtype, device="cuda")
        s["d_a"] = torch.zeros((n, r, inner), device="cuda")
        s["d_b"] = torch.zeros((n, outer, r), device="cuda")
    return s


# -------------------------------------------------------------------------------------- plain forms

def _plain_dispatch(s):
    offsets, pos, src, expert = _order(s["ids"], s["case"]["E"])
    rows, k = s["rows"], s["case"]["k"]
    token = src.long().clamp(min=0) // k
    rows = torch.where((src >= 0)[:, None], s["x"][token], rows)
    return {"rows": rows, "offsets": offsets, "pos": pos, "src": src, "expert": expert}


def _plain_weighted(rows, pos, gate, base, dtype):
    T, k = pos.shape
    ok = pos >= 0
    picked = rows[pos.long().clamp(min=0)].float()
    picked = torch.where(ok[:, :, None], picked if gate is None else picked * gate[:, :, None], 0.0)
    out = picked.sum(1)
    return (out if base is None else base.float() + out).to(dtype)


def _plain_combine_backward(s):
    pos, gate, rows = s["pos"], s["gate"], s["rows"]
    T, k = pos.shape
    ok, at = pos >= 0, pos.long().clamp(min=0)
    d_out = s["d_out"].float()
    d_gate = torch.where(ok, (rows[at].float() * d_out[:, None, :]).sum(-1), 0.0)
    flat = ok.reshape(-1)
    d_rows = s["d_rows"].clone()
    grads = (gate[:, :, None] * d_out[:, None, :]).to(rows.dtype).reshape(T * k, -1)
    d_rows[pos.reshape(-1)[flat].long()] = grads[flat]
    return {"d_rows": d_rows, "d_gate": d_gate}


def _one_hot(s):
    n = s["a"].shape[0]
    return (s["adapter"].long()[:, None] == torch.arange(n, device="cuda")).float()


def _plain_adapters(s):
    n, r, inner = s["a"].shape
    outer, T = s["b"].shape[1], s["x"].shape[0]
    x = s["x"].float()
    if T <= 64:   # few rows: each row's matrices picked out
        at = s["adapter"].long().clamp(min=0)
        v = (s["a"][at].float() * x[:, None, :]).sum(-1)
        delta = (s["b"][at].float() * v[:, None, :]).sum(-1) * s["scale"][at][:, None]
        delta = torch.where((s["adapter"] >= 0)[:, None], delta, 0.0)
    else:         # all adapters side by side, each row's own kept
        v = (x @ s["a"].float().reshape(n * r, inner).T).reshape(T, n, r)
        v = v * (_one_hot(s) * s["scale"])[:, :, None]
        delta = v.reshape(T, n * r) @ s["b"].float().transpose(1, 2).reshape(n * r, outer)
    return {"out": (s["base"].float() + delta).to(s["x"].dtype)}


def _plain_adapters_backward(s):
    n, r, inner = s["a"].shape
    outer, T = s["b"].shape[1], s["x"].shape[0]
    x, d_out = s["x"].float(), s["d_out"].float()
    a = s["a"].float().reshape(n * r, inner)
    b = s["b"].float().transpose(1, 2).reshape(n * r, outer)
    mine = (_one_hot(s) * s["scale"])[:, :, None]
    v = ((x @ a.T).reshape(T, n, r) * mine).reshape(T, n * r)
    u = ((d_out @ b.T).reshape(T, n, r) * mine).reshape(T, n * r)
    return {"d_x": (s["dx_base"].float() + u @ a).to(s["x"].dtype),
            "d_a": (u.T @ x).reshape(n, r, inner),
            "d_b": (v.T @ d_out).reshape(n, r, outer).transpose(1, 2).contiguous()}


def _plain(s):
    op = s["case"]["op"]
    if op == "dispatch":
        return _plain_dispatch(s)
    if op == "dispatch_backward":
        return {"d_x": _plain_weighted(s["d_rows"], s["pos"], None, None, s["d_rows"].dtype)}
    if op == "combine":
        return {"out": _plain_weighted(s["rows"], s["pos"], s["gate"], s["base"], s["rows"].dtype)}
    if op == "combine_backward":
        return _plain_combine_backward(s)
    return _plain_adapters(s) if op == "adapters" else _plain_adapters_backward(s)


# ------------------------------------------------------------------------------------ library calls

def _own(s):
    import expert_offload_lru_amd as moe
    op = s["case"]["op"]
    if op == "dispatch":
        moe.tokens_dispatch(s["x"], s["ids"], s["case"]["E"], s["rows"], s["offsets"], s["pos"], s["src"], s["expert"])
        return {n: s[n] for n in ("rows", "offsets", "pos", "src", "expert")}
    if op == "dispatch_backward":
        moe.tokens_dispatch_backward(s["d_rows"], s["pos"], s["d_x"])
        return {"d_x": s["d_x"]}
    if op == "combine":
        moe.tokens_combine(s["rows"], s["pos"], s["gate"], s["out"], base=s["base"])
        return {"out": s["out"]}
    if op == "combine_backward":
        moe.tokens_combine_backward(s["d_out"], s["rows"], s["pos"], s["gate"], s["d_rows"], s["d_gate"])
        return {"d_rows": s["d_rows"], "d_gate": s["d_gate"]}
    if op == "adapters":
        moe.adapters_forward(s["x"], s["adapter"], s["a"], s["b"], s["scale"], s["out"], base=s["base"])
        return {"out": s["out"]}
    moe.adapters_backward(s["d_out"], s["x"], s["adapter"], s["a"], s["b"], s["scale"], s["d_x"], s["d_a"], s["d_b"],
                          dx_base=s["dx_base"])
    return {"d_x": s["d_x"], "d_a": s["d_a"], "d_b": s["d_b"]}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------------------------- work

def work(case):
    c, z = case, SIZE[case["dtype"]]
    if c["op"] in TOKEN_OPS:
        T, k, E, H = c["T"], c["k"], c["E"], c["H"]
        P, picks = T * k * (1 - c["drop"]), T * k
        if c["op"] == "dispatch":
            return {"bytes": z * H * (T + P) + 4 * (4 * picks + E + 1), "flops": 0}
        if c["op"] == "dispatch_backward":
            return {"bytes": z * H * (T + P) + 4 * picks, "flops": P * H}
        if c["op"] == "combine":
            return {"bytes": z * H * (T + P + (T if c["base"] else 0)) + 8 * picks, "flops": 2 * P * H}
        return {"bytes": z * H * (T + 2 * P) + 12 * picks, "flops": 3 * P * H}
    T, n, r, inner, outer = (c[m] for m in ("T", "n", "r", "inner", "outer"))
    used = min(n, T)   # adapters that rows name, at most
    weights = used * r * (inner + outer) * SIZE[c["wtype"]] + 4 * (T + used)
    if c["op"] == "adapters":
        return {"bytes": z * T * (inner + 2 * outer) + weights, "flops": 2 * T * r * (inner + outer)}
    return {"bytes": z * T * (3 * inner + outer) + weights + 4 * n * r * (inner + outer),
            "flops": 6 * T * r * (inner + outer)}


# -------------------------------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        ids, x = s["ids"].cpu().numpy(), s["x"].double()
        T, k = ids.shape
        picks = [np.flatnonzero(ids.reshape(-1) == e) for e in range(case["E"])]
        order = np.concatenate(picks).astype(np.int64)
        offsets = np.concatenate([[0], np.cumsum([len(p) for p in picks])]).astype(np.int32)
        m = len(order)
        pos, src, expert = (np.full(T * k, -1, dtype=np.int32) for _ in range(3))
        pos[order] = np.arange(m)
        src[:m] = order
        expert[:m] = ids.reshape(-1)[order]
        rows = s["rows"].double()
        rows[:m] = x[torch.from_numpy(order // k).cuda()]
        return {"rows": rows, "offsets": offsets, "pos": pos.reshape(T, k), "src": src, "expert": expert}
    if op in ("dispatch_backward", "combine"):
        rows = s["d_rows" if op == "dispatch_backward" else "rows"]
        T, k = s["pos"].shape
        weight = torch.ones((T, k), dtype=torch.float64, device="cuda") if op != "combine" else s["gate"].double()
        base = s.get("base")
        out = torch.zeros((T, rows.shape[1]), dtype=torch.float64, device="cuda") if base is None else base.double()
        for j in range(k):
            at = torch.nonzero(s["pos"][:, j] >= 0)[:, 0]
            out[at] += weight[at, j, None] * rows[s["pos"][at, j].long()].double()
        return {"out" if op == "combine" else "d_x": out}
    if op == "combine_backward":
        T, k = s["pos"].shape
        d_rows = s["d_rows"].double()
        d_gate = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        d_out = s["d_out"].double()
        for j in range(k):
            at = torch.nonzero(s["pos"][:, j] >= 0)[:, 0]
            to = s["pos"][at, j].long()
            d_gate[at, j] = torch.linalg.vecdot(d_out[at], s["rows"][to].double())
            d_rows[to] = s["gate"][at, j, None].double() * d_out[at]
        return {"d_rows": d_rows, "d_gate": d_gate}
    x, a, b = s["x"].double(), s["a"].double(), s["b"].double()
    scale, which = s["scale"].double().tolist(), s["adapter"]
    if op == "adapters":
        out = s["base"].double()
        for e in range(case["n"]):
            at = torch.nonzero(which == e)[:, 0]
            out[at] += scale[e] * ((x[at] @ a[e].T.contiguous()) @ b[e].T.contiguous())
        return {"out": out}
    d_out, d_x = s["d_out"].double(), s["dx_base"].double()
    d_a, d_b = torch.zeros_like(a), torch.zeros_like(b)
    for e in range(case["n"]):
        at = torch.nonzero(which == e)[:, 0]
        v = x[at] @ a[e].T.contiguous()
        u = scale[e] * (d_out[at] @ b[e])
        d_x[at] += u @ a[e]
        d_a[e] = u.T.contiguous() @ x[at]
        d_b[e] = scale[e] * (d_out[at].T.contiguous() @ v)
    return {"d_x": d_x, "d_a": d_a, "d_b": d_b}
