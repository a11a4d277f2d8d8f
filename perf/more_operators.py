"""Cases of the experts' feed-forward, 8-bit row and block-norm operators, for measuring and comparing them.

Rows are sorted by expert: rows offsets[e] .. offsets[e+1] are expert e's; rows outside stay as they were.

* ``hidden``: w [E, 2I, H] holds an expert's gate rows, then its up rows.  g = w[:I] x, u = w[I:] x,
  hidden = act(g) u.  ``keep``: the pre-activations [g, u] too, in the type or in 8 bits.
* ``hidden_backward``: from d_out [R, H], the down projection w [E, H, I] and the kept [g, u]:
  d_h = w^T d_out, d_pre = [d_h u act'(g), d_h act(g)], and hidden again for the down projection's gradient.
* ``product``: out = w_e x, w [E, outer, inner].
* ``product_backward``: d_x = w_e^T d_out, d_w[e] = sum of d_out x^T over e's rows (fp32); x may be kept in 8 bits.
* ``encode``: a matrix kept in 8 bits and read back.  A block of 32 columns (the last one shorter) has the
  scale 2^e, e the least for which the block's largest size over 2^e rounds to 127 or less, and holds
  whole numbers x / 2^e rounded to nearest, ties to even.
* ``norm``: out = alpha x + gate (w_post y r_y), normed = w_pre out r_out, with r the inverse root of a
  row's mean square; rows_per_gate rows share a row of gate.
* ``norm_backward``: its gradients from those of out and normed.

``own`` chooses between the plain form in torch and the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32
EPS = 1e-6


def listed():
    def experts(name, op, T, k, E, inner, outer, dtype, keep="none", act="silu", drop=0.0):
        return dict(name=name, op=op, T=T, k=k, E=E, inner=inner, outer=outer, dtype=dtype, keep=keep, act=act, drop=drop)

    def norm(name, op, T, H, dtype, post=True, gate=0, alpha=False, pre=True):
        return dict(name=name, op=op, T=T, H=H, dtype=dtype, post=post, gate=gate, alpha=alpha, pre=pre)

    return [
        # one decoded token of the Qwen3-30B-A3B shape: eight experts' gate and up rows are read
        experts("hidden one token", "hidden", 1, 8, 128, 2048, 768, "bf16"),
        # a training micro-batch of 8192 tokens, what the backward pass needs kept in 8 bits
        experts("hidden 65536 kept in 8 bits", "hidden", 8192, 8, 128, 2048, 768, "bf16", keep="8 bits"),
        # a small model's step with odd sizes, picks dropped by a capacity limit; inner is the block's hidden width
        experts("hidden back odd", "hidden_backward", 333, 3, 16, 770, 333, "f16", keep="type", act="gelu", drop=0.1),
        # the backward pass of the large micro-batch
        experts("hidden back 65536", "hidden_backward", 8192, 8, 128, 2048, 768, "bf16", keep="8 bits"),
        # 32 requests decoded together: the down projection of the experts that they pick
        experts("product decode 32", "product", 32, 8, 128, 768, 2048, "bf16"),
        # a short fine-tuning step in fp32
        experts("product back f32", "product_backward", 667, 3, 8, 770, 1001, "f32"),
        # a dense block's gate and up projections over four prompts of 2048 tokens, the input kept in 8 bits
        experts("product back dense", "product_backward", 8192, 1, 1, 2048, 1536, "bf16", keep="8 bits"),
        # a few rows of odd length
        dict(name="encode 59 odd", op="encode", T=59, H=1001, dtype="f32"),
        # the dispatched rows of the large micro-batch
        dict(name="encode 65536", op="encode", T=65536, H=2048, dtype="bf16"),
        # one decoded token: the norm after one block and before the next
        norm("norm one token", "norm", 1, 2048, "bf16"),
        # four packed prompts, each with a gate of its own (2048 rows a gate), and a learned residual scale
        norm("norm 8192", "norm", 8192, 2048, "bf16", gate=2048, alpha=True),
        # the large training micro-batch, every parameter with its gradient; one gate for all rows
        norm("norm back 16384", "norm_backward", 16384, 2048, "bf16", gate=16384, alpha=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["hidden", "hidden_backward", "product", "product_backward", "encode", "norm", "norm_backward"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "encode" or op.startswith("norm"):
        H = _spread(rng, 64, 8192)
        if rng.random() < 0.7:
            H = max(64, H // 32 * 32)
        T = _spread(rng, 1, min(65536, (1 << 25) // H))
        if op == "encode":
            return dict(op=op, T=T, H=H, dtype=dtype)
        post = rng.random() < 0.8
        pre = not post or rng.random() < 0.8
        return dict(op=op, T=T, H=H, dtype=dtype, post=post, gate=rng.choice([0, T, max(1, T // 3), min(T, 512)]),
                    alpha=rng.random() < 0.5, pre=pre)
    E = _spread(rng, 1, 128)
    k = rng.randint(1, min(8, E))
    inner, outer = _spread(rng, 64, 4096), _spread(rng, 64, 4096)
    if rng.random() < 0.7:
        inner, outer = max(64, inner // 64 * 64), max(64, outer // 64 * 64)
    # fp32 products run at a sixteenth of the 16-bit types' rate; weights of all experts stay under 0.4 GB
    E = max(k, min(E, (400 << 20) // (inner * outer * 2 * SIZE[dtype])))
    most = min(65536, (60 << 30) // (inner * outer) // (8 if dtype == "f32" else 1), (120 << 20) // max(inner, outer))
    T = _spread(rng, 1, max(2, most // k))
    keep = {"hidden": ["none", "type", "8 bits"], "hidden_backward": ["type", "8 bits"], "product": ["none"],
            "product_backward": ["none", "8 bits"]}[op]
    if op == "hidden" and dtype == "f32":
        keep = ["none", "type"]
    return dict(op=op, T=T, k=k, E=E, inner=inner, outer=outer, dtype=dtype, keep=rng.choice(keep),
                act=rng.choice(["silu", "gelu"]), drop=rng.choice([0.0, 0.0, 0.1]))


# ------------------------------------------------------------------------------------------ inputs

def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _two_to(e):
    """2^e without a rounding, in 64 bits (borders between whole numbers hang on it)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _encode(x):
    """Whole numbers (as floats) and exponents of the blocks of x."""
    T, H = x.shape
    nb = -(-H // BLOCK)
    v = torch.zeros((T, nb * BLOCK), device=x.device)
    v[:, :H] = x.float()
    v = v.reshape(T, nb, BLOCK)
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax)[1] - 7
    e = torch.where(torch.round(amax * _two_to(-e)) > 127, e + 1, e).clamp(-133, 121)
    return torch.round(v * _two_to(-e)).float(), e


def _kept(x):
    """x in 8 bits: codes int8 [T, H] and scales uint8 [T, blocks], 2^(scale - 133)."""
    q, e = _encode(x)
    T, H = x.shape
    return q.reshape(T, -1)[:, :H].to(torch.int8).contiguous(), (e[:, :, 0] + 133).to(torch.uint8).contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[c["dtype"]]
    new = dict(dtype=dtype, device="cuda")
    s = {"case": c}
    if c["op"] == "encode":
        # activations: some channels are far larger than others
        T, H = c["T"], c["H"]
        s["x"] = _normal(g, (T, H), torch.float32).mul_(torch.exp(torch.randn(H, generator=g, device="cuda"))).to(dtype)
        s["codes"] = torch.zeros((T, H), dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros((T, -(-H // BLOCK)), dtype=torch.uint8, device="cuda")
        s["out"] = torch.zeros((T, H), **new)
        return s
    if c["op"] in ("norm", "norm_backward"):
        T, H = c["T"], c["H"]
        s["x"] = _normal(g, (T, H), dtype, 2.0)
        s["y"] = _normal(g, (T, H), dtype)
        near_one = lambda: 1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")  # noqa: E731
        s["w_post"] = near_one() if c["post"] else None
        s["w_pre"] = near_one() if c["pre"] else None
        s["alpha"] = near_one() if c["alpha"] else None
        s["gate"] = 0.5 * torch.randn((-(-T // c["gate"]), H), generator=g, device="cuda") if c["gate"] else None
        s["stats"] = torch.zeros((T, 2), device="cuda")
        if c["op"] == "norm":
            s["out"] = torch.zeros((T, H), **new)
            s["normed"] = torch.zeros((T, H), **new) if c["pre"] else None
            return s
        _, s["stats"][:, 0], s["stats"][:, 1] = _norm_parts(s)[1:]
        s["d_out"] = _normal(g, (T, H), dtype)
        s["d_normed"] = _normal(g, (T, H), dtype) if c["pre"] else None
        s["d_x"], s["d_y"] = torch.zeros((T, H), **new), torch.zeros((T, H), **new)
        for n in ("w_post", "w_pre", "alpha", "gate"):
            s["d_" + n] = None if s[n] is None else torch.zeros_like(s[n])
        return s
    T, k, E, inner, outer = (c[n] for n in ("T", "k", "E", "inner", "outer"))
    R = T * k
    # a trained router's load: nearly even
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.1 * torch.randn((1, E), generator=g, device="cuda")
    ids = torch.topk(logits, k, dim=-1)[1]
    if c["drop"]:
        ids = torch.where(torch.rand((T, k), generator=g, device="cuda") < c["drop"], E, ids)
    counts = torch.bincount(ids.reshape(-1), minlength=E + 1)[:E]
    s["offsets"] = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).int().contiguous()
    s["most"] = int(counts.max())   # the program's capacity of an expert, for the plain form's layout
    if c["op"] == "hidden":
        s["x"] = _normal(g, (R, inner), dtype)
        s["w"] = _normal(g, (E, 2 * outer, inner), dtype, inner ** -0.5)
        s["hidden"] = torch.zeros((R, outer), **new)
        if c["keep"] != "none":
            s["pre"] = torch.zeros((R, 2 * outer), **new)
        if c["keep"] == "8 bits":
            s["codes"] = torch.zeros((R, 2 * outer), dtype=torch.int8, device="cuda")
            s["scales"] = torch.zeros((R, 2 * -(-outer // BLOCK)), dtype=torch.uint8, device="cuda")
        return s
    s["w"] = _normal(g, (E, inner, outer) if c["op"] == "hidden_backward" else (E, outer, inner), dtype, inner ** -0.5)
    if c["op"] == "hidden_backward":
        s["d_out"] = _normal(g, (R, inner), dtype)
        pre = _normal(g, (R, 2 * outer), dtype)
        if c["keep"] == "8 bits":
            halves = [_kept(h) for h in (pre[:, :outer], pre[:, outer:])]
            s["codes"], s["scales"] = (torch.cat(h, 1).contiguous() for h in zip(*halves))
        else:
            s["pre"] = pre
        s["d_pre"], s["hidden"] = torch.zeros((R, 2 * outer), **new), torch.zeros((R, outer), **new)
        return s
    x = _normal(g, (R, inner), dtype)
    if c["op"] == "product":
        s["x"], s["out"] = x, torch.zeros((R, outer), **new)
        return s
    if c["keep"] == "8 bits":
        s["codes"], s["scales"] = _kept(x)
    else:
        s["x"] = x
    s["d_out"] = _normal(g, (R, outer), dtype)
    s["d_x"], s["d_w"] = torch.zeros((R, inner), **new), torch.zeros((E, outer, inner), device="cuda")
    return s


# -------------------------------------------------------------------------------------- plain forms

def _decode(codes, scales):
    """The values of rows kept in 8 bits, fp32."""
    T, H = codes.shape
    wide = torch.repeat_interleave(scales.int() - 133, BLOCK, dim=1)[:, :H]
    return (codes * _two_to(wide)).float()


def _halves(codes, scales):
    I, nb = codes.shape[1] // 2, scales.shape[1] // 2
    return _decode(codes[:, :I], scales[:, :nb]), _decode(codes[:, I:], scales[:, nb:])


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))


def _act_slope(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return p * (1 + g * (1 - p))
    t = torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * g * g)


def _place(s, R):
    """Each row's expert and its place in the layout [experts, most rows of one]; rows of no expert go behind it."""
    off = s["offsets"].long()
    E, M = off.shape[0] - 1, s["most"]
    row = torch.arange(R, device=off.device)
    expert = (torch.searchsorted(off, row, right=True) - 1).clamp(0, E - 1)
    mine = (row >= off[0]) & (row < off[-1])
    return expert, torch.where(mine, expert * M + row - off[expert], E * M), mine


def _spread_rows(x, slot, E, M):
    p = torch.zeros((E * M + 1, x.shape[1]), device=x.device)
    p[slot] = x
    return p[:E * M].reshape(E, M, -1)


def _rows_product(s, x, w):
    """Row i times its expert's matrix w [E, inner, outer], fp32; rows of no expert are undefined."""
    R, (E, inner, outer) = x.shape[0], w.shape
    expert, slot, _ = _place(s, R)
    if R <= 64:   # few rows: each row's matrix picked out
        return (w[expert].float() * x[:, :, None]).sum(1)
    out = torch.bmm(_spread_rows(x, slot, E, s["most"]), w.float().contiguous())
    return torch.cat([out.reshape(-1, outer), out.new_zeros(1, outer)])[slot]


def _rows_product_t(s, x, w):
    """The same with w [E, outer, inner]."""
    R, (E, outer, inner) = x.shape[0], w.shape
    expert, slot, _ = _place(s, R)
    if R <= 64:
        return (w[expert].float() * x[:, None, :]).sum(-1)
    out = torch.bmm(_spread_rows(x, slot, E, s["most"]), w.float().transpose(1, 2).contiguous())
    return torch.cat([out.reshape(-1, outer), out.new_zeros(1, outer)])[slot]


def _keep_others(s, new, old):
    mine = _place(s, new.shape[0])[2]
    return torch.where(mine[:, None], new.to(old.dtype), old)


def _plain_hidden(s):
    c = s["case"]
    pre = _rows_product_t(s, s["x"].float(), s["w"])
    g, u = pre[:, :c["outer"]], pre[:, c["outer"]:]
    out = {"hidden": _keep_others(s, _act(g, c["act"]) * u, s["hidden"])}
    if c["keep"] == "8 bits":
        pre = torch.cat([(lambda q, e: (q * _two_to(e)).float().reshape(q.shape[0], -1)[:, :c["outer"]])(*_encode(h))
                         for h in (g, u)], 1)
    if c["keep"] != "none":
        out["pre"] = _keep_others(s, pre, s["pre"])
    return out


def _plain_hidden_backward(s):
    c = s["case"]
    d_h = _rows_product(s, s["d_out"].float(), s["w"])
    if c["keep"] == "8 bits":
        g, u = _halves(s["codes"], s["scales"])
    else:
        g, u = s["pre"][:, :c["outer"]].float(), s["pre"][:, c["outer"]:].float()
    a = _act(g, c["act"])
    d_pre = torch.cat([d_h * u * _act_slope(g, c["act"]), d_h * a], 1)
    return {"d_pre": _keep_others(s, d_pre, s["d_pre"]), "hidden": _keep_others(s, a * u, s["hidden"])}


def _plain_product_backward(s):
    c = s["case"]
    x = _decode(s["codes"], s["scales"]) if c["keep"] == "8 bits" else s["x"].float()
    d_out = s["d_out"].float()
    _, slot, _ = _place(s, x.shape[0])
    E, M = c["E"], s["most"]
    d_w = torch.bmm(_spread_rows(d_out, slot, E, M).transpose(1, 2).contiguous(), _spread_rows(x, slot, E, M))
    return {"d_x": _keep_others(s, _rows_product(s, d_out, s["w"]), s["d_x"]), "d_w": d_w}


def _norm_parts(s):
    """gate spread over the rows, out, and the two inverse roots."""
    c = s["case"]
    x, y = s["x"].float(), s["y"].float()
    gate = None if s["gate"] is None else torch.repeat_interleave(s["gate"], c["gate"], dim=0)[:c["T"]]
    r_y = torch.rsqrt((y * y).mean(1) + EPS) if c["post"] else torch.zeros_like(y[:, 0])
    z = y * r_y[:, None] * s["w_post"] if c["post"] else y
    z = z if gate is None else z * gate
    out = z + (x if s["alpha"] is None else x * s["alpha"])
    r_out = torch.rsqrt((out * out).mean(1) + EPS) if c["pre"] else torch.zeros_like(r_y)
    return gate, out, r_y, r_out


def _plain_norm(s):
    _, out, r_y, r_out = _norm_parts(s)
    got = {"out": out.to(s["x"].dtype), "stats": torch.stack([r_y, r_out], 1)}
    if s["w_pre"] is not None:
        got["normed"] = (out * r_out[:, None] * s["w_pre"]).to(s["x"].dtype)
    return got


def _plain_norm_backward(s):
    c = s["case"]
    T, H = c["T"], c["H"]
    x, y = s["x"].float(), s["y"].float()
    gate, out, _, _ = _norm_parts(s)
    r_y, r_out = s["stats"][:, :1], s["stats"][:, 1:]
    d = s["d_out"].float()
    got = {}
    if c["pre"]:
        dn = s["d_normed"].float()
        t = dn * s["w_pre"]
        d = d + r_out * t - out * (r_out ** 3 / H * (t * out).sum(1, keepdim=True))
        got["d_w_pre"] = (dn * out * r_out).sum(0)
    got["d_x"] = (d if s["alpha"] is None else d * s["alpha"]).to(s["x"].dtype)
    if c["alpha"]:
        got["d_alpha"] = (x * d).sum(0)
    z = y * r_y if c["post"] else y
    scale = s["w_post"] if gate is None else gate if s["w_post"] is None else gate * s["w_post"]
    dz = d if scale is None else d * scale
    got["d_y"] = (r_y * dz - y * (r_y ** 3 / H * (dz * y).sum(1, keepdim=True)) if c["post"] else dz).to(s["y"].dtype)
    if c["post"]:
        got["d_w_post"] = (d * z if gate is None else d * z * gate).sum(0)
    if gate is not None:
        n = c["gate"]
        dg = d * z if s["w_post"] is None else d * z * s["w_post"]
        G = -(-T // n)
        got["d_gate"] = torch.cat([dg, dg.new_zeros(G * n - T, H)]).reshape(G, n, H).sum(1)
    return got


def _plain(s):
    op = s["case"]["op"]
    if op == "encode":
        q, e = _encode(s["x"])
        return {"out": (q * _two_to(e)).reshape(q.shape[0], -1)[:, :s["case"]["H"]].to(s["x"].dtype)}
    if op == "product":
        return {"out": _keep_others(s, _rows_product_t(s, s["x"].float(), s["w"]), s["out"])}
    return {"hidden": _plain_hidden, "hidden_backward": _plain_hidden_backward, "norm": _plain_norm,
            "product_backward": _plain_product_backward, "norm_backward": _plain_norm_backward}[op](s)


# ------------------------------------------------------------------------------------ library calls

def _own(s):
    import expert_offload_lru_amd as moe
    c = s["case"]
    op = c["op"]
    if op == "encode":
        moe.rows_encode(s["x"], s["codes"], s["scales"])
        moe.rows_decode(s["codes"], s["scales"], s["out"])
        return {"out": s["out"]}
    if op == "hidden":
        I, nb = c["outer"], -(-c["outer"] // BLOCK)
        if c["keep"] == "8 bits":
            moe.experts_hidden(s["x"], s["offsets"], s["w"], s["hidden"], activation=c["act"], codes=s["codes"],
                               scales=s["scales"])
            if I % BLOCK == 0:   # the halves' blocks lie side by side
                moe.rows_decode(s["codes"], s["scales"], s["pre"])
            else:
                moe.rows_decode(s["codes"][:, :I], s["scales"][:, :nb], s["pre"][:, :I])
                moe.rows_decode(s["codes"][:, I:], s["scales"][:, nb:], s["pre"][:, I:])
        else:
            moe.experts_hidden(s["x"], s["offsets"], s["w"], s["hidden"], activation=c["act"], pre=s.get("pre"))
        return {n: s[n] for n in ("hidden", "pre") if n in s}
    if op == "hidden_backward":
        moe.experts_hidden_backward(s["d_out"], s["offsets"], s["w"], s["d_pre"], hidden=s["hidden"],
                                    activation=c["act"], pre=s.get("pre"), codes=s.get("codes"), scales=s.get("scales"))
        return {"d_pre": s["d_pre"], "hidden": s["hidden"]}
    if op == "product":
        moe.experts_product(s["x"], s["offsets"], s["w"], s["out"])
        return {"out": s["out"]}
    if op == "product_backward":
        moe.experts_product_backward(s["d_out"], s["offsets"], s["w"], x=s.get("x"), codes=s.get("codes"),
                                     scales=s.get("scales"), d_x=s["d_x"], d_w=s["d_w"])
        return {"d_x": s["d_x"], "d_w": s["d_w"]}
    parts = {n: s[n] for n in ("w_post", "gate", "alpha", "w_pre")}
    if op == "norm":
        moe.block_norm(s["x"], s["y"], s["out"], normed=s["normed"], stats=s["stats"], rows_per_gate=c["gate"], eps=EPS,
                       **parts)
        return {n: s[n] for n in ("out", "normed", "stats") if s[n] is not None}
    grads = {"d_" + n: s["d_" + n] for n in parts}
    moe.block_norm_backward(s["d_out"], s["x"], s["y"], s["stats"], s["d_x"], s["d_y"], d_normed=s["d_normed"],
                            rows_per_gate=c["gate"], **parts, **grads)
    return {n: v for n, v in {"d_x": s["d_x"], "d_y": s["d_y"], **grads}.items() if v is not None}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------------------------- work

def work(case):
    c, z = case, SIZE[case["dtype"]]
    if c["op"] == "encode":
        return {"bytes": 2 * z * c["T"] * c["H"] + 2 * c["T"] * (c["H"] + -(-c["H"] // BLOCK)), "flops": 0}
    if c["op"] in ("norm", "norm_backward"):
        n = c["T"] * c["H"]
        vectors = c["post"] + c["pre"] + c["alpha"] + (-(-c["T"] // c["gate"]) if c["gate"] else 0)
        if c["op"] == "norm":
            return {"bytes": z * n * (3 + c["pre"]) + 4 * c["H"] * vectors + 8 * c["T"], "flops": 10 * n}
        return {"bytes": z * n * (5 + c["pre"]) + 8 * c["H"] * vectors + 8 * c["T"], "flops": 25 * n}
    E, inner, outer = c["E"], c["inner"], c["outer"]
    R = c["T"] * c["k"] * (1 - c["drop"])
    used = min(E, R)
    kept = {"none": 0, "type": z, "8 bits": 1 + 1 / BLOCK}[c["keep"]]
    if c["op"] == "hidden":
        back = z if c["keep"] == "8 bits" else 0   # the read back
        return {"bytes": z * (R * (inner + outer) + used * 2 * outer * inner) + R * 2 * outer * (kept * (1 + (back > 0)) + back),
                "flops": 4 * R * inner * outer}
    if c["op"] == "hidden_backward":
        return {"bytes": z * (R * (inner + 3 * outer) + used * outer * inner) + R * 2 * outer * kept,
                "flops": 2 * R * inner * outer}
    if c["op"] == "product":
        return {"bytes": z * (R * (inner + outer) + used * outer * inner), "flops": 2 * R * inner * outer}
    return {"bytes": z * (R * (inner + outer) + used * outer * inner) + R * inner * (kept or z) + 4 * E * outer * inner,
            "flops": 4 * R * inner * outer}


# -------------------------------------------------------------------------- the definition, 64 bits

def _exact_values(codes, scales):
    T, H = codes.shape
    at = torch.arange(H, device=codes.device) // BLOCK
    return codes.double() * torch.pow(2.0, scales.double() - 133)[:, at]


def _exact_encode(x):
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for b in range(0, x.shape[1], BLOCK):
        v = x[:, b:b + BLOCK].double()
        top = v.abs().max(dim=1, keepdim=True)[0]
        step = 2.0 ** -7 / _two_to(-torch.floor(torch.log2(top.clamp(min=1e-200))))   # too small by one at least
        for _ in range(2):
            step = torch.where(torch.round(top / step) > 127, 2 * step, step)
        out[:, b:b + BLOCK] = torch.where(top > 0, torch.round(v / step) * step, 0.0)
    return out


def _exact_norm(s, x, y, w_post, gate, alpha, w_pre):
    c = s["case"]
    z = y
    rms = lambda v: torch.sqrt(v.square().sum(1, keepdim=True) / c["H"] + EPS)  # noqa: E731
    if c["post"]:
        z = w_post * (y / rms(y))
    if gate is not None:
        z = gate[torch.arange(c["T"], device=x.device) // c["gate"]] * z
    out = z + (x if alpha is None else alpha * x)
    return out, (w_pre * (out / rms(out)) if c["pre"] else None), rms


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "encode":
        return {"out": _exact_encode(s["x"])}
    if op in ("norm", "norm_backward"):
        names = ("x", "y", "w_post", "gate", "alpha", "w_pre")
        v = {n: None if s[n] is None else s[n].double() for n in names}
        if op == "norm":
            out, normed, rms = _exact_norm(s, **v)
            none = torch.zeros((c["T"], 1), dtype=torch.float64, device="cuda")
            stats = torch.cat([1 / rms(v["y"]) if c["post"] else none, 1 / rms(out) if c["pre"] else none], 1)
            return {n: t for n, t in {"out": out, "normed": normed, "stats": stats}.items() if t is not None}
        with torch.enable_grad():   # the gradients by differentiating the definition
            leaves = {n: t.requires_grad_() for n, t in v.items() if t is not None}
            out, normed, _ = _exact_norm(s, **v)
            total = (out * s["d_out"].double()).sum()
            if normed is not None:
                total = total + (normed * s["d_normed"].double()).sum()
            grads = torch.autograd.grad(total, list(leaves.values()))
        return {"d_" + n: g for n, g in zip(leaves, grads)}
    off = s["offsets"].tolist()
    w = s["w"].double()
    segments = [(e, slice(off[e], off[e + 1])) for e in range(c["E"]) if off[e + 1] > off[e]]

    def act(g):
        if c["act"] == "silu":
            return g * torch.sigmoid(g)
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))

    if op == "hidden":
        hidden, I = s["hidden"].double(), c["outer"]
        pre = torch.zeros((hidden.shape[0], 2 * I), dtype=torch.float64, device="cuda")
        for e, at in segments:
            pre[at] = s["x"][at].double() @ w[e].T.contiguous()
            hidden[at] = act(pre[at, :I]) * pre[at, I:]
        # in 8 bits a value next to a border falls to either side
        return {"hidden": hidden, "pre": pre} if c["keep"] == "type" else {"hidden": hidden, "pre": None}
    if op == "product":
        out = s["out"].double()
        for e, at in segments:
            out[at] = s["x"][at].double() @ w[e].T.contiguous()
        return {"out": out}
    d_out = s["d_out"].double()
    if op == "hidden_backward":
        d_pre, hidden, I = s["d_pre"].double(), s["hidden"].double(), c["outer"]
        if c["keep"] == "8 bits":
            nb = s["scales"].shape[1] // 2
            pre = torch.cat([_exact_values(s["codes"][:, :I], s["scales"][:, :nb]),
                             _exact_values(s["codes"][:, I:], s["scales"][:, nb:])], 1)
        else:
            pre = s["pre"].double()
        for e, at in segments:
            with torch.enable_grad():
                p = pre[at].detach().requires_grad_()
                h = act(p[:, :I]) * p[:, I:]
                d_pre[at] = torch.autograd.grad(h, p, d_out[at] @ w[e])[0]
            hidden[at] = h.detach()
        return {"d_pre": d_pre, "hidden": hidden}
    x = _exact_values(s["codes"], s["scales"]) if c["keep"] == "8 bits" else s["x"].double()
    d_x, d_w = s["d_x"].double(), torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    for e, at in segments:
        d_x[at] = d_out[at] @ w[e]
        d_w[e] = d_out[at].T.contiguous() @ x[at]
    return {"d_x": d_x, "d_w": d_w}
