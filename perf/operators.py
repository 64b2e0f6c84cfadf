"""The operators around the grouped GEMMs, as workloads to time and compare.

A mixture-of-experts layer needs four things next to its expert products:
a router, the move of token rows into the GEMMs' layouts and back, and, for
training, the experts' activations kept in 8 bits and read by the backward
pass.  Each case below is one call of one of them as a model makes it:

  route          scores, bias, groups, top-k and weights of T tokens
  route_bwd      the gradient of those weights with respect to the logits
  dispatch       the slot map of the top-k choices (counts, row of every
                 choice, choice of every row), and the token rows moved into
                 the contiguous or masked layout, as bf16 or as E4M3 with one
                 power-of-two scale per (row, 128 columns)
  combine        the weighted sum of every token's expert rows (with unit
                 weights also the gradient of dispatch)
  combine_bwd    its gradients: expert rows and weights
  swiglu_save    SwiGLU of GEMM1's rows, which are kept in 8 bits
  swiglu_bwd     SwiGLU's backward pass from the 8-bit rows: the gradient of
                 GEMM1's rows, the weighted activations that GEMM2's weight
                 gradient reads, and the gradient of the routing weights

`own` chooses between the plain torch form of a case (32-bit arithmetic,
rounded once) and the library's calls.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
F32_TINY = 1.1754943508222875e-38      # smallest normal float32


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a serving batch (a graph of fixed size, its last
        # tokens unused): grouped sigmoid routing with a balance bias
        dict(name="route_decode", op="route", T=48, unused=5, E=256, k=8, score="sigmoid", groups=8, top_groups=4,
             group_top=2, bias=True, renorm=True, scale=2.5, logits="f32"),
        # a long prefill: softmax top-8 of 128 experts
        dict(name="route_prefill", op="route", T=32768, unused=0, E=128, k=8, score="softmax", groups=1, top_groups=1,
             group_top=1, bias=False, renorm=True, scale=1.0, logits="bf16"),
        # a training micro-batch of odd length, softmax weights without
        # renormalisation (every logit of a token has a gradient)
        dict(name="route_bwd_train", op="route_bwd", T=8191, unused=0, E=160, k=6, score="softmax", groups=8,
             top_groups=3, group_top=1, bias=False, renorm=False, scale=16.0, logits="bf16"),
        # the decode step's tokens into the masked buffers of an FP8 GEMM
        dict(name="dispatch_decode", op="dispatch", T=61, unused=3, E=16, k=4, K=7168, layout="masked", align=0,
             m_max=256, src="bf16", dst="e4m3", ckpt=False),
        # the FP8 prefill workload: 32768 choices over 64 experts
        dict(name="dispatch_prefill", op="dispatch", T=4096, unused=0, E=64, k=8, K=7168, layout="contiguous",
             align=128, m_max=0, src="bf16", dst="e4m3", ckpt=False),
        # backward pass of a training step: 65536 packed rows rebuilt from the
        # tokens' 8-bit checkpoint, for the K-grouped weight gradient
        dict(name="dispatch_ckpt", op="dispatch", T=8192, unused=0, E=32, k=8, K=2048, layout="contiguous", align=1,
             m_max=0, src="e4m3", dst="bf16", ckpt=False),
        # the decode step's expert rows back to its tokens
        dict(name="combine_decode", op="combine", T=61, unused=3, E=16, k=4, K=7168, layout="masked", align=0,
             m_max=256, weights=True),
        # the prefill's expert rows back to its tokens
        dict(name="combine_prefill", op="combine", T=4096, unused=0, E=64, k=8, K=7168, layout="contiguous",
             align=128, m_max=0, weights=True),
        # training: gradients of the expert rows and of the routing weights
        dict(name="combine_bwd_train", op="combine_bwd", T=8192, unused=0, E=32, k=8, K=2048, layout="contiguous",
             align=1, m_max=0),
        # training forward: GEMM1's rows to activations and 8-bit checkpoint
        dict(name="swiglu_save_train", op="swiglu_save", T=8192, unused=0, E=32, k=8, N=4096, layout="contiguous",
             align=1, m_max=0, out="bf16"),
        # training backward of the same rows
        dict(name="swiglu_bwd_train", op="swiglu_bwd", T=8192, unused=0, E=32, k=8, N=4096, layout="contiguous",
             align=1, m_max=0),
        # the backward of a small fine-tuning batch, ragged aligned segments
        dict(name="swiglu_bwd_small", op="swiglu_bwd", T=259, unused=0, E=16, k=2, N=4096, layout="contiguous",
             align=16, m_max=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _choices(rng, most, width):
    """Tokens, experts, choices per token: at most `most` values of T * k * width."""
    E = rng.choice([8, 16, 24, 32, 64, 96, 128, 160, 256])
    k = rng.randint(1, min(8, E))
    T = _log_int(rng, 1, max(2, min(16384, most // (k * width))))
    return T, E, k


def _layout(rng, T, E, fp8):
    if T <= 512 and E * T <= 16384 and rng.random() < 0.5:
        return dict(layout="masked", align=0, m_max=max(16, (T + 15) // 16 * 16))
    return dict(layout="contiguous", align=rng.choice([16, 32, 128] if fp8 else [1, 8, 16, 128]), m_max=0)


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "dispatch", "dispatch", "combine", "combine_bwd", "swiglu_save",
                     "swiglu_bwd"])
    if op in ("route", "route_bwd"):
        E = rng.choice([8, 12, 16, 32, 60, 64, 96, 128, 160, 192, 256, 384])
        k = rng.randint(1, min(8, E // 4))
        groups = rng.choice([1, 1, 4])
        T = _log_int(rng, 1, 65536)
        bias = rng.random() < 0.5
        return dict(op=op, T=T, unused=rng.choice([0, T // 9]), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    groups=groups, top_groups=max(1, groups // 2), group_top=2 if bias and E // groups > 1 else 1,
                    bias=bias, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    logits=rng.choice(["bf16", "f32"]))
    if op in ("dispatch", "combine", "combine_bwd"):
        K = rng.choice([256, 640, 1024, 2048, 2176, 4096, 5120, 7168])
        T, E, k = _choices(rng, 8192 * 8 * 2048, K)
        unused = rng.choice([0, T // 7])
        if op == "dispatch":
            src, dst = rng.choice([("bf16", "e4m3"), ("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "e4m3")])
            return dict(op=op, T=T, unused=unused, E=E, k=k, K=K, **_layout(rng, T, E, dst == "e4m3"), src=src,
                        dst=dst, ckpt=src == "bf16" and rng.random() < 0.5)
        d = dict(op=op, T=T, unused=unused, E=E, k=k, K=K, **_layout(rng, T, E, False))
        return dict(d, weights=rng.random() < 0.7) if op == "combine" else d
    N = rng.choice([512, 1536, 2816, 4096])
    T, E, k = _choices(rng, 8192 * 8 * 4096, N)
    d = dict(op=op, T=T, unused=0, E=E, k=k, N=N)
    if op == "swiglu_save":
        out = rng.choice(["bf16", "e4m3"])
        return dict(d, **_layout(rng, T, E, out == "e4m3"), out=out)
    return dict(d, **_layout(rng, T, E, False))


def _rows_total(c):
    """Rows of the layout's buffers, known without the counts."""
    if c["layout"] == "masked":
        return c["E"] * c["m_max"]
    return (c["T"] * c["k"] + c["E"] * (c["align"] - 1) + 15) // 16 * 16


def _group_rows(c):
    return c["m_max"] if c["layout"] == "masked" else _rows_total(c)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _zeros(*shape, dtype):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _skew(g, E):
    """A lasting preference of the router: some experts are hot."""
    return 0.8 * _normal(g, E)


def _separated(c, logits, bias):
    """Tokens whose choice of experts does not hang on the last bits of a score: the gaps next to every cut are
    zero (equal inputs: the lowest index wins) or well above a rounding of exp or of a sum."""
    key, s = _keys64(c, logits.double(), bias)
    T, E = key.shape
    fine = torch.ones(T, dtype=torch.bool, device=key.device)

    def gaps(v, n):
        v = torch.sort(v, dim=1, descending=True).values[:, :n + 1]
        d = v[:, :-1] - v[:, 1:]
        d = torch.where(torch.isnan(d), torch.zeros_like(d), d)
        return ((d == 0) | (d > 4e-6 * v[:, :-1].abs().clamp(max=1e30))).all(1)
    if c["groups"] > 1:
        grp = _group_scores64(c, key)
        fine &= gaps(grp, c["top_groups"])
        key = _drop_groups64(c, key, grp)
    return fine & gaps(key, c["k"])


def _route_inputs(c, g):
    T, E = c["T"], c["E"]
    logits = 1.5 * _normal(g, T, E) + _skew(g, E)
    # the balance bias moves by fixed small steps during training
    bias = (torch.round(20 * _normal(g, E)) * 1e-3).contiguous() if c["bias"] else None
    logits = logits.to(torch.bfloat16 if c["logits"] == "bf16" else torch.float32)
    fine = _separated(c, logits, bias)
    at = fine.nonzero().flatten()
    if at.numel():
        bad = (~fine).nonzero().flatten()
        logits[bad] = logits[at[torch.arange(bad.numel(), device="cuda") % at.numel()]]
    if c["unused"]:
        logits[T - c["unused"]:] = -math.inf      # an unused token chooses nothing
    return logits.contiguous(), bias


def _choose(c, g):
    """Every token's k distinct experts (-1 for unused tokens), int32 [T, k]."""
    s = _normal(g, c["T"], c["E"]) + _skew(g, c["E"])
    idx = torch.topk(s, c["k"], dim=1).indices.to(torch.int32)
    if c["unused"]:
        idx[c["T"] - c["unused"]:] = -1
    return idx.contiguous()


def _weights(c, g):
    w = torch.rand(c["T"], c["k"], generator=g, device="cuda") + 0.05
    return (w / w.sum(1, keepdim=True)).contiguous()


def _tokens(c, g, T, K):
    """Normalised hidden states: unit variance, a few large channels."""
    x = _normal(g, T, K)
    x *= 1.0 + 7.0 * (torch.rand(K, generator=g, device="cuda") < 0.01)
    return x.to(torch.bfloat16)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] in ("route", "route_bwd"):
        s["logits"], s["bias"] = _route_inputs(c, g)
        s["status"] = _zeros(1, dtype=torch.int32)
        s["idx"] = _zeros(T, k, dtype=torch.int32)
        s["w"] = _zeros(T, k, dtype=torch.float32)
        if c["op"] == "route_bwd":
            idx, w = _plain_route(c, s["logits"], s["bias"])
            s["idx"].copy_(idx)
            s["w"].copy_(w)
            s["dw"] = _normal(g, T, k).contiguous()
            s["dlogits"] = torch.zeros_like(s["logits"])
        return s
    idx = _choose(c, g)
    R = _rows_total(c)
    s["status"] = _zeros(1, dtype=torch.int32)
    if c["op"] == "dispatch":
        K = c["K"]
        s["idx"] = idx
        s["counts"] = _zeros(E, dtype=torch.int32)
        s["rows"] = _zeros(T, k, dtype=torch.int32)
        s["src"] = _zeros(R, dtype=torch.int32)
        # the slot map's scratch: 4 bytes per (block of 4096 choices, expert)
        s["work"] = _zeros(((T * k + 4095) // 4096) * E, dtype=torch.int32)
        x = _tokens(c, g, T, K)
        if c["src"] == "e4m3":
            s["X"], s["SX"] = _plain_quantize(x.float())
        else:
            s["X"], s["SX"] = x, None
        lead = (E, c["m_max"]) if c["layout"] == "masked" else (R,)
        s["A"] = _zeros(*lead, K, dtype=torch.uint8 if c["dst"] == "e4m3" else torch.bfloat16)
        s["SFA"] = None
        if c["dst"] == "e4m3":
            s["SFA"] = _zeros(*lead[:-1], K // 128, _group_rows(c), dtype=torch.uint8)
        s["CX"] = _zeros(T, K, dtype=torch.uint8) if c["ckpt"] else None
        s["SCX"] = _zeros(T, K // 128, dtype=torch.uint8) if c["ckpt"] else None
        return s
    _, s["rows"], s["src"] = _plain_slots(c, idx)
    s["w"] = _weights(c, g)
    if c["op"] in ("combine", "combine_bwd"):
        K = c["K"]
        s["D"] = _normal(g, R, K).to(torch.bfloat16)
        if c["op"] == "combine":
            if not c["weights"]:
                s["w"] = None
            s["out"] = _zeros(T, K, dtype=torch.bfloat16)
        else:
            s["dout"] = (1e-3 * _normal(g, T, K)).to(torch.bfloat16)
            s["dD"] = _zeros(R, K, dtype=torch.bfloat16)
            s["dw"] = _zeros(T, k, dtype=torch.float32)
        return s
    N = c["N"]
    if c["op"] == "swiglu_save":
        s["H"] = (1.3 * _normal(g, R, N)).to(torch.bfloat16)
        s["Y"] = _zeros(R, N // 2, dtype=torch.uint8 if c["out"] == "e4m3" else torch.bfloat16)
        s["SFY"] = None
        if c["out"] == "e4m3":
            G = _group_rows(c)
            s["SFY"] = _zeros(R // G, N // 256, G, dtype=torch.uint8)
        s["HC"] = _zeros(R, N, dtype=torch.uint8)
        s["SHC"] = _zeros(R, N // 128, dtype=torch.uint8)
    else:
        s["HC"], s["SHC"] = _plain_quantize((1.3 * _normal(g, R, N)).to(torch.bfloat16).float())
        s["dY"] = (1e-3 * _normal(g, R, N // 2)).to(torch.bfloat16)
        s["dH"] = _zeros(R, N, dtype=torch.bfloat16)
        s["Y"] = _zeros(R, N // 2, dtype=torch.bfloat16)
        s["dw"] = _zeros(T, k, dtype=torch.float32)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _codes(t):
    """8-bit codes as the numbers they stand for (no copy)."""
    return None if t is None else t.view(torch.float8_e4m3fn)


def _scales(t):
    """UE8M0 bytes as the powers of two they stand for (no copy)."""
    return None if t is None else t.view(torch.float8_e8m0fnu)


def run(state):
    return (_run_own if own else _run_plain)(state["case"], state)


def _run_own(c, s):
    from moe_grouped_gemm_side_gb300 import binding as mb
    op = c["op"]
    if op == "route":
        mb.route(s["logits"], s["idx"], s["w"], score=c["score"], bias=s["bias"], groups=c["groups"],
                 top_groups=c["top_groups"], group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"],
                 status=s["status"])
        return {"idx": s["idx"], "w": s["w"]}
    if op == "route_bwd":
        mb.route_backward(s["logits"], s["idx"], s["dw"], s["dlogits"], score=c["score"], renorm=c["renorm"],
                          scale=c["scale"], status=s["status"])
        return {"dlogits": s["dlogits"]}
    if op == "dispatch":
        if c["layout"] == "masked":
            mb.slots_masked(s["idx"], s["rows"], s["counts"], c["m_max"], src=s["src"], work=s["work"],
                            status=s["status"])
        else:
            mb.slots_contiguous(s["idx"], s["rows"], s["counts"], c["align"], _rows_total(c), src=s["src"],
                                work=s["work"], status=s["status"])
        mb.dispatch(s["X"], s["rows"], s["A"], SX=s["SX"], SFA=s["SFA"], CX=s["CX"], SCX=s["SCX"],
                    status=s["status"])
    elif op == "combine":
        mb.combine(s["D"], s["rows"], s["out"], w=s["w"], status=s["status"])
    elif op == "combine_bwd":
        mb.combine_backward(s["dout"], s["D"], s["rows"], s["w"], s["dD"], s["dw"], status=s["status"])
    elif op == "swiglu_save":
        mb.swiglu_save(s["H"], s["Y"], s["HC"], s["SHC"], SFY=s["SFY"], src=s["src"])
    else:
        mb.swiglu_backward(s["dY"], s["HC"], s["SHC"], s["dH"], w=s["w"], src=s["src"], Y=s["Y"], dw=s["dw"],
                           status=s["status"])
    return _outputs(c, s)


def _outputs(c, s):
    op = c["op"]
    if op == "dispatch":
        out = {"counts": s["counts"], "rows": s["rows"], "src": s["src"]}
        if c["dst"] == "e4m3":
            out.update(A=_codes(s["A"]), SFA=_scales(s["SFA"]))
        else:
            out["A"] = s["A"]
        if c["ckpt"]:
            out.update(CX=_codes(s["CX"]), SCX=_scales(s["SCX"]))
        return out
    if op == "combine":
        return {"out": s["out"]}
    if op == "combine_bwd":
        return {"dD": s["dD"], "dw": s["dw"]}
    if op == "swiglu_save":
        out = {"HC": _codes(s["HC"]), "SHC": _scales(s["SHC"])}
        if c["out"] == "e4m3":
            out.update(Y=_codes(s["Y"]), SFY=_scales(s["SFY"]))
        else:
            out["Y"] = s["Y"]
        return out
    return {"dH": s["dH"], "Y": s["Y"], "dw": s["dw"]}


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _plain_scores(c, x):
    """float32 scores of float32 logits; experts at -inf score 0."""
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.max(dim=1, keepdim=True).values
    e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return e / e.sum(dim=1, keepdim=True).clamp(min=F32_TINY)


def _plain_route(c, logits, bias):
    x = logits.float()
    T, E = x.shape
    s = _plain_scores(c, x)
    out = torch.full_like(x, -math.inf)
    key = torch.where(x == -math.inf, out, s if bias is None else s + bias)
    if c["groups"] > 1:
        by = key.view(T, c["groups"], E // c["groups"])
        top = torch.sort(by, dim=2, descending=True).values[:, :, :c["group_top"]]
        # a group's score: the sum of its largest keys; no member left: -inf
        grp = torch.where(torch.isinf(top), torch.zeros_like(top), top).sum(2)
        grp = torch.where(torch.isinf(top[:, :, 0]), torch.full_like(grp, -math.inf), grp)
        kept = torch.sort(grp, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros_like(grp, dtype=torch.bool).scatter_(1, kept, True)
        key = torch.where(keep[:, :, None].expand_as(by).reshape(T, E), key, out)
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    val, idx = val[:, :c["k"]], idx[:, :c["k"]]
    w = torch.where(torch.isinf(val), torch.zeros_like(val), s.gather(1, idx))
    idx = torch.where(torch.isinf(val), torch.full_like(idx, -1), idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=F32_TINY)
    return idx.to(torch.int32), w * c["scale"]


def _plain_route_bwd(c, logits, idx, dw):
    x = logits.float()
    s = _plain_scores(c, x)
    there = idx >= 0
    at = idx.clamp(min=0).long()
    sel = torch.where(there, s.gather(1, at), torch.zeros_like(dw))
    ds = c["scale"] * torch.where(there, dw, torch.zeros_like(dw))
    if c["renorm"]:
        total = sel.sum(1, keepdim=True).clamp(min=F32_TINY)
        ds = (ds - (ds * (sel / total)).sum(1, keepdim=True)) / total
        ds = torch.where(there, ds, torch.zeros_like(ds))
    full = torch.zeros_like(x).scatter_add_(1, at, ds)
    if c["score"] == "sigmoid":
        dx = full * s * (1.0 - s)
    else:
        dx = s * (full - (ds * sel).sum(1, keepdim=True))
    return dx.to(logits.dtype)


def _plain_quantize(x):
    """E4M3 codes and one UE8M0 byte per (row, 128 columns) of float32 x."""
    R, C = x.shape
    b = x.view(R, C // 128, 128)
    m, e = torch.frexp(b.abs().amax(2) / E4M3_MAX)
    s = torch.where(m == 0.5, e - 1, e) + 127            # smallest power of two that holds the block
    s = torch.where(m == 0, torch.full_like(s, 127), s.clamp(1, 254))
    codes = (b / torch.exp2(s.float() - 127.0)[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(R, C), s.to(torch.uint8)


def _plain_dequantize(codes, s):
    R, C = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(R, C // 128, 128)
    return (v * torch.exp2(s.float() - 127.0)[:, :, None]).view(R, C)


def _plain_slots(c, idx):
    """counts [E], rows [T, k], src [R]: choices of one expert keep their order."""
    E, dev = c["E"], idx.device
    e = idx.reshape(-1).long()
    key = torch.where(e < 0, torch.full_like(e, E), e)
    counts = (key[:, None] == torch.arange(E, device=dev)).sum(0)
    first = torch.cumsum(counts, 0) - counts
    if c["layout"] == "masked":
        base = torch.arange(E, device=dev) * c["m_max"]
    else:
        padded = (counts + c["align"] - 1) // c["align"] * c["align"]
        base = torch.cumsum(padded, 0) - padded
    key, order = torch.sort(key, stable=True)
    at = (key < E).nonzero().flatten()
    key, order = key[at], order[at]
    row = base[key] + torch.arange(key.numel(), device=dev) - first[key]
    rows = torch.full((idx.numel(),), -1, dtype=torch.int32, device=dev)
    rows[order] = row.to(torch.int32)
    src = torch.full((_rows_total(c),), -1, dtype=torch.int32, device=dev)
    src[row] = order.to(torch.int32)
    return counts.to(torch.int32), rows.view(idx.shape), src


def _pairs(rows):
    """Row and flat choice index of every choice that has a row."""
    flat = rows.reshape(-1)
    at = (flat >= 0).nonzero().flatten()
    return flat[at].long(), at


def _put_scales(c, sf, row, s):
    """One row's scales [rows, blocks] into the GEMM's layout [.., blocks, rows]."""
    G = _group_rows(c)
    sf.view(-1, s.shape[1], G)[row // G, :, row % G] = s


def _swiglu32(h):
    R, N = h.shape
    b = h.view(R, N // 256, 2, 128)
    return b[:, :, 0], b[:, :, 1]


def _run_plain(c, s):
    op = c["op"]
    if op == "route":
        idx, w = _plain_route(c, s["logits"], s["bias"])
        return {"idx": idx, "w": w}
    if op == "route_bwd":
        return {"dlogits": _plain_route_bwd(c, s["logits"], s["idx"], s["dw"])}
    if op == "dispatch":
        K = c["K"]
        counts, rows, src = _plain_slots(c, s["idx"])
        s["counts"].copy_(counts)
        s["rows"].copy_(rows)
        s["src"].copy_(src)
        row, at = _pairs(rows)
        tok = at // c["k"]
        A = s["A"].view(-1, K)
        x = s["X"].float() if c["src"] == "bf16" else _plain_dequantize(s["X"], s["SX"])
        if c["ckpt"] or c["dst"] == "e4m3":
            q, sc = _plain_quantize(x) if c["src"] == "bf16" else (s["X"], s["SX"])
        if c["dst"] == "e4m3":
            A[row] = q[tok]
            _put_scales(c, s["SFA"], row, sc[tok])
        else:
            A[row] = x.to(torch.bfloat16)[tok]
        if c["ckpt"]:
            s["CX"].copy_(q)
            s["SCX"].copy_(sc)
    elif op == "combine":
        T, k, K = c["T"], c["k"], c["K"]
        there = (s["rows"] >= 0).float()
        w = there if s["w"] is None else s["w"] * there
        got = s["D"][s["rows"].clamp(min=0).long()].float()
        s["out"].copy_((got * w[:, :, None]).sum(1))
    elif op == "combine_bwd":
        row, at = _pairs(s["rows"])
        g = s["dout"].float()[at // c["k"]]
        s["dw"].view(-1)[at] = (g * s["D"][row].float()).sum(1)
        s["dD"][row] = (g * s["w"].view(-1)[at][:, None]).to(torch.bfloat16)
    elif op == "swiglu_save":
        row = (s["src"] >= 0).nonzero().flatten()
        h = s["H"][row].float()
        g, u = _swiglu32(h)
        y = (g / (1.0 + torch.exp(-g)) * u).reshape(h.shape[0], -1)
        q, sc = _plain_quantize(h)
        s["HC"][row] = q
        s["SHC"][row] = sc
        if c["out"] == "e4m3":
            q, sc = _plain_quantize(y)
            s["Y"][row] = q
            _put_scales(c, s["SFY"], row, sc)
        else:
            s["Y"][row] = y.to(torch.bfloat16)
    else:
        row = (s["src"] >= 0).nonzero().flatten()
        at = s["src"][row].long()
        h = _plain_dequantize(s["HC"][row], s["SHC"][row])
        g, u = _swiglu32(h)
        dy = s["dY"][row].float().view(g.shape)
        w = s["w"].view(-1)[at][:, None, None]
        sig = 1.0 / (1.0 + torch.exp(-g))
        y = g * sig * u
        s["dw"].view(-1)[at] = (dy * y).sum((1, 2))
        d = dy * w
        dh = torch.stack([d * u * sig * (1.0 + g * (1.0 - sig)), d * g * sig], 2)
        s["dH"][row] = dh.view(h.shape).to(torch.bfloat16)
        s["Y"][row] = (y * w).reshape(h.shape[0], -1).to(torch.bfloat16)
    return _outputs(c, s)


# --------------------------------------------------------------------------
# bytes and operations
# --------------------------------------------------------------------------

def work(case):
    c = case
    T, E, k = c["T"], c["E"], c["k"]
    n = T * k
    if c["op"] in ("route", "route_bwd"):
        size = 2 if c["logits"] == "bf16" else 4
        if c["op"] == "route":
            return {"bytes": T * E * size + (4 * E if c["bias"] else 0) + 8 * n, "flops": 6 * T * E}
        # with renormalised or sigmoid weights only the chosen logits matter
        read = T * E if c["score"] == "softmax" and not c["renorm"] else n
        return {"bytes": read * size + T * E * size + 8 * n, "flops": 6 * read + 2 * T * E}
    live = (T - c["unused"]) * k
    if c["op"] == "dispatch":
        K = c["K"]
        one = {"bf16": 2 * K, "e4m3": K + K // 128}
        ckpt = T * one["e4m3"] if c["ckpt"] else 0
        tokens = (T - c["unused"]) if not c["ckpt"] else T
        return {"bytes": 8 * n + 4 * E + 4 * _rows_total(c) + tokens * one[c["src"]] + live * one[c["dst"]] + ckpt,
                "flops": 3 * T * K}
    if c["op"] == "combine":
        return {"bytes": live * 2 * c["K"] + T * 2 * c["K"] + 4 * n + (4 * n if c["weights"] else 0),
                "flops": 2 * live * c["K"]}
    if c["op"] == "combine_bwd":
        return {"bytes": (T - c["unused"]) * 2 * c["K"] + live * 4 * c["K"] + 12 * n, "flops": 3 * live * c["K"]}
    N = c["N"]
    one = N + N // 128
    if c["op"] == "swiglu_save":
        y = N if c["out"] == "bf16" else N // 2 + N // 256
        return {"bytes": live * (2 * N + one + y) + 4 * _rows_total(c), "flops": 8 * live * N}
    return {"bytes": live * (N + one + 2 * N + N + 8) + 4 * _rows_total(c), "flops": 10 * live * N}


# --------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------

def _scores64(c, x):
    if c["score"] == "sigmoid":
        return torch.where(x == -math.inf, torch.zeros_like(x), torch.special.expit(x))
    dead = (x == -math.inf).all(1, keepdim=True)
    return torch.where(dead, torch.zeros_like(x), torch.softmax(torch.where(dead, torch.zeros_like(x), x), 1))


def _keys64(c, x, bias):
    s = _scores64(c, x)
    key = s if bias is None else s + bias.double()
    return torch.where(x == -math.inf, torch.full_like(x, -math.inf), key), s


def _group_scores64(c, key):
    v = torch.sort(key.view(key.shape[0], c["groups"], -1), dim=2, descending=True).values
    tail = v[:, :, 1] if c["group_top"] == 2 else torch.zeros_like(v[:, :, 0])
    return v[:, :, 0] + torch.where(torch.isinf(tail), torch.zeros_like(tail), tail)


def _drop_groups64(c, key, grp):
    rank = torch.argsort(torch.argsort(grp, dim=1, descending=True, stable=True), dim=1)
    gone = (rank >= c["top_groups"]).repeat_interleave(c["E"] // c["groups"], 1)
    return torch.where(gone, torch.full_like(key, -math.inf), key)


def _round_e4m3(v):
    """The nearest E4M3 value of float64 v, ties to even, at most 448."""
    e = (torch.frexp(v).exponent - 1).clamp(min=-6).double()
    q = torch.exp2(e - 3)
    return (torch.round(v / q) * q).clamp(-E4M3_MAX, E4M3_MAX)


def _quantize64(x):
    """E4M3 values and power-of-two scales of float64 x [R, C]."""
    b = x.view(x.shape[0], -1, 128)
    top = b.abs().amax(2)
    e = torch.ceil(torch.log2(torch.where(top == 0, torch.ones_like(top), top) / E4M3_MAX))
    e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where(top <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
    s = torch.where(top == 0, torch.ones_like(e), torch.exp2(e.clamp(-126, 127)))
    return _round_e4m3(b / s[:, :, None]).view(x.shape), s


def _e4m3_value(codes):
    """E4M3 bytes as float64, from the format's definition."""
    v = codes.to(torch.int64)
    e, m = (v >> 3) & 15, (v & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    return torch.where(v >= 128, -mag, mag)


def _load64(codes, s):
    b = _e4m3_value(codes).view(codes.shape[0], -1, 128)
    return (b * torch.exp2(s.double() - 127)[:, :, None]).view(codes.shape)


def _like(t, row, values):
    """A buffer of zeros with `values` in its rows `row`, float64."""
    out = torch.zeros(t.shape, dtype=torch.float64, device=t.device)
    out.view(-1, values.shape[1])[row] = values
    return out


def _scales_like(c, t, row, s):
    out = torch.full(t.shape, 2.0 ** -127, dtype=torch.float64, device=t.device)   # byte 0
    G = _group_rows(c)
    out.view(-1, s.shape[1], G)[row // G, :, row % G] = s
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    op = c["op"]
    if op == "route":
        x = s["logits"].double()
        key, sc = _keys64(c, x, s["bias"])
        if c["groups"] > 1:
            key = _drop_groups64(c, key, _group_scores64(c, key))
        order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :c["k"]]
        w = sc.gather(1, order) * torch.isfinite(key.gather(1, order))
        if c["renorm"]:
            tot = w.sum(1, keepdim=True)
            w = torch.where(tot > 0, w / torch.where(tot > 0, tot, torch.ones_like(tot)), w)
        return {"idx": None, "w": c["scale"] * w}
    if op == "route_bwd":
        x = s["logits"].double()
        sc = _scores64(c, x)
        there = (s["idx"] >= 0).double()
        at = s["idx"].clamp(min=0).long()
        hit = torch.zeros_like(x).scatter_add_(1, at, there)                        # 1 at the chosen experts
        up = torch.zeros_like(x).scatter_add_(1, at, there * s["dw"].double()) * c["scale"]
        if c["renorm"]:
            tot = (hit * sc).sum(1, keepdim=True)
            tot = torch.where(tot > 0, tot, torch.ones_like(tot))
            up = hit * (up * tot - (up * sc).sum(1, keepdim=True)) / tot ** 2
        if c["score"] == "sigmoid":
            return {"dlogits": up * sc * torch.special.expit(-x)}
        return {"dlogits": sc * up - sc * (sc * up).sum(1, keepdim=True)}
    if op == "dispatch":
        _, rows, _ = _plain_slots(c, s["idx"])
        row, at = _pairs(rows)
        tok = at // c["k"]
        x = s["X"].double() if c["src"] == "bf16" else _load64(s["X"], s["SX"])
        if c["src"] == "bf16":
            q, sc = _quantize64(x) if c["ckpt"] or c["dst"] == "e4m3" else (None, None)
        else:
            q, sc = _e4m3_value(s["X"]), torch.exp2(s["SX"].double() - 127)
        out = {"A": _like(s["A"], row, q[tok] if c["dst"] == "e4m3" else x[tok])}
        if c["dst"] == "e4m3":
            out["SFA"] = _scales_like(c, s["SFA"], row, sc[tok])
        if c["ckpt"]:
            out.update(CX=q, SCX=sc)
        return out
    if op == "combine":
        there = (s["rows"] >= 0).double()
        w = there if s["w"] is None else there * s["w"].double()
        got = s["D"][s["rows"].clamp(min=0).long()].double()
        return {"out": torch.einsum("tkc,tk->tc", got, w)}
    if op == "combine_bwd":
        row, at = _pairs(s["rows"])
        g = s["dout"][at // c["k"]].double()
        dw = torch.zeros(c["T"] * c["k"], dtype=torch.float64, device=g.device)
        dw[at] = (g * s["D"][row].double()).sum(1)
        return {"dD": _like(s["dD"], row, g * s["w"].view(-1)[at].double()[:, None]), "dw": dw.view(c["T"], c["k"])}
    row = (s["src"] >= 0).nonzero().flatten()
    if op == "swiglu_save":
        h = s["H"][row].double()
        b = h.view(h.shape[0], -1, 256)
        y = (b[..., :128] * torch.special.expit(b[..., :128]) * b[..., 128:]).reshape(h.shape[0], -1)
        q, sc = _quantize64(h)
        out = {"HC": _like(s["HC"], row, q)}
        out["SHC"] = torch.full(s["SHC"].shape, 2.0 ** -127, dtype=torch.float64, device=h.device)
        out["SHC"][row] = sc
        if c["out"] == "e4m3":
            q, sc = _quantize64(y)
            out.update(Y=_like(s["Y"], row, q), SFY=_scales_like(c, s["SFY"], row, sc))
        else:
            out["Y"] = _like(s["Y"], row, y)
        return out
    at = s["src"][row].long()
    b = _load64(s["HC"][row], s["SHC"][row]).view(row.numel(), -1, 256)
    g, u = b[..., :128], b[..., 128:]
    p = torch.special.expit(g)
    dy = s["dY"][row].double().view(g.shape)
    w = s["w"].view(-1)[at].double()[:, None, None]
    dw = torch.zeros(c["T"] * c["k"], dtype=torch.float64, device=g.device)
    dw[at] = (dy * g * p * u).sum((1, 2))
    slope = p + g * p * torch.special.expit(-g)                                      # SiLU'
    dh = torch.cat([w * dy * u * slope, w * dy * g * p], 2).reshape(row.numel(), -1)
    y = (w * g * p * u).reshape(row.numel(), -1)
    return {"dH": _like(s["dH"], row, dh), "Y": _like(s["Y"], row, y), "dw": dw.view(c["T"], c["k"])}
