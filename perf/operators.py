"""The microscaled 4-bit and expert-routing operators, as they are measured.

Five operators of large language models, each with its plain form, its call through this
package and its definition in 64 bits:

  quantise  rows of a matrix to 4-bit floating point (E2M1) in blocks of 16 or 32 columns with
            8-bit block scales, and the values the codes stand for
  linear    Y = Xq Wq^T with both operands held in that form; X is quantised in the call
  route     (token, choice) slots sorted by expert, and the token rows gathered in that order
  combine   expert outputs back in token order, summed with the routing weights, and the
            gradients of the combination and of the gather
  experts   the whole pass of a layer of experts: sort, quantise in sorted order, one product
            per expert, combine

A number format is "nv" (blocks of 16, E4M3 scales, one fp32 scale for the tensor) or "mx"
(blocks of 32, power-of-two scales).  For "nv", in IEEE fp32 arithmetic with a = max |x| of a block
and g the tensor's scale: s = e4m3(min(a / (6 g), 448)), d = s g, and each code is x / d rounded to
the nearest E2M1 value, ties to even, at most 6 in size.  For "mx": d = 2^(floor(log2 a) - 2).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"nv": 16, "mx": 32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a prefill batch's activations before a projection of 8192 columns
        {"name": "quantise-prefill", "op": "quantise", "rows": 4096, "K": 8192, "fmt": "nv", "dtype": "bf16", "pad": 0},
        # a ragged handful of rows out of a wider buffer, the last block cut short
        {"name": "quantise-ragged", "op": "quantise", "rows": 37, "K": 4107, "fmt": "mx", "dtype": "fp16", "pad": 21},
        # one new token through the largest projection: the weights' bytes are the time
        {"name": "linear-token", "op": "linear", "M": 1, "N": 28672, "K": 8192, "fmt": "nv", "dtype": "bf16"},
        # a small decoding batch
        {"name": "linear-decode", "op": "linear", "M": 16, "N": 14336, "K": 4096, "fmt": "mx", "dtype": "fp16"},
        # an odd batch through an odd layer, in and out in fp32
        {"name": "linear-ragged", "op": "linear", "M": 333, "N": 4100, "K": 4104, "fmt": "nv", "dtype": "fp32"},
        # a prefill batch through the largest projection: the tensor cores' rate is the time
        {"name": "linear-prefill", "op": "linear", "M": 4096, "N": 28672, "K": 8192, "fmt": "nv", "dtype": "bf16"},
        # one decoding step's routing: latency
        {"name": "route-step", "op": "route", "T": 5, "k": 2, "E": 8, "H": 4096, "dtype": "bf16", "drop": 0.0},
        # a training batch's routing over many experts, some choices beyond capacity dropped
        {"name": "route-batch", "op": "route", "T": 8192, "k": 8, "E": 128, "H": 2048, "dtype": "bf16", "drop": 0.03},
        # a short sequence's combination and gradients, odd width
        {"name": "combine-short", "op": "combine", "T": 77, "k": 3, "E": 10, "H": 1031, "dtype": "fp32", "drop": 0.1},
        # a training batch's combination and gradients
        {"name": "combine-batch", "op": "combine", "T": 8192, "k": 4, "E": 64, "H": 4096, "dtype": "bf16", "drop": 0.0},
        # one decoding step through a few large experts: only the chosen experts' weights are read
        {"name": "experts-step", "op": "experts", "T": 4, "k": 2, "E": 8, "N": 14336, "K": 4096, "fmt": "nv",
         "dtype": "bf16"},
        # a prefill batch through many small experts, unevenly loaded
        {"name": "experts-prefill", "op": "experts", "T": 2048, "k": 4, "E": 64, "N": 2048, "K": 2048, "fmt": "mx",
         "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantise", "linear", "linear", "route", "combine", "experts", "experts"))
    dtype = rng.choice(("bf16", "fp16", "fp32"))
    fmt = rng.choice(("nv", "mx"))
    drop = rng.choice((0.0, 0.0, 0.05, 0.5))
    if op == "quantise":
        K = _log(rng, 24, 16384)
        rows = min(_log(rng, 1, 8192), 4096 * 8192 // K)
        return {"op": op, "rows": rows, "K": K, "fmt": fmt, "dtype": dtype, "pad": rng.choice((0, 0, 8, 13))}
    if op == "linear":
        M, N, K = _log(rng, 1, 4096), _log(rng, 64, 28672), _log(rng, 64, 14336)
        if rng.random() < 0.5:
            N, K = max(64, N // 128 * 128), max(64, K // 256 * 256)
        N = min(N, 28672 * 8192 // K)
        return {"op": op, "M": M, "N": N, "K": K, "fmt": fmt, "dtype": dtype}
    E = _log(rng, 2, 128)
    k = rng.randint(1, min(8, E))
    if op == "experts":
        E = min(E, 64)
        k = min(k, E)
        T, N, K = _log(rng, 1, 2048), _log(rng, 64, 4096), _log(rng, 64, 4096)
        E = max(k, min(E, 64 * 2048 * 2048 // (N * K)))
        return {"op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "fmt": fmt, "dtype": dtype}
    T, H = _log(rng, 1, 8192), _log(rng, 24, 4096)
    return {"op": op, "T": T, "k": k, "E": E, "H": H, "dtype": dtype, "drop": drop}


def _held(rows, K, fmt):
    """bytes of rows x K codes with their block scales"""
    return rows * (K / 2 + math.ceil(K / BLOCK[fmt]))


def work(case):
    op = case["op"]
    if op == "quantise":
        n, b = case["rows"] * case["K"], SIZE[case["dtype"]]
        # the matrix in and the values out; the codes and scales written and read back between them
        return {"bytes": 2 * n * b + 2 * _held(case["rows"], case["K"], case["fmt"]), "flops": 4 * n}
    if op == "linear":
        M, N, K, b = case["M"], case["N"], case["K"], SIZE[case["dtype"]]
        return {"bytes": _held(N, K, case["fmt"]) + b * M * (K + N), "flops": 2 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    n, b = T * k, SIZE[case["dtype"]]
    if op == "route":
        H, kept = case["H"], n * (1 - case["drop"])
        return {"bytes": 4 * n + 8 * n + 4 * (E + 1) + b * H * (T + kept), "flops": n}
    if op == "combine":
        H, kept = case["H"], n * (1 - case["drop"])
        # y and dx are written, dy read; expert outputs and dxs read, dys written; weights and positions
        return {"bytes": b * H * (3 * T + 3 * kept) + 16 * n, "flops": H * kept * 6}
    N, K = case["N"], case["K"]
    hit = min(E, E * (1 - (1 - k / E) ** T))          # experts that some token chose, on average
    return {"bytes": hit * _held(N, K, case["fmt"]) + b * T * (K + N) + 8 * n, "flops": 2 * n * N * K + 2 * n * N}


# ------------------------------------------------------------------ inputs, from the seed alone
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _activations(g, rows, K, dtype):
    """normal values with one column in a hundred twenty times as large"""
    x = torch.randn(rows, K, generator=g, device=DEV)
    big = torch.rand(K, generator=g, device=DEV) < 0.01
    return torch.where(big, x * 20, x).to(TYPES[dtype])


def _weights(g, shape, dtype):
    """normal weights of deviation 0.02 with one in a thousand ten times as large"""
    w = torch.randn(*shape, generator=g, device=DEV) * 0.02
    return torch.where(torch.rand(*shape, generator=g, device=DEV) < 0.001, w * 10, w).to(TYPES[dtype])


def _scale_of(t):
    """the tensor's scale: its largest value lands on the largest E4M3 scale"""
    return (t.abs().amax().float() / (6.0 * 448.0)).reshape(1)


def _choices(g, T, k, E, drop):
    """k different experts of every token, some experts favoured, some slots dropped (-1), and weights"""
    favour = torch.randn(E, generator=g, device=DEV)
    score = torch.randn(T, E, generator=g, device=DEV) + favour
    top = torch.topk(score, k, dim=1)
    ids = top.indices.to(torch.int32)
    if drop:
        ids = torch.where(torch.rand(T, k, generator=g, device=DEV) < drop, torch.full_like(ids, -1), ids)
    return ids.contiguous(), torch.softmax(top.values, dim=1).contiguous()


def _inputs(case, seed):
    g, op, d = _gen(seed), case["op"], case["dtype"]
    if op == "quantise":
        x = _activations(g, case["rows"], case["K"] + case["pad"], d)[:, :case["K"]]
        return {"x": x, "g": _scale_of(x)}
    if op == "linear":
        x = _activations(g, case["M"], case["K"], d)
        w = _weights(g, (case["N"], case["K"]), d)
        return {"x": x, "w": w, "g": _scale_of(x) * 1.25}
    ids, wt = _choices(g, case["T"], case["k"], case["E"], case.get("drop", 0.0))
    if op == "experts":
        x = _activations(g, case["T"], case["K"], d)
        w = _weights(g, (case["E"], case["N"], case["K"]), d)
        return {"x": x, "w": w, "g": _scale_of(x) * 1.25, "ids": ids, "wt": wt}
    T, n, H = case["T"], case["T"] * case["k"], case["H"]
    if op == "route":
        return {"ids": ids, "x": torch.randn(T, H, generator=g, device=DEV).to(TYPES[d])}
    rnd = [torch.randn(r, H, generator=g, device=DEV).to(TYPES[d]) for r in (n, T, n)]
    return {"ids": ids, "wt": wt, "ys": rnd[0], "dy": rnd[1], "dxs": rnd[2]}


# ------------------------------------------------------------------ the plain forms
def _blocks(x, block):
    """[..., K] as [..., blocks, block], the last block filled with zeros"""
    K = x.shape[-1]
    fill = -K % block
    if fill:
        x = torch.cat([x, x.new_zeros(*x.shape[:-1], fill)], -1)
    return x.reshape(*x.shape[:-1], -1, block)


def _fp4_values(x, fmt, g):
    """what the codes of x's rows stand for, in fp32"""
    K = x.shape[-1]
    b = _blocks(x.float(), BLOCK[fmt])
    a = b.abs().amax(-1, keepdim=True)
    if fmt == "nv":
        s = (a / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        d = s * g
    else:
        e = (torch.frexp(a).exponent - 3).clamp(min=-127)      # a = m 2^e with m in [1/2, 1): floor(log2 a) = e - 1
        power = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)
        d = torch.where(a > 0, power, torch.zeros_like(a))
    y = torch.where(d > 0, b / d, torch.zeros_like(b))
    m = y.abs()
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int()
            + (m >= 3.5).int() + (m > 5.0).int())
    v = torch.tensor(GRID, device=x.device)[code.long()]
    v = torch.where(y < 0, -v, v) * d
    return v.reshape(*x.shape[:-1], -1)[..., :K]


def _fp4_weights(w, fmt):
    """weights as they are held: each matrix with its own scale; [.., N, K] fp32 values"""
    if w.dim() == 2:
        return _fp4_values(w, fmt, _scale_of(w))
    return torch.stack([_fp4_values(m, fmt, _scale_of(m)) for m in w])


def _sorted_slots(ids, E):
    """order [n] (slot of each sorted row, -1 behind the last), pos [n] (row of each slot, -1 where
    dropped), offsets [E + 1]"""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    key, order = torch.sort(key, stable=True)
    count = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)])
    kept = torch.arange(flat.numel(), device=ids.device) < offsets[E]
    pos = torch.full_like(flat, -1)
    pos[order] = torch.where(kept, torch.arange(flat.numel(), device=ids.device), torch.full_like(flat, -1))
    order = torch.where(kept, order, torch.full_like(order, -1))
    return order.int(), pos.int(), offsets.int()


def _combine(ys, pos, wt):
    """sum over a token's slots of weight times row, in fp32; ys [n, H], pos [T, k]"""
    out = torch.zeros(pos.shape[0], ys.shape[1], device=ys.device)
    for j in range(pos.shape[1]):
        at = pos[:, j].long()
        row = ys[at.clamp(min=0)].float()
        w = wt[:, j:j + 1] if wt is not None else 1.0
        out = out + torch.where((at >= 0)[:, None], row * w, torch.zeros_like(row))
    return out


def _run_plain(st):
    c, op = st["case"], st["case"]["op"]
    out_t = TYPES[c["dtype"]]
    if op == "quantise":
        return _fp4_values(st["x"], c["fmt"], st["g"]).to(out_t)
    if op == "linear":
        return (_fp4_values(st["x"], c["fmt"], st["g"]) @ st["w"].t()).to(out_t)
    if op == "route":
        order, pos, offsets = _sorted_slots(st["ids"], c["E"])
        src = torch.div(order.long(), c["k"], rounding_mode="floor").clamp(min=0)
        xs = torch.where((order >= 0)[:, None], st["x"][src], torch.zeros_like(st["x"][:1]))
        return {"order": order, "pos": pos, "offsets": offsets, "xs": xs}
    if op == "combine":
        pos, wt, ys, dy = st["pos"], st["wt"], st["ys"], st["dy"]
        y = _combine(ys, pos, wt).to(out_t)
        dys = torch.zeros(ys.shape, device=ys.device)
        dwt = torch.zeros_like(wt)
        for j in range(pos.shape[1]):
            at = pos[:, j].long()
            kept = at >= 0
            dwt[:, j] = torch.where(kept, (dy.float() * ys[at.clamp(min=0)].float()).sum(-1), dwt[:, j])
            dys[at[kept]] = dy[kept].float() * wt[kept, j:j + 1]
        return {"y": y, "dys": dys.to(out_t), "dwt": dwt, "dx": _combine(st["dxs"], pos, None).to(out_t)}
    # experts: one product per expert over the tokens that chose it
    xq = _fp4_values(st["x"], c["fmt"], st["g"])
    y = torch.zeros(c["T"], c["N"], device=xq.device)
    rows = torch.zeros(c["T"], c["k"], c["N"], device=xq.device)
    for e in range(c["E"]):
        t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        if t.numel():
            rows[t, j] = xq[t] @ st["w"][e].t()
    for j in range(c["k"]):
        y = y + rows[:, j] * st["wt"][:, j:j + 1]
    return y.to(out_t)


# ------------------------------------------------------------------ the framework's calls
def _run_own(st):
    from mixed_precision_quantized_mx_b200 import binding as mx
    c, op = st["case"], st["case"]["op"]
    if op == "quantise":
        mx.mx_fp4_quant(st["L"], st["x"], st["blob"], gscale=st["g"] if c["fmt"] == "nv" else None)
        return mx.mx_fp4_dequant(st["L"], st["blob"], TYPES[c["dtype"]])
    if op == "linear":
        return st["layer"].forward(st["x"], out_dtype=TYPES[c["dtype"]])
    if op == "route":
        plan = st["plan"]
        mx.mx_experts_sort(plan, st["ids"])
        mx.mx_experts_gather(plan, st["x"], st["xs"])
        return {"order": plan.order, "pos": plan.pos, "offsets": plan.offsets, "xs": st["xs"]}
    if op == "combine":
        plan = st["plan"]
        y = mx.mx_experts_combine(plan, st["ys"], st["wt"])
        dys, dwt = mx.mx_experts_combine_bwd(plan, st["dy"], st["ys"], st["wt"], dYs=st["dys"])
        dx = mx.mx_experts_gather_bwd(plan, st["dxs"])
        return {"y": y, "dys": dys, "dwt": dwt, "dx": dx}
    return st["layer"].forward(st["x"], st["ids"], st["wt"], out_dtype=TYPES[c["dtype"]])


def _with_own_layer(st):
    """A layer of the "nv" format, its weights held with the scales that the plain form takes: a layer's own
    scale is the quotient max / 2688 rounded once, the plain form's on a GPU the product with 1 / 2688, and
    where their last bits differ, blocks next to a tie of E4M3 get other scales."""
    from mixed_precision_quantized_mx_b200 import binding as mx
    from mixed_precision_quantized_mx_b200 import layer
    w = st.pop("w")
    kind, scale = ((layer.MicroscaledLinear, _scale_of(w)) if w.dim() == 2 else
                   (layer.MicroscaledExperts, torch.cat([_scale_of(m) for m in w])))
    st["layer"] = kind(w, mx.FP4_E4M3_16, act_scale=st["g"], weight_scale=scale)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    op = case["op"]
    if not own:
        if op in ("linear", "experts"):
            st["w"] = _fp4_weights(st["w"], case["fmt"])
        if op == "combine":
            order, pos, offsets = _sorted_slots(st["ids"], case["E"])
            st["pos"] = pos.reshape(case["T"], case["k"])
        return st
    elif op in ("linear", "experts") and case["fmt"] == "nv":
        return _with_own_layer(st)
    from mixed_precision_quantized_mx_b200 import binding as mx
    from mixed_precision_quantized_mx_b200 import layer
    fmt = {"nv": mx.FP4_E4M3_16, "mx": mx.FP4_E8M0_32}[case["fmt"]] if "fmt" in case else None
    if op == "quantise":
        st["L"] = mx.mx_fp4_layout_init(case["rows"], case["K"], fmt)
        st["blob"] = torch.empty(st["L"].total_bytes, dtype=torch.uint8, device=DEV)
    elif op == "linear":
        st["layer"] = layer.MicroscaledLinear(st.pop("w"), fmt, act_scale=st["g"] if case["fmt"] == "nv" else None)
    elif op == "experts":
        st["layer"] = layer.MicroscaledExperts(st.pop("w"), fmt, act_scale=st["g"] if case["fmt"] == "nv" else None)
    else:
        st["plan"] = mx.ExpertsPlan(mx.mx_experts_layout_init(case["T"], case["k"], case["E"]))
        if op == "route":
            st["xs"] = torch.zeros(case["T"] * case["k"], case["H"], dtype=TYPES[case["dtype"]], device=DEV)
        else:
            mx.mx_experts_sort(st["plan"], st["ids"])
            st["dys"] = torch.zeros_like(st["ys"])
    return st


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ the definition, in 64 bits
def _floor_log2(v):
    """of positive normal values, from their exponent bits: torch.log2 is not exact at powers of two"""
    return (v.double().view(torch.int64) >> 52) - 1023


def _power(e):
    """2^e, from exponent bits: pow is not exact either"""
    return ((e + 1023) << 52).view(torch.float64)


def _round_to(v, step):
    return torch.round(v / step) * step            # torch.round takes ties to even


def _fp4_exact(x, fmt, g):
    """the values of the codes in 64 bits, with the definition's own roundings to fp32"""
    def f32(t):
        return t.float().double()
    K, block = x.shape[-1], BLOCK[fmt]
    v = torch.nn.functional.pad(x.double(), (0, -K % block)).unflatten(-1, (-1, block))
    a = v.abs().max(-1, keepdim=True).values
    if fmt == "nv":
        g = g.double()
        r = f32(a / f32(6.0 * g)).clamp(max=448.0)
        step = _power(_floor_log2(r.clamp(min=2.0 ** -6)) - 3)
        d = f32(_round_to(r, step).clamp(max=448.0) * g)
    else:
        d = torch.where(a > 0, _power((_floor_log2(a.clamp(min=2.0 ** -140)) - 2).clamp(min=-127)), a)
    y = f32(v / torch.where(d > 0, d, torch.ones_like(d)))
    m = y.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    q = _round_to(m, step).clamp(max=6.0) * torch.sign(y)
    return torch.where(d > 0, q * d, torch.zeros_like(q)).flatten(-2)[..., :K]


def exact(case, seed):
    st, op = _inputs(case, seed), case["op"]
    if op == "quantise":
        return _fp4_exact(st["x"], case["fmt"], st["g"])
    if op == "linear":
        return _fp4_exact(st["x"], case["fmt"], st["g"]) @ _fp4_exact(st["w"], case["fmt"], _scale_of(st["w"])).T
    T, k, E = case["T"], case["k"], case["E"]
    if op == "experts":
        xq = _fp4_exact(st["x"], case["fmt"], st["g"])
        y = torch.zeros(T, case["N"], dtype=torch.float64, device=DEV)
        for e in range(E):
            share = (st["wt"].double() * (st["ids"] == e)).sum(1)      # a token's weight on this expert
            t = torch.nonzero((st["ids"] == e).any(1)).flatten()
            if t.numel():
                y[t] += share[t, None] * (xq[t] @ _fp4_exact(st["w"][e], case["fmt"], _scale_of(st["w"][e])).T)
        return y
    ids = st["ids"].flatten().tolist()
    by_expert = _slots_of(ids, E)
    rows = [s for slots in by_expert for s in slots]
    n = len(ids)
    pos = [-1] * n
    for p, s in enumerate(rows):
        pos[s] = p
    if op == "route":
        offsets, total = [0], 0
        for slots in by_expert:
            total += len(slots)
            offsets.append(total)
        order = rows + [-1] * (n - len(rows))
        xs = torch.zeros(n, case["H"], dtype=torch.float64, device=DEV)
        if rows:
            xs[:len(rows)] = st["x"].double()[torch.tensor([s // k for s in rows], device=DEV)]

        def i32(a):
            return torch.tensor(a, dtype=torch.int32, device=DEV)
        return {"order": i32(order), "pos": i32(pos), "offsets": i32(offsets), "xs": xs}
    ys, dy, dxs, wt = st["ys"].double(), st["dy"].double(), st["dxs"].double(), st["wt"].double()
    at = torch.tensor(pos, device=DEV).view(T, k)
    kept = (at >= 0).double()
    y, dx = torch.zeros_like(dy), torch.zeros_like(dy)
    dwt, dys = torch.zeros_like(wt), torch.zeros_like(ys)
    for j in range(k):
        p, on = at[:, j].clamp(min=0), kept[:, j, None]
        y += on * wt[:, j, None] * ys[p]
        dx += on * dxs[p]
        dwt[:, j] = kept[:, j] * torch.einsum("th,th->t", dy, ys[p])
        dys.index_add_(0, p, on * wt[:, j, None] * dy)
    return {"y": y, "dys": dys, "dwt": dwt, "dx": dx}


def _slots_of(ids, E):
    slots = [[] for _ in range(E)]
    for s, e in enumerate(ids):
        if 0 <= e < E:
            slots[e].append(s)
    return slots
