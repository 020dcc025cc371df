"""The expert layer's operators as a program calls them: what is timed, on which sizes.

Four operators stand around the dispatch plan of this package:

  gate       routing scores (softmax or sigmoid) with a balance bias, expert
             groups, top-k and renormalised weights, and its gradient
  quantize   e4m3 values with one power-of-two scale per block of 128: of
             expert weights (128 x 128 blocks, both layouts) and, fused with
             the gated activation and with its gradient, of rows (1 x 128)
  matmul     the experts' products over the plan's instances from such blocks,
             forward, and as a backward step (input and weight gradients)
  combine    the sum of expert rows by given weights, and its gradient

`run` computes them in elementary torch operations, or, where `own` is true,
through load_balance_planning_amd.Layer.
"""
import math

import numpy as np
import torch

own = False
BLK = 128          # columns (and, for weights, rows) of one scale
E4M3_MAX = 448.0


# ---- cases -------------------------------------------------------------------

def _gate(name, T, E, k, R, score, bias, n_group, topk_group, renorm, scale, train):
    return dict(name=name, op="gate", T=T, E=E, k=k, R=R, score=score, bias=bias, n_group=n_group,
                topk_group=topk_group, renorm=renorm, scale=scale, train=train)


def _rows(name, op, rows, F):
    return dict(name=name, op=op, rows=rows, F=F)


def _experts(name, op, T, E, k, B, N, K, skew):
    return dict(name=name, op=op, T=T, E=E, k=k, B=B, N=N, K=K, skew=skew)


def listed():
    return [
        # one decoding step of 64 sequences on the DeepSeek-V3-shaped layer: latency
        _gate("gate_decode", 64, 256, 8, 8, "sigmoid", True, 8, 4, True, 2.5, False),
        # a prefill batch of the Qwen3-shaped layer: plain softmax routing
        _gate("gate_prefill", 16384, 128, 8, 8, "softmax", False, 1, 1, True, 1.0, False),
        # a training batch of the DeepSeek-V3-shaped layer, forward and backward
        _gate("gate_train", 32768, 256, 8, 64, "sigmoid", True, 8, 4, True, 2.5, True),
        # the Qwen3-shaped layer's gate and up weights, both layouts, as after an optimizer step
        dict(name="quantize_weights", op="quantize_weights", E=128, N=1536, K=2048),
        # between the two products of the Qwen3-shaped layer, a training batch
        _rows("swiglu", "swiglu", 131072, 768),
        # its gradient at the DeepSeek-V3-shaped width, a ragged number of rows
        _rows("swiglu_grad", "swiglu_grad", 5003, 2688),
        # first product of a decoding step of 64 sequences: a few rows an expert, bound by the weights
        _experts("matmul_decode", "matmul", 64, 128, 8, 16, 1536, 2048, 1.0),
        # first product of a prefill chunk: 32 experts of the DeepSeek-V3-shaped width, four replicas
        _experts("matmul_prefill", "matmul", 4096, 32, 8, 4, 5376, 7168, 0.5),
        # backward of a small odd layer: widths that are no multiple of a block, an odd number of tokens
        _experts("grads_odd", "grads", 999, 8, 2, 0, 760, 1000, 0.7),
        # backward of the Qwen3-shaped layer's first product, a training batch with its replicas
        _experts("grads_train", "grads", 16384, 128, 8, 16, 1536, 2048, 0.5),
        # the return path of a decoding step of 64 sequences, DeepSeek-V3-shaped rows, forward and backward
        dict(name="combine_small", op="combine", T=64, k=8, H=7168),
        # the return path of a training batch, forward and backward
        dict(name="combine_train", op="combine", T=8192, k=8, H=7168),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate", "quantize_weights", "swiglu", "swiglu_grad", "matmul", "matmul", "grads",
                     "combine"])
    if op == "gate":
        E = rng.choice([8, 64, 100, 128, 160, 256, 384, 512, 896])
        k = min(rng.choice([1, 2, 4, 6, 8, 16]), E // 4)
        n_group = rng.choice([g for g in (1, 1, 4, 8) if E % g == 0 and E // g >= 2])
        need = -(-k * n_group // E)
        topk_group = n_group if n_group == 1 else rng.randint(max(1, need), n_group)
        T = _log_int(rng, 1, 32768)
        while T * E > 32768 * 256:
            T //= 2
        R = rng.choice([r for r in (1, 2, 4, 8) if T % r == 0 and E % r == 0])
        c = _gate("", T, E, k, R, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, n_group, topk_group,
                  k > 1 and rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.random() < 0.5)
    elif op == "quantize_weights":
        c = dict(op=op, E=_log_int(rng, 1, 64), N=_log_int(rng, 40, 2000), K=_log_int(rng, 40, 2400))
    elif op in ("swiglu", "swiglu_grad"):
        rows = _log_int(rng, 1, 60000)
        c = _rows("", op, rows, _log_int(rng, 20, max(21, min(5000, 100663296 // rows))))
    elif op in ("matmul", "grads"):
        E = rng.choice([1, 4, 8, 16, 32, 64])
        k = min(E, rng.choice([1, 2, 4, 8]))
        T = _log_int(rng, 1, 32768 // k)
        N, K = _log_int(rng, 64, 3000), _log_int(rng, 64, 4000)
        c = _experts("", op, T, E, k, rng.choice([0, 0, min(E, 3)]), N, K, rng.choice([0.0, 0.5, 1.0]))
    else:
        T = _log_int(rng, 1, 8192)
        c = dict(op=op, T=T, k=rng.choice([1, 2, 4, 6, 8]), H=_log_int(rng, 24, 7168))
    c.pop("name", None)
    return c


# ---- inputs ------------------------------------------------------------------

def _device():
    return torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")


def _pad(n, m):
    return -(-n // m) * m


def _scale_exp(amax):
    """Exponent s of the smallest power of two with amax <= 448 * 2^s (0 for a block of zeros)."""
    m, e = torch.frexp(amax)                       # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    s = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _over(v, s):
    """v / 2^s without rounding: the power of two from its bits."""
    return v * ((127 - s).to(torch.int32) << 23).view(torch.float32)


def _quantize_rows(x):
    """fp32 rows [.., C] -> e4m3 [.., C padded to 128] and E8M0 [.., blocks padded to 4], one scale per 1 x 128."""
    C = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, _pad(C, BLK) - C))
    b = x.unflatten(-1, (-1, BLK))
    s = _scale_exp(b.abs().amax(-1))
    q = _over(b, s.unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)
    s = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, _pad(s.shape[-1], 4) - s.shape[-1]), value=127)
    return q, s.view(torch.float8_e8m0fnu)


def _quantize_weights(w):
    """bf16 [E, N, K] -> e4m3 [E, N, Kp] with E8M0 [E, N/128, K/128 padded to 4], and the same of the transpose."""
    E, N, K = w.shape
    Np, Kp = _pad(N, BLK), _pad(K, BLK)
    b = torch.nn.functional.pad(w.float(), (0, Kp - K, 0, Np - N)).view(E, Np // BLK, BLK, Kp // BLK, BLK)
    s = _scale_exp(b.abs().amax(4).amax(2))
    q = _over(b, s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(E, Np, Kp)
    pad4 = lambda v: torch.nn.functional.pad((v + 127).to(torch.uint8), (0, _pad(v.shape[-1], 4) - v.shape[-1]),
                                             value=127).contiguous().view(torch.float8_e8m0fnu)
    e4m3 = torch.float8_e4m3fn
    return (q[:, :N].contiguous().view(e4m3), pad4(s),
            q.transpose(1, 2)[:, :K].contiguous().view(e4m3), pad4(s.transpose(1, 2)))


def _instances(case, seed):
    """Rows per instance of a skewed layer: T * k rows over E experts, some with a replica, in rank-major order."""
    rng = np.random.RandomState(seed % (1 << 31))
    E, B, rows = case["E"], min(case["B"], case["E"]), case["T"] * case["k"]
    p = (1.0 + rng.permutation(E)) ** -case["skew"]
    count = rng.multinomial(rows, p / p.sum())
    hot = np.sort(np.argsort(-count, kind="stable")[:B])
    expert = np.concatenate([np.arange(E), hot])   # the last rank holds the replicas
    load = np.concatenate([count, count[hot] // 2])
    load[hot] -= count[hot] // 2
    return expert.astype(np.int32), np.concatenate([[0], np.cumsum(load)]).astype(np.int32), int(load.max())


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(int(seed))
    normal = lambda *s, dt=torch.float32: torch.randn(*s, generator=g, device=dev, dtype=torch.float32).to(dt)
    bf = torch.bfloat16
    op, st = case["op"], dict(case=case)
    shape = dict(T=8, E=8, k=1, R=1, G=1, H=8, B=0)  # the layer a handle is made for
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        shape.update(T=T, E=E, k=k, R=case["R"])
        st["logits"] = normal(T, E) + 0.5 * normal(E)
        st["bias"] = 0.05 * normal(E) if case["bias"] else None
        st["grad_weight"] = normal(T, k) if case["train"] else None
    elif op == "quantize_weights":
        st["w"] = 0.03 * normal(case["E"], case["N"], case["K"], dt=bf)
    elif op in ("swiglu", "swiglu_grad"):
        st["y"] = normal(case["rows"], 2 * case["F"], dt=bf)
        if op == "swiglu_grad":
            st["grad"] = (1e-3 * normal(case["rows"], case["F"])).to(bf)
    elif op in ("matmul", "grads"):
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        shape.update(T=T, E=E, k=k, B=case["B"])
        expert, offset, most = _instances(case, int(seed))
        pad = lambda a, n: torch.from_numpy(np.concatenate([a, np.full(n - len(a), -1, np.int32)])).to(dev)
        st["most_rows"], st["instances"] = most, len(expert)
        st["n_inst"] = torch.tensor([len(expert)], dtype=torch.int32, device=dev)
        st["inst_expert"], st["inst_offset"] = pad(expert, E + case["B"]), pad(offset, E + case["B"] + 1)
        st["x"] = _quantize_rows(normal(T * k, K, dt=bf).float())
        w = _quantize_weights((normal(E, N, K) / math.sqrt(K)).to(bf))
        if op == "matmul":
            st["w"] = w[:2]
        else:
            st["wt"], st["dy"] = w[2:], (1e-3 * normal(T * k, N)).to(bf)
    else:
        T, k, H = case["T"], case["k"], case["H"]
        shape.update(T=T, E=max(8, k), k=k, H=H)
        st["expert_out"], st["grad_out"] = normal(T * k, H, dt=bf), normal(T, H, dt=bf)
        st["weight"] = torch.softmax(normal(T, k), -1)
        st["slot_pos"] = torch.randperm(T * k, generator=g, device=dev).to(torch.int32)
    if own:
        import load_balance_planning_amd as mp
        layer = st["layer"] = mp.Layer(mp.make_config(**shape), cooc=False, topk_val=False)
        if op == "gate":
            st["gate"] = mp.make_gate(case["score"], case["n_group"], case["topk_group"], 2, case["renorm"],
                                      case["scale"])
        elif op in ("matmul", "grads"):
            st["plan"] = mp.PlanBuffers(st["n_inst"], st["inst_expert"], None, None, None, None, None, None)
            st["x"] = mp.Blocks(*st["x"], case["K"])
            if op == "matmul":
                st["w"] = mp.Blocks(*st["w"], case["K"])
            else:
                st["wt"] = mp.Blocks(*st["wt"], case["N"])
        layer.status()
    return st


# ---- one pass ----------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st, st["layer"])
    return _PLAIN[op](st, st["case"])


def _own_gate(st, layer):
    r, weight = layer.gate(st["logits"], st["gate"], bias=st["bias"])
    out = dict(topk_idx=r.topk_idx, weight=weight, expert_count=r.expert_count, omega=r.omega)
    if st["grad_weight"] is not None:
        out["grad_logits"] = layer.gate_grad(st["logits"], st["gate"], st["grad_weight"])
    return out


def _own_quantize_weights(st, layer):
    w, wt = layer.quantize_weights(st["w"], transposed=True)
    return dict(q=w.q, scale=w.scale, qt=wt.q, scale_t=wt.scale)


def _own_swiglu(st, layer):
    b = layer.swiglu(st["y"])
    return dict(q=b.q, scale=b.scale)


def _own_swiglu_grad(st, layer):
    b = layer.swiglu_grad(st["y"], st["grad"])
    return dict(q=b.q, scale=b.scale)


def _own_matmul(st, layer):
    return dict(y=layer.matmul(st["x"], st["w"], plan=st["plan"], inst_offset=st["inst_offset"]))


def _own_grads(st, layer):
    dy = layer.quantize(st["dy"])
    return dict(dx=layer.matmul(dy, st["wt"], plan=st["plan"], inst_offset=st["inst_offset"]),
                dw=layer.wgrad(dy, st["x"], plan=st["plan"], inst_offset=st["inst_offset"]))


def _own_combine(st, layer):
    out = layer.combine_weighted(st["expert_out"], st["weight"], slot_pos=st["slot_pos"])
    grad_rows, grad_weight = layer.combine_grad(st["expert_out"], st["grad_out"], st["weight"],
                                                slot_pos=st["slot_pos"])
    return dict(out=out, grad_expert_out=grad_rows, grad_weight=grad_weight)


_OWN = dict(gate=_own_gate, quantize_weights=_own_quantize_weights, swiglu=_own_swiglu, swiglu_grad=_own_swiglu_grad,
            matmul=_own_matmul, grads=_own_grads, combine=_own_combine)


def _scores(logits, case):
    if case["score"] == "softmax":
        z = torch.exp(logits - logits.amax(-1, keepdim=True))
        return z / z.sum(-1, keepdim=True)
    return 1.0 / (1.0 + torch.exp(-logits))


def _plain_gate(st, case):
    # 64 bits: two experts' choice values may lie closer than 32 bits tell apart
    T, E, k, G = case["T"], case["E"], case["k"], case["n_group"]
    score = _scores(st["logits"].double(), case)
    choice = score if st["bias"] is None else score + st["bias"].double()
    order = st["logits"].double() if st["bias"] is None else choice
    if G > 1:
        best = torch.sort(choice.view(T, G, E // G), dim=-1, descending=True).values[..., :2].sum(-1)
        at = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :case["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=at.device).scatter_(1, at, True)
        order = torch.where(keep.repeat_interleave(E // G, 1), order, torch.full_like(order, -math.inf))
    idx = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :k]
    s = score.gather(1, idx)
    weight = case["scale"] * (s / (s.sum(-1, keepdim=True) + 1e-20) if case["renorm"] else s)
    slot = torch.arange(T * k, device=idx.device)
    source = slot // k // (T // case["R"])
    flat = source * E + idx.reshape(-1)
    omega = torch.zeros(case["R"] * E, dtype=torch.int32, device=idx.device)
    omega = omega.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32)).view(case["R"], E)
    out = dict(topk_idx=idx.to(torch.int32), weight=weight.float(), expert_count=omega.sum(0, dtype=torch.int32),
               omega=omega)
    if st["grad_weight"] is not None:
        out["grad_logits"] = _plain_gate_grad(st["logits"], idx, st["grad_weight"], case)
    return out


def _plain_gate_grad(logits, idx, grad_weight, case):
    score = _scores(logits, case)
    s = score.gather(1, idx)
    if case["renorm"]:
        total = s.sum(-1, keepdim=True) + 1e-20
        ds = case["scale"] / total * (grad_weight - (grad_weight * s).sum(-1, keepdim=True) / total)
    else:
        ds = case["scale"] * grad_weight
    grad = torch.zeros_like(score).scatter_(1, idx, ds)
    if case["score"] == "softmax":
        return score * (grad - (s * ds).sum(-1, keepdim=True))
    return grad * score * (1.0 - score)


def _plain_quantize_weights(st, case):
    q, s, qt, t = _quantize_weights(st["w"])
    return dict(q=q, scale=s, qt=qt, scale_t=t)


def _plain_swiglu(st, case):
    gate, up = st["y"].float().split(case["F"], -1)
    q, s = _quantize_rows(gate / (1.0 + torch.exp(-gate)) * up)
    return dict(q=q, scale=s)


def _plain_swiglu_grad(st, case):
    gate, up = st["y"].float().split(case["F"], -1)
    da = st["grad"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dgate = da * up * (sig * (1.0 + gate * (1.0 - sig)))
    q, s = _quantize_rows(torch.cat([dgate, da * (gate * sig)], -1))
    return dict(q=q, scale=s)


def _values(q, s, rows=None):
    """fp32 values of e4m3 rows [.., C] with their E8M0 scales (rows: scales of 128-row blocks)."""
    s = s[..., : q.shape[-1] // BLK].float()
    if rows is not None:
        s = s.repeat_interleave(BLK, -2)[..., :rows, :]
    return (q.float().unflatten(-1, (-1, BLK)) * s.unsqueeze(-1)).flatten(-2)


def _place(st):
    """Instance of every row and its place in it."""
    n = st["instances"]
    row = torch.arange(st["case"]["T"] * st["case"]["k"], device=st["inst_offset"].device)
    inst = torch.searchsorted(st["inst_offset"][1:n + 1].contiguous(), row.to(torch.int32), right=True)
    return inst, row - st["inst_offset"][inst]


def _padded(v, inst, at, st):
    out = torch.zeros(st["instances"], st["most_rows"], v.shape[1], device=v.device)
    out[inst, at] = v
    return out


def _plain_product(q, w, rows, cols, st):
    inst, at = _place(st)
    x = _padded(_values(*q), inst, at, st)
    wv = _values(*w, rows=rows)[st["inst_expert"][:st["instances"]].long()]
    return torch.bmm(x, wv.transpose(1, 2).contiguous())[inst, at].to(torch.bfloat16)


def _plain_matmul(st, case):
    return dict(y=_plain_product(st["x"], st["w"], case["N"], case["K"], st))


def _plain_grads(st, case):
    dy = _quantize_rows(st["dy"].float())
    dx = _plain_product(dy, st["wt"], case["K"], case["N"], st)
    inst, at = _place(st)
    a = _padded(_values(*dy)[:, :case["N"]], inst, at, st)
    b = _padded(_values(*st["x"])[:, :case["K"]], inst, at, st)
    each = torch.bmm(a.transpose(1, 2).contiguous(), b)
    dw = torch.zeros(case["E"], case["N"], case["K"], device=each.device)
    dw.index_add_(0, st["inst_expert"][:st["instances"]], each)
    return dict(dx=dx, dw=dw.to(torch.bfloat16))


def _plain_combine(st, case):
    T, k, H = case["T"], case["k"], case["H"]
    pos = st["slot_pos"].long()
    rows, w, g = st["expert_out"][pos].float().view(T, k, H), st["weight"], st["grad_out"].float()
    out = (w.unsqueeze(-1) * rows).sum(1)
    grad_rows = torch.empty_like(st["expert_out"])
    grad_rows[pos] = (w.unsqueeze(-1) * g.unsqueeze(1)).view(T * k, H).to(torch.bfloat16)
    return dict(out=out.to(torch.bfloat16), grad_expert_out=grad_rows, grad_weight=(rows * g.unsqueeze(1)).sum(-1))


_PLAIN = dict(gate=_plain_gate, quantize_weights=_plain_quantize_weights, swiglu=_plain_swiglu,
              swiglu_grad=_plain_swiglu_grad, matmul=_plain_matmul, grads=_plain_grads, combine=_plain_combine)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        b = T * E * 4 + T * k * 8 + (case["R"] + 1) * E * 4
        if case["train"]:
            b += T * k * 8 + T * E * 8
        return dict(bytes=b, flops=T * E * (20 if case["train"] else 10))
    if op == "quantize_weights":
        return dict(bytes=case["E"] * case["N"] * case["K"] * 4, flops=case["E"] * case["N"] * case["K"] * 4)
    if op == "swiglu":
        return dict(bytes=case["rows"] * case["F"] * 5, flops=case["rows"] * case["F"] * 12)
    if op == "swiglu_grad":
        return dict(bytes=case["rows"] * case["F"] * 8, flops=case["rows"] * case["F"] * 20)
    if op in ("matmul", "grads"):
        rows, E, N, K = case["T"] * case["k"], case["E"], case["N"], case["K"]
        used = min(E, rows)
        if op == "matmul":
            return dict(bytes=rows * K + used * N * K + 2 * rows * N, flops=2 * rows * N * K)
        return dict(bytes=rows * K + used * N * K + 2 * rows * N + 2 * rows * K + 2 * E * N * K, flops=4 * rows * N * K)
    T, k, H = case["T"], case["k"], case["H"]
    return dict(bytes=T * k * H * 4 + T * H * 4 + T * k * 12, flops=T * k * H * 5)


# ---- the definitions in 64 bits ----------------------------------------------

def _e4m3(v):
    """Nearest e4m3 value of |v| <= 448, ties to the even one, as float64."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _blocks64(v, rows=1):
    """(values of e4m3, scales) of float64 [.., n, C] in blocks of rows x 128, padded with zeros."""
    n, C = v.shape[-2:]
    np_, cp = _pad(n, rows), _pad(C, BLK)
    p = torch.zeros(*v.shape[:-2], np_, cp, dtype=torch.float64, device=v.device)
    p[..., :n, :C] = v
    p = p.unflatten(-1, (-1, BLK)).unflatten(-3, (-1, rows))            # .., n/rows, rows, C/128, 128
    top = p.abs().amax(-1).amax(-2)
    s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -130) / E4M3_MAX)).clamp(min=-126))
    s = torch.where(top > 0, s, torch.ones_like(s))
    q = _e4m3(p / s.unsqueeze(-2).unsqueeze(-1)).flatten(-2).flatten(-3, -2)[..., :n, :]
    full = torch.ones(*s.shape[:-1], _pad(s.shape[-1], 4), dtype=torch.float64, device=v.device)
    full[..., : s.shape[-1]] = s
    return q, full


def _read64(blocks, rows, n, cols):
    """float64 [.., n, cols] of stored blocks."""
    q, s = blocks[0].double()[..., :n, :cols], blocks[1].double()
    s = s.repeat_interleave(rows, -2)[..., :n, :] if rows > 1 else s
    return q * s.repeat_interleave(BLK, -1)[..., :cols]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return _exact_gate(st, case)
    if op == "quantize_weights":
        w = st["w"].double()
        q, s = _blocks64(w, BLK)
        qt, t = _blocks64(w.transpose(1, 2).contiguous(), BLK)
        return dict(q=q, scale=s, qt=qt, scale_t=t)
    if op in ("swiglu", "swiglu_grad"):
        y = st["y"].double().requires_grad_(op == "swiglu_grad")
        a = torch.nn.functional.silu(y[:, : case["F"]]) * y[:, case["F"]:]
        if op == "swiglu_grad":
            a, = torch.autograd.grad(a, y, st["grad"].double())
        q, s = _blocks64(a)
        return dict(q=q, scale=s)
    if op in ("matmul", "grads"):
        return _exact_experts(st, case)
    T, k, H = case["T"], case["k"], case["H"]
    rows, w = st["expert_out"].double().requires_grad_(), st["weight"].double().requires_grad_()
    out = (rows[st["slot_pos"].long()].view(T, k, H) * w[:, :, None]).sum(1)
    grad_rows, grad_weight = torch.autograd.grad(out, (rows, w), st["grad_out"].double())
    return dict(out=out.detach(), grad_expert_out=grad_rows, grad_weight=grad_weight)


def _exact_gate(st, case):
    T, E, k, G = case["T"], case["E"], case["k"], case["n_group"]
    x = st["logits"].double().requires_grad_(bool(case["train"]))
    score = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    with torch.no_grad():
        choice = score if st["bias"] is None else score + st["bias"].double()
        rank = x.detach().clone() if st["bias"] is None else choice.clone()
        if G > 1:
            total = choice.view(T, G, -1).topk(2, -1).values.sum(-1)
            # place of a group: the groups with a larger sum, and the earlier ones with the same
            ahead = (total[:, None, :] > total[:, :, None]).sum(-1)
            same = ((total[:, None, :] == total[:, :, None]) & torch.ones(G, G, device=x.device).tril(-1).bool()).sum(-1)
            rank.view(T, G, -1)[(ahead + same) >= case["topk_group"]] = -math.inf
        idx = rank.argsort(dim=-1, descending=True, stable=True)[:, :k]
    s = score.gather(1, idx)
    weight = case["scale"] * (s / (s.sum(-1, keepdim=True) + 1e-20) if case["renorm"] else s)
    count = torch.nn.functional.one_hot(idx, E).sum(1).view(case["R"], -1, E).sum(1)
    out = dict(topk_idx=idx.to(torch.int32), weight=weight.detach(), expert_count=count.sum(0).to(torch.int32),
               omega=count.to(torch.int32))
    if case["train"]:
        out["grad_logits"], = torch.autograd.grad(weight, x, st["grad_weight"].double())
    return out


def _exact_experts(st, case):
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    if T * k * N * K > 3e12:
        return None
    offset, expert = st["inst_offset"].tolist(), st["inst_expert"].tolist()
    x = _read64(st["x"], 1, T * k, K)
    spans = [(expert[i], offset[i], offset[i + 1]) for i in range(st["instances"])]
    if case["op"] == "matmul":
        y = torch.zeros(T * k, N, dtype=torch.float64, device=x.device)
        for e, a, b in spans:
            y[a:b] = x[a:b] @ _read64((st["w"][0][e], st["w"][1][e]), BLK, N, K).t()
        return dict(y=y)
    dy = _read64(_blocks64(st["dy"].double()), 1, T * k, N)
    dx = torch.zeros(T * k, K, dtype=torch.float64, device=x.device)
    dw = torch.zeros(E, N, K, dtype=torch.float64, device=x.device)
    for e, a, b in spans:
        dx[a:b] = dy[a:b] @ _read64((st["wt"][0][e], st["wt"][1][e]), BLK, K, N).t()
        dw[e] += dy[a:b].t() @ x[a:b]
    return dict(dx=dx, dw=dw)
