"""The expert layer's 4-bit operators, and the layer of a few tokens, as a program calls them: what is timed, on which sizes.

  quantize  e2m1 values with one power-of-two scale per block of 32 along the
            summed axis: of rows, and of expert matrices in both layouts; and
            the values back
  down      the gated activation quantized so, and the experts' product after it
  product   the experts' products of rows in 4 or 8 bits with 4-bit matrices;
            as a training step also the input gradient
  few       a whole layer's experts for at most 64 tokens, from their top-k and
            weights to the combined rows, matrices in 4 or 8 bits

`run` computes them in elementary torch operations, or, where `own` is true,
through load_balance_planning_amd.Layer.
"""
import math

import numpy as np
import torch

own = False
E2M1_MAX, E4M3_MAX = 6.0, 448.0


# ---- cases -------------------------------------------------------------------

def _rows(name, rows, K):
    return dict(name=name, op="rows", rows=rows, K=K)


def _down(name, T, E, k, B, N, F, skew):
    return dict(name=name, op="down", T=T, E=E, k=k, B=B, N=N, K=F, skew=skew)


def _product(name, T, E, k, B, N, K, skew, bits, train):
    return dict(name=name, op="product", T=T, E=E, k=k, B=B, N=N, K=K, skew=skew, bits=bits, train=train)


def _few(name, T, E, k, H, F, bits, skew):
    return dict(name=name, op="few", T=T, E=E, k=k, H=H, F=F, bits=bits, skew=skew)


def listed():
    return [
        # the Qwen3-shaped layer's gate and up matrices, both layouts, as quantization-aware training takes them
        dict(name="weights_train", op="weights", E=128, N=1536, K=2048),
        # the rows of a decoding step of 64 sequences of that layer: latency
        _rows("rows_decode", 512, 2048),
        # activation and second product of a prefill chunk: 32 experts of the DeepSeek-V3-shaped width, four replicas
        _down("down_prefill", 4096, 32, 8, 4, 7168, 2688, 0.5),
        # the same of a small odd layer: widths that are no multiple of a block
        _down("down_odd", 999, 8, 2, 0, 1000, 380, 0.7),
        # first product of a decoding step of 64 sequences, rows in 8 bits: bound by the matrices
        _product("product_decode", 64, 128, 8, 16, 1536, 2048, 1.0, 8, False),
        # first product of a prefill chunk at the DeepSeek-V3-shaped width, rows in 4 bits
        _product("product_prefill", 4096, 32, 8, 4, 5376, 7168, 0.5, 4, False),
        # a training batch through the Qwen3-shaped layer's first product and back, rows and gradients in 8 bits
        _product("product_train", 16384, 128, 8, 16, 1536, 2048, 0.5, 8, True),
        # one sequence's next token through the Qwen3-shaped layer: latency
        _few("few_one", 1, 128, 8, 2048, 768, 4, 0.0),
        # a small batch of sequences, matrices in 8 bits
        _few("few_eight_bit", 16, 128, 8, 2048, 768, 8, 0.5),
        # the most sequences that the call takes: nearly every expert has a token
        _few("few_most", 64, 128, 8, 2048, 768, 4, 0.5),
        # wide rows: eight sequences at the DeepSeek-V3-shaped width, 32 experts
        _few("few_wide", 8, 32, 8, 7168, 2688, 4, 0.0),
        # a small layer of odd widths, matrices in 8 bits
        _few("few_odd", 7, 8, 2, 1000, 380, 8, 0.7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weights", "rows", "down", "product", "product", "product", "few", "few", "few", "few"])
    if op == "weights":
        return dict(op=op, E=_log_int(rng, 1, 64), N=_log_int(rng, 40, 2000), K=_log_int(rng, 40, 2400))
    if op == "rows":
        rows = _log_int(rng, 1, 60000)
        c = _rows("", rows, _log_int(rng, 20, max(21, min(7168, 100663296 // rows))))
    elif op == "few":
        E = rng.choice([1, 4, 8, 16, 32, 64, 100, 128])
        k = min(E, rng.choice([1, 2, 4, 6, 8]))
        H = _log_int(rng, 64, 4000)
        F = _log_int(rng, 32, max(33, min(2700, 402653184 // (E * H))))
        c = _few("", _log_int(rng, 1, 64), E, k, H, F, rng.choice([4, 4, 8]), rng.choice([0.0, 0.5, 1.0]))
    else:
        E = rng.choice([1, 4, 8, 16, 32, 64])
        k = min(E, rng.choice([1, 2, 4, 8]))
        T = _log_int(rng, 1, 32768 // k)
        N, K, B, skew = _log_int(rng, 64, 3000), _log_int(rng, 64, 4000), rng.choice([0, 0, min(E, 3)]), \
            rng.choice([0.0, 0.5, 1.0])
        if op == "down":
            c = _down("", T, E, k, B, N, K, skew)
        else:
            c = _product("", T, E, k, B, N, K, skew, rng.choice([4, 8]), rng.random() < 0.4)
    c.pop("name")
    return c


# ---- inputs ------------------------------------------------------------------

def _device():
    return torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")


def _pad(n, m):
    return -(-n // m) * m


def _scale_exp(amax, most):
    """Exponent s of the smallest power of two with amax <= most * 2^s, at least -126 (0 for a block of zeros)."""
    m, e = torch.frexp(amax)                          # amax = m * 2^e, 0.5 <= m < 1
    mm, me = math.frexp(most)
    s = (e - me + (m > mm).to(e.dtype)).clamp(min=-126)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _over(v, s):
    """v / 2^s without rounding: the power of two from its bits."""
    return v * ((127 - s).to(torch.int32) << 23).view(torch.float32)


def _two(s):
    """2^s in fp32, s from -126 to 127."""
    return ((127 + s).to(torch.int32) << 23).view(torch.float32)


def _to_e2m1(v):
    """Nearest e2m1 value of |v| <= 6, ties to the even one: steps of 0.5 below 2, 1 below 4, 2 above."""
    a = v.abs()
    step = 0.5 + 0.5 * (a >= 2).float() + (a >= 4).float()
    return torch.round(v / step) * step


def _blocks(x, width, size, most):
    """fp32 [.., C] padded with zeros to a multiple of width, in blocks of size: (blocks over their scale, exponents)."""
    x = torch.nn.functional.pad(x, (0, _pad(x.shape[-1], width) - x.shape[-1]))
    b = x.unflatten(-1, (-1, size))
    s = _scale_exp(b.abs().amax(-1), most)
    return _over(b, s.unsqueeze(-1)), s


def _scale_rows(s):
    """Exponents [.., rows, Kp/32] as scale bytes [.., Kp/256, rows, 8]."""
    return (s + 127).to(torch.uint8).unflatten(-1, (-1, 8)).transpose(-2, -3).contiguous().view(torch.float8_e8m0fnu)


def _pack4(v):
    """e2m1 values [.., 2 n] as n bytes, the first value in the low half: an e4m3 byte of v / 64 holds the code."""
    b = (v / 64).to(torch.float8_e4m3fn).view(torch.uint8)
    code = ((b >> 4) & 8) | ((b >> 2) & 7)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _quantize4(x):
    """fp32 rows [.., C] -> packed e2m1 [.., Kp/2] and E8M0 [.., Kp/256, rows, 8]."""
    b, s = _blocks(x, 256, 32, E2M1_MAX)
    return _pack4(_to_e2m1(b).flatten(-2)), _scale_rows(s)


def _quantize8(x):
    """fp32 rows [.., C] -> e4m3 [.., C padded to 128] and E8M0 [.., blocks padded to 4], one scale per 1 x 128."""
    b, s = _blocks(x, 128, 128, E4M3_MAX)
    s = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, _pad(s.shape[-1], 4) - s.shape[-1]), value=127)
    return b.to(torch.float8_e4m3fn).flatten(-2), s.view(torch.float8_e8m0fnu)


def _quantize8_weights(w):
    """fp32 [E, N, K] -> e4m3 [E, N, Kp] with E8M0 [E, N/128, K/128 padded to 4]."""
    E, N, K = w.shape
    Np, Kp = _pad(N, 128), _pad(K, 128)
    b = torch.nn.functional.pad(w, (0, Kp - K, 0, Np - N)).view(E, Np // 128, 128, Kp // 128, 128)
    s = _scale_exp(b.abs().amax(4).amax(2), E4M3_MAX)
    q = _over(b, s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(E, Np, Kp)[:, :N].contiguous()
    s = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, _pad(s.shape[-1], 4) - s.shape[-1]), value=127)
    return q.view(torch.float8_e4m3fn), s.contiguous().view(torch.float8_e8m0fnu)


def _matrices(normal, E, N, K, bits):
    """Quantized normal matrices of variance 1 / K, some experts at a time (fp32 copies of all would not fit three times)."""
    q, s = [], []
    some = max(1, (1 << 28) // (N * K))
    for e in range(0, E, some):
        w = (normal(min(some, E - e), N, K) / math.sqrt(K)).to(torch.bfloat16).float()
        a, b = _quantize4(w) if bits == 4 else _quantize8_weights(w)
        q.append(a)
        s.append(b.view(torch.uint8))
    q = torch.cat([v.view(torch.uint8) for v in q])
    return q if bits == 4 else q.view(torch.float8_e4m3fn), torch.cat(s).view(torch.float8_e8m0fnu)


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
    normal = lambda *s: torch.randn(*s, generator=g, device=dev, dtype=torch.float32)
    bf = torch.bfloat16
    op, st = case["op"], dict(case=case)
    shape = dict(T=8, E=8, k=1, R=1, G=1, H=8, B=0)  # the layer a handle is made for
    if op == "weights":
        st["w"] = (0.03 * normal(case["E"], case["N"], case["K"])).to(bf)
    elif op == "rows":
        st["x"] = normal(case["rows"], case["K"]).to(bf)
    elif op == "few":
        T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
        shape.update(T=T, E=E, k=k, H=H)
        hot = torch.log(1.0 + torch.randperm(E, generator=g, device=dev).float())
        top = torch.sort(normal(T, E) - case["skew"] * hot, dim=-1, descending=True)
        st["topk_idx"] = top.indices[:, :k].to(torch.int32).contiguous()
        st["weight"] = torch.softmax(top.values[:, :k], -1).contiguous()
        st["most_rows"] = int(torch.bincount(st["topk_idx"].reshape(-1), minlength=E).max())
        st["hidden"] = normal(T, H).to(bf)
        st["w1"] = _matrices(normal, E, 2 * F, H, case["bits"])
        st["w2"] = _matrices(normal, E, H, F, case["bits"])
    else:
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        shape.update(T=T, E=E, k=k, B=case["B"])
        expert, offset, most = _instances(case, int(seed))
        pad = lambda a, n: torch.from_numpy(np.concatenate([a, np.full(n - len(a), -1, np.int32)])).to(dev)
        st["most_rows"], st["instances"] = most, len(expert)
        st["n_inst"] = torch.tensor([len(expert)], dtype=torch.int32, device=dev)
        st["inst_expert"], st["inst_offset"] = pad(expert, E + case["B"]), pad(offset, E + case["B"] + 1)
        st["w"] = _matrices(normal, E, N, K, 4)
        if op == "down":
            st["y"] = normal(T * k, 2 * K).to(bf)
        else:
            rows8 = lambda cols, by: _quantize8((by * normal(T * k, cols)).to(bf).float())
            st["x"] = rows8(K, 1.0) if case["bits"] == 8 else _quantize4(normal(T * k, K).to(bf).float())
            if case["train"]:
                st["wt"], st["dy"] = _matrices(normal, E, K, N, 4), rows8(N, 1e-3)
    if own:
        import load_balance_planning_amd as mp
        layer = st["layer"] = mp.Layer(mp.make_config(**shape), cooc=False, topk_val=False)
        four = lambda b, cols: mp.Blocks4(b[0].view(torch.float4_e2m1fn_x2), b[1], cols)
        rows = lambda b, cols: four(b, cols) if case["bits"] == 4 else mp.Blocks(*b, cols)
        if op == "few":
            st["w1"], st["w2"] = rows(st["w1"], case["H"]), rows(st["w2"], case["F"])
        elif op in ("down", "product"):
            st["plan"] = mp.PlanBuffers(st["n_inst"], st["inst_expert"], None, None, None, None, None, None)
            st["w"] = four(st["w"], case["K"])
            if op == "product":
                st["x"] = rows(st["x"], case["K"])
                if case["train"]:
                    st["wt"], st["dy"] = four(st["wt"], case["N"]), mp.Blocks(*st["dy"], case["N"])
        layer.status()
    return st


# ---- one pass ----------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st, st["layer"])
    return _PLAIN[op](st, st["case"])


def _own_weights(st, layer):
    w, wt = layer.quantize_weights4(st["w"], transposed=True)
    return dict(scale=w.scale, values=layer.values4(w), scale_t=wt.scale, values_t=layer.values4(wt))


def _own_rows(st, layer):
    b = layer.quantize4(st["x"])
    return dict(scale=b.scale, values=layer.values4(b))


def _own_down(st, layer):
    return dict(y=layer.matmul4(layer.swiglu4(st["y"]), st["w"], plan=st["plan"], inst_offset=st["inst_offset"]))


def _own_product(st, layer):
    on = dict(plan=st["plan"], inst_offset=st["inst_offset"])
    out = dict(y=layer.matmul4(st["x"], st["w"], **on))
    if st["case"]["train"]:
        out["dx"] = layer.matmul4(st["dy"], st["wt"], **on)
    return out


def _own_few(st, layer):
    return dict(out=layer.experts(st["hidden"], st["weight"], st["w1"], st["w2"], topk_idx=st["topk_idx"]))


_OWN = dict(weights=_own_weights, rows=_own_rows, down=_own_down, product=_own_product, few=_own_few)


def _fake4(x):
    """(scale bytes, bf16 values) of fp32 [.., rows, C] in 4-bit blocks."""
    b, s = _blocks(x, 256, 32, E2M1_MAX)
    v = (_to_e2m1(b) * _two(s).unsqueeze(-1)).flatten(-2)[..., : x.shape[-1]]
    return _scale_rows(s), v.to(torch.bfloat16)


def _plain_weights(st, case):
    w = st["w"].float()
    s, v = _fake4(w)
    t, vt = _fake4(w.transpose(1, 2).contiguous())
    return dict(scale=s, values=v, scale_t=t, values_t=vt)


def _plain_rows(st, case):
    s, v = _fake4(st["x"].float())
    return dict(scale=s, values=v)


def _values4(q, s, cols):
    """fp32 values [.., rows, cols] of packed e2m1 (as e4m3 bytes of their 64th part) with their scales."""
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    v = (((code & 8) << 4) | ((code & 7) << 2)).view(torch.float8_e4m3fn).float() * 64
    s = s.float().transpose(-2, -3).flatten(-2)                      # [.., rows, Kp/32]
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)[..., :cols]


def _values8(q, s, cols, rows=None):
    """fp32 values [.., cols] of e4m3 rows with their scales (rows: scales of 128-row blocks)."""
    s = s[..., : q.shape[-1] // 128].float()
    if rows is not None:
        s = s.repeat_interleave(128, -2)[..., :rows, :]
    return (q.float().unflatten(-1, (-1, 128)) * s.unsqueeze(-1)).flatten(-2)[..., :cols]


def _place(st):
    """Instance of every row and its place in it."""
    n = st["instances"]
    row = torch.arange(st["case"]["T"] * st["case"]["k"], device=st["inst_offset"].device)
    inst = torch.searchsorted(st["inst_offset"][1:n + 1].contiguous(), row.to(torch.int32), right=True)
    return inst, row - st["inst_offset"][inst]


def _plain_experts(x, w, rows, cols, st):
    """Rows [T*k, cols] by their instances' matrices [rows, cols] in fp32."""
    inst, at = _place(st)
    p = torch.zeros(st["instances"], st["most_rows"], cols, device=x.device)
    p[inst, at] = x
    wv = _values4(*w, cols)[st["inst_expert"][:st["instances"]].long()]
    return torch.bmm(p, wv.transpose(1, 2).contiguous())[inst, at].to(torch.bfloat16)


def _silu_times(y, F):
    gate, up = y[..., :F], y[..., F:]
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_down(st, case):
    b, s = _blocks(_silu_times(st["y"].float(), case["K"]), 256, 32, E2M1_MAX)
    a = (_to_e2m1(b) * _two(s).unsqueeze(-1)).flatten(-2)[..., : case["K"]]
    return dict(y=_plain_experts(a, st["w"], case["N"], case["K"], st))


def _plain_product(st, case):
    x = _values4(*st["x"], case["K"]) if case["bits"] == 4 else _values8(*st["x"], case["K"])
    out = dict(y=_plain_experts(x, st["w"], case["N"], case["K"], st))
    if case["train"]:
        out["dx"] = _plain_experts(_values8(*st["dy"], case["N"]), st["wt"], case["K"], case["N"], st)
    return out


def _through8(x):
    """fp32 rows after rounding to e4m3 with one scale per 1 x 32."""
    b, s = _blocks(x, 32, 32, E4M3_MAX)
    return (b.to(torch.float8_e4m3fn).float() * _two(s).unsqueeze(-1)).flatten(-2)[..., : x.shape[-1]]


def _plain_few(st, case):
    T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
    expert = st["topk_idx"].reshape(-1).long()
    if T * k < E:  # a matrix for every slot
        used, at = expert, (torch.arange(T * k, device=expert.device), torch.zeros_like(expert))
        n, most = T * k, 1
    else:          # every expert's rows one behind the other
        order = torch.sort(expert, stable=True).indices
        ahead = torch.cumsum(torch.bincount(expert, minlength=E), 0) - torch.bincount(expert, minlength=E)
        place = torch.empty_like(expert)
        place[order] = torch.arange(T * k, device=expert.device) - ahead[expert[order]]
        used, at = torch.arange(E, device=expert.device), (expert, place)
        n, most = E, st["most_rows"]

    def product(rows, w, N, K):
        p = torch.zeros(n, most, K, device=rows.device)
        p[at] = rows
        q, s = w[0].view(torch.uint8)[used], w[1].view(torch.uint8)[used].view(torch.float8_e8m0fnu)
        wv = _values4(q, s, K) if case["bits"] == 4 else _values8(q.view(torch.float8_e4m3fn), s, K, rows=N)
        return torch.bmm(p, wv.transpose(1, 2).contiguous())[at]

    x = _through8(st["hidden"].float()).repeat_interleave(k, 0)
    a = _through8(_silu_times(product(x, st["w1"], 2 * F, H), F))
    y = product(a, st["w2"], H, F).view(T, k, H)
    return dict(out=(st["weight"].unsqueeze(-1) * y).sum(1).to(torch.bfloat16))


_PLAIN = dict(weights=_plain_weights, rows=_plain_rows, down=_plain_down, product=_plain_product, few=_plain_few)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    op, four = case["op"], 0.5 + 1 / 32
    if op in ("weights", "rows"):
        n = case["rows"] * case["K"] if op == "rows" else case["E"] * case["N"] * case["K"]
        each = 2 + 2 + 1 / 32 if op == "rows" else 2 + 2 * (2 + 1 / 32)
        return dict(bytes=n * each, flops=n * (4 if op == "rows" else 8))
    if op == "few":
        T, k, H, F = (case[n] for n in ("T", "k", "H", "F"))
        used = min(case["E"], T * k)
        return dict(bytes=used * 3 * F * H * (four if case["bits"] == 4 else 1) + 4 * T * H + 8 * T * k,
                    flops=2 * T * k * 3 * F * H)
    rows, N, K = case["T"] * case["k"], case["N"], case["K"]
    matrices = min(case["E"], rows) * N * K * four
    if op == "down":
        return dict(bytes=4 * rows * K + matrices + 2 * rows * N, flops=2 * rows * N * K + 12 * rows * K)
    b = rows * K * (four if case["bits"] == 4 else 1) + matrices + 2 * rows * N
    if case["train"]:
        b += rows * N + matrices + 2 * rows * K
    return dict(bytes=b, flops=2 * rows * N * K * (2 if case["train"] else 1))


# ---- the definitions in 64 bits ----------------------------------------------

_CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_blocks(v, most):
    """Blocks of 32 of float64 [.., C] (C padded with zeros) and the power of two that each is divided by."""
    p = torch.zeros(*v.shape[:-1], _pad(v.shape[-1], 256), dtype=torch.float64, device=v.device)
    p[..., : v.shape[-1]] = v
    p = p.unflatten(-1, (-1, 32))
    top = p.abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -150) / most)).clamp(min=-126))
    return p, torch.where(top > 0, s, torch.ones_like(s))


def _exact4(v):
    """float64 [.., C] rounded in 4-bit blocks, and the scales [.., Cp/32]: the nearest of eight magnitudes."""
    p, s = _exact_blocks(v, E2M1_MAX)
    a, out = (p / s).abs(), torch.zeros_like(p)
    for i in range(1, 8):  # a midpoint goes to the code that is even
        mid = (_CODES[i - 1] + _CODES[i]) / 2
        out = torch.where((a > mid) | ((a == mid) if i % 2 == 0 else torch.zeros_like(a, dtype=torch.bool)),
                          torch.full_like(out, _CODES[i]), out)
    return (torch.sign(p) * out * s).flatten(-2)[..., : v.shape[-1]], s.squeeze(-1)


def _exact8(v):
    """float64 [.., C] rounded to e4m3 in blocks of 32."""
    p, s = _exact_blocks(v, E4M3_MAX)
    q = p / s
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step * s).flatten(-2)[..., : v.shape[-1]]


def _layout(s):
    """Scales [.., rows, Kp/32] as they are kept."""
    return s.unflatten(-1, (-1, 8)).transpose(-2, -3).contiguous()


def _stored4(b, cols):
    """float64 [rows, cols] of one stored 4-bit matrix."""
    q, s = b[0].view(torch.uint8), b[1]
    table = torch.tensor(_CODES + tuple(-c for c in _CODES), dtype=torch.float64, device=q.device)
    v = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
    v[:, 0::2], v[:, 1::2] = table[(q & 15).long()], table[(q >> 4).long()]
    s = s.double().transpose(0, 1).reshape(q.shape[0], -1)
    return (v * s.repeat_interleave(32, -1))[:, :cols]


def _stored8(b, cols, n=None):
    """float64 [rows, cols] of stored 8-bit rows, or of one matrix of n rows."""
    s = b[1].double().repeat_interleave(128, -1)
    s = s if n is None else s.repeat_interleave(128, 0)[:n]
    return (b[0].double() * s[:, : b[0].shape[1]])[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    pair = lambda b: (b.q, b.scale) if hasattr(b, "q") else b
    op = case["op"]
    if op == "weights":
        v, s = _exact4(st["w"].double())
        out = dict(values=v, scale=_layout(s))
        v, s = _exact4(st["w"].double().transpose(1, 2).contiguous())
        return dict(values_t=v, scale_t=_layout(s), **out)
    if op == "rows":
        v, s = _exact4(st["x"].double())
        return dict(values=v, scale=_layout(s))
    if op == "few":
        T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
        x, out = _exact8(st["hidden"].double()), torch.zeros(T, H, dtype=torch.float64, device=st["hidden"].device)
        read = lambda b, e, N, K: _stored4((b[0][e], b[1][e]), K) if case["bits"] == 4 else \
            _stored8((b[0][e], b[1][e]), K, N)
        w1, w2 = pair(st["w1"]), pair(st["w2"])
        if hasattr(st["w1"], "q") and case["bits"] == 4:
            w1, w2 = (w1[0].view(torch.uint8), w1[1]), (w2[0].view(torch.uint8), w2[1])
        for e in torch.unique(st["topk_idx"]).tolist():
            t, j = (st["topk_idx"] == e).nonzero(as_tuple=True)
            y = x[t] @ read(w1, e, 2 * F, H).t()
            a = _exact8(torch.nn.functional.silu(y[:, :F]) * y[:, F:])
            out.index_put_((t,), st["weight"][t, j].double()[:, None] * (a @ read(w2, e, H, F).t()), accumulate=True)
        return dict(out=out)
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    if T * k * N * K > 3e12:
        return None
    if op == "down":
        y = st["y"].double()
        x = _exact4(torch.nn.functional.silu(y[:, :K]) * y[:, K:])[0]
    else:
        b = pair(st["x"])
        x = _stored8(b, K) if case["bits"] == 8 else _stored4(b, K)
    offset, expert = st["inst_offset"].tolist(), st["inst_expert"].tolist()

    def products(rows, w, n, cols):
        q, s = pair(w)
        q, out = q.view(torch.uint8), torch.zeros(T * k, n, dtype=torch.float64, device=rows.device)
        for i in range(st["instances"]):
            a, z = offset[i], offset[i + 1]
            if a < z:
                out[a:z] = rows[a:z] @ _stored4((q[expert[i]], s[expert[i]]), cols).t()
        return out

    out = dict(y=products(x, st["w"], N, K))
    if case.get("train"):
        out["dx"] = products(_stored8(pair(st["dy"]), N), st["wt"], K, N)
    return out
