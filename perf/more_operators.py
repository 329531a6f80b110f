"""The products over 4-bit weights, and the way from a step's logits to its tokens, as they are measured.

* ``mul``    -- y = x . W over 4-bit weights with a scale (and a zero point) a group of rows;
* ``pair``   -- silu(x . Wg) * (x . Wu) over two of them;
* ``rules``  -- penalties of a request's tokens, biases and grammar masks on its logits;
* ``sample`` -- a token a row from its logits: temperature, top-k, top-p, min-p, one random number.

Where ``own`` is false ``run`` computes them with elementary torch operations in 32 bits (the
probabilities that a token is drawn by in 64), where it is true through the package's entry points,
on the same buffers.

A 4-bit weight of K rows and N columns is held as bytes [K/2, N], row 2j in the low four bits and row
2j + 1 in the high ones, 2-byte scales [ceil(K/group), N] and, where it has them, zero points of a
byte each of the same shape: w = scale * (u - zero), zero 8 where there are none.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LARGEST = 2048 * 4096 * 14336        # products of the largest listed case
NEG = -math.inf


# ---- cases ------------------------------------------------------------------------

def _mul(name, m, k, n, *, op="mul", group=128, zeros=False, scale="f16", act="bf16", extra=False):
    """``extra``: a bias and a residual are added (calls of up to 32 rows)."""
    return {"name": name, "op": op, "m": m, "k": k, "n": n, "group": group, "zeros": zeros,
            "scale": scale, "act": act, "extra": extra}


def _logits(name, op, m, vocab, shape, *, history=0, biases=0, mask=False):
    return {"name": name, "op": op, "m": m, "vocab": vocab, "shape": shape, "history": history,
            "biases": biases, "mask": mask}


def listed():
    return [
        # one request's smallest projection: the latency of the call
        _mul("mul_1_k1024_n1024", 1, 1024, 1024, group=32),
        # a feed-forward projection of a decode batch, zero points
        _mul("mul_16_k4096_n14336", 16, 4096, 14336, zeros=True),
        # the last projection of a batch whose activation comes quantized, the width odd
        _mul("mul_32_k5120_n32001_q8", 32, 5120, 32001, group=32, scale="bf16", act="q8_0", extra=True),
        # prompts: a chunk of rows
        _mul("mul_2048_k4096_n14336", 2048, 4096, 14336),
        # the gated half of a feed-forward block for one request
        _mul("pair_1_k4096_n14336", 1, 4096, 14336, op="pair", group=64),
        # the same for a batch with quantized activations and an odd width
        _mul("pair_24_k4096_n11000_q8", 24, 4096, 11000, op="pair", group=32, zeros=True, act="q8_0"),
        # and for a chunk of a prompt
        _mul("pair_512_k4096_n14336", 512, 4096, 14336, op="pair"),
        # one request behind a grammar, its own short history
        _logits("rules_1_v32000", "rules", 1, 32000, 1, history=700, biases=20, mask=True),
        # a batch over a large odd vocabulary, histories up to 4096 tokens
        _logits("rules_192_v130001", "rules", 192, 130001, 2, history=4096, biases=300, mask=True),
        # one request: the latency of the call
        _logits("sample_1_v32000", "sample", 1, 32000, 3),
        # a batch, every kind of request in it
        _logits("sample_40_v50001", "sample", 40, 50001, 4),
        # a large batch over a large vocabulary
        _logits("sample_256_v131072", "sample", 256, 131072, 5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mul", "mul", "pair", "rules", "sample", "sample"])
    if op in ("mul", "pair"):
        weights = 2 if op == "pair" else 1
        k = 32 * _log(rng, 8, 512)
        n = _log(rng, 40, min(32768, 5120 * 32000 // (k * weights)))
        m = rng.choice([1, _log(rng, 2, 32), _log(rng, 33, 2048)])
        m = max(1, min(m, LARGEST // (k * n * weights)))
        c = _mul("", m, k, n, op=op, group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5,
                 scale=rng.choice(["f16", "bf16"]), act=rng.choice(["bf16", "bf16", "q8_0"]),
                 extra=op == "mul" and m <= 32 and rng.random() < 0.5)
    else:
        m = rng.choice([1, _log(rng, 2, 256)])
        vocab = min(_log(rng, 1000, 160000), 192 * 130001 // m)
        rules = op == "rules"
        c = _logits("", op, m, vocab, rng.randrange(1 << 30),
                    history=rng.choice([0, _log(rng, 16, 4096)]) if rules else 0,
                    biases=rng.choice([0, _log(rng, 1, 300)]) if rules else 0,
                    mask=rules and rng.random() < 0.6)
    del c["name"]
    return c


def _pad64(n):
    return -(-n // 64) * 64


def _requests(case):
    """The histories, biases and masks of each row of a ``rules`` case: part of the case."""
    r = np.random.default_rng(case["shape"])
    m, most = case["m"], case["history"]
    total = r.integers(most // 2, most + 1, m)
    total[1::7] = 0                                    # requests without any tokens yet
    prompt = (total * r.random(m)).astype(np.int64)
    bias = r.integers(case["biases"] // 2, case["biases"] + 1, m)
    bias[::3] = case["biases"]
    bias[2::5] = 0
    masked = r.random(m) < 0.7 if case["mask"] else np.zeros(m, bool)
    masked[:1] = case["mask"]
    return total, prompt, np.minimum(bias, case["vocab"]), masked


def work(case):
    if case["op"] in ("mul", "pair"):
        m, k, n = case["m"], case["k"], case["n"]
        w = 2 if case["op"] == "pair" else 1
        groups = -(-k // case["group"])
        x = m * k * (2 if case["act"] == "bf16" else 1.125)
        extra = 4 * (n + m * n) if case["extra"] else 0
        return {"bytes": w * (k * n / 2 + groups * n * (3 if case["zeros"] else 2)) + x + 4 * m * n + extra,
                "flops": 2.0 * w * m * k * n}
    m, v = case["m"], case["vocab"]
    if case["op"] == "rules":
        total, _, bias, masked = _requests(case)
        return {"bytes": 8 * m * v + 4 * int(total.sum()) + 8 * int(bias.sum()) + int(masked.sum()) * v / 8,
                "flops": 2 * m * v}
    return {"bytes": 4 * m * v, "flops": 4 * m * v}


# ---- inputs -----------------------------------------------------------------------

def _round_up(v, to):
    return -(-v // to) * to


def _quantized(x):
    """The buffer of a quantized activation: codes [m, K], scales [m, K/32] at the next 256 bytes, the
    codes block by block behind them."""
    m, k = x.shape
    b = x.float().unflatten(-1, (-1, 32))
    d = b.abs().amax(-1) / 127.0
    quot = b / torch.where(d == 0, 1.0, d)[..., None]
    code = torch.copysign((quot.abs() + 0.5).floor(), quot).clamp(-127, 127).to(torch.int8)
    at = _round_up(m * k, 256)
    view = _round_up(at + m * (k // 32) * 4, 256)
    buf = torch.zeros(view + m * k, dtype=torch.uint8, device=DEV)
    buf[:m * k] = code.flatten().view(torch.uint8)
    buf[at:at + m * (k // 32) * 4] = d.flatten().view(torch.uint8)
    buf[view:] = code.permute(1, 0, 2).contiguous().flatten().view(torch.uint8)
    return buf, code.flatten(1), d


def _weight(case, g):
    """(bytes, scales, zero points) of a weight whose values spread as a layer's do."""
    k, n, groups = case["k"], case["n"], -(-case["k"] // case["group"])
    u = torch.randint(0, 256, (k // 2, n), device=DEV, generator=g, dtype=torch.uint8)
    s = torch.exp(torch.randn((groups, n), device=DEV, generator=g) * 0.4) * (0.2 / math.sqrt(k))
    s = s.to(torch.float16 if case["scale"] == "f16" else torch.bfloat16)
    z = torch.randint(5, 11, (groups, n), device=DEV, generator=g, dtype=torch.uint8) if case["zeros"] else None
    return u, s, z


def _prepare_product(case, g):
    m, k, n = case["m"], case["k"], case["n"]
    s = {"case": case, "w": [_weight(case, g) for _ in range(2 if case["op"] == "pair" else 1)]}
    s["x"] = torch.randn((m, k), device=DEV, generator=g).to(torch.bfloat16)
    if case["act"] == "q8_0":
        s["x_q8"], s["codes"], s["dx"] = _quantized(s["x"])
    s["bias"] = s["residual"] = None
    if case["extra"]:
        s["bias"] = torch.randn(n, device=DEV, generator=g)
        s["residual"] = torch.zeros((m, _pad64(n)), device=DEV)
        s["residual"][:, :n] = torch.randn((m, n), device=DEV, generator=g)
    s["y"] = torch.zeros((m, _pad64(n)), device=DEV)
    return s


def _prepare_logits(case, seed, g):
    m, v = case["m"], case["vocab"]
    ld = _pad64(v)                                     # the last product's rows
    r = np.random.default_rng([seed, case["shape"]])
    logits = torch.randn((m, ld), device=DEV, generator=g) * 2.5
    top = torch.randint(0, v, (m, 24), device=DEV, generator=g)
    logits.scatter_add_(1, top, torch.rand((m, 24), device=DEV, generator=g) * 12)
    s = {"case": case, "logits": logits, "ld": ld}

    def f32(a):
        return torch.tensor(np.asarray(a, np.float32), device=DEV)

    def i32(a):
        return torch.tensor(np.asarray(a, np.int32), device=DEV)

    if case["op"] == "rules":
        total, prompt, bias, masked = _requests(case)
        width = max(1, int(total.max()))
        # words of a text: a few are most of it
        words = np.minimum((v ** r.random((m, width))).astype(np.int64) - 1, v - 1)
        words = (words * 7919 + 13) % v
        s |= {"tokens": i32(np.where(np.arange(width) < total[:, None], words, -1)), "width": width,
              "len": i32(total), "prompt_len": i32(prompt)}
        plain = r.random(m) < 0.2
        s["repetition"] = f32(np.where(plain, 1.0, 1.0 + 0.3 * r.random(m)))
        s["presence"] = f32(np.where(plain, 0.0, r.random(m)))
        s["frequency"] = f32(np.where(plain, 0.0, 0.5 * r.random(m)))
        start = np.concatenate([[0], np.cumsum(bias)])
        s["bias_start"] = i32(start)
        ids = torch.rand((m, v), device=DEV, generator=g).argsort(1)[:, :max(1, case["biases"])]
        at = torch.arange(ids.shape[1], device=DEV)[None, :] < torch.tensor(bias, device=DEV)[:, None]
        s["bias_token"] = torch.zeros(max(1, int(start[-1])), dtype=torch.int32, device=DEV)
        s["bias_token"][:int(start[-1])] = ids[at].to(torch.int32)
        s["bias_value"] = torch.randn(max(1, int(start[-1])), device=DEV, generator=g) * 4
        s["mask"] = s["mask_row"] = None
        if case["mask"]:
            row = np.where(masked, np.cumsum(masked) - 1, -1)
            words = -(-v // 32)
            bits = [torch.randint(-(1 << 31), 1 << 31, (int(masked.sum()), words), device=DEV,
                                  generator=g, dtype=torch.int64).to(torch.int32) for _ in range(2)]
            s["mask"] = bits[0] & bits[1]              # a quarter of the tokens may follow
            s["mask_row"] = i32(row)
        s["out"] = torch.zeros((m, ld), device=DEV)
        return s
    # a batch holds requests of every kind
    kind = r.integers(0, 6, m)
    s["temperature"] = f32(np.where(kind == 0, 0.0, 0.5 + r.random(m)))
    s["top_k"] = i32(np.where((kind == 1) | (kind == 3), r.integers(1, 200, m), 0))
    s["top_p"] = f32(np.where((kind == 2) | (kind == 3), 0.5 + 0.5 * r.random(m), 1.0))
    s["min_p"] = f32(np.where(kind == 4, 0.2 * r.random(m), 0.0))
    s["u"] = torch.rand(m, device=DEV, generator=g, dtype=torch.float64)
    s["token"] = torch.zeros(m, dtype=torch.int32, device=DEV)
    s["logprob"] = torch.zeros(m, device=DEV)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = _prepare_product(case, g) if case["op"] in ("mul", "pair") else _prepare_logits(case, seed, g)
    if own:
        _prepare_own(s)
    return s


# ---- the plain forms ----------------------------------------------------------------

def _plain_product(s, w):
    c = s["case"]
    u, scale, z = w
    q = torch.stack([u & 15, u >> 4], 1).flatten(0, 1).float()          # [K, N]
    row = torch.arange(c["k"], device=DEV) // c["group"]
    q = (q - (8.0 if z is None else z[row].float())) * scale[row].float()
    if c["act"] == "bf16":
        x = s["x"].float()
    else:
        x = (s["codes"].float().unflatten(-1, (-1, 32)) * s["dx"][..., None]).flatten(1)
    return x @ q


def _plain_mul(s):
    n = s["case"]["n"]
    y = _plain_product(s, s["w"][0])
    if s["bias"] is not None:
        y = y + s["bias"] + s["residual"][:, :n]
    s["y"][:, :n] = y
    return s["y"]


def _plain_pair(s):
    g, u = _plain_product(s, s["w"][0]), _plain_product(s, s["w"][1])
    s["y"][:, :s["case"]["n"]] = g / (1.0 + torch.exp(-g)) * u
    return s["y"]


def _plain_rules(s):
    c = s["case"]
    m, v = c["m"], c["vocab"]
    x = s["logits"][:, :v]
    at = torch.arange(s["width"], device=DEV)[None, :]
    tok, here = s["tokens"].long().clamp(min=0), at < s["len"][:, None]
    made = here & (at >= s["prompt_len"][:, None])
    seen = torch.zeros((m, v), device=DEV).scatter_add_(1, tok, here.float())
    count = torch.zeros((m, v), device=DEV).scatter_add_(1, tok, made.float())
    rep = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count - torch.where(count > 0, s["presence"][:, None], 0.0)
    n = int(s["bias_token"].numel())
    j = torch.arange(n, device=DEV, dtype=torch.int32)
    row = torch.searchsorted(s["bias_start"][1:].contiguous(), j, right=True).clamp(max=m - 1)
    value = torch.where(j < s["bias_start"][-1], s["bias_value"], 0.0)
    x = x.flatten().scatter_add(0, row * v + s["bias_token"].long(), value).unflatten(0, (m, v))
    if s["mask"] is not None:
        t = torch.arange(v, device=DEV)
        allowed = (s["mask"][:, t // 32] >> (t % 32).to(torch.int32)) & 1
        row = s["mask_row"].long()
        allowed = allowed[row.clamp(min=0)].bool() | (row < 0)[:, None]
        x = torch.where(allowed, x, NEG)
    s["out"][:, :v] = x
    return s["out"]


def _plain_sample(s):
    v = s["case"]["vocab"]
    x = s["logits"][:, :v]
    temp = s["temperature"].double()[:, None]
    greedy = temp <= 0
    order, index = torch.sort(x, dim=1, descending=True, stable=True)
    top = order[:, :1]
    w = torch.exp((order.double() - top.double()) / torch.where(greedy, 1.0, temp))
    before = w.cumsum(1) - w
    rank = torch.arange(v, device=DEV)[None, :]
    k = s["top_k"].long()[:, None]
    p = s["top_p"].double()[:, None]
    keep = (rank < torch.where(k > 0, k, v)) & (w >= s["min_p"].double()[:, None])
    keep &= (p >= 1) | (before < p * w.sum(1, keepdim=True)) | (rank == 0)
    keep &= ~greedy | (rank == 0)
    w = torch.zeros_like(w).scatter(1, index, torch.where(keep, w, 0.0)).cumsum(1)   # by token
    token = (w <= s["u"][:, None] * w[:, -1:]).sum(1).clamp(max=v - 1)
    s["token"].copy_(token)
    total = torch.exp(x - top).sum(1)
    s["logprob"].copy_(x.gather(1, token[:, None])[:, 0] - top[:, 0] - torch.log(total))
    return {"token": s["token"], "logprob": s["logprob"]}


# ---- the framework's calls ------------------------------------------------------------

def _prepare_own(s):
    """What a program keeps: the weights in their packed layout, workspaces, the calls' descriptions."""
    import block_quantized_weight_02_amd as q8
    c = s["case"]
    if c["op"] in ("mul", "pair"):
        k, n, zeros = c["k"], c["n"], c["zeros"]
        fmt = q8.Q8_W4_SCALE_F16 if c["scale"] == "f16" else q8.Q8_W4_SCALE_BF16
        s["packed"] = []
        for u, scale, z in s["w"]:
            values = torch.empty(q8.q8_w4_values_bytes(k, n), dtype=torch.uint8, device=DEV)
            scales = torch.empty(q8.q8_w4_scales_bytes(k, n, c["group"], zeros), dtype=torch.uint8, device=DEV)
            w = q8.make_w4_weight(values, scales, k, n, c["group"], fmt, zeros)
            q8.q8_w4_repack(u, scale, z, w)
            s["packed"].append((w, values, scales))
        s["act"] = q8.Q8_ACT_BF16 if c["act"] == "bf16" else q8.Q8_ACT_Q8_0
        s["in"] = s["x"] if c["act"] == "bf16" else s["x_q8"]
        s["epilogue"] = q8.make_epilogue(s["bias"], s["residual"]) if c["extra"] else None
        s["need"] = 0
        if c["m"] <= q8.Q8_MAX_ROWS:
            size = q8.q8_w4_gemv_workspace_bytes if c["op"] == "mul" else q8.q8_w4_glu_workspace_bytes
            s["need"] = size(c["m"], s["packed"][0][0], s["act"])
        s["ws"] = torch.zeros(max(16, s["need"]), dtype=torch.uint8, device=DEV)
    elif c["op"] == "rules":
        s["rules"] = q8.make_logit_rules(
            tokens=s["tokens"], ld_tokens=s["width"], lens=s["len"], prompt_lens=s["prompt_len"],
            repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
            bias_start=s["bias_start"], bias_token=s["bias_token"], bias_value=s["bias_value"],
            mask=s["mask"], ld_mask=0 if s["mask"] is None else s["mask"].shape[1],
            mask_row=s["mask_row"], mask_rows=0 if s["mask"] is None else s["mask"].shape[0])
    else:
        s["sampling"] = q8.make_sampling(s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                         top_p=s["top_p"], min_p=s["min_p"])
        s["need"] = q8.q8_sample_workspace_bytes(c["m"], c["vocab"])
        s["ws"] = torch.zeros(max(16, s["need"]), dtype=torch.uint8, device=DEV)


def _own(s):
    import block_quantized_weight_02_amd as q8
    c = s["case"]
    if c["op"] == "mul":
        w = s["packed"][0][0]
        if c["m"] <= q8.Q8_MAX_ROWS:
            q8.q8_w4_gemv(s["in"], w, s["y"], c["m"], s["act"], s["epilogue"], None, s["ws"], s["need"])
        else:
            q8.q8_w4_gemm(s["in"], w, s["y"], c["m"], s["act"])
        return s["y"]
    if c["op"] == "pair":
        g, u = s["packed"][0][0], s["packed"][1][0]
        if c["m"] <= q8.Q8_MAX_ROWS:
            q8.q8_w4_gemv_glu(s["in"], g, u, s["y"], c["m"], s["act"], None, None, s["ws"], s["need"])
        else:
            q8.q8_w4_gemm_glu(s["in"], g, u, s["y"], c["m"], s["act"])
        return s["y"]
    if c["op"] == "rules":
        q8.q8_logits_rules(s["logits"], s["ld"], c["m"], c["vocab"], s["rules"], s["out"], s["ld"])
        return s["out"]
    q8.q8_sample(s["logits"], s["ld"], c["m"], c["vocab"], s["sampling"], s["token"], s["logprob"],
                 None, s["ws"], s["need"])
    return {"token": s["token"], "logprob": s["logprob"]}


def run(state):
    if own:
        return _own(state)
    return {"mul": _plain_mul, "pair": _plain_pair, "rules": _plain_rules,
            "sample": _plain_sample}[state["case"]["op"]](state)


# ---- the definition, in 64 bits ---------------------------------------------------------

def _exact_product(case, s, w):
    """sum over the groups of scale * (x . u - zero * sum x)."""
    u, scale, z = w
    k, n, group = case["k"], case["n"], case["group"]
    if case["act"] == "bf16":
        x = s["x"].double()
    else:
        x = s["codes"].double() * s["dx"].double().repeat_interleave(32, 1)
    y = torch.zeros((case["m"], n), dtype=torch.float64, device=DEV)
    for i in range(scale.shape[0]):
        a, b = i * group, min(k, (i + 1) * group)
        part = x[:, a:b]
        dot = part[:, 0::2].contiguous() @ (u[a // 2:b // 2] % 16).double()
        dot += part[:, 1::2].contiguous() @ (u[a // 2:b // 2] // 16).double()
        zero = 8.0 if z is None else z[i].double()
        y += scale[i].double() * (dot - part.sum(1, keepdim=True) * zero)
    return y


def _exact_rules(case, s):
    m, v = case["m"], case["vocab"]
    out = torch.zeros((m, s["ld"]), dtype=torch.float64, device=DEV)
    tokens, total, prompt = (s[x].cpu().numpy() for x in ("tokens", "len", "prompt_len"))
    start, word, value = (s[x].cpu().numpy() for x in ("bias_start", "bias_token", "bias_value"))
    rep, pres, freq = (s[x].double().cpu().numpy() for x in ("repetition", "presence", "frequency"))
    logits = s["logits"].double().cpu().numpy()[:, :v]
    mask = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint8)
    which = None if mask is None else s["mask_row"].cpu().numpy()
    for i in range(m):
        x = logits[i].copy()
        seen = np.unique(tokens[i, :total[i]])
        x[seen] = np.where(x[seen] > 0, x[seen] / rep[i], x[seen] * rep[i])
        made, count = np.unique(tokens[i, prompt[i]:total[i]], return_counts=True)
        x[made] -= freq[i] * count + pres[i]
        x[word[start[i]:start[i + 1]]] += value[start[i]:start[i + 1]]
        if mask is not None and which[i] >= 0:
            x[np.unpackbits(mask[which[i]], bitorder="little")[:v] == 0] = NEG
        out[i, :v] = torch.from_numpy(x).to(DEV)
    return out


def _exact_sample(case, s):
    v = case["vocab"]
    host = {x: s[x].cpu().numpy() for x in ("temperature", "top_k", "top_p", "min_p", "u")}
    tokens, probs = [], []
    for i, x in enumerate(s["logits"].cpu().numpy()[:, :v].astype(np.float64)):
        t = float(host["temperature"][i])
        top = x.max()
        if t <= 0:
            token = int(x.argmax())
        else:
            w = np.exp((x - top) / t)
            by = np.argsort(-x, kind="stable")
            mass = np.cumsum(w[by])
            n = int(host["top_k"][i]) if 0 < host["top_k"][i] < v else v
            p = float(host["top_p"][i])
            if p < 1:
                n = min(n, max(1, 1 + int(np.searchsorted(mass, p * mass[-1], side="left"))))
            kept = np.zeros(v, bool)
            kept[by[:n]] = True
            cdf = np.cumsum(np.where(kept & (w >= float(host["min_p"][i])), w, 0.0))
            token = int(np.searchsorted(cdf, host["u"][i] * cdf[-1], side="right"))
        tokens.append(token)
        probs.append(x[token] - top - math.log(np.exp(x - top).sum()))
    return {"token": torch.tensor(tokens, dtype=torch.int32, device=DEV),
            "logprob": torch.tensor(probs, dtype=torch.float64, device=DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rules":
        return _exact_rules(case, s)
    if case["op"] == "sample":
        return _exact_sample(case, s)
    y = torch.zeros((case["m"], _pad64(case["n"])), dtype=torch.float64, device=DEV)
    if case["op"] == "mul":
        y[:, :case["n"]] = _exact_product(case, s, s["w"][0])
        if case["extra"]:
            y[:, :case["n"]] += s["bias"].double() + s["residual"][:, :case["n"]].double()
        return y
    a = _exact_product(case, s, s["w"][0])
    y[:, :case["n"]] = a / (1 + torch.exp(-a)) * _exact_product(case, s, s["w"][1])
    return y
