"""Cases of the serving operators: rotary positions, the quantized KV cache, attention over packed prompts and
attention of single tokens over the cache.

Each case is run either in a plain form (elementary torch operations in 32 bits, 64 where angles need them) or, with
`own` set, through the library's entry points.  Inputs are seeded; the library is imported only where `own` is true.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


# ---------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One decoding step of a small batch far into a stretched context: 8 tokens, grouped heads.
        {"name": "rope_step", "op": "rope", "T": 8, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "layout": "half",
         "scaling": "yarn", "factor": 8.0, "far": 200000, "axes": 1, "dtype": "bf16"},
        # A joint video sequence with (t, h, w, l) positions, every head rotated in adjacent pairs.
        {"name": "rope_joint", "op": "rope", "T": 20480, "Hq": 24, "Hk": 24, "D": 128, "rot": 128,
         "layout": "pairs", "scaling": "none", "factor": 1.0, "far": 0, "axes": 4, "dtype": "bf16"},
        # A long prompt whose heads are rotated in part, FP16, an odd number of tokens.
        {"name": "rope_part", "op": "rope", "T": 16381, "Hq": 32, "Hk": 4, "D": 128, "rot": 64, "layout": "half",
         "scaling": "ntk", "factor": 4.0, "far": 30000, "axes": 1, "dtype": "fp16"},
        # The cache write of one decoding step of 64 sequences.
        {"name": "write_step", "op": "write", "T": 64, "Hk": 8, "D": 128, "page": 16, "codes": "int8",
         "dtype": "bf16"},
        # The cache write of a long prompt.
        {"name": "write_prompt", "op": "write", "T": 32768, "Hk": 8, "D": 128, "page": 64, "codes": "e4m3",
         "dtype": "bf16"},
        # A short cached prefix read back, narrow heads.
        {"name": "read_prefix", "op": "read", "T": 517, "Hk": 4, "D": 64, "page": 16, "codes": "e4m3",
         "dtype": "fp16"},
        # A long cached context read back before the next part of the prompt.
        {"name": "read_context", "op": "read", "T": 32768, "Hk": 8, "D": 128, "page": 64, "codes": "int8",
         "dtype": "bf16"},
        # A batch of short captions of uneven lengths, narrow heads.
        {"name": "prompt_captions", "op": "prompt", "lens": "77,130,1,333,64,19,256,100", "past": "0", "Hq": 16,
         "Hk": 4, "D": 64, "dtype": "bf16"},
        # Parts of prompts continued after what the cache already held (queries at the end of longer keys).
        {"name": "prompt_continued", "op": "prompt", "lens": "1504,512,32,1000", "past": "2592,0,3000,77", "Hq": 24,
         "Hk": 8, "D": 128, "dtype": "fp16"},
        # One long prompt.
        {"name": "prompt_long", "op": "prompt", "lens": "8192", "past": "0", "Hq": 32, "Hk": 8, "D": 128,
         "dtype": "bf16"},
        # One sequence decoding alone in a middling context: latency.
        {"name": "token_single", "op": "token", "B": 1, "shortest": 3999, "longest": 3999, "Hq": 32, "Hk": 8,
         "D": 128, "page": 16, "codes": "int8", "dtype": "bf16"},
        # A decoding batch of uneven contexts.
        {"name": "token_batch", "op": "token", "B": 64, "shortest": 300, "longest": 8192, "Hq": 32, "Hk": 8,
         "D": 128, "page": 64, "codes": "e4m3", "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "write", "read", "prompt", "token", "prompt", "token"])
    Hk = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rope":
        axes = rng.choice([1, 1, 4])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return {"op": op, "T": log(1, 16384), "Hq": Hk * rng.choice([1, 3, 4]), "Hk": Hk, "D": D,
                "rot": rng.choice([16, 40, 64, D]), "layout": rng.choice(["half", "pairs"]), "scaling": scaling,
                "factor": 1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                "far": 0 if axes == 4 else log(1, 1000000), "axes": axes,
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op in ("write", "read"):
        return {"op": op, "T": log(1, 32768), "Hk": Hk, "D": D, "page": rng.choice([16, 32, 64, 128]),
                "codes": rng.choice(["int8", "e4m3"]), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op == "prompt":
        n = rng.choice([1, 1, 2, 3, 5, 8])
        lens = [log(1, 6000 // n) for _ in range(n)]
        past = [rng.choice([0, 0, log(1, 2000 // n + 1)]) for _ in range(n)]
        return {"op": op, "lens": ",".join(map(str, lens)), "past": ",".join(map(str, past)),
                "Hq": min(G, 32 // Hk) * Hk, "Hk": Hk, "D": D, "dtype": dtype}
    B = log(1, 64)
    longest = log(1, 8192)
    return {"op": op, "B": B, "shortest": max(1, longest // rng.choice([1, 3, 20])), "longest": longest, "Hq": G * Hk,
            "Hk": Hk, "D": D, "page": rng.choice([16, 32, 64, 128]), "codes": rng.choice(["int8", "e4m3"]),
            "dtype": dtype}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _prompt_lens(case):
    """Query and key counts of each packed sequence."""
    lens = _ints(case["lens"])
    past = _ints(case["past"])
    past = past * len(lens) if len(past) == 1 else past
    return lens, [n + p for n, p in zip(lens, past)]


def _token_lens(case, seed):
    g = torch.Generator().manual_seed(seed + 17)
    lens = torch.randint(case["shortest"], case["longest"] + 1, (case["B"],), generator=g)
    lens[0] = case["longest"]
    return lens


def work(case):
    op, e = case["op"], {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if op == "rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": 2 * n * e + 8 * case["T"] * case["axes"], "flops": 0}
    if op in ("write", "read"):
        n = 2 * case["T"] * case["Hk"]
        return {"bytes": n * case["D"] * e + n * (case["D"] + 4) + 8 * case["T"], "flops": 0}
    if op == "prompt":
        lq, lk = _prompt_lens(case)
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))
        rows = sum(lq) * case["Hq"] * 2 + sum(lk) * case["Hk"] * 2
        return {"bytes": rows * case["D"] * e + 4 * sum(lq) * case["Hq"], "flops": 4 * case["D"] * case["Hq"] * pairs}
    mean = (case["longest"] + (case["B"] - 1) * (case["shortest"] + case["longest"]) / 2) / case["B"]
    n = case["B"] * mean * case["Hk"] * 2 * (case["D"] + 4)
    return {"bytes": n + case["B"] * case["Hq"] * (2 * case["D"] * e + 4),
            "flops": 4 * case["D"] * case["Hq"] * case["B"] * mean}


# --------------------------------------------------------------------------------------------------------- inputs
def _frequencies(case):
    """Rotation per position of each channel pair, and the factor on cos and sin."""
    r, s, base = case["rot"], case["factor"], 10000.0
    if case["scaling"] == "ntk" and r > 2:
        base = base * s ** (r / (r - 2))
    f = base ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
    m = 1.0
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "yarn":
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = keep * f + (1 - keep) * f / s
        m = 0.1 * math.log(s) + 1.0
    return f, m


def _axis_of_pair(case):
    """Position axis of each pair: equal runs of pairs, the remainder on the last axis."""
    n, a = case["rot"] // 2, case["axes"]
    run_ = max(1, n // a)
    return [min(i // run_, a - 1) for i in range(n)]


def _random_pool(case, pages, g, dev):
    """A cache that holds earlier tokens: codes and one scale per token and head, as quantized N(0, 1) rows."""
    dt, top = _CODES[case["codes"]]
    x = torch.randn(pages, case["Hk"], case["page"], case["D"], generator=g, device=dev)
    amax = x.abs().amax(-1, keepdim=True)
    y = x * (top / amax)
    codes = y.round().to(dt) if dt == torch.int8 else y.to(dt)
    scale = amax[..., 0] / top * (0.5 + torch.rand(amax.shape[:-1], generator=g, device=dev))
    return codes, scale.contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op, t = case["op"], _TYPES[case["dtype"]]
    s = {"case": case}
    if op == "rope":
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        qkv = torch.randn(T, (Hq + 2 * Hk) * D, generator=g, device=dev).to(t)       # one fused projection
        s["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D : (Hq + Hk) * D].view(T, Hk, D)
        s["q_out"] = torch.empty(T, Hq, D, dtype=t, device=dev)
        s["k_out"] = torch.empty(T, Hk, D, dtype=t, device=dev)
        if case["axes"] == 1:
            first = int(torch.randint(0, case["far"] + 1, (1,), generator=host))
            s["pos"] = torch.arange(first, first + T, device=dev)
        else:
            n = torch.arange(T, device=dev)                                          # a raster of 32 x 56 frames
            s["pos"] = torch.stack([n // 1792, n % 1792 // 56, n % 56, n % 7 + seed % 100])[: case["axes"]].contiguous()
        f, s["m"] = _frequencies(case)
        s["f"] = f.to(dev)
        s["axis"] = torch.tensor(_axis_of_pair(case), device=dev)
        if own:
            import action_diffusion_transformers_b200 as adt
            s["plan"] = adt.RopePlan(case["rot"], base=10000.0, interleaved=case["layout"] == "pairs",
                                     scaling=None if case["scaling"] == "none" else case["scaling"],
                                     factor=case["factor"], orig_len=8192,
                                     axis=None if case["axes"] == 1 else _axis_of_pair(case))
    elif op in ("write", "read"):
        T, Hk, D, ps = case["T"], case["Hk"], case["D"], case["page"]
        pages = -(-T // ps) + 2
        table = torch.randperm(pages, generator=host)[: -(-T // ps)].to(dev)
        n = torch.arange(T, device=dev)
        s["slots"] = table[n // ps] * ps + n % ps                                    # a sequence in shuffled pages
        s["k_codes"], s["k_scale"] = _random_pool(case, pages, g, dev)
        s["v_codes"], s["v_scale"] = _random_pool(case, pages, g, dev)
        if op == "write":
            kv = torch.randn(T, 2 * Hk * D, generator=g, device=dev)
            kv += 2 * torch.randn(2 * Hk * D, generator=g, device=dev)               # channel offsets, as K has
            kv = kv.to(t)
            s["k"] = kv[:, : Hk * D].view(T, Hk, D)
            s["v"] = kv[:, Hk * D :].view(T, Hk, D)
        else:
            s["k_out"] = torch.empty(T, Hk, D, dtype=t, device=dev)
            s["v_out"] = torch.empty(T, Hk, D, dtype=t, device=dev)
    elif op == "prompt":
        Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
        lq, lk = _prompt_lens(case)
        s["cu_q"] = [0]
        s["cu_k"] = [0]
        for a, b in zip(lq, lk):
            s["cu_q"].append(s["cu_q"][-1] + a)
            s["cu_k"].append(s["cu_k"][-1] + b)
        s["q"] = (1.5 * torch.randn(sum(lq), Hq, D, generator=g, device=dev)).to(t)
        kv = torch.randn(sum(lk), 2 * Hk * D, generator=g, device=dev).to(t)
        s["k"] = kv[:, : Hk * D].view(sum(lk), Hk, D)
        s["v"] = kv[:, Hk * D :].view(sum(lk), Hk, D)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(Hq, sum(lq), dtype=torch.float32, device=dev)
        # Sequence and place of each query and key, for the mask.
        at = lambda ls: (torch.cat([torch.full((n,), i) for i, n in enumerate(ls)]).to(dev),  # noqa: E731
                         torch.cat([torch.arange(n) for n in ls]).to(dev))
        s["q_seq"], s["q_at"] = at(lq)
        s["k_seq"], s["k_at"] = at(lk)
        s["q_at"] = s["q_at"] + torch.tensor([b - a for a, b in zip(lq, lk)], device=dev)[s["q_seq"]]
    else:
        B, Hq, Hk, D, ps = case["B"], case["Hq"], case["Hk"], case["D"], case["page"]
        lens = _token_lens(case, seed)
        per = -(-case["longest"] // ps)
        used = [-(-int(n) // ps) for n in lens]
        order = torch.randperm(sum(used) + 1, generator=host).to(torch.int32)
        table = torch.zeros(B, per, dtype=torch.int32)
        a = 0
        for b, n in enumerate(used):
            table[b, :n] = order[a : a + n]
            a += n
        s["table"] = table.to(dev)
        s["lens"] = lens.to(torch.int32).to(dev)
        s["k_codes"], s["k_scale"] = _random_pool(case, sum(used) + 1, g, dev)
        s["v_codes"], s["v_scale"] = _random_pool(case, sum(used) + 1, g, dev)
        s["q"] = (1.5 * torch.randn(B, Hq, D, generator=g, device=dev)).to(t)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, Hq, dtype=torch.float32, device=dev)
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=dev)        # kept for every step
    return s


# ------------------------------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return _OWN[case["op"]](s)
    return _PLAIN[case["op"]](s)


def _own_rope(s):
    import action_diffusion_transformers_b200 as adt
    adt.sage_rope(s["q"], s["k"], s["pos"], s["plan"], s["q_out"], s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_write(s):
    import action_diffusion_transformers_b200 as adt
    adt.sage_kv_write(s["k"], s["v"], s["slots"], s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"])
    return {n: s[n] for n in ("k_codes", "k_scale", "v_codes", "v_scale")}


def _own_read(s):
    import action_diffusion_transformers_b200 as adt
    adt.sage_kv_read(s["slots"], s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_prompt(s):
    import action_diffusion_transformers_b200 as adt
    adt.sage_attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_token(s):
    import action_diffusion_transformers_b200 as adt
    adt.sage_attn_token(s["q"], s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"], s["table"], s["lens"],
                        s["out"], s["workspace"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _rotate(x, c, sn, r, pairs):
    y = x[..., :r].float()
    if pairs:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    else:
        a, b = y[..., : r // 2], y[..., r // 2 :]
        y = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    return torch.cat([y.to(x.dtype), x[..., r:]], -1)


def _plain_rope(s):
    case = s["case"]
    pos = s["pos"][None].expand(len(s["axis"]), -1) if s["pos"].dim() == 1 else s["pos"][s["axis"]]
    angle = pos.t().double() * s["f"]
    c = (angle.cos() * s["m"]).float()[:, None]
    sn = (angle.sin() * s["m"]).float()[:, None]
    pairs = case["layout"] == "pairs"
    return {"q": _rotate(s["q"], c, sn, case["rot"], pairs), "k": _rotate(s["k"], c, sn, case["rot"], pairs)}


def _plain_write(s):
    dt, top = _CODES[s["case"]["codes"]]
    page, at = s["slots"] // s["case"]["page"], s["slots"] % s["case"]["page"]
    for x, codes, scale in ((s["k"], s["k_codes"], s["k_scale"]), (s["v"], s["v_codes"], s["v_scale"])):
        x = x.float()
        amax = x.abs().amax(-1)
        tops = torch.full_like(amax, top)                # a division by a tensor is rounded once
        y = x * (tops / amax)[..., None]
        y = y.round().to(dt) if dt == torch.int8 else y.to(dt)
        codes.view(torch.uint8)[page, :, at] = y.view(torch.uint8)
        scale[page, :, at] = amax / tops
    return {n: s[n] for n in ("k_codes", "k_scale", "v_codes", "v_scale")}


def _plain_read(s):
    t = _TYPES[s["case"]["dtype"]]
    page, at = s["slots"] // s["case"]["page"], s["slots"] % s["case"]["page"]
    out = {}
    for n in "kv":
        codes = s[n + "_codes"].view(torch.uint8)[page, :, at].view(s[n + "_codes"].dtype).float()
        out[n] = (codes * s[n + "_scale"][page, :, at][..., None]).to(t)
    return out


def _plain_prompt(s):
    case = s["case"]
    G, D = case["Hq"] // case["Hk"], case["D"]
    q = s["q"].float().unflatten(1, (case["Hk"], G)).permute(1, 2, 0, 3)             # Hk, G, Tq, D
    k, v = (s[n].float().transpose(0, 1)[:, None] for n in "kv")                     # Hk, 1, Tk, D
    sc = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5)
    seen = (s["q_seq"][:, None] == s["k_seq"]) & (s["k_at"] <= s["q_at"][:, None])
    sc.masked_fill_(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / l
    return {"out": o.permute(2, 0, 1, 3).flatten(1, 2).to(s["q"].dtype), "lse": (m + l.log())[..., 0].flatten(0, 1)}


def _plain_token(s):
    case = s["case"]
    G, D, ps = case["Hq"] // case["Hk"], case["D"], case["page"]
    table = s["table"].long()
    kv = []
    for n in "kv":
        codes = s[n + "_codes"].view(torch.uint8)[table].view(s[n + "_codes"].dtype).float()
        x = codes * s[n + "_scale"][table][..., None]                                # B, pages, Hk, ps, D
        kv.append(x.transpose(1, 2).flatten(2, 3))                                   # B, Hk, L, D
    q = s["q"].float().unflatten(1, (case["Hk"], G))
    sc = torch.matmul(q, kv[0].transpose(-1, -2)) * D ** -0.5
    at = torch.arange(table.shape[1] * ps, device=table.device)
    sc = sc.masked_fill(at >= s["lens"][:, None, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[1]) / l
    return {"out": o.flatten(1, 2).to(s["q"].dtype), "lse": (m + l.log())[..., 0].flatten(1, 2)}


_OWN = {"rope": _own_rope, "write": _own_write, "read": _own_read, "prompt": _own_prompt, "token": _own_token}
_PLAIN = {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "prompt": _plain_prompt,
          "token": _plain_token}


# ------------------------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "write":
        return _exact_write(case, s)
    if case["op"] == "read":
        return _exact_read(case, s)
    return _exact_prompt(case, s) if case["op"] == "prompt" else _exact_token(case, s)


def _exact_rope(case, s):
    """Each pair as a complex number, turned by exp(i * position * frequency)."""
    f, m = s["f"], s["m"]
    pos = s["pos"].double().reshape(-1, case["T"])
    angle = torch.stack([pos[a] * f[i] for i, a in enumerate(_axis_of_pair(case))], -1)
    turn = torch.polar(torch.full_like(angle, m), angle)[:, None]
    r, out = case["rot"], {}
    for n in "qk":
        x = s[n].double().clone()
        if case["layout"] == "pairs":
            z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * turn
            x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., : r // 2], x[..., r // 2 : r]) * turn
            x[..., :r] = torch.cat([z.real, z.imag], -1)
        out[n] = x
    return out


def _rn32(x):
    return x.float().double()


def _exact_write(case, s):
    """The rule with its 32-bit roundings, each formed in 64 bits: scale = RN(amax / top), code = nearest of
    RN(x * RN(top / amax)), ties to even."""
    dt, top = _CODES[case["codes"]]
    out = {}
    for n in "kv":
        x = s[n].double()
        amax = x.abs().max(-1).values
        y = _rn32(x * _rn32(top / amax)[..., None])
        if dt == torch.int8:
            y = y.round()
        else:                                             # E4M3: 3 bits behind the first, none below 2^-9
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            y = (y / step).round() * step
        codes, scale = s[n + "_codes"].double(), s[n + "_scale"].double()
        for i in range(case["Hk"]):
            flat = codes[:, i].reshape(-1, case["D"])
            flat[s["slots"]] = y[:, i]
            codes[:, i] = flat.view(codes[:, i].shape)
            flat = scale[:, i].reshape(-1)
            flat[s["slots"]] = _rn32(amax[:, i] / top)
            scale[:, i] = flat.view(scale[:, i].shape)
        out[n + "_codes"] = codes.to(torch.int64) if dt == torch.int8 else codes
        out[n + "_scale"] = scale
    return out


def _exact_read(case, s):
    out = {}
    for n in "kv":
        x = s[n + "_codes"].double() * s[n + "_scale"].double()[..., None]
        out[n] = x.transpose(1, 2).reshape(-1, case["Hk"], case["D"])[s["slots"]]
    return out


def _attend(q, k, v, first):
    """One head: softmax attention where query i sees keys 0 .. first + i, 1024 queries at a time."""
    o, lse = [], []
    at = torch.arange(k.shape[0], device=q.device)
    for a in range(0, q.shape[0], 1024):
        x = q[a : a + 1024] @ k.t() / math.sqrt(q.shape[1])
        x = torch.where(at <= (first + a + torch.arange(x.shape[0], device=q.device))[:, None], x, -math.inf)
        lse.append(torch.logsumexp(x, -1))
        o.append(torch.softmax(x, -1) @ v)
    return torch.cat(o), torch.cat(lse)


def _exact_prompt(case, s):
    G = case["Hq"] // case["Hk"]
    q, k, v = (s[n].double() for n in "qkv")
    out = torch.zeros_like(q)
    lse = torch.zeros(case["Hq"], q.shape[0], dtype=torch.float64, device=q.device)
    for i in range(len(s["cu_q"]) - 1):
        a, b, c, d = s["cu_q"][i], s["cu_q"][i + 1], s["cu_k"][i], s["cu_k"][i + 1]
        for h in range(case["Hq"]):
            out[a:b, h], lse[h, a:b] = _attend(q[a:b, h], k[c:d, h // G], v[c:d, h // G], (d - c) - (b - a))
    return {"out": out, "lse": lse}


def _exact_token(case, s):
    G, B = case["Hq"] // case["Hk"], case["B"]
    out = torch.zeros(B, case["Hq"], case["D"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, case["Hq"], dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for b in range(B):
        rows = s["table"][b].long()
        kv = []
        for n in "kv":
            x = s[n + "_codes"].view(torch.uint8)[rows].view(s[n + "_codes"].dtype).double()
            x = x * s[n + "_scale"][rows].double()[..., None]
            kv.append(x.transpose(0, 1).reshape(case["Hk"], -1, case["D"])[:, : lens[b]])
        x = torch.einsum("hgd,hld->hgl", s["q"][b].double().view(case["Hk"], G, -1), kv[0]) / math.sqrt(case["D"])
        lse[b] = torch.logsumexp(x, -1).flatten()
        out[b] = torch.einsum("hgl,hld->hgd", torch.softmax(x, -1), kv[1]).flatten(0, 1)
    return {"out": out, "lse": lse}
