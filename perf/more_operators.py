"""Work that the 4-bit KV cache does, and the reading back of packed caches, as cases to be timed and compared.

Three operators over a cache whose rows are packed: 4-bit codes (e2m1) of all KV heads, one e4m3
scale for each 16 of them, padding to 16 bytes, one exponent byte for each head (a power of two for a
block of 64 slab tokens or a single COLD token), padding to 16 bytes.  An element stands for
code * scale * 2^(exponent - 127).

  store   K/V of new tokens into the 4-bit cache and out again: a prefix slab or single tokens at
          their COLD slots
  read    rows of a packed cache (4 or 8 bits) back in the type of q: a slab, or COLD tokens by slot
  decode  decode-step attention over the 4-bit cache: shared prefix slabs, then each request's COLD
          tokens through its token table; o and lse.  With `append`, the step's new K/V are given too
          and end up in the cache

``run`` computes them from elementary torch operations in fp32, or with the library's calls where
``own`` is true.
"""

import math
import random

import torch

own = False

BLOCK = 64            # tokens of a slab block that share a head's exponent (4 bits) or scale (8 bits)
GROUP = 16            # elements that share an e4m3 scale (4 bits)
E2M1_MAX, E4M3_MAX, E4M3_MIN = 6.0, 448.0, 2.0 ** -9
EXP_MIN, EXP_MAX = -100, 116
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------------------------

def listed():
    head = {"n_q": 32, "n_kv": 8, "d": 128, "dtype": "bf16"}
    return [
        # a 16K shared prefix admitted to its slab, one layer
        {"name": "store_prefix_16k", "op": "store", "kind": "slab", "tokens": 16384, **head},
        # the new tokens of one decode step of 64 requests
        {"name": "store_step_64", "op": "store", "kind": "cold", "tokens": 64, **head},
        # an fp32 prefix of odd length with 64-dim heads
        {"name": "store_prefix_f32", "op": "store", "kind": "slab", "tokens": 1501, "n_q": 8, "n_kv": 2, "d": 64, "dtype": "f32"},
        # a 16K prefix taken out of the 4-bit cache, for a 16-bit one
        {"name": "read_prefix_16k", "op": "read", "cache": "kv4", "kind": "slab", "tokens": 16384, **head},
        # the tokens of a request that leaves the 8-bit cache, at scattered slots
        {"name": "read_request_kv8", "op": "read", "cache": "kv8", "kind": "cold", "tokens": 3001, **head},
        # one agent alone on a long prefix: latency
        {"name": "decode_one", "op": "decode", "append": False, "prefixes": "8192", "B": 1, "suffix": "uniform", "lo": 200, "hi": 300, **head},
        # 64 agents on one 16K prefix, chat-like suffixes
        {"name": "decode_one_prefix_64", "op": "decode", "append": False, "prefixes": "16384", "B": 64, "suffix": "lognormal", "lo": 32, "hi": 2048, **head},
        # the same with the step's new tokens written by the call, as a decode loop makes it
        {"name": "decode_step_64", "op": "decode", "append": True, "prefixes": "16384", "B": 64, "suffix": "lognormal", "lo": 32, "hi": 2048, **head},
        # 128 agents on one 16K prefix, five query heads a KV head
        {"name": "decode_one_prefix_128", "op": "decode", "append": False, "prefixes": "16384", "B": 128, "suffix": "uniform", "lo": 64, "hi": 1024, **head, "n_q": 40},
        # eight ragged prefixes, 160 agents
        {"name": "decode_eight_prefixes", "op": "decode", "append": False, "prefixes": "2048,3001,5000,7777,9216,11111,14000,16384", "B": 160, "suffix": "lognormal", "lo": 32, "hi": 2048, **head},
        # prefixes that found no slab: COLD rows alone
        {"name": "decode_cold", "op": "decode", "append": False, "prefixes": "", "B": 16, "suffix": "uniform", "lo": 6000, "hi": 9000, **head},
        # fp32, small heads, a ragged prefix
        {"name": "decode_f32", "op": "decode", "append": True, "prefixes": "1500", "B": 48, "suffix": "uniform", "lo": 1, "hi": 80, "n_q": 8, "n_kv": 2, "d": 64, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "read", "decode", "decode", "decode"])
    heads = rng.choice([(1, 1), (8, 2), (16, 8), (32, 8), (40, 8), (16, 4), (24, 8), (64, 8)])
    head = {"n_q": heads[0], "n_kv": heads[1], "d": 128, "dtype": "bf16"}
    if op != "decode":
        kind = rng.choice(["slab", "cold"])
        if rng.random() < 0.3:
            head = {"n_q": 8, "n_kv": 2, "d": rng.choice([32, 64, 96]), "dtype": "f32"}
        case = {"op": op, "kind": kind, "tokens": _log(rng, 1, 16384 if kind == "slab" else 8192), **head}
        return {**case, "cache": rng.choice(["kv4", "kv8"])} if op == "read" else case
    if rng.random() < 0.2:
        head = {"n_q": 8, "n_kv": 2, "d": rng.choice([32, 64, 128]), "dtype": "f32"}
        n = rng.choice([1, 2])
        top, many, tail = 3000, 64, 300
    else:
        n = rng.choice([0, 1, 1, 2, 3, 6])
        top, many, tail = 16384, 160, 2048
    prefixes = ",".join(str(_log(rng, 16, top // max(1, n // 2))) for _ in range(n))
    hi = _log(rng, 1, tail)
    append = rng.random() < 0.4
    lo = rng.choice([0 if n and not append else 1, 1, max(1, hi // 2)])
    return {"op": op, "append": append, "prefixes": prefixes, "B": _log(rng, max(1, n), many), "suffix": "uniform", "lo": lo, "hi": hi, **head}


def _up16(n):
    return -(-n // 16) * 16


def _bits(case):
    return 8 if case.get("cache") == "kv8" else 4


def _row_bytes(case):
    """Bytes of one slot of the packed cache."""
    n_kv, d = case["n_kv"], case["d"]
    if _bits(case) == 8:
        return _up16(n_kv * (d + 4))
    return _up16(_up16(n_kv * (d // 2 + d // GROUP)) + n_kv)


def _layout(case):
    """The lengths of a case, the same for every seed: (prefix lengths, prefix of each request, COLD tokens of each)."""
    rng = random.Random("lengths of %s" % sorted((k, v) for k, v in case.items() if k not in ("name", "append")))
    prefixes = [int(x) for x in str(case.get("prefixes", "")).split(",") if x]
    B = case["B"]
    of = [b % len(prefixes) if prefixes else -1 for b in range(B)]
    lens = []
    for _ in range(B):
        if case.get("suffix") == "lognormal":
            n = int(round(math.exp(rng.gauss(math.log(300.0), 1.0))))
            n = min(max(n, case["lo"]), case["hi"])
        else:
            n = rng.randint(case["lo"], case["hi"])
        lens.append(n)
    return prefixes, of, lens


def work(case):
    n_kv, d = case["n_kv"], case["d"]
    width = 2 if case["dtype"] == "bf16" else 4
    # a token's K or V: codes, scales of 16 elements, and an exponent (or scale) for each head and block
    token = n_kv * (d if _bits(case) == 8 else d // 2 + d // GROUP)
    per = 4 * n_kv if _bits(case) == 8 else n_kv
    if case["op"] != "decode":
        n = case["tokens"]
        packed = n * token + per * (n if case["kind"] == "cold" else -(-n // BLOCK))
        plain = n * n_kv * d * width
        elements = n * n_kv * d
        if case["op"] == "read":
            return {"bytes": 2 * (packed + plain) + (4 * n if case["kind"] == "cold" else 0), "flops": 2 * 2 * elements}
        return {"bytes": 2 * 2 * (packed + plain), "flops": 2 * 5 * elements}
    prefixes, of, lens = _layout(case)
    q = case["B"] * case["n_q"] * d * width
    slab = sum(2 * (L * token + -(-L // BLOCK) * per) for L in prefixes)
    cold = sum(lens) * (2 * (token + per) + 4)
    new = case["B"] * 2 * 2 * n_kv * d * width if case["append"] else 0  # given, and read back
    keys = sum(n + (prefixes[p] if p >= 0 else 0) for n, p in zip(lens, of))
    return {"bytes": slab + cold + 2 * q + case["B"] * case["n_q"] * 4 + new, "flops": 4 * d * case["n_q"] * keys}


# ---- the packed forms -------------------------------------------------------------------------

def _heads_apart(gen, n, n_kv, d, dtype):
    """K or V as projections give them: a few channels of each head far larger than the rest."""
    x = torch.randn(n, n_kv, d, generator=gen, device="cuda")
    channel = torch.exp(0.5 * torch.randn(n_kv, d, generator=gen, device="cuda"))
    return (x * channel).to(dtype)


def _amax(x, per_block):
    """The largest finite magnitude of each head, over a block of slab tokens or over one token: [n, n_kv]."""
    n, n_kv, _ = x.shape
    size = x.abs()
    amax = torch.where(torch.isfinite(size), size, torch.zeros_like(size)).amax(dim=2)
    if per_block:
        blocks = -(-n // BLOCK)
        full = torch.zeros(blocks * BLOCK, n_kv, device=x.device)
        full[:n] = amax
        amax = full.view(blocks, BLOCK, n_kv).amax(dim=1).repeat_interleave(BLOCK, dim=0)[:n]
    return amax


def _pack4(x, per_block):
    """x [n, n_kv, d] as codes (0..15), e4m3 scales [n, n_kv, d / 16] and exponents [n, n_kv] (biased by 127)."""
    x = x.float()
    n, n_kv, d = x.shape
    # the smallest power of two with amax <= 6 * 448 of it
    mantissa, e = torch.frexp(_amax(x, per_block).double() / (E2M1_MAX * E4M3_MAX))
    e = torch.where(mantissa == 0.5, e - 1, e)
    e = torch.where(mantissa == 0, torch.full_like(e, EXP_MIN), e).clamp(EXP_MIN, EXP_MAX)
    unit = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    y = (x / unit[..., None]).view(n, n_kv, d // GROUP, GROUP)
    size = y.abs()
    top = torch.where(torch.isfinite(size), size, torch.zeros_like(size)).amax(dim=3)
    scale = (top / E2M1_MAX).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn).float().clamp(min=E4M3_MIN)
    scale = torch.where(torch.isnan(y).any(dim=3), torch.full_like(scale, math.nan), scale)
    z = size / scale[..., None]
    # the nearest of 0, 0.5, 1, 1.5, 2, 3, 4 and 6, ties to the even code
    code = ((z > 0.25).int() + (z >= 0.75).int() + (z > 1.25).int() + (z >= 1.75).int() + (z > 2.5).int()
            + (z >= 3.5).int() + (z > 5.0).int()) + 8 * torch.signbit(y).int()
    return code.view(n, n_kv, d), scale.to(torch.float8_e4m3fn), e + 127


def _store4(pool, at, x, per_block):
    """Packs the rows of x into the 4-bit pool's slots `at` (a slice or slot ids)."""
    n, n_kv, d = x.shape
    code, scale, e = _pack4(x, per_block)
    a, b = n_kv * d // 2, n_kv * (d // 2 + d // GROUP)
    pool[at, :a] = (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8).reshape(n, a)
    pool[at, a:b] = scale.view(torch.uint8).reshape(n, b - a)
    pool[at, _up16(b) : _up16(b) + n_kv] = e.to(torch.uint8)


def _store8(pool, at, x, per_block):
    """Packs the rows of x into the 8-bit pool's slots `at`."""
    n, n_kv, d = x.shape
    amax = _amax(x.float(), per_block).clamp(min=2.0 ** -96)
    codes = (x.float() * (E4M3_MAX / amax)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    pool[at, : n_kv * d] = codes.view(torch.uint8).reshape(n, n_kv * d)
    pool[at, n_kv * d : n_kv * (d + 4)] = (amax / E4M3_MAX).view(torch.uint8).reshape(n, n_kv * 4)


def _values(rows, n_kv, d, bits=4):
    """fp32 values of packed rows [..., row bytes] -> [..., n_kv, d]."""
    lead = rows.shape[:-1]
    if bits == 8:
        codes = rows[..., : n_kv * d].contiguous().view(torch.float8_e4m3fn).float()
        scales = rows[..., n_kv * d : n_kv * (d + 4)].contiguous().view(torch.float32)
        return codes.reshape(*lead, n_kv, d) * scales.reshape(*lead, n_kv, 1)
    a, b = n_kv * d // 2, n_kv * (d // 2 + d // GROUP)
    packed = rows[..., :a].int()
    code = torch.stack([packed & 15, packed >> 4], dim=-1).reshape(*lead, n_kv, d // GROUP, GROUP)
    # sign, two exponent bits, one of significance: twice the magnitude is m, or (2 + m) 2^(e - 1)
    e, m = (code >> 1) & 3, code & 1
    codes = 0.5 * torch.where(e == 0, m, (2 + m) << (e - 1).clamp(min=0)).float()
    codes = torch.where(code >= 8, -codes, codes)
    scale = rows[..., a:b].contiguous().view(torch.float8_e4m3fn).float().reshape(*lead, n_kv, d // GROUP, 1)
    e = rows[..., _up16(b) : _up16(b) + n_kv].int() - 127
    unit = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return (codes * scale).reshape(*lead, n_kv, d) * unit[..., None]


# ---- inputs -----------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    s = {"case": case}
    n_q, n_kv, d, dtype = case["n_q"], case["n_kv"], case["d"], DTYPES[case["dtype"]]
    bits = _bits(case)
    store = _store8 if bits == 8 else _store4
    if case["op"] != "decode":
        n = case["tokens"]
        prefixes, lens = ([n] if case["kind"] == "slab" else []), []
        n_hot, n_slots = sum(prefixes), n + 2 if case["kind"] == "slab" else 2 * n + 2
    else:
        prefixes, of, lens = _layout(case)
        n_hot, n_slots = sum(prefixes), sum(prefixes) + sum(lens) + 2
    k_pool, v_pool = (torch.zeros(n_slots, _row_bytes(case), dtype=torch.uint8, device="cuda") for _ in range(2))
    if case["op"] == "store":
        s["k_in"], s["v_in"] = _heads_apart(gen, n, n_kv, d, dtype), _heads_apart(gen, n, n_kv, d, dtype)
    else:
        for pool in (k_pool, v_pool):
            at = 0
            for L in prefixes:
                store(pool, slice(at, at + L), _heads_apart(gen, L, n_kv, d, dtype), True)
                at += L
            for i in range(n_hot, n_slots, 16384):
                end = min(n_slots, i + 16384)
                store(pool, slice(i, end), _heads_apart(gen, end - i, n_kv, d, dtype), False)
    if case["op"] != "decode":
        s["slots"] = (n_hot + torch.randperm(n_slots - n_hot, generator=gen, device="cuda")[:n]).to(torch.int32)
        s["k"], s["v"] = (torch.empty(n, n_kv, d, dtype=dtype, device="cuda") for _ in range(2))
    else:
        cap = max(max(lens), 1)
        order = (n_hot + torch.randperm(sum(lens), generator=gen, device="cuda")).to(torch.int32)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["table"] = torch.zeros(case["B"], cap, dtype=torch.int32, device="cuda")
        s["live"] = torch.arange(cap, device="cuda")[None] < s["lens"][:, None]
        s["table"][s["live"]] = order
        s["of"], s["prefixes"] = of, prefixes
        s["q"] = (torch.randn(case["B"], n_q, d, generator=gen, device="cuda") / math.sqrt(d)).to(dtype)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["B"], n_q, dtype=torch.float32, device="cuda")
        s["members"] = [torch.tensor([b for b, p in enumerate(of) if p == i], device="cuda") for i in range(len(prefixes))]
        if case["append"]:
            s["k_in"], s["v_in"] = (_heads_apart(gen, case["B"], n_kv, d, dtype) for _ in range(2))
            s["slots"] = s["table"].gather(1, (s["lens"][:, None] - 1).long())[:, 0].contiguous()
            s["k"], s["v"] = torch.empty_like(s["k_in"]), torch.empty_like(s["v_in"])
    s["k_pool"], s["v_pool"] = k_pool, v_pool
    if own:
        import shared_prefix_kv_decode_gb300 as G

        ctx = s["ctx"] = G.Context(
            n_layers=1, n_q=n_q, n_kv=n_kv, head_dim=d, dtype=G.DTYPE_BF16 if case["dtype"] == "bf16" else G.DTYPE_F32,
            n_slots=n_slots, k_pools=[k_pool], v_pools=[v_pool], hot_fraction=(n_hot + 0.5) / n_slots, max_batch=max(1, case.get("B", 1)),
            device=torch.cuda.current_device(), kv8=bits == 8, kv4=bits == 4)
        s["slabs"] = [ctx.hot_alloc(L)[0] for L in prefixes]
        if case["op"] == "decode":
            s["batch"] = G.Batch([s["slabs"][p] if p >= 0 else -1 for p in of], lens, s["table"], s["table"].shape[1], s["lens"])
            s["plan"] = ctx.dispatch(s["batch"])
            s["ws"] = torch.empty(ctx.workspace_size(s["plan"]), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _own_store(s):
    ctx, n, stream = s["ctx"], s["case"]["tokens"], torch.cuda.current_stream()
    if s["case"]["kind"] == "slab":
        ctx.hot_fill(0, s["slabs"][0], s["k_in"], s["v_in"], stream)
    else:
        ctx.cold_append(0, s["k_in"], s["v_in"], s["slots"], n, stream)
    return _own_read(s)


def _own_read(s):
    ctx, n, stream = s["ctx"], s["case"]["tokens"], torch.cuda.current_stream()
    if s["case"]["kind"] == "slab":
        ctx.hot_read(0, s["slabs"][0], 0, n, s["k"], s["v"], stream)
    else:
        ctx.cold_read(0, s["slots"], n, s["k"], s["v"], stream)
    return s["k"], s["v"]


def _own_decode(s):
    stream = torch.cuda.current_stream()
    if not s["case"]["append"]:
        s["ctx"].decode_attention(0, s["q"], s["batch"], s["plan"], s["o"], s["lse"], s["ws"], s["ws"].numel(), stream)
        return s["o"], s["lse"]
    s["ctx"].decode_attention_append(0, s["q"], s["k_in"], s["v_in"], s["batch"], s["plan"], s["o"], s["lse"], s["ws"], s["ws"].numel(), stream)
    s["ctx"].cold_read(0, s["slots"], s["case"]["B"], s["k"], s["v"], stream)
    return s["o"], s["lse"], s["k"], s["v"]


def _plain_store(s):
    slab = s["case"]["kind"] == "slab"
    at = slice(0, s["case"]["tokens"]) if slab else s["slots"].long()
    _store4(s["k_pool"], at, s["k_in"], slab)
    _store4(s["v_pool"], at, s["v_in"], slab)
    return _plain_read(s)


def _plain_read(s):
    c = s["case"]
    at = slice(0, c["tokens"]) if c["kind"] == "slab" else s["slots"].long()
    for name in ("k", "v"):
        s[name].copy_(_values(s[name + "_pool"][at], c["n_kv"], c["d"], _bits(c)))
    return s["k"], s["v"]


def _gathered(s, pool):
    """Each request's COLD rows [B, cap, n_kv, d] in fp32."""
    rows = pool[torch.where(s["live"], s["table"], s["table"].new_zeros(())).long()]
    return _values(rows, s["case"]["n_kv"], s["case"]["d"])


def _plain_decode(s):
    c = s["case"]
    n_q, n_kv, d, B = c["n_q"], c["n_kv"], c["d"], c["B"]
    g = n_q // n_kv
    if c["append"]:
        for name in ("k", "v"):
            _store4(s[name + "_pool"], s["slots"].long(), s[name + "_in"], False)
            s[name].copy_(_values(s[name + "_pool"][s["slots"].long()], n_kv, d))
    q = s["q"].float()
    # the COLD tokens
    k = _gathered(s, s["k_pool"])
    x = torch.matmul(q.view(B, n_kv, g, d), k.permute(0, 2, 3, 1)).reshape(B, n_q, -1)
    del k
    x = (x / math.sqrt(d)).masked_fill(~s["live"][:, None], -math.inf)
    top = x.amax(dim=2)
    at = 0
    parts = []
    for L, who in zip(s["prefixes"], s["members"]):
        rows = slice(at, at + L)
        at += L
        if who.numel():
            kp = _values(s["k_pool"][rows], n_kv, d)
            qg = q[who].view(-1, n_kv, g, d).transpose(0, 1).reshape(n_kv, -1, d)
            xp = torch.matmul(qg, kp.permute(1, 2, 0)) / math.sqrt(d)
            peak = xp.amax(dim=2).view(n_kv, -1, g).transpose(0, 1).reshape(-1, n_q)
            top[who] = torch.maximum(top[who], peak)
            parts.append((rows, who, xp))
    x = torch.exp(x - top[..., None])
    total = x.sum(dim=2)
    v = _gathered(s, s["v_pool"])
    o = torch.matmul(x.view(B, n_kv, g, -1), v.permute(0, 2, 1, 3)).reshape(B, n_q, d)
    del v
    for rows, who, xp in parts:
        m = top[who].view(-1, n_kv, g).transpose(0, 1).reshape(n_kv, -1, 1)
        w = torch.exp(xp - m)
        vp = _values(s["v_pool"][rows], n_kv, d)
        total[who] += w.sum(dim=2).view(n_kv, -1, g).transpose(0, 1).reshape(-1, n_q)
        o[who] += torch.matmul(w, vp.permute(1, 0, 2)).view(n_kv, -1, g, d).transpose(0, 1).reshape(-1, n_q, d)
    s["o"].copy_(o / total[..., None])
    s["lse"].copy_(top + torch.log(total))
    return (s["o"], s["lse"], s["k"], s["v"]) if c["append"] else (s["o"], s["lse"])


_run_own = {"store": _own_store, "read": _own_read, "decode": _own_decode}
_run_plain = {"store": _plain_store, "read": _plain_read, "decode": _plain_decode}


# ---- 64-bit values ----------------------------------------------------------------------------

def _nearest64(y, digits, least, largest):
    """The nearest value (ties to even) of a float with `digits` significant bits, subnormal below 2^least, saturated."""
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=least) - (digits - 1))
    return (torch.round(y / step) * step).clamp(-largest, largest)


def _through4_64(x, per_block):
    """What rows x [n, n_kv, d] stand for once they are held in 4 bits, in doubles."""
    x = x.double()
    n, n_kv, d = x.shape
    amax = x.abs().amax(dim=2)
    if per_block:
        amax = torch.cat([part.amax(dim=0, keepdim=True).expand_as(part) for part in amax.split(BLOCK)])
    unit = torch.exp2(torch.ceil(torch.log2(amax / 2688)).clamp(EXP_MIN, EXP_MAX))
    unit = torch.where(amax <= 2688 * unit / 2, unit / 2, torch.where(amax > 2688 * unit, unit * 2, unit))
    unit = unit.clamp(min=2.0 ** EXP_MIN)[..., None, None]
    groups = x.view(n, n_kv, -1, GROUP)
    scale = _nearest64(groups.abs().amax(dim=3, keepdim=True) / (6 * unit), 4, -6, E4M3_MAX).clamp(min=E4M3_MIN) * unit
    return (_nearest64(groups / scale, 2, 0, E2M1_MAX) * scale).view(n, n_kv, d)


def exact(case, seed):
    s = prepare(case, seed)
    op, n_q, n_kv, d = case["op"], case["n_q"], case["n_kv"], case["d"]

    def held(rows):
        if _bits(case) == 8:
            codes = rows[:, : n_kv * d].contiguous().view(torch.float8_e4m3fn).double().view(-1, n_kv, d)
            return codes * rows[:, n_kv * d : n_kv * (d + 4)].contiguous().view(torch.float32).double()[..., None]
        nibbles = torch.empty(rows.shape[0], n_kv * d, dtype=torch.long, device="cuda")
        nibbles[:, 0::2], nibbles[:, 1::2] = rows[:, : n_kv * d // 2].long() % 16, rows[:, : n_kv * d // 2].long() // 16
        sign, e, m = 1 - 2 * (nibbles // 8), nibbles // 2 % 4, nibbles % 2
        code = sign * torch.where(e == 0, 0.5 * m, torch.exp2((e - 1).double()) * (1 + 0.5 * m))
        first = n_kv * d // 2
        scale = rows[:, first : first + n_kv * d // GROUP].contiguous().view(torch.float8_e4m3fn).double()
        unit = torch.exp2(rows[:, _up16(first + n_kv * d // GROUP) :][:, :n_kv].double() - 127)
        return code.view(-1, n_kv, d) * scale.repeat_interleave(GROUP, dim=1).view(-1, n_kv, d) * unit[..., None]

    if op == "store":
        return _through4_64(s["k_in"], case["kind"] == "slab"), _through4_64(s["v_in"], case["kind"] == "slab")
    if op == "read":
        at = torch.arange(case["tokens"], device="cuda") if case["kind"] == "slab" else s["slots"].long()
        return held(s["k_pool"][at]), held(s["v_pool"][at])
    start = [0]
    for L in s["prefixes"]:
        start.append(start[-1] + L)
    lens = s["lens"].tolist()
    new = [_through4_64(s[name], False) for name in ("k_in", "v_in")] if case["append"] else None
    o = torch.zeros(case["B"], n_q, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(case["B"], n_q, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        slots = s["table"][b, : lens[b]].long()
        p = s["of"][b]
        if p >= 0:
            slots = torch.cat([torch.arange(start[p], start[p + 1], device="cuda"), slots])
        k, v = held(s["k_pool"][slots]), held(s["v_pool"][slots])
        if new:
            k[-1], v[-1] = new[0][b], new[1][b]
        qb = s["q"][b].double().view(n_kv, n_q // n_kv, d)
        x = torch.einsum("hgd,lhd->hgl", qb, k) * d ** -0.5
        lse[b] = torch.logsumexp(x, dim=2).flatten()
        o[b] = torch.einsum("hgl,lhd->hgd", torch.softmax(x, dim=2), v).reshape(n_q, d)
    return (o, lse, *new) if new else (o, lse)
