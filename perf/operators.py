"""Cases of the 8-bit key/value cache and of the shared-prefix decode.

The operators, each in a plain form (elementary torch operations in 32 bits) and
as the library's calls:

  append   new tokens' K and V rows written into an 8-bit cache: each row of d
           values gets the power-of-two scale 2^(e - 127), e the smallest byte
           >= 1 with max|x| <= 448 * 2^(e - 127), and is held as e4m3 codes of
           x / 2^(e - 127) (round to nearest even).
  read     the cached rows back as bf16 (code * 2^(e - 127)).
  decode   softmax(Q K^T * scale) V and the log-sum-exp straight from that cache.
  prefix   the decode of a batch whose sequences share one long prefix (bf16)
           and go on with a cache of their own.

``page`` = 0 is a contiguous cache [B, Hkv, Lk, d]; otherwise pages of that many
keys, [num_pages, Hkv, page, d], found through a block table.
"""
import math

import torch

own = False

DEVICE = "cuda"


def _case(name, op, **kw):
    c = {"name": name, "op": op, "B": 1, "Hq": 8, "Hkv": 8, "Lq": 1, "Lk": 128, "lo": 1, "d": 128,
         "page": 0, "Lp": 0}
    c.update(kw)
    return c


def listed():
    return [
        # One generated token for each of 64 sequences: the write that precedes every
        # decode step; a few kilobytes, so latency is all there is.
        _case("append_step_b64_h8_d128", "append", B=64, Hkv=8, Lq=1, Lk=4096, lo=1024),
        # Ragged prompts of up to 8K tokens going into 64-key pages after their prefill.
        _case("append_prompts_b4_h8_l8192_d128_page64", "append", B=4, Hkv=8, Lq=8192, Lk=8192,
              lo=2000, page=64),
        # Prompts at the small head size, an odd number of tokens, 16-key pages.
        _case("append_prompts_b7_h4_l2064_d64_page16", "append", B=7, Hkv=4, Lq=2064, Lk=4096,
              lo=2064, d=64, page=16),
        # Contexts read back for a prefill over them: long, contiguous.
        _case("read_b8_h8_l32768_d128", "read", B=8, Hkv=8, Lk=32768, lo=8192),
        # Short ragged contexts in 16-key pages.
        _case("read_b5_h4_l2064_d64_page16", "read", B=5, Hkv=4, Lk=2064, lo=1, d=64, page=16),
        # Two sequences of a few hundred keys: one decode step at the lowest load.
        _case("decode_b2hq16hkv2_lq1_lk1000_d128", "decode", B=2, Hq=16, Hkv=2, Lk=1000),
        # The benchmark's decode workload, its cache in 8 bits.
        _case("decode_b64hq64hkv8_lq1_lk32768_d128", "decode", B=64, Hq=64, Hkv=8, Lk=32768,
              lo=8192),
        # The same heads with 16 drafted tokens per sequence (128 rows share each key),
        # 16-key pages.
        _case("decode_b16hq64hkv8_lq16_lk32768_d128_page16", "decode", B=16, Hq=64, Hkv=8, Lq=16,
              Lk=32768, lo=8192, page=16),
        # One query head per key head, d = 64, ragged lengths from one key up.
        _case("decode_b16hq16hkv16_lq1_lk4099_d64", "decode", B=16, Hq=16, Hkv=16, Lk=4099, d=64),
        # Four sequences behind a system prompt of 2064 tokens, a few tokens into their answers.
        _case("prefix_b4hq32hkv8_lp2064_lk129_d128", "prefix", B=4, Hq=32, Hkv=8, Lk=129, Lp=2064),
        # 64 sequences that answer questions on one document of 32K tokens.
        _case("prefix_b64hq64hkv8_lp32768_lk1024_d128", "prefix", B=64, Hq=64, Hkv=8, Lk=1024,
              Lp=32768),
        # Four drafted tokens each, d = 64, prefix and suffixes in 64-key pages of one pool.
        _case("prefix_b24hq16hkv4_lq4_lp8190_lk2064_d64_page64", "prefix", B=24, Hq=16, Hkv=4,
              Lq=4, Lk=2064, Lp=8190, d=64, page=64),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["append", "read", "decode", "decode", "prefix", "prefix"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([0, 0, 16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    group = rng.choice([1, 2, 4, 5, 8, 8])
    B = log_int(1, 64)
    c = _case("", op, B=B, Hkv=Hkv, Hq=Hkv * group, d=d, page=page)
    del c["name"]
    if op == "append":
        c["Lq"] = rng.choice([1, log_int(1, 8192)])
        while B * Hkv * c["Lq"] > 64 * 8192:
            c["Lq"] = max(1, c["Lq"] // 3)
        c["Lk"] = c["Lq"] + log_int(1, 4096)
        c["lo"] = rng.randint(1, c["Lk"])
    elif op == "read":
        c["Lk"] = log_int(1, 32768)
        while B * Hkv * c["Lk"] > 64 * 32768:
            c["Lk"] = max(1, c["Lk"] // 3)
        c["lo"] = rng.randint(1, c["Lk"])
    elif op == "decode":
        c["Lq"] = rng.choice([1, 1, 2, 3, 8, 16])
        c["Lk"] = log_int(1, 32768)
        while B * Hkv * c["Lk"] * (c["Lq"] * group + 8) > 8 * 32768 * 64 * 16:
            c["Lk"] = max(1, c["Lk"] // 3)
        c["lo"] = rng.randint(1, c["Lk"])
    else:
        c["Lq"] = rng.choice([1, 1, 2, 4, 7])
        c["Lp"] = log_int(1, 32768)
        c["Lk"] = log_int(1, 4096)
        while B * Hkv * group * c["Lq"] * (c["Lp"] + c["Lk"]) > 64 * 64 * 33792:
            c["Lp"] = max(1, c["Lp"] // 3)
            c["Lk"] = max(1, c["Lk"] // 3)
        c["lo"] = rng.randint(1, c["Lk"])
    return c


# ------------------------------------------------------------------ inputs
def _rows(shape, g):
    """K or V rows as a model's projections give them: normal channels, a few of
    them several times larger than the rest, and token norms that vary."""
    d = shape[-1]
    ch = 1.0 + 5.0 * (torch.rand(d, generator=g, device=DEVICE) < 0.04).float()
    tok = torch.exp(0.5 * torch.randn(shape[:-1], generator=g, device=DEVICE))
    x = torch.randn(shape, generator=g, device=DEVICE)
    return (x.mul_(ch).mul_(tok.unsqueeze(-1)) * 0.7).to(torch.bfloat16)


def _quantise(x):
    """bf16 rows [..., d] -> (e4m3 codes, scale bytes [...])."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    byte = torch.where(m > 0.875, e - 8, e - 9) + 127  # 448 = 0.875 * 2^9
    byte = torch.where(m > 0, byte, 1).clamp(min=1)
    codes = torch.ldexp(x, 127 - byte.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, byte.to(torch.uint8)


def _pages(c):
    return -(-c["Lk"] // c["page"])


def _table(c, g, extra=0):
    """A block table of distinct shuffled pages, and the pages of a shared prefix."""
    n = c["B"] * _pages(c)
    perm = torch.randperm(n + extra + 3, generator=g, device=DEVICE).to(torch.int32)
    return perm[:n].view(c["B"], -1).contiguous(), perm[n:n + extra].contiguous(), n + extra + 3


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 7919 + 13)
    B, Hq, Hkv, Lq, Lk, d, page = (c[k] for k in ("B", "Hq", "Hkv", "Lq", "Lk", "d", "page"))
    s = {"case": c, "scale": 1.0 / math.sqrt(d)}
    s["kv_lens"] = torch.randint(c["lo"], Lk + 1, (B,), generator=g, device=DEVICE).to(torch.int32)
    n_prefix = -(-c["Lp"] // page) if page and c["Lp"] else 0
    if page:
        s["table"], s["prefix_table"], n_pages = _table(c, g, n_prefix)
        shape = (n_pages, Hkv, page, d)
    else:
        shape = (B, Hkv, Lk, d)
    if c["op"] == "prefix":
        s["k"], s["v"] = _rows(shape, g), _rows(shape, g)
        if not page:
            s["kp"], s["vp"] = _rows((Hkv, c["Lp"], d), g), _rows((Hkv, c["Lp"], d), g)
    else:  # an 8-bit cache in use: every row holds something
        for name in ("k", "v"):
            codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEVICE)
            exps = torch.empty(shape[:-1], dtype=torch.uint8, device=DEVICE)
            per = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
            for i in range(0, shape[0], per):
                n = min(per, shape[0] - i)
                q, e = _quantise(_rows((n,) + shape[1:], g))
                codes.view(torch.uint8)[i:i + n].copy_(q.view(torch.uint8))
                exps[i:i + n].copy_(e)
            s[name], s[name + "_exp"] = codes, exps
    if c["op"] == "append":
        s["k_new"], s["v_new"] = _rows((B, Hkv, Lq, d), g), _rows((B, Hkv, Lq, d), g)
        new = torch.randint(max(1, Lq // 2), Lq + 1, (B,), generator=g, device=DEVICE)
        s["new_lens"] = torch.minimum(new.to(torch.int32), s["kv_lens"]).contiguous()
    elif c["op"] == "read":
        s["k_out"] = torch.zeros((B, Hkv, page * _pages(c) if page else Lk, d),
                                 dtype=torch.bfloat16, device=DEVICE)
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        s["q"] = torch.randn((B, Hq, Lq, d), generator=g, device=DEVICE).to(torch.bfloat16)
    return s


# -------------------------------------------------------------- plain forms
def _where(s):
    """Row of the flat [rows, d] cache that holds key j of head h of sequence b:
    [B, Hkv, L], L = the longest a sequence can be."""
    c = s["case"]
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    h = torch.arange(Hkv, device=DEVICE).view(1, -1, 1)
    if not page:
        b = torch.arange(B, device=DEVICE).view(-1, 1, 1)
        return (b * Hkv + h) * c["Lk"] + torch.arange(c["Lk"], device=DEVICE)
    j = torch.arange(page * _pages(c), device=DEVICE)
    pg = s["table"].long()[:, j // page].view(B, 1, -1)
    return (pg * Hkv + h) * page + j % page


def _cached(s, name, at, live):
    """Rows `at` of an 8-bit cache in 32 bits, zero where not `live`."""
    d = s["case"]["d"]
    codes = s[name].view(torch.uint8).view(-1, d)[at].view(torch.float8_e4m3fn).float()
    x = torch.ldexp(codes, s[name + "_exp"].view(-1)[at].int().unsqueeze(-1) - 127)
    return torch.where(live.unsqueeze(-1), x, 0.0)


def _softmax_v(scores, values):
    """Rows of scores (-inf where masked) and [(columns, product with V)] ->
    (sum of softmax * V, log-sum-exp)."""
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    return values(p) / total, (m + torch.log(total)).squeeze(-1)


def _plain_append(s):
    c = s["case"]
    i = torch.arange(c["Lq"], device=DEVICE)
    at = (s["kv_lens"] - s["new_lens"]).long().view(-1, 1) + i
    live = (i < s["new_lens"].view(-1, 1)).unsqueeze(1).expand(-1, c["Hkv"], -1)
    rows = torch.gather(_where(s), 2, at.clamp(max=c["Lk"] - 1).unsqueeze(1).expand(
        -1, c["Hkv"], -1))[live]
    for name in ("k", "v"):
        codes, exps = _quantise(s[name + "_new"])
        s[name].view(torch.uint8).view(-1, c["d"])[rows] = codes.view(torch.uint8)[live]
        s[name + "_exp"].view(-1)[rows] = exps[live]
    return s["k"], s["v"], s["k_exp"], s["v_exp"]


def _live(s, L):
    return (torch.arange(L, device=DEVICE) < s["kv_lens"].view(-1, 1)).unsqueeze(1)


def _plain_read(s):
    at = _where(s)
    live = _live(s, at.shape[-1])
    for name in ("k", "v"):
        s[name + "_out"].copy_(_cached(s, name, at, live))
    return s["k_out"], s["v_out"]


def _plain_decode(s):
    c = s["case"]
    at = _where(s)
    live = _live(s, at.shape[-1])
    q = s["q"].float().view(c["B"], c["Hkv"], -1, c["d"])
    sc = q @ _cached(s, "k", at, live).transpose(-1, -2) * s["scale"]
    sc = sc.masked_fill(~live.unsqueeze(2), -math.inf)
    o, lse = _softmax_v(sc, lambda p: p @ _cached(s, "v", at, live))
    return o.view(s["q"].shape).to(torch.bfloat16), lse.view(s["q"].shape[:3])


def _plain_prefix(s):
    c = s["case"]
    B, Hkv, d, Lp, page = c["B"], c["Hkv"], c["d"], c["Lp"], c["page"]
    at = _where(s)
    live = _live(s, at.shape[-1])

    def suffix(x):
        return torch.where(live.unsqueeze(-1), x.view(-1, d)[at].float(), 0.0)

    def prefix(x, xp):
        if page:
            xp = x[s["prefix_table"].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :Lp]
        return xp.float()

    q = s["q"].float().view(B, Hkv, -1, d)
    qh = q.transpose(0, 1).reshape(Hkv, -1, d)  # every sequence's rows of a KV head
    sp = (qh @ prefix(s["k"], s.get("kp")).transpose(-1, -2)).view(Hkv, B, -1, Lp).transpose(0, 1)
    ss = (q @ suffix(s["k"]).transpose(-1, -2)).masked_fill(~live.unsqueeze(2), -math.inf)

    def values(p):
        pp = p[..., :Lp].transpose(0, 1).reshape(Hkv, -1, Lp)
        op = (pp @ prefix(s["v"], s.get("vp"))).view(Hkv, B, -1, d).transpose(0, 1)
        return op + p[..., Lp:] @ suffix(s["v"])

    o, lse = _softmax_v(torch.cat([sp, ss], -1) * s["scale"], values)
    return o.reshape(s["q"].shape).to(torch.bfloat16), lse.reshape(s["q"].shape[:3])


# ------------------------------------------------------- the library's calls
def _own(s):
    import sm_attn_fwd_b200 as ab
    c = s["case"]
    op, page = c["op"], c["page"]
    if op == "append":
        if page:
            ab.attn_cache_append_paged_q8(s["k_new"], s["v_new"], s["k"], s["v"], s["k_exp"],
                                          s["v_exp"], s["table"], s["kv_lens"],
                                          new_lens=s["new_lens"])
        else:
            ab.attn_cache_append_q8(s["k_new"], s["v_new"], s["k"], s["v"], s["k_exp"],
                                    s["v_exp"], s["kv_lens"], new_lens=s["new_lens"])
        return s["k"], s["v"], s["k_exp"], s["v_exp"]
    if op == "read":
        if page:
            return ab.attn_cache_read_paged_q8(s["k"], s["v"], s["k_exp"], s["v_exp"], s["table"],
                                               s["kv_lens"], k=s["k_out"], v=s["v_out"])
        return ab.attn_cache_read_q8(s["k"], s["v"], s["k_exp"], s["v_exp"], s["kv_lens"],
                                     k=s["k_out"], v=s["v_out"])
    if op == "decode":
        if page:
            return ab.attn_decode_paged_q8(s["q"], s["k"], s["v"], s["k_exp"], s["v_exp"],
                                           s["table"], s["kv_lens"], scale=s["scale"])
        return ab.attn_decode_splitkv_q8(s["q"], s["k"], s["v"], s["k_exp"], s["v_exp"],
                                         s["kv_lens"], scale=s["scale"])
    if page:
        return ab.attn_decode_shared_prefix_paged(s["q"], s["k"], s["v"], s["prefix_table"],
                                                  c["Lp"], s["table"], s["kv_lens"],
                                                  scale=s["scale"])
    return ab.attn_decode_shared_prefix(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["kv_lens"],
                                        scale=s["scale"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "read": _plain_read, "decode": _plain_decode,
            "prefix": _plain_prefix}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    B, Hq, Hkv, Lq, d = c["B"], c["Hq"], c["Hkv"], c["Lq"], c["d"]
    mean = (c["lo"] + c["Lk"]) / 2  # lengths are uniform on [lo, Lk]
    if c["op"] == "append":
        rows = 2 * B * Hkv * min((max(1, Lq // 2) + Lq) / 2, mean)
        return {"bytes": rows * (3 * d + 1), "flops": rows * 2 * d}
    if c["op"] == "read":
        rows = 2 * B * Hkv * mean
        return {"bytes": rows * (3 * d + 1), "flops": rows * d}
    io = B * Hq * Lq * (4 * d + 4)  # Q, O, LSE
    if c["op"] == "decode":
        return {"bytes": io + 2 * B * Hkv * mean * (d + 1), "flops": 4 * d * B * Hq * Lq * mean}
    return {"bytes": io + 4 * Hkv * d * (c["Lp"] + B * mean),
            "flops": 4 * d * B * Hq * Lq * (c["Lp"] + mean)}


# ------------------------------------------------ the definitions in 64 bits
def _e4m3_of(y):
    """The e4m3 value nearest to each float64 |y| <= 448, ties to the even code."""
    a = y.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    return torch.copysign(torch.round(a / step) * step, y)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    B, Hq, Hkv, Lq, d, page = (c[k] for k in ("B", "Hq", "Hkv", "Lq", "d", "page"))
    lens = s["kv_lens"].tolist()

    def keys(x, b, h, n):
        """The first n rows of head h of sequence b of a cache tensor."""
        if not page:
            return x[b, h, :n]
        return x.view(torch.uint8)[s["table"][b].long(), h].flatten(0, 1)[:n].view(x.dtype) \
            if x.dtype == torch.float8_e4m3fn else x[s["table"][b].long(), h].flatten(0, 1)[:n]

    def value(name, b, h, n):
        scale = torch.exp2(keys(s[name + "_exp"], b, h, n).double() - 127.0)
        return keys(s[name], b, h, n).double() * scale.unsqueeze(-1)

    if c["op"] == "append":
        new = s["new_lens"].tolist()
        out = {}
        for name in ("k", "v"):
            codes, exps = s[name].double(), s[name + "_exp"].clone()
            for b in range(B):
                x = s[name + "_new"][b, :, :new[b]].double()
                top = x.abs().amax(-1)
                e = torch.full_like(top, 1.0)
                big = top > 0
                e[big] = (torch.ceil(torch.log2(top[big] / 448.0)) + 127.0).clamp(min=1.0)
                e = torch.where(top > 448.0 * torch.exp2(e - 127.0), e + 1, e)
                low = (e > 1) & (top <= 448.0 * torch.exp2(e - 128.0))
                e = torch.where(low, e - 1, e)
                q = _e4m3_of(x * torch.exp2(127.0 - e).unsqueeze(-1))
                j = torch.arange(lens[b] - new[b], lens[b], device=DEVICE)
                if page:
                    pg, r = s["table"][b].long()[j // page], j % page
                    codes[pg, :, r] = q.transpose(0, 1)
                    exps[pg, :, r] = e.transpose(0, 1).to(torch.uint8)
                else:
                    codes[b, :, j] = q
                    exps[b, :, j] = e.to(torch.uint8)
            out[name], out[name + "_exp"] = codes, exps
        return out["k"], out["v"], out["k_exp"], out["v_exp"]

    if c["op"] == "read":
        got = []
        for name in ("k", "v"):
            x = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device=DEVICE)
            for b in range(B):
                for h in range(Hkv):
                    x[b, h, :lens[b]] = value(name, b, h, lens[b])
            got.append(x)
        return tuple(got)

    o = torch.empty((B, Hkv, Hq // Hkv * Lq, d), dtype=torch.float64, device=DEVICE)
    lse = torch.empty(o.shape[:-1], dtype=torch.float64, device=DEVICE)
    q = s["q"].double().view(o.shape)
    for h in range(Hkv):
        if c["op"] == "prefix":
            if page:
                ids = s["prefix_table"].long()
                kp = s["k"][ids, h].flatten(0, 1)[:c["Lp"]].double()
                vp = s["v"][ids, h].flatten(0, 1)[:c["Lp"]].double()
            else:
                kp, vp = s["kp"][h].double(), s["vp"][h].double()
        for b in range(B):
            if c["op"] == "prefix":
                k = torch.cat([kp, keys(s["k"], b, h, lens[b]).double()])
                v = torch.cat([vp, keys(s["v"], b, h, lens[b]).double()])
            else:
                k, v = value("k", b, h, lens[b]), value("v", b, h, lens[b])
            z = torch.einsum("rd,kd->rk", q[b, h], k) * s["scale"]
            lse[b, h] = torch.logsumexp(z, -1)
            o[b, h] = torch.exp(z - lse[b, h].unsqueeze(-1)) @ v
    return o.view(s["q"].shape), lse.view(s["q"].shape[:3])
