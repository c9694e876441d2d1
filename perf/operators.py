"""The 4-bit key/value cache and the adapter projections, as they are measured.

Four kinds of case:

  store   new tokens' keys and values are quantized into a paged 4-bit cache
          and read back as bf16 (``qz_kv4_append``, ``qz_kv4_read``)
  read    whole cached sequences are read back as bf16 (``qz_kv4_read``)
  attend  attention of one or several new tokens a sequence over the cache
          (``qz_kv4_attention``)
  lora    a packed int4 or int8 projection with a low-rank adapter per token
          (``qz_w4a16_lora_gemv``, ``qz_w8a16_lora_gemv``)

The cache holds each head's vector of a token in groups of ``group`` values:
4-bit codes 0..15, a bf16 scale S and a zero-point Z per group, with
S = (max - min) / 15 over the range widened to 0 (fp32, stored as bf16 rounded
up, 0 -> 1), Z = -round(min / S), code = clamp(round(x / S + Z), 0, 15), and it
stands for S (code - Z).
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a batch of 32 requests writes its new tokens
        dict(name="store_decode", kind="store", seqs=32, lens_seed=11, len_lo=200, len_hi=1500,
             new_lo=1, new_hi=1, kv_heads=8, dim=128, group=128, page=16),
        # five prompts of odd lengths are written at once
        dict(name="store_prompt", kind="store", seqs=5, lens_seed=12, len_lo=1, len_hi=1,
             new_lo=900, new_hi=2500, kv_heads=8, dim=128, group=64, page=64),
        # short cached prefixes with small heads, read back for a prefill
        dict(name="read_prefix", kind="read", seqs=9, lens_seed=13, len_lo=3, len_hi=700,
             kv_heads=4, dim=64, group=32, page=16),
        # two long documents read back
        dict(name="read_long", kind="read", seqs=2, lens_seed=14, len_lo=15000, len_hi=20000,
             kv_heads=8, dim=128, group=128, page=64),
        # one request decoding: the smallest call, latency counts
        dict(name="attend_single", kind="attend", seqs=1, lens_seed=15, len_lo=777, len_hi=777,
             new_lo=1, new_hi=1, heads=32, kv_heads=8, dim=128, group=128, page=16, window=0),
        # one request with a very long context
        dict(name="attend_long", kind="attend", seqs=1, lens_seed=16, len_lo=131001,
             len_hi=131001, new_lo=1, new_hi=1, heads=64, kv_heads=8, dim=128, group=64,
             page=64, window=0),
        # a large ragged decode batch: the largest call
        dict(name="attend_batch", kind="attend", seqs=128, lens_seed=17, len_lo=1000,
             len_hi=16000, new_lo=1, new_hi=1, heads=32, kv_heads=8, dim=128, group=128,
             page=16, window=0),
        # several draft tokens verified at once, one head per key head, a sliding window
        dict(name="attend_verify", kind="attend", seqs=17, lens_seed=18, len_lo=30, len_hi=9000,
             new_lo=2, new_hi=6, heads=32, kv_heads=32, dim=64, group=32, page=32,
             window=2000),
        # mixed batch: single tokens beside short prompt pieces, wide heads
        dict(name="attend_mixed", kind="attend", seqs=12, lens_seed=19, len_lo=64, len_hi=6000,
             new_lo=1, new_hi=48, heads=16, kv_heads=2, dim=256, group=64, page=16, window=0),
        # one token through a 4096 x 4096 int4 layer with one adapter
        dict(name="lora_single", kind="lora", bits=4, tokens=1, n=4096, k=4096, group=128,
             rank=16, adapters=4, run=1, ids_seed=1),
        # 16 requests with adapters of their own beside a 28672 x 8192 int4 layer
        dict(name="lora_batch", kind="lora", bits=4, tokens=16, n=28672, k=8192, group=128,
             rank=64, adapters=24, run=1, ids_seed=2),
        # 45 tokens in short runs beside an int8 layer
        dict(name="lora_int8", kind="lora", bits=8, tokens=45, n=11008, k=4096, group=4096,
             rank=32, adapters=10, run=4, ids_seed=3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(case):
    """Lengths before the new tokens, and new tokens, of each sequence."""
    r = random.Random(case["lens_seed"])
    old = [_log_int(r, case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    if case["kind"] == "read":
        return [0] * case["seqs"], old
    new = [_log_int(r, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    if case["kind"] == "store":
        return old, new
    # attend: the length drawn counts the new tokens
    return [max(0, n - m) for n, m in zip(old, new)], [min(n, m) for n, m in zip(old, new)]


def _adapter_ids(case):
    """Adapter of every token, -1 for none; tokens of a request follow one another."""
    r = random.Random(case["ids_seed"])
    ids = []
    while len(ids) < case["tokens"]:
        one = -1 if len(ids) > 0 and r.random() < 0.125 else r.randrange(case["adapters"])
        ids += [one] * r.randint(1, case["run"])
    return ids[:case["tokens"]]


def draw(rng):
    kind = rng.choice(["store", "read", "attend", "attend", "lora"])
    if kind == "lora":
        bits = rng.choice([4, 8])
        while True:
            k = 128 * _log_int(rng, 2, 86)
            n = _log_int(rng, 33, 28672)
            if n * k <= 8192 * 14336:
                break
        rank = 8 * _log_int(rng, 1, 16)
        return dict(kind="lora", bits=bits, tokens=_log_int(rng, 1, 64), n=n, k=k,
                    group=k if bits == 8 else rng.choice([32, 64, 128]), rank=rank,
                    adapters=_log_int(rng, 1, min(40, 1536 // rank)),
                    run=rng.choice([1, 1, 3, 8]), ids_seed=rng.randrange(10 ** 6))
    dim = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if dim // 4 <= g <= dim])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    case = dict(kind=kind, lens_seed=rng.randrange(10 ** 6), kv_heads=kv_heads, dim=dim,
                group=group, page=rng.choice([16, 32, 48, 64, 128]))
    budget = 64 * 1024 * 1024          # cached values of one kind (keys or values)
    if kind == "store":
        hi = _log_int(rng, 1, 3000)
        seqs = _log_int(rng, 1, 64)
        while seqs * hi * kv_heads * dim > budget:
            seqs, hi = (seqs + 1) // 2, (hi + 1) // 2
        case.update(seqs=seqs, len_lo=1, len_hi=_log_int(rng, 1, 800),
                    new_lo=max(1, hi // rng.choice([1, 2, 8])), new_hi=hi)
        return case
    hi = _log_int(rng, 1, 40000)
    seqs = _log_int(rng, 1, 100)
    while seqs * hi * kv_heads * dim > 4 * budget:
        seqs, hi = (seqs + 1) // 2, (hi + 1) // 2
    case.update(seqs=seqs, len_lo=max(1, hi // rng.choice([1, 4, 16])), len_hi=hi)
    if kind == "attend":
        share = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        new_hi = rng.choice([1, 1, 1, 4, 9, 40])
        while seqs * new_hi * share * kv_heads * hi > 2 ** 30 and new_hi > 1:
            new_hi = (new_hi + 1) // 2
        case.update(heads=kv_heads * share, new_lo=1, new_hi=new_hi,
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]))
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * int(seed) + salt)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _keys_values(case, total, seed):
    """Keys with a few large and shifted channels a head, plain values."""
    h, d = case["kv_heads"], case["dim"]
    g = _generator(seed, 1)
    gain = 1.0 + 6.0 * (torch.rand((h, d), generator=g, device=DEV) < 0.03)
    shift = _randn((h, d), g)
    k = (_randn((total, h, d), g).mul_(gain).add_(shift)).to(torch.bfloat16)
    v = _randn((total, h, d), g).mul_(0.5).to(torch.bfloat16)
    return k, v


def _prefix(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return cu


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pages(case, lens, seed):
    """Page table: every sequence's pages, scattered over the cache."""
    page = case["page"]
    need = [(n + page - 1) // page for n in lens]
    width = max(1, max(need))
    total = max(1, sum(need))
    order = list(range(total))
    random.Random(seed).shuffle(order)
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return _int32(table), total


def _slots(table, page, start, count):
    """Places in the cache (page * page size + offset) of tokens start.. of a sequence."""
    pos = torch.arange(start, start + count, device=table.device)
    return table[pos // page].long() * page + pos % page


def _queries(case, tokens, seed):
    return _randn((tokens, case["heads"], case["dim"]), _generator(seed, 2)).to(torch.bfloat16)


def _layer(case, seed):
    """Weights, activations and adapters of a projection."""
    n, k, r = case["n"], case["k"], case["rank"]
    g = _generator(seed, 3)
    w = _randn((n, k), g).mul_(0.02)
    w = torch.where(torch.rand((n, k), generator=g, device=DEV) < 1e-3, w * 20.0, w)
    a = _randn((case["tokens"], k), g).to(torch.bfloat16)
    down = _randn((case["adapters"], r, k), g).mul_(k ** -0.5).to(torch.bfloat16)
    up = _randn((case["adapters"], n, r), g).mul_(0.05).to(torch.bfloat16)
    scale = torch.rand((case["adapters"],), generator=g, device=DEV) * 1.75 + 0.25
    return w.to(torch.bfloat16), a, down, up, scale


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------
def _round_up_bf16(s):
    """fp32 -> the smallest bf16 at or above it (s >= 0), as fp32."""
    bits = s.view(torch.int32)
    up = torch.where((bits & 0xFFFF) != 0, (bits | 0xFFFF) + 1, bits)
    return up.view(torch.float32)


def _over(x, number):
    """x / number, rounded once (a division by a number may become a product
    with its rounded inverse; one by a tensor does not)."""
    return x / torch.full_like(x, number)


def _quantize_plain(x, group):
    """(..., D) bf16 -> packed codes (..., D/2), scales (..., D/group) bf16, zeros uint8."""
    x = x.float()
    x = x.view(*x.shape[:-1], x.shape[-1] // group, group)
    lo = x.amin(-1).clamp_max(0.0)
    hi = x.amax(-1).clamp_min(0.0)
    s = _over(hi - lo, 15.0)
    s = _round_up_bf16(torch.where(s == 0, torch.ones_like(s), s))
    z = -torch.round(lo / s)
    c = torch.round(x / s[..., None] + z[..., None]).clamp_(0, 15).to(torch.uint8)
    c = c.view(*c.shape[:-2], -1)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.to(torch.bfloat16), z.to(torch.uint8)


def _dequantize_plain(codes, s, z, group):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    c = c.view(*c.shape[:-1], -1, group).float()
    return ((c - z.float()[..., None]) * s.float()[..., None]).flatten(-2)


def _quantize_int8_plain(w):
    """Symmetric int8 per row."""
    x = w.float()
    s = _over(x.abs().amax(1, keepdim=True), 127.0)
    s = _round_up_bf16(torch.where(s == 0, torch.ones_like(s), s))
    return torch.round(x / s).to(torch.int8).view(torch.uint8), s.to(torch.bfloat16)


def _plain_store(st):
    codes = _quantize_plain(st["k"], st["group"]), _quantize_plain(st["v"], st["group"])
    out = []
    for (c, s, z), cache in zip(codes, st["plain"]):
        for part, new in zip(cache, (c, s, z)):
            part[st["slots"]] = new
        out.append(_dequantize_plain(*[p[st["slots"]] for p in cache],
                                     st["group"]).to(torch.bfloat16))
    return out


def _plain_read(st):
    return [_dequantize_plain(*[p[st["slots"]] for p in cache], st["group"]).to(torch.bfloat16)
            for cache in st["plain"]]


def _plain_attend(st):
    q, group, window, page = st["q"], st["group"], st["window"], st["page"]
    heads, kv = q.shape[1], st["kv_heads"]
    out = torch.zeros_like(q)
    for b, (n, m) in enumerate(zip(st["lens"], st["new"])):
        if n == 0 or m == 0:
            continue
        first = max(0, n - m - window + 1) if window else 0
        slots = _slots(st["table"][b], page, first, n - first)
        k, v = (_dequantize_plain(*[p[slots] for p in cache], group) for cache in st["plain"])
        rows = q[st["cu"][b]:st["cu"][b] + m].float().view(m, kv, heads // kv, -1)
        rows = rows.permute(1, 2, 0, 3).reshape(kv, -1, q.shape[2])
        s = torch.bmm(rows, k.permute(1, 2, 0)) * st["scale"]
        at = torch.arange(n - m, n, device=q.device).repeat(heads // kv)[:, None]
        key = torch.arange(first, n, device=q.device)[None, :]
        seen = key <= at
        if window:
            seen = seen & (key > at - window)
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.bmm(p, v.permute(1, 0, 2)) / p.sum(-1, keepdim=True)
        o = o.view(kv, heads // kv, m, -1).permute(2, 0, 1, 3).reshape(m, heads, -1)
        out[st["cu"][b]:st["cu"][b] + m] = o.to(torch.bfloat16)
    return out


def _plain_lora(st):
    if st["bits"] == 4:
        w = _dequantize_plain(st["codes"], st["scales"], st["zeros"], st["group"])
    else:
        w = st["codes"].view(torch.int8).float() * st["scales"].float()
    w = w.to(torch.bfloat16).float()               # the weight a packed layer stands for
    a = st["a"].float()
    y = a @ w.T
    ids = st["ids"].long().clamp_min(0)            # a token without an adapter gets factor 0
    factor = torch.where(st["ids"] >= 0, st["lora_scale"][ids], 0.0)
    h = torch.bmm(st["down"][ids].float(), a[:, :, None])
    y = y + torch.bmm(st["up"][ids].float(), h)[:, :, 0] * factor[:, None]
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the measured interface
# ---------------------------------------------------------------------------
def _prepare_cache(case, seed):
    old, new = _lens(case)
    lens = [a + b for a, b in zip(old, new)]
    table, pages = _pages(case, lens, seed)
    st = dict(kind=case["kind"], group=case["group"], page=case["page"], dim=case["dim"],
              kv_heads=case["kv_heads"], lens=lens, new=new, table=table,
              kv_lens=_int32(lens), cu=_prefix(new))
    st["cu_dev"] = _int32(st["cu"])
    h, d, g, page = case["kv_heads"], case["dim"], case["group"], case["page"]
    if own:
        import weight_only_quantization_wise_b200 as qz
        st["qz"] = qz
        st["cache"] = torch.zeros(qz.qz_kv4_cache_bytes(pages, h, d, page, g),
                                  dtype=torch.uint8, device=DEV)
    else:
        st["plain"] = [(torch.zeros((pages * page, h, d // 2), dtype=torch.uint8, device=DEV),
                        torch.zeros((pages * page, h, d // g), dtype=torch.bfloat16, device=DEV),
                        torch.zeros((pages * page, h, d // g), dtype=torch.uint8, device=DEV))
                       for _ in range(2)]
    if case["kind"] == "store":
        st["k"], st["v"] = _keys_values(case, st["cu"][-1], seed)
        if not own:
            st["slots"] = torch.cat([_slots(table[b], page, old[b], new[b])
                                     for b in range(case["seqs"])])
        return st
    # read, attend: the cached tokens were appended before
    k, v = _keys_values(case, sum(lens), seed)
    if own:
        qz.qz_kv4_append(st["cache"], k, v, table, st["kv_lens"], _int32(_prefix(lens)), page, g)
    else:
        at = 0
        for b, n in enumerate(lens):
            slots = _slots(table[b], page, 0, n)
            for x, cache in zip((k, v), st["plain"]):
                for part, fill in zip(cache, _quantize_plain(x[at:at + n], g)):
                    part[slots] = fill
            at += n
    if case["kind"] == "read":
        if not own:
            st["slots"] = torch.cat([_slots(table[b], page, 0, n) for b, n in enumerate(lens)])
        return st
    st["q"] = _queries(case, st["cu"][-1], seed)
    st["window"] = case["window"]
    st["scale"] = case["dim"] ** -0.5
    if own:
        st["ws"] = qz.Workspace(DEV)
    return st


def prepare(case, seed):
    if case["kind"] != "lora":
        return _prepare_cache(case, seed)
    w, a, down, up, scale = _layer(case, seed)
    st = dict(kind="lora", bits=case["bits"], n=case["n"], k=case["k"], group=case["group"],
              a=a, down=down, up=up, lora_scale=scale, ids=_int32(_adapter_ids(case)))
    if case["bits"] == 4:
        st["codes"], st["scales"], st["zeros"] = _quantize_plain(w, case["group"])
    else:
        st["codes"], st["scales"] = _quantize_int8_plain(w)
    if own:
        import weight_only_quantization_wise_b200 as qz
        st["qz"], st["ws"] = qz, qz.Workspace(DEV)
    return st


def run(st):
    kind = st["kind"]
    if not own:
        return {"store": _plain_store, "read": _plain_read, "attend": _plain_attend,
                "lora": _plain_lora}[kind](st)
    qz = st["qz"]
    if kind == "lora":
        if st["bits"] == 4:
            return qz.qz_w4a16_lora_gemv(st["a"], st["codes"], st["scales"], st["zeros"],
                                         st["n"], st["k"], st["down"], st["up"], st["ids"],
                                         st["lora_scale"], group_size=st["group"],
                                         workspace=st["ws"])
        return qz.qz_w8a16_lora_gemv(st["a"], st["codes"], st["scales"], st["n"], st["k"],
                                     st["down"], st["up"], st["ids"], st["lora_scale"],
                                     workspace=st["ws"])
    if kind == "attend":
        return qz.qz_kv4_attention(st["q"], st["cache"], st["table"], st["kv_lens"],
                                   st["cu_dev"], st["kv_heads"], st["page"], st["group"],
                                   scale=st["scale"], window=st["window"], workspace=st["ws"])
    if kind == "store":
        qz.qz_kv4_append(st["cache"], st["k"], st["v"], st["table"], st["kv_lens"],
                         st["cu_dev"], st["page"], st["group"])
    return list(qz.qz_kv4_read(st["cache"], st["table"], st["kv_lens"], st["cu_dev"],
                               st["cu"][-1], st["kv_heads"], st["dim"], st["page"],
                               st["group"]))


def work(case):
    if case["kind"] == "lora":
        m, n, k, r = case["tokens"], case["n"], case["k"], case["rank"]
        ids = _adapter_ids(case)
        used = sum(1 for i in ids if i >= 0)
        weights = n * k * case["bits"] // 8 + n * (k // case["group"]) * (
            3 if case["bits"] == 4 else 2)
        adapters = len({i for i in ids if i >= 0}) * (2 * r * (n + k) + 4)
        return dict(bytes=weights + adapters + 2 * m * (k + n) + 4 * m,
                    flops=2 * m * n * k + 2 * used * r * (n + k))
    old, new = _lens(case)
    h, d, g = case["kv_heads"], case["dim"], case["group"]
    packed = 2 * h * (d // 2 + 3 * (d // g))       # key and value of a token, all heads
    dense = 2 * h * d * 2
    tokens = sum(new)
    if case["kind"] == "store":
        return dict(bytes=tokens * 2 * (dense + packed), flops=tokens * 2 * h * d * 8)
    if case["kind"] == "read":
        return dict(bytes=tokens * (dense + packed), flops=tokens * 2 * h * d * 2)
    cached = pairs = 0
    w = case["window"]
    for a, m in zip(old, new):
        n = a + m
        cached += n - (max(0, a - w + 1) if w else 0)
        for p in range(a, n):
            pairs += min(p + 1, w) if w else p + 1
    return dict(bytes=cached * packed + 2 * tokens * case["heads"] * d * 2 +
                4 * case["seqs"] * 3 + 4 * (cached // case["page"]),
                flops=4 * d * pairs * case["heads"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _held_values(x, group):
    """The values S (code - Z) that the 4-bit form of x stands for, float64.

    S is part of the format: the fp32 quotient, rounded up to 8 significant
    bits."""
    x = x.double().unflatten(-1, (-1, group))
    top = torch.maximum(x.max(-1, keepdim=True).values, x.new_zeros(()))
    low = torch.minimum(x.min(-1, keepdim=True).values, x.new_zeros(()))
    width = (top - low).float().double()
    m, e = torch.frexp(torch.div(width, torch.full_like(width, 15)).float().double())
    s = torch.ldexp(torch.ceil(m * 256) / 256, e)
    s = torch.where(width == 0, torch.ones_like(s), s)
    z = -torch.round(low / s)
    c = torch.round(x / s + z).clamp(0, 15)
    return (s * (c - z)).flatten(-2)


def _exact_cache(case, seed):
    old, new = _lens(case)
    lens = [a + b for a, b in zip(old, new)]
    if case["kind"] != "attend":
        k, v = _keys_values(case, sum(new), seed)
        return [_held_values(k, case["group"]), _held_values(v, case["group"])]
    k, v = _keys_values(case, sum(lens), seed)
    q = _queries(case, sum(new), seed)
    heads, kv, d = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros((sum(new), heads, d), dtype=torch.float64, device=DEV)
    at = row = 0
    for n, m in zip(lens, new):
        kk, vv = _held_values(k[at:at + n], case["group"]), _held_values(v[at:at + n],
                                                                          case["group"])
        pos = torch.arange(n, device=DEV)
        for h in range(kv):
            qs = q[row:row + m, h * (heads // kv):(h + 1) * (heads // kv)].double()
            for i in range(m):
                p = n - m + i
                keep = pos <= p
                if case["window"]:
                    keep &= pos > p - case["window"]
                logits = (qs[i] @ kk[keep, h].T) / math.sqrt(d)
                prob = torch.softmax(logits, -1)
                out[row + i, h * (heads // kv):(h + 1) * (heads // kv)] = prob @ vv[keep, h]
        at += n
        row += m
    return out


def exact(case, seed):
    if case["kind"] != "lora":
        return _exact_cache(case, seed)
    w, a, down, up, scale = _layer(case, seed)
    if case["bits"] == 4:
        held = _held_values(w, case["group"])
    else:
        x = w.double()
        top = x.abs().max(1, keepdim=True).values
        m, e = torch.frexp((top / torch.full_like(top, 127)).float().double())
        s = torch.ldexp(torch.ceil(m * 256) / 256, e)
        held = s * torch.round(x / s)
    held = held.to(torch.bfloat16).double()        # a packed layer's weights are bf16 values
    y = a.double() @ held.T
    for i, r in enumerate(_adapter_ids(case)):
        if r >= 0:
            y[i] += scale[r].double() * (up[r].double() @ (down[r].double() @ a[i].double()))
    return y
