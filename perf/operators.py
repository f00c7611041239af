"""Measured cases of the 4-bit paged cache's operators: storing tokens and reading them back,
attention of packed 16-bit queries over it, and the management of its pages.

The cache (pages of 64 tokens, head dimension 128) holds K and V in NVFP4: per token, KV head and
16 channels E2M1 codes under one E4M3 scale, and one FP32 scale for the whole cache.

  K codes  [pages, heads, 64, 64]   byte i of a token: channels 2i (low nibble) and 2i + 1
  K scales [pages, heads, 64, 8]
  V codes  [pages, heads, 32, 128]  byte c of a token pair: channel c of the even (low) and odd token
  V scales [pages, heads, 8, 64]

Operators ("op" of a case):
  attend   causal attention of packed sequences, each one's query tokens the last of its context
  store    new tokens quantized into their pages, then read back
  fork     sequences dropped, others forked into their places, the shared tails' pages copied
  compact  live pages moved to the lowest page numbers
"""
import math
import random

import torch

own = False

DEV = "cuda"
PAGE, D = 64, 128
K_SCALE, V_SCALE = 2.0 ** -4, 2.0 ** -6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HEAD_BYTES = PAGE * 2 * (D // 2 + D // 16)      # one page of one KV head: K and V codes and scales


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def attend(seqs, steps, q, past, heads, dtype, lens):
    """The first `steps` sequences bring one query token, the others q[0]..q[1]; past: cached before."""
    return dict(op="attend", seqs=seqs, steps=steps, q_lo=q[0], q_hi=q[1], past_lo=past[0], past_hi=past[1],
                hq=heads[0], hkv=heads[1], dtype=dtype, lens=lens)


def store(seqs, q, past, hkv, dtype, lens):
    return dict(op="store", seqs=seqs, steps=0, q_lo=q[0], q_hi=q[1], past_lo=past[0], past_hi=past[1],
                hq=hkv, hkv=hkv, dtype=dtype, lens=lens)


def listed():
    return [
        # one user's next token in a short chat: latency
        dict(name="attend_1x1k", **attend(1, 1, (1, 1), (1000, 1000), (32, 8), "bf16", 1)),
        # a served batch's next tokens over long contexts: the cache is read once
        dict(name="attend_64x32k", **attend(64, 64, (1, 1), (8191, 32767), (32, 8), "bf16", 2)),
        # several proposed tokens per sequence checked at once
        dict(name="attend_verify", **attend(24, 0, (2, 5), (700, 9000), (64, 8), "fp16", 3)),
        # short prompts of different lengths, as many KV heads as query heads
        dict(name="attend_ragged_mha", **attend(7, 0, (17, 900), (0, 0), (16, 16), "fp16", 4)),
        # one long prompt
        dict(name="attend_prompt_16k", **attend(1, 0, (16384, 16384), (0, 0), (32, 8), "bf16", 5)),
        # a chunk of a long prompt whose beginning is in the cache
        dict(name="attend_chunk_32k", **attend(1, 0, (512, 512), (32000, 32000), (32, 8), "bf16", 6)),
        # a running batch's next tokens together with two prompts' chunks; five query heads a KV head
        dict(name="attend_mixed", **attend(34, 32, (300, 512), (500, 8000), (40, 8), "bf16", 7)),
        # the batch's new tokens, one each
        dict(name="store_64x1", **store(64, (1, 1), (8191, 32767), 8, "bf16", 8)),
        # prompts of different lengths
        dict(name="store_prompts", **store(9, (100, 6000), (0, 130), 8, "fp16", 9)),
        # parallel answers: four continuations of each of 16 prompts
        dict(name="fork_64", op="fork", seqs=80, keep=16, past_lo=200, past_hi=4000, hkv=8, free=1.2, lens=10),
        # a cache whose sequences came and went, a third of it live
        dict(name="compact_6k", op="compact", seqs=48, keep=48, past_lo=500, past_hi=5000, hkv=8, free=3.0, lens=11),
    ]


def spread(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = work(listed()[4])["flops"]
    while True:
        op = rng.choice(["attend", "attend", "attend", "attend", "store", "fork", "compact"])
        dtype, lens = rng.choice(["bf16", "fp16"]), rng.randrange(1 << 20)
        if op == "store":
            hi = spread(rng, 1, 6000)
            past = spread(rng, 1, 8000)
            c = store(spread(rng, 1, 64), (rng.randint(1, hi), hi), (rng.randint(0, past), past), rng.choice([1, 2, 5, 8, 16]), dtype, lens)
            if sum(n for n, _ in lengths(c)) > 30000 or sum(n for _, n in lengths(c)) > 400000:
                continue
            return c
        if op in ("fork", "compact"):
            keep = spread(rng, 1, 24)
            seqs = keep + spread(rng, 1, 60) if op == "fork" else keep
            hi = spread(rng, 40, 5000)
            return dict(op=op, seqs=seqs, keep=keep, past_lo=rng.randint(1, hi), past_hi=hi, hkv=rng.choice([1, 2, 8]),
                        free=round(rng.uniform(1.3, 4.0), 2), lens=lens)
        heads = rng.choice([(32, 8), (16, 16), (64, 8), (8, 1), (40, 8), (6, 2), (28, 4), (16, 1)])
        seqs = spread(rng, 1, 64)
        steps = rng.choice([0, seqs, rng.randint(0, seqs)])
        q_hi, past_hi = spread(rng, 1, 12000), spread(rng, 1, 32767)
        c = attend(seqs, steps, (rng.randint(1, q_hi), q_hi), (rng.randint(0, past_hi), past_hi), heads, dtype, lens)
        ls = lengths(c)
        q_max, most_ctx = max(n for n, _ in ls), max(n for _, n in ls)
        if seqs * q_max * most_ctx * heads[0] > 16384 * 16384 * 32 or seqs * most_ctx * heads[1] > 64 * 32768 * 8:
            continue                                   # the padded plain form has to fit
        if work(c)["flops"] > most:
            continue
        return c


def lengths(case):
    """[(new tokens, context with them)] of each sequence: part of the case, whatever the seed."""
    r = random.Random(case["lens"])
    got = []
    for s in range(case["seqs"]):
        n = 1 if s < case["steps"] else r.randint(case["q_lo"], case["q_hi"])
        got.append((n, n + r.randint(case["past_lo"], case["past_hi"])))
    return got


def pages_of(n):
    return (n + PAGE - 1) // PAGE


def pool_layout(case):
    """Lengths and page lists of a pool case, and the number of its pages."""
    r = random.Random(case["lens"])
    lens = [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["keep"])] + [0] * (case["seqs"] - case["keep"])
    used = sum(pages_of(n) for n in lens)
    total = int(used * case["free"]) + case["seqs"] + 1
    ids = r.sample(range(total), used)
    rows, at = [], 0
    for n in lens:
        rows.append(ids[at:at + pages_of(n)])
        at += pages_of(n)
    src = [r.randrange(case["keep"]) for _ in range(case["seqs"] - case["keep"])]
    return lens, rows, src, total


def work(case):
    op = case["op"]
    if op in ("fork", "compact"):
        lens, rows, src, total = pool_layout(case)
        ids = [p for row in rows for p in row]
        table = 4 * len(rows) * max(map(len, rows))
        moved = sum(lens[s] % PAGE != 0 for s in src) if op == "fork" else sum(p >= len(ids) for p in ids)
        return {"bytes": 2.0 * moved * case["hkv"] * HEAD_BYTES + 2 * table + 8 * total, "flops": 0.0}
    ls = lengths(case)
    t = sum(n for n, _ in ls)
    if op == "store":
        return {"bytes": 2.0 * t * case["hkv"] * (2 * 2 * D + HEAD_BYTES // PAGE), "flops": 0.0}
    ctx = sum(n for _, n in ls)
    seen = sum(n * (c - n) + n * (n + 1) // 2 for n, c in ls)
    return {"bytes": ctx * case["hkv"] * HEAD_BYTES / PAGE + 2.0 * 2 * t * case["hq"] * D, "flops": 4.0 * D * case["hq"] * seen}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def keys_values(n, hkv, gen, shape):
    """K with per-channel means and a few outlier channels, V normal: [n, ...]."""
    mean, outlier = shape
    k = (torch.randn(n, hkv, D, generator=gen, device=DEV) + mean) * outlier
    v = torch.randn(n, hkv, D, generator=gen, device=DEV)
    return k, v


def channel_shape(hkv, gen):
    mean = 0.5 * torch.randn(1, hkv, D, generator=gen, device=DEV)
    outlier = torch.ones(1, hkv, D, device=DEV)
    at = torch.randint(0, D, (1, hkv, 4), generator=gen, device=DEV)
    outlier.scatter_(2, at, 10.0)
    return mean, outlier


def filled_cache(pages, hkv, gen, shape):
    """Pages of quantized K and V."""
    kp = torch.empty(pages, hkv, PAGE, D // 2, dtype=torch.uint8, device=DEV)
    ks = torch.empty(pages, hkv, PAGE, D // 16, dtype=torch.uint8, device=DEV)
    vp = torch.empty(pages, hkv, PAGE // 2, D, dtype=torch.uint8, device=DEV)
    vs = torch.empty(pages, hkv, D // 16, PAGE, dtype=torch.uint8, device=DEV)
    for a in range(0, pages, 256):
        n = min(256, pages - a)
        k, v = keys_values(n * PAGE, hkv, gen, shape)
        kc, kx = encode(k, K_SCALE)
        vc, vx = encode(v, V_SCALE)
        kc = kc[..., 0::2] | (kc[..., 1::2] << 4)
        kp[a:a + n] = kc.view(n, PAGE, hkv, D // 2).transpose(1, 2)
        ks[a:a + n] = kx.view(n, PAGE, hkv, D // 16).transpose(1, 2)
        vc = vc.view(n, PAGE // 2, 2, hkv, D)
        vp[a:a + n] = (vc[:, :, 0] | (vc[:, :, 1] << 4)).transpose(1, 2)
        vs[a:a + n] = vx.view(n, PAGE, hkv, D // 16).permute(0, 2, 3, 1)
    return dict(k_pages=kp, k_scales=ks, k_tensor_scale=torch.full((1,), K_SCALE, device=DEV),
                v_pages=vp, v_scales=vs, v_tensor_scale=torch.full((1,), V_SCALE, device=DEV))


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hkv = case["hkv"]
    shape = channel_shape(hkv, gen)
    if case["op"] in ("fork", "compact"):
        lens, rows, src, total = pool_layout(case)
        width = max(map(len, rows)) + 1
        refs = [0] * total
        for row in rows:
            for p in row:
                refs[p] = 1
        table = int32([row + [-1] * (width - len(row)) for row in rows])
        st = dict(case=case, cache=filled_cache(total, hkv, gen, shape), refs=int32(refs), table=table, lens=int32(lens))
        if case["op"] == "fork":
            st.update(src=int32(src), dst=int32(list(range(case["keep"], case["seqs"]))))
        else:
            st.update(refs0=st["refs"].clone(), table0=table.clone())
        return st
    ls = lengths(case)
    count = [pages_of(c) for _, c in ls]
    total = sum(count) + 3
    ids = torch.randperm(total, generator=gen, device=DEV)[: sum(count)].tolist()
    width, rows, at = max(count), [], 0
    for n in count:
        rows.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    cu = [0]
    for n, _ in ls:
        cu.append(cu[-1] + n)
    st = dict(case=case, cache=filled_cache(total, hkv, gen, shape), table=int32(rows), cu=int32(cu))
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "attend":
        q = torch.randn(cu[-1], case["hq"], D, generator=gen, device=DEV).to(dtype)
        st.update(q=q, ctx=int32([c for _, c in ls]), max_q=max(n for n, _ in ls), max_ctx=max(c for _, c in ls))
    else:
        k, v = keys_values(cu[-1], hkv, gen, shape)
        st.update(k=k.to(dtype), v=v.to(dtype), before=int32([c - n for n, c in ls]))
    return st


# ------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------
def encode(x, tensor_scale):
    """NVFP4 along the last axis in single FP32 steps: codes (one per byte) and E4M3 scale codes."""
    x = x.float()
    b = x.unflatten(-1, (D // 16, 16))
    s = (b.abs().amax(-1) / 6.0 / tensor_scale).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = s.float() * tensor_scale
    y = b / den.unsqueeze(-1)
    a = y.abs()
    # nearest, ties to the even code, saturating
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
    code += (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte()
    code += torch.signbit(b).byte() * 8
    code = torch.where(den.unsqueeze(-1) == 0, torch.zeros_like(code), code)
    return code.flatten(-2), s.view(torch.uint8)


def e2m1_values():
    half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(half + [-h for h in half], device=DEV)


def decoded(cache, pages):
    """K and V of `pages` [S, n] in FP32 without the tensor scales: [S, heads, n * 64, D] each."""
    S, n = pages.shape
    value = e2m1_values()
    kc = cache["k_pages"][pages]
    k = value[torch.stack((kc & 15, kc >> 4), -1).int()].flatten(-2).unflatten(-1, (D // 16, 16))
    k = k * cache["k_scales"][pages].view(torch.float8_e4m3fn).float().unsqueeze(-1)
    vc = cache["v_pages"][pages]
    v = value[torch.stack((vc & 15, vc >> 4), -2).int()].flatten(-3, -2).unflatten(-1, (D // 16, 16))
    v = v * cache["v_scales"][pages].view(torch.float8_e4m3fn).float().transpose(-1, -2).unsqueeze(-1)
    heads = kc.shape[2]
    return (t.flatten(-2).transpose(1, 2).reshape(S, heads, n * PAGE, D) for t in (k, v))


def plain_attend(st):
    q, cu, ctx, cache = st["q"], st["cu"].long(), st["ctx"].long(), st["cache"]
    S, n, hq, hkv = len(ctx), st["max_q"], st["case"]["hq"], st["case"]["hkv"]
    g = hq // hkv
    k, v = decoded(cache, st["table"].long().clamp(min=0))
    row = torch.arange(len(q), device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pad = torch.zeros(S, n, hq, D, device=DEV)
    pad[seq, row - cu[seq]] = q.float()
    pad = pad.view(S, n, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(S, hkv, n * g, D)
    s = (pad @ k.transpose(-1, -2)).view(S, hkv, n, g, -1)
    del k
    s *= cache["k_tensor_scale"] / math.sqrt(D)
    last = (ctx - (cu[1:] - cu[:-1])).unsqueeze(1) + torch.arange(n, device=DEV)      # last key a token sees
    hidden = torch.arange(s.shape[-1], device=DEV) > last.unsqueeze(-1)
    s.masked_fill_(hidden.view(S, 1, n, 1, -1), -math.inf)
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    o = (s.view(S, hkv, n * g, -1) @ v) / s.sum(-1).view(S, hkv, n * g, 1) * cache["v_tensor_scale"]
    o = o.view(S, hkv, n, g, D).permute(0, 2, 1, 3, 4).reshape(S, n, hq, D)
    return o[seq, row - cu[seq]].to(q.dtype)


def plain_store(st):
    k, v, cu, cache = st["k"], st["v"], st["cu"].long(), st["cache"]
    row = torch.arange(len(k), device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = st["before"].long()[seq] + row - cu[seq]
    page, slot = st["table"].long()[seq, pos // PAGE], pos % PAGE
    kc, kx = encode(k, cache["k_tensor_scale"])
    vc, vx = encode(v, cache["v_tensor_scale"])
    cache["k_pages"][page, :, slot] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    cache["k_scales"][page, :, slot] = kx
    cache["v_scales"][page, :, :, slot] = vx
    even, odd = slot % 2 == 0, slot % 2 == 1
    pe, he, po, ho = page[even], slot[even] // 2, page[odd], slot[odd] // 2
    cache["v_pages"][pe, :, he] = (cache["v_pages"][pe, :, he] & 0xF0) | vc[even]
    cache["v_pages"][po, :, ho] = (cache["v_pages"][po, :, ho] & 0x0F) | (vc[odd] << 4)
    # read back
    value = e2m1_values()
    kb = cache["k_pages"][page, :, slot]
    k4 = value[torch.stack((kb & 15, kb >> 4), -1).int()].flatten(-2).unflatten(-1, (D // 16, 16))
    k4 = k4 * cache["k_scales"][page, :, slot].view(torch.float8_e4m3fn).float().unsqueeze(-1) * cache["k_tensor_scale"]
    vb = cache["v_pages"][page, :, slot // 2]
    v4 = value[torch.where(odd.view(-1, 1, 1), vb >> 4, vb & 15).int()].unflatten(-1, (D // 16, 16))
    v4 = v4 * cache["v_scales"][page, :, :, slot].view(torch.float8_e4m3fn).float().unsqueeze(-1) * cache["v_tensor_scale"]
    return dict(k=k4.flatten(-2).to(k.dtype), v=v4.flatten(-2).to(v.dtype))


def plain_fork(st):
    refs, table, lens, src, dst = st["refs"], st["table"], st["lens"], st["src"].long(), st["dst"].long()
    slot = torch.arange(table.shape[1], device=DEV)

    def held(rows):                                    # which entries of these rows hold a page
        return slot < ((lens[rows] + PAGE - 1) // PAGE).unsqueeze(1)

    # the places of the new sequences are emptied
    had = held(dst)
    refs.index_put_((table[dst].clamp(min=0).long(),), -had.int(), accumulate=True)
    table[dst] = torch.where(had, torch.full_like(table[dst], -1), table[dst])
    lens[dst] = 0
    # whole pages are shared; a page that is not full gets the lowest free page as its copy
    n = lens[src]
    part = n % PAGE != 0
    free = torch.argsort((refs != 0).byte(), stable=True)[: len(src)].int()
    fresh = torch.where(part, free[(part.cumsum(0) - 1).clamp(min=0)], torch.full_like(free, -1))
    whole = slot < (n // PAGE).unsqueeze(1)
    tail = part.unsqueeze(1) & (slot == (n // PAGE).unsqueeze(1))
    from_ = torch.where(part, table[src, (n // PAGE).long().clamp(max=table.shape[1] - 1)], torch.full_like(fresh, -1))
    refs.index_put_((table[src].clamp(min=0).long(),), whole.int(), accumulate=True)
    refs.index_put_((fresh.clamp(min=0).long(),), part.int(), accumulate=True)
    row = torch.where(whole, table[src], table[dst])
    table[dst] = torch.where(tail, fresh.unsqueeze(1), row)
    lens[dst] = n
    return from_, fresh


def plain_compact(st):
    refs, table, lens = st["refs"], st["table"], st["lens"]
    live = refs != 0
    n = live.sum()
    page = torch.arange(len(refs), device=DEV)
    move, hole = live & (page >= n), ~live & (page < n)
    # the i-th live page behind the first n goes to the i-th hole among them
    holes = torch.argsort((~hole).byte(), stable=True)
    to = torch.where(move, holes[(move.cumsum(0) - 1).clamp(min=0)], page)
    held = torch.arange(table.shape[1], device=DEV) < ((lens + PAGE - 1) // PAGE).unsqueeze(1)
    table.copy_(torch.where(held, to[table.clamp(min=0).long()].int(), table))
    new = torch.zeros_like(refs)
    new[to[live]] = refs[live]
    refs.copy_(new)
    return page[move], to[move]


def plain_copy(cache, src, dst):
    real = src >= 0
    src, dst = src[real].long(), dst[real].long()
    for name in ("k_pages", "k_scales", "v_pages", "v_scales"):
        cache[name][dst] = cache[name][src]


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(st):
    op, c = st["case"]["op"], st["cache"]
    if op == "compact":                                # a cache as its sequences left it
        st["refs"].copy_(st["refs0"])
        st["table"].copy_(st["table0"])
    if own:
        from bit_block_scaled_nvfp4_b200 import api, paged

        if "handle" not in st:                         # what a program makes once for its cache
            st["handle"] = api.PagedKV4(**c)
            if op == "attend":
                st["plan"] = api.KV4AttentionPlan(st["handle"], st["table"], st["ctx"], st["max_ctx"], st["case"]["hq"],
                                                  max_q=st["max_q"], max_tokens=len(st["q"]), dtype=st["q"].dtype)
            elif op != "store":
                st["pool"] = paged.PagePool(st["refs"])
        cache = st["handle"]
        if op == "attend":
            return st["plan"].run(st["q"], st["cu"])
        if op == "store":
            api.kv4_append_paged(cache, st["k"], st["v"], st["cu"], st["before"], st["table"])
            k, v = api.kv4_read_paged(cache, st["cu"], st["before"], st["table"], len(st["k"]), dtype=st["k"].dtype)
            return dict(k=k, v=v)
        if op == "fork":
            api.kv_pages_free(st["pool"], st["table"], st["lens"], st["dst"])
            moves = api.kv_pages_fork(st["pool"], st["table"], st["lens"], st["src"], st["dst"])
        else:
            moves = api.kv_pages_compact(st["pool"], st["table"], st["lens"])
        api.kv_pages_copy(cache, moves)
    elif op == "attend":
        return plain_attend(st)
    elif op == "store":
        return plain_store(st)
    else:
        plain_copy(c, *(plain_fork(st) if op == "fork" else plain_compact(st)))
    return dict(refs=st["refs"], table=st["table"], lens=st["lens"],
                pages=[c["k_pages"], c["k_scales"], c["v_pages"], c["v_scales"]])


# ------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------
def float_of(code, exponent, mantissa, bias):
    """The value of a small float's bits: sign, `exponent` bits, `mantissa` bits."""
    code = code.to(torch.int64)
    m = (code & ((1 << mantissa) - 1)).double()
    e = (code >> mantissa) & ((1 << exponent) - 1)
    sign = 1.0 - 2.0 * (code >> (exponent + mantissa)).double()
    one = 2.0 ** mantissa
    return sign * torch.where(e == 0, m / one * 2.0 ** (1 - bias), (1 + m / one) * torch.exp2((e - bias).double()))


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None
    st = prepare(case, seed)
    cache, ls = st["cache"], lengths(case)
    if op == "store":
        got = {}
        for name, tensor_scale in (("k", K_SCALE), ("v", V_SCALE)):
            x = st[name].double().unflatten(-1, (D // 16, 16))
            top = x.abs().amax(-1) / 6 / tensor_scale
            # E4M3 to nearest even: a step of 2^(e - 3), e at least -6, at most 448
            step = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -6))) - 3)
            s = (torch.round(top / step) * step).clamp(max=448.0).unsqueeze(-1) * tensor_scale
            y = torch.where(s == 0, torch.zeros_like(x), x / torch.where(s == 0, torch.ones_like(s), s))
            a = y.abs().clamp(max=6.0)
            step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
            got[name] = (torch.round(a / step) * step * torch.sign(y) * s).flatten(-2)
        return got
    out, at = torch.empty(len(st["q"]), case["hq"], D, dtype=torch.float64, device=DEV), 0
    g = case["hq"] // case["hkv"]
    for s, (n, ctx) in enumerate(ls):
        pages = st["table"][s, : pages_of(ctx)].long()
        q = st["q"][at:at + n].double()
        for h in range(case["hkv"]):
            kb = cache["k_pages"][pages, h].flatten(0, 1)[:ctx]
            k = float_of(torch.stack((kb & 15, kb >> 4), -1).flatten(1), 2, 1, 1).view(ctx, D // 16, 16)
            k = k * float_of(cache["k_scales"][pages, h].flatten(0, 1)[:ctx], 4, 3, 7).unsqueeze(-1) * K_SCALE
            vb = cache["v_pages"][pages, h].flatten(0, 1)
            v = float_of(torch.stack((vb & 15, vb >> 4), 1).flatten(0, 1)[:ctx], 2, 1, 1).view(ctx, D // 16, 16)
            v = v * float_of(cache["v_scales"][pages, h].transpose(1, 2).flatten(0, 1)[:ctx], 4, 3, 7).unsqueeze(-1) * V_SCALE
            seen = torch.arange(ctx, device=DEV) <= torch.arange(ctx - n, ctx, device=DEV).unsqueeze(1)
            for i in range(h * g, (h + 1) * g):
                w = (q[:, i] @ k.view(ctx, D).T) / math.sqrt(D)
                w = torch.softmax(w.masked_fill(~seen, -math.inf), -1)
                out[at:at + n, i] = w @ v.view(ctx, D)
        at += n
    return out
