"""The 4-bit cache, the attention that reads it and the pages that hold it, as measured work.

Each case is one call sequence of a serving loop:

  write    encode new K and V vectors into 4-bit caches and read them back
  attend   one decode step's attention over 4-bit caches (one query a sequence)
  step     append a few (or a chunk of) tokens to 4-bit caches and attend with as many queries, causally
  fork     a beam step on the pages: losing beams take their parents' pages, then every beam's next
           token is made writable (copy on write of the shared tail pages)
  compact  defragment the pools: live pages move into the lowest places, the table follows

``own`` false: the plain form, elementary torch operations in fp32 on the same packed bytes.
``own`` true: the framework's calls.

The 4-bit format: groups of ``group`` consecutive values of a vector share an fp16 scale and an fp16
zero (the group's minimum); a value stands for zero + scale * code.  A cache block holds 64 tokens:
64 x d/2 bytes of codes, then 64 x d/group (scale, zero) pairs.  Byte j of token tau's codes (values
2j in the low and 2j + 1 in the high nibble) is stored at j ^ 16 s(tau), with s(tau) = (tau & 2 where
d >= 128) + ((tau & 1) << 2 where d = 256).
"""
import math

import torch

own = False

BLOCK = 64
FIFTEENTH = 0.06666667014360428          # 1/15 in fp32, a constant of the format
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a long prompt's keys and values of one layer, as prefill hands them over
        dict(name="write_b1_hkv8_t32768_d128_bf16", kind="write", B=1, Hkv=8, T=32768, d=128, group=64, dtype="bf16",
             token_major=False, ragged=False, paged=False),
        # a batch of prompts appended behind different prefixes, token-major projections, odd length
        dict(name="write_b6_hkv4_t777_d64_f16", kind="write", B=6, Hkv=4, T=777, d=64, group=32, dtype="f16",
             token_major=True, ragged=True, paged=True),
        # one user, short context: latency of a single call
        dict(name="attend_b1_hq32_hkv8_t1000_d128", kind="attend", B=1, Hq=32, Hkv=8, T=1000, d=128, group=64,
             dtype="bf16", ragged=False, paged=False),
        # long context, four users
        dict(name="attend_b4_hq16_hkv8_t102400_d128", kind="attend", B=4, Hq=16, Hkv=8, T=102400, d=128, group=64,
             dtype="bf16", ragged=False, paged=False),
        # a serving batch: lengths all different, pages anywhere in the pool
        dict(name="attend_b64_hq32_hkv8_ragged8198_d128", kind="attend", B=64, Hq=32, Hkv=8, T=8198, d=128, group=128,
             dtype="f16", ragged=True, paged=True),
        # fp32 queries, seven query heads a kv head, odd length, small groups
        dict(name="attend_b3_hq21_hkv3_t4133_d64_f32", kind="attend", B=3, Hq=21, Hkv=3, T=4133, d=64, group=32,
             dtype="f32", ragged=False, paged=False),
        # chunked prefill: 512 new tokens after 40448
        dict(name="step_b1_hq32_hkv8_l512_t40448_d128", kind="step", B=1, Hq=32, Hkv=8, L=512, T=40448, d=128,
             group=64, dtype="bf16", ragged=False, paged=False),
        # speculative decoding: five drafted tokens of sixteen sequences checked at once
        dict(name="step_b16_hq32_hkv8_l5_t4000_d128", kind="step", B=16, Hq=32, Hkv=8, L=5, T=4000, d=128, group=64,
             dtype="bf16", ragged=True, paged=True),
        # beam search over two prompts: latency of the page bookkeeping
        dict(name="fork_b8_hkv2_t900", kind="fork", B=8, beams=4, Hkv=2, T=900, d=128, group=64, spare=256),
        # beam search over a batch of long prompts
        dict(name="fork_b64_hkv8_t8198", kind="fork", B=64, beams=4, Hkv=8, T=8198, d=128, group=64, spare=4096),
        # a pool that served many requests, a third of it live
        dict(name="compact_p49152_live33", kind="compact", B=32, Hkv=8, pool=49152, live=0.33, d=128, group=64),
        # a small pool, mostly live
        dict(name="compact_p1000_live90", kind="compact", B=5, Hkv=2, pool=1000, live=0.9, d=64, group=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["write", "attend", "attend", "step", "step", "fork", "compact"])
    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
    if kind == "write":
        B = _log(rng, 1, 16)
        T = max(1, min(_log(rng, 1, 32768), (16 << 20) // (B * Hkv * d)))
        return dict(kind=kind, B=B, Hkv=Hkv, T=T, d=d, group=group, dtype=dtype, token_major=rng.random() < 0.5,
                    ragged=rng.random() < 0.5, paged=rng.random() < 0.5)
    if kind == "attend":
        B = _log(rng, 1, 64)
        T = max(1, min(_log(rng, 1, 102400), (200 << 20) // (B * Hkv * d), (1 << 27) // (B * Hkv * G)))
        return dict(kind=kind, B=B, Hq=Hkv * G, Hkv=Hkv, T=T, d=d, group=group, dtype=dtype,
                    ragged=rng.random() < 0.6, paged=rng.random() < 0.6)
    if kind == "step":
        B = _log(rng, 1, 16)
        L = _log(rng, 1, 512)
        rows = B * Hkv * G * L
        T = max(1, min(_log(rng, 1, 40448), (64 << 20) // (B * Hkv * d), (1 << 29) // rows))
        return dict(kind=kind, B=B, Hq=Hkv * G, Hkv=Hkv, L=L, T=T, d=d, group=group, dtype=dtype,
                    ragged=rng.random() < 0.5, paged=rng.random() < 0.5)
    if kind == "fork":
        beams = rng.choice([2, 4, 6, 8])
        T = _log(rng, 70, 8198)
        return dict(kind=kind, B=beams * _log(rng, 1, 12), beams=beams, Hkv=Hkv, T=T + (T % 64 == 0), d=d, group=group,
                    spare=rng.choice([1024, 3000, 4096]))
    return dict(kind=kind, B=_log(rng, 1, 32), Hkv=Hkv, pool=_log(rng, 500, 24576), live=round(rng.uniform(0.1, 0.95), 2),
                d=d, group=group)


# ------------------------------------------------------------------ the packed format, in torch

def _block_bytes(d, group):
    return BLOCK * (d // 2 + 4 * (d // group))


def _swizzle(d, device):
    """[64, d/32]: place of 16-byte chunk c of token tau."""
    tau = torch.arange(BLOCK, device=device)
    s = (tau & 2 if d >= 128 else tau * 0) | ((tau & 1) << 2 if d == 256 else tau * 0)
    return torch.arange(d // 32, device=device)[None, :] ^ s[:, None]


def _quantise(x, group):
    """x [..., d] -> codes uint8 [..., d], scale and zero fp16 [..., d/group]."""
    g = x.float().clamp(-65504.0, 65504.0).unflatten(-1, (-1, group))
    zero = g.amin(-1).half()
    scale = ((g.amax(-1) - zero.float()) * FIFTEENTH).half()
    s = scale.float()
    r = torch.where(s > 0, 1.0 / s, 0.0)
    c = ((g - zero.float()[..., None]) * r[..., None]).round().clamp(0, 15)
    return c.to(torch.uint8).flatten(-2), scale, zero


def _code_bytes(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _pairs(scale, zero):
    return torch.stack([scale, zero], -1).flatten(-2).view(torch.uint8)


def _pack(x, group):
    """x [N, NB * 64, d] -> packed blocks [N, NB, block bytes]."""
    n, t, d = x.shape
    codes, scale, zero = _quantise(x, group)
    raw = _code_bytes(codes).view(n, t // BLOCK, BLOCK, d // 32, 16)
    tau = torch.arange(BLOCK, device=x.device)[:, None]
    raw = raw[:, :, tau, _swizzle(d, x.device)]           # an involution: stored chunk c holds chunk c ^ s
    return torch.cat([raw.reshape(n, t // BLOCK, -1), _pairs(scale, zero).reshape(n, t // BLOCK, -1)], -1)


def _unpack(blocks, d, group):
    """Packed blocks [..., NB, block bytes] -> fp32 values [..., NB * 64, d]."""
    lead = blocks.shape[:-1]
    raw = blocks[..., :BLOCK * d // 2].reshape(*lead, BLOCK, d // 32, 16)
    tau = torch.arange(BLOCK, device=blocks.device)[:, None]
    raw = raw[..., tau, _swizzle(d, blocks.device), :].reshape(*lead, BLOCK, d // 2)
    codes = torch.stack([raw & 15, raw >> 4], -1).reshape(*lead, BLOCK, d // group, group)
    pairs = blocks[..., BLOCK * d // 2:].contiguous().view(torch.float16).reshape(*lead, BLOCK, d // group, 2).float()
    x = codes.float() * pairs[..., :1] + pairs[..., 1:]
    return x.reshape(*lead[:-1], lead[-1] * BLOCK, d)


def _gather(s, name):
    """The blocks of every sequence in order: [B, Hkv, NB, block bytes]."""
    c = s["case"]
    pool = s[name].view(-1, _block_bytes(c["d"], c["group"]))
    b = pool[s["table"].long()] if s["table"] is not None else pool
    return b.view(c["B"], c["Hkv"], -1, b.shape[-1])


def _at(s, n):
    """(block, token in block) of the n tokens from s["pos"] on: [B, Hkv, n] each."""
    c = s["case"]
    t = s["pos"].long()[:, None] + torch.arange(n, device=s["pos"].device)
    nb = s["NB"]
    row = torch.arange(c["B"] * c["Hkv"], device=t.device).view(c["B"], c["Hkv"], 1)
    at = row * nb + (t // BLOCK)[:, None, :]
    block = s["table"].view(-1)[at].long() if s["table"] is not None else at
    return block, (t % BLOCK)[:, None, :].expand_as(block)


def _places(s, n):
    """Byte offsets of the codes [B, Hkv, n, d/2] and of the pairs [B, Hkv, n, 4 d/group]."""
    c = s["case"]
    d, group = c["d"], c["group"]
    block, tau = _at(s, n)
    base = block[..., None] * _block_bytes(d, group)
    chunk = _swizzle(d, block.device)[tau]                                       # [B, Hkv, n, d/32]
    byte = (chunk[..., None] * 16 + torch.arange(16, device=block.device)).flatten(-2)
    pair = BLOCK * (d // 2) + tau[..., None] * (4 * (d // group)) + torch.arange(4 * (d // group), device=block.device)
    return base + tau[..., None] * (d // 2) + byte, base + pair


def _append(s, name, x):
    codes, scale, zero = _quantise(x, s["case"]["group"])
    at_codes, at_pairs = _places(s, x.shape[2])
    s[name][at_codes] = _code_bytes(codes)
    s[name][at_pairs] = _pairs(scale.contiguous(), zero.contiguous()).view(at_pairs.shape)


def _read(s, name, n, dtype):
    c = s["case"]
    at_codes, at_pairs = _places(s, n)
    raw = s[name][at_codes]
    pairs = s[name][at_pairs].view(torch.float16).unflatten(-1, (-1, 2)).float()
    codes = torch.stack([raw & 15, raw >> 4], -1).flatten(-2).unflatten(-1, (-1, c["group"])).float()
    return (codes * pairs[..., :1] + pairs[..., 1:]).flatten(-2).to(dtype)


# ------------------------------------------------------------------ inputs

def _values(gen, shape, keys):
    """Gaussian values; keys have per-channel offsets and a few strong channels, as projections with rotary
    embeddings give them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if keys:
        d = shape[-1]
        x *= torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
        x += 2.0 * torch.randn(d, generator=gen, device="cuda") * (torch.rand(d, generator=gen, device="cuda") < 0.1)
    else:
        x *= 0.3
    return x


def _blocks(t):
    return (t + BLOCK - 1) // BLOCK


def _cache_state(case, seed, tokens):
    """State shared by the cache cases; `tokens`: the most tokens of a sequence."""
    B, Hkv = case["B"], case["Hkv"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    NB = _blocks(tokens)
    s = dict(case=case, NB=NB, table=None, pool=0)
    if case["paged"]:
        s["pool"] = B * Hkv * NB + 7
        s["table"] = torch.randperm(s["pool"], generator=gen, device="cuda")[:B * Hkv * NB].to(torch.int32).view(B * Hkv, NB)
    return s, gen


def _lengths(case, gen):
    B, T = case["B"], case["T"]
    n = torch.full((B,), T, dtype=torch.int32, device="cuda")
    if case["ragged"]:
        n = (T * (0.25 + 0.75 * torch.rand(B, generator=gen, device="cuda"))).to(torch.int32).clamp(1, T)
        n[0] = T
    return n


def _fill(s, gen, name, keys):
    """Cache `name` full of encoded vectors, one sequence at a time."""
    c = s["case"]
    bb = _block_bytes(c["d"], c["group"])
    blocks = torch.empty((c["B"], c["Hkv"], s["NB"], bb), dtype=torch.uint8, device="cuda")
    for b in range(c["B"]):
        blocks[b] = _pack(_values(gen, (c["Hkv"], s["NB"] * BLOCK, c["d"]), keys), c["group"])
    if s["table"] is None:
        s[name] = blocks.view(-1)
    else:
        pool = torch.zeros((s["pool"], bb), dtype=torch.uint8, device="cuda")
        pool[s["table"].view(-1).long()] = blocks.view(-1, bb)
        s[name] = pool.view(-1)


def _handles(s):
    """What a program keeps: the handle, the cache descriptors, outputs and workspace."""
    from kv_cache_vector_14_b200 import tq
    c = s["case"]
    s["tq"] = tq
    s["h"] = tq.tq_init(c["d"], 0)
    for name in ("k", "v"):
        s[name + "c"] = tq.Int4Cache(c["d"], c["group"], c["B"], c["Hkv"], s["NB"] * BLOCK, buf=s[name],
                                     block_table=s["table"], pool_blocks=s["pool"])
    if "q" in s:
        L = s["q"].shape[1]
        s["out"] = torch.empty_like(s["q"])
        s["ws"] = torch.empty(tq.tq_attend_int4_workspace_bytes(s["h"], c["B"], L, c["Hq"], c["Hkv"]),
                              dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    kind, d = case["kind"], case["d"]
    if kind in ("fork", "compact"):
        s = _fork_state(case, seed) if kind == "fork" else _compact_state(case, seed)
        if own:
            from kv_cache_vector_14_b200 import tq
            s["tq"], s["h"] = tq, tq.tq_init(d, 0)
            bb = _block_bytes(d, case["group"])
            s["pages"] = tq.Pages(s["table"], s["refs"], case["Hkv"], [(s["k"], bb), (s["v"], bb)])
            s["ws"] = torch.empty(tq.tq_pages_workspace_bytes(s["pages"]), dtype=torch.uint8, device="cuda")
        return s
    B, Hkv, dtype = case["B"], case["Hkv"], TYPES[case["dtype"]]
    if kind == "write":
        s, gen = _cache_state(case, seed, case["T"] + 100)
        s["pos"] = torch.randint(0, 100, (B,), generator=gen, device="cuda", dtype=torch.int32) * int(case["ragged"])
        size = (s["pool"] or B * Hkv * s["NB"]) * _block_bytes(d, case["group"])
        for name in ("k", "v"):
            s[name] = torch.zeros(size, dtype=torch.uint8, device="cuda")
            if case["token_major"]:
                s[name + "_new"] = _values(gen, (B, case["T"], Hkv, d), name == "k").to(dtype).transpose(1, 2)
            else:
                s[name + "_new"] = _values(gen, (B, Hkv, case["T"], d), name == "k").to(dtype)
            s[name + "_out"] = torch.empty((B, Hkv, case["T"], d), dtype=dtype, device="cuda")
    elif kind == "attend":
        s, gen = _cache_state(case, seed, case["T"])
        s["lens"] = _lengths(case, gen)
        _fill(s, gen, "k", True)
        _fill(s, gen, "v", False)
        s["q"] = torch.randn((B, 1, case["Hq"], d), generator=gen, device="cuda").to(dtype)
    else:
        L = case["L"]
        s, gen = _cache_state(case, seed, case["T"] + L)
        s["pos"] = _lengths(case, gen)
        _fill(s, gen, "k", True)
        _fill(s, gen, "v", False)
        s["q"] = torch.randn((B, L, case["Hq"], d), generator=gen, device="cuda").to(dtype)
        for name in ("k", "v"):
            s[name + "_new"] = _values(gen, (B, L, Hkv, d), name == "k").to(dtype).transpose(1, 2)
            s[name + "_out"] = torch.empty((B, Hkv, L, d), dtype=dtype, device="cuda")
    s["scale"] = d ** -0.5
    if own:
        _handles(s)
    return s


def _fork_state(case, seed):
    """Groups of beams that share their prompt's pages and hold one generated page run each."""
    B, W, Hkv, T = case["B"], case["beams"], case["Hkv"], case["T"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nb, NB = _blocks(T), _blocks(T + 1) + 1
    shared = max(0, nb - 2)                              # prompt pages; the last two are each beam's own
    groups = B // W
    live = groups * Hkv * shared + B * Hkv * (nb - shared)
    pool = live + B * Hkv + case["spare"]
    place = torch.randperm(pool, generator=gen, device="cuda")[:live].to(torch.int32)
    table = torch.full((B, Hkv, NB), -1, dtype=torch.int32, device="cuda")
    prompt = place[:groups * Hkv * shared].view(groups, 1, Hkv, shared)
    table[:, :, :shared] = prompt.expand(groups, W, Hkv, shared).reshape(B, Hkv, shared)
    table[:, :, shared:nb] = place[groups * Hkv * shared:].view(B, Hkv, nb - shared)
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    used = table[table >= 0].long()
    refs.index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
    # half of each group's beams survive; every survivor has one more child among the losing places
    order = torch.rand((groups, W), generator=gen, device="cuda").argsort(-1)
    keep, lose = order[:, :W // 2], order[:, W // 2:]
    parent = torch.arange(W, device="cuda").expand(groups, W).clone()
    parent.scatter_(1, lose, keep)
    parent = (parent + torch.arange(groups, device="cuda")[:, None] * W).view(-1).to(torch.int32)
    bb = _block_bytes(case["d"], case["group"])
    return dict(case=case, NB=NB, pool=pool, table=table.view(B * Hkv, NB), refs=refs, parent=parent,
                lo=torch.full((B,), T, dtype=torch.int32, device="cuda"),
                hi=torch.full((B,), T + 1, dtype=torch.int32, device="cuda"),
                info=torch.zeros(2, dtype=torch.int32, device="cuda"),
                k=torch.randint(0, 256, (pool * bb,), generator=gen, device="cuda", dtype=torch.uint8),
                v=torch.randint(0, 256, (pool * bb,), generator=gen, device="cuda", dtype=torch.uint8))


def _compact_state(case, seed):
    """A pool in which the share `live` of the pages, at random places, belongs to the table's rows."""
    B, Hkv, pool = case["B"], case["Hkv"], case["pool"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = B * Hkv
    live = max(1, int(pool * case["live"]))
    NB = -(-live // rows) + 2
    table = torch.full((rows * NB,), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(live, device="cuda")
    place = torch.randperm(pool, generator=gen, device="cuda")[:live].to(torch.int32)
    table[(at % rows) * NB + at // rows] = place
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    refs[place.long()] = 1
    bb = _block_bytes(case["d"], case["group"])
    return dict(case=case, NB=NB, pool=pool, table=table.view(rows, NB), refs=refs, table0=table.clone().view(rows, NB),
                refs0=refs.clone(), info=torch.zeros(2, dtype=torch.int32, device="cuda"),
                k=torch.randint(0, 256, (pool * bb,), generator=gen, device="cuda", dtype=torch.uint8),
                v=torch.randint(0, 256, (pool * bb,), generator=gen, device="cuda", dtype=torch.uint8))


# ------------------------------------------------------------------ one pass

def run(s):
    kind = s["case"]["kind"]
    if kind == "write":
        return _write(s)
    if kind == "attend":
        return _attend_case(s)
    if kind == "step":
        return _step(s)
    return _fork(s) if kind == "fork" else _compact(s)


def _write(s):
    if own:
        tq, h, pos = s["tq"], s["h"], s["pos"]
        tq.tq_encode_int4(h, s["k_new"], s["kc"], pos=pos)
        tq.tq_encode_int4(h, s["v_new"], s["vc"], pos=pos)
        tq.tq_expand_int4(h, s["kc"], s["k_out"], pos=pos)
        tq.tq_expand_int4(h, s["vc"], s["v_out"], pos=pos)
        return s["k_out"], s["v_out"]
    _append(s, "k", s["k_new"])
    _append(s, "v", s["v_new"])
    n, dtype = s["case"]["T"], s["k_new"].dtype
    return _read(s, "k", n, dtype), _read(s, "v", n, dtype)


def _attention(s, lens):
    """Plain attention over the packed caches; lens [B]: tokens of each sequence, the queries' own included."""
    c, q = s["case"], s["q"]
    B, L, Hq, d = q.shape
    Hkv = c["Hkv"]
    k = _unpack(_gather(s, "k"), d, c["group"])
    x = q.float().view(B, L, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)   # rows (head, query)
    a = (x @ k.transpose(-1, -2)) * s["scale"]
    del k
    last = lens.long()[:, None] - L + 1 + torch.arange(L, device=q.device)                       # [B, L]
    seen = torch.arange(a.shape[-1], device=q.device) < last.repeat(1, Hq // Hkv)[..., None]     # [B, rows, T]
    a.masked_fill_(~seen[:, None], float("-inf"))
    m = a.amax(-1, keepdim=True).clamp_min(-3e38)
    a = a.sub_(m).exp_()
    total = a.sum(-1, keepdim=True)
    out = (a @ _unpack(_gather(s, "v"), d, c["group"])) / total.clamp_min(1e-30)
    return out.view(B, Hkv, Hq // Hkv, L, d).permute(0, 3, 1, 2, 4).reshape(B, L, Hq, d).to(q.dtype)


def _attend_case(s):
    if own:
        s["tq"].tq_attend_int4(s["h"], s["q"], s["kc"], s["vc"], s["out"], s["ws"], seq_lens=s["lens"], scale=s["scale"])
        return s["out"]
    return _attention(s, s["lens"])


def _step(s):
    if own:
        tq, h, pos = s["tq"], s["h"], s["pos"]
        tq.tq_append_attend_int4(h, s["k_new"], s["v_new"], s["kc"], s["vc"], s["q"], s["out"], s["ws"], pos=pos,
                                 scale=s["scale"])
        tq.tq_expand_int4(h, s["kc"], s["k_out"], pos=pos)
        tq.tq_expand_int4(h, s["vc"], s["v_out"], pos=pos)
        return s["out"], s["k_out"], s["v_out"]
    L = s["case"]["L"]
    _append(s, "k", s["k_new"])
    _append(s, "v", s["v_new"])
    out = _attention(s, s["pos"] + L)
    return out, _read(s, "k", L, s["k_new"].dtype), _read(s, "v", L, s["k_new"].dtype)


def _count(refs, entries, by):
    """refs[e] += by for every entry e >= 0."""
    e = entries.reshape(-1).long()
    refs.index_add_(0, e.clamp_min(0), torch.where(e >= 0, by, 0).to(torch.int32))


def _fork(s):
    if own:
        tq, h = s["tq"], s["h"]
        tq.tq_pages_fork(h, s["pages"], s["parent"])
        tq.tq_pages_alloc(h, s["pages"], s["lo"], s["hi"], s["info"], s["ws"])
        return s["table"], s["refs"], s["info"], s["k"], s["v"]
    c, refs, pool = s["case"], s["refs"], s["pool"]
    B, Hkv, NB = c["B"], c["Hkv"], s["NB"]
    table = s["table"].view(B, Hkv, NB)
    old = table.clone()
    table.copy_(old[s["parent"].long()])
    _count(refs, old, -1)
    _count(refs, table, 1)
    # every block of [lo, hi) that is missing or shared gets a fresh page, lowest first
    lb = torch.arange(NB, device=refs.device)
    lo, hi = s["lo"].long()[:, None, None], s["hi"].long()[:, None, None]
    need = (lb >= lo // BLOCK) & (lb * BLOCK < hi)
    entry = table.long()
    shared = (entry >= 0) & (refs[entry.clamp_min(0)] > 1)
    ask = (need & ((entry < 0) | shared)).view(-1)
    free = refs == 0
    place = torch.where(free, free.cumsum(0) - 1, pool)
    fresh = torch.full((pool + 1,), -1, dtype=torch.int64, device=refs.device)
    fresh[place] = torch.arange(pool, device=refs.device)
    fresh[pool] = -1
    have = free.sum()
    rank = ask.long().cumsum(0) - 1
    get = ask & (rank < have)
    new = torch.where(get, fresh[rank.clamp(0, pool - 1)], entry.view(-1))
    was = entry.view(-1)
    table.view(-1).copy_(new)
    _count(refs, torch.where(get, was, -1), -1)
    _count(refs, torch.where(get, new, -1), 1)
    s["info"][0] = (refs == 0).sum()
    s["info"][1] = (ask & ~get).sum()
    # the copies: the blocks that any row may ask for are the one or two that hold [lo, hi)
    first = (s["lo"].long() // BLOCK)[:, None, None].expand(B, Hkv, 1)
    at = torch.cat([first, (first + 1).clamp_max(NB - 1)], -1)
    src, dst = was.view(B, Hkv, NB).gather(-1, at).view(-1), new.view(B, Hkv, NB).gather(-1, at).view(-1)
    quiet = (~free).long().argmax()               # a page in use before: no fresh page, so nobody's destination
    src = torch.where(src >= 0, src, dst)
    dst = torch.where(dst >= 0, dst, quiet)       # nothing to copy: that page onto itself
    src = torch.where(src >= 0, src, quiet)
    bb = _block_bytes(c["d"], c["group"])
    for name in ("k", "v"):
        data = s[name].view(pool, bb)
        data[dst] = data[src]
    return s["table"], refs, s["info"], s["k"], s["v"]


def _compact(s):
    s["table"].copy_(s["table0"])                 # the scheduler's table of this moment
    s["refs"].copy_(s["refs0"])
    if own:
        s["tq"].tq_pages_compact(s["h"], s["pages"], s["info"], s["ws"])
        return s["table"], s["refs"], s["info"], s["k"], s["v"]
    c, refs, table, pool = s["case"], s["refs"], s["table"], s["pool"]
    live = refs > 0
    total = live.sum()
    at = torch.arange(pool, device=refs.device)
    to = torch.nonzero(~live & (at < total)).view(-1)
    frm = torch.nonzero(live & (at >= total)).view(-1).flip(0)
    bb = _block_bytes(c["d"], c["group"])
    for name in ("k", "v"):
        data = s[name].view(pool, bb)
        data[to] = data[frm]
    refs[to] = refs[frm]
    refs[frm] = 0
    moved = at.to(torch.int32)
    moved[frm] = to.to(torch.int32)
    e = table.long()
    table.copy_(torch.where(e >= 0, moved[e.clamp_min(0)], table))
    s["info"][0] = pool - total
    s["info"][1] = to.numel()
    return s["table"], refs, s["info"], s["k"], s["v"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    d, group = case["d"], case["group"]
    vec = d // 2 + 4 * (d // group)
    bb = _block_bytes(d, group)
    kind = case["kind"]
    if kind == "fork":
        nb, rows = _blocks(case["T"]), case["B"] * case["Hkv"]
        # half of the rows replaced (their entries and their parents' read, theirs written), every row's tail page
        # copied for K and V, one look at the reference counts
        pool = case["B"] // case["beams"] * case["Hkv"] * max(0, nb - 2) + 3 * rows + case["spare"]
        return dict(bytes=rows // 2 * nb * 12 + 2 * 2 * rows * bb + 4 * pool, flops=0)
    if kind == "compact":
        pool, live = case["pool"], case["live"]
        moves = pool * live * (1 - live)
        return dict(bytes=int(2 * 2 * moves * bb + 2 * 4 * pool * live + 4 * pool + 8 * moves), flops=0)
    item = torch.finfo(TYPES[case["dtype"]]).bits // 8
    B, Hkv, T = case["B"], case["Hkv"], case["T"]
    if kind == "write":
        n = 2 * B * Hkv * T
        return dict(bytes=n * (2 * d * item + 2 * vec), flops=n * d * 6)
    mean = T * (0.625 if case["ragged"] else 1.0)
    Hq = case["Hq"]
    if kind == "attend":
        return dict(bytes=int(2 * B * Hkv * mean * vec + 2 * B * Hq * d * item), flops=int(4 * B * Hq * mean * d))
    L = case["L"]
    pairs = B * Hq * L * (mean + (L + 1) / 2)
    return dict(bytes=int(2 * B * Hkv * (mean + 2 * L) * vec + 2 * B * L * Hq * d * item + 4 * B * L * Hkv * d * item),
                flops=int(4 * pairs * d))


# ------------------------------------------------------------------ from the definition, in 64 bits

def _grid64(x, group):
    """What x [..., d] stands for after the 4-bit format, from its definition: every step that the format rounds to
    fp32 is computed in 64 bits and then rounded (products, sums and quotients of fp32 numbers round through
    fp64 as they do directly)."""
    def f32(v):
        return v.to(torch.float32).double()

    g = torch.minimum(torch.maximum(x.double(), torch.tensor(-65504.0, device=x.device, dtype=torch.float64)),
                      torch.tensor(65504.0, device=x.device, dtype=torch.float64))
    g = g.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    lowest = g.min(-1, keepdim=True).values.to(torch.float16).double()
    step = f32(f32(g.max(-1, keepdim=True).values - lowest) * FIFTEENTH).to(torch.float16).double()
    inverse = torch.where(step == 0, torch.zeros_like(step), f32(1.0 / step))
    code = torch.round(f32(f32(g - lowest) * inverse)).clamp(0.0, 15.0)
    return (lowest + step * code).reshape(x.shape)


def _stored64(s, name, b, h, n):
    """Tokens [0, n) of one sequence as the packed bytes have them, in 64 bits."""
    c = s["case"]
    d, group, bb = c["d"], c["group"], _block_bytes(c["d"], c["group"])
    row = b * c["Hkv"] + h
    ids = s["table"][row].long() if s["table"] is not None else row * s["NB"] + torch.arange(s["NB"], device="cuda")
    raw = s[name].view(-1, bb)[ids[:_blocks(n)]]
    t = torch.arange(BLOCK, device="cuda")
    turn = torch.zeros_like(t)
    if d >= 128:
        turn = turn + 2 * ((t // 2) % 2)
    if d == 256:
        turn = turn + 4 * (t % 2)
    j = torch.arange(d, device="cuda")
    byte = t[:, None] * (d // 2) + ((j // 2)[None, :] ^ (16 * turn[:, None]))
    code = (raw[:, byte.view(-1)].view(-1, BLOCK, d).to(torch.int64) >> (4 * (j % 2))) % 16
    half = raw[:, BLOCK * d // 2:].contiguous().view(torch.float16).double().view(-1, BLOCK, d // group, 2)
    x = half[..., 1].repeat_interleave(group, -1) + half[..., 0].repeat_interleave(group, -1) * code.double()
    return x.view(-1, d)[:n]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    kind = case["kind"]
    if kind in ("fork", "compact"):
        return None                                # whole numbers: the plain form says them
    if kind == "write":
        return _grid64(s["k_new"], case["group"]), _grid64(s["v_new"], case["group"])
    B, L, Hq, d = s["q"].shape
    Hkv, G = case["Hkv"], Hq // case["Hkv"]
    before = (s["pos"] if kind == "step" else s["lens"]).tolist()
    new = {n: _grid64(s[n + "_new"], case["group"]) for n in ("k", "v")} if kind == "step" else None
    out = torch.zeros((B, L, Hq, d), dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(Hkv):
            k, v = _stored64(s, "k", b, h, before[b]), _stored64(s, "v", b, h, before[b])
            if new is not None:
                k, v = torch.cat([k, new["k"][b, h]]), torch.cat([v, new["v"][b, h]])
            for g in range(G):
                x = s["q"][b, :, h * G + g].double()
                a = torch.einsum("ld,td->lt", x, k) * s["scale"]
                beyond = torch.arange(len(k), device="cuda")[None, :] > len(k) - L + torch.arange(L, device="cuda")[:, None]
                a = torch.softmax(a.masked_fill(beyond, -math.inf), -1)
                out[b, :, h * G + g] = torch.einsum("lt,td->ld", a, v)
    return (out, new["k"], new["v"]) if new is not None else out
