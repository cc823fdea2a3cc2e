"""Cases of the operators on a key/value cache held in 4 bits: what is timed, their
plain form in elementary torch operations, and their exact values in 64 bits.

  write   quantise new keys and values into the cache, then read the whole cache back
          (a chunk of a long prompt: append it, and have bf16 K, V for the forward)
  read    the cache as bf16 K, V, every query head with its own copy of a shared head
  attend  attention of a few query rows over the cache (one decoding step), O and LSE

The cache's format (one uint8 tensor [B, H_kv, ceil(m / 64), 34 (d_k + d_v)], a block of
64 slots each): K codes, K group words, V codes, V group words. A group is 64 channels
of one slot: lo = min(0, x), hi = max(0, x), step s = (hi - lo) / 15 rounded up to four
significant bits, zero u0 = rint(-lo / s), code u = clamp(rint(x / s) + u0, 0, 15),
value s (u - u0); its 16-bit word is s as bf16 with u0 in the four free low bits.
"""

import math

import torch

own = False

GROUP = 64
BLOCK = 64
LENGTH_MASKS = ("key_padding", "causal_key_padding", "causal_cache")
CAUSAL_MASKS = ("causal", "causal_key_padding", "causal_cache")


# ------------------------------------------------------------------------- cases

def listed():
    c = []

    def attend(name, B, H, H_kv, n, m, d_k, d_v, mask, lo, hi, slopes=False):
        c.append(dict(name=name, op="attend", B=B, H=H, H_kv=H_kv, n=n, m=m, d_k=d_k, d_v=d_v, mask=mask,
                      len_lo=lo, len_hi=hi, slopes=slopes))

    def write(name, B, H_kv, n, m, d_k, d_v, lo, hi, counts_lo):
        c.append(dict(name=name, op="write", B=B, H=H_kv, H_kv=H_kv, n=n, m=m, d_k=d_k, d_v=d_v,
                      len_lo=lo, len_hi=hi, counts_lo=counts_lo))

    def read(name, B, H, H_kv, m, d_k, d_v, lo, hi):
        c.append(dict(name=name, op="read", B=B, H=H, H_kv=H_kv, n=0, m=m, d_k=d_k, d_v=d_v, len_lo=lo, len_hi=hi))

    # the first tokens of a single sequence: all latency
    attend("attend_first_tokens", 1, 8, 8, 1, 64, 64, 64, "causal_cache", 33, 33)
    # one decoding step of a served batch (64 sequences x 16 heads, 4096 to 8192 filled slots)
    attend("attend_kv_cache", 64, 16, 16, 1, 8192, 128, 128, "key_padding", 4096, 8192)
    # the same step of a model whose 32 query heads share 8 cache heads
    attend("attend_shared_heads", 32, 32, 8, 1, 8192, 128, 128, "causal_cache", 512, 8192)
    # four draft tokens a sequence, checked at once
    attend("attend_draft_tokens", 64, 16, 16, 4, 8192, 128, 128, "causal_cache", 4096, 8192)
    # two long sequences: few heads, the work split over the slots
    attend("attend_long_context", 2, 16, 16, 1, 32768, 128, 128, "none", 32768, 32768)
    # odd sizes: 5 rows, 3 query heads to a cache head, wide values, distance bias, ragged lengths from 0 on
    attend("attend_odd", 7, 12, 4, 5, 1037, 64, 128, "causal_cache", 0, 1037, True)
    # a chunk of a prompt against what is there already: many rows
    attend("attend_prompt_chunk", 4, 16, 4, 256, 4096, 128, 128, "causal_cache", 1000, 4096)
    # one new token of a few short sequences
    write("write_token", 8, 8, 1, 256, 64, 64, 1, 255, 1)
    # a padded batch of prompts into an empty cache
    write("write_prompts", 16, 8, 1000, 2048, 128, 128, 0, 0, 1)
    # a chunk of long prompts, value heads of another width
    write("write_chunk", 4, 16, 2048, 8192, 64, 128, 2048, 6144, 2048)
    # a short cache of odd size
    read("read_odd", 5, 6, 3, 777, 64, 128, 0, 777)
    # long sequences, four query heads to a cache head
    read("read_long", 4, 16, 4, 8192, 128, 128, 4096, 8192)
    return c


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "write", "read"))
    d_k, d_v = rng.choice(((64, 64), (128, 128), (128, 128), (64, 128), (128, 64)))
    while True:
        B, H_kv = _log(rng, 1, 64), rng.choice((1, 2, 3, 4, 8, 16))
        m = _log(rng, 32, 32768)
        group = rng.choice((1, 1, 2, 3, 4, 8))
        if B * H_kv * m * (d_k + d_v) <= 64 * 16 * 4096 * 256 and B * H_kv * group * m <= 1 << 22:
            break
    lo = rng.randint(0, m)
    hi = rng.randint(lo, m)
    case = dict(op=op, B=B, H=H_kv * group, H_kv=H_kv, m=m, d_k=d_k, d_v=d_v, len_lo=lo, len_hi=hi)
    if op == "attend":
        case.update(n=rng.choice((1, 1, 1, 2, 3, 4, 5, 7, 8, 8, rng.randint(9, 40))),
                    mask=rng.choice(("none", "causal") + 2 * LENGTH_MASKS), slopes=rng.random() < 0.25)
    elif op == "write":
        n = _log(rng, 1, m)
        lo = rng.randint(0, m - n)
        case.update(n=n, H=H_kv, len_lo=lo, len_hi=rng.randint(lo, m - n), counts_lo=rng.randint(0, n))
    else:
        case.update(n=0)
    return case


def _spread(lo, hi, B, k):
    """B whole numbers spread evenly over [lo, hi], in an order of their own (k: which)."""
    v = [lo + (hi - lo) * i // max(1, B - 1) if B > 1 else hi for i in range(B)]
    step = next(s for s in range(k, k + B + 2) if math.gcd(s, B) == 1)
    return [v[(i * step + k) % B] for i in range(B)]


def _lengths(case):
    return _spread(case["len_lo"], case["len_hi"], case["B"], 3)


def _counts(case):
    return _spread(case["counts_lo"], case["n"], case["B"], 5)


# ----------------------------------------------------------------- the plain form

def _block_bytes(d_k, d_v):
    return 34 * (d_k + d_v)


def _quantise(x):
    """x [..., d] (d a multiple of 64): codes [..., d] and group words [..., d / 64], int32."""
    x = x.float().unflatten(-1, (-1, GROUP))
    bad = ~(x.abs().amax(-1) < 2.0 ** 127)
    x = torch.where(bad[..., None], torch.zeros_like(x), x)
    lo = x.amin(-1).clamp(max=0)
    hi = x.amax(-1).clamp(min=0)
    t = ((hi - lo) / torch.full_like(lo, 15.0)).contiguous().view(torch.int32)    # a scalar would become a product
    bits = (t + 0xFFFFF) & -0x100000
    s = bits.view(torch.float32)
    flat = s == 0
    div = torch.where(flat, torch.ones_like(s), s)
    u0 = torch.round(-lo / div)
    u = (torch.round(x / div[..., None]) + u0[..., None]).clamp(0, 15)
    word = torch.where(bad, torch.full_like(bits, 0x7FC0), ((bits >> 16) & 0xFFFF) | u0.int())
    return u.int().flatten(-2), word


def _k_order(d_k, dev):
    """For each slot of a block its row in the K codes."""
    k = torch.arange(BLOCK, device=dev)
    return k ^ (((k >> 2) & 1) * (128 // d_k))


def _pack_k(u):
    """Codes [..., 64, d_k] of a block's slots -> bytes [..., 32 d_k]."""
    d = u.shape[-1]
    ng = d // GROUP
    u = u.unflatten(-1, (ng, 4, 16)).transpose(-3, -2).flatten(-3)            # 8-byte units, group innermost
    u = u[..., _k_order(d, u.device), :]                                      # the order is its own inverse
    return (u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8).flatten(-2)


def _unpack_k(b, d):
    ng = d // GROUP
    b = b.unflatten(-1, (BLOCK, d // 2)).int()
    u = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    u = u[..., _k_order(d, u.device), :]
    return u.unflatten(-1, (4, ng, 16)).transpose(-3, -2).flatten(-3)


def _v_swap(d, dev):
    """Slots whose 8-byte units change halves (d_v = 128)."""
    return (((torch.arange(BLOCK, device=dev) >> 1) & 1) * (d == 128)).bool()[:, None]


def _pack_v(u):
    d = u.shape[-1]
    ng = d // GROUP
    u = u.unflatten(-1, (ng, 8, 8)).transpose(-3, -2).flatten(-3)
    u = torch.where(_v_swap(d, u.device), u.roll(d // 2, -1), u)
    return (u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8).flatten(-2)


def _unpack_v(b, d):
    ng = d // GROUP
    b = b.unflatten(-1, (BLOCK, d // 2)).int()
    u = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    u = torch.where(_v_swap(d, u.device), u.roll(d // 2, -1), u)
    return u.unflatten(-1, (8, ng, 8)).transpose(-3, -2).flatten(-3)


def _words_to_bytes(w):
    return torch.stack((w & 255, w >> 8), -1).to(torch.uint8).flatten(-3)


def _values(u, words):
    """Codes [..., 64, d], group words as bytes [..., 64 d / 32] -> values fp32 [..., 64, d]."""
    b = words.int().unflatten(-1, (BLOCK, -1, 2))
    w = b[..., 0] | (b[..., 1] << 8)
    s = ((w & 0xFFF0) << 16).contiguous().view(torch.float32)
    v = (u.unflatten(-1, (-1, GROUP)) - (w & 15)[..., None]).float() * s[..., None]
    return v.flatten(-2)


def _blocks(K, V):
    """bf16 K, V [..., 64 k, d] -> the bytes of their blocks [..., k, block bytes]."""
    out = []
    for x, pack in ((K, _pack_k), (V, _pack_v)):
        u, w = _quantise(x.unflatten(-2, (-1, BLOCK)))
        out += [pack(u), _words_to_bytes(w)]
    return torch.cat(out, -1)


def _read_blocks(cache, d_k, d_v):
    """The blocks' values, fp32 [..., slots, d_k] and [..., slots, d_v]."""
    ck, wk, cv, wv = cache.split((32 * d_k, 2 * d_k, 32 * d_v, 2 * d_v), -1)
    return (_values(_unpack_k(ck, d_k), wk).flatten(-3, -2), _values(_unpack_v(cv, d_v), wv).flatten(-3, -2))


def _entries(case):
    """How many batch entries the plain form takes at once."""
    a = case["H"] * case["m"] * (case["d_k"] + case["d_v"] + case["n"] + 1)
    return max(1, min(case["B"], (1 << 27) // a))


def _plain_read(case, cache, lens):
    B, H, H_kv, m, d_k, d_v = (case[k] for k in ("B", "H", "H_kv", "m", "d_k", "d_v"))
    K = torch.empty(B, H, m, d_k, dtype=torch.bfloat16, device=cache.device)
    V = torch.empty(B, H, m, d_v, dtype=torch.bfloat16, device=cache.device)
    e = _entries(case)
    for b in range(0, B, e):
        live = (torch.arange(m, device=cache.device) < lens[b:b + e, None])[:, None, :, None]
        for out, x in zip((K, V), _read_blocks(cache[b:b + e], d_k, d_v)):
            x = torch.where(live, x[:, :, :m], torch.zeros((), device=x.device))
            out[b:b + e] = x.repeat_interleave(H // H_kv, 1).to(torch.bfloat16)
    return K, V


def _plain_write(case, st):
    """Quantises the new rows and puts their bytes where the format has them."""
    B, H_kv, n, m, d_k, d_v = (case[k] for k in ("B", "H_kv", "n", "m", "d_k", "d_v"))
    cache, dev = st["cache"], st["cache"].device
    i = torch.arange(n, device=dev)
    slot = st["starts"][:, None] + i
    b, i = torch.nonzero((i < st["counts"][:, None]) & (slot >= 0) & (slot < m), as_tuple=True)
    slot = slot[b, i].long()
    blk, k = slot // BLOCK, slot % BLOCK
    at = torch.arange(H_kv, device=dev)[None, :, None]
    base = 0
    for x, d, is_k in ((st["K"], d_k, True), (st["V"], d_v, False)):
        u, w = _quantise(x[b, :, i])                                           # [tokens, H_kv, d]
        ng = d // GROUP
        if is_k:
            u = u.unflatten(-1, (ng, 4, 16)).transpose(-3, -2).flatten(-3)
            row = _k_order(d, dev)[k]
        else:
            u = u.unflatten(-1, (ng, 8, 8)).transpose(-3, -2).flatten(-3)
            u = torch.where(_v_swap(d, dev)[k][:, None], u.roll(d // 2, -1), u)
            row = k
        codes = (u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8)
        where = base + row[:, None] * (d // 2) + torch.arange(d // 2, device=dev)
        cache[b[:, None, None], at, blk[:, None, None], where[:, None, :]] = codes
        words = torch.stack((w & 255, w >> 8), -1).to(torch.uint8).flatten(-2)
        where = base + 32 * d + k[:, None] * (2 * ng) + torch.arange(2 * ng, device=dev)
        cache[b[:, None, None], at, blk[:, None, None], where[:, None, :]] = words
        base += 34 * d


def _visible(case, lens, dev, b, e):
    """[e, n, m] truth values, and the distance |position - slot| [e, n, m]."""
    n, m, mask = case["n"], case["m"], case["mask"]
    j = torch.arange(m, device=dev)
    i = torch.arange(n, device=dev)
    ln = lens[b:b + e, None, None].long()
    off = ln - n if mask == "causal_cache" else torch.full_like(ln, m - n)
    pos = i[None, :, None] + off
    vis = torch.ones(e, n, m, dtype=torch.bool, device=dev)
    if mask in LENGTH_MASKS:
        vis &= j < ln
    if mask in CAUSAL_MASKS:
        vis &= j <= pos
    return vis, (pos - j).abs()


def _plain_attend(case, st):
    B, H, H_kv, n, m, d_k, d_v = (case[k] for k in ("B", "H", "H_kv", "n", "m", "d_k", "d_v"))
    dev = st["cache"].device
    O = torch.empty(B, H, n, d_v, dtype=torch.bfloat16, device=dev)
    LSE = torch.empty(B, H, n, device=dev)
    step = _entries(case)
    for b in range(0, B, step):
        e = min(step, B - b)
        K, V = _read_blocks(st["cache"][b:b + e], d_k, d_v)
        K, V = K[:, :, :m], V[:, :, :m]
        vis, dist = _visible(case, st["lens"], dev, b, e)
        V = torch.where(vis.any(1)[:, None, :, None], V, torch.zeros((), device=dev))   # masked slots may hold anything
        Q = st["Q"][b:b + e].float().unflatten(1, (H_kv, -1)).flatten(2, 3)             # [e, H_kv, group n, d_k]
        S = (Q @ K.transpose(-1, -2)) / math.sqrt(d_k)
        S = S.unflatten(2, (-1, n)).flatten(1, 2)                                       # [e, H, n, m]
        if st["slopes"] is not None:
            S = S - st["slopes"][:, None, None] * dist[:, None]
        S = torch.where(vis[:, None], S, torch.full((), -math.inf, device=dev))
        top = S.amax(-1, keepdim=True)
        P = torch.exp(S - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = P.sum(-1, keepdim=True)
        out = P.unflatten(1, (H_kv, -1)).flatten(2, 3) @ V
        out = out.unflatten(2, (-1, n)).flatten(1, 2) / torch.where(total == 0, torch.ones_like(total), total)
        O[b:b + e] = out.to(torch.bfloat16)
        LSE[b:b + e] = (top + torch.log(total)).squeeze(-1)
    return O, LSE


# ------------------------------------------------------------------ prepare and run

def _draws(g, shape, channels):
    """Keys or values as a model makes them: normal, each channel with an offset and a
    width of its own, a few channels far wider than the rest."""
    off, width = channels
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * width + off).to(torch.bfloat16)


def _channels(g, H_kv, d):
    off = torch.randn(H_kv, 1, d, generator=g, device="cuda") * 0.5
    width = torch.exp(torch.randn(H_kv, 1, d, generator=g, device="cuda") * 0.3)
    wide = torch.rand(H_kv, 1, d, generator=g, device="cuda") < 0.03
    return off, torch.where(wide, 3 * width, width)


def prepare(case, seed):
    B, H, H_kv, n, m, d_k, d_v = (case[k] for k in ("B", "H", "H_kv", "n", "m", "d_k", "d_v"))
    g = torch.Generator("cuda").manual_seed(seed)
    blocks = -(-m // BLOCK)
    chan_k, chan_v = _channels(g, H_kv, d_k), _channels(g, H_kv, d_v)
    lens = _lengths(case)
    # slots that nothing has written yet hold whatever the memory held
    cache = torch.randint(0, 256, (B, H_kv, blocks, _block_bytes(d_k, d_v)), generator=g, device="cuda", dtype=torch.uint8)
    for b in range(B):
        filled = -(-(lens[b] if case["op"] != "attend" or case["mask"] in LENGTH_MASKS else m) // BLOCK)
        if filled:
            K = _draws(g, (H_kv, filled * BLOCK, d_k), chan_k)
            V = _draws(g, (H_kv, filled * BLOCK, d_v), chan_v)
            cache[b, :, :filled] = _blocks(K, V)
    st = dict(case=case, cache=cache, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["op"] == "attend":
        st["Q"] = torch.randn(B, H, n, d_k, generator=g, device="cuda").to(torch.bfloat16)
        st["slopes"] = None
        if case["slopes"]:
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")
    if case["op"] == "write":
        st["K"] = _draws(g, (B, H_kv, n, d_k), chan_k)
        st["V"] = _draws(g, (B, H_kv, n, d_v), chan_v)
        st["starts"] = st["lens"]
        st["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device="cuda")
        st["lens"] = st["starts"] + st["counts"]                               # filled once the rows are in
    if own and case["op"] == "attend":
        from transformer_scaled_dot_03_gb300 import attn
        size = attn.decode_q4_workspace_size(B, H, H_kv, n, m, d_k, d_v)
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    return st


def run(state):
    case, st = state["case"], state
    if not own:
        if case["op"] == "attend":
            return _plain_attend(case, st)
        if case["op"] == "write":
            _plain_write(case, st)
        return _plain_read(case, st["cache"], st["lens"])
    from transformer_scaled_dot_03_gb300 import attn
    if case["op"] == "attend":
        lens = st["lens"] if case["mask"] in LENGTH_MASKS else None
        return attn.decode_q4(st["Q"], st["cache"], case["mask"], lens, m=case["m"], slopes=st["slopes"],
                              workspace=st["workspace"])
    if case["op"] == "write":
        attn.cache_q4_write(st["cache"], st["K"], st["V"], st["starts"], st["counts"], m=case["m"])
    return attn.cache_q4_read(st["cache"], case["d_k"], case["m"], st["lens"], H=case["H"])


def _pairs(case):
    """Visible (row, slot) pairs of one query head, and the slots that any row sees, over the batch."""
    n, m, mask = case["n"], case["m"], case["mask"]
    pairs = slots = 0
    for ln in _lengths(case):
        ln = ln if mask in LENGTH_MASKS else m
        off = (ln if mask == "causal_cache" else m) - n
        seen = [max(0, min(ln, i + off + 1)) if mask in CAUSAL_MASKS else ln for i in range(n)]
        pairs += sum(seen)
        slots += max(seen)
    return pairs, slots


def work(case):
    B, H, H_kv, n, d_k, d_v = (case[k] for k in ("B", "H", "H_kv", "n", "d_k", "d_v"))
    slot = 17 * (d_k + d_v) // 32
    if case["op"] == "attend":
        pairs, slots = _pairs(case)
        return {"bytes": slots * H_kv * slot + B * H * n * (2 * d_k + 2 * d_v + 4), "flops": 2 * (d_k + d_v) * H * pairs}
    out = B * H * case["m"] * 2 * (d_k + d_v)
    if case["op"] == "read":
        rows = sum(_lengths(case)) * H_kv
        return {"bytes": rows * slot + out, "flops": 2 * rows * (d_k + d_v)}
    new = sum(_counts(case)) * H_kv
    rows = sum(_lengths(case)) * H_kv                                          # what was there: read, the new rows: written
    return {"bytes": new * (2 * (d_k + d_v) + slot) + rows * slot + out, "flops": (rows + 3 * new) * (d_k + d_v)}


# -------------------------------------------------------------------------- exact

def _addresses(d, is_k, dev):
    """Byte and bit of every code of a block's 64 slots, from the format's formulas."""
    k = torch.arange(BLOCK, device=dev)[:, None]
    e = torch.arange(d, device=dev)[None, :]
    ng, q, c = d // GROUP, e // GROUP, e % GROUP
    if is_k:
        row = k ^ (((k >> 2) & 1) * (128 // d))
        return row * (d // 2) + ((c // 16) * ng + q) * 8 + (c % 16) // 2, (c % 2) * 4
    unit = (c // 8) ^ (4 * ((k >> 1) & 1) if d == 128 else 0 * k)
    return k * (d // 2) + unit * (4 * ng) + q * 4 + (c % 8) // 2, (c % 2) * 4 + 0 * k


def _exact_side(cache, base, d, is_k):
    """fp64 values [e, H_kv, slots, d] of the K (or V) part of the blocks."""
    byte, shift = _addresses(d, is_k, cache.device)
    u = (cache[..., base + byte].short() >> shift.short()) & 15
    k = torch.arange(BLOCK, device=cache.device)[:, None]
    at = base + 32 * d + 2 * (k * (d // GROUP) + torch.arange(d // GROUP, device=cache.device)[None, :])
    w = cache[..., at].int() + 256 * cache[..., at + 1].int()
    frac, ex = (w >> 4) & 7, (w >> 7) & 255
    s = torch.where(ex == 0, frac.double() * 2.0 ** -129, (8 + frac).double() * torch.exp2(ex.double() - 130))
    s = torch.where(ex == 255, torch.full_like(s, math.nan), s)
    v = (u - (w & 15).repeat_interleave(GROUP, -1)).double() * s.repeat_interleave(GROUP, -1)
    return v.flatten(-3, -2)


def _exact_quantised(x):
    """The value that each element of x [..., d] is stored as, fp64."""
    g = x.double().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, True).clamp(max=0), g.amax(-1, True).clamp(min=0)
    t = (hi - lo).float().double() / 15
    frac, ex = torch.frexp(t)                                                  # t = frac 2^ex, frac in [0.5, 1)
    s = torch.ceil(frac * 16) * torch.exp2(ex.double() - 4)
    one = torch.where(s == 0, torch.ones_like(s), s)
    u0 = torch.round(-lo / one)
    return (((torch.round(g / one) + u0).clamp(0, 15) - u0) * s).flatten(-2)


def exact(case, seed):
    B, H, H_kv, n, m, d_k, d_v = (case[k] for k in ("B", "H", "H_kv", "n", "m", "d_k", "d_v"))
    if B * H * m * (d_k + d_v) * (1 + (n // 8 if case["op"] == "attend" else 0)) > 5 * 10 ** 9:
        return None                                                            # over the time that this may take
    st = prepare(case, seed)
    dev = st["cache"].device
    outs = ([], [])
    for b in range(B):
        cache = st["cache"][b]
        K, V = _exact_side(cache, 0, d_k, True)[:, :m], _exact_side(cache, 34 * d_k, d_v, False)[:, :m]
        ln = int(st["lens"][b])
        if case["op"] != "attend":
            if case["op"] == "write":
                a, c = int(st["starts"][b]), int(st["counts"][b])
                K[:, a:a + c] = _exact_quantised(st["K"][b, :, :c])
                V[:, a:a + c] = _exact_quantised(st["V"][b, :, :c])
            K[:, ln:], V[:, ln:] = 0, 0
            for out, x in zip(outs, (K, V)):
                out.append(x.repeat_interleave(H // H_kv, 0))
            continue
        O = torch.zeros(H, n, d_v, dtype=torch.float64, device=dev)
        L = torch.full((H, n), -math.inf, dtype=torch.float64, device=dev)
        mask = case["mask"]
        ln = ln if mask in LENGTH_MASKS else m
        for i in range(n):
            pos = i + (ln if mask == "causal_cache" else m) - n
            end = max(0, min(ln, pos + 1)) if mask in CAUSAL_MASKS else ln
            if end == 0:
                continue
            q = st["Q"][b, :, i].double().unflatten(0, (H_kv, -1))
            s = (torch.einsum("hgd,hjd->hgj", q, K[:, :end]) / math.sqrt(d_k)).flatten(0, 1)
            if st["slopes"] is not None:
                away = (pos - torch.arange(end, device=dev)).abs().double()
                s = s - st["slopes"].double()[:, None] * away
            L[:, i] = torch.logsumexp(s, -1)
            p = torch.exp(s - L[:, i, None]).unflatten(0, (H_kv, -1))
            O[:, i] = torch.einsum("hgj,hjd->hgd", p, V[:, :end]).flatten(0, 1)
        outs[0].append(O)
        outs[1].append(L)
    return tuple(torch.stack(o) for o in outs)
