"""Measured cases of the 4-bit key/value cache: storing rows in it, attention
over it, the attention weight its entries accumulate, and the eviction that
goes by that weight.

`run` computes a case in its plain form (elementary torch operations in 32
bits) or, with `own` true, by the library's entry points.  `exact` gives the
same results from the definitions in 64 bits.

The cache's format.  A row (one token of one key/value head) is cut into
blocks of 16 consecutive channels.  A block holds one scale s in e4m3 (the
block's largest magnitude divided by 6, rounded to the nearest e4m3 value,
ties to even, at most 448) and 16 codes in e2m1 (x / s rounded to the nearest
of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with its sign, ties to the even code); two codes
share a byte, the even channel in its low half.  A block whose scale rounds
to 0 holds zeros.

Every pass leaves what it reads as it was (counts and accumulated weights go
to tensors of their own; the eviction in place reads only slots that it does
not move), so that the same pass can be repeated.
"""
import math

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's new token of eight sequences stored and read back: latency
        dict(name="append_b8_n1", op="append", B=8, H_kv=8, n=1, length=16384, d=128, dtype="bf16"),
        # the prompts of two sequences stored in one call and read back as attention will see them
        dict(name="append_b2_n8192", op="append", B=2, H_kv=8, n=8192, length=0, d=128, dtype="bf16"),
        # a single short conversation, small heads: latency
        dict(name="attend_b1_n1000", op="attend", B=1, H=8, H_kv=2, N_q=1, length=1000, ragged=False, d=64, dtype="f16",
             causal=False, weights=False),
        # the decode step the library measures on its 16-bit cache
        dict(name="attend_b8_n16384", op="attend", B=8, H=32, H_kv=8, N_q=1, length=16384, ragged=False, d=128,
             dtype="bf16", causal=False, weights=False),
        # a serving batch of sequences of different lengths that accumulates the weight eviction goes by
        dict(name="attend_b16_ragged_weights", op="attend", B=16, H=32, H_kv=8, N_q=1, length=8192, ragged=True, d=128,
             dtype="bf16", causal=False, weights=True),
        # four draft tokens verified in one step, each sees the ones before it
        dict(name="attend_b4_draft4", op="attend", B=4, H=16, H_kv=4, N_q=4, length=2048, ragged=True, d=64, dtype="f16",
             causal=True, weights=False),
        # one long document, its weights accumulated: the work has to be split over the sequence
        dict(name="attend_b1_n131071_weights", op="attend", B=1, H=32, H_kv=8, N_q=1, length=131071, ragged=False, d=128,
             dtype="bf16", causal=False, weights=True),
        # weights of a whole prompt, every query counted
        dict(name="weights_b2_n8192_causal", op="weights", B=2, H=32, H_kv=8, N_q=8192, N_kv=8192, first=0, d=128,
             dtype="bf16", causal=True),
        # weights by the last 64 queries of a short prompt alone
        dict(name="weights_b1_n1000_last64", op="weights", B=1, H=16, H_kv=16, N_q=1000, N_kv=1000, first=936, d=64,
             dtype="f16", causal=True),
        # a batch whose caches grew one entry past their bound: the lightest leaves, in place
        dict(name="evict_b8_4097_to_4096", op="evict", B=8, H_kv=8, length=4097, ragged=False, keep=4096, sinks=4,
             recent=0, d=64, in_place=True),
        # prompts compressed after they were read, into the smaller caches that decoding then uses
        dict(name="evict_b8_16384_to_2048", op="evict", B=8, H_kv=8, length=16384, ragged=True, keep=2048, sinks=4,
             recent=256, d=128, in_place=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weights", "evict"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    if op == "append":
        n = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(16, 16384 // n)))
        return dict(op=op, B=B, H_kv=rng.choice([1, 2, 5, 8]), n=n, length=_log(rng, 1, 4096) - 1, d=d, dtype=dtype)
    if op == "attend":
        H_kv, N_q = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 1, 2, 3, 4])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        length = _log(rng, 1, 131071)
        B = _log(rng, 1, max(1, min(32, 131071 // length)))
        return dict(op=op, B=B, H=H_kv * group, H_kv=H_kv, N_q=N_q, length=length, ragged=rng.random() < 0.5, d=d,
                    dtype=dtype, causal=N_q > 1 and rng.random() < 0.7, weights=rng.random() < 0.4)
    if op == "weights":
        H_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4])
        N_kv = _log(rng, 1, 8192)
        N_q = N_kv if rng.random() < 0.7 else _log(rng, 1, N_kv)
        first = 0 if rng.random() < 0.5 else N_q - _log(rng, 1, N_q)
        return dict(op=op, B=rng.choice([1, 2]), H=H_kv * group, H_kv=H_kv, N_q=N_q, N_kv=N_kv, first=first, d=d,
                    dtype=dtype, causal=rng.random() < 0.7)
    length = _log(rng, 2, 16384)
    in_place = rng.random() < 0.5
    keep = max(1, length - _log(rng, 1, 64)) if in_place else _log(rng, 1, length)
    return dict(op="evict", B=rng.choice([1, 2, 3, 8]), H_kv=rng.choice([1, 2, 8]), length=length,
                ragged=rng.random() < 0.5, keep=keep, sinks=rng.choice([0, 1, 4]),
                recent=0 if in_place else min(keep, rng.choice([0, 16, 256])), d=d, in_place=in_place)


def _padded(n):
    """Slots of a cache that holds n rows: capacities are multiples of 128."""
    return max(128, -(-n // 128) * 128)


def _lengths(c):
    """Rows held per sequence: the case's length, or spread below it."""
    if not c["ragged"]:
        return [c["length"]] * c["B"]
    return [max(1, c["length"] * (2 * (i * 7 % c["B"]) + 2) // (2 * c["B"]) - 13 * i % 7) for i in range(c["B"])]


# ------------------------------------------------------- format, plain form
def _round_scale(a):
    """Nonnegative fp32 rounded to e4m3 (nearest, ties to even, at most 448)."""
    _, e = torch.frexp(a)                          # a = m 2^e, m in [0.5, 1)
    step = torch.exp2((e - 1).clamp(min=-6).float() - 3)
    return (torch.round(a / step) * step).clamp(max=448.0)


def _scale_byte(s):
    """The e4m3 bits of values that are e4m3 already."""
    m, e = torch.frexp(s)
    e = e - 1
    normal = ((e + 7) * 8 + torch.round((2 * m - 1) * 8).int())
    small = torch.round(s * 512).int()             # multiples of 2^-9 below 2^-6
    return torch.where(s >= 2.0 ** -6, normal, small).to(torch.uint8)


def _scale_value(byte):
    b = byte.int()
    e, m = (b >> 3) & 15, (b & 7).float()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).float()), m * 2.0 ** -9)


def _quantise(x):
    """(codes 0..15, scales as fp32) of x [..., d]: blocks of 16 channels."""
    x = x.float().unflatten(-1, (-1, 16))
    s = _round_scale(x.abs().amax(-1) / 6)
    y = torch.where(s[..., None] > 0, x / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    a = y.abs()
    code = (a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() \
        + (a >= 3.5).int() + (a > 5).int()
    return (code + 8 * (y < 0).int()).flatten(-2), s


def _pack(code, s):
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), _scale_byte(s)


def _values(code, s):
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=code.device)
    return (table[code.long()].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _unpack(codes, scales):
    """fp32 values of packed rows."""
    c = codes.int()
    return _values(torch.stack((c & 15, c >> 4), -1).flatten(-2), _scale_value(scales))


# ------------------------------------------------------------------- states
def _rows(g, shape, dtype):
    """Key- or value-like rows: unit normal with a few strong channels."""
    x = torch.randn(shape, generator=g, device="cuda")
    gain = torch.exp(0.5 * torch.randn(shape[1], 1, shape[3], generator=g, device="cuda"))
    return (x * gain).to(dtype)


def _cache(g, B, H_kv, capacity, d, lengths, seen):
    st = {}
    for part in ("k", "v"):
        st[part + "_codes"], st[part + "_scales"] = _pack(*_quantise(_rows(g, (B, H_kv, capacity, d), torch.bfloat16)))
    st["counts"] = torch.tensor([lengths, seen], dtype=torch.int32, device="cuda")
    st["pos"] = torch.arange(capacity, dtype=torch.int32, device="cuda").expand(B, H_kv, capacity).contiguous()
    w = torch.rand(B, H_kv, capacity, generator=g, device="cuda")
    st["weight"] = -torch.log1p(-w) * 0.5          # exponential: most entries are light
    return st


def _handle(st):
    from exact_tiled_attention_04_gb300 import KV4Cache
    return KV4Cache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], st["counts"], pos=st["pos"],
                    weight=st["weight"])


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(int(seed))
    st = dict(case=c)
    if c["op"] == "append":
        cap = _padded(c["length"] + c["n"])
        st.update(_cache(g, c["B"], c["H_kv"], cap, c["d"], [c["length"]] * c["B"], [c["length"] + 5] * c["B"]))
        st["k"] = _rows(g, (c["B"], c["H_kv"], c["n"], c["d"]), DTYPES[c["dtype"]])
        st["v"] = _rows(g, (c["B"], c["H_kv"], c["n"], c["d"]), DTYPES[c["dtype"]])
        st["counts_out"] = torch.empty_like(st["counts"])
    elif c["op"] == "attend":
        lengths = _lengths(c)
        st.update(_cache(g, c["B"], c["H_kv"], _padded(max(lengths)), c["d"], lengths, lengths))
        st["q"] = torch.randn(c["B"], c["H"], c["N_q"], c["d"], generator=g, device="cuda").to(DTYPES[c["dtype"]])
        st["weight_out"] = torch.zeros_like(st["weight"]) if c["weights"] else None
    elif c["op"] == "weights":
        st["q"] = torch.randn(c["B"], c["H"], c["N_q"], c["d"], generator=g, device="cuda").to(DTYPES[c["dtype"]])
        st["k"] = _rows(g, (c["B"], c["H_kv"], c["N_kv"], c["d"]), DTYPES[c["dtype"]])
        st["weight_in"] = torch.rand(c["B"], c["H_kv"], c["N_kv"], generator=g, device="cuda")
        st["weight_out"] = torch.zeros_like(st["weight_in"])
        # the log-sum-exp that the forward pass over the prompt has returned
        lse = [torch.logsumexp(_prompt_scores(st, b), -1) for b in range(c["B"])]
        st["lse"] = torch.stack(lse).reshape(c["B"], c["H"], c["N_q"]).contiguous()
    else:
        lengths = _lengths(c)
        st.update(_cache(g, c["B"], c["H_kv"], _padded(max(lengths)), c["d"], lengths, lengths))
        st["rank_by"] = st["weight"].clone()
        st["counts_out"] = torch.empty_like(st["counts"])
        if not c["in_place"]:
            st["to"] = _cache(g, c["B"], c["H_kv"], _padded(c["keep"]), c["d"], [0] * c["B"], [0] * c["B"])
    if own:
        if c["op"] != "weights":
            st["cache"] = _handle(st)
        if "to" in st:
            st["to_cache"] = _handle(st["to"])
    return st


# --------------------------------------------------------------------- runs
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import exact_tiled_attention_04_gb300 as fa
    c = st["case"]
    if c["op"] == "append":
        fa.kv4_append(st["cache"], st["k"], st["v"], counts_out=st["counts_out"])
        k, v = fa.kv4_read(st["cache"], c["n"], first=st["counts"][0], dtype=st["k"].dtype)
        return {"k": k, "v": v, "counts": st["counts_out"], "pos": st["pos"], "weight": st["weight"]}
    if c["op"] == "attend":
        out, lse = fa.kv4_attention(st["q"], st["cache"], causal=c["causal"], weight_out=st["weight_out"])
        return {"out": out, "lse": lse, "weight": st["weight_out"]}
    if c["op"] == "weights":
        return {"weight": fa.attention_weights(st["q"], st["k"], st["lse"], causal=c["causal"], first_query=c["first"],
                                               weight_in=st["weight_in"], out=st["weight_out"])}
    src = fa.kv4_evict(st["cache"], c["keep"], sinks=c["sinks"], recent=c["recent"], weight=st["rank_by"],
                       out=st.get("to_cache"), counts_out=st["counts_out"])
    return _evicted(st, src)


def _evicted(st, src):
    to = st.get("to", st)
    return {"src": src, "counts": st["counts_out"], "pos": to["pos"], "weight": to["weight"], "k_codes": to["k_codes"],
            "k_scales": to["k_scales"], "v_codes": to["v_codes"], "v_scales": to["v_scales"]}


def _run_plain(st):
    return {"append": _append, "attend": _attend, "weights": _weights, "evict": _evict}[st["case"]["op"]](st)


def _append(st):
    c = st["case"]
    slots = st["counts"][0][:, None].long() + torch.arange(c["n"], device="cuda")            # [B, n]
    slots = slots[:, None].expand(c["B"], c["H_kv"], c["n"])
    got = []
    for part in ("k", "v"):
        code, s = _quantise(st[part])
        codes, scales = _pack(code, s)
        st[part + "_codes"].scatter_(2, slots[..., None].expand(codes.shape), codes)
        st[part + "_scales"].scatter_(2, slots[..., None].expand(scales.shape), scales)
        got.append(_values(code, s).to(st[part].dtype))
    pos = st["counts"][1][:, None] + torch.arange(c["n"], dtype=torch.int32, device="cuda")
    st["pos"].scatter_(2, slots, pos[:, None].expand(slots.shape).contiguous())
    st["weight"].scatter_(2, slots, torch.zeros(slots.shape, device="cuda"))
    torch.add(st["counts"], c["n"], out=st["counts_out"])
    return {"k": got[0], "v": got[1], "counts": st["counts_out"], "pos": st["pos"], "weight": st["weight"]}


def _visible(c, lengths, slots):
    """[B, 1, 1, N_q, slots]: what each query sees."""
    last = lengths[:, None] - (torch.arange(c["N_q"] - 1, -1, -1, device="cuda") if c["causal"] else
                               torch.zeros(c["N_q"], dtype=torch.int32, device="cuda"))       # [B, N_q]
    return (torch.arange(slots, device="cuda") < last[..., None])[:, None, None]


def _attend(st):
    c = st["case"]
    B, H_kv, d = c["B"], c["H_kv"], c["d"]
    k, v = _unpack(st["k_codes"], st["k_scales"]), _unpack(st["v_codes"], st["v_scales"])
    q = st["q"].float().reshape(B, H_kv, -1, d)
    s = (q @ k.transpose(-1, -2)) * (1 / math.sqrt(d))
    s = s.reshape(B, H_kv, -1, c["N_q"], k.shape[2]).masked_fill(~_visible(c, st["counts"][0], k.shape[2]), -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, 1.0)
    out = (p.reshape(B, H_kv, -1, k.shape[2]) @ v).reshape(st["q"].shape).to(st["q"].dtype)
    lse = (m + torch.log(l)).reshape(B, c["H"], c["N_q"])
    if c["weights"]:
        used = torch.arange(k.shape[2], device="cuda") < st["counts"][0][:, None, None]
        torch.where(used, st["weight"] + p.sum((2, 3)), st["weight_out"], out=st["weight_out"])
    return {"out": out, "lse": lse, "weight": st["weight_out"]}


def _prompt_scores(st, b):
    """[H_kv, group, N_q, N_kv] of sequence b in 32 bits, masked."""
    c = st["case"]
    q = st["q"][b].float().reshape(c["H_kv"], -1, c["d"])
    s = (q @ st["k"][b].float().transpose(-1, -2)) * (1 / math.sqrt(c["d"]))
    s = s.reshape(c["H_kv"], -1, c["N_q"], c["N_kv"])
    if c["causal"]:
        i = torch.arange(c["N_q"], device="cuda")[:, None] + (c["N_kv"] - c["N_q"])
        s.masked_fill_(torch.arange(c["N_kv"], device="cuda") > i, -math.inf)
    return s


def _weights(st):
    c = st["case"]
    for b in range(c["B"]):
        p = torch.exp(_prompt_scores(st, b) - st["lse"][b].reshape(c["H_kv"], -1, c["N_q"], 1))
        st["weight_out"][b] = st["weight_in"][b] + p[:, :, c["first"]:].sum((1, 2))
    return {"weight": st["weight_out"]}


def _selection(st):
    """src [B, H_kv, keep] (-1 behind the last) and the new counts."""
    c = st["case"]
    n = st["counts"][0][:, None, None]
    cap, keep = st["pos"].shape[2], c["keep"]
    slot = torch.arange(cap, device="cuda")
    held = slot < n
    first = held & ((st["pos"] < c["sinks"]) | (st["pos"] >= st["counts"][1][:, None, None] - c["recent"]))
    rank = torch.where(first, math.inf, torch.where(held, st["rank_by"], -math.inf))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.zeros(rank.shape, dtype=torch.bool, device="cuda").scatter_(2, order, True) & held
    new = torch.clamp(n, max=keep)
    # holes take the kept entries at or behind the new length, both in order
    hole = ~kept & (slot < new)
    behind = kept & (slot >= new)
    queue = torch.sort(behind.int(), dim=-1, descending=True, stable=True).indices
    nth = (torch.cumsum(hole.int(), -1) - 1).clamp(min=0)
    src = torch.where(hole, queue.gather(2, nth), torch.where(slot < new, slot, -1))
    src = torch.nn.functional.pad(src, (0, max(0, keep - cap)), value=-1)[..., :keep]
    return src.int(), torch.stack((new[:, 0, 0], st["counts"][1]))


def _evict(st):
    c = st["case"]
    src, counts = _selection(st)
    to, w = st.get("to", st), min(c["keep"], st["pos"].shape[2])
    at = src[..., :w].long().clamp(min=0)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        x = st[name].gather(2, at[..., None].expand(*at.shape, st[name].shape[3]))
        to[name][:, :, :w] = torch.where(src[..., :w, None] >= 0, x, to[name][:, :, :w])
    for name in ("pos", "weight"):
        to[name][:, :, :w] = torch.where(src[..., :w] >= 0, st[name].gather(2, at), to[name][:, :, :w])
    st["counts_out"].copy_(counts)
    return _evicted(st, src)


# -------------------------------------------------------------------- exact
def _exact_values(codes, scales):
    """fp64 values of packed rows, by the fields of the two formats."""
    c = torch.empty(*codes.shape, 2, dtype=torch.int64, device="cuda")
    c[..., 0], c[..., 1] = codes % 16, codes // 16
    c = c.reshape(*codes.shape[:-1], -1)
    e, m = (c // 2) % 4, c % 2
    x = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e - 1).double()) * (1 - 2 * (c // 8)).double()
    b = scales.long()
    e, m = (b // 8) % 16, (b % 8).double() / 8
    s = torch.where(e == 0, m * 2.0 ** -6, (1 + m) * 2.0 ** (e - 7).double())
    return x * s.repeat_interleave(16, -1)


def _nearest(x, grid):
    """Each x >= 0 at the nearest point of the grid, ties to the even index, none past its end."""
    grid = torch.tensor(grid, dtype=torch.float64, device="cuda")
    hi = torch.bucketize(x, grid).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = x - grid[lo], grid[hi] - x
    return grid[torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)]


def _exact_stored(x):
    x = x.double().unflatten(-1, (-1, 16))
    e4m3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    s = _nearest(x.abs().amax(-1, keepdim=True) / 6, e4m3[:-1])
    y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    return (_nearest(y, LEVELS) * torch.sign(x) * s).flatten(-2)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "append":
        n, at = c["n"], c["length"]
        st["pos"][:, :, at:at + n] = torch.arange(at + 5, at + 5 + n, dtype=torch.int32, device="cuda")
        st["weight"][:, :, at:at + n] = 0
        return {"k": _exact_stored(st["k"]), "v": _exact_stored(st["v"]), "counts": st["counts"] + n, "pos": st["pos"],
                "weight": st["weight"].double()}
    if c["op"] == "attend":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(st["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
        weight = torch.zeros(st["weight"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(c)):
            for h in range(c["H"]):
                g = h // (c["H"] // c["H_kv"])
                k = _exact_values(st["k_codes"][b, g, :n], st["k_scales"][b, g, :n])
                v = _exact_values(st["v_codes"][b, g, :n], st["v_scales"][b, g, :n])
                if h % (c["H"] // c["H_kv"]) == 0:
                    weight[b, g, :n] += st["weight"][b, g, :n]
                for i in range(c["N_q"]):
                    m = n - (c["N_q"] - 1 - i) if c["causal"] else n
                    if m > 0:
                        s = k[:m] @ st["q"][b, h, i].double() / math.sqrt(c["d"])
                        lse[b, h, i] = torch.logsumexp(s, 0)
                        p = torch.exp(s - lse[b, h, i])
                        out[b, h, i] = p @ v[:m]
                        weight[b, g, :m] += p
        return {"out": out, "lse": lse, "weight": weight if c["weights"] else None}
    if c["op"] == "weights":
        weight = st["weight_in"].double()
        rows = torch.arange(c["first"], c["N_q"], device="cuda")[:, None] + (c["N_kv"] - c["N_q"])
        for b in range(c["B"]):
            for h in range(c["H"]):
                g = h // (c["H"] // c["H_kv"])
                s = st["q"][b, h, c["first"]:].double() @ st["k"][b, g].double().T / math.sqrt(c["d"])
                p = torch.exp(s - st["lse"][b, h, c["first"]:, None].double())
                if c["causal"]:
                    p = torch.where(torch.arange(c["N_kv"], device="cuda") <= rows, p, 0.0)
                weight[b, g] += p.sum(0)
        return {"weight": weight}
    to = st.get("to", st)
    src = torch.full((c["B"], c["H_kv"], c["keep"]), -1, dtype=torch.int32)
    counts = st["counts"].clone()
    for b, n in enumerate(_lengths(c)):
        counts[0, b] = new = min(n, c["keep"])
        for h in range(c["H_kv"]):
            w, pos = st["rank_by"][b, h, :n].tolist(), st["pos"][b, h, :n].tolist()
            best = sorted(range(n), key=lambda j: (not (pos[j] < c["sinks"] or pos[j] >= n - c["recent"]), -w[j], j))
            kept = set(best[:new])
            late = iter(sorted(j for j in kept if j >= new))
            src[b, h, :new] = torch.tensor([j if j in kept else next(late) for j in range(new)], dtype=torch.int32)
            at = src[b, h, :new].long().cuda()
            for name in ("k_codes", "k_scales", "v_codes", "v_scales", "pos", "weight"):
                to[name][b, h, :new] = st[name][b, h][at]
    got = {name: to[name] for name in ("pos", "weight", "k_codes", "k_scales", "v_codes", "v_scales")}
    return {"src": src.cuda(), "counts": counts, **got}


# --------------------------------------------------------------------- work
def work(case):
    c, d = case, case["d"]
    row = d // 2 + d // 16
    if c["op"] == "append":     # 16-bit rows in, packed rows out and in again, 16-bit values out; pos and weight
        return {"bytes": c["B"] * c["H_kv"] * c["n"] * (2 * (2 * d + 2 * row + 2 * d) + 8), "flops": 0}
    if c["op"] == "attend":
        held, rows = sum(_lengths(c)), c["B"] * c["H"] * c["N_q"]
        return {"bytes": held * c["H_kv"] * (2 * row + (8 if c["weights"] else 0)) + rows * (4 * d + 4),
                "flops": 4 * d * c["H"] * c["N_q"] * held}
    if c["op"] == "weights":
        counted = c["N_q"] - c["first"]
        seen = counted * c["N_kv"]
        if c["causal"]:
            seen -= counted * (counted - 1) // 2
        return {"bytes": 2 * d * c["B"] * (c["H"] * counted + c["H_kv"] * c["N_kv"]) + 4 * c["B"] * c["H"] * counted
                + 8 * c["B"] * c["H_kv"] * c["N_kv"], "flops": 2 * d * c["B"] * c["H"] * seen}
    held, kept = sum(_lengths(c)), sum(min(n, c["keep"]) for n in _lengths(c))
    moved = sum(min(n - k, k) for n, k in ((n, min(n, c["keep"])) for n in _lengths(c))) if c["in_place"] else kept
    return {"bytes": c["H_kv"] * (8 * held + 4 * kept + 2 * moved * (2 * row + 8)), "flops": 0}
