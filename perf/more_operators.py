"""Measured cases of attention over packed sequences (a prompt's forward pass
and its gradients) and of a paged 16-bit key/value cache: rows rotated and
stored in it, and decode steps over it, alone or behind a prefix that the whole
batch shares.

`run` computes a case in its plain form (elementary torch operations in 32
bits) or, with `own` true, by the library's entry points.  `exact` gives the
same results from the definitions in 64 bits.

Packed sequences.  Rows of all sequences lie one behind the other, [rows,
heads, d]; sequence b has rows cu[b] .. cu[b + 1] - 1.  Query i of a sequence
sees its own sequence's keys, under the causal mask those with
j <= i + n_k - n_q.

Paged cache.  Pages [pages, H_kv, page, d]; slot s of sequence b is row
s % page of page block_table[b, s // page].

Rotation.  The first `rot` channels of a row at position p are turned in pairs,
(x, y) -> (x cos - y sin, x sin + y cos), by row p of a table of cosines and
sines that the program keeps; pair j is channels (j, j + rot / 2), or
(2j, 2j + 1) where interleaved.

Every pass leaves what it reads as it was (lengths go to a tensor of their own),
so that the same pass can be repeated.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a few short requests, one of a single token: latency
        dict(name="prompt_b3_short", op="prompt", lens="1,37,200", lens_k="", H=8, H_kv=2, d=64, dtype="f16",
             causal=True, fused=False),
        # a serving batch's prompts, q, k and v as one projection leaves them
        dict(name="prompt_b16_ragged", op="prompt",
             lens="2048,1999,1531,1200,1024,777,700,640,513,384,300,255,200,129,64,17", lens_k="", H=32, H_kv=8, d=128,
             dtype="bf16", causal=True, fused=True),
        # one long document beside shorter ones: the work lies in a few rows of blocks
        dict(name="prompt_b4_n16384", op="prompt", lens="16384,8191,4096,1000", lens_k="", H=32, H_kv=8, d=128,
             dtype="bf16", causal=True, fused=False),
        # gradients of a small batch whose keys are another text's (encoder and decoder), one pair without keys
        dict(name="grad_b5_cross", op="grad", lens="100,33,257,1,64", lens_k="300,0,128,77,64", H=8, H_kv=8, d=64,
             dtype="f16", causal=False, fused=False),
        # a training step's packed documents
        dict(name="grad_b8_docs", op="grad", lens="4096,3500,2777,2048,1600,1111,777,475", lens_k="", H=32, H_kv=8,
             d=128, dtype="bf16", causal=True, fused=True),
        # long sequences read in both directions, a key/value head to each query head
        dict(name="grad_b2_n8192_full", op="grad", lens="8192,8000", lens_k="", H=16, H_kv=16, d=64, dtype="bf16",
             causal=False, fused=False),
        # one decode step's new tokens of 32 sequences: latency
        dict(name="append_b32_step", op="append", lens=",".join(["1"] * 32), held=2048, H=32, H_kv=8, d=128, rot=128,
             page=16, dtype="bf16", interleaved=False),
        # chunks of three prompts rotated and stored, q rotated beside them
        dict(name="append_b3_n8192", op="append", lens="5000,3000,192", held=500, H=32, H_kv=8, d=128, rot=128, page=64,
             dtype="bf16", interleaved=False),
        # a decode step of a few short conversations: latency
        dict(name="step_b4_n1000", op="step", B=4, H=8, H_kv=2, N_q=1, length=1000, ragged=True, prefix=0, d=64,
             page=16, dtype="f16", causal=False),
        # a decode step of a serving batch of different lengths
        dict(name="step_b32_n16384", op="step", B=32, H=32, H_kv=8, N_q=1, length=16384, ragged=True, prefix=0, d=128,
             page=64, dtype="bf16", causal=False),
        # drafted tokens of requests behind a system prompt that ends inside a page
        dict(name="prefix_b8_draft4", op="step", B=8, H=16, H_kv=4, N_q=4, length=100, ragged=True, prefix=2000, d=64,
             page=16, dtype="f16", causal=True),
        # a large batch behind a long shared document
        dict(name="prefix_b64_n8192", op="step", B=64, H=32, H_kv=8, N_q=1, length=512, ragged=True, prefix=8192, d=128,
             page=64, dtype="bf16", causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "grad", "append", "step", "step"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    H_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4])
    if op in ("prompt", "grad"):
        causal = rng.random() < 0.7
        total, lens = {("prompt", True): 24000, ("prompt", False): 16000, ("grad", True): 10000,
                       ("grad", False): 7000}[op, causal], []
        longest = _log(rng, 1, total // 2)
        while len(lens) < 48 and (not lens or rng.random() < 0.85):
            n = 0 if rng.random() < 0.05 else _log(rng, 1, longest)
            if sum(lens) + n > total:
                break
            lens.append(n)
        if max(lens) == 0:
            lens[0] = 1
        lens_k = ""
        if rng.random() < 0.25:  # keys of another length: chunks behind earlier tokens, other texts
            lens_k = ",".join(str(max(0, n + rng.choice([0, 1, -1, 127, 500]))) for n in lens)
        return dict(op=op, lens=",".join(map(str, lens)), lens_k=lens_k, H=H_kv * group, H_kv=H_kv, d=d, dtype=dtype,
                    causal=causal, fused=lens_k == "" and rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 64)
        longest = _log(rng, 1, max(1, 8192 // B))
        lens = [1] * B if rng.random() < 0.4 else [0 if rng.random() < 0.1 else _log(rng, 1, longest) for _ in range(B)]
        if max(lens) == 0:
            lens[0] = 1
        return dict(op=op, lens=",".join(map(str, lens)), held=_log(rng, 1, 2048) - 1, H=H_kv * group, H_kv=H_kv, d=d,
                    rot=rng.choice([d, d, d // 2, 32]), page=page, dtype=dtype, interleaved=rng.random() < 0.3)
    N_q = rng.choice([1, 1, 1, 2, 4])
    prefix = _log(rng, 1, 8192) if rng.random() < 0.4 else 0
    length = _log(rng, 1, 16384)
    B = _log(rng, 1, max(1, min(64, 250000 // (length + prefix))))
    return dict(op="step", B=B, H=H_kv * rng.choice([1, 2, 4, 5, 8]), H_kv=H_kv, N_q=N_q, length=length,
                ragged=rng.random() < 0.7, prefix=prefix, d=d, page=page, dtype=dtype,
                causal=N_q > 1 and rng.random() < 0.7)


def _list(text):
    return [int(x) for x in text.split(",")]


def _seqs(c):
    """(first query row, queries, first key row, keys) of each sequence."""
    nq, out, a, b = _list(c["lens"]), [], 0, 0
    nk = _list(c["lens_k"]) if c["lens_k"] else nq
    for x, y in zip(nq, nk):
        out.append((a, x, b, y))
        a, b = a + x, b + y
    return out


def _held(c):
    """Slots in use per sequence: a step's cases the length or spread below it, an append's around `held`."""
    if c["op"] == "append":
        return [max(0, c["held"] - 37 * (i % 5)) for i in range(len(_list(c["lens"])))]
    if not c["ragged"]:
        return [c["length"]] * c["B"]
    return [max(1, c["length"] * (2 * (i * 7 % c["B"]) + 2) // (2 * c["B"]) - 13 * i % 7) for i in range(c["B"])]


# ------------------------------------------------------------------- states
def _rows(g, shape, dtype):
    """Key- or value-like rows: unit normal with a few strong channels."""
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp(0.3 * torch.randn(shape[-1], generator=g, device="cuda"))).to(dtype)


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def _table(n, rot, base=10000.0):
    """fp32 [n, rot]: the cosines of a position's rot / 2 angles, then their sines (angles in 64 bits)."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def _pages(c, g, lens, prefix=0):
    """Page pool and block tables in a shuffled order, as a server's free list leaves them."""
    need = [max(1, -(-n // c["page"])) for n in lens]
    shared = -(-prefix // c["page"])
    pool = sum(need) + shared + 3
    order = torch.randperm(pool, generator=g, device="cuda").int()
    st = {p: _rows(g, (pool, c["H_kv"], c["page"], c["d"]), DTYPES[c["dtype"]]) for p in ("k_pages", "v_pages")}
    st["block_table"] = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    at = shared
    for b, n in enumerate(need):
        st["block_table"][b, :n] = order[at:at + n]
        at += n
    st["prefix_pages"] = order[:shared].contiguous() if prefix else None
    return st


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(int(seed))
    st, t, d = dict(case=c), DTYPES[c["dtype"]], c["d"]
    if c["op"] in ("prompt", "grad"):
        seqs = _seqs(c)
        Tq, Tk = sum(s[1] for s in seqs), sum(s[3] for s in seqs)
        if c["fused"]:
            qkv = _rows(g, (Tq, c["H"] + 2 * c["H_kv"], d), t)
            st["q"], st["k"], st["v"] = qkv.split([c["H"], c["H_kv"], c["H_kv"]], 1)
        else:
            st["q"], st["k"], st["v"] = (_rows(g, (n, h, d), t) for n, h in
                                         ((Tq, c["H"]), (Tk, c["H_kv"]), (Tk, c["H_kv"])))
        st["cu_q"] = _cu([s[1] for s in seqs])
        st["cu_k"] = _cu([s[3] for s in seqs]) if c["lens_k"] else st["cu_q"]
        if c["op"] == "grad":  # what the forward pass has returned, and the gradient that comes back
            st["out"], st["lse"] = _prompt(st)
            st["dout"] = torch.randn(Tq, c["H"], d, generator=g, device="cuda").to(t)
        return st
    held = _held(c)
    if c["op"] == "append":
        lens = _list(c["lens"])
        st.update(_pages(c, g, [a + b for a, b in zip(held, lens)]))
        st["q"], st["k"], st["v"] = (_rows(g, (sum(lens), h, d), t) for h in (c["H"], c["H_kv"], c["H_kv"]))
        st["cu"] = None if min(lens) == max(lens) == 1 else _cu(lens)
        st["table"] = _table(max(a + b for a, b in zip(held, lens)), c["rot"])
        st["lengths_out"] = torch.empty(len(lens), dtype=torch.int32, device="cuda")
    else:
        st.update(_pages(c, g, held, c["prefix"]))
        st["q"] = torch.randn(c["B"], c["H"], c["N_q"], d, generator=g, device="cuda").to(t)
    st["lengths"] = torch.tensor(held, dtype=torch.int32, device="cuda")
    if own:
        from exact_tiled_attention_04_gb300 import PagedKVCache
        st["cache"] = PagedKVCache(st["k_pages"], st["v_pages"], st["block_table"], st["lengths"])
    return st


# --------------------------------------------------------------------- runs
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import exact_tiled_attention_04_gb300 as fa
    c = st["case"]
    if c["op"] == "prompt":
        out, lse = fa.packed_attention(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], causal=c["causal"])
        return {"out": out, "lse": lse}
    if c["op"] == "grad":
        dq, dk, dv = fa.packed_attention_backward(st["q"], st["k"], st["v"], st["out"], st["lse"], st["dout"],
                                                  st["cu_q"], st["cu_k"], causal=c["causal"])
        return {"dq": dq, "dk": dk, "dv": dv}
    if c["op"] == "append":
        q = fa.paged_append(st["cache"], st["k"], st["v"], cu=st["cu"], q=st["q"], table=st["table"],
                            interleaved=c["interleaved"], lengths_out=st["lengths_out"])
        return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"], "lengths": st["lengths_out"]}
    out, lse = fa.paged_attention(st["q"], st["cache"], causal=c["causal"], prefix_pages=st["prefix_pages"],
                                  prefix_length=c["prefix"])
    return {"out": out, "lse": lse}


def _run_plain(st):
    c = st["case"]
    if c["op"] == "prompt":
        out, lse = _prompt(st)
        return {"out": out, "lse": lse}
    return {"grad": _grad, "append": _append, "step": _step}[c["op"]](st)


def _scores(q, k, causal):
    """[heads, n_q, n_k] of one key/value head and its query heads, masked, in 32 bits."""
    s = (q @ k.transpose(-1, -2)) * (1 / math.sqrt(q.shape[-1]))
    if causal:
        n_q, n_k = s.shape[-2:]
        i = torch.arange(n_q, device="cuda")[:, None] + (n_k - n_q)
        s.masked_fill_(torch.arange(n_k, device="cuda") > i, -math.inf)
    return s


def _softmax(s):
    """Weights and log-sum-exp; a row that sees nothing has weights 0 and -inf."""
    if s.shape[-1] == 0:
        return s, torch.full(s.shape[:-1], -math.inf, device="cuda")
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l > 0, l, 1.0), (m + torch.log(l))[..., 0]


def _prompt(st):
    c, group = st["case"], st["case"]["H"] // st["case"]["H_kv"]
    out = torch.empty(st["q"].shape, dtype=st["q"].dtype, device="cuda")
    lse = torch.empty(c["H"], st["q"].shape[0], device="cuda")
    for a, n, b, m in _seqs(c):
        for g in range(c["H_kv"]):
            h = slice(g * group, (g + 1) * group)
            q = st["q"][a:a + n, h].float().transpose(0, 1)
            k, v = st["k"][b:b + m, g].float(), st["v"][b:b + m, g].float()
            p, lse[h, a:a + n] = _softmax(_scores(q, k, c["causal"]))
            out[a:a + n, h] = (p @ v).transpose(0, 1).to(out.dtype)
    return out, lse


def _grad(st):
    c, group, scale = st["case"], st["case"]["H"] // st["case"]["H_kv"], 1 / math.sqrt(st["case"]["d"])
    dq, dk, dv = (torch.empty(st[x].shape, dtype=st[x].dtype, device="cuda") for x in ("q", "k", "v"))
    for a, n, b, m in _seqs(c):
        for g in range(c["H_kv"]):
            h = slice(g * group, (g + 1) * group)
            q, o, do = (st[x][a:a + n, h].float().transpose(0, 1) for x in ("q", "out", "dout"))
            k, v = st["k"][b:b + m, g].float(), st["v"][b:b + m, g].float()
            lse = st["lse"][h, a:a + n, None]
            p = torch.where(lse == -math.inf, 0.0, torch.exp(_scores(q, k, c["causal"]) - lse))
            ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
            dq[a:a + n, h] = (ds @ k * scale).transpose(0, 1).to(dq.dtype)
            dk[b:b + m, g] = ((ds.transpose(-1, -2) @ q).sum(0) * scale).to(dk.dtype)
            dv[b:b + m, g] = (p.transpose(-1, -2) @ do).sum(0).to(dv.dtype)
    return {"dq": dq, "dk": dk, "dv": dv}


def _rotate(x, table, positions, c):
    """Rows x [rows, heads, d] turned by their positions' angles; in x's precision."""
    half = c["rot"] // 2
    cos, sin = (t.to(x.dtype)[:, None] for t in table[positions].split(half, 1))
    turned, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if c["interleaved"] else turned.split(half, -1)
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1)


def _append(st):
    c, lens = st["case"], _list(st["case"]["lens"])
    n = torch.tensor(lens, device="cuda")
    b = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n, output_size=sum(lens))
    slot = st["lengths"].long()[b] + torch.arange(sum(lens), device="cuda") - (torch.cumsum(n, 0) - n)[b]
    page, row = st["block_table"].long()[b, slot // c["page"]], slot % c["page"]
    q, k = (_rotate(st[x].float(), st["table"], slot, c).to(st[x].dtype) for x in ("q", "k"))
    st["k_pages"][page, :, row] = k
    st["v_pages"][page, :, row] = st["v"]
    torch.add(st["lengths"], n.int(), out=st["lengths_out"])
    return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"], "lengths": st["lengths_out"]}


def _gather(pages, table, n):
    """[H_kv, n, d] of the first n slots that a row of page numbers holds."""
    page = pages.shape[2]
    x = pages[table[:-(-n // page)].long()]
    return x.transpose(0, 1).reshape(pages.shape[1], -1, pages.shape[3])[:, :n]


def _step(st):
    c, out, lse = st["case"], [], []
    H_kv, N_q, d, P = c["H_kv"], c["N_q"], c["d"], c["prefix"]
    shared = [_gather(st[x], st["prefix_pages"], P).float() for x in ("k_pages", "v_pages")] if P else None
    for b, n in enumerate(_held(c)):
        k, v = (_gather(st[x], st["block_table"][b], n).float() for x in ("k_pages", "v_pages"))
        if P:
            k, v = torch.cat((shared[0], k), 1), torch.cat((shared[1], v), 1)
        s = (st["q"][b].float().reshape(H_kv, -1, d) @ k.transpose(-1, -2)) * (1 / math.sqrt(d))
        if c["causal"]:  # query i sees the own slots j < n - (N_q - 1 - i), and the whole prefix
            last = torch.arange(n - N_q + 1, n + 1, device="cuda").clamp(min=0)[:, None] + P
            hidden = torch.arange(P + n, device="cuda") >= last
            s = s.reshape(H_kv, -1, N_q, P + n).masked_fill(hidden, -math.inf).reshape(H_kv, -1, P + n)
        p, l = _softmax(s)
        out.append((p @ v).reshape(c["H"], N_q, d).to(st["q"].dtype))
        lse.append(l.reshape(c["H"], N_q))
    return {"out": torch.stack(out), "lse": torch.stack(lse)}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    c = case
    if work(c)["flops"] > 3.5e12:  # 64-bit products of more would take over 20 seconds
        return None
    st, f64, scale = prepare(c, seed), dict(dtype=torch.float64, device="cuda"), 1 / math.sqrt(c["d"])
    if c["op"] == "append":
        half = c["rot"] // 2
        pages = {x: st[x].double() for x in ("k_pages", "v_pages")}
        out = {"q": st["q"].double(), **pages, "lengths": st["lengths"] + torch.tensor(_list(c["lens"]), device="cuda")}
        turned = {"q": out["q"], "k": st["k"].double()}
        at = 0
        for b, (held, n) in enumerate(zip(_held(c), _list(c["lens"]))):
            cos, sin = st["table"][held:held + n, None, :half].double(), st["table"][held:held + n, None, half:].double()
            for x in turned.values():
                rows = x[at:at + n]
                a = rows[..., 0:c["rot"]:2].clone() if c["interleaved"] else rows[..., :half].clone()
                e = rows[..., 1:c["rot"]:2].clone() if c["interleaved"] else rows[..., half:c["rot"]].clone()
                first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else \
                    (slice(0, half), slice(half, c["rot"]))
                rows[..., first], rows[..., second] = cos * a - sin * e, sin * a + cos * e
            for s0 in range(held - held % c["page"], held + n, c["page"]):  # page by page
                lo, hi = max(s0, held), min(s0 + c["page"], held + n)
                page = int(st["block_table"][b, s0 // c["page"]])
                for name, x in (("k_pages", turned["k"]), ("v_pages", st["v"].double())):
                    pages[name][page, :, lo - s0:hi - s0] = x[at + lo - held:at + hi - held].transpose(0, 1)
            at += n
        return {**out, "lengths": out["lengths"].int()}
    if c["op"] == "step":
        out, lse = torch.zeros(st["q"].shape, **f64), torch.full(st["q"].shape[:3], -math.inf, **f64)
        group = c["H"] // c["H_kv"]

        def rows(pages, numbers, g, n):  # n slots of head g, page after page
            got = [pages[p, g] for p in numbers[:-(-n // c["page"])]]
            return torch.cat(got)[:n].double() if got else torch.zeros(0, c["d"], **f64)

        order = st["prefix_pages"].tolist() if c["prefix"] else []
        for b, n in enumerate(_held(c)):
            table = st["block_table"][b].tolist()
            for g in range(c["H_kv"]):
                k, v = (rows(st[x], order, g, c["prefix"]) for x in ("k_pages", "v_pages"))
                ko, vo = (rows(st[x], table, g, n) for x in ("k_pages", "v_pages"))
                for i in range(c["N_q"]):
                    seen = max(0, n - (c["N_q"] - 1 - i)) if c["causal"] else n
                    keys, vals = torch.cat((k, ko[:seen])), torch.cat((v, vo[:seen]))
                    if len(keys):
                        s = st["q"][b, g * group:(g + 1) * group, i].double() @ keys.T * scale
                        lse[b, g * group:(g + 1) * group, i] = top = torch.logsumexp(s, -1)
                        out[b, g * group:(g + 1) * group, i] = torch.exp(s - top[:, None]) @ vals
        return {"out": out, "lse": lse}
    group = c["H"] // c["H_kv"]
    out, lse = torch.zeros(st["q"].shape, **f64), torch.full((c["H"], st["q"].shape[0]), -math.inf, **f64)
    dq, dk, dv = (torch.zeros(st[x].shape, **f64) for x in ("q", "k", "v"))
    for a, n, b, m in _seqs(c):
        for h in range(c["H"]):
            k, v = st["k"][b:b + m, h // group].double(), st["v"][b:b + m, h // group].double()
            for r in range(0, n, 2048):  # rows of queries at a time, with the keys that they see
                rows = slice(a + r, a + min(n, r + 2048))
                at = torch.arange(r, min(n, r + 2048), device="cuda") + m - n if c["causal"] else \
                    torch.full((min(n - r, 2048),), m, device="cuda")
                w = max(0, min(m, int(at[-1]) + 1))
                if w == 0:
                    continue
                s = st["q"][rows, h].double() @ k[:w].T * scale
                hidden = torch.arange(w, device="cuda") > at[:, None]
                if c["op"] == "prompt":
                    lse[h, rows] = top = torch.logsumexp(s.masked_fill(hidden, -math.inf), -1)
                    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top)[:, None]).masked_fill(hidden, 0.0)
                    out[rows, h] = p @ v[:w]
                else:  # the gradient for the out and lse that are given
                    top = st["lse"][h, rows].double()
                    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top)[:, None]).masked_fill(hidden, 0.0)
                    do = st["dout"][rows, h].double()
                    ds = p * (do @ v[:w].T - (do * st["out"][rows, h].double()).sum(-1, keepdim=True)) * scale
                    dq[rows, h] = ds @ k[:w]
                    dk[b:b + w, h // group] += ds.T @ st["q"][rows, h].double()
                    dv[b:b + w, h // group] += p.T @ do
    return {"out": out, "lse": lse} if c["op"] == "prompt" else {"dq": dq, "dk": dk, "dv": dv}


# --------------------------------------------------------------------- work
def work(case):
    c, d = case, case["d"]
    if c["op"] in ("prompt", "grad"):
        pairs = 0  # visible (query, key)
        for _, n, _, m in _seqs(c):
            # row i from the last sees m - i keys under the mask
            full = min(n, m)
            pairs += full * m - full * (full - 1) // 2 if c["causal"] else n * m
        Tq, Tk = sum(s[1] for s in _seqs(c)), sum(s[3] for s in _seqs(c))
        k = 2 if c["op"] == "prompt" else 4
        return {"bytes": 2 * d * k * (c["H"] * Tq + c["H_kv"] * Tk) + 4 * c["H"] * Tq,
                "flops": (4 if c["op"] == "prompt" else 10) * d * c["H"] * pairs}
    if c["op"] == "append":  # rows in and out, and a row of the table for each token
        T = sum(_list(c["lens"]))
        return {"bytes": T * (4 * d * (c["H"] + 2 * c["H_kv"]) + 4 * c["rot"]),
                "flops": 3 * T * c["rot"] * (c["H"] + c["H_kv"])}
    held, rows = sum(_held(c)), c["B"] * c["H"] * c["N_q"]
    return {"bytes": 4 * d * c["H_kv"] * (held + c["prefix"]) + rows * (4 * d + 4),
            "flops": 4 * d * c["H"] * c["N_q"] * (held + c["B"] * c["prefix"])}
