"""What the dense latent attention and the page tables cost: cases, plain forms, calls.

Four operators of a serving step over the latent cache of this library:

* ``tables``   block tables, cache slots, positions and offsets of the new
               tokens from the requests' lengths (``page_tables``);
* ``dense``    latent attention in the absorbed form: every head of a token
               attends the 576-d cache rows of all positions up to its own,
               value = first 512 dims (``dense_mla``);
* ``prefix``   the same for a batch whose sequences share their first
               positions, read and multiplied once for all (``prefix_mla``);
* ``expanded`` latent attention in the expanded form: 128-d keys and values of
               each head made from the latent rows, plus the 64 RoPE dims that
               all heads share (``expanded_mla``).

Sequence b has ``q_len[b]`` new tokens at the end of its ``kv_len[b]``
positions; query i sits at t = kv_len - q_len + i and sees positions 0..t.

``run`` computes a case in its plain form (elementary torch operations in
32-bit arithmetic, sequences padded to the longest) or, with ``own`` set, by
the library's entry points.  ``exact`` restates the definitions in 64 bits, a
sequence at a time.
"""

import math
import random

import numpy as np
import torch

own = False

LATENT, VALUE, ROPE, HEAD = 576, 512, 64, 128
SCALE = 1.0 / math.sqrt(192.0)
NEG = float("-inf")


# ---------------------------------------------------------------- the cases --
def listed():
    return [
        # one decode step's bookkeeping: 64 requests of 16K-32K positions take a token each
        {"name": "tables_decode", "op": "tables", "seqs": 64, "q_lo": 1, "q_hi": 1, "before_lo": 16384,
         "before_hi": 32767, "page": 64, "pad": 0, "lengths": 1},
        # a mixed step: 500 requests, decode tokens and prompt chunks, padded to a captured graph's token count
        {"name": "tables_mixed", "op": "tables", "seqs": 500, "q_lo": 1, "q_hi": 130, "before_lo": 0,
         "before_hi": 9000, "page": 128, "pad": 777, "lengths": 2},
        # one request, one token, one rank's 16 heads of a short conversation: latency
        {"name": "dense_one", "op": "dense", "seqs": 1, "heads": 16, "q_lo": 1, "q_hi": 1, "kv_lo": 1000,
         "kv_hi": 1000, "page": 0, "lengths": 3},
        # decode on one of eight ranks: 16 heads, very uneven contexts, paged
        {"name": "dense_decode_16", "op": "dense", "seqs": 64, "heads": 16, "q_lo": 1, "q_hi": 1, "kv_lo": 1024,
         "kv_hi": 32768, "page": 64, "lengths": 4},
        # decode with all 128 heads, the 64 x 16K-32K workload of the benchmark
        {"name": "dense_decode_128", "op": "dense", "seqs": 64, "heads": 128, "q_lo": 1, "q_hi": 1, "kv_lo": 16384,
         "kv_hi": 32768, "page": 64, "lengths": 5},
        # speculative decode, 8 x 2 tokens at 128K, flat caches
        {"name": "dense_spec_128k", "op": "dense", "seqs": 8, "heads": 128, "q_lo": 2, "q_hi": 2, "kv_lo": 131072,
         "kv_hi": 131072, "page": 0, "lengths": 6},
        # a handful of requests behind a system prompt that ends inside a page
        {"name": "prefix_small", "op": "prefix", "seqs": 6, "heads": 16, "q_lo": 1, "q_hi": 1, "prefix": 1000,
         "tail_lo": 1, "tail_hi": 100, "page": 64, "lengths": 7},
        # 64 requests over one 32K document, one of eight ranks
        {"name": "prefix_doc_16", "op": "prefix", "seqs": 64, "heads": 16, "q_lo": 1, "q_hi": 1, "prefix": 32768,
         "tail_lo": 64, "tail_hi": 2048, "page": 128, "lengths": 8},
        # parallel samples of one 16K prompt with two tokens each, all heads
        {"name": "prefix_samples_128", "op": "prefix", "seqs": 32, "heads": 128, "q_lo": 2, "q_hi": 2,
         "prefix": 16384, "tail_lo": 2, "tail_hi": 512, "page": 64, "lengths": 9},
        # short ragged prompts, some after earlier turns
        {"name": "expanded_ragged", "op": "expanded", "seqs": 6, "heads": 16, "q_lo": 1, "q_hi": 500, "before_lo": 0,
         "before_hi": 700, "lengths": 10},
        # an 8K prompt on one of eight ranks
        {"name": "expanded_8k_16", "op": "expanded", "seqs": 1, "heads": 16, "q_lo": 8192, "q_hi": 8192,
         "before_lo": 0, "before_hi": 0, "lengths": 11},
        # a 4K prompt with all heads
        {"name": "expanded_4k_128", "op": "expanded", "seqs": 1, "heads": 128, "q_lo": 4096, "q_hi": 4096,
         "before_lo": 0, "before_hi": 0, "lengths": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "dense", "dense", "prefix", "expanded", "expanded"])
    seed = rng.randrange(1 << 30)
    if op == "tables":
        q = _log(rng, 1, 400)
        before = _log(rng, 1, 30000)
        return {"op": op, "seqs": _log(rng, 1, 500), "q_lo": min(q, rng.choice([0, 1, 1])), "q_hi": q, "before_lo": 0,
                "before_hi": before, "page": rng.choice([64, 128, 256]), "pad": rng.choice([0, 0, _log(rng, 1, 900)]),
                "lengths": seed}
    if op == "dense":
        seqs = _log(rng, 1, 64)
        heads = rng.choice([_log(rng, 1, 128), 16, 128])
        q = rng.choice([1, 1, 2, _log(rng, 1, 9)])
        top = max(64, min(131072, (1 << 20) // seqs, (1 << 27) // (seqs * q * heads)))
        hi = _log(rng, max(q, 16), top)
        lo = rng.choice([hi, max(q, hi // 2), q])
        return {"op": op, "seqs": seqs, "heads": heads, "q_lo": rng.choice([1, q]), "q_hi": q, "kv_lo": lo,
                "kv_hi": hi, "page": rng.choice([0, 64, 128, 192]), "lengths": seed}
    if op == "prefix":
        seqs = _log(rng, 2, 64)
        heads = rng.choice([_log(rng, 1, 128), 16, 128])
        q = rng.choice([1, 1, 2, 3])
        top = max(64, min(32768, (1 << 20) // seqs, (1 << 26) // (seqs * q * heads)))
        return {"op": op, "seqs": seqs, "heads": heads, "q_lo": 1, "q_hi": q, "prefix": _log(rng, 1, top),
                "tail_lo": q, "tail_hi": q + _log(rng, 1, 700), "page": rng.choice([64, 128]), "lengths": seed}
    seqs = _log(rng, 1, 8)
    heads = rng.choice([_log(rng, 1, 64), 16, 128])
    q = _log(rng, 1, min(4096, int(math.sqrt((1 << 29) / (seqs * heads)))))
    before = rng.choice([0, _log(rng, 1, max(1, min(8192, (1 << 29) // (seqs * heads * q))))])
    return {"op": op, "seqs": seqs, "heads": heads, "q_lo": rng.choice([1, q]), "q_hi": q, "before_lo": 0,
            "before_hi": before, "lengths": seed}


def _lengths(case):
    """(new tokens, positions already there) of every sequence: part of the case, whatever the seed."""
    rng = random.Random(case["lengths"])
    n = case["seqs"]
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(n)]
    if case["op"] in ("tables", "expanded"):
        before = [rng.randint(case["before_lo"], case["before_hi"]) for _ in range(n)]
    elif case["op"] == "dense":
        kv = [max(x, rng.randint(case["kv_lo"], case["kv_hi"])) for x in q]
        before = [k - x for k, x in zip(kv, q)]
    else:
        tail = [max(x, rng.randint(case["tail_lo"], case["tail_hi"])) for x in q]
        before = [case["prefix"] + t - x for t, x in zip(tail, q)]
    return q, before


def work(case):
    q, before = _lengths(case)
    n, rows = case["seqs"], sum(q)
    if case["op"] == "tables":
        page = case["page"]
        new = sum((b + x + page - 1) // page - (b + page - 1) // page for x, b in zip(q, before))
        # lengths in and out, offsets, free pages in and table entries out, a position and a slot a token
        return {"bytes": 4 * (4 * n + 1) + 8 * new + 12 * (rows + case["pad"]), "flops": 0}
    pairs = sum(x * b + x * (x + 1) // 2 for x, b in zip(q, before))
    keys = rows + sum(before)
    heads = case["heads"]
    if case["op"] == "expanded":
        per_key = (2 * HEAD * heads + ROPE) * 2
        per_row = heads * ((HEAD + ROPE) * 2 + HEAD * 2 + 4)
        return {"bytes": keys * per_key + rows * per_row, "flops": pairs * heads * 2 * (HEAD + ROPE + HEAD)}
    if case["op"] == "prefix":
        keys -= (n - 1) * case["prefix"]
    return {"bytes": keys * LATENT * 2 + rows * heads * (LATENT * 2 + VALUE * 2 + 4),
            "flops": pairs * heads * 2 * (LATENT + VALUE)}


# --------------------------------------------------------------- the inputs --
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, before = _lengths(case)
    n, rows = case["seqs"], sum(q)
    kv = [b + x for x, b in zip(q, before)]
    st = {"case": case, "rows": rows, "max_q": max(q), "max_kv": max(kv), "kept": {}}
    cu = np.concatenate([[0], np.cumsum(q)])
    page = case.get("page", 0)
    if case["op"] == "tables":
        have = [(b + page - 1) // page for b in before]
        blocks = max((k + page - 1) // page for k in kv) + 1
        need = sum((k + page - 1) // page for k in kv)
        pages = need + 7
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        held = sum(have)
        mine = np.arange(blocks)[None, :] < np.array(have)[:, None]
        table = torch.full((n, blocks), -1, dtype=torch.int32, device="cuda")
        table[torch.from_numpy(mine).cuda()] = order[:held]
        cap = rows + case["pad"]
        st.update(q_len=_ints(q), before=_ints(before), free=order[held:].contiguous(), table=table, cap=cap,
                  cu_q=_ints([0] * (n + 1)), kv_len=_ints([0] * n), pos=_ints([0] * cap),
                  slots=_ints([0] * cap, torch.int64), used=_ints([0]))
        return st

    heads = case["heads"]
    st.update(cu_q=_ints(cu.tolist()), kv_len=_ints(kv), q_len=_ints(q), page=page)
    if page:
        prefix = case.get("prefix", 0)
        whole = prefix // page                       # pages that all sequences share
        blocks = [(k + page - 1) // page for k in kv]
        pages = whole + sum(b - whole for b in blocks) + 5
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).cpu().numpy()
        table = np.full((n, max(blocks)), -1, np.int32)
        table[:, :whole] = order[:whole]
        own_pages = np.arange(table.shape[1])[None, :] < np.array(blocks)[:, None]
        own_pages[:, :whole] = False
        table[own_pages] = order[whole:whole + int(own_pages.sum())]
        st["keys"] = pages * page
        st["table"] = torch.from_numpy(table).cuda()
        st["start"] = None
    else:
        start = np.concatenate([[0], np.cumsum(np.array(kv) + 3)[:-1]])     # a few spare rows between sequences
        st["keys"] = int(start[-1]) + kv[-1]
        st["start"] = _ints(start.tolist(), torch.int64)
    st["cache"] = _normal(gen, st["keys"], LATENT)
    if case["op"] == "prefix" and case["prefix"] % page:
        # the prefix ends inside a page: every sequence's own page begins with a copy of those rows
        rest = case["prefix"] % page
        firsts = st["table"][:, case["prefix"] // page].long() * page
        at = firsts[:, None] + torch.arange(rest, device="cuda")
        st["cache"][at] = st["cache"][at[0]].clone()
    if case["op"] == "expanded":
        st["q"] = _normal(gen, rows, heads, HEAD + ROPE)
        st["kv_up"] = _normal(gen, st["keys"], heads, 2 * HEAD)
        st["out"] = torch.empty((rows, heads, HEAD), dtype=torch.bfloat16, device="cuda")
    else:
        st["q"] = _normal(gen, rows, heads, LATENT)
        st["out"] = torch.empty((rows, heads, VALUE), dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty((rows, heads), dtype=torch.float32, device="cuda")
    return st


# ------------------------------------------------------------ the plain forms --
def _padded(st):
    """Row of the caches for position s of every sequence [n, max_kv], row of q for its i-th token [n, max_q] (any
    row where there is none), whether token i sees position s [n, max_q, max_kv], which tokens there are."""
    n, mq, mk, page = st["case"]["seqs"], st["max_q"], st["max_kv"], st["page"]
    s = torch.arange(mk, device="cuda")
    i = torch.arange(mq, device="cuda")
    kv, q_len, cu = st["kv_len"].long(), st["q_len"].long(), st["cu_q"].long()
    if page:
        at = st["table"].long()[:, s // page].clamp(min=0) * page + s % page
    else:
        at = (st["start"][:, None] + s).clamp(max=st["keys"] - 1)
    qat = (cu[:n, None] + i).clamp(max=max(st["rows"] - 1, 0))
    t = kv[:, None] - q_len[:, None] + i
    there = i < q_len[:, None]
    sees = (s <= t[:, :, None]) & there[:, :, None]
    return at, qat, sees, there


def _plain_softmax(x, sees):
    """exp(x - max) where seen (in place), its sums and the log-sum-exp, over the last dim."""
    x.masked_fill_(~sees, NEG)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == NEG, torch.zeros_like(m), m)).exp_()
    l = x.sum(-1, keepdim=True)
    return x, l, (m + l.log())[..., 0]


def _plain_dense(st):
    at, qat, sees, there = _padded(st)
    n, mq, heads = at.shape[0], qat.shape[1], st["q"].shape[1]
    c = st["cache"][at].float()                                           # [n, max_kv, 576]
    q = st["q"][qat].float().reshape(n, mq * heads, LATENT)
    x = torch.matmul(q, c.transpose(1, 2)).mul_(SCALE).view(n, mq, heads, -1)
    p, l, lse = _plain_softmax(x, sees[:, :, None, :])
    o = torch.matmul(p.view(n, mq * heads, -1), c[..., :VALUE]).view(n, mq, heads, VALUE).div_(l)
    return {"out": o[there].to(torch.bfloat16), "lse": lse[there]}


def _plain_expanded(st):
    at, qat, sees, there = _padded(st)
    up = st["kv_up"][at]                                                  # [n, max_kv, heads, 256]
    rope = st["cache"][at, VALUE:].float()                                # [n, max_kv, 64]
    q = st["q"][qat].float().transpose(1, 2)                              # [n, heads, max_q, 192]
    x = torch.matmul(q[..., :HEAD], up[..., :HEAD].float().permute(0, 2, 3, 1))
    x += torch.matmul(q[..., HEAD:], rope.transpose(1, 2)[:, None])
    p, l, lse = _plain_softmax(x.mul_(SCALE), sees[:, None])
    o = torch.matmul(p, up[..., HEAD:].float().transpose(1, 2)).div_(l)   # [n, heads, max_q, 128]
    return {"out": o.transpose(1, 2)[there].to(torch.bfloat16), "lse": lse.transpose(1, 2)[there]}


def _plain_tables(st):
    page, cap, n = st["case"]["page"], st["cap"], st["case"]["seqs"]
    q_len, before = st["q_len"].long(), st["before"].long()
    kv = before + q_len
    cu = torch.cat([q_len.new_zeros(1), q_len.cumsum(0)])
    have, upto = (before + page - 1) // page, (kv + page - 1) // page
    first = (upto - have).cumsum(0) - (upto - have)                       # pages taken by earlier sequences
    j = torch.arange(st["table"].shape[1], device="cuda")
    new = (j >= have[:, None]) & (j < upto[:, None])
    take = (first[:, None] + j - have[:, None]).clamp(0, st["free"].numel() - 1)
    table = torch.where(new, st["free"][take], st["table"])
    r = torch.arange(cap, device="cuda")
    seq = torch.searchsorted(cu[1:], r, right=True).clamp(max=n - 1)
    pos = before[seq] + r - cu[seq]
    there = r < cu[-1]
    pos = torch.where(there, pos, torch.zeros_like(pos))
    slots = torch.where(there, table[seq, pos // page].long() * page + pos % page, torch.full_like(pos, -1))
    return {"table": table, "cu_q": cu.int(), "kv_len": kv.int(), "pos": pos.int(), "slots": slots,
            "used": (upto - have).sum().reshape(1).int()}


# ------------------------------------------------------ the library's calls --
def _batch(dsa, st, op):
    """The batch descriptor and the workspace, made once as a serving loop keeps them."""
    kept = st["kept"]
    if "batch" not in kept:
        kept["batch"] = dsa.Batch(st["cu_q"], st["kv_len"], st["start"], st["rows"], st["max_q"], st["max_kv"],
                                  st["keys"], block_table=st.get("table"), page_size=st["page"])
        kept["ws"] = dsa.workspace(op, kept["batch"], n_heads=st["q"].shape[1])
    return kept["batch"], kept["ws"]


def _own(st):
    import long_context_sparse_lightning_b200 as dsa
    case = st["case"]
    if case["op"] == "tables":
        if "ws" not in st["kept"]:
            st["kept"]["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        dsa.page_tables(st["q_len"], st["before"], st["free"], case["page"], st["table"], st["cu_q"], st["kv_len"],
                        st["pos"], st["slots"], st["used"], st["kept"]["ws"])
        return {k: st[k] for k in ("table", "cu_q", "kv_len", "pos", "slots", "used")}
    if case["op"] == "dense":
        batch, ws = _batch(dsa, st, dsa.OP_DENSE_MLA)
        dsa.dense_mla(batch, st["q"], st["cache"], SCALE, st["out"], st["lse"], ws)
    elif case["op"] == "prefix":
        batch, ws = _batch(dsa, st, dsa.OP_PREFIX_MLA)
        dsa.prefix_mla(batch, case["prefix"], st["q"], st["cache"], SCALE, st["out"], st["lse"], ws)
    else:
        batch, ws = _batch(dsa, st, dsa.OP_EXPANDED_MLA)
        dsa.expanded_mla(batch, st["q"], st["kv_up"], st["cache"][:, VALUE:], SCALE, st["out"], st["lse"], ws)
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "tables":
        return _plain_tables(state)
    return _plain_expanded(state) if op == "expanded" else _plain_dense(state)


# ------------------------------------------------------------ in 64 bits --
def exact(case, seed):
    st = prepare(case, seed)
    q_len, before = _lengths(case)
    if case["op"] == "tables":
        return _exact_tables(case, st, q_len, before)
    heads, page = case["heads"], st["page"]
    out, lse, row = [], [], 0
    for b, (n, pre) in enumerate(zip(q_len, before)):
        pos = torch.arange(pre + n, device="cuda")
        if page:
            at = st["table"][b].long()[pos // page] * page + pos % page
        else:
            at = st["start"][b] + pos
        hidden = pos[None, :] > (pre + torch.arange(n, device="cuda"))[:, None]
        rows = st["cache"][at].double()
        o = torch.empty((n, heads, st["out"].shape[2]), dtype=torch.float64, device="cuda")
        z = torch.empty((n, heads), dtype=torch.float64, device="cuda")
        for h in range(heads):
            q = st["q"][row:row + n, h].double()
            if case["op"] == "expanded":
                up = st["kv_up"][at, h].double()
                keys, values = torch.cat([up[:, :HEAD], rows[:, VALUE:]], 1), up[:, HEAD:]
            else:
                keys, values = rows, rows[:, :VALUE]
            x = (q @ keys.T / math.sqrt(192.0)).masked_fill(hidden, NEG)
            z[:, h] = torch.logsumexp(x, 1)
            o[:, h] = torch.softmax(x, 1) @ values
        out.append(o)
        lse.append(z)
        row += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_tables(case, st, q_len, before):
    page = case["page"]
    table, free = st["table"].cpu().tolist(), st["free"].cpu().tolist()
    cu, pos, slots, used = [0], [], [], 0
    for b, (n, pre) in enumerate(zip(q_len, before)):
        for p in range(pre, pre + n):
            if p % page == 0:
                table[b][p // page] = free[used]
                used += 1
            pos.append(p)
            slots.append(table[b][p // page] * page + p % page)
        cu.append(cu[-1] + n)
    kv = [n + p for n, p in zip(q_len, before)]
    pos += [0] * case["pad"]
    slots += [-1] * case["pad"]
    return {"table": torch.tensor(table), "cu_q": torch.tensor(cu), "kv_len": torch.tensor(kv),
            "pos": torch.tensor(pos), "slots": torch.tensor(slots), "used": torch.tensor([used])}
