"""What the prompt-side operators of the paged KV cache cost, case by case.

Four operators bring requests into the paged cache that tree decoding reads: the page plan (block tables and slot
maps from request lengths), the append of new K/V rows to their slots, causal attention over packed whole prompts,
and causal attention of chunks of new tokens (one token: plain decoding) over the paged cache.

With ``own`` false every pass runs the operators' plain form: elementary torch operations in 32 bits.  With ``own``
true it makes the calls a user makes: a ``PromptStep`` (buffers allocated once for a batch capacity) whose methods
issue one library call each.
"""
import math

import torch

own = False

# Head layouts and page sizes are those of the repository's workloads (32/8 and 64/8 heads of 128, 4/4 of 64; pages
# of 16 and 64 rows), prefix lengths those of its prefixes (1024 to 131072).


def listed():
    return [
        # --- kv_page_plan: one launch per scheduler step
        # 64 sequences in decode: each gets room for a committed path of 5, some finish and give their pages back
        {"name": "plan_decode_b64", "op": "plan", "B": 64, "prefix": 1024, "new": 0, "room": 5, "page": 16,
         "finished": 5, "spread": True},
        # a full scheduler step: 300 requests, prompts of very different lengths beside decoding sequences
        {"name": "plan_mixed_b300", "op": "plan", "B": 300, "prefix": 2048, "new": 700, "room": 5, "page": 16,
         "finished": 23, "spread": True},
        # --- kv_append_paged: once per layer
        # the new token of each of 64 decoding sequences
        {"name": "append_decode_b64", "op": "append", "dtype": "bf16", "N": 64, "Hkv": 8, "D": 128, "page": 16,
         "fused": False},
        # a 32k prompt, K and V read out of the fused projection's rows, some rows refused (slot -1)
        {"name": "append_prompt_32k", "op": "append", "dtype": "bf16", "N": 32768, "Hkv": 8, "D": 128, "page": 16,
         "fused": True},
        # --- prompt_attention
        # one short fp32 batch (the tiny workload's heads), odd lengths
        {"name": "prompt_f32_tiny", "op": "prompt", "dtype": "f32", "B": 3, "len": 149, "Hq": 4, "Hkv": 4, "D": 64,
         "spread": True},
        # one llama8b prompt of 2048 tokens
        {"name": "prompt_2k", "op": "prompt", "dtype": "bf16", "B": 1, "len": 2048, "Hq": 32, "Hkv": 8, "D": 128,
         "spread": False},
        # a packed batch of prompts between one and 4096 tokens, odd lengths
        {"name": "prompt_packed_b16", "op": "prompt", "dtype": "bf16", "B": 16, "len": 4096, "Hq": 32, "Hkv": 8,
         "D": 128, "spread": True},
        # one long prompt
        {"name": "prompt_32k", "op": "prompt", "dtype": "bf16", "B": 1, "len": 32768, "Hq": 32, "Hkv": 8, "D": 128,
         "spread": False},
        # --- chunk_attention_paged
        # one new token per sequence, 8 sequences of the ragged_paged_b8 workload's lengths
        {"name": "decode_b8", "op": "chunk", "dtype": "bf16", "B": 8, "new": 1, "prefix": 8192, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 16, "spread": True},
        # one new token over one 128k prefix
        {"name": "decode_128k", "op": "chunk", "dtype": "bf16", "B": 1, "new": 1, "prefix": 131071, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "spread": False},
        # a chunk of 1024 tokens of a long prompt whose first 32k are cached (64 query heads)
        {"name": "chunk_1k_over_32k", "op": "chunk", "dtype": "bf16", "B": 1, "new": 1024, "prefix": 32768, "Hq": 64,
         "Hkv": 8, "D": 128, "page": 16, "spread": False},
        # a mixed step: 24 sequences, chunks of one to 1024 tokens over prefixes of nothing to 8192
        {"name": "chunk_mixed_b24", "op": "chunk", "dtype": "bf16", "B": 24, "new": 1024, "prefix": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 16, "spread": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "prompt", "prompt", "chunk", "chunk", "chunk"])
    page = rng.choice([8, 16, 16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 300)
        return {"op": "plan", "B": B, "prefix": _log(rng, 1, 8192), "new": rng.choice([0, _log(rng, 1, 1024)]),
                "room": rng.randint(0, 8), "page": page, "finished": rng.randint(0, B // 3), "spread": True}
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    if op == "append":
        return {"op": "append", "dtype": dtype, "N": _log(rng, 1, 16384), "Hkv": Hkv, "D": D, "page": page,
                "fused": rng.random() < 0.5}
    Hq = Hkv * rng.choice([1, 3, 4, 4, 5, 7, 8])
    B = _log(rng, 1, 32)
    few = dtype == "f32"
    if op == "prompt":
        return {"op": "prompt", "dtype": dtype, "B": B, "len": _log(rng, 1, (1024 if few else 16384) // B), "Hq": Hq,
                "Hkv": Hkv, "D": D, "spread": rng.random() < 0.7}
    new = rng.choice([1, rng.randint(1, 8), _log(rng, 1, (256 if few else 2048) // B)])
    return {"op": "chunk", "dtype": dtype, "B": B, "new": new, "prefix": _log(rng, 1, (8192 if few else 65536) // B),
            "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "spread": rng.random() < 0.7}


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _lengths(n, top, spread, low, gen):
    """n lengths: all `top`, or spread over [low, top] by their logarithm, the first of them `top`."""
    if not spread:
        return [top] * n
    u = torch.rand(n, generator=gen, dtype=torch.float64).tolist()
    lo = max(low, 1)
    got = [max(low, min(top, int(round(lo * (max(top, 1) / lo) ** x)) if top else 0)) for x in u]
    return [top] + got[1:]


def _shape(case):
    """The lengths of a case: prefix and new tokens of each sequence (from the case alone)."""
    gen = torch.Generator().manual_seed(20)
    if case["op"] == "prompt":
        return [0] * case["B"], _lengths(case["B"], case["len"], case["spread"], 1, gen)
    prefix = _lengths(case["B"], case["prefix"], case["spread"], min(64, case["prefix"]), gen)
    if case["op"] == "plan":
        new = _lengths(case["B"], case["new"], case["spread"], 0, gen)
        for b in range(case["B"]):  # finished sequences, and every third one decodes beside the prompts
            if b % 3 == 2 and new[b] > 1:
                new[b] = 1
            elif b % 3 == 1 and new[b] > 1:
                prefix[b] = 0
        for b in range(case["finished"]):
            new[(b * 3 + 1) % case["B"]] = -1
        return prefix, new
    new = _lengths(case["B"], case["new"], case["spread"] and case["new"] > 8, 1, gen)
    if case["spread"]:  # a request's first chunk has nothing cached
        prefix[-1] = 0 if case["B"] > 2 else prefix[-1]
    return prefix, new


def _pages(n, page):
    return -(-n // page)


def _randn(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _starts(new):
    row = [0]
    for n in new:
        row.append(row[-1] + max(n, 0))
    return row


def _step(case, **kw):
    if not own:
        return None
    from medusa_tree_speculative_heads_b200 import api
    return api.PromptStep(**kw)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    st = {"case": case}
    if case["op"] == "append":
        N, Hkv, D, page, dt = case["N"], case["Hkv"], case["D"], case["page"], _dtype(case)
        num_pages = _pages(N, page) + 9
        if case["fused"]:  # rows of a projection that holds Q (4 heads a group), K and V
            rows = _randn((N, Hkv * 6, D), gen, dt)
            st["k"], st["v"] = rows[:, Hkv * 4:Hkv * 5], rows[:, Hkv * 5:]
        else:
            st["k"], st["v"] = _randn((N, Hkv, D), gen, dt), _randn((N, Hkv, D), gen, dt)
        st["k_pages"], st["v_pages"] = (_randn((num_pages, Hkv, page, D), gen, dt) for _ in range(2))
        # a prompt's tokens run through pages taken in any order; the first page is entered in its middle
        perm = torch.randperm(num_pages, generator=gen, device="cuda")
        pos = torch.arange(N, device="cuda") + page // 2
        slot = perm[pos // page] * page + pos % page
        st["slot_map"] = torch.where(torch.arange(N, device="cuda") % 1021 == 1020, -1, slot)
        st["step"] = _step(case, B=1, Hq=Hkv, Hkv=Hkv, D=D, max_tokens=N, dtype=dt, page_size=page,
                           max_pages=num_pages, num_pages=num_pages)
        return st
    prefix, new = _shape(case)
    row = _starts(new)
    st["prefix"], st["new"], st["row"] = prefix, new, row
    if case["op"] == "plan":
        B, page, room = case["B"], case["page"], case["room"]
        have = [_pages(p, page) for p in prefix]  # the pages of the cached positions are owned
        max_pages = max(_pages(p + max(n, 0) + room, page) for p, n in zip(prefix, new)) + 1
        grow = sum(_pages(p + max(n, 0) + room, page) - h for p, n, h in zip(prefix, new, have))
        num_pages = sum(have) + grow + 7
        perm = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(max_pages, device="cuda")[None] < ints(have)[:, None]
        table[at] = perm[:sum(have)]
        free = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
        free[:num_pages - sum(have)] = perm[sum(have):]
        st.update(prefix_len=ints(prefix), new_len=ints(new), block_table=table, owned=ints(have), free_list=free,
                  free_count=ints([num_pages - sum(have)]), max_tokens=max(row[-1], 1),
                  owned_out=ints([0] * B), free_count_out=ints([0]))
        st["step"] = _step(case, B=B, Hq=1, Hkv=1, D=64, max_tokens=st["max_tokens"], dtype=torch.bfloat16,
                           page_size=page, max_pages=max_pages, num_pages=num_pages, room=room)
        return st
    B, N, Hq, Hkv, D, dt = case["B"], row[-1], case["Hq"], case["Hkv"], case["D"], _dtype(case)
    st["q"] = _randn((N, Hq, D), gen, dt)
    st["row_start"] = ints(row)
    if case["op"] == "prompt":
        st["k"], st["v"] = _randn((N, Hkv, D), gen, dt), _randn((N, Hkv, D), gen, dt)
        st["step"] = _step(case, B=B, Hq=Hq, Hkv=Hkv, D=D, max_tokens=N, dtype=dt, max_new=max(new), want_lse=True)
        return st
    page = case["page"]
    need = [_pages(p + n, page) for p, n in zip(prefix, new)]
    num_pages, max_pages = sum(need) + 3, max(need)
    perm = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max_pages, device="cuda")[None] < ints(need)[:, None]] = perm[:sum(need)]
    st["k_pages"], st["v_pages"] = (_randn((num_pages, Hkv, page, D), gen, dt) for _ in range(2))
    st["block_table"], st["prefix_len"] = table, ints(prefix)
    st["step"] = _step(case, B=B, Hq=Hq, Hkv=Hkv, D=D, max_tokens=N, dtype=dt, page_size=page, max_pages=max_pages,
                       num_pages=num_pages, max_new=max(new), max_prefix=max(prefix), want_lse=True)
    return st


def run(st):
    op, step = st["case"]["op"], st["step"]
    if not own:
        return {"plan": _plan, "append": _append, "prompt": _prompt, "chunk": _chunk}[op](st)
    if op == "plan":
        step.plan(st["prefix_len"], st["new_len"], st["block_table"], st["owned"], st["free_list"], st["free_count"],
                  owned_out=st["owned_out"], free_count_out=st["free_count_out"])
        return {"row_start": step.row_start, "slot_map": step.slot_map, "block_table": st["block_table"],
                "owned": st["owned_out"], "free_count": st["free_count_out"], "free_list": st["free_list"]}
    if op == "append":
        step.append(st["k"], st["v"], st["k_pages"], st["v_pages"], slot_map=st["slot_map"])
        return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    if op == "prompt":
        step.prompt_attention(st["q"], st["k"], st["v"], row_start=st["row_start"])
    else:
        step.chunk_attention(st["q"], st["k_pages"], st["v_pages"], st["block_table"], st["prefix_len"],
                             row_start=st["row_start"])
    return {"out": step.out, "lse": step.lse}


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _plan(st):
    page, room = st["case"]["page"], st["case"]["room"]
    prefix, new, owned, table = st["prefix_len"].long(), st["new_len"].long(), st["owned"].long(), st["block_table"]
    B, max_pages = table.shape
    num_pages = st["free_list"].numel()
    gone, rows = new < 0, new.clamp(min=0)
    row_start = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    # released pages go on the stack, sequence by sequence
    col = torch.arange(max_pages, device=table.device)[None]
    back = (col < owned[:, None]) & gone[:, None]
    rank = back.reshape(-1).long().cumsum(0) - 1
    at = torch.where(back.reshape(-1), st["free_count"].long() + rank, num_pages)
    stack = torch.cat([st["free_list"], st["free_list"].new_zeros(1)]).scatter(0, at, table.reshape(-1))
    stack = stack[:num_pages]
    avail = st["free_count"].long() + back.sum()
    # growth, taken from the top of the stack
    want = (prefix + rows + room + page - 1) // page
    fits = want <= max_pages
    grow = torch.where(gone | ~fits, 0, (want - owned).clamp(min=0))
    off = grow.cumsum(0) - grow
    served = ~gone & fits & ((grow == 0) | (off + grow <= avail))
    grow = torch.where(served, grow, 0)
    fresh = (col >= owned[:, None]) & (col < (owned + grow)[:, None])
    src = (avail - 1 - (off[:, None] + col - owned[:, None])).clamp(0, num_pages - 1)
    table = torch.where(fresh, stack[src], table)
    owned_out = torch.where(gone, 0, owned + grow)
    # slots of the packed new tokens
    t = torch.arange(st["max_tokens"], device=table.device)
    b = torch.searchsorted(row_start[1:], t, right=True).clamp(max=B - 1)
    pos = prefix[b] + t - row_start[b]
    slot = table[b, (pos // page).clamp(0, max_pages - 1)].long() * page + pos % page
    slot = torch.where((t < row_start[-1]) & served[b], slot, -1)
    return {"row_start": row_start.int(), "slot_map": slot, "block_table": table, "owned": owned_out.int(),
            "free_count": (avail - grow.sum()).int(), "free_list": stack}


def _append(st):
    page = st["case"]["page"]
    rows = (st["slot_map"] >= 0).nonzero()[:, 0]
    slot = st["slot_map"][rows]
    st["k_pages"][slot // page, :, slot % page] = st["k"][rows]
    st["v_pages"][slot // page, :, slot % page] = st["v"][rows]
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}


_BLOCK_BYTES = 4 << 30  # scores held at once


def _attend(q, k, v, pos, scale):
    """q [..., n, D] at positions pos [..., n], keys k, v [..., m, D] at 0 .. m: output and log-sum-exp."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    hidden = torch.arange(k.shape[-2], device=k.device) > pos[..., None]
    s = s.masked_fill_(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s.sub_(top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / total, (top + torch.log(total))[..., 0]


def _one(q, k, v, first):
    """One sequence: q [n, Hq, D] at positions first .., k, v [Hkv, m, D] (32 bits); rows taken in blocks."""
    n, Hq, D = q.shape
    Hkv, m, _ = k.shape
    out = torch.empty((n, Hq, D), device=q.device)
    lse = torch.empty((n, Hq), device=q.device)
    rows = max(1, min(n, _BLOCK_BYTES // (4 * Hq * m)))
    for r in range(0, n, rows):
        blk = q[r:r + rows].float().reshape(-1, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
        pos = torch.arange(first + r, first + r + blk.shape[2], device=q.device)
        o, l = _attend(blk, k[:, None], v[:, None], pos, D ** -0.5)
        out[r:r + rows] = o.permute(2, 0, 1, 3).reshape(-1, Hq, D)
        lse[r:r + rows] = l.permute(2, 0, 1).reshape(-1, Hq)
    return out.to(q.dtype), lse


def _prompt(st):
    outs = [_one(st["q"][a:b], st["k"][a:b].float().transpose(0, 1), st["v"][a:b].float().transpose(0, 1), 0)
            for a, b in zip(st["row"], st["row"][1:])]
    return {"out": torch.cat([o for o, _ in outs]), "lse": torch.cat([l for _, l in outs])}


def _gathered(pages, table):
    """[..., n] page ids -> [..., Hkv, n * page, D] in 32 bits."""
    got = pages[table.long().clamp(min=0)].float().transpose(-4, -3)
    return got.reshape(*got.shape[:-3], -1, got.shape[-1])


def _chunk(st):
    Hq, Hkv, D, page = (st["case"][x] for x in ("Hq", "Hkv", "D", "page"))
    prefix, new, row = st["prefix"], st["new"], st["row"]
    top = max(p + n for p, n in zip(prefix, new))
    if len(set(new)) == 1 and len(new) * Hkv * top * (Hq // Hkv * new[0] + 2 * D) * 4 <= _BLOCK_BYTES:
        # the same few tokens for every sequence: one padded batch
        n = new[0]
        used = st["block_table"][:, :_pages(top, page)]
        k, v = _gathered(st["k_pages"], used), _gathered(st["v_pages"], used)  # [B, Hkv, m, D]
        real = torch.arange(k.shape[2], device=k.device) < (st["prefix_len"] + n)[:, None]
        v = v * real[:, None, :, None]
        q = st["q"].float().reshape(-1, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
        pos = (st["prefix_len"][:, None] + torch.arange(n, device=k.device))[:, None, None]
        o, l = _attend(q, k[:, :, None], v[:, :, None], pos, D ** -0.5)
        return {"out": o.permute(0, 3, 1, 2, 4).reshape(-1, Hq, D).to(st["q"].dtype),
                "lse": l.permute(0, 3, 1, 2).reshape(-1, Hq)}
    outs = []
    for b in range(len(new)):
        used = st["block_table"][b, :_pages(prefix[b] + new[b], page)]
        m = prefix[b] + new[b]
        outs.append(_one(st["q"][row[b]:row[b + 1]], _gathered(st["k_pages"], used)[:, :m],
                         _gathered(st["v_pages"], used)[:, :m], prefix[b]))
    return {"out": torch.cat([o for o, _ in outs]), "lse": torch.cat([l for _, l in outs])}


# ----------------------------------------------------------------------------
# work, and the definition in 64 bits
# ----------------------------------------------------------------------------

def work(case):
    if case["op"] == "append":
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["N"] * (8 + 4 * case["Hkv"] * case["D"] * e), "flops": 0}
    prefix, new = _shape(case)
    N = sum(max(n, 0) for n in new)
    if case["op"] == "plan":
        page, room = case["page"], case["room"]
        pages = sum(abs(_pages(p + max(n, 0) + room, page) - _pages(p, page)) if n >= 0 else _pages(p, page)
                    for p, n in zip(prefix, new))
        # lengths and owned counts in and out, row starts, each moved page read and written, each slot written
        return {"bytes": case["B"] * 20 + 16 + 8 * pages + 8 * N, "flops": 0}
    e = 4 if case["dtype"] == "f32" else 2
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    keys = sum(p + n for p, n in zip(prefix, new))
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(prefix, new))
    table = 4 * sum(_pages(p + n, case["page"]) for p, n in zip(prefix, new)) if case["op"] == "chunk" else 0
    return {"bytes": e * D * (2 * N * Hq + 2 * keys * Hkv) + 4 * N * Hq + table + 4 * (2 * case["B"] + 1),
            "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    """Attention from its definition in 64 bits, one sequence and query head at a time; the append as rows of the
    pool laid out slot by slot.  The page plan moves whole numbers."""
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        got = {}
        keep = st["slot_map"] != -1
        for rows, pool in (("k", "k_pages"), ("v", "v_pages")):
            slots = st[pool].double().transpose(1, 2).reshape(-1, case["Hkv"], case["D"])
            slots.index_copy_(0, st["slot_map"][keep], st[rows].double()[keep])
            got[pool] = slots.reshape(-1, case["page"], case["Hkv"], case["D"]).transpose(1, 2).contiguous()
        return got
    group = case["Hq"] // case["Hkv"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["new"]):
        r0, m = st["row"][b], st["prefix"][b] + n
        at = torch.arange(m, device="cuda")
        for g in range(case["Hkv"]):
            if case["op"] == "prompt":
                k, v = st["k"][r0:r0 + n, g].double(), st["v"][r0:r0 + n, g].double()
            else:
                page = st["block_table"][b].long()[at // case["page"]]
                k, v = (st[x][page, g, at % case["page"]].double() for x in ("k_pages", "v_pages"))
            for h in range(g * group, (g + 1) * group):
                for i in range(0, n, 4096):
                    q = st["q"][r0 + i:r0 + min(i + 4096, n), h].double()
                    last = st["prefix"][b] + i + q.shape[0]  # no row of this block sees a later key
                    score = (q @ k[:last].T) / math.sqrt(case["D"])
                    seen = at[:last][None] <= (last - q.shape[0] + torch.arange(q.shape[0], device="cuda"))[:, None]
                    score[~seen] = -math.inf
                    z = torch.logsumexp(score, 1)
                    lse[r0 + i:r0 + i + q.shape[0], h] = z
                    out[r0 + i:r0 + i + q.shape[0], h] = torch.exp(score - z[:, None]) @ v[:last]
    return {"out": out, "lse": lse}
