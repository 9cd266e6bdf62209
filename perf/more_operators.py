"""The operators at both ends of a request's life, as cases that can be timed.

Three operators, which a serving loop runs before its draft-tree rounds and after them:

  prompt    dt_prompt_attention: causal attention over the packed prompts of a batch, grouped heads, each prompt (or
            chunk of one) behind the tokens that its request already has in the pages.
  logprobs  dt_token_logprobs: log probabilities of given tokens under the target's rows, with the row's entropy, the
            token's rank and the best alternatives: along a round's accepted paths, or over prompts.
  fork      dt_kv_fork / dt_kv_release_shared: requests that continue another one: whole pages shared, the last one
            copied; and pages given back by requests that share them.

With ``own`` false, ``run`` computes them from elementary torch operations; with ``own`` true it makes the library's
calls. Ragged lengths follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases --
def listed():
    return [
        # one short question to an idle server: latency
        dict(name="prompt_one", op="prompt", B=1, len=93, ragged=False, ones=False, cached=0, page=16, H_kv=8, G=4, D=128,
             dtype="bf16"),
        # a batch of prompts of different lengths, nothing cached
        dict(name="prompt_batch", op="prompt", B=16, len=2000, ragged=True, ones=False, cached=0, page=16, H_kv=8, G=4,
             D=128, dtype="bf16"),
        # one long document
        dict(name="prompt_long", op="prompt", B=1, len=16384, ragged=False, ones=False, cached=0, page=16, H_kv=8, G=4,
             D=128, dtype="bf16"),
        # chunks of long prompts behind what earlier chunks left in the pages
        dict(name="prompt_chunk", op="prompt", B=4, len=512, ragged=False, ones=False, cached=8192, page=64, H_kv=8, G=4,
             D=128, dtype="fp16"),
        # a mixed step: most requests bring one token, some a prompt; odd heads and head size, empty caches too
        dict(name="prompt_mixed", op="prompt", B=32, len=700, ragged=True, ones=True, cached=1003, page=32, H_kv=3, G=5,
             D=80, dtype="fp16"),
        # one request's next token: the smallest call
        dict(name="logprobs_one", op="logprobs", B=1, P=1, V=32000, K=0, dtype="bf16", form="path", packed=False,
             grammar=False),
        # a round's accepted paths of up to 9 positions, five alternatives each
        dict(name="logprobs_round", op="logprobs", B=8, P=61, V=128256, K=5, dtype="bf16", form="path", packed=True,
             grammar=False),
        # the rows of eight prompts, every token's log probability with one alternative
        dict(name="logprobs_prompts", op="logprobs", B=8, P=400, V=128256, K=1, dtype="bf16", form="next", packed=True,
             grammar=False),
        # fp32 rows of an odd vocabulary after a grammar, given labels, twenty alternatives
        dict(name="logprobs_stress", op="logprobs", B=16, P=65, V=128255, K=20, dtype="fp32", form="labels", packed=False,
             grammar=True),
        # one request branches: two planes, a short context
        dict(name="fork_one", op="fork", B=2, parents=1, planes=2, H=8, D=128, page=16, len=100, heads_first=False),
        # eight samples of one prompt, 32 layers
        dict(name="fork_samples", op="fork", B=8, parents=1, planes=64, H=8, D=128, page=16, len=1000, heads_first=False),
        # eight prompts with eight samples each, large pages with the heads first
        dict(name="fork_batch", op="fork", B=64, parents=8, planes=32, H=8, D=128, page=64, len=2000, heads_first=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "logprobs", "logprobs", "fork"])
    if op == "prompt":
        B = _log(rng, 1, 48)
        H_kv, G = rng.choice([(1, 8), (2, 7), (2, 16), (3, 5), (4, 1), (4, 8), (5, 4), (8, 1), (8, 2), (8, 4)])
        return dict(op=op, B=B, len=_log(rng, 1, 8000 // B), ragged=rng.random() < 0.7, ones=rng.random() < 0.3,
                    cached=_log(rng, 1, 6000) if rng.random() < 0.5 else 0, page=rng.choice([16, 32, 64, 128]), H_kv=H_kv, G=G,
                    D=rng.choice([64, 80, 96, 128, 128]), dtype=rng.choice(["bf16", "fp16"]))
    if op == "logprobs":
        form = rng.choice(["path", "next", "labels"])
        return dict(op=op, B=_log(rng, 1, 16), P=_log(rng, 1, 65) if form == "path" else _log(rng, 1, 200),
                    V=_log(rng, 1000, 152000), K=rng.choice([0, 1, rng.randint(2, 20)]), dtype=rng.choice(["bf16", "fp32"]),
                    form=form, packed=rng.random() < 0.5, grammar=rng.random() < 0.3)
    parents = _log(rng, 1, 8)
    return dict(op=op, B=parents * rng.randint(2, 8), parents=parents, planes=2 * _log(rng, 1, 16), H=rng.choice([1, 2, 3, 5, 8]),
                D=rng.choice([64, 80, 96, 128]), page=rng.choice([16, 32, 64, 128]), len=_log(rng, 1, 3000),
                heads_first=rng.random() < 0.5)


# ------------------------------------------------------------ what the case alone determines -------
def _own_rng(case):
    return random.Random(" ".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))


def _up(a, b):
    return -(-a // b)


def _offsets(n):
    off = [0]
    for k in n:
        off.append(off[-1] + k)
    return off


def _shape(case):
    """Lengths of a case: plain lists."""
    rng = _own_rng(case)
    B = case["B"]
    if case["op"] == "prompt":
        n = [rng.randint(max(1, case["len"] // 8), case["len"]) if case["ragged"] else case["len"] for _ in range(B)]
        if case["ones"]:
            n = [x if rng.random() < 0.25 else 1 for x in n]
        n[rng.randrange(B)] = case["len"]
        c = case["cached"]
        lens = [rng.randint(c // 4, c) if case["ragged"] else c for _ in range(B)]
        if c and case["ragged"] and B > 2:
            lens[:2] = [0, 1]
        return dict(n=n, lens=lens)
    if case["op"] == "logprobs":
        P = case["P"]
        used = [rng.randint(max(1, P // 4), P) for _ in range(B)]  # rows of a request
        used[rng.randrange(B)] = P
        n = [rng.randint(1, min(9, u)) for u in used] if case["form"] == "path" else used
        return dict(used=used, n=n)
    lens = [rng.randint(1, case["len"]) for _ in range(case["parents"])]
    lens[rng.randrange(case["parents"])] = case["len"]
    per = case["B"] // case["parents"]  # a parent and its forks stand next to one another
    src = [b // per * per for b in range(B) if b % per]
    dst = [b for b in range(B) if b % per]
    return dict(lens=lens, per=per, src=src, dst=dst)


def work(case):
    s = _shape(case)
    if case["op"] == "prompt":
        H_kv, G, D = case["H_kv"], case["G"], case["D"]
        rows, tokens = sum(s["n"]), sum(s["lens"])
        pairs = sum(x * k + k * (k + 1) // 2 for x, k in zip(s["lens"], s["n"]))
        nbytes = 2 * D * (2 * H_kv * (tokens + rows) + 2 * H_kv * G * rows)
        nbytes += 4 * sum(_up(x, case["page"]) for x in s["lens"])
        return {"bytes": nbytes, "flops": 4 * D * H_kv * G * pairs}
    if case["op"] == "logprobs":
        rows, V, K = sum(s["n"]), case["V"], case["K"]
        return {"bytes": rows * (V * (2 if case["dtype"] == "bf16" else 4) + 16 + 8 * K), "flops": 6 * rows * V}
    page = case["page"]
    lens = [s["lens"][p // s["per"]] for p in s["src"]]
    tails = sum(x % page for x in lens)
    entries = sum(_up(x, page) for x in lens)
    # tail rows read and written; per shared page: its entry written, its count up and down; back: entry read and cleared
    return {"bytes": 2 * tails * case["planes"] * case["H"] * case["D"] * 2 + 28 * entries, "flops": 0}


# ---------------------------------------------------------------------------------------- inputs --
class State:
    pass


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    s = State()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s.case, s.op, shape = case, case["op"], _shape(case)
    B = case["B"]

    def randn(*size, dtype):
        return torch.randn(*size, generator=g, device="cuda", dtype=dtype)

    if s.op == "prompt":
        dt_, H_kv, H, D, page = TYPES[case["dtype"]], case["H_kv"], case["H_kv"] * case["G"], case["D"], case["page"]
        s.n, s.lens = shape["n"], shape["lens"]
        off = _offsets(s.n)
        rows = off[-1] + 3  # room behind the last prompt
        s.row_off, s.seq_len = _i32(off), _i32(s.lens)
        s.q = randn(rows, H, D, dtype=dt_) * 2  # scores spread by about two, as after query and key norms
        s.k_new, s.v_new = randn(rows, H_kv, D, dtype=dt_), randn(rows, H_kv, D, dtype=dt_)
        s.out = torch.zeros(rows, H, D, dtype=dt_, device="cuda")
        s.scale = D ** -0.5
        s.k_pages = s.v_pages = s.table = None
        if case["cached"]:
            need = [_up(x, page) for x in s.lens]
            n_blocks, mb = sum(need) + 5, max(1, max(need))
            perm = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)
            e = torch.arange(mb, device="cuda")[None, :]
            first = torch.tensor(_offsets(need)[:-1], device="cuda")[:, None]
            have = e < torch.tensor(need, device="cuda")[:, None]
            s.table = torch.where(have, perm[(first + e).clamp(max=n_blocks - 1)], -1).to(torch.int32).contiguous()
            s.k_pages = randn(n_blocks, page, H_kv, D, dtype=dt_)
            s.v_pages = randn(n_blocks, page, H_kv, D, dtype=dt_)
        if own:
            import dynamic_draft_tree_gb300 as dt
            s.h = dt.Handle(B, 2, 1, 1, 1, 1)
            s.ws = dt.dt_prompt_attention_workspace(s.h, B, H, H_kv, D)
    elif s.op == "logprobs":
        V, P, K, dt_ = case["V"], case["P"], case["K"], TYPES[case["dtype"]]
        used, n = shape["used"], shape["n"]
        off = _offsets(used)
        s.n, s.used = n, used
        lead = (off[-1] + 2,) if case["packed"] else (B, P)
        s.row_off = _i32(off) if case["packed"] else None
        s.logits = randn(*lead, V, dtype=dt_) * 3
        if case["grammar"]:  # one token in four is allowed
            s.logits.masked_fill_(torch.rand(*lead, V, generator=g, device="cuda", dtype=dt_) < 0.75, -math.inf)
        s.path = s.last = None
        s.shift = 0 if case["form"] == "labels" else 1
        s.n_extra = 0
        if case["form"] == "path":  # accepted positions, root first; tokens of the tree's positions, and the bonus token
            s.n_extra = 1
            key = torch.rand(B, P, generator=g, device="cuda")
            key.masked_fill_(torch.arange(P, device="cuda")[None, :] >= _i32(used)[:, None], 2.0)
            key[:, 0] = -1.0
            S = max(n)
            s.path = key.argsort(1)[:, :S].sort(1).values.to(torch.int32).contiguous()
            for b in range(B):  # the first n of a request's are its used positions in ascending order
                s.path[b, : n[b]] = key[b].argsort()[: n[b]].sort().values.to(torch.int32)
                s.path[b, n[b]:] = -1
            s.tokens = torch.randint(0, V, (B, P), generator=g, device="cuda", dtype=torch.int32)
            out = (B, S)
        else:
            s.tokens = torch.randint(0, V, lead, generator=g, device="cuda", dtype=torch.int32)
            out = lead
        if s.shift:
            s.last = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
        s.n_new = _i32(n) - s.n_extra
        f32 = dict(dtype=torch.float32, device="cuda")
        s.logp, s.entropy = torch.zeros(*out, **f32), torch.zeros(*out, **f32)
        s.rank = torch.zeros(*out, dtype=torch.int32, device="cuda")
        s.top_ids = torch.zeros(*out, K, dtype=torch.int32, device="cuda") if K else None
        s.top_logp = torch.zeros(*out, K, **f32) if K else None
        if own:
            import dynamic_draft_tree_gb300 as dt
            s.h = dt.Handle(B, V, 1, 1, 1, 1, dt.DT_BF16 if case["dtype"] == "bf16" else dt.DT_F32)
            s.ws = dt.dt_token_logprobs_workspace(s.h, s.logp.numel(), K)
    else:
        planes, H, D, page, per = case["planes"], case["H"], case["D"], case["page"], shape["per"]
        lens = [shape["lens"][b // per] if b % per == 0 else 0 for b in range(B)]
        need = [_up(x, page) for x in lens]
        mb = max(need) + 1
        tails = sum(1 for p in shape["src"] if lens[p] % page)
        n_blocks = sum(need) + tails + 4
        pages = randn(planes, n_blocks, H, page, D, dtype=torch.bfloat16) if case["heads_first"] else \
            randn(planes, n_blocks, page, H, D, dtype=torch.bfloat16)
        s.cache = pages.transpose(2, 3) if case["heads_first"] else pages
        perm = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)
        e = torch.arange(mb, device="cuda")[None, :]
        first = torch.tensor(_offsets(need)[:-1], device="cuda")[:, None]
        s.n_owned, s.seq_len = _i32(need), _i32(lens)
        s.table = torch.where(e < s.n_owned[:, None], perm[(first + e).clamp(max=n_blocks - 1)], -1).to(torch.int32).contiguous()
        s.free_list = torch.full((n_blocks,), -1, dtype=torch.int32, device="cuda")
        s.free_list[: n_blocks - sum(need)] = perm[sum(need):]
        s.free_count = _i32([n_blocks - sum(need)])
        s.refs = torch.zeros(n_blocks, dtype=torch.int32, device="cuda")
        s.src, s.dst = _i32(shape["src"]), _i32(shape["dst"])
        s.keep = s.seq_len.clone()  # the last samples end, their parents stay
        if own:
            import dynamic_draft_tree_gb300 as dt
            s.h = dt.Handle(B, 2, 1, 1, 1, 1)
            s.pool = dt.BlockPool(s.table, s.n_owned, s.free_list, s.free_count, page)
    return s


# ------------------------------------------------------------------------------------------- run --
def run(s):
    return {"prompt": _prompt, "logprobs": _logprobs, "fork": _fork}[s.op](s)


def _prompt(s):
    if own:
        import dynamic_draft_tree_gb300 as dt
        cached = {}
        if s.table is not None:
            cached = dict(k_pages=s.k_pages, v_pages=s.v_pages, block_table=s.table, seq_len=s.seq_len)
        dt.dt_prompt_attention(s.h, s.q, s.k_new, s.v_new, s.row_off, s.out, s.ws, scale=s.scale, **cached)
        return s.out
    H, D = s.q.shape[1:]
    H_kv, page = s.k_new.shape[1], s.case["page"]
    G, r0 = H // H_kv, 0
    for b, (n, L) in enumerate(zip(s.n, s.lens)):
        k, v = s.k_new[r0: r0 + n].float(), s.v_new[r0: r0 + n].float()
        if s.table is not None and L:
            blocks = s.table[b, : _up(L, page)].long()
            k = torch.cat([s.k_pages[blocks].flatten(0, 1)[:L].float(), k])
            v = torch.cat([s.v_pages[blocks].flatten(0, 1)[:L].float(), v])
        above = None
        if n > 1:
            above = torch.ones(n, n, dtype=torch.bool, device="cuda").triu_(1)
        for h in range(H_kv):
            q = s.q[r0: r0 + n, h * G: h * G + G].float().transpose(0, 1)  # [G][n][D]
            w = torch.matmul(q, k[:, h].T).mul_(s.scale)
            if above is not None:
                w[:, :, -n:].masked_fill_(above, -math.inf)
            w = w.sub_(w.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(w, v[:, h]).div_(w.sum(-1, keepdim=True))
            s.out[r0: r0 + n, h * G: h * G + G] = o.transpose(0, 1).to(s.out.dtype)
        r0 += n
    return s.out


def _entries(s):
    """Buffer row, token and output place of every entry, requests in ascending order."""
    rows, toks, outs = [], [], []
    base = _offsets(s.used) if s.row_off is not None else [b * s.case["P"] for b in range(s.case["B"])]
    tokens = s.tokens.reshape(-1).long()
    for b, n in enumerate(s.n):
        if s.path is not None:
            pos = s.path[b, :n].long()
            rows.append(base[b] + pos)
            toks.append(torch.cat([tokens[b * s.case["P"] + pos[1:]], s.last[b: b + 1].long()]))
            outs.append(torch.arange(n, device="cuda") + b * s.path.shape[1])
        else:
            row = torch.arange(base[b], base[b] + n, device="cuda")
            rows.append(row)
            toks.append(torch.cat([tokens[row[1:]], s.last[b: b + 1].long()]) if s.shift else tokens[row])
            outs.append(row)
    return torch.cat(rows), torch.cat(toks), torch.cat(outs)


def _logprobs(s):
    if own:
        import dynamic_draft_tree_gb300 as dt
        dt.dt_token_logprobs(s.h, s.logits, s.n_new, s.logp, s.ws, tokens=s.tokens, last=s.last, shift=s.shift, n_extra=s.n_extra,
                             path=s.path, row_off=s.row_off, entropy=s.entropy, rank=s.rank, top_ids=s.top_ids,
                             top_logp=s.top_logp)
    else:
        V, K = s.case["V"], s.case["K"]
        flat = s.logits.reshape(-1, V)
        rows, toks, outs = _entries(s)
        for at in range(0, rows.numel(), 256):  # as many rows at a time as keep the temporaries moderate
            x, t, o = flat[rows[at: at + 256]].float(), toks[at: at + 256, None], outs[at: at + 256]
            d = x - x.amax(1, keepdim=True)
            e = d.exp()
            S = e.sum(1, keepdim=True)
            xt = x.gather(1, t)
            v = torch.arange(V, device="cuda")[None, :]
            s.logp.view(-1)[o] = (d.gather(1, t) - S.log())[:, 0]
            s.entropy.view(-1)[o] = (S.log() - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / S)[:, 0]
            s.rank.view(-1)[o] = ((x > xt) | ((x == xt) & (v < t))).sum(1).to(torch.int32)
            if K:
                bits = (x + 0.0).view(torch.int32)  # -0 as +0; an order of whole numbers, and the lower id first
                order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
                ids = (order * (1 << 32) - v).topk(K, dim=1).indices
                some = x.gather(1, ids) > -math.inf
                s.top_ids.view(-1, K)[o] = torch.where(some, ids, -1).to(torch.int32)
                s.top_logp.view(-1, K)[o] = torch.where(some, d.gather(1, ids) - S.log(), -math.inf)
    return [s.logp, s.entropy, s.rank] + ([s.top_ids, s.top_logp] if s.case["K"] else [])


def _fork(s):
    """The samples of the last prompts end, then those of the next ones begin. (The first call finds none to end.)"""
    if own:
        import dynamic_draft_tree_gb300 as dt
        dt.dt_kv_release_shared(s.h, s.pool, s.refs, s.keep)
        dt.dt_kv_fork(s.h, s.pool, s.refs, s.cache, s.src, s.dst, s.seq_len)
    else:
        page, (B, MB), N = s.case["page"], s.table.shape, s.refs.numel()
        e = torch.arange(MB, device="cuda")[None, :]
        # release: who gives a page back; a page that nobody keeps goes to the list, at the place of the last who gave it
        kept = torch.minimum((s.keep + page - 1) // page, s.n_owned)
        back = (e >= kept[:, None]) & (e < s.n_owned[:, None])
        block = s.table.clamp(min=0).long()
        gave = torch.zeros(N, dtype=torch.int32, device="cuda").index_add_(0, block[back], torch.ones_like(s.table[back]))
        freed = back & (gave[block] > s.refs[block])
        place = torch.arange(B * MB, device="cuda").view(B, MB)
        last = torch.full((N,), -1, device="cuda").scatter_reduce_(0, block[back], place[back], "amax")
        freed &= last[block] == place
        total = freed.sum()
        at = s.free_count + total - torch.cumsum(freed.view(-1), 0).view(B, MB)
        s.free_list[at[freed]] = s.table[freed]
        s.refs.sub_(gave).clamp_(min=0)
        s.table.masked_fill_(back, -1)
        s.n_owned.copy_(kept)
        s.free_count += total
        # fork: whole pages shared, a page of its own for the tokens of the last one
        src, dst = s.src.long(), s.dst.long()
        length = s.seq_len[src]
        full, tail = length // page, length % page
        need = (tail > 0).to(torch.int32)
        upto = torch.cumsum(need, 0)
        ok = (need == 0) | (upto <= s.free_count)
        new = s.free_list[(s.free_count - upto).clamp(min=0).long()]
        shared = (e < full[:, None]) & ok[:, None]
        table = torch.where(shared, s.table[src], -1)
        s.refs.index_add_(0, table[shared].long(), torch.ones_like(table[shared]))
        copied = ok & (need > 0)
        old = s.table[src].gather(1, full.long()[:, None])[:, 0].long()
        s.table[dst] = torch.where((e == full[:, None]) & copied[:, None], new[:, None], table)
        f, t = torch.nonzero((torch.arange(page, device="cuda")[None, :] < tail[:, None]) & copied[:, None], as_tuple=True)
        s.cache[:, new.long()[f], t] = s.cache[:, old[f], t]
        s.n_owned[dst] = torch.where(ok, full + need, s.n_owned[dst])
        s.seq_len[dst] = torch.where(ok, length, s.seq_len[dst])
        s.free_count -= torch.where(copied, need, 0).sum()
    return [s.cache, s.table, s.n_owned, s.seq_len, s.refs, s.free_list, s.free_count]


# ----------------------------------------------------------------------------------------- exact --
def exact(case, seed):
    """The definitions, one request after another, in 64 bits."""
    if case["op"] == "fork":
        return None  # whole numbers and copies
    s = prepare(case, seed)
    if case["op"] == "prompt":
        out = torch.zeros(s.out.shape, dtype=torch.float64, device="cuda")
        G, first = case["G"], 0
        for b, n in enumerate(s.n):
            L = s.lens[b]
            rows = slice(first, first + n)
            first += n
            key, val = s.k_new[rows].double(), s.v_new[rows].double()
            if L:
                at = torch.arange(L, device="cuda")
                blk = s.table[b].long()[at // case["page"]]
                key = torch.cat([s.k_pages[blk, at % case["page"]].double(), key])
                val = torch.cat([s.v_pages[blk, at % case["page"]].double(), val])
            j, i = torch.arange(L + n, device="cuda"), torch.arange(n, device="cuda")
            for x in range(s.q.shape[1]):
                for i0 in range(0, n, 2048):
                    i1 = min(n, i0 + 2048)
                    seen = L + i1  # tokens that some row of these attends to
                    z = (s.q[rows, x][i0:i1].double() * s.scale) @ key[:seen, x // G].T
                    z = torch.where(j[None, :seen] <= L + i[i0:i1, None], z, -math.inf)
                    out[rows, x][i0:i1] = torch.softmax(z, 1) @ val[:seen, x // G]
        return out
    V, K = case["V"], case["K"]
    x = s.logits.reshape(-1, V)
    f64 = dict(dtype=torch.float64, device="cuda")
    n_out = s.logp.numel()
    logp, entropy = torch.zeros(n_out, **f64), torch.zeros(n_out, **f64)
    rank = torch.zeros(n_out, dtype=torch.int64, device="cuda")
    ids, alt = torch.zeros(n_out, K, dtype=torch.int64, device="cuda"), torch.zeros(n_out, K, **f64)
    S = s.path.shape[1] if s.path is not None else case["P"]
    first = s.row_off.tolist() if s.row_off is not None else [b * case["P"] for b in range(case["B"])]
    for b, n in enumerate(s.n):
        pos = s.path[b, :n].tolist() if s.path is not None else list(range(n))
        own_tokens = s.tokens[b].tolist() if s.tokens.dim() == 2 else s.tokens[first[b]: first[b] + n].tolist()
        tok = [own_tokens[p] for p in pos]
        if s.shift:
            tok = tok[1:] + [s.last[b].item()]
        o0 = first[b] if s.path is None and s.row_off is not None else b * S
        y = x[torch.tensor([first[b] + p for p in pos], device="cuda")].double()
        t = torch.tensor(tok, device="cuda")
        z = torch.log_softmax(y, 1)
        logp[o0: o0 + n] = z[torch.arange(n, device="cuda"), t]
        entropy[o0: o0 + n] = -torch.special.xlogy(z.exp(), z.exp()).sum(1)
        ordered, by = torch.sort(y, dim=1, descending=True, stable=True)  # equal logits: the lower id first
        rank[o0: o0 + n] = (by == t[:, None]).to(torch.uint8).argmax(1)
        if K:
            some = ordered[:, :K] > -math.inf
            ids[o0: o0 + n] = torch.where(some, by[:, :K], -1)
            alt[o0: o0 + n] = torch.where(some, z.gather(1, by[:, :K]), -math.inf)
    shape = s.logp.shape
    res = [logp.view(shape), entropy.view(shape), rank.view(shape).to(torch.int32)]
    return res + ([ids.view(*shape, K).to(torch.int32), alt.view(*shape, K)] if K else [])
