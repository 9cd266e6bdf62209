"""The operators around the target model's verify forward, as cases that can be timed.

Four operators, which a serving loop runs next to the draft-tree round:

  attend   dt_tree_attention: the tree's query rows against a paged KV cache and the tree's own keys
           and values under the ancestor mask; a prefix that all requests share is read once for all.
  logits   dt_logits_process: penalties for repeated tokens (history counts and the row's own tree
           path), sparse biases and grammar bit masks on the target rows, before dt_verify.
  reserve  dt_kv_reserve / dt_kv_release: pages for the tokens to come, block tables and slot maps.
  commit   dt_commit_kv_paged: the accepted positions' KV rows moved into the pages of the slot map.

With ``own`` false, ``run`` computes them from elementary torch operations; with ``own`` true it makes
the library's calls. Ragged lengths and tree shapes follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

SEEN = 0x40000000  # a token of the prompt, in a counts entry (the low bits count generated tokens)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases --
def listed():
    return [
        # one request, one new token, a short context: the latency of a decode step
        dict(name="attend_one", op="attend", B=1, P=1, tree=False, packed=False, len=511, ragged=False, shared=0,
             page=16, H_kv=8, G=4, D=128, dtype="bf16", holes=False),
        # a full batch decoding single tokens over long contexts: the cache's bandwidth
        dict(name="attend_decode", op="attend", B=64, P=1, tree=False, packed=False, len=8192, ragged=True, shared=0,
             page=16, H_kv=8, G=4, D=128, dtype="bf16", holes=False),
        # the CAST batch: trees of up to 60 nodes, padding-free rows, contexts up to 8192
        dict(name="attend_cast", op="attend", B=8, P=61, tree=True, packed=True, len=8192, ragged=True, shared=0,
             page=64, H_kv=8, G=4, D=128, dtype="bf16", holes=False),
        # the stress batch behind one system prompt that all 64 requests share
        dict(name="attend_prefix", op="attend", B=64, P=65, tree=True, packed=True, len=5120, ragged=True,
             shared=4096, page=32, H_kv=8, G=4, D=128, dtype="fp16", holes=False),
        # odd head counts and head size, empty and one-token caches, rows whose mask leaves nothing
        dict(name="attend_odd", op="attend", B=5, P=23, tree=True, packed=False, len=1003, ragged=True, shared=0,
             page=32, H_kv=3, G=5, D=80, dtype="fp16", holes=True),
        # one request without a tree: penalties on one row
        dict(name="logits_one", op="logits", B=1, P=1, packed=False, V=32000, dtype="bf16", hist=300, bias=0,
             grammar=False),
        # the CAST batch's target rows: penalties, 64 biases a request, a grammar state for every position
        dict(name="logits_cast", op="logits", B=8, P=61, packed=True, V=128256, dtype="bf16", hist=4000, bias=64,
             grammar=True),
        # fp32 rows of the stress shape, 16 requests, an odd vocabulary (rows without 16-byte alignment)
        dict(name="logits_stress", op="logits", B=16, P=65, packed=False, V=128255, dtype="fp32", hist=8000, bias=300,
             grammar=True),
        # a round's reservation: at most nine tokens a request
        dict(name="reserve_round", op="reserve", B=8, S=9, page=16, len=8192, packed=False),
        # prompts of up to 8000 tokens for 64 requests, packed slot map
        dict(name="reserve_prompts", op="reserve", B=64, S=8000, page=16, len=1, packed=True),
        # a round's commit: accepted paths of 32 layers' keys and values
        dict(name="commit_round", op="commit", B=8, P=61, S=9, planes=64, H=8, D=128, page=16, tree=True,
             heads_first=False),
        # prompts' KV into pages whose heads come before the tokens
        dict(name="commit_prompts", op="commit", B=16, P=1500, S=1500, planes=16, H=5, D=96, page=32, tree=False,
             heads_first=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "logits", "reserve", "commit"])
    if op == "attend":
        B = _log(rng, 1, 64)
        P = rng.choice([1, 1, min(_log(rng, 2, 128), 4096 // B)])
        page = rng.choice([16, 32, 64, 128])
        shared = page * _log(rng, 1, 2048 // page) if rng.random() < 0.3 else 0
        H_kv, G = rng.choice([(1, 8), (2, 7), (2, 16), (3, 5), (4, 1), (4, 8), (5, 4), (8, 1), (8, 2), (8, 4)])
        return dict(op=op, B=B, P=P, tree=P > 1, packed=rng.random() < 0.5, len=shared + _log(rng, 1, 4000),
                    ragged=rng.random() < 0.8, shared=shared, page=page, H_kv=H_kv, G=G, D=rng.choice([64, 80, 96, 128, 128]),
                    dtype=rng.choice(["bf16", "fp16"]), holes=P > 1 and rng.random() < 0.3)
    if op == "logits":
        return dict(op=op, B=_log(rng, 1, 16), P=rng.choice([1, _log(rng, 2, 65)]), packed=rng.random() < 0.5,
                    V=_log(rng, 1000, 152000), dtype=rng.choice(["bf16", "fp32"]), hist=_log(rng, 1, 8000),
                    bias=rng.choice([0, _log(rng, 1, 300)]), grammar=rng.random() < 0.6)
    if op == "reserve":
        return dict(op=op, B=_log(rng, 1, 128), S=_log(rng, 1, 4000), page=rng.choice([16, 32, 64, 128]),
                    len=_log(rng, 1, 8192), packed=rng.random() < 0.5)
    tree = rng.random() < 0.6
    S = rng.randint(1, 17) if tree else _log(rng, 20, 1500)
    return dict(op=op, B=_log(rng, 1, 16), P=max(S, rng.randint(17, 85)) if tree else S, S=S,
                planes=_log(rng, 2, 16) * (4 if tree else 1), H=rng.choice([1, 2, 3, 5, 8]),
                D=rng.choice([64, 80, 96, 128]), page=rng.choice([16, 32, 64, 128]), tree=tree,
                heads_first=rng.random() < 0.5)


# ------------------------------------------------------------ what the case alone determines -------
def _own_rng(case):
    return random.Random(" ".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))


def _positions(rng, case):
    """Used positions of each request, between a quarter of P and P (P itself once)."""
    B, P = case["B"], case["P"]
    n = [rng.randint(max(1, P // 4), P) for _ in range(B)]
    n[rng.randrange(B)] = P
    return n


def _parents(rng, n):
    """A tree in breadth order: every position hangs from one of the last ten before it."""
    return [-1] + [rng.randint(max(0, i - 10), i - 1) for i in range(1, n)]


def _shape(case):
    """Lengths and trees of a case: plain lists."""
    rng = _own_rng(case)
    B = case["B"]
    if case["op"] == "attend":
        lo = max(case["shared"], case["len"] // 4) if case["ragged"] else case["len"]
        lens = [rng.randint(min(lo, case["len"]), case["len"]) for _ in range(B)]
        lens[rng.randrange(B)] = case["len"]
        if case["holes"] and not case["shared"] and B > 2:
            lens[:2] = [0, 1]
        n = _positions(rng, case) if case["tree"] else [case["P"]] * B
        parents = [_parents(rng, k) for k in n] if case["tree"] else None
        return dict(lens=lens, n=n, parents=parents)
    if case["op"] == "logits":
        n = _positions(rng, case)
        return dict(n=n, parents=[_parents(rng, k) for k in n])
    lens = [rng.randint(0, case.get("len", 1000)) for _ in range(B)]
    n = [rng.randint(1, case["S"]) for _ in range(B)]
    n[rng.randrange(B)] = case["S"]
    return dict(lens=lens, n=n)


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _up(a, b):
    return -(-a // b)


def work(case):
    s = _shape(case)
    if case["op"] == "attend":
        H_kv, G, D, P = case["H_kv"], case["G"], case["D"], case["P"]
        tokens = case["shared"] + sum(x - case["shared"] for x in s["lens"])
        rows = sum(s["n"])
        pairs = sum(x * n for x, n in zip(s["lens"], s["n"]))
        if case["tree"]:
            pairs += sum(d + 1 for p in s["parents"] for d in _depths(p))
        else:
            pairs += sum(n * (n + 1) // 2 for n in s["n"])
        nbytes = 2 * 2 * D * H_kv * (tokens + rows) + 2 * 2 * D * H_kv * G * rows
        nbytes += sum(n * n for n in s["n"]) if case["tree"] else 0
        nbytes += 4 * (case["shared"] // case["page"] + sum(_up(x - case["shared"], case["page"]) for x in s["lens"]))
        return {"bytes": nbytes, "flops": 4 * D * H_kv * G * pairs}
    if case["op"] == "logits":
        rows, V, B = sum(s["n"]), case["V"], case["B"]
        e = 2 if case["dtype"] == "bf16" else 4
        nbytes = rows * V * 2 * e + 4 * V * B + 8 * case["bias"] * B + (rows * 4 * _up(V, 32) if case["grammar"] else 0)
        return {"bytes": nbytes + sum(n * n for n in s["n"]), "flops": 4 * rows * V}
    if case["op"] == "reserve":
        page = case["page"]
        new = sum(_up(x + n, page) - _up(x, page) for x, n in zip(s["lens"], s["n"]))
        slots = sum(s["n"]) if case["packed"] else case["B"] * case["S"]
        # per granted page: taken from the stack and written to the table; then back; per request: lengths
        return {"bytes": 8 * slots + 16 * new + 24 * case["B"], "flops": 0}
    rows = sum(s["n"])
    return {"bytes": 2 * rows * case["planes"] * case["H"] * case["D"] * 2 + 20 * rows, "flops": 0}


# ---------------------------------------------------------------------------------------- inputs --
class State:
    pass


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tree_mask(parents, P):
    """[B][P][P] uint8, 1 where the column is an ancestor of the row or the row itself."""
    B = len(parents)
    up = torch.tensor([[max(p, 0) for p in row] + [0] * (P - len(row)) for row in parents], device="cuda")
    used = torch.tensor([[1] * len(row) + [0] * (P - len(row)) for row in parents], device="cuda").bool()
    anc = torch.zeros(B, P, P, dtype=torch.bool, device="cuda")
    at = torch.arange(P, device="cuda").expand(B, P)
    for _ in range(max(max(_depths(row)) for row in parents) + 1):
        anc.scatter_(2, at.unsqueeze(2), True)
        at = torch.gather(up, 1, at)
    anc &= used.unsqueeze(2)
    return anc.to(torch.uint8)


def _row_off(n):
    off = [0]
    for k in n:
        off.append(off[-1] + k)
    return off


def prepare(case, seed):
    s = State()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s.case, shape = case, _shape(case)
    s.op = case["op"]
    B = case["B"]

    def randn(*size, dtype):
        return torch.randn(*size, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)

    def randint(lo, hi, size, dtype=torch.int32):
        return torch.randint(lo, hi, size, generator=g, device="cuda", dtype=dtype)

    if s.op == "attend":
        dt_, H_kv, H, D, P, page = TYPES[case["dtype"]], case["H_kv"], case["H_kv"] * case["G"], case["D"], case["P"], case["page"]
        lens, n = shape["lens"], shape["n"]
        off = _row_off(n)
        rows = off[-1] + 3 if case["packed"] else B * P  # a packed buffer has room behind its last row
        s.row_off = _i32(off) if case["packed"] else None
        s.n_pos, s.seq_len = _i32(n), _i32(lens)
        s.shared = case["shared"]
        ns, mb = s.shared // page, max(1, max(_up(x, page) for x in lens))
        need = [_up(x, page) - ns for x in lens]
        n_blocks = ns + sum(need) + 5
        perm = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)
        e = torch.arange(mb, device="cuda")[None, :]
        first = torch.tensor(_row_off(need)[:-1], device="cuda")[:, None] + ns
        idx = torch.where(e < ns, e, first + e - ns)
        have = e < torch.tensor(need, device="cuda")[:, None] + ns
        s.table = torch.where(have, perm[idx.clamp(max=n_blocks - 1)], -1).to(torch.int32).contiguous()
        s.k_pages = randn(n_blocks, page, H_kv, D, dtype=dt_)
        s.v_pages = randn(n_blocks, page, H_kv, D, dtype=dt_)
        lead = (rows,) if case["packed"] else (B, P)
        s.q = randn(*lead, H, D, dtype=dt_) * 2  # scores spread by about two, as after query and key norms
        s.k_new = randn(*lead, H_kv, D, dtype=dt_)
        s.v_new = randn(*lead, H_kv, D, dtype=dt_)
        s.out = torch.zeros(*lead, H, D, dtype=dt_, device="cuda")
        s.mask = _tree_mask(shape["parents"], P) if case["tree"] else None
        if case["holes"]:  # rows of invalid nodes: nothing to attend to in the tree
            s.mask[:, 2::5] = 0
        s.P, s.scale = P, D ** -0.5
        if own:
            import dynamic_draft_tree_gb300 as dt
            s.h = dt.Handle(B, 2, 1, 1, 1, P)
            s.ws = dt.dt_tree_attention_workspace(s.h, B, P, H, H_kv, D, shared=s.shared > 0)
    elif s.op == "logits":
        V, P, dt_ = case["V"], case["P"], TYPES[case["dtype"]]
        n = shape["n"]
        off = _row_off(n)
        lead = (off[-1] + 2,) if case["packed"] else (B, P)
        s.row_off = _i32(off) if case["packed"] else None
        s.n_pos, s.P = _i32(n), P
        s.logits = randn(*lead, V, dtype=dt_) * 3
        s.out = torch.zeros(*lead, V, dtype=dt_, device="cuda")
        s.mask = _tree_mask(shape["parents"], P)
        s.tokens = randint(0, V, (B, P))
        # history: prompt tokens and generated ones, repeated as text repeats (squared uniform ranks)
        ids = (torch.rand(B, case["hist"], generator=g, device="cuda").square() * V).long().clamp(max=V - 1)
        half = case["hist"] // 2
        s.counts = torch.zeros(B, V, dtype=torch.int32, device="cuda")
        s.counts.scatter_add_(1, ids[:, half:], torch.ones_like(ids[:, half:], dtype=torch.int32))
        s.counts |= torch.zeros_like(s.counts).scatter_(1, ids[:, :half], SEEN)
        s.rep = 1 + torch.rand(B, generator=g, device="cuda") * 0.5
        s.freq = torch.rand(B, generator=g, device="cuda")
        s.pres = torch.rand(B, generator=g, device="cuda")
        s.bias_ids = s.bias_vals = s.allow = None
        if case["bias"]:
            k = min(case["bias"], V)
            s.bias_ids = torch.rand(B, V, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32).contiguous()
            s.bias_vals = torch.randn(B, k, generator=g, device="cuda") * 5
        if case["grammar"]:
            w = randint(-2 ** 31, 2 ** 31, (*lead, _up(V, 32)), torch.int64).to(torch.int32)
            s.allow = w & randint(-2 ** 31, 2 ** 31, (*lead, _up(V, 32)), torch.int64).to(torch.int32)
        if own:
            import dynamic_draft_tree_gb300 as dt
            s.h = dt.Handle(B, V, 1, 1, 1, P, dt.DT_BF16 if case["dtype"] == "bf16" else dt.DT_F32)
    elif s.op == "reserve":
        page, S, lens, n = case["page"], case["S"], shape["lens"], shape["n"]
        s.seq_len, s.n_new = _i32(lens), _i32(n)
        s.max_blocks = max(_up(x + k, page) for x, k in zip(lens, n)) + 1
        owned = [_up(x, page) for x in lens]
        total = sum(_up(x + k, page) for x, k in zip(lens, n)) + 7
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        s.n_owned = _i32(owned)
        first = torch.tensor(_row_off(owned)[:-1], device="cuda")[:, None]
        e = torch.arange(s.max_blocks, device="cuda")[None, :]
        s.table = torch.where(e < s.n_owned[:, None], perm[(first + e).clamp(max=total - 1)], -1).to(torch.int32).contiguous()
        s.n_blocks = total
        s.free_list = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        s.free_list[: total - sum(owned)] = perm[sum(owned):]
        s.free_count = _i32([total - sum(owned)])
        off = _row_off(n)
        s.slot_off = _i32(off) if case["packed"] else None
        s.S = S
        s.slots = torch.full((off[-1] + 2,) if case["packed"] else (B, S), -7, dtype=torch.int64, device="cuda")
        if own:
            import dynamic_draft_tree_gb300 as dt
            s.h = dt.Handle(B, 2, 1, 1, 1, 1)
            s.pool = dt.BlockPool(s.table, s.n_owned, s.free_list, s.free_count, page)
    else:
        planes, H, D, page, S, P = (case[k] for k in ("planes", "H", "D", "page", "S", "P"))
        n = shape["n"]
        off = _row_off([P] * B if case["tree"] else n)
        s.row_off = _i32(off)
        s.tmp = randn(planes, off[-1], H, D, dtype=torch.bfloat16)
        n_blocks = sum(_up(x, page) + 1 for x in n) + 3
        pages = randn(planes, n_blocks, H, page, D, dtype=torch.bfloat16) if case["heads_first"] else \
            randn(planes, n_blocks, page, H, D, dtype=torch.bfloat16)
        s.cache = pages.transpose(2, 3) if case["heads_first"] else pages
        # request b's tokens start somewhere inside its first page
        start = randint(0, page, (B,), torch.int64)
        base = torch.tensor(_row_off([_up(x, page) + 1 for x in n])[:-1], device="cuda")
        perm = torch.randperm(n_blocks, generator=g, device="cuda")
        j = torch.arange(S, device="cuda")[None, :]
        pos = start[:, None] + j
        blk = perm[(base[:, None] + pos // page).clamp(max=n_blocks - 1)]
        s.slots = torch.where(j < _i32(n)[:, None], blk * page + pos % page, -1).contiguous()
        s.n_new, s.seq_len = _i32(n), start.to(torch.int32)
        s.path = None
        if case["tree"]:  # accepted positions, root first, in ascending order
            s.path = torch.rand(B, P, generator=g, device="cuda").argsort(1)[:, :S].sort(1).values.to(torch.int32).contiguous()
            s.path[:, 0] = 0
        s.len_out = torch.zeros_like(s.seq_len)
        if own:
            import dynamic_draft_tree_gb300 as dt
            s.h = dt.Handle(B, 2, 1, 1, 1, min(P, 512))
    return s


# ------------------------------------------------------------------------------------------- run --
def run(s):
    return {"attend": _attend, "logits": _logits, "reserve": _reserve, "commit": _commit}[s.op](s)


def _rows_of(n_pos, row_off, P):
    """Buffer row, request and position of every used row."""
    b = torch.repeat_interleave(torch.arange(n_pos.numel(), device="cuda"), n_pos)
    first = torch.cumsum(n_pos, 0) - n_pos
    i = torch.arange(b.numel(), device="cuda") - first[b]
    return (row_off[b] if row_off is not None else b * P) + i, b, i


def _attend(s):
    if own:
        import dynamic_draft_tree_gb300 as dt
        dt.dt_tree_attention(s.h, s.q, s.k_new, s.v_new, s.k_pages, s.v_pages, s.table, s.seq_len, s.n_pos, s.out,
                             mask=s.mask, row_off=s.row_off, shared_len=s.shared, scale=s.scale, workspace=s.ws)
        return s.out
    H, D = s.q.shape[-2:]
    H_kv, page = s.k_pages.shape[2], s.k_pages.shape[1]
    B, P, G = s.n_pos.numel(), s.P, H // H_kv
    L = s.table.shape[1] * page
    q, kn, vn = (x.reshape(-1, *x.shape[-2:]) for x in (s.q, s.k_new, s.v_new))
    row, b, i = _rows_of(s.n_pos, s.row_off, P)
    at = torch.zeros(B, P, dtype=torch.long, device="cuda")
    at[b, i] = row.long()  # padded position -> buffer row (0 where unused)
    Q = q[at].float().reshape(B, P, H_kv, G, D).permute(0, 2, 3, 1, 4).reshape(B, H_kv, G * P, D)
    table = s.table.clamp(min=0).long()
    keys = torch.cat([s.k_pages[table].reshape(B, L, H_kv, D), kn[at]], 1).float().transpose(1, 2)
    vals = torch.cat([s.v_pages[table].reshape(B, L, H_kv, D), vn[at]], 1).float().transpose(1, 2)
    ok = torch.zeros(B, P, L + P, dtype=torch.bool, device="cuda")
    ok[:, :, :L] = (torch.arange(L, device="cuda")[None, :] < s.seq_len[:, None])[:, None, :]
    j = torch.arange(P, device="cuda")
    tree = s.mask.bool() if s.mask is not None else (j[None, :, None] >= j[None, None, :])
    ok[:, :, L:] = tree & (j[None, None, :] < s.n_pos[:, None, None])
    seen = torch.cat([torch.arange(L, device="cuda")[None, :] < s.seq_len[:, None], j[None, :] < s.n_pos[:, None]], 1)
    vals = torch.where(seen[:, None, :, None], vals, 0.0)  # what no row attends to is not a number to be added
    score = torch.matmul(Q, keys.transpose(2, 3)).mul_(s.scale).reshape(B, H_kv, G, P, L + P)
    score.masked_fill_(~ok[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    w = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.reshape(B, H_kv, G * P, L + P), vals).reshape(B, H_kv, G, P, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, P, H, D)
    s.out.view(-1, H, D)[row.long()] = o[b, i].to(s.out.dtype)
    return s.out


def _logits(s):
    if own:
        import dynamic_draft_tree_gb300 as dt
        dt.dt_logits_process(s.h, s.logits, s.out, s.n_pos, tokens=s.tokens, mask=s.mask, row_off=s.row_off,
                             counts=s.counts, repetition=s.rep, frequency=s.freq, presence=s.pres,
                             bias_ids=s.bias_ids, bias_vals=s.bias_vals, allow=s.allow)
        return s.out
    V, P = s.logits.shape[-1], s.P
    row, b, i = _rows_of(s.n_pos, s.row_off, P)
    row = row.long()
    x = s.logits.reshape(-1, V)[row].float()
    counts = s.counts[b]
    on_path = s.mask[b, i].to(torch.int32)
    made = (counts & (SEEN - 1)).scatter_add_(1, s.tokens[b].long(), on_path)
    seen = (made > 0) | (counts >= SEEN)
    rep = s.rep[b, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s.freq[b, None] * made - s.pres[b, None] * (made > 0)
    if s.bias_ids is not None:
        bias = torch.zeros(s.n_pos.numel(), V, device="cuda").scatter_add_(1, s.bias_ids.long(), s.bias_vals)
        x = x + bias[b]
    if s.allow is not None:
        v = torch.arange(V, device="cuda")
        x.masked_fill_((s.allow.reshape(-1, s.allow.shape[-1])[row][:, v >> 5] >> (v & 31)) & 1 == 0, -math.inf)
    s.out.view(-1, V)[row] = x.to(s.out.dtype)
    return s.out


def _reserve(s):
    """Reserves the new tokens' pages and writes their slots; then gives the pages back (a reservation that
    a round rolls back), which leaves the pool as it was."""
    if own:
        import dynamic_draft_tree_gb300 as dt
        dt.dt_kv_reserve(s.h, s.pool, s.seq_len, s.n_new, s.slots, slot_off=s.slot_off)
        dt.dt_kv_release(s.h, s.pool, s.seq_len)
        return [s.slots, s.table, s.n_owned, s.free_list, s.free_count]
    page, B, MB = s.case["page"], s.case["B"], s.max_blocks
    want = (s.seq_len + s.n_new + page - 1) // page
    need = (want - s.n_owned).clamp(min=0)
    need = torch.where(want <= MB, need, 0)
    upto = torch.cumsum(need, 0)
    ok = (want <= MB) & ((need == 0) | (upto <= s.free_count))
    e = torch.arange(MB, device="cuda")[None, :]
    grant = ok[:, None] & (e >= s.n_owned[:, None]) & (e < want[:, None])
    q = (upto - need)[:, None] + e - s.n_owned[:, None]
    table = torch.where(grant, s.free_list[(s.free_count - 1 - q).clamp(0, s.n_blocks - 1).long()], s.table)
    owned = torch.where(ok, torch.maximum(want, s.n_owned), s.n_owned)
    count = s.free_count - (grant.sum())
    j = torch.arange(s.S, device="cuda")[None, :]
    pos = s.seq_len[:, None] + j
    slot = torch.gather(table, 1, (pos // page).clamp(max=MB - 1).long()).long() * page + pos % page
    slot = torch.where(ok[:, None] & (j < s.n_new[:, None]), slot, -1)
    if s.slot_off is None:
        s.slots.copy_(slot)
    else:
        row, b, i = _rows_of(s.n_new, s.slot_off, s.S)
        s.slots[row.long()] = slot[b, i]
    keep = torch.minimum((s.seq_len + page - 1) // page, owned)
    back = (e >= keep[:, None]) & (e < owned[:, None])
    order = torch.cumsum(back.reshape(-1), 0).reshape(B, MB) - 1
    total = back.sum()
    free = s.free_list.clone()
    free[(count + total - 1 - order)[back]] = table[back]
    return [s.slots, torch.where(back, -1, table).to(torch.int32), keep.to(torch.int32), free, (count + total).to(torch.int32)]


def _commit(s):
    if own:
        import dynamic_draft_tree_gb300 as dt
        dt.dt_commit_kv_paged(s.h, s.tmp, s.cache, s.slots, s.n_new, s.seq_len, s.len_out, path=s.path,
                              row_off=s.row_off)
        return [s.cache, s.len_out]
    page, S = s.case["page"], s.case["S"]
    j = torch.arange(S, device="cuda")[None, :].expand(s.case["B"], S)
    used = (j < s.n_new[:, None]) & (s.slots >= 0)
    pos = s.path if s.path is not None else j
    rows = (s.row_off[:-1, None] + pos)[used].long()
    slot = s.slots[used]
    s.cache[:, slot // page, slot % page] = s.tmp[:, rows]
    s.len_out.copy_(s.seq_len + s.n_new)
    return [s.cache, s.len_out]


# ----------------------------------------------------------------------------------------- exact --
def exact(case, seed):
    """The definitions, one request after another, in 64 bits."""
    s = prepare(case, seed)
    n = s.n_pos.tolist() if case["op"] in ("attend", "logits") else s.n_new.tolist()
    if case["op"] == "attend":
        H, D = s.q.shape[-2:]
        G, page = case["G"], case["page"]
        q, kn, vn = (x.reshape(-1, *x.shape[-2:]) for x in (s.q, s.k_new, s.v_new))
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        for b, L in enumerate(s.seq_len.tolist()):
            r0 = s.row_off[b].item() if s.row_off is not None else b * s.P
            blocks = s.table[b, : _up(L, page)].long()
            k = torch.cat([s.k_pages[blocks].flatten(0, 1)[:L], kn[r0: r0 + n[b]]])
            v = torch.cat([s.v_pages[blocks].flatten(0, 1)[:L], vn[r0: r0 + n[b]]])
            ok = torch.ones(n[b], L + n[b], dtype=torch.bool, device="cuda")
            ok[:, L:] = s.mask[b, : n[b], : n[b]].bool() if s.mask is not None else ok[:, L:].tril()
            for h in range(H):
                z = q[r0: r0 + n[b], h].double() @ k[:, h // G].double().T * s.scale
                z = z.masked_fill(~ok, -math.inf)
                some = ok.any(1, keepdim=True)
                p = torch.softmax(torch.where(some, z, 0.0), 1) * some
                out[r0: r0 + n[b], h] = p @ v[:, h // G].double()
        return out.reshape(s.q.shape)
    if case["op"] == "logits":
        V = case["V"]
        x, out = s.logits.reshape(-1, V), torch.zeros(s.out.numel() // V, V, dtype=torch.float64, device="cuda")
        for b, k in enumerate(n):
            r0 = s.row_off[b].item() if s.row_off is not None else b * s.P
            y = x[r0: r0 + k].double()
            path = s.mask[b, :k, :k].double()
            hit = torch.zeros(k, V, dtype=torch.float64, device="cuda")
            hit.index_add_(1, s.tokens[b, :k].long(), path)
            hit += (s.counts[b] % SEEN).double()
            known = (hit > 0) | (s.counts[b] // SEEN > 0)
            r = s.rep[b].double()
            y = torch.where(known & (y > 0), y / r, torch.where(known, y * r, y))
            y -= s.freq[b].double() * hit + s.pres[b].double() * (hit > 0)
            if s.bias_ids is not None:
                y[:, s.bias_ids[b].long()] += s.bias_vals[b].double()
            if s.allow is not None:
                bits = s.allow.reshape(-1, s.allow.shape[-1])[r0: r0 + k]
                bits = torch.stack([(bits >> t) & 1 for t in range(32)], 2).flatten(1)[:, :V]
                y[bits == 0] = -math.inf
            out[r0: r0 + k] = y
        return out.reshape(s.out.shape)
    return None  # whole numbers and copies
