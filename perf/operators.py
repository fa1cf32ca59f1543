"""Measured cases of the paged KV cache: attention for a tree of drafted tokens
over it, and the operators that write, compact, fork, extend and free its pages.

A cache keeps its K and V rows in pages, k_pages and v_pages
[layers][n_pages][hkv][page_rows][head_dim].  Row t of sequence s is row
t % page_rows of page page_table[s][t // page_rows], for every layer and KV
head; seq_lens[s] rows are valid, page_refs[p] sequences hold page p.

  kind "tree"     tree_attention: n_nodes drafted tokens a sequence attend to
                  the sequence's cached rows and to their ancestors in the
                  tree (with "plan": the visibility words come from
                  tree_mask, in the same pass)
  kind "prompt"   kv_pages_write: a prompt's K/V rows into the pages
  kind "commit"   kv_pages_free + kv_pages_reserve + kv_pages_write: back to
                  the committed length, room for the accepted tokens, their rows
  kind "compact"  kv_pages_compact: the selected rows into pages of their own
  kind "fork"     kv_pages_fork + kv_pages_reserve: sequences that share their
                  pages, each extended on its own (the shared last page is copied)

`own` chooses between the plain forms (elementary torch operations, 32-bit)
and the framework's operators.
"""
import math
import random

import torch

own = False

LOG2E = 1.4426950408889634


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one new token over a 16K cache: the single-token form, one layer a call as a model runs it
        dict(name="token_16k", kind="tree", batch=1, layers=1, hq=32, hkv=8, d=128, nodes=1, rows=16384,
             page=64, ragged=False, fp16=False, plan=False),
        # the smallest call: a small draft model's layer, 8 drafted tokens over a 2K prompt, with the tree's words
        dict(name="tree8_draft_2k", kind="tree", batch=1, layers=1, hq=14, hkv=2, d=64, nodes=8, rows=2048,
             page=16, ragged=False, fp16=False, plan=True),
        # 16 drafted tokens over the compressed cache (C_max 256 and the window of 64), all layers in a call
        dict(name="tree16_compressed", kind="tree", batch=1, layers=64, hq=40, hkv=8, d=128, nodes=16, rows=320,
             page=64, ragged=False, fp16=False, plan=False),
        # a batch of ragged sequences and trees, fp16, one layer
        dict(name="tree24_batch16", kind="tree", batch=16, layers=1, hq=32, hkv=8, d=128, nodes=24, rows=8192,
             page=32, ragged=True, fp16=True, plan=True),
        # 64 drafted tokens over the uncompressed 64K cache, one layer
        dict(name="tree64_64k", kind="tree", batch=2, layers=1, hq=40, hkv=8, d=128, nodes=64, rows=65536,
             page=128, ragged=False, fp16=False, plan=False),
        # an odd tree size over odd lengths, two layers
        dict(name="tree33_odd", kind="tree", batch=5, layers=2, hq=32, hkv=8, d=128, nodes=33, rows=4999,
             page=48, ragged=True, fp16=False, plan=False),
        # a 16K prompt's rows into the pages, all layers
        dict(name="prompt_16k", kind="prompt", batch=1, layers=32, hkv=8, d=128, rows=16384, page=64),
        # the accepted tokens of a batch's trees join the cache
        dict(name="commit_batch32", kind="commit", batch=32, layers=16, hkv=8, d=128, rows=1024, nodes=16, page=16),
        # the rows that each KV head keeps of a 16K prompt (C_max 256 and the window of 64)
        dict(name="compact_16k_320", kind="compact", batch=1, layers=32, hkv=8, d=128, rows=16384, keep=320,
             page=64, shared=False),
        # 2048 prompt tokens kept for every layer and head, two sequences of a 32K prompt
        dict(name="compact_32k_2048", kind="compact", batch=2, layers=8, hkv=8, d=128, rows=32768, keep=2048,
             page=128, shared=True),
        # one layer of a draft model: four continuations of a sequence
        dict(name="fork_4", kind="fork", batch=4, layers=1, hkv=2, d=64, rows=777, new=5, page=16),
        # 32 continuations of long sequences
        dict(name="fork_32", kind="fork", batch=32, layers=4, hkv=8, d=128, rows=8192, new=16, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "tree", "prompt", "commit", "compact", "fork"])
    page = rng.choice([16, 24, 32, 48, 64, 128])
    if kind == "tree":
        hq, hkv, d = rng.choice([(14, 2, 64), (32, 8, 128), (40, 8, 128), (8, 8, 128), (16, 2, 64)])
        nodes = _log(rng, 1, 64)
        batch, layers = _log(rng, 1, 24), _log(rng, 1, 16)
        rows = _log(rng, 64, 65536)
        rows = max(64, min(rows, (2 * 8 * 65536 * 128 * 320) // (batch * layers * hkv * d * (hq // hkv) * max(nodes, 16))))
        rows = max(64, min(rows, (4 << 30) // (batch * layers * hkv * d * 4)))
        return dict(kind=kind, batch=batch, layers=layers, hq=hq, hkv=hkv, d=d, nodes=nodes, rows=rows, page=page,
                    ragged=rng.random() < 0.5, fp16=rng.random() < 0.3, plan=nodes > 1 and rng.random() < 0.5)
    hkv, d = rng.choice([(8, 128), (2, 64), (4, 128)])
    layers = _log(rng, 1, 24)
    if kind == "prompt":
        rows = _log(rng, 64, 16384)
        return dict(kind=kind, batch=max(1, min(_log(rng, 1, 8), 16384 // rows)), layers=layers, hkv=hkv, d=d,
                    rows=rows, page=page)
    if kind == "commit":
        return dict(kind=kind, batch=_log(rng, 1, 48), layers=layers, hkv=hkv, d=d, rows=_log(rng, 32, 2048),
                    nodes=_log(rng, 1, 64), page=page)
    if kind == "compact":
        rows, batch = _log(rng, 512, 16384), rng.randint(1, 3)
        return dict(kind=kind, batch=batch, layers=max(1, layers // batch), hkv=hkv, d=d, rows=rows,
                    keep=max(1, min(rows, _log(rng, 64, 2048))), page=page, shared=rng.random() < 0.4)
    return dict(kind=kind, batch=_log(rng, 2, 32), layers=max(1, layers // 4), hkv=hkv, d=d, rows=_log(rng, 64, 8192),
                new=_log(rng, 1, 48), page=page)


# --------------------------------------------------------------------- inputs
def _lens(case):
    """Rows cached for each sequence, and live nodes of each tree (fixed by the case)."""
    B, n, T = case["batch"], case["rows"], case.get("nodes", 1)
    r = random.Random(n * 1009 + B * 31 + T)
    if not case.get("ragged"):
        return [n] * B, [T] * B
    lens = [n] + [_log(r, max(1, n // 16), n) for _ in range(B - 1)]
    return lens, [T] + [max(1, T - r.randrange(1 + T // 3)) for _ in range(B - 1)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _empty_cache(case, n_pages, n_seqs, max_pages, g, dtype):
    shape = (case["layers"], n_pages, case["hkv"], case["page"], case["d"])
    return dict(k_pages=_randn(shape, g, dtype), v_pages=_randn(shape, g, dtype),
                page_refs=torch.zeros(n_pages, dtype=torch.int32, device="cuda"),
                page_table=torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device="cuda"),
                seq_lens=torch.zeros(n_seqs, dtype=torch.int32, device="cuda"))


def _fill(st, seqs, lens, page, seed):
    """Give sequences `seqs` their pages, at places drawn from the seed."""
    order = list(range(st["page_refs"].numel()))
    random.Random(seed).shuffle(order)
    table, at = st["page_table"].cpu(), 0
    for s, n in zip(seqs, lens):
        k = -(-n // page)
        table[s, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
        at += k
    st["page_table"].copy_(table)
    st["page_refs"][torch.tensor(order[:at], device="cuda")] = 1
    st["seq_lens"][torch.tensor(seqs, device="cuda")] = torch.tensor(lens, dtype=torch.int32, device="cuda")


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    kind, B, page = case["kind"], case["batch"], case["page"]
    L, H, d = case["layers"], case["hkv"], case["d"]
    if kind == "tree":
        return _prepare_tree(case, seed, g)
    if kind == "prompt":
        n = case["rows"]
        per = -(-n // page)
        st = _empty_cache(case, B * per + 3, B, per + 1, g, torch.bfloat16)
        _fill(st, list(range(B)), [n] * B, page, seed)
        st.update(kind=kind, page=page, k=_randn((B, L, H, n, d), g, torch.bfloat16),
                  v=_randn((B, L, H, n, d), g, torch.bfloat16), seqs=_i32(list(range(B))))
        return st
    if kind == "commit":
        n, T = case["rows"], case["nodes"]
        r = random.Random(n + 7 * T + B)
        lens = [_log(r, max(1, n // 8), n) for _ in range(B)]
        most = min(T, 8)
        counts = [r.randint(1, most) for _ in range(B)]
        per = -(-(n + T) // page)
        st = _empty_cache(case, sum(-(-(m + T) // page) for m in lens) + 5, B, per, g, torch.bfloat16)
        _fill(st, list(range(B)), lens, page, seed)
        path = torch.sort(torch.argsort(torch.rand((B, T), generator=g, device="cuda"), 1)[:, :most], 1)[0]
        st.update(kind=kind, page=page, k=_randn((B, L, H, T, d), g, torch.bfloat16),
                  v=_randn((B, L, H, T, d), g, torch.bfloat16), seqs=_i32(list(range(B))), keep=_i32(lens),
                  idx=path.to(torch.int32).contiguous(), counts=_i32(counts),
                  result=_i32([0]))
        return st
    if kind == "compact":
        n, keep = case["rows"], case["keep"]
        per, kp = -(-n // page), -(-keep // page)
        st = _empty_cache(case, B * (per + kp) + 4, 2 * B, per, g, torch.bfloat16)
        _fill(st, list(range(B)), [n] * B, page, seed)
        lists = B if case["shared"] else B * L * H
        idx = torch.stack([torch.randperm(n, generator=g, device="cuda")[:keep] for _ in range(lists)])
        st.update(kind=kind, page=page, src=_i32(list(range(B))), dst=_i32(list(range(B, 2 * B))),
                  idx=torch.sort(idx, 1)[0].to(torch.int32).contiguous(), units_per_idx=L * H if case["shared"] else 1,
                  result=_i32([0]))
        return st
    n, new = case["rows"], case["new"]                    # fork: B continuations of max(1, B // 4) sequences
    S = max(1, B // 4)
    lens = [n - (n * i) // (3 * S) for i in range(S)]
    per = -(-(n + new) // page)
    own_pages = 1 + -(-new // page)
    st = _empty_cache(case, sum(-(-m // page) for m in lens) + B * own_pages + 2, S + B, per, g, torch.bfloat16)
    _fill(st, list(range(S)), lens, page, seed)
    parent = torch.randint(0, S, (B,), generator=g, device="cuda").to(torch.int32)
    st.update(kind=kind, page=page, src=parent, dst=_i32(list(range(S, S + B))), new=_i32([new] * B), result=_i32([0]),
              result2=_i32([0]))
    return st


def _prepare_tree(case, seed, g):
    B, L, hq, H, d, T, page = (case[x] for x in ("batch", "layers", "hq", "hkv", "d", "nodes", "page"))
    dtype = torch.float16 if case["fp16"] else torch.bfloat16
    lens, live = _lens(case)
    n_pages = sum(-(-n // page) for n in lens) + 2
    st = _empty_cache(case, n_pages, B, -(-max(lens) // page) + 1, g, dtype)
    _fill(st, list(range(B)), lens, page, seed)
    # the queries share a direction with some of the keys, and strongly with each sequence's first row
    u = torch.randn((L, H, d), generator=g, device="cuda")
    u = u / u.norm(dim=-1, keepdim=True)
    heavy = torch.rand((L, n_pages, H, page), generator=g, device="cuda") < 0.01
    st["k_pages"].add_((3.0 * heavy[..., None] * u[:, None, :, None, :]).to(dtype))
    st["k_pages"][:, :, :, 0][:, st["page_table"][:, 0].long()] += (4.0 * u)[:, None].to(dtype)
    q = torch.randn((B, L, H, hq // H, T, d), generator=g, device="cuda") + 1.5 * u[None, :, :, None, None, :]
    parents = (torch.rand((B, T), generator=g, device="cuda") * (torch.arange(T, device="cuda") + 1)).floor()
    parents = (parents.to(torch.int32) - 1).contiguous()
    n_live = _i32(live)
    st.update(kind="tree", plan=case["plan"], q=q.reshape(B, L, hq, T, d).to(dtype).contiguous(), n_live=n_live,
              k_tree=_randn((B, L, H, T, d), g, dtype), v_tree=_randn((B, L, H, T, d), g, dtype), parents=parents,
              mask=_plain_tree_mask(parents, n_live)[0], scale=d ** -0.5,
              out=torch.full((B, L, hq, T, d), 2.0 ** -10, dtype=dtype, device="cuda"),
              lse2=torch.full((B, L, hq, T), 2.0 ** -10, dtype=torch.float32, device="cuda"))
    return st


# --------------------------------------------------------------------- one pass
def run(st):
    return (_own_run if own else _plain_run)(st)


def _own_run(st):
    import prompt_compression_b200 as P
    kind = st["kind"]
    cache = (st["k_pages"], st["v_pages"], st["page_refs"], st["page_table"], st["seq_lens"])
    if kind == "tree":
        mask, depth = st["mask"], None
        if st["plan"]:
            mask, depth = P.tree_mask(st["parents"], n_live=st["n_live"])
        out = P.tree_attention(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["seq_lens"],
                               st["k_tree"], st["v_tree"], mask=mask, n_live=st["n_live"], out=st["out"],
                               lse2=st["lse2"], scale=st["scale"])
        return (out, st["lse2"], mask, depth) if st["plan"] else (out, st["lse2"])
    if kind == "prompt":
        P.kv_pages_write(st["k"], st["v"], *cache, st["seqs"])
    elif kind == "commit":
        P.kv_pages_free(*cache[2:], st["seqs"], page_rows=st["page"], keep_rows=st["keep"])
        P.kv_pages_reserve(*cache, st["seqs"], st["counts"], result=st["result"])
        P.kv_pages_write(st["k"], st["v"], *cache, st["seqs"], idx=st["idx"], counts=st["counts"],
                         units_per_idx=st["k"].shape[1] * st["k"].shape[2])
    elif kind == "compact":
        P.kv_pages_compact(*cache, st["src"], st["dst"], st["idx"], units_per_idx=st["units_per_idx"],
                           result=st["result"])
    else:
        P.kv_pages_fork(*cache[2:], st["src"], st["dst"], page_rows=st["page"], result=st["result"])
        P.kv_pages_reserve(*cache, st["dst"], st["new"], result=st["result2"])
    return _cache_outputs(st)


def _cache_outputs(st):
    return tuple(st[x] for x in ("k_pages", "v_pages", "page_refs", "page_table", "seq_lens", "result", "result2")
                 if x in st)


def _plain_run(st):
    kind = st["kind"]
    if kind == "tree":
        mask, depth = st["mask"], None
        if st["plan"]:
            mask, depth = _plain_tree_mask(st["parents"], st["n_live"])
        _plain_tree_attention(st, mask)
        return (st["out"], st["lse2"], mask, depth) if st["plan"] else (st["out"], st["lse2"])
    if kind == "prompt":
        _plain_write(st, None, torch.full_like(st["seqs"], st["k"].shape[3]))
    elif kind == "commit":
        _plain_free(st, st["seqs"], st["keep"])
        st["result"].copy_(_plain_reserve(st, st["seqs"], st["counts"]))
        _plain_write(st, st["idx"][:, None, None], st["counts"])
    elif kind == "compact":
        _plain_compact(st)
    else:
        _plain_fork(st)
        st["result2"].copy_(_plain_reserve(st, st["dst"], st["new"]))
    return _cache_outputs(st)


# --------------------------------------------------------------------- plain forms
def _plain_tree_mask(parents, n_live):
    """mask int32 [B][T][ceil(T/32)]: bit j of row i = node j is node i or an ancestor of it; depth [B][T]."""
    B, T = parents.shape
    node = torch.arange(T, device=parents.device)
    sees = (parents[:, :, None] == node) | (node[:, None] == node)
    for _ in range(max(1, (T - 1).bit_length())):                        # paths of twice the length a turn
        sees = (sees.float() @ sees.float()) > 0
    live = node < n_live[:, None]
    sees &= live[:, :, None]
    depth = (sees.sum(-1) - live.long()).to(torch.int32)
    words = -(-T // 32)
    bits = torch.zeros((B, T, words * 32), dtype=torch.int64, device=parents.device)
    bits[:, :, :T] = sees
    mask = (bits.view(B, T, words, 32) << torch.arange(32, device=parents.device)).sum(-1)
    return torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32), depth


def _plain_tree_attention(st, mask):
    q, kt, vt, table, lens = st["q"], st["k_tree"], st["v_tree"], st["page_table"], st["seq_lens"]
    B, L, hq, T, d = q.shape
    H, page = kt.shape[2], st["k_pages"].shape[3]
    n = table.shape[1] * page
    at = torch.arange(n, device=q.device)
    valid = at < lens[:, None]                                           # [B][n]
    pages = torch.where(valid, table[:, at // page], table[:, :1]).long()
    bits = (mask[..., None] >> torch.arange(32, device=q.device)) & 1
    node = torch.arange(T, device=q.device)
    live = node < st["n_live"][:, None]
    sees = (bits.flatten(2)[:, :, :T] > 0) & live[:, None, :]            # [B][T][T]

    def rows(pool, tree):                                                # [B][L][H][n + T][d], 0 where no row is
        r = pool[:, pages, :, at % page]                                 # [B][n][L][H][d]
        r = torch.where(valid[:, :, None, None, None], r, 0).permute(0, 2, 3, 1, 4)
        t = torch.where(live[:, None, None, :, None], tree, 0)
        return torch.cat([r, t], 3).float()

    k, v = rows(st["k_pages"], kt), rows(st["v_pages"], vt)
    visible = torch.cat([valid[:, None, :].expand(B, T, n), sees], 2)    # [B][T][n + T]
    qf = q.float().view(B, L, H, hq // H, T, d)
    s = qf.reshape(B, L, H, -1, d) @ k.transpose(-1, -2) * st["scale"]
    s = s.view(B, L, H, hq // H, T, -1).masked_fill(~visible[:, None, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    lse2 = ((m + torch.log(z)) * LOG2E).squeeze(-1).reshape(B, L, hq, T)
    p = e / torch.where(z == 0, 1.0, z)
    o = (p.view(B, L, H, -1, n + T) @ v).view(B, L, hq, T, d)
    keep = live[:, None, None, :]
    st["out"].copy_(torch.where(keep[..., None], o.to(q.dtype), st["out"]))
    st["lse2"].copy_(torch.where(keep, lse2, st["lse2"]))


def _plain_free(st, seqs, keep):
    page, table, refs, lens, s = st["page"], st["page_table"], st["page_refs"], st["seq_lens"], seqs.long()
    new = torch.minimum(lens[s], keep)
    drop = (torch.arange(table.shape[1], device=table.device) * page >= new[:, None]) & (table[s] >= 0)
    refs.index_add_(0, table[s].clamp(min=0).flatten().long(), -drop.flatten().to(torch.int32))
    table[s] = torch.where(drop, -1, table[s])
    lens[s] = new


def _plain_alloc(refs, want):
    """The `want` lowest-numbered free pages, and how many are missing."""
    free = torch.sort((refs != 0).to(torch.int8), stable=True)[1]
    missing = (want - (refs == 0).sum()).clamp(min=0)
    return free, missing


def _plain_reserve(st, seqs, n_new):
    page, table, refs, lens, s = st["page"], st["page_table"], st["page_refs"], st["seq_lens"], seqs.long()
    old, grows = lens[s], n_new > 0
    have = (old + page - 1) // page
    need = (old + n_new + page - 1) // page - have
    at = (old // page).clamp(max=table.shape[1] - 1)
    tail = table[s].gather(1, at[:, None].long()).squeeze(1)
    part = grows & (old % page > 0)
    same = (tail[:, None] == tail) & part[:, None] & part
    before = same.tril(-1).sum(1)
    copy = part & (refs[tail.clamp(min=0).long()] - before > 1)
    want = need + copy
    first = torch.cumsum(want, 0) - want
    free, missing = _plain_alloc(refs, want.sum())
    pos = torch.arange(table.shape[1], device=table.device)
    fresh = (pos >= have[:, None]) & (pos < (have + need)[:, None])
    takes = (fresh | (copy[:, None] & (pos == at[:, None]))) & (missing == 0)
    rank = torch.where(fresh, pos - have[:, None] + copy[:, None], 0) + first[:, None]
    page_of = free[rank.clamp(0, free.numel() - 1)].to(torch.int32)
    refs.index_add_(0, tail.clamp(min=0).long(), -(copy & (missing == 0)).to(torch.int32))
    refs.index_add_(0, page_of.flatten().long(), takes.flatten().to(torch.int32))
    table[s] = torch.where(takes, page_of, table[s])
    lens[s] = torch.where(missing == 0, old + n_new, old)
    i = torch.nonzero(copy & (missing == 0)).squeeze(1)                  # the shared last pages, copied up to the length
    to, frm = table[s[i]].gather(1, at[i, None].long()).squeeze(1).long(), tail[i].long()
    rows = (torch.arange(page, device=table.device) < (old[i] % page)[:, None])[None, :, None, :, None]
    for pool in (st["k_pages"], st["v_pages"]):
        pool[:, to] = torch.where(rows, pool[:, frm], pool[:, to])
    return missing.to(torch.int32)


def _plain_write(st, idx, counts):
    """Rows idx[i][l][h][t] (or t), t < counts[i], of k and v become sequence i's newest rows."""
    page, table, s = st["page"], st["page_table"], st["seqs"].long()
    B, L, H, n, _ = st["k"].shape
    n = n if idx is None else idx.shape[-1]
    item, layer, head = (torch.arange(m, device=table.device) for m in (B, L, H))
    t = torch.arange(n, device=table.device)
    pos = st["seq_lens"][s][:, None] - counts[:, None] + t               # [B][n]
    put = (t < counts[:, None]) & (pos >= 0)
    b, t = torch.nonzero(put, as_tuple=True)
    where = pos[b, t].long()
    to = table[s[b], where // page].long()
    for src, pool in ((st["k"], st["k_pages"]), (st["v"], st["v_pages"])):
        picked = src if idx is None else src[item[:, None, None, None], layer[:, None, None], head[:, None], idx.long()]
        pool[:, to, :, where % page] = picked[b, :, :, t]


def _plain_compact(st):
    page, table, refs, lens = st["page"], st["page_table"], st["page_refs"], st["seq_lens"]
    src, dst, idx = st["src"].long(), st["dst"].long(), st["idx"]
    L, H, d, n, keep = st["k_pages"].shape[0], st["k_pages"].shape[2], st["k_pages"].shape[4], src.numel(), idx.shape[1]
    old, gone = table[src], table[dst]
    # pages of the sources are held while the destinations' old pages are released and new ones taken
    held = refs.index_add(0, old.clamp(min=0).flatten().long(), (old >= 0).flatten().to(torch.int32))
    held.index_add_(0, gone.clamp(min=0).flatten().long(), -(gone >= 0).flatten().to(torch.int32))
    per = -(-keep // page)
    free, missing = _plain_alloc(held, torch.tensor(n * per, device="cuda"))
    fresh = free[:n * per].view(n, per).to(torch.int32)
    done = missing == 0
    new = refs.index_add(0, gone.clamp(min=0).flatten().long(), -(gone >= 0).flatten().to(torch.int32))
    new.index_add_(0, fresh.flatten().long(), torch.ones_like(fresh).flatten())
    refs.copy_(torch.where(done, new, refs))
    rows = torch.full_like(gone, -1)
    rows[:, :per] = fresh
    table[dst] = torch.where(done, rows, gone)
    lens[dst] = torch.where(done, keep, lens[dst]).to(torch.int32)
    st["result"].copy_(missing.to(torch.int32))
    at = (idx.view(n, 1, 1, keep) if st["units_per_idx"] > 1 else idx.view(n, L, H, keep)).expand(n, L, H, keep)
    at = at.permute(1, 0, 2, 3).long()                                   # [L][n][H][keep]
    frm = old[torch.arange(n, device="cuda")[:, None, None], at // page].long()
    t = torch.arange(keep, device="cuda")
    to = fresh[:, t // page].long()[None, :, None].expand_as(at)
    layer = torch.arange(L, device="cuda")[:, None, None, None]
    head = torch.arange(H, device="cuda")[:, None]
    for pool in (st["k_pages"], st["v_pages"]):
        pool[layer, to, head, (t % page).expand_as(at)] = pool[layer, frm, head, at % page]


def _plain_fork(st):
    table, refs, lens, src, dst = st["page_table"], st["page_refs"], st["seq_lens"], st["src"].long(), st["dst"].long()
    new, gone, n = table[src], table[dst], lens[src]
    refs.index_add_(0, new.clamp(min=0).flatten().long(), (new >= 0).flatten().to(torch.int32))
    refs.index_add_(0, gone.clamp(min=0).flatten().long(), -(gone >= 0).flatten().to(torch.int32))
    table[dst] = new
    lens[dst] = n
    st["result"].zero_()


# --------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return _exact_tree(case, st) if case["kind"] == "tree" else _exact_pages(case, st)


def _exact_tree(case, st):
    B, L, hq, H, d, T, page = (case[x] for x in ("batch", "layers", "hq", "hkv", "d", "nodes", "page"))
    lens, live = _lens(case)
    parents = st["parents"].tolist()
    out, lse2 = st["out"].double(), st["lse2"].double()
    words, depth = [], []
    for b in range(B):
        sees = []                                                        # the nodes on the way up, each node's own first
        for i in range(T):
            p = parents[b][i]
            sees.append([i] + (sees[p] if p >= 0 else []))
        w = [[0] * (-(-T // 32)) for _ in range(T)]
        for i in range(live[b]):
            for j in sees[i]:
                w[i][j // 32] |= 1 << (j % 32)
        words.append([[x - (1 << 32) if x >> 31 else x for x in row] for row in w])
        depth.append([len(sees[i]) - 1 if i < live[b] else 0 for i in range(T)])
        n, t = lens[b], live[b]
        hidden = torch.ones((t, t), dtype=torch.bool)
        for i in range(t):
            hidden[i, sees[i]] = False
        hidden = hidden.to("cuda")
        used = st["page_table"][b, :-(-n // page)].long()
        for l in range(L):
            for h in range(H):
                k = torch.cat([st["k_pages"][l, used, h].reshape(-1, d)[:n], st["k_tree"][b, l, h, :t]]).double()
                v = torch.cat([st["v_pages"][l, used, h].reshape(-1, d)[:n], st["v_tree"][b, l, h, :t]]).double()
                g = slice(h * (hq // H), (h + 1) * (hq // H))
                s = torch.einsum("gtd,nd->gtn", st["q"][b, l, g, :t].double(), k) * st["scale"]
                s[:, :, n:].masked_fill_(hidden, -math.inf)
                lse = torch.logsumexp(s, -1)
                lse2[b, l, g, :t] = lse / math.log(2.0)
                out[b, l, g, :t] = torch.einsum("gtn,nd->gtd", (s - lse[..., None]).exp(), v)
    if not case["plan"]:
        return out, lse2
    return out, lse2, torch.tensor(words, dtype=torch.int32), torch.tensor(depth, dtype=torch.int32)


def _exact_pages(case, st):
    """The pages after a pass, sequence by sequence on the host's lists, rows copied as they are."""
    kind, page = case["kind"], case["page"]
    refs, table, lens = st["page_refs"].tolist(), st["page_table"].tolist(), st["seq_lens"].tolist()
    pools = [st["k_pages"], st["v_pages"]]

    def take():
        p = refs.index(0)
        refs[p] = 1
        return p

    def grow(s, n):
        at = lens[s] // page
        if n and lens[s] % page and refs[table[s][at]] > 1:
            old, table[s][at] = table[s][at], take()
            refs[old] -= 1
            for x in pools:
                x[:, table[s][at], :, :lens[s] % page] = x[:, old, :, :lens[s] % page]
        for p in range(-(-lens[s] // page), -(-(lens[s] + n) // page)):
            table[s][p] = take()
        lens[s] += n

    def put(s, first, k, v):                                             # k, v [L][H][rows][d]
        for x, y in zip(pools, (k, v)):
            done = 0
            while done < y.shape[2]:
                r = (first + done) % page
                m = min(page - r, y.shape[2] - done)
                x[:, table[s][(first + done) // page], :, r:r + m] = y[:, :, done:done + m]
                done += m

    if kind == "prompt":
        for b in range(case["batch"]):
            put(b, 0, st["k"][b], st["v"][b])
    elif kind == "commit":
        counts, idx = st["counts"].tolist(), st["idx"].long()
        for b in range(case["batch"]):
            grow(b, counts[b])
        for b in range(case["batch"]):
            pick = idx[b, :counts[b]]
            put(b, lens[b] - counts[b], st["k"][b][:, :, pick], st["v"][b][:, :, pick])
    elif kind == "compact":
        B, L, H, d, keep = case["batch"], case["layers"], case["hkv"], case["d"], case["keep"]
        for b in range(B):
            used = torch.tensor(table[b][:-(-case["rows"] // page)], device="cuda")
            for p in range(-(-keep // page)):
                table[B + b][p] = take()
            lens[B + b] = keep
            at = st["idx"][b].expand(L * H, keep) if case["shared"] else st["idx"].view(B, L * H, keep)[b]
            at = at.long().reshape(L, H, keep, 1).expand(L, H, keep, d)
            put(B + b, 0, *(x[:, used].transpose(1, 2).reshape(L, H, -1, d).gather(2, at) for x in pools))
    else:
        src, dst = st["src"].tolist(), st["dst"].tolist()
        for a, b in zip(src, dst):
            table[b], lens[b] = list(table[a]), lens[a]
            for p in table[b]:
                if p >= 0:
                    refs[p] += 1
        for b in dst:
            grow(b, case["new"])
    got = [pools[0], pools[1], _i32(refs), _i32(table), _i32(lens)]
    return tuple(got + [_i32([0]) for x in ("result", "result2") if x in st])


# --------------------------------------------------------------------- work
def work(case):
    B, L, H, d, page = (case[x] for x in ("batch", "layers", "hkv", "d", "page"))
    row = 2 * 2 * d * L * H                                              # K and V of a token, all layers and heads
    if case["kind"] == "tree":
        lens, live = _lens(case)
        hq, T = case["hq"], case["nodes"]
        bytes_, flops = 0, 0
        for n, t in zip(lens, live):
            bytes_ += (n + t) * row + L * hq * t * (2 * d * 2 + 4) + 4 * (-(-n // page)) + 4 * t * (-(-T // 32))
            flops += 4 * L * hq * t * d * (n + 1)
        return dict(bytes=bytes_, flops=flops)
    if case["kind"] == "prompt":
        return dict(bytes=2 * B * case["rows"] * row + 4 * B * -(-case["rows"] // page), flops=0)
    if case["kind"] == "commit":
        T = case["nodes"]
        r = random.Random(case["rows"] + 7 * T + B)
        for _ in range(B):
            _log(r, max(1, case["rows"] // 8), case["rows"])
        n = sum(r.randint(1, min(T, 8)) for _ in range(B))
        return dict(bytes=2 * n * row + 4 * (3 * B + n), flops=0)
    if case["kind"] == "compact":
        return dict(bytes=2 * B * case["keep"] * row + 4 * case["keep"] * B * (1 if case["shared"] else L * H), flops=0)
    S = max(1, B // 4)
    lens = [case["rows"] - (case["rows"] * i) // (3 * S) for i in range(S)]
    tail = sum(n % page for n in lens) / S                               # rows of a shared last page, on average
    table = sum(-(-n // page) for n in lens) / S
    return dict(bytes=B * (2 * tail * row + 4 * 4 * table), flops=0)
