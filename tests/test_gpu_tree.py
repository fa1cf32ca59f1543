"""Tree attention over a paged cache and the trees' visibility words, through
the C ABI, against plain 64-bit implementations: both element types and head
sizes, groups of 1 to 8 heads, one node to many, empty sequences, rows that see
nothing, nodes that do not count, pages that end inside a tile, NaN wherever
no row may look.

Tolerance of out, per element, with e = half a step of the element type and
A = the weights' sum of |v|: the result's rounding e |out|; the weights'
rounding e A; the logits, fp32 sums of up to 128 products (at most 2^-24 * 128
of the sum of |q||k|, below 4e-5 at the tests' scales) and the exponential's
2^-22: together below 2e-4 of A + |out|, the |out| through the normaliser.
Weights below the smallest normal number of fp16 keep 2^-25 of the largest:
n * 2^-25 * max|v|.  lse2: fp32 sums, 2e-4 by the same bound."""
import numpy as np
import pytest

from tests import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    from prompt_compression_b200 import build
    build.build_library()
    import prompt_compression_b200 as P
    P.spk_device_error(clear=True)
    return P


def build_case(seed, dtype, B, L, hq, hkv, d, T, page, lens, live=None, mask="tree", tree=True, spare=1, scale=None,
               seqs=None, n_seqs=None):
    """Tensors on the GPU, with NaN in every row that no result may look at,
    and their fp64 copies by sequence."""
    import torch
    rng = np.random.default_rng(seed)
    live = [T] * B if live is None else live
    seqs_l = list(range(B)) if seqs is None else seqs
    n_seqs = max(seqs_l) + 1 if n_seqs is None else n_seqs
    max_pages = max(1, max(-(-n // page) for n in lens)) + spare
    need = sum(-(-n // page) for n in lens)
    n_pages = need + 2
    order = rng.permutation(n_pages)[:need]
    table = np.full((n_seqs, max_pages), -1, np.int32)
    seq_lens = np.zeros(n_seqs, np.int32)

    def half(x):
        return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype)

    kp = torch.full((L, n_pages, hkv, page, d), float("nan"), dtype=dtype)
    vp = torch.full_like(kp, float("nan"))
    at = 0
    for b, n in zip(seqs_l, lens):
        seq_lens[b] = n
        for x in range(-(-n // page)):
            pg = int(order[at])
            at += 1
            table[b, x] = pg
            r = min(page, n - x * page)
            kp[:, pg, :, :r] = half(rng.standard_normal((L, hkv, r, d)))
            vp[:, pg, :, :r] = half(rng.standard_normal((L, hkv, r, d)))
    q = half(rng.standard_normal((B, L, hq, T, d)))
    kt = vt = None
    if tree:
        kt, vt = half(rng.standard_normal((B, L, hkv, T, d))), half(rng.standard_normal((B, L, hkv, T, d)))
        for b in range(B):
            kt[b, :, :, live[b]:] = float("nan")
            vt[b, :, :, live[b]:] = float("nan")
    sees = np.zeros((B, T, T), bool)
    words = np.zeros((B, T, (T + 31) // 32), np.int32)
    parents = np.array([[int(rng.integers(-1, i)) for i in range(T)] for _ in range(B)], np.int32)
    for b in range(B):
        if mask == "tree":
            words[b], _ = R.mask_words(parents[b], live[b])
        elif mask == "random":                       # any bits, some rows empty, some beyond the live nodes
            w = rng.integers(0, 1 << 32, size=words[b].shape, dtype=np.uint64).astype(np.uint32)
            w[rng.random(T) < 0.3] = 0
            words[b] = w.view(np.int32)
        else:
            for i in range(T):
                sees[b, i, :i + 1] = True
        if mask != "chain":
            for i in range(T):
                for j in range(T):
                    sees[b, i, j] = (int(words[b, i, j // 32]) >> (j % 32)) & 1
        sees[b, :, live[b]:] = False
    t = dict(q=q.cuda(), k_pages=kp.cuda(), v_pages=vp.cuda(), page_table=torch.from_numpy(table).cuda(),
             seq_lens=torch.from_numpy(seq_lens).cuda(), k_tree=None if kt is None else kt.cuda(),
             v_tree=None if vt is None else vt.cuda(),
             mask=None if mask == "chain" else torch.from_numpy(words).cuda(),
             n_live=torch.tensor(live, dtype=torch.int32, device="cuda"), scale=d ** -0.5 if scale is None else scale,
             seqs=None if seqs is None else torch.tensor(seqs, dtype=torch.int32, device="cuda"))
    host = dict(q=q.double().numpy(), kp=kp.double().numpy(), vp=vp.double().numpy(), table=table, lens=lens, live=live,
                kt=None if kt is None else kt.double().numpy(), vt=None if vt is None else vt.double().numpy(),
                sees=sees, page=page, seqs=seqs_l, scale=t["scale"])
    return t, host


def reference(h, units=None):
    B, L, hq, T, d = h["q"].shape
    hkv = h["kp"].shape[2]
    g = hq // hkv
    out, lse2, mag = np.zeros(h["q"].shape), np.zeros((B, L, hq, T)), np.zeros(h["q"].shape)
    for b in range(B):
        n, lv = h["lens"][b], h["live"][b]
        pages = h["table"][h["seqs"][b], :-(-n // h["page"])]
        for l in range(L):
            for x in range(hkv):
                k = h["kp"][l, pages, x].reshape(-1, d)[:n]
                v = h["vp"][l, pages, x].reshape(-1, d)[:n]
                s = slice(x * g, (x + 1) * g)
                kt = None if h["kt"] is None else h["kt"][b, l, x, :lv]
                vt = None if h["vt"] is None else h["vt"][b, l, x, :lv]
                o, ls, a = R.tree_rows(h["q"][b, l, s, :lv], k, v, kt, vt, h["sees"][b][:lv, :lv], h["scale"])
                out[b, l, s, :lv], lse2[b, l, s, :lv], mag[b, l, s, :lv] = o, ls, a
    return out, lse2, mag


def check(P, t, h, dtype, **more):
    import torch
    out = torch.full_like(t["q"], 7.0)
    lse2 = torch.full(t["q"].shape[:-1], 7.0, dtype=torch.float32, device="cuda")
    got = P.tree_attention(**t, out=out, lse2=lse2, **more)
    torch.cuda.synchronize()
    assert got is out
    assert P.spk_device_error() == (0, 0)
    compare(out, lse2, h, dtype)
    return out, lse2


def compare(out, lse2, h, dtype):
    import torch
    ref, ref_lse, mag = reference(h)
    o, ls = out.double().cpu().numpy(), lse2.double().cpu().numpy()
    e = torch.finfo(dtype).eps / 2
    vmax = 6.0
    n = max(h["lens"]) + h["q"].shape[3]
    tol = e * (np.abs(ref) + mag) + 2e-4 * (mag + np.abs(ref))
    if dtype == torch.float16:
        tol = tol + n * 2.0 ** -25 * vmax
    for b, lv in enumerate(h["live"]):
        assert (o[b, :, :, lv:] == 7.0).all() and (ls[b, :, :, lv:] == 7.0).all(), "rows of dead nodes were written"
        err, ok = np.abs(o[b] - ref[b])[:, :, :lv], tol[b][:, :, :lv]
        assert (err <= ok).all(), f"element {b}: worst {np.nanmax(err / np.maximum(ok, 1e-30)):.2f} of the tolerance, " \
            f"{np.isnan(err).sum()} NaN"
        a, r = ls[b, :, :, :lv], ref_lse[b, :, :, :lv]
        assert np.array_equal(np.isneginf(a), np.isneginf(r))
        fin = np.isfinite(r)
        assert (np.abs(a[fin] - r[fin]) <= 2e-4).all()


CASES = [
    # seed, dtype, B, L, hq, hkv, d, T, page, lens, live, mask, tree
    (1, "bf16", 1, 1, 8, 8, 128, 1, 16, [1], None, "tree", True),              # one row, one token
    (2, "bf16", 1, 1, 8, 2, 128, 1, 64, [300], None, "chain", True),           # single-token decoding
    (3, "bf16", 2, 1, 4, 2, 64, 1, 32, [0, 65], None, "tree", False),          # an empty cache and no tree: zeros
    (4, "bf16", 1, 2, 10, 2, 128, 7, 64, [320], None, "tree", True),           # g = 5, 35 rows: a 64-row tile
    (5, "fp16", 3, 1, 8, 2, 128, 4, 16, [129, 64, 3], [4, 2, 1], "tree", True),
    (6, "bf16", 2, 1, 14, 2, 64, 8, 48, [500, 47], [8, 5], "tree", True),      # g = 7, pages across tiles
    (7, "fp16", 1, 1, 8, 1, 64, 33, 128, [257], None, "tree", True),           # 264 rows: five row tiles
    (8, "bf16", 2, 2, 4, 4, 128, 64, 24, [63, 200], [64, 1], "random", True),  # rows that see only the cache
    (9, "bf16", 2, 1, 4, 4, 128, 16, 8, [0, 0], [16, 9], "random", True),      # no cache: some rows see nothing
    (10, "bf16", 1, 1, 2, 1, 128, 130, 64, [100], None, "chain", True),        # three node tiles, words 0 .. 4
    (11, "bf16", 3, 1, 16, 2, 128, 2, 16, [2500, 1, 900], [2, 2, 0], "tree", True),  # split over shares; no live node
    (12, "fp16", 1, 1, 5, 1, 128, 13, 64, [4097], [12], "random", True),       # 65 rows
    (13, "bf16", 1, 1, 8, 8, 64, 5, 40, [511], None, "chain", True),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c[0]) for c in CASES])
def test_tree_attention_parity(P, case):
    import torch
    seed, dt, B, L, hq, hkv, d, T, page, lens, live, mask, tree = case
    dtype = torch.bfloat16 if dt == "bf16" else torch.float16
    t, h = build_case(seed, dtype, B, L, hq, hkv, d, T, page, lens, live, mask, tree)
    check(P, t, h, dtype)


def test_sequences_of_a_larger_table_and_peaked_rows(P):
    import torch
    t, h = build_case(20, torch.bfloat16, 3, 1, 8, 2, 128, 6, 32, [70, 1000, 31], [6, 3, 6], seqs=[5, 0, 2], n_seqs=9,
                      scale=1.0)
    check(P, t, h, torch.bfloat16)


def test_the_same_sequence_twice(P):
    # two trees over one sequence: the batch elements read the same pages
    import torch
    t, h = build_case(21, torch.bfloat16, 2, 1, 4, 2, 64, 3, 16, [90, 90], seqs=[0, 1])
    t["seqs"] = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    h["seqs"] = [1, 1]
    check(P, t, h, torch.bfloat16)


def test_results_do_not_depend_on_the_workspace(P):
    import torch
    t, h = build_case(22, torch.bfloat16, 1, 1, 8, 2, 128, 9, 64, [3000])
    shape = P.tree_shape(t["q"], t["k_pages"], t["page_table"], t["scale"])
    ws = torch.full((P.tree_attention_workspace_size(shape),), 255, dtype=torch.uint8, device="cuda")
    a, la = check(P, t, h, torch.bfloat16, workspace=ws)
    b, lb = check(P, t, h, torch.bfloat16)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_captured_and_replayed_with_a_longer_sequence(P):
    # the lengths are read when the graph runs: a captured call serves every step
    import torch
    t, h = build_case(23, torch.bfloat16, 2, 1, 8, 2, 128, 3, 16, [700, 40], spare=2)
    full = t["seq_lens"].clone()
    shape = P.tree_shape(t["q"], t["k_pages"], t["page_table"], t["scale"])
    ws = torch.empty(P.tree_attention_workspace_size(shape), dtype=torch.uint8, device="cuda")
    out, lse2 = torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:-1], 7.0, device="cuda")
    t["seq_lens"].copy_(torch.tensor([1, 40], dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        P.tree_attention(**t, out=out, lse2=lse2, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.tree_attention(**t, out=out, lse2=lse2, workspace=ws)
    for lens in ([1, 40], full.tolist()):
        t["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        h["lens"] = lens
        graph.replay()
        torch.cuda.synchronize()
        compare(out, lse2, h, torch.bfloat16)
    assert P.spk_device_error() == (0, 0)


def test_on_another_stream(P):
    import torch
    t, h = build_case(24, torch.bfloat16, 1, 1, 8, 2, 128, 5, 16, [400])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = P.tree_attention(**t, stream=side)
    side.synchronize()
    ref = P.tree_attention(**t)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


@pytest.mark.parametrize("T,hq,lens,dt", [(6, 4, [200, 9], "bf16"), (40, 4, [300, 64], "fp16"), (40, 16, [500, 3], "bf16"),
                                          (150, 8, [129, 0], "bf16")])
def test_nodes_that_a_row_does_not_see_may_hold_anything(P, T, hq, lens, dt):
    # node 2 has NaN, infinities and huge values in K and V: the rows that see it
    # get what the sums give, the others do not notice
    import torch
    dtype = torch.bfloat16 if dt == "bf16" else torch.float16
    t, h = build_case(30 + T, dtype, 2, 1, hq, 2, 128, T, 32, lens, mask="random")
    seen = h["sees"][:, :, 2].copy()
    clean = {x: t[x].clone() for x in ("k_tree", "v_tree")}
    t["v_tree"][:, :, :, 2, 0] = float("nan")
    t["v_tree"][:, :, :, 2, 1] = float("inf")
    t["v_tree"][:, :, :, 2, 2] = float("-inf")
    out, lse2 = (torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:-1], 7.0, device="cuda"))
    P.tree_attention(**t, out=out, lse2=lse2)
    torch.cuda.synchronize()
    got = out.float().cpu().numpy()
    for b in range(2):
        rows = got[b][:, :, seen[b], :]
        assert np.isnan(rows[..., 0]).all() and np.isposinf(rows[..., 1]).all() and np.isneginf(rows[..., 2]).all()
    t["v_tree"], h["vt"] = clean["v_tree"], clean["v_tree"].double().cpu().numpy()
    ref = torch.full_like(t["q"], 7.0)
    P.tree_attention(**t, out=ref)
    torch.cuda.synchronize()
    ref = ref.float().cpu().numpy()
    for b in range(2):
        assert np.array_equal(got[b][:, :, ~seen[b]], ref[b][:, :, ~seen[b]])
        assert np.array_equal(got[b][:, :, seen[b], 3:], ref[b][:, :, seen[b], 3:])
    t["k_tree"][:, :, :, 2] = float("nan")                          # hidden keys: not even the maximum sees them
    bad = torch.full_like(t["q"], 7.0)
    P.tree_attention(**t, out=bad)
    torch.cuda.synchronize()
    bad = bad.float().cpu().numpy()
    for b in range(2):
        assert np.array_equal(bad[b][:, :, ~seen[b]], ref[b][:, :, ~seen[b]])
        assert np.isnan(bad[b][:, :, seen[b]]).all()
    assert P.spk_device_error() == (0, 0)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,hq,lens", [(6, 4, [40]), (6, 4, [3000]), (40, 4, [40]), (40, 4, [3000]), (40, 16, [60]),
                                       (40, 16, [3000, 50]), (150, 8, [2500])],
                         ids=["narrow", "narrow-cut", "wide", "wide-cut", "pair", "pair-cut", "nodes-cut"])
def test_what_is_not_finite_adds_up_whole_or_cut(P, T, hq, lens, dt):
    import torch
    dtype = torch.bfloat16 if dt == "bf16" else torch.float16
    t, h = build_case(70 + T, dtype, len(lens), 1, hq, 2, 64, T, 32, lens, mask="random")
    not_finite_adds_up(P, t, h)


@pytest.mark.parametrize("B,hq,T,most", [(80, 16, 3, 700), (40, 32, 10, 900), (40, 64, 20, 900)], ids=["narrow", "wide", "pair"])
def test_what_is_not_finite_adds_up_where_the_main_kernel_joins(P, B, hq, T, most):
    import torch
    rng = np.random.default_rng(170 + T)
    t, h = build_case(170 + T, torch.bfloat16, B, 1, hq, 8, 64, T, 32, [int(x) for x in rng.integers(40, most, B)], mask="random")
    not_finite_adds_up(P, t, h)


def not_finite_adds_up(P, t, h):
    # in one share or in many: NaN logits beside an infinite V, infinities of both signs,
    # an infinite V whose weight is too small for 32 bits
    import torch
    B, T = t["q"].shape[0], t["q"].shape[3]
    t["q"] = t["q"].abs()
    t["mask"][:, :, 0] &= ~4                                         # odd nodes see node 2, even ones do not
    t["mask"][:, 1::2, 0] |= 4
    seen = np.broadcast_to(np.arange(T) % 2 == 1, (B, T))
    names = ("k_tree", "v_tree", "v_pages")

    def call(**change):
        a = dict(t, **change)
        out, lse2 = torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:-1], 7.0, device="cuda")
        P.tree_attention(**a, out=out, lse2=lse2)
        torch.cuda.synchronize()
        return out.float().cpu().numpy(), lse2.cpu().numpy()

    ref, ref_lse = call()
    clean = {x: t[x].clone() for x in names}

    k, v = clean["k_tree"].clone(), clean["v_tree"].clone()          # a NaN logit: the row is NaN, infinite V or not
    k[:, :, :, 2], v[:, :, :, 2, 0] = float("nan"), float("inf")
    out, lse2 = call(k_tree=k, v_tree=v)
    for b in range(B):
        assert np.isnan(out[b][:, :, seen[b]]).all() and np.isnan(lse2[b][:, :, seen[b]]).all()
        assert np.array_equal(out[b][:, :, ~seen[b]], ref[b][:, :, ~seen[b]])
        assert np.array_equal(lse2[b][:, :, ~seen[b]], ref_lse[b][:, :, ~seen[b]])

    v, pages = clean["v_tree"].clone(), clean["v_pages"].clone()     # -inf in the cache, +inf in the node: NaN for who sees both
    v[:, :, :, 2, 1] = float("inf")
    for b in range(B):
        pages[:, h["table"][b][0], :, 3, 1] = float("-inf")
    out, lse2 = call(v_tree=v, v_pages=pages)
    assert np.array_equal(lse2, ref_lse)
    for b in range(B):
        assert np.isnan(out[b][:, :, seen[b], 1]).all()
        assert np.isneginf(out[b][:, :, ~seen[b], 1]).all()
        rest = [x for x in range(64) if x != 1]
        assert np.array_equal(out[b][..., rest], ref[b][..., rest])

    k, v = clean["k_tree"].clone(), clean["v_tree"].clone()          # a weight below 2^-1000: infinity all the same
    k[:, :, :, 2], v[:, :, :, 2, 0] = -1000.0, float("inf")
    out, lse2 = call(k_tree=k, v_tree=v)
    for b in range(B):
        assert np.isposinf(out[b][:, :, seen[b], 0]).all()
        assert np.isfinite(out[b][:, :, seen[b], 1:]).all() and np.isfinite(lse2[b]).all()
        assert np.array_equal(out[b][:, :, ~seen[b]], ref[b][:, :, ~seen[b]])
    assert P.spk_device_error() == (0, 0)


@pytest.mark.parametrize("T,hq", [(6, 4), (40, 4), (40, 16)], ids=["narrow", "wide", "pair"])
@pytest.mark.parametrize("lens", [[500], [4000]], ids=["few-tiles", "cut"])
def test_a_tile_of_keys_whose_logits_are_all_minus_infinity(P, T, hq, lens):
    # the first 128 rows have infinite K against the queries' sign: their weights are 0, the others as without them
    import torch
    t, h = build_case(90 + T, torch.bfloat16, 1, 1, hq, 2, 64, T, 32, lens)
    t["q"] = t["q"].abs() + 0.25
    h["q"] = t["q"].double().cpu().numpy()
    pages = h["table"][0][:4]
    t["k_pages"][:, pages.tolist()] = float("-inf")
    out, lse2 = torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:-1], 7.0, device="cuda")
    P.tree_attention(**t, out=out, lse2=lse2)
    torch.cuda.synchronize()
    assert P.spk_device_error() == (0, 0)
    h["table"] = h["table"][:, 4:]
    h["lens"] = [lens[0] - 128]
    compare(out, lse2, h, torch.bfloat16)


@pytest.mark.parametrize("case", [
    # seed, B, L, hq, hkv, d, T, page, lens: many units, ragged, so that shares cut them in two
    (40, 40, 2, 16, 8, 64, 1, 16, 300),          # 640 units of 2 rows
    (41, 44, 1, 32, 8, 128, 5, 32, 700),         # 352 units of 20 rows, items cut where a share ends
    (42, 20, 2, 40, 8, 128, 9, 64, 520),         # 320 units of 45 rows
    (43, 38, 1, 16, 4, 64, 40, 24, 400),         # 152 units of 160 rows: pairs of query tiles
    (44, 19, 1, 64, 8, 128, 40, 16, 300),        # 152 units of 320 rows: a pair and a single
])
def test_many_ragged_units(P, case):
    import torch
    seed, B, L, hq, hkv, d, T, page, most = case
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(0, most, B)]
    live = [int(x) for x in rng.integers(1, T + 1, B)]
    t, h = build_case(seed, torch.bfloat16, B, L, hq, hkv, d, T, page, lens, live, "tree")
    check(P, t, h, torch.bfloat16)


def test_many_runs_of_one_query_tile_that_end_in_ragged_tiles(P):
    # 128 units of 96 rows, several runs of each block: a run's last V is cleared behind its
    # keys, which must wait for the products of the V before it in the same place
    import torch
    rng = np.random.default_rng(45)
    lens = [int(x) for x in rng.integers(200, 3000 + 1, 16)]
    live = [int(x) for x in rng.integers(12, 25, 16)]
    t, h = build_case(45, torch.float16, 16, 1, 32, 8, 128, 24, 32, lens, live, "tree")
    out, lse2 = check(P, t, h, torch.float16)
    for _ in range(30):
        o, l = torch.full_like(out, 7.0), torch.full_like(lse2, 7.0)
        P.tree_attention(**t, out=o, lse2=l)
        assert torch.equal(o, out) and torch.equal(l, lse2)


@pytest.mark.parametrize("case", [
    # seed, B, hq, hkv, d, T, page, most: shares of a few jobs more than an item's start
    # counts for, so that borders fall before an item's first tile
    (60, 24, 32, 8, 128, 24, 32, 900),           # tcgen05, one query tile
    (61, 10, 32, 8, 64, 40, 24, 1100),           # pairs of query tiles
    (62, 40, 16, 8, 128, 3, 16, 800),            # 320 units of six rows
])
def test_borders_before_the_first_tile_of_an_item(P, case):
    import torch
    seed, B, hq, hkv, d, T, page, most = case
    rng = np.random.default_rng(seed)
    lens = [0 if b % 7 == 3 else int(x) for b, x in enumerate(rng.integers(1, most, B))]
    live = [0 if b % 11 == 5 else int(x) for b, x in enumerate(rng.integers(1, T + 1, B))]
    t, h = build_case(seed, torch.bfloat16, B, 1, hq, hkv, d, T, page, lens, live, "tree")
    out, lse2 = check(P, t, h, torch.bfloat16)
    o, l = torch.full_like(out, 7.0), torch.full_like(lse2, 7.0)
    P.tree_attention(**t, out=o, lse2=l)
    assert torch.equal(o, out) and torch.equal(l, lse2)


def test_long_rows_of_two_query_tiles_and_more(P):
    import torch
    t, h = build_case(50, torch.bfloat16, 1, 1, 10, 2, 64, 64, 64, [6000], None, "tree")      # 320 rows, 47 tiles
    check(P, t, h, torch.bfloat16)


def test_two_calls_at_once(P):
    # different streams, workspaces of their own
    import torch
    a, ha = build_case(51, torch.bfloat16, 2, 1, 8, 2, 128, 5, 16, [700, 90])
    b, hb = build_case(52, torch.float16, 1, 1, 16, 2, 64, 20, 32, [900])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):
        outs.append((P.tree_attention(**a, stream=s1), P.tree_attention(**b, stream=s2)))
    torch.cuda.synchronize()
    ra, rb = P.tree_attention(**a), P.tree_attention(**b)
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, ra) and torch.equal(y, rb)


def test_a_pool_beyond_32_bit_offsets(P):
    # the sequence's pages lie behind 2^31 elements of the pool
    import torch
    t, h = build_case(53, torch.bfloat16, 1, 1, 4, 1, 128, 3, 64, [200])
    n_pages = (1 << 31) // (64 * 128) + 10
    kp = torch.zeros((1, n_pages, 1, 64, 128), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    old = t["k_pages"].shape[1]
    kp[:, n_pages - old:], vp[:, n_pages - old:] = t["k_pages"], t["v_pages"]
    t["page_table"] = torch.where(t["page_table"] >= 0, t["page_table"] + (n_pages - old), t["page_table"])
    t["k_pages"], t["v_pages"] = kp, vp
    check(P, t, h, torch.bfloat16)


def test_bad_elements_keep_their_rows_and_are_recorded(P):
    import torch
    t, h = build_case(25, torch.bfloat16, 3, 1, 4, 2, 64, 2, 16, [60, 60, 60], seqs=[0, 1, 2])
    t["seqs"] = torch.tensor([0, 7, 2], dtype=torch.int32, device="cuda")
    out = torch.full_like(t["q"], 7.0)
    P.tree_attention(**t, out=out)
    st, _ = P.spk_device_error(clear=True)
    assert st == P.binding.SPK_ERR_ARG
    assert (out[1] == 7.0).all() and not (out[0] == 7.0).any() and not (out[2] == 7.0).any()
    t["seqs"] = None
    t["n_live"] = torch.tensor([2, 2, 3], dtype=torch.int32, device="cuda")
    out = torch.full_like(t["q"], 7.0)
    P.tree_attention(**t, out=out)
    st, _ = P.spk_device_error(clear=True)
    assert st == P.binding.SPK_ERR_ARG
    assert (out[2] == 7.0).all() and not (out[0] == 7.0).any()


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 200, 1024])
def test_tree_mask(P, T):
    import torch
    rng = np.random.default_rng(T)
    B = 3
    parents = np.array([[int(rng.integers(-1, i)) for i in range(T)] for _ in range(B)], np.int32)
    parents[1] = np.arange(T) - 1                                   # a chain
    live = [T, max(0, T - 3), (T + 1) // 2]
    mask, depth = P.tree_mask(torch.from_numpy(parents).cuda(), torch.tensor(live, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert P.spk_device_error() == (0, 0)
    for b in range(B):
        w, dp = R.mask_words(parents[b], live[b])
        assert np.array_equal(mask[b].cpu().numpy(), w)
        assert np.array_equal(depth[b].cpu().numpy(), dp)


def test_tree_mask_of_wrong_parents(P):
    import torch
    parents = torch.tensor([[-1, 1, 0, 7, -2]], dtype=torch.int32, device="cuda")
    mask, depth = P.tree_mask(parents)
    st, _ = P.spk_device_error(clear=True)
    assert st == P.binding.SPK_ERR_ARG
    assert mask[0, :, 0].tolist() == [1, 2, 5, 8, 16] and depth[0].tolist() == [0, 0, 1, 0, 0]


GIVE_UP = [
    # seed, B, L, hq, hkv, T, page, most, sites: shares that cut items; both ways of joining them
    (80, 20, 2, 32, 8, 10, 16, 700, range(620, 690)),     # tcgen05, 320 items, joined inside
    (81, 2, 1, 32, 8, 10, 16, 6000, range(620, 690)),     # tcgen05, 16 items
    (82, 40, 2, 16, 8, 3, 16, 700, range(600, 620)),      # mma.sync, 640 items, joined inside
    (83, 1, 1, 16, 8, 3, 16, 6000, range(600, 620)),      # mma.sync, 8 items
]


@pytest.mark.parametrize("case", GIVE_UP, ids=["wide-inside", "wide", "narrow-inside", "narrow"])
def test_waits_that_run_out_end_the_kernel(P, case):
    # two CTAs lose work: their waits give up after 2 s and say so, and the same call behind it is right
    import time

    import torch
    seed, B, L, hq, hkv, T, page, most, sites = case
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(most // 2, most, B)]
    t, h = build_case(seed, torch.bfloat16, B, L, hq, hkv, 64, T, page, lens)
    shape = P.tree_shape(t["q"], t["k_pages"], t["page_table"], t["scale"])
    ws = torch.full((P.tree_attention_workspace_size(shape),), 255, dtype=torch.uint8, device="cuda")
    out, lse2 = torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:-1], 7.0, device="cuda")
    torch.cuda.synchronize()
    t0 = time.monotonic()
    P.spk_selftest_tree_give_up(**t, out=out, lse2=lse2, workspace=ws)
    torch.cuda.synchronize()
    assert 1.5 < time.monotonic() - t0 < 10.0
    status, where = P.spk_device_error(clear=True)
    assert status == P.binding.SPK_ERR_TIMEOUT and where in sites
    compare(out, lse2, h, torch.bfloat16)
    # the words that count a cut item's shares lie behind the partial results: none is left in between
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ctas, item_rows = (sms, 128) if hq // hkv * T > 32 else (2 * sms, 8)
    counts = ws[ctas * 2 * item_rows * (64 + 2) * 4:][:ctas * 8].view(torch.int64)
    used = counts != -1
    assert bool(used.any()) == (B * L * hkv >= 2 * ctas) and not (counts[used] & 0xffff).any()
    assert P.spk_device_error() == (0, 0)


@pytest.mark.parametrize("case", [
    # seed, B, hq, T, long, short, dead: twice as many items as CTAs, and one sequence whose items lie in tens of shares
    (100, 74, 16, 1, 16384, 40, True),           # mma.sync, one element with a live node
    (101, 80, 16, 3, 9000, 200, False),
    (102, 37, 32, 10, 16384, 40, True),          # tcgen05
    (103, 40, 32, 10, 12000, 200, False),
    (104, 40, 64, 20, 8000, 100, False),         # pairs of query tiles: 160 rows
], ids=["narrow-dead", "narrow", "wide-dead", "wide", "pair"])
def test_one_long_sequence_among_many_short_ones(P, case):
    import torch
    seed, B, hq, T, most, short, dead = case
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(1, short, B)]
    live = [0 if dead else int(x) for x in rng.integers(0, T + 1, B)]
    lens[B // 3], live[B // 3] = most, T
    t, h = build_case(seed, torch.bfloat16, B, 1, hq, 8, 64, T, 64, lens, live)
    out, lse2 = check(P, t, h, torch.bfloat16)
    for _ in range(5):
        o, l = torch.full_like(out, 7.0), torch.full_like(lse2, 7.0)
        P.tree_attention(**t, out=o, lse2=l)
        assert torch.equal(o, out) and torch.equal(l, lse2)


@pytest.mark.parametrize("case", [
    # seed, dtype, B, hq, hkv, d, T, page, lens, live, mask: forms that the cases above leave out
    (110, "fp16", 2, 8, 2, 128, 1, 16, [700, 1], None, "tree"),           # one token in fp16
    (111, "fp16", 1, 8, 8, 64, 1, 24, [65], None, "chain"),
    (112, "fp16", 2, 16, 2, 128, 33, 48, [300, 129], [33, 20], "tree"),   # 264 rows, fp16, head size 128
    (113, "fp16", 1, 4, 1, 128, 40, 64, [5000], None, "random"),          # 160 rows, cut
    (114, "bf16", 1, 2, 1, 64, 1024, 16, [77], None, "tree"),             # the most nodes: 2048 rows, 8 node tiles
    (115, "bf16", 2, 1, 1, 128, 700, 8, [0, 333], [700, 513], "random"),
    (116, "fp16", 1, 1, 1, 64, 257, 32, [96], [256], "chain"),
], ids=[str(x) for x in range(110, 117)])
def test_more_forms(P, case):
    import torch
    seed, dt, B, hq, hkv, d, T, page, lens, live, mask = case
    dtype = torch.bfloat16 if dt == "bf16" else torch.float16
    t, h = build_case(seed, dtype, B, 1, hq, hkv, d, T, page, lens, live, mask)
    check(P, t, h, dtype)


@pytest.mark.parametrize("T,hq", [(3, 4), (12, 16), (40, 16)], ids=["narrow", "wide", "pair"])
@pytest.mark.parametrize("page", [24, 128])
def test_pages_out_of_range_are_read_as_zeros_and_recorded(P, T, hq, page):
    import torch
    t, h = build_case(120 + T, torch.bfloat16, 2, 1, hq, 2, 64, T, page, [5 * page + 7, 100])
    n_pages = t["k_pages"].shape[1]
    zero = np.zeros_like(h["kp"][:, :1])
    h["kp"], h["vp"] = np.concatenate([h["kp"], zero], 1), np.concatenate([h["vp"], zero], 1)
    for at, bad in ((0, n_pages), (2, -1), (4, 0x7fffffff), (5, -0x80000000)):
        t["page_table"][0, at] = bad
        h["table"][0, at] = n_pages                                  # the zeros
    out, lse2 = torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:-1], 7.0, device="cuda")
    P.tree_attention(**t, out=out, lse2=lse2)
    torch.cuda.synchronize()
    assert P.spk_device_error(clear=True)[0] == P.binding.SPK_ERR_ARG
    compare(out, lse2, h, torch.bfloat16)


@pytest.mark.parametrize("T,hq", [(3, 4), (12, 16), (40, 16)], ids=["narrow", "wide", "pair"])
@pytest.mark.parametrize("length", [-1, -0x80000000, 161, 0x7fffffff])
def test_lengths_out_of_range_keep_their_rows_and_are_recorded(P, T, hq, length):
    import torch
    t, h = build_case(130 + T, torch.bfloat16, 3, 1, hq, 2, 64, T, 16, [140, 100, 9], spare=1)      # ten pages of 16 rows
    assert t["page_table"].shape[1] == 10
    t["seq_lens"][1] = length
    h["live"] = [T, 0, T]                                            # element 1 has no rows
    out, lse2 = torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:-1], 7.0, device="cuda")
    P.tree_attention(**t, out=out, lse2=lse2)
    torch.cuda.synchronize()
    assert P.spk_device_error(clear=True)[0] == P.binding.SPK_ERR_ARG
    compare(out, lse2, h, torch.bfloat16)


@pytest.mark.parametrize("T,hq", [(3, 4), (12, 16), (40, 16)], ids=["narrow", "wide", "pair"])
def test_no_keys_at_all(P, T, hq):
    # an empty sequence beside one with rows, and no nodes to see: zeros, and -inf
    import torch
    t, h = build_case(140 + T, torch.bfloat16, 3, 2, hq, 2, 64, T, 16, [0, 140, 0], tree=False)
    out, lse2 = check(P, t, h, torch.bfloat16)
    assert (out[0] == 0).all() and torch.isneginf(lse2[0]).all()
    t, h = build_case(141 + T, torch.float16, 1, 1, hq, 2, 128, T, 16, [0], tree=False)
    check(P, t, h, torch.float16)
