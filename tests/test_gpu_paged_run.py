"""The paged cache as a decoding loop uses it: a prompt compressed into pages,
trees of drafted tokens checked against it, the accepted path committed, the
sequence forked, rolled back, compacted again and freed; and where the paged
operators meet the contiguous ones (kv_compact's rows, decode_attention)."""
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


def _randn(shape, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(cache, s):
    """K and V of a sequence, [L][Hkv][n][d]."""
    n, page = int(cache.seq_lens[s]), cache.page_rows
    pages = cache.page_table[s, :-(-n // page)].long()
    out = []
    for pool in (cache.k_pages, cache.v_pages):
        x = pool[:, pages].transpose(1, 2)
        out.append(x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])[:, :, :n])
    return out


def test_a_decoding_loop(P):
    import torch
    B, L, hq, hkv, d, n_in, nw, nl, c_max, page, T = 2, 2, 8, 2, 64, 900, 32, 32, 100, 16, 7
    cache = P.PagedCache(L, 100, hkv, page, d, n_seqs=5, max_pages=20)
    q, k, v = _randn((B, L, hq, nw + nl, d), 1, d ** -0.5), _randn((B, L, hkv, n_in, d), 2), _randn((B, L, hkv, n_in, d), 3)
    scores, idx, result = P.speckv_compress_pages(q, k, v, nw, c_max, cache, _i32([3, 1]))
    buf = P.speckv_compress(q, k, v, nw, c_max)
    assert result.item() == 0 and torch.equal(idx, buf.idx) and torch.equal(scores, buf.scores)
    for b, s in enumerate((3, 1)):
        kr, vr = _rows(cache, s)
        assert torch.equal(kr, buf.k_out[b]) and torch.equal(vr, buf.v_out[b])

    rng = np.random.default_rng(7)
    seqs, held = _i32([3, 1]), {s: [x.clone() for x in _rows(cache, s)] for s in (3, 1)}
    for step in range(4):
        parents = np.array([[int(rng.integers(-1, i)) for i in range(T)] for _ in range(B)], np.int32)
        live = [T, int(rng.integers(2, T + 1))]
        mask, depth = P.tree_mask(torch.from_numpy(parents).cuda(), n_live=_i32(live))
        qt, kt, vt = (_randn((B, L, h, T, d), 10 * step + x) for x, h in ((4, hq), (5, hkv), (6, hkv)))
        lse2 = torch.empty((B, L, hq, T), device="cuda")
        out = cache.attend(qt, kt, vt, mask=mask, n_live=_i32(live), seqs=seqs, lse2=lse2, scale=d ** -0.5)
        for l in range(L):                                        # a layer at a time: the same
            one = P.tree_attention(qt[:, l:l + 1].contiguous(), cache.k_pages[l:l + 1], cache.v_pages[l:l + 1],
                                   cache.page_table, cache.seq_lens, kt[:, l:l + 1].contiguous(),
                                   vt[:, l:l + 1].contiguous(), mask=mask, n_live=_i32(live), seqs=seqs, scale=d ** -0.5)
            for b in range(B):
                diff = (one[b, 0, :, :live[b]].float() - out[b, l, :, :live[b]].float()).abs().max()
                assert diff <= 2 ** -6                            # other shares, other roundings: a step of values below 2
        paths = []
        for b, s in enumerate((3, 1)):
            sees = R.ancestors(parents[b])
            kr, vr = _rows(cache, s)
            assert torch.equal(kr, held[s][0]) and torch.equal(vr, held[s][1])
            vis = np.zeros((live[b], live[b]), bool)
            for i in range(live[b]):
                vis[i, sees[i]] = True
            for l in range(L):
                for h in range(hkv):
                    g = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                    ref, rl, mag = R.tree_rows(qt[b, l, g, :live[b]].double().cpu().numpy(), kr[l, h].double().cpu().numpy(),
                                               vr[l, h].double().cpu().numpy(), kt[b, l, h, :live[b]].double().cpu().numpy(),
                                               vt[b, l, h, :live[b]].double().cpu().numpy(), vis, d ** -0.5)
                    got = out[b, l, g, :live[b]].double().cpu().numpy()
                    # half a step for the result and half a step of the weights' sum of |v|; 2e-4 as in the parity tests
                    assert (np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + mag) + 2e-4 * (np.abs(ref) + mag)).all()
                    assert (np.abs(lse2[b, l, g, :live[b]].cpu().numpy() - rl) <= 2e-4).all()
            leaf = int(rng.integers(0, live[b]))
            paths.append(sees[leaf][::-1])
        counts = [len(x) for x in paths]
        path = _i32([x + [0] * (T - len(x)) for x in paths])
        assert cache.reserve(seqs, _i32(counts)).item() == 0
        cache.write(kt, vt, seqs, idx=path, counts=_i32(counts), units_per_idx=L * hkv)
        for b, s in enumerate((3, 1)):
            for x, new in ((0, kt), (1, vt)):
                held[s][x] = torch.cat([held[s][x], new[b][:, :, paths[b]]], 2)
            kr, vr = _rows(cache, s)
            assert torch.equal(kr, held[s][0]) and torch.equal(vr, held[s][1])

    n3 = int(cache.seq_lens[3])
    assert cache.fork(_i32([3, 3]), _i32([0, 4])).item() == 0     # two continuations
    assert cache.reserve(_i32([0, 3]), _i32([2, 1])).item() == 0  # each grows on its own
    extra = [_randn((2, L, hkv, 2, d), 90 + x) for x in range(2)]
    cache.write(*extra, _i32([0, 3]), counts=_i32([2, 1]))
    for s, b, c in ((0, 0, 2), (3, 1, 1), (4, 0, 0)):
        for x, rows in enumerate(_rows(cache, s)):
            assert torch.equal(rows[:, :, :n3], held[3][x]) and torch.equal(rows[:, :, n3:], extra[x][b][:, :, :c])
    cache.free(_i32([3, 0]), keep_rows=_i32([n3 - 3, 0]))         # rolled back; dropped
    for x, rows in enumerate(_rows(cache, 3)):
        assert torch.equal(rows, held[3][x][:, :, :n3 - 3])
    sel = torch.sort(torch.stack([torch.randperm(n3 - 3, device="cuda")[:50] for _ in range(L * hkv)]), 1)[0].to(torch.int32)
    assert cache.compact(_i32([3]), _i32([3]), sel).item() == 0   # compressed once more, in place
    for x, rows in enumerate(_rows(cache, 3)):
        want = held[3][x][:, :, :n3 - 3].gather(2, sel.view(L, hkv, 50, 1).long().expand(L, hkv, 50, d))
        assert torch.equal(rows, want)
    for x, rows in enumerate(_rows(cache, 4)):                    # the other continuation has its rows
        assert torch.equal(rows, held[3][x])
    cache.free(_i32([0, 1, 2, 3, 4]))
    assert int(cache.page_refs.abs().sum()) == 0 and int(cache.seq_lens.sum()) == 0
    assert P.spk_device_error() == (0, 0)


def test_a_single_token_is_decode_attention(P):
    # decode_attention's cache as one page a sequence: the same sums, rounded to bf16
    import torch
    L, hq, hkv, d, n = 3, 16, 4, 128, 328
    q, k, v = _randn((1, L, hq, d), 1), _randn((1, L, hkv, n, d), 2), _randn((1, L, hkv, n, d), 3)
    want = P.decode_attention(q, k, v, scale=d ** -0.5)
    got = P.tree_attention(q.view(1, L, hq, 1, d), k.view(L, 1, hkv, n, d), v.view(L, 1, hkv, n, d), _i32([[0]]), _i32([n]),
                           scale=d ** -0.5)
    # the result's rounding and the weights' (half a step each, of at most max|v|), decode_attention's own 1e-4
    bound = 2.0 ** -8 * (want.abs() + v.abs().max().float()) + 1e-4 * v.abs().max().float()
    assert ((got.view(1, L, hq, d).float() - want).abs() <= bound).all()
    assert P.spk_device_error() == (0, 0)


def test_two_graphs_of_a_step(P):
    # two captured steps that share the cache but not their workspaces, replayed in turn
    import torch
    L, hq, hkv, d, page = 1, 8, 2, 128, 32
    cache = P.PagedCache(L, 40, hkv, page, d, n_seqs=2, max_pages=16)
    seqs = [_i32([0]), _i32([1])]
    k, v = _randn((2, L, hkv, 70, d), 1), _randn((2, L, hkv, 70, d), 2)
    assert cache.reserve(_i32([0, 1]), _i32([70, 70])).item() == 0
    cache.write(k, v, _i32([0, 1]))
    qs = [_randn((1, L, hq, 3, d), 3 + s) for s in range(2)]
    kts, vts = [_randn((1, L, hkv, 3, d), 5 + s) for s in range(2)], [_randn((1, L, hkv, 3, d), 7 + s) for s in range(2)]
    outs = [torch.empty_like(x) for x in qs]
    one, ress = _i32([1]), [_i32([9]), _i32([9])]
    graphs = []
    for s in range(2):
        cache.attend(qs[s], kts[s], vts[s], seqs=seqs[s], out=outs[s], scale=0.1)      # before the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.attend(qs[s], kts[s], vts[s], seqs=seqs[s], out=outs[s], scale=0.1)
            cache.reserve(seqs[s], one, result=ress[s])
            cache.write(kts[s], vts[s], seqs[s], counts=one)
        graphs.append(g)
    for _ in range(5):
        for s in range(2):
            want = cache.attend(qs[s], kts[s], vts[s], seqs=seqs[s], scale=0.1)
            graphs[s].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[s], want) and ress[s].item() == 0
    assert cache.seq_lens.tolist() == [75, 75]
    for s in range(2):
        kr, _ = _rows(cache, s)
        assert torch.equal(kr[:, :, :70], k[s]) and torch.equal(kr[:, :, 70:], kts[s][0][:, :, :1].expand(-1, -1, 5, -1))
    assert P.spk_device_error() == (0, 0)


def test_rows_without_room_leave_the_cache_as_it_was(P):
    # a prompt whose kept rows find too few pages, and a list that names a sequence twice:
    # what the sequences hold is not written over; on a stream of its own too
    import torch
    L, hq, hkv, d, page, n_in, window = 2, 4, 2, 64, 16, 300, 16
    q, k, v = _randn((2, L, hq, 20, d), 1), _randn((2, L, hkv, n_in, d), 2), _randn((2, L, hkv, n_in, d), 3)
    kw = dict(n_window=window, c_max=32, scale=0.125)
    cache = P.PagedCache(L, 14, hkv, page, d, n_seqs=3, max_pages=12)
    both, side = _i32([0, 2]), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, idx, result = P.speckv_compress_pages(q, k, v, cache=cache, seqs=both, stream=side, **kw)
    side.synchronize()
    assert result.item() == 0 and cache.seq_lens.tolist() == [48, 0, 48]       # 6 of the 14 pages
    assert P.speckv_compress_pages(q, k, v, cache=cache, seqs=_i32([0, 2]), **kw)[2].item() == 0
    held = [x.clone() for x in cache.tensors]
    for seqs, want in (([0, 2], 4), ([0, 0], -1), ([0, 1], 4)):
        assert P.speckv_compress_pages(q, k, v, cache=cache, seqs=_i32(seqs), **kw)[2].item() == want
        for a, b in zip(cache.tensors[2:], held[2:]):
            assert torch.equal(a, b)
        for a, b in zip(cache.tensors[:2], held[:2]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert P.spk_device_error(clear=True)[0] == (0 if want > 0 else P.binding.SPK_ERR_ARG)
    assert torch.equal(_rows(cache, 0)[0][:, :, :48],
                       k[0].gather(2, idx.view(2, L, hkv, 48, 1)[0].long().expand(L, hkv, 48, d)))
    with pytest.raises(ValueError):
        P.speckv_compress_pages(q, k, v[:, :1], cache=cache, seqs=_i32([0, 1]), **kw)
    with pytest.raises(ValueError):
        P.speckv_compress_pages(q, k, v, cache=cache, seqs=_i32([0]), **kw)
    assert cache.seq_lens.tolist() == [96, 0, 96]
