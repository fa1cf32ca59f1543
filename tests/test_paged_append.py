"""PagedCache.append: room and rows together, so that a list that finds no room
writes over nothing that the sequences hold."""
import pytest
import torch

from prompt_compression_b200.pipeline import PagedCache


def test_append_writes_under_the_reserves_result(monkeypatch):
    cache, calls = PagedCache(1, 4, 1, 16, 64, n_seqs=2, max_pages=2, device="cpu"), []
    monkeypatch.setattr(cache, "reserve", lambda *a, **k: calls.append(("reserve", a, k)) or "result", raising=False)
    monkeypatch.setattr(cache, "write", lambda *a, **k: calls.append(("write", a, k)), raising=False)
    assert cache.append("k", "v", "seqs", "counts", idx="idx", units_per_idx=2, stream=5) == "result"
    assert calls == [("reserve", ("seqs", "counts"), dict(stream=5)),
                     ("write", ("k", "v", "seqs"), dict(idx="idx", counts="counts", units_per_idx=2, reserved="result",
                                                        stream=5))]


@pytest.mark.gpu
def test_append_to_a_full_pool_leaves_the_rows():
    from prompt_compression_b200 import build
    build.build_library()
    import prompt_compression_b200 as P
    P.spk_device_error(clear=True)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    cache = PagedCache(2, 5, 2, 16, 64, n_seqs=3, max_pages=4)
    cache.k_pages.zero_(), cache.v_pages.zero_()
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn((2, 2, 2, 40, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    assert cache.append(k, v, i32([2, 0]), i32([40, 17])).item() == 0            # all five pages
    for s, b, n in ((2, 0, 40), (0, 1, 17)):
        for pool, x in ((cache.k_pages, k), (cache.v_pages, v)):
            rows = pool[:, cache.page_table[s, :-(-n // 16)].long()].transpose(1, 2).reshape(2, 2, -1, 64)
            assert torch.equal(rows[:, :, :n], x[b, :, :, :n])
    held = [x.clone() for x in cache.tensors]
    for seqs, counts, want in (([1, 2], [16, 1], 1), ([0], [32], 2), ([2, 2], [1, 1], -1)):
        assert cache.append(k[:len(seqs)], v[:len(seqs)], i32(seqs), i32(counts)).item() == want
        for a, b in zip(cache.tensors, held):
            assert torch.equal(a, b)
        assert P.spk_device_error(clear=True)[0] == (0 if want > 0 else P.binding.SPK_ERR_ARG)
    rows = i32([[3, 1, 0], [5, 9, 0]])                                           # chosen rows, in the last pages' room
    assert cache.append(k, v, i32([0, 2]), i32([3, 2]), idx=rows, units_per_idx=4).item() == 0
    assert cache.seq_lens.tolist() == [20, 0, 42]
    last = cache.k_pages[:, int(cache.page_table[0, 1]), :, 1:4]
    assert torch.equal(last, k[0][:, :, [3, 1, 0]])
    assert P.spk_device_error() == (0, 0)
