"""The pipelines on a stream that is not the caller's: what they allocate must
be known to both streams, so that the allocator does not hand its memory to
either while the other still uses it."""
import contextlib

import pytest
import torch

from prompt_compression_b200 import binding as B
from prompt_compression_b200 import pipeline


@pytest.fixture
def recorded(monkeypatch):
    """Operators replaced by recorders; the tensors that _new_on hands out."""
    made, used = [], []

    def new_on(stream, t, shape, dtype):
        assert stream == 1234
        made.append(torch.empty(shape, dtype=dtype))
        return made[-1]

    monkeypatch.setattr(B, "_new_on", new_on)
    monkeypatch.setattr(B, "_stream_object", lambda stream, device: stream)
    monkeypatch.setattr(B.torch.cuda, "stream", lambda s: contextlib.nullcontext())
    for name, outs in (("speckv_score", (3,)), ("specpc_score", (3,)), ("topk_select", (0, 3)), ("kv_compact", (2, 3, 4))):
        monkeypatch.setattr(B, name, lambda *a, _o=outs, **k: used.extend(a[x] for x in _o if x < len(a)))
    return made, used


class _Cache:
    k_pages = torch.zeros((2, 9, 2, 16, 64), dtype=torch.bfloat16)

    def append(self, k, v, seqs, counts, idx=None, stream=None):
        self.idx = idx
        return torch.zeros(1, dtype=torch.int32)


def _inputs():
    q = torch.zeros((1, 2, 4, 20, 64), dtype=torch.bfloat16)
    k = torch.zeros((1, 2, 2, 300, 64), dtype=torch.bfloat16)
    return q, k, torch.zeros_like(k)


def test_scores_and_rows_of_speckv_compress_pages_belong_to_both_streams(recorded):
    made, used = recorded
    cache, seqs = _Cache(), torch.zeros(1, dtype=torch.int32)
    scores, idx, _ = pipeline.speckv_compress_pages(*_inputs(), 16, 32, cache, seqs, stream=1234)
    known = {id(t) for t in made}
    assert id(scores) in known and id(idx) in known and id(cache.idx) in known
    assert {id(t) for t in used} <= known


def test_what_the_other_pipelines_allocate_belongs_to_both_streams(recorded, monkeypatch):
    made, used = recorded
    monkeypatch.setattr(B, "speckv_workspace_size", lambda shape: 1000)
    monkeypatch.setattr(B, "topk_workspace_size", lambda units, n: 1000)
    q, k, v = _inputs()
    buf = pipeline.speckv_compress(q, k, v, 16, 32, stream=1234)
    assert {id(x) for x in vars(buf).values() if torch.is_tensor(x)} <= {id(t) for t in made}
    scores, idx = pipeline.specpc_select(q, k, torch.ones(4), 0, 40, stream=1234)
    pc_scores, pc_idx, k_g, v_g, buf = pipeline.cascade_compress(q, k, torch.ones(4), 0, 200, q, k, v, 16, 32, stream=1234)
    known = {id(t) for t in made}
    assert {id(t) for t in (scores, idx, pc_scores, pc_idx, k_g, v_g, buf.scores, buf.ws_score)} <= known
    assert {id(t) for t in used if t is not None} <= known


def test_outputs_that_the_binding_makes_belong_to_both_streams(recorded, monkeypatch):
    made, _ = recorded

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(B, "load_library", Library)
    monkeypatch.setattr(B, "_dev", lambda t, *a: 0)
    q, k, v = _inputs()
    rows = torch.zeros((4, 3), dtype=torch.int32)
    outs = [B.decode_attention(q[:, :, :, 0].contiguous(), k, v, stream=1234),
            B.vs_sparse_attention(q, k, v, rows, rows, workspace=torch.zeros(8), stream=1234),
            B.speckv_prefill_attention(q, k, v, k[:, :, :, :4], v[:, :, :, :4], 16, stream=1234)]
    assert {id(t) for t in outs} <= {id(t) for t in made}


@pytest.mark.gpu
def test_speckv_compress_pages_whose_results_are_dropped():
    # the side stream is kept busy, the call's outputs are dropped and their sizes allocated and
    # filled again on the caller's stream before the side stream comes to the call
    from prompt_compression_b200 import build
    build.build_library()
    import prompt_compression_b200 as P
    P.spk_device_error(clear=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
               for s in ((1, 2, 4, 20, 64), (1, 2, 2, 300, 64), (1, 2, 2, 300, 64)))
    seqs, caches = torch.zeros(1, dtype=torch.int32, device="cuda"), []
    side = torch.cuda.Stream()
    for stream in (None, side):
        cache = P.PagedCache(2, 8, 2, 16, 64, n_seqs=1, max_pages=8)
        cache.k_pages.zero_(), cache.v_pages.zero_()
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(side):
                torch.cuda._sleep(200_000_000)                      # about 0.1 s
        P.speckv_compress_pages(q, k, v, 16, 32, cache, seqs, stream=stream)
        again = [torch.full(s, 7, dtype=t, device="cuda")
                 for s, t in (((4, 284), torch.float32), ((4, 48), torch.int32)) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(bool((x == 7).all()) for x in again)
        caches.append(cache)
    for a, b in zip(caches[0].tensors, caches[1].tensors):
        assert torch.equal(a, b)
    assert P.spk_device_error() == (0, 0)


def test_handle_0_is_the_default_stream(monkeypatch):
    monkeypatch.setattr(B.torch.cuda, "default_stream", lambda device: ("default", device))
    monkeypatch.setattr(B.torch.cuda, "ExternalStream", lambda handle, device: ("external", handle, device))
    assert B._stream_object(0, "cuda:1") == ("default", "cuda:1")
    assert B._stream_object(5, "cuda:1") == ("external", 5, "cuda:1")


@pytest.mark.gpu
def test_the_default_streams_handle_names_that_stream():
    default = torch.cuda.default_stream()
    assert default.cuda_stream == 0
    assert B._stream_object(0, torch.device("cuda", 0)).cuda_stream == 0
    side = torch.cuda.Stream()
    assert B._stream_object(side.cuda_stream, torch.device("cuda", 0)).cuda_stream == side.cuda_stream


@pytest.mark.gpu
def test_speckv_compress_pages_on_handle_0():
    # from a stream that is not the default one: the fill of the new lengths, the workspaces and the kernels
    # all go to the default stream, behind what keeps it busy
    from prompt_compression_b200 import build
    build.build_library()
    import prompt_compression_b200 as P
    P.spk_device_error(clear=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
               for s in ((2, 2, 4, 20, 64), (2, 2, 2, 300, 64), (2, 2, 2, 300, 64)))
    seqs, caches, got = torch.tensor([1, 0], dtype=torch.int32, device="cuda"), [], []
    side = torch.cuda.Stream()
    for handle in (None, 0):
        cache = P.PagedCache(2, 8, 2, 16, 64, n_seqs=2, max_pages=8)
        cache.k_pages.zero_(), cache.v_pages.zero_()
        torch.cuda.synchronize()
        if handle is None:
            out = P.speckv_compress_pages(q, k, v, 16, 32, cache, seqs)
        else:
            torch.cuda._sleep(100_000_000)
            with torch.cuda.stream(side):
                out = P.speckv_compress_pages(q, k, v, 16, 32, cache, seqs, stream=handle)
        torch.cuda.synchronize()
        assert out[2].item() == 0
        caches.append(cache)
        got.append(out[:2])
    for a, b in zip(caches[0].tensors + got[0], caches[1].tensors + got[1]):
        assert torch.equal(a, b)
    assert P.spk_device_error() == (0, 0)
