"""The C-ABI library loads and exports every symbol include/speckv.h declares,
and argument errors are reported before anything touches a GPU (no GPU needed)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "speckv.h")


def declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text)) - {"if", "sizeof"})


@pytest.fixture(scope="module")
def lib():
    from prompt_compression_b200 import build
    build.build_library()
    from prompt_compression_b200 import binding
    return binding.load_library()


def test_header_declares_the_boundary():
    names = declared_functions()
    for f in ("speckv_score", "specpc_score", "topk_select", "topk_select_pool", "kv_compact", "spk_last_error",
              "speckv_workspace_size", "specpc_workspace_size", "topk_workspace_size"):
        assert f in names


def test_every_declared_symbol_is_exported(lib):
    for name in declared_functions():
        assert hasattr(lib, name), f"{name} declared in speckv.h but not exported"


def test_workspace_sizes(lib):
    from prompt_compression_b200 import binding as B
    s = B.SpeckvShape(1, 64, 40, 8, 128, 65536, 64, 128, 1.0)
    assert B.speckv_workspace_size(s) == 512 * 1024 * 32    # 32 B per row, rows padded to 128
    s = B.SpecpcShape(1, 24, 4, 14, 2, 64, 32768, 256, 1, 1.0)
    # row offsets (40 units x 1792 rows x 32 B) + on 148 SMs the 128 key blocks
    # are split into 8 segment groups: 128 x 8 x 14 heads x 1 KB of partial sums
    assert B.specpc_workspace_size(s) == 40 * 1792 * 32 + 128 * 8 * 14 * 1024
    s = B.SpecpcShape(2, 24, 4, 14, 2, 64, 131072, 256, 1, 1.0)
    assert B.specpc_workspace_size(s) == 80 * 1792 * 32      # 1024 blocks fill 148 SMs: no split
    assert B.topk_workspace_size(512, 65472) == 512 * 65472 * 4


@pytest.mark.parametrize("fields,status,needle", [
    ((1, 1, 4, 2, 96, 64, 8, 8, 1.0), 2, "head_dim"),
    ((1, 1, 4, 3, 64, 64, 8, 8, 1.0), 1, "multiple"),
    ((1, 1, 4, 2, 64, 64, 80, 8, 1.0), 1, "n_window"),
    ((1, 1, 4, 2, 64, 64, 8, 8, -1.0), 1, "scale"),
    ((1, 1, 64, 2, 64, 64, 64, 8, 1.0), 2, "exceeds"),
    ((1, 1, 4, 2, 64, 64, 0, 0, 1.0), 1, ">= 1"),
])
def test_speckv_argument_errors(lib, fields, status, needle):
    from prompt_compression_b200 import binding as B
    s = B.SpeckvShape(*fields)
    rc = lib.speckv_score(ctypes.byref(s), 16, 16, 16, None, 16, 1 << 20, None)
    assert rc == status
    assert needle in lib.spk_last_error().decode()
    assert lib.speckv_workspace_size(ctypes.byref(s)) == 0


def test_speckv_workspace_and_pointer_errors(lib):
    from prompt_compression_b200 import binding as B
    s = B.SpeckvShape(1, 1, 4, 2, 64, 64, 8, 8, 1.0)
    assert lib.speckv_score(ctypes.byref(s), 16, 16, 16, None, 16, 8, None) == B.SPK_ERR_WORKSPACE
    assert lib.speckv_score(ctypes.byref(s), 16, 16, None, None, 16, 1 << 20, None) == B.SPK_ERR_ARG
    assert lib.speckv_score(ctypes.byref(s), 18, 16, 16, None, 16, 1 << 20, None) == B.SPK_ERR_ARG


def test_specpc_argument_errors(lib):
    from prompt_compression_b200 import binding as B
    bad = [((1, 4, 4, 4, 2, 64, 100, 16, 1, 1.0), 1),      # l_skip == layers
           ((1, 4, 1, 4, 2, 96, 100, 16, 1, 1.0), 2),      # head_dim 96 unsupported
           ((1, 4, 1, 4, 2, 64, 100, 101, 1, 1.0), 1),     # window longer than the input
           ((1, 4, 1, 34, 2, 64, 100, 16, 1, 1.0), 2),     # group of 17 query heads
           ((1, 4, 1, 4, 2, 64, 100, 16, 0, 1.0), 1)]      # no lookahead token
    for fields, status in bad:
        s = B.SpecpcShape(*fields)
        assert lib.specpc_score(ctypes.byref(s), 16, 16, 16, 16, 16, 1 << 30, None) == status, fields


def test_topk_and_compact_argument_errors(lib):
    from prompt_compression_b200 import binding as B
    assert lib.topk_select(16, 4, 100, 4, 10, 0, 16, None, 16, 1 << 20, None) == B.SPK_ERR_ARG  # even pool
    assert lib.topk_select(16, 4, 100, 7, 10, 0, 16, None, 16, 8, None) == B.SPK_ERR_WORKSPACE
    assert lib.topk_select(16, 4, 100, 7, -1, 0, 16, None, 16, 1 << 20, None) == B.SPK_ERR_ARG
    assert lib.topk_select_pool(16, 4, 100, 2, 7, 10, 0, 16, None, 16, 1 << 20, None) == B.SPK_ERR_ARG   # mode
    assert "pool_mode" in lib.spk_last_error().decode()
    assert lib.topk_select_pool(16, 4, 100, 1, 6, 10, 0, 16, None, 16, 1 << 20, None) == B.SPK_ERR_ARG   # even
    assert lib.kv_compact(16, 16, 4, 10, 60, 2, 16, 3, 1, 16, 16, None) == B.SPK_ERR_UNSUPPORTED
    assert lib.kv_compact(16, 16, 5, 10, 64, 2, 16, 3, 2, 16, 16, None) == B.SPK_ERR_ARG
    assert lib.kv_compact(16, None, 4, 10, 64, 2, 16, 3, 1, 16, 16, None) == B.SPK_ERR_ARG
    assert lib.kv_compact(24, 16, 4, 10, 64, 2, 16, 3, 1, 16, 16, None) == B.SPK_ERR_ARG


def test_mapped_host_pointer_rejects_unmapped_memory(lib):
    # ordinary (pageable) host memory is not mapped into any device: the call
    # reports an error and leaves the output alone (here, or on a GPU machine)
    import numpy as np
    buf = np.zeros(64, dtype=np.uint8)
    out = ctypes.c_void_p(12345)
    rc = lib.spk_mapped_host_pointer(ctypes.c_void_p(buf.ctypes.data), ctypes.byref(out))
    assert rc != 0
    assert out.value == 12345
    assert lib.spk_mapped_host_pointer(None, ctypes.byref(out)) == 1   # SPK_ERR_ARG


@pytest.mark.parametrize("args,status,needle", [
    ((1, 1, 4, 3, 128, 10, 1.0), 1, "multiple"),
    ((1, 1, 36, 2, 128, 10, 1.0), 2, "exceeds 8"),
    ((1, 1, 4, 2, 96, 10, 1.0), 2, "head_dim"),
    ((1, 1, 4, 2, 128, 0, 1.0), 1, ">= 1"),
    ((1, 1, 4, 2, 128, 10, -1.0), 1, "scale"),
    ((1, 1, 4, 2, 128, 10, 1.0), 1, "non-NULL"),
])
def test_decode_argument_errors(lib, args, status, needle):
    B, L, hq, hkv, d, n_kv, scale = args
    rc = lib.decode_attention(B, L, hq, hkv, d, n_kv, ctypes.c_float(scale), None, None, None, None, None)
    assert rc == status
    assert needle in lib.spk_last_error().decode()


def _prototypes():
    """name -> number of parameters, from the header's declarations."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    protos = {}
    for m in re.finditer(r"\b([a-z_][a-z0-9_]*)\s*\(([^;{}]*?)\)\s*;", text, flags=re.S):
        name, params = m.group(1), m.group(2).strip()
        protos[name] = 0 if params in ("", "void") else params.count(",") + 1
    return protos


def test_binding_signatures_match_the_header(lib):
    # every function the Python binding declares takes as many arguments as
    # its prototype in include/speckv.h (the boundary cannot drift silently)
    protos = _prototypes()
    checked = 0
    for name, n in protos.items():
        fn = getattr(lib, name)
        if fn.argtypes is None:
            continue
        assert len(fn.argtypes) == n, f"{name}: header has {n} parameters, binding {len(fn.argtypes)}"
        checked += 1
    assert checked >= 10


def _pages(**change):
    from prompt_compression_b200 import binding as B
    f = dict(layers=2, n_pages=10, hkv=2, page_rows=16, head_dim=64, elem_bytes=2, n_seqs=4, max_pages=5)
    f.update(change)
    return B.PagesShape(*f.values())


@pytest.mark.parametrize("change,n,status,needle", [
    (dict(n_pages=0), 2, 1, ">= 1"),
    (dict(page_rows=0), 2, 1, ">= 1"),
    (dict(max_pages=0), 2, 1, ">= 1"),
    (dict(layers=0), 2, 1, ">= 1"),
    (dict(), -1, 1, "n must be"),
    (dict(), 1025, 2, "1025 sequences"),
    (dict(head_dim=7), 2, 2, "multiple of 16"),
    (dict(max_pages=1 << 20, page_rows=1 << 12), 2, 2, "too large"),
    (dict(layers=1 << 12, n_pages=1 << 20), 2, 2, "too large"),
])
def test_pages_shape_errors(lib, change, n, status, needle):
    s = _pages(**change)
    assert lib.kv_pages_reserve(ctypes.byref(s), 16, 16, 16, 16, 16, 16, 16, n, 16, 16, 1 << 30, None) == status
    assert needle in lib.spk_last_error().decode()
    assert lib.kv_pages_write(ctypes.byref(s), 16, 16, 4, None, 4, 1, None, 16, 16, 16, 16, n, 16, 16, None, None) == status
    assert lib.kv_pages_compact(ctypes.byref(s), 16, 16, 16, 16, 16, 16, 16, n, 16, 3, 1, 16, 16, 1 << 30, None) == status


def test_pages_pointer_and_workspace_errors(lib):
    from prompt_compression_b200 import binding as B
    s = ctypes.byref(_pages())
    need = 4 * (2 * 5 + 2 + 4 * 2)                   # two table rows (rounded up to 4 words) and 4 words a sequence
    assert lib.kv_pages_workspace_size(s, 2) == 256
    assert lib.kv_pages_workspace_size(ctypes.byref(_pages(max_pages=0)), 2) == 0
    assert lib.kv_pages_reserve(s, 16, 16, 16, 16, 16, 16, 16, 2, 16, 16, need - 1, None) == B.SPK_ERR_WORKSPACE
    assert lib.kv_pages_fork(s, 16, 16, 16, 16, 16, None, 2, 16, None, 1 << 20, None) == B.SPK_ERR_WORKSPACE
    assert lib.kv_pages_fork(s, 16, 16, 16, 16, 16, None, 2, 16, 24, 1 << 20, None) == B.SPK_ERR_ARG     # workspace alignment
    assert lib.kv_pages_reserve(s, 16, 24, 16, 16, 16, 16, 16, 2, 16, 16, 1 << 20, None) == B.SPK_ERR_ARG
    assert lib.kv_pages_reserve(s, 16, 16, 18, 16, 16, 16, 16, 2, 16, 16, 1 << 20, None) == B.SPK_ERR_ARG
    assert lib.kv_pages_reserve(s, 16, 16, 16, 16, 16, 16, 16, 2, None, 16, 1 << 20, None) == B.SPK_ERR_ARG
    assert lib.kv_pages_reserve(s, 16, 16, 16, 16, 16, None, 16, 2, 16, 16, 1 << 20, None) == B.SPK_ERR_ARG
    assert lib.kv_pages_free(s, 16, None, 16, 16, None, 2, None) == B.SPK_ERR_ARG
    assert lib.kv_pages_free(s, 16, 16, 16, None, None, 2, None) == B.SPK_ERR_ARG
    assert lib.kv_pages_free(s, 16, 16, 16, None, None, 0, None) == B.SPK_OK                             # nothing to do
    book = (16, 16, 16)
    for bad in ((18, 16, 16), (16, 18, 16), (16, 16, 18)):            # a list or *result off its alignment
        assert lib.kv_pages_reserve(s, 16, 16, *book, bad[0], bad[1], 2, bad[2], 16, 1 << 20, None) == B.SPK_ERR_ARG
        assert lib.kv_pages_fork(s, *book, bad[0], 16, bad[1], 2, bad[2], 16, 1 << 20, None) == B.SPK_ERR_ARG
        assert lib.kv_pages_compact(s, 16, 16, *book, bad[0], 16, 2, bad[1], 3, 1, bad[2], 16, 1 << 20, None) == B.SPK_ERR_ARG
        assert lib.kv_pages_write(s, 16, 16, 4, bad[0], 4, 1, bad[1], *book, 16, 2, 16, 16, bad[2], None) == B.SPK_ERR_ARG
    assert lib.kv_pages_free(s, *book, 18, None, 2, None) == B.SPK_ERR_ARG
    assert lib.kv_pages_free(s, *book, 16, 18, 2, None) == B.SPK_ERR_ARG
    w = lambda **k: lib.kv_pages_write(s, k.get("k", 16), 16, k.get("n_src", 4), k.get("idx"), k.get("n_idx", 4),  # noqa: E731
                                       k.get("per", 1), None, 16, 16, 16, 16, 2, 16, 16, None, None)
    assert w(per=3) == B.SPK_ERR_ARG and w(per=0) == B.SPK_ERR_ARG and w(n_idx=5) == B.SPK_ERR_ARG
    assert w(k=None) == B.SPK_ERR_ARG and w(k=8) == B.SPK_ERR_ARG and w(n_src=-1) == B.SPK_ERR_ARG
    assert w(n_idx=0) == B.SPK_OK
    c = lambda n_idx, per=1, idx=16: lib.kv_pages_compact(s, 16, 16, 16, 16, 16, 16, 16, 2, idx, n_idx, per, 16, 16,  # noqa: E731
                                                          1 << 20, None)
    assert c(81) == B.SPK_ERR_ARG and c(-1) == B.SPK_ERR_ARG and c(3, per=5) == B.SPK_ERR_ARG
    assert c(3, idx=None) == B.SPK_ERR_ARG


def _tree(**change):
    from prompt_compression_b200 import binding as B
    f = dict(batch=2, layers=1, hq=8, hkv=2, head_dim=128, n_nodes=4, n_pages=10, page_rows=16, n_seqs=2, max_pages=5,
             dtype=0, scale=1.0)
    f.update(change)
    return B.TreeShape(*f.values())


@pytest.mark.parametrize("change,status,needle", [
    (dict(n_nodes=0), 1, ">= 1"),
    (dict(max_pages=0), 1, ">= 1"),
    (dict(hq=7), 1, "multiple"),
    (dict(dtype=2), 1, "dtype"),
    (dict(scale=0.0), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"),
    (dict(head_dim=96), 2, "head_dim"),
    (dict(n_nodes=1025), 2, "exceeds 1024"),
    (dict(batch=1025, n_seqs=1025), 2, "exceeds 1024"),
    (dict(page_rows=12), 2, "multiple of 8"),
    (dict(layers=1 << 20, n_pages=1 << 20), 2, "too many"),
    (dict(layers=1 << 16, max_pages=1 << 16, n_pages=1 << 13), 2, "too many"),
])
def test_tree_shape_errors(lib, change, status, needle):
    s = _tree(**change)
    assert lib.tree_attention(ctypes.byref(s), 16, 16, 16, 16, 16, None, 16, 16, None, None, 16, None, 16, 1 << 40,
                              None) == status
    assert needle in lib.spk_last_error().decode()
    assert lib.tree_attention_workspace_size(ctypes.byref(s)) == 0


def test_tree_pointer_and_workspace_errors(lib):
    from prompt_compression_b200 import binding as B
    s = _tree()
    base = dict(q=16, kp=16, vp=16, table=16, lens=16, seqs=None, kt=16, vt=16, mask=None, live=None, out=16, lse=None,
                ws=16, n=1 << 40)

    def call(shape=s, **k):
        a = dict(base, **k)
        return lib.tree_attention(ctypes.byref(shape), a["q"], a["kp"], a["vp"], a["table"], a["lens"], a["seqs"],
                                  a["kt"], a["vt"], a["mask"], a["live"], a["out"], a["lse"], a["ws"], a["n"], None)

    assert lib.tree_attention_workspace_size(ctypes.byref(s)) > 0
    for k in (dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(out=None),
              dict(kt=None), dict(vt=None), dict(q=24), dict(kt=8), dict(out=8), dict(table=18), dict(seqs=2),
              dict(mask=6), dict(live=1), dict(lse=2), dict(ws=24)):
        assert call(**k) == B.SPK_ERR_ARG, k
    assert call(ws=None) == B.SPK_ERR_WORKSPACE
    assert call(n=lib.tree_attention_workspace_size(ctypes.byref(s)) - 256) == B.SPK_ERR_WORKSPACE
    assert call(shape=_tree(batch=3)) == B.SPK_ERR_ARG and "n_seqs" in lib.spk_last_error().decode()
    assert lib.tree_mask(0, 4, 16, None, 16, None, None) == B.SPK_ERR_ARG
    assert lib.tree_mask(1, 1025, 16, None, 16, None, None) == B.SPK_ERR_UNSUPPORTED
    assert lib.tree_mask(65536, 4, 16, None, 16, None, None) == B.SPK_ERR_UNSUPPORTED
    assert lib.tree_mask(1, 4, None, None, 16, None, None) == B.SPK_ERR_ARG
    assert lib.tree_mask(1, 4, 16, None, 18, None, None) == B.SPK_ERR_ARG


def test_the_tree_self_test_refuses_what_it_has_no_kernel_for(lib):
    from prompt_compression_b200 import binding as B
    for change in (dict(), dict(head_dim=64, dtype=1), dict(head_dim=64, n_nodes=5), dict(head_dim=64, n_nodes=33)):
        s = _tree(**change)
        assert lib.spk_selftest_tree_give_up(ctypes.byref(s), 16, 16, 16, 16, 16, None, 16, 16, None, None, 16, None, 16,
                                             1 << 40, None) == B.SPK_ERR_UNSUPPORTED
    s = _tree(head_dim=64, n_nodes=2)
    assert lib.spk_selftest_tree_give_up(ctypes.byref(s), None, 16, 16, 16, 16, None, 16, 16, None, None, 16, None, 16,
                                         1 << 40, None) == B.SPK_ERR_ARG
