"""Checks of the 8-bit paged cache and the prompts' attention at the edges of
their headers that need no GPU."""
import ctypes as C
import os

import pytest

from conftest import ROOT
from test_operators_cpu import A16, declared
from test_serving_cpu import APPEND, LAYOUT, lib  # noqa: F401


# ---------------------------------------------------------------------------
# pages of several geometries
# ---------------------------------------------------------------------------
def test_page_set_symbols_are_bound(lib):  # noqa: F811
    from gather_concat_cache_amd import _operators
    names = declared("gcache_page_sets.h")
    assert sorted(names) == sorted(_operators._SET_SIGS) and all(hasattr(lib, n) for n in names)


def test_page_set_header_compiles_as_c(tmp_path):
    import shutil
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "gcache_page_sets.h"\nint main(void) { gcache_page_caches s[2]; return (int)sizeof s == 0; }\n')
    subprocess.run([shutil.which("gcc"), "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", "-fsyntax-only", str(src)], check=True)


def test_page_set_refusals(lib):  # noqa: F811
    """Every set is checked, not the first alone."""
    from gather_concat_cache_amd._operators import PageCaches, PageState
    ptrs = (C.c_void_p * 2)(A16, A16 + 64)
    good = dict(caches=C.cast(ptrs, C.c_void_p), num_caches=2, block_stride=96, page_bytes=96)
    state = PageState(block_table=A16, block_table_stride=4, seq_lens=A16, ref_counts=A16, num_blocks=9, num_rows=3, block_size=16)
    W = lib.gcache_pages_workspace_bytes(9, 3, 2)

    def sets(**bad):
        return (PageCaches * 2)(PageCaches(**good), PageCaches(**{**good, **bad}))

    def fork(s, n, forks=2):
        return lib.gcache_fork_page_sets(C.byref(state), s, n, A16, A16, forks, A16, A16, W, None)

    def compact(s, n):
        return lib.gcache_compact_page_sets(C.byref(state), s, n, A16, A16, W, None)

    def copy(s, n, pairs=2):
        return lib.gcache_copy_page_sets(s, n, 9, A16, A16, pairs, None)
    for bad, status in ((dict(caches=None), -1), (dict(num_caches=-1), -2), (dict(page_bytes=97), -2), (dict(page_bytes=-1), -2),
                        (dict(block_stride=1 << 62), -2)):
        for f in (fork, compact, copy):
            assert f(sets(**bad), 2) == status, (f.__name__, bad)
    for f in (fork, compact, copy):
        assert f(sets(), -1) == -2 and f(None, 1) == -1
    assert fork(sets(), 2, 0) == 0 and copy(sets(), 2, 0) == 0 and copy(None, 0) == 0
    assert copy(sets(page_bytes=0), 0) == 0


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def test_append_without_rotation_looks_at_no_table(lib):  # noqa: F811
    """rot 0: positions and cos_sin may be anything.  The calls are refused for
    their layout, which is checked behind the pointers."""
    from gather_concat_cache_amd._serving import AppendArgs, Fp8KvLayout
    bad = Fp8KvLayout(**{**LAYOUT, "block_stride": 1 << 62})
    for change in (dict(positions=A16 + 4), dict(cos_sin=A16 + 2), dict(cos_sin=A16 + 1, cos_sin_bf16=1, max_position=-1, cos_sin_stride=-5)):
        a = AppendArgs(**{**APPEND, "rot": 0, **change})
        assert lib.gcache_rope_append_fp8_kv(C.byref(a), A16, A16, C.byref(bad), None) == -2, change
        if "max_position" not in change:
            a.rot = 16
            assert lib.gcache_rope_append_fp8_kv(C.byref(a), A16, A16, C.byref(bad), None) == -3, change


# ---------------------------------------------------------------------------
# inline assembly
# ---------------------------------------------------------------------------
def test_assembly_that_writes_m0_says_so():
    """The compiler keeps values in m0 over a statement that does not name it."""
    import glob
    import re
    found = 0
    for path in glob.glob(os.path.join(ROOT, "gather_concat_cache_amd", "csrc", "*.h*")):
        for asm in re.findall(r"\basm\b[^;]*?\((.*?)\);", open(path).read(), flags=re.S):
            if re.search(r"s_mov_b32 m0", asm):
                found += 1
                assert '"m0"' in asm.split(":")[-1], (path, asm)
    assert found
