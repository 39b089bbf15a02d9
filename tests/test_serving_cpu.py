"""Checks of the 8-bit paged cache and the prompts' attention that need no GPU:
exported symbols, refusals on the host before any HIP call, workspaces, and the
references' own definitions."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

import serving_refs as ref
from conftest import ROOT
from test_operators_cpu import declared

A16 = 0x10000      # never dereferenced: every call below is refused or empty


@pytest.fixture(scope="module")
def lib():
    from gather_concat_cache_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    from gather_concat_cache_amd import _serving
    return _serving._load()


def test_declared_symbols_are_bound(lib):
    import gather_concat_cache_amd as g
    from gather_concat_cache_amd import _serving
    names = declared("gcache_fp8_kv.h") + declared("gcache_prompt.h")
    assert sorted(names) == sorted(_serving._SIGS)
    for n in names:
        assert hasattr(lib, n)
        if not n.endswith("workspace_bytes"):
            assert getattr(g, n) is getattr(g, n[len("gcache_"):]) and n[len("gcache_"):] in g.__all__


def test_public_headers_compile_as_c(tmp_path):
    import shutil
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "gcache_fp8_kv.h"\n#include "gcache_prompt.h"\nint main(void) { gcache_append_args a; '
                   "gcache_prompt_args p; gcache_fp8_kv_layout l; return (int)(sizeof a + sizeof p + sizeof l) == 0; }\n")
    subprocess.run([shutil.which("gcc"), "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", "-fsyntax-only", str(src)], check=True)


def test_structs_match_the_headers(tmp_path):
    """Sizes and the last field's offset as the C compiler lays them out."""
    import shutil
    import subprocess
    from gather_concat_cache_amd import _serving as s
    src, exe = tmp_path / "t.c", tmp_path / "t"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gcache_fp8_kv.h"\n#include "gcache_prompt.h"\n'
                   "int main(void) { printf(\"%zu %zu %zu %zu %zu %zu\\n\", sizeof(gcache_append_args), "
                   "offsetof(gcache_append_args, cos_sin_bf16), sizeof(gcache_prompt_args), offsetof(gcache_prompt_args, "
                   "accumulate), sizeof(gcache_fp8_kv_layout), offsetof(gcache_fp8_kv_layout, scale_block_stride)); return 0; }\n")
    subprocess.run([shutil.which("gcc"), "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [C.sizeof(s.AppendArgs), s.AppendArgs.cos_sin_bf16.offset, C.sizeof(s.PromptArgs),
                   s.PromptArgs.accumulate.offset, C.sizeof(s.Fp8KvLayout), s.Fp8KvLayout.scale_block_stride.offset]


LAYOUT = dict(token_stride=256, head_stride=128, side_stride=16 * 256, block_stride=2 * 16 * 256, scale_head_stride=1,
              scale_side_stride=2, scale_block_stride=4)
APPEND = dict(q=A16, k=A16, v=A16, q_out=A16, k_out=A16, q_token_stride=1024, q_head_stride=128, k_token_stride=256,
              k_head_stride=128, v_token_stride=256, v_head_stride=128, q_out_token_stride=1024, q_out_head_stride=128,
              k_out_token_stride=256, k_out_head_stride=128, query_starts=A16, seq_lens=A16, block_table=A16,
              block_table_stride=4, positions=A16, cos_sin=A16, max_position=100, cos_sin_stride=128, num_tokens=5,
              num_blocks=9, batch_size=2, num_q_heads=8, num_kv_heads=2, head_size=128, block_size=16, rot=128,
              interleaved=0, cos_sin_bf16=0)
BAD_APPEND = [
    (dict(num_tokens=-1), -2), (dict(batch_size=-1), -2), (dict(k=None), -1), (dict(v=None), -1), (dict(q=None), -1),
    (dict(q_out=None), -1), (dict(query_starts=None), -1), (dict(seq_lens=None), -1), (dict(block_table=None), -1),
    (dict(cos_sin=None), -1), (dict(num_q_heads=-1), -2), (dict(num_kv_heads=0), -2), (dict(head_size=120), -2),
    (dict(head_size=0), -2), (dict(head_size=272, rot=0, k_head_stride=272), -4), (dict(rot=120), -2), (dict(rot=144), -2),
    (dict(block_size=0), -2), (dict(block_size=65537), -2), (dict(block_table_stride=0), -2), (dict(num_blocks=-1), -2),
    (dict(max_position=-1), -2), (dict(cos_sin_stride=127), -2), (dict(num_tokens=1 << 30), -2), (dict(k_token_stride=-8), -2),
    (dict(v_head_stride=132), -3), (dict(q_token_stride=1028), -3), (dict(k=A16 + 8), -3), (dict(k_out=A16 + 2), -3),
    (dict(q_out_head_stride=120), -2), (dict(k_out_token_stride=0), -2), (dict(positions=A16 + 4), -3), (dict(cos_sin=A16 + 2), -3),
    (dict(seq_lens=A16 + 2), -3),
]


@pytest.mark.parametrize("change,status", BAD_APPEND)
def test_append_refusals(lib, change, status):
    from gather_concat_cache_amd._serving import AppendArgs, Fp8KvLayout
    a = AppendArgs(**{**APPEND, **change})
    assert lib.gcache_rope_append_fp8_kv(C.byref(a), A16, A16, C.byref(Fp8KvLayout(**LAYOUT)), None) == status


BAD_LAYOUT = [
    (dict(token_stride=-16), -2), (dict(token_stride=264), -3), (dict(side_stride=8), -3), (dict(block_stride=1 << 62), -2),
    (dict(head_stride=(1 << 62) + 16), -2), (dict(scale_block_stride=-1), -2),
]
OVERLAPS = [dict(token_stride=128), dict(head_stride=112), dict(side_stride=15 * 256), dict(block_stride=4096),
            dict(scale_head_stride=0), dict(scale_side_stride=1), dict(scale_block_stride=3)]


@pytest.mark.parametrize("change,status", BAD_LAYOUT)
def test_layout_refusals(lib, change, status):
    from gather_concat_cache_amd._serving import AppendArgs, Fp8KvLayout
    from test_operators_cpu import _args
    L = Fp8KvLayout(**{**LAYOUT, **change})
    assert lib.gcache_rope_append_fp8_kv(C.byref(AppendArgs(**APPEND)), A16, A16, C.byref(L), None) == status
    assert lib.gcache_attention_fp8_kv(C.byref(_args()), A16, A16, C.byref(L), 2, 128, 0, 0, None, 0, 0, None) == status


@pytest.mark.parametrize("change", OVERLAPS)
def test_append_refuses_rows_that_meet(lib, change):
    from gather_concat_cache_amd._serving import AppendArgs, Fp8KvLayout
    L = Fp8KvLayout(**{**LAYOUT, **change})
    assert lib.gcache_rope_append_fp8_kv(C.byref(AppendArgs(**APPEND)), A16, A16, C.byref(L), None) == -2


def test_empty_calls(lib):
    from gather_concat_cache_amd._serving import AppendArgs, Fp8KvLayout, PromptArgs
    L = Fp8KvLayout(**LAYOUT)
    for change in (dict(num_tokens=0, q=None), dict(batch_size=0, k=None)):
        assert lib.gcache_rope_append_fp8_kv(C.byref(AppendArgs(**{**APPEND, **change})), A16, A16, C.byref(L), None) == 0
    assert lib.gcache_rope_append_fp8_kv(None, A16, A16, C.byref(L), None) == -1
    for change in (dict(total_q=0, q=None), dict(batch_size=0, q=None)):
        assert lib.gcache_prompt_attention(C.byref(PromptArgs(**{**PROMPT, **change})), None) == 0
    assert lib.gcache_prompt_attention(None, None) == -1


def test_cache_attention_refusals(lib):
    from gather_concat_cache_amd._serving import Fp8KvLayout
    from test_operators_cpu import BAD_ARGS, _args
    L = Fp8KvLayout(**LAYOUT)

    def call(a, cache=A16, scales=A16, layout=L, hk=2, hs=128, w=0, s=0, mask=None, ts=0, cols=0):
        return lib.gcache_attention_fp8_kv(a and C.byref(a), cache, scales, layout and C.byref(layout), hk, hs, w, s, mask, ts,
                                           cols, None)
    for change, status in BAD_ARGS:
        assert call(_args(**change)) == status, change
    a = _args()
    assert call(None) == -1 and call(a, cache=None) == -1 and call(a, scales=None) == -1 and call(a, layout=None) == -1
    assert call(a, hs=120) == -2 and call(a, hs=0) == -2 and call(a, hs=272) == -4 and call(a, hk=3) == -2
    assert call(a, w=-1) == -2 and call(a, s=-1) == -2 and call(a, cache=A16 + 8) == -3 and call(a, scales=A16 + 2) == -3
    assert call(a, mask=A16, ts=7, cols=8) == -2 and call(a, mask=A16, ts=8, cols=-1) == -2 and call(a, w=4, mask=A16, ts=8, cols=8) == -2
    assert call(_args(total_q=0, q=None)) == 0 and call(_args(batch_size=0, q=None)) == 0


PROMPT = dict(q=A16, k=A16, v=A16, out=A16, lse=A16, q_token_stride=1024, q_head_stride=128, k_token_stride=256,
              k_head_stride=128, v_token_stride=256, v_head_stride=128, out_token_stride=1024, out_head_stride=128,
              lse_token_stride=8, query_starts=A16, key_starts=A16, total_q=5, total_k=7, max_key_len=7, batch_size=2,
              num_q_heads=8, num_kv_heads=2, key_size=128, value_size=128, softmax_scale=0.1, causal=1, window=0, num_sinks=0,
              accumulate=0, workspace=None, workspace_bytes=0)
BAD_PROMPT = [
    (dict(total_q=-1), -2), (dict(total_k=-1), -2), (dict(batch_size=-1), -2), (dict(q=None), -1), (dict(k=None), -1),
    (dict(v=None), -1), (dict(out=None), -1), (dict(query_starts=None), -1), (dict(key_starts=None), -1),
    (dict(lse=None, accumulate=1), -1), (dict(num_q_heads=0), -2), (dict(num_kv_heads=3), -2), (dict(num_kv_heads=0), -2),
    (dict(key_size=124), -2), (dict(key_size=0), -2), (dict(value_size=4), -2), (dict(key_size=264), -4),
    (dict(value_size=264, out_head_stride=264, out_token_stride=8 * 264), -4), (dict(max_key_len=-1), -2),
    (dict(workspace_bytes=-4), -2), (dict(window=-1), -2), (dict(num_sinks=-1), -2), (dict(window=3, causal=0), -2),
    (dict(softmax_scale=float("nan")), -2), (dict(total_q=1 << 29), -2), (dict(total_k=(1 << 31) - 200), -2),
    (dict(q_token_stride=-8), -2), (dict(k_token_stride=260), -3), (dict(v=A16 + 8), -3), (dict(out=A16 + 2), -3),
    (dict(out_head_stride=120), -2), (dict(out_token_stride=64), -2), (dict(lse_token_stride=7), -2), (dict(lse=A16 + 2), -3),
    (dict(k_token_stride=(1 << 23) + 8), -4), (dict(v_token_stride=1 << 24), -4), (dict(workspace=A16 + 8), -3),
    (dict(key_starts=A16 + 2), -3),
]


@pytest.mark.parametrize("change,status", BAD_PROMPT)
def test_prompt_refusals(lib, change, status):
    from gather_concat_cache_amd._serving import PromptArgs
    assert lib.gcache_prompt_attention(C.byref(PromptArgs(**{**PROMPT, **change})), None) == status


def test_workspace_bytes(lib):
    ws = lib.gcache_prompt_workspace_bytes
    assert ws(1, 1, 32, 8, 128, 128, 100, 0, 0) == 0 and ws(0, 1, 32, 8, 128, 128, 100, 0, 0) == 0
    assert ws(1, 1, 32, 8, 128, 128, 65536, 0, 0) > 0 and ws(16384, 4, 32, 8, 128, 128, 4096, 0, 0) == 0
    assert ws(1, 1, 32, 7, 128, 128, 65536, 0, 0) == 0 and ws(1, 1, 32, 8, 128, 128, -1, 0, 0) == 0
    ws = lib.gcache_attention_fp8_kv_workspace_bytes
    assert ws(1, 1, 32, 8, 128, 65536, 0, 0) > 0 and ws(1, 1, 32, 8, 128, 64, 0, 0) == 0 and ws(1, 1, 32, 8, 128, 65536, 64, 4) == 0


def test_python_refusals():
    """CPU tensors and wrong types never reach the library."""
    import gather_concat_cache_amd as g
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cache, scales = torch.zeros(3, 2, 16, 2, 64, dtype=torch.uint8), torch.zeros(3, 2, 2)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.prompt_attention(q, q, q, i, i, 2, 1.0)
    with pytest.raises(TypeError):
        g.prompt_attention(q.float(), q, q, i, i, 2, 1.0)
    with pytest.raises(TypeError):
        g.attention_fp8_kv(q, cache.float(), scales, i[None], i, i[:1], 2, 1.0)
    with pytest.raises(ValueError):
        g.attention_fp8_kv(q, cache, scales, i[None], i, i[:1], 2, 1.0)
    with pytest.raises(ValueError):
        g.rope_append_fp8_kv(q, q, q, cache, scales, i[None], i, i[:1], None)


def test_page_units_cover_every_split():
    """The units that the append launches for a request are at least the pages
    its tokens can touch: floor((n + 2 bs - 2) / bs) from the first unit on."""
    for bs in (1, 2, 3, 16):
        for n in range(1, 40):
            most = max((ctx + n - 1) // bs - ctx // bs + 1 for ctx in range(bs))
            for before in range(3 * bs):                     # first units of two neighbours
                assert (before + n + 2 * bs - 2) // bs - before // bs >= most


def test_reference_codes_are_the_nearest():
    x = np.concatenate([np.linspace(-500, 500, 4001), 2.0 ** np.linspace(-14, 9, 999)])
    grid = np.unique(ref.e4m3(np.array([b for b in range(256) if b & 127 != 127], np.uint8)))
    near = np.abs(grid[None] - np.clip(x, -448, 448)[:, None]).min(1)
    assert np.array_equal(np.abs(ref.codes(x) - np.clip(x, -448, 448)), near) and np.isin(ref.codes(x), grid).all()
    t = torch.from_numpy(x).float().clamp(-448, 448)
    assert np.array_equal(ref.codes(t.double().numpy()), t.to(torch.float8_e4m3fn).double().numpy())


def test_reference_append_keeps_within_half_a_step():
    rng = np.random.default_rng(0)
    cache, scales = np.zeros((4, 2, 4, 1, 16)), np.zeros((4, 2, 1))
    k, v = rng.standard_normal((11, 1, 16)), rng.standard_normal((11, 1, 16)) * 30
    table = np.array([[2, 0, 3]])
    for t in range(11):
        ref.append(cache, scales, k[t:t + 1], v[t:t + 1], table, [0, 1], [t + 1], 4)
    for t in range(11):
        blk = table[0, t // 4]
        for side, x in enumerate((k[t], v[t])):
            got = cache[blk, side, t % 4] * scales[blk, side]
            assert (np.abs(got - x) <= 2.0 ** -4 * np.abs(x) * 1.0001 + 2.0 ** -9 * scales[blk, side]).all()
