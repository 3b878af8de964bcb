"""The paged-cache entry points (include/hc_paged.h) reject bad arguments on the host before any launch (CPU only; no compute
calls)."""
import os
import re

import pytest

from hyper_connection_rank_gb300 import _binding as B
from hyper_connection_rank_gb300 import _paged as P
from hyper_connection_rank_gb300 import build as gpu_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORMAT = {"hc_rotary_t": P._ROTARY, "hc_rotary_append_t": P._APPEND, "hc_paged_attention_t": P._ATTENTION,
          "hc_pages_t": P._PAGES}


@pytest.fixture(scope="module")
def L():
    gpu_build.build()
    return B.load_library()


def fields(struct_name):
    """Names of a struct's fields in include/hc_paged.h, in order, with whether each is a pointer."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hc_paged.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + struct_name + ";", text).group(1)
    got = []
    for decl in body.split(";"):
        words = decl.replace("const ", "").strip()
        if words:
            kind, rest = words.split(None, 1)
            got += [(name.strip(" *\n"), kind, "*" in name or "*" in kind) for name in rest.split(",")]
    return got


def pack(name, **values):
    have = fields(name)
    assert set(values) <= {f for f, _, _ in have}, set(values) - {f for f, _, _ in have}
    return FORMAT[name].pack(*[values.get(f, 0.0 if kind == "float" and not ptr else 0) for f, kind, ptr in have])


@pytest.mark.parametrize("name", sorted(FORMAT))
def test_packed_structs_have_the_header_s_fields(name):
    """Field by field: pointers and 8-byte integers are 8 bytes, the others 4, in the header's order."""
    codes = re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), FORMAT[name].format.lstrip("@").replace("0q", ""))
    want = "".join("P" if ptr else {"int64_t": "q", "int32_t": "i", "uint32_t": "I", "float": "f", "size_t": "N"}[kind]
                   for _, kind, ptr in [(f, k, p) for f, k, p in fields(name)])
    assert codes == want


ROT = dict(x=0x1000000, positions=0x2000000, inv_freq=0x3000000, out=0x4000000, tokens=4, x_token_stride=128,
           x_head_stride=64, out_token_stride=128, out_head_stride=64, heads=2, head_dim=64, rot_dim=64, dtype=B.HC_BF16,
           amplitude=1.0)


@pytest.mark.parametrize("over", [dict(x=0), dict(positions=0), dict(inv_freq=0), dict(out=0), dict(tokens=-1), dict(heads=0),
                                  dict(head_dim=0), dict(rot_dim=3), dict(rot_dim=66), dict(rot_dim=-2), dict(dtype=7),
                                  dict(x_token_stride=-1), dict(out_token_stride=64), dict(out_head_stride=32),
                                  dict(out=ROT["x"] + 128), dict(out=ROT["positions"]), dict(x=ROT["x"] + 1)], ids=str)
def test_rotary_rejects(L, over):
    assert L.hc_rotary(pack("hc_rotary_t", **{**ROT, **over}), None) == B.HC_ERR_INVALID_ARG
    assert L.hc_last_error()


APP = dict(q=0x1000000, k=0x2000000, v=0x3000000, q_out=0x4000000, k_cache=0x5000000, v_cache=0x6000000, inv_freq=0x7000000,
           page_table=0x7100000, kv_lens=0x7200000, cu_q=0x7300000, tokens=4, num_pages=9, table_stride=5, q_token_stride=128,
           q_head_stride=64, k_token_stride=64, k_head_stride=64, v_token_stride=64, v_head_stride=64, out_token_stride=128,
           out_head_stride=64, cache_page_stride=1024, cache_token_stride=64, cache_head_stride=64, seqs=2, max_pages=5,
           page_size=16, heads=2, kv_heads=1, head_dim=64, rot_dim=64, dtype=B.HC_BF16, amplitude=1.0)


@pytest.mark.parametrize("over", [dict(q=0), dict(k=0), dict(v=0), dict(q_out=0), dict(k_cache=0), dict(v_cache=0),
                                  dict(inv_freq=0), dict(page_table=0), dict(kv_lens=0), dict(cu_q=0), dict(tokens=-1),
                                  dict(seqs=-1), dict(num_pages=0), dict(max_pages=0), dict(page_size=0),
                                  dict(table_stride=4), dict(rot_dim=128), dict(dtype=3), dict(cache_token_stride=32),
                                  dict(cache_page_stride=0), dict(q_out=APP["k"]), dict(k_cache=APP["v_cache"]),
                                  dict(k_cache=APP["q"]), dict(v_cache=APP["page_table"] - 64), dict(kv_heads=0)], ids=str)
def test_rotary_append_rejects(L, over):
    assert L.hc_rotary_append(pack("hc_rotary_append_t", **{**APP, **over}), None) == B.HC_ERR_INVALID_ARG
    assert L.hc_last_error()


ATT = dict(q=0x1000000, k_cache=0x5000000, v_cache=0x6000000, page_table=0x7100000, kv_lens=0x7200000, cu_q=0x7300000,
           out=0x4000000, tokens=4, num_pages=9, table_stride=5, q_token_stride=128, q_head_stride=64, out_token_stride=128,
           out_head_stride=64, cache_page_stride=1024, cache_token_stride=64, cache_head_stride=64, seqs=2, max_pages=5,
           page_size=16, heads=2, kv_heads=1, head_dim=64, dtype=B.HC_BF16, scale=0.125)


@pytest.mark.parametrize("over", [dict(q=0), dict(k_cache=0), dict(v_cache=0), dict(page_table=0), dict(kv_lens=0), dict(out=0),
                                  dict(cu_q=0), dict(tokens=-1), dict(heads=3, kv_heads=2), dict(heads=0), dict(window=-1),
                                  dict(softcap=-1.0), dict(softcap=float("nan")), dict(scale=float("inf")), dict(max_q=-1),
                                  dict(max_kv=-1), dict(flags=4), dict(dtype=9), dict(out_head_stride=63),
                                  dict(table_stride=1), dict(max_pages=2 ** 21)], ids=str)
def test_attention_rejects(L, over):
    assert L.hc_paged_attention(pack("hc_paged_attention_t", **{**ATT, **over}), None) == B.HC_ERR_INVALID_ARG
    assert L.hc_last_error()
    assert L.hc_paged_attention_workspace_size(pack("hc_paged_attention_t", **{**ATT, **over})) == 0


@pytest.mark.parametrize("over", [dict(head_dim=257, cache_token_stride=257, cache_head_stride=257, cache_page_stride=9000,
                                       q_head_stride=257, q_token_stride=514, out_head_stride=257, out_token_stride=514),
                                  dict(tokens=2 ** 30)], ids=["head_dim", "tokens"])
def test_attention_limits(L, over):
    assert L.hc_paged_attention(pack("hc_paged_attention_t", **{**ATT, **over}), None) == B.HC_ERR_UNSUPPORTED


PAG = dict(page_table=0x1000000, lens=0x1100000, refs=0x1200000, page_table_out=0x1300000, lens_out=0x1400000,
           refs_out=0x1500000, num_pages=9, table_stride=5, seqs=2, max_pages=5, page_size=16)
WS, POOL, LIST, ONE = 0x2000000, 0x3000000, 0x4000000, 0x5000000
BAD_PAGES = [dict(refs=0), dict(refs_out=0), dict(page_table=0), dict(lens=0), dict(page_table_out=0), dict(num_pages=0),
             dict(seqs=-1), dict(max_pages=0), dict(page_size=0), dict(table_stride=3), dict(refs_out=PAG["refs"]),
             dict(page_table_out=PAG["page_table"] + 8)]


@pytest.mark.parametrize("over", BAD_PAGES, ids=str)
def test_pages_reject(L, over):
    p = pack("hc_pages_t", **{**PAG, **over})
    n = 1 << 20
    assert L.hc_page_fork(p, LIST, 2, ONE, POOL, 2, 64, WS, n, None) == B.HC_ERR_INVALID_ARG
    assert L.hc_page_extend(p, LIST, ONE, WS, n, None) == B.HC_ERR_INVALID_ARG
    assert L.hc_page_release(p, LIST, None) == B.HC_ERR_INVALID_ARG
    assert L.hc_page_compact(p, LIST, ONE, POOL, 2, 64, WS, n, None) == B.HC_ERR_INVALID_ARG


def test_pages_reject_their_other_arguments(L):
    p = pack("hc_pages_t", **PAG)
    need = L.hc_pages_workspace_size(9, 2)
    assert need > 0 and L.hc_pages_workspace_size(0, 2) == 0 and L.hc_pages_workspace_size(9, -1) == 0
    bad = [
        L.hc_page_fork(p, None, 2, ONE, POOL, 2, 64, WS, need, None), L.hc_page_fork(p, LIST, 2, None, POOL, 2, 64, WS, need, None),
        L.hc_page_fork(p, LIST, -1, ONE, POOL, 2, 64, WS, need, None), L.hc_page_fork(p, LIST, 2, ONE, None, 2, 64, WS, need, None),
        L.hc_page_fork(p, LIST, 2, ONE, POOL, 2, 0, WS, need, None), L.hc_page_fork(p, LIST, 2, ONE, POOL, -1, 64, WS, need, None),
        L.hc_page_fork(None, LIST, 2, ONE, POOL, 2, 64, WS, need, None),
        L.hc_page_extend(p, None, ONE, WS, need, None), L.hc_page_extend(p, LIST, None, WS, need, None),
        L.hc_page_release(p, None, None), L.hc_page_compact(p, None, ONE, POOL, 2, 64, WS, need, None),
        L.hc_page_compact(p, LIST, None, POOL, 2, 64, WS, need, None),
        L.hc_page_copy(None, 2, 9, 64, LIST, LIST, 3, None), L.hc_page_copy(POOL, 2, 9, 64, None, LIST, 3, None),
        L.hc_page_copy(POOL, 2, 9, 64, LIST, LIST, 10, None), L.hc_page_copy(POOL, 2, 9, 64, LIST, LIST, -1, None),
        L.hc_page_copy(POOL, 2, 0, 64, LIST, LIST, 3, None), L.hc_page_copy(POOL, 2, 9, 64, POOL + 64, LIST, 3, None),
    ]
    assert bad == [B.HC_ERR_INVALID_ARG] * len(bad)
    short = [L.hc_page_fork(p, LIST, 2, ONE, POOL, 2, 64, WS, need - 1, None),
             L.hc_page_fork(p, LIST, 2000, ONE, POOL, 2, 64, WS, need, None),
             L.hc_page_fork(p, LIST, 2, ONE, POOL, 2, 64, WS + 8, need, None),
             L.hc_page_extend(p, LIST, ONE, None, need, None),
             L.hc_page_compact(p, LIST, ONE, POOL, 2, 64, WS, need - 1, None)]
    assert short == [B.HC_ERR_WORKSPACE] * len(short)


def test_nothing_to_do_is_ok(L):
    assert L.hc_rotary(pack("hc_rotary_t", **{**ROT, "tokens": 0, "x": 0, "out": 0}), None) == B.HC_OK
    assert L.hc_rotary_append(pack("hc_rotary_append_t", **{**APP, "tokens": 0, "q": 0}), None) == B.HC_OK
    assert L.hc_paged_attention(pack("hc_paged_attention_t", **{**ATT, "tokens": 0, "q": 0, "out": 0}), None) == B.HC_OK
    assert L.hc_page_copy(POOL, 2, 9, 64, None, None, 0, None) == B.HC_OK
