"""The paged-cache entry points on the host at the ends of their ranges (CPU only; no compute calls): sizes whose products
pass 64 bits, and outputs that overlap."""
import pytest

from hyper_connection_rank_gb300 import _binding as B
from test_abi_paged import APP, ATT, LIST, ONE, PAG, POOL, ROT, WS, L, pack  # noqa: F401 (L is a fixture)

BIG, FAR = 2 ** 62, 2 ** 45  # tokens; a stride within the limit of one


def refused(status):
    return status in (B.HC_ERR_INVALID_ARG, B.HC_ERR_UNSUPPORTED)


@pytest.mark.parametrize("over", [dict(tokens=BIG), dict(tokens=2 ** 31), dict(tokens=2 ** 61 + 1, heads=8),
                                  dict(tokens=2 ** 29, heads=1, x_token_stride=FAR, out_token_stride=64),
                                  dict(tokens=2 ** 29, heads=1, out_token_stride=FAR),
                                  dict(heads=65535, tokens=1, x_head_stride=FAR, out_head_stride=64),
                                  dict(heads=65535, tokens=1, out_head_stride=FAR)], ids=str)
def test_rotary_sizes_beyond_64_bits(L, over):  # noqa: F811
    # (the outputs lie far above the inputs, so that no overlap is found by chance)
    assert refused(L.hc_rotary(pack("hc_rotary_t", **{**ROT, "out": 2 ** 48, **over}), None))


@pytest.mark.parametrize("over", [dict(tokens=BIG), dict(tokens=2 ** 60, cu_q=0, seqs=0), dict(tokens=2 ** 29, heads=1, q_token_stride=FAR),
                                  dict(tokens=2 ** 29, heads=1, k_token_stride=FAR), dict(tokens=2 ** 29, heads=1, v_token_stride=FAR),
                                  dict(tokens=2 ** 29, heads=1, out_token_stride=FAR),
                                  dict(page_size=2 ** 20, cache_token_stride=FAR), dict(kv_heads=65535, cache_head_stride=FAR),
                                  dict(seqs=2 ** 30, table_stride=FAR)], ids=str)
def test_append_sizes_beyond_64_bits(L, over):  # noqa: F811
    app = {**APP, "q_out": 2 ** 48, "k_cache": 2 ** 49, "v_cache": 2 ** 50}
    assert refused(L.hc_rotary_append(pack("hc_rotary_append_t", **{**app, **over}), None))


@pytest.mark.parametrize("over", [dict(tokens=BIG), dict(tokens=2 ** 61 + 4), dict(tokens=2 ** 29, heads=1, q_token_stride=FAR),
                                  dict(tokens=2 ** 29, heads=1, out_token_stride=FAR), dict(heads=65535, q_head_stride=FAR, tokens=1),
                                  dict(page_size=2 ** 20, cache_token_stride=FAR), dict(kv_heads=2, heads=2, cache_head_stride=2 ** 47),
                                  dict(seqs=2 ** 24, table_stride=FAR)], ids=str)
def test_attention_sizes_beyond_64_bits(L, over):  # noqa: F811
    att = {**ATT, "out": 2 ** 48}
    assert refused(L.hc_paged_attention(pack("hc_paged_attention_t", **{**att, **over}), None))
    assert L.hc_paged_attention_workspace_size(pack("hc_paged_attention_t", **{**att, **over})) == 0


def test_pools_beyond_64_bits(L):  # noqa: F811
    many = 2 ** 31 - 1
    assert refused(L.hc_page_copy(POOL, 1, many, 2 ** 36, LIST, LIST, 3, None))
    assert refused(L.hc_page_copy(POOL, 2 ** 31, many, 2 ** 33, LIST, LIST, 3, None))
    p = pack("hc_pages_t", **{**PAG, "num_pages": many, "refs": 2 ** 40, "refs_out": 2 ** 41})
    need = L.hc_pages_workspace_size(many, 2)
    assert refused(L.hc_page_fork(p, LIST, 2, ONE, 2 ** 44, 1, 2 ** 36, 2 ** 42, need, None))
    assert refused(L.hc_page_compact(p, LIST, ONE, 2 ** 44, 1, 2 ** 36, 2 ** 42, need, None))
    p = pack("hc_pages_t", **{**PAG, "seqs": 2 ** 24, "table_stride": FAR, "page_table_out": 2 ** 40, "lens_out": 2 ** 50})
    assert refused(L.hc_page_release(p, 2 ** 51, None))


# ------------------------------------------------------------------------------- outputs that overlap --

# Places apart from one another.
AT = dict(table=0x1000000, lens=0x1100000, refs=0x1200000, table_out=0x1300000, lens_out=0x1400000, refs_out=0x1500000,
          ws=0x2000000, cache=0x3000000, list=0x4000000, missing=0x5000000, remap=0x5100000, live=0x5200000)
SIZE = dict(table=(5 + 5) * 4, lens=8, refs=36, table_out=40, lens_out=8, refs_out=36, cache=2 * 9 * 64, list=8, missing=4, remap=36,
            live=4)


def page_call(L, what, at):  # noqa: F811
    p = pack("hc_pages_t", page_table=at["table"], lens=at["lens"], refs=at["refs"], page_table_out=at["table_out"],
             lens_out=at["lens_out"], refs_out=at["refs_out"], num_pages=9, table_stride=5, seqs=2, max_pages=5, page_size=16)
    n = L.hc_pages_workspace_size(9, 2)
    if what == "fork":
        return L.hc_page_fork(p, at["list"], 2, at["missing"], at["cache"], 2, 64, at["ws"], n, None)
    if what == "extend":
        return L.hc_page_extend(p, at["list"], at["missing"], at["ws"], n, None)
    if what == "release":
        return L.hc_page_release(p, at["list"], None)
    return L.hc_page_compact(p, at["remap"], at["live"], at["cache"], 2, 64, at["ws"], n, None)


INPUTS = ["table", "lens", "refs"]
OUTPUTS = {"fork": ["table_out", "lens_out", "refs_out", "missing", "cache", "ws"],
           "extend": ["table_out", "lens_out", "refs_out", "missing", "ws"],
           "release": ["table_out", "lens_out", "refs_out"],
           "compact": ["table_out", "refs_out", "remap", "live", "cache", "ws"]}
READS = {"fork": ["list"], "extend": ["list"], "release": ["list"], "compact": []}


@pytest.mark.parametrize("what", sorted(OUTPUTS))
def test_page_operators_refuse_overlaps(L, what):  # noqa: F811
    """Every output against every input and every other output: at the same place, and ending or beginning inside it."""
    size = {**SIZE, "ws": L.hc_pages_workspace_size(9, 2)}
    for out in OUTPUTS[what]:
        for other in INPUTS + READS[what] + OUTPUTS[what]:
            if other == out:
                continue
            last = 2 if what == "release" and other == "list" else size[other]  # (a byte to a sequence there)
            for place in (AT[other], AT[other] + last - 1, AT[other] - size[out] + 1):
                if out == "ws" and place % 256:
                    continue  # refused for its alignment
                got = page_call(L, what, {**AT, out: place})
                assert got == B.HC_ERR_INVALID_ARG, (out, other, hex(place))
                assert b"overlaps" in L.hc_last_error(), (out, other)


# q (2 heads of 64), k and v (one each) as the columns of one matrix's rows, q rotated in place
ONE_MATRIX = {**APP, "q_out": APP["q"], "k": APP["q"] + 256, "v": APP["q"] + 384, "q_token_stride": 256, "k_token_stride": 256,
              "v_token_stride": 256, "out_token_stride": 256}


@pytest.mark.parametrize("over", [dict(k=APP["q"]), dict(v=APP["q"] + 128), dict(k=APP["q"] + 254), dict(v=APP["q"] + 2 * 512 + 128),
                                  dict(k=APP["q"] - 126), dict(k=APP["q"] - 512 + 386), dict(v_token_stride=320),
                                  dict(tokens=1, seqs=1, k=APP["q"] + 128), dict(k_cache=APP["v_cache"] + 64),
                                  dict(k_cache=APP["v_cache"] - 126)], ids=str)
def test_append_in_place_refuses_overlaps(L, over):  # noqa: F811
    assert L.hc_rotary_append(pack("hc_rotary_append_t", **{**ONE_MATRIX, **over}), None) == B.HC_ERR_INVALID_ARG
    assert b"overlaps" in L.hc_last_error()


@pytest.mark.parametrize("over", [dict(), dict(k=APP["q"] - 512 + 256), dict(k=APP["q"] - 128, v=APP["q"] - 256),
                                  dict(tokens=1, seqs=1), dict(k=0x2000000)], ids=str)
def test_append_in_place_takes_one_matrix(L, over):  # noqa: F811
    """What is refused of these is the check after it (so that nothing is launched where there is a GPU): the caches are one."""
    args = {**ONE_MATRIX, **over, "k_cache": APP["v_cache"]}
    if over.get("tokens") == 1:
        args["cu_q"] = 0
    assert L.hc_rotary_append(pack("hc_rotary_append_t", **args), None) == B.HC_ERR_INVALID_ARG
    assert L.hc_last_error() == b"k_cache overlaps v_cache"
