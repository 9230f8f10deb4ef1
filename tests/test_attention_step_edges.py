"""The operators over a paged cache refuse calls whose rows would be read and written, or written twice, in no order; on
the host, none of these calls reaches a device."""
import pytest

from tests.test_attention_step_abi import (ALIASING, D, GOT_TO_THE_DEVICE, HEADS, K, KC, KS, PAGE, Q, SCRATCH, V, attend, write,
                                            ws_bytes)

# (64 tokens, 4 query heads and 2 key heads of 128 elements of 2 bytes)
IN_PLACE = dict(QO=Q, q_t=1024, qo_t=1024)


@pytest.mark.parametrize("kw", [
    dict(K=Q, k_t=1024), dict(V=Q, v_t=1024), dict(K=Q + 2 * 2 * D, k_t=1024), dict(K=Q + 3 * 2 * D, k_t=1024),
    dict(V=Q + 3 * 2 * D, v_t=1024), dict(K=Q + 7 * 2 * D, k_t=1024), dict(V=Q - 2 * D, v_t=1024),
    dict(K=Q - 1024, k_t=1024, k_h=512), dict(K=Q + 5 * 2048, k_t=1024), dict(V=Q + 63 * 2048, v_t=1024),
    dict(K=Q + 1024 - 16, k_t=1024), dict(V=Q + 1024, v_t=512), dict(V=Q + 1024, v_t=1024 + 8), dict(K=Q + 512, k_t=0),
    dict(K=Q, k_t=1024, q_heads=1), dict(K=Q, k_t=1024, T=1), dict(V=Q + 3 * 2 * D, v_t=0, T=1),
    dict(K=Q + 2 * 64 * D, k_t=D, k_h=64 * D, q_t=D, q_h=64 * D, qo_t=D, qo_h=64 * D),     # heads before tokens
    dict(K=Q + 2 * 64 * D * 2, k_t=D, k_h=2 * 64 * D, q_t=D, q_h=2 * 64 * D, qo_t=D, qo_h=2 * 64 * D),
])
def test_write_refuses_keys_among_queries_turned_in_place(kw):
    assert write(**{**IN_PLACE, **kw}) == ALIASING


def test_write_in_place_accepted():
    for kw in (dict(K=Q + 4 * 2 * D, k_t=1024, V=Q + 6 * 2 * D, v_t=1024),               # [queries, keys, values]
               dict(K=Q - 4 * 2 * D, k_t=1024, V=Q - 2 * 2 * D, v_t=1024),               # [keys, values, queries]
               dict(q_heads=2, q_h=384, qo_h=384, q_t=768, qo_t=768, K=Q + 256, k_h=384, k_t=768, V=Q + 512, v_h=384,
                    v_t=768),                                                           # [head, query key value]
               dict(K=Q + 4 * 2 * D, k_t=0, V=Q + 6 * 2 * D, v_t=2048, v_h=128),         # a token's, every second token's
               dict(K=Q + 4 * 64 * 2 * D, k_t=D, k_h=64 * D, V=Q + 6 * 64 * 2 * D, v_t=D, v_h=64 * D, q_t=D, qo_t=D,
                    q_h=64 * D, qo_h=64 * D),                                           # heads before tokens
               dict(K=Q + 64 * 2 * D, k_t=D, k_h=3 * 64 * D, V=Q + 2 * 64 * 2 * D, v_t=D, v_h=3 * 64 * D, q_t=D, qo_t=D,
                    q_h=3 * 64 * D, qo_h=3 * 64 * D, q_heads=HEADS),
               dict(K=Q + 4 * 2 * D, V=Q + 6 * 2 * D, T=1), dict(K=Q + 1024 * 2 * 64, k_t=1024), dict(K=K, V=V)):
        assert write(**{**IN_PLACE, **kw}) in GOT_TO_THE_DEVICE


# A cache [8, 16, 2, 128] of codes and [8, 16, 2] of scales: strides of a page, a token and a head.
P, PS = PAGE * HEADS * D, PAGE * HEADS


@pytest.mark.parametrize("vc", [
    dict(codes=KC + 16), dict(codes=KC - 16), dict(codes=KC + D), dict(codes=KC + HEADS * D), dict(codes=KC + P),
    dict(codes=KC - 7 * P), dict(codes=KC + 7 * P + 15 * HEADS * D + D), dict(scales=KS + 4), dict(scales=KS - 4),
    dict(scales=KS + 4 * HEADS), dict(scales=KS + 4 * PS), dict(scales=KS + 4 * (8 * PS - 1)),
    dict(codes=KC + P, stride_page=2 * P), dict(codes=KC + D, stride_token=2 * HEADS * D, stride_page=2 * P),
    dict(codes=KC + 16, stride_head=PAGE * D, stride_token=D)])
def test_write_refuses_caches_among_each_other(vc):
    assert write(vc=vc) == ALIASING


def test_write_accepts_halves_of_one_tensor():
    pages = dict(stride_page=2 * P, s_stride_page=2 * PS)
    rows = dict(stride_page=2 * P, stride_token=2 * HEADS * D, s_stride_page=2 * PS, s_stride_token=2 * HEADS)
    heads = dict(rows, stride_head=2 * D, s_stride_head=2)
    first = dict(stride_head=PAGE * D, stride_token=D, s_stride_head=PAGE, s_stride_token=1)    # heads before tokens
    for strides, codes, scales in ((pages, P, PS), (rows, HEADS * D, HEADS), (heads, D, 1), ({}, 8 * P, 8 * PS),
                                   (pages, 5 * P, 5 * PS), (rows, 7 * HEADS * D, 7 * HEADS),
                                   (dict(first, **pages), P, PS),
                                   (dict(first, stride_page=2 * P, stride_head=2 * PAGE * D, s_stride_page=2 * PS,
                                         s_stride_head=2 * PAGE), PAGE * D, PAGE)):
        for sign in (1, -1):
            vc = dict(codes=KC + sign * codes, scales=KS + sign * 4 * scales)
            assert write(kc=strides, vc=dict(strides, **vc)) in GOT_TO_THE_DEVICE
    # keys with tokens before heads, values with heads before tokens
    assert write(kc=pages, vc=dict(first, **pages, codes=KC + P, scales=KS + 4 * PS)) in GOT_TO_THE_DEVICE


# ---------------------------------------------------------------- attention's workspace

def needed(**kw):
    """Workspace bytes that an attention call needs: with fewer it is refused for them, with as many for its output in
    the queries' place."""
    low, high = -1, ws_bytes(**kw)
    strides = dict(q_t=kw["q_heads"] * D, o_t=kw["q_heads"] * D, out=Q)
    sizes = dict(T=kw["T"], B=kw["B"], q_heads=kw["q_heads"], longest=kw["longest"],
                 kc=dict(heads=kw["heads"]), vc=dict(heads=kw["heads"]))
    assert attend(**sizes, **strides, ws_bytes=high) == ALIASING
    while high - low > 1:
        mid = (low + high) // 2
        status = attend(**sizes, **strides, ws_bytes=mid)
        assert status in (SCRATCH, ALIASING)
        low, high = (mid, high) if status == SCRATCH else (low, mid)
    return high


@pytest.mark.parametrize("singles", [1, 100, 500, 5000])
def test_chunks_are_cut_beside_any_number_of_single_tokens(singles):
    """A chunk's tiles of rows can be cut, for which the workspace has room, whatever else is in the batch."""
    alone = needed(T=64, B=1, q_heads=64, heads=8, longest=64)
    assert alone >= 768 * 256 * (D + 2) * 4
    others = needed(T=singles, B=singles, q_heads=64, heads=8, longest=1)
    assert needed(T=singles + 64, B=singles + 1, q_heads=64, heads=8, longest=64) >= alone + others
