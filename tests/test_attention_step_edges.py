"""The operators over a paged cache refuse calls whose rows would be read and written, or written twice, in no order; on
the host, none of these calls reaches a device."""
import pytest

from tests.test_attention_step_abi import ALIASING, D, GOT_TO_THE_DEVICE, HEADS, K, Q, V, write

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
