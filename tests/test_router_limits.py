"""Router arguments that no 32-bit or 64-bit product may hide: refused before any launch."""
import pytest

P = 4096  # an aligned address that a refused call never follows


@pytest.fixture(scope="module")
def ep():
    from combine_ep_prepare_gb300 import build
    build.build()
    import combine_ep_prepare_gb300 as ep
    return ep


@pytest.mark.parametrize("top_k,tokens", [(4, 1 << 62), (4, (1 << 62) + 5), (2, (1 << 63) - 1), (32, 1 << 59), (3, (1 << 62) - 1),
                                          (8, (1 << 21) + 1), (7, (1 << 24) // 7 + 1)])
def test_token_counts_whose_product_wraps_are_refused(ep, top_k, tokens):
    from combine_ep_prepare_gb300._libep import RouterConfig
    c = RouterConfig(64, top_k, 1, 1, 0, 1, 2, 1.0)
    before = ep.ep_launch_count()
    for rc in (ep.lib().ep_router(c, P, None, tokens, P, P, None), ep.lib().ep_router_bwd(c, P, P, P, tokens, P, None)):
        assert rc == 2 and "num_tokens" in ep.ep_last_error()
    assert ep.ep_launch_count() == before
