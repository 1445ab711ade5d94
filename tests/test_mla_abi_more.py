"""Further refusals and arguments of the attention, weights and eviction calls,
on the host (the pointers are placeholders that are never dereferenced)."""

from test_mla_abi import lib, tree, weights  # noqa: F401  (the fixture)


def test_weights_without_query_tokens(lib):
    nothing = dict(T=0, lse=None, ql=None, qr=None)
    assert weights(lib, **nothing) == 0                      # in place with a decay of 1
    # the sums decay, so what that takes is checked
    for over, status in ((dict(cache=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(wo=None), 1),
                         (dict(start=None), 1), (dict(cache=0x10008), 2)):
        assert weights(lib, **{**nothing, "decay": 0.5, **over}) == status
    assert tree(lib, T=0, ql=None, qr=None, out=None, cache=None) == 0
